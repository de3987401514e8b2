// Host side of the operators around attention and recurrences declared in include/kda.h (norms,
// rotary positions, 4-bit caches): argument validation, schedule selection and launches.
// Nothing here touches device memory.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/kda.h"
#include "api_util.h"
#include "layer_params.h"

namespace {

using kda::aligned16;
using kda::any_overlap;
using kda::kCache4Tile;
using kda::kMaxBytes;
using kda::make_range;
using kda::overlaps;
using kda::Range;
using kda::row_ok;
using kda::span_bytes;
using kda::status;

constexpr int64_t kMostItems = ((int64_t)1 << 32) - 1;  // work-items of a launch

// ---- kda_norm

bool norm_group_ok(int64_t W, int64_t group) {
  if (group == W) return true;
  return group >= 32 && group <= 512 && (group & (group - 1)) == 0 && W % group == 0;
}

int norm_check(const void* x, int64_t x_row, const void* gate, int64_t gate_row, int gate_fn,
               const void* post_weight, int64_t group, const void* weight, int weight_dtype,
               float eps, const void* residual, const void* residual_out, int residual_dtype,
               float residual_scale, const void* out, int64_t R, int64_t W) {
  if (R < 0 || W < 8 || W % 8 != 0 || W > kda::kNormMaxW) return KDA_ERR_BAD_SHAPE;
  if (post_weight && !norm_group_ok(W, group)) return KDA_ERR_BAD_SHAPE;
  if (R > kMostItems / kda::norm_threads(W) / 8) return KDA_ERR_BAD_SHAPE;
  if (gate && gate_fn != KDA_GATE_SIGMOID && gate_fn != KDA_GATE_SILU) return KDA_ERR_BAD_DTYPE;
  if ((post_weight || weight) && weight_dtype != KDA_DTYPE_BF16 && weight_dtype != KDA_DTYPE_FP32)
    return KDA_ERR_BAD_DTYPE;
  if (residual && residual_dtype != KDA_DTYPE_BF16 && residual_dtype != KDA_DTYPE_FP32)
    return KDA_ERR_BAD_DTYPE;
  if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(residual_scale))
    return KDA_ERR_BAD_SCALE;
  if (!post_weight && !gate && !weight && !residual) return KDA_ERR_NULL_ARG;
  if ((residual == nullptr) != (residual_out == nullptr)) return KDA_ERR_NULL_ARG;
  if (R > 0 && (!x || (!out && (weight || !residual)))) return KDA_ERR_NULL_ARG;
  if (!row_ok(x_row, 1, W) || (gate && !row_ok(gate_row, 1, W)) || !aligned16(x) ||
      !aligned16(gate) || !aligned16(post_weight) || !aligned16(weight) || !aligned16(residual) ||
      !aligned16(residual_out) || !aligned16(out))
    return KDA_ERR_BAD_LAYOUT;
  const int64_t bx = span_bytes(R, x_row, 1, W), bg = gate ? span_bytes(R, gate_row, 1, W) : 0;
  if (bx < 0 || bg < 0) return KDA_ERR_BAD_SHAPE;
  const int64_t wb = weight_dtype == KDA_DTYPE_FP32 ? 4 : 2;
  const int64_t rb = residual ? R * W * (residual_dtype == KDA_DTYPE_FP32 ? 4 : 2) : 0;
  const Range ro = make_range(out, out ? R * W * 2 : 0), rh = make_range(residual_out, rb),
              rr = make_range(residual, rb);
  const Range ins[] = {make_range(x, bx), make_range(gate, bg),
                       make_range(post_weight, post_weight ? group * wb : 0),
                       make_range(weight, weight ? W * wb : 0)};
  if (any_overlap(ro, ins, 4) || any_overlap(rh, ins, 4) || overlaps(ro, rh) || overlaps(ro, rr))
    return KDA_ERR_BAD_ALIAS;
  if (overlaps(rh, rr) && residual != residual_out) return KDA_ERR_BAD_ALIAS;
  return KDA_OK;
}

// ---- kda_rope

// Strided rows of one tensor: n rows of `len` elements, `row` apart.
struct Rows {
  const void* at;
  int64_t row, len;
};

// Whether two tensors of n rows share a byte.  Rows of one stride that lie in other columns of
// the same wider rows do not, though their ranges overlap.
bool share(const Rows& a, const Rows& b, int64_t n) {
  if (!overlaps(make_range(a.at, span_bytes(n, a.row, 1, a.len)),
                make_range(b.at, span_bytes(n, b.row, 1, b.len))))
    return false;
  if (a.row != b.row) return true;
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.at)) -
                    static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.at));
  const int64_t row = a.row * 2, shift = ((d % row) + row) % row;
  return !(shift >= a.len * 2 && row - shift >= b.len * 2);
}

bool in_place(const Rows& a, const Rows& b) { return a.at == b.at && a.row == b.row; }

int rope_check(const void* q, int64_t q_row, const void* q_out, int64_t q_out_row, const void* k,
               int64_t k_row, const void* k_out, int64_t k_out_row, const double* freqs,
               int64_t rot, float amplitude, const int64_t* positions, const int64_t* offsets,
               const int64_t* cu, int64_t N, int64_t B, int64_t T, int64_t Hq, int64_t Hk,
               int64_t D) {
  if (D < 8 || D % 8 != 0 || D > kda::kRopeMaxD || rot < 2 || rot % 2 != 0 || rot > D)
    return KDA_ERR_BAD_SHAPE;
  if (Hq < 1 || Hk < 0 || Hq > (1 << 20) || Hk > (1 << 20)) return KDA_ERR_BAD_SHAPE;
  const int sizes = kda::batch_ok(cu, N, B, T);
  if (sizes != KDA_OK) return sizes;
  if (N >= ((int64_t)1 << 31)) return KDA_ERR_BAD_SHAPE;
  const int64_t tok = B * T;
  // a workgroup for each token at most, or a few that share a token's heads
  if (tok >= ((int64_t)1 << 24)) return KDA_ERR_BAD_SHAPE;
  if (positions && (offsets || cu)) return KDA_ERR_BAD_VARLEN;
  if (!std::isfinite(amplitude)) return KDA_ERR_BAD_SCALE;
  if (!freqs || (tok > 0 && (!q || !q_out || (Hk > 0 && (!k || !k_out)))))
    return KDA_ERR_NULL_ARG;
  const Rows a = {q, q_row, Hq * D}, ao = {q_out, q_out_row, Hq * D}, b = {k, k_row, Hk * D},
             bo = {k_out, k_out_row, Hk * D};
  const Rows both[] = {a, ao, b, bo};
  for (int i = 0; i < (Hk > 0 ? 4 : 2); ++i) {
    if (!row_ok(both[i].row, 1, both[i].len) || !aligned16(both[i].at)) return KDA_ERR_BAD_LAYOUT;
    if (span_bytes(tok, both[i].row, 1, both[i].len) < 0) return KDA_ERR_BAD_SHAPE;
  }
  if (tok == 0) return KDA_OK;
  const Range small[] = {make_range(freqs, rot / 2 * 8),
                         make_range(positions, positions ? tok * 8 : 0),
                         make_range(offsets, offsets ? N * 8 : 0),
                         make_range(cu, cu ? (N + 1) * 8 : 0)};
  if (any_overlap(make_range(q_out, span_bytes(tok, q_out_row, 1, ao.len)), small, 4) ||
      (share(a, ao, tok) && !in_place(a, ao)))
    return KDA_ERR_BAD_ALIAS;
  if (Hk > 0) {
    if (any_overlap(make_range(k_out, span_bytes(tok, k_out_row, 1, bo.len)), small, 4) ||
        (share(b, bo, tok) && !in_place(b, bo)) || share(a, bo, tok) || share(b, ao, tok) ||
        share(ao, bo, tok))
      return KDA_ERR_BAD_ALIAS;
  }
  return KDA_OK;
}

// ---- caches in 4 bits

struct CacheRanges {
  Range r[4];
};

// Sizes and pointers of a cache; its ranges.
int cache4_check(const void* k4, const void* ks, const void* v4, const void* vs, int64_t slots,
                 int64_t cap, int64_t Hk, int64_t D, CacheRanges* out) {
  if (D != 64 && D != 128) return KDA_ERR_BAD_SHAPE;
  if (slots < 1 || Hk < 1 || Hk >= (1 << 24) || cap < kCache4Tile || cap % kCache4Tile != 0 ||
      cap > ((int64_t)1 << 30))
    return KDA_ERR_BAD_SHAPE;
  if (slots > kMaxBytes / cap / Hk / D) return KDA_ERR_BAD_SHAPE;
  if (!k4 || !ks || !v4 || !vs) return KDA_ERR_NULL_ARG;
  if (!aligned16(k4) || !aligned16(ks) || !aligned16(v4) || !aligned16(vs))
    return KDA_ERR_BAD_LAYOUT;
  const int64_t rows = slots * Hk * cap;
  out->r[0] = make_range(k4, rows * (D / 2));
  out->r[1] = make_range(ks, rows * (D / 32));
  out->r[2] = make_range(v4, rows * (D / 2));
  out->r[3] = make_range(vs, rows * (D / 32));
  return KDA_OK;
}

int put4_check(const void* k, int64_t k_row, const void* v, int64_t v_row, const void* k4,
               const void* ks, const void* v4, const void* vs, int64_t num_slots, int64_t cap,
               const void* k_out, const void* v_out, const int64_t* offsets, const int64_t* slots,
               const int64_t* cu, int64_t N, int64_t B, int64_t T, int64_t Hk, int64_t D) {
  CacheRanges c;
  const int st = cache4_check(k4, ks, v4, vs, num_slots, cap, Hk, D, &c);
  if (st == KDA_ERR_BAD_SHAPE) return st;
  const int sizes = kda::batch_ok(cu, N, B, T);
  if (sizes != KDA_OK) return sizes;
  const int64_t tok = B * T;
  if (N >= ((int64_t)1 << 31) || (!slots && N > num_slots)) return KDA_ERR_BAD_SHAPE;
  if (kda::put4_tiles(tok, T, N, cu != nullptr) > kMostItems / kda::put4_threads((int)D) / Hk)
    return KDA_ERR_BAD_SHAPE;
  if (st != KDA_OK) return st;
  if ((tok > 0 && (!k || !v)) || (k_out == nullptr) != (v_out == nullptr)) return KDA_ERR_NULL_ARG;
  if (!row_ok(k_row, Hk, D) || !row_ok(v_row, Hk, D) || !aligned16(k) || !aligned16(v) ||
      !aligned16(k_out) || !aligned16(v_out))
    return KDA_ERR_BAD_LAYOUT;
  const int64_t bk = span_bytes(tok, k_row, Hk, D), bv = span_bytes(tok, v_row, Hk, D);
  if (bk < 0 || bv < 0) return KDA_ERR_BAD_SHAPE;
  const int64_t bo = k_out ? tok * Hk * D * 2 : 0;
  const Range ins[] = {make_range(k, bk), make_range(v, bv),
                       make_range(offsets, offsets ? N * 8 : 0),
                       make_range(slots, slots ? N * 8 : 0), make_range(cu, cu ? (N + 1) * 8 : 0)};
  const Range outs[] = {c.r[0], c.r[1], c.r[2], c.r[3], make_range(k_out, bo),
                        make_range(v_out, bo)};
  for (int i = 0; i < 6; ++i)
    if (any_overlap(outs[i], ins, 5) || any_overlap(outs[i], outs + i + 1, 5 - i))
      return KDA_ERR_BAD_ALIAS;
  return KDA_OK;
}

// How a kda_attn4_fwd call runs: keys in parts of `part` straight from the cache; or
// (expand) keys and values to a bf16 workspace first and then the kernel of
// kda_attn_fwd's prompts with `splits` parts of each row's keys.
struct Plan4 {
  bool expand;
  int64_t part, splits;
  kda::AttnSchedule sched;
  int64_t bytes;  // of the workspace
};

// Keys of a part when the caller leaves the choice, for `units` (tile of rows, key/value head)
// pairs.  Parts are of equally many keys, not as many for each sequence, whose lengths differ.
// One part up to 1280 positions (16 units, D 64: 7.5 us, 8.7 in three).  Up to a quarter of the
// compute units: a workgroup for each, and at least 512 keys (D 128; 8 units, 2048 positions, in one
// part and in parts of 1024, 512, 256: 13.6, 11.6, 9.7, 8.9 us; 32 units, 8192: 37, 13.2, 14.3, 18.4;
// 8 units, 131072, parts of 8192, 4096, 2048: 43, 33, 39).  Up to two units each: five workgroups and
// at least 1024 keys (256 units, 8192 positions, in one part and parts of 4096, 1536, 1024: 46, 43,
// 39.8, 41.5), but more units than half of them with 2048 positions or fewer in one (256 units 15.5,
// 18.2 in two).  Beyond: one part (512 units of 4096 positions 37.6, in four 49).
// The figures are of lengths from an eighth of the capacity to all of it.  Where all caches are full
// one part gains at 4096 positions, having no uneven lengths to level (256 units in one part and by
// this rule, D 64: 17.4 and 21.0, D 128: 28.0 and 32.0; 192 units, three tiles of rows over the same
// keys: 17.1 and 20.7, 22.8 and 29.1), and D 64 with 2048 positions would rather have one part or
// parts of 512 (64 units: 10.0 and 9.7, by this rule 11.4).
int64_t attn4_auto_part(int64_t units, int64_t cap) {
  const int64_t cus = kda::device_cus();
  if (units < 1 || units >= 2 * cus || cap <= (2 * units > cus ? 2048 : 1280)) return cap;
  const bool few = 4 * units <= cus;
  int64_t parts = (few ? 1 : 5) * cus / units;
  if (parts > cap / (few ? 512 : 1024)) parts = cap / (few ? 512 : 1024);
  if (parts > 64) parts = 64;
  if (parts < 1) parts = 1;
  const int64_t part = (cap + parts - 1) / parts;
  return (part + 63) / 64 * 64;
}

constexpr int64_t kExpandMax = (int64_t)8 << 30;  // bytes of expanded keys and values, at most

int64_t round16(int64_t x) { return (x + 15) / 16 * 16; }

int64_t parts_bytes(int64_t parts, int64_t rows, int64_t D) {
  return parts > 1 ? parts * rows * (D + 2) * 4 : 0;
}

int attn4_plan(int64_t N, int64_t Bq, int64_t Tq, int64_t cap, int64_t Hq, int64_t Hk, int64_t D,
               int64_t part, bool workspace, Plan4* plan) {
  if (D != 64 && D != 128) return KDA_ERR_BAD_SHAPE;
  if (Hk < 1 || Hq < 1 || Hq % Hk != 0 || Hq >= (1 << 24)) return KDA_ERR_BAD_SHAPE;
  if (N < 1 || N >= ((int64_t)1 << 31) || Bq < 1 || Tq < 0) return KDA_ERR_BAD_SHAPE;
  if (Bq != 1 && Bq != N) return KDA_ERR_BAD_VARLEN;
  if (cap < kCache4Tile || cap % kCache4Tile != 0 || cap > ((int64_t)1 << 30))
    return KDA_ERR_BAD_SHAPE;
  // rows of a sequence are 32-bit numbers
  if (Tq > ((int64_t)1 << 30) / (Hq / Hk) || Tq > ((int64_t)1 << 40) / Bq)
    return KDA_ERR_BAD_SHAPE;
  if (part < 0 || part % kCache4Tile != 0 || (part && (cap + part - 1) / part > 64))
    return KDA_ERR_BAD_SCHEDULE;
  const int64_t G = Hq / Hk, total = Bq * Tq, most = kMostItems / kda::kAttnThreads;
  const int64_t tiles = kda::attn_slots(total, N, G, kda::kAttn4Rows) + (Bq == N ? N : 0);
  if (tiles > most / Hk) return KDA_ERR_BAD_SHAPE;
  plan->expand = false;
  plan->splits = 1;
  const int64_t units = Bq == N ? N * ((Tq * G + kda::kAttn4Rows - 1) / kda::kAttn4Rows) * Hk
                                : tiles * Hk;
  // Expanded keys pay from some 450 rows of a sequence and key/value head on (32 sequences of 4096
  // positions, 8 heads, D 128, 256 rows: 241 us, from the cache 210; 512 rows: 376 and 405), and
  // only where their tiles fill the device many times over (1 sequence of 8192, 512 rows: 36 and
  // 21, 2048 rows: 52 and 60; 3 sequences of 2208, D 64, 1024 rows: 45 and 32, 2048 rows: 53, 57).
  // p has one bf16 part then, as in that kernel's own calls: packed [300, 700, 1024] queries over
  // [300, 2200, 1101] keys, 96/8 heads, 119 us with an error of 2.1e-3; two parts there 149 and 1.6e-3.
  // Both conditions go by the call's mean, as the host knows no lengths: a prompt of 2048 beside 31 single
  // tokens over 1024-3904 positions, 32/8 heads, takes 116 us, in two calls 58 and 28; one of 8192
  // expands all 32 caches, 625 us, in two calls 498 and 27.
  const int64_t row_bytes = Hk * D * 4;
  if (part == 0 && workspace && total * G > N * kda::kExpand4Rows &&
      units > (D == 128 ? 3 : 8) * kda::device_cus() &&
      Hk * D < (1 << 24) && N <= kExpandMax / row_bytes / cap &&
      N * Hk <= most / (cap / kCache4Tile)) {
    plan->expand = true;
    plan->sched = kda::AttnSchedule{0, 2, 128};
    const int64_t slots = Bq == N ? N * ((Tq * G + 127) / 128) : kda::attn_slots(total, N, G, 128);
    int64_t sp = kda::attn_auto_splits(plan->sched, slots, Hk, cap);
    if (sp > 1 && (slots * Hk > most / sp || total > 4 * most / Hq)) sp = 1;
    plan->splits = sp;
    plan->part = cap;
    plan->bytes = N * cap * row_bytes + round16(N * 8) + parts_bytes(sp, total * Hq, D);
    return KDA_OK;
  }
  int64_t pt = part ? part : workspace ? attn4_auto_part(units, cap) : cap;
  if (pt > cap) pt = cap;
  const int64_t parts = (cap + pt - 1) / pt;
  if (parts > 1 && (tiles * Hk > most / parts || total > 4 * most / Hq)) {
    if (part) return KDA_ERR_BAD_SHAPE;
    pt = cap;
  }
  plan->part = pt;
  plan->bytes = parts_bytes((cap + pt - 1) / pt, total * Hq, D);
  return KDA_OK;
}

int attn4_check(const void* q, int64_t q_row, const void* k4, const void* ks, const void* v4,
                const void* vs, int64_t num_slots, int64_t cap, float scale, const void* out,
                const float* lse, const int64_t* cu_q, const int64_t* k_lens, const int64_t* slots,
                int64_t N, int64_t Bq, int64_t Tq, int64_t Hq, int64_t Hk, int64_t D, int64_t part,
                const void* workspace, int64_t workspace_bytes, Plan4* plan) {
  // left to the library: without a workspace, neither parts nor expanded keys
  int st = attn4_plan(N, Bq, Tq, cap, Hq, Hk, D, part, workspace != nullptr, plan);
  if (st != KDA_OK) return st;
  if (cu_q ? Bq != 1 : Bq != N) return KDA_ERR_BAD_VARLEN;
  if (!slots && N > num_slots) return KDA_ERR_BAD_SHAPE;
  CacheRanges c;
  st = cache4_check(k4, ks, v4, vs, num_slots, cap, Hk, D, &c);
  if (st != KDA_OK) return st;
  if (!std::isfinite(kda::attn_c(scale)) || scale < 0.f) return KDA_ERR_BAD_SCALE;
  const int64_t nq = Bq * Tq;
  if (nq > 0 && (!q || !out)) return KDA_ERR_NULL_ARG;
  if (q_row >= (1 << 24)) return KDA_ERR_BAD_SHAPE;
  if (!row_ok(q_row, Hq, D) || !aligned16(q) || !aligned16(out) || !aligned16(workspace))
    return KDA_ERR_BAD_LAYOUT;
  const int64_t bq = span_bytes(nq, q_row, Hq, D);
  if (bq < 0) return KDA_ERR_BAD_SHAPE;
  const int64_t need = plan->bytes;
  if (need > 0 && !workspace) return KDA_ERR_NULL_ARG;
  if (need > workspace_bytes) return KDA_ERR_BAD_WORKSPACE;
  const Range ins[] = {make_range(q, bq),
                       c.r[0],
                       c.r[1],
                       c.r[2],
                       c.r[3],
                       make_range(cu_q, cu_q ? (N + 1) * 8 : 0),
                       make_range(k_lens, k_lens ? N * 8 : 0),
                       make_range(slots, slots ? N * 8 : 0)};
  const Range outs[] = {make_range(out, nq * Hq * D * 2), make_range(lse, lse ? nq * Hq * 4 : 0),
                        make_range(workspace, need)};
  for (int i = 0; i < 3; ++i)
    if (any_overlap(outs[i], ins, 8) || any_overlap(outs[i], outs + i + 1, 2 - i))
      return KDA_ERR_BAD_ALIAS;
  return KDA_OK;
}

kda::Cache4 cache_of(const void* k4, const void* ks, const void* v4, const void* vs, int64_t slots,
                     int64_t cap) {
  auto u8 = [](const void* x) { return static_cast<uint8_t*>(const_cast<void*>(x)); };
  return kda::Cache4{u8(k4), u8(ks), u8(v4), u8(vs), slots, cap};
}

}  // namespace

extern "C" {

int kda_norm_check(const void* x, int64_t x_row, const void* gate, int64_t gate_row, int gate_fn,
                   const void* post_weight, int64_t group, const void* weight, int weight_dtype,
                   float eps, const void* residual, const void* residual_out, int residual_dtype,
                   float residual_scale, const void* out, int64_t R, int64_t W) {
  return norm_check(x, x_row, gate, gate_row, gate_fn, post_weight, group, weight, weight_dtype,
                    eps, residual, residual_out, residual_dtype, residual_scale, out, R, W);
}

int kda_norm(const void* x, int64_t x_row, const void* gate, int64_t gate_row, int gate_fn,
             const void* post_weight, int64_t group, const void* weight, int weight_dtype,
             float eps, const void* residual, void* residual_out, int residual_dtype,
             float residual_scale, void* out, int64_t R, int64_t W, void* stream) {
  const int st = norm_check(x, x_row, gate, gate_row, gate_fn, post_weight, group, weight,
                            weight_dtype, eps, residual, residual_out, residual_dtype,
                            residual_scale, out, R, W);
  if (st != KDA_OK || R == 0) return st;
  kda::NormParams p = {};
  p.x = static_cast<const uint16_t*>(x);
  p.gate = static_cast<const uint16_t*>(gate);
  p.post_w = post_weight;
  p.w = weight;
  p.res = residual;
  p.res_out = residual_out;
  p.out = static_cast<uint16_t*>(out);
  p.x_row = x_row;
  p.gate_row = gate_row;
  p.group = static_cast<int32_t>(post_weight ? group : 8);
  p.pieces = 1;
  // groups that nothing couples: pieces of a row fill the device as rows of their own
  const int64_t piece = weight || (post_weight && group == W) ? W : kda::norm_piece(W, p.group);
  if (W > 2048 && piece >= 512) p.pieces = static_cast<int32_t>(W / piece);
  p.W = static_cast<int32_t>(W / p.pieces);
  p.items = R * p.pieces;
  p.silu = gate_fn == KDA_GATE_SILU;
  p.w_fp32 = weight_dtype == KDA_DTYPE_FP32;
  p.res_fp32 = residual_dtype == KDA_DTYPE_FP32;
  p.eps = eps;
  p.alpha = residual_scale;
  return status(kda::launch_norm(p, static_cast<hipStream_t>(stream)));
}

int kda_rope_check(const void* q, int64_t q_row, const void* q_out, int64_t q_out_row,
                   const void* k, int64_t k_row, const void* k_out, int64_t k_out_row,
                   const double* freqs, int64_t rot, float amplitude, int interleaved, int inverse,
                   const int64_t* positions, const int64_t* offsets, const int64_t* cu_seqlens,
                   int64_t num_seqs, int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t D) {
  (void)interleaved;
  (void)inverse;
  return rope_check(q, q_row, q_out, q_out_row, k, k_row, k_out, k_out_row, freqs, rot, amplitude,
                    positions, offsets, cu_seqlens, num_seqs, B, T, Hq, Hk, D);
}

int kda_rope(const void* q, int64_t q_row, void* q_out, int64_t q_out_row, const void* k,
             int64_t k_row, void* k_out, int64_t k_out_row, const double* freqs, int64_t rot,
             float amplitude, int interleaved, int inverse, const int64_t* positions,
             const int64_t* offsets, const int64_t* cu_seqlens, int64_t num_seqs, int64_t B,
             int64_t T, int64_t Hq, int64_t Hk, int64_t D, void* stream) {
  const int st = rope_check(q, q_row, q_out, q_out_row, k, k_row, k_out, k_out_row, freqs, rot,
                            amplitude, positions, offsets, cu_seqlens, num_seqs, B, T, Hq, Hk, D);
  if (st != KDA_OK || B * T == 0) return st;
  kda::RopeParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_out = static_cast<uint16_t*>(k_out);
  p.freqs = freqs;
  p.pos = positions;
  p.offsets = offsets;
  p.cu = cu_seqlens;
  p.q_row = q_row;
  p.k_row = k_row;
  p.q_out_row = q_out_row;
  p.k_out_row = k_out_row;
  p.T = T;
  p.tokens = B * T;
  p.N = static_cast<int32_t>(num_seqs);
  p.Hq = static_cast<int32_t>(Hq);
  p.Hk = static_cast<int32_t>(Hk);
  p.D = static_cast<int32_t>(D);
  p.rot = static_cast<int32_t>(rot);
  p.q_copy = q != q_out;
  p.k_copy = k != k_out;
  p.interleaved = interleaved != 0;
  p.amplitude = amplitude;
  p.sign = inverse ? -1.f : 1.f;
  kda::rope_schedule(p);
  return status(kda::launch_rope(p, static_cast<hipStream_t>(stream)));
}

int kda_cache4_put_check(const void* k, int64_t k_row, const void* v, int64_t v_row,
                         const void* k4, const void* ks, const void* v4, const void* vs,
                         int64_t num_slots, int64_t cap, const void* k_out, const void* v_out,
                         const int64_t* offsets, const int64_t* slots, const int64_t* cu_seqlens,
                         int64_t num_seqs, int64_t B, int64_t T, int64_t Hk, int64_t D) {
  return put4_check(k, k_row, v, v_row, k4, ks, v4, vs, num_slots, cap, k_out, v_out, offsets,
                    slots, cu_seqlens, num_seqs, B, T, Hk, D);
}

int kda_cache4_put(const void* k, int64_t k_row, const void* v, int64_t v_row, void* k4, void* ks,
                   void* v4, void* vs, int64_t num_slots, int64_t cap, void* k_out, void* v_out,
                   const int64_t* offsets, const int64_t* slots, const int64_t* cu_seqlens,
                   int64_t num_seqs, int64_t B, int64_t T, int64_t Hk, int64_t D, void* stream) {
  const int st = put4_check(k, k_row, v, v_row, k4, ks, v4, vs, num_slots, cap, k_out, v_out,
                            offsets, slots, cu_seqlens, num_seqs, B, T, Hk, D);
  if (st != KDA_OK || B * T == 0) return st;
  kda::Put4Params p = {};
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.c = cache_of(k4, ks, v4, vs, num_slots, cap);
  p.k_out = static_cast<uint16_t*>(k_out);
  p.v_out = static_cast<uint16_t*>(v_out);
  p.offsets = offsets;
  p.slot = slots;
  p.cu = cu_seqlens;
  p.k_row = k_row;
  p.v_row = v_row;
  p.T = T;
  p.tokens = B * T;
  p.N = static_cast<int32_t>(num_seqs);
  p.Hk = static_cast<int32_t>(Hk);
  return status(kda::launch_put4(p, static_cast<int>(D), static_cast<hipStream_t>(stream)));
}

int64_t kda_attn4_workspace_bytes(int64_t num_seqs, int64_t Bq, int64_t Tq, int64_t cap,
                                  int64_t Hq, int64_t Hk, int64_t D, int64_t part) {
  Plan4 plan = {};
  const int st = attn4_plan(num_seqs, Bq, Tq, cap, Hq, Hk, D, part, true, &plan);
  return st != KDA_OK ? st : plan.bytes;
}

int kda_attn4_fwd_check(const void* q, int64_t q_row, const void* k4, const void* ks,
                        const void* v4, const void* vs, int64_t num_slots, int64_t cap,
                        float scale, const void* out, const float* lse,
                        const int64_t* cu_seqlens_q, const int64_t* k_lens, const int64_t* slots,
                        int64_t num_seqs, int64_t Bq, int64_t Tq, int64_t Hq, int64_t Hk,
                        int64_t D, int64_t part, const void* workspace, int64_t workspace_bytes) {
  Plan4 plan = {};
  return attn4_check(q, q_row, k4, ks, v4, vs, num_slots, cap, scale, out, lse, cu_seqlens_q,
                     k_lens, slots, num_seqs, Bq, Tq, Hq, Hk, D, part, workspace, workspace_bytes,
                     &plan);
}

int kda_attn4_fwd(const void* q, int64_t q_row, const void* k4, const void* ks, const void* v4,
                  const void* vs, int64_t num_slots, int64_t cap, float scale, void* out,
                  float* lse, const int64_t* cu_seqlens_q, const int64_t* k_lens,
                  const int64_t* slots, int64_t num_seqs, int64_t Bq, int64_t Tq, int64_t Hq,
                  int64_t Hk, int64_t D, int64_t part, void* workspace, int64_t workspace_bytes,
                  void* stream) {
  Plan4 plan = {};
  const int st = attn4_check(q, q_row, k4, ks, v4, vs, num_slots, cap, scale, out, lse,
                             cu_seqlens_q, k_lens, slots, num_seqs, Bq, Tq, Hq, Hk, D, part,
                             workspace, workspace_bytes, &plan);
  if (st != KDA_OK || Bq * Tq == 0) return st;
  kda::Attn4Params p = {};
  kda::AttnParams& a = p.a;
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.cu_q = cu_seqlens_q;
  a.k_lens = k_lens;
  a.q_row = q_row;
  a.Tq = Tq;
  a.Tk = cap;
  a.Tq_total = Bq * Tq;
  a.N = static_cast<int32_t>(num_seqs);
  a.Hq = static_cast<int32_t>(Hq);
  a.Hk = static_cast<int32_t>(Hk);
  a.G = static_cast<int32_t>(Hq / Hk);
  a.c = kda::attn_factor(scale);
  p.c = cache_of(k4, ks, v4, vs, num_slots, cap);
  p.slot = slots;
  p.part = static_cast<int32_t>(plan.part / kCache4Tile);
  // loads that do not stay in the caches: 10% of a batch of single tokens over long caches, but
  // several tiles of rows read a sequence's keys from there (their times rise by up to a sixth)
  p.once = a.Tq_total * a.G <= num_seqs * kda::kAttn4Rows;
  hipStream_t const on = static_cast<hipStream_t>(stream);
  a.splits = static_cast<int32_t>(plan.expand ? plan.splits : (cap + plan.part - 1) / plan.part);
  char* ws = static_cast<char*>(workspace);
  if (plan.expand) {
    const int64_t half = num_seqs * cap * Hk * D * 2;
    p.k_ws = reinterpret_cast<uint16_t*>(ws);
    p.v_ws = reinterpret_cast<uint16_t*>(ws + half);
    p.lens = reinterpret_cast<int64_t*>(ws + 2 * half);
    ws += 2 * half + round16(num_seqs * 8);
  }
  if (a.splits > 1) {
    a.ws_o = reinterpret_cast<float*>(ws);
    a.ws_ml = a.ws_o + a.splits * a.Tq_total * Hq * D;
  }
  if (!plan.expand) return status(kda::launch_attn4(p, static_cast<int>(D), on));
  const hipError_t e = kda::launch_expand4(p, static_cast<int>(D), on);
  if (e != hipSuccess) return status(e);
  a.k = p.k_ws;
  a.v = p.v_ws;
  a.k_row = a.v_row = Hk * D;
  a.k_lens = p.lens;
  return status(kda::launch_attn(a, plan.sched, static_cast<int>(D), on));
}

}  // extern "C"
