// Host side of the serving operators declared in include/kda.h: argument validation,
// schedule selection and launches.  Nothing here touches device memory.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <limits>

#include "../../include/kda.h"
#include "api_util.h"
#include "ops_params.h"

namespace {

using kda::make_range;
using kda::overlaps;
using kda::Range;

constexpr int64_t kMaxBytes = (int64_t)1 << 62;  // of one tensor: the range arithmetic cannot wrap

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

bool state_dtype_ok(int dtype) { return dtype == KDA_DTYPE_BF16 || dtype == KDA_DTYPE_FP32; }

// A row stride in elements: whole 16-byte units, at least the row itself.
bool row_ok(int64_t row, int64_t heads, int64_t D) { return row >= heads * D && row % 8 == 0; }

// Bytes from the first element of `rows` bf16 rows to the last, or -1 beyond kMaxBytes.
int64_t span_bytes(int64_t rows, int64_t row, int64_t heads, int64_t D) {
  if (rows <= 0) return 0;
  if (row > kMaxBytes / 2 / rows) return -1;
  return ((rows - 1) * row + heads * D) * 2;
}

bool any_overlap(Range out, const Range* ins, int n) {
  for (int i = 0; i < n; ++i)
    if (overlaps(out, ins[i])) return true;
  return false;
}

// What kda_step and kda_la_step share: sizes, the pool, the slots.
int step_resolve(const void* state, int state_dtype, int64_t num_slots, const int64_t* slot_in,
                 const int64_t* slot_out, float scale, int64_t N, int64_t H, int64_t D) {
  if (N < 0 || H < 1 || num_slots < 1) return KDA_ERR_BAD_SHAPE;
  if (D != 32 && D != 64 && D != 128) return KDA_ERR_BAD_SHAPE;
  // one launch covers at most 2^32 - 1 work-items: N * H workgroups of up to 256 threads
  // (more, smaller ones only while they are few)
  if (H >= ((int64_t)1 << 24) || (N > 0 && N > (((int64_t)1 << 24) - 1) / H))
    return KDA_ERR_BAD_SHAPE;
  if (num_slots > kMaxBytes / (H * D * D * 4)) return KDA_ERR_BAD_SHAPE;
  if (!state_dtype_ok(state_dtype)) return KDA_ERR_BAD_DTYPE;
  if (!std::isfinite(scale)) return KDA_ERR_BAD_SCALE;
  // without slots request n reads (and without slot_out writes) slot n
  if (!slot_in && N > num_slots) return KDA_ERR_BAD_SHAPE;
  if (!state) return KDA_ERR_NULL_ARG;
  if (!aligned16(state)) return KDA_ERR_BAD_LAYOUT;
  return KDA_OK;
}

int step_check(const void* q, const void* k, const void* v, const void* g, const void* beta,
               float scale, const void* out, const float* A_log, const float* dt_bias,
               float lower_bound, const void* state, int state_dtype, int64_t num_slots,
               const int64_t* slot_in, const int64_t* slot_out, int64_t N, int64_t H, int64_t D) {
  const int st = step_resolve(state, state_dtype, num_slots, slot_in, slot_out, scale, N, H, D);
  if (st != KDA_OK) return st;
  if (!A_log || !dt_bias || (N > 0 && (!q || !k || !v || !g || !beta || !out)))
    return KDA_ERR_NULL_ARG;
  if (!std::isfinite(lower_bound) || !(lower_bound < 0.f)) return KDA_ERR_BAD_LOWER_BOUND;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(out))
    return KDA_ERR_BAD_LAYOUT;
  const int64_t act = N * H * D * 2;
  const Range ro = make_range(out, act),
              rp = make_range(state, num_slots * H * D * D * (state_dtype ? 4 : 2));
  const Range ins[] = {make_range(q, act), make_range(k, act), make_range(v, act),
                       make_range(g, act), make_range(beta, N * H * 2), make_range(A_log, H * 4),
                       make_range(dt_bias, H * D * 4), make_range(slot_in, slot_in ? N * 8 : 0),
                       make_range(slot_out, slot_out ? N * 8 : 0)};
  if (any_overlap(ro, ins, 9) || any_overlap(rp, ins, 9) || overlaps(ro, rp))
    return KDA_ERR_BAD_ALIAS;
  return KDA_OK;
}

int la_step_check(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
                  int64_t v_row, const float* g, const float* decay, float scale, const void* out,
                  const void* state, int state_dtype, int64_t num_slots, const int64_t* slot_in,
                  const int64_t* slot_out, int64_t N, int64_t H, int64_t Hk, int64_t D) {
  const int st = step_resolve(state, state_dtype, num_slots, slot_in, slot_out, scale, N, H, D);
  if (st != KDA_OK) return st;
  if (Hk < 1 || H % Hk != 0) return KDA_ERR_BAD_SHAPE;
  if (N > 0 && (!q || !k || !v || !out)) return KDA_ERR_NULL_ARG;
  if (!row_ok(q_row, Hk, D) || !row_ok(k_row, Hk, D) || !row_ok(v_row, H, D) || !aligned16(q) ||
      !aligned16(k) || !aligned16(v) || !aligned16(out))
    return KDA_ERR_BAD_LAYOUT;
  const int64_t bq = span_bytes(N, q_row, Hk, D), bk = span_bytes(N, k_row, Hk, D),
                bv = span_bytes(N, v_row, H, D);
  if (bq < 0 || bk < 0 || bv < 0) return KDA_ERR_BAD_SHAPE;
  const Range ro = make_range(out, N * H * D * 2),
              rp = make_range(state, num_slots * H * D * D * (state_dtype ? 4 : 2));
  const Range ins[] = {make_range(q, bq), make_range(k, bk), make_range(v, bv),
                       make_range(g, g ? N * H * 4 : 0), make_range(decay, decay ? H * 4 : 0),
                       make_range(slot_in, slot_in ? N * 8 : 0),
                       make_range(slot_out, slot_out ? N * 8 : 0)};
  if (any_overlap(ro, ins, 7) || any_overlap(rp, ins, 7) || overlaps(ro, rp))
    return KDA_ERR_BAD_ALIAS;
  return KDA_OK;
}

// Tokens per segment of kda_la_fwd when the caller leaves the choice, 0 for none: the least
// estimated time.  The host knows the sequences' mean length only.  The constants
// (microseconds, bytes per microsecond) are fitted to 130 measured calls, 1-4 sequences of
// 512-32,768 tokens, 1-128 heads, D 64 and 128, with and without segments: the choice costs
// 2% over the best of each on average.  (23.4: 21 as fitted, and 2.4 for the launch that carries
// infinities and NaN on, 2.2 to 2.6 in the same calls.)
int64_t la_auto_segment(int64_t T_total, int64_t N, int64_t H, int64_t D) {
  const double units = double(N) * H, mean = double(T_total) / N, chunk = kda::kLaChunk;
  const double room = 2.0 * kda::device_cus();  // workgroups at once
  const double bytes = 8.0 * T_total * H * D;
  // one workgroup walks a sequence's chunks, unless HBM bounds the call
  double best = 9.0 + std::fmax((2.2 + 0.0136 * D) * std::ceil(mean / chunk) *
                                    std::fmax(1.0, units / room), bytes / 4.4e6);
  int64_t choice = 0;
  for (int64_t seg = 2 * kda::kLaChunk; 2 * seg <= mean && seg <= (1 << 20); seg *= 2) {
    // two passes over a segment's chunks and a scan over the segments, or the bytes: k and v
    // twice (the first pass ends where the decay is zero), each segment's state four times
    const double walk = (2.1 + 0.017 * D) * (seg / chunk) + 0.25 * mean / seg;
    const double move = (1.35 * bytes + 16.0 * D * D * H * (double(T_total) / seg)) / 4.6e6;
    const double t = 23.4 + std::fmax(walk, move) + 0.13 * std::fmin(walk, move);
    if (t < best) {
      best = t;
      choice = seg;
    }
  }
  return choice;
}

// A segment length as given (0: automatic) to the one used, or a negative status.
int64_t la_segment(int64_t T_total, int64_t N, int64_t H, int64_t D, int64_t segment) {
  if (segment < 0 || segment % kda::kLaChunk != 0 || segment > (1 << 20))
    return KDA_ERR_BAD_SCHEDULE;
  return segment ? segment : la_auto_segment(T_total, N, H, D);
}

// Whether every launch of a la call stays below 2^32 work-items and its slots in range.
bool la_grid_ok(int64_t T_total, int64_t N, int64_t H, int64_t seg) {
  const int64_t most = (((int64_t)1 << 32) - 1) / 512 / 8;  // eight workgroups of 512 threads
  const int64_t items = seg ? kda::la_slots(T_total, N, seg) : N;
  if (items > most * 8 / H - 8) return false;
  return !seg || N <= most / H / 2;  // the scan: up to 16 workgroups per (sequence, head)
}

// Bytes of the workspace of a la call in segments of seg tokens, or a negative status.
int64_t la_ws_bytes(int64_t T_total, int64_t N, int64_t H, int64_t D, int64_t seg) {
  if (seg == 0) return 0;
  if (!la_grid_ok(T_total, N, H, seg)) return KDA_ERR_BAD_SHAPE;
  return kda::la_ws_floats(kda::la_slots(T_total, N, seg), H, D) * 4;
}

// The sizes of a packed or batched call; num_seqs sequences.
int batch_ok(const int64_t* cu, int64_t N, int64_t B, int64_t T) {
  if (B < 1 || T < 0) return KDA_ERR_BAD_SHAPE;
  if (T == 0 && !cu) return KDA_ERR_BAD_SHAPE;
  if (T > ((int64_t)1 << 40) / B) return KDA_ERR_BAD_SHAPE;
  if (cu ? (B != 1 || N < 1) : N != B) return KDA_ERR_BAD_VARLEN;
  return KDA_OK;
}

int la_check(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
             int64_t v_row, const float* g, const float* decay, float scale, const void* out,
             const void* s_in, int in_dtype, const void* s_out, int out_dtype, const int64_t* cu,
             int64_t N, int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t D, int64_t segment,
             const void* workspace, int64_t workspace_bytes, int64_t* seg_out) {
  if (D != 32 && D != 64 && D != 128) return KDA_ERR_BAD_SHAPE;
  if (H < 1 || Hk < 1 || H % Hk != 0) return KDA_ERR_BAD_SHAPE;
  // a chunk's 64 token rows are addressed with 32-bit byte offsets
  if (H >= ((int64_t)1 << 24) / D || q_row >= (1 << 24) || k_row >= (1 << 24) ||
      v_row >= (1 << 24))
    return KDA_ERR_BAD_SHAPE;
  const int sizes = batch_ok(cu, N, B, T);
  if (sizes != KDA_OK) return sizes;
  const int64_t tok = B * T;
  if (N > (((int64_t)1 << 31) - 1) / H || !la_grid_ok(tok, N, H, 0)) return KDA_ERR_BAD_SHAPE;
  if ((s_in && !state_dtype_ok(in_dtype)) || (s_out && !state_dtype_ok(out_dtype)))
    return KDA_ERR_BAD_DTYPE;
  if (!std::isfinite(scale)) return KDA_ERR_BAD_SCALE;
  if (tok > 0 && (!q || !k || !v || !out)) return KDA_ERR_NULL_ARG;
  if (!row_ok(q_row, Hk, D) || !row_ok(k_row, Hk, D) || !row_ok(v_row, H, D) || !aligned16(q) ||
      !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(s_in) || !aligned16(s_out) ||
      !aligned16(workspace))
    return KDA_ERR_BAD_LAYOUT;
  int64_t seg = la_segment(tok, N, H, D, segment);
  if (seg < 0) return static_cast<int>(seg);
  if (segment == 0 && !workspace) seg = 0;  // left to the library: without one, no segments
  const int64_t need = la_ws_bytes(tok, N, H, D, seg);
  if (need < 0) return static_cast<int>(need);
  if (need > 0 && !workspace) return KDA_ERR_NULL_ARG;
  if (need > workspace_bytes) return KDA_ERR_BAD_WORKSPACE;

  const int64_t st = N * H * D * D;
  const Range ro = make_range(out, tok * H * D * 2),
              rs = make_range(s_out, s_out ? st * (out_dtype ? 4 : 2) : 0),
              ri = make_range(s_in, s_in ? st * (in_dtype ? 4 : 2) : 0),
              rw = make_range(workspace, need);
  const Range ins[] = {make_range(q, span_bytes(tok, q_row, Hk, D)),
                       make_range(k, span_bytes(tok, k_row, Hk, D)),
                       make_range(v, span_bytes(tok, v_row, H, D)),
                       make_range(g, g ? tok * H * 4 : 0),
                       make_range(decay, decay ? H * 4 : 0),
                       make_range(cu, cu ? (N + 1) * 8 : 0)};
  if (any_overlap(ro, ins, 6) || any_overlap(rs, ins, 6) || any_overlap(rw, ins, 6))
    return KDA_ERR_BAD_ALIAS;
  if (overlaps(ro, rs) || overlaps(ro, ri) || overlaps(ro, rw) || overlaps(rs, rw) ||
      overlaps(ri, rw))
    return KDA_ERR_BAD_ALIAS;
  if (overlaps(rs, ri) && !(s_in == s_out && in_dtype == out_dtype)) return KDA_ERR_BAD_ALIAS;
  *seg_out = seg;
  return KDA_OK;
}

// Parts of each row's keys when the caller leaves the choice, from a sequence's mean number
// of keys.  Single tokens: one workgroup per compute unit, from 1024 keys on and at least 256
// a part (8192 keys, 8 key/value heads: 80 us in one part, 14 in 32; 4 such sequences of 4096
// keys: 48 and 16 in 8; 32 sequences: more parts only cost).  Tiles of rows: two workgroups
// per compute unit and at least 512 keys a part, or 1024 when every second unit has a tile
// anyway (256 queries, 8192 keys, 32/8 heads: 161 us in one part, 51 in 8; 1024 queries and
// keys: 27 in one, 38 in two, whose partial results cost more than they save).
int64_t attn_auto_splits(const kda::AttnSchedule& s, int64_t slots, int64_t Hk, int64_t mean_k) {
  const int64_t units = slots * Hk, cus = kda::device_cus();
  if (units < 1 || (s.tokens && mean_k < 1024)) return 1;
  int64_t n = (s.tokens ? cus : 2 * cus) / units;
  const int64_t least = s.tokens ? 256 : 2 * units < cus ? 512 : 1024;
  if (n > mean_k / least) n = mean_k / least;
  return n < 1 ? 1 : n > 64 ? 64 : n;
}

// Sizes of a kda_attn_fwd call to its schedule and splits.  Keys are packed when one row of
// keys serves several sequences (Bk == 1).
int attn_sizes(int64_t N, int64_t Bq, int64_t Tq, int64_t Bk, int64_t Tk, int64_t Hq, int64_t Hk,
               int64_t D, int64_t splits, kda::AttnSchedule* sched, int64_t* splits_out) {
  if (D != 64 && D != 128) return KDA_ERR_BAD_SHAPE;
  if (Hk < 1 || Hq < 1 || Hq % Hk != 0 || Hq >= (1 << 24)) return KDA_ERR_BAD_SHAPE;
  if (N < 1 || N >= ((int64_t)1 << 31) || Bq < 1 || Bk < 1 || Tq < 0 || Tk < 0)
    return KDA_ERR_BAD_SHAPE;
  if ((Bq != 1 && Bq != N) || (Bk != 1 && Bk != N)) return KDA_ERR_BAD_VARLEN;
  // rows and keys of a sequence are 32-bit numbers
  if (Tk > ((int64_t)1 << 30) || Tq > ((int64_t)1 << 30) / (Hq / Hk)) return KDA_ERR_BAD_SHAPE;
  if (Tq > ((int64_t)1 << 40) / Bq || Tk > ((int64_t)1 << 40) / Bk) return KDA_ERR_BAD_SHAPE;
  if (splits < 0 || splits > 64) return KDA_ERR_BAD_SCHEDULE;
  const int64_t G = Hq / Hk, total = Bq * Tq;
  *sched = kda::attn_schedule(total, N, G);
  // tiles of rows: for batch rows as many as each has, for packed ones a bound
  const int64_t slots = Bq == N ? N * ((Tq * G + sched->rows - 1) / sched->rows)
                                : kda::attn_slots(total, N, G, sched->rows);
  const int64_t mean_k = Bk == 1 ? Tk / N : Tk;
  int64_t sp = splits ? splits : attn_auto_splits(*sched, slots, Hk, mean_k);
  // every launch below 2^32 work-items
  const int64_t most = (((int64_t)1 << 32) - 1) / kda::kAttnThreads;
  const int64_t tiles = kda::attn_slots(total, N, G, sched->rows) + (Bq == N ? N : 0);
  if (tiles > most / Hk) return KDA_ERR_BAD_SHAPE;
  // ... the join's of four rows a workgroup among them
  if (sp > 1 && (tiles * Hk > most / sp || total > 4 * most / Hq)) {
    if (splits) return KDA_ERR_BAD_SHAPE;
    sp = 1;
  }
  *splits_out = sp;
  return KDA_OK;
}

int64_t attn_ws_bytes(int64_t total, int64_t Hq, int64_t D, int64_t splits) {
  return splits > 1 ? splits * total * Hq * (D + 2) * 4 : 0;
}

// The factor of the scores in base 2.
float attn_c(float scale) { return static_cast<float>(scale * 1.4426950408889634); }

int attn_check(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
               int64_t v_row, float scale, const void* out, const float* lse, const int64_t* cu_q,
               const int64_t* cu_k, const int64_t* k_lens, int64_t N, int64_t Bq, int64_t Tq,
               int64_t Bk, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, int64_t splits,
               const void* workspace, int64_t workspace_bytes, kda::AttnSchedule* sched,
               int64_t* splits_out) {
  int64_t sp = 1;
  const int st = attn_sizes(N, Bq, Tq, Bk, Tk, Hq, Hk, D, splits, sched, &sp);
  if (st != KDA_OK) return st;
  if ((cu_q ? Bq != 1 : Bq != N) || (cu_k ? Bk != 1 : Bk != N) || (cu_k && k_lens))
    return KDA_ERR_BAD_VARLEN;
  if (!std::isfinite(attn_c(scale)) || scale < 0.f) return KDA_ERR_BAD_SCALE;
  const int64_t nq = Bq * Tq, nk = Bk * Tk;
  if ((nq > 0 && (!q || !out)) || (nq > 0 && nk > 0 && (!k || !v))) return KDA_ERR_NULL_ARG;
  if (q_row >= (1 << 24) || k_row >= (1 << 24) || v_row >= (1 << 24)) return KDA_ERR_BAD_SHAPE;
  if (!row_ok(q_row, Hq, D) || !row_ok(k_row, Hk, D) || !row_ok(v_row, Hk, D) || !aligned16(q) ||
      !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(workspace))
    return KDA_ERR_BAD_LAYOUT;
  if (splits == 0 && !workspace) sp = 1;  // left to the library: without one, no splits
  const int64_t need = attn_ws_bytes(nq, Hq, D, sp);
  if (need > 0 && !workspace) return KDA_ERR_NULL_ARG;
  if (need > workspace_bytes) return KDA_ERR_BAD_WORKSPACE;
  const Range ro = make_range(out, nq * Hq * D * 2), rl = make_range(lse, lse ? nq * Hq * 4 : 0),
              rw = make_range(workspace, need);
  const Range ins[] = {make_range(q, span_bytes(nq, q_row, Hq, D)),
                       make_range(k, span_bytes(nk, k_row, Hk, D)),
                       make_range(v, span_bytes(nk, v_row, Hk, D)),
                       make_range(cu_q, cu_q ? (N + 1) * 8 : 0),
                       make_range(cu_k, cu_k ? (N + 1) * 8 : 0),
                       make_range(k_lens, k_lens ? N * 8 : 0)};
  if (any_overlap(ro, ins, 6) || any_overlap(rl, ins, 6) || any_overlap(rw, ins, 6) ||
      overlaps(ro, rl) || overlaps(ro, rw) || overlaps(rl, rw))
    return KDA_ERR_BAD_ALIAS;
  *splits_out = sp;
  return KDA_OK;
}

int status(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

}  // namespace

extern "C" {

int kda_step_check(const void* q, const void* k, const void* v, const void* g, const void* beta,
                   float scale, const void* out, const float* A_log, const float* dt_bias,
                   float lower_bound, const void* state, int state_dtype, int64_t num_slots,
                   const int64_t* slot_in, const int64_t* slot_out, int64_t N, int64_t H,
                   int64_t D) {
  return step_check(q, k, v, g, beta, scale, out, A_log, dt_bias, lower_bound, state, state_dtype,
                    num_slots, slot_in, slot_out, N, H, D);
}

int kda_step(const void* q, const void* k, const void* v, const void* g, const void* beta,
             float scale, void* out, const float* A_log, const float* dt_bias, float lower_bound,
             void* state, int state_dtype, int64_t num_slots, const int64_t* slot_in,
             const int64_t* slot_out, int64_t N, int64_t H, int64_t D, void* stream) {
  const int st = step_check(q, k, v, g, beta, scale, out, A_log, dt_bias, lower_bound, state,
                            state_dtype, num_slots, slot_in, slot_out, N, H, D);
  if (st != KDA_OK || N == 0) return st;
  kda::StepParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.gate = static_cast<const uint16_t*>(g);
  p.beta = static_cast<const uint16_t*>(beta);
  p.A_log = A_log;
  p.dt_bias = dt_bias;
  p.out = static_cast<uint16_t*>(out);
  p.state = state;
  p.slot_in = slot_in;
  p.slot_out = slot_out;
  p.num_slots = num_slots;
  p.q_row = p.k_row = p.v_row = H * D;
  p.N = static_cast<int32_t>(N);
  p.H = static_cast<int32_t>(H);
  p.group = 1;
  p.scale = scale;
  p.lower_bound = lower_bound;
  return status(kda::launch_step(p, true, static_cast<int>(D), state_dtype == KDA_DTYPE_FP32,
                                 static_cast<hipStream_t>(stream)));
}

int kda_la_step_check(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
                      int64_t v_row, const float* g, const float* decay, float scale,
                      const void* out, const void* state, int state_dtype, int64_t num_slots,
                      const int64_t* slot_in, const int64_t* slot_out, int64_t N, int64_t H,
                      int64_t Hk, int64_t D) {
  return la_step_check(q, q_row, k, k_row, v, v_row, g, decay, scale, out, state, state_dtype,
                       num_slots, slot_in, slot_out, N, H, Hk, D);
}

int kda_la_step(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
                int64_t v_row, const float* g, const float* decay, float scale, void* out,
                void* state, int state_dtype, int64_t num_slots, const int64_t* slot_in,
                const int64_t* slot_out, int64_t N, int64_t H, int64_t Hk, int64_t D,
                void* stream) {
  const int st = la_step_check(q, q_row, k, k_row, v, v_row, g, decay, scale, out, state,
                               state_dtype, num_slots, slot_in, slot_out, N, H, Hk, D);
  if (st != KDA_OK || N == 0) return st;
  kda::StepParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.g = g;
  p.decay = decay;
  p.out = static_cast<uint16_t*>(out);
  p.state = state;
  p.slot_in = slot_in;
  p.slot_out = slot_out;
  p.num_slots = num_slots;
  p.q_row = q_row;
  p.k_row = k_row;
  p.v_row = v_row;
  p.N = static_cast<int32_t>(N);
  p.H = static_cast<int32_t>(H);
  p.group = static_cast<int32_t>(H / Hk);
  p.scale = scale;
  return status(kda::launch_step(p, false, static_cast<int>(D), state_dtype == KDA_DTYPE_FP32,
                                 static_cast<hipStream_t>(stream)));
}

int64_t kda_la_workspace_bytes(int64_t T_total, int64_t num_seqs, int64_t H, int64_t D,
                               int64_t segment) {
  if (T_total < 0 || T_total > ((int64_t)1 << 40) || num_seqs < 1 || H < 1 ||
      (D != 32 && D != 64 && D != 128) || H >= ((int64_t)1 << 24) / D ||
      num_seqs > (((int64_t)1 << 31) - 1) / H)
    return KDA_ERR_BAD_SHAPE;
  const int64_t seg = la_segment(T_total, num_seqs, H, D, segment);
  return seg < 0 ? seg : la_ws_bytes(T_total, num_seqs, H, D, seg);
}

int kda_la_fwd_check(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
                     int64_t v_row, const float* g, const float* decay, float scale,
                     const void* out, const void* initial_state, int initial_state_dtype,
                     const void* final_state, int final_state_dtype, const int64_t* cu_seqlens,
                     int64_t num_seqs, int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t D,
                     int64_t segment, const void* workspace, int64_t workspace_bytes) {
  int64_t seg = 0;
  return la_check(q, q_row, k, k_row, v, v_row, g, decay, scale, out, initial_state,
                  initial_state_dtype, final_state, final_state_dtype, cu_seqlens, num_seqs, B, T,
                  H, Hk, D, segment, workspace, workspace_bytes, &seg);
}

int kda_la_fwd(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
               int64_t v_row, const float* g, const float* decay, float scale, void* out,
               const void* initial_state, int initial_state_dtype, void* final_state,
               int final_state_dtype, const int64_t* cu_seqlens, int64_t num_seqs, int64_t B,
               int64_t T, int64_t H, int64_t Hk, int64_t D, int64_t segment, void* workspace,
               int64_t workspace_bytes, void* stream) {
  int64_t seg = 0;
  const int st = la_check(q, q_row, k, k_row, v, v_row, g, decay, scale, out, initial_state,
                          initial_state_dtype, final_state, final_state_dtype, cu_seqlens,
                          num_seqs, B, T, H, Hk, D, segment, workspace, workspace_bytes, &seg);
  if (st != KDA_OK) return st;
  kda::LaParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.g = g;
  p.decay = decay;
  p.out = static_cast<uint16_t*>(out);
  p.s_in = initial_state;
  p.s_out = final_state;
  p.cu = cu_seqlens;
  p.q_row = q_row;
  p.k_row = k_row;
  p.v_row = v_row;
  p.T = T;
  p.T_total = B * T;
  p.N = static_cast<int32_t>(num_seqs);
  p.H = static_cast<int32_t>(H);
  p.group = static_cast<int32_t>(H / Hk);
  p.s_in_fp32 = initial_state_dtype == KDA_DTYPE_FP32 ? 1 : 0;
  p.s_out_fp32 = final_state_dtype == KDA_DTYPE_FP32 ? 1 : 0;
  p.scale = scale;
  p.seg = static_cast<int32_t>(seg);
  if (seg) {
    p.slots = kda::la_slots(B * T, num_seqs, seg);
    p.ws = static_cast<float*>(workspace);
    p.ws_decay = p.ws + p.slots * H * D * D;
  }
  return status(kda::launch_la(p, static_cast<int>(D), static_cast<hipStream_t>(stream)));
}

int64_t kda_attn_workspace_bytes(int64_t num_seqs, int64_t Bq, int64_t Tq, int64_t Bk, int64_t Tk,
                                 int64_t Hq, int64_t Hk, int64_t D, int64_t splits) {
  kda::AttnSchedule sched;
  int64_t sp = 1;
  const int st = attn_sizes(num_seqs, Bq, Tq, Bk, Tk, Hq, Hk, D, splits, &sched, &sp);
  return st != KDA_OK ? st : attn_ws_bytes(Bq * Tq, Hq, D, sp);
}

int kda_attn_fwd_check(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
                       int64_t v_row, float scale, const void* out, const float* lse,
                       const int64_t* cu_seqlens_q, const int64_t* cu_seqlens_k,
                       const int64_t* k_lens, int64_t num_seqs, int64_t Bq, int64_t Tq, int64_t Bk,
                       int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, int64_t splits,
                       const void* workspace, int64_t workspace_bytes) {
  kda::AttnSchedule sched;
  int64_t sp = 1;
  return attn_check(q, q_row, k, k_row, v, v_row, scale, out, lse, cu_seqlens_q, cu_seqlens_k,
                    k_lens, num_seqs, Bq, Tq, Bk, Tk, Hq, Hk, D, splits, workspace,
                    workspace_bytes, &sched, &sp);
}

int kda_attn_fwd(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
                 int64_t v_row, float scale, void* out, float* lse, const int64_t* cu_seqlens_q,
                 const int64_t* cu_seqlens_k, const int64_t* k_lens, int64_t num_seqs, int64_t Bq,
                 int64_t Tq, int64_t Bk, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D,
                 int64_t splits, void* workspace, int64_t workspace_bytes, void* stream) {
  kda::AttnSchedule sched;
  int64_t sp = 1;
  const int st = attn_check(q, q_row, k, k_row, v, v_row, scale, out, lse, cu_seqlens_q,
                            cu_seqlens_k, k_lens, num_seqs, Bq, Tq, Bk, Tk, Hq, Hk, D, splits,
                            workspace, workspace_bytes, &sched, &sp);
  if (st != KDA_OK || Bq * Tq == 0) return st;
  kda::AttnParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k;
  p.k_lens = k_lens;
  p.q_row = q_row;
  p.k_row = k_row;
  p.v_row = v_row;
  p.Tq = Tq;
  p.Tk = Tk;
  p.Tq_total = Bq * Tq;
  p.N = static_cast<int32_t>(num_seqs);
  p.Hq = static_cast<int32_t>(Hq);
  p.Hk = static_cast<int32_t>(Hk);
  p.G = static_cast<int32_t>(Hq / Hk);
  // never zero: minus infinity times it stands for a masked score.  The smallest float in
  // place of zero moves a finite score by 2^-21 at most, six roundings of its exponential.
  p.c = std::fmax(attn_c(scale), std::numeric_limits<float>::denorm_min());
  p.splits = static_cast<int32_t>(sp);
  p.ws_o = static_cast<float*>(workspace);
  p.ws_ml = sp > 1 ? p.ws_o + sp * p.Tq_total * Hq * D : nullptr;
  return status(
      kda::launch_attn(p, sched, static_cast<int>(D), static_cast<hipStream_t>(stream)));
}

}  // extern "C"
