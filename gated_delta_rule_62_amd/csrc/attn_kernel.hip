// Causal softmax attention with grouped heads (kda_attn_fwd), for gfx950.
//
// Query i of a sequence with Lq queries and Lk keys sees keys j <= i + Lk - Lq:
//     x_ij = scale q_i . k_j,   out_i = sum_j e^{x_ij} v_j / sum_j e^{x_ij},
//     lse_i = log sum_j e^{x_ij}     (no visible key: out 0, lse minus infinity).
//
// Rows.  The G query heads of a key/value head read the same keys, so a row is a pair
// (query token, head of the group): row r is token r / G, head r % G.  A workgroup owns a
// tile of rows of one key/value head whatever G is, and a single token already fills G of
// them.
//
// One pass over the keys with a running maximum and sum.  Both products keep the row in
// the accumulator's column, x^T = K Q^T and out^T = V^T P^T: a lane then holds one row
// (l % 16) and four keys, so the maximum, the sum and the rescaling factor are one value
// per lane and tile, two cross-lane steps reduce a row, and two accumulator tiles of P^T
// pack into the operand of the second product without passing through LDS (V^T is read
// transposed from LDS in the same key order).  The maximum is only raised when a row
// outgrows it by 2^8 (a published refinement of the running maximum): p then reaches 256 at
// most, which costs no accuracy in a float, and almost every step skips the rescaling of the
// output.  p is rounded to bf16 for the product, at most half a bf16 step of each term's
// absolute value (the sum uses the unrounded p); a second part would be half as many products
// again.  The kernel for few rows, bound by its loads, takes a second bf16 part of p.
//
// Infinities and NaN of v behind a row's last key would reach it through the product, as zero
// times them.  On the diagonal's tiles they are dropped from LDS, and what they mean for the
// rows that do see them is added after the loop (looking for them: under 1% of a prompt).
//
// Few rows leave the device idle; then `splits` workgroups share a tile's keys, write
// unnormalised fp32 outputs with their maximum and sum, and a second kernel joins them.
//
// Measured (D 128): 8192 tokens of 32/8 heads 520-542 us, 1.01-1.05 PFLOP/s, where the matrix
// products alone take 400 at the clock they bring the card down to; one token of each of 32
// requests over 1024-8192 keys, 32/8 heads, 121 us, 5.0 TB/s, as its loads alone.
#include "api_util.h"
#include "attn_rows.h"
#include "gfx950.h"
#include "ops_params.h"

namespace kda {
namespace {

using namespace dev;

// Tile number `slot` with the tiles that see the most keys first, as workgroups start in order and a
// long one that starts last would set the time: batch rows by their tile, packed sequences
// (of up to 16: the ranking costs a short workgroup more than it gains with many) longest
// keys first, each from its last tile.  Whole waves call it.
__device__ __forceinline__ bool find_tile_longest_first(const AttnParams& p, unsigned slot,
                                                        unsigned slots, int tile_rows, Tile& t) {
  int n;
  int64_t row0;
  if (p.cu_q == nullptr) {
    const int64_t per = (p.Tq * p.G + tile_rows - 1) / tile_rows;
    n = (int)(slot % (unsigned)p.N);
    row0 = (per - 1 - slot / (unsigned)p.N) * tile_rows;
  } else if (p.N > 16) {
    return find_tile(p, slots - 1 - slot, tile_rows, t);
  } else {
    // lane l: keys and tiles of sequence l, and the tiles of all that come before it
    const int lane = threadIdx.x & 63;
    int64_t a = 0, b = 0, c = 0, d = 0;
    if (lane < p.N) {
      query_bounds(p, lane, a, b);
      key_bounds(p, lane, c, d);
    }
    const int keys = (int)(d - c), tiles = (int)(((b - a) * p.G + tile_rows - 1) / tile_rows);
    int before = 0;
    for (int m = 0; m < p.N; ++m) {
      const int k = __builtin_amdgcn_readlane(keys, m), x = __builtin_amdgcn_readlane(tiles, m);
      if (k > keys || (k == keys && m < lane)) before += x;
    }
    const int mine = (int)slot - before;
    const uint64_t has = __ballot(lane < p.N && mine >= 0 && mine < tiles);
    if (has == 0) return false;
    n = __builtin_ctzll(has);
    row0 = (int64_t)(__builtin_amdgcn_readlane(tiles, n) - 1 -
                     __builtin_amdgcn_readlane(mine, n)) * tile_rows;
  }
  return set_tile(p, __builtin_amdgcn_readfirstlane(n), row0, t);
}

// Descriptor of `tokens` rows of one head from `base`; nothing when there are none.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const u16* base, int64_t row,
                                                            int tokens, int D) {
  return make_rsrc(base, tokens > 0 ? (uint32_t)(tokens - 1) * (uint32_t)(row * 2) + D * 2u : 0u);
}

__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// Probability tiles 2 js and 2 js + 1 as the operand of 32 keys.
__device__ __forceinline__ u32x4_t p_op(f32x4_t a, f32x4_t b) {
  return u32x4_t{pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(b[0], b[1]),
                 pack_bf16(b[2], b[3])};
}

// What infinities and NaN of v add to the rows that see them, 32 keys: `key` is the first of
// this lane's (key .. + 3 and key + 16 .. + 19), vt(d) the operand of v's 16-column tile d.
template <int D, int NI, class V>
__device__ __forceinline__ void add_odd(Acc<D, NI>& acc, int key, const int (&last)[NI], V vt) {
  u32x4_t sees[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int k = key + 16 * (e >> 1) + 2 * (e & 1);
      sees[i][e] = (k <= last[i] ? 0x3f80u : 0u) | (k + 1 <= last[i] ? 0x3f800000u : 0u);
    }
#pragma unroll
  for (int d = 0; d < D / 16; ++d) {
    u32x4_t code = vt(d);
#pragma unroll
    for (int e = 0; e < 4; ++e) code[e] = odd_split(code[e]).code;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const f32x4_t n = mfma(code, sees[i], f32x4_t{0.f, 0.f, 0.f, 0.f});
#pragma unroll
      for (int r = 0; r < 4; ++r)
        acc.o[d][i][r] += odd_value(n[r]);
    }
  }
}

// Lane `lane` of a group of `lanes` looks at its part of n bf16 in LDS; whether its wave found
// any that is not finite.
__device__ __forceinline__ bool any_odd(const u16* v, int n, int lane, int lanes) {
  float zero = 0.f;
#pragma unroll 4
  for (int e = lane * 8; e < n; e += lanes * 8) {
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(v + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) zero = dot_zero(w[i], zero);
  }
  return __any(zero != zero);
}
// The same part with zeros in their place.
__device__ __forceinline__ void drop_odd(u16* v, int n, int lane, int lanes) {
#pragma unroll 1
  for (int e = lane * 8; e < n; e += lanes * 8) {
    u32x4_t w = *reinterpret_cast<const u32x4_t*>(v + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = odd_split(w[i]).finite;
    *reinterpret_cast<u32x4_t*>(v + e) = w;
  }
}

// One row's outputs, or with several splits its partial ones.  l is the whole sum.
template <int D>
__device__ __forceinline__ void store_row(const AttnParams& p, int64_t token, int head, int split,
                                          int lg, const f32x4_t* o, float m, float l) {
  const int64_t at = token * p.Hq + head;
  if (p.splits > 1) {
    const int64_t w = (int64_t)split * p.Tq_total * p.Hq + at;
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
      *reinterpret_cast<f32x4_t*>(p.ws_o + w * D + 16 * d + 4 * lg) = o[d];
    if (lg == 0) *reinterpret_cast<f32x2_t*>(p.ws_ml + 2 * w) = f32x2_t{m, l};
    return;
  }
  const float f = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // no key: zero; NaN stays
#pragma unroll
  for (int d = 0; d < D / 16; ++d)
    *reinterpret_cast<u32x2_t*>(p.out + at * D + 16 * d + 4 * lg) =
        u32x2_t{pack_bf16(o[d][0] * f, o[d][1] * f), pack_bf16(o[d][2] * f, o[d][3] * f)};
  if (p.lse != nullptr && lg == 0)
    p.lse[at] = l == 0.f ? kNone : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// ---- prompts: four waves share the keys' tiles in LDS, each owns NI 16-row tiles.
template <int D, int NI>
__global__ __launch_bounds__(kAttnThreads, 2) void attn_tile_kernel(AttnParams p) {
  constexpr int BN = kAttnKeys, JT = BN / 16, KS = D / 32, DT = D / 16;
  constexpr int ROWS = 4 * 16 * NI;
  __shared__ alignas(1024) u16 sk[2][BN][D];
  __shared__ alignas(1024) u16 sv[2][BN][D];
  __shared__ unsigned sodd[2][4];  // per wave: its quarter of a v tile is not all finite

  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // a key/value head's tiles share an XCD and its L2 (blocks go to the XCDs round robin)
  const unsigned units = gridDim.x / (unsigned)p.splits;
  const int split = (int)(blockIdx.x / units);
  const unsigned unit = blockIdx.x % units;
  const int hk = (int)(unit % (unsigned)p.Hk);
  Tile t;
  if (!find_tile_longest_first(p, unit / (unsigned)p.Hk, units / (unsigned)p.Hk, ROWS, t)) return;

  // ---- this wave's rows: their operand of the first product, their last visible key
  const int off = t.Lk - t.Lq;
  const int wrow = t.row0 + wave * 16 * NI;
  u32x4_t q[KS][NI];
  int last[NI];
  int64_t tok[NI];
  int head[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = wrow + 16 * i + l16;
    const int w = r / p.G;
    tok[i] = t.q0 + w;
    head[i] = hk * p.G + r % p.G;
    last[i] = r < t.rows ? w + off : -1;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) q[ks][i] = u32x4_t{0u, 0u, 0u, 0u};
    if (r < t.rows) {
      const u16* src = p.q + tok[i] * p.q_row + head[i] * D + 8 * lg;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) q[ks][i] = *reinterpret_cast<const u32x4_t*>(src + 32 * ks);
    }
  }
  end_loads(q);
  // keys some row of the tile, of this wave sees; keys every row of this wave sees
  const int tile_end = min(t.rows, t.row0 + ROWS) - 1;
  const int keys = max(0, min(t.Lk, tile_end / p.G + off + 1));
  const int wave_keys =
      wrow < t.rows ? max(0, min(t.Lk, (min(t.rows, wrow + 16 * NI) - 1) / p.G + off + 1)) : 0;
  const int all_keys = wrow / p.G + off + 1, tile_all_keys = t.row0 / p.G + off + 1;
  // this split's steps
  const int steps = (keys + BN - 1) / BN, per = (steps + p.splits - 1) / p.splits;
  const int first = min(steps, split * per), end = min(steps, first + per);

  // ---- K and V tiles go from memory straight into LDS, 1 KB (512 / D rows) per wave
  // instruction: through registers and back the copies cost an eighth of the time.  The
  // 16-byte pieces of a row are permuted, by exclusive or with the row, so that operand
  // reads of 16 rows fall in distinct banks without padding.
  constexpr int RPI = 512 / D;         // rows per instruction
  constexpr int IPW = BN / RPI / 4;    // instructions per wave and tile
  constexpr int PPR = D / 8;           // pieces per row
  auto swz = [](int row) { return D == 128 ? row & 15 : (row >> 1) & 7; };
  uint32_t koff[IPW], voff[IPW];
#pragma unroll
  for (int i = 0; i < IPW; ++i) {
    const int r = (wave * IPW + i) * RPI + lane / PPR;
    const uint32_t col = (uint32_t)((lane % PPR) ^ swz(r)) * 16u;
    koff[i] = (uint32_t)r * (uint32_t)(p.k_row * 2) + col;
    voff[i] = (uint32_t)r * (uint32_t)(p.v_row * 2) + col;
  }
  const u16* kb = p.k + t.k0 * p.k_row + hk * D;
  const u16* vb = p.v + t.k0 * p.v_row + hk * D;
  auto load = [&](int s) {
    const int valid = min(BN, t.Lk - s * BN);
    const u32x4_t dk = rows_words(kb + (int64_t)s * BN * p.k_row, p.k_row, valid, D),
                  dv = rows_words(vb + (int64_t)s * BN * p.v_row, p.v_row, valid, D);
#pragma unroll
    for (int i = 0; i < IPW; ++i) {
      load_lds<false>(dk, &sk[s & 1][(wave * IPW + i) * RPI][0], koff[i]);
      load_lds<false>(dv, &sv[s & 1][(wave * IPW + i) * RPI][0], voff[i]);
    }
  };

  Acc<D, NI> acc;
  acc.init();
  auto v_op = [&](int b, int row, int d) {
    const int c = ((2 * d + ((l16 & 3) >> 1)) ^ swz(row)) * 8 + 4 * (l16 & 1);
    const u32x2_t lo = ds_read_tr(&sv[b][row][c]), hi = ds_read_tr(&sv[b][row + 16][c]);
    return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
  };
  bool odd = false;  // some step dropped infinities or NaN of v
  if (first < end) load(first);
  for (int s = first; s < end; ++s) {
    const int b = s & 1;
    // this wave's part of tile s is in LDS; behind the barrier every wave's is, and all have
    // read tile s - 1, whose buffer takes tile s + 1
    wait_loads();
    const bool diagonal = (s + 1) * BN > tile_all_keys;  // some row does not see all these keys
    if (diagonal) {
      const bool any = any_odd(&sv[b][BN / 4 * wave][0], BN / 4 * D, lane, 64);
      if (lane == 0) sodd[b][wave] = any;
    }
    lds_barrier();
    if (s + 1 < end) load(s + 1);
    if (diagonal && __builtin_amdgcn_readfirstlane(sodd[b][0] | sodd[b][1] | sodd[b][2] |
                                                   sodd[b][3])) {
      odd = true;
      drop_odd(&sv[b][0][0], BN * D, tid, kAttnThreads);
      lds_barrier();
    }
    if (s * BN < wave_keys) {  // uniform per wave
      f32x4_t x[JT][NI];
#pragma unroll
      for (int j = 0; j < JT; ++j) {
#pragma unroll
        for (int i = 0; i < NI; ++i) x[j][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const u32x4_t k = *reinterpret_cast<const u32x4_t*>(
              &sk[b][16 * j + l16][((4 * ks + lg) ^ swz(l16)) * 8]);
#pragma unroll
          for (int i = 0; i < NI; ++i) x[j][i] = mfma(k, q[ks][i], x[j][i]);
        }
      }
      __builtin_amdgcn_iglp_opt(1);  // operand reads ahead of the products: 2% of the time
      if ((s + 1) * BN > all_keys) {  // uniform: some row does not see all of these keys
        asm volatile("");  // keeps this a branch
#pragma unroll
        for (int j = 0; j < JT; ++j)
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (s * BN + 16 * j + 4 * lg + r > last[i]) x[j][i][r] = kNone;
      }
      acc.raise(x, p.c);
#pragma unroll
      for (int j = 0; j < JT; ++j) acc.exps(x[j], p.c);
#pragma unroll
      for (int js = 0; js < JT / 2; ++js) {
        u32x4_t pr[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) pr[i] = p_op(x[2 * js][i], x[2 * js + 1][i]);
        const int row = 32 * js + 4 * lg + (l16 >> 2);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const u32x4_t vt = v_op(b, row, d);
#pragma unroll
          for (int i = 0; i < NI; ++i) acc.o[d][i] = mfma(vt, pr[i], acc.o[d][i]);
        }
      }
    }
  }
  // what was dropped, after the loop, where it takes no registers from it
  for (int s = max(first, tile_all_keys / BN); odd && s < end; ++s) {
    lds_barrier();  // reads of the tiles before are done
    load(s);
    wait_loads();
    lds_barrier();
#pragma unroll
    for (int js = 0; js < JT / 2; ++js)
      add_odd(acc, s * BN + 32 * js + 4 * lg, last,
              [&](int d) { return v_op(s & 1, 32 * js + 4 * lg + (l16 >> 2), d); });
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const float l = sum_over_groups(acc.l[i]);
    if (wrow + 16 * i + l16 < t.rows) {
      f32x4_t o[DT];
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] = acc.o[d][i];
      store_row<D>(p, tok[i], head[i], split, lg, o, acc.m[i], l);
    }
  }
}

// ---- single tokens: the four waves share NI 16-row tiles and take 32 keys each in turn.
// Bound by HBM.  A key is read by one wave of a workgroup (and by one workgroup, but for a
// long sequence among many short ones), so each wave brings its keys and values into a piece
// of LDS of its own, two steps deep, and waits for nobody until the waves join
// their results; one workgroup of a compute unit keeps up to 128 KB in flight.
template <int D, int NI>
__global__ __launch_bounds__(kAttnThreads, 1) void attn_token_kernel(AttnParams p) {
  constexpr int KEYS = 32, JT = 2, KS = D / 32, DT = D / 16;
  constexpr int ROWS = 16 * NI;
  constexpr int RPI = 512 / D, IPT = KEYS / RPI;  // rows per load instruction, of them per tile
  constexpr int PPR = D / 8;
  constexpr int LO = D + 4;  // row stride of the join buffer (floats)
  struct Keys {
    u16 k[4][2][KEYS][D], v[4][2][KEYS][D];
  };
  union Smem {
    Keys s;
    float o[4][16][LO];
  };
  __shared__ alignas(1024) Smem sm;
  __shared__ float sml[4][ROWS][2];

  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const unsigned units = gridDim.x / (unsigned)p.splits;
  const int split = (int)(blockIdx.x / units);
  const unsigned unit = blockIdx.x % units;
  const int hk = (int)(unit % (unsigned)p.Hk);
  Tile t;
  if (!find_tile(p, unit / (unsigned)p.Hk, ROWS, t)) return;

  const int off = t.Lk - t.Lq;
  u32x4_t q[KS][NI];
  int last[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = t.row0 + 16 * i + l16;
    last[i] = r < t.rows ? r / p.G + off : -1;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) q[ks][i] = u32x4_t{0u, 0u, 0u, 0u};
    if (r < t.rows) {
      const u16* src = p.q + (t.q0 + r / p.G) * p.q_row + (hk * p.G + r % p.G) * D + 8 * lg;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) q[ks][i] = *reinterpret_cast<const u32x4_t*>(src + 32 * ks);
    }
  }
  end_loads(q);
  const int keys = max(0, min(t.Lk, (min(t.rows, t.row0 + ROWS) - 1) / p.G + off + 1));
  const int all_keys = t.row0 / p.G + off + 1;
  const int steps = (keys + KEYS - 1) / KEYS, per = (steps + p.splits - 1) / p.splits;
  const int first = min(steps, split * per), end = min(steps, first + per);

  auto swz = [](int row) { return D == 128 ? row & 15 : (row >> 1) & 7; };
  uint32_t koff[IPT], voff[IPT];
#pragma unroll
  for (int i = 0; i < IPT; ++i) {
    const int r = i * RPI + lane / PPR;
    const uint32_t col = (uint32_t)((lane % PPR) ^ swz(r)) * 16u;
    koff[i] = (uint32_t)r * (uint32_t)(p.k_row * 2) + col;
    voff[i] = (uint32_t)r * (uint32_t)(p.v_row * 2) + col;
  }
  const u16* kb = p.k + t.k0 * p.k_row + hk * D;
  const u16* vb = p.v + t.k0 * p.v_row + hk * D;
  auto load = [&](int s, int buf) {
    const int valid = min(KEYS, t.Lk - s * KEYS);
    const u32x4_t dk = rows_words(kb + (int64_t)s * KEYS * p.k_row, p.k_row, valid, D),
                  dv = rows_words(vb + (int64_t)s * KEYS * p.v_row, p.v_row, valid, D);
#pragma unroll
    for (int i = 0; i < IPT; ++i) load_lds<true>(dk, &sm.s.k[wave][buf][i * RPI][0], koff[i]);
#pragma unroll
    for (int i = 0; i < IPT; ++i) load_lds<true>(dv, &sm.s.v[wave][buf][i * RPI][0], voff[i]);
  };

  Acc<D, NI> acc;
  acc.init();
  if (first + wave < end) load(first + wave, 0);
  if (first + wave + 4 < end) load(first + wave + 4, 1);
  auto v_op = [&](int buf, int d) {
    const int row = 4 * lg + (l16 >> 2);
    const int c = ((2 * d + ((l16 & 3) >> 1)) ^ swz(row)) * 8 + 4 * (l16 & 1);
    const u32x2_t lo = ds_read_tr(&sm.s.v[wave][buf][row][c]),
                  hi = ds_read_tr(&sm.s.v[wave][buf][row + 16][c]);
    return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
  };
  bool odd = false;  // some step dropped infinities or NaN of v
  int buf = 0;
  for (int s = first + wave; s < end; s += 4, buf ^= 1) {
    // the oldest step is in place when only the next one's loads are in flight
    if (s + 4 < end) wait_loads<2 * IPT>();
    else wait_loads();
    // some row does not see all of these keys
    if ((s + 1) * KEYS > all_keys && any_odd(&sm.s.v[wave][buf][0][0], KEYS * D, lane, 64)) {
      odd = true;
      drop_odd(&sm.s.v[wave][buf][0][0], KEYS * D, lane, 64);
      asm volatile("" ::: "memory");  // a wave's LDS accesses stay in order
    }
    f32x4_t x[JT][NI];
#pragma unroll
    for (int j = 0; j < JT; ++j) {
#pragma unroll
      for (int i = 0; i < NI; ++i) x[j][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const u32x4_t k = *reinterpret_cast<const u32x4_t*>(
            &sm.s.k[wave][buf][16 * j + l16][((4 * ks + lg) ^ swz(l16)) * 8]);
#pragma unroll
        for (int i = 0; i < NI; ++i) x[j][i] = mfma(k, q[ks][i], x[j][i]);
      }
    }
    if ((s + 1) * KEYS > all_keys) {
      asm volatile("");  // keeps this a branch
#pragma unroll
      for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (s * KEYS + 16 * j + 4 * lg + r > last[i]) x[j][i][r] = kNone;
    }
    acc.raise(x, p.c);
#pragma unroll
    for (int j = 0; j < JT; ++j) acc.exps(x[j], p.c);
    // p in two bf16 parts, its upper half and the rest: the products are free beside the
    // loads.  No part of a positive p is zero, so an infinity of v stays one.
    u32x4_t pr[NI], pr2[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float lo = x[e >> 1][i][2 * (e & 1)], hi = x[e >> 1][i][2 * (e & 1) + 1];
        pr[i][e] = __float_as_uint(lo) >> 16 | (__float_as_uint(hi) & 0xffff0000u);
        pr2[i][e] = pack_bf16(__builtin_amdgcn_fmed3f(lo - bf_lo(pr[i][e]), 1.2e-38f, lo),
                              __builtin_amdgcn_fmed3f(hi - bf_hi(pr[i][e]), 1.2e-38f, hi));
      }
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const u32x4_t v = v_op(buf, d);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        acc.o[d][i] = mfma(v, pr2[i], acc.o[d][i]);
        acc.o[d][i] = mfma(v, pr[i], acc.o[d][i]);
      }
    }
    // this step's reads are done before its place is written again
    wait_lds();
    if (s + 8 < end) load(s + 8, buf);
  }

  // what was dropped, after the loop, where it takes no registers from it
  for (int s = first + wave; odd && s < end; s += 4) {
    if ((s + 1) * KEYS <= all_keys) continue;
    load(s, 0);
    wait_loads();
    add_odd(acc, s * KEYS + 4 * lg, last, [&](int d) { return v_op(0, d); });
    wait_lds();
  }

  // ---- join the waves: maxima and sums first, then the outputs, one 16-row tile at a time
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const float l = sum_over_groups(acc.l[i]);
    if (lg == 0) {
      sml[wave][16 * i + l16][0] = acc.m[i];
      sml[wave][16 * i + l16][1] = l;
    }
  }
  lds_barrier();  // also: every wave's reads of v are done
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    float m = kNone, l = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) m = fmaxf(m, sml[w][16 * i + l16][0]);
    const float base = m == kNone ? 0.f : m;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      l += sml[w][16 * i + l16][1] * __builtin_amdgcn_exp2f(sml[w][16 * i + l16][0] - base);
    const float f = __builtin_amdgcn_exp2f(acc.m[i] - base);
#pragma unroll
    for (int d = 0; d < DT; ++d)
      *reinterpret_cast<f32x4_t*>(&sm.o[wave][l16][16 * d + 4 * lg]) = acc.o[d][i] * f;
    lds_barrier();
    // thread: row tid / 16, D / 16 columns from (tid % 16) * 4 in strides of 64
    const int rr = tid >> 4, r = t.row0 + 16 * i + rr;
    float mr = kNone, lr = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) mr = fmaxf(mr, sml[w][16 * i + rr][0]);
    const float br = mr == kNone ? 0.f : mr;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      lr += sml[w][16 * i + rr][1] * __builtin_amdgcn_exp2f(sml[w][16 * i + rr][0] - br);
    if (r < t.rows) {
      const int64_t at = (t.q0 + r / p.G) * p.Hq + hk * p.G + r % p.G;
      const int64_t w = (int64_t)split * p.Tq_total * p.Hq + at;
      const float g = lr > 0.f ? 1.f / lr : lr == 0.f ? 0.f : lr;
#pragma unroll
      for (int cc = 0; cc < D / 64; ++cc) {
        const int c = 64 * cc + 4 * (tid & 15);
        f32x4_t o = *reinterpret_cast<const f32x4_t*>(&sm.o[0][rr][c]);
#pragma unroll
        for (int ww = 1; ww < 4; ++ww) o += *reinterpret_cast<const f32x4_t*>(&sm.o[ww][rr][c]);
        if (p.splits > 1) {
          *reinterpret_cast<f32x4_t*>(p.ws_o + w * D + c) = o;
        } else {
          *reinterpret_cast<u32x2_t*>(p.out + at * D + c) =
              u32x2_t{pack_bf16(o[0] * g, o[1] * g), pack_bf16(o[2] * g, o[3] * g)};
        }
      }
      if ((tid & 15) == 0) {
        if (p.splits > 1) *reinterpret_cast<f32x2_t*>(p.ws_ml + 2 * w) = f32x2_t{mr, lr};
        else if (p.lse != nullptr)
          p.lse[at] = lr == 0.f ? kNone : (mr + __builtin_amdgcn_logf(lr)) * kLn2;
      }
    }
    if (i + 1 < NI) lds_barrier();
  }
}

// Joins the splits of a row, one wave per (query token, head): lane s weighs split s (there
// are at most 64), then the lanes share the row's D values.  GAPS: what the outputs of a
// split without keys hold is loaded (the loads do not wait for the sums) but not used.  Each of
// its two callers keeps the order in which its results' normalisers have always been summed.
template <int D, bool GAPS>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnParams p) {
  constexpr int V = D / 64;  // values per lane
  typedef float vec __attribute__((ext_vector_type(V)));
  const int lane = threadIdx.x & 63;
  const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t rows = p.Tq_total * p.Hq;
  if (at >= rows) return;
  // every load that does not wait for another one first
  bool there = true;  // a query outside every sequence keeps its rows
  if (p.cu_q != nullptr) {
    const int64_t token = (uint32_t)at / (uint32_t)p.Hq;  // split calls have fewer than 2^26 rows
    there = token >= p.cu_q[0] && token < p.cu_q[p.N];
  }
  f32x2_t ml = {kNone, 0.f};
  if (lane < p.splits) ml = *reinterpret_cast<const f32x2_t*>(p.ws_ml + 2 * (lane * rows + at));
  const float* o = p.ws_o + at * D + lane * V;
  vec x[8];  // eight loads in flight
  auto load = [&](int s0) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = s0 + i < p.splits ? *reinterpret_cast<const vec*>(o + (s0 + i) * rows * D) : vec{};
  };
  load(0);
  const uint64_t filled = GAPS ? __ballot(!(ml[0] == kNone && ml[1] == 0.f)) : ~0ull;
  const float m = wave_max(ml[0]);
  const float f = __builtin_amdgcn_exp2f(ml[0] - (m == kNone ? 0.f : m));
  const float l = GAPS ? wave_sum_mirrored(ml[1] * f) : wave_sum(ml[1] * f);
  vec sum = {};
  for (int s0 = 0; s0 < p.splits; s0 += 8) {
    if (s0 > 0) load(s0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (GAPS && !(filled >> ((s0 + i) & 63) & 1)) x[i] = vec{};
      sum += x[i] * __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), (s0 + i) & 63));
    }
  }
  if (!there) return;
  const float g = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
  u16* out = p.out + at * D + lane * V;
  if constexpr (V == 2) *reinterpret_cast<unsigned*>(out) = pack_bf16(sum[0] * g, sum[1] * g);
  else out[0] = (u16)pack_bf16(sum[0] * g, 0.f);
  if (p.lse != nullptr && lane == 0)
    p.lse[at] = l == 0.f ? kNone : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

template <int D, bool GAPS>
void join(const AttnParams& p, hipStream_t stream) {
  const int64_t rows = p.Tq_total * p.Hq;
  attn_join_kernel<D, GAPS><<<dim3((unsigned)((rows + 3) / 4)), 256, 0, stream>>>(p);
}

template <int D>
hipError_t go(const AttnParams& p, const AttnSchedule& s, hipStream_t stream) {
  int64_t slots = attn_slots(p.Tq_total, p.N, p.G, s.rows);
  if (p.cu_q == nullptr) slots = p.N * ((p.Tq * p.G + s.rows - 1) / s.rows);
  const dim3 grid((unsigned)(slots * p.Hk * p.splits));
  if (s.tokens) {
    if (s.tiles16 == 1) attn_token_kernel<D, 1><<<grid, kAttnThreads, 0, stream>>>(p);
    else if (s.tiles16 == 2) attn_token_kernel<D, 2><<<grid, kAttnThreads, 0, stream>>>(p);
    else attn_token_kernel<D, 4><<<grid, kAttnThreads, 0, stream>>>(p);
  } else {
    attn_tile_kernel<D, 2><<<grid, kAttnThreads, 0, stream>>>(p);
  }
  if (p.splits > 1) join<D, false>(p, stream);
  return hipGetLastError();
}

}  // namespace

AttnSchedule attn_schedule(int64_t Tq_total, int64_t N, int64_t G) {
  const int64_t mean = (Tq_total * G + N - 1) / N;  // rows of a sequence and key/value head
  if (mean <= 64) {
    const int tiles = mean <= 16 ? 1 : mean <= 32 ? 2 : 4;
    return AttnSchedule{1, tiles, 16 * tiles};
  }
  return AttnSchedule{0, 2, 128};
}

hipError_t launch_attn(const AttnParams& p, const AttnSchedule& s, int D, hipStream_t stream) {
  return D == 64 ? go<64>(p, s, stream) : go<128>(p, s, stream);
}

hipError_t launch_attn_join(const AttnParams& p, int D, hipStream_t stream) {
  if (D == 64) join<64, true>(p, stream);
  else join<128, true>(p, stream);
  return hipGetLastError();
}

}  // namespace kda
