// Causal softmax attention with grouped heads over caches held in 4 bits (kda_attn4_fwd), for
// gfx950: the formulas and the rows of attn_kernel.hip, keys and values as codes times powers of
// two (cache4_kernel.hip).  Their bf16 values are exact, so the products are those of a bf16 cache
// that holds the same values, and the bytes read are 17/64 of its.
//
// The waves of a workgroup share a tile of 16 rows and take 64 keys, two tiles of the cache, each in
// turn.  Codes and scales go from memory straight into a ring in LDS, two such steps ahead, every
// lane its own 16 bytes of 16 keys' rows and of the values of eight channels at four keys: the places
// in the cache are those of the matrix products' operands, so nothing is exchanged.
//   x^T = K Q^T: lane (g, c) holds channels D/4 g .. of key 4 (c % 4) + c / 4 of sixteen, so that
//     accumulator row 4 g + r is key 4 r + g;
//   out^T = V^T P^T: lane (g, c) holds channels D/16 c .. of the keys 4 r + g, and product e gives
//     the channels D/16 m + e, m its row.  The conversion yields two channels of one key, an
//     operand word wants two keys of one channel: a byte permutation between two keys' words.
// Long caches are split into parts of equally many keys (not into equally many parts: lengths
// differ), which a second kernel joins.  Prompts bring the keys to bf16 once (expand4_kernel) and run
// kda_attn_fwd's kernel for them.
//
// p keeps two bf16 parts, as in kda_attn_fwd's kernel for few rows: error 1.65e-3, that of rounding
// the output, where one part has 2.3e-3.  One part takes 38.9 instead of 41.2 us for the single tokens
// below, and 18.2 instead of 17.5 for the drafted ones.
//
// Measured (calls): one token of each of 32 requests over 1024-8192 keys, 32/8 heads, D 128, 40.8 us
// (161 MB, 4.0 TB/s; the loads alone and the join 33.5): a byte of codes asks for four times the
// arithmetic of one of bf16, vector instructions are busy 56%, matrix products 21%, and the join takes
// 4.6 us; five tokens of each of 16 over 512-4096 keys, 32/4 heads, D 64, 17.2; two requests of 200 and
// 77 keys 4.4; packed [300, 700, 1024] queries over [300, 2200, 1101] keys, 96/8 heads, 118, of which 8 expand
// the keys.  Two and four tiles of rows a wave, which convert a key once for more rows, were slower with
// codes in registers (256 of them and spills: the drafted tokens 21 and 32 us, 19 in tiles of 16 then)
// and have not been measured since codes wait in LDS.  Slower too: registers instead of LDS for what is
// on its way (45.9 us, 37.6 two steps ahead without the second path for infinities, whose registers do
// not fit beside it), 16 waves, and one tile a step (19-20 us for the drafted tokens).
#include "api_util.h"
#include "attn_rows.h"
#include "cache4.h"
#include "layer_params.h"

#include <utility>

namespace kda {
namespace {

using namespace dev;

// A lane's codes and scales of a tile of 32 keys: D / 4 channels of two keys, and D / 16 of the values
// at eight.
template <int D>
struct Keys4 {
  typedef unsigned part __attribute__((ext_vector_type(D / 32)));
  part k[2];
  unsigned scale;
};
template <int D>
struct Values4 {
  u32x4_t v[D / 64];
  u32x2_t scale;
};

// One word a lane from memory to LDS, as load_lds.
template <bool ONCE>
__device__ __forceinline__ void load_lds_word(const uint8_t* at, const uint8_t* to) {
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)to;
  const uint32_t m0 = (uint32_t)__builtin_amdgcn_readfirstlane(lds);
  if constexpr (ONCE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off nt"
                 :
                 : "s"(m0), "v"(at)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
                 :
                 : "s"(m0), "v"(at)
                 : "memory", "m0");
}

// A tile of 32 keys on its way from a cache through LDS.  Every lane brings its own 16 (keys of
// 64 channels: 8) bytes of each instruction and reads them back from where they land, so reads
// meet no bank twice; the scales' two words of 32 positions lie side by side.
template <int D>
struct Tile4 {
  uint8_t k[16 * D], v[16 * D], s[256];
};
template <int D, bool ONCE>
struct View4 {
  static constexpr int LOADS = D == 128 ? 5 : 3;  // instructions of a tile
  const uint8_t *k4, *v4, *sc;
  uint32_t k_at, v_at, k_lds, ks_lds, vs_lds;

  __device__ __forceinline__ View4(const Cache4& c, int64_t unit, int lane) {
    const uint32_t g = lane >> 4, l = lane & 15;
    const int64_t at = unit * (c.cap / kCache4Tile);
    k4 = c.k4 + at * (16 * D);
    v4 = c.v4 + at * (16 * D);
    // lanes of the first half bring the keys' scales (a word each, D / 4 of them), of the second
    // the values'; what lanes behind them bring lands behind and is not used
    const uint32_t word = lane & 31;
    sc = (lane < 32 ? c.ks : c.vs) + at * D + (word < D / 4 ? 4 * word : 0);
    v_at = lane * 16;
    const uint32_t row = 4 * (l & 3) + (l >> 2);  // the key of sixteen
    if constexpr (D == 128) {
      k_at = row * 64 + g * 16;
      k_lds = v_at;
    } else {
      k_at = v_at;  // 32 keys at once, a lane the halves of two operands
      k_lds = row * 32 + g * 8;
    }
    ks_lds = g * (D / 32) / 4 * 32 + 2 * l;
    vs_lds = 128 + l * (D / 32) / 16 * 32 + 8 * g;
  }
  static __device__ __forceinline__ u32x4_t words(const uint8_t* base) {
    const uint64_t at = reinterpret_cast<uint64_t>(base);
    return u32x4_t{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)at),
                   (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(at >> 32) & 0xffffu),
                   16u * D, 0x00020000u};
  }
  __device__ __forceinline__ void load(int tile, const Tile4<D>& to) const {
    const u32x4_t dk = words(k4 + (int64_t)tile * (16 * D)),
                  dv = words(v4 + (int64_t)tile * (16 * D));
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      load_lds<ONCE>(dk, reinterpret_cast<const u16*>(to.k + 1024 * i), k_at + 1024 * i);
      load_lds<ONCE>(dv, reinterpret_cast<const u16*>(to.v + 1024 * i), v_at + 1024 * i);
    }
    load_lds_word<ONCE>(sc + (int64_t)tile * D, to.s);
  }
  __device__ __forceinline__ Keys4<D> keys(const Tile4<D>& from) const {
    Keys4<D> s;
    if constexpr (D == 128) {
      s.k[0] = *reinterpret_cast<const u32x4_t*>(from.k + k_lds);
      s.k[1] = *reinterpret_cast<const u32x4_t*>(from.k + k_lds + 1024);
    } else {
      s.k[0] = *reinterpret_cast<const u32x2_t*>(from.k + k_lds);
      s.k[1] = *reinterpret_cast<const u32x2_t*>(from.k + k_lds + 512);
    }
    s.scale = *reinterpret_cast<const u16*>(from.s + ks_lds);
    return s;
  }
  __device__ __forceinline__ Values4<D> values(const Tile4<D>& from) const {
    Values4<D> s;
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
      s.v[i] = *reinterpret_cast<const u32x4_t*>(from.v + v_at + 1024 * i);
    s.scale = *reinterpret_cast<const u32x2_t*>(from.s + vs_lds);
    return s;
  }
};

// Codes of channels D/16 c .. at key 16 j + 4 i + g, from bit 0, and their scale.
template <int D>
__device__ __forceinline__ unsigned v_codes(const Values4<D>& s, int j, int i) {
  if constexpr (D == 128) {
    return s.v[j][i];
  } else {
    const unsigned w = s.v[0][2 * j + (i >> 1)];
    return i & 1 ? w >> 16 : w;
  }
}
template <int D>
__device__ __forceinline__ float v_scale(const Values4<D>& s, int j, int i) {
  const int byte = 2 * i + j;
  return scale_of(s.scale[byte >> 2], byte & 3);
}

// Operands of out^T's products 2 M and 2 M + 1.
struct VOps {
  u32x4_t a, b;
};
template <int D, int M>
__device__ __forceinline__ VOps v_ops(const Values4<D>& s) {
  VOps r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int j = e >> 1, i = 2 * (e & 1);
    const unsigned lo = two_values<M>(v_codes<D>(s, j, i), v_scale<D>(s, j, i)),
                   hi = two_values<M>(v_codes<D>(s, j, i + 1), v_scale<D>(s, j, i + 1));
    r.a[e] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
    r.b[e] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
  }
  return r;
}
template <class F, int... M>
__device__ __forceinline__ void each(F f, std::integer_sequence<int, M...>) {
  (f(std::integral_constant<int, M>{}), ...);
}

// Whether a scale of these values may give infinities or NaN (a byte of 252 and more).
template <int D>
__device__ __forceinline__ bool may_be_odd(const Values4<D>& s) {
  bool any = false;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const unsigned z = ~s.scale[w] & 0xfcfcfcfcu;  // a zero byte where the six bits are ones
    any |= ((z - 0x01010101u) & ~z & 0x80808080u) != 0u;
  }
  return __any(any);
}

// Waits for a row's loads before the loop over the keys: their first use inside it would make every
// step wait for all loads in flight.
template <int KS>
__device__ __forceinline__ void end_row_loads(u32x4_t (&q)[KS]) {
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) asm volatile("" : "+v"(q[ks]));
}

template <int D, int WAVES, bool ONCE>
__global__ __launch_bounds__(64 * WAVES, 2) void attn4_kernel(Attn4Params q4) {
  constexpr int KS = D / 32, DT = D / 16, ROWS = kAttn4Rows;
  constexpr int AHEAD = 2;  // pairs of tiles of a wave on their way
  constexpr int LO = D + 4;  // row stride of the join buffer (floats)
  union Smem {
    Tile4<D> tile[WAVES][AHEAD][2];
    float o[WAVES][ROWS][LO];
  };
  __shared__ alignas(16) Smem sm;
  __shared__ float sml[WAVES][ROWS][2];
  const AttnParams& p = q4.a;

  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const unsigned units = gridDim.x / (unsigned)p.splits;
  const int split = (int)(blockIdx.x / units);
  const unsigned unit = blockIdx.x % units, tile_no = unit / (unsigned)p.Hk;
  const int hk = (int)(unit % (unsigned)p.Hk);
  Tile t;
  if (p.cu_q == nullptr) {
    const unsigned n = tile_no / (unsigned)q4.row_tiles;
    if (!set_tile(p, (int)n, (int64_t)(tile_no % (unsigned)q4.row_tiles) * ROWS, t)) return;
  } else {
    // the last sequence whose first slot is not behind this one (first slots grow strictly)
    const int n = find_last(p.N, [&](int i) {
      return clamp64(p.cu_q[i], 0, p.Tq_total) * p.G / ROWS + i <= tile_no;
    });
    int64_t a, b;
    query_bounds(p, n, a, b);
    if (!set_tile(p, n, (tile_no - (a * p.G / ROWS + n)) * ROWS, t)) return;
  }
  // this lane's row
  const int row = t.row0 + l16, token = row / p.G;
  u32x4_t q[KS];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) q[ks] = u32x4_t{0u, 0u, 0u, 0u};
  if (row < t.rows) {
    const u16* src =
        p.q + (t.q0 + token) * p.q_row + (hk * p.G + row - token * p.G) * D + D / 4 * lg;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) q[ks] = *reinterpret_cast<const u32x4_t*>(src + 8 * ks);
  }
  const int64_t slot = q4.slot != nullptr ? q4.slot[t.n] : t.n;
  if (slot < 0 || slot >= q4.c.slots) t.Lk = 0;
  const int off = t.Lk - t.Lq, last = row < t.rows ? token + off : -1;
  const int keys = max(0, min(t.Lk, (min(t.rows, t.row0 + ROWS) - 1) / p.G + off + 1));
  const int all_keys = t.row0 / p.G + off + 1;
  const int steps = (keys + kCache4Tile - 1) / kCache4Tile;
  const int first = min(steps, split * q4.part), end = min(steps, first + q4.part);
  if (split > 0 && first == end) {  // no keys in this part: the join uses no outputs of it
    if (tid < ROWS && row < t.rows) {
      const int64_t at = (t.q0 + token) * p.Hq + hk * p.G + row - token * p.G;
      *reinterpret_cast<f32x2_t*>(p.ws_ml + 2 * ((int64_t)split * p.Tq_total * p.Hq + at)) =
          f32x2_t{kNone, 0.f};
    }
    return;
  }

  const View4<D, ONCE> view(q4.c, slot * p.Hk + hk, lane);
  end_row_loads(q);
  Acc<D, 1> acc;
  acc.init();
  bool odd = false;  // some step dropped infinities or NaN of v
  // One step: a pair of tiles, the second there or not.  Two tiles at once give the matrix products,
  // exponentials and conversions twice the independent work to fill their latencies with.
  const int limit = min(last, end * kCache4Tile - 1);
  const int all = min(all_keys, end * kCache4Tile);
  auto step = [&](const Tile4<D> (&tile)[2], int s) {
    f32x4_t x[4][1];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const Keys4<D> k = view.keys(tile[h]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float scale = scale_of(k.scale, j);
        f32x4_t y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) y = mfma(eight_values(k.k[j][ks], scale), q[ks], y);
        x[2 * h + j][0] = y;
      }
    }
    const Values4<D> v[2] = {view.values(tile[0]), view.values(tile[1])};
    bool drop = false;
    if ((s + 2) * kCache4Tile > all) {  // some row does not see all of these keys
      asm volatile("");  // keeps this a branch
      drop = may_be_odd<D>(v[0]) || may_be_odd<D>(v[1]);
      odd |= drop;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (s * kCache4Tile + 16 * j + 4 * r + lg > limit) x[j][0][r] = kNone;
    }
    acc.raise(x, p.c);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc.exps(x[j], p.c);
    // p in two bf16 parts, its upper half and the rest.  No part of a positive p is zero, so an
    // infinity of v stays one.
    u32x4_t pr[2], pr2[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float lo = x[2 * h + (e >> 1)][0][2 * (e & 1)],
                    hi = x[2 * h + (e >> 1)][0][2 * (e & 1) + 1];
        pr[h][e] = __float_as_uint(lo) >> 16 | (__float_as_uint(hi) & 0xffff0000u);
        pr2[h][e] = pack_bf16(__builtin_amdgcn_fmed3f(lo - bf_lo(pr[h][e]), 1.2e-38f, lo),
                              __builtin_amdgcn_fmed3f(hi - bf_hi(pr[h][e]), 1.2e-38f, hi));
      }
    auto products = [&](auto dropped) {
      each(
          [&](auto m) {
            constexpr int M = decltype(m)::value;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              VOps o = v_ops<D, M>(v[h]);
              if constexpr (decltype(dropped)::value) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  o.a[e] = odd_split(o.a[e]).finite;
                  o.b[e] = odd_split(o.b[e]).finite;
                }
              }
              acc.o[2 * M][0] = mfma(o.a, pr2[h], acc.o[2 * M][0]);
              acc.o[2 * M + 1][0] = mfma(o.b, pr2[h], acc.o[2 * M + 1][0]);
              acc.o[2 * M][0] = mfma(o.a, pr[h], acc.o[2 * M][0]);
              acc.o[2 * M + 1][0] = mfma(o.b, pr[h], acc.o[2 * M + 1][0]);
            }
          },
          std::make_integer_sequence<int, DT / 2>{});
    };
    if (drop) products(std::true_type{});
    else products(std::false_type{});
  };

  // AHEAD pairs are on their way, or what is left; a missing second tile takes the first's place
  auto load = [&](int s, Tile4<D> (&to)[2]) {
    view.load(s, to[0]);
    view.load(min(s + 1, end - 1), to[1]);
  };
  constexpr int NEXT = 2 * WAVES, L = 2 * View4<D, ONCE>::LOADS;
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (first + 2 * wave + i * NEXT < end) load(first + 2 * wave + i * NEXT, sm.tile[wave][i]);
  int buf = 0;
  for (int s = first + 2 * wave; s < end; s += NEXT, buf ^= 1) {
    if (s + NEXT < end) wait_loads<L>();
    else wait_loads();
    step(sm.tile[wave][buf], s);
    wait_lds();  // this pair's reads are done before its place is written again
    if (s + AHEAD * NEXT < end) load(s + AHEAD * NEXT, sm.tile[wave][buf]);
  }

  // what was dropped, after the loop, where it takes no registers from it
  for (int pair = first + 2 * wave, s = pair; odd && s < end; s = s == pair ? s + 1 : pair += NEXT) {
    if ((pair + 2) * kCache4Tile <= all) continue;
    view.load(s, sm.tile[wave][0][0]);
    wait_loads();
    const Values4<D> v = view.values(sm.tile[wave][0][0]);
    wait_lds();
    if (!may_be_odd<D>(v)) continue;
    u32x4_t sees;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int k = s * kCache4Tile + lg + 16 * (e >> 1) + 8 * (e & 1);
      sees[e] = (k <= last ? 0x3f80u : 0u) | (k + 4 <= last ? 0x3f800000u : 0u);
    }
    each(
        [&](auto m) {
          constexpr int M = decltype(m)::value;
          VOps o = v_ops<D, M>(v);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o.a[e] = odd_split(o.a[e]).code;
            o.b[e] = odd_split(o.b[e]).code;
          }
          const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
          const f32x4_t na = mfma(o.a, sees, zero), nb = mfma(o.b, sees, zero);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            acc.o[2 * M][0][r] += odd_value(na[r]);
            acc.o[2 * M + 1][0][r] += odd_value(nb[r]);
          }
        },
        std::make_integer_sequence<int, DT / 2>{});
  }

  // ---- join the waves (behind the barrier every wave's reads of its tiles are done): maxima and
  // sums first, then the outputs
  const float l = sum_over_groups(acc.l[0]);
  if (lg == 0) {
    sml[wave][l16][0] = acc.m[0];
    sml[wave][l16][1] = l;
  }
  lds_barrier();
  float m = kNone;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) m = fmaxf(m, sml[w][l16][0]);
  const float f = __builtin_amdgcn_exp2f(acc.m[0] - (m == kNone ? 0.f : m));
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int e = 0; e < DT; e += 4)
      *reinterpret_cast<f32x4_t*>(&sm.o[wave][l16][DT * (4 * lg + r) + e]) =
          f32x4_t{acc.o[e][0][r], acc.o[e + 1][0][r], acc.o[e + 2][0][r], acc.o[e + 3][0][r]} * f;
  lds_barrier();
  // a thread: four columns of a row
  for (int i = tid; i < ROWS * D / 4; i += 64 * WAVES) {
    const int rr = i / (D / 4), c = i % (D / 4) * 4, r = t.row0 + rr;
    if (r >= t.rows) break;
    float mr = kNone, lr = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) mr = fmaxf(mr, sml[w][rr][0]);
    const float br = mr == kNone ? 0.f : mr;
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
      lr += sml[w][rr][1] * __builtin_amdgcn_exp2f(sml[w][rr][0] - br);
    f32x4_t o = *reinterpret_cast<const f32x4_t*>(&sm.o[0][rr][c]);
#pragma unroll
    for (int w = 1; w < WAVES; ++w) o += *reinterpret_cast<const f32x4_t*>(&sm.o[w][rr][c]);
    const int tk = r / p.G;
    const int64_t at = (t.q0 + tk) * p.Hq + hk * p.G + r - tk * p.G;
    const int64_t w = (int64_t)split * p.Tq_total * p.Hq + at;
    if (p.splits > 1) {
      *reinterpret_cast<f32x4_t*>(p.ws_o + w * D + c) = o;
      if (c == 0) *reinterpret_cast<f32x2_t*>(p.ws_ml + 2 * w) = f32x2_t{mr, lr};
    } else {
      const float g = lr > 0.f ? 1.f / lr : lr == 0.f ? 0.f : lr;
      *reinterpret_cast<u32x2_t*>(p.out + at * D + c) =
          u32x2_t{pack_bf16(o[0] * g, o[1] * g), pack_bf16(o[2] * g, o[3] * g)};
      if (p.lse != nullptr && c == 0)
        p.lse[at] = lr == 0.f ? kNone : (mr + __builtin_amdgcn_logf(lr)) * kLn2;
    }
  }
}

// ---- many rows: keys and values in bf16 to a workspace once, [N, cap, Hk, D], for the kernel of
// kda_attn_fwd's prompts.  A workgroup takes a tile of 32 keys of one head; lengths go along.
template <int D>
__global__ __launch_bounds__(kAttnThreads) void expand4_kernel(Attn4Params q4) {
  constexpr int LPT = D / 16;  // threads of a key, 16 channels each
  const AttnParams& p = q4.a;
  const int tid = threadIdx.x;
  const unsigned tiles = (unsigned)(p.Tk / kCache4Tile);
  const int hk = (int)(blockIdx.x % (unsigned)p.Hk);
  const unsigned at = blockIdx.x / (unsigned)p.Hk;
  const int n = (int)(at / tiles), tile = (int)(at % tiles);
  const int64_t slot = q4.slot != nullptr ? q4.slot[n] : n;
  const bool there = slot >= 0 && slot < q4.c.slots;
  const int64_t len = !there ? 0 : p.k_lens != nullptr ? clamp64(p.k_lens[n], 0, p.Tk) : p.Tk;
  if (tile == 0 && hk == 0 && tid == 0) q4.lens[n] = len;
  if ((int64_t)tile * kCache4Tile >= len) return;

  const int64_t unit = slot * p.Hk + hk, t = unit * tiles + tile;
  const uint8_t *kc = q4.c.k4 + t * (16 * D), *vc = q4.c.v4 + t * (16 * D),
                *ks = q4.c.ks + t * D, *vs = q4.c.vs + t * D;
  for (int x = tid / LPT; x < kCache4Tile; x += kAttnThreads / LPT) {
    const int c = tid % LPT, j = x >> 4, i = x >> 2 & 3, g = x & 3, place = 8 * g + 2 * i + j;
    const int64_t to = (((int64_t)n * p.Tk + tile * kCache4Tile + x) * p.Hk + hk) * D + 16 * c;
    const float fk = scale_of(ks[c / 2 * 32 + place], 0), fv = scale_of(vs[c / 2 * 32 + place], 0);
    const u32x2_t wk = *reinterpret_cast<const u32x2_t*>(kc + x * (D / 2) + 8 * c);
    unsigned v0, v1;
    if constexpr (D == 128) {
      const uint8_t* from = vc + 1024 * j + 256 * g + 32 * c + 4 * i;
      v0 = *reinterpret_cast<const unsigned*>(from);
      v1 = *reinterpret_cast<const unsigned*>(from + 16);
    } else {
      const uint8_t* from = vc + 256 * g + 64 * c + 8 * j + 2 * i;
      const u16* h = reinterpret_cast<const u16*>(from);
      v0 = h[0] | (unsigned)h[8] << 16;
      v1 = h[16] | (unsigned)h[24] << 16;
    }
    u32x4_t* ko = reinterpret_cast<u32x4_t*>(q4.k_ws + to);
    u32x4_t* vo = reinterpret_cast<u32x4_t*>(q4.v_ws + to);
    ko[0] = eight_values(wk[0], fk);
    ko[1] = eight_values(wk[1], fk);
    vo[0] = eight_values(v0, fv);
    vo[1] = eight_values(v1, fv);
  }
}

template <int D, int WAVES>
void start(const Attn4Params& p, dim3 grid, hipStream_t stream) {
  if (p.once) attn4_kernel<D, WAVES, true><<<grid, 64 * WAVES, 0, stream>>>(p);
  else attn4_kernel<D, WAVES, false><<<grid, 64 * WAVES, 0, stream>>>(p);
}

template <int D>
hipError_t go(Attn4Params p, hipStream_t stream) {
  const AttnParams& a = p.a;
  p.row_tiles = (int32_t)((a.Tq * a.G + kAttn4Rows - 1) / kAttn4Rows);
  const int64_t slots = a.cu_q == nullptr ? a.N * (int64_t)p.row_tiles
                                          : attn_slots(a.Tq_total, a.N, a.G, kAttn4Rows);
  const int64_t groups = slots * a.Hk * a.splits;
  // one workgroup a compute unit at most: eight waves instead of four share its keys (16 tokens, 8
  // heads, D 64, 2048 positions, one part: 10.1 us, 11.6 with four; 8 units of 1024: 6.9 and 7.4)
  const dim3 grid((unsigned)groups);
  if (groups <= device_cus()) start<D, 8>(p, grid, stream);
  else start<D, 4>(p, grid, stream);
  if (a.splits > 1) return launch_attn_join(a, D, stream);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_expand4(const Attn4Params& p, int D, hipStream_t stream) {
  const dim3 grid((unsigned)(p.a.N * (p.a.Tk / kCache4Tile) * p.a.Hk));
  if (D == 64) expand4_kernel<64><<<grid, kAttnThreads, 0, stream>>>(p);
  else expand4_kernel<128><<<grid, kAttnThreads, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_attn4(const Attn4Params& p, int D, hipStream_t stream) {
  return D == 64 ? go<64>(p, stream) : go<128>(p, stream);
}

}  // namespace kda
