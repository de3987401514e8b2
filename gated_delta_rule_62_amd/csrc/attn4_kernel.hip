// Causal softmax attention with grouped heads over caches held in 4 bits (kda_attn4_fwd), for
// gfx950: the formulas and the rows of attn_kernel.hip, keys and values as codes times powers of
// two (cache4_kernel.hip).  Their bf16 values are exact, so the products are those of a bf16 cache
// that holds the same values, and the bytes read are 17/64 of its.
//
// The four waves of a workgroup share a tile of rows and take 32 keys each in turn, straight from
// memory into registers, a step ahead.  One 16-byte load a lane is a lane's part of 16 keys' rows,
// one is the values of eight channels at four keys: the places of codes and scales in the cache are
// those of the matrix products' operands.
//   x^T = K Q^T: lane (g, c) holds channels D/4 g .. of key 4 (c % 4) + c / 4 of sixteen, so that
//     accumulator row 4 g + r is key 4 r + g;
//   out^T = V^T P^T: lane (g, c) holds channels D/16 c .. of the keys 4 r + g, and product e gives
//     the channels D/16 m + e, m its row.  The conversion yields two channels of one key, an
//     operand word wants two keys of one channel: a byte permutation between two keys' words.
// Long caches are split into parts of equally many keys (not into equally many parts: lengths
// differ), which a second kernel joins.
#include "api_util.h"
#include "attn_rows.h"
#include "cache4.h"
#include "layer_params.h"

#include <utility>

namespace kda {
namespace {

using namespace dev;

// A lane's codes and scales of 32 keys.
template <int D>
struct Step4;
template <>
struct Step4<128> {
  u32x4_t k[2], v[2];
  u32x2_t vs;
  unsigned ks;
};
template <>
struct Step4<64> {
  u32x2_t k[2];
  u32x4_t v;
  u32x2_t vs;
  unsigned ks;
};

// One (slot, key/value head) of a cache, and where this lane's parts of a tile lie.
template <int D>
struct View4 {
  const uint8_t *k4, *v4, *ks, *vs;

  __device__ __forceinline__ View4(const Cache4& c, int64_t unit, int lane) {
    const int g = lane >> 4, l = lane & 15;
    const int64_t tiles = c.cap / kCache4Tile;
    k4 = c.k4 + unit * c.cap * (D / 2) + (4 * (l & 3) + (l >> 2)) * (D / 2) + g * (D / 8);
    v4 = c.v4 + unit * tiles * (16 * D) + lane * 16;
    ks = c.ks + unit * tiles * D + g * (D / 32) / 4 * 32 + 2 * l;
    vs = c.vs + unit * tiles * D + l * (D / 32) / 16 * 32 + 8 * g;
  }
  __device__ __forceinline__ Step4<D> load(int tile) const {
    Step4<D> s;
    const int64_t at = (int64_t)tile * (16 * D), sc = (int64_t)tile * D;
    if constexpr (D == 128) {
      s.k[0] = *reinterpret_cast<const u32x4_t*>(k4 + at);
      s.k[1] = *reinterpret_cast<const u32x4_t*>(k4 + at + 1024);
      s.v[0] = *reinterpret_cast<const u32x4_t*>(v4 + at);
      s.v[1] = *reinterpret_cast<const u32x4_t*>(v4 + at + 1024);
    } else {
      s.k[0] = *reinterpret_cast<const u32x2_t*>(k4 + at);
      s.k[1] = *reinterpret_cast<const u32x2_t*>(k4 + at + 512);
      s.v = *reinterpret_cast<const u32x4_t*>(v4 + at);
    }
    s.ks = *reinterpret_cast<const u16*>(ks + sc);
    s.vs = *reinterpret_cast<const u32x2_t*>(vs + sc);
    return s;
  }
};

// Codes of channels D/16 c .. at key 16 j + 4 i + g, from bit 0.
__device__ __forceinline__ unsigned v_codes(const Step4<128>& s, int j, int i) {
  return s.v[j][i];
}
__device__ __forceinline__ unsigned v_codes(const Step4<64>& s, int j, int i) {
  const unsigned w = s.v[2 * j + (i >> 1)];
  return i & 1 ? w >> 16 : w;
}
template <int D>
__device__ __forceinline__ float v_scale(const Step4<D>& s, int j, int i) {
  const int byte = 2 * i + j;
  return scale_of(s.vs[byte >> 2], byte & 3);
}

// Operands of out^T's products 2 M and 2 M + 1.
struct VOps {
  u32x4_t a, b;
};
template <int D, int M>
__device__ __forceinline__ VOps v_ops(const Step4<D>& s) {
  VOps r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int j = e >> 1, i = 2 * (e & 1);
    const unsigned lo = two_values<M>(v_codes(s, j, i), v_scale<D>(s, j, i)),
                   hi = two_values<M>(v_codes(s, j, i + 1), v_scale<D>(s, j, i + 1));
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
__device__ __forceinline__ bool may_be_odd(const Step4<D>& s) {
  bool any = false;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const unsigned z = ~s.vs[w] & 0xfcfcfcfcu;  // a zero byte where the six bits are ones
    any |= ((z - 0x01010101u) & ~z & 0x80808080u) != 0u;
  }
  return __any(any);
}

template <int D, int NI>
__global__ __launch_bounds__(kAttnThreads, NI == 1 ? 3 : 2) void attn4_kernel(
    Attn4Params q4) {
  constexpr int WAVES = kAttnThreads / 64;
  constexpr int KS = D / 32, DT = D / 16, ROWS = 16 * NI;
  constexpr int LO = D + 4;  // row stride of the join buffer (floats)
  __shared__ alignas(16) float so[WAVES][16][LO];
  __shared__ float sml[WAVES][ROWS][2];
  const AttnParams& p = q4.a;

  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const unsigned units = gridDim.x / (unsigned)p.splits;
  const int split = (int)(blockIdx.x / units);
  const unsigned unit = blockIdx.x % units;
  const int hk = (int)(unit % (unsigned)p.Hk);
  Tile t;
  if (!find_tile(p, unit / (unsigned)p.Hk, ROWS, t)) return;
  const int64_t slot = q4.slot != nullptr ? q4.slot[t.n] : t.n;
  if (slot < 0 || slot >= q4.c.slots) t.Lk = 0;

  const int off = t.Lk - t.Lq;
  const int keys = max(0, min(t.Lk, (min(t.rows, t.row0 + ROWS) - 1) / p.G + off + 1));
  const int all_keys = t.row0 / p.G + off + 1;
  const int steps = (keys + kCache4Tile - 1) / kCache4Tile;
  const int first = min(steps, split * q4.part), end = min(steps, first + q4.part);
  if (split > 0 && first == end) {  // no keys in this part: the join reads no outputs of it
    for (int i = tid; i < ROWS; i += kAttnThreads) {
      const int r = t.row0 + i;
      if (r < t.rows) {
        const int64_t at = (t.q0 + r / p.G) * p.Hq + hk * p.G + r % p.G;
        const int64_t w = (int64_t)split * p.Tq_total * p.Hq + at;
        *reinterpret_cast<f32x2_t*>(p.ws_ml + 2 * w) = f32x2_t{kNone, 0.f};
      }
    }
    return;
  }

  u32x4_t q[KS][NI];
  int last[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = t.row0 + 16 * i + l16;
    last[i] = r < t.rows ? r / p.G + off : -1;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) q[ks][i] = u32x4_t{0u, 0u, 0u, 0u};
    if (r < t.rows) {
      const u16* src = p.q + (t.q0 + r / p.G) * p.q_row + (hk * p.G + r % p.G) * D + D / 4 * lg;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) q[ks][i] = *reinterpret_cast<const u32x4_t*>(src + 8 * ks);
    }
  }
  const View4<D> view(q4.c, slot * p.Hk + hk, lane);
  Step4<D> now = {}, next = {};
  if (first + wave < end) now = view.load(first + wave);
  end_loads(q);

  Acc<D, NI> acc;
  acc.init();
  bool odd = false;  // some step dropped infinities or NaN of v
  for (int s = first + wave; s < end; s += WAVES) {
    if (s + WAVES < end) next = view.load(s + WAVES);
    f32x4_t x[2][NI];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float scale = scale_of(now.ks, j);
#pragma unroll
      for (int i = 0; i < NI; ++i) x[j][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const u32x4_t k = eight_values(now.k[j][ks], scale);
#pragma unroll
        for (int i = 0; i < NI; ++i) x[j][i] = mfma(k, q[ks][i], x[j][i]);
      }
    }
    bool drop = false;
    if ((s + 1) * kCache4Tile > all_keys) {  // some row does not see all of these keys
      asm volatile("");  // keeps this a branch
      drop = may_be_odd<D>(now);
      odd |= drop;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int key = s * kCache4Tile + 16 * j + 4 * r + lg;
            if (key > last[i]) x[j][i][r] = kNone;
          }
    }
    acc.raise(x, p.c);
    acc.exps(x[0], p.c);
    acc.exps(x[1], p.c);
    // p in two bf16 parts, its upper half and the rest.  No part of a positive p is zero, so an
    // infinity of v stays one.
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
    auto products = [&](auto dropped) {
      each(
          [&](auto m) {
            constexpr int M = decltype(m)::value;
            VOps v = v_ops<D, M>(now);
            if constexpr (decltype(dropped)::value) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v.a[e] = odd_split(v.a[e]).finite;
                v.b[e] = odd_split(v.b[e]).finite;
              }
            }
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              acc.o[2 * M][i] = mfma(v.a, pr2[i], acc.o[2 * M][i]);
              acc.o[2 * M][i] = mfma(v.a, pr[i], acc.o[2 * M][i]);
              acc.o[2 * M + 1][i] = mfma(v.b, pr2[i], acc.o[2 * M + 1][i]);
              acc.o[2 * M + 1][i] = mfma(v.b, pr[i], acc.o[2 * M + 1][i]);
            }
          },
          std::make_integer_sequence<int, DT / 2>{});
    };
    if (drop) products(std::true_type{});
    else products(std::false_type{});
    now = next;
  }

  // what was dropped, after the loop, where it takes no registers from it
  for (int s = first + wave; odd && s < end; s += WAVES) {
    if ((s + 1) * kCache4Tile <= all_keys) continue;
    now = view.load(s);
    if (!may_be_odd<D>(now)) continue;
    u32x4_t sees[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = s * kCache4Tile + lg + 16 * (e >> 1) + 8 * (e & 1);
        sees[i][e] = (k <= last[i] ? 0x3f80u : 0u) | (k + 4 <= last[i] ? 0x3f800000u : 0u);
      }
    each(
        [&](auto m) {
          constexpr int M = decltype(m)::value;
          VOps v = v_ops<D, M>(now);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v.a[e] = odd_split(v.a[e]).code;
            v.b[e] = odd_split(v.b[e]).code;
          }
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
            const f32x4_t na = mfma(v.a, sees[i], zero), nb = mfma(v.b, sees[i], zero);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              acc.o[2 * M][i][r] += odd_value(na[r]);
              acc.o[2 * M + 1][i][r] += odd_value(nb[r]);
            }
          }
        },
        std::make_integer_sequence<int, DT / 2>{});
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
  lds_barrier();
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    float m = kNone;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) m = fmaxf(m, sml[w][16 * i + l16][0]);
    const float f = __builtin_amdgcn_exp2f(acc.m[i] - (m == kNone ? 0.f : m));
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int e = 0; e < DT; e += 4)
        *reinterpret_cast<f32x4_t*>(&so[wave][l16][DT * (4 * lg + r) + e]) =
            f32x4_t{acc.o[e][i][r], acc.o[e + 1][i][r], acc.o[e + 2][i][r], acc.o[e + 3][i][r]} *
            f;
    lds_barrier();
    // thread: row tid / TPT, D / TPT columns from (tid % TPT) * 4 in strides of 4 TPT
    constexpr int TPT = kAttnThreads / 16;
    const int rr = tid / TPT, r = t.row0 + 16 * i + rr;
    float mr = kNone, lr = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) mr = fmaxf(mr, sml[w][16 * i + rr][0]);
    const float br = mr == kNone ? 0.f : mr;
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
      lr += sml[w][16 * i + rr][1] * __builtin_amdgcn_exp2f(sml[w][16 * i + rr][0] - br);
    if (r < t.rows) {
      const int64_t at = (t.q0 + r / p.G) * p.Hq + hk * p.G + r % p.G;
      const int64_t w = (int64_t)split * p.Tq_total * p.Hq + at;
      const float g = lr > 0.f ? 1.f / lr : lr == 0.f ? 0.f : lr;
#pragma unroll
      for (int cc = 0; cc < D / (4 * TPT); ++cc) {
        const int c = 4 * TPT * cc + 4 * (tid % TPT);
        f32x4_t o = *reinterpret_cast<const f32x4_t*>(&so[0][rr][c]);
#pragma unroll
        for (int ww = 1; ww < WAVES; ++ww) o += *reinterpret_cast<const f32x4_t*>(&so[ww][rr][c]);
        if (p.splits > 1) {
          *reinterpret_cast<f32x4_t*>(p.ws_o + w * D + c) = o;
        } else {
          *reinterpret_cast<u32x2_t*>(p.out + at * D + c) =
              u32x2_t{pack_bf16(o[0] * g, o[1] * g), pack_bf16(o[2] * g, o[3] * g)};
        }
      }
      if (tid % TPT == 0) {
        if (p.splits > 1) *reinterpret_cast<f32x2_t*>(p.ws_ml + 2 * w) = f32x2_t{mr, lr};
        else if (p.lse != nullptr)
          p.lse[at] = lr == 0.f ? kNone : (mr + __builtin_amdgcn_logf(lr)) * kLn2;
      }
    }
    if (i + 1 < NI) lds_barrier();
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

template <int D>
hipError_t go(const Attn4Params& p, int rows, hipStream_t stream) {
  const AttnParams& a = p.a;
  int64_t slots = attn_slots(a.Tq_total, a.N, a.G, rows);
  if (a.cu_q == nullptr) slots = a.N * ((a.Tq * a.G + rows - 1) / rows);
  const dim3 grid((unsigned)(slots * a.Hk * a.splits));
  if (rows == 16) attn4_kernel<D, 1><<<grid, kAttnThreads, 0, stream>>>(p);
  else attn4_kernel<D, 2><<<grid, kAttnThreads, 0, stream>>>(p);
  if (a.splits > 1) return launch_attn_join(a, D, stream);
  return hipGetLastError();
}

}  // namespace

int attn4_rows(int64_t Tq_total, int64_t N, int64_t G) {
  const int64_t mean = (Tq_total * G + N - 1) / N;  // rows of a sequence and key/value head
  return mean <= 16 ? 16 : 32;
}

hipError_t launch_expand4(const Attn4Params& p, int D, hipStream_t stream) {
  const dim3 grid((unsigned)(p.a.N * (p.a.Tk / kCache4Tile) * p.a.Hk));
  if (D == 64) expand4_kernel<64><<<grid, kAttnThreads, 0, stream>>>(p);
  else expand4_kernel<128><<<grid, kAttnThreads, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_attn4(const Attn4Params& p, int rows, int D, hipStream_t stream) {
  return D == 64 ? go<64>(p, rows, stream) : go<128>(p, rows, stream);
}

}  // namespace kda
