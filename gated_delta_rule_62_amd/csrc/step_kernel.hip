// The single-token recurrences for gfx950: kda_step (per-key decay, delta rule) and
// kda_la_step (one decay per head).  Per request and head, on a V x K state S:
//
//   kda_step      a = exp(lb sigmoid(exp(A_log) (g + dt_bias)))       per key
//                 u = sigmoid(beta) (v - (S diag(a)) kh),  S' = S diag(a) + u kh^T
//                 out = scale S' qh        (qh, kh: L2-normalised rows)
//   kda_la_step   a = exp(g + decay),  S' = a S + v k^T,  out = scale S' q
//
// Bound by HBM: the state is read and written once and everything else is D-long.  A
// state row of D keys lies across D / VEC neighbouring lanes, 16 bytes in each, so one
// wave instruction moves whole rows; the lanes of a row hold the same keys for every
// row, so each lane prepares only its own VEC components of a, kh and qh, in registers,
// and no LDS or barrier is used.  All of a wave's rows are requested before the gate is
// computed, so their latency covers it.  The two row sums a lane group needs,
// p = (S diag(a)) kh and o = (S diag(a)) qh, are formed together: out's second term is
// u (kh . qh), a scalar of the head, which leaves one reduction latency per row and not
// two dependent ones.  A state is read once and written once, long before its next use:
// both accesses are marked non-temporal (96 requests, 96 heads, fp32: 231 to 215 us, 5.6
// TB/s read and written; 256 requests, 32 heads, bf16: 109 to 102 us).  State arithmetic is fp32 for either storage type; out is
// computed from the fp32 state before a bf16 state is rounded.
#include "api_util.h"
#include "gfx950.h"
#include "ops_params.h"

namespace kda {
namespace {

using namespace dev;

// VEC consecutive elements of a state row as floats, from and to 16 bytes.
template <bool FP32>
struct Row;
template <>
struct Row<true> {
  static constexpr int VEC = 4, BYTES = 4;
  static __device__ __forceinline__ void widen(u32x4_t w, float* x) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(w[e]);
  }
  static __device__ __forceinline__ u32x4_t narrow(const float* x) {
    return u32x4_t{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                   __float_as_uint(x[3])};
  }
};
template <>
struct Row<false> {
  static constexpr int VEC = 8, BYTES = 2;
  static __device__ __forceinline__ void widen(u32x4_t w, float* x) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = bf_lo(w[e]);
      x[2 * e + 1] = bf_hi(w[e]);
    }
  }
  static __device__ __forceinline__ u32x4_t narrow(const float* x) {
    return u32x4_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                   pack_bf16(x[6], x[7])};
  }
};

// VEC consecutive bf16 as floats.
template <int VEC>
__device__ __forceinline__ void load_bf16(const u16* p, float* x) {
  if constexpr (VEC == 4) {
    const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      x[2 * e] = bf_lo(w[e]);
      x[2 * e + 1] = bf_hi(w[e]);
    }
  } else {
    Row<false>::widen(*reinterpret_cast<const u32x4_t*>(p), x);
  }
}

// A workgroup owns GROUPS * PASSES value rows of one (request, head): each lane group
// walks PASSES consecutive rows.
template <int D, bool FP32>
struct Cfg {
  static constexpr int LPR = D / Row<FP32>::VEC;                 // lanes per row
  static constexpr int THREADS = D * LPR < kStepThreads ? D * LPR : kStepThreads;
  static constexpr int GROUPS = THREADS / LPR;                   // lane groups of the workgroup
  static constexpr int MOST = D / GROUPS;                        // rows per lane group, one workgroup
};

template <int D, bool FP32, bool DELTA, int PASSES>
__global__ __launch_bounds__((Cfg<D, FP32>::THREADS)) void step_kernel(StepParams p) {
  using R = Row<FP32>;
  using C = Cfg<D, FP32>;
  constexpr int VEC = R::VEC, LPR = C::LPR, GROUPS = C::GROUPS;
  constexpr int TILES = C::MOST / PASSES;  // workgroups per (request, head)
  static_assert(TILES * PASSES == C::MOST, "tiling");

  const unsigned unit = blockIdx.x / TILES;
  const int n = (int)(unit / (unsigned)p.H), h = (int)(unit % (unsigned)p.H);
  const int k0 = ((int)threadIdx.x % LPR) * VEC;  // this lane's keys
  const int row0 = ((int)(blockIdx.x % TILES) * GROUPS + (int)threadIdx.x / LPR) * PASSES;

  const int64_t src = p.slot_in ? p.slot_in[n] : n;
  const int64_t dst = p.slot_out ? p.slot_out[n] : src;
  const bool has_src = src >= 0 && src < p.num_slots, has_dst = dst >= 0 && dst < p.num_slots;
  const int64_t at = (int64_t)row0 * D + k0;  // inside the head's state
  char* const pool = static_cast<char*>(p.state);

  u32x4_t raw[PASSES];
  if (has_src) {
    const char* s = pool + ((src * p.H + h) * (int64_t)(D * D) + at) * R::BYTES;
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
      raw[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(s + i * D * R::BYTES));
  } else {
#pragma unroll
    for (int i = 0; i < PASSES; ++i) raw[i] = u32x4_t{0u, 0u, 0u, 0u};
  }

  const int hk = h / p.group;
  const int64_t nh = (int64_t)n * p.H + h;
  float q[VEC], k[VEC], a[VEC];
  load_bf16<VEC>(p.q + n * p.q_row + hk * D + k0, q);
  load_bf16<VEC>(p.k + n * p.k_row + hk * D + k0, k);
  float v[PASSES];
  {
    const u16* pv = p.v + n * p.v_row + h * D + row0;  // PASSES * 2 bytes, so aligned
    if constexpr (PASSES == 1) {
      v[0] = bf2f(pv[0]);
    } else {
#pragma unroll
      for (int i = 0; i < PASSES; i += 2) {
        const unsigned w = *reinterpret_cast<const unsigned*>(pv + i);
        v[i] = bf_lo(w);
        v[i + 1] = bf_hi(w);
      }
    }
  }
  float b = 1.f;
  if constexpr (DELTA) {
    float x[VEC];
    load_bf16<VEC>(p.gate + nh * D + k0, x);
    const float rate = expf(p.A_log[h]);
    const float* bias = p.dt_bias + h * D + k0;
    float qq = 0.f, kk = 0.f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      a[e] = expf(p.lower_bound / (1.f + expf(-rate * (x[e] + bias[e]))));
      qq = fmaf(q[e], q[e], qq);
      kk = fmaf(k[e], k[e], kk);
    }
    const float rq = 1.f / sqrtf(group_sum<LPR>(qq) + 1e-6f);
    const float rk = 1.f / sqrtf(group_sum<LPR>(kk) + 1e-6f);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      q[e] *= rq;
      k[e] *= rk;
    }
    b = 1.f / (1.f + expf(-bf2f(p.beta[nh])));
  } else {
    const float lam = (p.g ? p.g[nh] : 0.f) + (p.decay ? p.decay[h] : 0.f);
    a[0] = expf(lam > 0.f ? 0.f : lam);  // log decays above zero count as zero; NaN stays
  }
  float kq = 0.f;
#pragma unroll
  for (int e = 0; e < VEC; ++e) kq = fmaf(k[e], q[e], kq);
  kq = group_sum<LPR>(kq);

  float o[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    float s[VEC];
    R::widen(raw[i], s);
    float pk = 0.f, pq = 0.f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      s[e] *= DELTA ? a[e] : a[0];
      if constexpr (DELTA) pk = fmaf(s[e], k[e], pk);
      pq = fmaf(s[e], q[e], pq);
    }
    float u = v[i];
    if constexpr (DELTA) u = b * (u - group_sum<LPR>(pk));
    o[i] = p.scale * fmaf(u, kq, group_sum<LPR>(pq));
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[e] = fmaf(u, k[e], s[e]);
    raw[i] = R::narrow(s);
  }
  if (has_dst) {
    char* s = pool + ((dst * p.H + h) * (int64_t)(D * D) + at) * R::BYTES;
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
      __builtin_nontemporal_store(raw[i], reinterpret_cast<u32x4_t*>(s + i * D * R::BYTES));
  }
  if (k0 == 0) {
    u16* out = p.out + nh * D + row0;
    if constexpr (PASSES == 1) {
      out[0] = (u16)pack_bf16(o[0], 0.f);
    } else {
#pragma unroll
      for (int i = 0; i < PASSES; i += 2)
        *reinterpret_cast<unsigned*>(out + i) = pack_bf16(o[i], o[i + 1]);
    }
  }
}

template <int D, bool FP32, bool DELTA, int PASSES>
hipError_t go(const StepParams& p, hipStream_t stream) {
  using C = Cfg<D, FP32>;
  const dim3 grid((unsigned)((int64_t)p.N * p.H * (C::MOST / PASSES)));
  step_kernel<D, FP32, DELTA, PASSES><<<grid, C::THREADS, 0, stream>>>(p);
  return hipGetLastError();
}

// The fewest workgroups per head that still give every compute unit kWant of them, and
// the most (one row per lane group) when even those do not.
template <int D, bool FP32, bool DELTA>
hipError_t pick(const StepParams& p, hipStream_t stream) {
  constexpr int MOST = Cfg<D, FP32>::MOST;
  constexpr int kWant = 4;
  const int64_t units = (int64_t)p.N * p.H, want = (int64_t)kWant * device_cus();
  if constexpr (MOST >= 16)
    if (units >= want) return go<D, FP32, DELTA, 16>(p, stream);
  if constexpr (MOST >= 8)
    if (units * (MOST / 8) >= want) return go<D, FP32, DELTA, 8>(p, stream);
  if constexpr (MOST >= 4)
    if (units * (MOST / 4) >= want) return go<D, FP32, DELTA, 4>(p, stream);
  if constexpr (MOST >= 2)
    if (units * (MOST / 2) >= want) return go<D, FP32, DELTA, 2>(p, stream);
  return go<D, FP32, DELTA, 1>(p, stream);
}

template <int D, bool FP32>
hipError_t by_rule(const StepParams& p, bool delta, hipStream_t stream) {
  return delta ? pick<D, FP32, true>(p, stream) : pick<D, FP32, false>(p, stream);
}

}  // namespace

hipError_t launch_step(const StepParams& p, bool delta, int D, bool fp32_state,
                       hipStream_t stream) {
  switch (D) {
    case 32:
      return fp32_state ? by_rule<32, true>(p, delta, stream) : by_rule<32, false>(p, delta, stream);
    case 64:
      return fp32_state ? by_rule<64, true>(p, delta, stream) : by_rule<64, false>(p, delta, stream);
    default:
      return fp32_state ? by_rule<128, true>(p, delta, stream)
                        : by_rule<128, false>(p, delta, stream);
  }
}

}  // namespace kda
