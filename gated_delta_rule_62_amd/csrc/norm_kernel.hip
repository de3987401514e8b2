// The norms before and after a block, fused with its gate and the residual sum (kda_norm), for
// gfx950.  Per row of W channels, each part there or not:
//
//     u = x                                              bf16
//     u = u / sqrt(mean_group(u^2) + eps) post_w         norm behind the block, by groups
//     u = u act(gate)                                    act: sigmoid, or silu
//     h = residual + alpha u                             -> residual_out
//     y = h / sqrt(mean_W(h^2) + eps) w                  norm before the next block -> out
//
// One pass: a row stays in registers between its loads and its stores, so every input is read
// once and every output written once, and HBM bounds it.  Everything between is fp32; h enters
// the second norm as it is before residual_out is rounded.
//
// Measured: 8192 rows of 4096 with both norms, gate and an fp32 residual 85 us (5.5 TB/s, above a
// plain copy's 5.1: loads that do not stay in the caches); 2048 rows of 96 gated heads of 128, views
// of wider rows, 30.1 us (5.0 TB/s; as pieces of 2048 channels to a workgroup 32.8; with a full
// division in the gate and two more selections an element, bound by arithmetic, 36); four rows 3.7.
#include "gfx950.h"
#include "layer_params.h"

namespace kda {
namespace {

using namespace dev;

// Eight channels as floats: bf16 or fp32 in memory.
struct F8 {
  float v[8];
};
__device__ __forceinline__ F8 widen(u32x4_t w) {
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = bf_lo(w[i]);
    r.v[2 * i + 1] = bf_hi(w[i]);
  }
  return r;
}
// ONCE: not to stay in the caches.
template <bool ONCE, class T>
__device__ __forceinline__ T get(const T* at) {
  if constexpr (ONCE) return __builtin_nontemporal_load(at);
  else return *at;
}
template <bool ONCE>
__device__ __forceinline__ F8 load8(const void* at, int64_t e, bool fp32) {
  if (!fp32)
    return widen(get<ONCE>(reinterpret_cast<const u32x4_t*>(static_cast<const u16*>(at) + e)));
  const f32x4_t* f = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(at) + e);
  const f32x4_t a = get<ONCE>(f), b = get<ONCE>(f + 1);
  return F8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
__device__ __forceinline__ u32x4_t narrow(const F8& r) {
  return u32x4_t{pack_bf16(r.v[0], r.v[1]), pack_bf16(r.v[2], r.v[3]), pack_bf16(r.v[4], r.v[5]),
                 pack_bf16(r.v[6], r.v[7])};
}

// Sum over aligned groups of `lanes` lanes (a power of two from 4 to 64, the same for the wave).
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  v = group_sum<4>(v);
  if (lanes >= 8) v += dpp<0x141>(v);
  if (lanes >= 16) v += dpp<0x140>(v);
  if (lanes >= 32) {
    const Two t = swap16(v);
    v = t.a + t.b;
  }
  if (lanes >= 64) {
    const Two t = swap32(v);
    v = t.a + t.b;
  }
  return v;
}

// TPR threads own a row, C chunks of 8 channels each; a workgroup holds max(TPR, 256) threads, and
// several rows of a wave or less.
template <int TPR, int C>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_kernel(NormParams p) {
  constexpr int WG = TPR < 256 ? 256 : TPR, WAVES = TPR < 64 ? 1 : TPR / 64;
  __shared__ float part[2][WAVES];
  const int tid = threadIdx.x, t = tid % TPR;
  int64_t item = (int64_t)blockIdx.x * (WG / TPR) + tid / TPR;
  const int W = item < p.items ? p.W : 0;  // a row that is not there has no channels
  if (item >= p.items) item = p.items - 1;
  const int64_t row = p.pieces == 1 ? item : item / p.pieces;
  const int first = p.pieces == 1 ? 0 : (int)(item % p.pieces) * p.W;
  const int64_t at = item * p.W;  // rows of res, res_out and out follow each other

  // a sum over the row's threads
  auto row_sum = [&](float v, int which) {
    v = lanes_sum(v, TPR < 64 ? TPR : 64);
    if constexpr (WAVES > 1) {
      if ((tid & 63) == 0) part[which][t >> 6] = v;
      lds_barrier();
      v = 0.f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) v += part[which][w];
    }
    return v;
  };

  F8 u[C], r[C];
  u32x4_t gate[C];
  const u16 *x = p.x + row * p.x_row + first,
            *g = p.gate != nullptr ? p.gate + row * p.gate_row + first : nullptr;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = (c * TPR + t) * 8;
    const bool in = e < W;
    u32x4_t w = u32x4_t{0u, 0u, 0u, 0u};
    gate[c] = w;
    r[c] = F8{};
    if (in) {
      w = get<true>(reinterpret_cast<const u32x4_t*>(x + e));
      if (g != nullptr) gate[c] = get<true>(reinterpret_cast<const u32x4_t*>(g + e));
      if (p.res != nullptr) r[c] = load8<true>(p.res, at + e, p.res_fp32);
    }
    u[c] = widen(w);
  }

  if (p.post_w != nullptr) {
    float s[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      s[c] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s[c] = fmaf(u[c].v[i], u[c].v[i], s[c]);
    }
    if (p.group < p.W) {  // groups of 4 to 64 lanes
#pragma unroll
      for (int c = 0; c < C; ++c) s[c] = lanes_sum(s[c], p.group / 8);
    } else {
      float all = s[0];
#pragma unroll
      for (int c = 1; c < C; ++c) all += s[c];
      all = row_sum(all, 0);
#pragma unroll
      for (int c = 0; c < C; ++c) s[c] = all;
    }
    const float n = (float)p.group;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = (c * TPR + t) * 8;
      if (e < W) {
        const float f = rsqrtf(s[c] / n + p.eps);
        const F8 w = load8<false>(p.post_w, p.group < p.W ? e & (p.group - 1) : e, p.w_fp32);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[c].v[i] = u[c].v[i] * f * w.v[i];
      }
    }
  }
  if (g != nullptr) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const F8 z = widen(gate[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // sigmoid(z) = s s / (1 + t t) with t = e^(-|z| / 2) and s = t or 1: factors that underflow
        // only where the result does
        const float t = __builtin_amdgcn_exp2f(-0.5f * kLog2e * fabsf(z.v[i]));
        const float s = z.v[i] < 0.f ? t : 1.f;
        u[c].v[i] = u[c].v[i] * s * (s * __builtin_amdgcn_rcpf(fmaf(t, t, 1.f)));
      }
      if (p.silu) {  // after the sigmoid, so that a large u does not overflow on the way to zero
#pragma unroll
        for (int i = 0; i < 8; ++i) u[c].v[i] *= z.v[i];
      }
    }
  }
  if (p.res != nullptr) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = (c * TPR + t) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) u[c].v[i] = fmaf(p.alpha, u[c].v[i], r[c].v[i]);
      if (e < W) {
        if (p.res_fp32) {
          f32x4_t* to = reinterpret_cast<f32x4_t*>(static_cast<float*>(p.res_out) + at + e);
          to[0] = f32x4_t{u[c].v[0], u[c].v[1], u[c].v[2], u[c].v[3]};
          to[1] = f32x4_t{u[c].v[4], u[c].v[5], u[c].v[6], u[c].v[7]};
        } else {
          *reinterpret_cast<u32x4_t*>(static_cast<u16*>(p.res_out) + at + e) = narrow(u[c]);
        }
      }
    }
  }
  if (p.w != nullptr) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(u[c].v[i], u[c].v[i], s);
    const float f = rsqrtf(row_sum(s, 1) / (float)p.W + p.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = (c * TPR + t) * 8;
      if (e < W) {
        const F8 w = load8<false>(p.w, e, p.w_fp32);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[c].v[i] = u[c].v[i] * f * w.v[i];
      }
    }
  }
  if (p.out != nullptr) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = (c * TPR + t) * 8;
      if (e < W) *reinterpret_cast<u32x4_t*>(p.out + at + e) = narrow(u[c]);
    }
  }
}

}  // namespace

// A wave for rows of up to 1024 channels (32,768 rows of 800: 39 us, 49 by workgroups), else a
// workgroup: 512 threads from 2048 on (8192 rows of 4096: 85 us, 87 with 256; more threads gain half
// a microsecond with few rows and lose 4-17% of many).
int norm_threads(int64_t W) {
  return W <= 64 ? 8 : W <= 128 ? 16 : W <= 256 ? 32 : W <= 1024 ? 64 : W <= 2048 ? 256 : 512;
}

int norm_piece(int64_t W, int64_t group) {
  int64_t piece = group;
  while (piece * 2 <= 1024 && W % (piece * 2) == 0) piece *= 2;
  return (int)piece;
}

hipError_t launch_norm(const NormParams& p, hipStream_t stream) {
  const int W = p.W, threads = norm_threads(W);
  const int64_t per = threads < 256 ? 256 / threads : 1;
  const dim3 grid((unsigned)((p.items + per - 1) / per));
  if (W <= 64) norm_kernel<8, 1><<<grid, 256, 0, stream>>>(p);
  else if (W <= 128) norm_kernel<16, 1><<<grid, 256, 0, stream>>>(p);
  else if (W <= 256) norm_kernel<32, 1><<<grid, 256, 0, stream>>>(p);
  else if (W <= 512) norm_kernel<64, 1><<<grid, 256, 0, stream>>>(p);
  else if (W <= 1024) norm_kernel<64, 2><<<grid, 256, 0, stream>>>(p);
  else if (W <= 2048) norm_kernel<256, 1><<<grid, 256, 0, stream>>>(p);
  else if (W <= 4096) norm_kernel<512, 1><<<grid, 512, 0, stream>>>(p);
  else if (W <= 8192) norm_kernel<512, 2><<<grid, 512, 0, stream>>>(p);
  else norm_kernel<512, 4><<<grid, 512, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace kda
