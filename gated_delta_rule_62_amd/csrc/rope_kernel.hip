// Rotary positions of queries and keys (kda_rope), for gfx950.
//
//     angle = position f_i,   (a, b) -> amplitude (a cos - b sin, a sin + b cos)
//
// for the pairs (i, i + rot / 2) or (2 i, 2 i + 1) of a head's first rot channels; the rest is
// copied.  The angle of a far position has more digits than fp32: position and frequency are
// multiplied in 64 bits and reduced to a fraction of a turn there, whose sine and cosine are
// fp32.  They are the same for all heads of a token: a workgroup forms those of its tokens once,
// in LDS, then streams the heads past them, bound by HBM.
#include "gfx950.h"
#include "layer_params.h"

namespace kda {
namespace {

using namespace dev;

__device__ __forceinline__ int64_t position(const RopeParams& p, int64_t token) {
  if (p.pos != nullptr) return p.pos[token];
  int64_t n, first;
  if (p.cu == nullptr) {
    n = token / p.T;
    first = n * p.T;
  } else {  // the last sequence that starts at or before the token
    int lo = 0, hi = p.N - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.cu[mid] <= token) lo = mid;
      else hi = mid - 1;
    }
    n = lo;
    first = p.cu[lo];
  }
  const uint64_t from = p.offsets != nullptr ? (uint64_t)p.offsets[n] : 0u;
  return (int64_t)(from + (uint64_t)(token - first));
}

// Whether some sequence holds the token (with cu: one between its ends).
__device__ __forceinline__ bool in_batch(const RopeParams& p, int64_t token) {
  return p.cu == nullptr || (token >= p.cu[0] && token < p.cu[p.N]);
}

// VEC: units of 8 pairs (rot a multiple of 16), 16-byte accesses; else of one pair.
template <bool VEC, bool INTER>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeParams p) {
  __shared__ f32x2_t turn[kRopePairs];
  const int tid = threadIdx.x, half = p.rot / 2;
  const int64_t token0 = (int64_t)(blockIdx.x / (unsigned)p.splits) * p.tpb;
  const int tokens = (int)min((int64_t)p.tpb, p.tokens - token0);
  const int split = (int)(blockIdx.x % (unsigned)p.splits);

  for (int e = tid; e < tokens * half; e += kRopeThreads) {
    const int tk = e / half, i = e - tk * half;
    const double turns = (double)position(p, token0 + tk) * (p.freqs[i] * 0.15915494309189535);
    float s, c;
    sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
    turn[e] = f32x2_t{c * p.amplitude, s * p.amplitude * p.sign};
  }
  lds_barrier();

  // a thread's unit: 8 pairs (or one) of a head, or behind them 16 copied channels (or one)
  constexpr int P = VEC ? 8 : 1, CP = VEC ? 16 : 1;
  const int turned = half / P, rest = p.D - p.rot, units = turned + (rest + CP - 1) / CP;
  const int heads = p.Hq + p.Hk, rows = tokens * heads;
  const int per = max(1, kRopeThreads / units);
  const int stride = p.splits * per;
  for (int unit = tid % units; unit < units; unit += kRopeThreads) {
    if (tid / units >= per) break;
    for (int r = split * per + tid / units; r < rows; r += stride) {
      const int tk = r / heads, h = r - tk * heads;
      const int64_t token = token0 + tk;
      const bool is_q = h < p.Hq;
      const u16* in = is_q ? p.q + token * p.q_row + (int64_t)h * p.D
                           : p.k + token * p.k_row + (int64_t)(h - p.Hq) * p.D;
      u16* out = is_q ? p.q_out + token * p.q_out_row + (int64_t)h * p.D
                      : p.k_out + token * p.k_out_row + (int64_t)(h - p.Hq) * p.D;
      if (!in_batch(p, token)) continue;
      if (unit >= turned) {
        if (!(is_q ? p.q_copy : p.k_copy)) continue;
        const int e = p.rot + (unit - turned) * CP;
        if constexpr (VEC) {
          *reinterpret_cast<u32x4_t*>(out + e) = *reinterpret_cast<const u32x4_t*>(in + e);
          if (e + 8 < p.D)
            *reinterpret_cast<u32x4_t*>(out + e + 8) =
                *reinterpret_cast<const u32x4_t*>(in + e + 8);
        } else {
          out[e] = in[e];
        }
        continue;
      }
      const f32x2_t* cs = turn + tk * half + unit * P;
      if constexpr (VEC) {
        const int e0 = INTER ? unit * 16 : unit * 8, e1 = INTER ? e0 + 8 : half + e0;
        u32x4_t a = *reinterpret_cast<const u32x4_t*>(in + e0),
                b = *reinterpret_cast<const u32x4_t*>(in + e1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (INTER) {  // a word is a pair
            const f32x2_t ca = cs[i], cb = cs[4 + i];
            const float a0 = bf_lo(a[i]), a1 = bf_hi(a[i]), b0 = bf_lo(b[i]), b1 = bf_hi(b[i]);
            a[i] = pack_bf16(a0 * ca[0] - a1 * ca[1], a0 * ca[1] + a1 * ca[0]);
            b[i] = pack_bf16(b0 * cb[0] - b1 * cb[1], b0 * cb[1] + b1 * cb[0]);
          } else {
            const f32x2_t cl = cs[2 * i], ch = cs[2 * i + 1];
            const float a0 = bf_lo(a[i]), a1 = bf_hi(a[i]), b0 = bf_lo(b[i]), b1 = bf_hi(b[i]);
            a[i] = pack_bf16(a0 * cl[0] - b0 * cl[1], a1 * ch[0] - b1 * ch[1]);
            b[i] = pack_bf16(a0 * cl[1] + b0 * cl[0], a1 * ch[1] + b1 * ch[0]);
          }
        }
        *reinterpret_cast<u32x4_t*>(out + e0) = a;
        *reinterpret_cast<u32x4_t*>(out + e1) = b;
      } else {
        const int e0 = INTER ? 2 * unit : unit, e1 = INTER ? e0 + 1 : e0 + half;
        const float a = bf2f(in[e0]), b = bf2f(in[e1]);
        const f32x2_t c = cs[0];
        out[e0] = (u16)pack_bf16(a * c[0] - b * c[1], 0.f);
        out[e1] = (u16)pack_bf16(a * c[1] + b * c[0], 0.f);
      }
    }
  }
}

}  // namespace

void rope_schedule(RopeParams& p) {
  const int half = p.rot / 2;
  // one cosine and sine a thread, and as many workgroups as there are tokens for
  int64_t tpb = kRopeThreads / half;
  if (tpb < 1) tpb = 1;
  const int64_t fill = p.tokens / 2048;
  if (tpb > fill) tpb = fill < 1 ? 1 : fill;
  p.tpb = (int32_t)tpb;
  p.splits = 1;
}

hipError_t launch_rope(const RopeParams& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.tokens + p.tpb - 1) / p.tpb * p.splits));
  const bool vec = p.rot % 16 == 0;
  if (vec && p.interleaved) rope_kernel<true, true><<<grid, kRopeThreads, 0, stream>>>(p);
  else if (vec) rope_kernel<true, false><<<grid, kRopeThreads, 0, stream>>>(p);
  else if (p.interleaved) rope_kernel<false, true><<<grid, kRopeThreads, 0, stream>>>(p);
  else rope_kernel<false, false><<<grid, kRopeThreads, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace kda
