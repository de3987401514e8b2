// Rotary positions of queries and keys (kda_rope), for gfx950.
//
//     angle = position f_i,   (a, b) -> amplitude (a cos - b sin, a sin + b cos)
//
// for the pairs (i, i + rot / 2) or (2 i, 2 i + 1) of a head's first rot channels; the rest is
// copied.  The angle of a far position has more digits than fp32: position and frequency are
// multiplied in 64 bits and reduced to a fraction of a turn there, whose sine and cosine are
// fp32.  They are the same for all heads of a token: a workgroup forms those of its tokens once,
// in LDS, then streams the heads past them, bound by HBM.
//
// Measured: 2024 tokens of 96/8 heads, D 128, 21.6 us, 8192 tokens of 32/8 heads, half of each turned
// in pairs side by side, 32.1 us: 5.0 and 5.2 TB/s, a copy's rate.  Loads that do not stay in the
// caches gave a tenth; stores that do not would lose a fifth where a row's turned part is half a
// cache line.
#include "gfx950.h"
#include "layer_params.h"

namespace kda {
namespace {

using namespace dev;

// Position of a token; with cu, `near` is the sequence of the workgroup's first token.
__device__ __forceinline__ int64_t position(const RopeParams& p, int64_t token, int near) {
  if (p.pos != nullptr) return p.pos[token];
  int64_t n, first;
  if (p.cu == nullptr) {
    n = token / p.T;
    first = n * p.T;
  } else {  // the last sequence that starts at or before the token
    int lo = near, hi = near + 1 < p.N && p.cu[near + 1] <= token ? p.N - 1 : near;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.cu[mid] <= token) lo = mid;
      else hi = mid - 1;
    }
    n = lo;
    first = p.cu[lo];
  }
  const uint64_t from = p.offsets != nullptr ? (uint64_t)p.offsets[n] : 0u;
  return (int64_t)(from + (uint64_t)token - (uint64_t)first);
}

// Cosines and sines of `tokens` tokens from token0 on, in LDS.
__device__ __forceinline__ void turns_of(const RopeParams& p, int64_t token0, int tokens,
                                         f32x2_t* turn) {
  const int half = p.rot / 2;
  const int near =
      p.cu == nullptr ? 0 : find_last(p.N, [&](int i) { return p.cu[i] <= token0; });
  for (int e = threadIdx.x; e < tokens * half; e += kRopeThreads) {
    const int tk = e / half, i = e - tk * half;
    const double turns =
        (double)position(p, token0 + tk, near) * (p.freqs[i] * 0.15915494309189535);  // 1 / (2 pi)
    float s, c;
    sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
    turn[e] = f32x2_t{c * p.amplitude, s * p.amplitude * p.sign};
  }
}

// The tokens of a workgroup that some sequence holds: [first, last) of its p.tpb.
struct Span {
  int first, last;
};
__device__ __forceinline__ Span span_of(const RopeParams& p, int64_t token0) {
  auto in_group = [&](int64_t token) {  // token of the batch, clamped, as one of the group
    const int64_t t = token < token0 ? token0 : token;
    return (int)(min(t, min(token0 + p.tpb, p.tokens)) - token0);
  };
  if (p.cu == nullptr) return Span{0, in_group(p.tokens)};
  return Span{in_group(p.cu[0]), in_group(p.cu[p.N])};
}

// A head's row of a token: h counts the query heads, then the key heads.
__device__ __forceinline__ const u16* in_row(const RopeParams& p, int64_t token, int h) {
  return h < p.Hq ? p.q + token * p.q_row + (int64_t)h * p.D
                  : p.k + token * p.k_row + (int64_t)(h - p.Hq) * p.D;
}
__device__ __forceinline__ u16* out_row(const RopeParams& p, int64_t token, int h) {
  return h < p.Hq ? p.q_out + token * p.q_out_row + (int64_t)h * p.D
                  : p.k_out + token * p.k_out_row + (int64_t)(h - p.Hq) * p.D;
}

// 16 bytes that this call reads once.
__device__ __forceinline__ u32x4_t load_once(const u16* x) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(x));
}

// 8 pairs, or 16 channels to copy, a thread and head (rot a multiple of 16): 16-byte accesses.  A
// thread keeps its place in the head and walks the heads, eight of them in flight; the first eight
// are asked for before the turns are formed.
template <bool INTER>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeParams p) {
  __shared__ f32x2_t turn[kRopePairs];
  constexpr int AT_ONCE = 8;
  const int tid = threadIdx.x, half = p.rot / 2;
  const int64_t token0 = (int64_t)blockIdx.x * p.tpb;
  const Span in = span_of(p, token0);
  const int turned = half / 8, units = turned + (p.D - p.rot + 15) / 16;
  const int heads = p.Hq + p.Hk, per = kRopeThreads / units;
  const int unit = tid % units, row0 = in.first * heads + tid / units;
  const int rows = tid < per * units ? in.last * heads : 0;
  const bool turns = unit < turned;
  // two pieces of 8 channels, one in each half of what is turned (also of pairs side by side, so
  // that neighbours' pieces touch), or of what is copied
  const int e0 = turns ? unit * 8 : p.rot + (unit - turned) * 8;
  const int e1 = e0 + (turns ? half : (p.D - p.rot + 15) / 16 * 8);
  const bool two = e1 < p.D;

  u32x4_t a[AT_ONCE], b[AT_ONCE];
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int r = r0 + i * per;
      a[i] = b[i] = u32x4_t{0u, 0u, 0u, 0u};
      if (r < rows) {
        const u16* x = in_row(p, token0 + r / heads, r % heads);
        a[i] = load_once(x + e0);
        if (two) b[i] = load_once(x + e1);
      }
    }
  };
  load(row0);
  turns_of(p, token0, in.last, turn);
  lds_barrier();
  for (int r0 = row0; r0 < rows; r0 += AT_ONCE * per) {
    if (r0 > row0) load(r0);
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int r = r0 + i * per;
      if (r >= rows) break;
      const int tk = r / heads, h = r - tk * heads;
      if (turns) {
        const f32x2_t* cs = turn + tk * half + unit * (INTER ? 4 : 8);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float a0 = bf_lo(a[i][w]), a1 = bf_hi(a[i][w]), b0 = bf_lo(b[i][w]),
                      b1 = bf_hi(b[i][w]);
          if constexpr (INTER) {  // a word is a pair
            const f32x2_t ca = cs[w], cb = cs[half / 2 + w];
            a[i][w] = pack_bf16(a0 * ca[0] - a1 * ca[1], a0 * ca[1] + a1 * ca[0]);
            b[i][w] = pack_bf16(b0 * cb[0] - b1 * cb[1], b0 * cb[1] + b1 * cb[0]);
          } else {
            const f32x2_t cl = cs[2 * w], ch = cs[2 * w + 1];
            a[i][w] = pack_bf16(a0 * cl[0] - b0 * cl[1], a1 * ch[0] - b1 * ch[1]);
            b[i][w] = pack_bf16(a0 * cl[1] + b0 * cl[0], a1 * ch[1] + b1 * ch[0]);
          }
        }
      } else if (!(h < p.Hq ? p.q_copy : p.k_copy)) {
        continue;
      }
      u16* y = out_row(p, token0 + tk, h);
      *reinterpret_cast<u32x4_t*>(y + e0) = a[i];
      if (two) *reinterpret_cast<u32x4_t*>(y + e1) = b[i];
    }
  }
}

// Any even rot: pieces of 8 channels as above, whose partners lie at any distance, so rows go
// through LDS.  8192 tokens of 32/8 heads, 50 of 128 channels: 42 us, pairs side by side 45 (187 with
// a pair a thread; 48 channels by the kernel above 39; the bytes 33).  Two barriers for every four rows
// of a thread are the likely difference; pairs side by side would need neither them nor the LDS.
template <bool INTER>
__global__ __launch_bounds__(kRopeThreads) void rope_any_kernel(RopeParams p) {
  constexpr int AT_ONCE = 4;
  __shared__ f32x2_t turn[kRopePairs];
  __shared__ alignas(16) u16 rows_of[AT_ONCE][kRopeThreads * 8];
  const int tid = threadIdx.x, half = p.rot / 2;
  const int64_t token0 = (int64_t)blockIdx.x * p.tpb;
  const Span in = span_of(p, token0);
  const int units = p.D / 8, per = kRopeThreads / units, heads = p.Hq + p.Hk;
  const int unit = tid % units, first = in.first * heads, rows = in.last * heads;
  const int mine = tid < per * units ? tid / units : rows;  // rows: none
  const int c0 = 8 * unit;

  u32x4_t x[AT_ONCE];
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int r = r0 + mine + i * per;
      x[i] = u32x4_t{0u, 0u, 0u, 0u};
      if (r < rows) x[i] = load_once(in_row(p, token0 + r / heads, r % heads) + c0);
    }
  };
  load(first);
  turns_of(p, token0, in.last, turn);
  for (int r0 = first; r0 < rows; r0 += AT_ONCE * per) {  // the same for the workgroup
    if (r0 > first) load(r0);
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i)
      *reinterpret_cast<u32x4_t*>(&rows_of[i][8 * tid]) = x[i];
    lds_barrier();
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int r = r0 + mine + i * per;
      if (r >= rows) break;
      const int tk = r / heads, h = r - tk * heads;
      if (c0 < p.rot) {
        const u16* row = &rows_of[i][8 * (tid - unit)];
        const f32x2_t* cs = turn + tk * half;
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = c0 + e;
          const float mine_x = e & 1 ? bf_hi(x[i][e >> 1]) : bf_lo(x[i][e >> 1]);
          y[e] = mine_x;
          if (c < p.rot) {
            const bool second = INTER ? e & 1 : c >= half;
            const int pair = INTER ? c >> 1 : second ? c - half : c;
            const float other = INTER ? (e & 1 ? bf_lo(x[i][e >> 1]) : bf_hi(x[i][e >> 1]))
                                      : bf2f(row[second ? c - half : c + half]);
            const f32x2_t t = cs[pair];
            // first: a cos - b sin; second: a sin + b cos
            y[e] = second ? other * t[1] + mine_x * t[0] : mine_x * t[0] - other * t[1];
          }
        }
        x[i] = u32x4_t{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                       pack_bf16(y[6], y[7])};
      } else if (!(h < p.Hq ? p.q_copy : p.k_copy)) {
        continue;
      }
      *reinterpret_cast<u32x4_t*>(out_row(p, token0 + tk, h) + c0) = x[i];
    }
    lds_barrier();
  }
}

}  // namespace

void rope_schedule(RopeParams& p) {
  const int half = p.rot / 2;
  // one cosine and sine a thread at most, and two workgroups a compute unit first (2024 tokens of
  // 104 heads: three tokens each 21.6 us, one 23.6)
  int64_t tpb = kRopeThreads / half;
  const int64_t fill = p.tokens / 512;
  if (tpb > fill) tpb = fill;
  p.tpb = tpb < 1 ? 1 : (int32_t)tpb;
}

hipError_t launch_rope(const RopeParams& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.tokens + p.tpb - 1) / p.tpb));
  const bool any = p.rot % 16 != 0;
  if (any && p.interleaved) rope_any_kernel<true><<<grid, kRopeThreads, 0, stream>>>(p);
  else if (any) rope_any_kernel<false><<<grid, kRopeThreads, 0, stream>>>(p);
  else if (p.interleaved) rope_kernel<true><<<grid, kRopeThreads, 0, stream>>>(p);
  else rope_kernel<false><<<grid, kRopeThreads, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace kda
