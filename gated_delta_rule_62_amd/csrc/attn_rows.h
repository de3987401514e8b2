// What the attention kernels share (gfx950): tiles of rows, and one pass over the keys with a
// running maximum and sum, a row per accumulator column.
#ifndef KDA_ATTN_ROWS_H_
#define KDA_ATTN_ROWS_H_

#include "gfx950.h"
#include "ops_params.h"

namespace kda {
namespace dev {

constexpr float kRaise = 8.f;  // base-2 slack of the running maximum
constexpr float kNone = -__builtin_inff();

// A tile of rows: its sequence's queries and keys, its rows.
struct Tile {
  int n;            // its sequence
  int64_t q0, k0;   // first query and key token
  int Lq, Lk;       // lengths
  int row0, rows;   // first row of the tile, rows of the sequence (Lq * G)
};

__device__ __forceinline__ int64_t clamp64(int64_t x, int64_t lo, int64_t hi) {
  return x < lo ? lo : (x > hi ? hi : x);
}

__device__ __forceinline__ void query_bounds(const AttnParams& p, int n, int64_t& a, int64_t& b) {
  if (p.cu_q != nullptr) {
    a = clamp64(p.cu_q[n], 0, p.Tq_total);
    b = clamp64(p.cu_q[n + 1], a, p.Tq_total);
  } else {
    a = (int64_t)n * p.Tq;
    b = a + p.Tq;
  }
}

__device__ __forceinline__ void key_bounds(const AttnParams& p, int n, int64_t& a, int64_t& b) {
  if (p.cu_k != nullptr) {
    a = clamp64(p.cu_k[n], 0, p.Tk);
    b = clamp64(p.cu_k[n + 1], a, p.Tk);
  } else {
    a = (int64_t)n * p.Tk;
    b = a + (p.k_lens != nullptr ? clamp64(p.k_lens[n], 0, p.Tk) : p.Tk);
  }
}

// The tile of `tile_rows` rows that starts at row row0 of sequence n; false if there is none.
__device__ __forceinline__ bool set_tile(const AttnParams& p, int n, int64_t row0, Tile& t) {
  int64_t a, b;
  query_bounds(p, n, a, b);
  if (row0 < 0 || row0 >= (b - a) * p.G) return false;
  t.n = n;
  t.row0 = (int)row0;
  t.q0 = a;
  t.Lq = (int)(b - a);
  t.rows = t.Lq * p.G;
  key_bounds(p, n, a, b);
  t.k0 = a;
  t.Lk = (int)(b - a);
  return true;
}

// Tile number `slot` of a key/value head, in any order; false if it has none.
__device__ __forceinline__ bool find_tile(const AttnParams& p, unsigned slot, int tile_rows,
                                          Tile& t) {
  if (p.cu_q == nullptr) {
    const unsigned per = (unsigned)((p.Tq * p.G + tile_rows - 1) / tile_rows), n = slot / per;
    return n < (unsigned)p.N && set_tile(p, (int)n, (int64_t)(slot % per) * tile_rows, t);
  }
  // the last sequence whose first slot is not behind this one (first slots grow strictly)
  int lo = 0, hi = p.N - 1;
  int64_t a, b;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    query_bounds(p, mid, a, b);
    if (a * p.G / tile_rows + mid <= slot) lo = mid;
    else hi = mid - 1;
  }
  query_bounds(p, lo, a, b);
  return set_tile(p, lo, (slot - (a * p.G / tile_rows + lo)) * tile_rows, t);
}

__device__ __forceinline__ float max_over_groups(float x) {
  Two t = swap16(x);
  x = fmaxf(t.a, t.b);
  t = swap32(x);
  return fmaxf(t.a, t.b);
}
__device__ __forceinline__ float sum_over_groups(float x) {
  Two t = swap16(x);
  x = t.a + t.b;
  t = swap32(x);
  return t.a + t.b;
}

// Waits for the loads of a tile of rows before the loop over the keys: their first use inside
// it would make every step wait for all loads in flight.
template <int KS, int NI>
__device__ __forceinline__ void end_loads(u32x4_t (&q)[KS][NI]) {
#pragma unroll
  for (int ks = 0; ks < KS; ++ks)
#pragma unroll
    for (int i = 0; i < NI; ++i) asm volatile("" : "+v"(q[ks][i]));
}

// Descriptor of `tokens` rows of one head from `base` as four words, for load_lds; nothing when
// there are none.
__device__ __forceinline__ u32x4_t rows_words(const u16* base, int64_t row, int tokens, int D) {
  const uint64_t at = reinterpret_cast<uint64_t>(base);
  const uint32_t bytes = tokens > 0 ? (uint32_t)(tokens - 1) * (uint32_t)(row * 2) + D * 2u : 0u;
  return u32x4_t{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)at),
                 (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(at >> 32) & 0xffffu),
                 (uint32_t)__builtin_amdgcn_readfirstlane(bytes), 0x00020000u};
}

// 16 bytes per lane from memory to LDS: lane l's land 16 l bytes behind `to` (uniform);
// zeros where `off` is behind the descriptor's end.  It has no result the compiler could
// track: wait_loads ends it, and a barrier shows it to the other waves.  ONCE (non-temporal)
// is for what one workgroup alone reads as a rule, so that it does not displace what others do.
template <bool ONCE>
__device__ __forceinline__ void load_lds(u32x4_t rsrc, const u16* to, uint32_t off) {
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const u16*)to;
  const uint32_t m0 = (uint32_t)__builtin_amdgcn_readfirstlane(at);
  if constexpr (ONCE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
                 :
                 : "s"(m0), "v"(off), "s"(rsrc)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(m0), "v"(off), "s"(rsrc)
                 : "memory", "m0");
}

// Waits until at most the N youngest of this wave's vector memory accesses are in flight, and
// until its LDS accesses are done.  The compiler moves no access over either.
template <int N = 0>
__device__ __forceinline__ void wait_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | (N >> 4 << 14));
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void wait_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);
  asm volatile("" ::: "memory");
}

// Row state and output tiles of NI 16-row tiles: lane = row l16, d = 16 dt + 4 lg + i.
template <int D, int NI>
struct Acc {
  static constexpr int DT = D / 16;
  f32x4_t o[DT][NI];
  float m[NI], l[NI];  // maximum of the scaled scores (base 2), this lane's part of the sum

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      m[i] = kNone;
      l[i] = 0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
  }

  // Raises the running maximum where a row of x (scores, masked ones minus infinity) outgrows
  // it.
  template <int JT>
  __device__ __forceinline__ void raise(const f32x4_t (&x)[JT][NI], float c) {
    float top[NI];
    bool any = false;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float t = kNone;
#pragma unroll
      for (int j = 0; j < JT; ++j) {
        t = fmaxf(t, fmaxf(x[j][i][0], x[j][i][1]));
        t = fmaxf(t, fmaxf(x[j][i][2], x[j][i][3]));
      }
      top[i] = max_over_groups(t) * c;
      any |= top[i] > m[i] + kRaise;  // minus infinity plus kRaise: any score raises it
    }
    if (__any(any)) {  // uniform
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const float now = fmaxf(m[i], top[i]);
        const float f = now == kNone ? 1.f : __builtin_amdgcn_exp2f(m[i] - now);
        m[i] = now;
        l[i] *= f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d][i] *= f;
      }
    }
  }

  // One 16-key tile of scores to probabilities, in place.
  __device__ __forceinline__ void exps(f32x4_t (&x)[NI], float c) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const float base = m[i] == kNone ? 0.f : -m[i];
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[i][r] = __builtin_amdgcn_exp2f(fmaf(x[i][r], c, base));
        s += x[i][r];
      }
      l[i] += s;
    }
  }
};

}  // namespace dev
}  // namespace kda

#endif  // KDA_ATTN_ROWS_H_
