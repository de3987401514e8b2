// New keys and values into caches held in 4 bits (kda_cache4_put), for gfx950.
//
// A block of 32 channels of one token and head shares the scale 2^e, the smallest with
// max |x| <= 6 2^e, and holds the codes of x / 2^e: 0, .5, 1, 1.5, 2, 3, 4, 6 and their
// negatives, nearest, ties to even.  The inputs are bf16 and the scale a power of two, so every
// step is exact and the codes do not depend on the machine's rounding.
//
// A workgroup owns a tile of 32 cache positions of one head, whatever tokens of the call fall
// into it: position 16 j + 4 i + g of a tile.  Lanes of a wave hold the 8-channel pieces of the
// four tokens i of one g, for both j, so that 256 contiguous bytes of the values' codes (whose
// places put the four together) and whole rows of the keys' are written by one instruction.
// 2 bytes an element are read, 17/32 written (and 2 more with the values).
//
// Measured: 2024 tokens of 8 heads, D 128, with their values 5.9 us (18.8 MB, 3.2 TB/s), one token of
// each of 32 requests 4.2: the launch and three loads that wait for each other (the sequence, its
// position and slot, its rows).  Even fewer bytes would not make such calls shorter; larger ones come to
// a copy's rate (16,384 tokens 17.6 us, 85 MB, 4.8 TB/s).
#include "cache4.h"
#include "layer_params.h"

namespace kda {
namespace {

using namespace dev;

__device__ __forceinline__ int64_t clip(int64_t x, int64_t lo, int64_t hi) {
  return x < lo ? lo : (x > hi ? hi : x);
}

// First token of sequence n, or the end of the last for n == N.
__device__ __forceinline__ int64_t starts(const Put4Params& p, int n) {
  return p.cu != nullptr ? clip(p.cu[n], 0, p.tokens) : (int64_t)n * p.T;
}

__device__ __forceinline__ unsigned top_of(u32x4_t x) {
  unsigned t = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) t = max(t, max(x[i] & 0x7fffu, x[i] >> 16 & 0x7fffu));
  return t;
}
template <int CTRL>
__device__ __forceinline__ unsigned dpp_max(unsigned v) {
  return max(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, false));
}

template <int D>
__global__ __launch_bounds__(put4_threads(D)) void put4_kernel(Put4Params p) {
  constexpr int PPT = D / 8, LPG = 4 * PPT;  // pieces of a token, lanes of one g
  const int tid = threadIdx.x;
  const unsigned tile_no = blockIdx.x / (unsigned)p.Hk;
  const int h = (int)(blockIdx.x % (unsigned)p.Hk);

  // the sequence of this tile: the last whose first slot is not behind it
  int n;
  int64_t nth;
  if (p.cu == nullptr) {
    const unsigned per = (unsigned)((p.T + 62) / kCache4Tile);
    n = (int)(tile_no / per);
    nth = tile_no % per;
  } else {
    n = find_last(p.N, [&](int i) {
      return starts(p, i) / kCache4Tile + 2 * (int64_t)i <= tile_no;
    });
    nth = tile_no - (starts(p, n) / kCache4Tile + 2 * (int64_t)n);
  }
  const int64_t t0 = starts(p, n);
  int64_t len = starts(p, n + 1) - t0;
  if (len <= 0) return;
  const int64_t from = p.offsets != nullptr ? p.offsets[n] : 0;
  const int64_t slot = p.slot != nullptr ? p.slot[n] : n;
  // token of the tile's first position, counted from the sequence's first
  const int in_tile = (int)(from & (kCache4Tile - 1));
  const int64_t rel0 = nth * kCache4Tile - in_tile;
  if (rel0 >= len) return;
  const int64_t tile = (from >> 5) + nth;
  const bool kept = slot >= 0 && slot < p.c.slots && tile >= 0 && tile < p.c.cap / kCache4Tile;
  if (!kept && p.k_out == nullptr) return;

  const int g = tid / LPG, i = tid % LPG / PPT, piece = tid % PPT;
  u32x4_t x[2][2];  // key or value, j
  bool has[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t rel = rel0 + 16 * j + 4 * i + g;
    has[j] = rel >= 0 && rel < len;
    x[0][j] = x[1][j] = u32x4_t{0u, 0u, 0u, 0u};
    if (has[j]) {
      const int64_t e = (int64_t)h * D + 8 * piece;
      x[0][j] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4_t*>(p.k + (t0 + rel) * p.k_row + e));
      x[1][j] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4_t*>(p.v + (t0 + rel) * p.v_row + e));
    }
  }
  unsigned code[2][2], byte[2][2];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const unsigned top = dpp_max<0x4E>(dpp_max<0xB1>(top_of(x[s][j])));  // over four lanes
      byte[s][j] = scale_byte(top);
      code[s][j] = eight_codes(x[s][j], byte[s][j]);
    }
  if (kept) {
    const int64_t unit = slot * p.Hk + h, tiles = p.c.cap / kCache4Tile;
    uint8_t* kc = p.c.k4 + (unit * p.c.cap + tile * kCache4Tile) * (D / 2) + 4 * piece;
    uint8_t* vc = p.c.v4 + (unit * tiles + tile) * (16 * D);
    const int64_t sc = (unit * tiles + tile) * D + (piece / 4) * 32 + 8 * g + 2 * i;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (has[j]) {
        *reinterpret_cast<unsigned*>(kc + (16 * j + 4 * i + g) * (D / 2)) = code[0][j];
        if constexpr (D == 128) {
          *reinterpret_cast<unsigned*>(vc + j * 1024 + (g * 16 + piece) * 16 + i * 4) = code[1][j];
        } else {
          u16* to = reinterpret_cast<u16*>(vc + (g * 16 + 2 * piece) * 16 + (j * 4 + i) * 2);
          to[0] = (u16)code[1][j];
          to[8] = (u16)(code[1][j] >> 16);
        }
        if ((piece & 3) == 0) {
          p.c.ks[sc + j] = (uint8_t)byte[0][j];
          p.c.vs[sc + j] = (uint8_t)byte[1][j];
        }
      }
  }
  if (p.k_out != nullptr) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (has[j]) {
        const int64_t e =
            ((t0 + rel0 + 16 * j + 4 * i + g) * p.Hk + h) * D + 8 * piece;
        *reinterpret_cast<u32x4_t*>(p.k_out + e) =
            eight_values(code[0][j], __uint_as_float(byte[0][j] << 23));
        *reinterpret_cast<u32x4_t*>(p.v_out + e) =
            eight_values(code[1][j], __uint_as_float(byte[1][j] << 23));
      }
  }
}

}  // namespace

hipError_t launch_put4(const Put4Params& p, int D, hipStream_t stream) {
  const dim3 grid((unsigned)(put4_tiles(p.tokens, p.T, p.N, p.cu != nullptr) * p.Hk));
  if (D == 64) put4_kernel<64><<<grid, put4_threads(64), 0, stream>>>(p);
  else put4_kernel<128><<<grid, put4_threads(128), 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace kda
