// Launch parameters shared by the host API and the kernels of the operators around attention
// and recurrences: norms, rotary positions, 4-bit caches.
#ifndef KDA_LAYER_PARAMS_H_
#define KDA_LAYER_PARAMS_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_params.h"

namespace kda {

// kda_norm.  A row is `pieces` pieces of W channels; a workgroup (or wave) owns one of them.
struct NormParams {
  const uint16_t* x;       // bf16 [R, pieces * W], rows x_row elements apart
  const uint16_t* gate;    // the same, rows gate_row apart, or nullptr
  const void* post_w;      // [group] or nullptr
  const void* w;           // [W] or nullptr (then pieces may exceed one)
  const void* res;         // [R, pieces * W] or nullptr
  void* res_out;           // the same
  uint16_t* out;           // bf16 [R, pieces * W] or nullptr
  int64_t x_row, gate_row;
  int64_t items;           // R * pieces
  int32_t W, group, pieces;
  int32_t silu, w_fp32, res_fp32;
  float eps, alpha;
};
constexpr int kNormMaxW = 16384;
// Channels of a workgroup's piece when nothing couples a row's groups.
int norm_piece(int64_t W, int64_t group);
// Threads of a row of W channels.
int norm_threads(int64_t W);
hipError_t launch_norm(const NormParams& p, hipStream_t stream);

// kda_rope.
struct RopeParams {
  const uint16_t* q;       // bf16 [tokens, Hq, D], rows q_row elements apart
  const uint16_t* k;       // bf16 [tokens, Hk, D], rows k_row apart (Hk 0: none)
  uint16_t* q_out;
  uint16_t* k_out;
  const double* freqs;     // [rot / 2] radians per position
  const int64_t* pos;      // [tokens] or nullptr
  const int64_t* offsets;  // [N] first positions or nullptr (0)
  const int64_t* cu;       // [N + 1] or nullptr (batch rows of T tokens)
  int64_t q_row, k_row, q_out_row, k_out_row;
  int64_t T, tokens;
  int32_t N, Hq, Hk, D, rot;
  int32_t q_copy, k_copy;  // whether the channels behind rot are copied (not in place)
  int32_t interleaved;
  float amplitude, sign;   // sign -1 turns back
  int32_t tpb;             // tokens of a workgroup
};
constexpr int kRopeThreads = 256;
constexpr int kRopePairs = 512;   // cosines and sines of a workgroup, at most
constexpr int kRopeMaxD = 1024;
void rope_schedule(RopeParams& p);
hipError_t launch_rope(const RopeParams& p, hipStream_t stream);

// A cache of keys and values in 4 bits: see kda.h for the places of codes and scales.
struct Cache4 {
  uint8_t* k4;  // [slots, Hk, cap, D / 2]
  uint8_t* ks;  // [slots, Hk, cap / 32, D / 32, 32]
  uint8_t* v4;  // [slots, Hk, cap / 32, 16 D]
  uint8_t* vs;  // [slots, Hk, cap / 32, D / 32, 32]
  int64_t slots, cap;
};
constexpr int kCache4Tile = 32;

// kda_cache4_put.
struct Put4Params {
  const uint16_t* k;       // bf16 [tokens, Hk, D], rows k_row elements apart
  const uint16_t* v;       // the same, rows v_row apart
  Cache4 c;
  uint16_t* k_out;         // bf16 [tokens, Hk, D] or nullptr
  uint16_t* v_out;
  const int64_t* offsets;  // [N] first positions or nullptr (0)
  const int64_t* slot;     // [N] or nullptr (n)
  const int64_t* cu;       // [N + 1] or nullptr (batch rows of T tokens)
  int64_t k_row, v_row;
  int64_t T, tokens;
  int32_t N, Hk;
};
// Tiles that the tokens of a call touch, at most; a sequence's never share a slot.
constexpr int64_t put4_tiles(int64_t tokens, int64_t T, int64_t N, bool packed) {
  return packed ? tokens / kCache4Tile + 2 * N : N * ((T + 62) / kCache4Tile);
}
constexpr int put4_threads(int D) { return 2 * D; }  // a piece of 8 channels of two positions each
hipError_t launch_put4(const Put4Params& p, int D, hipStream_t stream);

// kda_attn4_fwd: the rows and outputs of AttnParams (its k, v and cu_k are unused, Tk is cap).
struct Attn4Params {
  AttnParams a;
  Cache4 c;
  const int64_t* slot;     // [N] or nullptr (n)
  int32_t part;            // tiles of 32 keys per part
  uint16_t* k_ws;          // expanded keys and values [N, cap, Hk, D] (many rows)
  uint16_t* v_ws;
  int64_t* lens;           // [N] their lengths
  int32_t row_tiles;       // tiles of rows of a batch row
  int32_t once;            // one tile of rows a sequence: its keys are read once
};
// Rows of a sequence and key/value head from which on keys and values are expanded.
constexpr int kExpand4Rows = 448;
constexpr int kAttn4Rows = 16;  // rows of a workgroup
hipError_t launch_expand4(const Attn4Params& p, int D, hipStream_t stream);
hipError_t launch_attn4(const Attn4Params& p, int D, hipStream_t stream);

}  // namespace kda

#endif  // KDA_LAYER_PARAMS_H_
