// Launch parameters shared by the host API and the kernels of the serving operators.
#ifndef KDA_OPS_PARAMS_H_
#define KDA_OPS_PARAMS_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// One token of each request: kda_step (delta rule, per-key decay) and kda_la_step.
struct StepParams {
  const uint16_t* q;       // bf16 [N, Hk, D], rows q_row elements apart
  const uint16_t* k;       // bf16 [N, Hk, D], rows k_row apart
  const uint16_t* v;       // bf16 [N, H, D], rows v_row apart
  const uint16_t* gate;    // kda_step: bf16 [N, H, D]
  const uint16_t* beta;    // kda_step: bf16 [N, H] (logits)
  const float* A_log;      // kda_step: [H]
  const float* dt_bias;    // kda_step: [H, D]
  const float* g;          // kda_la_step: fp32 [N, H] log decays or nullptr
  const float* decay;      // kda_la_step: fp32 [H] log decays or nullptr
  uint16_t* out;           // bf16 [N, H, D]
  void* state;             // [num_slots, H, D(v), D(k)], bf16 or fp32
  const int64_t* slot_in;  // [N] or nullptr (identity)
  const int64_t* slot_out; // [N] or nullptr (slot_in)
  int64_t num_slots;
  int64_t q_row, k_row, v_row;
  int32_t N, H, group;     // group: heads that share a q/k head
  float scale, lower_bound;
};

// delta: kda_step's rule, else kda_la_step's.  Returns a hipError_t.
hipError_t launch_step(const StepParams& p, bool delta, int D, bool fp32_state,
                       hipStream_t stream);
constexpr int kStepThreads = 256;  // threads of its workgroups, at most

// Prompts through linear attention with one decay per head: kda_la_fwd.
struct LaParams {
  const uint16_t* q;       // bf16 [tokens, Hk, D], rows q_row elements apart
  const uint16_t* k;       // bf16 [tokens, Hk, D], rows k_row apart
  const uint16_t* v;       // bf16 [tokens, H, D], rows v_row apart
  const float* g;          // fp32 [tokens, H] log decays or nullptr
  const float* decay;      // fp32 [H] log decays or nullptr
  uint16_t* out;           // bf16 [tokens, H, D]
  const void* s_in;        // [N, H, D(v), D(k)] bf16/fp32 or nullptr
  void* s_out;             // [N, H, D(v), D(k)] bf16/fp32 or nullptr
  const int64_t* cu;       // [N + 1] or nullptr (batched)
  int64_t q_row, k_row, v_row;
  int64_t T;               // tokens per batch row (batched mode)
  int64_t T_total;
  int32_t N, H, group;     // group: heads that share a q/k head
  int32_t s_in_fp32, s_out_fp32;
  float scale;
  // Segments (split over the tokens): 0, or tokens per segment.  Segment s of sequence n
  // sits in slot floor(start(n) / seg) + n + s; slot j of head h owns D * D floats of ws
  // (in the kernels' accumulator order) and one of ws_decay, both at [j * H + h].
  int32_t seg;
  int64_t slots;
  float* ws;
  float* ws_decay;
};

constexpr int kLaChunk = 64;  // tokens per chunk

// Slots of a segmented launch: segment starts never share one.
constexpr int64_t la_slots(int64_t T_total, int64_t N, int64_t seg) {
  return T_total / seg + N + 1;
}
// Floats of its workspace.
constexpr int64_t la_ws_floats(int64_t slots, int64_t H, int64_t D) {
  return slots * H * (D * D + 1);
}

hipError_t launch_la(const LaParams& p, int D, hipStream_t stream);

// Causal softmax attention with grouped heads: kda_attn_fwd.
struct AttnParams {
  const uint16_t* q;       // bf16 [query tokens, Hq, D], rows q_row elements apart
  const uint16_t* k;       // bf16 [key tokens, Hk, D], rows k_row apart
  const uint16_t* v;       // bf16 [key tokens, Hk, D], rows v_row apart
  uint16_t* out;           // bf16 [query tokens, Hq, D]
  float* lse;              // fp32 [query tokens, Hq] or nullptr
  const int64_t* cu_q;     // [N + 1] or nullptr (every sequence has Tq queries)
  const int64_t* cu_k;     // [N + 1] or nullptr (sequence n has row n of Tk keys)
  const int64_t* k_lens;   // [N] keys in use of each row, or nullptr (all)
  int64_t q_row, k_row, v_row;
  int64_t Tq, Tk;          // query and key tokens of one batch row
  int64_t Tq_total;
  int32_t N, Hq, Hk, G;    // G = Hq / Hk query heads share a key/value head
  float c;                 // scale * log2(e)
  int32_t splits;          // parts of a row's keys, joined by a second kernel when above 1
  float* ws_o;             // [splits, query tokens, Hq, D] unnormalised outputs
  float* ws_ml;            // [splits, query tokens, Hq, 2] running maximum (base 2) and sum
};

// The schedule of a call: rows are (query token, head of the group) pairs of one key/value
// head; a workgroup owns a tile of them.
struct AttnSchedule {
  int tokens;              // 1: the kernel whose waves split the keys; 0: the tile kernel
  int tiles16;             // 16-row tiles per wave (tile kernel) or workgroup (token kernel)
  int rows;                // rows per workgroup
};

AttnSchedule attn_schedule(int64_t Tq_total, int64_t N, int64_t G);
// Tiles of one key/value head: a sequence's tiles never share a slot with another's.
constexpr int64_t attn_slots(int64_t Tq_total, int64_t N, int64_t G, int64_t rows) {
  return Tq_total * G / rows + N;
}
constexpr int kAttnThreads = 256;
constexpr int kAttnKeys = 64;  // keys per step of the tile kernel

hipError_t launch_attn(const AttnParams& p, const AttnSchedule& s, int D, hipStream_t stream);

}  // namespace kda

#endif  // KDA_OPS_PARAMS_H_
