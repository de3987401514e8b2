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

}  // namespace kda

#endif  // KDA_OPS_PARAMS_H_
