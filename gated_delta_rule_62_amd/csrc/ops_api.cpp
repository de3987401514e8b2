// Host side of the serving operators declared in include/kda.h: argument validation,
// schedule selection and launches.  Nothing here touches device memory.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/kda.h"
#include "api_util.h"
#include "ops_params.h"

namespace {

using kda::make_range;
using kda::overlaps;
using kda::Range;

constexpr int64_t kMaxBytes = (int64_t)1 << 62;  // of one tensor: the range arithmetic cannot wrap

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

bool state_dtype_ok(int dtype) { return dtype == KDA_DTYPE_BF16 || dtype == KDA_DTYPE_FP32; }

// A row stride in elements: whole 16-byte units, at least the row itself.
bool row_ok(int64_t row, int64_t heads, int64_t D) { return row >= heads * D && row % 8 == 0; }

// Bytes from the first element of `rows` bf16 rows to the last, or -1 beyond kMaxBytes.
int64_t span_bytes(int64_t rows, int64_t row, int64_t heads, int64_t D) {
  if (rows <= 0) return 0;
  if (row > kMaxBytes / 2 / rows) return -1;
  return ((rows - 1) * row + heads * D) * 2;
}

bool any_overlap(Range out, const Range* ins, int n) {
  for (int i = 0; i < n; ++i)
    if (overlaps(out, ins[i])) return true;
  return false;
}

// What kda_step and kda_la_step share: sizes, the pool, the slots.
int step_resolve(const void* state, int state_dtype, int64_t num_slots, const int64_t* slot_in,
                 const int64_t* slot_out, float scale, int64_t N, int64_t H, int64_t D) {
  if (N < 0 || H < 1 || num_slots < 1) return KDA_ERR_BAD_SHAPE;
  if (D != 32 && D != 64 && D != 128) return KDA_ERR_BAD_SHAPE;
  // one launch covers at most 2^32 - 1 work-items: N * H workgroups of up to 256 threads
  // (more, smaller ones only while they are few)
  if (H >= ((int64_t)1 << 24) || (N > 0 && N > (((int64_t)1 << 24) - 1) / H))
    return KDA_ERR_BAD_SHAPE;
  if (num_slots > kMaxBytes / (H * D * D * 4)) return KDA_ERR_BAD_SHAPE;
  if (!state_dtype_ok(state_dtype)) return KDA_ERR_BAD_DTYPE;
  if (!std::isfinite(scale)) return KDA_ERR_BAD_SCALE;
  // without slots request n reads (and without slot_out writes) slot n
  if (!slot_in && N > num_slots) return KDA_ERR_BAD_SHAPE;
  if (!state) return KDA_ERR_NULL_ARG;
  if (!aligned16(state)) return KDA_ERR_BAD_LAYOUT;
  return KDA_OK;
}

int step_check(const void* q, const void* k, const void* v, const void* g, const void* beta,
               float scale, const void* out, const float* A_log, const float* dt_bias,
               float lower_bound, const void* state, int state_dtype, int64_t num_slots,
               const int64_t* slot_in, const int64_t* slot_out, int64_t N, int64_t H, int64_t D) {
  const int st = step_resolve(state, state_dtype, num_slots, slot_in, slot_out, scale, N, H, D);
  if (st != KDA_OK) return st;
  if (!A_log || !dt_bias || (N > 0 && (!q || !k || !v || !g || !beta || !out)))
    return KDA_ERR_NULL_ARG;
  if (!std::isfinite(lower_bound) || !(lower_bound < 0.f)) return KDA_ERR_BAD_LOWER_BOUND;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(out))
    return KDA_ERR_BAD_LAYOUT;
  const int64_t act = N * H * D * 2;
  const Range ro = make_range(out, act),
              rp = make_range(state, num_slots * H * D * D * (state_dtype ? 4 : 2));
  const Range ins[] = {make_range(q, act), make_range(k, act), make_range(v, act),
                       make_range(g, act), make_range(beta, N * H * 2), make_range(A_log, H * 4),
                       make_range(dt_bias, H * D * 4), make_range(slot_in, slot_in ? N * 8 : 0),
                       make_range(slot_out, slot_out ? N * 8 : 0)};
  if (any_overlap(ro, ins, 9) || any_overlap(rp, ins, 9) || overlaps(ro, rp))
    return KDA_ERR_BAD_ALIAS;
  return KDA_OK;
}

int la_step_check(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
                  int64_t v_row, const float* g, const float* decay, float scale, const void* out,
                  const void* state, int state_dtype, int64_t num_slots, const int64_t* slot_in,
                  const int64_t* slot_out, int64_t N, int64_t H, int64_t Hk, int64_t D) {
  const int st = step_resolve(state, state_dtype, num_slots, slot_in, slot_out, scale, N, H, D);
  if (st != KDA_OK) return st;
  if (Hk < 1 || H % Hk != 0) return KDA_ERR_BAD_SHAPE;
  if (N > 0 && (!q || !k || !v || !out)) return KDA_ERR_NULL_ARG;
  if (!row_ok(q_row, Hk, D) || !row_ok(k_row, Hk, D) || !row_ok(v_row, H, D) || !aligned16(q) ||
      !aligned16(k) || !aligned16(v) || !aligned16(out))
    return KDA_ERR_BAD_LAYOUT;
  const int64_t bq = span_bytes(N, q_row, Hk, D), bk = span_bytes(N, k_row, Hk, D),
                bv = span_bytes(N, v_row, H, D);
  if (bq < 0 || bk < 0 || bv < 0) return KDA_ERR_BAD_SHAPE;
  const Range ro = make_range(out, N * H * D * 2),
              rp = make_range(state, num_slots * H * D * D * (state_dtype ? 4 : 2));
  const Range ins[] = {make_range(q, bq), make_range(k, bk), make_range(v, bv),
                       make_range(g, g ? N * H * 4 : 0), make_range(decay, decay ? H * 4 : 0),
                       make_range(slot_in, slot_in ? N * 8 : 0),
                       make_range(slot_out, slot_out ? N * 8 : 0)};
  if (any_overlap(ro, ins, 7) || any_overlap(rp, ins, 7) || overlaps(ro, rp))
    return KDA_ERR_BAD_ALIAS;
  return KDA_OK;
}

int status(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

}  // namespace

extern "C" {

int kda_step_check(const void* q, const void* k, const void* v, const void* g, const void* beta,
                   float scale, const void* out, const float* A_log, const float* dt_bias,
                   float lower_bound, const void* state, int state_dtype, int64_t num_slots,
                   const int64_t* slot_in, const int64_t* slot_out, int64_t N, int64_t H,
                   int64_t D) {
  return step_check(q, k, v, g, beta, scale, out, A_log, dt_bias, lower_bound, state, state_dtype,
                    num_slots, slot_in, slot_out, N, H, D);
}

int kda_step(const void* q, const void* k, const void* v, const void* g, const void* beta,
             float scale, void* out, const float* A_log, const float* dt_bias, float lower_bound,
             void* state, int state_dtype, int64_t num_slots, const int64_t* slot_in,
             const int64_t* slot_out, int64_t N, int64_t H, int64_t D, void* stream) {
  const int st = step_check(q, k, v, g, beta, scale, out, A_log, dt_bias, lower_bound, state,
                            state_dtype, num_slots, slot_in, slot_out, N, H, D);
  if (st != KDA_OK || N == 0) return st;
  kda::StepParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.gate = static_cast<const uint16_t*>(g);
  p.beta = static_cast<const uint16_t*>(beta);
  p.A_log = A_log;
  p.dt_bias = dt_bias;
  p.out = static_cast<uint16_t*>(out);
  p.state = state;
  p.slot_in = slot_in;
  p.slot_out = slot_out;
  p.num_slots = num_slots;
  p.q_row = p.k_row = p.v_row = H * D;
  p.N = static_cast<int32_t>(N);
  p.H = static_cast<int32_t>(H);
  p.group = 1;
  p.scale = scale;
  p.lower_bound = lower_bound;
  return status(kda::launch_step(p, true, static_cast<int>(D), state_dtype == KDA_DTYPE_FP32,
                                 static_cast<hipStream_t>(stream)));
}

int kda_la_step_check(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
                      int64_t v_row, const float* g, const float* decay, float scale,
                      const void* out, const void* state, int state_dtype, int64_t num_slots,
                      const int64_t* slot_in, const int64_t* slot_out, int64_t N, int64_t H,
                      int64_t Hk, int64_t D) {
  return la_step_check(q, q_row, k, k_row, v, v_row, g, decay, scale, out, state, state_dtype,
                       num_slots, slot_in, slot_out, N, H, Hk, D);
}

int kda_la_step(const void* q, int64_t q_row, const void* k, int64_t k_row, const void* v,
                int64_t v_row, const float* g, const float* decay, float scale, void* out,
                void* state, int state_dtype, int64_t num_slots, const int64_t* slot_in,
                const int64_t* slot_out, int64_t N, int64_t H, int64_t Hk, int64_t D,
                void* stream) {
  const int st = la_step_check(q, q_row, k, k_row, v, v_row, g, decay, scale, out, state,
                               state_dtype, num_slots, slot_in, slot_out, N, H, Hk, D);
  if (st != KDA_OK || N == 0) return st;
  kda::StepParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.g = g;
  p.decay = decay;
  p.out = static_cast<uint16_t*>(out);
  p.state = state;
  p.slot_in = slot_in;
  p.slot_out = slot_out;
  p.num_slots = num_slots;
  p.q_row = q_row;
  p.k_row = k_row;
  p.v_row = v_row;
  p.N = static_cast<int32_t>(N);
  p.H = static_cast<int32_t>(H);
  p.group = static_cast<int32_t>(H / Hk);
  p.scale = scale;
  return status(kda::launch_step(p, false, static_cast<int>(D), state_dtype == KDA_DTYPE_FP32,
                                 static_cast<hipStream_t>(stream)));
}

}  // extern "C"
