// Linear attention with one decay per head over prompts (kda_la_fwd), for gfx950.
//
// Per sequence and head, on a V x K state S with log decays lam_t <= 0:
//     S_t = e^{lam_t} S_{t-1} + v_t k_t^T,      out_t = scale S_t q_t
// evaluated in chunks of C = 64 tokens.  With G the inclusive prefix sum of lam in the
// chunk and S the state before it,
//     out_i = scale (e^{G_i} S q_i + sum_{j<=i} e^{G_i - G_j} (q_i . k_j) v_j)
//     S'    = e^{G_C} S + sum_j e^{G_C - G_j} v_j k_j^T.
//
// One workgroup owns one (sequence, head) and walks its chunks; its D / 16 waves hold the
// fp32 state in accumulators, S^T, all D keys by 16 values a wave (lane l: value l%16, four
// keys of each 16-key tile).  The keys are ordered so that two tiles of accumulators pack
// into a matrix operand whose reduction slots are eight consecutive keys, a 16-byte read of
// a q row in LDS: row 4g + i of an even tile is key 8g + i of its 32-key block, and of an
// odd tile key 8g + 4 + i.
//
// Decay weights never exceed one and never come from a difference of long sums.  Inside
// each 16-token tile p is the inclusive prefix of lam and s the sum of what follows, each
// summed directly; across tiles e^{G_i - G_j} = e^{p_i} (whole tiles between) e^{s_j}.
// Only pairs inside one tile take e^{p_i - p_j}, a difference of at most 16 terms.  So an
// underflowing factor belongs to a weight below the fp32 range, and 16 + 16 + 4
// exponentials stand for a row of 64.
//
// Roundings.  Scores times weights, and the state as an operand of S q, are rounded to
// bf16 once each, at most half a bf16 step of each term's absolute value (second parts of
// both cost 11-29% of a large call; small ones have them).  The state itself must not lose bits at each of thousands of chunks:
// its update multiplies k (exact in bf16) by the weighted v in two or three bf16 parts,
// whose sum holds the fp32 product to 2^-17 or 2^-25.
//
// Infinities and NaN of v would reach earlier tokens of their chunk, as zero times them in the
// products.  A wave that finds any in its values of a chunk drops them and sets the outputs
// from their tokens on, and the state, to NaN there.  Looking for them takes 1-2% of a large
// call.
//
// Segments.  One workgroup per (sequence, head) leaves most of the device idle for a few
// long sequences.  Then launches split the tokens: a state-only pass sums every
// segment's own contribution from a zero state (k and v only), an elementwise scan turns
// these into the state before each segment, and the main pass runs all segments at once.
// The state-only pass goes backwards from the segment's end and stops once the decay of
// what it has passed is zero in fp32: all earlier weights are.  Infinities and NaN of the tokens
// it never reads belong in every later state all the same (a zero weight times one is NaN).
// The main pass meets them: a segment whose true end state is not all finite leaves it in its
// place of the workspace, and a fourth launch, a look at one flag per segment otherwise,
// carries it to the outputs and the final state behind.
//
// Measured (D 128, bf16 states): 2 x 1024 tokens of 96 heads 58 us, where loads and stores alone
// take 50; 32,768 tokens of 32 heads 353 us, 3.1 TB/s of q, k, v and out and 4.2 of all that
// the passes move, a copy's rate in their access pattern; 64 prompts of 1-512 tokens, 32
// heads, fp32 states 160 us, 4.1 TB/s, loads and stores alone 136.
#include "api_util.h"
#include "gfx950.h"
#include "ops_params.h"

namespace kda {
namespace {

using namespace dev;

constexpr int C = kLaChunk;
constexpr int RT = C / 16;    // 16-token tiles of a chunk
constexpr int kOnce = 2;      // a buffer access's flags: non-temporal

template <int D>
struct LaCfg {
  static constexpr int NW = D / 16;              // waves, 16 values each
  static constexpr int THREADS = NW * 64;
  static constexpr int KT = D / 16;              // key tiles
  static constexpr int KS = D / 32;              // 32-key steps
  static constexpr int LD = D + 16;              // row stride of the token tiles (bf16)
  static constexpr int LDA = C + 8;              // row stride of the score tile
  static constexpr int TPR = D / 8;              // threads per token row (16 bytes each)
  static constexpr int RPP = THREADS / TPR;      // rows per pass of the workgroup
  static constexpr int PASSES = C / RPP;
};

template <int D, bool STATE_ONLY, bool FINE>
struct alignas(16) LaSmem {
  using F = LaCfg<D>;
  float p[C];       // inclusive prefix of the base-2 log decay inside its 16-token tile
  float ep[C];      // 2^p
  float es[C];      // 2^(sum of what follows in the tile)
  float w[C];       // 2^(sum of what follows in the chunk): weight of a token in the state
  float tile[RT];   // 2^(sum of the tile)
  int from[D];      // first token of the chunk with an infinity or NaN of v, per value
  u16 Q[STATE_ONLY ? 1 : C][F::LD];
  u16 K[C][F::LD];
  u16 V[C][F::LD];
  u16 A[STATE_ONLY ? 1 : C][F::LDA];  // scores; columns in the order of a reduction's slots
  u16 A2[FINE ? C : 1][F::LDA];       // their second parts
};

// One launch unit: which sequence and head, its tokens [t0, t1), its segment.
struct Unit {
  int n, h, hk;
  int64_t t0, t1;
  int64_t slot;  // of this segment
  int nseg, s;
};

__device__ __forceinline__ void seq_bounds(const LaParams& p, int n, int64_t& a, int64_t& b) {
  if (p.cu != nullptr) {
    a = p.cu[n];
    b = p.cu[n + 1];
    a = a < 0 ? 0 : (a > p.T_total ? p.T_total : a);
    b = b < a ? a : (b > p.T_total ? p.T_total : b);
  } else {
    a = (int64_t)n * p.T;
    b = a + p.T;
  }
}

// The heads of one group read the same q and k: blocks go to the eight XCDs round robin,
// so a group's heads sit 8 blocks apart, on one XCD and its L2.  False: no such unit.
__device__ __forceinline__ bool find_unit(const LaParams& p, unsigned block, Unit& u) {
  const unsigned run = 8u * (unsigned)p.group;
  const unsigned c = block / run * 8u + block % 8u, Hk = (unsigned)(p.H / p.group);
  const int64_t item = c / Hk;
  u.hk = (int)(c % Hk);
  u.h = u.hk * p.group + (int)((block / 8) % (unsigned)p.group);
  if (p.seg == 0) {
    if (item >= p.N) return false;
    u.n = (int)item;
    u.nseg = 1;
    u.s = 0;
    u.slot = 0;
    seq_bounds(p, u.n, u.t0, u.t1);
    return true;
  }
  if (item >= p.slots) return false;
  // the last sequence whose first slot is not behind this one (first slots grow strictly)
  int lo = 0, hi = p.N - 1;
  int64_t a, b;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    seq_bounds(p, mid, a, b);
    if (a / p.seg + mid <= item) lo = mid;
    else hi = mid - 1;
  }
  seq_bounds(p, lo, a, b);
  const int64_t s = item - (a / p.seg + lo);
  const int64_t nseg = b > a ? (b - a + p.seg - 1) / p.seg : 1;  // an empty sequence keeps one
  if (s < 0 || s >= nseg) return false;
  u.n = lo;
  u.slot = item;
  u.nseg = (int)nseg;
  u.s = (int)s;
  u.t0 = a + s * p.seg;
  u.t1 = u.t0 + p.seg < b ? u.t0 + p.seg : b;
  return true;
}

// First of the four keys that row 4g + i of key tile kt holds for lane group g.
__device__ __forceinline__ constexpr int key0(int kt, int g) {
  return 32 * (kt >> 1) + 8 * g + 4 * (kt & 1);
}

template <int CTRL>
__device__ __forceinline__ float dpp0(float v) {  // lanes without a source read zero
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL,
                                                               0xf, 0xf, true));
}

// Loads and stores of the state as accumulators: `at` is the element of the lane's value and
// lane group in a [V, K] state.
template <int KT>
__device__ __forceinline__ void state_load(f32x4_t (&S)[KT], const void* src, int64_t at,
                                           int fp32) {
  if (fp32) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
      S[kt] = *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(src) + at + key0(kt, 0));
  } else {
    u32x2_t w[KT];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
      w[kt] = *reinterpret_cast<const u32x2_t*>(static_cast<const u16*>(src) + at + key0(kt, 0));
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
      S[kt] = f32x4_t{bf_lo(w[kt][0]), bf_hi(w[kt][0]), bf_lo(w[kt][1]), bf_hi(w[kt][1])};
  }
}
template <int KT>
__device__ __forceinline__ void state_store(const f32x4_t (&S)[KT], void* dst, int64_t at,
                                            int fp32) {
  if (fp32) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
      *reinterpret_cast<f32x4_t*>(static_cast<float*>(dst) + at + key0(kt, 0)) = S[kt];
  } else {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
      *reinterpret_cast<u32x2_t*>(static_cast<u16*>(dst) + at + key0(kt, 0)) =
          u32x2_t{pack_bf16(S[kt][0], S[kt][1]), pack_bf16(S[kt][2], S[kt][3])};
  }
}

// The part of a pair that its bf16 rounding w leaves, as another bf16 pair.
__device__ __forceinline__ unsigned rest(float lo, float hi, unsigned w) {
  return pack_bf16(lo - bf_lo(w), hi - bf_hi(w));
}

// PARTS: bf16 parts of the weighted v in the state update.  FINE: second parts of the scores
// and of the state operand.
template <int D, bool STATE_ONLY, int PARTS, bool FINE>
__global__ __launch_bounds__(LaCfg<D>::THREADS,
                             (D == 128 || STATE_ONLY ? 4 : D == 64 ? 3 : 2)) void la_kernel(LaParams p) {
  using F = LaCfg<D>;
  __shared__ LaSmem<D, STATE_ONLY, FINE> sm;
  Unit u;
  if (!find_unit(p, blockIdx.x, u)) return;  // uniform per workgroup
  if (STATE_ONLY && u.s == u.nseg - 1) return;  // no segment starts from this one's end

  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t H = p.H;

  // ---- the state before the segment: tile kt holds keys key0(kt, lg) .. +3 of value
  // 16 wave + l16
  f32x4_t S[F::KT];
#pragma unroll
  for (int kt = 0; kt < F::KT; ++kt) S[kt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  float* const wseg = p.ws + (u.slot * H + u.h) * (int64_t)(D * D) + tid * 4;
  const int64_t head = ((int64_t)u.n * H + u.h) * (D * D) + (16 * wave + l16) * D + 8 * lg;
  if constexpr (!STATE_ONLY) {
    if (u.nseg > 1) {
#pragma unroll
      for (int kt = 0; kt < F::KT; ++kt)
        S[kt] = *reinterpret_cast<const f32x4_t*>(wseg + kt * F::THREADS * 4);
    } else if (p.s_in != nullptr) {
      state_load(S, p.s_in, head, p.s_in_fp32);
    }
  }

  // ---- raw chunk loads, one chunk ahead: 16 bytes per thread and pass; rows past the end
  // read zero
  const int lrow = tid / F::TPR, lcol = (tid % F::TPR) * 8;
  u32x4_t rq[F::PASSES], rk[F::PASSES], rv[F::PASSES];
  float rg = 0.f;
  auto fetch = [&](u32x4_t* r, const u16* base, int64_t row, int heads_off, int64_t t, int valid) {
    const uint32_t row_bytes = (uint32_t)row * 2u;  // below 2^25
    const __amdgpu_buffer_rsrc_t rs =
        make_rsrc(base + t * row + heads_off, (uint32_t)(valid - 1) * row_bytes + D * 2u);
#pragma unroll
    for (int i = 0; i < F::PASSES; ++i)
      r[i] = __builtin_bit_cast(
          u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                       rs, (uint32_t)(lrow + i * F::RPP) * row_bytes + lcol * 2u, 0, 0));
  };
  const float dec = p.decay ? p.decay[u.h] : 0.f;
  auto load_q = [&](int64_t t) {
    if constexpr (!STATE_ONLY)
      fetch(rq, p.q, p.q_row, u.hk * D, t, (int)(u.t1 - t < C ? u.t1 - t : C));
  };
  auto load_kv = [&](int64_t t) {
    const int valid = (int)(u.t1 - t < C ? u.t1 - t : C);
    fetch(rk, p.k, p.k_row, u.hk * D, t, valid);
    fetch(rv, p.v, p.v_row, u.h * D, t, valid);
    if (wave == 0 && p.g != nullptr) rg = lane < valid ? p.g[(t + lane) * H + u.h] : 0.f;
  };

  // the main pass goes forwards, the state-only pass backwards
  constexpr int STEP = STATE_ONLY ? -C : C;
  auto inside = [&](int64_t t) { return STATE_ONLY ? t >= u.t0 : t < u.t1; };
  const int64_t first =
      STATE_ONLY && u.t0 < u.t1 ? u.t0 + (u.t1 - u.t0 - 1) / C * C : u.t0;
  if (u.t0 < u.t1) {
    load_q(first);
    load_kv(first);
  }
  // the state's loads end here: their first use inside the loop would make every chunk wait
  // for all loads in flight
#pragma unroll
  for (int kt = 0; kt < F::KT; ++kt) asm volatile("" : "+v"(S[kt]));
  // the outputs of the chunk at t, from LDS: each thread reads the pieces that it will write
  // next
  const uint32_t out_row = (uint32_t)H * D * 2u;
  auto store_out = [&](int64_t t) {
    const int valid = (int)(u.t1 - t < C ? u.t1 - t : C);
    const __amdgpu_buffer_rsrc_t ro =
        make_rsrc(p.out + (t * H + u.h) * D, (uint32_t)(valid - 1) * out_row + D * 2u);
#pragma unroll
    for (int i = 0; i < F::PASSES; ++i) {
      const int r = lrow + i * F::RPP;
      __builtin_amdgcn_raw_buffer_store_b128(*reinterpret_cast<const u32x4_t*>(&sm.Q[r][lcol]), ro,
                                             (uint32_t)r * out_row + lcol * 2u, 0, kOnce);
    }
  };
  float after = 1.f;  // state-only: decay of the chunks passed, which follow this one
  for (int64_t t = first; u.t0 < u.t1 && inside(t); t += STEP) {
    const int valid = (int)(u.t1 - t < C ? u.t1 - t : C);
    lds_barrier();  // the previous chunk's reads are done, its outputs in place
    if constexpr (!STATE_ONLY)
      if (t > first) store_out(t - C);
#pragma unroll
    for (int i = 0; i < F::PASSES; ++i) {
      const int r = lrow + i * F::RPP;
      if constexpr (!STATE_ONLY) *reinterpret_cast<u32x4_t*>(&sm.Q[r][lcol]) = rq[i];
      *reinterpret_cast<u32x4_t*>(&sm.K[r][lcol]) = rk[i];
      *reinterpret_cast<u32x4_t*>(&sm.V[r][lcol]) = rv[i];
    }
    if (wave == 0) {  // lane = token: the chunk's decays
      float lam = rg + dec;
      lam = (lam > 0.f ? 0.f : lam) * kLog2e;
      lam = lam < -126.f ? -126.f : lam;  // 2^-126: zero to every weight; keeps sums finite
      if (lane >= valid) lam = 0.f;
      float pre = lam, suf = dpp0<0x101>(lam);  // row_shl:1, what follows
      pre += dpp0<0x111>(pre);                  // row_shr:1, 2, 4, 8
      pre += dpp0<0x112>(pre);
      pre += dpp0<0x114>(pre);
      pre += dpp0<0x118>(pre);
      suf += dpp0<0x101>(suf);
      suf += dpp0<0x102>(suf);
      suf += dpp0<0x104>(suf);
      suf += dpp0<0x108>(suf);
      const float ep = __builtin_amdgcn_exp2f(pre), es = __builtin_amdgcn_exp2f(suf);
      sm.p[lane] = pre;
      sm.ep[lane] = ep;
      sm.es[lane] = es;
      if (l16 == 15) sm.tile[lg] = ep;
      // weight of a token in the state: the tiles behind its own
      float w = es;
      const float e1 = __shfl(ep, 31), e2 = __shfl(ep, 47), e3 = __shfl(ep, 63);
      if (lg < 3) w *= e3;
      if (lg < 2) w *= e2;
      if (lg < 1) w *= e1;
      sm.w[lane] = w;
    }
    lds_barrier();
    if (inside(t + STEP)) load_kv(t + STEP);

    const float d0 = sm.tile[0], d1 = sm.tile[1], d2 = sm.tile[2], d3 = sm.tile[3];
    float d_all = d0 * d1 * d2 * d3;
    f32x4_t O[RT];
    if constexpr (!STATE_ONLY) {
      // ---- scores: ten 16x16 tiles (i, j <= i) over the waves, the four diagonal ones first,
      // as K Q^T: lane holds token i = l16 and four j
#pragma unroll F::NW <= 4 ? 5 : 1
      for (int x = 0; x < (10 + F::NW - 1) / F::NW; ++x) {
        const int m = wave + x * F::NW;
        if ((x + 1) * F::NW > 10 && m >= 10) break;
        const bool diagonal = F::NW <= 4 ? x < 4 / F::NW : m < 4;  // known for few waves
        const int i = diagonal ? m : m < 5 ? 1 : m < 7 ? 2 : 3,
                  j = diagonal ? m : m - 4 - i * (i - 1) / 2;
        f32x4_t a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < F::KS; ++ks)
          a = mfma(*reinterpret_cast<const u32x4_t*>(&sm.K[16 * j + l16][32 * ks + 8 * lg]),
                   *reinterpret_cast<const u32x4_t*>(&sm.Q[16 * i + l16][32 * ks + 8 * lg]), a);
        const int ti = 16 * i + l16, tj = 16 * j + 4 * lg;
        if (diagonal) {
          const float pi = sm.p[ti];
          const f32x4_t pj = *reinterpret_cast<const f32x4_t*>(&sm.p[tj]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float f = __builtin_amdgcn_exp2f(pi - pj[r]);
            a[r] = tj + r <= ti ? a[r] * f : 0.f;
          }
        } else {
          const float t1 = sm.tile[(j + 1) % RT], t2 = sm.tile[(j + 2) % RT];
          const float f = sm.ep[ti] * (i - j > 1 ? t1 : 1.f) * (i - j > 2 ? t2 : 1.f);
          const f32x4_t ej = *reinterpret_cast<const f32x4_t*>(&sm.es[tj]);
#pragma unroll
          for (int r = 0; r < 4; ++r) a[r] *= f * ej[r];
        }
        const u32x2_t w = {pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3])};
        const int col = 32 * (j >> 1) + 8 * lg + 4 * (j & 1);
        *reinterpret_cast<u32x2_t*>(&sm.A[ti][col]) = w;
        if constexpr (FINE)
          *reinterpret_cast<u32x2_t*>(&sm.A2[ti][col]) =
              u32x2_t{rest(a[0], a[1], w[0]), rest(a[2], a[3], w[1])};
      }
      // ---- the state's part: O^T = S Q^T, lane holds token l16 and four values
#pragma unroll
      for (int i = 0; i < RT; ++i) O[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < F::KS; ++ks) {
        const f32x4_t x = S[2 * ks], y = S[2 * ks + 1];
        const u32x4_t s_op = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                              pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
        u32x4_t s2;
        if constexpr (FINE)
          s2 = u32x4_t{rest(x[0], x[1], s_op[0]), rest(x[2], x[3], s_op[1]),
                       rest(y[0], y[1], s_op[2]), rest(y[2], y[3], s_op[3])};
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const u32x4_t q = *reinterpret_cast<const u32x4_t*>(&sm.Q[16 * i + l16][32 * ks + 8 * lg]);
          if constexpr (FINE) O[i] = mfma(s2, q, O[i]);
          O[i] = mfma(s_op, q, O[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        float f = sm.ep[16 * i + l16];
        if (i > 0) f *= d0;
        if (i > 1) f *= d1;
        if (i > 2) f *= d2;
        O[i] *= f;
      }
      lds_barrier();  // the scores are written
      // the loads of a chunk keep the address unit busy for 800 cycles, which its waves would
      // wait for if they were all asked for at once (8% of a call with a workgroup per unit)
      if (inside(t + STEP)) load_q(t + STEP);
    }

    // ---- V^T, from transposed reads: rows are values, slots tokens 32 b + 4g + i and
    // 32 b + 16 + 4g + i
    const int tr = 4 * lg + (l16 >> 2);
    u32x4_t vt[C / 32];
    auto read_v = [&]() {
#pragma unroll
      for (int b = 0; b < C / 32; ++b) {
        const int c = 16 * wave + 4 * (l16 & 3);
        const u32x2_t lo = ds_read_tr(&sm.V[32 * b + tr][c]),
                      hi = ds_read_tr(&sm.V[32 * b + tr + 16][c]);
        vt[b] = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
      }
    };
    read_v();
    bool odd = false;
    if constexpr (!STATE_ONLY) {
      float zero = 0.f;
#pragma unroll
      for (int b = 0; b < C / 32; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) zero = dot_zero(vt[b][e], zero);
      odd = __any(zero != zero);
      if (odd) {  // a wave's own values: nobody else reads them
        const int c = 16 * wave + l16;
        if (lg == 0) {
          int from = C;
#pragma unroll 1
          for (int j = C - 1; j >= 0; --j)
            if ((sm.V[j][c] & 0x7f80u) == 0x7f80u) {
              sm.V[j][c] = 0;
              from = j;
            }
          sm.from[c] = from;
        }
        asm volatile("" ::: "memory");  // a wave's LDS accesses stay in order
        read_v();
      }
    }
    if constexpr (!STATE_ONLY) {
      // ---- the chunk's own part of the output; the columns behind the diagonal tile are not
      // written in the first row tile of each 32: slots 4-7 zero
#pragma unroll
      for (int b = 0; b < C / 32; ++b)
#pragma unroll
        for (int i = 2 * b; i < RT; ++i) {
          u32x4_t a = *reinterpret_cast<const u32x4_t*>(&sm.A[16 * i + l16][32 * b + 8 * lg]);
          if (i == 2 * b) a = u32x4_t{a[0], a[1], 0u, 0u};
          if constexpr (FINE) {
            u32x4_t a2 = *reinterpret_cast<const u32x4_t*>(&sm.A2[16 * i + l16][32 * b + 8 * lg]);
            if (i == 2 * b) a2 = u32x4_t{a2[0], a2[1], 0u, 0u};
            O[i] = mfma(vt[b], a2, O[i]);
          }
          O[i] = mfma(vt[b], a, O[i]);
        }
      // into the place of Q, whose reads are done: whole rows leave with the next chunk
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const f32x4_t o = O[i] * p.scale;
        *reinterpret_cast<u32x2_t*>(&sm.Q[16 * i + l16][16 * wave + 4 * lg]) =
            u32x2_t{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
      }
      if (odd) {
#pragma unroll 1
        for (int r = 0; r < 4; ++r) {
          const int c = 16 * wave + 4 * lg + r, from = sm.from[c];
#pragma unroll 1
          for (int i = l16; i < C; i += 16)
            if (i >= from) sm.Q[i][c] = 0x7fc0u;
        }
        if (sm.from[16 * wave + l16] < C) d_all = __builtin_nanf("");
      }
      // the output's registers are free from here: the compiler does not mix the phases, and
      // two workgroups of eight waves stay on a compute unit (128 registers)
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int kt = 0; kt < F::KT; ++kt) S[kt] *= d_all;
    }
    // ---- the state update
#pragma unroll
    for (int b = 0; b < C / 32; ++b) {
      f32x4_t wa = *reinterpret_cast<const f32x4_t*>(&sm.w[32 * b + 4 * lg]);
      f32x4_t wb = *reinterpret_cast<const f32x4_t*>(&sm.w[32 * b + 16 + 4 * lg]);
      if constexpr (STATE_ONLY) {
        wa *= after;
        wb *= after;
      }
      u32x4_t w[PARTS];  // weight times v
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = bf_lo(vt[b][e]) * (e < 2 ? wa[2 * e] : wb[2 * e - 4]);
        float y = bf_hi(vt[b][e]) * (e < 2 ? wa[2 * e + 1] : wb[2 * e - 3]);
#pragma unroll
        for (int m = 0; m < PARTS; ++m) {
          w[m][e] = pack_bf16(x, y);
          x -= bf_lo(w[m][e]);
          y -= bf_hi(w[m][e]);
        }
      }
#pragma unroll
      for (int kt = 0; kt < F::KT; ++kt) {
        const int c = key0(kt, l16 & 3);
        const u32x2_t lo = ds_read_tr(&sm.K[32 * b + tr][c]),
                      hi = ds_read_tr(&sm.K[32 * b + tr + 16][c]);
        const u32x4_t kop = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
        for (int m = PARTS - 1; m >= 0; --m) S[kt] = mfma(kop, w[m], S[kt]);
      }
    }
    if constexpr (STATE_ONLY) {
      after *= d_all;
      if (__builtin_amdgcn_readfirstlane(after == 0.f)) break;  // the same in every lane
    }
  }

  if constexpr (!STATE_ONLY)
    if (u.t0 < u.t1) {
      lds_barrier();
      store_out(u.t0 + (u.t1 - u.t0 - 1) / C * C);
    }
  if constexpr (STATE_ONLY) {
#pragma unroll
    for (int kt = 0; kt < F::KT; ++kt)
      *reinterpret_cast<f32x4_t*>(wseg + kt * F::THREADS * 4) = S[kt];
    if (tid == 0) p.ws_decay[u.slot * H + u.h] = after;
  } else {
    const bool inner = u.s < u.nseg - 1;
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));  // addresses are formed anew, not kept through the loop
    if (inner) {
      // whether the state behind this segment is all finite, for la_carry_kernel; the scan is
      // done with the segment's place and decay
      float zero = 0.f;
#pragma unroll
      for (int kt = 0; kt < F::KT; ++kt)
#pragma unroll
        for (int i = 0; i < 4; ++i) zero = fmaf(S[kt][i], 0.f, zero);
      const bool odd = __any(zero != zero);
      if ((t & 63) == 0) sm.from[t >> 6] = odd;  // behind the barrier above nobody reads sm.from
      lds_barrier();
      int any = 0;
#pragma unroll
      for (int w = 0; w < F::NW; ++w) any |= sm.from[w];
      if (t == 0) p.ws_decay[u.slot * H + u.h] = any ? 1.f : 0.f;
      if (!any) return;
    } else if (p.s_out == nullptr) {
      return;
    }
    const int64_t at = inner ? u.slot * H + u.h : (int64_t)u.n * H + u.h;
    const int row = 16 * (t >> 6) + (t & 15), key = 8 * (t >> 4 & 3);
    state_store(S, inner ? p.ws : p.s_out, at * (D * D) + row * D + key, inner ? 1 : p.s_out_fp32);
  }
}

// Turns the segments' own sums into the state before each segment, in place: four
// consecutive floats of one head's accumulator image per thread, segments in order.  Also
// reads the initial state, so that the main pass never does when it runs in segments and
// final_state may be the same buffer.
template <int D>
__global__ __launch_bounds__(256) void la_scan_kernel(LaParams p) {
  using F = LaCfg<D>;
  constexpr int QUADS = D * D / 4, BLOCKS = (QUADS + 255) / 256;
  const int64_t unit = blockIdx.x / BLOCKS;
  const int n = (int)(unit / p.H), h = (int)(unit % p.H);
  const int e = (int)(blockIdx.x % BLOCKS) * 256 + threadIdx.x;
  int64_t a, b;
  seq_bounds(p, n, a, b);
  const int nseg = (int)((b - a + p.seg - 1) / p.seg);
  if (nseg <= 1 || e >= QUADS) return;
  const int64_t slot = a / p.seg + n;
  f32x4_t S = {0.f, 0.f, 0.f, 0.f};
  if (p.s_in != nullptr) {
    const int tid = e % F::THREADS, kt = e / F::THREADS;
    f32x4_t one[1];
    state_load(one, p.s_in,
               ((int64_t)n * p.H + h) * (D * D) + (16 * (tid >> 6) + (tid & 15)) * D +
                   key0(kt, (tid & 63) >> 4),
               p.s_in_fp32);
    S = one[0];
  }
  const int64_t step = (int64_t)p.H * (D * D);
  float* w = p.ws + (slot * p.H + h) * (int64_t)(D * D) + e * 4;
  const float* d = p.ws_decay + slot * p.H + h;
  for (int s = 0; s < nseg - 1; ++s) {
    const f32x4_t own = *reinterpret_cast<const f32x4_t*>(w);
    *reinterpret_cast<f32x4_t*>(w) = S;
    S = S * d[(int64_t)s * p.H] + own;
    w += step;
  }
  *reinterpret_cast<f32x4_t*>(w) = S;
}

// Carries what is not finite in the state behind a segment to the outputs of the segments after
// it, a value's from each of its keys, and to the final state.  One workgroup per (sequence,
// head), its lanes as in la_kernel; without a flag it leaves.
template <int D>
__global__ __launch_bounds__(LaCfg<D>::THREADS) void la_carry_kernel(LaParams p) {
  using F = LaCfg<D>;
  const int64_t H = p.H;
  const int n = (int)(blockIdx.x / (unsigned)p.H), h = (int)(blockIdx.x % (unsigned)p.H);
  int64_t a, b;
  seq_bounds(p, n, a, b);
  const int nseg = (int)((b - a + p.seg - 1) / p.seg);
  const int64_t slot = a / p.seg + n;
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, lg = lane >> 4, wave = tid >> 6;
  const int at = (16 * wave + l16) * D + 8 * lg;  // the lane's first element of a state
  const float* flags = p.ws_decay + slot * H + h;
  uint32_t bad = 0;    // bit 4 kt + i: element i of the lane's tile kt
  int from = nseg;     // the first segment that its value's outputs are spoilt in
  for (int s0 = 0; s0 < nseg - 1; s0 += 64) {
    const bool flag = s0 + lane < nseg - 1 && flags[(int64_t)(s0 + lane) * H] != 0.f;
    for (uint64_t left = __ballot(flag); left != 0; left &= left - 1) {
      const int s = s0 + __builtin_ctzll(left);
      const float* w = p.ws + ((slot + s) * H + h) * (int64_t)(D * D) + at;
#pragma unroll
      for (int kt = 0; kt < F::KT; ++kt) {
        const f32x4_t x = *reinterpret_cast<const f32x4_t*>(w + key0(kt, 0));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!(fabsf(x[i]) < __builtin_inff())) bad |= 1u << (4 * kt + i);
      }
      const uint64_t value = __ballot(bad != 0) >> l16 & 0x0001000100010001ull;
      if (value != 0 && from == nseg) from = s + 1;
    }
  }
  u16* out = p.out + h * D + 16 * wave + l16;
  if (from < nseg)
    for (int64_t t = a + (int64_t)from * p.seg + lg; t < b; t += 4) out[t * H * D] = 0x7fc0u;
  if (bad != 0 && p.s_out != nullptr) {
    const int64_t head = ((int64_t)n * H + h) * (D * D) + at;
#pragma unroll
    for (int kt = 0; kt < F::KT; ++kt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (bad >> (4 * kt + i) & 1u) {
          if (p.s_out_fp32)
            static_cast<float*>(p.s_out)[head + key0(kt, 0) + i] = __builtin_nanf("");
          else
            static_cast<u16*>(p.s_out)[head + key0(kt, 0) + i] = 0x7fc0u;
        }
  }
}

template <int D, int PARTS, bool FINE>
hipError_t go(const LaParams& p, hipStream_t stream) {
  using F = LaCfg<D>;
  const int64_t run = 8 * (int64_t)p.group;
  const int64_t items = p.seg ? p.slots : p.N;
  const int64_t blocks = (items * (p.H / p.group) + 7) / 8 * run;
  if (p.seg) {
    la_kernel<D, true, PARTS, false><<<dim3((unsigned)blocks), F::THREADS, 0, stream>>>(p);
    constexpr int BLOCKS = (D * D / 4 + 255) / 256;
    la_scan_kernel<D><<<dim3((unsigned)((int64_t)p.N * p.H * BLOCKS)), 256, 0, stream>>>(p);
  }
  la_kernel<D, false, PARTS, FINE><<<dim3((unsigned)blocks), F::THREADS, 0, stream>>>(p);
  if (p.seg)
    la_carry_kernel<D><<<dim3((unsigned)((int64_t)p.N * p.H)), F::THREADS, 0, stream>>>(p);
  return hipGetLastError();
}

// An fp32 final state keeps three parts; where none leaves, or one rounded to bf16, two
// parts hold it to 2^-17 and save a third of the update's products.
// Calls of few outputs take every second part.  It costs them 0.8 to 2.4 us (128 tokens of 2
// heads, D 32: 7.0 and 7.8 us; 512 tokens of 4 heads, D 128: 24.0 and 26.4), as it would a
// little beyond the limit (8 heads: 24.9 and 27.2), and large calls in proportion (2 x 1024
// tokens of 96 heads 58.8 and 75.7 us; 64 short prompts of 32 heads 161 and 178): the limit is
// a choice between accuracy and time, and stands in the operator's description.
template <int D>
hipError_t by_parts(const LaParams& p, hipStream_t stream) {
  if (p.T_total * p.H <= 2048) return go<D, 3, true>(p, stream);
  return p.s_out != nullptr && p.s_out_fp32 ? go<D, 3, false>(p, stream)
                                             : go<D, 2, false>(p, stream);
}

}  // namespace

hipError_t launch_la(const LaParams& p, int D, hipStream_t stream) {
  return D == 32   ? by_parts<32>(p, stream)
         : D == 64 ? by_parts<64>(p, stream)
                   : by_parts<128>(p, stream);
}

}  // namespace kda
