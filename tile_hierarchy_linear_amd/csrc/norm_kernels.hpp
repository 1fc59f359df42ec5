// norm_kernels.hpp -- the kernels of the per-token norms (norm.hip: root mean
// square; layernorm.hip: centred) and of their gradients, and the choice of
// their variants.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/thl.h"
#include "host_checks.hpp"
#include "rows.hpp"

namespace thl {
namespace {

enum : int { Y_FLOAT = 0, Y_FP8 = 1, Y_MX = 2 };

struct NormArgs {
  const void* x;
  const void* r;  // NULL: no residual
  void* s;        // NULL: the sum is not stored
  const void* w;  // centred norm: NULL for ones
  const void* b;  // centred norm: NULL for zeros; w's type
  void* y;
  uint8_t* sf;
  int64_t ldx, ldr, lds, ldy, ld_sf;
  int64_t n;
  int32_t m;
  float eps, inv_scale;
  int32_t x_type, r_type, w_type, y_type, y_mode;
};

// Features e .. e+7 of a token's output (those past m take part in the
// block maximum as zeros and are not stored).  Called by whole groups of
// four consecutive lanes, which hold one MX block.  A block with a NaN has the
// scale NaN and elements of zero; not centred, of 8 bits, elements of NaN under the
// others' scale.  Measured, centred, 16,384 x 4,096 bf16 with residual and its sum:
// to bf16 97 us, to E4M3 87 under one scale and 89 in blocks (93 at a copy's rate), to
// E2M1 102 (87 at a copy's rate: its codes' comparisons take the rest).
template <bool CENTRED>
__device__ __forceinline__ void store_out(const NormArgs& a, int64_t row, int e, const float (&v)[8]) {
  const int valid = a.m - e;
  if (a.y_mode == Y_FLOAT) {
    if (valid > 0) store8_f(a.y, a.y_type, row * a.ldy + e, v, valid < 8 ? valid : 8);
    return;
  }
  uint8_t* y = static_cast<uint8_t*>(a.y);
  if (a.y_mode == Y_FP8) {
    // times the rounded 1 / scale: a quotient next to the midpoint of two codes
    // may take the other one.  Divided instead, 8,192 tokens of 4,096 bf16
    // features take 28.0 us for 23.9, 16,384 of 16,384 to e5m2 226 for 174 (25.5
    // and 187 with the product corrected by its remainder).
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = v[i] * a.inv_scale;
    if (valid > 0) store_codes8(y + row * a.ldy + e, fp8_codes(q, a.y_type == THL_E4M3), valid);
    return;
  }
  // (the maximum that keeps a NaN: two values an instruction)
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < valid) amax = __builtin_elementwise_maximum(amax, __builtin_fabsf(v[i]));
  amax = __builtin_elementwise_maximum(amax, __shfl_xor(amax, 1));
  amax = __builtin_elementwise_maximum(amax, __shfl_xor(amax, 2));
  bool nan = amax != amax;
  if (!CENTRED && a.y_type != THL_E2M1X2 && __ballot(nan) != 0) {
    amax = 0.0f, nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) amax = __builtin_fmaxf(amax, __builtin_fabsf(v[i]));
    amax = __builtin_fmaxf(amax, __shfl_xor(amax, 1));
    amax = __builtin_fmaxf(amax, __shfl_xor(amax, 2));
  }
  if (valid <= 0) return;
  const int emax = a.y_type == THL_E2M1X2 ? 2 : (a.y_type == THL_E4M3 ? 8 : 15);
  const int code = nan ? 255 : mx_scale_code(amax, emax);
  const float inv = __builtin_ldexpf(1.0f, 127 - code);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = v[i] * inv;
  if (a.y_type == THL_E2M1X2) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) w |= e2m1_code(q[i]) << (4 * i);
    store_codes4(y + (row * a.ldy + e) / 2, nan ? 0u : w, valid);
  } else {
    v2u_a1 w = fp8_codes(q, a.y_type == THL_E4M3);
    if (nan) w = v2u_a1{0, 0};
    store_codes8(y + row * a.ldy + e, w, valid);
  }
  if ((e & 31) == 0) a.sf[row * a.ld_sf + (e >> 5)] = static_cast<uint8_t>(code);
}

// Features e .. e+7 of the centred norm's weight and bias (m of them), ones
// and zeros where there is none.
template <int RUNS>
struct Affine {
  RawAny w, b;
  __device__ __forceinline__ void load(const void* pw, const void* pb, int type, int e, int m) {
    if (pw) w = load_any<RUNS>(pw, type, e, m);
    if (pb) b = load_any<RUNS>(pb, type, e, m);
  }
  __device__ __forceinline__ void weight(const void* pw, int type, int e, int m, float (&v)[8]) const {
    if (pw) {
      any_f8<RUNS>(w, type, e, m, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 1.0f;
    }
  }
  __device__ __forceinline__ void bias(const void* pb, int type, int e, int m, float (&v)[8]) const {
    if (pb) {
      any_f8<RUNS>(b, type, e, m, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    }
  }
};

// v - mu for the features that exist, zeros for the others.
template <int RUNS>
__device__ __forceinline__ void centre(float (&v)[8], float mu, int e, int m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (RUNS == RUNS_WHOLE ? e < m : e + i < m) ? v[i] - mu : 0.0f;
}

// XB, RB: bytes of an element of X and of R / S (0: no residual).  CENTRED:
// the layer norm.  CH = 0: any number of features, read twice (centred: three
// times).
template <bool CENTRED, int XB, int RB, int WPR, int CH, int RUNS>
__global__ void __launch_bounds__(WPR * 64) norm_kernel(NormArgs a) {
  constexpr int T = WPR * 64;
  __shared__ float red[2][WPR];
  __shared__ float red_mean[CENTRED ? WPR : 1];
  const int t = static_cast<int>(threadIdx.x), m = a.m;
  const bool x_bf = a.x_type == THL_BF16, r_bf = a.r_type == THL_BF16;
  int parity = 0;

  // x + r of features e .. e+7
  auto add = [&](Raw8<XB>& x, Raw8<RB>& r, int e, float (&v)[8]) {
    settle<XB, RUNS>(x, e, m);
    to_f8<XB>(x, x_bf, v);
    if constexpr (RB != 0) {
      float u[8];
      settle<RB, RUNS>(r, e, m);
      to_f8<RB>(r, r_bf, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += u[i];
    }
  };
  auto store_sum = [&](int64_t row, int e, const float (&v)[8]) {
    if constexpr (RB != 0) {
      if (a.s && e < m) store8_f(a.s, a.r_type, row * a.lds + e, v, m - e < 8 ? m - e : 8);
    }
  };

  if constexpr (CH > 0) {
    RawAny wr[CENTRED ? 1 : CH];
    Affine<RUNS> affine[CENTRED ? CH : 1];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if constexpr (CENTRED)
        affine[c].load(a.w, a.b, a.w_type, 8 * (t + T * c), m);
      else
        wr[c] = load_any<RUNS>(a.w, a.w_type, 8 * (t + T * c), m);
    }
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x, parity ^= 1) {
      Raw8<XB> x[CH];
      Raw8<RB> r[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        x[c] = load_run<XB, RUNS>(a.x, row * a.ldx, 8 * (t + T * c), m);
        r[c] = load_run<RB, RUNS>(a.r, row * a.ldr, 8 * (t + T * c), m);
      }
      float v[CH][8], ss[1] = {0.0f}, mu = 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        add(x[c], r[c], 8 * (t + T * c), v[c]);
        if constexpr (!CENTRED) {
#pragma unroll
          for (int i = 0; i < 8; ++i) ss[0] += v[c][i] * v[c][i];
        }
      }
      if constexpr (CENTRED) {
        // The mean first, then the squares of the differences: nothing cancels
        // where the mean is far from zero.  (S rounds v, not v - mu + mu.)
        float sum[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[0] += v[c][i];
        row_sum<1, WPR>(sum, red_mean);
        mu = sum[0] / static_cast<float>(m);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int e = 8 * (t + T * c);
          store_sum(row, e, v[c]);
          centre<RUNS>(v[c], mu, e, m);
#pragma unroll
          for (int i = 0; i < 8; ++i) ss[0] += v[c][i] * v[c][i];
        }
      }
      // Past this sum every lane has read its run: with ragged runs the last
      // two overlap, and S may be stored over X or R.
      row_sum<1, WPR>(ss, red[parity]);
      const float rho = rsqrtf(ss[0] / static_cast<float>(m) + a.eps);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int e = 8 * (t + T * c);
        float w[8], o[8];
        if constexpr (CENTRED) {
          float b[8];
          affine[c].weight(a.w, a.w_type, e, m, w);
          affine[c].bias(a.b, a.w_type, e, m, b);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = v[c][i] * rho * w[i] + b[i];
        } else {
          store_sum(row, e, v[c]);
          any_f8<RUNS>(wr[c], a.w_type, e, m, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = v[c][i] * rho * w[i];
        }
        store_out<CENTRED>(a, row, e, o);
      }
    }
  } else {
    // S may be X or R, and Y may be X: the second pass reads an element
    // before the same lane overwrites it, and no lane reads another's (whole
    // runs, or element by element in the last one).
    auto run = [&](int64_t row, int e, float (&v)[8]) {
      if (RUNS == RUNS_WHOLE || e + 8 <= m) {
        Raw8<XB> x = load_run<XB, RUNS_WHOLE>(a.x, row * a.ldx, e, m);
        Raw8<RB> r = load_run<RB, RUNS_WHOLE>(a.r, row * a.ldr, e, m);
        to_f8<XB>(x, x_bf, v);
        if constexpr (RB != 0) {
          float u[8];
          to_f8<RB>(r, r_bf, u);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += u[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = 0.0f;
          if (e + i < m) {
            v[i] = load_f(a.x, a.x_type, row * a.ldx + e + i);
            if constexpr (RB != 0) v[i] += load_f(a.r, a.r_type, row * a.ldr + e + i);
          }
        }
      }
    };
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x, parity ^= 1) {
      float ss[1] = {0.0f}, mu = 0.0f;
      if constexpr (CENTRED) {
        float sum[1] = {0.0f};
        for (int e = 8 * t; e < m; e += 8 * T) {
          float v[8];
          run(row, e, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[0] += v[i];
        }
        row_sum<1, WPR>(sum, red_mean);
        mu = sum[0] / static_cast<float>(m);
      }
      for (int e = 8 * t; e < m; e += 8 * T) {
        float v[8];
        run(row, e, v);
        if constexpr (CENTRED) centre<RUNS>(v, mu, e, m);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] += v[i] * v[i];
      }
      row_sum<1, WPR>(ss, red[parity]);
      const float rho = rsqrtf(ss[0] / static_cast<float>(m) + a.eps);
      // whole groups of four lanes stay together for the block maximum
      for (int e = 8 * t; (e & ~31) < m; e += 8 * T) {
        const int valid = m - e;
        float v[8] = {}, w[8] = {}, b[8] = {};
        if constexpr (CENTRED) {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = 1.0f;
        }
        if (valid > 0) {
          run(row, e, v);
          if (!CENTRED || a.w) load8_f(a.w, a.w_type, e, valid < 8 ? valid : 8, w);
          if (CENTRED && a.b) load8_f(a.b, a.w_type, e, valid < 8 ? valid : 8, b);
        }
        store_sum(row, e, v);
        if constexpr (CENTRED) {
          centre<RUNS>(v, mu, e, m);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = v[i] * rho * w[i] + b[i];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = v[i] * rho * w[i];
        }
        store_out<CENTRED>(a, row, e, v);
      }
    }
  }
}

// ---- gradient

struct NormGradArgs {
  const void* s;
  const void* dy;
  const void* dr;  // NULL: none
  const void* w;  // centred norm: NULL for ones
  void* dx;
  float* part;  // partial dw, one row of m floats per workgroup (centred norm: 2 m, then db); NULL: not wanted
  int64_t lds, lddy, lddr, lddx;
  int64_t n;
  int32_t m;
  float eps;
  int32_t s_type, g_type, w_type;
};

// Tokens that one wavefront holds go to a workgroup's wavefronts side by side:
// a quarter of the rows of partial dw for as many wavefronts.
constexpr int tokens_at_once(int wpr) { return wpr == 1 ? 4 : 1; }

// SB, GB: bytes of an element of S and of the gradients.  CH = 0: any number
// of features; dw then accumulates in the workgroup's row of `part`.
// CENTRED: the layer norm's, with db.
template <bool CENTRED, int SB, int GB, int WPR, int CH, int RUNS>
__global__ void __launch_bounds__(WPR * tokens_at_once(WPR) * 64) norm_grad_kernel(NormGradArgs a) {
  constexpr int T = WPR * 64, TOKENS = tokens_at_once(WPR);
  constexpr int NC = CH > 0 ? CH : 1;
  constexpr int NS = CENTRED ? 3 : 2;  // sums of a token: of squares, of t and s, centred of t
  constexpr int NP = CENTRED ? 2 : 1;  // sums over tokens: dw, db
  __shared__ float red[2][NS * WPR];
  __shared__ float red_mean[CENTRED && TOKENS == 1 ? WPR : 1];
  const int t = static_cast<int>(threadIdx.x) % T, m = a.m;
  const int which = TOKENS > 1 ? static_cast<int>(threadIdx.x) / T : 0;
  const bool s_bf = a.s_type == THL_BF16, g_bf = a.g_type == THL_BF16;
  int parity = 0;

  // dx of features e .. e+7 (d: the gradient past the norm), with h = rho * s
  // and mean = mean(w * dy * h); dw's terms of this token in h.  Centred: s
  // less its mean, and level = mean(w * dy).
  auto emit = [&](int64_t row, int e, const float (&s)[8], const float (&g)[8], const float (&w)[8], float (&d)[8],
                  float rho, float mean, float level, float (&h)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[i] = s[i] * rho;
      if constexpr (CENTRED)
        d[i] += rho * (w[i] * g[i] - level - h[i] * mean);
      else
        d[i] += rho * (w[i] * g[i] - h[i] * mean);
      h[i] *= g[i];
    }
    if (e < m) store8_f(a.dx, a.g_type, row * a.lddx + e, d, m - e < 8 ? m - e : 8);
  };

  float* part = a.part ? a.part + static_cast<int64_t>(blockIdx.x) * NP * m : nullptr;
  if constexpr (CH > 0) {
    RawAny wr[NC];
    // dw's sums: of one run a lane in registers, of two in LDS, and the weights
    // in fp32 in registers instead (with dr, and with the second launch: 4,096
    // tokens of 8,192 bf16 features 52 us, 63 with one run a lane on twice the
    // wavefronts; 2,048 of 16,384 58 us, 108 with everything in registers, of
    // which 30 spill)
    constexpr bool IN_LDS = NC > 1;
    float acc[IN_LDS ? 1 : NC][8] = {}, acc_b[CENTRED && !IN_LDS ? NC : 1][8] = {};
    __shared__ __attribute__((aligned(16))) v4f held[IN_LDS ? 2 * NP * NC * T : 1];
    if constexpr (IN_LDS) {
#pragma unroll
      for (int c = 0; c < 2 * NP * NC; ++c) held[c * T + t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const bool has_w = !CENTRED || a.w;
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (has_w) wr[c] = load_any<RUNS>(a.w, a.w_type, 8 * (t + T * c), m);
    float w[NC][8];
    auto weights = [&](int c) {
      if (has_w) {
        any_f8<RUNS>(wr[c], a.w_type, 8 * (t + T * c), m, w[c]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[c][i] = 1.0f;
      }
    };
    if constexpr (IN_LDS) {
#pragma unroll
      for (int c = 0; c < NC; ++c) weights(c);
    }
    // without a gradient past the norm, dy is loaded in its place and not used
    const void* dr = a.dr ? a.dr : a.dy;
    const int64_t lddr = a.dr ? a.lddr : a.lddy;
    const int64_t step = static_cast<int64_t>(gridDim.x) * TOKENS;
    Raw8<SB> sr[NC];
    Raw8<GB> gr[NC], rr[NC];
    auto load_row = [&](int64_t row, Raw8<SB> (&s)[NC], Raw8<GB> (&g)[NC], Raw8<GB> (&r)[NC]) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int e = 8 * (t + T * c);
        s[c] = load_run<SB, RUNS>(a.s, row * a.lds, e, m);
        g[c] = load_run<GB, RUNS>(a.dy, row * a.lddy, e, m);
        r[c] = load_run<GB, RUNS>(dr, row * lddr, e, m);
      }
    };
    // Centred, with a second sum across the workgroup, a token waits long enough
    // to ask for the next one first (the last one asks for itself again): with dr
    // 8,192 x 4,096 bf16 58 us for 66, 16,384 x 2,048 54 for 56 (fp32 108 for 111),
    // x 1,024 31 for 32.  Not on one wavefront, nor fp32 on two, which have others
    // to wait beside: 20,000 x 500 fp32 46 for 37, 16,384 x 1,001 66 for 62.  Nor two
    // runs a lane, whose registers then leave one workgroup a CU: 8,192 x 6,144 bf16
    // 105 for 85, 2,048 x 8,192 fp32 71 for 60.
    constexpr bool AHEAD = CENTRED && NC == 1 && SB + 2 * GB <= 3 * WPR;
    // On sixteen wavefronts two 16-bit runs stay as loaded across the sums and are
    // converted again after each: in fp32 they spill 100 registers.  2,048 x 12,288
    // bf16 58 us for 88, fp32 with bf16 gradients 72 for 85; bf16 with fp32
    // gradients 97 for 89.
    constexpr bool AGAIN = CENTRED && WPR == 16 && GB == 2;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * TOKENS + which;
    Raw8<SB> sn[AHEAD ? NC : 1];
    Raw8<GB> gn[AHEAD ? NC : 1], rn[AHEAD ? NC : 1];
    if constexpr (AHEAD) {
      if (row0 < a.n) load_row(row0, sn, gn, rn);
    }
    for (int64_t row = row0; row < a.n; row += step, parity ^= 1) {
      if constexpr (AHEAD) {
#pragma unroll
        for (int c = 0; c < NC; ++c) sr[c] = sn[c], gr[c] = gn[c], rr[c] = rn[c];
        load_row(row + step < a.n ? row + step : row, sn, gn, rn);
      } else {
        load_row(row, sr, gr, rr);
      }
      float s[NC][8], g[NC][8], sum[NS] = {}, mu = 0.0f;
      if constexpr (CENTRED) {
        float total[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          settle<SB, RUNS>(sr[c], 8 * (t + T * c), m);
          to_f8<SB>(sr[c], s_bf, s[c]);
#pragma unroll
          for (int i = 0; i < 8; ++i) total[0] += s[c][i];
        }
        row_sum<1, WPR>(total, red_mean);
        mu = total[0] / static_cast<float>(m);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          if constexpr (AGAIN) {
            arrived(sr[c]);
            to_f8<SB>(sr[c], s_bf, s[c]);
          }
          centre<RUNS>(s[c], mu, 8 * (t + T * c), m);
        }
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int e = 8 * (t + T * c);
        if constexpr (!CENTRED) settle<SB, RUNS>(sr[c], e, m);
        settle<GB, RUNS>(gr[c], e, m);
        if constexpr (!CENTRED) to_f8<SB>(sr[c], s_bf, s[c]);
        to_f8<GB>(gr[c], g_bf, g[c]);
        if constexpr (!IN_LDS) weights(c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum[0] += s[c][i] * s[c][i];
          sum[1] += w[c][i] * g[c][i] * s[c][i];
          if constexpr (CENTRED) sum[2] += w[c][i] * g[c][i];
        }
        settle<GB, RUNS>(rr[c], e, m);
      }
      // Past these sums every lane has read its runs (dx may be stored over
      // any of them).
      if constexpr (RUNS == RUNS_RAGGED) {
#pragma unroll
        for (int c = 0; c < NC; ++c) arrived(rr[c]);
      }
      row_sum<NS, WPR>(sum, red[parity]);
      const float rho = rsqrtf(sum[0] / static_cast<float>(m) + a.eps);
      const float mean = rho * sum[1] / static_cast<float>(m);
      const float level = CENTRED ? sum[NS - 1] / static_cast<float>(m) : 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float d[8] = {}, h[8];
        if constexpr (AGAIN) {
          arrived(sr[c]), arrived(gr[c]), arrived(rr[c]);
          to_f8<SB>(sr[c], s_bf, s[c]);
          centre<RUNS>(s[c], mu, 8 * (t + T * c), m);
          to_f8<GB>(gr[c], g_bf, g[c]);
        }
        if (a.dr) to_f8<GB>(rr[c], g_bf, d);
        emit(row, 8 * (t + T * c), s[c], g[c], w[c], d, rho, mean, level, h);
        if constexpr (IN_LDS) {
          held[2 * c * T + t] += v4f{h[0], h[1], h[2], h[3]};
          held[(2 * c + 1) * T + t] += v4f{h[4], h[5], h[6], h[7]};
          if constexpr (CENTRED) {
            held[2 * (NC + c) * T + t] += v4f{g[c][0], g[c][1], g[c][2], g[c][3]};
            held[(2 * (NC + c) + 1) * T + t] += v4f{g[c][4], g[c][5], g[c][6], g[c][7]};
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[c][i] += h[i];
          if constexpr (CENTRED) {
#pragma unroll
            for (int i = 0; i < 8; ++i) acc_b[c][i] += g[c][i];
          }
        }
      }
    }
    if (!part) return;
    if constexpr (TOKENS > 1) {  // the wavefronts' sums, in their order
      __shared__ float sums[NP][TOKENS][NC * 8 * 64];
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sums[0][which][8 * (t + T * c) + i] = acc[c][i];
          if constexpr (CENTRED) sums[NP - 1][which][8 * (t + T * c) + i] = acc_b[c][i];
        }
      __syncthreads();
#pragma unroll
      for (int p = 0; p < NP; ++p)
        for (int e = static_cast<int>(threadIdx.x); e < m; e += TOKENS * 64) {
          float v = 0.0f;
#pragma unroll
          for (int w = 0; w < TOKENS; ++w) v += sums[p][w][e];
          part[p * m + e] = v;
        }
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int e = 8 * (t + T * c);
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = IN_LDS ? held[IN_LDS ? (2 * c + i / 4) * T + t : 0][i % 4] : acc[IN_LDS ? 0 : c][i];
        if (e < m) store8_f(part, THL_F32, e, p, m - e < 8 ? m - e : 8);
        if constexpr (CENTRED) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            p[i] = IN_LDS ? held[IN_LDS ? (2 * (NC + c) + i / 4) * T + t : 0][i % 4] : acc_b[IN_LDS ? 0 : c][i];
          if (e < m) store8_f(part, THL_F32, static_cast<int64_t>(m) + e, p, m - e < 8 ? m - e : 8);
        }
      }
    }
  } else {
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x, parity ^= 1) {
      float sum[NS] = {}, mu = 0.0f;
      if constexpr (CENTRED) {
        float total[1] = {0.0f};
        for (int e = 8 * t; e < m; e += 8 * T) {
          float s[8];
          load8_f(a.s, a.s_type, row * a.lds + e, m - e < 8 ? m - e : 8, s);
#pragma unroll
          for (int i = 0; i < 8; ++i) total[0] += s[i];
        }
        row_sum<1, WPR>(total, red_mean);
        mu = total[0] / static_cast<float>(m);
      }
      auto load_w = [&](int e, int k, float (&w)[8]) {
        if (!CENTRED || a.w) {
          load8_f(a.w, a.w_type, e, k, w);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = 1.0f;
        }
      };
      for (int e = 8 * t; e < m; e += 8 * T) {
        const int k = m - e < 8 ? m - e : 8;
        float s[8], g[8], w[8];
        load8_f(a.s, a.s_type, row * a.lds + e, k, s);
        load8_f(a.dy, a.g_type, row * a.lddy + e, k, g);
        load_w(e, k, w);
        if constexpr (CENTRED) centre<RUNS>(s, mu, e, m);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum[0] += s[i] * s[i];
          sum[1] += w[i] * g[i] * s[i];
          if constexpr (CENTRED) sum[2] += w[i] * g[i];
        }
      }
      row_sum<NS, WPR>(sum, red[parity]);
      const float rho = rsqrtf(sum[0] / static_cast<float>(m) + a.eps);
      const float mean = rho * sum[1] / static_cast<float>(m);
      const float level = CENTRED ? sum[NS - 1] / static_cast<float>(m) : 0.0f;
      for (int e = 8 * t; e < m; e += 8 * T) {
        const int k = m - e < 8 ? m - e : 8;
        float s[8], g[8], w[8], d[8] = {}, h[8];
        load8_f(a.s, a.s_type, row * a.lds + e, k, s);
        load8_f(a.dy, a.g_type, row * a.lddy + e, k, g);
        load_w(e, k, w);
        if (a.dr) load8_f(a.dr, a.g_type, row * a.lddr + e, k, d);
        if constexpr (CENTRED) centre<RUNS>(s, mu, e, m);
        emit(row, e, s, g, w, d, rho, mean, level, h);
        if (part) {  // this lane's own features of the workgroup's own row
          float p[8];
          if (row >= gridDim.x) {
            load8_f(part, THL_F32, e, k, p);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] += p[i];
          }
          store8_f(part, THL_F32, e, h, k);
          if constexpr (CENTRED) {
            const int64_t at = static_cast<int64_t>(m) + e;
            if (row >= gridDim.x) {
              load8_f(part, THL_F32, at, k, p);
#pragma unroll
              for (int i = 0; i < 8; ++i) g[i] += p[i];
            }
            store8_f(part, THL_F32, at, g, k);
          }
        }
      }
    }
  }
}

// dw = the sum of `rows` partial rows `pitch` apart, in a fixed order: a
// workgroup adds 32 columns, 32 slices of the rows side by side, then the
// slices.  Workgroups (., 1) add the rows' second m columns to db.
__global__ void __launch_bounds__(1024) norm_grad_reduce(const float* part, int rows, int64_t pitch, int m, void* dw,
                                                         void* db, int dw_type) {
  if (blockIdx.y != 0) dw = db, part += m;
  if (!dw) return;
  __shared__ float slice[32][33];
  const int col = static_cast<int>(threadIdx.x) & 31, sl = static_cast<int>(threadIdx.x) >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + col;
  float t = 0.0f;
  const int64_t cc = c < m ? c : m - 1;
  for (int r = sl; r < rows; r += 8 * 32) {  // eight loads at a time, of rows that exist
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = part[static_cast<int64_t>(r + 32 * i < rows ? r + 32 * i : r) * pitch + cc];
#pragma unroll
    for (int i = 0; i < 8; ++i) t += r + 32 * i < rows ? v[i] : 0.0f;
  }
  slice[sl][col] = t;
  __syncthreads();
  if (sl != 0 || c >= m) return;
  t = 0.0f;
  for (int i = 0; i < 32; ++i) t += slice[i][col];
  if (dw_type == THL_F32)
    static_cast<float*>(dw)[c] = t;
  else if (dw_type == THL_F16)
    static_cast<_Float16*>(dw)[c] = static_cast<_Float16>(t);
  else
    static_cast<__bf16*>(dw)[c] = static_cast<__bf16>(t);
}

// ---- launch

hipError_t launch(const void* f, int64_t grid, int block, void* arg, hipStream_t st) {
  void* args[] = {arg};
  return hipLaunchKernel(f, dim3(static_cast<unsigned>(grid)), dim3(block), args, 0, st);
}

// Workgroups: one per token up to what keeps the device full several times
// over; each then walks its tokens.  Weights and biases, which a workgroup loads
// once, want a quarter as many: with residual and its sum, bf16, 8,192 x 5,003 86 us
// for 106, 4,096 x 12,288 94 for 101, 65,536 x 256 37 for 43, 1,024 x 8,192 19.5 for
// 21.7.  From 1,025 to 4,096 features all are better for the larger half, a
// quarter and all: 16,384 x 4,096 104.6 and 100.5, 20,000 x 3,200 100.9 and 94.4,
// 24,576 x 2,560 103.4 and 97.1 (but 20,000 x 2,501 101.9 and 115.6); for the smaller,
// fp32 (16,384 x 2,048 107.8 and 104.9, 32,768 x 1,280 147.9 and 141.4) and without a
// residual (32,768 x 2,048 bf16 64.2 and 60.9, x 1,280 58.8 and 57.3), where bf16 with
// one has it the other way round (96.0 and 98.3, 77.0 and 81.9).
int64_t norm_grid(bool centred, int64_t m, int64_t n, int wpr) {
  const int64_t most = (centred && (m <= 1024 || m > 4096) ? 8192 : 32768) / wpr;
  return n < most ? n : most;
}

// A token goes to as few wavefronts as hold it at 32 features a lane where
// there are tokens to fill the device, and to as many as hold it at 8 or 16
// where there are not: one token of 8,192 takes 7.4 us on four wavefronts.
template <bool CENTRED, int XB, int RB, int RUNS>
hipError_t launch_norm(NormArgs& a, hipStream_t st) {
#define THL_NORM(WPR, CH)                                                                                            \
  return launch(reinterpret_cast<const void*>(&norm_kernel<CENTRED, XB, RB, WPR, CH, RUNS>),                         \
                norm_grid(CENTRED, a.m, a.n, WPR), WPR * 64, &a, st)
  const bool few = a.n <= 1024;
  if (a.m <= 512) THL_NORM(1, 1);
  if constexpr (RUNS != RUNS_TINY) {
    if (a.m <= 1024) THL_NORM(1, 2);
    if (a.m <= 2048) THL_NORM(4, 1);
    if (few && a.m <= 4096) THL_NORM(8, 1);
    if (few && a.m <= 8192) THL_NORM(16, 1);
    if (a.m <= 4096) THL_NORM(4, 2);
    if (a.m <= 6144) THL_NORM(4, 3);
    if (a.m <= 8192) THL_NORM(4, 4);
    if (a.m <= 16384) THL_NORM(16, 2);
    THL_NORM(16, 0);
  }
  return hipErrorInvalidValue;
#undef THL_NORM
}
template <bool CENTRED, int XB, int RB>
hipError_t launch_norm(NormArgs& a, hipStream_t st) {
  const int runs = runs_of(a.m);
  if (runs == RUNS_TINY) return launch_norm<CENTRED, XB, RB, RUNS_TINY>(a, st);
  return runs == RUNS_WHOLE ? launch_norm<CENTRED, XB, RB, RUNS_WHOLE>(a, st)
                            : launch_norm<CENTRED, XB, RB, RUNS_RAGGED>(a, st);
}

// Workgroups of the gradient, and rows of partial dw: enough to fill the
// device, few enough that the partial rows stay a small part of the traffic.
// Short tokens leave few bytes in flight a workgroup and want more of them:
// 16,384 tokens of 1,024 bf16 features take 33.8 us with 2,048 rows on two
// wavefronts each and 41.5 with 1,024 rows on four.  From 8,193 to 16,384 a
// workgroup fills a compute unit, and 256 are all that run at a time: 2,048
// tokens of 16,384 features (both launches, with dr) take 58 us and 66 with 512
// rows, of 12,288 features 48 and 53.
int64_t grad_rows(int64_t m, int64_t n) {
  const int64_t tokens = m <= 512 ? (n + tokens_at_once(1) - 1) / tokens_at_once(1) : n;
  int64_t most = 512;
  if (m <= 2048 && n >= 4096) most = m <= 1024 ? 2048 : 1024;
  if (m > 8192 && m <= 16384) most = 256;
  return tokens < most ? tokens : most;
}

template <bool CENTRED, int SB, int GB, int RUNS>
hipError_t launch_grad(NormGradArgs& a, int64_t grid, hipStream_t st) {
#define THL_GRAD(WPR, CH) \
  return launch(reinterpret_cast<const void*>(&norm_grad_kernel<CENTRED, SB, GB, WPR, CH, RUNS>), grid, \
                WPR * tokens_at_once(WPR) * 64, &a, st)
  if (a.m <= 512) THL_GRAD(1, 1);
  if constexpr (RUNS != RUNS_TINY) {
    if (a.m <= 1024) THL_GRAD(2, 1);
    if (a.m <= 2048) THL_GRAD(4, 1);
    if (a.m <= 4096) THL_GRAD(8, 1);
    if (a.m <= 8192) THL_GRAD(8, 2);
    if (a.m <= 16384) THL_GRAD(16, 2);
    THL_GRAD(16, 0);
  }
  return hipErrorInvalidValue;
#undef THL_GRAD
}
template <bool CENTRED, int SB, int GB>
hipError_t launch_grad(NormGradArgs& a, int64_t grid, hipStream_t st) {
  const int runs = runs_of(a.m);
  if (runs == RUNS_TINY) return launch_grad<CENTRED, SB, GB, RUNS_TINY>(a, grid, st);
  return runs == RUNS_WHOLE ? launch_grad<CENTRED, SB, GB, RUNS_WHOLE>(a, grid, st)
                            : launch_grad<CENTRED, SB, GB, RUNS_RAGGED>(a, grid, st);
}

template <bool CENTRED>
hipError_t launch_norm(NormArgs& a, hipStream_t st) {
  if (a.x_type == THL_F32) return a.r ? launch_norm<CENTRED, 4, 4>(a, st) : launch_norm<CENTRED, 4, 0>(a, st);
  if (!a.r) return launch_norm<CENTRED, 2, 0>(a, st);
  return a.r_type == THL_F32 ? launch_norm<CENTRED, 2, 4>(a, st) : launch_norm<CENTRED, 2, 2>(a, st);
}
template <bool CENTRED>
hipError_t launch_grad(NormGradArgs& a, int64_t grid, hipStream_t st) {
  if (a.s_type == THL_F32)
    return a.g_type == THL_F32 ? launch_grad<CENTRED, 4, 4>(a, grid, st) : launch_grad<CENTRED, 4, 2>(a, grid, st);
  return a.g_type == THL_F32 ? launch_grad<CENTRED, 2, 4>(a, grid, st) : launch_grad<CENTRED, 2, 2>(a, grid, st);
}

// The gradient's second launch: dw (and db) from `rows` partial rows.
hipError_t launch_grad_reduce(const float* part, int64_t rows, int64_t pitch, int64_t m, void* dw, void* db, int type,
                              hipStream_t st) {
  int r = static_cast<int>(rows), cols = static_cast<int>(m);
  void* args[] = {&part, &r, &pitch, &cols, &dw, &db, &type};
  return hipLaunchKernel(reinterpret_cast<const void*>(&norm_grad_reduce),
                         dim3(static_cast<unsigned>((m + 31) / 32), db ? 2 : 1), dim3(1024), args, 0, st);
}

bool bad_ld(int64_t ld, int64_t m) { return ld < (m > 1 ? m : 1); }
bool big(int64_t v) { return v > INT32_MAX; }
bool misaligned(const void* p, thl_dtype t) { return reinterpret_cast<uintptr_t>(p) % bytes_of(t, 1) != 0; }


}  // namespace
}  // namespace thl
