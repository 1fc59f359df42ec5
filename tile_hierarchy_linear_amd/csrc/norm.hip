// norm.hip -- the root-mean-square norm of each token, with the residual's
// addition before it and its output in 32, 16, 8 or 4 bits, and its gradient.
//
//   s = x + r,   rho = 1 / sqrt(mean(s^2) + eps),   y_i = q(s_i * rho * w_i)
//
// with q the rounding to Y's format: a float type, fp8 under one scale for
// the tensor, or MX blocks of 32 consecutive features (the operand formats of
// the matrix products, with the scales in the layout they read).
//
// Gradient: with h = rho * s and t = w * dy,
//   dx = rho * (t - h * mean(t * h)) + dr,   dw = sum over tokens of dy * h.
//
// Both are bound by HBM: every input is read once and every output written
// once.  One token is held in registers by WPR wavefronts, 8 CH features a
// lane, so the values that the sum of squares needs are still there when the
// outputs are formed.  Only tokens of more than 16,384 features are read
// twice (the second time from L2).
//
// Measured on bf16: the norm of 16,384 tokens of 8,192 features with residual
// 187 us (5.7 TB/s; a large copy runs at 5.0), of one token 4.4 us (a launch
// alone takes 3.9); the gradient of 8,192 tokens of 4,096 features 52.8 us
// (5.1 TB/s).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

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
  const void* w;
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
// four consecutive lanes, which hold one MX block.
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
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < valid) amax = __builtin_fmaxf(amax, __builtin_fabsf(v[i]));
  amax = __builtin_fmaxf(amax, __shfl_xor(amax, 1));
  amax = __builtin_fmaxf(amax, __shfl_xor(amax, 2));
  if (valid <= 0) return;
  const int emax = a.y_type == THL_E2M1X2 ? 2 : (a.y_type == THL_E4M3 ? 8 : 15);
  const int code = mx_scale_code(amax, emax);
  const float inv = __builtin_ldexpf(1.0f, 127 - code);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = v[i] * inv;
  if (a.y_type == THL_E2M1X2) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) w |= e2m1_code(q[i]) << (4 * i);
    store_codes4(y + (row * a.ldy + e) / 2, w, valid);
  } else {
    store_codes8(y + row * a.ldy + e, fp8_codes(q, a.y_type == THL_E4M3), valid);
  }
  if ((e & 31) == 0) a.sf[row * a.ld_sf + (e >> 5)] = static_cast<uint8_t>(code);
}

// XB, RB: bytes of an element of X and of R / S (0: no residual).  CH = 0:
// any number of features, read twice.
template <int XB, int RB, int WPR, int CH, int RUNS>
__global__ void __launch_bounds__(WPR * 64) rmsnorm_kernel(NormArgs a) {
  constexpr int T = WPR * 64;
  __shared__ float red[2][WPR];
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
    RawAny wr[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) wr[c] = load_any<RUNS>(a.w, a.w_type, 8 * (t + T * c), m);
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x, parity ^= 1) {
      Raw8<XB> x[CH];
      Raw8<RB> r[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        x[c] = load_run<XB, RUNS>(a.x, row * a.ldx, 8 * (t + T * c), m);
        r[c] = load_run<RB, RUNS>(a.r, row * a.ldr, 8 * (t + T * c), m);
      }
      float v[CH][8], ss[1] = {0.0f};
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        add(x[c], r[c], 8 * (t + T * c), v[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] += v[c][i] * v[c][i];
      }
      // Past this sum every lane has read its run: with ragged runs the last
      // two overlap, and S may be stored over X or R.
      row_sum<1, WPR>(ss, red[parity]);
      const float rho = rsqrtf(ss[0] / static_cast<float>(m) + a.eps);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int e = 8 * (t + T * c);
        store_sum(row, e, v[c]);
        float w[8], o[8];
        any_f8<RUNS>(wr[c], a.w_type, e, m, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = v[c][i] * rho * w[i];
        store_out(a, row, e, o);
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
      float ss[1] = {0.0f};
      for (int e = 8 * t; e < m; e += 8 * T) {
        float v[8];
        run(row, e, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] += v[i] * v[i];
      }
      row_sum<1, WPR>(ss, red[parity]);
      const float rho = rsqrtf(ss[0] / static_cast<float>(m) + a.eps);
      // whole groups of four lanes stay together for the block maximum
      for (int e = 8 * t; (e & ~31) < m; e += 8 * T) {
        const int valid = m - e;
        float v[8] = {}, w[8] = {};
        if (valid > 0) {
          run(row, e, v);
          load8_f(a.w, a.w_type, e, valid < 8 ? valid : 8, w);
        }
        store_sum(row, e, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * rho * w[i];
        store_out(a, row, e, v);
      }
    }
  }
}

// ---- gradient

struct NormGradArgs {
  const void* s;
  const void* dy;
  const void* dr;  // NULL: none
  const void* w;
  void* dx;
  float* part;  // partial dw, one row of m floats per workgroup; NULL: dw is not wanted
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
template <int SB, int GB, int WPR, int CH, int RUNS>
__global__ void __launch_bounds__(WPR * tokens_at_once(WPR) * 64) rmsnorm_grad_kernel(NormGradArgs a) {
  constexpr int T = WPR * 64, TOKENS = tokens_at_once(WPR);
  constexpr int NC = CH > 0 ? CH : 1;
  __shared__ float red[2][2 * WPR];
  const int t = static_cast<int>(threadIdx.x) % T, m = a.m;
  const int which = TOKENS > 1 ? static_cast<int>(threadIdx.x) / T : 0;
  const bool s_bf = a.s_type == THL_BF16, g_bf = a.g_type == THL_BF16;
  int parity = 0;

  // dx of features e .. e+7 (d: the gradient past the norm), with h = rho * s
  // and mean = mean(w * dy * h); dw's terms of this token in h
  auto emit = [&](int64_t row, int e, const float (&s)[8], const float (&g)[8], const float (&w)[8], float (&d)[8],
                  float rho, float mean, float (&h)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[i] = s[i] * rho;
      d[i] += rho * (w[i] * g[i] - h[i] * mean);
      h[i] *= g[i];
    }
    if (e < m) store8_f(a.dx, a.g_type, row * a.lddx + e, d, m - e < 8 ? m - e : 8);
  };

  float* part = a.part ? a.part + static_cast<int64_t>(blockIdx.x) * m : nullptr;
  if constexpr (CH > 0) {
    RawAny wr[NC];
    // dw's sums: of one run a lane in registers, of two in LDS, and the weights
    // in fp32 in registers instead (with dr, and with the second launch: 4,096
    // tokens of 8,192 bf16 features 52 us, 63 with one run a lane on twice the
    // wavefronts; 2,048 of 16,384 58 us, 108 with everything in registers, of
    // which 30 spill)
    constexpr bool IN_LDS = NC > 1;
    float acc[IN_LDS ? 1 : NC][8] = {};
    __shared__ __attribute__((aligned(16))) v4f held[IN_LDS ? 2 * NC * T : 1];
    if constexpr (IN_LDS) {
#pragma unroll
      for (int c = 0; c < 2 * NC; ++c) held[c * T + t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) wr[c] = load_any<RUNS>(a.w, a.w_type, 8 * (t + T * c), m);
    float w[NC][8];
    if constexpr (IN_LDS) {
#pragma unroll
      for (int c = 0; c < NC; ++c) any_f8<RUNS>(wr[c], a.w_type, 8 * (t + T * c), m, w[c]);
    }
    // without a gradient past the norm, dy is loaded in its place and not used
    const void* dr = a.dr ? a.dr : a.dy;
    const int64_t lddr = a.dr ? a.lddr : a.lddy;
    const int64_t step = static_cast<int64_t>(gridDim.x) * TOKENS;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * TOKENS + which; row < a.n; row += step, parity ^= 1) {
      Raw8<SB> sr[NC];
      Raw8<GB> gr[NC], rr[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int e = 8 * (t + T * c);
        sr[c] = load_run<SB, RUNS>(a.s, row * a.lds, e, m);
        gr[c] = load_run<GB, RUNS>(a.dy, row * a.lddy, e, m);
        rr[c] = load_run<GB, RUNS>(dr, row * lddr, e, m);
      }
      float s[NC][8], g[NC][8], sum[2] = {0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int e = 8 * (t + T * c);
        settle<SB, RUNS>(sr[c], e, m);
        settle<GB, RUNS>(gr[c], e, m);
        to_f8<SB>(sr[c], s_bf, s[c]);
        to_f8<GB>(gr[c], g_bf, g[c]);
        if constexpr (!IN_LDS) any_f8<RUNS>(wr[c], a.w_type, e, m, w[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum[0] += s[c][i] * s[c][i];
          sum[1] += w[c][i] * g[c][i] * s[c][i];
        }
        settle<GB, RUNS>(rr[c], e, m);
      }
      // Past these sums every lane has read its runs (dx may be stored over
      // any of them).
      if constexpr (RUNS == RUNS_RAGGED) {
#pragma unroll
        for (int c = 0; c < NC; ++c) arrived(rr[c]);
      }
      row_sum<2, WPR>(sum, red[parity]);
      const float rho = rsqrtf(sum[0] / static_cast<float>(m) + a.eps);
      const float mean = rho * sum[1] / static_cast<float>(m);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float d[8] = {}, h[8];
        if (a.dr) to_f8<GB>(rr[c], g_bf, d);
        emit(row, 8 * (t + T * c), s[c], g[c], w[c], d, rho, mean, h);
        if constexpr (IN_LDS) {
          held[2 * c * T + t] += v4f{h[0], h[1], h[2], h[3]};
          held[(2 * c + 1) * T + t] += v4f{h[4], h[5], h[6], h[7]};
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[c][i] += h[i];
        }
      }
    }
    if (!part) return;
    if constexpr (TOKENS > 1) {  // the wavefronts' sums, in their order
      __shared__ float sums[TOKENS][NC * 8 * 64];
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[which][8 * (t + T * c) + i] = acc[c][i];
      __syncthreads();
      for (int e = static_cast<int>(threadIdx.x); e < m; e += TOKENS * 64) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < TOKENS; ++w) v += sums[w][e];
        part[e] = v;
      }
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int e = 8 * (t + T * c);
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = IN_LDS ? held[IN_LDS ? (2 * c + i / 4) * T + t : 0][i % 4] : acc[IN_LDS ? 0 : c][i];
        if (e < m) store8_f(part, THL_F32, e, p, m - e < 8 ? m - e : 8);
      }
    }
  } else {
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x, parity ^= 1) {
      float sum[2] = {0.0f, 0.0f};
      for (int e = 8 * t; e < m; e += 8 * T) {
        const int k = m - e < 8 ? m - e : 8;
        float s[8], g[8], w[8];
        load8_f(a.s, a.s_type, row * a.lds + e, k, s);
        load8_f(a.dy, a.g_type, row * a.lddy + e, k, g);
        load8_f(a.w, a.w_type, e, k, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum[0] += s[i] * s[i];
          sum[1] += w[i] * g[i] * s[i];
        }
      }
      row_sum<2, WPR>(sum, red[parity]);
      const float rho = rsqrtf(sum[0] / static_cast<float>(m) + a.eps);
      const float mean = rho * sum[1] / static_cast<float>(m);
      for (int e = 8 * t; e < m; e += 8 * T) {
        const int k = m - e < 8 ? m - e : 8;
        float s[8], g[8], w[8], d[8] = {}, h[8];
        load8_f(a.s, a.s_type, row * a.lds + e, k, s);
        load8_f(a.dy, a.g_type, row * a.lddy + e, k, g);
        load8_f(a.w, a.w_type, e, k, w);
        if (a.dr) load8_f(a.dr, a.g_type, row * a.lddr + e, k, d);
        emit(row, e, s, g, w, d, rho, mean, h);
        if (part) {  // this lane's own features of the workgroup's own row
          float p[8];
          if (row >= gridDim.x) {
            load8_f(part, THL_F32, e, k, p);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] += p[i];
          }
          store8_f(part, THL_F32, e, h, k);
        }
      }
    }
  }
}

// dw = the sum of `rows` partial rows, in a fixed order: a workgroup adds 32
// columns, 32 slices of the rows side by side, then the slices.
__global__ void __launch_bounds__(1024) rmsnorm_grad_reduce(const float* part, int rows, int m, void* dw,
                                                            int dw_type) {
  __shared__ float slice[32][33];
  const int col = static_cast<int>(threadIdx.x) & 31, sl = static_cast<int>(threadIdx.x) >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + col;
  float t = 0.0f;
  const int64_t cc = c < m ? c : m - 1;
  for (int r = sl; r < rows; r += 8 * 32) {  // eight loads at a time, of rows that exist
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = part[static_cast<int64_t>(r + 32 * i < rows ? r + 32 * i : r) * m + cc];
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
// over; each then walks its tokens.
int64_t norm_grid(int64_t n, int wpr) {
  const int64_t most = 32768 / wpr;
  return n < most ? n : most;
}

// A token goes to as few wavefronts as hold it at 32 features a lane where
// there are tokens to fill the device, and to as many as hold it at 8 or 16
// where there are not: one token of 8,192 takes 7.4 us on four wavefronts.
template <int XB, int RB, int RUNS>
hipError_t launch_norm(NormArgs& a, hipStream_t st) {
#define THL_NORM(WPR, CH)                                                                                            \
  return launch(reinterpret_cast<const void*>(&rmsnorm_kernel<XB, RB, WPR, CH, RUNS>), norm_grid(a.n, WPR), WPR * 64, \
                &a, st)
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
template <int XB, int RB>
hipError_t launch_norm(NormArgs& a, hipStream_t st) {
  const int runs = runs_of(a.m);
  if (runs == RUNS_TINY) return launch_norm<XB, RB, RUNS_TINY>(a, st);
  return runs == RUNS_WHOLE ? launch_norm<XB, RB, RUNS_WHOLE>(a, st) : launch_norm<XB, RB, RUNS_RAGGED>(a, st);
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

template <int SB, int GB, int RUNS>
hipError_t launch_grad(NormGradArgs& a, int64_t grid, hipStream_t st) {
#define THL_GRAD(WPR, CH) \
  return launch(reinterpret_cast<const void*>(&rmsnorm_grad_kernel<SB, GB, WPR, CH, RUNS>), grid, \
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
template <int SB, int GB>
hipError_t launch_grad(NormGradArgs& a, int64_t grid, hipStream_t st) {
  const int runs = runs_of(a.m);
  if (runs == RUNS_TINY) return launch_grad<SB, GB, RUNS_TINY>(a, grid, st);
  return runs == RUNS_WHOLE ? launch_grad<SB, GB, RUNS_WHOLE>(a, grid, st)
                            : launch_grad<SB, GB, RUNS_RAGGED>(a, grid, st);
}

bool bad_ld(int64_t ld, int64_t m) { return ld < (m > 1 ? m : 1); }
bool big(int64_t v) { return v > INT32_MAX; }
bool misaligned(const void* p, thl_dtype t) { return reinterpret_cast<uintptr_t>(p) % bytes_of(t, 1) != 0; }

}  // namespace
}  // namespace thl

using namespace thl;

extern "C" {

thl_status thl_rmsnorm(int64_t m, int64_t n, const void* X, int64_t ldx, const void* R, int64_t ldr, void* S,
                       int64_t lds, const void* W, float eps, float y_scale, void* Y, int64_t ldy, uint8_t* sfy,
                       int64_t ld_sfy, const thl_norm_types* ty, struct ihipStream_t* stream) {
  // ---- arguments
  if (!ty || m < 0 || n < 0) return THL_ERR_INVALID;
  if (m > kMaxFeatures || big(n) || big(ldx) || big(ldr) || big(lds) || big(ldy) || big(ld_sfy)) return THL_ERR_UNSUPPORTED;
  if (!is_float_io(ty->x) || !is_float_io(ty->w)) return THL_ERR_UNSUPPORTED;
  if (R && ty->r != ty->x && ty->r != THL_F32) return THL_ERR_UNSUPPORTED;
  const bool fp8 = ty->y == THL_E4M3 || ty->y == THL_E5M2, fp4 = ty->y == THL_E2M1X2;
  if (!is_float_io(ty->y) && !fp8 && !fp4) return THL_ERR_UNSUPPORTED;
  const bool mx = sfy != nullptr;
  if (is_float_io(ty->y) ? mx : (fp4 && !mx)) return THL_ERR_UNSUPPORTED;
  if (!(eps >= 0.0f) || std::isinf(eps)) return THL_ERR_INVALID;
  const float inv_scale = 1.0f / y_scale;
  if (!(y_scale > 0.0f) || std::isinf(y_scale) || std::isinf(inv_scale)) return THL_ERR_INVALID;
  if (y_scale != 1.0f && (!fp8 || mx)) return THL_ERR_UNSUPPORTED;
  if (bad_ld(ldx, m) || bad_ld(ldy, m)) return THL_ERR_INVALID;
  if (fp4 && ldy % 2 != 0) return THL_ERR_INVALID;
  if (R ? (bad_ld(ldr, m) || (S && bad_ld(lds, m))) : S != nullptr) return THL_ERR_INVALID;
  if (mx && ld_sfy < (m + 31) / 32) return THL_ERR_INVALID;
  if (m == 0 || n == 0) return THL_OK;
  if (!X || !W || !Y) return THL_ERR_INVALID;
  if (misaligned(X, ty->x) || misaligned(W, ty->w) || (is_float_io(ty->y) && misaligned(Y, ty->y)) ||
      (R && (misaligned(R, ty->r) || misaligned(S, ty->r))))
    return THL_ERR_MISALIGNED;

  // ---- overlap: S may be X or R exactly, Y may be X exactly
  const Range rx = matrix_range(X, ty->x, m, n, ldx), rw = matrix_range(W, ty->w, m, 1, m);
  const Range rr = R ? matrix_range(R, ty->r, m, n, ldr) : Range{};
  const Range rs = R ? matrix_range(S, ty->r, m, n, lds) : Range{};
  const Range ry = matrix_range(Y, ty->y, m, n, ldy);
  const Range rf = mx ? matrix_range(sfy, THL_E8M0, (m + 31) / 32, n, ld_sfy) : Range{};
  const bool s_is_x = S == X && lds == ldx && ty->r == ty->x, s_is_r = S == R && lds == ldr;
  const bool y_is_x = Y == X && ldy == ldx && ty->y == ty->x;
  if ((!s_is_x && overlaps(rs, rx)) || (!s_is_r && overlaps(rs, rr)) || overlaps(rs, rw)) return THL_ERR_INVALID;
  if ((!y_is_x && overlaps(ry, rx)) || overlaps(ry, rr) || overlaps(ry, rs) || overlaps(ry, rw)) return THL_ERR_INVALID;
  if (overlaps(rf, rx) || overlaps(rf, rr) || overlaps(rf, rs) || overlaps(rf, rw) || overlaps(rf, ry))
    return THL_ERR_INVALID;

  NormArgs a{};
  a.x = X, a.r = R, a.s = S, a.w = W, a.y = Y, a.sf = sfy;
  a.ldx = ldx, a.ldr = ldr, a.lds = lds, a.ldy = ldy, a.ld_sf = ld_sfy;
  a.n = n, a.m = static_cast<int32_t>(m), a.eps = eps, a.inv_scale = inv_scale;
  a.x_type = ty->x, a.r_type = ty->r, a.w_type = ty->w, a.y_type = ty->y;
  a.y_mode = mx ? Y_MX : (fp8 ? Y_FP8 : Y_FLOAT);
  hipError_t e;
  if (ty->x == THL_F32)
    e = R ? launch_norm<4, 4>(a, stream) : launch_norm<4, 0>(a, stream);
  else if (!R)
    e = launch_norm<2, 0>(a, stream);
  else
    e = ty->r == THL_F32 ? launch_norm<2, 4>(a, stream) : launch_norm<2, 2>(a, stream);
  return e == hipSuccess ? THL_OK : THL_ERR_HIP;
}

size_t thl_rmsnorm_backward_workspace(int64_t m, int64_t n) {
  if (m <= 0 || n <= 0) return 0;
  return static_cast<size_t>(grad_rows(m, n)) * static_cast<size_t>(m) * sizeof(float);
}

thl_status thl_rmsnorm_backward(int64_t m, int64_t n, const void* S, int64_t lds, const void* DY, int64_t lddy,
                                const void* DR, int64_t lddr, const void* W, float eps, void* DX, int64_t lddx,
                                void* DW, void* workspace, size_t workspace_bytes, const thl_norm_grad_types* ty,
                                struct ihipStream_t* stream) {
  if (!ty || m < 0 || n < 0) return THL_ERR_INVALID;
  if (m > kMaxFeatures || big(n) || big(lds) || big(lddy) || big(lddr) || big(lddx)) return THL_ERR_UNSUPPORTED;
  if (!is_float_io(ty->s) || !is_float_io(ty->w) || !is_float_io(ty->g)) return THL_ERR_UNSUPPORTED;
  if (DW && ty->dw != THL_F32 && ty->dw != ty->w) return THL_ERR_UNSUPPORTED;
  if (!(eps >= 0.0f) || std::isinf(eps)) return THL_ERR_INVALID;
  if (bad_ld(lds, m) || bad_ld(lddy, m) || bad_ld(lddx, m) || (DR && bad_ld(lddr, m))) return THL_ERR_INVALID;
  if (m == 0) return THL_OK;
  if (DW && misaligned(DW, ty->dw)) return THL_ERR_MISALIGNED;
  const size_t need = DW ? thl_rmsnorm_backward_workspace(m, n) : 0;
  if (n > 0) {
    if (!S || !DY || !W || !DX) return THL_ERR_INVALID;
    if (need && (!workspace || workspace_bytes < need)) return THL_ERR_INVALID;
    if (misaligned(S, ty->s) || misaligned(DY, ty->g) || misaligned(W, ty->w) || misaligned(DX, ty->g) ||
        misaligned(DR, ty->g) || (need && reinterpret_cast<uintptr_t>(workspace) % 4 != 0))
      return THL_ERR_MISALIGNED;
    // DX may be DY, DR or S exactly; nothing else may overlap an output
    const Range rs = matrix_range(S, ty->s, m, n, lds), rg = matrix_range(DY, ty->g, m, n, lddy);
    const Range rr = matrix_range(DR, ty->g, m, n, lddr), rw = matrix_range(W, ty->w, m, 1, m);
    const Range rx = matrix_range(DX, ty->g, m, n, lddx);
    const Range rd = DW ? matrix_range(DW, ty->dw, m, 1, m) : Range{};
    const Range rp = need ? vector_range(workspace, static_cast<int64_t>(need), 1) : Range{};
    if ((overlaps(rx, rs) && !(DX == S && lddx == lds && ty->g == ty->s)) ||
        (overlaps(rx, rg) && !(DX == DY && lddx == lddy)) || (overlaps(rx, rr) && !(DX == DR && lddx == lddr)) ||
        overlaps(rx, rw))
      return THL_ERR_INVALID;
    for (const Range& o : {rs, rg, rr, rw, rx})
      if (overlaps(rd, o) || overlaps(rp, o)) return THL_ERR_INVALID;
    if (overlaps(rd, rp)) return THL_ERR_INVALID;
  }

  hipError_t e = hipSuccess;
  const int64_t grid = n > 0 ? grad_rows(m, n) : 0;
  if (n > 0) {
    NormGradArgs a{};
    a.s = S, a.dy = DY, a.dr = DR, a.w = W, a.dx = DX, a.part = DW ? static_cast<float*>(workspace) : nullptr;
    a.lds = lds, a.lddy = lddy, a.lddr = lddr, a.lddx = lddx;
    a.n = n, a.m = static_cast<int32_t>(m), a.eps = eps;
    a.s_type = ty->s, a.g_type = ty->g, a.w_type = ty->w;
    if (ty->s == THL_F32)
      e = ty->g == THL_F32 ? launch_grad<4, 4>(a, grid, stream) : launch_grad<4, 2>(a, grid, stream);
    else
      e = ty->g == THL_F32 ? launch_grad<2, 4>(a, grid, stream) : launch_grad<2, 2>(a, grid, stream);
  }
  if (e == hipSuccess && DW) {
    const float* part = static_cast<const float*>(workspace);
    int rows = static_cast<int>(grid), cols = static_cast<int>(m), type = ty->dw;
    void* args[] = {&part, &rows, &cols, &DW, &type};
    e = hipLaunchKernel(reinterpret_cast<const void*>(&rmsnorm_grad_reduce), dim3(static_cast<unsigned>((m + 31) / 32)),
                        dim3(1024), args, 0, stream);
  }
  return e == hipSuccess ? THL_OK : THL_ERR_HIP;
}

}  // extern "C"
