// experts.hip -- a whole mixture-of-experts layer for a few tokens:
//
//   u_t = act(W1g_e x + b1g_e) * (W1u_e x + b1u_e)   or   act(W1_e x + b1_e),   e = ids[j, t]
//   y_j = sum over t of w[j, t] * (W2_e u_t + b2_e)
//
// With a few tokens every weight of a chosen expert is used a few times, so
// the layer is a stream over those weights, bound by HBM.  Nothing is sorted
// and no size passes through the host: a workgroup takes sixteen features of
// one expert, finds that expert's choices among the ids itself, and multiplies
// them, sixteen at a time, on the matrix cores (choices are the rows of the
// tile, features its columns), its wavefronts splitting K.
//
// Three launches: W1 with the activation into the workspace, W2 into the
// workspace, and the choices of each token added in their order.
//
// All products are bf16 by bf16 with fp32 sums, and exact, of one or two
// planes a side: what has more than eight significant bits (fp16 activations
// and weights; u, which is computed in fp32) is a sum of two bf16 numbers, its
// value rounded to eight bits and the rest.  For fp16 that is exact; for u it
// leaves 2^-17 of the value.  fp16 activations meet fp16 weights as they are.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/thl.h"
#include "host_checks.hpp"
#include "rows.hpp"

namespace thl {
namespace {

enum : int { W_B16 = 0, W_H16 = 1, W_E4M3 = 2, W_E2M1 = 3 };
enum : int { X_B16 = 0, X_H16 = 1, X_PAIR = 2 };  // PAIR: u as two planes

constexpr int64_t kMaxPairs = 1024;  // choices of all tokens
constexpr int kWaves = 4;

// Values of K in 16 bytes of a row.
constexpr int piece_of(int wk) { return wk == W_E2M1 ? 32 : (wk == W_E4M3 ? 16 : 8); }

struct ExpertArgs {
  const uint8_t* w;
  const uint8_t* sf;
  const void* bias;
  const uint16_t* x;   // X, or u's first plane
  const uint16_t* lo;  // u's second plane
  const void* ids;
  uint16_t* u_hi;  // outputs: u's planes, or z
  uint16_t* u_lo;
  float* z;
  int64_t w_row, w_expert;  // bytes
  int64_t ld_sf, sf_expert, bias_expert;
  int64_t ldx, ld_u, ld_z, ld_ids;
  int64_t row_bytes;        // of K weights
  int32_t k, features;      // of an output: hidden features, or the layer's
  int32_t pairs, topk, experts, ids_bytes, by_choice;
  int32_t act, bias_type;
};

__device__ __forceinline__ int64_t id_of(const ExpertArgs& a, int p) {
  const int64_t at = static_cast<int64_t>(p / a.topk) * a.ld_ids + p % a.topk;
  return a.ids_bytes == 8 ? static_cast<const int64_t*>(a.ids)[at] : static_cast<const int32_t*>(a.ids)[at];
}

__device__ __forceinline__ v4f mfma_bf(v4i a, v4i b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}
__device__ __forceinline__ v4f mfma_h(v4i a, v4i b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// Eight fp16 numbers as two planes of bf16: the value without its last three
// bits, and those.  Infinities and NaN have no rest.
__device__ __forceinline__ void split_h(v4i x, v4i& hi, v4i& lo) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    uint32_t h[2], l[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint16_t b = static_cast<uint16_t>(static_cast<uint32_t>(x[d]) >> (16 * q));
      const float f = static_cast<float>(__builtin_bit_cast(_Float16, b));
      h[q] = __builtin_bit_cast(uint32_t, f) & 0xffff0000u;
      const float rest = (b & 0x7c00u) == 0x7c00u ? 0.0f : f - __builtin_bit_cast(float, h[q]);
      if ((b & 0x7fffu) > 0x7c00u) h[q] |= 0x00400000u;  // a NaN stays one
      l[q] = __builtin_bit_cast(uint32_t, rest);
    }
    hi[d] = static_cast<int>(__builtin_amdgcn_perm(h[1], h[0], 0x07060302u));
    lo[d] = static_cast<int>(__builtin_amdgcn_perm(l[1], l[0], 0x07060302u));
  }
}

// u as two planes.
__device__ __forceinline__ void split_f(float v, uint16_t& hi, uint16_t& lo) {
  const __bf16 h = static_cast<__bf16>(v);
  const float f = static_cast<float>(h);
  hi = __builtin_bit_cast(uint16_t, h);
  lo = __builtin_fabsf(f) < INFINITY ? __builtin_bit_cast(uint16_t, static_cast<__bf16>(v - f)) : 0;
}

// Codes 8 s .. 8 s + 7 of a piece as bf16, times `scale`, a power of two.
template <int WK>
__device__ __forceinline__ v4i decode(v4i w, int s, float scale) {
  v4i o;
  if constexpr (WK == W_E2M1) {
    const uint32_t v = static_cast<uint32_t>(w[s]);
    o[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 0));
    o[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 1));
    o[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 2));
    o[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 3));
  } else {
    const uint32_t a = static_cast<uint32_t>(w[2 * s]), b = static_cast<uint32_t>(w[2 * s + 1]);
    o[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, false));
    o[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true));
    o[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false));
    o[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true));
  }
  return o;
}

// E8M0 code 1 .. 254 in fp32: 2^(b - 127).
__device__ __forceinline__ float e8m0(uint32_t b) { return __builtin_bit_cast(float, b << 23); }
// The scale next to this one under which every element is a normal bf16
// number, and what it lacks: a factor of the sums.
template <int WK>
__device__ __forceinline__ uint32_t tame(uint32_t b) {
  constexpr uint32_t lo = WK == W_E2M1 ? 2 : 10, hi = WK == W_E2M1 ? 252 : 246;
  return b < lo ? lo : (b > hi ? hi : b);
}
template <int WK>
__device__ __forceinline__ float lacking(uint32_t b) {
  return b == 255 ? __builtin_nanf("") : __builtin_bit_cast(float, (127 + b - tame<WK>(b)) << 23);
}

__device__ __forceinline__ float activated(float v, int act) {
  if (act & THL_MOE_RELU) return v > 0.0f ? v : 0.0f;
  if (act & THL_MOE_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752440f));
  if (act & THL_MOE_SILU) return v / (1.0f + expf(-v));
  return v;
}

// A chunk of K is 128 bytes of every row: lane (feature l % 16, group g = l / 16)
// holds its row's pieces g and 4 + g, whole lines of HBM.  Piece order is K
// order within a lane, so step s of half h multiplies values
// chunk + PK (4 h + g) + 8 s .. + 7 of choices and features alike.
//
// GATED: tiles 0 .. RT/2-1 are gates, the others what they multiply.  UP: the
// first product (u), else the second (z).
template <int WK, int XK, bool UP, bool GATED, int RT>
__global__ void __launch_bounds__(64 * kWaves) experts_kernel(ExpertArgs a) {
  constexpr int PK = piece_of(WK), KC = 8 * PK, STEPS = PK / 8;
  constexpr int OUT = GATED ? RT / 2 : RT;  // tiles of outputs
  constexpr bool MX = WK == W_E4M3 || WK == W_E2M1;
  constexpr bool HALF = WK == W_H16 && XK == X_H16;  // fp16 by fp16
  constexpr int XP = XK == X_B16 || HALF ? 1 : 2;
  __shared__ int list[kMaxPairs];
  __shared__ int hits[kWaves];
  __shared__ float part[kWaves][RT][4][64];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, g = lane >> 4;

  // This workgroup's expert: the y-th, or that of choice y, if y is the first
  // choice of it; and its choices in order.
  int64_t expert = blockIdx.y;
  if (a.by_choice) {
    expert = id_of(a, static_cast<int>(blockIdx.y));
    if (expert < 0 || expert >= a.experts) return;
  }
  int count = 0;
  for (int base = 0; base < a.pairs; base += 64 * kWaves) {
    const int p = base + tid;
    const bool hit = p < a.pairs && id_of(a, p) == expert;
    const uint64_t who = __ballot(hit);
    if (lane == 0) hits[wave] = __popcll(who);
    __syncthreads();
    int at = count, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) at += hits[w];
      all += hits[w];
    }
    if (hit) list[at + __popcll(who & ((1ull << lane) - 1))] = p;
    count += all;
    __syncthreads();
  }
  if (count == 0 || (a.by_choice && list[0] != static_cast<int>(blockIdx.y))) return;

  // Rows of weights: features past the last repeat it, and are not stored.
  const int f0 = static_cast<int>(blockIdx.x) * 16 * OUT;
  const uint8_t* w[RT];
  const uint8_t* sf[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    int f = f0 + 16 * (r % OUT) + col;
    f = f < a.features ? f : a.features - 1;
    const int64_t row = static_cast<int64_t>(f) + (GATED && r >= OUT ? a.features : 0);
    w[r] = a.w + expert * a.w_expert + row * a.w_row;
    sf[r] = MX ? a.sf + expert * a.sf_expert + row * a.ld_sf : nullptr;
  }
  const int whole = a.k / KC;

  for (int first = 0; first < count; first += 16) {
    const int rows = count - first < 16 ? count - first : 16;
    const int p = list[first + (col < rows ? col : rows - 1)];
    const int64_t xrow = XK == X_PAIR ? p : p / a.topk;
    const uint16_t* x = a.x + xrow * a.ldx;
    const uint16_t* xl = XK == X_PAIR ? a.lo + xrow * a.ldx : nullptr;
    v4f acc[RT] = {};

    auto use = [&](const v4i (&wq)[RT][2], const uint32_t (&sc)[RT][2], auto load_x) {
      bool rare = false;
      if constexpr (MX) {
#pragma unroll
        for (int r = 0; r < RT; ++r) rare |= sc[r][0] != tame<WK>(sc[r][0]) || sc[r][1] != tame<WK>(sc[r][1]);
        rare = __ballot(rare) != 0;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        v4f alone[RT][4];  // rare scales: the sums of each lane group's block by themselves
        if (MX && rare) {
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int q = 0; q < 4; ++q) alone[r][q] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          v4i xf[2];
          load_x(h, s, xf);
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            if constexpr (HALF) {
              acc[r] = mfma_h(xf[0], wq[r][h], acc[r]);
            } else if constexpr (WK == W_H16) {
              v4i hi, lo;
              split_h(wq[r][h], hi, lo);
              acc[r] = mfma_bf(xf[0], hi, acc[r]);
              acc[r] = mfma_bf(xf[0], lo, acc[r]);
              if constexpr (XP == 2) {
                acc[r] = mfma_bf(xf[1], hi, acc[r]);
                acc[r] = mfma_bf(xf[1], lo, acc[r]);
              }
            } else if constexpr (WK == W_B16) {
              acc[r] = mfma_bf(xf[0], wq[r][h], acc[r]);
              if constexpr (XP == 2) acc[r] = mfma_bf(xf[1], wq[r][h], acc[r]);
            } else if (!rare) {
              const v4i v = decode<WK>(wq[r][h], s, e8m0(sc[r][h]));
              acc[r] = mfma_bf(xf[0], v, acc[r]);
              if constexpr (XP == 2) acc[r] = mfma_bf(xf[1], v, acc[r]);
            } else {
              const v4i v = decode<WK>(wq[r][h], s, e8m0(tame<WK>(sc[r][h])));
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const v4i mine = g == q ? v : v4i{0, 0, 0, 0};
                alone[r][q] = mfma_bf(xf[0], mine, alone[r][q]);
                if constexpr (XP == 2) alone[r][q] = mfma_bf(xf[1], mine, alone[r][q]);
              }
            }
          }
        }
        if (MX && rare) {
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float factor = lacking<WK>(static_cast<uint32_t>(__shfl(static_cast<int>(sc[r][h]), 16 * q + col)));
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[r][e] += factor * alone[r][q][e];
            }
        }
      }
    };
    // The eight values from k on of this lane's choice, as planes.
    auto planes = [&](v4i v, v4i l, v4i (&xf)[2]) {
      if constexpr (XK == X_H16 && !HALF) {
        split_h(v, xf[0], xf[1]);
      } else {
        xf[0] = v;
        xf[1] = l;
      }
    };

    for (int c = wave; c < whole; c += kWaves) {
      v4i wq[RT][2];
      uint32_t sc[RT][2] = {};
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          wq[r][h] = __builtin_nontemporal_load(
              reinterpret_cast<const v4i_a1*>(w[r] + 128 * static_cast<int64_t>(c) + 64 * h + 16 * g));
          if constexpr (MX) sc[r][h] = sf[r][static_cast<int64_t>(c) * (KC / 32) + (4 * h + g) * PK / 32];
        }
      use(wq, sc, [&](int h, int s, v4i (&xf)[2]) {
        const int64_t k = static_cast<int64_t>(c) * KC + PK * (4 * h + g) + 8 * s;
        v4i v = *reinterpret_cast<const v4i_a2*>(x + k), l = {};
        if constexpr (XK == X_PAIR) l = *reinterpret_cast<const v4i_a2*>(xl + k);
        planes(v, l, xf);
      });
    }
    if (whole * KC < a.k && wave == whole % kWaves) {  // K's partial chunk
      const int c = whole;
      v4i wq[RT][2];
      uint32_t sc[RT][2];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t at = 128 * static_cast<int64_t>(c) + 64 * h + 16 * g;
          load_codes_at(w[r] + at, a.row_bytes - at, wq[r][h]);
          sc[r][h] = 127;
          if constexpr (MX) {
            const int64_t k = static_cast<int64_t>(c) * KC + (4 * h + g) * PK;
            if (k < a.k) sc[r][h] = sf[r][k / 32];
          }
        }
      use(wq, sc, [&](int h, int s, v4i (&xf)[2]) {
        const int64_t k = static_cast<int64_t>(c) * KC + PK * (4 * h + g) + 8 * s, left = a.k - k;
        const int valid = left < 8 ? static_cast<int>(left < 0 ? 0 : left) : 8;
        v4i v = load_x8(x + k, valid), l = {};
        if constexpr (XK == X_PAIR) l = load_x8(xl + k, valid);
        planes(v, l, xf);
      });
    }

    // The wavefronts' sums in their order: register e of lane l is choice
    // 4 (l / 16) + e and feature l % 16.
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[wave][r][e][lane] = acc[r][e];
    __syncthreads();
    auto sum = [&](int r) {
      float v = 0.0f;
#pragma unroll
      for (int w2 = 0; w2 < kWaves; ++w2) v += part[w2][r][wave][lane];
      return v;
    };
    static_assert(kWaves == 4, "a wavefront finishes one register");
    const int row = 4 * g + wave;
#pragma unroll
    for (int r = 0; r < OUT; ++r) {
      const int f = f0 + 16 * r + col;
      if (row >= rows || f >= a.features) continue;
      const int64_t at = list[first + row], b = expert * a.bias_expert + f;
      float v = sum(r);
      if (a.bias) v += load_f(a.bias, a.bias_type, b);
      if constexpr (UP) {
        v = activated(v, a.act);
        if constexpr (GATED) {
          float m = sum(OUT + r);
          if (a.bias) m += load_f(a.bias, a.bias_type, b + a.features);
          v *= m;
        }
        uint16_t hi, lo;
        split_f(v, hi, lo);
        a.u_hi[at * a.ld_u + f] = hi;
        a.u_lo[at * a.ld_u + f] = lo;
      } else {
        a.z[at * a.ld_z + f] = v;
      }
    }
  }
}

struct JoinArgs {
  const float* z;
  const float* weights;
  const void* ids;
  void* y;
  int64_t ldy, ld_ids;
  int32_t m, n, topk, experts, ids_bytes, y_type;
};

// y_j = the sum over its choices, in their order.
__global__ void __launch_bounds__(256) experts_join_kernel(JoinArgs a) {
  const int64_t total = static_cast<int64_t>(a.n) * a.m;
  for (int64_t q = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; q < total;
       q += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t j = q / a.m, i = q - j * a.m;
    float v = 0.0f;
    for (int t = 0; t < a.topk; ++t) {
      const int64_t at = j * a.ld_ids + t;
      const int64_t e = a.ids_bytes == 8 ? static_cast<const int64_t*>(a.ids)[at] : static_cast<const int32_t*>(a.ids)[at];
      if (e >= 0 && e < a.experts) v += a.weights[j * a.topk + t] * a.z[(j * a.topk + t) * a.m + i];
    }
    const int64_t to = j * a.ldy + i;
    if (a.y_type == THL_F32)
      static_cast<float*>(a.y)[to] = v;
    else if (a.y_type == THL_F16)
      static_cast<_Float16*>(a.y)[to] = static_cast<_Float16>(v);
    else
      static_cast<__bf16*>(a.y)[to] = static_cast<__bf16>(v);
  }
}

template <int WK, int XK, bool UP, bool GATED, int RT>
hipError_t launch(ExpertArgs& a, hipStream_t st) {
  constexpr int OUT = 16 * (GATED ? RT / 2 : RT);
  const int64_t tiles = (static_cast<int64_t>(a.features) + OUT - 1) / OUT;
  const int slots = a.by_choice ? a.pairs : a.experts;
  void* args[] = {&a};
  return hipLaunchKernel(reinterpret_cast<const void*>(&experts_kernel<WK, XK, UP, GATED, RT>),
                         dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(slots)), dim3(64 * kWaves), args, 0,
                         st);
}
template <int WK, int XK>
hipError_t launch_up(ExpertArgs& a, bool gated, hipStream_t st) {
  return gated ? launch<WK, XK, true, true, 2>(a, st) : launch<WK, XK, true, false, 2>(a, st);
}
hipError_t launch_up(ExpertArgs& a, thl_dtype w, bool x_bf, bool gated, hipStream_t st) {
  switch (w) {
    case THL_BF16:
      return launch_up<W_B16, X_B16>(a, gated, st);
    case THL_F16:
      return launch_up<W_H16, X_H16>(a, gated, st);
    case THL_E4M3:
      return x_bf ? launch_up<W_E4M3, X_B16>(a, gated, st) : launch_up<W_E4M3, X_H16>(a, gated, st);
    default:
      return x_bf ? launch_up<W_E2M1, X_B16>(a, gated, st) : launch_up<W_E2M1, X_H16>(a, gated, st);
  }
}
hipError_t launch_down(ExpertArgs& a, thl_dtype w, hipStream_t st) {
  switch (w) {
    case THL_BF16:
      return launch<W_B16, X_PAIR, false, false, 2>(a, st);
    case THL_F16:
      return launch<W_H16, X_PAIR, false, false, 2>(a, st);
    case THL_E4M3:
      return launch<W_E4M3, X_PAIR, false, false, 2>(a, st);
    default:
      return launch<W_E2M1, X_PAIR, false, false, 2>(a, st);
  }
}

bool big(int64_t v) { return v > INT32_MAX; }
int64_t at_least_one(int64_t v) { return v > 1 ? v : 1; }
bool off(const void* p, thl_dtype t) { return reinterpret_cast<uintptr_t>(p) % bytes_of(t, 1) != 0; }
bool is_mx(thl_dtype t) { return t == THL_E4M3 || t == THL_E2M1X2; }

constexpr int64_t kMaxStride = INT64_C(1) << 40;

// One of the layer's matrices of `rows` rows of k.
thl_status check(const thl_expert_matrix& w, int64_t rows, int64_t k, thl_dtype x) {
  if (!is_mx(w.type) && w.type != x) return THL_ERR_UNSUPPORTED;
  if (big(w.ld) || big(w.ld_sf) || w.stride > kMaxStride || w.stride_sf > kMaxStride || w.stride_bias > kMaxStride)
    return THL_ERR_UNSUPPORTED;
  if (w.bias && !is_float_io(w.type_bias)) return THL_ERR_UNSUPPORTED;
  if (is_mx(w.type) != (w.sf != nullptr)) return THL_ERR_INVALID;
  if (w.ld < at_least_one(k) || w.stride < 0 || w.stride_sf < 0 || w.stride_bias < 0) return THL_ERR_INVALID;
  if (w.type == THL_E2M1X2 && (w.ld % 2 != 0 || w.stride % 2 != 0)) return THL_ERR_INVALID;
  if (is_mx(w.type) && w.ld_sf < (k + 31) / 32) return THL_ERR_INVALID;
  if (!w.w) return THL_ERR_INVALID;
  if (!is_mx(w.type) && off(w.w, w.type)) return THL_ERR_MISALIGNED;
  if (w.bias && off(w.bias, w.type_bias)) return THL_ERR_MISALIGNED;
  return THL_OK;
}
// What it reads: weights, scales, bias.
void ranges(const thl_expert_matrix& w, int64_t experts, int64_t rows, int64_t k, Range (&o)[3]) {
  o[0] = vector_range(w.w, bytes_of(w.type, (experts - 1) * w.stride + (rows - 1) * w.ld + k), 1);
  o[1] = w.sf ? vector_range(w.sf, (experts - 1) * w.stride_sf + (rows - 1) * w.ld_sf + (k + 31) / 32, 1) : Range{};
  o[2] = w.bias ? vector_range(w.bias, bytes_of(w.type_bias, (experts - 1) * w.stride_bias + rows), 1) : Range{};
}
void matrix(ExpertArgs& a, const thl_expert_matrix& w, int64_t k) {
  a.w = static_cast<const uint8_t*>(w.w), a.sf = w.sf, a.bias = w.bias, a.bias_type = w.type_bias;
  a.w_row = bytes_of(w.type, w.ld), a.w_expert = bytes_of(w.type, w.stride);
  a.ld_sf = w.ld_sf, a.sf_expert = w.stride_sf, a.bias_expert = w.stride_bias;
  a.row_bytes = bytes_of(w.type, k), a.k = static_cast<int32_t>(k);
}

int64_t pitch(int64_t hidden) { return (hidden + 63) / 64 * 64; }

}  // namespace
}  // namespace thl

using namespace thl;

extern "C" {

size_t thl_moe_layer_workspace(int64_t m, int64_t hidden, int64_t n, int64_t topk) {
  if (m <= 0 || m > kMaxFeatures || hidden <= 0 || hidden > kMaxFeatures || n <= 0 || topk <= 0) return 0;
  if (n > kMaxPairs || topk > kMaxPairs || n * topk > kMaxPairs) return 0;
  return static_cast<size_t>(n * topk) * 4 * static_cast<size_t>(pitch(hidden) + m);
}

thl_status thl_moe_layer(int64_t m, int64_t hidden, int64_t n, int64_t topk, int64_t experts, const void* X,
                         int64_t ldx, const void* ids, int64_t ld_ids, int ids_bytes, const float* weights,
                         const thl_expert_matrix* up, const thl_expert_matrix* down, unsigned flags, void* Y,
                         int64_t ldy, thl_dtype type_x, thl_dtype type_y, void* workspace, size_t workspace_bytes,
                         struct ihipStream_t* stream) {
  // ---- arguments
  if (!up || !down || m < 0 || hidden < 0 || n < 0 || topk < 0 || experts < 1) return THL_ERR_INVALID;
  if (m > kMaxFeatures || hidden > kMaxFeatures || experts > INT32_MAX / 2 || big(ldx) || big(ldy) || big(ld_ids))
    return THL_ERR_UNSUPPORTED;
  if (n > kMaxPairs || topk > kMaxPairs || n * topk > kMaxPairs) return THL_ERR_UNSUPPORTED;
  if (type_x != THL_F16 && type_x != THL_BF16) return THL_ERR_UNSUPPORTED;
  if (!is_float_io(type_y)) return THL_ERR_UNSUPPORTED;
  if (ids_bytes != 4 && ids_bytes != 8) return THL_ERR_UNSUPPORTED;
  if (flags & ~static_cast<unsigned>(THL_MOE_GATED | THL_MOE_RELU | THL_MOE_GELU | THL_MOE_SILU)) return THL_ERR_INVALID;
  const unsigned act = flags & (THL_MOE_RELU | THL_MOE_GELU | THL_MOE_SILU);
  if ((act & (act - 1)) != 0) return THL_ERR_INVALID;  // one at most
  const bool gated = (flags & THL_MOE_GATED) != 0;
  if (ldx < at_least_one(m) || ldy < at_least_one(m) || ld_ids < at_least_one(topk)) return THL_ERR_INVALID;
  if (m == 0 || n == 0) return THL_OK;
  if (hidden == 0 || topk == 0) return THL_ERR_INVALID;
  const int64_t rows1 = gated ? 2 * hidden : hidden;
  thl_status s = check(*up, rows1, m, type_x);
  if (s == THL_OK) s = check(*down, m, hidden, type_x);
  if (s != THL_OK) return s;
  if (!X || !ids || !weights || !Y) return THL_ERR_INVALID;
  const size_t need = thl_moe_layer_workspace(m, hidden, n, topk);
  if (!workspace || workspace_bytes < need) return THL_ERR_INVALID;
  if (off(X, type_x) || off(Y, type_y) || off(weights, THL_F32) ||
      reinterpret_cast<uintptr_t>(ids) % static_cast<unsigned>(ids_bytes) != 0 ||
      reinterpret_cast<uintptr_t>(workspace) % 4 != 0)
    return THL_ERR_MISALIGNED;

  // ---- Y and the workspace overlap nothing
  Range r1[3], r2[3];
  ranges(*up, experts, rows1, m, r1);
  ranges(*down, experts, m, hidden, r2);
  const Range ry = matrix_range(Y, type_y, m, n, ldy), rp = vector_range(workspace, static_cast<int64_t>(need), 1);
  const Range rest[] = {matrix_range(X, type_x, m, n, ldx),
                        vector_range(ids, (n - 1) * ld_ids + topk, ids_bytes), vector_range(weights, n * topk, 4),
                        r1[0], r1[1], r1[2], r2[0], r2[1], r2[2]};
  if (overlaps(ry, rp)) return THL_ERR_INVALID;
  for (const Range& o : rest)
    if (overlaps(ry, o) || overlaps(rp, o)) return THL_ERR_INVALID;

  const int64_t pairs = n * topk, ld_u = pitch(hidden);
  ExpertArgs a{};
  a.ids = ids, a.ld_ids = ld_ids, a.ids_bytes = ids_bytes;
  a.pairs = static_cast<int32_t>(pairs), a.topk = static_cast<int32_t>(topk), a.experts = static_cast<int32_t>(experts);
  // a workgroup for each choice where they are fewer than the experts (grid rows)
  a.by_choice = pairs < experts;
  a.u_hi = static_cast<uint16_t*>(workspace), a.u_lo = a.u_hi + pairs * ld_u;
  a.z = reinterpret_cast<float*>(a.u_lo + pairs * ld_u);
  a.ld_u = ld_u, a.ld_z = m;

  matrix(a, *up, m);
  a.x = static_cast<const uint16_t*>(X), a.ldx = ldx, a.features = static_cast<int32_t>(hidden);
  a.act = static_cast<int32_t>(act);
  hipError_t e = launch_up(a, up->type, type_x == THL_BF16, gated, stream);
  if (e == hipSuccess) {
    matrix(a, *down, hidden);
    a.x = a.u_hi, a.lo = a.u_lo, a.ldx = ld_u, a.features = static_cast<int32_t>(m);
    e = launch_down(a, down->type, stream);
  }
  if (e == hipSuccess) {
    JoinArgs j{};
    j.z = a.z, j.weights = weights, j.ids = ids, j.y = Y, j.ldy = ldy, j.ld_ids = ld_ids;
    j.m = static_cast<int32_t>(m), j.n = static_cast<int32_t>(n), j.topk = a.topk, j.experts = a.experts;
    j.ids_bytes = ids_bytes, j.y_type = type_y;
    void* args[] = {&j};
    const int64_t blocks = (n * m + 255) / 256;
    e = hipLaunchKernel(reinterpret_cast<const void*>(&experts_join_kernel),
                        dim3(static_cast<unsigned>(blocks < 8192 ? blocks : 8192)), dim3(256), args, 0, stream);
  }
  return e == hipSuccess ? THL_OK : THL_ERR_HIP;
}

}  // extern "C"
