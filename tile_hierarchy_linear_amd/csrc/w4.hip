// w4.hip -- the product of a few tokens with a matrix of 4-bit weights under
// group scales (16-bit activations, fp32 sums):
//
//   D(i,j) = act(alpha * sum_g s(i,g) * sum_{p in g} (q(i,p) - z(i,g)) X(p,j) + beta C(i,j) + bias_i)
//
// With a few tokens every weight is used a few times, so the product is a
// stream over the weights: bound by HBM.  As in the small-M kernel, weights
// go from memory straight into matrix-core operand registers, a whole
// 128-byte line (256 codes) of each of 16 features per K unit, with K spread
// over the wavefronts of a workgroup so that enough lines are in flight.
// Tokens are the rows of the matrix-core tile, features its columns: a lane
// then holds sums of one feature, and needs one scale a group.
//
// Codes become 16-bit floats without a conversion instruction: placed in the
// upper mantissa bits of 16.0 an unsigned code q reads as 16 + q, exactly, in
// bf16 and in fp16, two codes per shift and and-or.  The offset leaves with
// the zero point, (16 + z) * sum_p X(p,j), the sum of X over a group coming
// from a product with a matrix of ones in the same layout.  Signed codes are
// q + 8 with their top bit turned.  E2M1 codes are converted two at a time
// by the hardware's own instruction (exact).
//
// Every product is exact in fp32; sums within a group, its scaling and the
// sum over groups round in fp32 like any fp32 product does.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/thl.h"
#include "host_checks.hpp"
#include "rows.hpp"

namespace thl {
namespace {

typedef int v4i_a1 __attribute__((ext_vector_type(4), aligned(1)));

struct W4Args {
  const uint8_t* w;
  const void* scales;
  const uint8_t* zeros;  // unsigned codes only
  const uint16_t* x;
  const void* c;
  void* d;
  const void* bias;
  int64_t ldw_bytes, ld_scales, ld_zeros, ldx, ldc, ldd;
  int32_t m, n, k, groups;
  int32_t group_shift;  // log2 of the group length (31: one group a feature)
  uint32_t flip;        // signed codes: the bits that turn q into q + 8
  int32_t s_type, c_type, d_type, bias_type, flags;
  float alpha, beta;
};

enum : int { W_INT = 0, W_E2M1 = 1 };

template <bool BF>
__device__ __forceinline__ v4f mfma16(v4i a, v4i b, v4f c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0,
                                                   0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// Eight codes as eight 16-bit floats.  Integer codes come out as 16 + q in
// the order 0, 4, 1, 5, 2, 6, 3, 7, E2M1 codes in order.
template <int WT, bool BF>
__device__ __forceinline__ v4i decode(uint32_t v) {
  v4i o;
  if constexpr (WT == W_E2M1) {
    if constexpr (BF) {
      o[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 0));
      o[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 1));
      o[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 2));
      o[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 3));
    } else {
      o[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, 1.0f, 0));
      o[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, 1.0f, 1));
      o[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, 1.0f, 2));
      o[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, 1.0f, 3));
    }
  } else if constexpr (BF) {  // 16.0 = 0x4180, units at mantissa bit 3
    o[0] = static_cast<int>(((v << 3) & 0x00780078u) | 0x41804180u);
    o[1] = static_cast<int>(((v >> 1) & 0x00780078u) | 0x41804180u);
    o[2] = static_cast<int>(((v >> 5) & 0x00780078u) | 0x41804180u);
    o[3] = static_cast<int>(((v >> 9) & 0x00780078u) | 0x41804180u);
  } else {  // 16.0 = 0x4c00, units at mantissa bit 6
    o[0] = static_cast<int>(((v << 6) & 0x03c003c0u) | 0x4c004c00u);
    o[1] = static_cast<int>(((v << 2) & 0x03c003c0u) | 0x4c004c00u);
    o[2] = static_cast<int>(((v >> 2) & 0x03c003c0u) | 0x4c004c00u);
    o[3] = static_cast<int>(((v >> 6) & 0x03c003c0u) | 0x4c004c00u);
  }
  return o;
}

// Eight activations in decode's order.
template <int WT>
__device__ __forceinline__ v4i in_order(v4i x) {
  if constexpr (WT == W_E2M1) {
    return x;
  } else {
    v4i o;
    o[0] = static_cast<int>(__builtin_amdgcn_perm(x[2], x[0], 0x05040100u));
    o[1] = static_cast<int>(__builtin_amdgcn_perm(x[2], x[0], 0x07060302u));
    o[2] = static_cast<int>(__builtin_amdgcn_perm(x[3], x[1], 0x05040100u));
    o[3] = static_cast<int>(__builtin_amdgcn_perm(x[3], x[1], 0x07060302u));
    return o;
  }
}

// Lane group g (of 16 lanes), register s  <->  lane group s, register g.
__device__ __forceinline__ v4i turn(v4i w) {
  typedef unsigned v2 __attribute__((ext_vector_type(2)));
  v2 a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  v2 b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  v2 c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  v2 d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return v4i{static_cast<int>(c[0]), static_cast<int>(c[1]), static_cast<int>(d[0]), static_cast<int>(d[1])};
}

__device__ __forceinline__ uint32_t scale_bits(const void* p, int type, int64_t i) {
  if (type == THL_F32) return static_cast<const uint32_t*>(p)[i];
  if (type == THL_E8M0) return static_cast<const uint8_t*>(p)[i];
  return static_cast<const uint16_t*>(p)[i];
}
__device__ __forceinline__ float scale_value(uint32_t b, int type) {
  if (type == THL_F32) return __builtin_bit_cast(float, b);
  if (type == THL_BF16) return __builtin_bit_cast(float, b << 16);
  if (type == THL_F16) return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(b)));
  // E8M0: 2^(b - 127), 2^-127 a subnormal, 255 NaN
  return __builtin_bit_cast(float, b == 255 ? 0x7fc00000u : (b == 0 ? 0x00400000u : b << 23));
}

// GPU: scale groups in a unit of 256 codes (1 also for longer groups).
// MT: sixteen-token tiles.  NB: sixteen-feature tiles per wavefront.
template <int WT, bool BF, int GPU, int MT, int NB>
__global__ void __launch_bounds__(512) w4_kernel(W4Args a) {
  extern __shared__ float part[];  // [wavefront][NB][MT][4][64]
  constexpr int LEN = 256 / GPU;   // codes per group within a unit
  constexpr bool TURN = LEN < 128;
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int waves = static_cast<int>(blockDim.x) >> 6;
  const int col = lane & 15, g = lane >> 4;
  const int i0 = static_cast<int>(blockIdx.x) * 16 * NB, j0 = static_cast<int>(blockIdx.y) * 16 * MT;
  const int units = (a.k + 255) >> 8;
  const int u_beg = static_cast<int>(static_cast<int64_t>(wave) * units / waves);
  const int u_end = static_cast<int>(static_cast<int64_t>(wave + 1) * units / waves);

  // Features past m and tokens past n repeat the last one; nothing of them
  // is stored.
  const uint8_t* w[NB];
  int64_t srow[NB], zrow[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int i = i0 + 16 * b + col < a.m ? i0 + 16 * b + col : a.m - 1;
    w[b] = a.w + static_cast<int64_t>(i) * a.ldw_bytes;
    srow[b] = static_cast<int64_t>(i) * a.ld_scales;
    zrow[b] = static_cast<int64_t>(i) * a.ld_zeros;
  }
  // Row `col` of the token tile is token 4 (col % 4) + col / 4, so that
  // register r of lane group g of the sums is token 4 r + g.
  const uint16_t* x[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int j = j0 + 16 * t + 4 * (col & 3) + (col >> 2);
    x[t] = a.x + static_cast<int64_t>(j < a.n ? j : a.n - 1) * a.ldx;
  }

  v4f tot[NB][MT] = {};
  const v4i ones = BF ? v4i{0x3f803f80, 0x3f803f80, 0x3f803f80, 0x3f803f80}
                      : v4i{0x3c003c00, 0x3c003c00, 0x3c003c00, 0x3c003c00};

  struct Unit {
    v4i w[NB][2];
    uint32_t s[NB][GPU], z[NB][GPU];
  };
  // A whole unit's loads; codes past K (FULL = false) read as zero codes and
  // are met by zero activations.
  auto load = [&](int u, auto full_tag, Unit& o) {
    constexpr bool FULL = decltype(full_tag)::value;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t at = 128 * static_cast<int64_t>(u) + 64 * h + 16 * g;
        if (FULL || at + 16 <= (a.k >> 1)) {
          o.w[b][h] = *reinterpret_cast<const v4i_a1*>(w[b] + at);
        } else {
          uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
          for (int q = 0; q < 16; ++q)
            if (at + q < (a.k + 1) >> 1) v[q / 4] |= static_cast<uint32_t>(w[b][at + q]) << (8 * (q & 3));
          o.w[b][h] = v4i{static_cast<int>(v[0]), static_cast<int>(v[1]), static_cast<int>(v[2]),
                          static_cast<int>(v[3])};
        }
      }
#pragma unroll
      for (int q = 0; q < GPU; ++q) {
        int at = static_cast<int>((256 * static_cast<int64_t>(u) + LEN * q) >> a.group_shift);
        if (!FULL && at >= a.groups) at = a.groups - 1;
        o.s[b][q] = scale_bits(a.scales, a.s_type, srow[b] + at);
        o.z[b][q] = WT == W_INT ? (a.zeros ? a.zeros[zrow[b] + at] : 8u) : 0u;
      }
    }
  };
  auto use = [&](int u, auto full_tag, Unit& o) {
    constexpr bool FULL = decltype(full_tag)::value;
    v4f acc[NB][MT] = {}, xs[MT] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v4i wq[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        wq[b] = TURN ? turn(o.w[b][h]) : o.w[b][h];
        if constexpr (WT == W_INT) {
#pragma unroll
          for (int s = 0; s < 4; ++s) wq[b][s] ^= static_cast<int>(a.flip);
        }
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        // the eight K this lane holds of this product
        const int64_t p = 256 * static_cast<int64_t>(u) + 128 * h + (TURN ? 32 * s + 8 * g : 32 * g + 8 * s);
        v4i xa[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t)
          xa[t] = in_order<WT>(load_raw8<2>(x[t], p, FULL ? 8 : static_cast<int>(a.k - p)).w);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const v4i wf = decode<WT, BF>(static_cast<uint32_t>(wq[b][s]));
#pragma unroll
          for (int t = 0; t < MT; ++t) acc[b][t] = mfma16<BF>(xa[t], wf, acc[b][t]);
        }
        if constexpr (WT == W_INT) {
#pragma unroll
          for (int t = 0; t < MT; ++t) xs[t] = mfma16<BF>(xa[t], ones, xs[t]);
        }
        // end of a group: its sums leave under its scale
        const int done = 128 * h + 32 * (s + 1);
        if ((TURN && done % LEN == 0) || (!TURN && s == 3 && (LEN == 128 || h == 1))) {
          const int q = (done - 1) / LEN;
          if (FULL || 256 * static_cast<int64_t>(u) + LEN * q < a.k) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              const float sv = scale_value(o.s[b][q], a.s_type);
              const float zv = static_cast<float>(16u + o.z[b][q]);
#pragma unroll
              for (int t = 0; t < MT; ++t) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                  float v = acc[b][t][r];
                  if constexpr (WT == W_INT) v -= zv * xs[t][r];
                  tot[b][t][r] += sv * v;
                }
                acc[b][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
              }
            }
          }
#pragma unroll
          for (int t = 0; t < MT; ++t) xs[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
      }
    }
  };

  // Whole units, the next one's loads out before this one's products; then
  // the last, partial unit of K.
  const int u_full = u_end < (a.k >> 8) ? u_end : (a.k >> 8);
  Unit cur, next;
  if (u_beg < u_full) load(u_beg, std::true_type{}, cur);
  for (int u = u_beg; u < u_full; ++u) {
    if (u + 1 < u_full) load(u + 1, std::true_type{}, next);
    use(u, std::true_type{}, cur);
    cur = next;
  }
  if (u_full < u_end && u_beg < u_end) {
    load(u_end - 1, std::false_type{}, cur);
    use(u_end - 1, std::false_type{}, cur);
  }

  // The wavefronts' partial sums, added in wavefront order.
  constexpr int TILE = NB * MT * 256;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wave * TILE + ((b * MT + t) * 4 + r) * 64 + lane] = tot[b][t][r];
  __syncthreads();
  for (int q = static_cast<int>(threadIdx.x); q < TILE; q += static_cast<int>(blockDim.x)) {
    const int l = q & 63, r = (q >> 6) & 3, t = (q >> 8) % MT, b = (q >> 8) / MT;
    const int i = i0 + 16 * b + (l & 15), j = j0 + 16 * t + 4 * r + (l >> 4);
    if (i >= a.m || j >= a.n) continue;
    float v = part[q];
    for (int s = 1; s < waves; ++s) v += part[s * TILE + q];
    v *= a.alpha;
    if (nonzero_f32(a.beta)) v += a.beta * load_f(a.c, a.c_type, static_cast<int64_t>(j) * a.ldc + i);
    if (a.flags & EPI_BIAS) v += load_f(a.bias, a.bias_type, i);
    v = activate(v, a.flags);
    const int64_t at = static_cast<int64_t>(j) * a.ldd + i;
    if (a.d_type == THL_F32)
      static_cast<float*>(a.d)[at] = v;
    else if (a.d_type == THL_F16)
      static_cast<_Float16*>(a.d)[at] = static_cast<_Float16>(v);
    else
      static_cast<__bf16*>(a.d)[at] = static_cast<__bf16>(v);
  }
}

template <int WT, bool BF, int GPU, int MT, int NB>
hipError_t launch_one(W4Args& a, hipStream_t st) {
  const int units = (a.k + 255) / 256;
  int waves = 8;
  while (waves > 1 && waves > units) waves /= 2;
  const int64_t gx = (static_cast<int64_t>(a.m) + 16 * NB - 1) / (16 * NB), gy = (static_cast<int64_t>(a.n) + 16 * MT - 1) / (16 * MT);
  void* args[] = {&a};
  return hipLaunchKernel(reinterpret_cast<const void*>(&w4_kernel<WT, BF, GPU, MT, NB>),
                         dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), dim3(waves * 64), args,
                         static_cast<size_t>(waves) * NB * MT * 256 * sizeof(float), st);
}

template <int WT, bool BF, int GPU>
hipError_t launch_tokens(W4Args& a, hipStream_t st) {
  if (a.n <= 16) return launch_one<WT, BF, GPU, 1, 1>(a, st);
  if (a.n <= 32) return launch_one<WT, BF, GPU, 2, 1>(a, st);
  return launch_one<WT, BF, GPU, 4, 2>(a, st);
}

template <bool BF>
hipError_t launch_type(W4Args& a, int wt, hipStream_t st) {
  if (wt == W_E2M1) return launch_tokens<W_E2M1, BF, 8>(a, st);
  switch (a.group_shift) {
    case 5:
      return launch_tokens<W_INT, BF, 8>(a, st);
    case 6:
      return launch_tokens<W_INT, BF, 4>(a, st);
    case 7:
      return launch_tokens<W_INT, BF, 2>(a, st);
    default:
      return launch_tokens<W_INT, BF, 1>(a, st);
  }
}

constexpr int64_t kMaxTokens = INT64_C(1) << 21;  // grid rows of 64

bool big(int64_t v) { return v > INT32_MAX; }
int64_t at_least_one(int64_t v) { return v > 1 ? v : 1; }
bool misaligned(const void* p, thl_dtype t) { return reinterpret_cast<uintptr_t>(p) % bytes_of(t, 1) != 0; }

}  // namespace
}  // namespace thl

using namespace thl;

extern "C" thl_status thl_gemm_w4(int64_t m, int64_t n, int64_t k, const void* W, int64_t ldw,
                                  const thl_group_scales* gs, const void* X, int64_t ldx, const void* C, int64_t ldc,
                                  void* D, int64_t ldd, float alpha, float beta, const thl_dtypes* dt,
                                  const thl_epilogue* epi, struct ihipStream_t* stream) {
  // ---- arguments
  if (!dt || !gs || m < 0 || n < 0 || k < 0) return THL_ERR_INVALID;
  if (m > kMaxFeatures || n > kMaxTokens || big(k) || big(ldw) || big(ldx) || big(ldc) || big(ldd) || big(gs->ld_scales) ||
      big(gs->ld_zeros))
    return THL_ERR_UNSUPPORTED;
  const unsigned flags = epi ? epi->flags : 0;
  if (flags & ~static_cast<unsigned>(THL_EPI_BIAS | THL_EPI_RELU | THL_EPI_GELU)) return THL_ERR_INVALID;
  if ((flags & THL_EPI_RELU) && (flags & THL_EPI_GELU)) return THL_ERR_INVALID;
  const bool has_bias = (flags & THL_EPI_BIAS) != 0;
  const void* bias = has_bias ? epi->bias : nullptr;

  // ---- supported combinations
  const bool e2m1 = dt->a == THL_E2M1X2, u4 = dt->a == THL_U4X2;
  if (!e2m1 && !u4 && dt->a != THL_I4X2) return THL_ERR_UNSUPPORTED;
  if (dt->b != THL_F16 && dt->b != THL_BF16) return THL_ERR_UNSUPPORTED;
  if (dt->acc != THL_F32 || !is_float_io(dt->d)) return THL_ERR_UNSUPPORTED;
  if (beta != 0.0f && !is_float_io(dt->c)) return THL_ERR_UNSUPPORTED;
  if (has_bias && !is_float_io(dt->bias)) return THL_ERR_UNSUPPORTED;
  if (e2m1 ? gs->type != THL_E8M0 : !is_float_io(gs->type)) return THL_ERR_UNSUPPORTED;
  if (!u4 && gs->zeros) return THL_ERR_UNSUPPORTED;
  // group length: a power of two from 32 on, or one group for the whole of K
  if (gs->group < 1) return THL_ERR_INVALID;
  int shift = 31;
  if (e2m1) {
    if (gs->group != 32) return THL_ERR_UNSUPPORTED;
    shift = 5;
  } else if (gs->group < k || gs->group == 32 || gs->group == 64 || gs->group == 128) {
    if (gs->group < 32 || (gs->group & (gs->group - 1)) != 0) return THL_ERR_UNSUPPORTED;
    shift = __builtin_ctzll(static_cast<uint64_t>(gs->group));
  }
  const int64_t groups = k == 0 ? 0 : (shift == 31 ? 1 : ((k - 1) >> shift) + 1);

  // ---- leading dimensions and pointers
  if (ldw < at_least_one(k) || ldw % 2 != 0 || ldx < at_least_one(k) || ldd < at_least_one(m)) return THL_ERR_INVALID;
  if (beta != 0.0f && ldc < at_least_one(m)) return THL_ERR_INVALID;
  if (gs->ld_scales < at_least_one(groups) || (u4 && gs->ld_zeros < at_least_one(groups))) return THL_ERR_INVALID;
  if (m == 0 || n == 0) return THL_OK;
  if (!D || (beta != 0.0f && !C) || (has_bias && !bias)) return THL_ERR_INVALID;
  if (k > 0 && (!W || !X || !gs->scales || (u4 && !gs->zeros))) return THL_ERR_INVALID;
  if (misaligned(X, dt->b) || misaligned(D, dt->d) || (beta != 0.0f && misaligned(C, dt->c)) ||
      (has_bias && misaligned(bias, dt->bias)) || misaligned(gs->scales, gs->type))
    return THL_ERR_MISALIGNED;

  // ---- overlap: D may alias C exactly
  const Range rd = matrix_range(D, dt->d, m, n, ldd);
  if (beta != 0.0f && !(C == D && ldc == ldd && dt->c == dt->d) && overlaps(rd, matrix_range(C, dt->c, m, n, ldc)))
    return THL_ERR_INVALID;
  if (overlaps(rd, matrix_range(W, dt->a, k, m, ldw)) || overlaps(rd, matrix_range(X, dt->b, k, n, ldx)) ||
      overlaps(rd, matrix_range(gs->scales, gs->type, groups, m, gs->ld_scales)) ||
      (u4 && overlaps(rd, matrix_range(gs->zeros, THL_I8, groups, m, gs->ld_zeros))) ||
      (has_bias && overlaps(rd, matrix_range(bias, dt->bias, m, 1, m))))
    return THL_ERR_INVALID;

  W4Args a{};
  a.w = static_cast<const uint8_t*>(W), a.scales = gs->scales, a.zeros = u4 ? gs->zeros : nullptr;
  a.x = static_cast<const uint16_t*>(X), a.c = C, a.d = D, a.bias = bias;
  a.ldw_bytes = ldw / 2, a.ld_scales = gs->ld_scales, a.ld_zeros = u4 ? gs->ld_zeros : 0;
  a.ldx = ldx, a.ldc = ldc, a.ldd = ldd;
  a.m = static_cast<int32_t>(m), a.n = static_cast<int32_t>(n), a.k = static_cast<int32_t>(k);
  a.groups = static_cast<int32_t>(groups), a.group_shift = shift;
  a.flip = dt->a == THL_I4X2 ? 0x88888888u : 0u;
  a.s_type = gs->type, a.c_type = dt->c, a.d_type = dt->d, a.bias_type = dt->bias;
  a.flags = static_cast<int32_t>(flags), a.alpha = alpha, a.beta = beta;
  const hipError_t e = dt->b == THL_BF16 ? launch_type<true>(a, e2m1 ? W_E2M1 : W_INT, stream)
                                         : launch_type<false>(a, e2m1 ? W_E2M1 : W_INT, stream);
  return e == hipSuccess ? THL_OK : THL_ERR_HIP;
}
