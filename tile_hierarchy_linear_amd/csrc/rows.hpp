// rows.hpp -- device helpers of the per-token kernels (norm.hip, moe.hip):
// runs of eight consecutive features moved in one or two 16-byte accesses,
// and sums over the lanes that share a token.
#pragma once

#include "gemm_kernels.hpp"

namespace thl {

// Eight consecutive elements as loaded: 16-bit (B = 2) or fp32 (B = 4).
// Kept apart from their conversion, so that every load of a token is in
// flight before the first value is used.  B = 0: no such operand.
template <int B>
struct Raw8;
template <>
struct Raw8<0> {};
template <>
struct Raw8<2> {
  v4i w;
};
template <>
struct Raw8<4> {
  v4f lo, hi;
};

// Elements off .. off+valid-1 of a 16-bit or fp32 array (valid > 8 reads 8;
// what lies past them is not read and comes back as zero).
template <int B>
__device__ __forceinline__ Raw8<B> load_raw8(const void* base, int64_t off, int valid) {
  Raw8<B> r;
  if constexpr (B == 2) {
    const uint16_t* q = static_cast<const uint16_t*>(base) + off;
    if (valid >= 8) {
      r.w = *reinterpret_cast<const v4i_a2*>(q);
    } else {
      unsigned u[4] = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < valid) u[e / 2] |= static_cast<unsigned>(q[e]) << (16 * (e & 1));
      r.w = v4i{static_cast<int>(u[0]), static_cast<int>(u[1]), static_cast<int>(u[2]), static_cast<int>(u[3])};
    }
  } else if constexpr (B == 4) {
    const float* q = static_cast<const float*>(base) + off;
    if (valid >= 8) {
      r.lo = *reinterpret_cast<const v4f_a4*>(q);
      r.hi = *reinterpret_cast<const v4f_a4*>(q + 4);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        r.lo[e] = e < valid ? q[e] : 0.0f;
        r.hi[e] = 4 + e < valid ? q[4 + e] : 0.0f;
      }
    }
  }
  return r;
}

// The eight values in fp32 (`bf`: the 16-bit type is bf16, uniform).
template <int B>
__device__ __forceinline__ void to_f8(const Raw8<B>& r, bool bf, float (&v)[8]) {
  if constexpr (B == 2) {
    if (bf) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const unsigned u = static_cast<unsigned>(r.w[e / 2]);
        v[e] = __builtin_bit_cast(float, (e & 1) ? (u & 0xffff0000u) : (u << 16));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const unsigned u = static_cast<unsigned>(r.w[e / 2]);
        v[e] = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(u >> (16 * (e & 1)))));
      }
    }
  } else if constexpr (B == 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = r.lo[e];
      v[4 + e] = r.hi[e];
    }
  }
}

// v + v of the lane that `ctrl` (a DPP control) names.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(
                 float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// Sum over each aligned 16 lanes, in all of them: neighbours, pairs, then
// halves of eight and of sixteen mirrored.
__device__ __forceinline__ float sum16(float v) {
  v = dpp_add<0xb1>(v);
  v = dpp_add<0x4e>(v);
  v = dpp_add<0x141>(v);
  return dpp_add<0x140>(v);
}

// Sum of NV values over the WPR wavefronts of a workgroup (every lane gets
// it), always in the same order.  `slot` is an LDS area of NV * WPR floats
// that no lane of the workgroup may still be reading.
template <int NV, int WPR>
__device__ __forceinline__ void row_sum(float (&v)[NV], float* slot) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v[i] += __shfl_xor(v[i], d);
  }
  if constexpr (WPR > 1) {
    const int lane = static_cast<int>(threadIdx.x) & 63, wave = static_cast<int>(threadIdx.x) >> 6;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) slot[i * WPR + wave] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) t += slot[i * WPR + w];
      v[i] = t;
    }
  }
}

// Eight bytes at any address.
typedef uint32_t v2u_a1 __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));

// Codes of eight values (already divided by their scale) in E4M3 or E5M2:
// round to nearest even, magnitudes past the largest finite value clamped to
// it, NaN kept.
__device__ __forceinline__ v2u_a1 fp8_codes(const float (&v)[8], bool e4m3) {
  const float top = e4m3 ? 448.0f : 57344.0f;
  float t[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] = __builtin_fabsf(v[e]) > top ? __builtin_copysignf(top, v[e]) : v[e];
  v2u_a1 w;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int x;
    if (e4m3) {
      x = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * h], t[4 * h + 1], 0, false);
      x = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * h + 2], t[4 * h + 3], x, true);
    } else {
      x = __builtin_amdgcn_cvt_pk_bf8_f32(t[4 * h], t[4 * h + 1], 0, false);
      x = __builtin_amdgcn_cvt_pk_bf8_f32(t[4 * h + 2], t[4 * h + 3], x, true);
    }
    w[h] = static_cast<uint32_t>(x);
  }
  return w;
}

// The first `valid` (up to 8) of eight byte codes to p, or of eight 4-bit
// codes (the odd one out's high nibble zero).
__device__ __forceinline__ void store_codes8(uint8_t* p, v2u_a1 w, int valid) {
  if (valid >= 8) {
    *reinterpret_cast<v2u_a1*>(p) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < valid) p[e] = static_cast<uint8_t>(w[e / 4] >> (8 * (e & 3)));
  }
}
__device__ __forceinline__ void store_codes4(uint8_t* p, uint32_t w, int valid) {
  if (valid >= 8) {
    *reinterpret_cast<u32_a1*>(p) = w;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (2 * q < valid) p[q] = static_cast<uint8_t>(w >> (8 * q));
  }
}

}  // namespace thl
