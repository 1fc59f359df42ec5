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

// The load of r has returned: nothing after this statement moves before it.
__device__ __forceinline__ void arrived(Raw8<2>& r) { asm volatile("" : "+v"(r.w)::"memory"); }
__device__ __forceinline__ void arrived(Raw8<4>& r) { asm volatile("" : "+v"(r.lo), "+v"(r.hi)::"memory"); }

// How a row of m features splits into runs of eight (chosen by the host).
// Loads are unconditional: behind branches the compiler waits for each before
// the next goes out.  So a lane past the row's end loads a run that exists,
// and settle() makes the values zero (or shifts a run that ends the row into
// place) when they are used.
enum : int {
  RUNS_WHOLE = 0,  // m % 8 == 0
  RUNS_RAGGED = 1, // m > 8: the last run is the row's last eight elements, shifted
  RUNS_TINY = 2    // m < 8: element by element
};
inline int runs_of(int64_t m) { return m % 8 == 0 ? RUNS_WHOLE : (m > 8 ? RUNS_RAGGED : RUNS_TINY); }

// Elements e .. e+7 of a row of m that starts at element `row` of a 16-bit or
// fp32 array, as loaded.  Read once: marked to leave L2 first.
template <int B, int RUNS>
__device__ __forceinline__ Raw8<B> load_run(const void* base, int64_t row, int e, int m) {
  Raw8<B> r;
  if constexpr (RUNS == RUNS_TINY) {
    if constexpr (B == 2) {
      const uint16_t* q = static_cast<const uint16_t*>(base) + row;
      unsigned u[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i < m) u[i / 2] |= static_cast<unsigned>(q[e + i]) << (16 * (i & 1));
#pragma unroll
      for (int i = 0; i < 4; ++i) r.w[i] = static_cast<int>(u[i]);
    } else if constexpr (B == 4) {
      const float* q = static_cast<const float*>(base) + row;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r.lo[i] = e + i < m ? q[e + i] : 0.0f;
        r.hi[i] = e + 4 + i < m ? q[e + 4 + i] : 0.0f;
      }
    }
  } else {
    const int64_t off = row + (e < m - 8 ? e : m - 8);
    if constexpr (B == 2) {
      r.w = __builtin_nontemporal_load(reinterpret_cast<const v4i_a2*>(static_cast<const uint16_t*>(base) + off));
    } else if constexpr (B == 4) {
      const v4f_a4* q = reinterpret_cast<const v4f_a4*>(static_cast<const float*>(base) + off);
      r.lo = __builtin_nontemporal_load(q);
      r.hi = __builtin_nontemporal_load(q + 1);
    }
  }
  return r;
}

// Words w[0 .. N-1] of elements of 32 / PER bits: element i becomes element
// i + sh, zeros behind the last; sh >= 8: all zeros.
template <int N, int PER>
__device__ __forceinline__ void shift_run(uint32_t (&w)[N], int sh) {
#pragma unroll
  for (int bit = 4; bit >= PER; bit /= 2) {  // whole words
    const int by = bit / PER;
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = (sh & bit) ? (i + by < N ? w[i + by] : 0u) : w[i];
  }
  if constexpr (PER == 2) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t t = __builtin_amdgcn_alignbit(i + 1 < N ? w[i + 1] : 0u, w[i], 16);
      w[i] = (sh & 1) ? t : w[i];
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = sh >= 8 ? 0u : w[i];
}

// The loaded run as elements e .. e+7, zeros past m.
template <int B, int RUNS>
__device__ __forceinline__ void settle(Raw8<B>& r, int e, int m) {
  if constexpr (RUNS == RUNS_TINY || B == 0) return;
  const int sh = RUNS == RUNS_WHOLE ? (e < m ? 0 : 8) : (e < m - 8 ? 0 : e - (m - 8));
  if constexpr (B == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = static_cast<uint32_t>(r.w[i]);
    if constexpr (RUNS == RUNS_RAGGED) {
      shift_run<4, 2>(w, sh);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = sh ? 0u : w[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = static_cast<int>(w[i]);
  } else if constexpr (B == 4) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = r.lo[i], hi = r.hi[i];
      w[i] = __builtin_bit_cast(uint32_t, lo);
      w[4 + i] = __builtin_bit_cast(uint32_t, hi);
    }
    if constexpr (RUNS == RUNS_RAGGED) {
      shift_run<8, 1>(w, sh);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = sh ? 0u : w[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.lo[i] = __builtin_bit_cast(float, w[i]);
      r.hi[i] = __builtin_bit_cast(float, w[4 + i]);
    }
  }
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

// Elements e .. e+7 of a vector of m whose type is only known at run time
// (uniform): two loads for fp32, the same one twice for 16 bits.
struct RawAny {
  v4i lo, hi;
};
template <int RUNS>
__device__ __forceinline__ RawAny load_any(const void* base, int type, int e, int m) {
  RawAny r;
  if constexpr (RUNS == RUNS_TINY) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = e + i < m ? __builtin_bit_cast(uint32_t, load_f(base, type, e + i)) : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.lo[i] = static_cast<int>(w[i]);
      r.hi[i] = static_cast<int>(w[4 + i]);
    }
  } else {
    const int off = e < m - 8 ? e : m - 8, size = type == DT_F32 ? 4 : 2;
    const uint8_t* p = static_cast<const uint8_t*>(base) + static_cast<int64_t>(off) * size;
    r.lo = *reinterpret_cast<const v4i_a2*>(p);
    r.hi = *reinterpret_cast<const v4i_a2*>(p + (type == DT_F32 ? 16 : 0));
  }
  return r;
}
template <int RUNS>
__device__ __forceinline__ void any_f8(const RawAny& r, int type, int e, int m, float (&v)[8]) {
  if (RUNS == RUNS_TINY || type == DT_F32) {
    Raw8<4> x;
    x.lo = __builtin_bit_cast(v4f, r.lo);
    x.hi = __builtin_bit_cast(v4f, r.hi);
    settle<4, RUNS>(x, e, m);
    to_f8<4>(x, false, v);
  } else {
    Raw8<2> x;
    x.w = r.lo;
    settle<2, RUNS>(x, e, m);
    to_f8<2>(x, type == DT_BF16, v);
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
    v[i] = sum16(v[i]);
    v[i] += __shfl_xor(v[i], 16);
    v[i] += __shfl_xor(v[i], 32);
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
typedef uint16_t u16_a1 __attribute__((aligned(1)));

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
