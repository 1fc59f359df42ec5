// mx.hip -- arrays to MX blocks: along the features (the rows' blocks), along
// the tokens (the columns' blocks, of the transposed array), or both in one
// read.
//
//   X = floor(log2 max|v|) - emax in [-127, 127],   element = rne(v / 2^X), clamped
//
// over each 32 consecutive values v, the rule of the products' MX output: the
// quotient by a power of two is exact, so an element rounds once.
//
// Bound by HBM: each value is read once.  A wavefront's lanes hold eight
// consecutive features each, four lanes a block of a row; for the columns'
// blocks a tile of 128 x 128 values turns through LDS as it was read, and a
// thread then holds 32 tokens of two neighbouring features.  16-bit values stay
// packed: magnitudes are compared two at a time, and E2M1 codes converted two at
// a time under their scale by the hardware's instruction.
//
// Measured: 2,048 x 8,192 bf16 values to E2M1 10.0 us (4.2 TB/s), 8,192 x 8,192
// both ways 48 us (4.3 TB/s; a large copy runs at 5.0), 1,531 x 5,003 fp32 values
// to E4M3 8.5 us (4.5 TB/s).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/thl.h"
#include "host_checks.hpp"
#include "rows.hpp"

namespace thl {
namespace {

struct MxArgs {
  const void* x;
  uint8_t* y;    // NULL: no blocks along the features
  uint8_t* sf;
  uint8_t* yt;   // NULL: no blocks along the tokens
  uint8_t* sft;
  int64_t ldx, ldy, ld_sf, ldyt, ld_sft;  // ldy, ldyt in elements
  int64_t n;
  int32_t m, x_type, y_type;
  int32_t lanes_shift;  // log2 of the lanes that share a row
};

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef uint16_t v2us __attribute__((ext_vector_type(2)));

enum : int { X_BF16 = 0, X_F16 = 1, X_F32 = 2 };

// Eight consecutive values as loaded.
template <int X>
struct Run {
  static constexpr int WORDS = X == X_F32 ? 8 : 4;
  uint32_t w[WORDS];
};

// The magnitudes' bits order like the magnitudes, infinity above every number
// and NaN above infinity: the largest of a block tells both its scale and
// whether it holds a NaN.  16-bit values two at a time.
template <int X>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  if constexpr (X == X_F32) {
    return max(a, b);
  } else {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(v2us, a), __builtin_bit_cast(v2us, b)));
  }
}
template <int X>
__device__ __forceinline__ uint32_t magnitude(uint32_t w) {
  return w & (X == X_F32 ? 0x7fffffffu : 0x7fff7fffu);
}
// A 16-bit magnitude's (low half) as fp32 bits.
template <int X>
__device__ __forceinline__ uint32_t as_f32(uint32_t m) {
  if constexpr (X == X_BF16) return m << 16;
  if constexpr (X == X_F16)
    return __builtin_bit_cast(uint32_t, static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(m))));
  return m;
}
// v of the lane next to this one, and of the one after that pair.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, true));
}

// A block's E8M0 code from the fp32 bits of its largest magnitude: the biased
// exponent less emax, 0 where that is negative (and for a block of zeros; a
// subnormal's floor(log2) is below -126), 255 with a NaN.
struct Scale {
  int code;
  float inv;    // 2^(127 - code), 0 with a NaN
  float value;  // 2^(code - 127) for code > 0
  __device__ __forceinline__ Scale(uint32_t most, int emax) {
    const int x = static_cast<int>(most >> 23) - emax;
    code = most > 0x7f800000u ? 255 : (x > 0 ? x : 0);
    inv = __builtin_bit_cast(float, code == 255 ? 0u : static_cast<uint32_t>(254 - code) << 23);
    value = __builtin_bit_cast(float, static_cast<uint32_t>(code) << 23);
  }
};

__device__ __forceinline__ int emax_of(int type) { return type == THL_E2M1X2 ? 2 : (type == THL_E4M3 ? 8 : 15); }

// v under the scale (a NaN and its neighbours become zeros).
__device__ __forceinline__ float under(float v, const Scale& s) { return s.inv != 0.0f ? v * s.inv : 0.0f; }

// The value of a 16-bit half.
template <int X>
__device__ __forceinline__ float value16(uint32_t w, int hi) {
  if constexpr (X == X_BF16) return __builtin_bit_cast(float, hi ? w & 0xffff0000u : w << 16);
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(hi ? w >> 16 : w)));
}

// The E2M1 codes of two values into byte SEL of `old`.  The conversion divides by
// the scale (exactly) and rounds once, to nearest even, larger magnitudes to 6.
// `w`: two 16-bit values; `tiny`: a scale of 2^-127, which as an fp32 is no normal
// number, so that the values are multiplied first.
template <int X, int SEL>
__device__ __forceinline__ uint32_t fp4_pair(uint32_t old, uint32_t w, const Scale& s, bool tiny) {
  if (tiny) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, value16<X>(w, 0) * s.inv, value16<X>(w, 1) * s.inv, 1.0f, SEL);
  }
  if constexpr (X == X_BF16)
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(v2bf, w), s.value, SEL);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(v2h, w), s.value, SEL);
}
template <int SEL>
__device__ __forceinline__ uint32_t fp4_pair(uint32_t old, float a, float b, const Scale& s) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a * s.inv, b * s.inv, 1.0f, SEL);
}
// Eight codes: of four words of two values, or of eight fp32 values.
template <int X>
__device__ __forceinline__ uint32_t fp4_codes(const uint32_t (&w)[Run<X>::WORDS], const Scale& s, bool tiny) {
  uint32_t o = 0;
  if constexpr (X == X_F32) {
    (void)tiny;
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __builtin_bit_cast(float, w[i]);
    o = fp4_pair<0>(o, f[0], f[1], s);
    o = fp4_pair<1>(o, f[2], f[3], s);
    o = fp4_pair<2>(o, f[4], f[5], s);
    o = fp4_pair<3>(o, f[6], f[7], s);
  } else {
    o = fp4_pair<X, 0>(o, w[0], s, tiny);
    o = fp4_pair<X, 1>(o, w[1], s, tiny);
    o = fp4_pair<X, 2>(o, w[2], s, tiny);
    o = fp4_pair<X, 3>(o, w[3], s, tiny);
  }
  return s.code == 255 ? 0u : o;
}
template <int X>
__device__ __forceinline__ v2u_a1 fp8_codes_of(const uint32_t (&w)[Run<X>::WORDS], const Scale& s, bool e4m3) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    q[i] = under(X == X_F32 ? __builtin_bit_cast(float, w[X == X_F32 ? i : 0]) : value16<X>(w[X == X_F32 ? 0 : i / 2], i & 1), s);
  return fp8_codes(q, e4m3);
}

// Eight elements to y at element `at`; `valid` of them exist (the values of the
// others are zeros).
template <int X, bool FP4>
__device__ __forceinline__ void store_elements(uint8_t* y, int64_t at, int type, const uint32_t (&w)[Run<X>::WORDS],
                                               const Scale& s, bool tiny, int valid) {
  if constexpr (FP4)
    store_codes4(y + at / 2, fp4_codes<X>(w, s, tiny), valid);
  else
    store_codes8(y + at, fp8_codes_of<X>(w, s, type == THL_E4M3), valid);
}

// Eight features of a row, all of them there.
template <int X>
__device__ __forceinline__ void load_run8(const MxArgs& a, int64_t row, int e, Run<X>& o) {
  if constexpr (X == X_F32) {
    const v4f_a4* p = reinterpret_cast<const v4f_a4*>(static_cast<const float*>(a.x) + row * a.ldx + e);
    const v4f_a4 lo = p[0], hi = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float l = lo[i], h = hi[i];
      o.w[i] = __builtin_bit_cast(uint32_t, l);
      o.w[4 + i] = __builtin_bit_cast(uint32_t, h);
    }
  } else {
    // (read once: marked to leave L2 first.  Not the two halves of eight fp32
    // values, which share lines: 10.9 us for 8.5)
    const v4i_a2 v = __builtin_nontemporal_load(
        reinterpret_cast<const v4i_a2*>(static_cast<const uint16_t*>(a.x) + row * a.ldx + e));
#pragma unroll
    for (int i = 0; i < 4; ++i) o.w[i] = static_cast<uint32_t>(v[i]);
  }
}
// The first `valid` of them, zeros for the others.
template <int X>
__device__ __forceinline__ void load_some8(const MxArgs& a, int64_t row, int e, int valid, Run<X>& o) {
  if (valid >= 8) {
    load_run8<X>(a, row, e, o);
    return;
  }
#pragma unroll
  for (int i = 0; i < Run<X>::WORDS; ++i) o.w[i] = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i >= valid) continue;
    if constexpr (X == X_F32)
      o.w[i] = static_cast<const uint32_t*>(a.x)[row * a.ldx + e + i];
    else
      o.w[i / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(a.x)[row * a.ldx + e + i]) << (16 * (i & 1));
  }
}

// A row's block of four lanes: its elements and, by the first lane, its scale.
template <int X, bool FP4>
__device__ __forceinline__ void store_block(const MxArgs& a, int64_t row, int e, int valid, const Run<X>& r) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < Run<X>::WORDS; ++i) most = larger<X>(most, magnitude<X>(r.w[i]));
  most = larger<X>(most, dpp<0xb1>(most));
  most = larger<X>(most, dpp<0x4e>(most));
  if constexpr (X != X_F32) most = max(most & 0xffffu, most >> 16);
  if (valid <= 0) return;
  const Scale s(as_f32<X>(most), emax_of(a.y_type));
  const bool tiny = __ballot(s.code == 0 && most != 0) != 0;
  store_elements<X, FP4>(a.y, row * a.ldy + e, a.y_type, r.w, s, tiny, valid);
  if ((e & 31) == 0) a.sf[row * a.ld_sf + (e >> 5)] = static_cast<uint8_t>(s.code);
}

// Blocks along the features only.  A row goes to 4 to 64 lanes, and a lane takes
// ROWS rows at a time, their loads together.
template <int X, bool FP4, int ROWS>
__global__ void __launch_bounds__(256) mx_rows_kernel(MxArgs a) {
  const int lanes = 1 << a.lanes_shift, tid = static_cast<int>(threadIdx.x);
  const int64_t chunks = (static_cast<int64_t>(a.m) + 8 * lanes - 1) >> (a.lanes_shift + 3);
  const int at_once = 256 >> a.lanes_shift;  // rows
  const int64_t groups = (a.n + ROWS * at_once - 1) / (ROWS * at_once), units = groups * chunks;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t group = u / chunks, chunk = u - group * chunks;
    const int64_t row0 = group * ROWS * at_once + (tid >> a.lanes_shift);
    const int64_t e64 = chunk * 8 * lanes + 8 * (tid & (lanes - 1));
    const int e = static_cast<int>(e64), there = e64 < a.m ? static_cast<int>(a.m - e64) : 0;
    Run<X> r[ROWS];
    // (loads behind branches are waited for one by one)
    if ((group + 1) * ROWS * at_once <= a.n && (chunk + 1) * 8 * lanes <= a.m) {
#pragma unroll
      for (int i = 0; i < ROWS; ++i) load_run8<X>(a, row0 + i * at_once, e, r[i]);
    } else {
#pragma unroll
      for (int i = 0; i < ROWS; ++i) load_some8<X>(a, row0 + i * at_once, e, row0 + i * at_once < a.n ? there : 0, r[i]);
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      store_block<X, FP4>(a, row0 + i * at_once, e, row0 + i * at_once < a.n ? there : 0, r[i]);
  }
}

constexpr int kTile = 128, kPanel = 8;

// Blocks along the tokens, and along the features if y is given: a tile of 128 x
// 128 values.  16 lanes hold a row's 128 features; behind LDS a lane holds
// two neighbouring features of 32 tokens, a wavefront's 64 lanes a whole row.
template <int X, bool FP4>
__global__ void __launch_bounds__(256) mx_turn_kernel(MxArgs a) {
  constexpr int WORDS = Run<X>::WORDS, ROW = WORDS * 16;  // words of a tile's row
  __shared__ __attribute__((aligned(16))) uint32_t tile[kTile * ROW];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
  const int64_t tiles_m = (static_cast<int64_t>(a.m) + kTile - 1) / kTile, tiles_n = (a.n + kTile - 1) / kTile;
  // Tiles next to one another share lines of yt along the tokens, and along the
  // features lines of y and of the scales (four bytes of a tile's row): to each
  // XCD a stretch of them (workgroups go round the eight), in panels of kPanel
  // tiles of features.  8,192 x 8,192 bf16 to E2M1 56 us in the workgroups' order,
  // 51 with stretches along the tokens, 48 with panels; 4,096 x 8,192 fp32 48 and
  // 43 with panels.
  const int64_t tiles = tiles_m * tiles_n, stretch = tiles / 8;
  for (int64_t u0 = blockIdx.x; u0 < tiles; u0 += gridDim.x) {
    const int64_t u = u0 < 8 * stretch ? (u0 & 7) * stretch + (u0 >> 3) : u0;
    const int64_t panel = u / (kPanel * tiles_n), in = u - panel * kPanel * tiles_n;
    const int64_t wide = tiles_m - panel * kPanel < kPanel ? tiles_m - panel * kPanel : kPanel;
    const int64_t tn = in / wide, tm = panel * kPanel + in - tn * wide;
    const int64_t row0 = kTile * tn + (tid >> 4);
    const int e = static_cast<int>(tm) * kTile + 8 * (tid & 15), there = e < a.m ? a.m - e : 0;
    Run<X> r[8];
    if ((tn + 1) * kTile <= a.n && (tm + 1) * kTile <= a.m) {
#pragma unroll
      for (int i = 0; i < 8; ++i) load_run8<X>(a, row0 + 16 * i, e, r[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) load_some8<X>(a, row0 + 16 * i, e, row0 + 16 * i < a.n ? there : 0, r[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (a.y) store_block<X, FP4>(a, row0 + 16 * i, e, row0 + 16 * i < a.n ? there : 0, r[i]);
      v4u* to = reinterpret_cast<v4u*>(tile + ((tid >> 4) + 16 * i) * ROW + WORDS * (tid & 15));
#pragma unroll
      for (int k = 0; k < WORDS / 4; ++k) to[k] = v4u{r[i].w[4 * k], r[i].w[4 * k + 1], r[i].w[4 * k + 2], r[i].w[4 * k + 3]};
    }
    __syncthreads();
    const uint32_t* from = tile + 32 * wave * ROW + (WORDS / 4) * lane;
    uint32_t c[2][X == X_F32 ? 32 : 16];  // two features: fp32 values, or two tokens' a word
    uint32_t most[2] = {0, 0};
    if constexpr (X == X_F32) {
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        typedef uint32_t v2u __attribute__((ext_vector_type(2)));
        const v2u v = *reinterpret_cast<const v2u*>(from + k * ROW);
        c[0][k] = v[0], c[1][k] = v[1];
#pragma unroll
        for (int h = 0; h < 2; ++h) most[h] = max(most[h], magnitude<X>(c[h][k]));
      }
    } else {
      uint32_t both = 0;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const uint32_t p = from[2 * k * ROW], q = from[(2 * k + 1) * ROW];
        both = larger<X>(both, larger<X>(magnitude<X>(p), magnitude<X>(q)));
        c[0][k] = __builtin_amdgcn_perm(q, p, 0x05040100u);
        c[1][k] = __builtin_amdgcn_perm(q, p, 0x07060302u);
      }
      most[0] = both & 0xffffu, most[1] = both >> 16;
    }
    // Codes go back through LDS, a feature's 128 tokens side by side, so that a
    // feature's lanes store neighbouring bytes (16 bytes a lane and feature took
    // 89 us for 8,192 x 8,192 bf16 values to E2M1 both ways).
    constexpr int BYTES = FP4 ? kTile / 2 : kTile, PITCH = BYTES + 16;  // of a feature
    uint8_t* out = reinterpret_cast<uint8_t*>(tile);
    uint8_t* scales = out + kTile * PITCH;
    __syncthreads();  // the tile has been read
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const Scale s(as_f32<X>(most[h]), emax_of(a.y_type));
      const bool tiny = __ballot(s.code == 0 && most[h] != 0) != 0;
      scales[4 * (2 * lane + h) + wave] = static_cast<uint8_t>(s.code);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t w[WORDS];
#pragma unroll
        for (int k = 0; k < WORDS; ++k) w[k] = c[h][WORDS * q + k];
        uint8_t* to = out + (2 * lane + h) * PITCH + (BYTES / 4) * wave + (BYTES / 16) * q;
        if constexpr (FP4)
          *reinterpret_cast<uint32_t*>(to) = fp4_codes<X>(w, s, tiny);
        else
          *reinterpret_cast<uint64_t*>(to) = __builtin_bit_cast(uint64_t, fp8_codes_of<X>(w, s, a.y_type == THL_E4M3));
      }
    }
    __syncthreads();
    const int tokens = a.n - kTile * tn < kTile ? static_cast<int>(a.n - kTile * tn) : kTile;
    const int bytes = FP4 ? (tokens + 1) / 2 : tokens, blocks = (tokens + 31) / 32;
#pragma unroll
    for (int k = 0; k < kTile * BYTES / 16 / 256; ++k) {
      const int piece = tid + 256 * k, at = 16 * (piece % (BYTES / 16)), row = piece / (BYTES / 16);
      const int64_t f = tm * kTile + row;
      if (f >= a.m || at >= bytes) continue;
      const v4i v = *reinterpret_cast<const v4i*>(out + row * PITCH + at);
      uint8_t* to = a.yt + f * (FP4 ? a.ldyt / 2 : a.ldyt) + (FP4 ? kTile / 2 : kTile) * tn + at;
      if (at + 16 <= bytes) {
        *reinterpret_cast<v4i_a1*>(to) = v;
      } else {
#pragma unroll
        for (int b = 0; b < 16; ++b)
          if (at + b < bytes) to[b] = static_cast<uint8_t>(static_cast<uint32_t>(v[b / 4]) >> (8 * (b & 3)));
      }
    }
    if (tid < kTile && tm * kTile + tid < a.m) {
      const uint32_t v = *reinterpret_cast<const uint32_t*>(scales + 4 * tid);
      uint8_t* to = a.sft + (tm * kTile + tid) * a.ld_sft + 4 * tn;
      if (blocks == 4) {
        *reinterpret_cast<u32_a1*>(to) = v;
      } else {
        for (int b = 0; b < blocks; ++b) to[b] = static_cast<uint8_t>(v >> (8 * b));
      }
    }
    __syncthreads();
  }
}

hipError_t launch(const void* f, int64_t units, MxArgs& a, hipStream_t st) {
  void* args[] = {&a};
  const int64_t grid = units < (1 << 20) ? units : (1 << 20);
  return hipLaunchKernel(f, dim3(static_cast<unsigned>(grid)), dim3(256), args, 0, st);
}
template <int X, bool FP4>
hipError_t launch(MxArgs& a, hipStream_t st) {
  if (a.yt)
    return launch(reinterpret_cast<const void*>(&mx_turn_kernel<X, FP4>),
                  (static_cast<int64_t>(a.m) + kTile - 1) / kTile * ((a.n + kTile - 1) / kTile), a, st);
  a.lanes_shift = 2;
  while (a.lanes_shift < 6 && (8 << a.lanes_shift) < a.m) ++a.lanes_shift;
  const int64_t chunks = (static_cast<int64_t>(a.m) + (8 << a.lanes_shift) - 1) >> (a.lanes_shift + 3);
  const int64_t rows = 256 >> a.lanes_shift, four = (a.n + 4 * rows - 1) / (4 * rows) * chunks;
  // Four rows at a time where there are workgroups for it: 2,048 x 8,192 bf16
  // values to E2M1 10.0 us, 19.7 one by one; 1,531 x 5,003 fp32 values to E4M3,
  // 960 workgroups, 10.9 and 8.8.
  if (four >= 2048) return launch(reinterpret_cast<const void*>(&mx_rows_kernel<X, FP4, 4>), four, a, st);
  return launch(reinterpret_cast<const void*>(&mx_rows_kernel<X, FP4, 1>), (a.n + rows - 1) / rows * chunks, a, st);
}
template <int X>
hipError_t launch(MxArgs& a, hipStream_t st) {
  return a.y_type == THL_E2M1X2 ? launch<X, true>(a, st) : launch<X, false>(a, st);
}

bool big(int64_t v) { return v > INT32_MAX; }
int64_t at_least_one(int64_t v) { return v > 1 ? v : 1; }

}  // namespace
}  // namespace thl

using namespace thl;

extern "C" {

thl_status thl_mx_quantize(int64_t m, int64_t n, const void* X, int64_t ldx, void* Y, int64_t ldy, uint8_t* sfy,
                           int64_t ld_sfy, void* YT, int64_t ldyt, uint8_t* sfyt, int64_t ld_sfyt, thl_dtype type_x,
                           thl_dtype type_y, struct ihipStream_t* stream) {
  // ---- arguments
  if (m < 0 || n < 0) return THL_ERR_INVALID;
  if (m > kMaxFeatures || big(n) || big(ldx) || big(ldy) || big(ld_sfy) || big(ldyt) || big(ld_sfyt))
    return THL_ERR_UNSUPPORTED;
  if (!is_float_io(type_x)) return THL_ERR_UNSUPPORTED;
  const bool fp4 = type_y == THL_E2M1X2;
  if (!fp4 && type_y != THL_E4M3 && type_y != THL_E5M2) return THL_ERR_UNSUPPORTED;
  if (ldx < at_least_one(m)) return THL_ERR_INVALID;
  if ((Y != nullptr) != (sfy != nullptr) || (YT != nullptr) != (sfyt != nullptr)) return THL_ERR_INVALID;
  if (Y && (ldy < at_least_one(m) || (fp4 && ldy % 2 != 0) || ld_sfy < (m + 31) / 32)) return THL_ERR_INVALID;
  if (YT && (ldyt < at_least_one(n) || (fp4 && ldyt % 2 != 0) || ld_sfyt < (n + 31) / 32)) return THL_ERR_INVALID;
  if (m == 0 || n == 0) return THL_OK;
  if (!Y && !YT) return THL_ERR_INVALID;
  if (!X) return THL_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(X) % bytes_of(type_x, 1) != 0) return THL_ERR_MISALIGNED;

  // ---- no output overlaps another array
  const Range all[] = {matrix_range(X, type_x, m, n, ldx), Y ? matrix_range(Y, type_y, m, n, ldy) : Range{},
                       Y ? matrix_range(sfy, THL_E8M0, (m + 31) / 32, n, ld_sfy) : Range{},
                       YT ? matrix_range(YT, type_y, n, m, ldyt) : Range{},
                       YT ? matrix_range(sfyt, THL_E8M0, (n + 31) / 32, m, ld_sfyt) : Range{}};
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < i; ++j)
      if (overlaps(all[i], all[j])) return THL_ERR_INVALID;

  MxArgs a{};
  a.x = X, a.y = static_cast<uint8_t*>(Y), a.sf = sfy, a.yt = static_cast<uint8_t*>(YT), a.sft = sfyt;
  a.ldx = ldx, a.ldy = ldy, a.ld_sf = ld_sfy, a.ldyt = ldyt, a.ld_sft = ld_sfyt;
  a.n = n, a.m = static_cast<int32_t>(m), a.x_type = type_x, a.y_type = type_y;
  const hipError_t e = type_x == THL_F32 ? launch<X_F32>(a, stream)
                                         : (type_x == THL_BF16 ? launch<X_BF16>(a, stream) : launch<X_F16>(a, stream));
  return e == hipSuccess ? THL_OK : THL_ERR_HIP;
}

}  // extern "C"
