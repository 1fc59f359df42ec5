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
// thread then holds 32 tokens of two neighbouring features.
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

// The bits of |v| order like |v|, infinity above every number and NaN above
// infinity: the largest of a block tells both its scale and whether it holds
// a NaN.
__device__ __forceinline__ uint32_t magnitude(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }

// A block's E8M0 code, and what its values are multiplied by: 0 for a block
// of zeros, 255 with a NaN in it (whose elements then are zeros).
__device__ __forceinline__ int block_scale(uint32_t most, int emax, float& inv) {
  if (most > 0x7f800000u) {
    inv = 0.0f;
    return 255;
  }
  const int code = mx_scale_code(__builtin_bit_cast(float, most), emax);
  inv = __builtin_bit_cast(float, static_cast<uint32_t>(254 - code) << 23);  // code <= 253: never subnormal
  return code;
}
// v times it: a NaN and its neighbours become zeros.
__device__ __forceinline__ float scaled(float v, float inv) { return inv != 0.0f ? v * inv : 0.0f; }

// Eight E2M1 codes of values already divided by their scale.
__device__ __forceinline__ uint32_t fp4_codes(const float (&q)[8]) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) w |= e2m1_code(q[i]) << (4 * i);
  return w;
}

// Eight values of a block's row to y at element `at`; `valid` of them exist.
__device__ __forceinline__ void store_elements(uint8_t* y, int64_t at, int type, const float (&v)[8], float inv,
                                               int valid) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = i < valid ? scaled(v[i], inv) : 0.0f;
  if (type == THL_E2M1X2)
    store_codes4(y + at / 2, fp4_codes(q), valid);
  else
    store_codes8(y + at, fp8_codes(q, type == THL_E4M3), valid);
}

__device__ __forceinline__ int emax_of(int type) { return type == THL_E2M1X2 ? 2 : (type == THL_E4M3 ? 8 : 15); }

// Eight features of a row, 0 .. 8 of which exist.
__device__ __forceinline__ void load_row8(const MxArgs& a, int64_t row, int e, int valid, float (&v)[8]) {
  if (valid > 0) {
    load8_f(a.x, a.x_type, row * a.ldx + e, valid < 8 ? valid : 8, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  }
}

// A row's block of four lanes: its elements and, by the first lane, its scale.
__device__ __forceinline__ void store_block(const MxArgs& a, int64_t row, int e, int valid, const float (&v)[8]) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = max(most, magnitude(v[i]));
  most = max(most, static_cast<uint32_t>(__shfl_xor(static_cast<int>(most), 1)));
  most = max(most, static_cast<uint32_t>(__shfl_xor(static_cast<int>(most), 2)));
  if (valid <= 0) return;
  float inv;
  const int code = block_scale(most, emax_of(a.y_type), inv);
  store_elements(a.y, row * a.ldy + e, a.y_type, v, inv, valid);
  if ((e & 31) == 0) a.sf[row * a.ld_sf + (e >> 5)] = static_cast<uint8_t>(code);
}

// Blocks along the features only.  A row goes to 4 to 64 lanes.
__global__ void __launch_bounds__(256) mx_rows_kernel(MxArgs a) {
  const int lanes = 1 << a.lanes_shift, tid = static_cast<int>(threadIdx.x);
  const int64_t chunks = (static_cast<int64_t>(a.m) + 8 * lanes - 1) >> (a.lanes_shift + 3);
  const int at_once = 256 >> a.lanes_shift;  // rows
  const int64_t groups = (a.n + at_once - 1) / at_once, units = groups * chunks;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t group = u / chunks, chunk = u - group * chunks;
    const int64_t row = group * at_once + (tid >> a.lanes_shift);
    const int64_t e64 = chunk * 8 * lanes + 8 * (tid & (lanes - 1));
    const int e = static_cast<int>(e64), valid = row < a.n ? static_cast<int>(e64 < a.m ? a.m - e64 : 0) : 0;
    float v[8];
    load_row8(a, row, e, valid, v);
    store_block(a, row, e, valid, v);
  }
}

constexpr int kTile = 128;

// Blocks along the tokens, and along the features if y is given.
__global__ void __launch_bounds__(256) mx_turn_kernel(MxArgs a) {
  __shared__ float tile[32][kTile];
  const int tid = static_cast<int>(threadIdx.x);
  const int64_t tiles_m = (static_cast<int64_t>(a.m) + kTile - 1) / kTile, tiles_n = (a.n + 31) / 32;
  for (int64_t u = blockIdx.x; u < tiles_m * tiles_n; u += gridDim.x) {
    const int64_t tn = u / tiles_m, tm = u - tn * tiles_m;
    const int e = static_cast<int>(tm) * kTile + 8 * (tid & 15);
    for (int i = 0; i < 2; ++i) {
      const int r = (tid >> 4) + 16 * i;
      const int64_t row = 32 * tn + r;
      const int valid = row < a.n ? (e < a.m ? a.m - e : 0) : 0;
      float v[8];
      load_row8(a, row, e, valid, v);
      if (a.y) store_block(a, row, e, valid, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) tile[r][8 * (tid & 15) + k] = v[k];
    }
    __syncthreads();
    const int64_t f = tm * kTile + (tid >> 1);  // two threads a feature, 16 tokens each
    {
      float v[16];
      uint32_t most = 0;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        v[k] = tile[16 * (tid & 1) + k][tid >> 1];
        most = max(most, magnitude(v[k]));
      }
      most = max(most, static_cast<uint32_t>(__shfl_xor(static_cast<int>(most), 1)));
      if (f < a.m) {
        float inv;
        const int code = block_scale(most, emax_of(a.y_type), inv);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t row = 32 * tn + 16 * (tid & 1) + 8 * h;
          float w[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) w[k] = v[8 * h + k];
          const int64_t left = a.n - row;
          if (left > 0) store_elements(a.yt, f * a.ldyt + row, a.y_type, w, inv, left < 8 ? static_cast<int>(left) : 8);
        }
        if ((tid & 1) == 0) a.sft[f * a.ld_sft + tn] = static_cast<uint8_t>(code);
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
  hipError_t e;
  if (YT) {
    e = launch(reinterpret_cast<const void*>(&mx_turn_kernel), (m + kTile - 1) / kTile * ((n + 31) / 32), a, stream);
  } else {
    a.lanes_shift = 2;
    while (a.lanes_shift < 6 && (8 << a.lanes_shift) < m) ++a.lanes_shift;
    const int64_t chunks = (m + (8 << a.lanes_shift) - 1) >> (a.lanes_shift + 3), rows = 256 >> a.lanes_shift;
    e = launch(reinterpret_cast<const void*>(&mx_rows_kernel), (n + rows - 1) / rows * chunks, a, stream);
  }
  return e == hipSuccess ? THL_OK : THL_ERR_HIP;
}

}  // extern "C"
