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
  uint8_t* packed;       // more than 16 tokens: X in operand order
  const void* c;
  void* d;
  const void* bias;
  int64_t ldw_bytes, ld_scales, ld_zeros, ldx, ldc, ldd;
  int32_t m, n, k, groups;
  int32_t group_shift;  // log2 of the group length (31: one group a feature)
  uint32_t s_bf;        // all ones when the scales are bf16
  int32_t c_type, d_type, bias_type, flags;
  float alpha, beta;
};

enum : int { W_U4 = 0, W_I4 = 1, W_E2M1 = 2 };

// Codes are integers (E2M1 codes otherwise).
constexpr bool is_int(int wt) { return wt != W_E2M1; }

template <bool BF>
__device__ __forceinline__ v4f mfma16(v4i a, v4i b, v4f c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0,
                                                   0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// A constant in a vector register: an instruction takes one scalar, and with
// both the mask and the base scalars a pair of codes would take two.
__device__ __forceinline__ uint32_t vector_constant(uint32_t c) {
  uint32_t v = c;
  asm("" : "+v"(v));
  return v;
}

// Eight codes as eight 16-bit floats.  Integer codes come out as 16 + q in
// the order 0, 4, 1, 5, 2, 6, 3, 7, E2M1 codes in order and times `scale`, a
// power of two.
template <int WT, bool BF>
__device__ __forceinline__ v4i decode(uint32_t v, float scale) {
  v4i o;
  if constexpr (WT == W_E2M1) {
    if constexpr (BF) {
      o[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 0));
      o[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 1));
      o[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 2));
      o[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 3));
    } else {
      o[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, scale, 0));
      o[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, scale, 1));
      o[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, scale, 2));
      o[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, scale, 3));
    }
  } else {
    // bf16: 16.0 = 0x4180, units at mantissa bit 3; fp16: 0x4c00, bit 6.
    // (v & mask) ^ base: a signed code's top bit turned gives q + 8.
    constexpr uint32_t one = BF ? 0x41804180u : 0x4c004c00u, unit = BF ? 0x00080008u : 0x00400040u;
    constexpr uint32_t mask = unit * 15u, base = one | (WT == W_I4 ? unit * 8u : 0u);
    const uint32_t b = vector_constant(base);
    if constexpr (BF) {
      o[0] = static_cast<int>(((v << 3) & mask) ^ b);
      o[1] = static_cast<int>(((v >> 1) & mask) ^ b);
      o[2] = static_cast<int>(((v >> 5) & mask) ^ b);
      o[3] = static_cast<int>(((v >> 9) & mask) ^ b);
    } else {
      o[0] = static_cast<int>(((v << 6) & mask) ^ b);
      o[1] = static_cast<int>(((v << 2) & mask) ^ b);
      o[2] = static_cast<int>(((v >> 2) & mask) ^ b);
      o[3] = static_cast<int>(((v >> 6) & mask) ^ b);
    }
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

// Eight activations of which the first `valid` exist, the others zero.
__device__ __forceinline__ v4i load_x8(const uint16_t* p, int valid) {
  if (valid >= 8) return *reinterpret_cast<const v4i_a2*>(p);
  uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < valid) u[e / 2] |= static_cast<uint32_t>(p[e]) << (16 * (e & 1));
  return v4i{static_cast<int>(u[0]), static_cast<int>(u[1]), static_cast<int>(u[2]), static_cast<int>(u[3])};
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

// The scales (and zero points) of the GPU groups in a unit of 256 codes of
// one feature, as stored: two 16-bit scales or four E8M0 bytes a word.
// Groups past the last read as zero.
template <int WT, int GPU>
struct Groups {
  uint32_t s[WT == W_E2M1 ? GPU / 4 : (GPU + 1) / 2];
  uint32_t z[WT == W_U4 ? (GPU + 3) / 4 : 1];
};

typedef uint16_t u16_a1 __attribute__((aligned(1)));

// W words from any address.
template <int W>
__device__ __forceinline__ void words(const void* p, uint32_t* o) {
  if constexpr (W == 1) {
    o[0] = *static_cast<const u32_a1*>(p);
  } else if constexpr (W == 2) {
    const v2u_a1 v = *static_cast<const v2u_a1*>(p);
    o[0] = v[0], o[1] = v[1];
  } else {
    static_assert(W == 4, "one access");
    const v4i_a1 v = *static_cast<const v4i_a1*>(p);
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = static_cast<uint32_t>(v[q]);
  }
}

// A whole unit's, of the lane's own feature.
template <int WT, int GPU>
__device__ __forceinline__ void load_groups(const W4Args& a, int64_t srow, int64_t zrow, int u, Groups<WT, GPU>& o) {
  const int first = static_cast<int>((256 * static_cast<int64_t>(u)) >> a.group_shift);
  if constexpr (WT == W_E2M1) {
    words<GPU / 4>(static_cast<const uint8_t*>(a.scales) + srow + first, o.s);
  } else {
    const uint16_t* s = static_cast<const uint16_t*>(a.scales) + srow + first;
    if constexpr (GPU == 1)
      o.s[0] = s[0];
    else
      words<GPU / 2>(s, o.s);
  }
  if constexpr (WT == W_U4) {
    const uint8_t* z = a.zeros + zrow + first;
    if constexpr (GPU == 1)
      o.z[0] = z[0];
    else if constexpr (GPU == 2)
      o.z[0] = *reinterpret_cast<const u16_a1*>(z);
    else
      words<GPU / 4>(z, o.z);
  }
}
// Those of the partial unit at K's end.
template <int WT, int GPU>
__device__ __forceinline__ void load_groups_end(const W4Args& a, int64_t srow, int64_t zrow, int u,
                                                Groups<WT, GPU>& o) {
  const int first = static_cast<int>((256 * static_cast<int64_t>(u)) >> a.group_shift);
  for (uint32_t& v : o.s) v = 0;
  for (uint32_t& v : o.z) v = 0;
#pragma unroll
  for (int q = 0; q < GPU; ++q) {
    if (first + q >= a.groups) continue;
    if constexpr (WT == W_E2M1)
      o.s[q / 4] |= static_cast<uint32_t>(static_cast<const uint8_t*>(a.scales)[srow + first + q]) << (8 * (q & 3));
    else
      o.s[q / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(a.scales)[srow + first + q]) << (16 * (q & 1));
    if constexpr (WT == W_U4) o.z[q / 4] |= static_cast<uint32_t>(a.zeros[zrow + first + q]) << (8 * (q & 3));
  }
}

// Lane group j's value in all four lane groups (of 16 lanes), j = 0 .. 3.
__device__ __forceinline__ void spread(uint32_t v, uint32_t (&o)[4]) {
  typedef unsigned v2 __attribute__((ext_vector_type(2)));
  const v2 h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  const v2 a = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
  const v2 b = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
  o[0] = a[0], o[1] = a[1], o[2] = b[0], o[3] = b[1];
}

// A scale as stored (its low 8 or 16 bits) in fp32.
template <int WT>
__device__ __forceinline__ float scale_of(const W4Args& a, uint32_t b) {
  if constexpr (WT == W_E2M1) {
    // E8M0: 2^(b - 127), 2^-127 a subnormal, 255 NaN
    return __builtin_bit_cast(float, b == 255 ? 0x7fc00000u : (b == 0 ? 0x00400000u : b << 23));
  } else {
    const float f = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(b)));
    return __builtin_bit_cast(float, bsel(a.s_bf, b << 16, __builtin_bit_cast(uint32_t, f)));
  }
}
// Scale q of the unit.
template <int WT, int GPU>
__device__ __forceinline__ float group_scale(const W4Args& a, const Groups<WT, GPU>& o, int q) {
  if constexpr (WT == W_E2M1)
    return scale_of<WT>(a, (o.s[q / 4] >> (8 * (q & 3))) & 255u);
  else
    return scale_of<WT>(a, (o.s[q / 2] >> (16 * (q & 1))) & 0xffffu);
}
// 16 + the zero point of group q (8 for signed codes, decoded as q + 8).
template <int WT, int GPU>
__device__ __forceinline__ float group_offset(const Groups<WT, GPU>& o, int q) {
  if constexpr (WT == W_U4) return static_cast<float>(16u + ((o.z[q / 4] >> (8 * (q & 3))) & 255u));
  return 24.0f;
}

// 16 bytes of codes of which `left` exist; the others read as zero.
__device__ __forceinline__ void load_codes_at(const uint8_t* p, int64_t left, v4i& o) {
  o = v4i{0, 0, 0, 0};
  uint32_t part = 0;
#pragma unroll
  for (int q = 0; q < 3; ++q)
    if (left > 0 && left < 16 && q < (left & 3)) part |= static_cast<uint32_t>(p[(left & 12) + q]) << (8 * q);
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    if (4 * d + 4 <= left)
      o[d] = static_cast<int>(*reinterpret_cast<const u32_a1*>(p + 4 * d));
    else if (4 * d < left)
      o[d] = static_cast<int>(part);
  }
}
// load_codes of the partial unit at K's end.
__device__ __forceinline__ void load_codes_end(const W4Args& a, const uint8_t* row, int u, int g, v4i (&o)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t at = 128 * static_cast<int64_t>(u) + 64 * h + 16 * g;
    load_codes_at(row + at, ((static_cast<int64_t>(a.k) + 1) >> 1) - at, o[h]);
  }
}

// One tile's sums of a group leave under its scale.
template <int WT>
__device__ __forceinline__ void leave(v4f& tot, const v4f& acc, const v4f& xs, float scale, float offset) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    float v = acc[r];
    if constexpr (is_int(WT)) v -= offset * xs[r];
    tot[r] += scale * v;
  }
  // here, and not where the totals are next used: until then every group's
  // sums would stay in registers
  asm volatile("" : "+v"(tot));
}

template <bool BF>
__device__ __forceinline__ v4i ones() {
  const int o = BF ? 0x3f803f80 : 0x3c003c00;
  return v4i{o, o, o, o};
}

// The epilogue of one product, if there is such a feature and token.
__device__ __forceinline__ void store_result(const W4Args& a, float v, int64_t i, int64_t j) {
  if (i >= a.m || j >= a.n) return;
  v *= a.alpha;
  if (nonzero_f32(a.beta)) v += a.beta * load_f(a.c, a.c_type, j * a.ldc + i);
  if (a.flags & EPI_BIAS) v += load_f(a.bias, a.bias_type, i);
  v = activate(v, a.flags);
  const int64_t at = j * a.ldd + i;
  if (a.d_type == THL_F32)
    static_cast<float*>(a.d)[at] = v;
  else if (a.d_type == THL_F16)
    static_cast<_Float16*>(a.d)[at] = static_cast<_Float16>(v);
  else
    static_cast<__bf16*>(a.d)[at] = static_cast<__bf16>(v);
}

// Sums of TILE = tiles * 256 values over the wavefronts, in wavefront order,
// and the epilogue.  Value q of `part` is register r, lane l of tile (b, t).
template <int MT, int NB>
__device__ __forceinline__ void finish(const W4Args& a, const float* part, int waves, int i0, int j0) {
  constexpr int TILE = NB * MT * 256;
  for (int q = static_cast<int>(threadIdx.x); q < TILE; q += static_cast<int>(blockDim.x)) {
    const int l = q & 63, r = (q >> 6) & 3, t = (q >> 8) % MT, b = (q >> 8) / MT;
    const int i = i0 + 16 * b + (l & 15), j = j0 + 16 * t + 4 * r + (l >> 4);
    float v = part[q];
    for (int s = 1; s < waves; ++s) v += part[s * TILE + q];
    store_result(a, v, i, j);
  }
}

// ---- up to four tokens
// No matrix cores: a lane takes 32 consecutive codes of a row, the lanes of a
// wavefront a run of 2,048 codes (1 KB), so that loads are whole lines in lane
// order, and its 32 activations a token stay in registers while the wavefront
// goes down the rows, four at a time.  Two products an instruction (exact,
// summed in fp32), one scale a lane, and the lanes' sums added in a fixed
// order: four rows' trees share their first two levels.  The wavefronts of a
// workgroup split K `ks` ways, and the rows otherwise.
//
// Matrix-core operands would have neighbouring lanes read different rows: one
// cache access a lane instead of one for four (m = 28672, k = 8192, n = 1,
// signed codes in groups of 128: 36 us that way).
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

template <bool BF>
__device__ __forceinline__ float dot2(int x, int w, float c) {
  if constexpr (BF)
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2bf, x), __builtin_bit_cast(v2bf, w), c, false);
  else
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(v2h, x), __builtin_bit_cast(v2h, w), c, false);
}

// The sums of four values over the 64 lanes: lanes 16 g .. 16 g + 15 get that
// of value (g & 1) * 2 + (g >> 1).
__device__ __forceinline__ float sum_rows(const float (&v)[4]) {
  typedef unsigned v2 __attribute__((ext_vector_type(2)));
  auto halves = [](float x, float y) {  // lanes 0 .. 31: x of both halves; 32 .. 63: y
    const v2 p = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, y),
                                                  false, false);
    const unsigned lo = p[0], hi = p[1];
    return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
  };
  const float a = halves(v[0], v[1]), b = halves(v[2], v[3]);
  const v2 q =
      __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b), false, false);
  const unsigned lo = q[0], hi = q[1];
  return sum16(__builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi));
}

constexpr int kOneWaves = 8;

// TAIL: K is not whole pieces of 32 codes.
template <int WT, bool BF, int NT, bool TAIL>
__global__ void __launch_bounds__(kOneWaves * 64) w4_one_kernel(W4Args a, int ks) {
  __shared__ float part[2][kOneWaves][4][NT];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kw = wave & (ks - 1), rg = wave / ks, groups_of_rows = kOneWaves / ks;
  const int rows = 4 * groups_of_rows;  // a workgroup's rows at a time
  const int pieces = a.k >> 5, slices = (pieces + 63) >> 6;
  const int blocks = (a.m + rows - 1) / rows, step = static_cast<int>(gridDim.x);

  // This lane's activations of a slice, and their sum.  Lanes past K's whole
  // pieces hold zeros.
  int x[NT][16];
  float xs[NT];
  auto load_x = [&](int slice) {
    const int piece = 64 * slice + lane;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int64_t at = static_cast<int64_t>(t < a.n ? t : a.n - 1) * a.ldx + 32 * static_cast<int64_t>(piece);
      xs[t] = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const Raw8<2> r{load_x8(a.x + at + 8 * q, piece < pieces ? 8 : 0)};
        const v4i o = in_order<WT>(r.w);
#pragma unroll
        for (int d = 0; d < 4; ++d) x[t][4 * q + d] = o[d];
        if constexpr (is_int(WT)) {
          float f[8];
          to_f8<2>(r, BF, f);
#pragma unroll
          for (int d = 0; d < 8; ++d) xs[t] += f[d];
        }
      }
    }
  };

  struct Rows {
    v4i w[4];
    uint32_t s[4], z[4];
  } ring[2];
  // The next (block of rows, slice of K) to load.  Every load is issued
  // whatever the position, of rows and pieces that exist: with loads behind
  // branches the compiler waits for all of them at each use.
  int l_block = static_cast<int>(blockIdx.x), l_slice = kw;
  auto load_next = [&](Rows& o) {
    int piece = 64 * l_slice + lane;
    piece = piece < pieces ? piece : 0;
    const int group = static_cast<int>((32 * static_cast<int64_t>(piece)) >> a.group_shift);
    const int64_t r0 = static_cast<int64_t>(l_block) * rows + 4 * rg;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t i = r0 + r < a.m ? r0 + r : static_cast<int64_t>(a.m) - 1;
      o.w[r] = __builtin_nontemporal_load(
          reinterpret_cast<const v4i_a1*>(a.w + i * a.ldw_bytes + 16 * static_cast<int64_t>(piece)));
      if constexpr (WT == W_E2M1)
        o.s[r] = (static_cast<const uint8_t*>(a.scales) + i * a.ld_scales)[group];
      else
        o.s[r] = (static_cast<const uint16_t*>(a.scales) + i * a.ld_scales)[group];
      if constexpr (WT == W_U4) o.z[r] = (a.zeros + i * a.ld_zeros)[group];
    }
    l_slice += ks;
    if (l_slice >= slices) {
      l_slice = kw;
      l_block += step;
    }
  };

  float sum[NT][4] = {};
  auto use = [&](const Rows& o, bool live) {
    const uint32_t keep = live ? ~0u : 0u;  // lanes past K: a scale of zero
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float d[NT] = {};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const v4i w = decode<WT, BF>(static_cast<uint32_t>(o.w[r][q]), 1.0f);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int e = 0; e < 4; ++e) d[t] = dot2<BF>(x[t][4 * q + e], w[e], d[t]);
        }
      }
      const float scale = scale_of<WT>(a, o.s[r] & keep);
      const float offset = WT == W_U4 ? static_cast<float>(16u + o.z[r]) : 24.0f;
#pragma unroll
      for (int t = 0; t < NT; ++t) sum[t][r] += scale * (is_int(WT) ? d[t] - offset * xs[t] : d[t]);
    }
  };

  // The last, partial piece of K: a code a lane.
  auto use_tail = [&](int block) {
    const int64_t at = 32 * static_cast<int64_t>(pieces) + lane;
    if (at >= a.k) return;
    const int group = static_cast<int>(at >> a.group_shift);
    for (int r = 0; r < 4; ++r) {
      const int64_t i0 = static_cast<int64_t>(block) * rows + 4 * rg + r, i = i0 < a.m ? i0 : static_cast<int64_t>(a.m) - 1;
      const uint32_t q = (a.w[i * a.ldw_bytes + (at >> 1)] >> (4 * (at & 1))) & 15u;
      uint32_t s;
      float v;
      if constexpr (WT == W_E2M1) {
        s = (static_cast<const uint8_t*>(a.scales) + i * a.ld_scales)[group];
        // the magnitude bits as an fp32's, times 2^126
        v = __builtin_bit_cast(float, ((q & 7u) << 22) | ((q & 8u) << 28)) * 0x1p126f;
      } else {
        s = (static_cast<const uint16_t*>(a.scales) + i * a.ld_scales)[group];
        v = WT == W_U4 ? static_cast<float>(q) - static_cast<float>((a.zeros + i * a.ld_zeros)[group])
                       : static_cast<float>(static_cast<int>(q ^ 8u) - 8);
      }
      const float scale = scale_of<WT>(a, s);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int64_t j = t < a.n ? t : a.n - 1;
        const float xv = load_f(a.x, BF ? DT_BF16 : DT_F16, j * a.ldx + at);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e == r) sum[t][e] += scale * (v * xv);
      }
    }
  };

  int block = static_cast<int>(blockIdx.x), slice = kw, parity = 0;
  const bool one_slice = kw + ks >= slices;
  if (pieces > 0) {
    load_next(ring[0]);
    load_x(kw);
  }
  while (block < blocks) {
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      if (block >= blocks) break;
      if (pieces > 0) {
        load_next(ring[d ^ 1]);
        if (!one_slice) load_x(slice);
        use(ring[d], 64 * slice + lane < pieces);
      }
      slice += ks;
      if (slice < slices) continue;
      // these rows' end
      slice = kw;
      if (TAIL && kw == 0) use_tail(block);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float v = sum_rows(sum[t]);
        const int g = lane >> 4;
        if ((lane & 15) == 0) part[parity][wave][(g & 1) * 2 + (g >> 1)][t] = v;
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[t][r] = 0.0f;
      }
      __syncthreads();  // (the sums before the last have long been read)
      if (tid < rows * NT) {
        const int t = tid / rows, row = tid - t * rows;
        float v = 0.0f;
        for (int w = 0; w < ks; ++w) v += part[parity][(row >> 2) * ks + w][row & 3][t];
        store_result(a, v, static_cast<int64_t>(block) * rows + row, t);
      }
      parity ^= 1;
      block += step;
    }
  }
}

// ---- more tokens
// A wavefront takes 32 features and all of the workgroup's 16 MT tokens over
// its share of K: a weight is decoded once for all of them, an activation
// fragment serves both feature tiles.  Every wavefront reads every
// activation of its units, from L2: read where they lie, 16 rows of 64 bytes
// an instruction, they would set the pace (8192 x 48 x 8192 on E2M1: 33 us).
// So a first kernel writes them in operand order, a fragment's 64 lanes side
// by side, padded with zeros to whole units and tiles.

// Fragment (tile, unit, step): 64 pieces of eight activations, lane l's at
// 16 l bytes, for row l % 16 of the tile and lane group l / 16.
__device__ __forceinline__ int64_t fragment(int64_t tile, int64_t units, int64_t u, int step) {
  return ((tile * units + u) * 8 + step) * 64;
}

// One workgroup per unit and tile: 16 tokens x 256 K.
template <int WT>
__global__ void __launch_bounds__(256) w4_pack_kernel(W4Args a, int turned) {
  const int64_t u = blockIdx.x, tile = blockIdx.y, units = gridDim.x;
  v4i* out = reinterpret_cast<v4i*>(a.packed);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int p = static_cast<int>(threadIdx.x) + 256 * q, kp = p & 31, row = p >> 5;
    const int64_t k0 = 256 * u + 8 * kp, j = 16 * tile + 4 * (row & 3) + (row >> 2);
    v4i x = {0, 0, 0, 0};
    if (j < a.n && k0 < a.k) x = load_x8(a.x + j * a.ldx + k0, a.k - k0 < 8 ? static_cast<int>(a.k - k0) : 8);
    const int h = kp >> 4, hi = (kp >> 2) & 3, lo = kp & 3;
    out[fragment(tile, units, u, 4 * h + (turned ? hi : lo)) + 16 * (turned ? lo : hi) + row] = in_order<WT>(x);
  }
}

template <int WT, bool BF, int GPU, int MT, int NB>
__global__ void __launch_bounds__(512) w4_many_kernel(W4Args a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t area[];  // the codes of a unit by wavefront, then the sums
  constexpr int LEN = 256 / GPU;
  constexpr bool TURN = LEN < 128, FOLD = WT == W_E2M1 && BF;
  constexpr int RING = MT == 4 && !FOLD ? 4 : 8;  // steps of activations on their way (registers allow)
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int waves = static_cast<int>(blockDim.x) >> 6;
  const int col = lane & 15, g = lane >> 4;
  const int i0 = static_cast<int>(blockIdx.x) * 16 * NB, j0 = static_cast<int>(blockIdx.y) * 16 * MT;
  const int units = static_cast<int>((static_cast<int64_t>(a.k) + 255) >> 8), whole = a.k >> 8;

  // Codes are loaded along the rows, eight lanes a row's 128 bytes of a unit,
  // and turned into operand order through LDS (in operand order neighbouring
  // lanes hold different rows, and a load takes a cache access a lane instead
  // of one for four).  Position p of row r holds its 16-byte chunk p ^ (r % 8),
  // so that neither the writes nor the reads meet in a bank.
  // Features past m repeat the last one; nothing of them is stored.
  auto feature = [&](int i) { return static_cast<int64_t>(i < a.m ? i : a.m - 1); };
  const uint8_t* w[NB][2];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w[b][h] = a.w + feature(i0 + 16 * b + 8 * h + (lane >> 3)) * a.ldw_bytes + 16 * (lane & 7);
  v4i* const turned = reinterpret_cast<v4i*>(area) + wave * NB * 128;
  const int put = (lane >> 3) * 8 + ((lane & 7) ^ (lane >> 3));  // row lane / 8 of the first eight
  const int get = col * 8 + (g ^ (col & 7));                     // chunk g of row col (chunk 4 + g: ^ 4)
  // Scales: lane group g asks for tile g % NB of the unit g / NB turns on,
  // 4 / NB units at a time.
  constexpr int UNITS = 4 / NB;
  const int64_t gi = feature(i0 + 16 * (g % NB) + col);
  const int64_t srow = gi * a.ld_scales, zrow = gi * a.ld_zeros;
  const v4i* x = reinterpret_cast<const v4i*>(a.packed) + fragment(blockIdx.y * MT, units, 0, 0) + lane;

  v4i ring[2][NB][2];
  // Every load is issued whatever the position, of a unit that exists: with
  // loads behind branches the compiler waits for all of them at each use.
  auto load = [&](int v, v4i (&o)[NB][2]) {
    const int64_t u = v < whole ? v : whole - 1;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        o[b][h] = __builtin_nontemporal_load(reinterpret_cast<const v4i_a1*>(w[b][h] + 128 * u));
  };
  auto load_scales = [&](int v, Groups<WT, GPU>& o) {
    const int u = v + waves * (g / NB);
    load_groups<WT, GPU>(a, srow, zrow, u < whole ? u : whole - 1, o);
  };
  // Fragments of step s (0 .. 7) of unit u.
  v4i xa[RING][MT];
  auto fetch = [&](int v, int s, v4i (&o)[MT]) {
    const int u = v < units ? v : units - 1;
#pragma unroll
    for (int t = 0; t < MT; ++t) o[t] = x[fragment(t, units, u, s)];
  };

  v4f tot[NB][MT] = {}, acc[NB][MT] = {}, xs[MT] = {};
  // Unit u of this wavefront, its codes in operand order.
  auto use = [&](int u, const v4i (&codes)[NB][2], const Groups<WT, GPU> (&groups)[NB]) {
#pragma unroll
    for (int s8 = 0; s8 < 8; ++s8) {
      const int h = s8 >> 2, s = s8 & 3;
      // one step's operands at a time: mixing the steps costs more registers
      // than there are
      __builtin_amdgcn_sched_barrier(0);
      v4i (&xf)[MT] = xa[s8 % RING];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const v4i wq = TURN ? turn(codes[b][h]) : codes[b][h];
        const uint32_t c = static_cast<uint32_t>(wq[s]);
        const v4i wf = decode<WT, BF>(c, FOLD ? group_scale<WT, GPU>(a, groups[b], s8) : 1.0f);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          if constexpr (FOLD)
            tot[b][t] = mfma16<BF>(xf[t], wf, tot[b][t]);
          else
            acc[b][t] = mfma16<BF>(xf[t], wf, acc[b][t]);
        }
      }
      if constexpr (is_int(WT)) {
#pragma unroll
        for (int t = 0; t < MT; ++t) xs[t] = mfma16<BF>(xf[t], ones<BF>(), xs[t]);
      }
      // this step's slot takes the activations RING steps on
      fetch(s8 + RING < 8 ? u : u + waves, (s8 + RING) & 7, xf);
      const int done = 32 * (s8 + 1);
      if (FOLD) {
        // the scales are in the products
      } else if (TURN ? done % LEN == 0 : (s == 3 && (LEN == 128 || h == 1))) {
        const int q = (done - 1) / LEN;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float sv = group_scale<WT, GPU>(a, groups[b], q);
          const float ov = group_offset<WT, GPU>(groups[b], q);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            leave<WT>(tot[b][t], acc[b][t], xs[t], sv, ov);
            acc[b][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
          }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) xs[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      }
    }
  };

  auto turn_and_use = [&](int u, const v4i (&in)[NB][2], const Groups<WT, GPU> (&groups)[NB]) {
    v4i codes[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h) turned[b * 128 + h * 64 + put] = in[b][h];
    __builtin_amdgcn_wave_barrier();  // a wavefront's LDS accesses run in order
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h) codes[b][h] = turned[b * 128 + (get ^ (4 * h))];
    __builtin_amdgcn_wave_barrier();
    use(u, codes, groups);
  };

  // The wavefronts take the units in turn.  Loads return in order, so a
  // unit's weights are asked for after the activations of the unit before:
  // those then do not wait for memory.
  if (wave < whole) {
    Groups<WT, GPU> asked;
    load_scales(wave, asked);
    load(wave, ring[0]);
#pragma unroll
    for (int s = 0; s < RING; ++s) fetch(wave, s, xa[s]);
    load(wave + waves, ring[1]);
    bool more = true;
    for (int u = wave; more;) {
      // the scales of the next UNITS units, one set of tiles a unit
      constexpr int SW = sizeof(asked.s) / 4, ZW = sizeof(asked.z) / 4;
      Groups<WT, GPU> groups[4];
#pragma unroll
      for (int q = 0; q < SW; ++q) {
        uint32_t o[4];
        spread(asked.s[q], o);
#pragma unroll
        for (int j = 0; j < 4; ++j) groups[j].s[q] = o[j];
      }
      if constexpr (WT == W_U4) {
#pragma unroll
        for (int q = 0; q < ZW; ++q) {
          uint32_t o[4];
          spread(asked.z[q], o);
#pragma unroll
          for (int j = 0; j < 4; ++j) groups[j].z[q] = o[j];
        }
      }
      load_scales(u + UNITS * waves, asked);
#pragma unroll
      for (int d = 0; d < UNITS; ++d) {
        Groups<WT, GPU> mine[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) mine[b] = groups[d * NB + b];
        turn_and_use(u, ring[d & 1], mine);
        load(u + 2 * waves, ring[d & 1]);
        u += waves;
        if (u >= whole) {
          more = false;
          break;
        }
      }
    }
  }
  if (whole < units && wave == whole % waves) {  // K's partial unit
    v4i codes[NB][2];
    Groups<WT, GPU> groups[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int64_t i = feature(i0 + 16 * b + col);
      load_codes_end(a, a.w + i * a.ldw_bytes, whole, g, codes[b]);
      load_groups_end<WT, GPU>(a, i * a.ld_scales, i * a.ld_zeros, whole, groups[b]);
    }
#pragma unroll
    for (int s = 0; s < RING; ++s) fetch(whole, s, xa[s]);
    use(whole, codes, groups);
  }

  float* const part = reinterpret_cast<float*>(area);  // [wavefront][NB][MT][4][64]
  __syncthreads();
  constexpr int TILE = NB * MT * 256;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wave * TILE + ((b * MT + t) * 4 + r) * 64 + lane] = tot[b][t][r];
  __syncthreads();
  finish<MT, NB>(a, part, waves, i0, j0);
}

template <int WT, bool BF, int NT>
hipError_t launch_one(W4Args& a, hipStream_t st) {
  // K split over as many wavefronts as it has slices; then workgroups for
  // two a CU, each with the same number of row blocks
  const int64_t slices = (static_cast<int64_t>(a.k) + 2047) / 2048;
  const void* f = a.k % 32 != 0 ? reinterpret_cast<const void*>(&w4_one_kernel<WT, BF, NT, true>)
                                : reinterpret_cast<const void*>(&w4_one_kernel<WT, BF, NT, false>);
  int ks = 1;
  while (ks < kOneWaves && 2 * ks <= slices) ks *= 2;
  const int rows = 4 * (kOneWaves / ks), blocks = (a.m + rows - 1) / rows;
  const int rounds = (blocks + 511) / 512, grid = (blocks + rounds - 1) / rounds;
  void* args[] = {&a, &ks};
  return hipLaunchKernel(f, dim3(static_cast<unsigned>(grid)),
                         dim3(kOneWaves * 64), args, 0, st);
}

// Tokens padded to whole tiles of the kernel that takes them.
int64_t padded_tokens(int64_t n) {
  const int64_t tile = n <= 16 ? 16 : (n <= 32 ? 32 : (n <= 48 ? 48 : 64));
  return (n + tile - 1) / tile * tile;
}

template <int WT, bool BF, int GPU, int MT, int NB>
hipError_t launch_many(W4Args& a, hipStream_t st) {
  const int64_t units = (static_cast<int64_t>(a.k) + 255) / 256, gy = padded_tokens(a.n) / (16 * MT);
  if (units > 0) {
    int turned = 256 / GPU < 128;
    void* args[] = {&a, &turned};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&w4_pack_kernel<WT>),
                                         dim3(static_cast<unsigned>(units), static_cast<unsigned>(gy * MT)), dim3(256),
                                         args, 0, st);
    if (e != hipSuccess) return e;
  }
  int waves = 8;
  while (waves > 1 && waves > units) waves /= 2;
  void* args[] = {&a};
  return hipLaunchKernel(reinterpret_cast<const void*>(&w4_many_kernel<WT, BF, GPU, MT, NB>),
                         dim3(static_cast<unsigned>((a.m + 16 * NB - 1) / (16 * NB)), static_cast<unsigned>(gy)), dim3(waves * 64), args,
                         static_cast<size_t>(waves) * NB * (MT > 2 ? MT : 2) * 1024, st);
}

// Two feature tiles a wavefront read each activation once for both; one
// where two would leave compute units without a workgroup.
template <int WT, bool BF, int GPU, int MT>
hipError_t launch_many(W4Args& a, hipStream_t st) {
  return a.m <= 4096 ? launch_many<WT, BF, GPU, MT, 1>(a, st) : launch_many<WT, BF, GPU, MT, 2>(a, st);
}

template <int WT, bool BF, int GPU>
hipError_t launch_tokens(W4Args& a, hipStream_t st) {
  if (a.n <= 16) return launch_many<WT, BF, GPU, 1>(a, st);
  if (a.n <= 32) return launch_many<WT, BF, GPU, 2>(a, st);
  if (a.n <= 48) return launch_many<WT, BF, GPU, 3, 2>(a, st);
  return launch_many<WT, BF, GPU, 4, 2>(a, st);
}

template <int WT, bool BF>
hipError_t launch_weights(W4Args& a, hipStream_t st) {
  if (a.n == 1) return launch_one<WT, BF, 1>(a, st);
  if (a.n == 2) return launch_one<WT, BF, 2>(a, st);
  if (a.n <= 4) return launch_one<WT, BF, 4>(a, st);
  if constexpr (WT == W_E2M1) {
    return launch_tokens<WT, BF, 8>(a, st);
  } else {
    switch (a.group_shift) {
      case 5:
        return launch_tokens<WT, BF, 8>(a, st);
      case 6:
        return launch_tokens<WT, BF, 4>(a, st);
      case 7:
        return launch_tokens<WT, BF, 2>(a, st);
      default:
        return launch_tokens<WT, BF, 1>(a, st);
    }
  }
}

template <bool BF>
hipError_t launch_type(W4Args& a, thl_dtype w, hipStream_t st) {
  if (w == THL_E2M1X2) return launch_weights<W_E2M1, BF>(a, st);
  return w == THL_U4X2 ? launch_weights<W_U4, BF>(a, st) : launch_weights<W_I4, BF>(a, st);
}

constexpr int64_t kMaxTokens = INT64_C(1) << 19;  // tiles of 16 in a grid's rows

bool big(int64_t v) { return v > INT32_MAX; }
int64_t at_least_one(int64_t v) { return v > 1 ? v : 1; }
bool misaligned(const void* p, thl_dtype t) { return reinterpret_cast<uintptr_t>(p) % bytes_of(t, 1) != 0; }

}  // namespace
}  // namespace thl

using namespace thl;

extern "C" {

size_t thl_gemm_w4_workspace(int64_t n, int64_t k) {
  if (n <= 4 || n > kMaxTokens || k <= 0 || big(k)) return 0;
  return static_cast<size_t>(padded_tokens(n)) * static_cast<size_t>((k + 255) / 256) * 512;
}

thl_status thl_gemm_w4(int64_t m, int64_t n, int64_t k, const void* W, int64_t ldw,
                       const thl_group_scales* gs, const void* X, int64_t ldx, const void* C, int64_t ldc, void* D,
                       int64_t ldd, float alpha, float beta, const thl_dtypes* dt, const thl_epilogue* epi,
                       void* workspace, size_t workspace_bytes, struct ihipStream_t* stream) {
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
  if (e2m1 ? gs->type != THL_E8M0 : gs->type != THL_F16 && gs->type != THL_BF16) return THL_ERR_UNSUPPORTED;
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

  const size_t need = thl_gemm_w4_workspace(n, k);
  if (need && (!workspace || workspace_bytes < need)) return THL_ERR_INVALID;
  if (need && reinterpret_cast<uintptr_t>(workspace) % 16 != 0) return THL_ERR_MISALIGNED;

  // ---- overlap: D may alias C exactly; the workspace overlaps nothing
  const Range rd = matrix_range(D, dt->d, m, n, ldd);
  if (need) {
    const Range rp = vector_range(workspace, static_cast<int64_t>(need), 1);
    if (overlaps(rp, rd) || overlaps(rp, matrix_range(W, dt->a, k, m, ldw)) ||
        overlaps(rp, matrix_range(X, dt->b, k, n, ldx)) ||
        overlaps(rp, matrix_range(gs->scales, gs->type, groups, m, gs->ld_scales)) ||
        (u4 && overlaps(rp, matrix_range(gs->zeros, THL_I8, groups, m, gs->ld_zeros))) ||
        (beta != 0.0f && overlaps(rp, matrix_range(C, dt->c, m, n, ldc))) ||
        (has_bias && overlaps(rp, matrix_range(bias, dt->bias, m, 1, m))))
      return THL_ERR_INVALID;
  }
  if (beta != 0.0f && !(C == D && ldc == ldd && dt->c == dt->d) && overlaps(rd, matrix_range(C, dt->c, m, n, ldc)))
    return THL_ERR_INVALID;
  if (overlaps(rd, matrix_range(W, dt->a, k, m, ldw)) || overlaps(rd, matrix_range(X, dt->b, k, n, ldx)) ||
      overlaps(rd, matrix_range(gs->scales, gs->type, groups, m, gs->ld_scales)) ||
      (u4 && overlaps(rd, matrix_range(gs->zeros, THL_I8, groups, m, gs->ld_zeros))) ||
      (has_bias && overlaps(rd, matrix_range(bias, dt->bias, m, 1, m))))
    return THL_ERR_INVALID;

  W4Args a{};
  a.w = static_cast<const uint8_t*>(W), a.scales = gs->scales, a.zeros = u4 ? gs->zeros : nullptr;
  a.x = static_cast<const uint16_t*>(X), a.packed = static_cast<uint8_t*>(workspace), a.c = C, a.d = D, a.bias = bias;
  a.ldw_bytes = ldw / 2, a.ld_scales = gs->ld_scales, a.ld_zeros = u4 ? gs->ld_zeros : 0;
  a.ldx = ldx, a.ldc = ldc, a.ldd = ldd;
  a.m = static_cast<int32_t>(m), a.n = static_cast<int32_t>(n), a.k = static_cast<int32_t>(k);
  a.groups = static_cast<int32_t>(groups), a.group_shift = shift;
  a.s_bf = gs->type == THL_BF16 ? ~0u : 0u, a.c_type = dt->c, a.d_type = dt->d, a.bias_type = dt->bias;
  a.flags = static_cast<int32_t>(flags), a.alpha = alpha, a.beta = beta;
  const hipError_t e = dt->b == THL_BF16 ? launch_type<true>(a, dt->a, stream) : launch_type<false>(a, dt->a, stream);
  return e == hipSuccess ? THL_OK : THL_ERR_HIP;
}

}  // extern "C"
