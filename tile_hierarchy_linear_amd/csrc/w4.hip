// w4.hip -- the product of a few tokens with a matrix of 4-bit weights under
// group scales (16-bit activations, fp32 sums):
//
//   D(i,j) = act(alpha * sum_g s(i,g) * sum_{p in g} (q(i,p) - z(i,g)) X(p,j) + beta C(i,j) + bias_i)
//
// With a few tokens every weight is used a few times, so the product is a
// stream over the weights: bound by HBM.  One or two tokens are multiplied
// without matrix cores, a wavefront going down the rows (w4_one_kernel); more
// go to the matrix cores in workgroups of 128 features (w4_many_kernel).
// There tokens are the rows of the matrix-core tile, features its columns: a
// lane then holds sums of one feature, and needs one scale a group.
// Measured: one token, signed codes in groups of 128, m = 28672, k = 8192 23.6
// us (5.1 TB/s); 48 tokens, MX fp4 weights, m = k = 8192 21.9 us, of which 6
// would be the stream's.
//
// Codes become 16-bit floats without a conversion instruction: placed in the
// upper mantissa bits of 16.0 an unsigned code q reads as 16 + q, exactly, in
// bf16 and in fp16, two codes per shift and and-or.  The offset leaves with
// the zero point, (16 + z) * sum_p X(p,j), the sum of X over a group coming
// from a product with a matrix of ones in the same layout.  Signed codes are
// q + 8 with their top bit turned.  E2M1 codes are converted two at a time
// by the hardware's own instruction (exact), under their block scale where
// the weight then is a normal bf16.
//
// Every product is exact in fp32; sums within a group, its scaling and the
// sum over groups round in fp32 like any fp32 product does.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

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
  float* sums;           // K split over workgroups: the splits' n x m sums
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

constexpr int64_t kMaxTokens = INT64_C(1) << 21;  // workgroups of 64 in a grid's rows

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

// Whether any of four E8M0 scales may take an E2M1 code out of bf16's normal
// range: 253 .. 255 and 0 .. 4 (0 and 1 would do; this way three bits are
// dropped from b + 3, and a zero byte is what is looked for).
__device__ __forceinline__ bool extreme(uint32_t s) {
  const uint32_t v = (((s & 0x7f7f7f7fu) + 0x03030303u) ^ (s & 0x80808080u)) & 0xf8f8f8f8u;
  return ((v - 0x01010101u) & ~v & 0x80808080u) != 0;
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
// A lane's codes of the partial unit at K's end, in operand order.
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

// ---- one or two tokens
// No matrix cores: a lane takes 32 consecutive codes of a row, the lanes of a
// wavefront a run of 2,048 codes (1 KB), so that loads are whole lines in lane
// order, and its 32 activations a token stay in registers while the wavefront
// goes down the rows, four at a time.  Two products an instruction (exact,
// summed in fp32), one scale a lane, and the lanes' sums added in a fixed
// order: four rows' trees share their first two levels.  The wavefronts of a
// workgroup split K `ks` ways, and the rows otherwise; K's slices are of equal
// length, so that with 4,480 codes three wavefronts hold 48 pieces each.
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
__global__ void __launch_bounds__(kOneWaves * 64) w4_one_kernel(W4Args a, int ks, int span) {
  __shared__ float part[2][kOneWaves][4][NT];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rg = wave / ks, kw = wave - rg * ks, groups_of_rows = static_cast<int>(blockDim.x) / (64 * ks);
  const int rows = 4 * groups_of_rows;  // a workgroup's rows at a time
  // K in slices of `span` pieces, a multiple of `ks` slices of equal length
  const int pieces = a.k >> 5, slices = (pieces + span - 1) / span;
  const int blocks = (a.m + rows - 1) / rows, step = static_cast<int>(gridDim.x);

  // This lane's activations of a slice, and their sum.  Lanes past K's whole
  // pieces hold zeros.
  int x[NT][16];
  float xs[NT];
  auto load_x = [&](int slice) {
    const int piece = lane < span ? span * slice + lane : pieces;
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
    int piece = span * l_slice + (lane < span ? lane : 0);
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
        use(ring[d], lane < span && span * slice + lane < pieces);
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
// On the matrix cores.  A workgroup takes 128 features, its wavefronts four
// groups of 32 times KW units of K; a weight is decoded once for all of the
// workgroup's 16 MT tokens, and the activations of KW units go through LDS
// once for all features, in operand order, the next ones on their way in
// registers.  KW is 1 with one token tile, where a CU holds several small
// workgroups whose barriers do not meet (8192 x 16 x 8192, signed codes, groups
// of 128: 16.8 against 19.5 us), and 2 with more (28672 x 64 x 8192: 67.6
// against 71.3 us).  (Read by each wavefront for itself they set the pace: 8192 x
// 48 x 8192 moved 200 MB of activations from L2 and took 21 us.)  Where the
// features alone leave compute units idle, K is split over workgroups too;
// the splits' sums then go to the workspace and a second kernel adds them in
// order.
//
// Codes are loaded along the rows, eight lanes a row's 128 bytes of a unit,
// and turned into operand order through LDS (in operand order neighbouring
// lanes hold different rows, and a load takes a cache access a lane instead of
// one for four).
constexpr int kManyFeatures = 128;

// What the row of an activation piece is turned by in LDS, by the two-bit
// halves of its place along K: sixteen values, and between the lane groups
// that read together none that maps their rows onto one another.
__device__ __forceinline__ int swizzle(int high, int low) {
  return ((high & 1) << 3) | (((high ^ (high >> 1)) & 1) << 2) | low;
}

constexpr int units_at_once(int mt) { return mt == 1 ? 1 : 2; }

template <int WT, bool BF, int GPU, int MT>
__global__ void __launch_bounds__(256 * units_at_once(MT)) w4_many_kernel(W4Args a) {
  constexpr int NB = 2, FW = 4, KW = units_at_once(MT);
  constexpr int PASSES = 2 / KW;  // to move sixteen rows of 32 pieces
  constexpr int LEN = 256 / GPU;  // codes per group within a unit
  constexpr bool TURN = LEN < 128;
  // Activations: [buffer][unit][tile][step][lane group][row],
  // eight a piece; piece kp of a row's unit lies at row ^ swizzle, so that neither
  // the writes (along kp) nor the reads (along the rows) meet in a bank.
  __shared__ __attribute__((aligned(16))) v4i xbuf[2][KW * MT * 512];
  // Codes of a wavefront's unit: position p of row r holds its 16-byte chunk p ^ (r % 8).
  __shared__ __attribute__((aligned(16))) v4i turned[FW * KW][NB * 128];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fw = wave % FW, kw = wave / FW;
  const int col = lane & 15, g = lane >> 4;
  const int i0 = static_cast<int>(blockIdx.x) * kManyFeatures + 32 * fw, j0 = static_cast<int>(blockIdx.y) * 16 * MT;
  const int split = static_cast<int>(blockIdx.z), splits = static_cast<int>(gridDim.z);
  const int units = static_cast<int>((static_cast<int64_t>(a.k) + 255) >> 8), whole = a.k >> 8;
  const int sets = (whole + KW - 1) / KW;  // of KW units
  const int beg = static_cast<int>(static_cast<int64_t>(split) * sets / splits);
  const int len = static_cast<int>(static_cast<int64_t>(split + 1) * sets / splits) - beg;

  // Features past m and tokens past n repeat the last one; nothing of them
  // is stored.
  auto feature = [&](int i) { return static_cast<int64_t>(i < a.m ? i : a.m - 1); };
  const uint8_t* w[NB][2];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w[b][h] = a.w + feature(i0 + 16 * b + 8 * h + (lane >> 3)) * a.ldw_bytes + 16 * (lane & 7);
  const int put = (lane >> 3) * 8 + ((lane & 7) ^ (lane >> 3));  // row lane / 8 of the first eight
  const int get = col * 8 + (g ^ (col & 7));                     // chunk g of row col (chunk 4 + g: ^ 4)
  // Scales: lane group g asks for tile g % NB of its wavefront's unit g / NB
  // sets on, 4 / NB units at a time.
  constexpr int UNITS = 4 / NB;
  const int64_t gi = feature(i0 + 16 * (g % NB) + col);
  const int64_t srow = gi * a.ld_scales, zrow = gi * a.ld_zeros;

  // Unit k2 of this workgroup's q-th set.  Every load of the loop is issued
  // whatever the position, of a unit that exists: with loads behind branches
  // the compiler waits for all of them at each use.
  auto unit_of = [&](int q, int k2) {
    const int u = KW * (beg + (q < len ? q : len - 1)) + k2;
    return u < whole ? u : whole - 1;
  };
  v4i ring[2][NB][2];
  auto load = [&](int q, v4i (&o)[NB][2]) {
    const int64_t u = unit_of(q, kw);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        o[b][h] = __builtin_nontemporal_load(reinterpret_cast<const v4i_a1*>(w[b][h] + 128 * u));
  };
  auto load_scales = [&](int q, Groups<WT, GPU>& o) {
    load_groups<WT, GPU>(a, srow, zrow, unit_of(q + g / NB, kw), o);
  };

  // A lane moves piece kp of row `row` (and row + 8, in two passes) of every
  // unit and tile.  Row r of a
  // token tile is token 4 (r % 4) + r / 4, so that register r of lane group g
  // of the sums is token 4 r + g.
  const int kp = tid & 31, row = tid >> 5;
  auto place_at = [&](int r) {
    return ((kp >> 4) * 4 + (TURN ? (kp >> 2) & 3 : kp & 3)) * 64 + (TURN ? kp & 3 : (kp >> 2) & 3) * 16 +
           (r ^ swizzle(kp >> 2 & 3, kp & 3));
  };
  const uint16_t* x[MT][PASSES];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int h = 0; h < PASSES; ++h) {
      const int r = row + 8 * h, j = j0 + 16 * t + 4 * (r & 3) + (r >> 2);
      x[t][h] = a.x + static_cast<int64_t>(j < a.n ? j : a.n - 1) * a.ldx + 8 * kp;
    }
  v4i pre[KW][MT][PASSES];
  auto fetch = [&](int q) {
#pragma unroll
    for (int k2 = 0; k2 < KW; ++k2) {
      const int64_t u = unit_of(q, k2);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int h = 0; h < PASSES; ++h) pre[k2][t][h] = *reinterpret_cast<const v4i_a2*>(x[t][h] + 256 * u);
    }
  };
  auto place = [&](int buffer) {
#pragma unroll
    for (int k2 = 0; k2 < KW; ++k2)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int h = 0; h < PASSES; ++h)
          xbuf[buffer][(k2 * MT + t) * 512 + place_at(row + 8 * h)] = in_order<WT>(pre[k2][t][h]);
  };

  v4f tot[NB][MT] = {}, acc[NB][MT] = {}, xs[MT] = {};
  // One unit: its codes in operand order, its activations as unit k2 of a
  // buffer.  `fold`: E2M1 codes times their scale are bf16 numbers.
  auto use = [&](int buffer, int k2, const v4i (&codes)[NB][2], const Groups<WT, GPU> (&groups)[NB], auto fold) {
    constexpr bool FOLD = decltype(fold)::value;
    v4i wq[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h) wq[b][h] = TURN ? turn(codes[b][h]) : codes[b][h];
    const v4i* from = &xbuf[buffer][k2 * MT * 512 + g * 16];
    auto read = [&](int s8, v4i (&o)[MT]) {
      const int at = s8 * 64 + (col ^ (TURN ? swizzle(s8 & 3, g) : swizzle(g, s8 & 3)));
#pragma unroll
      for (int t = 0; t < MT; ++t) o[t] = from[t * 512 + at];
    };
    // Step s8's weights as 16-bit floats.
    auto weights = [&](int s8, v4i (&o)[NB]) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
        o[b] = decode<WT, BF>(static_cast<uint32_t>(wq[b][s8 >> 2][s8 & 3]),
                              FOLD ? group_scale<WT, GPU>(a, groups[b], s8) : 1.0f);
    };
    v4i xa[2][MT], wf[2][NB];
    read(0, xa[0]);
    weights(0, wf[0]);
#pragma unroll
    for (int s8 = 0; s8 < 8; ++s8) {
      const int h = s8 >> 2, s = s8 & 3;
      // One step's products at a time (mixing the steps costs more registers
      // than there are), with the next step's operands made in their shadow.
      __builtin_amdgcn_sched_barrier(0);
      if (s8 < 7) {
        read(s8 + 1, xa[(s8 + 1) & 1]);
        weights(s8 + 1, wf[(s8 + 1) & 1]);
      }
      const v4i (&xf)[MT] = xa[s8 & 1];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          if constexpr (FOLD)
            tot[b][t] = mfma16<BF>(xf[t], wf[s8 & 1][b], tot[b][t]);
          else
            acc[b][t] = mfma16<BF>(xf[t], wf[s8 & 1][b], acc[b][t]);
        }
      }
      if constexpr (is_int(WT)) {
#pragma unroll
        for (int t = 0; t < MT; ++t) xs[t] = mfma16<BF>(xf[t], ones<BF>(), xs[t]);
      }
#pragma unroll
      for (int i = 0; i < (NB + (is_int(WT) ? 1 : 0)) * MT; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a product
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // a read of LDS
        __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);  // three vector instructions
      }
      const int done = 32 * (s8 + 1);
      if (FOLD) {
        // the scales are in the products
      } else if (TURN ? done % LEN == 0 : (s == 3 && (LEN == 128 || h == 1))) {
        __builtin_amdgcn_sched_barrier(0);
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
  auto turn_and_use = [&](int buffer, const v4i (&in)[NB][2], const Groups<WT, GPU> (&groups)[NB], bool whole_range) {
    v4i codes[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h) turned[wave][b * 128 + h * 64 + put] = in[b][h];
    __builtin_amdgcn_wave_barrier();  // a wavefront's LDS accesses run in order
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h) codes[b][h] = turned[wave][b * 128 + (get ^ (4 * h))];
    __builtin_amdgcn_wave_barrier();
    if constexpr (WT == W_E2M1 && BF) {
      if (!whole_range) return use(buffer, kw, codes, groups, std::true_type{});
    }
    use(buffer, kw, codes, groups, std::false_type{});
  };

  if (len > 0) {
    Groups<WT, GPU> asked;
    load_scales(0, asked);
    load(0, ring[0]);
    fetch(0);
    place(0);
    fetch(1);
    load(1, ring[1]);
    for (int q = 0; q < len;) {
      // the scales of the next UNITS units, one set of tiles a unit
      constexpr int SW = sizeof(asked.s) / 4, ZW = sizeof(asked.z) / 4;
      Groups<WT, GPU> groups[4];
#pragma unroll
      for (int i = 0; i < SW; ++i) {
        uint32_t o[4];
        spread(asked.s[i], o);
#pragma unroll
        for (int j = 0; j < 4; ++j) groups[j].s[i] = o[j];
      }
      if constexpr (WT == W_U4) {
#pragma unroll
        for (int i = 0; i < ZW; ++i) {
          uint32_t o[4];
          spread(asked.z[i], o);
#pragma unroll
          for (int j = 0; j < 4; ++j) groups[j].z[i] = o[j];
        }
      }
      bool whole_range = false;  // weights that are not all normal bf16 numbers
      if constexpr (WT == W_E2M1 && BF) {
#pragma unroll
        for (int i = 0; i < SW; ++i) whole_range |= extreme(asked.s[i]);
        whole_range = __ballot(whole_range) != 0;
      }
      load_scales(q + UNITS, asked);
#pragma unroll
      for (int d = 0; d < UNITS; ++d) {
        if (q >= len) break;
        // buffer d is whole, and nobody reads the other one any more
        __syncthreads();
        place(d ^ 1);
        fetch(q + 2);
        Groups<WT, GPU> mine[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) mine[b] = groups[d * NB + b];
        if (KW == 1 || KW * (beg + q) + kw < whole) turn_and_use(d, ring[d], mine, whole_range);
        load(q + 2, ring[d]);
        ++q;
      }
    }
  }
  if (whole < units && split == splits - 1) {  // K's partial unit
    __syncthreads();
    const int64_t left = a.k - (256 * static_cast<int64_t>(whole) + 8 * kp);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int h = 0; h < PASSES; ++h)
        xbuf[0][t * 512 + place_at(row + 8 * h)] = in_order<WT>(
            load_x8(x[t][h] + 256 * static_cast<int64_t>(whole), left < 8 ? static_cast<int>(left < 0 ? 0 : left) : 8));
    __syncthreads();
    if (kw == 0) {
      v4i codes[NB][2];
      Groups<WT, GPU> groups[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int64_t i = feature(i0 + 16 * b + col);
        load_codes_end(a, a.w + i * a.ldw_bytes, whole, g, codes[b]);
        load_groups_end<WT, GPU>(a, i * a.ld_scales, i * a.ld_zeros, whole, groups[b]);
      }
      use(0, 0, codes, groups, std::false_type{});
    }
  }

  if constexpr (KW == 2) {
    // The two units' sums, the first's first.
    float* const part = reinterpret_cast<float*>(&xbuf[0][0]) + fw * NB * MT * 256 + lane;
    static_assert(sizeof(xbuf) >= FW * NB * MT * 1024, "the sums fit the activations' area");
    __syncthreads();
    if (kw == 1) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) part[((b * MT + t) * 4 + r) * 64] = tot[b][t][r];
    }
    __syncthreads();
    if (kw != 0) return;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) tot[b][t][r] += part[((b * MT + t) * 4 + r) * 64];
  }
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t i = i0 + 16 * b + col, j = j0 + 16 * t + 4 * r + g;
        if (splits == 1)
          store_result(a, tot[b][t][r], i, j);
        else if (i < a.m && j < a.n)
          a.sums[(static_cast<int64_t>(split) * a.n + j) * a.m + i] = tot[b][t][r];
      }
}

// The splits' sums, in order, and the epilogue.
__global__ void __launch_bounds__(256) w4_splits_kernel(W4Args a, int splits) {
  const int64_t total = static_cast<int64_t>(a.n) * a.m;
  for (int64_t q = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; q < total;
       q += static_cast<int64_t>(gridDim.x) * 256) {
    float v = 0.0f;
    for (int s = 0; s < splits; s += 4) {
      float t[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = a.sums[(s + i < splits ? s + i : s) * total + q];
#pragma unroll
      for (int i = 0; i < 4; ++i) v += s + i < splits ? t[i] : 0.0f;
    }
    const int64_t j = q / a.m;
    store_result(a, v, q - j * a.m, j);
  }
}

template <int WT, bool BF, int NT>
hipError_t launch_one(W4Args& a, hipStream_t st) {
  // K split over as many wavefronts as it has slices; then workgroups for
  // two a CU, each with the same number of row blocks
  const int pieces = a.k / 32, slices = (pieces + 63) / 64;
  int ks = slices < kOneWaves ? (slices > 1 ? slices : 1) : kOneWaves;
  const int rounds_k = slices > 0 ? (slices + ks - 1) / ks : 1;
  int span = ((pieces + ks * rounds_k - 1) / (ks * rounds_k) + 7) / 8 * 8;  // whole 128-byte lines
  if (span < 1) span = 1;
  const int waves = kOneWaves / ks * ks, rows = 4 * (kOneWaves / ks), blocks = (a.m + rows - 1) / rows;
  const int rounds = (blocks + 511) / 512, grid = (blocks + rounds - 1) / rounds;
  const void* f = a.k % 32 != 0 ? reinterpret_cast<const void*>(&w4_one_kernel<WT, BF, NT, true>)
                                : reinterpret_cast<const void*>(&w4_one_kernel<WT, BF, NT, false>);
  void* args[] = {&a, &ks, &span};
  return hipLaunchKernel(f, dim3(static_cast<unsigned>(grid)), dim3(waves * 64), args, 0, st);
}

// Token tiles of sixteen per workgroup, and workgroups along the tokens.
int tiles_for(int64_t n) { return n <= 16 ? 1 : (n <= 32 ? 2 : (n <= 48 ? 3 : 4)); }

// Ways to split K over workgroups: as many as bring their number to one a CU
// (two with one token tile), of at least two units of K each.  More of them
// cost more in sums than they hide (8192 x 8 x 8192, signed codes: 15.5 us with
// two a CU, 18.8 with four).
int64_t splits_of(int64_t m, int64_t n, int64_t k) {
  const int mt = tiles_for(n);
  const int64_t blocks = (m + kManyFeatures - 1) / kManyFeatures * ((n + 16 * mt - 1) / (16 * mt));
  const int64_t most = k / 512, want = (mt == 1 ? 512 : 256) / blocks;
  const int64_t s = want < most ? want : most;
  return s > 1 ? s : 1;
}

template <int WT, bool BF, int GPU, int MT>
hipError_t launch_many(W4Args& a, hipStream_t st) {
  int splits = static_cast<int>(splits_of(a.m, a.n, a.k));
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.m) + kManyFeatures - 1) / kManyFeatures),
                  static_cast<unsigned>((static_cast<int64_t>(a.n) + 16 * MT - 1) / (16 * MT)),
                  static_cast<unsigned>(splits));
  void* args[] = {&a, &splits};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&w4_many_kernel<WT, BF, GPU, MT>), grid,
                                       dim3(256 * units_at_once(MT)), args, 0, st);
  if (e != hipSuccess || splits == 1) return e;
  const int64_t blocks = (static_cast<int64_t>(a.n) * a.m + 255) / 256;
  return hipLaunchKernel(reinterpret_cast<const void*>(&w4_splits_kernel),
                         dim3(static_cast<unsigned>(blocks < 8192 ? blocks : 8192)), dim3(256), args, 0, st);
}

template <int WT, bool BF, int GPU>
hipError_t launch_tokens(W4Args& a, hipStream_t st) {
  if (a.n <= 16) return launch_many<WT, BF, GPU, 1>(a, st);
  if (a.n <= 32) return launch_many<WT, BF, GPU, 2>(a, st);
  if (a.n <= 48) return launch_many<WT, BF, GPU, 3>(a, st);
  return launch_many<WT, BF, GPU, 4>(a, st);
}

// One and two tokens go down the rows, more to the matrix cores: with four
// tokens' activations in registers a CU holds half the wavefronts (8192 x 4 x
// 8192, unsigned codes, groups of 128: 21.2 us down the rows, 15.5 on the
// matrix cores; two tokens, 28672 x 2 x 8192: 30 against 36 us).
template <int WT, bool BF>
hipError_t launch_weights(W4Args& a, hipStream_t st) {
  if (a.n == 1) return launch_one<WT, BF, 1>(a, st);
  if (a.n == 2) return launch_one<WT, BF, 2>(a, st);
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

bool big(int64_t v) { return v > INT32_MAX; }
int64_t at_least_one(int64_t v) { return v > 1 ? v : 1; }
bool misaligned(const void* p, thl_dtype t) { return reinterpret_cast<uintptr_t>(p) % bytes_of(t, 1) != 0; }

}  // namespace
}  // namespace thl

using namespace thl;

extern "C" {

size_t thl_gemm_w4_workspace(int64_t m, int64_t n, int64_t k) {
  if (m <= 0 || m > kMaxFeatures || n <= 2 || n > kMaxTokens || k <= 0 || big(k)) return 0;
  const int64_t s = splits_of(m, n, k);
  return s == 1 ? 0 : static_cast<size_t>(s) * static_cast<size_t>(n) * static_cast<size_t>(m) * sizeof(float);
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

  const size_t need = thl_gemm_w4_workspace(m, n, k);
  if (need && (!workspace || workspace_bytes < need)) return THL_ERR_INVALID;
  if (need && reinterpret_cast<uintptr_t>(workspace) % 4 != 0) return THL_ERR_MISALIGNED;

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
  a.x = static_cast<const uint16_t*>(X), a.sums = static_cast<float*>(workspace), a.c = C, a.d = D, a.bias = bias;
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
