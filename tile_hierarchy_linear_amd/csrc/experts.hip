// experts.hip -- a whole mixture-of-experts layer for a few tokens:
//
//   u_t = act(W1g_e x + b1g_e) * (W1u_e x + b1u_e)   or   act(W1_e x + b1_e),   e = ids[j, t]
//   y_j = sum over t of w[j, t] * (W2_e u_t + b2_e)
//
// With a few tokens every weight of a chosen expert is used a few times, so
// the layer is a stream over those weights, bound by HBM.  Nothing is sorted
// and no size passes through the host: in the first launch a workgroup takes
// sixteen features of one expert, finds that expert's choices among the ids
// itself, and multiplies them on the matrix cores (choices are the rows of the
// tile, features its columns), its wavefronts splitting K; u goes to the
// workspace, with each expert's choices.  The second launch does the same with
// the second matrix, and a third adds each token's choices in their order; for
// few bytes of weights one launch does both.
//
// Products are exact and their sums fp32.  The first multiplies activations of
// bf16 or fp16 with weights of their type, or MX weights decoded to it.  u is
// computed in fp32 and taken as the sum of three bf16 numbers, eight of its bits
// each; the second product adds those of all three, and fp16 weights are,
// exactly, two bf16 numbers as well.
//
// Measured, silu, gated, bf16 activations: one token of 4096 features, 8 of 128
// experts of 1024 E2M1, 21.0 us (12 and 9; its 53 MB at the rate of large reads,
// 6.1 TB/s, are 8.8, and a wavefront's 8 KB of weights come after its ids, so two
// latencies are most of each launch).  48 tokens, 64 experts of bf16, 1.6 GB, 296 to
// 315 us: 5.1 to 5.4 TB/s (with u in two bf16 numbers instead of three 284 to 300).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/thl.h"
#include "host_checks.hpp"
#include "rows.hpp"

namespace thl {
namespace {

enum : int { W_B16 = 0, W_H16 = 1, W_E4M3 = 2, W_E2M1 = 3 };
enum : int { X_B16 = 0, X_H16 = 1, X_PLANES = 2 };  // PLANES: u as three bf16 numbers

constexpr int64_t kMaxPairs = 1024;  // choices of all tokens
constexpr int kWaves = 4;

// Tiles of choices that share a pass over an expert's weights.  A second one
// needs its activations, four times as many registers of them for E2M1 as for
// 16-bit weights, and costs wavefronts; without it an expert of more choices than
// a tile's is read again, from L2.  Both, of 64 experts of 2048 x 768, 4 and 16
// choices each, first product: E2M1 30.7 and 72.6 us with one tile, 34.6 and
// 69.6 with two; E4M3 50.2 and 117.6, 53.1 and 97.0.  bf16 with 128 experts,
// 3 choices each: 112.9 with one, 103.9 with two.
constexpr int most_tiles(int wk) { return wk == W_E2M1 ? 1 : 2; }

// Choices of a pass over an expert's weights in the second product.
constexpr int choices_of_pass(bool many) { return many ? 16 : 4; }

// Values of K in 16 bytes of a row.
constexpr int piece_of(int wk) { return wk == W_E2M1 ? 32 : (wk == W_E4M3 ? 16 : 8); }

// A slot's choices: their number, where they start in `order`, and their expert.
struct Slot {
  uint16_t count, start;
  int32_t expert;
};

struct ExpertArgs {
  const uint8_t* w;
  const uint8_t* sf;
  const void* bias;
  const uint16_t* x;  // X, or u's first plane
  const void* ids;
  const float* weights;
  void* y;
  // the workspace: u's planes, z of every choice, each slot, and the choices by
  // expert
  uint16_t* u;
  float* z;
  Slot* slots;
  int32_t* order;
  int64_t w_row, w_expert;  // bytes
  int64_t ld_sf, sf_expert, bias_expert;
  int64_t ldx, ldy, ld_u, ld_ids;
  int64_t plane;            // values from one of u's to the next
  int64_t row_bytes;        // of K weights
  int32_t k, features;      // of an output: hidden features, or the layer's
  int32_t pairs, topk, experts, ids_bytes;
  int32_t slot_count, by_choice;  // a slot is an expert, or where the choices are fewer, a choice
  int32_t act, bias_type, y_type;
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

// An fp16 number as two bf16: without its last three bits, and those.
// Infinities and NaN have no rest.
__device__ __forceinline__ void split_h1(uint16_t b, uint32_t& hi, uint32_t& lo) {
  const float f = static_cast<float>(__builtin_bit_cast(_Float16, b));
  hi = __builtin_bit_cast(uint32_t, f) & 0xffff0000u;
  lo = __builtin_bit_cast(uint32_t, (b & 0x7c00u) == 0x7c00u ? 0.0f : f - __builtin_bit_cast(float, hi));
  if ((b & 0x7fffu) > 0x7c00u) hi |= 0x00400000u;  // a NaN stays one
}
__device__ __forceinline__ void split_h(v4i x, v4i& hi, v4i& lo) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    uint32_t h[2], l[2];
    split_h1(static_cast<uint16_t>(x[d]), h[0], l[0]);
    split_h1(static_cast<uint16_t>(static_cast<uint32_t>(x[d]) >> 16), h[1], l[1]);
    hi[d] = static_cast<int>(__builtin_amdgcn_perm(h[1], h[0], 0x07060302u));
    lo[d] = static_cast<int>(__builtin_amdgcn_perm(l[1], l[0], 0x07060302u));
  }
}
// u as three planes: its first eight bits, the next eight and the last, exact
// but for what lies below 2^-133, the smallest bf16 number.  Infinities and NaN
// have no rest.
__device__ __forceinline__ void split_f(float v, uint16_t (&o)[3]) {
#pragma clang fp contract(off)  // (of v's value as rounded, not of the product that gave it)
  const bool rest = __builtin_fabsf(v) < INFINITY;
  const uint16_t quiet = v != v ? 0x0040 : 0;  // a NaN stays one
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const uint32_t top = __builtin_bit_cast(uint32_t, v) & 0xffff0000u;
    o[p] = static_cast<uint16_t>(top >> 16);
    v = rest ? v - __builtin_bit_cast(float, top) : 0.0f;
  }
  o[0] |= quiet;
}

// Sums of plane 0 and of the others.  An infinite weight makes the first infinite
// and, of planes of zeros, the others NaN.
__device__ __forceinline__ float planes_sum(float first, float rest) {
  return __builtin_fabsf(first) < INFINITY ? first + rest : first;
}

// Codes 8 s .. 8 s + 7 of a piece, times `scale`, a power of two: as fp16 if H,
// else as bf16.
template <int WK, bool H>
__device__ __forceinline__ v4i decode(v4i w, int s, float scale) {
  v4i o;
#define THL_TWO(i, codes, which)                                                                            \
  if constexpr (WK == W_E2M1 && H)                                                                          \
    o[i] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, which));          \
  else if constexpr (WK == W_E2M1)                                                                          \
    o[i] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, which));         \
  else if constexpr (H)                                                                                     \
    o[i] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes, scale, (which) != 0));   \
  else                                                                                                      \
    o[i] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, (which) != 0))
  if constexpr (WK == W_E2M1) {
    const uint32_t v = static_cast<uint32_t>(w[s]);
    THL_TWO(0, v, 0);
    THL_TWO(1, v, 1);
    THL_TWO(2, v, 2);
    THL_TWO(3, v, 3);
  } else {
    const uint32_t a = static_cast<uint32_t>(w[2 * s]), b = static_cast<uint32_t>(w[2 * s + 1]);
    THL_TWO(0, a, 0);
    THL_TWO(1, a, 1);
    THL_TWO(2, b, 0);
    THL_TWO(3, b, 1);
  }
#undef THL_TWO
  return o;
}

// fp32 numbers by their exponent: 2^(e - 127), e from 1 to 254.
__device__ __forceinline__ float exp2_of(uint32_t e) { return __builtin_bit_cast(float, e << 23); }

// MX blocks are decoded with 2^SHIFT times their scale, and the sums divided by
// it.  An E8M0 code b = LO .. HI so makes every element a number of the type:
// a normal bf16 number, or an fp16 number (of E4M3, down to its subnormal ones).
// With SHIFT the 23 or 27 powers of two that fp16 has room for lie where
// weights' scales do: 2^-21 to 2^1, or 2^-19 to 2^7 of E2M1.
template <int WK, bool H>
struct Scales {
  static constexpr int SHIFT = H ? 6 : 0;
  static constexpr uint32_t LO = !H ? (WK == W_E2M1 ? 2 : 10) : (WK == W_E2M1 ? 127 - 13 - SHIFT : 127 - 15 - SHIFT);
  static constexpr uint32_t HI = !H ? (WK == W_E2M1 ? 252 : 246) : (WK == W_E2M1 ? 127 + 13 - SHIFT : 127 + 7 - SHIFT);
  // The code next to b in that range, and what a sum decoded under it lacks.
  static __device__ __forceinline__ uint32_t tame(uint32_t b) { return b < LO ? LO : (b > HI ? HI : b); }
  static __device__ __forceinline__ float lacking(uint32_t b) {
    return b == 255 ? __builtin_nanf("") : exp2_of(127 + b - tame(b) - SHIFT);
  }
  static __device__ __forceinline__ float decoding(uint32_t b) { return exp2_of(b + SHIFT); }
};

__device__ __forceinline__ float activated(float v, int act) {
  if (act & THL_MOE_RELU) return v <= 0.0f ? 0.0f : v;  // (NaN stays)
  if (act & THL_MOE_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752440f));
  if (act & THL_MOE_SILU) return v / (1.0f + expf(-v));
  return v;
}

// A chunk of K is 128 bytes of every row: lane (feature l % 16, group g = l / 16)
// holds its row's pieces g and 4 + g, whole lines of HBM.  Piece order is K
// order within a lane, so step s of half h multiplies values
// chunk + PK (4 h + g) + 8 s .. + 7 of choices and features alike.
//
// A tile's sixteen rows are sixteen choices, and of u there are three such tiles,
// one of each plane.  Of up to four choices one tile holds all planes: rows
// 4 p .. 4 p + 3 are plane p of choices 0 .. 3 (the last four rows repeat plane 2 and
// are not used), so that lane group p ends with the sums of plane p, which are
// added at the end.  (Two such tiles for five to eight choices gave and took:
// 48 tokens, 8 of 64 experts of 4096 x 1024 bf16, 301 us for 305; 64 tokens, 4 of 32
// experts of 2048 x 1024, 113.5 for 111.6.)
template <int WK, int XK>
struct Kind {
  static constexpr bool MX = WK == W_E4M3 || WK == W_E2M1;
  static constexpr bool HALF = XK == X_H16;  // fp16 by fp16; else bf16 by bf16
  static constexpr int PK = piece_of(WK), KC = 8 * PK, STEPS = PK / 8;
};

// 16 bytes moved `by` (0 or more) towards the first, zeros behind them.
__device__ __forceinline__ v4i shift_bytes(v4i v, int by) {
  uint32_t w[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) w[d] = static_cast<uint32_t>(v[d]);
  shift_run<4, 1>(w, by < 16 ? by >> 2 : 8);
#pragma unroll
  for (int d = 0; d < 4; ++d)
    v[d] = static_cast<int>(__builtin_amdgcn_alignbyte(d < 3 ? w[d + 1] : 0u, w[d], by & 3));
  return v;
}

// Eight 16-bit values, likewise.
__device__ __forceinline__ v4i shift_values(v4i v, int by) {
  uint32_t w[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) w[d] = static_cast<uint32_t>(v[d]);
  shift_run<4, 2>(w, by);
#pragma unroll
  for (int d = 0; d < 4; ++d) v[d] = static_cast<int>(w[d]);
  return v;
}

// One chunk's weights of RT tiles of features with their scales (of half h in
// byte g of word h, or bytes 2 h + g / 2), and its activations of MT tiles of
// choices, as loaded.
template <int WK, int RT>
struct Weights {
  v4i w[2][RT];
  uint32_t sc[RT][WK == W_E2M1 ? 2 : 1];
};
template <int WK, int XK, int MT>
struct Values {
  v4i x[2][MT][Kind<WK, XK>::STEPS];
};

// Chunk c.  `there`: it exists; else every lane loads the matrix's first bytes
// (a load behind a branch would make the compiler wait for all of them, and a
// chunk loaded again is traffic).
template <int WK, int RT>
__device__ __forceinline__ void load_weights(const ExpertArgs& a, const uint8_t* const (&w)[RT],
                                             const uint8_t* const (&sf)[RT], int c, bool there, Weights<WK, RT>& o) {
  const int g = (static_cast<int>(threadIdx.x) & 63) >> 4;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const uint8_t* p = there ? w[r] + 128 * static_cast<int64_t>(c) + 16 * g : a.w;
    // (not marked to leave L2 first: the two halves of a line come apart)
    o.w[0][r] = *reinterpret_cast<const v4i_a1*>(p);
    o.w[1][r] = *reinterpret_cast<const v4i_a1*>(p + 64);
    if constexpr (WK == W_E2M1) {
      const v2u_a1 q = *reinterpret_cast<const v2u_a1*>(there ? sf[r] + 8 * static_cast<int64_t>(c) : a.sf);
      o.sc[r][0] = q[0], o.sc[r][1] = q[1];
    } else if constexpr (WK == W_E4M3) {
      o.sc[r][0] = *reinterpret_cast<const u32_a1*>(there ? sf[r] + 4 * static_cast<int64_t>(c) : a.sf);
    }
  }
}

// A wavefront's chunks c0, c0 + step, ... below `whole`, and its first ones on
// their way: asked for before it is known what they are multiplied with.
template <int WK, int RT, int D>
struct Stream {
  Weights<WK, RT> b[D];
  int c0, step, whole;
  bool tail;  // K's partial chunk is this wavefront's
  __device__ __forceinline__ Stream(const ExpertArgs& a, int first, int by)
      : c0(first), step(by), whole(a.k / (8 * piece_of(WK))) {
    tail = whole * 8 * piece_of(WK) < a.k && whole % by == first;
  }
  __device__ __forceinline__ int end() const { return c0 + (whole - 1 - c0) / step * step; }
  __device__ __forceinline__ void start(const ExpertArgs& a, const uint8_t* const (&w)[RT],
                                        const uint8_t* const (&sf)[RT]) {
    if (c0 >= whole) return;
#pragma unroll
    for (int d = 0; d < D - 1; ++d) load_weights<WK, RT>(a, w, sf, c0 + d * step, c0 + d * step < whole, b[d]);
  }
};

// The sums over a wavefront's started stream and, if it is its, K's partial
// chunk, of RT tiles of features (w, sf: this lane's rows) and MT tiles of
// choices (x: this lane's rows), each with its sums; or the last with its own and
// the others with one.
template <int WK, int XK, int RT, int MT, int AT, int D>
__device__ __forceinline__ void products(const ExpertArgs& a, const uint8_t* const (&w)[RT],
                                         const uint8_t* const (&sf)[RT], const uint16_t* const (&x)[MT],
                                         Stream<WK, RT, D>& st, v4f (&acc)[RT][AT]) {
  constexpr auto sum_of = [](int t) { return AT == MT ? t : (t == MT - 1 ? AT - 1 : 0); };
  using T = Kind<WK, XK>;
  constexpr int PK = T::PK, KC = T::KC, STEPS = T::STEPS;
  using S = Scales<WK, T::HALF>;
  const int lane = static_cast<int>(threadIdx.x) & 63, col = lane & 15, g = lane >> 4;
  const int c0 = st.c0, step = st.step, whole = st.whole;

  auto multiply = [](v4i x, v4i w, v4f sum) {
    if constexpr (T::HALF) return mfma_h(x, w, sum);
    return mfma_bf(x, w, sum);
  };
  // Half a chunk, `code`: the lane's scales.
  auto half = [&](const v4i (&wh)[RT], const uint32_t (&code)[RT], const v4i (&xh)[MT][STEPS]) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        if constexpr (WK == W_H16 && !T::HALF) {
          v4i hi, lo;
          split_h(wh[r], hi, lo);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            v4f& sum = acc[r][sum_of(t)];
            sum = mfma_bf(xh[t][s], lo, mfma_bf(xh[t][s], hi, sum));
          }
        } else {
          v4i q = wh[r];
          if constexpr (T::MX) q = decode<WK, T::HALF>(q, s, S::decoding(code[r]));
#pragma unroll
          for (int t = 0; t < MT; ++t) acc[r][sum_of(t)] = multiply(xh[t][s], q, acc[r][sum_of(t)]);
        }
      }
  };
  // The same under any scales: each lane group's blocks by themselves, under a
  // scale next to their own, and what that lacks applied to the sums.
  auto half_rare = [&](const v4i (&wh)[RT], const uint32_t (&code)[RT], const v4i (&xh)[MT][STEPS]) {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        const float factor = S::lacking(static_cast<uint32_t>(__shfl(static_cast<int>(code[r]), 16 * q + col)));
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          v4f alone = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int s = 0; s < STEPS; ++s) {
            v4i v = decode<WK, T::HALF>(wh[r], s, S::decoding(S::tame(code[r])));
            v4i u = xh[t][s];
            if (g != q) u = v = v4i{0, 0, 0, 0};  // (an infinity, NaN may be in either)
            alone = multiply(u, v, alone);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[r][sum_of(t)][e] += factor * alone[e];
        }
      }
    }
  };
  auto is_rare = [&](const uint32_t (&code)[RT]) {
    bool any = false;
#pragma unroll
    for (int r = 0; r < RT; ++r) any |= code[r] != S::tame(code[r]);
    return __ballot(any) != 0;
  };

  auto load_x = [&](int c, Values<WK, XK, MT>& o) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
          o.x[h][t][s] = *reinterpret_cast<const v4i_a2*>(x[t] + static_cast<int64_t>(c) * KC + PK * (4 * h + g) + 8 * s);
  };
  bool skipped = false;
  auto use = [&](const Weights<WK, RT>& b, const Values<WK, XK, MT>& v) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t code[RT] = {};
      if constexpr (T::MX) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
          code[r] = (WK == W_E2M1 ? b.sc[r][WK == W_E2M1 ? h : 0] >> (8 * g) : b.sc[r][0] >> (8 * (2 * h + (g >> 1)))) & 255u;
        if (is_rare(code)) {
          skipped = true;
          continue;
        }
      }
      half(b.w[h], code, v.x[h]);
    }
  };

  // D - 1 chunks' weights are on their way while one is used.  Its activations,
  // which L2 holds, are asked for just before: a second set of them would cost
  // the registers of a wavefront in three and gains nothing.
  if (c0 < whole) {
    const int end = st.end();
    Values<WK, XK, MT> v;
    for (int c = c0;;) {
      bool last = false;
#pragma unroll
      for (int d = 0; d < D; ++d) {
        load_x(c, v);
        load_weights<WK, RT>(a, w, sf, c + (D - 1) * step, c + (D - 1) * step < whole, st.b[(d + D - 1) % D]);
        use(st.b[d], v);
        last = c == end;
        c += step;
        if (last) break;
      }
      if (last) break;
    }
  }

  if constexpr (T::MX && S::SHIFT != 0) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < AT; ++t) acc[r][t] *= exp2_of(127 - S::SHIFT);
  }

  // The halves that were skipped, and K's partial chunk (whose number is
  // `whole`).  Loads that would pass a row's end end with it instead and are
  // shifted into place; rows shorter than a load go element by element.
  for (int c = skipped ? c0 : whole; c < whole || (c == whole && st.tail); c += step) {
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      const int64_t at = 128 * static_cast<int64_t>(c) + 64 * h + 16 * g, end = a.row_bytes - 16;
      const int k0 = c * KC + PK * (4 * h + g);
      v4i wh[RT], xh[MT][STEPS];
      uint32_t code[RT] = {};
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        if (end >= 0)
          wh[r] = *reinterpret_cast<const v4i_a1*>(w[r] + (at < end ? at : end));
        else
          load_codes_at(w[r] + at, a.row_bytes - at, wh[r]);
        if constexpr (T::MX) code[r] = sf[r][(k0 < a.k ? k0 : a.k - 1) / 32];
      }
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          const int k = k0 + 8 * s;
          if (a.k >= 8)
            xh[t][s] = *reinterpret_cast<const v4i_a2*>(x[t] + (k < a.k - 8 ? k : a.k - 8));
          else
            xh[t][s] = load_x8(x[t] + k, k < a.k ? a.k - k : 0);
        }
      if (end >= 0) {
#pragma unroll
        for (int r = 0; r < RT; ++r) wh[r] = shift_bytes(wh[r], at > end ? static_cast<int>(at - end) : 0);
      }
      if (a.k >= 8) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          const int by = k0 + 8 * s - (a.k - 8);
#pragma unroll
          for (int t = 0; t < MT; ++t) xh[t][s] = shift_values(xh[t][s], by > 0 ? by : 0);
        }
      }
      bool rare = false;
      if constexpr (T::MX) {
        rare = is_rare(code) || (S::SHIFT != 0 && c == whole);
        if (rare) half_rare(wh, code, xh);
      }
      if (c == whole && !rare) half(wh, code, xh);
    }
  }
}

// The lane's row of weights of tile r of features f0 .. (`features` in a part;
// part 1 of a gated matrix is what the gates multiply); features past the last
// repeat it and are not stored.
template <int WK>
__device__ __forceinline__ void row_of(const ExpertArgs& a, int64_t expert, int f, int part, const uint8_t*& w,
                                       const uint8_t*& sf) {
  f = f < a.features ? f : a.features - 1;
  const int64_t row = static_cast<int64_t>(f) + (part ? a.features : 0);
  w = a.w + expert * a.w_expert + row * a.w_row;
  sf = WK == W_E4M3 || WK == W_E2M1 ? a.sf + expert * a.sf_expert + row * a.ld_sf : nullptr;
}
// ---- the first product
// A workgroup takes sixteen features of one expert (and of a gated matrix what
// their gates multiply); its wavefronts split K.
template <int WK, int XK, bool GATED>
__global__ void __launch_bounds__(64 * kWaves, 2) experts_up_kernel(ExpertArgs a) {
  constexpr int RT = GATED ? 2 : 1, MOST = most_tiles(WK), D = 2;
  __shared__ int list[kMaxPairs];
  __shared__ int hits[2][kWaves];
  __shared__ float part[kWaves][RT][MOST][4][64];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, g = lane >> 4, slot = static_cast<int>(blockIdx.y);

  // This workgroup's expert: the slot's number, or that of choice `slot`, if it
  // is the first choice of it; and its choices in order.
  int64_t expert = slot;
  bool live = true;
  if (a.by_choice) {
    expert = id_of(a, slot);
    live = expert >= 0 && expert < a.experts;
  }
  const int f0 = static_cast<int>(blockIdx.x) * 16;
  const uint8_t* w[RT];
  const uint8_t* sf[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
    row_of<WK>(a, live ? expert : 0, f0 + col, r, w[r], sf[r]);
  Stream<WK, RT, D> st(a, wave, kWaves);
  // (of a choice that is not its expert's first these loads are for nothing)
  if (a.by_choice) st.start(a, w, sf);
  int count = 0, before = 0;  // choices of it, and of experts below it
  if (live) {
    for (int base = 0; base < a.pairs; base += 64 * kWaves) {
      const int p = base + tid;
      const int64_t id = p < a.pairs ? id_of(a, p) : -1;
      const bool hit = id == expert;
      const uint64_t who = __ballot(hit), less = __ballot(id >= 0 && id < expert);
      if (lane == 0) hits[0][wave] = __popcll(who), hits[1][wave] = __popcll(less);
      __syncthreads();
      int at = count, all = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        if (w < wave) at += hits[0][w];
        all += hits[0][w];
        before += hits[1][w];
      }
      if (hit) list[at + __popcll(who & ((1ull << lane) - 1))] = p;
      count += all;
      __syncthreads();
    }
    if (a.by_choice && count > 0 && list[0] != slot) count = 0;
  }
  // (for the second product)
  if (blockIdx.x == 0) {
    if (tid == 0)
      a.slots[slot] = Slot{static_cast<uint16_t>(count), static_cast<uint16_t>(before), static_cast<int32_t>(expert)};
    for (int i = tid; i < count; i += 64 * kWaves) a.order[before + i] = list[i];
  }
  if (count == 0) return;

  if (!a.by_choice) st.start(a, w, sf);

  auto run = [&](int first, auto tiles) {
    constexpr int MT = decltype(tiles)::value;
    const uint16_t* x[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int i = first + 16 * t + col;
      x[t] = a.x + static_cast<int64_t>(list[i < count ? i : count - 1] / a.topk) * a.ldx;
    }
    v4f acc[RT][MT] = {};
    products<WK, XK, RT, MT, MT, D>(a, w, sf, x, st, acc);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[wave][r][t][e][lane] = acc[r][t][e];
  };
  for (int first = 0; first < count;) {
    const int left = count - first, tiles = left > 16 ? MOST : 1;
    __syncthreads();  // the sums before these have been read
    if (MOST == 1 || tiles == 1)
      run(first, std::integral_constant<int, 1>{});
    else
      run(first, std::integral_constant<int, MOST>{});
    __syncthreads();
    // Register e of lane l is choice 4 (l / 16) + e of the tile and feature l % 16.
    static_assert(kWaves == 4, "a wavefront finishes one register");
    for (int t = 0; t < tiles; ++t) {
      const int i = 16 * t + 4 * g + wave;
      if (i >= left) continue;
      auto sum = [&](int r) {
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < kWaves; ++q) v += part[q][r][t][wave][lane];
        return v;
      };
      const int64_t at = list[first + i];
      const int f = f0 + col;
      if (f >= a.features) continue;
      const int64_t b = expert * a.bias_expert + f;
      float v = sum(0);
      if (a.bias) v += load_f(a.bias, a.bias_type, b);
      v = activated(v, a.act);
      if constexpr (GATED) {
        float m = sum(1);
        if (a.bias) m += load_f(a.bias, a.bias_type, b + a.features);
        v *= m;
      }
      uint16_t u[3];
      split_f(v, u);
#pragma unroll
      for (int p = 0; p < 3; ++p) a.u[p * a.plane + at * a.ld_u + f] = u[p];
    }
    first += 16 * tiles;
    if (first < count) st.start(a, w, sf);
  }
}

// ---- the second product
// The sums of an expert's choices over a wavefront's started stream, handed to
// `put(place in `order`, choice, tile, feature of it, value)` by the lanes that hold
// them, planes added.  MANY: up to sixteen choices a pass, else up to four.
template <int WK, bool MANY, int RT, int D, class Put>
__device__ __forceinline__ void down_choices(const ExpertArgs& a, const uint8_t* const (&w)[RT],
                                             const uint8_t* const (&sf)[RT], Stream<WK, RT, D>& st, const int* order,
                                             int count, Put put) {
  const int lane = static_cast<int>(threadIdx.x) & 63, col = lane & 15, g = lane >> 4;
  auto row = [&](int i, int p) {  // of u, of a choice that exists
    return a.x + p * a.plane + static_cast<int64_t>(order[i < count ? i : count - 1]) * a.ldx;
  };
  for (int first = 0; first < count; first += choices_of_pass(MANY)) {
    if (first > 0) st.start(a, w, sf);
    if (!MANY || count - first <= 4) {
      const uint16_t* x[1] = {row(first + (col & 3), col < 12 ? col >> 2 : 2)};
      v4f acc[RT][1] = {};
      products<WK, X_PLANES, RT, 1, 1, D>(a, w, sf, x, st, acc);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = acc[r][0][e], rest = __shfl_xor(v, 16) + __shfl_xor(v, 32);
          const int i = first + e;
          if (g == 0 && i < count) put(i, order[i], r, col, planes_sum(v, rest));
        }
    } else if constexpr (MANY) {
      const uint16_t* x[3];
#pragma unroll
      for (int p = 0; p < 3; ++p) x[p] = row(first + col, 2 - p);
      // of planes 1 and 2, and of plane 0 (of MX weights all in one: the registers of
      // two cost E4M3 a third of its wavefronts, 32 tokens, 8 of 128 experts of 2048 x
      // 768, 137 us for 129)
      constexpr int AT = Kind<WK, X_PLANES>::MX ? 1 : 2;
      v4f acc[RT][AT] = {};
      products<WK, X_PLANES, RT, 3, AT, D>(a, w, sf, x, st, acc);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = first + 4 * g + e;
          if (i < count) put(i, order[i], r, col, AT == 1 ? acc[r][0][e] : planes_sum(acc[r][AT - 1][e], acc[r][0][e]));
        }
    }
  }
}

__device__ __forceinline__ void store_y(const ExpertArgs& a, int64_t j, int64_t f, float v) {
  const int64_t to = j * a.ldy + f;
  if (a.y_type == THL_F32)
    static_cast<float*>(a.y)[to] = v;
  else if (a.y_type == THL_F16)
    static_cast<_Float16*>(a.y)[to] = static_cast<_Float16>(v);
  else
    static_cast<__bf16*>(a.y)[to] = static_cast<__bf16>(v);
}

// Few bytes: a workgroup takes sixteen features of every slot, its wavefronts
// the slots (`ks` of them share one slot's K), and adds each token's choices.
constexpr int kJoinWaves = 8;

template <int WK>
__global__ void __launch_bounds__(64 * kJoinWaves, 2) experts_down_join_kernel(ExpertArgs a, int ks) {
  constexpr int D = 2;
  extern __shared__ int shared[];
  int* order = shared;
  int* expert_of = order + a.pairs;                                 // -1: no expert of this layer
  float* share_of = reinterpret_cast<float*>(expert_of + a.pairs);  // the choices' weights
  float* z = share_of + a.pairs;                                    // [share of K][choice][feature]
  const int tid = static_cast<int>(threadIdx.x), col = tid & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int f0 = static_cast<int>(blockIdx.x) * 16, share = wave % ks;
  float* mine = z + share * a.pairs * 16;
  bool copied = false;
  for (int slot = wave / ks; slot < a.slot_count || !copied; slot += kJoinWaves / ks) {
    const Slot s = slot < a.slot_count ? a.slots[slot] : Slot{0, 0, 0};
    const uint8_t* w[1];
    const uint8_t* sf[1];
    Stream<WK, 1, D> st(a, share, ks);
    row_of<WK>(a, s.count > 0 ? s.expert : 0, f0 + col, 0, w[0], sf[0]);
    if (s.count > 0) st.start(a, w, sf);
    if (!copied) {  // (every wavefront comes here once)
      for (int i = tid; i < a.pairs; i += 64 * kJoinWaves) {
        const int64_t e = id_of(a, i);
        order[i] = a.order[i];
        expert_of[i] = e >= 0 && e < a.experts ? static_cast<int>(e) : -1;
        share_of[i] = a.weights[i];
      }
      __syncthreads();
      copied = true;
    }
    if (s.count > 0)
      down_choices<WK, false, 1, D>(a, w, sf, st, order + s.start, s.count,
                                    [&](int, int p, int, int f, float v) { mine[p * 16 + f] = v; });
  }
  __syncthreads();
  const int n = a.pairs / a.topk;
  for (int q = tid; q < n * 16; q += 64 * kJoinWaves) {
    const int j = q >> 4, f = f0 + (q & 15);
    if (f >= a.features) continue;
    float v = 0.0f;
    for (int t = 0; t < a.topk; ++t) {
      const int p = j * a.topk + t, e = expert_of[p];
      if (e < 0) continue;
      float u = 0.0f;
      for (int i = 0; i < ks; ++i) u += z[(i * a.pairs + p) * 16 + (q & 15)];
      if (a.bias) u += load_f(a.bias, a.bias_type, e * a.bias_expert + f);
      v += share_of[p] * u;
    }
    store_y(a, j, f, v);
  }
}

// More of them: a workgroup takes RT tiles of features of one slot, its
// wavefronts splitting K; z goes to the workspace, and a third launch adds
// each token's choices.
template <int WK, bool MANY>
__global__ void __launch_bounds__(64 * kWaves, 2) experts_down_kernel(ExpertArgs a) {
  constexpr int RT = 2, D = 2, ROWS = choices_of_pass(MANY);
  __shared__ float part[kWaves][ROWS][16 * RT];
  const int tid = static_cast<int>(threadIdx.x), col = tid & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Slot slot = a.slots[blockIdx.y];
  const int count = slot.count;
  const int* order = a.order + slot.start;
  if (count == 0) return;
  const int f0 = static_cast<int>(blockIdx.x) * 16 * RT;
  const uint8_t* w[RT];
  const uint8_t* sf[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) row_of<WK>(a, slot.expert, f0 + 16 * r + col, 0, w[r], sf[r]);
  Stream<WK, RT, D> st(a, wave, kWaves);
  for (int first = 0; first < count; first += ROWS) {
    st.start(a, w, sf);
    const int left = count - first < ROWS ? count - first : ROWS;
    __syncthreads();  // the sums before these have been read
    down_choices<WK, MANY, RT, D>(a, w, sf, st, order + first, left,
                                  [&](int i, int, int r, int f, float v) { part[wave][i][16 * r + f] = v; });
    __syncthreads();
    for (int q = tid; q < left * 16 * RT; q += 64 * kWaves) {
      const int i = q / (16 * RT), f = q % (16 * RT);
      if (f0 + f >= a.features) continue;
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) v += part[k][i][f];
      a.z[static_cast<int64_t>(order[first + i]) * a.features + f0 + f] = v;
    }
  }
}

// y_j = the sum over its choices, in their order: four choices' loads at a time
// (of a choice that does not count they are of what is there, and not used).
__global__ void __launch_bounds__(256) experts_join_kernel(ExpertArgs a) {
  const int64_t m = a.features, total = static_cast<int64_t>(a.pairs / a.topk) * m;
  for (int64_t q = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; q < total;
       q += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t j = q / m, f = q - j * m, base = j * a.topk;
    float v = 0.0f;
    for (int t0 = 0; t0 < a.topk; t0 += 4) {
      int64_t e[4];
      float weight[4], z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t p = base + (t0 + i < a.topk ? t0 + i : t0);
        e[i] = id_of(a, static_cast<int>(p));
        weight[i] = a.weights[p];
        z[i] = a.z[p * m + f];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (t0 + i >= a.topk || e[i] < 0 || e[i] >= a.experts) continue;
        if (a.bias) z[i] += load_f(a.bias, a.bias_type, e[i] * a.bias_expert + f);
        v += weight[i] * z[i];
      }
    }
    store_y(a, j, f, v);
  }
}

template <int WK, int XK, bool GATED>
hipError_t launch_up(ExpertArgs& a, hipStream_t st) {
  void* args[] = {&a};
  const int64_t tiles = (static_cast<int64_t>(a.features) + 15) / 16;
  return hipLaunchKernel(reinterpret_cast<const void*>(&experts_up_kernel<WK, XK, GATED>),
                         dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(a.slot_count)), dim3(64 * kWaves),
                         args, 0, st);
}
template <int WK, int XK>
hipError_t launch_up(ExpertArgs& a, bool gated, hipStream_t st) {
  return gated ? launch_up<WK, XK, true>(a, st) : launch_up<WK, XK, false>(a, st);
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

template <int WK, bool MANY>
hipError_t launch_down(ExpertArgs& a, hipStream_t st) {
  const int64_t tiles = (static_cast<int64_t>(a.features) + 15) / 16;
  // Products and joining in one launch save a launch of 4.7 us, but every
  // workgroup works through all slots, four choices at a time.  So by the bits of a
  // weight of every slot, and of every choice.  The layer in one launch and in two,
  // of 4096 x 1024 and of 2048 x 768: slots of one choice, sixteen of E2M1 39.1 for 43.6
  // us and 21.5 for 23.8, twenty-four 52.1 for 55.4 and 29.6 for 28.7, thirty-two 64.2
  // for 65.5 and 36.7 for 33.7; eight of E4M3 33.6 for 38.3 and 21.2 for 21.9, sixteen
  // 59.5 for 62.2 and 36.6 for 35.3; four of bf16 29.3 for 31.9 and 18.0 for 19.7, eight
  // 52.2 for 52.4 and 29.1 for 27.2.  Several choices a slot: sixteen of E2M1 of two
  // 36.5 for 38.2 and 25.4 for 24.4, of four 54.8 for 52.3 and 34.7 for 26.7; eight of
  // four 28.4 for 29.8 and 21.1 for 19.4; eight of E4M3 of two 31.2 for 34.7 and 21.1
  // for 21.5, of four 39.4 for 39.2 and 27.2 for 23.6.
  constexpr int kBits = 128 / piece_of(WK);
  if (a.slot_count * kBits <= 64 && a.pairs * kBits <= 128) {
    int ks = 1;
    while (2 * ks * a.slot_count <= kJoinWaves) ks *= 2;
    void* args[] = {&a, &ks};
    return hipLaunchKernel(reinterpret_cast<const void*>(&experts_down_join_kernel<WK>),
                           dim3(static_cast<unsigned>(tiles)), dim3(64 * kJoinWaves), args,
                           static_cast<unsigned>(4 * a.pairs * (3 + 16 * ks)), st);
  }
  void* args[] = {&a};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&experts_down_kernel<WK, MANY>),
                                       dim3(static_cast<unsigned>((tiles + 1) / 2), static_cast<unsigned>(a.slot_count)),
                                       dim3(64 * kWaves), args, 0, st);
  if (e != hipSuccess) return e;
  const int64_t blocks = (static_cast<int64_t>(a.pairs / a.topk) * a.features + 255) / 256;
  return hipLaunchKernel(reinterpret_cast<const void*>(&experts_join_kernel),
                         dim3(static_cast<unsigned>(blocks < 8192 ? blocks : 8192)), dim3(256), args, 0, st);
}
hipError_t launch_down(ExpertArgs& a, thl_dtype w, hipStream_t st) {
  switch (w) {
    case THL_BF16:
      return launch_down<W_B16, true>(a, st);
    case THL_F16:
      return launch_down<W_H16, true>(a, st);
    case THL_E4M3:
      return launch_down<W_E4M3, true>(a, st);
    default:
      // Sixteen choices a pass of E2M1 weights take 228 registers (146 with four) and
      // so a third of the wavefronts: at two choices a slot or fewer the passes are
      // four.  The layer of 2048 x 768, 8 of 128 experts, four a pass and sixteen: 4
      // tokens 33.9 and 36.7 us, 16 66.3 and 69.6, 32 (two a slot) 91.7 and 93.0, 48
      // 116 and 113, 96 179 and 164.
      return a.pairs > 2 * a.slot_count ? launch_down<W_E2M1, true>(a, st) : launch_down<W_E2M1, false>(a, st);
  }
}

bool big(int64_t v) { return v > INT32_MAX; }
int64_t at_least_one(int64_t v) { return v > 1 ? v : 1; }
bool off(const void* p, thl_dtype t) { return reinterpret_cast<uintptr_t>(p) % bytes_of(t, 1) != 0; }
bool is_mx(thl_dtype t) { return t == THL_E4M3 || t == THL_E2M1X2; }

constexpr int64_t kMaxSpan = INT64_C(1) << 40;  // values of all experts

// One of the layer's matrices, rows of k (of any number: `ranges` has it).
thl_status check(const thl_expert_matrix& w, int64_t experts, int64_t k, thl_dtype x) {
  if (!is_mx(w.type) && w.type != x) return THL_ERR_UNSUPPORTED;
  const int64_t most = kMaxSpan / experts;  // (their byte offsets stay in 64 bits)
  if (big(w.ld) || big(w.ld_sf) || w.stride > most || w.stride_sf > most || w.stride_bias > most)
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
  return static_cast<size_t>(n * topk) * static_cast<size_t>(6 * pitch(hidden) + 4 * (m + 3));
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
  thl_status s = check(*up, experts, m, type_x);
  if (s == THL_OK) s = check(*down, experts, hidden, type_x);
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
  a.by_choice = pairs < experts;
  a.slot_count = a.by_choice ? a.pairs : a.experts;
  a.weights = weights, a.y = Y, a.ldy = ldy, a.y_type = type_y;
  a.u = static_cast<uint16_t*>(workspace), a.ld_u = ld_u, a.plane = pairs * ld_u;
  a.z = reinterpret_cast<float*>(a.u + 3 * a.plane);
  a.slots = reinterpret_cast<Slot*>(a.z + pairs * m), a.order = reinterpret_cast<int32_t*>(a.slots + pairs);

  matrix(a, *up, m);
  a.x = static_cast<const uint16_t*>(X), a.ldx = ldx, a.features = static_cast<int32_t>(hidden);
  a.act = static_cast<int32_t>(act);
  hipError_t e = launch_up(a, up->type, type_x == THL_BF16, gated, stream);
  if (e == hipSuccess) {
    matrix(a, *down, hidden);
    a.x = a.u, a.ldx = ld_u, a.features = static_cast<int32_t>(m);
    e = launch_down(a, down->type, stream);
  }
  return e == hipSuccess ? THL_OK : THL_ERR_HIP;
}

}  // extern "C"
