// route.hip -- the router of a layer of experts: each token's choice of
// experts from its logits with their weights, and the gradient.
//
//   p = softmax(l) or sigmoid(l);   the topk experts of the largest p (+ bias)
//   w_t = scale * p_t,   or scale * p_t / (sum of the chosen p)
//
// One wavefront a token, its logits in registers (expert 64 i + lane in
// register i).  The values are compared as 32-bit keys of the same order.  The
// topk-th largest key is found by halving: between the largest key and the
// smallest maximum of as many groups of lanes, by the number of keys that are
// no less than the middle, done as soon as that number is topk (some six times
// for 8 of 256 experts).  The chosen ones then go to neighbouring lanes in
// the experts' order, and a lane's place is the number of chosen before it; so
// ties go to the lowest expert.  (One maximum over the wavefront a choice took
// twice the vector instructions, which bound it: 16.5 us for 16,384 tokens'
// 8 of 256 experts.)  Softmax and sigmoid keep the logits' order, so without a
// bias the logits themselves are compared, exactly.
//
// Measured, 16,384 tokens' 8 of 256 experts, fp32 logits: 11 us, bound by
// instructions (the logits' 17 MB take 3.3), and the gradient of sigmoid scores
// 7.7 us (its 17 MB and the chosen logits' lines: 5), of softmax ones 10.9 (34 MB:
// 6.7), instructions too: with every choice's value offered to every lane 12.1
// and 15.7.  With a bias the choice takes 14 us.  16 tokens' 8 of 128 3.9 us, a
// launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "../../include/thl.h"
#include "host_checks.hpp"
#include "rows.hpp"

namespace thl {
namespace {

constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxChoices = 64;

struct RouteArgs {
  const void* logits;
  const float* bias;  // NULL: none
  int32_t* ids;
  float* weights;
  const float* dweights;  // gradient only, with dlogits
  void* dlogits;
  int64_t ld, ldd, n;
  int32_t topk, experts, type, score, renormalize;
  float scale;
};

typedef unsigned v2u __attribute__((ext_vector_type(2)));

// Over the 64 lanes, in all of them: neighbours, pairs, then halves of eight and
// of sixteen mirrored, then the four rows of sixteen.
__device__ __forceinline__ float wave_sum(float v) {
  v = sum16(v);
  const unsigned u = __builtin_bit_cast(unsigned, v);
  const v2u h = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const unsigned h0 = h[0], h1 = h[1];
  v = __builtin_bit_cast(float, h0) + __builtin_bit_cast(float, h1);
  const unsigned w = __builtin_bit_cast(unsigned, v);
  const v2u a = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  const unsigned a0 = a[0], a1 = a[1];
  return __builtin_bit_cast(float, a0) + __builtin_bit_cast(float, a1);
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, true)));
}
// (over the sixteen lanes of a row)
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = dpp_max<0xb1>(v);
  v = dpp_max<0x4e>(v);
  v = dpp_max<0x141>(v);
  return dpp_max<0x140>(v);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max16(v);
  const v2u h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  v = max(h[0], h[1]);
  const v2u a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(max(a[0], a[1]))));
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_min(uint32_t v) {
  return min(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, true)));
}
// The largest of the lanes' keys, and a key that k (up to 64) keys or more
// reach: the smallest of the maxima of as many groups of lanes.
__device__ __forceinline__ uint32_t extent(uint32_t v, int k, uint32_t& least) {
  uint32_t low = v;  // per group the maximum; across groups the minimum of those
  v = dpp_max<0xb1>(v);
  low = k <= 32 ? v : dpp_min<0xb1>(low);
  v = dpp_max<0x4e>(v);
  low = k <= 16 ? v : dpp_min<0x4e>(low);
  v = dpp_max<0x141>(v);
  low = k <= 8 ? v : dpp_min<0x141>(low);
  v = dpp_max<0x140>(v);
  low = k <= 4 ? v : dpp_min<0x140>(low);
  const v2u h = __builtin_amdgcn_permlane32_swap(v, v, false, false), l = __builtin_amdgcn_permlane32_swap(low, low, false, false);
  v = max(h[0], h[1]);
  low = min(l[0], l[1]);
  const v2u a = __builtin_amdgcn_permlane16_swap(v, v, false, false), b = __builtin_amdgcn_permlane16_swap(low, low, false, false);
  least = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(min(b[0], b[1]))));
  return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(max(a[0], a[1]))));
}

// Between a wavefront's writes to LDS and its other lanes' reads of them: its
// accesses run in order, so this holds back the compiler alone.
__device__ __forceinline__ void lds_exchange() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The bits of `mask` below this lane's.
__device__ __forceinline__ uint32_t below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32),
                                   __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0));
}

// Unsigned keys that order like the values, equal ones alike (-0 and 0 too);
// 0 for an expert that cannot be chosen (-infinity or NaN).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
  const uint32_t k = b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
  return v > -INFINITY ? k : 0u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __builtin_bit_cast(float, k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// This token's logits: expert 64 i + lane, -infinity past the last.  Every load
// is issued whatever the lane, of a logit that exists, and the types part outside
// the loops: behind branches the compiler waits for each load.
template <int PER>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t row, int lane, float (&l)[PER]) {
  int at[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) at[i] = min(64 * i + lane, a.experts - 1);
  if (a.type == THL_F32) {
    const float* p = static_cast<const float*>(a.logits) + row * a.ld;
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = p[at[i]];
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(a.logits) + row * a.ld;
    uint32_t u[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) u[i] = p[at[i]];
#pragma unroll
    for (int i = 0; i < PER; ++i)
      l[i] = a.type == THL_BF16 ? __builtin_bit_cast(float, u[i] << 16)
                                : static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(u[i])));
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) l[i] = 64 * i + lane < a.experts ? l[i] : -INFINITY;
}

// The logits' exponentials under `top`, the largest one that is a number above
// -infinity, in their place (0 for one that is masked), and their sum.
template <int PER>
__device__ __forceinline__ float softmax_sum(float (&l)[PER], float top) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    l[i] = l[i] > -INFINITY ? expf(l[i] - top) : 0.0f;
    s += l[i];
  }
  return wave_sum(s);
}

template <int PER>
__global__ void __launch_bounds__(256) route_kernel(RouteArgs a) {
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int64_t waves = static_cast<int64_t>(gridDim.x) * 4;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6); row < a.n; row += waves) {
    float l[PER];
    uint32_t key[PER];
    load_logits<PER>(a, row, lane, l);
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      key[i] = key_of(l[i]);
      best = max(best, key[i]);
    }
    best = wave_max(best);
    const bool soft = a.score == THL_ROUTE_SOFTMAX;
    const float top = best ? value_of(best) : 0.0f;
    // A logit of +infinity makes every softmax score NaN, which masks no expert: the
    // logits are compared then, and the weights come out NaN.
    const bool scores = !soft || top < INFINITY;
    // with the chosen ones' sum alone in the quotient, the others' is not needed
    float x[PER], total = 1.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) x[i] = l[i];
    if (soft && (a.bias || !a.renormalize)) total = softmax_sum<PER>(x, top);
    if (a.bias && scores) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = 64 * i + lane;
        const float p = soft ? x[i] / total : sigmoid(l[i]);
        key[i] = key[i] && e < a.experts ? key_of(p + a.bias[e]) : 0u;
      }
    } else if (a.bias) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = 64 * i + lane;
        if (e < a.experts && key_of(a.bias[e]) == 0) key[i] = 0;
      }
    }
    auto count = [&](uint32_t least) {
      int c = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) c += __popcll(__ballot(key[i] >= least));
      return c;
    };
    // chosen: keys above `under`, and the first `equal` of those that are it
    const int left = count(1u), k = left < a.topk ? left : a.topk;
    uint32_t under = 0;
    int equal = 0;
    if (left > a.topk) {
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) most = max(most, key[i]);
      uint32_t above, from = 0;  // fewer than k keys are `above` or more, k or more are `from` or more
      above = extent(most, k, from) + 1;
      bool exact = false;
      while (above - from > 1 && !exact) {
        const uint32_t middle = from + (above - from) / 2;
        const int c = count(middle);
        exact = c == k;
        if (c >= k)
          from = middle;
        else
          above = middle;
      }
      under = exact ? from - 1 : from;
      if (!exact) equal = k - count(from + 1);  // (no key is the largest number: that would be a NaN's)
    }
    __shared__ uint32_t chosen[4][3][64];  // keys, experts, logits
    uint32_t(&mine)[3][64] = chosen[threadIdx.x >> 6];
    lds_exchange();
    int place = 0, same = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      bool in = key[i] > under;
      if (equal > 0) {
        const uint64_t eq = __ballot(key[i] == under);
        in = in || (key[i] == under && same + static_cast<int>(below(eq)) < equal);
        same += __popcll(eq);
      }
      const uint64_t who = __ballot(in);
      const int at = place + static_cast<int>(below(who));
      if (in) mine[0][at] = key[i], mine[1][at] = 64 * i + lane, mine[2][at] = __builtin_bit_cast(uint32_t, l[i]);
      place += __popcll(who);
    }
    lds_exchange();
    const bool one = lane < k;  // this lane's choice
    const int id = static_cast<int>(mine[1][lane]);
    const float v = __builtin_bit_cast(float, mine[2][lane]);
    int rank = 0;  // the chosen ones before it
    if (k <= 8) {  // every pair of them in one comparison: byte t is choice t's
      const int t = lane >> 3, o = lane & 7;
      const uint32_t a = mine[0][t], b = mine[0][o];
      const uint64_t before = __ballot(o < k && (b > a || (b == a && o < t)));
      rank = __popc(static_cast<uint32_t>(before >> (8 * o)) & 255u);
    } else {
      const uint32_t its = mine[0][lane];
      for (int t = 0; t < k; ++t) {
        const uint32_t other = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(its), t));
        rank += other > its || (other == its && t < lane);
      }
    }
    // Divided by the chosen ones' sum, the softmax's may be shifted by the largest of
    // them: with a bias that one can lie far below the largest of all.
    float shift = top, of = total;
    if (soft && scores && a.renormalize && a.bias) {
      const uint32_t most = wave_max(one ? key_of(v) : 0u);
      shift = most ? value_of(most) : 0.0f, of = 1.0f;
    }
    const float p = one ? (soft ? expf(v - shift) / of : sigmoid(v)) : 0.0f;
    const float sum = a.renormalize ? wave_sum(p) : 1.0f;
    if (lane < a.topk) {
      const int64_t at = row * a.topk + (one ? rank : lane);
      a.ids[at] = one ? id : -1;
      a.weights[at] = !one || sum == 0.0f ? 0.0f : a.scale * (p / sum);
    }
  }
}

// With w_t = scale * p_t / P (P = 1 where the sum is not divided by) and the
// gradient g_t of w_t, d p_t = scale * (g_t - sum_c g_c p_c / P) / P, or scale * g_t;
// then d l = p (d p - sum_e p_e d p_e) for the softmax and d p * p (1 - p) for
// the sigmoid.
//
// A wavefront takes 64 / G tokens, G lanes the choices of one: with G = 16 only
// where the choices alone have a gradient.
template <int PER, int G>
__global__ void __launch_bounds__(256) route_grad_kernel(RouteArgs a) {
  constexpr int TOKENS = 64 / G;
  __shared__ int values[4][TOKENS][64 * PER];
  int(&mine)[TOKENS][64 * PER] = values[threadIdx.x >> 6];
  const int lane = static_cast<int>(threadIdx.x) & 63, sub = lane & (G - 1);
  const int64_t step = static_cast<int64_t>(gridDim.x) * 4 * TOKENS;
  const bool soft = a.score == THL_ROUTE_SOFTMAX;
  const bool all = G == 64 && soft && !a.renormalize;  // the other experts have a gradient
  auto sum_of = [](float v) { return G == 64 ? wave_sum(v) : sum16(v); };
  auto max_of = [](uint32_t v) { return G == 64 ? wave_max(v) : max16(v); };
#pragma unroll
  for (int j = 0; j < TOKENS; ++j)
#pragma unroll
    for (int i = 0; i < PER; ++i) mine[j][64 * i + lane] = 0;
  for (int64_t row0 = (static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6)) * TOKENS; row0 < a.n; row0 += step) {
    const int64_t its = row0 + lane / G;
    int id = -1;
    float g = 0.0f, v = -INFINITY;
    if (sub < a.topk && its < a.n) {
      id = a.ids[its * a.topk + sub];
      if (id < 0 || id >= a.experts) {
        id = -1;
      } else {
        g = a.dweights[its * a.topk + sub];
        v = load_f(a.logits, a.type, its * a.ld + id);
      }
    }
    float o[PER] = {}, top = 0.0f, total = 1.0f;
    if (all) load_logits<PER>(a, row0, lane, o);
    if (soft) {
      uint32_t best = key_of(v);
      if (all) {
#pragma unroll
        for (int i = 0; i < PER; ++i) best = max(best, key_of(o[i]));
      }
      best = max_of(best);
      top = best ? value_of(best) : 0.0f;
      if (all) total = softmax_sum<PER>(o, top);
    }
    const float p = id < 0 ? 0.0f : (soft ? expf(v - top) / total : sigmoid(v));
    const float sum = a.renormalize ? sum_of(p) : 1.0f;
    float d = 0.0f;  // d l of this choice, less what all experts share
    if (a.renormalize) {
      const float w = sum == 0.0f ? 0.0f : p / sum, along = sum_of(w * g);
      if (soft)
        d = w * (g - along);
      else
        d = sum == 0.0f ? 0.0f : w * (g - along) * sigmoid(-v);
    } else if (soft) {
      const float shared = -a.scale * wave_sum(p * g) / total;
      d = p * g;
#pragma unroll
      for (int i = 0; i < PER; ++i) o[i] = o[i] != 0.0f ? shared * o[i] : 0.0f;  // (a masked one has none)
    } else {
      d = p * g * sigmoid(-v);
    }
    d = id < 0 ? 0.0f : a.scale * d;
    // The choices' values reach their experts' lanes through LDS, which is zero
    // before and after.  A lane number there first tells whether two choices of
    // a token share an expert; such are added one by one, in their order.
    int* const place = &mine[TOKENS > 1 ? lane / G : 0][id < 0 ? 0 : id];
    lds_exchange();
    if (id >= 0) *place = lane;
    lds_exchange();
    const bool twice = __ballot(id >= 0 && *place != lane) != 0;
    lds_exchange();
    if (id >= 0) *place = twice ? 0 : __builtin_bit_cast(int, d);
    lds_exchange();
#pragma unroll
    for (int j = 0; j < TOKENS; ++j) {
      const int64_t row = row0 + j;
      if (row >= a.n) break;
      float to[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) to[i] = o[i] + __builtin_bit_cast(float, mine[j][64 * i + lane]);
      if (twice) {
        for (int t = 0; t < a.topk; ++t) {
          const int e = __builtin_amdgcn_readlane(id, G * j + t);
          const float dt = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, d), G * j + t));
          const float one = (e & 63) == lane ? dt : 0.0f;
#pragma unroll
          for (int i = 0; i < PER; ++i)
            if (e >> 6 == i) to[i] += one;
        }
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = 64 * i + lane;
        if (e >= a.experts) continue;
        const int64_t at = row * a.ldd + e;
        if (a.type == THL_F32)
          static_cast<float*>(a.dlogits)[at] = to[i];
        else if (a.type == THL_F16)
          static_cast<_Float16*>(a.dlogits)[at] = static_cast<_Float16>(to[i]);
        else
          static_cast<__bf16*>(a.dlogits)[at] = static_cast<__bf16>(to[i]);
      }
    }
    lds_exchange();
    if (id >= 0) *place = 0;
  }
}

template <int PER>
hipError_t launch(RouteArgs& a, hipStream_t st) {
  const void* f = reinterpret_cast<const void*>(&route_kernel<PER>);
  int64_t tokens = 4;  // of a workgroup
  if (a.dlogits) {
    f = reinterpret_cast<const void*>(&route_grad_kernel<PER, 64>);
    // Four tokens a wavefront, where there are tokens for it: sigmoid scores of 64,
    // 128 and 256 experts, 32,768 tokens 6.3, 8.6 and 11.3 us, 10.8, 11.5 and 14.0
    // one a wavefront; 4,096 tokens 3.2, 3.8 and 4.9 us, 3.3, 3.6 and 4.3.  512
    // experts: 24.0 for 22.8.
    if constexpr (PER <= 4) {
      if (a.topk <= 16 && (a.score != THL_ROUTE_SOFTMAX || a.renormalize) && a.n >= 4096 * PER) {
        f = reinterpret_cast<const void*>(&route_grad_kernel<PER, 16>);
        tokens = 16;
      }
    }
  }
  void* args[] = {&a};
  const int64_t blocks = (a.n + tokens - 1) / tokens;
  return hipLaunchKernel(f, dim3(static_cast<unsigned>(blocks < 65536 ? blocks : 65536)), dim3(256), args, 0, st);
}
hipError_t launch(RouteArgs& a, hipStream_t st) {
  if (a.experts <= 64) return launch<1>(a, st);
  if (a.experts <= 128) return launch<2>(a, st);
  if (a.experts <= 256) return launch<4>(a, st);
  return a.experts <= 512 ? launch<8>(a, st) : launch<16>(a, st);
}

bool big(int64_t v) { return v > INT32_MAX; }
bool off(const void* p, thl_dtype t) { return reinterpret_cast<uintptr_t>(p) % bytes_of(t, 1) != 0; }

thl_status check(int64_t n, int64_t topk, int64_t experts, int64_t ldl, const thl_route* how) {
  if (!how || n < 0 || topk < 0 || experts < 1) return THL_ERR_INVALID;
  if (experts > kMaxExperts || topk > kMaxChoices || big(n) || big(ldl)) return THL_ERR_UNSUPPORTED;
  if (!is_float_io(how->type)) return THL_ERR_UNSUPPORTED;
  if (how->score != THL_ROUTE_SOFTMAX && how->score != THL_ROUTE_SIGMOID) return THL_ERR_INVALID;
  if (!std::isfinite(how->scale)) return THL_ERR_INVALID;
  return ldl < experts ? THL_ERR_INVALID : THL_OK;
}

}  // namespace
}  // namespace thl

using namespace thl;

extern "C" {

thl_status thl_moe_route(int64_t n, int64_t topk, int64_t experts, const void* L, int64_t ldl, const float* bias,
                         const thl_route* how, int32_t* ids, float* weights, struct ihipStream_t* stream) {
  const thl_status s = check(n, topk, experts, ldl, how);
  if (s != THL_OK) return s;
  if (n == 0 || topk == 0) return THL_OK;
  if (!L || !ids || !weights) return THL_ERR_INVALID;
  if (off(L, how->type) || off(bias, THL_F32) || off(ids, THL_I32) || off(weights, THL_F32)) return THL_ERR_MISALIGNED;
  const Range rl = matrix_range(L, how->type, experts, n, ldl), rb = vector_range(bias, experts, 4);
  const Range ri = vector_range(ids, n * topk, 4), rw = vector_range(weights, n * topk, 4);
  if (overlaps(ri, rl) || overlaps(ri, rb) || overlaps(rw, rl) || overlaps(rw, rb) || overlaps(ri, rw))
    return THL_ERR_INVALID;
  RouteArgs a{};
  a.logits = L, a.bias = bias, a.ids = ids, a.weights = weights, a.ld = ldl, a.n = n;
  a.topk = static_cast<int32_t>(topk), a.experts = static_cast<int32_t>(experts), a.type = how->type;
  a.score = how->score, a.renormalize = how->renormalize != 0, a.scale = how->scale;
  return launch(a, stream) == hipSuccess ? THL_OK : THL_ERR_HIP;
}

thl_status thl_moe_route_backward(int64_t n, int64_t topk, int64_t experts, const void* L, int64_t ldl,
                                  const thl_route* how, const int32_t* ids, const float* dweights, void* DL,
                                  int64_t lddl, struct ihipStream_t* stream) {
  const thl_status s = check(n, topk, experts, ldl, how);
  if (s != THL_OK) return s;
  if (big(lddl)) return THL_ERR_UNSUPPORTED;
  if (lddl < experts) return THL_ERR_INVALID;
  if (n == 0) return THL_OK;
  if (!L || !DL || (topk > 0 && (!ids || !dweights))) return THL_ERR_INVALID;
  if (off(L, how->type) || off(DL, how->type) || off(ids, THL_I32) || off(dweights, THL_F32)) return THL_ERR_MISALIGNED;
  // DL may be L exactly
  const Range rl = matrix_range(L, how->type, experts, n, ldl), rd = matrix_range(DL, how->type, experts, n, lddl);
  if ((overlaps(rd, rl) && !(DL == L && lddl == ldl)) || overlaps(rd, vector_range(ids, n * topk, 4)) ||
      overlaps(rd, vector_range(dweights, n * topk, 4)))
    return THL_ERR_INVALID;
  RouteArgs a{};
  a.logits = L, a.ids = const_cast<int32_t*>(ids), a.dweights = dweights, a.dlogits = DL, a.ld = ldl, a.ldd = lddl;
  a.n = n, a.topk = static_cast<int32_t>(topk), a.experts = static_cast<int32_t>(experts), a.type = how->type;
  a.score = how->score, a.renormalize = how->renormalize != 0, a.scale = how->scale;
  return launch(a, stream) == hipSuccess ? THL_OK : THL_ERR_HIP;
}

}  // extern "C"
