// moe.hip -- tokens sorted by expert and back: what stands before and after
// a grouped product whose problems are a layer's experts.
//
//   sort      each (token, choice)'s place in a stable order by expert, and
//             each expert's first place
//   gather    row place(j, t) of the experts' operand = token j's row
//   combine   token j's row = sum over t of weight(j, t) * row place(j, t);
//             without weights it is gather's gradient
//   gradient  of combine: row place(j, t) = weight(j, t) * dy(j), and
//             dweight(j, t) = <dy(j), row place(j, t)>
//
// The sort is bound by launch latency, the rest by HBM: each source row is
// read once and each destination row written once.  Nothing is added with
// atomics whose order could change a result: places come from counts, and
// sums over a token's choices run in the order of the choices.
//
// Measured with 4,096 bf16 features: sort and gather of 8,192 tokens' eight
// choices 122 us (4.9 TB/s, most of it writes; the sort is 10 us of it), of 24
// tokens 8.6 us (two launches), combine of the same 98 us (6.0 TB/s), its
// gradient for 4,096 tokens' two choices of 5,126 features 40 us (5.2 TB/s).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/thl.h"
#include "host_checks.hpp"
#include "rows.hpp"

namespace thl {
namespace {

// ---------------------------------------------------------------- sort
// A counting sort of n * topk entries, flat index f = token * topk + choice.
// Entries are cut into up to kSortBlocks contiguous chunks, one per
// workgroup, and a chunk into one contiguous segment per wavefront.  The
// place of an entry is the number of entries of smaller experts, plus those
// of its own expert in earlier workgroups, in earlier wavefronts, and earlier
// in its own wavefront: counts only, so the order is the stable one whatever
// the timing.  A single workgroup needs one launch; more need their counts
// first (sort_count).
constexpr int kSortWaves = 8;
constexpr int kSortThreads = kSortWaves * 64;
constexpr int kSortBlocks = 256;
constexpr int kMaxExperts = 1024;   // counts of eight wavefronts in 32 KB of LDS
constexpr int64_t kSortOne = 4096;  // entries one workgroup takes alone
constexpr int64_t kSortChunk = 1024;  // entries at least per workgroup otherwise

struct SortArgs {
  const void* ids;
  int64_t ld_ids;
  int32_t ids_bytes, topk, experts, total;
  int32_t chunk, blocks;  // entries per workgroup, workgroups
  int32_t* rows;
  int32_t* offsets;
  int32_t* order;   // NULL: not wanted
  int32_t* counts;  // blocks x experts, more than one workgroup only
};

// The experts of entries f, f + step, .. (four of them), -1 for one that is
// dropped or lies past `end`; the loads go out together.
__device__ __forceinline__ void experts_of(const SortArgs& a, int f, int step, int end, int (&e)[4]) {
  int64_t id[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = f + i * step < end ? f + i * step : end - 1;
    const int64_t k = a.ld_ids == a.topk ? at : static_cast<int64_t>(at / a.topk) * a.ld_ids + at % a.topk;
    // the low and the high half of a 64-bit id (of a 32-bit one the same word)
    const int32_t* p = static_cast<const int32_t*>(a.ids) + (a.ids_bytes == 8 ? 2 * k : k);
    const int32_t lo = p[0], hi = p[a.ids_bytes == 8 ? 1 : 0];
    id[i] = a.ids_bytes == 8 ? static_cast<int64_t>((static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32) |
                                                    static_cast<uint32_t>(lo))
                             : lo;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    e[i] = f + i * step < end && id[i] >= 0 && id[i] < a.experts ? static_cast<int>(id[i]) : -1;
}

__global__ void __launch_bounds__(kSortThreads) sort_count(SortArgs a) {
  __shared__ int count[kMaxExperts];
  const int t = static_cast<int>(threadIdx.x);
  for (int e = t; e < a.experts; e += kSortThreads) count[e] = 0;
  __syncthreads();
  const int lo = static_cast<int>(blockIdx.x) * a.chunk;
  const int hi = a.total - lo < a.chunk ? a.total : lo + a.chunk;
  for (int f = lo + t; f < hi; f += 4 * kSortThreads) {
    int e[4];
    experts_of(a, f, kSortThreads, hi, e);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e[i] >= 0) atomicAdd(&count[e[i]], 1);
  }
  __syncthreads();
  for (int e = t; e < a.experts; e += kSortThreads)
    a.counts[static_cast<int64_t>(blockIdx.x) * a.experts + e] = count[e];
}

__global__ void __launch_bounds__(kSortThreads) sort_place(SortArgs a) {
  __shared__ int next[kSortWaves][kMaxExperts];  // counts, then the next place, per wavefront and expert
  __shared__ int all[kMaxExperts], before[kMaxExperts];  // entries of an expert: all, and in earlier workgroups
  __shared__ int wave_sum[kSortWaves];
  const int t = static_cast<int>(threadIdx.x), lane = t & 63, wave = t >> 6;
  const int me = static_cast<int>(blockIdx.x);
  for (int e = t; e < a.experts; e += kSortThreads) {
    for (int w = 0; w < kSortWaves; ++w) next[w][e] = 0;
    all[e] = 0;
    before[e] = 0;
  }
  __syncthreads();

  // this wavefront's segment of this workgroup's chunk
  const int lo = me * a.chunk, hi = a.total - lo < a.chunk ? a.total : lo + a.chunk;
  const int seg = ((hi - lo + kSortWaves - 1) / kSortWaves + 63) & ~63;
  const int s0 = lo + wave * seg < hi ? lo + wave * seg : hi, s1 = hi - s0 < seg ? hi : s0 + seg;
  int first[4] = {-1, -1, -1, -1};  // the segment's first four runs of 64, kept for the second pass
  for (int f = s0; f < s1; f += 256) {
    int e[4];
    experts_of(a, f + lane, 64, s1, e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (f == s0) first[i] = e[i];
      if (e[i] >= 0) atomicAdd(&next[wave][e[i]], 1);
    }
  }
  if (a.blocks > 1) {
    // A thread adds one expert's counts of every `slices`-th workgroup.
    const int cols = a.experts < kSortThreads ? a.experts : kSortThreads, slices = kSortThreads / cols;
    const int sl = t / cols;
    for (int e = sl < slices ? t - sl * cols : a.experts; e < a.experts; e += cols) {
      int sum = 0, sum_before = 0;
      for (int b = sl; b < a.blocks; b += 16 * slices) {
        int c[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const int at = b + q * slices < a.blocks ? b + q * slices : b;
          c[q] = a.counts[static_cast<int64_t>(at) * a.experts + e];
        }
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const int at = b + q * slices;
          sum += at < a.blocks ? c[q] : 0;
          sum_before += at < me && at < a.blocks ? c[q] : 0;
        }
      }
      if (sum != 0) atomicAdd(&all[e], sum);
      if (sum_before != 0) atomicAdd(&before[e], sum_before);
    }
  }
  __syncthreads();

  // experts 2t, 2t+1: exclusive sum over the experts
  int mine[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 2 * t + i;
    if (e >= a.experts) continue;
    if (a.blocks > 1) {
      mine[i] = all[e];
    } else {
      for (int w = 0; w < kSortWaves; ++w) mine[i] += next[w][e];
    }
  }
  int run = mine[0] + mine[1];
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(run, d);
    if (lane >= d) run += o;
  }
  if (lane == 63) wave_sum[wave] = run;
  __syncthreads();
  int start = run - mine[0] - mine[1];
  for (int w = 0; w < wave; ++w) start += wave_sum[w];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 2 * t + i;
    if (e < a.experts) {
      if (me == 0) {
        a.offsets[e] = start;
        if (e == a.experts - 1) a.offsets[a.experts] = start + mine[i];
      }
      int p = start + before[e];
      for (int w = 0; w < kSortWaves; ++w) {
        const int c = next[w][e];
        next[w][e] = p;
        p += c;
      }
      start += mine[i];
    }
  }
  __syncthreads();

  // places: lanes with one expert take consecutive ones, in lane order
  const int bits = 32 - __builtin_clz(static_cast<unsigned>(a.experts));
  for (int f = s0; f < s1; f += 256) {
    int es[4];
    if (f == s0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) es[i] = first[i];
    } else {
      experts_of(a, f + lane, 64, s1, es);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = es[i], at = f + 64 * i + lane;
      uint64_t same = __ballot(e >= 0);
      for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((e >> b) & 1);
        same &= ((e >> b) & 1) ? set : ~set;
      }
      if (e >= 0) {
        const int rank = __popcll(same & ((1ull << lane) - 1ull));
        const int leader = __ffsll(static_cast<unsigned long long>(same)) - 1;
        int base = 0;
        if (rank == 0) base = atomicAdd(&next[wave][e], __popcll(same));
        const int place = __shfl(base, leader) + rank;
        a.rows[at] = place;
        if (a.order) a.order[place] = at;
      } else if (at < s1) {
        a.rows[at] = -1;
      }
    }
  }
}

// ---------------------------------------------------------------- gather
typedef uint32_t v4u_a1 __attribute__((ext_vector_type(4), aligned(1)));

struct GatherArgs {
  const uint8_t* x;
  uint8_t* y;
  const uint8_t* sfx;
  uint8_t* sfy;
  int64_t ldx, ldy, ld_sfx, ld_sfy;  // bytes
  const int32_t* rows;
  int64_t n, rows_y;
  int64_t row_bytes, sf_bytes;  // per row
  int64_t units, units_x;       // 16-byte units of a row with its scales, and of the row alone
  int32_t topk, lanes;          // lanes per token, a power of two up to the workgroup
};

// One piece of a short row, from s to every place of the token.
template <class V>
__device__ __forceinline__ void copy_piece(const GatherArgs& a, const uint8_t* s, uint8_t* dst, int64_t ld_dst,
                                           const int32_t* places) {
  const V v = *reinterpret_cast<const V*>(s);
  for (int c = 0; c < a.topk; ++c) {
    const int64_t p = places[c];
    if (p >= 0 && p < a.rows_y) *reinterpret_cast<V*>(dst + p * ld_dst) = v;
  }
}

// `lanes` lanes read a token's row in 16-byte units and write each unit to
// every place of the token.  The last unit of a row that is no multiple of 16
// bytes ends with it, over the unit before (the same bytes twice): byte by
// byte it took 16.8 us instead of 7.8 for 109 tokens of 843 bytes to six
// places each.  Rows below 16 bytes go in pieces of eight, four, two and one.
__global__ void __launch_bounds__(256) moe_gather_kernel(GatherArgs a) {
  const int t = static_cast<int>(threadIdx.x);
  const int per = 256 / a.lanes;
  for (int64_t u = static_cast<int64_t>(blockIdx.y) * a.lanes + (t & (a.lanes - 1)); u < a.units;
       u += static_cast<int64_t>(gridDim.y) * a.lanes) {
    const bool sf = u >= a.units_x;
    const int64_t bytes = sf ? a.sf_bytes : a.row_bytes, first = 16 * (sf ? u - a.units_x : u);
    const int64_t at = bytes < 16 ? 0 : (first + 16 <= bytes ? first : bytes - 16);
    const uint8_t* src = (sf ? a.sfx : a.x) + at;
    uint8_t* dst = (sf ? a.sfy : a.y) + at;
    const int64_t ld_src = sf ? a.ld_sfx : a.ldx, ld_dst = sf ? a.ld_sfy : a.ldy;
    for (int64_t j = static_cast<int64_t>(blockIdx.x) * per + t / a.lanes; j < a.n;
         j += static_cast<int64_t>(gridDim.x) * per) {
      const uint8_t* s = src + j * ld_src;
      const int32_t* places = a.rows + j * a.topk;
      if (bytes >= 16) {
        const v4u_a1 v = __builtin_nontemporal_load(reinterpret_cast<const v4u_a1*>(s));
        for (int c = 0; c < a.topk; ++c) {
          const int64_t p = places[c];
          if (p >= 0 && p < a.rows_y) *reinterpret_cast<v4u_a1*>(dst + p * ld_dst) = v;
        }
      } else {
        int64_t o = 0;
        if (bytes & 8) copy_piece<v2u_a1>(a, s, dst, ld_dst, places), o = 8;
        if (bytes & 4) copy_piece<u32_a1>(a, s + o, dst + o, ld_dst, places), o += 4;
        if (bytes & 2) copy_piece<u16_a1>(a, s + o, dst + o, ld_dst, places), o += 2;
        if (bytes & 1) copy_piece<uint8_t>(a, s + o, dst + o, ld_dst, places);
      }
    }
  }
}

// ---------------------------------------------------------------- combine
struct CombineArgs {
  const void* x;
  void* y;
  const int32_t* rows;
  const float* weights;  // NULL: ones
  int64_t ldx, ldy, n, rows_x;
  int32_t m, topk, lanes, x_type, y_type;
};

// `lanes` lanes take eight features each of a token's row; KB of the token's
// rows are in flight at a time.  ONE: a workgroup has one token, whose places
// and weights are then scalars.  Choices without a row load one that is there
// (a load behind a branch would be waited for by itself) and are not added.
template <int XB, int RUNS, int KB, bool ONE>
__global__ void __launch_bounds__(256) moe_combine_kernel(CombineArgs a) {
  const int t = static_cast<int>(threadIdx.x);
  const int per = ONE ? 1 : 256 / a.lanes;
  const int64_t e64 = 8 * (static_cast<int64_t>(blockIdx.y) * (ONE ? 256 : a.lanes) + (ONE ? t : t & (a.lanes - 1)));
  if (e64 >= a.m) return;
  const int e = static_cast<int>(e64), m = a.m;
  const bool bf = a.x_type == THL_BF16;
  for (int64_t j = static_cast<int64_t>(blockIdx.x) * per + (ONE ? 0 : t / a.lanes); j < a.n;
       j += static_cast<int64_t>(gridDim.x) * per) {
    float acc[8] = {};
    for (int c0 = 0; c0 < a.topk; c0 += KB) {
      Raw8<XB> r[KB];
      float w[KB];
      bool on[KB];
      int64_t last = 0;
#pragma unroll
      for (int i = 0; i < KB; ++i) {
        const int c = c0 + i < a.topk ? c0 + i : a.topk - 1;
        const int64_t p = a.rows[j * a.topk + c];
        on[i] = c0 + i < a.topk && p >= 0 && p < a.rows_x;
        last = on[i] ? p : last;
        r[i] = load_run<XB, RUNS>(a.x, last * a.ldx, e, m);
        w[i] = a.weights ? a.weights[j * a.topk + c] : 1.0f;
      }
#pragma unroll
      for (int i = 0; i < KB; ++i) {
        if (on[i]) {
          float v[8];
          settle<XB, RUNS>(r[i], e, m);
          to_f8<XB>(r[i], bf, v);
#pragma unroll
          for (int q = 0; q < 8; ++q) acc[q] += w[i] * v[q];
        }
      }
    }
    store8_f(a.y, a.y_type, j * a.ldy + e, acc, m - e < 8 ? m - e : 8);
  }
}

struct CombineGradArgs {
  const void* dy;
  const void* x;
  void* dx;         // NULL: not wanted
  float* dweights;  // NULL: not wanted
  const int32_t* rows;
  const float* weights;
  int64_t lddy, ldx, lddx, n, rows_x;
  int32_t m, topk, dy_type, x_type;
};

// WPT wavefronts per token; KB of its choices at a time share each read of
// dy.  XB, DB: bytes of an element of X / DX and of DY.  DOT: dweights is
// wanted (X is read).  Choices without a row as in combine.
template <int XB, int DB, int RUNS, int WPT, int KB, bool DOT>
__global__ void __launch_bounds__(WPT * 64) moe_combine_grad_kernel(CombineGradArgs a) {
  __shared__ float red[2][KB * WPT];
  const int t = static_cast<int>(threadIdx.x), m = a.m;
  const bool x_bf = a.x_type == THL_BF16, d_bf = a.dy_type == THL_BF16;
  int parity = 0;
  for (int64_t j = blockIdx.x; j < a.n; j += gridDim.x) {
    for (int c0 = 0; c0 < a.topk; c0 += KB, parity ^= 1) {
      int64_t place[KB], last = 0;
      float w[KB], dot[KB];
      bool on[KB];
#pragma unroll
      for (int i = 0; i < KB; ++i) {
        const int c = c0 + i < a.topk ? c0 + i : a.topk - 1;
        const int64_t p = a.rows[j * a.topk + c];
        on[i] = c0 + i < a.topk && p >= 0 && p < a.rows_x;
        last = on[i] ? p : last;
        place[i] = last;
        w[i] = a.dx ? a.weights[j * a.topk + c] : 0.0f;
        dot[i] = 0.0f;
      }
      for (int e = 8 * t; e < m; e += 8 * WPT * 64) {
        Raw8<DB> dr = load_run<DB, RUNS>(a.dy, j * a.lddy, e, m);
        Raw8<XB> xr[KB];
        if constexpr (DOT) {
#pragma unroll
          for (int i = 0; i < KB; ++i) xr[i] = load_run<XB, RUNS>(a.x, place[i] * a.ldx, e, m);
        }
        float d[8];
        settle<DB, RUNS>(dr, e, m);
        to_f8<DB>(dr, d_bf, d);
#pragma unroll
        for (int i = 0; i < KB; ++i) {
          if (!on[i]) continue;
          if constexpr (DOT) {
            float v[8];
            settle<XB, RUNS>(xr[i], e, m);
            to_f8<XB>(xr[i], x_bf, v);
#pragma unroll
            for (int q = 0; q < 8; ++q) dot[i] += d[q] * v[q];
          }
          if (a.dx) {
            float o[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] = w[i] * d[q];
            store8_f(a.dx, a.x_type, place[i] * a.lddx + e, o, m - e < 8 ? m - e : 8);
          }
        }
      }
      if constexpr (DOT) {
        row_sum<KB, WPT>(dot, red[parity]);
        if (t == 0) {
#pragma unroll
          for (int i = 0; i < KB; ++i)
            if (c0 + i < a.topk) a.dweights[j * a.topk + c0 + i] = dot[i];
        }
      }
    }
  }
}

// ---------------------------------------------------------------- launch

hipError_t launch(const void* f, dim3 grid, int block, void* arg, hipStream_t st) {
  void* args[] = {arg};
  return hipLaunchKernel(f, grid, dim3(block), args, 0, st);
}

__global__ void __launch_bounds__(256) zeros_kernel(float* p, int64_t n) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256)
    p[i] = 0.0f;
}
hipError_t launch_zeros(float* p, int64_t n, hipStream_t st) {
  void* args[] = {&p, &n};
  const int64_t blocks = (n + 255) / 256;
  return hipLaunchKernel(reinterpret_cast<const void*>(&zeros_kernel),
                         dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), dim3(256), args, 0, st);
}

// Lanes per token for `units` pieces of work: a power of two up to 256.
int lanes_for(int64_t units) {
  int l = 1;
  while (l < 256 && l < units) l *= 2;
  return l;
}

// Tokens in x (each workgroup then walks on), pieces of a token in y (a
// gather of 2^26 features of four bytes walks on there too; combine's pieces,
// of eight features, are 2^15 workgroups at most).
dim3 token_grid(int64_t n, int64_t units, int lanes) {
  const int64_t per = 256 / lanes, gy = (units + lanes - 1) / lanes;
  int64_t gx = (n + per - 1) / per;
  if (gx > 65536) gx = 65536;
  return dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy < 65535 ? gy : 65535));
}

// A token of up to 1,024 features goes to one wavefront, longer ones to four.
template <int XB, int DB, int RUNS, bool DOT>
hipError_t launch_combine_grad(CombineGradArgs& a, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.n < 65536 ? a.n : 65536));
#define THL_CGRAD(WPT, KB)                                                                                         \
  return launch(reinterpret_cast<const void*>(&moe_combine_grad_kernel<XB, DB, RUNS, WPT, KB, DOT>), grid, WPT * 64, \
                &a, st)
  if (a.m <= 1024) {
    if (a.topk <= 2) THL_CGRAD(1, 2);
    THL_CGRAD(1, 8);
  }
  if constexpr (RUNS != RUNS_TINY) {
    if (a.topk <= 2) THL_CGRAD(4, 2);
    if (a.topk <= 4) THL_CGRAD(4, 4);
    THL_CGRAD(4, 8);
  }
  return hipErrorInvalidValue;
#undef THL_CGRAD
}
template <int XB, int DB>
hipError_t launch_combine_grad(CombineGradArgs& a, hipStream_t st) {
  const int runs = runs_of(a.m);
  if (a.dweights) {
    if (runs == RUNS_TINY) return launch_combine_grad<XB, DB, RUNS_TINY, true>(a, st);
    return runs == RUNS_WHOLE ? launch_combine_grad<XB, DB, RUNS_WHOLE, true>(a, st)
                              : launch_combine_grad<XB, DB, RUNS_RAGGED, true>(a, st);
  }
  if (runs == RUNS_TINY) return launch_combine_grad<XB, DB, RUNS_TINY, false>(a, st);
  return runs == RUNS_WHOLE ? launch_combine_grad<XB, DB, RUNS_WHOLE, false>(a, st)
                            : launch_combine_grad<XB, DB, RUNS_RAGGED, false>(a, st);
}

template <int XB, int RUNS>
hipError_t launch_combine(CombineArgs& a, dim3 grid, hipStream_t st) {
#define THL_COMBINE(KB, ONE) \
  return launch(reinterpret_cast<const void*>(&moe_combine_kernel<XB, RUNS, KB, ONE>), grid, 256, &a, st)
  if (a.lanes == 256) {
    if constexpr (RUNS != RUNS_TINY) {
      if (a.topk <= 2) THL_COMBINE(2, true);
      if (a.topk <= 4) THL_COMBINE(4, true);
      THL_COMBINE(8, true);
    }
    return hipErrorInvalidValue;
  }
  if (a.topk <= 2) THL_COMBINE(2, false);
  THL_COMBINE(8, false);
#undef THL_COMBINE
}
template <int XB>
hipError_t launch_combine(CombineArgs& a, dim3 grid, hipStream_t st) {
  const int runs = runs_of(a.m);
  if (runs == RUNS_TINY) return launch_combine<XB, RUNS_TINY>(a, grid, st);
  return runs == RUNS_WHOLE ? launch_combine<XB, RUNS_WHOLE>(a, grid, st)
                            : launch_combine<XB, RUNS_RAGGED>(a, grid, st);
}

bool big(int64_t v) { return v > INT32_MAX; }
bool bad_ld(int64_t ld, int64_t m) { return ld < (m > 1 ? m : 1); }
bool off4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 != 0; }
bool misaligned(const void* p, thl_dtype t) { return reinterpret_cast<uintptr_t>(p) % bytes_of(t, 1) != 0; }

// Sizes every entry point shares: tokens, choices, and rows of the experts'
// array (entries are counted in 32 bits: up to 2^30 of them).
thl_status check_sizes(int64_t n, int64_t topk, int64_t rows) {
  if (n < 0 || topk < 0 || rows < 0) return THL_ERR_INVALID;
  if (big(n) || big(topk) || big(rows) || (topk > 0 && n > (INT64_C(1) << 30) / topk)) return THL_ERR_UNSUPPORTED;
  return THL_OK;
}

// Workgroups of the sort and entries per workgroup.
void sort_split(int64_t total, int32_t* blocks, int32_t* chunk) {
  int64_t c = kSortOne;
  if (total > kSortOne) {
    c = (total + kSortBlocks - 1) / kSortBlocks;
    c = c < kSortChunk ? kSortChunk : (c + kSortThreads - 1) / kSortThreads * kSortThreads;
  }
  *chunk = static_cast<int32_t>(c);
  *blocks = static_cast<int32_t>((total + c - 1) / c);
}

}  // namespace
}  // namespace thl

using namespace thl;

extern "C" {

size_t thl_moe_sort_workspace(int64_t n, int64_t topk, int64_t experts) {
  if (check_sizes(n, topk, 0) != THL_OK || n * topk == 0 || experts <= 0 || experts > kMaxExperts) return 0;
  int32_t blocks, chunk;
  sort_split(n * topk, &blocks, &chunk);
  return blocks == 1 ? 0 : static_cast<size_t>(blocks) * static_cast<size_t>(experts) * sizeof(int32_t);
}

thl_status thl_moe_sort(int64_t n, int64_t topk, int64_t experts, const void* ids, int64_t ld_ids, int ids_bytes,
                        int32_t* rows, int32_t* offsets, int32_t* order, void* workspace, size_t workspace_bytes,
                        struct ihipStream_t* stream) {
  const thl_status st = check_sizes(n, topk, 0);
  if (st != THL_OK) return st;
  if (experts < 1) return THL_ERR_INVALID;
  if (experts > kMaxExperts || big(ld_ids)) return THL_ERR_UNSUPPORTED;
  if (ids_bytes != 4 && ids_bytes != 8) return THL_ERR_UNSUPPORTED;
  if (bad_ld(ld_ids, topk) || !offsets) return THL_ERR_INVALID;
  const int64_t total = n * topk;
  if (total > 0 && (!ids || !rows)) return THL_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(ids) % static_cast<unsigned>(ids_bytes) != 0 || off4(rows) || off4(offsets) ||
      off4(order))
    return THL_ERR_MISALIGNED;
  const size_t need = thl_moe_sort_workspace(n, topk, experts);
  if (need && (!workspace || workspace_bytes < need)) return THL_ERR_INVALID;
  if (need && off4(workspace)) return THL_ERR_MISALIGNED;
  const Range r[] = {vector_range(ids, total > 0 ? (n - 1) * ld_ids + topk : 0, ids_bytes), vector_range(rows, total, 4),
                     vector_range(offsets, experts + 1, 4), vector_range(order, total, 4),
                     need ? vector_range(workspace, static_cast<int64_t>(need), 1) : Range{}};
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < i; ++j)
      if (overlaps(r[i], r[j])) return THL_ERR_INVALID;

  SortArgs a{};
  a.ids = ids, a.ld_ids = ld_ids, a.ids_bytes = ids_bytes;
  a.topk = static_cast<int32_t>(topk), a.experts = static_cast<int32_t>(experts);
  a.total = static_cast<int32_t>(total);
  a.rows = rows, a.offsets = offsets, a.order = order, a.counts = static_cast<int32_t*>(workspace);
  sort_split(total, &a.blocks, &a.chunk);
  if (total == 0) a.blocks = 1;  // no entries: the offsets are still written
  hipError_t e = hipSuccess;
  if (a.blocks > 1)
    e = launch(reinterpret_cast<const void*>(&sort_count), dim3(a.blocks), kSortThreads, &a, stream);
  if (e == hipSuccess) e = launch(reinterpret_cast<const void*>(&sort_place), dim3(a.blocks), kSortThreads, &a, stream);
  return e == hipSuccess ? THL_OK : THL_ERR_HIP;
}

thl_status thl_moe_gather(int64_t m, int64_t n, int64_t topk, const void* X, int64_t ldx, const uint8_t* sfx,
                          int64_t ld_sfx, const int32_t* rows, int64_t rows_y, void* Y, int64_t ldy, uint8_t* sfy,
                          int64_t ld_sfy, thl_dtype type, struct ihipStream_t* stream) {
  const thl_status st = check_sizes(n, topk, rows_y);
  if (st != THL_OK) return st;
  if (m < 0) return THL_ERR_INVALID;
  if (m > kMaxFeatures || big(ldx) || big(ldy) || big(ld_sfx) || big(ld_sfy)) return THL_ERR_UNSUPPORTED;
  if (bytes_of(type, 1) == 0) return THL_ERR_UNSUPPORTED;
  // rows start on whole bytes
  const int64_t whole = bytes_of(type, 2) == 1 ? 2 : (type == THL_E2M3 || type == THL_E3M2 ? 4 : 1);
  if (bad_ld(ldx, m) || bad_ld(ldy, m) || ldx % whole != 0 || ldy % whole != 0) return THL_ERR_INVALID;
  if (!sfx != !sfy) return THL_ERR_INVALID;
  if (sfx && (bad_ld(ld_sfx, (m + 31) / 32) || bad_ld(ld_sfy, (m + 31) / 32))) return THL_ERR_INVALID;
  if (m == 0 || n == 0 || topk == 0 || rows_y == 0) return THL_OK;
  if (!X || !Y || !rows) return THL_ERR_INVALID;
  if (off4(rows)) return THL_ERR_MISALIGNED;
  const Range rx = matrix_range(X, type, m, n, ldx), rr = vector_range(rows, n * topk, 4);
  const Range ry = matrix_range(Y, type, m, rows_y, ldy);
  const Range fx = matrix_range(sfx, THL_E8M0, (m + 31) / 32, n, ld_sfx);
  const Range fy = matrix_range(sfy, THL_E8M0, (m + 31) / 32, rows_y, ld_sfy);
  for (const Range& o : {rx, rr, fx})
    if (overlaps(ry, o) || overlaps(fy, o)) return THL_ERR_INVALID;
  if (overlaps(ry, fy)) return THL_ERR_INVALID;

  GatherArgs a{};
  a.x = static_cast<const uint8_t*>(X), a.y = static_cast<uint8_t*>(Y), a.sfx = sfx, a.sfy = sfy;
  a.ldx = bytes_of(type, ldx), a.ldy = bytes_of(type, ldy), a.ld_sfx = ld_sfx, a.ld_sfy = ld_sfy;
  a.rows = rows, a.n = n, a.rows_y = rows_y, a.topk = static_cast<int32_t>(topk);
  a.row_bytes = bytes_of(type, m), a.sf_bytes = sfx ? (m + 31) / 32 : 0;
  a.units_x = (a.row_bytes + 15) / 16, a.units = a.units_x + (a.sf_bytes + 15) / 16;
  a.lanes = lanes_for(a.units);
  const dim3 grid = token_grid(n, a.units, a.lanes);
  return launch(reinterpret_cast<const void*>(&moe_gather_kernel), grid, 256, &a, stream) == hipSuccess ? THL_OK
                                                                                                         : THL_ERR_HIP;
}

thl_status thl_moe_combine(int64_t m, int64_t n, int64_t topk, const void* X, int64_t ldx, int64_t rows_x,
                           const int32_t* rows, const float* weights, void* Y, int64_t ldy, thl_dtype type_x,
                           thl_dtype type_y, struct ihipStream_t* stream) {
  const thl_status st = check_sizes(n, topk, rows_x);
  if (st != THL_OK) return st;
  if (m < 0) return THL_ERR_INVALID;
  if (m > kMaxFeatures || big(ldx) || big(ldy)) return THL_ERR_UNSUPPORTED;
  if (!is_float_io(type_x) || !is_float_io(type_y)) return THL_ERR_UNSUPPORTED;
  if (bad_ld(ldx, m) || bad_ld(ldy, m)) return THL_ERR_INVALID;
  if (m == 0 || n == 0) return THL_OK;
  if (!Y || (topk > 0 && (!rows || (rows_x > 0 && !X)))) return THL_ERR_INVALID;
  if (misaligned(X, type_x) || misaligned(Y, type_y) || off4(rows) || off4(weights)) return THL_ERR_MISALIGNED;
  const Range ry = matrix_range(Y, type_y, m, n, ldy);
  if (overlaps(ry, matrix_range(X, type_x, m, rows_x, ldx)) || overlaps(ry, vector_range(rows, n * topk, 4)) ||
      overlaps(ry, vector_range(weights, n * topk, 4)))
    return THL_ERR_INVALID;

  CombineArgs a{};
  a.x = X, a.y = Y, a.rows = rows, a.weights = weights, a.ldx = ldx, a.ldy = ldy, a.n = n, a.rows_x = rows_x;
  a.m = static_cast<int32_t>(m), a.topk = static_cast<int32_t>(topk), a.x_type = type_x, a.y_type = type_y;
  const int64_t units = (m + 7) / 8;
  a.lanes = lanes_for(units);
  const dim3 grid = token_grid(n, units, a.lanes);
  if (rows_x == 0) a.topk = 0;  // no row to add
  const hipError_t e = type_x == THL_F32 ? launch_combine<4>(a, grid, stream) : launch_combine<2>(a, grid, stream);
  return e == hipSuccess ? THL_OK : THL_ERR_HIP;
}

thl_status thl_moe_combine_backward(int64_t m, int64_t n, int64_t topk, const void* DY, int64_t lddy, const void* X,
                                    int64_t ldx, int64_t rows_x, const int32_t* rows, const float* weights, void* DX,
                                    int64_t lddx, float* dweights, thl_dtype type_dy, thl_dtype type_x,
                                    struct ihipStream_t* stream) {
  const thl_status st = check_sizes(n, topk, rows_x);
  if (st != THL_OK) return st;
  if (m < 0) return THL_ERR_INVALID;
  if (m > kMaxFeatures || big(lddy) || big(ldx) || big(lddx)) return THL_ERR_UNSUPPORTED;
  if (!is_float_io(type_dy) || !is_float_io(type_x)) return THL_ERR_UNSUPPORTED;
  if (bad_ld(lddy, m) || (dweights && bad_ld(ldx, m)) || (DX && bad_ld(lddx, m))) return THL_ERR_INVALID;
  if (n == 0 || topk == 0 || (!DX && !dweights)) return THL_OK;
  if (m > 0 && (!DY || (dweights && rows_x > 0 && !X))) return THL_ERR_INVALID;
  if (!rows || (DX && !weights)) return THL_ERR_INVALID;
  if (misaligned(DY, type_dy) || (dweights && misaligned(X, type_x)) || misaligned(DX, type_x) || off4(rows) ||
      off4(weights) || off4(dweights))
    return THL_ERR_MISALIGNED;
  const Range rg = matrix_range(DY, type_dy, m, n, lddy), rr = vector_range(rows, n * topk, 4);
  const Range rx = dweights ? matrix_range(X, type_x, m, rows_x, ldx) : Range{};
  const Range rw = DX ? vector_range(weights, n * topk, 4) : Range{};
  const Range rd = matrix_range(DX, type_x, m, rows_x, lddx), rv = vector_range(dweights, n * topk, 4);
  if (overlaps(rd, rx)) return THL_ERR_INVALID;
  for (const Range& o : {rg, rr, rw})
    if (overlaps(rd, o) || overlaps(rv, o)) return THL_ERR_INVALID;
  if (overlaps(rv, rx) || overlaps(rv, rd)) return THL_ERR_INVALID;

  if (rows_x == 0) {  // no row has a place
    if (!dweights) return THL_OK;
    const hipError_t e = launch_zeros(dweights, n * topk, stream);
    return e == hipSuccess ? THL_OK : THL_ERR_HIP;
  }
  CombineGradArgs a{};
  a.dy = DY, a.x = X, a.dx = DX, a.dweights = dweights, a.rows = rows, a.weights = weights;
  a.lddy = lddy, a.ldx = ldx, a.lddx = lddx, a.n = n, a.rows_x = rows_x;
  a.m = static_cast<int32_t>(m), a.topk = static_cast<int32_t>(topk), a.dy_type = type_dy, a.x_type = type_x;
  hipError_t e;
  if (type_x == THL_F32)
    e = type_dy == THL_F32 ? launch_combine_grad<4, 4>(a, stream) : launch_combine_grad<4, 2>(a, stream);
  else
    e = type_dy == THL_F32 ? launch_combine_grad<2, 4>(a, stream) : launch_combine_grad<2, 2>(a, stream);
  return e == hipSuccess ? THL_OK : THL_ERR_HIP;
}

}  // extern "C"
