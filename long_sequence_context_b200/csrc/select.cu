// select.cu -- which pages of a long cache one new token attends to.
//
// A page's score for kv head h is the largest q.k that any key inside the
// page's bounds could have, over the query heads of the group:
//     score = max_i sum_d max(q_id lo_d, q_id hi_d)
//           = max_i sum_d (min(q_id, 0) lo_d + max(q_id, 0) hi_d)
// summed in 64 bits and rounded once to fp32: products of 16-bit values are
// exact there and their sums almost always, so that the order of summation
// does not decide between near pages.  The `budget` pages with the largest
// scores are listed in ascending order, ties to the lower page; the newest
// page and the first keep_first pages are always among them.
//
// One cluster of thread blocks takes one (request, kv head): every block scores
// a stretch of pages and sends the scores to the first block's shared memory,
// which finds the threshold by a radix search of eight bits at a time and lists
// the pages.  A page's bounds are read once; what bounds the kernel is the
// chain of latencies from the lengths over the page table and the bounds to the
// search, so the loads of a warp's next pages are under way while it sums, and
// the pages are spread over as many blocks as the device holds at once.
#include <cooperative_groups.h>

#include <algorithm>

#include "cpattn.h"
#include "kernels.h"
#include "paged.cuh"

namespace cg = cooperative_groups;

namespace cpattn {
namespace {

using namespace paged;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPages = 49152;  // scores that a block's shared memory holds
constexpr int kMaxCluster = 16;

struct SelectArgs {
  const void *q, *bounds;
  const int32_t *table, *lens;
  int32_t* sel;
  unsigned* err;
  int R, Hq, Hkv, group, shift, max_pages, num_pages, budget, keep_first, q_bf16;
};

// unsigned order of the keys = order of the scores; NaN is below every number
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 counts as 0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// W consecutive words, in place.
template <int W>
__device__ __forceinline__ void load_packed(const void* p, uint32_t (&w)[W]) {
#pragma unroll
  for (int i = 0; i < W; i += 4)
    asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                 : "l"(static_cast<const char*>(p) + 4 * i));
}

// c (8 pages x 8 heads, 64 bits) += a (8 pages x 4 columns) b (4 columns x 8 heads)
__device__ __forceinline__ void mma_f64(double (&c)[2], double a, double b) {
  asm volatile("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0,%1}, {%2}, {%3}, {%0,%1};"
               : "+d"(c[0]), "+d"(c[1])
               : "d"(a), "d"(b));
}

template <typename CT, int D>
__global__ void __launch_bounds__(kThreads) select_kernel(const SelectArgs a) {
  // A warp takes 8 pages at a time, 4 lanes each, in steps of W words (E columns) of
  // a lane's low and high bounds.
  constexpr int P = Unpack<CT>::kPerWord;
  constexpr int W = D / (4 * P) < 8 ? D / (4 * P) : 8, E = W * P, STEPS = D / (4 * E);
  extern __shared__ uint32_t s_key[];      // the first block's: the keys of all pages
  __shared__ double2 s_q[STEPS * E][32];   // (min(q, 0), max(q, 0)) of 4 columns x 8 heads
  __shared__ uint32_t s_hist[256], s_bin[kThreads];
  __shared__ uint32_t s_pick[3], s_found, s_warp[kWarps], s_warp2[kWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int pair = blockIdx.x / ranks, r = pair / a.Hkv, h = pair % a.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* out = a.sel + (size_t)pair * a.budget;

  after_previous();
  const long long cap = (long long)a.max_pages << a.shift;
  long long len = a.lens[r];
  if (len < 0 || len > cap) {
    if (tid == 0) atomicOr(a.err, kErrPage);
    len = len < 0 ? 0 : cap;
  }
  const int held = (int)((len + (1 << a.shift) - 1) >> a.shift);
  if (held <= a.budget) {  // everything is selected (the whole cluster leaves here)
    for (int j = rank * kThreads + tid; j < a.budget; j += ranks * kThreads) out[j] = j < held ? j : -1;
    return;
  }

  cluster.barrier_arrive();  // no block writes to the first one before that has started

  const int per = (held + ranks - 1) / ranks;
  const int first = min(rank * per, held), n = min(per, held - first);
  const int g = lane >> 2, t = lane & 3;
  uint32_t* keys = cluster.map_shared_rank(s_key, 0);
  const int32_t* table = a.table + (size_t)r * a.max_pages + first;
  auto page_of = [&](int i) { return table[min(i, n - 1)]; };  // only for n > 0
  auto load = [&](int page, int step, uint32_t (&lo)[W], uint32_t (&hi)[W]) {
    const int p = page >= 0 && page < a.num_pages ? page : 0;
    const CT* b = static_cast<const CT*>(a.bounds) + ((size_t)p * a.Hkv + h) * 2 * D + step * 4 * E + t * E;
    load_packed(b, lo);
    load_packed(b + D, hi);
  };
  for (int h0 = 0; h0 < a.group; h0 += 8) {
    uint32_t lo[W], hi[W];
    int i0 = warp * 8, page = 0, page_next = 0;
    if (i0 < n) {
      page = page_of(i0 + g);
      page_next = page_of(i0 + kWarps * 8 + g);
      load(page, 0, lo, hi);
    }
    __syncthreads();
    for (int i = tid; i < 8 * D; i += kThreads) {
      const int head = i / D, d = i % D;
      float x = 0.f;
      if (h0 + head < a.group) {
        const size_t at = ((size_t)r * a.Hq + (size_t)h * a.group + h0 + head) * D + d;
        x = a.q_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at])
                     : static_cast<const float*>(a.q)[at];
      }
      s_q[d / (4 * E) * E + d % E][head * 4 + d / E % 4] = make_double2(fminf(x, 0.f), fmaxf(x, 0.f));
    }
    if (h0 == 0) cluster.barrier_wait();
    __syncthreads();
    for (; i0 < n; i0 += kWarps * 8) {
      const int i = i0 + g, j = first + i;
      const bool there = page >= 0 && page < a.num_pages;
      if (!there && t == 0) atomicOr(a.err, kErrPage);
      double acc[4][2] = {};
#pragma unroll
      for (int step = 0; step < STEPS; ++step) {
        float flo[E], fhi[E];
#pragma unroll
        for (int w = 0; w < W; ++w) {
          Unpack<CT>::word(lo[w], flo + w * P);
          Unpack<CT>::word(hi[w], fhi + w * P);
        }
        if (step + 1 < STEPS) {
          load(page, step + 1, lo, hi);
        } else {
          page = page_next;
          if (i0 + kWarps * 8 < n) {
            load(page, 0, lo, hi);
            page_next = page_of(i0 + 2 * kWarps * 8 + g);
          }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const double2 q = s_q[step * E + e][lane];
          mma_f64(acc[2 * (e & 1)], (double)flo[e], q.x);
          mma_f64(acc[2 * (e & 1) + 1], (double)fhi[e], q.y);
        }
      }
      // lane 4g + t has page g with heads 2t and 2t + 1
      uint32_t key = 0u;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const float x = (float)((acc[0][m] + acc[1][m]) + (acc[2][m] + acc[3][m]));
        if (there && h0 + 2 * t + m < a.group) key = max(key, order_key(x));
      }
      key = max(key, __shfl_xor_sync(0xffffffffu, key, 1));
      key = max(key, __shfl_xor_sync(0xffffffffu, key, 2));
      if (t == 0 && i < n) {
        if (j < a.keep_first || j == held - 1) key = 0xffffffffu;
        keys[j] = h0 == 0 ? key : max(key, keys[j]);
      }
    }
  }
  cluster.sync();
  if (rank != 0) return;

  // The pages that are always listed need no search: their key is the largest.
  // The others: first the leading bits that all keys share, then eight bits at a
  // time until the bin of the threshold is small enough to rank its keys directly.
  const int always = min(a.keep_first, held - 1) + 1;
  const uint32_t kAlways = 0xffffffffu;
  uint32_t any = 0u, all = 0xffffffffu;
  for (int i = tid; i < held; i += kThreads) {
    const uint32_t key = s_key[i];
    if (key != kAlways) any |= key, all &= key;
  }
  s_hist[tid] = 0;
  any = __reduce_or_sync(0xffffffffu, any);
  all = __reduce_and_sync(0xffffffffu, all);
  if (lane == 0) s_warp[warp] = any, s_warp2[warp] = all;
  if (tid == 0) s_found = 0;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) any |= s_warp[w], all &= s_warp2[w];
  int low = 32 - __clz(any ^ all);               // bits below `low` differ
  uint32_t prefix = low < 32 ? any >> low : 0u;  // of the threshold
  int need = a.budget - always;                  // keys wanted among those that share the prefix
  uint32_t threshold = any;                      // every key above it, and `need` equal to it
  if (need == 0) low = 0, threshold = kAlways - 1u;
  while (low > 0) {
    const int above = low;
    low = max(0, low - 8);
    const uint32_t digits = (1u << (above - low)) - 1u;
    for (int i = tid; i < held; i += kThreads) {
      const uint32_t key = s_key[i];
      if (key != kAlways && (above == 32 || (key >> above) == prefix)) atomicAdd(&s_hist[(key >> low) & digits], 1u);
    }
    __syncthreads();
    // thread b: keys in bin 255 - b; inclusive sums from the top
    const uint32_t c = s_hist[255 - tid];
    uint32_t up = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += x;
    }
    if (lane == 31) s_warp[warp] = up;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (w < warp) up += s_warp[w];
    if (up >= (uint32_t)need && up - c < (uint32_t)need) s_pick[0] = 255 - tid, s_pick[1] = need - (up - c), s_pick[2] = c;
    s_hist[255 - tid] = 0;
    __syncthreads();
    prefix = (above == 32 ? 0u : prefix << (above - low)) | s_pick[0];
    need = (int)s_pick[1];
    threshold = prefix << low;
    const uint32_t in_bin = s_pick[2];
    if (low == 0) break;
    if (in_bin == (uint32_t)need) {  // the whole bin is taken; a key below it exists, so threshold > 0
      threshold -= 1u;
      need = 0;
      break;
    }
    if (in_bin <= (uint32_t)kThreads) {  // rank the bin's keys: one for each thread
      for (int i = tid; i < held; i += kThreads) {
        const uint32_t key = s_key[i];
        if (key != kAlways && (key >> low) == prefix) s_bin[atomicAdd(&s_found, 1u)] = key;
      }
      __syncthreads();
      if (tid < (int)in_bin) {
        const uint32_t key = s_bin[tid];
        uint32_t more = 0, same = 0;
        for (uint32_t i = 0; i < in_bin; ++i) more += s_bin[i] > key, same += s_bin[i] == key;
        // equal keys write the same two numbers
        if (more < (uint32_t)need && more + same >= (uint32_t)need) s_pick[0] = key, s_pick[1] = need - more;
      }
      __syncthreads();
      threshold = s_pick[0];
      need = (int)s_pick[1];
      break;
    }
  }

  // every key above the threshold and the first `need` equal to it, in order: a
  // stretch of pages for each warp
  const int stretch = ((held + kWarps - 1) / kWarps + 31) & ~31;
  const int w0 = min(warp * stretch, held), w1 = min(w0 + stretch, held);
  uint32_t above = 0, equal = 0;
  for (int i = w0; i < w1; i += 32) {
    const uint32_t key = i + lane < w1 ? s_key[i + lane] : 0u;
    above += __popc(__ballot_sync(0xffffffffu, i + lane < w1 && key > threshold));
    equal += __popc(__ballot_sync(0xffffffffu, i + lane < w1 && key == threshold));
  }
  __syncthreads();  // s_warp of the last pass is read
  if (lane == 0) s_warp[warp] = above, s_warp2[warp] = equal;
  __syncthreads();
  above = equal = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < warp) above += s_warp[w], equal += s_warp2[w];
  const uint32_t below = (1u << lane) - 1u;
  for (int i = w0; i < w1; i += 32) {
    const uint32_t key = i + lane < w1 ? s_key[i + lane] : 0u;
    const bool gt = i + lane < w1 && key > threshold, eq = i + lane < w1 && key == threshold;
    const uint32_t gts = __ballot_sync(0xffffffffu, gt), eqs = __ballot_sync(0xffffffffu, eq);
    const uint32_t eq_at = equal + __popc(eqs & below);
    if (gt || (eq && eq_at < (uint32_t)need)) out[above + __popc(gts & below) + min(eq_at, (uint32_t)need)] = i + lane;
    above += __popc(gts);
    equal += __popc(eqs);
  }
}

template <typename CT, int D>
int launch_dim(const SelectArgs& a, int cluster, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  auto* kernel = select_kernel<CT, D>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
  if (!(done.load() & (1ull << dev)) &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return -1;
  if (!smem_attr_once(kernel, kMaxPages * (int)sizeof(uint32_t), done)) return -1;
  prof_begin(kKSelect, s);
  const cudaError_t e = launch_chained(kernel, dim3((unsigned)((long long)a.R * a.Hkv * cluster)), kThreads,
                                       a.max_pages * sizeof(uint32_t), cluster, s, a);
  prof_end(kKSelect, s);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? 1 : -1;
}

template <typename CT>
int launch_select(const SelectArgs& a, int D, int cluster, cudaStream_t s) {
  return D == 64 ? launch_dim<CT, 64>(a, cluster, s) : launch_dim<CT, 128>(a, cluster, s);
}

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" int cpattn_select_pages(const void* q, const void* k_bounds, const int32_t* block_table,
                                   const int32_t* lens, int32_t* pages, int R, int Hq, int Hkv, int D,
                                   int page_size, int max_pages, int num_pages, int budget, int keep_first,
                                   int dtype, int cache_dtype, void* stream) {
  NvtxRange nv("cpattn_select_pages");
  if (dtype != CPATTN_BF16 && dtype != CPATTN_FP32) return CPATTN_ERR_DTYPE;
  if (cache_dtype != dtype && !(cache_dtype == CPATTN_E4M3 && dtype == CPATTN_BF16)) return CPATTN_ERR_DTYPE;
  const int shift = paged::page_shift(page_size);
  if (R < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > 64 || (D != 64 && D != 128)) return CPATTN_ERR_SHAPE;
  if (shift < 0 || max_pages < 1 || max_pages > kMaxPages || num_pages < 1) return CPATTN_ERR_SHAPE;
  if (((long long)max_pages << shift) > 0x7fffffffLL || (long long)R * Hkv > (1LL << 27)) return CPATTN_ERR_SHAPE;
  if (keep_first < 0 || budget < 1 || budget - 1 < keep_first) return CPATTN_ERR_SHAPE;
  if (!q || !k_bounds || !block_table || !lens || !pages) return CPATTN_ERR_ARG;
  if (!paged::aligned_to(q, 16) || !paged::aligned_to(k_bounds, 16) || !paged::aligned_to(block_table, 4) ||
      !paged::aligned_to(lens, 4) || !paged::aligned_to(pages, 4))
    return CPATTN_ERR_ALIGN;
  unsigned* err = device_error_word();
  if (!err) return CPATTN_ERR_CUDA;
  SelectArgs a = {};
  a.q = q;
  a.bounds = k_bounds;
  a.table = block_table;
  a.lens = lens;
  a.sel = pages;
  a.err = err;
  a.R = R;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.group = Hq / Hkv;
  a.shift = shift;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.budget = budget;
  a.keep_first = keep_first;
  a.q_bf16 = dtype == CPATTN_BF16;
  int dev = 0;
  cudaGetDevice(&dev);
  // blocks per pair: while all blocks fit the device at once (four to an SM), and
  // a block still has two steps of its warps (64 pages); at most 8 where the
  // scores leave room for one block to an SM
  const int most = max_pages > kMaxPages / 2 ? 8 : kMaxCluster;
  int cluster = 1;
  while (cluster < most && (long long)a.R * a.Hkv * cluster * 2 <= 4LL * num_sms(dev) && max_pages > 64 * cluster)
    cluster *= 2;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int n = -1;
  if (cache_dtype == CPATTN_BF16) n = launch_select<__nv_bfloat16>(a, D, cluster, s);
  else if (cache_dtype == CPATTN_FP32) n = launch_select<float>(a, D, cluster, s);
  else n = launch_select<paged::E4m3>(a, D, cluster, s);
  if (n < 0) return CPATTN_ERR_CUDA;
  add_launches(n);
  return CPATTN_OK;
}
