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
// One cluster of thread blocks takes one (request, kv head): each block scores
// a stretch of pages and keeps the scores in its shared memory; the threshold
// is found by four passes of an 8-bit radix search whose histograms the blocks
// read from one another.
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
constexpr int kHeads = 8;       // query heads scored at a time
constexpr int kPerCta = 32768;  // scores a block can hold
constexpr int kMaxCluster = 8;

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

// E elements of a row of bounds, as 64-bit numbers
template <typename CT, int E>
__device__ __forceinline__ void load_wide(const CT* p, double (&f)[E]) {
  constexpr int W = E * (int)sizeof(CT) / 4, P = Unpack<CT>::kPerWord;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    float x[P];
    Unpack<CT>::word(__ldg(reinterpret_cast<const uint32_t*>(p) + i), x);
#pragma unroll
    for (int e = 0; e < P; ++e) f[i * P + e] = (double)x[e];
  }
}

template <typename CT, int D>
__global__ void __launch_bounds__(kThreads) select_kernel(const SelectArgs a) {
  constexpr int E = D / 8;  // columns of one lane; eight lanes share a page
  extern __shared__ uint32_t s_key[];
  __shared__ double2 s_q[kHeads][E][8];  // (min(q, 0), max(q, 0)) of column 8 lanes apart
  __shared__ uint32_t s_hist[4][256];
  __shared__ uint32_t s_count[2], s_pick[2], s_warp[2][kWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int pair = blockIdx.x / ranks, r = pair / a.Hkv, h = pair % a.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* out = a.sel + (size_t)pair * a.budget;

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

  const int per = (held + ranks - 1) / ranks;
  const int first = min(rank * per, held), n = min(per, held - first);
  for (int i = tid; i < 4 * 256; i += kThreads) (&s_hist[0][0])[i] = 0;
  const int sub = lane & 7;
  for (int h0 = 0; h0 < a.group; h0 += kHeads) {
    __syncthreads();
    for (int i = tid; i < kHeads * D; i += kThreads) {
      const int head = i / D, d = i % D;
      float x = 0.f;
      if (h0 + head < a.group) {
        const size_t at = ((size_t)r * a.Hq + (size_t)h * a.group + h0 + head) * D + d;
        x = a.q_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at])
                     : static_cast<const float*>(a.q)[at];
      }
      s_q[head][d % E][d / E] = make_double2(fminf(x, 0.f), fmaxf(x, 0.f));
    }
    __syncthreads();
    for (int i0 = warp * 4; i0 < n; i0 += kWarps * 4) {
      const int i = i0 + (lane >> 3);
      const int j = min(first + i, held - 1);
      const int page = a.table[(size_t)r * a.max_pages + j];
      const bool there = page >= 0 && page < a.num_pages;
      double acc[kHeads] = {};
      if (there) {
        const CT* b = static_cast<const CT*>(a.bounds) + ((size_t)page * a.Hkv + h) * 2 * D + sub * E;
        double lo[E], hi[E];
        load_wide<CT, E>(b, lo);
        load_wide<CT, E>(b + D, hi);
#pragma unroll
        for (int m = 0; m < kHeads; ++m)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const double2 q = s_q[m][e][sub];
            acc[m] = fma(q.x, lo[e], acc[m]);
            acc[m] = fma(q.y, hi[e], acc[m]);
          }
      } else if (sub == 0) {
        atomicOr(a.err, kErrPage);
      }
      // eight lanes, eight heads: lane `sub` is left with head sub
      double b4[4], b2[2];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const double keep = (sub & 4) ? acc[4 + m] : acc[m], give = (sub & 4) ? acc[m] : acc[4 + m];
        b4[m] = keep + __shfl_xor_sync(0xffffffffu, give, 4);
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const double keep = (sub & 2) ? b4[2 + m] : b4[m], give = (sub & 2) ? b4[m] : b4[2 + m];
        b2[m] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
      }
      const double keep = (sub & 1) ? b2[1] : b2[0], give = (sub & 1) ? b2[0] : b2[1];
      const float x = (float)(keep + __shfl_xor_sync(0xffffffffu, give, 1));
      uint32_t key = h0 + sub < a.group && there ? order_key(x) : 0u;
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
      if (sub == 0 && i < n) {
        if (j < a.keep_first || j == held - 1) key = 0xffffffffu;
        s_key[i] = h0 == 0 ? key : max(key, s_key[i]);
      }
    }
  }
  __syncthreads();

  // the budget-th largest key, eight bits at a time
  uint32_t prefix = 0;
  int need = a.budget;  // keys wanted among those that share the prefix
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int low = 24 - 8 * pass;
    for (int i = tid; i < n; i += kThreads) {
      const uint32_t key = s_key[i];
      if (pass == 0 || (key >> (low + 8)) == prefix) atomicAdd(&s_hist[pass][(key >> low) & 255u], 1u);
    }
    cluster.sync();
    // thread b: keys in bin 255 - b over the cluster; inclusive sums from the top
    uint32_t c = 0;
    for (int k = 0; k < ranks; ++k) c += *cluster.map_shared_rank(&s_hist[pass][255 - tid], k);
    uint32_t up = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += x;
    }
    if (lane == 31) s_warp[0][warp] = up;
    __syncthreads();
    for (int w = 0; w < warp; ++w) up += s_warp[0][w];
    if (up >= (uint32_t)need && up - c < (uint32_t)need) s_pick[0] = 255 - tid, s_pick[1] = need - (up - c);
    __syncthreads();
    prefix = (prefix << 8) | s_pick[0];
    need = (int)s_pick[1];
    __syncthreads();
  }

  // every key above the threshold, and the first `need` equal to it
  if (tid < 2) s_count[tid] = 0;
  __syncthreads();
  uint32_t above = 0, equal = 0;
  for (int i = tid; i < n; i += kThreads) above += s_key[i] > prefix, equal += s_key[i] == prefix;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    above += __shfl_xor_sync(0xffffffffu, above, o);
    equal += __shfl_xor_sync(0xffffffffu, equal, o);
  }
  if (lane == 0) {
    atomicAdd(&s_count[0], above);
    atomicAdd(&s_count[1], equal);
  }
  cluster.sync();
  uint32_t above_before = 0, equal_before = 0;
  for (int k = 0; k < rank; ++k) {
    above_before += *cluster.map_shared_rank(&s_count[0], k);
    equal_before += *cluster.map_shared_rank(&s_count[1], k);
  }
  uint32_t at = above_before + min(equal_before, (uint32_t)need);
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + tid;
    const uint32_t key = i < n ? s_key[i] : 0u;
    const bool eq = i < n && key == prefix, gt = i < n && key > prefix;
    const uint32_t eq_mask = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) s_warp[0][warp] = __popc(eq_mask);
    __syncthreads();
    uint32_t eq_at = equal_before + __popc(eq_mask & ((1u << lane) - 1u));
    uint32_t eq_all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) eq_at += s_warp[0][w];
      eq_all += s_warp[0][w];
    }
    const bool take = gt || (eq && eq_at < (uint32_t)need);
    const uint32_t mask = __ballot_sync(0xffffffffu, take);
    if (lane == 0) s_warp[1][warp] = __popc(mask);
    __syncthreads();
    uint32_t to = at + __popc(mask & ((1u << lane) - 1u));
    uint32_t all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) to += s_warp[1][w];
      all += s_warp[1][w];
    }
    if (take) out[to] = first + i;
    at += all;
    equal_before += eq_all;
    __syncthreads();
  }
  cluster.sync();  // no block leaves while another still reads its counts
}

template <typename CT>
int launch_select(const SelectArgs& a, int D, int cluster, cudaStream_t s) {
  static std::atomic<unsigned long long> done64{0}, done128{0};
  const int bytes = (int)(((a.max_pages + cluster - 1) / cluster) * sizeof(uint32_t));
  if (D == 64 ? !smem_attr_once(select_kernel<CT, 64>, kPerCta * 4, done64)
              : !smem_attr_once(select_kernel<CT, 128>, kPerCta * 4, done128))
    return -1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)a.R * a.Hkv * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  prof_begin(kKSelect, s);
  const cudaError_t e = D == 64 ? cudaLaunchKernelEx(&cfg, select_kernel<CT, 64>, a)
                                : cudaLaunchKernelEx(&cfg, select_kernel<CT, 128>, a);
  prof_end(kKSelect, s);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? 1 : -1;
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
  if (shift < 0 || max_pages < 1 || max_pages > kPerCta * kMaxCluster || num_pages < 1) return CPATTN_ERR_SHAPE;
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
  // blocks per pair: until the device is full twice over, and while a block
  // still has at least 64 pages; more where the scores would not fit
  int cluster = 1;
  while (cluster < kMaxCluster && (((long long)a.R * a.Hkv * cluster < 2LL * num_sms(dev) && max_pages > 64 * cluster) ||
                                   max_pages > kPerCta * cluster))
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
