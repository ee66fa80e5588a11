// cache.cu -- the paged key-value cache's books and its rows.
//
// cache_plan: from the requests' lengths and what each asks for (new tokens,
// or tokens taken back) the pages they take from and return to the pool, the
// new tokens' slots and the lengths afterwards.  Integer work of a few bytes
// per request and token: the launch and the prefix sums' latency bound it.
//
// cache_append: new K and V rows into their slots, quantised for an 8-bit
// cache, with the elementwise smallest and largest key of every page kept up
// to date.  Every row is read and written once: the memory bandwidth bounds it.
#include <algorithm>

#include "cpattn.h"
#include "kernels.h"
#include "paged.cuh"

namespace cpattn {
namespace {

using namespace paged;

constexpr int kPlanThreads = 1024;

// verdict bits of a plan
constexpr int kShort = 1, kBadLength = 2, kCapacity = 4, kBadState = 8;

struct PlanArgs {
  const int32_t *lens, *delta, *free_state;
  int32_t *table, *ring;
  int32_t *lens_out, *state_out, *cu, *verdict;
  int64_t* slots;
  // workspace: what the planning block leaves for the writing ones
  int32_t *head, *pop_at, *push_at;  // {ok, ring head, count}, [R + 1], [R + 1]
  unsigned* err;
  long long capacity;
  int R, max_pages, shift, num_pages;
};

struct Three {
  long long a, b, c;
};

__device__ __forceinline__ long long pages_of(long long n, int shift) { return (n + (1 << shift) - 1) >> shift; }

// What request r asks for: new tokens, pages taken, pages returned.
__device__ __forceinline__ Three request_of(const PlanArgs& a, int r, int* bad) {
  const long long n = a.lens[r], after = n + a.delta[r];
  if (n < 0 || after < 0 || after > ((long long)a.max_pages << a.shift)) {
    *bad |= kBadLength;
    return {0, 0, 0};
  }
  const long long p0 = pages_of(n, a.shift), p1 = pages_of(after, a.shift);
  return {max(0LL, after - n), max(0LL, p1 - p0), max(0LL, p0 - p1)};
}

// One block: prefix sums over the requests, the verdict, and everything that
// has one value per request.  Reads all lengths before it writes any, so that
// lens_out may be lens and state_out free_state.
__device__ __forceinline__ void plan_requests(const PlanArgs& a) {
  __shared__ Three s_sum[32];
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.R + blockDim.x - 1) / blockDim.x;
  const int lo = min(tid * per, a.R), hi = min(lo + per, a.R);
  if (tid == 0) s_bad = 0;
  int bad = 0;
  Three mine = {0, 0, 0};
  for (int r = lo; r < hi; ++r) {
    const Three x = request_of(a, r, &bad);
    mine.a += x.a, mine.b += x.b, mine.c += x.c;
  }
  Three up = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, up.a, o), y = __shfl_up_sync(0xffffffffu, up.b, o),
                    z = __shfl_up_sync(0xffffffffu, up.c, o);
    if (lane >= o) up.a += x, up.b += y, up.c += z;
  }
  if (lane == 31) s_sum[warp] = up;
  const int head = a.free_state[0], count = a.free_state[1];
  __syncthreads();
  if (bad) atomicOr(&s_bad, bad);
  Three all = {0, 0, 0};
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
    if (w < warp) up.a += s_sum[w].a, up.b += s_sum[w].b, up.c += s_sum[w].c;
    all.a += s_sum[w].a, all.b += s_sum[w].b, all.c += s_sum[w].c;
  }
  __syncthreads();
  int verdict = s_bad;
  if (all.b > count) verdict |= kShort;
  if (all.a > a.capacity) verdict |= kCapacity;
  if (head < 0 || head >= a.num_pages || count < 0 || count > a.num_pages || count + all.c > a.num_pages)
    verdict |= kBadState;
  const bool ok = verdict == 0;
  Three at = {up.a - mine.a, up.b - mine.b, up.c - mine.c};
  for (int r = lo; r < hi; ++r) {
    const int n = a.lens[r];
    int ignore = 0;
    const Three x = request_of(a, r, &ignore);
    a.cu[r] = ok ? (int)at.a : 0;
    a.pop_at[r] = ok ? (int)at.b : 0;
    a.push_at[r] = ok ? (int)at.c : 0;
    a.lens_out[r] = ok ? n + a.delta[r] : n;
    at.a += x.a, at.b += x.b, at.c += x.c;
  }
  if (tid == 0) {
    a.cu[a.R] = ok ? (int)all.a : 0;
    a.pop_at[a.R] = ok ? (int)all.b : 0;
    a.push_at[a.R] = ok ? (int)all.c : 0;
    a.head[0] = ok;
    a.head[1] = head;
    a.head[2] = count;
    a.state_out[0] = ok ? (int)(((long long)head + all.b) % a.num_pages) : head;
    a.state_out[1] = ok ? (int)(count - all.b + all.c) : count;
    *a.verdict = verdict;
  }
}

// The last r with at[r] <= i (at[0] = 0, not descending, i < at[R]).
__device__ __forceinline__ int find(const int32_t* at, int R, int i) {
  int lo = 0, hi = R;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Everything that has one value per token or page, dealt to `n` threads.
__device__ __forceinline__ void plan_items(const PlanArgs& a, long long i0, long long n) {
  const bool ok = a.head[0] != 0;
  const int head = a.head[1], count = a.head[2];
  const int tokens = a.cu[a.R], pops = a.pop_at[a.R], pushes = a.push_at[a.R];
  for (long long i = i0; i < a.capacity; i += n) {
    long long slot = -1;
    if (i < tokens) {
      const int r = find(a.cu, a.R, (int)i);
      const int before = a.lens_out[r] - a.delta[r];
      const int pos = before + ((int)i - a.cu[r]);
      const int j = pos >> a.shift, held = (int)pages_of(before, a.shift);
      const int page = j < held ? a.table[(size_t)r * a.max_pages + j]
                                : a.ring[((long long)head + a.pop_at[r] + (j - held)) % a.num_pages];
      if (page >= 0 && page < a.num_pages)
        slot = ((long long)page << a.shift) + (pos & ((1 << a.shift) - 1));
      else
        atomicOr(a.err, kErrPage);
    }
    a.slots[i] = slot;
  }
  if (!ok) return;
  for (long long i = i0; i < pops; i += n) {
    const int r = find(a.pop_at, a.R, (int)i);
    const int held = (int)pages_of(a.lens_out[r] - a.delta[r], a.shift);
    a.table[(size_t)r * a.max_pages + held + ((int)i - a.pop_at[r])] = a.ring[((long long)head + i) % a.num_pages];
  }
  // returned pages go behind the last free one: count + pushes <= num_pages, so
  // none of these places is read above
  for (long long i = i0; i < pushes; i += n) {
    const int r = find(a.push_at, a.R, (int)i);
    const int left = (int)pages_of(a.lens_out[r], a.shift);
    a.ring[((long long)head + count + i) % a.num_pages] =
        a.table[(size_t)r * a.max_pages + left + ((int)i - a.push_at[r])];
  }
}

__global__ void __launch_bounds__(kPlanThreads) plan_requests_kernel(const PlanArgs a) { plan_requests(a); }
__global__ void __launch_bounds__(256) plan_items_kernel(const PlanArgs a) {
  plan_items(a, (long long)blockIdx.x * blockDim.x + threadIdx.x, (long long)gridDim.x * blockDim.x);
}

struct AppendArgs {
  const void *k, *v;
  long long k_tok, k_head, v_tok, v_head;  // strides in elements
  const int64_t* slots;
  void *k_cache, *v_cache, *bounds;
  const float* kv_amax;
  unsigned* err;
  long long N, n_slots;
  int Hkv, shift;
};

template <typename T>
__device__ __forceinline__ void load_row(const T* p, float (&f)[4]);
template <>
__device__ __forceinline__ void load_row<float>(const float* p, float (&f)[4]) {
  const float4 x = __ldg(reinterpret_cast<const float4*>(p));
  f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w;
}
template <>
__device__ __forceinline__ void load_row<__nv_bfloat16>(const __nv_bfloat16* p, float (&f)[4]) {
  const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
  Unpack<__nv_bfloat16>::word(x.x, f);
  Unpack<__nv_bfloat16>::word(x.y, f + 2);
}

// four values as stored, and f as the numbers that are then stored (unscaled)
template <typename CT>
struct Store4;
template <>
struct Store4<float> {
  __device__ static __forceinline__ void put(float* p, float (&f)[4], float) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct Store4<__nv_bfloat16> {
  __device__ static __forceinline__ void put(__nv_bfloat16* p, float (&f)[4], float) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t*>(&a);
    w.y = *reinterpret_cast<const uint32_t*>(&b);
    *reinterpret_cast<uint2*>(p) = w;
  }
};
template <>
struct Store4<E4m3> {
  __device__ static __forceinline__ void put(E4m3* p, float (&f)[4], float s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __fmul_rn(f[i], s);
    const uint32_t w = (uint32_t)float2_to_e4m3x2(f[0], f[1]) | ((uint32_t)float2_to_e4m3x2(f[2], f[3]) << 16);
    *reinterpret_cast<uint32_t*>(p) = w;
    Unpack<E4m3>::word(w, f);
  }
};
template <typename CT>
__device__ __forceinline__ void load4(const CT* p, float (&f)[4]) {
  constexpr int W = (int)sizeof(CT);  // words of four elements
  const uint32_t* w = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
  for (int i = 0; i < W; ++i) Unpack<CT>::word(w[i], f + i * (4 / W));
}

// A group of D / 4 lanes takes the rows of one kv head that lie next to one
// another in one page, copies them and reduces their keys.
template <typename IT, typename CT, int D>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs a) {
  constexpr int kLanes = D / 4;
  const long long unit = ((long long)blockIdx.x * blockDim.x + threadIdx.x) / kLanes;
  const int d = (threadIdx.x % kLanes) * 4;
  const long long t = unit / a.Hkv;
  const int h = (int)(unit % a.Hkv);
  if (t >= a.N) return;
  const long long slot = a.slots[t];
  if (slot < 0) return;
  if (slot >= a.n_slots) {
    if (d == 0 && h == 0) atomicOr(a.err, kErrPage);
    return;
  }
  const int page_mask = (1 << a.shift) - 1;
  const long long page = slot >> a.shift;
  const int off = (int)(slot & page_mask);
  if (t > 0 && off > 0 && a.slots[t - 1] == slot - 1) return;  // the run begins before this row
  const float ks = sizeof(CT) == 1 ? e4m3_scale(a.kv_amax) : 1.f;
  const float vs = sizeof(CT) == 1 ? e4m3_scale(a.kv_amax + 1) : 1.f;
  float lo[4], hi[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) lo[e] = INFINITY, hi[e] = -INFINITY;
  for (int i = 0; off + i <= page_mask && t + i < a.N; ++i) {
    if (i > 0 && a.slots[t + i] != slot + i) break;
    float k[4], v[4];
    load_row(static_cast<const IT*>(a.k) + (t + i) * a.k_tok + h * a.k_head + d, k);
    load_row(static_cast<const IT*>(a.v) + (t + i) * a.v_tok + h * a.v_head + d, v);
    const size_t at = ((((size_t)page * a.Hkv + h) << a.shift) + off + i) * D + d;
    Store4<CT>::put(static_cast<CT*>(a.k_cache) + at, k, ks);
    Store4<CT>::put(static_cast<CT*>(a.v_cache) + at, v, vs);
#pragma unroll
    for (int e = 0; e < 4; ++e) lo[e] = fminf(lo[e], k[e]), hi[e] = fmaxf(hi[e], k[e]);
  }
  if (!a.bounds) return;
  CT* b = static_cast<CT*>(a.bounds) + ((size_t)page * a.Hkv + h) * 2 * D + d;
  if (off > 0) {  // the page held rows before: the first row of a page starts its bounds afresh
    float f[4];
    load4<CT>(b, f);
#pragma unroll
    for (int e = 0; e < 4; ++e) lo[e] = fminf(lo[e], f[e]);
    load4<CT>(b + D, f);
#pragma unroll
    for (int e = 0; e < 4; ++e) hi[e] = fmaxf(hi[e], f[e]);
  }
  // stored values: writing them again rounds nothing
  Store4<CT>::put(b, lo, 1.f);
  Store4<CT>::put(b + D, hi, 1.f);
}

template <typename IT, typename CT>
int launch_append(const AppendArgs& a, int D, cudaStream_t s) {
  const long long threads = a.N * a.Hkv * (D / 4);
  const unsigned blocks = (unsigned)((threads + 255) / 256);
  prof_begin(kKCacheAppend, s);
  if (D == 64)
    append_kernel<IT, CT, 64><<<blocks, 256, 0, s>>>(a);
  else
    append_kernel<IT, CT, 128><<<blocks, 256, 0, s>>>(a);
  prof_end(kKCacheAppend, s);
  return cudaGetLastError() == cudaSuccess ? 1 : -1;
}

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" {

size_t cpattn_cache_plan_workspace_bytes(int R) {
  if (R < 1) return 0;
  return (4 + 2 * ((size_t)R + 1)) * sizeof(int32_t);
}

int cpattn_cache_plan(const int32_t* lens, const int32_t* delta, int32_t* block_table, int R,
                      int max_pages, int page_size, int32_t* free_ring, const int32_t* free_state,
                      int num_pages, int32_t* lens_out, int32_t* free_state_out, int32_t* cu_new,
                      int64_t* slots, long capacity, int32_t* verdict, void* workspace,
                      size_t ws_bytes, void* stream) {
  NvtxRange nv("cpattn_cache_plan");
  const int shift = paged::page_shift(page_size);
  if (R < 1 || max_pages < 1 || num_pages < 1 || shift < 0) return CPATTN_ERR_SHAPE;
  if (capacity < 0 || capacity > 0x7fffffffL) return CPATTN_ERR_SHAPE;
  if (((long long)max_pages << shift) > 0x7fffffffLL) return CPATTN_ERR_SHAPE;
  if (!lens || !delta || !block_table || !free_ring || !free_state || !lens_out || !free_state_out || !cu_new ||
      (capacity > 0 && !slots) || !verdict)
    return CPATTN_ERR_ARG;
  for (const void* p : {(const void*)lens, (const void*)delta, (const void*)block_table, (const void*)free_ring,
                        (const void*)free_state, (const void*)lens_out, (const void*)free_state_out,
                        (const void*)cu_new, (const void*)verdict})
    if (!paged::aligned_to(p, 4)) return CPATTN_ERR_ALIGN;
  if (!paged::aligned_to(slots, 8)) return CPATTN_ERR_ALIGN;
  if (!workspace || ws_bytes < cpattn_cache_plan_workspace_bytes(R)) return CPATTN_ERR_WORKSPACE;
  if (!paged::aligned_to(workspace, 16)) return CPATTN_ERR_ALIGN;
  unsigned* err = device_error_word();
  if (!err) return CPATTN_ERR_CUDA;
  PlanArgs a = {};
  a.lens = lens;
  a.delta = delta;
  a.free_state = free_state;
  a.table = block_table;
  a.ring = free_ring;
  a.lens_out = lens_out;
  a.state_out = free_state_out;
  a.cu = cu_new;
  a.verdict = verdict;
  a.slots = slots;
  a.head = static_cast<int32_t*>(workspace);
  a.pop_at = a.head + 4;
  a.push_at = a.pop_at + R + 1;
  a.err = err;
  a.capacity = capacity;
  a.R = R;
  a.max_pages = max_pages;
  a.shift = shift;
  a.num_pages = num_pages;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int dev = 0;
  cudaGetDevice(&dev);
  prof_begin(kKCachePlan, s);
  plan_requests_kernel<<<1, kPlanThreads, 0, s>>>(a);
  prof_end(kKCachePlan, s);
  if (cudaGetLastError() != cudaSuccess) return CPATTN_ERR_CUDA;
  const long long items = std::max<long long>(capacity, std::min<long long>((long long)R * max_pages, num_pages));
  const int blocks = (int)std::min<long long>((items + 255) / 256, (long long)num_sms(dev) * 8);
  prof_begin(kKCachePlan, s);
  plan_items_kernel<<<std::max(blocks, 1), 256, 0, s>>>(a);
  prof_end(kKCachePlan, s);
  if (cudaGetLastError() != cudaSuccess) return CPATTN_ERR_CUDA;
  add_launches(2);
  return CPATTN_OK;
}

int cpattn_cache_append(const void* k_new, const void* v_new, long k_tok_stride, long k_head_stride,
                        long v_tok_stride, long v_head_stride, const int64_t* slots, long N,
                        void* k_cache, void* v_cache, void* k_bounds, int Hkv, int D, int page_size,
                        int num_pages, const float* kv_amax, int dtype, int cache_dtype, void* stream) {
  NvtxRange nv("cpattn_cache_append");
  if (dtype != CPATTN_BF16 && dtype != CPATTN_FP32) return CPATTN_ERR_DTYPE;
  if (cache_dtype != dtype && !(cache_dtype == CPATTN_E4M3 && dtype == CPATTN_BF16)) return CPATTN_ERR_DTYPE;
  const int shift = paged::page_shift(page_size);
  if (N < 0 || Hkv < 1 || (D != 64 && D != 128) || shift < 0 || num_pages < 1) return CPATTN_ERR_SHAPE;
  if (N > 0x7fffffffL || (long long)N * Hkv > (1LL << 34)) return CPATTN_ERR_SHAPE;
  const long step = 16 / (dtype == CPATTN_FP32 ? 4 : 2);
  for (long st : {k_tok_stride, k_head_stride, v_tok_stride, v_head_stride})
    if (st < 0 || st % step != 0) return CPATTN_ERR_SHAPE;
  if (N == 0) return CPATTN_OK;
  if (!k_new || !v_new || !slots || !k_cache || !v_cache) return CPATTN_ERR_ARG;
  if (cache_dtype == CPATTN_E4M3 && !kv_amax) return CPATTN_ERR_ARG;
  for (const void* p : {k_new, v_new, (const void*)k_cache, (const void*)v_cache, (const void*)k_bounds})
    if (!paged::aligned_to(p, 16)) return CPATTN_ERR_ALIGN;
  if (!paged::aligned_to(slots, 8) || !paged::aligned_to(kv_amax, 4)) return CPATTN_ERR_ALIGN;
  unsigned* err = device_error_word();
  if (!err) return CPATTN_ERR_CUDA;
  AppendArgs a = {};
  a.k = k_new;
  a.v = v_new;
  a.k_tok = k_tok_stride;
  a.k_head = k_head_stride;
  a.v_tok = v_tok_stride;
  a.v_head = v_head_stride;
  a.slots = slots;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.bounds = k_bounds;
  a.kv_amax = kv_amax;
  a.err = err;
  a.N = N;
  a.n_slots = (long long)num_pages << shift;
  a.Hkv = Hkv;
  a.shift = shift;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int n = -1;
  if (cache_dtype == CPATTN_BF16) n = launch_append<__nv_bfloat16, __nv_bfloat16>(a, D, s);
  else if (cache_dtype == CPATTN_FP32) n = launch_append<float, float>(a, D, s);
  else n = launch_append<__nv_bfloat16, paged::E4m3>(a, D, s);
  if (n < 0) return CPATTN_ERR_CUDA;
  add_launches(n);
  return CPATTN_OK;
}

}  // extern "C"
