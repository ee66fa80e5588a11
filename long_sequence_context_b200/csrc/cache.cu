// cache.cu -- the paged key-value cache's books and its rows.
//
// cache_plan: from the requests' lengths and what each asks for (new tokens,
// or tokens taken back) the pages they take from and return to the pool, the
// new tokens' slots and the lengths afterwards.  Integer work of a few bytes
// per request and token: the launch and the prefix sums' latency bound it (16
// requests: 2.9 us; 512 with 116,000 tokens: 5.1 us).
//
// cache_append: new K and V rows into their slots, quantised for an 8-bit
// cache, with the elementwise smallest and largest key of every page kept up
// to date.  Every row is read and written once: the memory bandwidth bounds it
// (8192 tokens x 16 heads x 128 bf16, 135 MB: 25.5 us, 5.3 TB/s, 0.82 of a plain
// copy; in fp32, 268 MB, 52 us; to e4m3, 101 MB, 20.5).
#include <algorithm>

#include "cpattn.h"
#include "kernels.h"
#include "paged.cuh"

namespace cpattn {
namespace {

using namespace paged;

constexpr int kPlanThreads = 1024;
// Up to kSmallR requests, each of many blocks sums them all for itself and takes its
// share of the tokens and pages: one launch.  A block that starts late must still find
// the lengths and the state as they were, so updating them in place takes one block up to
// kSmallTokens tokens, and above (or with more requests) one block that sums and a second
// launch for the rest.
// Measured, many blocks | one block | two launches (us): 16 requests 2.9 | 2.9 | 5.0; 256
// with 595 tokens 3.5 | 4.7 | 6.3; 1000 with 2276 4.6 | 7.7 | 8.0; 512 with 116,000
// 5.1 | 108 | 7.4; the end of a context of 524,288 tokens 3.0 | 7.2 | -.
constexpr int kSmallR = 1024;
constexpr long kSmallTokens = 2048;

// verdict bits of a plan
constexpr int kShort = 1, kBadLength = 2, kCapacity = 4, kBadState = 8;

struct PlanArgs {
  const int32_t *lens, *delta, *free_state;
  int32_t *table, *ring;
  int32_t *lens_out, *state_out, *cu, *verdict;
  int64_t* slots;
  int32_t *head, *pop_at, *push_at;  // workspace of two launches: see Prefix
  unsigned* err;
  long long capacity;
  int R, max_pages, shift, num_pages;
};

struct Three {
  long long a, b, c;
};

// What the requests' prefix sums leave for the items, in shared memory or in the
// workspace (two launches).
struct Prefix {
  int32_t *head;                     // {everything fits, the ring's head, its count}
  int32_t *cu, *pop_at, *push_at;    // [R + 1]: first new token, page taken, page returned
  int32_t *before;                   // [R]: lengths before the step, or null: from those after it
};

__device__ __forceinline__ long long pages_of(long long n, int shift) { return (n + (1 << shift) - 1) >> shift; }

// What request r asks for: new tokens, pages taken, pages returned.
__device__ __forceinline__ Three request_of(const PlanArgs& a, int r, int* bad) {
  const long long n = a.lens[r], after = n + a.delta[r], room = (long long)a.max_pages << a.shift;
  // n too: the pages that a request gives back are read from its row of the table
  if (n < 0 || n > room || after < 0 || after > room) {
    *bad |= kBadLength;
    return {0, 0, 0};
  }
  const long long p0 = pages_of(n, a.shift), p1 = pages_of(after, a.shift);
  return {max(0LL, after - n), max(0LL, p1 - p0), max(0LL, p0 - p1)};
}

// Place i of the ring of n entries (i < 2 n).
__device__ __forceinline__ int ring_at(long long i, int n) { return (int)(i >= n ? i - n : i); }

// One block: prefix sums over the requests, the verdict, and (`writes`) everything
// that has one value per request.  Reads all lengths before it writes any, so that
// lens_out may be lens and state_out free_state.
__device__ __forceinline__ void plan_requests(const PlanArgs& a, const Prefix& p, bool writes) {
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
  // every warp sums the warps' sums for itself
  const Three part = lane < (int)(blockDim.x >> 5) ? s_sum[lane] : Three{0, 0, 0};
  Three sums = part;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, sums.a, o), y = __shfl_up_sync(0xffffffffu, sums.b, o),
                    z = __shfl_up_sync(0xffffffffu, sums.c, o);
    if (lane >= o) sums.a += x, sums.b += y, sums.c += z;
  }
  const Three all = {__shfl_sync(0xffffffffu, sums.a, 31), __shfl_sync(0xffffffffu, sums.b, 31),
                     __shfl_sync(0xffffffffu, sums.c, 31)};
  up.a += __shfl_sync(0xffffffffu, sums.a - part.a, warp);
  up.b += __shfl_sync(0xffffffffu, sums.b - part.b, warp);
  up.c += __shfl_sync(0xffffffffu, sums.c - part.c, warp);
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
    p.cu[r] = ok ? (int)at.a : 0;
    p.pop_at[r] = ok ? (int)at.b : 0;
    p.push_at[r] = ok ? (int)at.c : 0;
    if (p.before) p.before[r] = n;
    if (writes) {
      a.cu[r] = ok ? (int)at.a : 0;
      a.lens_out[r] = ok ? n + a.delta[r] : n;
    }
    at.a += x.a, at.b += x.b, at.c += x.c;
  }
  if (tid == 0) {
    p.cu[a.R] = ok ? (int)all.a : 0;
    p.pop_at[a.R] = ok ? (int)all.b : 0;
    p.push_at[a.R] = ok ? (int)all.c : 0;
    p.head[0] = ok;
    p.head[1] = head;
    p.head[2] = count;
  }
  if (tid == 0 && writes) {
    a.cu[a.R] = ok ? (int)all.a : 0;
    a.state_out[0] = ok ? ring_at(head + all.b, a.num_pages) : head;
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
__device__ __forceinline__ void plan_items(const PlanArgs& a, const Prefix& p, long long i0, long long n) {
  const bool ok = p.head[0] != 0;
  const int head = p.head[1], count = p.head[2];
  const int tokens = p.cu[a.R], pops = p.pop_at[a.R], pushes = p.push_at[a.R];
  auto before_of = [&](int r) { return p.before ? p.before[r] : a.lens_out[r] - a.delta[r]; };  // (ok)
  for (long long i = i0; i < a.capacity; i += n) {
    long long slot = -1;
    if (i < tokens) {
      const int r = find(p.cu, a.R, (int)i);
      const int before = before_of(r);
      const int pos = before + ((int)i - p.cu[r]);
      const int j = pos >> a.shift, held = (int)pages_of(before, a.shift);
      const int page = j < held ? a.table[(size_t)r * a.max_pages + j]
                                : a.ring[ring_at((long long)head + p.pop_at[r] + (j - held), a.num_pages)];
      if (page >= 0 && page < a.num_pages)
        slot = ((long long)page << a.shift) + (pos & ((1 << a.shift) - 1));
      else
        atomicOr(a.err, kErrPage);
    }
    a.slots[i] = slot;
  }
  if (!ok) return;
  // Returned pages go behind the last free one: count + pushes <= num_pages, so none of
  // these places is read.
  auto find_page = [&](int k, const int32_t* at, bool back, size_t& cell, int& place) {
    const int r = find(at, a.R, k);
    const int first = (int)pages_of(back ? before_of(r) + a.delta[r] : before_of(r), a.shift);
    cell = (size_t)r * a.max_pages + first + (k - at[r]);
    place = ring_at((back ? ring_at((long long)head + count, a.num_pages) : head) + (long long)k, a.num_pages);
  };
  // A number outside of the pool is passed on as it is, so that the books still count, and
  // reported: nothing ever follows it.  (Of the pages taken the new tokens report it.)
  auto put_page = [&](bool back, size_t cell, int place, int page) {
    if (back && (unsigned)page >= (unsigned)a.num_pages) atomicOr(a.err, kErrPage);
    if (back) a.ring[place] = page;
    else a.table[cell] = page;
  };
  auto move = [&](int total, const int32_t* at, bool back) {
    // several at a time while there are: one block may have to return the pages of a long context
    constexpr int kAhead = 4;
    long long i = i0;
#pragma unroll 1
    for (; i + (kAhead - 1) * n < total; i += kAhead * n) {
      size_t cell[kAhead];
      int place[kAhead], page[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) find_page((int)(i + x * n), at, back, cell[x], place[x]);
#pragma unroll
      for (int x = 0; x < kAhead; ++x) page[x] = back ? a.table[cell[x]] : a.ring[place[x]];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) put_page(back, cell[x], place[x], page[x]);
    }
#pragma unroll 1
    for (; i < total; i += n) {
      size_t cell;
      int place;
      find_page((int)i, at, back, cell, place);
      put_page(back, cell, place, back ? a.table[cell] : a.ring[place]);
    }
  };
  move(pops, p.pop_at, false);
  move(pushes, p.push_at, true);
}

// Every block sums the requests for itself (lens_out and state_out are other memory than
// lens and free_state, or this is the only block) and takes its share of the items.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
  __shared__ int32_t s_at[4][kSmallR + 1], s_head[3];
  const Prefix p = {s_head, s_at[0], s_at[1], s_at[2], s_at[3]};
  after_previous();
  plan_requests(a, p, blockIdx.x == 0);
  __syncthreads();
  plan_items(a, p, (long long)blockIdx.x * blockDim.x + threadIdx.x, (long long)gridDim.x * blockDim.x);
}
__global__ void __launch_bounds__(kPlanThreads) plan_requests_kernel(const PlanArgs a) {
  after_previous();
  plan_requests(a, {a.head, a.cu, a.pop_at, a.push_at, nullptr}, true);
}
__global__ void __launch_bounds__(256) plan_items_kernel(const PlanArgs a) {
  __shared__ int32_t s_at[3][kSmallR + 1];
  after_previous();
  Prefix p = {a.head, a.cu, a.pop_at, a.push_at, nullptr};
  if (a.R <= kSmallR) {  // searched in shared memory: 512 requests with 80,000 tokens 8.9 us, else 10.9
    for (int i = threadIdx.x; i <= a.R; i += blockDim.x)
      s_at[0][i] = a.cu[i], s_at[1][i] = a.pop_at[i], s_at[2][i] = a.push_at[i];
    __syncthreads();
    p.cu = s_at[0], p.pop_at = s_at[1], p.push_at = s_at[2];
  }
  plan_items(a, p, (long long)blockIdx.x * blockDim.x + threadIdx.x, (long long)gridDim.x * blockDim.x);
}

struct Span {
  const void* p;
  size_t bytes;
};
bool overlap(const Span& x, const Span& y) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  return a < b + y.bytes && b < a + x.bytes;
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

// 16 bytes, in place
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[4]) {
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "l"(p));
}

// V floats as stored; f becomes the numbers that are then stored (unscaled).
template <typename CT, int V>
__device__ __forceinline__ void put(CT* p, float (&f)[V], float s) {
  if constexpr (sizeof(CT) == 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
  } else if constexpr (sizeof(CT) == 2) {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&x);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      w[i] = (uint32_t)float2_to_e4m3x2(__fmul_rn(f[4 * i], s), __fmul_rn(f[4 * i + 1], s)) |
             ((uint32_t)float2_to_e4m3x2(__fmul_rn(f[4 * i + 2], s), __fmul_rn(f[4 * i + 3], s)) << 16);
      Unpack<E4m3>::word(w[i], f + 4 * i);
    }
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

constexpr int kAppendWarps = 4;
constexpr int kTile = 32;  // tokens whose slots one block looks at

// The new rows fall into stretches: tokens next to one another in one page.  A warp
// takes a stretch of one kv head, copies it with kAhead rows' loads under way, 64 tokens
// with their slots in its lanes at a time, reduces its keys and writes the page's bounds:
// no other warp touches these.  Blocks (x: 32 tokens; y: a share of their stretches and
// heads) find the stretches that begin in their tokens by a vote over the slots.
template <typename IT, typename CT, int D>
__global__ void __launch_bounds__(kAppendWarps * 32) append_kernel(const AppendArgs a) {
  constexpr int V = 16 / (int)sizeof(IT);  // elements of a lane
  constexpr int kLanes = D / V, kRows = 32 / kLanes;  // lanes of a row, rows of a warp's load
  constexpr int kAhead = 4;
  after_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int page_mask = (1 << a.shift) - 1;
  const long long t0 = (long long)blockIdx.x * kTile;
  auto slot_of = [&](long long t) { return t < a.N ? a.slots[t] : -1; };
  const long long mine = slot_of(t0 + lane);
  long long before = __shfl_up_sync(0xffffffffu, mine, 1);
  if (lane == 0) before = t0 > 0 ? a.slots[t0 - 1] : -1;
  const bool bad = mine >= a.n_slots;
  if (bad && warp == 0 && blockIdx.y == 0) atomicOr(a.err, kErrPage);
  const bool first = mine >= 0 && !bad && before >> a.shift != mine >> a.shift;
  const uint32_t stretches = __ballot_sync(0xffffffffu, first);
  const int nth = __popc(stretches & ((1u << lane) - 1u));
  const float ks = sizeof(CT) == 1 ? e4m3_scale(a.kv_amax[0]) : 1.f;
  const float vs = sizeof(CT) == 1 ? e4m3_scale(a.kv_amax[1]) : 1.f;
  const int sub = lane / kLanes, d = lane % kLanes * V;

  const int items = __popc(stretches) * a.Hkv;
  for (int item = blockIdx.y * kAppendWarps + warp; item < items; item += gridDim.y * kAppendWarps) {
    const int stretch = item / a.Hkv, h = item % a.Hkv;
    const int from = __ffs(__ballot_sync(0xffffffffu, first && nth == stretch)) - 1;
    const long long t = t0 + from, page = __shfl_sync(0xffffffffu, mine, from) >> a.shift;
    const IT* k = static_cast<const IT*>(a.k) + t * a.k_tok + h * a.k_head + d;
    const IT* v = static_cast<const IT*>(a.v) + t * a.v_tok + h * a.v_head + d;
    const size_t at = (((size_t)page * a.Hkv + h) << a.shift) * D + d;  // of the page's first row
    CT* kc = static_cast<CT*>(a.k_cache) + at;
    CT* vc = static_cast<CT*>(a.v_cache) + at;
    float lo[V], hi[V];
#pragma unroll
    for (int e = 0; e < V; ++e) lo[e] = INFINITY, hi[e] = -INFINITY;
    bool fresh = false;  // the page's first row is among them
    long long slot0 = slot_of(t + lane), slot1 = slot_of(t + 32 + lane);
    for (long long u = t;; u += 64) {
      const uint32_t other0 = ~__ballot_sync(0xffffffffu, slot0 >> a.shift == page);
      const uint32_t other1 = ~__ballot_sync(0xffffffffu, slot1 >> a.shift == page);
      const int n = other0 ? __ffs(other0) - 1 : other1 ? 31 + __ffs(other1) : 64;
      const int row0 = (int)(slot0 & page_mask), row1 = (int)(slot1 & page_mask);
      fresh |= (lane < n && row0 == 0) || (lane + 32 < n && row1 == 0);
      // Rows without a gap are counted: shuffling each out of its lane costs 2 to 5% (5720
      // tokens of one head in pages of 128: 6.4 us, 6.7 with shuffles, 7.0 in steps of 32).
      const int from_row = __shfl_sync(0xffffffffu, row0, 0);
      const bool run = __all_sync(0xffffffffu, (lane >= n || row0 == from_row + lane) &&
                                                   (lane + 32 >= n || row1 == from_row + 32 + lane));
      if (n == 64) slot0 = slot_of(u + 64 + lane), slot1 = slot_of(u + 96 + lane);  // under way meanwhile
#pragma unroll 1
      for (int i0 = 0; i0 < n; i0 += kRows * kAhead) {
        uint32_t kw[kAhead][4], vw[kAhead][4];
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
          const int i = i0 + x * kRows + sub;
          if (i < n) {
            load_words(k + i * a.k_tok, kw[x]);
            load_words(v + i * a.v_tok, vw[x]);
          }
        }
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
          const int i = i0 + x * kRows + sub;
          int to = from_row + i;
          if (!run) to = __shfl_sync(0xffffffffu, i0 < 32 ? row0 : row1, i & 31);
          if (i < n) {
            float f[V], g[V];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              Unpack<IT>::word(kw[x][w], f + w * Unpack<IT>::kPerWord);
              Unpack<IT>::word(vw[x][w], g + w * Unpack<IT>::kPerWord);
            }
            put<CT, V>(kc + to * D, f, ks);
            put<CT, V>(vc + to * D, g, vs);
#pragma unroll
            for (int e = 0; e < V; ++e) lo[e] = fminf(lo[e], f[e]), hi[e] = fmaxf(hi[e], f[e]);
          }
        }
      }
      if (n < 64) break;
      k += 64 * a.k_tok;
      v += 64 * a.v_tok;
    }
    if (!a.bounds) continue;
#pragma unroll
    for (int o = kLanes; o < 32; o <<= 1)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        lo[e] = fminf(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], o));
        hi[e] = fmaxf(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], o));
      }
    fresh = __any_sync(0xffffffffu, fresh);
    if (sub != 0) continue;
    CT* b = static_cast<CT*>(a.bounds) + ((size_t)page * a.Hkv + h) * 2 * D + d;
    if (!fresh) {  // the page held rows before: its first row starts its bounds afresh
      constexpr int W = V * (int)sizeof(CT) / 4;
      uint32_t w[2][W];
#pragma unroll
      for (int i = 0; i < W; ++i) {
        w[0][i] = reinterpret_cast<const uint32_t*>(b)[i];
        w[1][i] = reinterpret_cast<const uint32_t*>(b + D)[i];
      }
#pragma unroll
      for (int i = 0; i < W; ++i) {
        constexpr int P = Unpack<CT>::kPerWord;
        float f[P], g[P];
        Unpack<CT>::word(w[0][i], f);
        Unpack<CT>::word(w[1][i], g);
#pragma unroll
        for (int e = 0; e < P; ++e) lo[i * P + e] = fminf(lo[i * P + e], f[e]), hi[i * P + e] = fmaxf(hi[i * P + e], g[e]);
      }
    }
    // a column of NaN keys alone has no bounds: NaN, which the next key's take the place of
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (lo[e] > hi[e]) lo[e] = hi[e] = NAN;
    // stored values: writing them again rounds nothing
    put<CT, V>(b, lo, 1.f);
    put<CT, V>(b + D, hi, 1.f);
  }
}

template <typename IT, typename CT>
int launch_append(const AppendArgs& a, int D, cudaStream_t s) {
  int dev = 0;
  cudaGetDevice(&dev);
  // A warp for every token and head, so that runs of one token do not queue, up to 32
  // warps an SM (8192 tokens x 16 heads in one run per page, ragged chunks in e4m3, us:
  // 8 warps an SM 30.0, 4.3; 32 25.6, 3.9; 64 25.5, 5.0; 512 39.9, 6.3)
  const long long tiles = (a.N + kTile - 1) / kTile;
  const long long warps = std::min<long long>(a.N * a.Hkv, (long long)num_sms(dev) * 32);
  const long long share = std::max<long long>(1, std::min<long long>(65535, (warps + tiles * kAppendWarps - 1) / (tiles * kAppendWarps)));
  const dim3 grid((unsigned)tiles, (unsigned)share);
  prof_begin(kKCacheAppend, s);
  const cudaError_t e = launch_chained(D == 64 ? append_kernel<IT, CT, 64> : append_kernel<IT, CT, 128>, grid,
                                       kAppendWarps * 32, 0, 0, s, a);
  prof_end(kKCacheAppend, s);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? 1 : -1;
}

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" {

size_t cpattn_cache_plan_workspace_bytes(int R, long capacity) {
  if (R < 1 || (R <= kSmallR && capacity <= kSmallTokens)) return 0;
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
  if (R > 1 << 30) return CPATTN_ERR_SHAPE;  // find() adds two request numbers
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
  const size_t need = cpattn_cache_plan_workspace_bytes(R, capacity);
  if (need && (!workspace || ws_bytes < need)) return CPATTN_ERR_WORKSPACE;
  if (!paged::aligned_to(workspace, 16)) return CPATTN_ERR_ALIGN;
  // Blocks read what others have not written yet: nothing that is written may lie in anything
  // else, but the lengths and the state in their own place.
  const size_t requests = (size_t)R * sizeof(int32_t);
  const Span written[] = {{lens_out, requests}, {free_state_out, 8}, {block_table, requests * max_pages},
                          {free_ring, (size_t)num_pages * 4}, {cu_new, requests + 4}, {slots, (size_t)capacity * 8},
                          {verdict, 4}, {workspace, need}};
  const Span read[] = {{lens, requests}, {free_state, 8}, {delta, requests}};
  for (int i = 0; i < 8; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(written[i], written[j])) return CPATTN_ERR_ARG;
    for (int j = 0; j < 3; ++j)
      if (overlap(written[i], read[j]) && !(i == j && j < 2 && written[i].p == read[j].p)) return CPATTN_ERR_ARG;
  }
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
  if (need) {
    a.head = static_cast<int32_t*>(workspace);
    a.pop_at = a.head + 4;
    a.push_at = a.pop_at + R + 1;
  }
  a.err = err;
  a.capacity = capacity;
  a.R = R;
  a.max_pages = max_pages;
  a.shift = shift;
  a.num_pages = num_pages;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int dev = 0;
  cudaGetDevice(&dev);
  const long long items = std::max<long long>(capacity, std::min<long long>((long long)R * max_pages, num_pages));
  const unsigned blocks =
      (unsigned)std::max<long long>(1, std::min<long long>((items + 255) / 256, (long long)num_sms(dev) * 2));
  const bool in_place = lens == lens_out || free_state == free_state_out;
  const bool many = R <= kSmallR && !in_place;
  if (many || !need) {
    // fewer warps' sums to add in a small block: 16 requests 3.0 us with 256 threads, 5.1 with 1024
    const unsigned threads = many || (R <= 256 && capacity <= 1024) ? 256 : kPlanThreads;
    prof_begin(kKCachePlan, s);
    const cudaError_t e = launch_chained(plan_kernel, dim3(many ? blocks : 1), threads, 0, 0, s, a);
    prof_end(kKCachePlan, s);
    if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return CPATTN_ERR_CUDA;
    add_launches(1);
    return CPATTN_OK;
  }
  prof_begin(kKCachePlan, s);
  cudaError_t e = launch_chained(plan_requests_kernel, dim3(1), kPlanThreads, 0, 0, s, a);
  prof_end(kKCachePlan, s);
  if (e != cudaSuccess) return CPATTN_ERR_CUDA;
  prof_begin(kKCachePlan, s);
  e = launch_chained(plan_items_kernel, dim3(blocks), 256, 0, 0, s, a);
  prof_end(kKCachePlan, s);
  if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return CPATTN_ERR_CUDA;
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
  if (Hkv > 1 << 25) return CPATTN_ERR_SHAPE;  // a block counts 32 stretches of so many heads
  // the stride of an axis of one says nothing
  if (N <= 1) k_tok_stride = v_tok_stride = 0;
  if (Hkv == 1) k_head_stride = v_head_stride = 0;
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
