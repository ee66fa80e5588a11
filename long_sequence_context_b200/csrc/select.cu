// select.cu -- which pages of a long cache one new token attends to.
//
// A page's score for kv head h is the largest q.k that any key inside the
// page's bounds could have, over the query heads of the group:
//     score = max_i sum_d max(q_id lo_d, q_id hi_d)
//           = max_i sum_d (min(q_id, 0) lo_d + max(q_id, 0) hi_d)      (lo <= hi, finite)
// in 64 bits, rounded once to fp32: products of 16-bit values are exact there and
// their sums almost always, so that the order of summation does not decide
// between near pages.  Beside an infinite bound the second form would multiply it by
// 0: there the first one is evaluated, with 0 for a zero of q (bound_of).  A head
// whose sum is NaN does not count.  The `budget` pages with the largest scores are listed in
// ascending order, ties to the lower page; the newest page and the first
// keep_first pages are always among them.
//
// Scoring every page in 64 bits is what that would cost most (64 products a cycle
// and SM).  For 16- and 8-bit bounds the tensor cores score in fp32 first, with an
// error below some eps (derived where it is computed).  The budget-th largest of these
// scores is then within eps of the exact one: of a page more than 2 eps above or below
// it is known on which side it stands, and only those between, a few, are scored in
// 64 bits.
//
// One cluster of thread blocks takes one (request, kv head): every block scores
// a stretch of pages and sends the scores to the first block's shared memory,
// which finds the threshold by a radix search of eight bits at a time and lists
// the pages.  A page's bounds are read once.  What bounds one request is the chain of
// latencies from the lengths over the page table and the bounds to the search, so the
// pages are spread over as many blocks as the device holds at once.  In a batch it is the
// scoring: a warp asks for a step's page numbers, then for its bounds, and only then
// multiplies (of some 11 cycles that a warp takes for an instruction 5.9 are waits for
// memory, which runs at 0.7 of a copy).  fp32 bounds are all scored in 64 bits.
// Measured (8 kv heads, 4 query heads each, D = 128, us; bf16 | e4m3 | fp32): 2048 pages
// 10.4 | 10.4 | 12.4, 8192 pages 25.3 | 24.0 | 37, 16 x 8192 pages 117 | 110 | 252 (bf16
// with every page scored in 64 bits: 33.8 for 8192 pages, 197 for 16 x 8192).
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

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
  int R, Hq, Hkv, group, shift, max_pages, num_pages, budget, keep_first;
};

// unsigned order of the keys = order of the scores; NaN is below every number
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 counts as 0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// the number that order_key maps to k
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// W (a multiple of 4) consecutive words, in place.
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
// c (16 pages x 8 heads, fp32) += a (16 pages x 16 columns) b (16 columns x 8 heads)
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct Pair {  // what a cluster works on
  int r, h, first, n;  // request, kv head; this block's stretch of pages
  const int32_t* table;
};

template <typename CT, int D>
__device__ __forceinline__ const CT* bounds_of(const SelectArgs& a, const Pair& p, int page) {
  return static_cast<const CT*>(a.bounds) + ((size_t)page * a.Hkv + p.h) * 2 * D;
}
// What q is multiplied by for max(q lo, q hi), lo <= hi; NaN if a bound is.
__device__ __forceinline__ float bound_of(float q, float lo, float hi) {
  if (lo != lo || hi != hi) return NAN;
  return q > 0.f ? hi : q < 0.f ? lo : 0.f;
}
__device__ __forceinline__ bool in_pool(const SelectArgs& a, int page) { return (unsigned)page < (unsigned)a.num_pages; }

// Scores of the block's pages in 64 bits on the tensor cores, 8 pages a warp: fp32 bounds.
template <int D>
struct Exact {
  // A warp takes 8 pages at a time, 4 lanes each, in steps of E columns of a lane's low
  // and high bounds.
  static constexpr int E = 8, STEPS = D / (4 * E);
  static constexpr int kQueryBytes = STEPS * E * 32 * 16;

  uint32_t lo[E], hi[E];
  int page, page_next;

  __device__ __forceinline__ int page_of(const Pair& p, int i) const { return p.table[p.first + min(i, p.n - 1)]; }
  __device__ __forceinline__ void load(const SelectArgs& a, const Pair& p, int step) {
    const float* b = bounds_of<float, D>(a, p, in_pool(a, page) ? page : 0) + step * 4 * E + (threadIdx.x & 3) * E;
    load_packed(b, lo);
    load_packed(b + D, hi);
  }
  __device__ __forceinline__ void queries(const SelectArgs&, int, int, int) {}
  // the first pages' loads
  __device__ __forceinline__ void begin(const SelectArgs& a, const Pair& p) {
    const int g = (threadIdx.x & 31) >> 2, i0 = (threadIdx.x >> 5) * 8;
    if (i0 >= p.n) return;
    page = page_of(p, i0 + g);
    page_next = page_of(p, i0 + kWarps * 8 + g);
    load(a, p, 0);
  }

  __device__ __forceinline__ void stage(const SelectArgs& a, const Pair& p, int h0, char* s, float*) {
    double2(*s_q)[32] = reinterpret_cast<double2(*)[32]>(s);  // (min(q, 0), max(q, 0)) of 4 columns x 8 heads
    for (int i = threadIdx.x; i < 8 * D; i += kThreads) {
      const int head = i / D, d = i % D;
      float x = 0.f;
      if (h0 + head < a.group)
        x = static_cast<const float*>(a.q)[((size_t)p.r * a.Hq + (size_t)p.h * a.group + h0 + head) * D + d];
      s_q[d / (4 * E) * E + d % E][head * 4 + d / E % 4] = make_double2(fminf(x, 0.f), fmaxf(x, 0.f));
    }
  }

  // One page's score for one head where the products gave NaN.
  __device__ __noinline__ static float by_terms(const SelectArgs& a, const Pair& p, int page, int head) {
    const float* b = bounds_of<float, D>(a, p, page);
    const float* q = static_cast<const float*>(a.q) + ((size_t)p.r * a.Hq + (size_t)p.h * a.group + head) * D;
    double sum = 0.;
    for (int d = 0; d < D; ++d) sum = fma((double)q[d], (double)bound_of(q[d], b[d], b[D + d]), sum);
    return (float)sum;
  }

  template <typename Put>
  __device__ __forceinline__ float score(const SelectArgs& a, const Pair& p, int h0, const char* s, Put put) {
    const double2(*s_q)[32] = reinterpret_cast<const double2(*)[32]>(s);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    for (int i0 = warp * 8; i0 < p.n; i0 += kWarps * 8) {
      const bool there = in_pool(a, page);
      const int here = page;
      if (!there && t == 0) atomicOr(a.err, kErrPage);
      double acc[4][2] = {};
#pragma unroll
      for (int step = 0; step < STEPS; ++step) {
        float flo[E], fhi[E];
#pragma unroll
        for (int e = 0; e < E; ++e) flo[e] = __uint_as_float(lo[e]), fhi[e] = __uint_as_float(hi[e]);
        if (step + 1 < STEPS) {
          load(a, p, step + 1);
        } else {
          page = page_next;
          if (i0 + kWarps * 8 < p.n) {
            load(a, p, 0);
            page_next = page_of(p, i0 + 2 * kWarps * 8 + g);
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
        float x = (float)((acc[0][m] + acc[1][m]) + (acc[2][m] + acc[3][m]));
        if (there && h0 + 2 * t + m < a.group) {
          if (x != x) x = by_terms(a, p, here, h0 + 2 * t + m);
          key = max(key, order_key(x));
        }
      }
      key = max(key, __shfl_xor_sync(0xffffffffu, key, 1));
      key = max(key, __shfl_xor_sync(0xffffffffu, key, 2));
      if (t == 0 && i0 + g < p.n) put(p.first + i0 + g, key);
    }
    return 0.f;
  }
};

// The same in fp32 with bf16 operands, 16 pages a warp; also the largest |bound|
// and, staging, the largest sum |q| of a head.
template <typename CT, int D>
struct Approx {
  static constexpr int W = D * (int)sizeof(CT) / 16;  // words of a lane's quarter of a row
  static constexpr int kQueryBytes = D / 32 * 2 * 32 * 16;

  // A lane's quarter of a row are its 16-byte pieces t, t + 4, ...: entry e of 8 columns is
  // piece e (bf16) or half of piece e / 2 (e4m3).
  __device__ static __forceinline__ void load(const CT* row, int t, uint32_t (&w)[W]) {
#pragma unroll
    for (int i = 0; i < W; i += 4)
      asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                   : "l"(reinterpret_cast<const char*>(row) + 16 * (i + t)));
  }

  uint32_t q[4], lo[2][W], hi[2][W];
  int page[2];

  // a warp's head and a lane's 8 columns of it
  __device__ __forceinline__ void queries(const SelectArgs& a, int r, int h, int h0) {
    static_assert(kWarps == 8, "a warp for each head");
    const int lane = threadIdx.x & 31, head = threadIdx.x >> 5;
    q[0] = q[1] = q[2] = q[3] = 0u;
    if (h0 + head < a.group && lane < D / 8)
      load_packed(static_cast<const __nv_bfloat16*>(a.q) + ((size_t)r * a.Hq + (size_t)h * a.group + h0 + head) * D + lane * 8, q);
  }
  __device__ __forceinline__ void pages(const SelectArgs& a, const Pair& p, int i0) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) page[r] = p.table[p.first + min(i0 + g + 8 * r, p.n - 1)];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const CT* b = bounds_of<CT, D>(a, p, in_pool(a, page[r]) ? page[r] : 0);
      load(b, t, lo[r]);
      load(b + D, t, hi[r]);
    }
  }
  // the first pages' loads
  __device__ __forceinline__ void begin(const SelectArgs& a, const Pair& p) {
    const int i0 = (threadIdx.x >> 5) * 16;
    if (i0 < p.n) pages(a, p, i0);
  }

  // s: [entry][min(q, 0), max(q, 0)][lane] 16 bytes
  __device__ __forceinline__ void stage(const SelectArgs&, const Pair&, int h0, char* s, float* norm) {
    const int lane = threadIdx.x & 31, head = threadIdx.x >> 5;
    // the lane and entry that columns 8 * lane .. + 7 belong to: see load()
    const int t = sizeof(CT) == 2 ? lane & 3 : (lane >> 1) & 3;
    const int e = sizeof(CT) == 2 ? lane >> 2 : (lane >> 3) * 2 + (lane & 1);
    float sum = 0.f;
    uint32_t neg[4], pos[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[2];
      Unpack<__nv_bfloat16>::word(q[i], f);
      sum += fabsf(f[0]) + fabsf(f[1]);
      const uint32_t minus = ((q[i] & 0x8000u) ? 0xffffu : 0u) | ((q[i] & 0x80000000u) ? 0xffff0000u : 0u);
      neg[i] = q[i] & minus;
      pos[i] = q[i] & ~minus;
    }
    if (lane < D / 8) {
      uint4* to = reinterpret_cast<uint4*>(s) + e * 64 + head * 4 + t;
      to[0] = make_uint4(neg[0], neg[1], neg[2], neg[3]);
      to[32] = make_uint4(pos[0], pos[1], pos[2], pos[3]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) norm[head] = h0 == 0 ? sum : fmaxf(norm[head], sum);
  }

  // words 2i, 2i + 1 (e4m3: word i) of a lane's quarter as two bf16 pairs
  __device__ static __forceinline__ void pairs(const uint32_t (&w)[W], int i, uint32_t& x, uint32_t& y) {
    if constexpr (sizeof(CT) == 2) {
      x = w[2 * i], y = w[2 * i + 1];
    } else {
      float f[4];
      Unpack<E4m3>::word(w[i], f);
      const __nv_bfloat162 u = __floats2bfloat162_rn(f[0], f[1]), v = __floats2bfloat162_rn(f[2], f[3]);
      x = *reinterpret_cast<const uint32_t*>(&u), y = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
  __device__ static __forceinline__ __nv_bfloat162 as2(uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); }

  template <typename Put>
  __device__ __forceinline__ float score(const SelectArgs& a, const Pair& p, int h0, const char* s, Put put) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    __nv_bfloat162 most = __float2bfloat162_rn(0.f);
    for (int i0 = warp * 16; i0 < p.n; i0 += kWarps * 16) {
      if (i0 > warp * 16) pages(a, p, i0);
      float c[4][4] = {};
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        const uint4 qn = reinterpret_cast<const uint4*>(s)[e * 64 + lane], qp = reinterpret_cast<const uint4*>(s)[e * 64 + 32 + lane];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t x[2], y[2], z[2], w[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            pairs(lo[r], 2 * e + half, x[r], y[r]);
            pairs(hi[r], 2 * e + half, z[r], w[r]);
            most = __hmax2(most, __hmax2(__hmax2(__habs2(as2(x[r])), __habs2(as2(y[r]))), __hmax2(__habs2(as2(z[r])), __habs2(as2(w[r])))));
          }
          mma_bf16(c[2 * half], x[0], x[1], y[0], y[1], half ? qn.z : qn.x, half ? qn.w : qn.y);
          mma_bf16(c[2 * half + 1], z[0], z[1], w[0], w[1], half ? qp.z : qp.x, half ? qp.w : qp.y);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const bool there = in_pool(a, page[r]);
        if (!there && t == 0) atomicOr(a.err, kErrPage);
        uint32_t key = 0u;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int i = 2 * r + m;
          if (there && h0 + 2 * t + m < a.group) key = max(key, order_key((c[0][i] + c[1][i]) + (c[2][i] + c[3][i])));
        }
        key = max(key, __shfl_xor_sync(0xffffffffu, key, 1));
        key = max(key, __shfl_xor_sync(0xffffffffu, key, 2));
        if (t == 0 && i0 + g + 8 * r < p.n) put(p.first + i0 + g + 8 * r, key);
      }
    }
    return fmaxf(__low2float(most), __high2float(most));
  }

  // The largest score of page j over heads h0 .. h1 - 1 in 64 bits, by a whole warp.
  __device__ static uint32_t rescore(const SelectArgs& a, const Pair& p, int j, int h0, int h1) {
    const int lane = threadIdx.x & 31;
    constexpr int V = D / 32;  // columns of a lane
    const int page = p.table[j];
    if (!in_pool(a, page)) return 0u;
    const CT* b = bounds_of<CT, D>(a, p, page) + lane * V;
    float lo[V], hi[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if constexpr (sizeof(CT) == 2) {
        lo[e] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(b)[e]);
        hi[e] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(b + D)[e]);
      } else {
        float f[4];
        Unpack<E4m3>::word(reinterpret_cast<const uint8_t*>(b)[e], f);
        lo[e] = f[0];
        Unpack<E4m3>::word(reinterpret_cast<const uint8_t*>(b + D)[e], f);
        hi[e] = f[0];
      }
    }
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + ((size_t)p.r * a.Hq + (size_t)p.h * a.group) * D + lane * V;
    uint32_t key = 0u;
    for (int m = h0; m < h1; ++m) {
      double sum = 0.;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float x = __bfloat162float(q[(size_t)m * D + e]);
        sum = fma((double)x, (double)bound_of(x, lo[e], hi[e]), sum);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      key = max(key, order_key((float)sum));
    }
    return key;
  }
};

constexpr uint32_t kAlways = 0xffffffffu;  // key of a page that is listed whatever its score

struct Search {
  uint32_t hist[256], bin[kThreads], warp[3][kWarps], pick[3], found;
};

// The budget-th largest of n keys: every key above `threshold` is taken, and the
// first `need` equal to it.  First the leading bits that all keys share, then
// eight bits at a time until the bin of the threshold is small enough to rank its
// keys directly.  `itself`: the threshold has to be that key itself, not a
// number below a bin that is taken whole.
__device__ __noinline__ void find_threshold(const uint32_t* keys, int n, int budget, bool itself, Search& s, uint32_t& threshold, int& need) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto each = [&](auto f) {
    for (int i = 4 * tid; i < n; i += 4 * kThreads) {
      const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
      f(k.x);
      if (i + 1 < n) f(k.y);
      if (i + 2 < n) f(k.z);
      if (i + 3 < n) f(k.w);
    }
  };
  uint32_t any = 0u, all = 0xffffffffu, always = 0u;
  each([&](uint32_t key) {
    if (key == kAlways) ++always;
    else any |= key, all &= key;
  });
  any = __reduce_or_sync(0xffffffffu, any);
  all = __reduce_and_sync(0xffffffffu, all);
  always = __reduce_add_sync(0xffffffffu, always);
  __syncthreads();
  s.hist[tid & 255] = 0;
  if (lane == 0) s.warp[0][warp] = any, s.warp[1][warp] = all, s.warp[2][warp] = always;
  if (tid == 0) s.found = 0;
  __syncthreads();
  always = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) any |= s.warp[0][w], all &= s.warp[1][w], always += s.warp[2][w];
  int low = 32 - __clz(any ^ all);               // bits below `low` differ
  uint32_t prefix = low < 32 ? any >> low : 0u;  // of the threshold
  need = budget - (int)always;                   // keys wanted among those that share the prefix
  threshold = any;
  if (need <= 0) low = 0, need = 0, threshold = kAlways - 1u;
  while (low > 0) {
    const int above = low;
    low = max(0, low - 8);
    const uint32_t digits = (1u << (above - low)) - 1u;
    each([&](uint32_t key) {
      if (key != kAlways && (above == 32 || (key >> above) == prefix)) atomicAdd(&s.hist[(key >> low) & digits], 1u);
    });
    __syncthreads();
    // thread b: keys in bin 255 - b; inclusive sums from the top
    const uint32_t c = s.hist[255 - tid];
    uint32_t up = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += x;
    }
    if (lane == 31) s.warp[0][warp] = up;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (w < warp) up += s.warp[0][w];
    if (up >= (uint32_t)need && up - c < (uint32_t)need) s.pick[0] = 255 - tid, s.pick[1] = need - (up - c), s.pick[2] = c;
    s.hist[255 - tid] = 0;
    __syncthreads();
    prefix = (above == 32 ? 0u : prefix << (above - low)) | s.pick[0];
    need = (int)s.pick[1];
    threshold = prefix << low;
    const uint32_t in_bin = s.pick[2];
    if (low == 0) break;
    if (in_bin == (uint32_t)need && !itself && threshold > 0u) {  // the whole bin is taken
      threshold -= 1u;
      need = 0;
      break;
    }
    if (in_bin <= (uint32_t)kThreads) {  // rank the bin's keys: one for each thread
      each([&](uint32_t key) {
        if (key != kAlways && (key >> low) == prefix) s.bin[atomicAdd(&s.found, 1u)] = key;
      });
      __syncthreads();
      if (tid < (int)in_bin) {
        const uint32_t key = s.bin[tid];
        uint32_t more = 0, same = 0;
        for (uint32_t i = 0; i < in_bin; ++i) more += s.bin[i] > key, same += s.bin[i] == key;
        // equal keys write the same two numbers
        if (more < (uint32_t)need && more + same >= (uint32_t)need) s.pick[0] = key, s.pick[1] = need - more;
      }
      __syncthreads();
      threshold = s.pick[0];
      need = (int)s.pick[1];
      break;
    }
  }
  __syncthreads();
}

template <typename CT, int D>
__global__ void __launch_bounds__(kThreads) select_kernel(const SelectArgs a) {
  constexpr bool kApprox = sizeof(CT) < 4;
  using Scores = std::conditional_t<kApprox, Approx<CT, D>, Exact<D>>;
  extern __shared__ __align__(16) uint32_t s_key[];  // the first block's: the keys of all pages
  __shared__ __align__(16) char s_q[Scores::kQueryBytes];
  __shared__ Search s_search;
  __shared__ uint32_t s_count[2][kWarps], s_list[kThreads], s_listed;
  __shared__ float s_most[kMaxCluster], s_warp_most[kWarps];
  __shared__ float s_norm[8];
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int pair = blockIdx.x / ranks;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* out = a.sel + (size_t)pair * a.budget;
  Scores scores;
  Pair p = {pair / a.Hkv, pair % a.Hkv, 0, 0, nullptr};

  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this block has started
  if (tid == 0) s_listed = 0u;
  after_previous();
  scores.queries(a, p.r, p.h, 0);
  p.table = a.table + (size_t)p.r * a.max_pages;
  for (int i = 32 * (rank * kThreads + tid); i < a.max_pages; i += 32 * kThreads * ranks)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.table + i));  // while the length is under way
  const long long cap = (long long)a.max_pages << a.shift;
  long long len = a.lens[p.r];
  if (len < 0 || len > cap) {
    if (tid == 0) atomicOr(a.err, kErrPage);
    len = len < 0 ? 0 : cap;
  }
  const int held = (int)((len + (1 << a.shift) - 1) >> a.shift);
  if (held <= a.budget) {  // everything is selected (the whole cluster leaves here)
    // unsigned: a step past a budget near 2^31 is no int
    for (unsigned j = rank * kThreads + tid; j < (unsigned)a.budget; j += ranks * kThreads) out[j] = (int)j < held ? (int)j : -1;
    __syncwarp();
    cluster.barrier_wait();
    return;
  }

  const int per = (held + ranks - 1) / ranks;
  p.first = min(rank * per, held);
  p.n = min(per, held - p.first);
  uint32_t* keys = cluster.map_shared_rank(s_key, 0);
  for (int h0 = 0; h0 < a.group; h0 += 8) {
    if (h0 > 0) {
      scores.queries(a, p.r, p.h, h0);
      __syncthreads();
    }
    scores.begin(a, p);
    scores.stage(a, p, h0, s_q, s_norm);
    if (h0 == 0) cluster.barrier_wait();  // no block writes to the first one before that has started
    __syncthreads();
    float most = scores.score(a, p, h0, s_q, [&](int j, uint32_t key) {
      if (j < a.keep_first || j == held - 1) key = kAlways;
      keys[j] = h0 == 0 ? key : max(key, keys[j]);
    });
    if constexpr (kApprox) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      if (lane == 0 && h0 == 0) s_warp_most[warp] = most;
    }
  }
  if constexpr (kApprox) {
    __syncthreads();
    if (tid == 0) {
      float most = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) most = fmaxf(most, s_warp_most[w]);
      *cluster.map_shared_rank(&s_most[rank], 0) = most;
    }
  }
  cluster.sync();
  if (rank != 0) return;

  uint32_t threshold;
  int need;
  find_threshold(s_key, held, a.budget, kApprox, s_search, threshold, need);
  // a stretch of pages for each thread
  const int mine = 4 * ((held + 4 * kThreads - 1) / (4 * kThreads));
  const int i0 = min(tid * mine, held), i1 = min(i0 + mine, held);
  auto each = [&](auto f) {
    for (int i = i0; i < i1; i += 4) {
      const uint4 k = *reinterpret_cast<const uint4*>(s_key + i);
      f(i, k.x);
      if (i + 1 < i1) f(i + 1, k.y);
      if (i + 2 < i1) f(i + 2, k.z);
      if (i + 3 < i1) f(i + 3, k.w);
    }
  };
  if constexpr (kApprox) {
    if (threshold != kAlways - 1u) {
      // [low, high]: the keys within 2 eps of the threshold
      float norm = 0.f, most = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) norm = fmaxf(norm, s_norm[i]);
      for (int i = 0; i < ranks; ++i) most = fmaxf(most, s_most[i]);
      const float at = key_value(threshold);
      // The error of a score in fp32.  Each of the four accumulators takes D / 2 products, exact
      // before they are added, by D / 32 instructions of 16.  Whatever order an instruction adds
      // its 17 numbers in, rounding or cutting off each sum to fp32, or cutting all of them off
      // at the largest one's last place: it loses at most 17 units of 2^-23 S_i, S_i the sum of
      // the accumulator's |terms|.  The three sums of the accumulators lose less than 2 2^-23
      // sum S_i, and sum S_i <= sum |q| max |bound|, whose own rounding the 1.01 covers.  Then the
      // rounding of the exact score, and products and operands below the normal range.  (A band
      // twice as wide: 2048 pages 10.8 us for 10.0.)
      const float eps = norm * most * ((17 * D / 32 + 3) * 0x1p-23f) * 1.01f + fabsf(at) * 0x1p-22f +
                        2 * D * 0x1p-126f * (norm + most + 1.f);
      uint32_t low = 0u, high = kAlways - 1u;
      if (threshold != 0u && eps < 1e37f && fabsf(at) < 1e37f)
        low = order_key(__fadd_rd(at, -2.f * eps)), high = min(high, order_key(__fadd_ru(at, 2.f * eps)));
      uint32_t above = 0;
      each([&](int i, uint32_t key) {
        above += key > high;
        if (key >= low && key <= high) {
          const uint32_t at = atomicAdd(&s_listed, 1u);
          if (at < (uint32_t)kThreads) s_list[at] = i, s_search.bin[at] = 0u;
        }
      });
      above = __reduce_add_sync(0xffffffffu, above);
      if (lane == 0) s_count[0][warp] = above;
      __syncthreads();
      const uint32_t within = s_listed;
      above = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) above += s_count[0][w];
      if (above + within == (uint32_t)a.budget) {  // those within are taken too
        threshold = low - 1u;
        need = 0;
        __syncthreads();
      } else if (within <= (uint32_t)kThreads) {
        // score some heads of a page with each warp, rank a page with each thread
        const int heads = max(1, min(a.group, (int)((within * a.group + kWarps - 1) / kWarps)));
        const int parts = (a.group + heads - 1) / heads;
        for (int i = warp; i < (int)within * parts; i += kWarps) {
          const int x = i / parts, h0 = (i - x * parts) * heads;
          const uint32_t exact = Scores::rescore(a, p, (int)s_list[x], h0, min(h0 + heads, a.group));
          if (lane == 0) atomicMax(&s_search.bin[x], exact);
        }
        __syncthreads();
        if (tid < (int)within) {
          const uint32_t key = s_search.bin[tid], page = s_list[tid];
          uint32_t before = above;
          for (uint32_t i = 0; i < within; ++i)
            before += s_search.bin[i] > key || (s_search.bin[i] == key && s_list[i] < page);
          s_key[page] = before < (uint32_t)a.budget ? kAlways : 0u;
        }
        __syncthreads();
        threshold = high;
        need = 0;
      } else {
        // a stretch of pages for each warp, in steps of 32
        const int stretch = ((held + kWarps - 1) / kWarps + 31) & ~31;
        const int w0 = min(warp * stretch, held), w1 = min(w0 + stretch, held);
        for (int j0 = w0; j0 < w1; j0 += 32) {
          const int i = j0 + lane;
          const uint32_t key = i < w1 ? s_key[i] : 0u;
          const bool mid = i < w1 && key >= low && key <= high;
          if (i < w1 && !mid) s_key[i] = key > high ? kAlways : 0u;
          uint32_t left = __ballot_sync(0xffffffffu, mid);
          while (left) {
            const int b = __ffs(left) - 1;
            left &= left - 1u;
            const uint32_t exact = Scores::rescore(a, p, j0 + b, 0, a.group);
            if (lane == 0) s_key[j0 + b] = exact;
          }
        }
        __syncthreads();
        find_threshold(s_key, held, a.budget, false, s_search, threshold, need);
      }
    }
  }

  // every key above the threshold and the first `need` equal to it, in order
  uint32_t count = 0;  // keys above (high half) and equal (low half): at most kMaxPages of each
  each([&](int, uint32_t key) { count += key > threshold ? 0x10000u : (key == threshold ? 1u : 0u); });
  uint32_t up = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += x;
  }
  if (lane == 31) s_count[0][warp] = up;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < warp) up += s_count[0][w];
  up -= count;
  uint32_t above = up >> 16, equal = up & 0xffffu;
  if (count != 0u)
    each([&](int i, uint32_t key) {
      if (key > threshold || (key == threshold && equal < (uint32_t)need)) out[above + min(equal, (uint32_t)need)] = i;
      above += key > threshold;
      equal += key == threshold;
    });
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
                                       ((size_t)a.max_pages + 3) / 4 * 16, cluster, s, a);
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
  int dev = 0;
  cudaGetDevice(&dev);
  // Blocks per pair: while there are at most four to an SM, and a block still has 64
  // pages; at most 8 where the scores leave room for one block to an SM.  Measured (us):
  // 8 pairs of 2048 pages with 2, 8, 16 blocks each 21.0, 12.7, 12.1; of 8192 pages 57.9,
  // 26.9, 25.6; 128 pairs of up to 1024 pages with 1, 2, 4, 8 blocks an SM (and the
  // attention) 54.1, 48.2, 44.1, 47.
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
