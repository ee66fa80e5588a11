// decode.cu -- attention of one new token per request over a paged key-value
// cache: for every (request r, query head i) with kv head h = i / group,
//     x_j = scale * q_i . k_j,   o_i = sum_j softmax_j(x) v_j,   lse_i = log sum_j e^{x_j}
// over the request's keys, or over the pages that a list selects.
//
// The keys are cut into units of 64 to 256 (16 KB of keys).  All units of all
// (request, kv head) pairs, with kPairCost more for each pair, form one line,
// which is dealt to the thread blocks in equal contiguous shares: a block finds
// its share from the lengths alone, on the device, so that a batch of very
// different lengths keeps every block equally busy and the host needs no length.
// A pair that lies inside one block is finished there; the others leave one
// partial result (running maximum, sum, unnormalised output, all fp32) per block,
// and join_kernel combines them by the log-sum-exp rule of cpattn_merge.
//
// Where the table (or the selection) has room for a few units a block only, a cluster
// of up to 16 blocks takes each pair instead and joins through shared memory: one
// launch, and no search for a share (see one_shape).
//
// What bounds it: K and V are read once, in bf16 and for up to 16 heads a group at
// 93 to 99% of a plain copy's bandwidth (32768 keys x 32 heads x 128: 537 MB in 84
// us, 6.4 TB/s; 131072 x 8 heads in e4m3, where the codes' widening doubles the
// instructions for a byte: 268 MB in 49 us), beside some 6 us of start, partial
// results and join.  Short contexts wait for a chain of latencies (launch, length,
// page, keys, join): 16 keys take 3.7 to 4.8 us, 257 keys x 16 heads 5.0.  Many heads a
// group wait for their instructions with two warps a scheduler: 268 MB with 32 heads take
// 66 us in bf16 (tensor pipe 38% busy, issue slots 37%), with 16 heads 56 in e4m3 (45%,
// 37%) and 97 in fp32 (FMA pipe 34%, issue slots 50%).  Sharing a ring between the warps
// of a group of 32 took longer (77 us for 70 at the time).
#include <cooperative_groups.h>

#include <algorithm>

#include "cpattn.h"
#include "kernels.h"
#include "paged.cuh"
#include "sm100.cuh"
#include "tmap.h"

namespace cpattn {
namespace {

using namespace paged;
namespace cg = cooperative_groups;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kNothing = -3.0e38f;  // the running maximum before any key: finite, so that no difference is inf - inf
constexpr int kChunk = 16;  // keys of one block; never straddles pages
// What starting and finishing a pair costs, in units of keys: without it a block
// that draws many short pairs ends last (48 requests of 1 to 16384 keys: 97 us with
// 0, 67.5 with 2, 66 to 66.6 with 3 to 8).
constexpr int kPairCost = 4;
constexpr int kMaxGroup = 64;
constexpr int kMostCluster = 16;

struct DecodeArgs {
  const void *q, *k, *v;
  const int32_t *table, *lens, *pages;
  void* o;
  float *lse, *part_o, *part_ml;
  int4* tail;  // notes for the join: {request, kv head, last block, first block} or {-1}
  int by_pair;  // one note for each pair (fewer pairs than blocks), else one for each block
  const float* kv_amax;
  unsigned* err;
  int R, Hq, Hkv, group, shift, max_pages, num_pages, budget;
  float scale_log2;
  int o_bf16, stall;
};

// Keys of request r in the order its page list gives them (whole pages where
// a selection is read: positions behind the length are masked one by one).
__device__ __forceinline__ int request_len(const DecodeArgs& a, int r, bool report) {
  int n = a.lens[r];
  const long long cap = (long long)a.max_pages << a.shift;
  if (n < 0 || n > cap) {
    if (report) atomicOr(a.err, kErrPage);
    n = n < 0 ? 0 : (int)cap;
  }
  return n;
}
__device__ __forceinline__ int listed_pages(const DecodeArgs& a, int len) {
  const int held = (int)(((long long)len + (1 << a.shift) - 1) >> a.shift);
  return a.pages ? min(held, a.budget) : held;
}
template <int UNIT>
__device__ __forceinline__ int request_units(const DecodeArgs& a, int len) {
  const unsigned keys = a.pages ? (unsigned)listed_pages(a, len) << a.shift : (unsigned)len;
  return (int)((keys + UNIT - 1) / UNIT);
}
// Length of a pair on the line: its units and what a pair costs by itself.
__device__ __forceinline__ int pair_weight(int units) { return units == 0 ? 0 : units + kPairCost; }

// 2^x, 0 below 2^-126
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// outputs i .. i + N - 1 (N = 2 or 4, i a multiple of N)
template <int N>
__device__ __forceinline__ void store_o(const DecodeArgs& a, size_t i, const float (&x)[N]) {
  if (a.o_bf16) {
    uint32_t w[N / 2];
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&y);
    }
    void* to = static_cast<__nv_bfloat16*>(a.o) + i;
    if constexpr (N == 4) *static_cast<uint2*>(to) = make_uint2(w[0], w[1]);
    else *static_cast<uint32_t*>(to) = w[0];
  } else {
    void* to = static_cast<float*>(a.o) + i;
    if constexpr (N == 4) *static_cast<float4*>(to) = make_float4(x[0], x[1], x[2], x[3]);
    else *static_cast<float2*>(to) = make_float2(x[0], x[1]);
  }
}
// A head's weighted sum and sum of weights (reference m) as the output and the
// log-sum-exp.  A head without a key: o = 0, lse = -inf.
template <int N>
__device__ __forceinline__ void finish(const DecodeArgs& a, size_t out, int D, int d, float (&o)[N], float m, float l) {
  const float f = l == 0.f ? 0.f : __frcp_rn(l);
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] *= f;
  store_o<N>(a, out * D + d, o);
  if (d == 0) a.lse[out] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// One warp's view of 16 keys in shared memory.  Lane 4g + t holds, for every 8
// heads, the scores of two keys (slots g and g + 8) with heads 2t and 2t + 1, and
// of the output 8 columns for every 64 (col()) of the same two heads: the
// accumulator layout of mma.m16n8k16 with the keys (scores) or the columns
// (output) as its 16 rows.
//
// The 16 rows of K, and those of V, are one contiguous block of the cache.  TMA
// brings it as lines of 128 bytes whose 16-byte pieces are permuted (piece p of
// line i stands at p ^ (i & 7)), and the lanes' order of keys and columns, which
// both products leave free, is chosen per type so that the pieces a quarter of a
// warp reads fall into different banks.
__device__ __forceinline__ const char* piece(const char* block, int line, int p) {
  return block + line * 128 + ((p ^ (line & 7)) << 4);
}

// FmaTile: fp32 caches, fp32 arithmetic throughout.
template <int D, int NT>
struct FmaTile {
  using CT = float;
  static constexpr int kQueryBytes = D * 4;  // shared memory of one head's query
  static constexpr float kLift = -4.f, kSlack = 4.f;  // weights up to 1: see MmaTile
  // Blocks of 16 keys a warp takes at a time, how many times that it has under way, and
  // thread blocks of an SM.  Many warps hide the arithmetic better than deep rings (268 MB,
  // D = 128: as here 55 us; two blocks one deep 59, one block two deep 62).
  static constexpr int kSub = 1, kDepth = D == 128 ? 1 : 2, kCtas = NT == 1 ? 3 : 2;
  static constexpr int kLineStart = 6;   // what the line's second launch costs: see one_shape
  static constexpr int kLines = D / 32;  // of a row

  __device__ static __forceinline__ int col(int h, int g, int e) { return 64 * h + 8 * g + e; }
  __device__ static __forceinline__ int key_of(int slot) { return slot; }
  // piece v of lane t's quarter of a line (two of eight)
  __device__ static __forceinline__ int quarter(int t, int v) {
    return kLines == 4 ? t + 4 * v : (t & 1) + 4 * (t >> 1) + 2 * v;
  }

  // the queries of `heads` heads from row `at` of q on, for all warps of this block
  __device__ static __forceinline__ void stage_queries(char* s, float*, const void* q, size_t at, int group, int heads) {
    for (int i = threadIdx.x; i < heads * D; i += kThreads)
      reinterpret_cast<float*>(s)[i] = i / D < group ? static_cast<const float*>(q)[at * D + i] : 0.f;
  }

  __device__ static __forceinline__ void scores(const char* k, const char* s_q, float (&s)[NT][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float acc[2][8] = {};
#pragma unroll
      for (int l = 0; l < kLines; ++l)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          float4 x[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) x[r] = *reinterpret_cast<const float4*>(piece(k, (g + 8 * r) * kLines + l, quarter(t, v)));
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const float4 f = *reinterpret_cast<const float4*>(s_q + (nt * 8 + n) * D * 4 + l * 128 + quarter(t, v) * 16);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              acc[r][n] = fmaf(f.x, x[r].x, acc[r][n]);
              acc[r][n] = fmaf(f.y, x[r].y, acc[r][n]);
              acc[r][n] = fmaf(f.z, x[r].z, acc[r][n]);
              acc[r][n] = fmaf(f.w, x[r].w, acc[r][n]);
            }
          }
        }
      // sum over the quad; lane t is left with heads 2t and 2t + 1
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float keep = (t & 2) ? acc[r][4 + i] : acc[r][i], give = (t & 2) ? acc[r][i] : acc[r][4 + i];
          b[i] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float keep = (t & 1) ? b[2 + i] : b[i], give = (t & 1) ? b[i] : b[2 + i];
          s[nt][2 * r + i] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
        }
      }
    }
  }

  // acc += p v; n_valid: rows behind it hold anything and count as zero
  __device__ static __forceinline__ void output(const char* v, const float (&p)[NT][4], int n_valid,
                                                float (&acc)[NT][D / 64][16]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll 4
    for (int kk = 0; kk < kChunk; ++kk) {
      float x[D / 64][8];
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          float4 u = *reinterpret_cast<const float4*>(piece(v, kk * kLines + 2 * h + (g >> 2), 2 * (g & 3) + e / 4));
          if (kk >= n_valid) u = make_float4(0.f, 0.f, 0.f, 0.f);
          x[h][e] = u.x, x[h][e + 1] = u.y, x[h][e + 2] = u.z, x[h][e + 3] = u.w;
        }
      const int src_lane = (kk & 7) * 4 + t;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float p0 = __shfl_sync(0xffffffffu, kk < 8 ? p[nt][0] : p[nt][2], src_lane);
        const float p1 = __shfl_sync(0xffffffffu, kk < 8 ? p[nt][1] : p[nt][3], src_lane);
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            acc[nt][h][2 * e] = fmaf(p0, x[h][e], acc[nt][h][2 * e]);
            acc[nt][h][2 * e + 1] = fmaf(p1, x[h][e], acc[nt][h][2 * e + 1]);
          }
      }
    }
  }
};

__device__ __forceinline__ void mma_16816(bool half, float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  if (half)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// MmaTile: bf16 and e4m3 caches on the tensor cores, S^T = K Q^T and O^T = V^T P^T
// with up to 8 heads as the narrow side, so that a group of few heads wastes
// little.  A lane's 16 bytes of consecutive columns are at once its share of one
// or more operands (the contraction index may be permuted at will).  8-bit codes
// are widened to half precision, which holds them exactly; the queries then are
// in half precision too, scaled per head by a power of two: entries down to 2^-31 of
// the head's largest keep all their bits, smaller ones are off by 2^-39 of it at most.
// The weights enter as the sum of two 16-bit numbers, off by at most 2^-17 relative in
// bf16 and by 2^-22, or 2^-39 of the largest weight, in half precision: the kernel waits
// for memory, the second product is free, and fp32 outputs stay good to that.
template <typename C, int D, int NT>
struct MmaTile {
  using CT = C;
  static constexpr bool kHalf = sizeof(C) == 1;
  static constexpr int kQueryBytes = D * 2;
  static constexpr int kRowBytes = D * (int)sizeof(C);  // 256, 128 or 64
  // 8 KB of K and V at a time and twice that under way for each warp, 128 KB for an SM.
  // Measured (32768 keys x 32 heads bf16; 131072 x 8 e4m3, us): as here 84.6, 51.0 (e4m3 has gained 2 since); three
  // blocks of an SM 86.4, 53.0 (more partial results); three deep 87.5, 53.2; one block
  // six deep 88.0, 65.2; e4m3 in steps of 16 keys, four deep, 54.3.  Rows of 64 bytes (e4m3,
  // D = 64), the most instructions for a byte, take a third block: 268 MB 51 us, else 58.
  static constexpr int kSub = 256 / kRowBytes;
  static constexpr int kDepth = 2;
  static constexpr int kLineStart = 12;  // what the line's second launch costs: see one_shape
  static constexpr int kCtas = NT == 1 && kRowBytes == 64 ? 3 : 2;
  // The largest weight lies between 2^kLift and 2^(kLift + kSlack): half precision ends at
  // 2^-24, which must be far below the largest weight of a long context.  bf16 reaches as far
  // as fp32, so there no weight is above 1 and the sums overflow only where n max|v| does.
  static constexpr float kLift = kHalf ? 14.f : -4.f, kSlack = kHalf ? 1.f : 4.f;

  __device__ static __forceinline__ int col(int h, int g, int e) {
    return kHalf ? D / 8 * g + 8 * h + e : 64 * h + 8 * g + e;
  }
  // The key of a row slot.  Rows of 256 bytes are two lines: keys 2t and 2t + 8 of the
  // natural order would share banks.
  __device__ static __forceinline__ int key_of(int slot) {
    if constexpr (kRowBytes == 256)
      return (slot & 8) + ((slot & 1) ? 4 + (((slot & 7) / 2 + 1) & 3) : (slot & 7) / 2);
    else
      return slot;
  }
  // the 8 columns of lane t's part of query entry e (a quarter of a row is D / 32 entries)
  __device__ static __forceinline__ int query_col(int e, int t) {
    if constexpr (kRowBytes == 256) return 64 * (e >> 1) + 8 * ((t & 1) + 4 * (t >> 1) + 2 * (e & 1));
    if constexpr (kHalf && D == 128) return 16 * (2 * t + (e >> 1)) + 8 * (e & 1);
    if constexpr (kHalf) return 16 * t + 8 * e;
    return 8 * (2 * t + e);
  }

  // s: [head / 8][entry][lane] 16 bytes, lane 4 * (head % 8) + t; unit[head]: what a score is multiplied by
  __device__ static __forceinline__ void stage_queries(char* s, float* unit, const void* q, size_t at, int group, int heads) {
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(q) + at * D;
    const int t = threadIdx.x & 3;
    for (int head = threadIdx.x >> 2; head < heads; head += kThreads / 4) {  // a quad per head
      uint4 w[D / 32];
#pragma unroll
      for (int e = 0; e < D / 32; ++e)
        w[e] = head < group ? __ldg(reinterpret_cast<const uint4*>(src + (size_t)head * D + query_col(e, t)))
                            : make_uint4(0, 0, 0, 0);
      if constexpr (kHalf) {
        float f[D / 32][8], m = 0.f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          const uint32_t u[4] = {w[e].x, w[e].y, w[e].z, w[e].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) Unpack<__nv_bfloat16>::word(u[i], &f[e][2 * i]);
#pragma unroll
          for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[e][i]));
        }
        const unsigned quad = 0xfu << (threadIdx.x & 28);
        m = fmaxf(m, __shfl_xor_sync(quad, m, 1));
        m = fmaxf(m, __shfl_xor_sync(quad, m, 2));
        // 2^up m in [2^14, 2^15), below it if m is subnormal; by two factors, since 2^up may
        // be no fp32 number (what the first one rounds ends as zero)
        const int up = m > 0.f && m < INFINITY ? 14 + 127 - (int)(__float_as_uint(m) >> 23) : 0;
        auto power = [](int n) { return __int_as_float((127 + n) << 23); };
        const float up0 = power(up / 2), up1 = power(up - up / 2);
        if (t == 0) unit[head] = power(-(up / 2)) * power(up / 2 - up);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          uint32_t u[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __half2 x = __floats2half2_rn(f[e][2 * i] * up0 * up1, f[e][2 * i + 1] * up0 * up1);
            u[i] = *reinterpret_cast<const uint32_t*>(&x);
          }
          w[e] = make_uint4(u[0], u[1], u[2], u[3]);
        }
      } else if (t == 0) {
        unit[head] = 1.f;
      }
#pragma unroll
      for (int e = 0; e < D / 32; ++e)
        reinterpret_cast<uint4*>(s)[((head >> 3) * (D / 32) + e) * 32 + (head & 7) * 4 + t] = w[e];
    }
  }

  __device__ static __forceinline__ void scores(const char* k, const char* s_q, float (&s)[NT][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
    uint32_t w[2][kRowBytes / 16];  // the lane's quarters of rows g, g + 8
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int key = key_of(g + 8 * r);
#pragma unroll
      for (int j = 0; j < kRowBytes / 64; ++j) {
        int line, p;
        if constexpr (kRowBytes == 256) line = 2 * key + (j >> 1), p = (t & 1) + 4 * (t >> 1) + 2 * (j & 1);
        else if constexpr (kRowBytes == 128) line = key, p = 2 * t + j;
        else line = key >> 1, p = 4 * (key & 1) + t;
        const uint4 u = *reinterpret_cast<const uint4*>(piece(k, line, p));
        w[r][4 * j] = u.x, w[r][4 * j + 1] = u.y, w[r][4 * j + 2] = u.z, w[r][4 * j + 3] = u.w;
      }
    }
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      uint32_t a[2][4];  // the operands of two steps of 16 columns
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if constexpr (kHalf) {
#pragma unroll
          for (int i = 0; i < 2; ++i) e4m3x4_to_half(w[r][2 * e + i], a[r][2 * i], a[r][2 * i + 1]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) a[r][i] = w[r][4 * e + i];
        }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 b = reinterpret_cast<const uint4*>(s_q)[(nt * (D / 32) + e) * 32 + lane];
        mma_16816(kHalf, s[nt], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
        mma_16816(kHalf, s[nt], a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
      }
    }
  }

  __device__ __forceinline__ static uint32_t pack(float x, float y) {
    if constexpr (kHalf) {
      const __half2 h = __floats2half2_rn(x, y);
      return *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
      return *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  __device__ __forceinline__ static float2 unpack(uint32_t w) {
    if constexpr (kHalf) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }

  __device__ static __forceinline__ void output(const char* block, const float (&p)[NT][4], int n_valid,
                                                float (&acc)[NT][D / 64][16]) {
    constexpr int kWords = kRowBytes / 32;  // of a lane's eighth of a row
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint32_t v[4][kWords];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = key_of(2 * t + (i & 1) + 8 * (i >> 1));
      if constexpr (kWords == 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(piece(block, key >> 1, 4 * (key & 1) + (g >> 1)) + 8 * (g & 1));
        v[i][0] = u.x, v[i][1] = u.y;
      } else {
#pragma unroll
        for (int h = 0; h < kWords / 4; ++h) {
          const uint4 u = *reinterpret_cast<const uint4*>(piece(block, key * (kWords / 4) + h, g));
          v[i][4 * h] = u.x, v[i][4 * h + 1] = u.y, v[i][4 * h + 2] = u.z, v[i][4 * h + 3] = u.w;
        }
      }
    }
    if (n_valid < kChunk) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (key_of(2 * t + (i & 1) + 8 * (i >> 1)) >= n_valid)
#pragma unroll
          for (int w = 0; w < kWords; ++w) v[i][w] = 0u;
    }
    uint32_t b[NT][2][2];  // [head tile][high, low part][keys 0-7, 8-15]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t hi = pack(p[nt][2 * r], p[nt][2 * r + 1]);
        const float2 f = unpack(hi);
        b[nt][0][r] = transpose8x8(hi);
        b[nt][1][r] = transpose8x8(pack(p[nt][2 * r] - f.x, p[nt][2 * r + 1] - f.y));
      }
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        // columns col(h, g, 2m) (a0, a2) and the next (a1, a3) of the lane's key pairs
        uint32_t a0, a1, a2, a3;
        if constexpr (kHalf) {
          const int w = 2 * h + (m >> 1);
          e4m3x4_to_half(__byte_perm(v[0][w], v[1][w], (m & 1) ? 0x7362 : 0x5140), a0, a1);
          e4m3x4_to_half(__byte_perm(v[2][w], v[3][w], (m & 1) ? 0x7362 : 0x5140), a2, a3);
        } else {
          a0 = __byte_perm(v[0][4 * h + m], v[1][4 * h + m], 0x5410), a1 = __byte_perm(v[0][4 * h + m], v[1][4 * h + m], 0x7632);
          a2 = __byte_perm(v[2][4 * h + m], v[3][4 * h + m], 0x5410), a3 = __byte_perm(v[2][4 * h + m], v[3][4 * h + m], 0x7632);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_16816(kHalf, &acc[nt][h][4 * m], a0, a1, a2, a3, b[nt][0][0], b[nt][0][1]);
          mma_16816(kHalf, &acc[nt][h][4 * m], a0, a1, a2, a3, b[nt][1][0], b[nt][1][1]);
        }
      }
  }
};

// ONE: a cluster of thread blocks takes one (request, kv head); else the line.
template <typename Tile, int D, int NT, bool ONE>
__global__ void __launch_bounds__(kThreads, Tile::kCtas)
    decode_kernel(const DecodeArgs a, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  using CT = typename Tile::CT;
  constexpr int HT = 8 * NT;                              // heads of one warp
  constexpr int kGroups = NT == 1 ? 1 : kMaxGroup / HT;   // head groups at most
  constexpr int kBlock = kChunk * D * (int)sizeof(CT);    // bytes of K (and of V) of 16 keys
  constexpr int SUB = Tile::kSub, kDepth = Tile::kDepth;
  constexpr int UNIT = kWarps * SUB * kChunk;             // keys of one unit
  // the warps' rings of K and V blocks; between pairs, when nothing is under way, the warps' outputs
  extern __shared__ char s_raw[];
  char* s_ring = s_raw + ((1024u - (sm100::smem_u32(s_raw) & 1023u)) & 1023u);
  constexpr int kRow = D + 4;  // of the outputs: the lanes' 16 bytes fall into different banks
  float(*s_buf)[kRow] = reinterpret_cast<float(*)[kRow]>(s_ring);
  static_assert(kWarps * HT * kRow * 4 <= kWarps * kDepth * SUB * 2 * kBlock, "the outputs fit into the rings");
  __shared__ __align__(16) char s_queries[kGroups * HT * Tile::kQueryBytes];
  __shared__ __align__(8) uint64_t s_full[kWarps][kDepth];
  __shared__ int s_valid[kWarps][kDepth][SUB], s_abort;
  __shared__ float s_unit[kGroups * HT];
  __shared__ float s_m[kWarps][HT], s_l[kWarps][HT];
  __shared__ int s_scan[kWarps], s_base;
  __shared__ int s_r;
  __shared__ float2 s_ml[ONE ? kGroups * HT : 1];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int cta = blockIdx.x;
  if (tid == 0) {
    for (int w = 0; w < kWarps; ++w)
      for (int i = 0; i < kDepth; ++i) sm100::mbar_init(&s_full[w][i], SUB);
    s_abort = 0;
    sm100::fence_barrier_init();
    sm100::prefetch_tensormap(&k_map);
    sm100::prefetch_tensormap(&v_map);
  }
  after_previous();

  int u = 0, u_end = 0, r = 0, base = 0, each = 0, more = 0;
  if constexpr (!ONE) {
    // requests without a key: o = 0, lse = -inf
    for (int r = cta; r < a.R; r += gridDim.x) {
      if (request_units<UNIT>(a, request_len(a, r, tid == 0)) != 0) continue;
      if (a.by_pair)
        for (int h = tid; h < a.Hkv; h += kThreads) a.tail[r * a.Hkv + h] = make_int4(-1, 0, 0, 0);
      const float none[4] = {0.f, 0.f, 0.f, 0.f};
      for (int i = 4 * tid; i < a.Hq * D; i += 4 * kThreads) store_o<4>(a, (size_t)r * a.Hq * D + i, none);
      for (int i = tid; i < a.Hq; i += kThreads) a.lse[(size_t)r * a.Hq + i] = -INFINITY;
    }

    // this block's share of the line
    auto weight = [&](int r) { return pair_weight(request_units<UNIT>(a, request_len(a, r, false))) * a.Hkv; };
    const int per = (a.R + kThreads - 1) / kThreads;
    const int r_lo = min(tid * per, a.R), r_hi = min(r_lo + per, a.R);
    int mine = 0;
    for (int r = r_lo; r < r_hi; ++r) mine += weight(r);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) s_scan[warp] = upto;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) upto += s_scan[w];
      total += s_scan[w];
    }
    // `each` units for every block and one more for the first `more`
    const int n_cta = max(1, min((int)gridDim.x, total));
    each = total / n_cta, more = total - each * n_cta;
    u = each * cta + min(cta, more);
    u_end = cta < n_cta ? u + each + (cta < more ? 1 : 0) : u;
    if (u >= u_end) {
      if (tid == 0 && !a.by_pair) a.tail[cta] = make_int4(-1, 0, 0, 0);
      return;
    }
    if (upto - mine <= u && u < upto) {  // one thread's requests hold the first unit
      int base = upto - mine, r = r_lo;
      for (; r < r_hi - 1; ++r) {
        const int n = weight(r);
        if (u < base + n) break;
        base += n;
      }
      s_r = r;
      s_base = base;
    }
    __syncthreads();
    r = s_r, base = s_base;
  }

  const int hgroups = a.group <= HT ? 1 : (a.group <= 2 * HT ? 2 : 4);  // head groups: warps share keys
  const int kwarps = kWarps / hgroups;
  const int hg = warp % hgroups, kw = warp / hgroups;
  float amax[2] = {0.f, 0.f};  // asked for here, looked at when the first keys are under way
  if constexpr (sizeof(CT) == 1) {
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(amax[0]) : "l"(a.kv_amax));
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(amax[1]) : "l"(a.kv_amax + 1));
  }
  int4 tail = make_int4(-1, 0, 0, 0);
  unsigned issued = 0, done = 0;  // blocks this warp has asked for and used

  const int ranks = ONE ? (int)cg::this_cluster().num_blocks() : 1;
  const int rank = ONE ? (int)cg::this_cluster().block_rank() : 0;
  for (bool once = true; ONE ? once : u < u_end; once = false) {
    int len, n_units, w_pair = 0, h, x0, x1;
    if constexpr (ONE) {
      const int pair = cta / ranks;
      r = pair / a.Hkv, h = pair - r * a.Hkv;
      len = request_len(a, r, tid == 0 && rank == 0);
      n_units = request_units<UNIT>(a, len);
      // A block without units goes on: all of the cluster meet at its barriers.
      x0 = (int)((long long)n_units * rank / ranks), x1 = (int)((long long)n_units * (rank + 1) / ranks);
    } else {
      len = request_len(a, r, false);
      n_units = request_units<UNIT>(a, len), w_pair = pair_weight(n_units);
      if (u >= base + w_pair * a.Hkv) {
        base += w_pair * a.Hkv;
        if (++r >= a.R) break;  // not with lengths that stand still
        continue;
      }
      h = (u - base) / w_pair;
      const int y0 = u - base - h * w_pair;
      const int y1 = min(w_pair, y0 + (u_end - u));
      u += y1 - y0;
      // the pair's own cost stands before its units
      x0 = max(0, y0 - kPairCost), x1 = max(0, y1 - kPairCost);
      if (x0 == x1) continue;
    }
    const int n_list = listed_pages(a, len), held = (int)(((unsigned)len + (1u << a.shift) - 1u) >> a.shift);
    const int32_t* table = a.table + (size_t)r * a.max_pages;
    const int32_t* list = a.pages ? a.pages + ((size_t)r * a.Hkv + h) * a.budget : nullptr;

    // The warps take the pair's blocks of 16 keys in turn, SUB at a time: this warp's
    // i-th turn are blocks (first + i * kwarps) * SUB and the next ones.  Each lane
    // knows where one of the next 32 blocks stands and asks for it when its turn is
    // kDepth away; the pages of the 32 after them are read half way.  Blocks that are
    // not there (behind the end, padding of the list, a page out of range) pass
    // through the ring empty.
    const int first = x0 * kWarps + kw, n_mine = (x1 * kWarps - first + kwarps - 1) / kwarps;
    constexpr int kTurns = 32 / SUB;  // whose blocks the lanes hold
    int line = 0, valid = 0, line_next = 0, valid_next = 0;
    auto look = [&](int turn0) {  // of the turns from turn0 on
      const int i = turn0 + lane / SUB;
      const unsigned at = ((unsigned)(first + i * kwarps) * SUB + lane % SUB) * kChunk;
      const int j = (int)(at >> a.shift), off = (int)(at & ((1u << a.shift) - 1u));
      valid_next = 0;
      if (i < n_mine && j < n_list) {
        const int logical = list ? list[j] : j;
        if ((unsigned)logical < (unsigned)held) {  // neither padding nor behind the end
          const int page = table[logical];
          valid_next = max(0, min(kChunk, len - ((logical << a.shift) + off)));
          if (valid_next > 0 && (unsigned)page >= (unsigned)a.num_pages) {
            atomicOr(a.err, kErrPage);
            valid_next = 0;
          }
          line_next = (int)(((((long long)page * a.Hkv + h) << a.shift) + off) * (D * (int)sizeof(CT)) / 128);
        }
      }
    };
    auto issue = [&](int i) {
      if (i % kTurns == 0) line = line_next, valid = valid_next;
      if (i % kTurns == kTurns / 2 && i / kTurns * kTurns + kTurns < n_mine) look(i / kTurns * kTurns + kTurns);
      if (lane / SUB == i % kTurns) {
        const int slot = (int)(issued % kDepth), sub = lane % SUB;
        char* to = s_ring + ((warp * kDepth + slot) * SUB + sub) * 2 * kBlock;
        s_valid[warp][slot][sub] = valid;
        if (valid > 0 && !s_abort) {
          sm100::mbar_expect_tx(&s_full[warp][slot], 2 * kBlock);
          if (!(a.stall && base + r + h + x0 + warp + i == 0))  // else: failure-detection tests only
            sm100::tma_load_2d(to, &k_map, &s_full[warp][slot], 0, line);
          sm100::tma_load_2d(to + kBlock, &v_map, &s_full[warp][slot], 0, line);
        } else {
          sm100::mbar_arrive(&s_full[warp][slot]);
        }
      }
      ++issued;
    };

    // the previous pair's outputs were written and read where the copies go now
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    look(0);
    for (int i = 0; i < min(kDepth, n_mine); ++i) issue(i);
    Tile::stage_queries(s_queries, s_unit, a.q, (size_t)r * a.Hq + (size_t)h * a.group, a.group,
                        hgroups * HT);
    __syncthreads();

    float m[NT][2], l[NT][2], acc[NT][D / 64][16];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) m[nt][i] = kNothing, l[nt][i] = 0.f;
#pragma unroll
      for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[nt][hh][e] = 0.f;
    }

    const float scale_log2 = sizeof(CT) == 1 ? a.scale_log2 / e4m3_scale(amax[0]) : a.scale_log2;
    const char* s_q = s_queries + hg * HT * Tile::kQueryBytes;
    float unit[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        // never 0: a masked score is -inf, and 0 times that is NaN.  (A product below 2^-149 takes
        // every score of a head, at most 2^31 in half precision, to 0 all the same.)
        unit[nt][i] = fmaxf(scale_log2 * (sizeof(CT) == 1 ? s_unit[hg * HT + nt * 8 + 2 * t + i] : 1.f), 0x1p-149f);

    for (int i = 0; i < n_mine; ++i, ++done) {
      const int slot = (int)(done % kDepth);
      if (!sm100::mbar_wait_warp(&s_full[warp][slot], (uint32_t)(done / kDepth) & 1u, &s_abort, a.err)) break;
      const char* block = s_ring + (warp * kDepth + slot) * SUB * 2 * kBlock;
      int n_valid[SUB], least = kChunk;
#pragma unroll
      for (int sub = 0; sub < SUB; ++sub) {
        n_valid[sub] = s_valid[warp][slot][sub];
        least = min(least, n_valid[sub]);
      }
      float s[SUB][NT][4];
#pragma unroll
      for (int sub = 0; sub < SUB; ++sub) Tile::scores(block + sub * 2 * kBlock, s_q, s[sub]);
      if (least < kChunk) {
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (Tile::key_of(g + 8 * (e >> 1)) >= n_valid[sub]) s[sub][nt][e] = -INFINITY;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // unit > 0: the largest product is the largest score
        float mx[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[e] = fmaxf(s[0][nt][e], s[0][nt][e + 2]);
#pragma unroll
          for (int sub = 1; sub < SUB; ++sub) mx[e] = fmaxf(mx[e], fmaxf(s[sub][nt][e], s[sub][nt][e + 2]));
          mx[e] *= unit[nt][e];
        }
        // The reference of the weights follows the largest score only when that has grown by
        // kSlack; a lane looks at its own keys first.
        if (__any_sync(0xffffffffu, mx[0] > m[nt][0] + (Tile::kLift + Tile::kSlack) ||
                                        mx[1] > m[nt][1] + (Tile::kLift + Tile::kSlack))) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
            const float mn = fmaxf(m[nt][e], mx[e] - Tile::kLift);
            const float alpha = exp2_fast(m[nt][e] - mn);
            m[nt][e] = mn;
            l[nt][e] *= alpha;
#pragma unroll
            for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
              for (int x = 0; x < 8; ++x) acc[nt][hh][2 * x + e] *= alpha;
          }
        }
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[sub][nt][e] = exp2_fast(fmaf(s[sub][nt][e], unit[nt][e & 1], -m[nt][e & 1]));
            l[nt][e & 1] += s[sub][nt][e];
          }
      }
#pragma unroll
      for (int sub = 0; sub < SUB; ++sub)
        Tile::output(block + sub * 2 * kBlock + kBlock, s[sub], n_valid[sub], acc);
      __syncwarp();  // the block is read
      if (i + kDepth < n_mine) issue(i + kDepth);
    }
    // After a wait that ran out nothing new is issued; what is under way is waited for, with the same limit.
    if (s_abort) {
      for (int i = 0; i < kDepth; ++i) {
        const unsigned long long t0 = sm100::globaltimer();
        while (i < issued - done && !sm100::mbar_try_wait(&s_full[warp][(done + i) % kDepth], (uint32_t)((done + i) / kDepth) & 1u) &&
               sm100::globaltimer() - t0 < sm100::kWaitLimitNs) {
        }
      }
      done = issued;
    }

    // the warps' results side by side, then one per head
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], o);
        const int head = nt * 8 + 2 * t + i;
        if (g == 0) s_m[warp][head] = m[nt][i], s_l[warp][head] = l[nt][i];
#pragma unroll
        for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
          for (int e = 0; e < 8; e += 4)
            *reinterpret_cast<float4*>(&s_buf[warp * HT + head][Tile::col(hh, g, e)]) =
                make_float4(acc[nt][hh][2 * e + i], acc[nt][hh][2 * e + 2 + i], acc[nt][hh][2 * e + 4 + i], acc[nt][hh][2 * e + 6 + i]);
      }
    __syncthreads();
    const float v_unit = sizeof(CT) == 1 ? __fdiv_rn(1.f, e4m3_scale(amax[1])) : 1.f;
    const bool whole = x0 == 0 && x1 == n_units;
    const int slot = 2 * cta + (x0 == 0 ? 1 : 0);
    for (int i = tid; i < a.group * (D / 4); i += kThreads) {
      const int head = i / (D / 4), d = i % (D / 4) * 4, hw = head / HT, hh = head % HT;
      float mm = kNothing, ll = 0.f, oo[4] = {0.f, 0.f, 0.f, 0.f};
      for (int w = hw; w < kWarps; w += hgroups) mm = fmaxf(mm, s_m[w][hh]);
      for (int w = hw; w < kWarps; w += hgroups) {
        const float f = exp2_fast(s_m[w][hh] - mm);
        const float4 x = *reinterpret_cast<const float4*>(&s_buf[w * HT + hh][d]);
        ll = fmaf(f, s_l[w][hh], ll);
        oo[0] = fmaf(f, x.x, oo[0]), oo[1] = fmaf(f, x.y, oo[1]), oo[2] = fmaf(f, x.z, oo[2]), oo[3] = fmaf(f, x.w, oo[3]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) oo[e] *= v_unit;
      if (ONE && ranks > 1) {  // in place: no other thread reads these four
        *reinterpret_cast<float4*>(&s_buf[hw * HT + hh][d]) = make_float4(oo[0], oo[1], oo[2], oo[3]);
        if (d == 0) s_ml[head] = make_float2(mm, ll);
      } else if (ONE || whole) {
        finish<4>(a, (size_t)r * a.Hq + (size_t)h * a.group + head, D, d, oo, mm, ll);
      } else {
        const size_t at = (size_t)slot * a.group + head;
        *reinterpret_cast<float4*>(a.part_o + at * D + d) = make_float4(oo[0], oo[1], oo[2], oo[3]);
        if (d == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(mm, ll);
      }
    }
    if (ONE && ranks == 1) break;
    if constexpr (ONE) {
      // every block joins a share of the outputs
      cg::cluster_group cluster = cg::this_cluster();
      __syncwarp();
      cluster.sync();
      const int n = a.group * (D / 4), share = (n + ranks - 1) / ranks;
      for (int i = rank * share + tid; i < min(n, (rank + 1) * share); i += kThreads) {
        const int head = i / (D / 4), d = i % (D / 4) * 4;
        float2* ml = &s_ml[head];
        float4* from = reinterpret_cast<float4*>(&s_buf[head / HT * HT + head % HT][d]);
        float mm = kNothing, ll = 0.f, oo[4] = {0.f, 0.f, 0.f, 0.f};
        float2 p[kMostCluster];  // all asked for at once
        float4 x[kMostCluster];
#pragma unroll
        for (int c = 0; c < kMostCluster; ++c) {
          p[c] = make_float2(kNothing, 0.f), x[c] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c < ranks) p[c] = *cluster.map_shared_rank(ml, c), x[c] = *cluster.map_shared_rank(from, c);
        }
#pragma unroll
        for (int c = 0; c < kMostCluster; ++c) mm = fmaxf(mm, p[c].x);
#pragma unroll
        for (int c = 0; c < kMostCluster; ++c) {
          const float f = exp2_fast(p[c].x - mm);
          ll = fmaf(f, p[c].y, ll);
          oo[0] = fmaf(f, x[c].x, oo[0]), oo[1] = fmaf(f, x[c].y, oo[1]), oo[2] = fmaf(f, x[c].z, oo[2]), oo[3] = fmaf(f, x[c].w, oo[3]);
        }
        finish<4>(a, (size_t)r * a.Hq + (size_t)h * a.group + head, D, d, oo, mm, ll);
      }
      // No block leaves while its results are read.  They have been when a thread arrives, and
      // nothing here is for the others to see: no release, which would wait for the outputs.
      __syncwarp();
      asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
      cluster.barrier_wait();
    } else if (x0 == 0) {
      if (!whole) {  // the block that holds the pair's last unit
        const int last = base + (h + 1) * w_pair - 1, long_ones = more * (each + 1);
        tail = make_int4(r, h, last < long_ones ? last / (each + 1) : more + (last - long_ones) / each, cta);
      }
      if (tid == 0 && a.by_pair) a.tail[r * a.Hkv + h] = whole ? make_int4(-1, 0, 0, 0) : tail;
    }
  }
  if (!ONE && tid == 0 && !a.by_pair) a.tail[cta] = tail;
}

// Combines the partial results of a pair that starts in one block and continues
// in the following ones: M = max m_c, o = sum e^{m_c - M} o_c / sum e^{m_c - M} l_c.
// Block x looks at the x-th note about such a pair, block y at a share of its
// heads; `ways` warps take a head's parts in turn, eight loads at a time.
constexpr int kJoinWarps = 16;  // at most
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const DecodeArgs a, int ways) {
  after_previous();
  const int4 tail = a.tail[blockIdx.x];
  if (tail.x < 0) return;
  __shared__ float s_o[kJoinWarps][D], s_m[kJoinWarps], s_l[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = tail.w, n_parts = tail.z - first + 1;
  constexpr int V = D / 32, kAhead = 8;
  const int head = blockIdx.y * ((blockDim.x >> 5) / ways) + warp / ways, way = warp % ways;
  auto part = [&](int c) { return (size_t)(c == 0 ? 2 * first + 1 : 2 * (first + c)) * a.group + head; };
  float m = kNothing, l = 0.f, o[V] = {};
  if (head < a.group) {
    for (int c0 = way; c0 < n_parts; c0 += ways * kAhead) {
      float pm[kAhead], pl[kAhead], po[kAhead][V];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int c = c0 + i * ways;
        pm[i] = kNothing, pl[i] = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) po[i][e] = 0.f;
        if (c < n_parts) {
          const size_t at = part(c);
          asm volatile("ld.global.v2.f32 {%0,%1}, [%2];" : "=f"(pm[i]), "=f"(pl[i]) : "l"(a.part_ml + at * 2));
          const float* from = a.part_o + at * D + lane * V;
          if constexpr (V == 4)
            asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(po[i][0]), "=f"(po[i][1]), "=f"(po[i][2]), "=f"(po[i][V - 1])
                         : "l"(from));
          else
            asm volatile("ld.global.v2.f32 {%0,%1}, [%2];" : "=f"(po[i][0]), "=f"(po[i][V - 1]) : "l"(from));
        }
      }
      float mn = m;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) mn = fmaxf(mn, pm[i]);
      const float f0 = exp2_fast(m - mn);
      m = mn;
      l *= f0;
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] *= f0;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float f = exp2_fast(pm[i] - mn);
        l = fmaf(f, pl[i], l);
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = fmaf(f, po[i][e], o[e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) s_o[warp][lane * V + e] = o[e];
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
  __syncthreads();
  if (way == 0 && head < a.group) {
    float mm = kNothing, ll = 0.f, oo[V] = {};
    for (int w = 0; w < ways; ++w) mm = fmaxf(mm, s_m[warp + w]);
    for (int w = 0; w < ways; ++w) {
      const float f = exp2_fast(s_m[warp + w] - mm);
      ll = fmaf(f, s_l[warp + w], ll);
#pragma unroll
      for (int e = 0; e < V; ++e) oo[e] = fmaf(f, s_o[warp + w][lane * V + e], oo[e]);
    }
    finish<V>(a, (size_t)tail.x * a.Hq + (size_t)tail.y * a.group + head, D, lane * V, oo, mm, ll);
  }
}

int decode_grid(int ctas, long long max_units) {
  int dev = 0;
  cudaGetDevice(&dev);
  return (int)std::min<long long>((long long)num_sms(dev) * ctas, std::max<long long>(1, max_units));
}

bool sizes_ok(int R, int Hq, int Hkv, int D) {
  if (R < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > kMaxGroup) return false;
  return D == 64 || D == 128;
}

// bytes of the workspace of a grid: partial outputs, (maximum, sum) pairs, tails
size_t ws_part_o(int grid, int group, int D) { return (size_t)2 * grid * group * D * sizeof(float); }
size_t ws_part_ml(int grid, int group) { return ((size_t)2 * grid * group * 2 * sizeof(float) + 15) & ~(size_t)15; }
constexpr int kMostCtas = 3;  // blocks of an SM, over all variants

// Clusters of `cluster` blocks that the current device runs at once, when it is empty.
template <typename Kernel>
int clusters_at_once(Kernel* kernel, int threads, int smem, int cluster) {
  cudaLaunchAttribute attr[1] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess) return n;
  cudaGetLastError();
  return 0;
}

// How a cluster for each pair would run: blocks of a cluster, blocks of an SM, and what it
// costs in quarters of a unit of keys.
struct OneShape {
  int cluster, per_sm, cost;
};
// A block's units cost 5 each, sharing an SM 4 for each block of it, and a cluster of one
// block saves the join: the choice that is best or within 5% of it at 1 to 200 pairs of 64
// to 4096 keys in bf16, e4m3 and fp32 (bf16, us: 16 pairs of 513 keys in clusters of 4, 8,
// 16 blocks 6.4, 6.1, 6.5; 96 pairs of 257 in clusters of 1, 2, 4 6.8, 7.7, 7.4).  `room`
// says how many clusters of 2^i blocks run at once; more blocks of an SM than that takes
// would crowd some SMs (32 clusters of 8: 7.0 us with two blocks of an SM, 7.7 with three).
// At most kOneUnits units a block: requests shorter than the table is wide leave clusters
// idle, which the line levels.
// Clusters | line (us): bf16, 8 heads of 257 keys 5.0 | 6.7, of 1024 5.6 | 7.4, of 4096 8.2 |
// 9.0; 32 requests x 4 heads of 257 keys 6.8 | 10.4, of 512 9.9 | 13.0; e4m3, the same of 1024
// keys 11.6 | 15; fp32, 8 heads of 1024 keys 6.1 | 8.1, of 4096 12.1 | 10.9.
constexpr int kOneUnits = 5, kNoJoin = 8;
template <typename Room>
OneShape one_shape(long long pairs, long long units, Room room) {
  OneShape best = {0, 0, 1 << 30};
  for (int i = 0; (1 << i) <= kMostCluster && (i == 0 || (1 << (i - 1)) < units); ++i) {
    const long long each = (units + (1 << i) - 1) >> i;
    if (each > kOneUnits) continue;
    for (int per_sm = 1; per_sm <= kMostCtas; ++per_sm)
      if (room(per_sm, i) >= pairs) {
        const int cost = (int)(5 * each + 4 * per_sm) - (i == 0 ? kNoJoin : 0);
        if (cost < best.cost) best = {1 << i, per_sm, cost};
        break;
      }
  }
  return best;
}

template <typename Tile, int D, int NT>
int launch_tile(DecodeArgs a, cudaStream_t s, long long max_units, char* ws) {
  static_assert(Tile::kCtas <= kMostCtas, "the workspace is sized for kMostCtas");
  CUtensorMap k_map, v_map;
  constexpr int kBlock = kChunk * D * (int)sizeof(typename Tile::CT), kUnit = kWarps * Tile::kSub * kChunk;
  constexpr int kBytes = kWarps * Tile::kDepth * Tile::kSub * 2 * kBlock + 1024;
  const uint64_t lines = ((uint64_t)a.num_pages * a.Hkv << a.shift) * (kBlock / kChunk) / 128;
  if (!make_tmap_u8_2d(&k_map, a.k, lines, 128, 128, kBlock / 128) || !make_tmap_u8_2d(&v_map, a.v, lines, 128, 128, kBlock / 128))
    return -1;
  cudaError_t e;
  const long long pairs = (long long)a.R * a.Hkv, places = decode_grid(Tile::kCtas, 1LL << 40);
  const long long listed = a.pages ? std::min(a.budget, a.max_pages) : a.max_pages;
  const long long pair_units = ((listed << a.shift) + kUnit - 1) / kUnit;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
  // shared memory that leaves an SM room for 1, 2 or 3 blocks
  constexpr int kOneBytes[kMostCtas] = {120 * 1024, 80 * 1024, kBytes};
  static_assert(kBytes <= 72 * 1024, "three blocks of an SM");
  auto* one = decode_kernel<Tile, D, NT, true>;
  static std::atomic<unsigned long long> one_done{0};
  static std::atomic<int> known[64][kMostCtas][5];  // clusters at once, and one more
  if (pair_units <= kOneUnits * kMostCluster) {
    if (!(one_done.load() & (1ull << dev)) &&
        cudaFuncSetAttribute(one, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
      return -1;
    if (!smem_attr_once(one, kOneBytes[0], one_done)) return -1;
    const OneShape shape = one_shape(pairs, pair_units, [&](int per_sm, int i) {
      std::atomic<int>& k = known[dev][per_sm - 1][i];
      if (k.load() == 0) k.store(1 + clusters_at_once(one, kThreads, kOneBytes[per_sm - 1], 1 << i));
      return k.load() - 1;
    });
    // the line: two launches and a join, kPairCost for each pair, every block the same
    const long long line = pairs * (pair_units + kPairCost), sms = places / Tile::kCtas;
    const long long line_cost = 5 * std::max(line, places) / places + 4 * std::min<long long>(Tile::kCtas, (line + sms - 1) / sms);
    if (shape.cluster && shape.cost < line_cost + Tile::kLineStart) {
      prof_begin(kKDecode, s);
      e = launch_chained(one, dim3((unsigned)(pairs * shape.cluster)), kThreads, kOneBytes[shape.per_sm - 1],
                         shape.cluster, s, a, k_map, v_map);
      prof_end(kKDecode, s);
      return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? 1 : -1;
    }
  }
  static std::atomic<unsigned long long> done{0};
  if (!smem_attr_once(decode_kernel<Tile, D, NT, false>, kBytes, done)) return -1;
  const int grid = decode_grid(Tile::kCtas, max_units);
  a.by_pair = pairs < grid;
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float*>(ws + ws_part_o(grid, a.group, D));
  a.tail = reinterpret_cast<int4*>(ws + ws_part_o(grid, a.group, D) + ws_part_ml(grid, a.group));
  prof_begin(kKDecode, s);
  e = launch_chained(decode_kernel<Tile, D, NT, false>, dim3(grid), kThreads, kBytes, 0, s, a, k_map, v_map);
  prof_end(kKDecode, s);
  if (e != cudaSuccess) return -1;
  // Few pairs can have many parts: a large block for each head.  Else blocks of
  // which most find nothing to do, small and with more heads each.
  const int notes = a.by_pair ? a.R * a.Hkv : grid, sms = decode_grid(1, 1LL << 40);
  const int warps = (long long)notes * a.group <= sms ? kJoinWarps : kJoinWarps / 2;
  int heads = 1;
  while (heads < warps / 2 && (long long)notes * ((a.group + heads - 1) / heads) > 2LL * sms) heads *= 2;
  prof_begin(kKDecodeJoin, s);
  e = launch_chained(join_kernel<D>, dim3(notes, (a.group + heads - 1) / heads), warps * 32, 0, 0, s, a, warps / heads);
  prof_end(kKDecodeJoin, s);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? 2 : -1;
}

template <int D>
int launch_decode(const DecodeArgs& a, int cache_dtype, cudaStream_t s, long long max_units, char* ws) {
  // One tile of 8 heads for a warp, or two: a group of 8 in two tiles takes 54 to 59 us
  // (e4m3) and 63 to 136 (fp32) for 268 MB, and as long in bf16.
  const bool one = a.group <= 8;
  switch (cache_dtype) {
    case CPATTN_BF16:
      return one ? launch_tile<MmaTile<__nv_bfloat16, D, 1>, D, 1>(a, s, max_units, ws)
                 : launch_tile<MmaTile<__nv_bfloat16, D, 2>, D, 2>(a, s, max_units, ws);
    case CPATTN_FP32:
      return one ? launch_tile<FmaTile<D, 1>, D, 1>(a, s, max_units, ws)
                 : launch_tile<FmaTile<D, 2>, D, 2>(a, s, max_units, ws);
    default:
      return one ? launch_tile<MmaTile<E4m3, D, 1>, D, 1>(a, s, max_units, ws)
                 : launch_tile<MmaTile<E4m3, D, 2>, D, 2>(a, s, max_units, ws);
  }
}

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" {

size_t cpattn_decode_workspace_bytes(int R, int Hq, int Hkv, int D) {
  if (!sizes_ok(R, Hq, Hkv, D)) return 0;
  const int grid = decode_grid(kMostCtas, 1LL << 40), group = Hq / Hkv;
  return ws_part_o(grid, group, D) + ws_part_ml(grid, group) + (size_t)grid * sizeof(int4);
}

int cpattn_decode(const void* q, const void* k_cache, const void* v_cache,
                  const int32_t* block_table, const int32_t* lens, const int32_t* pages, void* o,
                  float* lse, int R, int Hq, int Hkv, int D, int page_size, int max_pages,
                  int num_pages, int budget, float scale, const float* kv_amax, void* workspace,
                  size_t ws_bytes, int dtype, int cache_dtype, int o_dtype, void* stream) {
  NvtxRange nv("cpattn_decode");
  if (dtype != CPATTN_BF16 && dtype != CPATTN_FP32) return CPATTN_ERR_DTYPE;
  if (o_dtype != CPATTN_BF16 && o_dtype != CPATTN_FP32) return CPATTN_ERR_DTYPE;
  if (cache_dtype != dtype && !(cache_dtype == CPATTN_E4M3 && dtype == CPATTN_BF16)) return CPATTN_ERR_DTYPE;
  if (!(scale > 0.f) || !isfinite(scale)) return CPATTN_ERR_ARG;
  const int shift = paged::page_shift(page_size);
  if (!sizes_ok(R, Hq, Hkv, D) || shift < 0 || max_pages < 1 || num_pages < 1) return CPATTN_ERR_SHAPE;
  if (((long long)max_pages << shift) > 0x7fffffffLL) return CPATTN_ERR_SHAPE;
  if ((long long)R * Hq * D > (1LL << 40)) return CPATTN_ERR_SHAPE;
  if ((long long)Hq * D > (1LL << 30)) return CPATTN_ERR_SHAPE;  // a block counts a request's outputs in 31 bits
  // the kernel counts the cache's lines of 128 bytes in 31 bits (256 GB)
  const long long row_bytes = (long long)D * (cache_dtype == CPATTN_FP32 ? 4 : cache_dtype == CPATTN_BF16 ? 2 : 1);
  if ((long long)num_pages * Hkv > (1LL << 38) / row_bytes >> shift) return CPATTN_ERR_SHAPE;
  if (pages && budget < 1) return CPATTN_ERR_SHAPE;
  if (!q || !k_cache || !v_cache || !block_table || !lens || !o || !lse) return CPATTN_ERR_ARG;
  if (cache_dtype == CPATTN_E4M3 && !kv_amax) return CPATTN_ERR_ARG;
  if (!paged::aligned_to(q, 16) || !paged::aligned_to(k_cache, 16) || !paged::aligned_to(v_cache, 16) ||
      !paged::aligned_to(o, 16) || !paged::aligned_to(lse, 4) || !paged::aligned_to(block_table, 4) ||
      !paged::aligned_to(lens, 4) || !paged::aligned_to(pages, 4) || !paged::aligned_to(kv_amax, 4))
    return CPATTN_ERR_ALIGN;
  if (!workspace || ws_bytes < cpattn_decode_workspace_bytes(R, Hq, Hkv, D)) return CPATTN_ERR_WORKSPACE;
  if (!paged::aligned_to(workspace, 256)) return CPATTN_ERR_ALIGN;
  unsigned* err = device_error_word();
  if (!err) return CPATTN_ERR_CUDA;

  DecodeArgs a = {};
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  a.table = block_table;
  a.lens = lens;
  a.pages = pages;
  a.o = o;
  a.lse = lse;
  a.kv_amax = kv_amax;
  a.err = err;
  a.R = R;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.group = Hq / Hkv;
  a.shift = shift;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.budget = budget;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.o_bf16 = o_dtype == CPATTN_BF16;
  a.stall = take_stall();
  const long long listed = pages ? std::min(budget, max_pages) : max_pages;
  const long long max_units = (long long)R * Hkv * (((listed << shift) + kWarps * kChunk - 1) / (kWarps * kChunk) + kPairCost);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (max_units > 0x7fffffffLL) return CPATTN_ERR_SHAPE;
  char* ws = static_cast<char*>(workspace);
  const int n = D == 64 ? launch_decode<64>(a, cache_dtype, s, max_units, ws)
                        : launch_decode<128>(a, cache_dtype, s, max_units, ws);
  if (n < 0) return CPATTN_ERR_CUDA;
  add_launches(n);
  return CPATTN_OK;
}

}  // extern "C"
