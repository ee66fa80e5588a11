// decode.cu -- attention of one new token per request over a paged key-value
// cache: for every (request r, query head i) with kv head h = i / group,
//     x_j = scale * q_i . k_j,   o_i = sum_j softmax_j(x) v_j,   lse_i = log sum_j e^{x_j}
// over the request's keys, or over the pages that a list selects.
//
// The keys are cut into units of 64 to 256 (16 KB of keys).  All units of all
// (request, kv head) pairs, with kPairCost more for each pair, form one line,
// which is dealt to the thread blocks in equal contiguous shares: a block finds
// its share from the lengths alone, on the device, so that a batch of very
// different lengths keeps every block equally busy and the host needs no length.  A pair that lies inside one block is
// finished there; the others leave one partial result (running maximum, sum,
// unnormalised output, all fp32) per block, and join_kernel combines them by
// the log-sum-exp rule of cpattn_merge.
#include <algorithm>

#include "cpattn.h"
#include "kernels.h"
#include "paged.cuh"

namespace cpattn {
namespace {

using namespace paged;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 16;   // keys of one tile; never straddles pages
constexpr int kPairCost = 4;  // what starting and finishing a pair costs, in units of keys
constexpr int kMaxGroup = 64;

struct DecodeArgs {
  const void *q, *k, *v;
  const int32_t *table, *lens, *pages;
  void* o;
  float *lse, *part_o, *part_ml;
  int4* tail;
  const float* kv_amax;
  unsigned* err;
  int R, Hq, Hkv, group, shift, max_pages, num_pages, budget;
  float scale_log2;
  int o_bf16;
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

__device__ __forceinline__ void store_o(const DecodeArgs& a, size_t i, float x) {
  if (a.o_bf16)
    static_cast<__nv_bfloat16*>(a.o)[i] = __float2bfloat16_rn(x);
  else
    static_cast<float*>(a.o)[i] = x;
}

// One warp's view of 16 keys.  Lane 4g + t holds, for every 8 heads, the scores
// of keys g and g + 8 with heads 2t and 2t + 1, and of the output 8 columns for
// every 64 (col()) of the same two heads: the accumulator layout of mma.m16n8k16
// with the keys (scores) or the columns (output) as its 16 rows.
//
// FmaTile: fp32 caches, fp32 arithmetic throughout.
template <int D, int NT>
struct FmaTile {
  using CT = float;
  static constexpr int kQueryBytes = D * 4;  // shared memory of one head's query
  static constexpr float kLift = 0.f, kSlack = 8.f;
  static constexpr int kCtas = NT == 1 ? 3 : 2;  // blocks of an SM
  static constexpr int kSub = 1;
  static constexpr int kVecs = D / 16;  // 16-byte loads of a lane's quarter of a row

  float4 k[2][kVecs];
  const float* v_rows;

  __device__ static __forceinline__ int col(int h, int g, int e) { return 64 * h + 8 * g + e; }

  // the queries of `heads` heads from row `at` of q on, for all tiles of this block
  __device__ static __forceinline__ void stage_queries(char* s, float*, const void* q, size_t at, int group, int heads) {
    for (int i = threadIdx.x; i < heads * D; i += kThreads)
      reinterpret_cast<float*>(s)[i] = i / D < group ? static_cast<const float*>(q)[at * D + i] : 0.f;
  }

  __device__ __forceinline__ void load_k(const CT* p) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        k[r][j] = __ldg(reinterpret_cast<const float4*>(p + (g + 8 * r) * D + (j * 4 + t) * 4));
  }
  __device__ __forceinline__ void load_v(const CT* p) { v_rows = p; }

  __device__ __forceinline__ void scores(const char* s_q, float (&s)[NT][4]) const {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float acc[2][8] = {};
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const float4 f = *reinterpret_cast<const float4*>(s_q + (size_t)(nt * 8 + n) * D * 4 + (j * 4 + t) * 16);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            acc[r][n] = fmaf(f.x, k[r][j].x, acc[r][n]);
            acc[r][n] = fmaf(f.y, k[r][j].y, acc[r][n]);
            acc[r][n] = fmaf(f.z, k[r][j].z, acc[r][n]);
            acc[r][n] = fmaf(f.w, k[r][j].w, acc[r][n]);
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
  __device__ __forceinline__ void output(const float (&p)[NT][4], int n_valid, float (&acc)[NT][D / 64][16]) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int kk = 0; kk < kChunk; ++kk) {
      float x[D / 64][8];
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          float4 u = __ldg(reinterpret_cast<const float4*>(v_rows + kk * D + 64 * h + 8 * g + e));
          if (kk >= n_valid) u = make_float4(0.f, 0.f, 0.f, 0.f);
          x[h][e] = u.x, x[h][e + 1] = u.y, x[h][e + 2] = u.z, x[h][e + 3] = u.w;
        }
      const int src_lane = (kk & 7) * 4 + t;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float p0 = __shfl_sync(0xffffffffu, p[nt][(kk >> 3) * 2], src_lane);
        const float p1 = __shfl_sync(0xffffffffu, p[nt][(kk >> 3) * 2 + 1], src_lane);
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

// Loads whose place in the instruction stream is fixed: left to itself the
// compiler sinks a prefetch to its use and waits for each load in turn.
__device__ __forceinline__ void load16(const char* p, uint32_t* w) {
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "l"(p));
}
__device__ __forceinline__ void load8(const char* p, uint32_t* w) {
  asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
}

// MmaTile: bf16 and e4m3 caches on the tensor cores, S^T = K Q^T and O^T = V^T P^T
// with up to 8 heads as the narrow side, so that a group of few heads wastes
// little.  K and V go from global memory straight into the operand registers:
// the contraction index of a product and the row index of O^T may be permuted
// at will, so a lane's 16-byte load of consecutive columns is at once its share
// of one or more operands, and no shared memory, no wait and no barrier stands
// between memory and the tensor cores.  8-bit codes are widened to half
// precision, which holds them exactly; the queries then are in half precision
// too, scaled per head by a power of two so that none of their bits is lost.
// The weights enter as the sum of two 16-bit numbers (2^-17 relative or
// better): the kernel waits for memory, the second product is free, and fp32
// outputs stay good to that.
template <typename C, int D, int NT>
struct MmaTile {
  using CT = C;
  static constexpr bool kHalf = sizeof(C) == 1;
  static constexpr int kQueryBytes = D * 2;
  static constexpr int kCtas = NT == 1 ? 3 : 2;
  static constexpr int kSub = NT == 1 ? 256 / (D * (int)sizeof(C)) : 1;  // 4 KB of keys at a time
  // The largest weight lies between 2^kLift and 2^(kLift + kSlack) times 1: half precision
  // ends at 2^-24, which must be far below the largest weight of a long context.
  static constexpr float kLift = kHalf ? 14.f : 0.f, kSlack = kHalf ? 1.f : 8.f;
  static constexpr int kRowVecs = D * (int)sizeof(C) / 64;  // 16-byte loads of a lane's quarter of a key
  static constexpr int kVWords = D * (int)sizeof(C) / 32;   // words of a lane's eighth of a value row

  uint32_t k[2][kRowVecs * 4];
  uint32_t v[4][kVWords];

  __device__ static __forceinline__ int col(int h, int g, int e) {
    return kHalf ? D / 8 * g + 8 * h + e : 64 * h + 8 * g + e;
  }
  // the 8 columns that lane t's part of query entry e stands for
  __device__ static __forceinline__ int query_col(int e, int t) {
    return kHalf ? 64 * (e >> 1) + 16 * t + 8 * (e & 1) : 32 * e + 8 * t;
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
        // 2^up m in [2^14, 2^15)
        const int up = m > 0.f && m < INFINITY ? 14 - ilogbf(m) : 0;
        if (t == 0) unit[head] = ldexpf(1.f, -up);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          uint32_t u[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __half2 x = __floats2half2_rn(ldexpf(f[e][2 * i], up), ldexpf(f[e][2 * i + 1], up));
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

  __device__ __forceinline__ void load_k(const CT* p) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < kRowVecs; ++j)
        load16(reinterpret_cast<const char*>(p) + (g + 8 * r) * D * (int)sizeof(CT) + j * 64 + t * 16, &k[r][4 * j]);
  }
  __device__ __forceinline__ void load_v(const CT* p) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = 2 * t + (i & 1) + 8 * (i >> 1);
      const char* row = reinterpret_cast<const char*>(p) + key * D * (int)sizeof(CT);
      if constexpr (kVWords == 2) {
        load8(row + g * 8, v[i]);
      } else {
#pragma unroll
        for (int h = 0; h < kVWords / 4; ++h) load16(row + h * 128 + g * 16, &v[i][4 * h]);
      }
    }
  }

  __device__ __forceinline__ void scores(const char* s_q, float (&s)[NT][4]) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      uint32_t a[2][4];  // rows g, g + 8: the operands of two steps of 16 columns
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if constexpr (kHalf) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            a[r][2 * i] = e4m3x2_to_half2((uint16_t)(k[r][2 * e + i] & 0xffffu));
            a[r][2 * i + 1] = e4m3x2_to_half2((uint16_t)(k[r][2 * e + i] >> 16));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) a[r][i] = k[r][4 * e + i];
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

  __device__ __forceinline__ void output(const float (&p)[NT][4], int n_valid, float (&acc)[NT][D / 64][16]) {
    const int t = threadIdx.x & 3;
    if (n_valid < kChunk) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (2 * t + (i & 1) + 8 * (i >> 1) >= n_valid)
#pragma unroll
          for (int w = 0; w < kVWords; ++w) v[i][w] = 0u;
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
        uint32_t w[4];  // columns col(h, g, 2m), + 1 of the lane's four keys
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (kHalf) {
            const uint32_t x = v[i][2 * h + (m >> 1)];
            w[i] = e4m3x2_to_half2((uint16_t)((m & 1) ? x >> 16 : x & 0xffffu));
          } else {
            w[i] = v[i][4 * h + m];
          }
        }
        const uint32_t a0 = __byte_perm(w[0], w[1], 0x5410), a1 = __byte_perm(w[0], w[1], 0x7632);
        const uint32_t a2 = __byte_perm(w[2], w[3], 0x5410), a3 = __byte_perm(w[2], w[3], 0x7632);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_16816(kHalf, &acc[nt][h][4 * m], a0, a1, a2, a3, b[nt][0][0], b[nt][0][1]);
          mma_16816(kHalf, &acc[nt][h][4 * m], a0, a1, a2, a3, b[nt][1][0], b[nt][1][1]);
        }
      }
  }
};

template <typename Tile, int D, int NT>
__global__ void __launch_bounds__(kThreads, Tile::kCtas) decode_kernel(const DecodeArgs a) {
  using CT = typename Tile::CT;
  constexpr int HT = 8 * NT;                           // heads of one warp
  __shared__ __align__(16) float s_buf[kWarps * HT][D];  // the queries; then the warps' outputs
  __shared__ float s_unit[kWarps * HT];
  __shared__ float s_m[kWarps][HT], s_l[kWarps][HT];
  __shared__ long long s_scan[kWarps], s_base;
  __shared__ int s_r;

  constexpr int SUB = Tile::kSub;                // tiles a warp takes at a time
  constexpr int UNIT = kWarps * SUB * kChunk;    // keys of one unit

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int cta = blockIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may take its places

  // requests without a key: o = 0, lse = -inf
  for (int r = cta; r < a.R; r += gridDim.x) {
    if (request_units<UNIT>(a, request_len(a, r, tid == 0)) != 0) continue;
    for (int i = tid; i < a.Hq * D; i += kThreads) store_o(a, (size_t)r * a.Hq * D + i, 0.f);
    for (int i = tid; i < a.Hq; i += kThreads) a.lse[(size_t)r * a.Hq + i] = -INFINITY;
  }

  // this block's share of the line
  auto weight = [&](int r) { return (long long)pair_weight(request_units<UNIT>(a, request_len(a, r, false))) * a.Hkv; };
  const int per = (a.R + kThreads - 1) / kThreads;
  const int r_lo = min(tid * per, a.R), r_hi = min(r_lo + per, a.R);
  long long mine = 0;
  for (int r = r_lo; r < r_hi; ++r) mine += weight(r);
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) s_scan[warp] = upto;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += s_scan[w];
    total += s_scan[w];
  }
  const long long n_cta = min((long long)gridDim.x, total);
  long long u = 0, u_end = 0;
  if (cta < n_cta) u = total * cta / n_cta, u_end = total * (cta + 1) / n_cta;
  if (u >= u_end) {
    if (tid == 0) a.tail[cta] = make_int4(-1, 0, 0, 0);
    return;
  }
  if (upto - mine <= u && u < upto) {  // one thread's requests hold the first unit
    long long base = upto - mine;
    int r = r_lo;
    for (;; ++r) {
      const long long n = weight(r);
      if (u < base + n) break;
      base += n;
    }
    s_r = r;
    s_base = base;
  }
  __syncthreads();
  int r = s_r;
  long long base = s_base;

  const int hgroups = a.group <= HT ? 1 : (a.group <= 2 * HT ? 2 : 4);  // head groups: warps share keys
  const int kwarps = kWarps / hgroups;
  const int hg = warp % hgroups, kw = warp / hgroups;
  const float scale_log2 =
      sizeof(CT) == 1 ? a.scale_log2 / e4m3_scale(a.kv_amax) : a.scale_log2;
  const float v_unit = sizeof(CT) == 1 ? __fdiv_rn(1.f, e4m3_scale(a.kv_amax + 1)) : 1.f;
  int4 tail = make_int4(-1, 0, 0, 0);

  while (u < u_end) {
    const int len = request_len(a, r, false);
    const int n_units = request_units<UNIT>(a, len), w_pair = pair_weight(n_units);
    if (u >= base + (long long)w_pair * a.Hkv) {
      base += (long long)w_pair * a.Hkv;
      ++r;
      continue;
    }
    const int h = (int)((u - base) / w_pair), y0 = (int)((u - base) % w_pair);
    const int y1 = (int)min((long long)w_pair, y0 + (u_end - u));
    u += y1 - y0;
    // the pair's own cost stands before its units
    const int x0 = max(0, y0 - kPairCost), x1 = max(0, y1 - kPairCost);
    if (x0 == x1) continue;
    const int n_list = listed_pages(a, len);
    const int32_t* table = a.table + (size_t)r * a.max_pages;
    const int32_t* list = a.pages ? a.pages + ((size_t)r * a.Hkv + h) * a.budget : nullptr;

    __syncthreads();  // the previous pair's queries and partial outputs are read
    Tile::stage_queries(reinterpret_cast<char*>(s_buf), s_unit, a.q, (size_t)r * a.Hq + (size_t)h * a.group, a.group,
                        hgroups * HT);
    __syncthreads();

    float m[NT][2], l[NT][2], acc[NT][D / 64][16];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) m[nt][i] = -INFINITY, l[nt][i] = 0.f;
#pragma unroll
      for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[nt][hh][e] = 0.f;
    }

    const char* s_q = reinterpret_cast<const char*>(s_buf) + hg * HT * Tile::kQueryBytes;
    float unit[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        unit[nt][i] = scale_log2 * (sizeof(CT) == 1 ? s_unit[hg * HT + nt * 8 + 2 * t + i] : 1.f);

    // Tile c of the pair: its first row in the cache and how many of its 16 keys
    // count; tiles that are not there read row 0 and count none.
    const int c_end = x1 * kWarps * SUB;
    auto locate = [&](int c, int& n_valid) -> size_t {
      n_valid = 0;
      const int j = (int)((unsigned)c * kChunk >> a.shift);
      if (c >= c_end || j >= n_list) return 0;
      const int off = (int)((unsigned)c * kChunk) & ((1 << a.shift) - 1);
      const int logical = list ? list[j] : j;
      const long long pos = ((long long)logical << a.shift) + off;
      if (logical < 0 || pos >= len) return 0;  // padding of the list, or behind the end
      const int page = table[logical];
      if (page < 0 || page >= a.num_pages) {
        if (lane == 0) atomicOr(a.err, kErrPage);
        return 0;
      }
      n_valid = (int)min((long long)kChunk, len - pos);
      return ((((size_t)page * a.Hkv + h) << a.shift) + off) * D;
    };

    // The next tiles' K is on its way while these ones' softmax and output run;
    // where they stand is known one step earlier still.
    Tile tile[SUB];
    const CT* kc = static_cast<const CT*>(a.k);
    const CT* vc = static_cast<const CT*>(a.v);
    const int step = kwarps * SUB;
    int c = x0 * kWarps * SUB + kw * SUB, n_valid[SUB], n_next[SUB];
    size_t row[SUB], row_next[SUB];
#pragma unroll
    for (int i = 0; i < SUB; ++i) row[i] = locate(c + i, n_valid[i]);
#pragma unroll
    for (int i = 0; i < SUB; ++i) row_next[i] = locate(c + step + i, n_next[i]);
    if (c < c_end)
#pragma unroll
      for (int i = 0; i < SUB; ++i) tile[i].load_k(kc + row[i]);
    for (; c < c_end; c += step) {
      float s[SUB][NT][4];
#pragma unroll
      for (int i = 0; i < SUB; ++i) tile[i].load_v(vc + row[i]);
#pragma unroll
      for (int i = 0; i < SUB; ++i) tile[i].scores(s_q, s[i]);
      if (c + step < c_end)
#pragma unroll
        for (int i = 0; i < SUB; ++i) tile[i].load_k(kc + row_next[i]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float& x = s[sub][nt][i];
            x = (g + 8 * (i >> 1)) < n_valid[sub] ? x * unit[nt][i & 1] : -INFINITY;
            mx[i & 1] = fmaxf(mx[i & 1], x);
          }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
        // the reference of the weights follows the maximum only when that has grown by kSlack
        if (__any_sync(0xffffffffu, mx[0] > m[nt][0] + (Tile::kLift + Tile::kSlack) ||
                                        mx[1] > m[nt][1] + (Tile::kLift + Tile::kSlack))) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float mn = fmaxf(m[nt][i], mx[i] - Tile::kLift);
            const float alpha = exp2f(m[nt][i] - (mn == -INFINITY ? 0.f : mn));
            m[nt][i] = mn;
            l[nt][i] *= alpha;
#pragma unroll
            for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
              for (int e = 0; e < 8; ++e) acc[nt][hh][2 * e + i] *= alpha;
          }
        }
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float b = m[nt][i & 1];
            float& x = s[sub][nt][i];
            x = exp2f(x - (b == -INFINITY ? 0.f : b));
            l[nt][i & 1] += x;
          }
      }
#pragma unroll
      for (int i = 0; i < SUB; ++i) tile[i].output(s[i], n_valid[i], acc);
      int n_after[SUB];
      size_t row_after[SUB];
#pragma unroll
      for (int i = 0; i < SUB; ++i) row_after[i] = locate(c + 2 * step + i, n_after[i]);
#pragma unroll
      for (int i = 0; i < SUB; ++i) {
        row[i] = row_next[i], n_valid[i] = n_next[i];
        row_next[i] = row_after[i], n_next[i] = n_after[i];
      }
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
          for (int e = 0; e < 8; ++e) s_buf[warp * HT + head][Tile::col(hh, g, e)] = acc[nt][hh][2 * e + i];
      }
    __syncthreads();
    const bool whole = x0 == 0 && x1 == n_units;
    const int slot = 2 * cta + (x0 == 0 ? 1 : 0);
    for (int i = tid; i < a.group * D; i += kThreads) {
      const int head = i / D, d = i % D, hw = head / HT, hh = head % HT;
      float mm = -INFINITY, ll = 0.f, oo = 0.f;
      for (int w = 0; w < kwarps; ++w) mm = fmaxf(mm, s_m[w * hgroups + hw][hh]);
      const float b = mm == -INFINITY ? 0.f : mm;
      for (int w = 0; w < kwarps; ++w) {
        const float f = exp2f(s_m[w * hgroups + hw][hh] - b);
        ll = fmaf(f, s_l[w * hgroups + hw][hh], ll);
        oo = fmaf(f, s_buf[(w * hgroups + hw) * HT + hh][d], oo);
      }
      oo *= v_unit;
      if (whole) {
        const size_t out = (size_t)r * a.Hq + (size_t)h * a.group + head;
        store_o(a, out * D + d, ll == 0.f ? 0.f : oo / ll);
        if (d == 0) a.lse[out] = ll == 0.f ? -INFINITY : (b + log2f(ll)) * 0.69314718055994531f;
      } else {
        a.part_o[((size_t)slot * a.group + head) * D + d] = oo;
        if (d == 0) {
          a.part_ml[((size_t)slot * a.group + head) * 2] = mm;
          a.part_ml[((size_t)slot * a.group + head) * 2 + 1] = ll;
        }
      }
    }
    if (!whole && x0 == 0) {
      // the block that holds the pair's last unit: the largest c with total * c / n_cta <= last
      const long long last = base + (long long)(h + 1) * w_pair - 1;
      tail = make_int4(r, h, (int)(((last + 1) * n_cta - 1) / total), 0);
    }
  }
  if (tid == 0) a.tail[cta] = tail;
}

// Combines the partial results of the pair that starts in block blockIdx.x and
// continues in the following ones: M = max m_c, o = sum e^{m_c - M} o_c / sum
// e^{m_c - M} l_c.  Four heads for each blockIdx.y, four warps for each head,
// every fourth part for each warp.
constexpr int kJoinHeads = 4, kJoinWays = 4, kJoinWarps = kJoinHeads * kJoinWays;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const DecodeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 tail = a.tail[blockIdx.x];
  if (tail.x < 0) return;
  __shared__ float s_o[kJoinWarps][D], s_m[kJoinWarps], s_l[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = blockIdx.x, n_parts = tail.z - first + 1;
  constexpr int V = D / 32;
  const int head = blockIdx.y * kJoinHeads + warp / kJoinWays, way = warp % kJoinWays;
  auto part = [&](int c) { return (size_t)(c == 0 ? 2 * first + 1 : 2 * (first + c)) * a.group + head; };
  float m = -INFINITY, l = 0.f, o[V] = {};
  if (head < a.group) {
    for (int c = way + kJoinWays * lane; c < n_parts; c += kJoinWays * 32) m = fmaxf(m, a.part_ml[part(c) * 2]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    const float b = m == -INFINITY ? 0.f : m;
#pragma unroll 4
    for (int c = way; c < n_parts; c += kJoinWays) {
      const size_t at = part(c);
      const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + at * 2);
      const float f = exp2f(ml.x - b);
      l = fmaf(f, ml.y, l);
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = fmaf(f, a.part_o[at * D + e * 32 + lane], o[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) s_o[warp][e * 32 + lane] = o[e];
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
  __syncthreads();
  if (way == 0 && head < a.group) {
    float mm = -INFINITY, ll = 0.f, oo[V] = {};
#pragma unroll
    for (int w = 0; w < kJoinWays; ++w) mm = fmaxf(mm, s_m[warp + w]);
    const float b = mm == -INFINITY ? 0.f : mm;
#pragma unroll
    for (int w = 0; w < kJoinWays; ++w) {
      const float f = exp2f(s_m[warp + w] - b);
      ll = fmaf(f, s_l[warp + w], ll);
#pragma unroll
      for (int e = 0; e < V; ++e) oo[e] = fmaf(f, s_o[warp + w][e * 32 + lane], oo[e]);
    }
    const size_t out = (size_t)tail.x * a.Hq + (size_t)tail.y * a.group + head;
#pragma unroll
    for (int e = 0; e < V; ++e) store_o(a, out * D + e * 32 + lane, ll == 0.f ? 0.f : oo[e] / ll);
    if (lane == 0) a.lse[out] = ll == 0.f ? -INFINITY : (b + log2f(ll)) * 0.69314718055994531f;
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
constexpr int kMostCtas = 4;  // blocks of an SM, over all variants

template <typename Tile, int D, int NT>
int launch_tile(DecodeArgs a, cudaStream_t s, long long max_units, char* ws) {
  static_assert(Tile::kCtas <= kMostCtas, "the workspace is sized for kMostCtas");
  const int grid = decode_grid(Tile::kCtas, max_units);
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float*>(ws + ws_part_o(grid, a.group, D));
  a.tail = reinterpret_cast<int4*>(ws + ws_part_o(grid, a.group, D) + ws_part_ml(grid, a.group));
  prof_begin(kKDecode, s);
  decode_kernel<Tile, D, NT><<<grid, kThreads, 0, s>>>(a);
  prof_end(kKDecode, s);
  if (cudaGetLastError() != cudaSuccess) return -1;
  // the join starts while the last blocks finish and waits for them on the device
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, (a.group + kJoinHeads - 1) / kJoinHeads);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  prof_begin(kKDecodeJoin, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, join_kernel<D>, a);
  prof_end(kKDecodeJoin, s);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? 2 : -1;
}

template <int D>
int launch_decode(const DecodeArgs& a, int cache_dtype, cudaStream_t s, long long max_units, char* ws) {
  const bool one = a.group <= 8;  // head tiles of a warp
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
  const long long listed = pages ? std::min(budget, max_pages) : max_pages;
  const long long max_units = (long long)R * Hkv * (((listed << shift) + kWarps * kChunk - 1) / (kWarps * kChunk) + kPairCost);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  const int n = D == 64 ? launch_decode<64>(a, cache_dtype, s, max_units, ws)
                        : launch_decode<128>(a, cache_dtype, s, max_units, ws);
  if (n < 0) return CPATTN_ERR_CUDA;
  add_launches(n);
  return CPATTN_OK;
}

}  // extern "C"
