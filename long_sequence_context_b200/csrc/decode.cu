// decode.cu -- attention of one new token per request over a paged key-value
// cache: for every (request r, query head i) with kv head h = i / group,
//     x_j = scale * q_i . k_j,   o_i = sum_j softmax_j(x) v_j,   lse_i = log sum_j e^{x_j}
// over the request's keys, or over the pages that a list selects.
//
// The keys are cut into units of 64.  All units of all (request, kv head)
// pairs form one line, which is dealt to the thread blocks in equal
// contiguous shares: a block finds its share from the lengths alone, on the
// device, so that a batch of very different lengths keeps every block equally
// busy and the host needs no length.  A pair that lies inside one block is
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
constexpr int kUnit = 64;   // keys of one unit: four chunks of 16
constexpr int kChunk = 16;  // keys a warp takes at a time; never straddles pages
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
  int o_bf16, q_bf16;
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
__device__ __forceinline__ int request_units(const DecodeArgs& a, int len) {
  const long long keys = a.pages ? (long long)listed_pages(a, len) << a.shift : len;
  return (int)((keys + kUnit - 1) / kUnit);
}

__device__ __forceinline__ void store_o(const DecodeArgs& a, size_t i, float x) {
  if (a.o_bf16)
    static_cast<__nv_bfloat16*>(a.o)[i] = __float2bfloat16_rn(x);
  else
    static_cast<float*>(a.o)[i] = x;
}

// One warp's view of 16 keys, in fp32 arithmetic.  Lane 4g + t holds, for
// every 8 heads, the scores of keys g and g + 8 with heads 2t and 2t + 1, and
// of the output the 8 columns 64h + 8g .. + 7 of the same two heads.
template <typename CT, int D, int NT>
struct FmaTile {
  static constexpr int kEpv = 16 / sizeof(CT);      // elements of a 16-byte load
  static constexpr int kVecs = D / (4 * kEpv);      // loads of a lane's quarter of a row
  static constexpr int kWpv = 8 * sizeof(CT) / 4;   // words of 8 elements

  // qs: the heads of this warp, [8 * NT][D] fp32
  __device__ static __forceinline__ void scores(const CT* k, const float* qs, float (&s)[NT][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint4 w[2][kVecs];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        w[r][j] = __ldg(reinterpret_cast<const uint4*>(k + (g + 8 * r) * D + (j * 4 + t) * kEpv));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float acc[2][8] = {};
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        float x[2][kEpv];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          constexpr int P = Unpack<CT>::kPerWord;
          Unpack<CT>::word(w[r][j].x, x[r]);
          Unpack<CT>::word(w[r][j].y, x[r] + P);
          Unpack<CT>::word(w[r][j].z, x[r] + 2 * P);
          Unpack<CT>::word(w[r][j].w, x[r] + 3 * P);
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const float* q = qs + (nt * 8 + n) * D + (j * 4 + t) * kEpv;
#pragma unroll
          for (int e = 0; e < kEpv; e += 4) {
            const float4 f = *reinterpret_cast<const float4*>(q + e);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              acc[r][n] = fmaf(f.x, x[r][e], acc[r][n]);
              acc[r][n] = fmaf(f.y, x[r][e + 1], acc[r][n]);
              acc[r][n] = fmaf(f.z, x[r][e + 2], acc[r][n]);
              acc[r][n] = fmaf(f.w, x[r][e + 3], acc[r][n]);
            }
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
  __device__ static __forceinline__ void output(const CT* v, const float (&p)[NT][4], int n_valid,
                                                float (&acc)[NT][D / 64][16]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int kk = 0; kk < kChunk; ++kk) {
      float x[D / 64][8];
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(v + kk * D + 64 * h + 8 * g);
        uint32_t w[kWpv];
        if constexpr (kWpv == 2) {
          const uint2 u = __ldg(reinterpret_cast<const uint2*>(src));
          w[0] = u.x, w[1] = u.y;
        } else {
#pragma unroll
          for (int i = 0; i < kWpv; i += 4) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(src + i));
            w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
          }
        }
#pragma unroll
        for (int i = 0; i < kWpv; ++i) Unpack<CT>::word(w[i], x[h] + i * Unpack<CT>::kPerWord);
        if (kk >= n_valid)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[h][e] = 0.f;
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

template <typename CT, int D, int NT>
__global__ void __launch_bounds__(kThreads) decode_kernel(const DecodeArgs a) {
  constexpr int HT = 8 * NT;  // heads of one warp
  __shared__ float s_buf[kWarps * HT][D];  // the queries; then the warps' outputs
  __shared__ float s_m[kWarps][HT], s_l[kWarps][HT];
  __shared__ long long s_scan[kWarps], s_base;
  __shared__ int s_r;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int cta = blockIdx.x;

  // requests without a key: o = 0, lse = -inf
  for (int r = cta; r < a.R; r += gridDim.x) {
    if (request_units(a, request_len(a, r, tid == 0)) != 0) continue;
    for (int i = tid; i < a.Hq * D; i += kThreads) store_o(a, (size_t)r * a.Hq * D + i, 0.f);
    for (int i = tid; i < a.Hq; i += kThreads) a.lse[(size_t)r * a.Hq + i] = -INFINITY;
  }

  // this block's share of the line of units
  const int per = (a.R + kThreads - 1) / kThreads;
  const int r_lo = min(tid * per, a.R), r_hi = min(r_lo + per, a.R);
  long long mine = 0;
  for (int r = r_lo; r < r_hi; ++r) mine += (long long)request_units(a, request_len(a, r, false)) * a.Hkv;
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
      const long long n = (long long)request_units(a, request_len(a, r, false)) * a.Hkv;
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
    const int n_units = request_units(a, len);
    if (n_units == 0 || u >= base + (long long)n_units * a.Hkv) {
      base += (long long)n_units * a.Hkv;
      ++r;
      continue;
    }
    const int h = (int)((u - base) / n_units), x0 = (int)((u - base) % n_units);
    const int x1 = (int)min((long long)n_units, x0 + (u_end - u));
    const int n_list = listed_pages(a, len);
    const int32_t* table = a.table + (size_t)r * a.max_pages;
    const int32_t* list = a.pages ? a.pages + ((size_t)r * a.Hkv + h) * a.budget : nullptr;

    __syncthreads();  // the previous pair's queries and partial outputs are read
    for (int i = tid; i < hgroups * HT * D; i += kThreads) {
      const int head = i / D;
      float x = 0.f;
      if (head < a.group) {
        const size_t at = ((size_t)r * a.Hq + (size_t)h * a.group + head) * D + i % D;
        x = a.q_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at])
                     : static_cast<const float*>(a.q)[at];
      }
      s_buf[head][i % D] = x;
    }
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

    for (int c = x0 * 4 + kw; c < x1 * 4; c += kwarps) {
      const int j = (int)(((long long)c * kChunk) >> a.shift);
      if (j >= n_list) break;
      const int off = (c * kChunk) & ((1 << a.shift) - 1);
      const int logical = list ? list[j] : j;
      const long long pos = ((long long)logical << a.shift) + off;  // of the chunk's first key
      if (logical < 0 || pos >= len) continue;                        // padding of the list, or the end
      const int page = table[logical];
      if (page < 0 || page >= a.num_pages) {
        if (lane == 0) atomicOr(a.err, kErrPage);
        continue;
      }
      const int n_valid = (int)min((long long)kChunk, len - pos);
      const size_t row = ((((size_t)page * a.Hkv + h) << a.shift) + off) * D;
      const CT* k = static_cast<const CT*>(a.k) + row;
      const CT* v = static_cast<const CT*>(a.v) + row;

      float s[NT][4];
      FmaTile<CT, D, NT>::scores(k, s_buf[hg * HT], s);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = (g + 8 * (i >> 1)) < n_valid ? s[nt][i] * scale_log2 : -INFINITY;
        float base2[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float mx = fmaxf(s[nt][i], s[nt][i + 2]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          mx = fmaxf(mx, m[nt][i]);
          base2[i] = mx == -INFINITY ? 0.f : mx;
          const float alpha = exp2f(m[nt][i] - base2[i]);
          m[nt][i] = mx;
          l[nt][i] *= alpha;
#pragma unroll
          for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[nt][hh][2 * e + i] *= alpha;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[nt][i] = exp2f(s[nt][i] - base2[i & 1]);
          l[nt][i & 1] += s[nt][i];
        }
      }
      FmaTile<CT, D, NT>::output(v, s, n_valid, acc);
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
          for (int e = 0; e < 8; ++e) s_buf[warp * HT + head][64 * hh + 8 * g + e] = acc[nt][hh][2 * e + i];
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
      const long long last = base + (long long)(h + 1) * n_units - 1;
      tail = make_int4(r, h, (int)(((last + 1) * n_cta - 1) / total), 0);
    }
    u += x1 - x0;
  }
  if (tid == 0) a.tail[cta] = tail;
}

// Combines the partial results of the pair that starts in block blockIdx.x and
// continues in the following ones: M = max m_c, o = sum e^{m_c - M} o_c / sum
// e^{m_c - M} l_c.  A warp takes every kJoinWarps / heads-th part of a head.
constexpr int kJoinWarps = 16;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const DecodeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 tail = a.tail[blockIdx.x];
  if (tail.x < 0) return;
  __shared__ float s_o[kJoinWarps][D], s_m[kJoinWarps], s_l[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = blockIdx.x, n_parts = tail.z - first + 1;
  constexpr int V = D / 32;
  int ways = 1;  // warps that share a head
  while (ways * 2 * a.group <= kJoinWarps) ways *= 2;
  const int at_once = kJoinWarps / ways;
  for (int h0 = 0; h0 < a.group; h0 += at_once) {
    const int head = h0 + warp / ways, way = warp % ways;
    float m = -INFINITY, l = 0.f, o[V] = {};
    if (head < a.group) {
      for (int c = way; c < n_parts; c += ways) {
        const size_t slot = c == 0 ? 2 * first + 1 : 2 * (first + c);
        const size_t at = slot * a.group + head;
        const float mc = a.part_ml[at * 2], lc = a.part_ml[at * 2 + 1];
        const float mn = fmaxf(m, mc), b = mn == -INFINITY ? 0.f : mn;
        const float f0 = exp2f(m - b), f1 = exp2f(mc - b);
        m = mn;
        l = l * f0 + lc * f1;
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = o[e] * f0 + a.part_o[at * D + e * 32 + lane] * f1;
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) s_o[warp][e * 32 + lane] = o[e];
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
    __syncthreads();
    if (way == 0 && head < a.group) {
      float mm = -INFINITY, ll = 0.f, oo[V] = {};
      for (int w = 0; w < ways; ++w) mm = fmaxf(mm, s_m[warp + w]);
      const float b = mm == -INFINITY ? 0.f : mm;
      for (int w = 0; w < ways; ++w) {
        const float f = exp2f(s_m[warp + w] - b);
        ll += f * s_l[warp + w];
#pragma unroll
        for (int e = 0; e < V; ++e) oo[e] += f * s_o[warp + w][e * 32 + lane];
      }
      const size_t out = (size_t)tail.x * a.Hq + (size_t)tail.y * a.group + head;
#pragma unroll
      for (int e = 0; e < V; ++e) store_o(a, out * D + e * 32 + lane, ll == 0.f ? 0.f : oo[e] / ll);
      if (lane == 0) a.lse[out] = ll == 0.f ? -INFINITY : (b + log2f(ll)) * 0.69314718055994531f;
    }
  }
}

constexpr int kCtasPerSm = 3;

int decode_grid(long long max_units) {
  int dev = 0;
  cudaGetDevice(&dev);
  return (int)std::min<long long>((long long)num_sms(dev) * kCtasPerSm, std::max<long long>(1, max_units));
}

template <typename CT, int D>
void launch_nt(const DecodeArgs& a, int grid, cudaStream_t s) {
  if (a.group <= 8)
    decode_kernel<CT, D, 1><<<grid, kThreads, 0, s>>>(a);
  else
    decode_kernel<CT, D, 2><<<grid, kThreads, 0, s>>>(a);
}

template <typename CT>
int launch_decode(const DecodeArgs& a, int D, int grid, cudaStream_t s) {
  prof_begin(kKDecode, s);
  if (D == 64)
    launch_nt<CT, 64>(a, grid, s);
  else
    launch_nt<CT, 128>(a, grid, s);
  prof_end(kKDecode, s);
  if (cudaGetLastError() != cudaSuccess) return -1;
  // the join starts while the last blocks finish and waits for them on the device
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  prof_begin(kKDecodeJoin, s);
  const cudaError_t e = D == 64 ? cudaLaunchKernelEx(&cfg, join_kernel<64>, a) : cudaLaunchKernelEx(&cfg, join_kernel<128>, a);
  prof_end(kKDecodeJoin, s);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? 2 : -1;
}

bool sizes_ok(int R, int Hq, int Hkv, int D) {
  if (R < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > kMaxGroup) return false;
  return D == 64 || D == 128;
}

// bytes of the workspace of a grid: partial outputs, (maximum, sum) pairs, tails
size_t ws_part_o(int grid, int group, int D) { return (size_t)2 * grid * group * D * sizeof(float); }
size_t ws_part_ml(int grid, int group) { return ((size_t)2 * grid * group * 2 * sizeof(float) + 15) & ~(size_t)15; }

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" {

size_t cpattn_decode_workspace_bytes(int R, int Hq, int Hkv, int D) {
  if (!sizes_ok(R, Hq, Hkv, D)) return 0;
  const int grid = decode_grid(1LL << 40), group = Hq / Hkv;
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
  a.q_bf16 = dtype == CPATTN_BF16;
  const long long listed = pages ? std::min(budget, max_pages) : max_pages;
  const int grid = decode_grid((long long)R * Hkv * (((listed << shift) + kUnit - 1) / kUnit));
  char* ws = static_cast<char*>(workspace);
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float*>(ws + ws_part_o(grid, a.group, D));
  a.tail = reinterpret_cast<int4*>(ws + ws_part_o(grid, a.group, D) + ws_part_ml(grid, a.group));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int n = -1;
  if (cache_dtype == CPATTN_BF16) n = launch_decode<__nv_bfloat16>(a, D, grid, s);
  else if (cache_dtype == CPATTN_FP32) n = launch_decode<float>(a, D, grid, s);
  else n = launch_decode<paged::E4m3>(a, D, grid, s);
  if (n < 0) return CPATTN_ERR_CUDA;
  add_launches(n);
  return CPATTN_OK;
}

}  // extern "C"
