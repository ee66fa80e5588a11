// paged.cuh -- what the paged key-value cache's translation units share: the
// cache element types, the error bit of a page outside of the pool and small
// conversions.
//
// Layout of a cache: [num_pages][Hkv][page_size][D], K and V apart, so that the
// rows of one (page, kv head) are one contiguous block.  page_size is a power
// of two from 16 to 256: 16 consecutive keys never straddle two pages.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <utility>

namespace cpattn {
namespace paged {

// bit of the device error word: a page number, slot or length out of range
constexpr unsigned kErrPage = 4u;

// An element of an 8-bit cache: the e4m3 code of x * s, s = 448 * (1 / max|x|).
struct E4m3 {
  uint8_t code;
};

// log2 of a page size, or -1 for one that is not supported
inline int page_shift(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == (1 << s)) return s;
  return -1;
}

inline bool aligned_to(const void* p, unsigned n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// One token's step is a chain of short kernels.  Each is launched so that it may
// take its places while the kernel before it finishes, reads and writes nothing
// before after_previous(), and only then lets the next one in.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, unsigned cluster,
                           cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

// 448 * (1 / amax), both steps rounded to fp32: what 448.0 / amax gives for a
// tensor in PyTorch, so that codes a program writes with torch and codes written
// here agree bit for bit.  (The one-step quotient of cpattn_quantize_e4m3 can
// differ in the last bit.)
__device__ __forceinline__ float e4m3_scale(float amax) {
  return amax > 0.f ? __fmul_rn(__fdiv_rn(1.f, amax), 448.f) : 1.f;
}

// four e4m3 codes (low byte first) as two pairs in half precision, which holds every code exactly
__device__ __forceinline__ void e4m3x4_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ uint16_t float2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// the elements of a 32-bit word as floats
template <typename CT>
struct Unpack;
template <>
struct Unpack<float> {
  static constexpr int kPerWord = 1;
  __device__ static __forceinline__ void word(uint32_t w, float* f) { f[0] = __uint_as_float(w); }
};
template <>
struct Unpack<__nv_bfloat16> {
  static constexpr int kPerWord = 2;
  __device__ static __forceinline__ void word(uint32_t w, float* f) {
    f[0] = __uint_as_float(w << 16);
    f[1] = __uint_as_float(w & 0xffff0000u);
  }
};
template <>
struct Unpack<E4m3> {
  static constexpr int kPerWord = 4;
  __device__ static __forceinline__ void word(uint32_t w, float* f) {
    uint32_t a, b;
    e4m3x4_to_half(w, a, b);
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
    f[0] = x.x;
    f[1] = x.y;
    f[2] = y.x;
    f[3] = y.y;
  }
};

}  // namespace paged
}  // namespace cpattn
