// ops.cuh -- what the operators beside the products share (norm.cu, rope.cu,
// lora.cu, attend.cu): element types, 16-byte groups of them in f32, launches
// and the device status word they set.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace q1 {

// Status bit of an index on the device (a page, an adapter, a position) that
// lies outside what the call was given: the kernel skips it and sets this.
constexpr unsigned kStatusBadIndex = 2u;

// The device status word of these kernels on the current device (ops.cu).
int ops_status_ptr(unsigned** p);
int status_word_ops(unsigned* v, int clear);

template <class T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kGroup = 4;  // values in 16 bytes
  static __device__ __forceinline__ float to(float v) { return v; }
  static __device__ __forceinline__ float from(float v) { return v; }
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[4]) {
    v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kGroup = 8;
  static __device__ __forceinline__ float to(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b) {
    a = __uint_as_float(w << 16);  // bf16 is the upper half of an f32
    b = __uint_as_float(w & 0xffff0000u);
  }
  // two values rounded to nearest even, `a` in the low half
  static __device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[8]) {
    unpack2(r.x, v[0], v[1]), unpack2(r.y, v[2], v[3]), unpack2(r.z, v[4], v[5]), unpack2(r.w, v[6], v[7]);
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
  }
};
template <>
struct Elem<__half> {
  static constexpr int kGroup = 8;
  static __device__ __forceinline__ float to(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    a = f.x, b = f.y;
  }
  static __device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[8]) {
    unpack2(r.x, v[0], v[1]), unpack2(r.y, v[2], v[3]), unpack2(r.z, v[4], v[5]), unpack2(r.w, v[6], v[7]);
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
  }
};

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
inline bool aligned4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

// A launch with programmatic dependent launch (the kernel starts while its
// predecessor on the stream drains; every thread of it calls pdl_wait before
// it touches memory) and, where `cluster` > 1, in clusters of that many CTAs.
template <typename Args>
int launch_op(void (*kernel)(Args), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s,
              const char* who, const Args& args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, args), who);
}

}  // namespace q1
