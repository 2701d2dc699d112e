// norm.cu -- q8_add_rms_norm: h = x + r, y = h / sqrt(mean(h^2) + eps) * w, and
// the q8_0 form of y, in one pass over a row.
//
// A value costs about ten operations and 13 bytes (f32 in and out, one byte of
// quant), so bytes bound it: each thread keeps its part of the row in
// registers between the sum of squares and the scaling, and a row is read
// once.  One CTA takes one row.  The lanes of a warp hold consecutive 16-byte
// groups, so a q8_0 block of 32 values is 8 (f32) or 4 (16-bit) neighbouring
// lanes and its maximum costs 3 or 2 shuffles, as in quant.cu.
//
// Measured: 8191 rows of 4128 f32 values with residual, 442 MB, in 66.7 us: 6.6 TB/s,
// 0.99 of the copy bandwidth of the card (6.69 TB/s).  One row of 4096 takes 2.6 us a
// launch in a chain of them, 64 bf16 rows 2.4 us: the launch and one round of
// loads, not bytes.
//
// The order of every sum depends on n and the type alone (which thread holds
// which group, the warp's butterfly, then the warps in order), never on the
// number of rows: a row's outputs are the same bits in any batch.
#include "ops.cuh"

namespace q1 {

struct NormArgs {
  const void* x;
  const void* res;      // or null
  const float* w;
  void* res_out;        // or null
  void* y;              // or null
  int8_t* q;            // or null
  uint16_t* d;
  int64_t ldx, ldr, ldo, ldy;
  int n;
  float eps;
};

// Group g (kGroup values from element g*kGroup on) of a row; past n: zeros.
template <class T, bool VEC>
__device__ __forceinline__ void load_group(const T* row, int g, int n, float (&v)[Elem<T>::kGroup]) {
  constexpr int G = Elem<T>::kGroup;
  const int e = g * G;
  if constexpr (VEC) {
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    if (e < n) r = *reinterpret_cast<const uint4*>(row + e);
    Elem<T>::unpack(r, v);
  } else {
#pragma unroll
    for (int i = 0; i < G; ++i) v[i] = e + i < n ? Elem<T>::to(row[e + i]) : 0.f;
  }
}

template <class T, bool VEC>
__device__ __forceinline__ void store_group(T* row, int g, int n, const float (&v)[Elem<T>::kGroup]) {
  constexpr int G = Elem<T>::kGroup;
  const int e = g * G;
  if constexpr (VEC) {
    if (e < n) *reinterpret_cast<uint4*>(row + e) = Elem<T>::pack(v);
  } else {
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (e + i < n) row[e + i] = Elem<T>::from(v[i]);
  }
}

template <class T, bool VEC>
__device__ __forceinline__ void load_sum(const NormArgs& a, const T* x, const T* r, int g,
                                         float (&h)[Elem<T>::kGroup]) {
  load_group<T, VEC>(x, g, a.n, h);
  if (r) {
    float t[Elem<T>::kGroup];
    load_group<T, VEC>(r, g, a.n, t);
#pragma unroll
    for (int i = 0; i < Elem<T>::kGroup; ++i) h[i] = __fadd_rn(h[i], t[i]);
  }
}

// What follows the row's scale rs for one group: y, and its q8_0 form.  All
// lanes of the warp call it (groups past n hold zeros).
template <class T, bool VEC>
__device__ __forceinline__ void finish_group(const NormArgs& a, int64_t row, int g, float rs,
                                             const float (&h)[Elem<T>::kGroup],
                                             const float (&w)[Elem<T>::kGroup]) {
  constexpr int G = Elem<T>::kGroup;
  float y[G];
#pragma unroll
  for (int i = 0; i < G; ++i) y[i] = __fmul_rn(__fmul_rn(h[i], rs), w[i]);
  if (a.y) store_group<T, VEC>(static_cast<T*>(a.y) + row * a.ldy, g, a.n, y);
  if (a.q) {
    float amax = fabsf(y[0]);  // (not 0: the scale of values that are all NaN is NaN, as in quant.cu)
#pragma unroll
    for (int i = 1; i < G; ++i) amax = fmaxf(amax, fabsf(y[i]));
#pragma unroll
    for (int off = kSub / G / 2; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    if (g * G >= a.n) return;
    const float dd = __fdiv_rn(amax, 127.0f);
    const float id = dd != 0.0f ? __fdiv_rn(1.0f, dd) : 0.0f;
    uint32_t code[G / 4];
#pragma unroll
    for (int i = 0; i < G; i += 4) {
      uint32_t c = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        c |= uint32_t(uint8_t(static_cast<int8_t>(static_cast<int>(roundf(__fmul_rn(y[i + j], id)))))) << (8 * j);
      code[i / 4] = c;
    }
    int8_t* q = a.q + row * a.n + g * G;
    if constexpr (G == 4)
      *reinterpret_cast<uint32_t*>(q) = code[0];
    else
      *reinterpret_cast<uint2*>(q) = make_uint2(code[0], code[1]);
    if ((g * G) % kSub == 0) a.d[row * (a.n / kSub) + g * G / kSub] = __half_as_ushort(__float2half_rn(dd));
  }
}

template <class T, bool VEC>
__device__ __forceinline__ void load_weight(const NormArgs& a, int g, float (&w)[Elem<T>::kGroup]) {
  constexpr int G = Elem<T>::kGroup;
#pragma unroll
  for (int i = 0; i < G; i += 4) {
    if constexpr (VEC) {
      const float4 v = g * G < a.n ? *reinterpret_cast<const float4*>(a.w + g * G + i) : make_float4(0.f, 0.f, 0.f, 0.f);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    } else {
#pragma unroll
      for (int j = i; j < i + 4; ++j) w[j] = g * G + j < a.n ? a.w[g * G + j] : 0.f;
    }
  }
}

// The row's 1 / sqrt(mean + eps) from every thread's sum of squares.
__device__ __forceinline__ float row_scale(const NormArgs& a, float s) {
  __shared__ float part[32];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.f;
  for (unsigned i = 0; i < blockDim.x / 32; ++i) s = __fadd_rn(s, part[i]);
  return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(s, float(a.n)), a.eps)));
}

// K groups a thread, held in registers.
template <class T, int K>
__global__ void __launch_bounds__(1024) k_add_rms_norm(NormArgs a) {
  constexpr int G = Elem<T>::kGroup;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* r = a.res ? static_cast<const T*>(a.res) + row * a.ldr : nullptr;
  float h[K][G], w[K][G], s = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) load_sum<T, true>(a, x, r, k * blockDim.x + threadIdx.x, h[k]);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (K * G <= 32) load_weight<T, true>(a, k * blockDim.x + threadIdx.x, w[k]);
#pragma unroll
    for (int i = 0; i < G; ++i) s = __fmaf_rn(h[k][i], h[k][i], s);
  }
  if (a.res_out) {
    T* o = static_cast<T*>(a.res_out) + row * a.ldo;
#pragma unroll
    for (int k = 0; k < K; ++k) store_group<T, true>(o, k * blockDim.x + threadIdx.x, a.n, h[k]);
  }
  const float rs = row_scale(a, s);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int g = k * blockDim.x + threadIdx.x;
    if (K * G > 32) load_weight<T, true>(a, g, w[k]);
    finish_group<T, true>(a, row, g, rs, h[k], w[k]);
  }
}

// Rows too long for registers, and rows whose addresses allow no 16-byte
// access: the row is read twice (the second time from L2).
template <class T, bool VEC>
__global__ void __launch_bounds__(1024) k_add_rms_norm_long(NormArgs a) {
  constexpr int G = Elem<T>::kGroup;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* r = a.res ? static_cast<const T*>(a.res) + row * a.ldr : nullptr;
  const int groups = (a.n + G - 1) / G;
  float s = 0.f;
  for (int g = threadIdx.x; g < groups; g += blockDim.x) {
    float h[G];
    load_sum<T, VEC>(a, x, r, g, h);
#pragma unroll
    for (int i = 0; i < G; ++i) s = __fmaf_rn(h[i], h[i], s);
  }
  const float rs = row_scale(a, s);
  for (int g0 = 0; g0 < groups; g0 += blockDim.x) {
    const int g = g0 + threadIdx.x;
    float h[G], w[G];
    load_sum<T, VEC>(a, x, r, g, h);
    load_weight<T, VEC>(a, g, w);
    if (a.res_out) store_group<T, VEC>(static_cast<T*>(a.res_out) + row * a.ldo, g, a.n, h);
    finish_group<T, VEC>(a, row, g, rs, h, w);
  }
}

// Threads a row, from n and the type alone (not from the rows: their bits
// must not depend on the batch): two groups of 16 bytes a thread up to 256
// groups, three where that leaves fewer threads idle (8191 rows of 2048 bf16:
// 21.5 us against 26.2 with one, of 1024 f32 17.6 against 19.9, of 768 bf16 9.6
// against 11.0), then 256 threads of up to six groups, each count a form of its
// own (8191 x 4128 f32: 67.8 us with five, 71.9 in the form for six; 8000 x 5120
// bf16: 51.3 with three, 66.5 in the form for four), then 384 (4096 x 14336
// bf16: 74 us, 93 with 512; one row 4.5 and 4.8), then 1024 (14336 f32: 64 rows
// 5.1 us, 7.3 with 512; 2000 rows 71.5 and 67).
template <class T>
static int launch_norm(const NormArgs& a, int64_t nvec, bool vec, cudaStream_t s) {
  constexpr int G = Elem<T>::kGroup;
  const char* who = "q8_add_rms_norm launch";
  const int groups = (a.n + G - 1) / G;
  const auto each = [&](int k) { return (groups + 32 * k - 1) / (32 * k) * 32; };  // threads of k groups
  int threads = groups > 6 * 384 ? 1024 : groups > 6 * 256 ? 384 : 256;
  if (groups <= 256) threads = 3 * each(3) < 2 * each(2) ? each(3) : each(2);
  const int k = (groups + threads - 1) / threads;
  const dim3 grid{unsigned(nvec)};
  if (!vec) return launch_op(k_add_rms_norm_long<T, false>, grid, threads, 0, 1, s, who, a);
  if (k == 1) return launch_op(k_add_rms_norm<T, 1>, grid, threads, 0, 1, s, who, a);
  if (k == 2) return launch_op(k_add_rms_norm<T, 2>, grid, threads, 0, 1, s, who, a);
  if (k == 3) return launch_op(k_add_rms_norm<T, 3>, grid, threads, 0, 1, s, who, a);
  if (k == 4) return launch_op(k_add_rms_norm<T, 4>, grid, threads, 0, 1, s, who, a);
  if (k == 5) return launch_op(k_add_rms_norm<T, 5>, grid, threads, 0, 1, s, who, a);
  if (k == 6) return launch_op(k_add_rms_norm<T, 6>, grid, threads, 0, 1, s, who, a);
  return launch_op(k_add_rms_norm_long<T, true>, grid, threads, 0, 1, s, who, a);
}

}  // namespace q1

using namespace q1;

extern "C" int q8_add_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const float* weight,
                               float eps, int64_t nvec, int64_t n, int dtype, void* residual_out, int64_t ldo,
                               void* y, int64_t ldy, int8_t* q, uint16_t* d, void* stream) {
  const char* who = "q8_add_rms_norm";
  if (nvec < 1 || nvec > (int64_t(1) << 24) || n < 1 || n > (int64_t(1) << 24))
    return fail(Q1_ERR_ARG, "%s: bad shape nvec=%lld n=%lld", who, (long long)nvec, (long long)n);
  if (dtype != Q1_F32 && dtype != Q1_BF16 && dtype != Q1_F16) return fail(Q1_ERR_ARG, "%s: bad type %d", who, dtype);
  if (!x || !weight || (!q && !y && !residual_out) || (!q != !d)) return fail(Q1_ERR_ARG, "%s: null pointer", who);
  if (q && n % kSub) return fail(Q1_ERR_ARG, "%s: n=%lld is no multiple of 32", who, (long long)n);
  if (!(eps >= 0.f)) return fail(Q1_ERR_ARG, "%s: eps must not be negative", who);
  if (ldx < n || (residual && ldr < n) || (residual_out && ldo < n) || (y && ldy < n))
    return fail(Q1_ERR_ARG, "%s: a row stride is less than n", who);
  const int64_t size = dtype == Q1_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(x) % size || reinterpret_cast<uintptr_t>(residual) % size ||
      reinterpret_cast<uintptr_t>(residual_out) % size || reinterpret_cast<uintptr_t>(y) % size ||
      reinterpret_cast<uintptr_t>(weight) % 4 || !aligned16(q) || !aligned16(d))
    return fail(Q1_ERR_ARG, "%s: a misaligned pointer (q and d: 16 bytes, the others their type's size)", who);
  NormArgs a = {x, residual, weight, residual_out, y, q, d, ldx, ldr, ldo, ldy, int(n), eps};
  // 16-byte accesses where every row starts on 16 bytes and holds whole groups.
  const auto fits = [&](const void* p, int64_t ld) { return !p || (aligned16(p) && ld * size % 16 == 0); };
  const bool vec = n * size % 16 == 0 && fits(x, ldx) && fits(residual, ldr) && fits(residual_out, ldo) && fits(y, ldy) &&
                   aligned16(weight);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == Q1_F32) return launch_norm<float>(a, nvec, vec, s);
  if (dtype == Q1_BF16) return launch_norm<__nv_bfloat16>(a, nvec, vec, s);
  return launch_norm<__half>(a, nvec, vec, s);
}
