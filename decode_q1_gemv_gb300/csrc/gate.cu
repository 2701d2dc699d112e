// gate.cu -- q8_gated_act: y = act(gate) * up, and the q8_0 form of y.
//
// Elementwise but for a block's maximum: a value costs some forty instructions
// (the exponential, three divisions' worth of it a fourth each) and 9 bytes (f32 in,
// a quant out), so bytes bound it.  A thread takes 16-byte groups of gate and up;
// the lanes of a block exchange its maximum, as in norm.cu.
#include "q8.cuh"

namespace q1 {

struct GateArgs {
  const void *gate, *up;
  void* y;      // or null
  int8_t* q;    // or null
  uint16_t* d;
  int64_t ldg, ldu, ldy;
  int n, parts;  // parts: CTAs a row
};

constexpr int kGateThreads = 256;

template <int kAct>
__device__ __forceinline__ float activation(float x) {
  float e = -x;
  if constexpr (kAct == Q1_ACT_GELU)
    e = __fmul_rn(-1.5957691216057308f, __fmaf_rn(__fmul_rn(__fmul_rn(x, x), x), 0.044715f, x));  // -2 sqrt(2/pi)
  return __fdiv_rn(x, __fadd_rn(1.0f, expf(e)));
}

// Group g (16 bytes) of a row.
template <class T, int kAct, bool kVec>
__device__ __forceinline__ void gate_group(const GateArgs& a, int64_t row, int g, const float (&x)[Elem<T>::kGroup],
                                           const float (&u)[Elem<T>::kGroup]) {
  constexpr int G = Elem<T>::kGroup;
  const int e = g * G;
  float y[G];
#pragma unroll
  for (int i = 0; i < G; ++i) y[i] = __fmul_rn(activation<kAct>(x[i]), u[i]);
  if (a.y && e < a.n) {
    T* to = static_cast<T*>(a.y) + row * a.ldy + e;
    if constexpr (kVec) {
      *reinterpret_cast<uint4*>(to) = Elem<T>::pack(y);
    } else {
#pragma unroll
      for (int i = 0; i < G; ++i)
        if (e + i < a.n) to[i] = Elem<T>::from(y[i]);
    }
  }
  if (a.q) {  // the whole warp calls
    uint32_t code[G / 4];
    const float d = q8_block<G>(y, 0xffffffffu, code);
    if (e >= a.n) return;
    int8_t* to = a.q + row * a.n + e;
    if constexpr (G == 4)
      *reinterpret_cast<uint32_t*>(to) = code[0];
    else
      *reinterpret_cast<uint2*>(to) = make_uint2(code[0], code[1]);
    if (e % kSub == 0) a.d[row * (a.n / kSub) + e / kSub] = __half_as_ushort(__float2half_rn(d));
  }
}

// kGroups groups a thread, their loads side by side.
template <class T, int kAct, bool kVec, int kGroups>
__global__ void __launch_bounds__(kGateThreads) k_gated_act(GateArgs a) {
  constexpr int G = Elem<T>::kGroup;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t row = blockIdx.x / unsigned(a.parts);
  const int g0 = int(blockIdx.x - unsigned(row) * unsigned(a.parts)) * (kGateThreads * kGroups) + threadIdx.x;
  const T* gate = static_cast<const T*>(a.gate) + row * a.ldg;
  const T* up = static_cast<const T*>(a.up) + row * a.ldu;
  float x[kGroups][G], u[kGroups][G];
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const int e = (g0 + k * kGateThreads) * G;
    if constexpr (kVec) {
      uint4 r = make_uint4(0u, 0u, 0u, 0u), s = r;
      if (e < a.n) r = *reinterpret_cast<const uint4*>(gate + e), s = *reinterpret_cast<const uint4*>(up + e);
      Elem<T>::unpack(r, x[k]);
      Elem<T>::unpack(s, u[k]);
    } else {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        x[k][i] = e + i < a.n ? Elem<T>::to(gate[e + i]) : 0.f;
        u[k][i] = e + i < a.n ? Elem<T>::to(up[e + i]) : 0.f;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kGroups; ++k) gate_group<T, kAct, kVec>(a, row, g0 + k * kGateThreads, x[k], u[k]);
}

template <class T, int kAct, bool kVec, int kGroups>
static int launch_gate_as(GateArgs& a, int64_t nvec, cudaStream_t s) {
  constexpr int kPart = kGateThreads * kGroups * Elem<T>::kGroup;
  a.parts = (a.n + kPart - 1) / kPart;
  // (2^24 rows of 2^24 values are more bytes than any device has; parts of them fit 31 bits
  // for all that does.)
  if (nvec * a.parts >= (int64_t(1) << 31)) return fail(Q1_ERR_ARG, "q8_gated_act: too many values");
  return launch_op(k_gated_act<T, kAct, kVec, kGroups>, dim3(unsigned(nvec * a.parts)), kGateThreads, 0, 1, s,
                   "q8_gated_act launch", a);
}

template <class T>
static int launch_gate(GateArgs& a, int64_t nvec, int act, bool vec, cudaStream_t s) {
  if (!vec) return act == Q1_ACT_SILU ? launch_gate_as<T, Q1_ACT_SILU, false, 1>(a, nvec, s) : launch_gate_as<T, Q1_ACT_GELU, false, 1>(a, nvec, s);
  return act == Q1_ACT_SILU ? launch_gate_as<T, Q1_ACT_SILU, true, 1>(a, nvec, s) : launch_gate_as<T, Q1_ACT_GELU, true, 1>(a, nvec, s);
}

}  // namespace q1

using namespace q1;

extern "C" int q8_gated_act(const void* gate, int64_t ldg, const void* up, int64_t ldu, int64_t nvec, int64_t n, int dtype,
                            int activation, void* y, int64_t ldy, int8_t* q, uint16_t* d, void* stream) {
  const char* who = "q8_gated_act";
  if (nvec < 1 || nvec > (int64_t(1) << 24) || n < 1 || n > (int64_t(1) << 24))
    return fail(Q1_ERR_ARG, "%s: bad shape nvec=%lld n=%lld", who, (long long)nvec, (long long)n);
  if (dtype != Q1_F32 && dtype != Q1_BF16 && dtype != Q1_F16) return fail(Q1_ERR_ARG, "%s: bad type %d", who, dtype);
  if (activation != Q1_ACT_SILU && activation != Q1_ACT_GELU) return fail(Q1_ERR_ARG, "%s: bad activation %d", who, activation);
  if (!gate || !up || (!q && !y) || (!q != !d)) return fail(Q1_ERR_ARG, "%s: null pointer", who);
  if (q && n % kSub) return fail(Q1_ERR_ARG, "%s: n=%lld is no multiple of 32", who, (long long)n);
  if (ldg < n || ldu < n || (y && ldy < n)) return fail(Q1_ERR_ARG, "%s: a row stride is less than n", who);
  const int64_t size = dtype == Q1_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(gate) % size || reinterpret_cast<uintptr_t>(up) % size ||
      reinterpret_cast<uintptr_t>(y) % size || !aligned16(q) || !aligned16(d))
    return fail(Q1_ERR_ARG, "%s: a misaligned pointer (q and d: 16 bytes, the others their type's size)", who);
  GateArgs a = {gate, up, y, q, d, ldg, ldu, ldy, int(n), 0};
  // 16-byte accesses where every row starts on 16 bytes and holds whole groups.
  const auto fits = [&](const void* p, int64_t ld) { return !p || (aligned16(p) && ld * size % 16 == 0); };
  const bool vec = n * size % 16 == 0 && fits(gate, ldg) && fits(up, ldu) && fits(y, ldy);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == Q1_F32) return launch_gate<float>(a, nvec, activation, vec, s);
  if (dtype == Q1_BF16) return launch_gate<__nv_bfloat16>(a, nvec, activation, vec, s);
  return launch_gate<__half>(a, nvec, activation, vec, s);
}
