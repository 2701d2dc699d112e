// gate.cu -- q8_gated_act: y = act(gate) * up, and the q8_0 form of y.
//
// Elementwise but for a block's maximum: a value costs 9 bytes (f32 in, a quant out), which
// bound it, by little (profiled: instructions issued in 84 % of the cycles): with one 16-byte group a thread,
// eight lanes a block, and quants rounded by conversions it took 109 us where eight values a thread, four
// lanes a block, rounded on the FMA pipe, take 84.
//
// Measured: 4095 rows of 14336 f32 values to q8_0, 532 MB, 84 us: 6.3 TB/s, 0.94 of the copy
// bandwidth; 2000 x 11008 bf16, gelu, 132 MB, 20.6 us (0.95; 31.5 with an exact exponential and division);
// one row of 14336 1.9 us a launch in a chain of them.
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
constexpr int kGateValues = 8;  // consecutive ones a thread: four lanes a block

// silu: the same operations as torch's silu of f32 tensors, bit for bit.  gelu: x / (1 + e^-2u) with the
// exponential and the reciprocal of the special-function unit, off by some 2^-22 of itself each.
template <int kAct>
__device__ __forceinline__ float activation(float x) {
  if constexpr (kAct == Q1_ACT_SILU) {
    return __fdiv_rn(x, __fadd_rn(1.0f, expf(-x)));
  } else {
    // -2 sqrt(2/pi) log2(e) x (1 + 0.044715 x^2)
    const float t = __fmul_rn(__fmul_rn(x, -2.3022082f), __fmaf_rn(__fmul_rn(x, x), 0.044715f, 1.0f));
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.0f, e)));
    return __fmul_rn(x, r);
  }
}

// Values e .. e+7 of a row of n; past it: zeros.
template <class T, bool kVec>
__device__ __forceinline__ void load8(const T* row, int e, int n, float (&v)[kGateValues]) {
  constexpr int G = Elem<T>::kGroup;
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < kGateValues; i += G) {
      uint4 r = make_uint4(0u, 0u, 0u, 0u);
      if (e + i < n) r = *reinterpret_cast<const uint4*>(row + e + i);
      float part[G];
      Elem<T>::unpack(r, part);
#pragma unroll
      for (int j = 0; j < G; ++j) v[i + j] = part[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kGateValues; ++i) v[i] = e + i < n ? Elem<T>::to(row[e + i]) : 0.f;
  }
}

template <class T, int kAct, bool kVec>
__global__ void __launch_bounds__(kGateThreads) k_gated_act(GateArgs a) {
  constexpr int G = Elem<T>::kGroup;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t row = blockIdx.x / unsigned(a.parts);
  const int e = (int(blockIdx.x - unsigned(row) * unsigned(a.parts)) * kGateThreads + int(threadIdx.x)) * kGateValues;
  float x[kGateValues], u[kGateValues];
  load8<T, kVec>(static_cast<const T*>(a.gate) + row * a.ldg, e, a.n, x);
  load8<T, kVec>(static_cast<const T*>(a.up) + row * a.ldu, e, a.n, u);
#pragma unroll
  for (int i = 0; i < kGateValues; ++i) x[i] = __fmul_rn(activation<kAct>(x[i]), u[i]);
  if (a.y) {
    T* to = static_cast<T*>(a.y) + row * a.ldy + e;
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < kGateValues; i += G) {
        float part[G];
#pragma unroll
        for (int j = 0; j < G; ++j) part[j] = x[i + j];
        if (e + i < a.n) *reinterpret_cast<uint4*>(to + i) = Elem<T>::pack(part);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kGateValues; ++i)
        if (e + i < a.n) to[i] = Elem<T>::from(x[i]);
    }
  }
  if (a.q) {  // the whole warp is here
    uint32_t code[kGateValues / 4];
    const float d = q8_block<kGateValues>(x, 0xffffffffu, code);
    if (e >= a.n) return;  // (n is a multiple of 32)
    *reinterpret_cast<uint2*>(a.q + row * a.n + e) = make_uint2(code[0], code[1]);
    if (e % kSub == 0) a.d[row * (a.n / kSub) + e / kSub] = __half_as_ushort(__float2half_rn(d));
  }
}

template <class T, int kAct, bool kVec>
static int launch_gate_as(GateArgs& a, int64_t nvec, cudaStream_t s) {
  constexpr int kPart = kGateThreads * kGateValues;
  a.parts = (a.n + kPart - 1) / kPart;
  // (2^24 rows of 2^24 values are more bytes than any device has; parts of them fit 31 bits
  // for all that does.)
  if (nvec * a.parts >= (int64_t(1) << 31)) return fail(Q1_ERR_ARG, "q8_gated_act: too many values");
  return launch_op(k_gated_act<T, kAct, kVec>, dim3(unsigned(nvec * a.parts)), kGateThreads, 0, 1, s, "q8_gated_act launch", a);
}

template <class T>
static int launch_gate(GateArgs& a, int64_t nvec, int act, bool vec, cudaStream_t s) {
  if (!vec) return act == Q1_ACT_SILU ? launch_gate_as<T, Q1_ACT_SILU, false>(a, nvec, s) : launch_gate_as<T, Q1_ACT_GELU, false>(a, nvec, s);
  return act == Q1_ACT_SILU ? launch_gate_as<T, Q1_ACT_SILU, true>(a, nvec, s) : launch_gate_as<T, Q1_ACT_GELU, true>(a, nvec, s);
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
