// q8.cuh -- q8_0 within kernels: blocks of 32 values to quants and a scale, as
// quant.cu defines them, and quants back to numbers; the paged q8_0 cache.
#pragma once

#include <cfloat>

#include "paged.cuh"

namespace q1 {

// roundf(t), halves away from zero, in the last byte, |t| < 2^22: |t| + 1/2 and then the sum with
// 2^23, whose last bits are the whole part, both rounded toward zero, which keeps the whole
// part where |t| + 1/2 is no float.
__device__ __forceinline__ uint32_t q8_code(float t) {
  const uint32_t k = __float_as_uint(__fadd_rz(__fadd_rz(fabsf(t), 0.5f), 8388608.0f));
  const uint32_t sign = uint32_t(__float_as_int(t) >> 31);
  return (k ^ sign) - sign;
}

// Quants of `kCount` values of a block of 32 that 32 / kCount neighbouring lanes
// hold (`lanes`: the mask of those that call), four to a word, and the block's
// scale: NaN where one of the values is no number.
template <int kCount>
__device__ __forceinline__ float q8_block(const float (&x)[kCount], unsigned lanes, uint32_t (&code)[kCount / 4]) {
  uint32_t top = 0;  // bits of magnitudes are in the order of the magnitudes, with NaN above inf above all numbers
#pragma unroll
  for (int i = 0; i < kCount; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
  for (int off = kSub / kCount / 2; off > 0; off >>= 1) top = max(top, __shfl_xor_sync(lanes, top, off));
  const float amax = __uint_as_float(top >= 0x7f800000u ? 0x7fc00000u : top);
  const float d = __fdiv_rn(amax, 127.0f);
  const float id = d != 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
  if (id <= FLT_MAX) {
#pragma unroll
    for (int i = 0; i < kCount; i += 4) {
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = q8_code(__fmul_rn(x[i + j], id));
      code[i / 4] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    }
  } else {  // d is NaN, or so small (a scale of zero) that its inverse is infinite
#pragma unroll
    for (int i = 0; i < kCount; i += 4) {
      uint32_t c = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) c |= uint32_t(uint8_t(static_cast<int8_t>(static_cast<int>(roundf(__fmul_rn(x[i + j], id)))))) << (8 * j);
      code[i / 4] = c;
    }
  }
  return d;
}

// Four quants as floats: the byte b ^ 0x80 = b + 128 as the last bits of 2^23 + b + 128.
__device__ __forceinline__ void q8_floats(uint32_t w, float (&v)[4]) {
  w ^= 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __fadd_rn(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440u | uint32_t(i))), -8388736.0f);
}

struct Paged8 {
  Paged kv;  // k and v are int8; strides in values
  uint16_t *ks, *vs;
  int64_t s_page, s_slot, s_head;  // scales
};

// Checks the descriptor and fills in the kernels' form of it.
int check_paged_q8(const char* who, const q1_paged_q8* kv, Paged8& p);

// cache8.cu: f16 copies of the keys and values of the sequences of p with at least
// `least_rows` / group new tokens, for the tensor-core kernel: pages of 128 tokens,
// [part][sequence * pages + page][kv_heads][128][dim], `pages` of them a sequence, and their
// `table`.  Values of a sequence and head are divided by a power of two that brings the
// largest possible one near f16's, [sequence][kv_heads][keys, values] in `factors`; a second part
// holds what rounding to f16 took.
constexpr int kTopSlices = 16;
struct CopyQ8 {
  Paged8 p;
  __half *k, *v;
  int32_t* table;
  float* factors;
  uint32_t* tops;  // [sequence][kv_heads][keys, values][slices]: the largest scales
  unsigned* status;
  int pages, parts, dim, group, least_rows;
};
int launch_copy_q8(const CopyQ8& c, cudaStream_t s);

}  // namespace q1
