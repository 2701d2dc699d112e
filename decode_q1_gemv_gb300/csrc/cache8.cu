// cache8.cu -- the paged q8_0 cache: q1_rope_append_q8 (rotary positions, and
// keys and values into the cache), q1_cache_read_q8 (and back), the 16-bit copy
// that the attention of many rows works on, and the checks of the descriptor.
//
// All of them touch every value once with a few operations: bytes bound them
// when there are many tokens (4 in and 1.06 out a key or value on append, 1.06
// in and 2 or 4 out on reading), and the chain of small loads (which sequence,
// its length, its page) when there are few, as in rope.cu.
//
// Measured: 5751 tokens of seven prompts (32 + 8 + 8 heads of 64) appended in 18.1 us (102 MB, 0.83 of the copy
// bandwidth) and read back in 6.5; 64 single tokens (heads of 128) in 3.2 and 2.1 us a launch.  The copy of
// 16001 tokens of 8 heads of 128 to f16 with its scales' maxima takes 37 us in profiled launches (101 MB, most of it in L2), of 27000 tokens of 16
// heads of 64 in two parts 55 (283 MB); CTAs from 4 to 200 an SM and one to four tokens' loads at once change it by 10 %.
#include "q8.cuh"

namespace q1 {

struct Rope8Args {
  Paged8 p;
  const float *q, *k, *v;
  int64_t ldq, ldk, ldv;
  const float* cs;     // [positions][rot]: rot/2 cosines, then rot/2 sines
  void* q_out;
  unsigned* status;
  int heads, dim, rot, positions, interleaved;
  int shift, units;  // units of 8 values: log2 of a head's, of a token's q, k and v
};

constexpr int kCacheThreads = 128;

// The token's sequence, its position there (-1: none) and its page.  Every thread calls.
struct Place {
  int seq, pos, page;
  bool owned, good;
};
__device__ __forceinline__ Place place_of(const Paged& kv, int token, int positions) {
  int before = 0;  // sequences that end at or before the token
  for (int b0 = 0; b0 < kv.batch; b0 += kCacheThreads) {
    const int b = b0 + threadIdx.x;
    before += __syncthreads_count(b < kv.batch && kv.new_start[b + 1] <= token);
  }
  Place at = {before, -1, -1, before < kv.batch && kv.new_start[before < kv.batch ? before : 0] <= token, false};
  if (at.owned) {
    at.pos = kv.kv_len[before] - kv.new_start[before + 1] + token;
    if (at.pos >= 0 && at.pos < positions && at.pos < kv.table_tokens)
      at.page = kv.table[before * kv.table_stride + (at.pos >> kv.page_shift)];
  }
  at.good = at.page >= 0 && at.page < kv.pages;
  return at;
}
__device__ __forceinline__ int64_t value_offset(const Paged8& p, int page, int pos) {
  return int64_t(page) * p.kv.page_stride + int64_t(pos & ((1 << p.kv.page_shift) - 1)) * p.kv.slot_stride;
}
__device__ __forceinline__ int64_t scale_offset(const Paged8& p, int page, int pos) {
  return int64_t(page) * p.s_page + int64_t(pos & ((1 << p.kv.page_shift) - 1)) * p.s_slot;
}

// Values e .. e+3 (e a multiple of 4) of a head at `src`, turned: the same
// operations on the same values as in rope.cu.
__device__ __forceinline__ float4 turned4(const Rope8Args& a, const float* src, const float* cs, int e) {
  const float4 x = *reinterpret_cast<const float4*>(src + e);
  if (e >= a.rot) return x;
  const int half = a.rot >> 1;
  const auto first = [](float p, float q, float c, float s) { return __fmaf_rn(-q, s, __fmul_rn(p, c)); };
  const auto second = [](float p, float q, float c, float s) { return __fmaf_rn(p, s, __fmul_rn(q, c)); };
  if (a.interleaved) {
    const float2 c = *reinterpret_cast<const float2*>(cs + (e >> 1)), s = *reinterpret_cast<const float2*>(cs + half + (e >> 1));
    return make_float4(first(x.x, x.y, c.x, s.x), second(x.x, x.y, c.x, s.x), first(x.z, x.w, c.y, s.y), second(x.z, x.w, c.y, s.y));
  }
  const bool low = e < half;
  const int i = low ? e : e - half;
  const float4 y = *reinterpret_cast<const float4*>(src + (low ? e + half : i));
  const float4 c = *reinterpret_cast<const float4*>(cs + i), s = *reinterpret_cast<const float4*>(cs + half + i);
  if (low) return make_float4(first(x.x, y.x, c.x, s.x), first(x.y, y.y, c.y, s.y), first(x.z, y.z, c.z, s.z), first(x.w, y.w, c.w, s.w));
  return make_float4(second(y.x, x.x, c.x, s.x), second(y.y, x.y, c.y, s.y), second(y.z, x.z, c.z, s.z), second(y.w, x.w, c.w, s.w));
}

// One CTA takes a token (or a part of its units, blockIdx.y); a unit is 8
// consecutive values of one head, four lanes a block of the cache.  The halves of a
// split rotation are 4 to 64 values apart and then read twice, the second time from L1.
template <class T>
__global__ void __launch_bounds__(kCacheThreads) k_rope_append_q8(const __grid_constant__ Rope8Args a) {
  pdl_launch_dependents();
  pdl_wait();
  const Paged& kv = a.p.kv;
  const int token = blockIdx.x;
  const Place at = place_of(kv, token, a.positions);
  if (at.owned && !at.good && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(a.status, kStatusBadIndex);
  const int64_t slot = value_offset(a.p, at.page, at.pos), scale = scale_offset(a.p, at.page, at.pos);
  const float* cs = a.cs + int64_t(at.good ? at.pos : 0) * a.rot;

  const int qunits = a.heads << a.shift, kunits = kv.kv_heads << a.shift;
  for (int u = blockIdx.y * kCacheThreads + threadIdx.x; u < a.units; u += gridDim.y * kCacheThreads) {
    const int part = u < qunits ? 0 : u < qunits + kunits ? 1 : 2;  // the same for the four lanes of a block
    const int v = part == 0 ? u : part == 1 ? u - qunits : u - qunits - kunits;
    const int head = v >> a.shift, e = (v & ((1 << a.shift) - 1)) * 8;
    const float* src = (part == 0 ? a.q + token * a.ldq : part == 1 ? a.k + token * a.ldk : a.v + token * a.ldv) + head * a.dim;
    if (part != 0 && !at.good) continue;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    if (part == 2)
      x = *reinterpret_cast<const float4*>(src + e), y = *reinterpret_cast<const float4*>(src + e + 4);
    else if (at.good)
      x = turned4(a, src, cs, e), y = turned4(a, src, cs, e + 4);
    if (part == 0) {
      *reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + (int64_t(token) * a.heads + head) * a.dim + e) =
          make_uint4(Elem<T>::pack2(x.x, x.y), Elem<T>::pack2(x.z, x.w), Elem<T>::pack2(y.x, y.y), Elem<T>::pack2(y.z, y.w));
      continue;
    }
    const float w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    uint32_t code[2];
    const float d = q8_block<8>(w, 0xfu << (threadIdx.x & 28), code);
    int8_t* to = static_cast<int8_t*>(part == 1 ? kv.k : kv.v) + slot + head * kv.head_stride + e;
    *reinterpret_cast<uint2*>(to) = make_uint2(code[0], code[1]);
    if ((e & (kSub - 1)) == 0) (part == 1 ? a.p.ks : a.p.vs)[scale + head * a.p.s_head + e / kSub] = __half_as_ushort(__float2half_rn(d));
  }
}

// 16 values of a block: quants times the scale.
__device__ __forceinline__ void values16(const uint4& w, float s, float (&v)[16]) {
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[4];
    q8_floats(words[i], f);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[i * 4 + j] = __fmul_rn(f[j], s);
  }
}
template <class T>
__device__ __forceinline__ void write16(T* to, const float (&v)[16]) {
  constexpr int G = Elem<T>::kGroup;
#pragma unroll
  for (int i = 0; i < 16; i += G) {
    float part[G];
#pragma unroll
    for (int j = 0; j < G; ++j) part[j] = v[i + j];
    reinterpret_cast<uint4*>(to)[i / G] = Elem<T>::pack(part);
  }
}

struct Read8Args {
  Paged8 p;
  void *k, *v;  // [total_new][kv_heads][dim], or null
  unsigned* status;
  int dim, shift;  // log2 of a head's units of 16 values
};

// One CTA takes a token; a unit is 16 consecutive values of one head.
template <class T>
__global__ void __launch_bounds__(kCacheThreads) k_cache_read_q8(const __grid_constant__ Read8Args a) {
  pdl_launch_dependents();
  pdl_wait();
  const Paged& kv = a.p.kv;
  const int token = blockIdx.x;
  const Place at = place_of(kv, token, kv.table_tokens);
  if (at.owned && !at.good && threadIdx.x == 0) atomicOr(a.status, kStatusBadIndex);
  const int64_t slot = value_offset(a.p, at.page, at.pos), scale = scale_offset(a.p, at.page, at.pos);
  const int units = kv.kv_heads << a.shift;
  for (int u = threadIdx.x; u < 2 * units; u += kCacheThreads) {
    const bool second = u >= units;
    const int v = second ? u - units : u, head = v >> a.shift, e = (v & ((1 << a.shift) - 1)) * 16;
    T* out = static_cast<T*>(second ? a.v : a.k);
    if (!out) continue;
    float x[16] = {};
    if (at.good)
      values16(*reinterpret_cast<const uint4*>(static_cast<const int8_t*>(second ? kv.v : kv.k) + slot + head * kv.head_stride + e),
               __half2float(__ushort_as_half((second ? a.p.vs : a.p.ks)[scale + head * a.p.s_head + e / kSub])), x);
    write16(out + (int64_t(token) * kv.kv_heads + head) * a.dim + e, x);
  }
}

// The largest finite scales of keys and values of a sequence's head, a sixteenth
// of the tokens a CTA.
constexpr int kTopThreads = 256;
__global__ void __launch_bounds__(kTopThreads) k_scale_tops(const __grid_constant__ CopyQ8 a) {
  __shared__ uint32_t top_s[kTopThreads / 32][2];
  pdl_launch_dependents();
  pdl_wait();
  const Paged& kv = a.p.kv;
  const int slice = blockIdx.x, head = blockIdx.y, b = blockIdx.z;
  const SeqSpan s = seq_span(kv, b);  // (the attention reports what it changes)
  if (int64_t(s.count) * a.group < a.least_rows) return;
  const int32_t* table = kv.table + b * kv.table_stride;
  const int j0 = int(int64_t(s.len) * slice / kTopSlices), j1 = int(int64_t(s.len) * (slice + 1) / kTopSlices);
  uint32_t top[2] = {0u, 0u};
#pragma unroll 4
  for (int j = j0 + threadIdx.x; j < j1; j += kTopThreads) {
    const int page = table[j >> kv.page_shift];
    if (page < 0 || page >= kv.pages) continue;
    const int64_t at = scale_offset(a.p, page, j & ((1 << kv.page_shift) - 1)) + head * a.p.s_head;
#pragma unroll
    for (int second = 0; second < 2; ++second) {
      const uint32_t* d = reinterpret_cast<const uint32_t*>((second ? a.p.vs : a.p.ks) + at);
      for (int i = 0; i < a.dim / 64; ++i) {
        const uint32_t w = d[i], lo = w & 0x7fffu, hi = w >> 16 & 0x7fffu;
        if (lo < 0x7c00u) top[second] = max(top[second], lo);
        if (hi < 0x7c00u) top[second] = max(top[second], hi);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    top[i] = __reduce_max_sync(0xffffffffu, top[i]);
    if ((threadIdx.x & 31) == 0) top_s[threadIdx.x >> 5][i] = top[i];
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    uint32_t m = 0;
    for (int w = 0; w < kTopThreads / 32; ++w) m = max(m, top_s[w][threadIdx.x]);
    a.tops[((int64_t(b) * kv.kv_heads + head) * 2 + threadIdx.x) * kTopSlices + slice] = m;
  }
}

// A CTA takes 16 tokens for every dim threads; those of a sequence's head (blockIdx.x) take
// its tokens in turn, so that short sequences of a wide table cost little.
constexpr int kCopyThreads = 256;
template <int kParts>
__global__ void __launch_bounds__(kCopyThreads) k_copy_q8(const __grid_constant__ CopyQ8 a) {
  pdl_launch_dependents();
  pdl_wait();
  const Paged& kv = a.p.kv;
  const int head = blockIdx.y, b = blockIdx.z;
  if (head == 0)
    for (int i = blockIdx.x * kCopyThreads + threadIdx.x; i < a.pages; i += gridDim.x * kCopyThreads)
      a.table[int64_t(b) * a.pages + i] = b * a.pages + i;
  const SeqSpan s = seq_span(kv, b);
  if (int64_t(s.count) * a.group < a.least_rows) return;
  // Values are at most 127 scales: below 2^15 once divided by the largest scale's power of two and 2^-7.
  const uint32_t* tops = a.tops + (int64_t(b) * kv.kv_heads + head) * 2 * kTopSlices;
  float factor[2], inverse[2];
  {
    uint32_t top = tops[threadIdx.x & 31];
    static_assert(2 * kTopSlices == 32, "a lane a slice");
#pragma unroll
    for (int off = kTopSlices / 2; off > 0; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t t = __shfl_sync(0xffffffffu, top, i * kTopSlices);
      const uint32_t e = t ? (__float_as_uint(__half2float(__ushort_as_half(uint16_t(t)))) >> 23) - 7u : 127u;
      factor[i] = __uint_as_float(e << 23), inverse[i] = __uint_as_float((254u - e) << 23);
    }
  }
  if (blockIdx.x == 0 && threadIdx.x < 2) a.factors[(int64_t(b) * kv.kv_heads + head) * 2 + threadIdx.x] = threadIdx.x ? factor[1] : factor[0];
  const int units = a.dim / 16, page_mask = (1 << kv.page_shift) - 1, step = kCopyThreads / units;  // tokens at a time
  const int e = int(threadIdx.x) % units * 16;
  const int32_t* table = kv.table + b * kv.table_stride;
  const int64_t part = int64_t(kv.batch) * a.pages * kv.kv_heads * 128 * a.dim;
  // kAtOnce tokens' loads side by side.
  constexpr int kAtOnce = 2;
  for (int j0 = blockIdx.x * step + int(threadIdx.x) / units; j0 < s.len; j0 += kAtOnce * gridDim.x * step) {
    uint4 q[kAtOnce][2];
    uint16_t d[kAtOnce][2];
#pragma unroll
    for (int n = 0; n < kAtOnce; ++n) {
      const int j = j0 + n * int(gridDim.x) * step;
      q[n][0] = q[n][1] = make_uint4(0u, 0u, 0u, 0u), d[n][0] = d[n][1] = 0;
      if (j >= s.len) continue;
      const int page = table[j >> kv.page_shift];
      if (page < 0 || page >= kv.pages) {  // zeros
        atomicOr(a.status, kStatusBadIndex);
        continue;
      }
      const int64_t from = value_offset(a.p, page, j & page_mask) + head * kv.head_stride + e;
      const int64_t scale = scale_offset(a.p, page, j & page_mask) + head * a.p.s_head + e / kSub;
      q[n][0] = *reinterpret_cast<const uint4*>(static_cast<const int8_t*>(kv.k) + from), d[n][0] = a.p.ks[scale];
      q[n][1] = *reinterpret_cast<const uint4*>(static_cast<const int8_t*>(kv.v) + from), d[n][1] = a.p.vs[scale];
    }
#pragma unroll
    for (int n = 0; n < kAtOnce; ++n) {
      const int j = j0 + n * int(gridDim.x) * step;
      if (j >= s.len) break;
      const int64_t to = (((int64_t(b) * a.pages + j / 128) * kv.kv_heads + head) * 128 + j % 128) * a.dim + e;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x[16];
        values16(q[n][i], __fmul_rn(__half2float(__ushort_as_half(d[n][i])), inverse[i]), x);
        __half* out = (i ? a.v : a.k) + to;
        write16(out, x);
        if constexpr (kParts == 2) {
#pragma unroll
          for (int k = 0; k < 16; ++k) x[k] = __fsub_rn(x[k], __half2float(__float2half_rn(x[k])));
          write16(out + part, x);
        }
      }
    }
  }
}

int launch_copy_q8(const CopyQ8& c, cudaStream_t s) {
  const char* who = "q1_paged_attention_q8 launch";
  const Paged& kv = c.p.kv;
  if (int e = launch_op<CopyQ8>(k_scale_tops, dim3(kTopSlices, unsigned(kv.kv_heads), unsigned(kv.batch)), kTopThreads, 0, 1, s, who, c)) return e;
  const int64_t step = kCopyThreads / (c.dim / 16), most = (kv.table_tokens + step - 1) / step;
  const int64_t fill = (int64_t(8) * num_sms() + kv.batch * kv.kv_heads - 1) / (int64_t(kv.batch) * kv.kv_heads);  // eight CTAs an SM
  const dim3 grid(unsigned(most < fill ? most : fill), unsigned(kv.kv_heads), unsigned(kv.batch));
  if (c.parts == 2) return launch_op<CopyQ8>(k_copy_q8<2>, grid, kCopyThreads, 0, 1, s, who, c);
  return launch_op<CopyQ8>(k_copy_q8<1>, grid, kCopyThreads, 0, 1, s, who, c);
}

int check_paged_q8(const char* who, const q1_paged_q8* kv, Paged8& p) {
  if (!kv) return fail(Q1_ERR_ARG, "%s: null descriptor", who);
  q1_paged_kv c = {kv->k, kv->v, kv->page_stride, kv->slot_stride, kv->head_stride, kv->table, kv->table_width, kv->table_stride,
                   kv->kv_len, kv->new_start, kv->pages, kv->page_size, kv->kv_heads, kv->dim, kv->batch, kv->total_new, Q1_BF16};
  if (int e = check_paged(who, &c, p.kv)) return e;
  if (kv->page_stride % 16 || kv->slot_stride % 16 || kv->head_stride % 16)
    return fail(Q1_ERR_ARG, "%s: the cache's strides must be multiples of 16 values", who);
  if (!kv->k_scale || !kv->v_scale) return fail(Q1_ERR_ARG, "%s: null pointer", who);
  if (!aligned16(kv->k_scale) || !aligned16(kv->v_scale)) return fail(Q1_ERR_ARG, "%s: the cache must be 16-byte aligned", who);
  const int64_t each = kv->dim / kSub;
  for (const int64_t stride : {kv->scale_page_stride, kv->scale_slot_stride, kv->scale_head_stride})
    if (stride % each || stride < each || stride >= (int64_t(1) << 38))
      return fail(Q1_ERR_ARG, "%s: the scales' strides must be multiples of dim / 32, from that to 2^38", who);
  p.ks = kv->k_scale, p.vs = kv->v_scale;
  p.s_page = kv->scale_page_stride, p.s_slot = kv->scale_slot_stride, p.s_head = kv->scale_head_stride;
  return Q1_OK;
}

}  // namespace q1

using namespace q1;

extern "C" int q1_rope_append_q8(const float* q, int64_t ldq, const float* k, int64_t ldk, const float* v, int64_t ldv,
                                 const float* cos_sin, int64_t positions, int64_t rot, int interleaved, int64_t heads,
                                 void* q_out, int dtype, const q1_paged_q8* kv, void* stream) {
  const char* who = "q1_rope_append_q8";
  Rope8Args a = {};
  if (int e = check_paged_q8(who, kv, a.p)) return e;
  if (dtype != Q1_BF16 && dtype != Q1_F16) return fail(Q1_ERR_ARG, "%s: bad type %d", who, dtype);
  if (heads < 1 || heads > 4096) return fail(Q1_ERR_ARG, "%s: bad heads=%lld", who, (long long)heads);
  if (rot < 8 || rot > kv->dim || rot % 8 || positions < 1 || positions > (int64_t(1) << 30))
    return fail(Q1_ERR_ARG, "%s: rot=%lld must be a multiple of 8 in 8..dim, positions=%lld in 1..2^30", who,
                (long long)rot, (long long)positions);
  if (!q || !k || !v || !cos_sin || !q_out) return fail(Q1_ERR_ARG, "%s: null pointer", who);
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(cos_sin) || !aligned16(q_out) || ldq % 4 ||
      ldk % 4 || ldv % 4)
    return fail(Q1_ERR_ARG, "%s: buffers must be 16-byte aligned, row strides multiples of 4", who);
  if (ldq < heads * kv->dim || ldk < kv->kv_heads * kv->dim || ldv < kv->kv_heads * kv->dim)
    return fail(Q1_ERR_ARG, "%s: a row stride is less than its row", who);
  a.q = q, a.k = k, a.v = v, a.ldq = ldq, a.ldk = ldk, a.ldv = ldv;
  a.cs = cos_sin, a.q_out = q_out;
  if (int e = ops_status_ptr(&a.status)) return e;
  a.heads = int(heads), a.dim = int(kv->dim), a.rot = int(rot), a.positions = int(positions);
  a.interleaved = interleaved != 0;
  a.shift = a.dim == 64 ? 3 : 4;
  a.units = (a.heads + 2 * a.p.kv.kv_heads) << a.shift;
  const int per = (a.units + kCacheThreads - 1) / kCacheThreads;
  const dim3 grid(unsigned(a.p.kv.total_new), unsigned(a.p.kv.total_new < num_sms() ? per : 1));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == Q1_BF16) return launch_op<Rope8Args>(k_rope_append_q8<__nv_bfloat16>, grid, kCacheThreads, 0, 1, s, who, a);
  return launch_op<Rope8Args>(k_rope_append_q8<__half>, grid, kCacheThreads, 0, 1, s, who, a);
}

extern "C" int q1_cache_read_q8(const q1_paged_q8* kv, int dtype, void* k_out, void* v_out, void* stream) {
  const char* who = "q1_cache_read_q8";
  Read8Args a = {};
  if (int e = check_paged_q8(who, kv, a.p)) return e;
  if (dtype != Q1_F32 && dtype != Q1_BF16 && dtype != Q1_F16) return fail(Q1_ERR_ARG, "%s: bad type %d", who, dtype);
  if (!k_out && !v_out) return fail(Q1_ERR_ARG, "%s: null pointer", who);
  if (!aligned16(k_out) || !aligned16(v_out)) return fail(Q1_ERR_ARG, "%s: buffers must be 16-byte aligned", who);
  a.k = k_out, a.v = v_out, a.dim = int(kv->dim), a.shift = a.dim == 64 ? 2 : 3;
  if (int e = ops_status_ptr(&a.status)) return e;
  const dim3 grid{unsigned(a.p.kv.total_new)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == Q1_F32) return launch_op<Read8Args>(k_cache_read_q8<float>, grid, kCacheThreads, 0, 1, s, who, a);
  if (dtype == Q1_BF16) return launch_op<Read8Args>(k_cache_read_q8<__nv_bfloat16>, grid, kCacheThreads, 0, 1, s, who, a);
  return launch_op<Read8Args>(k_cache_read_q8<__half>, grid, kCacheThreads, 0, 1, s, who, a);
}
