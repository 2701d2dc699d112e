// attend8.cu -- q1_paged_attention_q8: new tokens attend to their sequence's
// paged q8_0 cache.  This file holds the kernel for few rows a key head (single
// tokens and short chunks) and the entry points; more rows go through a 16-bit
// copy of the sequence (cache8.cu) and the tensor-core kernel (attend_tc.cu).
//
// The formula, the split into items and units and the join are attend.cu's.
// Here a key and its value are 2 D (1 + 1/16) bytes, about half of a 16-bit
// cache's, so there is half the time for the same sums, and the instructions
// of a warp count.  A chunk of 16 keys therefore is the wide operand of the
// m16n8k16 MMAs and the rows the narrow one, eight at a time: S^T = K Q^T
// and O^T = V^T P^T, half of the MMAs and sums that 16 rows would take.
//   Keys: quants are whole numbers up to 127, exact in f16, two by a mask, an
//     exclusive or and a subtraction (0x6400 | b + 128 is 1152 + b).  q is f16 too, bf16 rows
//     divided by a power of two near their largest value, which f16's 11 bits hold exactly
//     down to 2^-14 of it.  The sums of 32 products are multiplied with the block's scale in f32.
//   Values: a block's scale depends on the key and the block, so it goes into
//     the weight: p d, rounded to f16.  So that its size does not matter, p is
//     relative not to the row's largest weight but to its largest product of a weight and
//     a key's largest scale: p d then is at most 2^8, off by 2^-11 of itself or, below 2^-14,
//     2^-25; the sum of p is f32, relative to the same.  (Relative to the largest scale of any key, a key
//     that weighs nothing in the row, or that it may not see, took bits from all others.)
// ldmatrix moves pairs of bytes as 16-bit elements: a lane gets four dims of a
// key, or (transposed) two dims of two keys; taking the even and the odd bytes of
// a word apart puts dims in the order 0 2 1 3 in both operands.
//
// Maxima are looked at by a vote: the ones in use move only when a product is 2^8 times
// beyond, so most chunks have no exchange between lanes for it.
//
// Measured (32 heads over 8 key heads of 128, bf16): one token of each of 64 sequences, 1.08 GB of keys and
// values, 177 us: 6.1 TB/s, 0.90 of the copy bandwidth (the 16-bit cache's kernel takes 312 us for 2.04 GB); one token over
// 8191 keys 11.8 us, over 1000 6.0 (16-bit: 11.9, 6.1).  Profiled with 16 of those sequences, instructions are issued
// in 59 % of the cycles and the pipe of masks and shifts, which take quants out of words, is 51 % active.  Rows past
// eight are further from their bytes (16 sequences of 4 tokens: 62 us, floor 21; of up to 12, f16: 50, floor 11).
// 2048 tokens over 16001 keys take 412 to 422 us (profiled: 37 of them the maxima and the copy).
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <type_traits>

#include <cooperative_groups.h>

#include "attend.cuh"
#include "q8.cuh"

namespace q1 {

namespace cg = cooperative_groups;

constexpr int kWarps8 = 4;
constexpr int kKeys8 = 16 * kWarps8;  // keys of a unit: 16 for each warp
constexpr int kWhole8 = 2;   // units of an item that is not split
constexpr float kGrow8 = 8.f;  // log2 units a maximum may be behind
// The log2 that a key's largest scale counts with at least: those of scales of zero have to be some number.  (Sums
// of weights are up to 2^(8 - this) times the number of keys.)
constexpr float kLeastScale8 = -40.f;

struct Attend8Args {
  AttendArgs a;        // kv.k and kv.v are quants
  const uint16_t *ks, *vs;
  int64_t s_page, s_slot, s_head;
};

// kWarps warps take chunks of 16 kHalves keys each.
template <int D, int NT, int kWarps = kWarps8, int kHalves = 1>
struct Shape8 {
  static constexpr int kRows = 8 * NT, kChunk = 16 * kHalves, kUnit = kChunk * kWarps;
  static constexpr int kRowBytes = D, kChunkBytes = kChunk * D, kScaleBytes = D / 16;  // a key's quants, a chunk's, a key's scales
  static constexpr int kStageBytes = 2 * kChunkBytes + 2 * kChunk * kScaleBytes;
  static constexpr int kCtas = kWarps == 2 * kWarps8 ? 1 : kHalves == 1 ? (NT == 1 ? 4 : 3) : D == 64 ? 4 - NT + 1 : 4 - NT;  // an SM
  static constexpr int kStages = (D == 64 ? 5 : NT == 1 ? 3 : 4) / kHalves + (kHalves == 2);
  static constexpr int kSmem = kWarps * kStages * kStageBytes;
  static_assert(kSmem >= kWarps * kRows * (D + 4) * 4, "the warps' outputs go over the ring");
  static_assert(kCtas * (kSmem + 2048) <= 227 * 1024, "");
};

template <int kBytes>
__device__ __forceinline__ void cp_async_scales(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes) : "memory");
}
template <int kBytes>
__device__ __forceinline__ void cp_async_scales(uint32_t dst, const void* src, uint32_t bytes) {  // zeros past `bytes`
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_whole(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// c += a b, and a b alone.
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_new(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transposed(uint32_t v) {  // of an 8x8 matrix of 16-bit elements
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Quants b0 and b2 of a word as f16; b1 and b3 those of the word shifted by a byte.
__device__ __forceinline__ uint32_t quants(uint32_t w) {
  const uint32_t biased = (w & 0x00ff00ffu) ^ 0x64806480u, bias = 0x64806480u;
  const __half2 r = __hsub2(reinterpret_cast<const __half2&>(biased), reinterpret_cast<const __half2&>(bias));
  return reinterpret_cast<const uint32_t&>(r);
}
// Scales of one key, kWords pairs of them, from shared memory; as f32.
template <int kWords>
__device__ __forceinline__ void scales_of(const unsigned char* at, uint32_t (&w)[kWords]) {
  if constexpr (kWords == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(at);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(at);
  }
}
// For keys an infinite scale is NaN, as the sum of the block's values is: the scale only meets the sum of the quants.
__device__ __forceinline__ uint32_t no_infinity(uint32_t w) {  // w * 0 + w
  const uint32_t zero = 0u;
  const __half2 r = __hfma2(reinterpret_cast<const __half2&>(w), reinterpret_cast<const __half2&>(zero), reinterpret_cast<const __half2&>(w));
  return reinterpret_cast<const uint32_t&>(r);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {  // of numbers, where there are some
  const __half2 r = __hmax2(reinterpret_cast<const __half2&>(a), reinterpret_cast<const __half2&>(b));
  return reinterpret_cast<const uint32_t&>(r);
}
// log2 of the largest magnitude of a key's scales that are numbers, kLeastScale8 at least.
template <int kWords>
__device__ __forceinline__ float log2_largest(const uint32_t (&w)[kWords]) {
  uint32_t tops = 0u;
#pragma unroll
  for (int k = 0; k < kWords; ++k) tops = max2(tops, no_infinity(w[k] & 0x7fff7fffu));  // (a NaN is passed over)
  float a, b, r;
  Elem<__half>::unpack2(tops, a, b);
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaxf(a, b)));  // -inf of zero
  return fmaxf(r, kLeastScale8);
}

// kCluster: not shares of the axis but a cluster of a.ctas CTAs for each
// sequence, key head and tile, which joins its own parts, as in attend.cu.
template <class T, int D, int NT, bool kCluster, int kWarps = kWarps8, int kHalves = 1>
__global__ void __launch_bounds__(kWarps * 32, Shape8<D, NT, kWarps, kHalves>::kCtas) k_attend_q8(const __grid_constant__ Attend8Args args) {
  using Shape = Shape8<D, NT, kWarps, kHalves>;
  constexpr int kUnit = Shape::kUnit, kChunk = Shape::kChunk;  // keys
  using Tile = Tiling<Shape::kRows, kUnit>;
  constexpr int kRows = Shape::kRows, kStages = Shape::kStages, kPieces = D / 16, kBlocks = D / 32, kWords = D / 64;
  const AttendArgs& a = args.a;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ LocateScratch scratch;
  __shared__ float ml[kWarps][kRows][2];
  __shared__ float2 own[kRows];  // kCluster: the CTA's maxima and sums
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  pdl_launch_dependents();
  if (!a.beside) pdl_wait();
  Cursor cur = {};
  int64_t u0, u1;
  int ctas = a.ctas;
  int64_t total = 0;
  if constexpr (kCluster) {
    const int item = int(blockIdx.x) / ctas, head = item / a.tiles;
    bool bad;
    cur.b = head / a.kv.kv_heads, cur.h = head - cur.b * a.kv.kv_heads;
    cur.s = seq_span(a.kv, cur.b, &bad);
    if (bad && threadIdx.x == 0) atomicOr(a.status, kStatusBadIndex);
    u0 = item - head * a.tiles, u1 = Tile::tiles(a, cur.s);  // tiles, here
  } else {
    total = locate<Tile, kWhole8 / kHalves>(a, blockIdx.x, ctas, scratch, cur, u0, u1);
    if (threadIdx.x == 0) a.joins[blockIdx.x].parts = 0;
  }
  unsigned char* my_ring = smem + warp * (kStages * Shape::kStageBytes);
  const uint32_t ring = smem_addr(my_ring);
  const int page_mask = (1 << a.kv.page_shift) - 1;
  // A key's 16-byte pieces trade places so that eight keys' same pieces, what ldmatrix reads, lie in different banks.
  const auto place = [](int piece, int r) { return piece ^ (D == 128 ? r & 7 : (r >> 1) & 3); };
  for (int64_t u = u0; u < u1;) {
    int take = 0;  // units of this item here
    if constexpr (kCluster) {
      const int i = int(blockIdx.x) % ctas;
      cur.m = int(u), cur.units = Tile::units(a, cur.s, cur.m);
      cur.unit = int(share(cur.units, i, ctas)), take = int(share(cur.units, i + 1, ctas)) - cur.unit;
    } else {
      take = int(min(int64_t(cur.units - cur.unit), u1 - u));
    }
    const int keys = Tile::keys(a, cur.s, cur.m), of_all = Tile::keys_of_all(a, cur.s, cur.m);
    const int32_t* table = a.kv.table + cur.b * a.kv.table_stride;

    // Chunk i of this warp: kChunk keys from j0 + kUnit i on, a multiple of 16.  16 of them lie in one page of 16
    // slots or more, which their lanes look up well before it is needed (of 8: each lane for row lane % kChunk).  A
    // lane copies piece lane % kPieces of rows lane / kPieces and on, and the scales of row lane % kChunk (of 16
    // rows: lanes from 16 on those of the values).
    constexpr int kRowsOnce = 32 / kPieces, kTimes = kChunk / kRowsOnce, kPlaces = 8 / kRowsOnce;
    const bool one_page = a.kv.page_shift >= 4;  // for 16
    const int j0 = cur.unit * kUnit + warp * kChunk, row0 = lane / kPieces, my_row = lane % kChunk;
    const int64_t rows_on = kRowsOnce * a.kv.slot_stride;
    const int8_t* kbase = static_cast<const int8_t*>(a.kv.k) + cur.h * a.kv.head_stride + lane % kPieces * 16;
    const int8_t* vbase = static_cast<const int8_t*>(a.kv.v) + cur.h * a.kv.head_stride + lane % kPieces * 16;
    const uint16_t* sbase = (lane < 16 || kHalves == 2 ? args.ks : args.vs) + cur.h * args.s_head;
    const uint16_t* sbase_v = args.vs + cur.h * args.s_head;  // kHalves == 2
    const auto page_of = [&](int i) {  // -1 past the keys
      const int j = j0 + i * kUnit + (one_page ? my_row & 16 : my_row);
      return i < take && j < keys ? table[j >> a.kv.page_shift] : -1;
    };
    const int64_t row_off = int64_t(row0) * a.kv.slot_stride;
    const bool dense = a.kv.slot_stride == D;  // a head's slots side by side: rows at constant distances
    uint32_t to[kPlaces];  // where this lane's pieces go in a stage: of its first rows, repeated every 8
#pragma unroll
    for (int k = 0; k < kPlaces; ++k)
      to[k] = ring + (k * kRowsOnce + row0) * Shape::kRowBytes + (place(lane % kPieces, k * kRowsOnce + row0) << 4);
    const auto dst_of = [&](int n) { return to[n % kPlaces] + n / kPlaces * 8 * Shape::kRowBytes; };
    const uint32_t scale_to = ring + 2 * Shape::kChunkBytes + lane * Shape::kScaleBytes;
    constexpr int kScaleV = kChunk * Shape::kScaleBytes;
    const auto fill = [&](int i, uint32_t stage, int page) {  // stage: its offset
      if (i < take) {
        const int j = j0 + i * kUnit;
        const bool usual = one_page && j + kChunk <= keys && page >= 0 && page < a.kv.pages;
        if (kHalves == 1 ? usual : __all_sync(0xffffffffu, usual)) {
          const int64_t soff = int64_t(page) * args.s_page + int64_t((j + my_row) & page_mask) * args.s_slot;
          cp_async_scales<Shape::kScaleBytes>(scale_to + stage, sbase + soff);
          if constexpr (kHalves == 2) cp_async_scales<Shape::kScaleBytes>(scale_to + stage + kScaleV, sbase_v + soff);
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            const int its_page = kHalves == 1 ? page : __shfl_sync(0xffffffffu, page, h * 16);
            const int64_t off = int64_t(its_page) * a.kv.page_stride + int64_t((j + h * 16) & page_mask) * a.kv.slot_stride + row_off;
            const int8_t *k = kbase + off, *v = vbase + off;
            if (dense) {
#pragma unroll
              for (int n = 0; n < 16 / kRowsOnce; ++n) {
                cp_async_whole(dst_of(h * 16 / kRowsOnce + n) + stage, k + n * kRowsOnce * D);
                cp_async_whole(dst_of(h * 16 / kRowsOnce + n) + stage + Shape::kChunkBytes, v + n * kRowsOnce * D);
              }
            } else {
#pragma unroll
              for (int n = 0; n < 16 / kRowsOnce; ++n, k += rows_on, v += rows_on) {
                cp_async_whole(dst_of(h * 16 / kRowsOnce + n) + stage, k);
                cp_async_whole(dst_of(h * 16 / kRowsOnce + n) + stage + Shape::kChunkBytes, v);
              }
            }
          }
        } else {  // the last chunk, or several pages, or none; rows that are not there read as zeros
          const int mine = j + my_row;
          int64_t off = -1, soff = 0;
          if (mine < keys) {
            if (page >= 0 && page < a.kv.pages) {
              off = int64_t(page) * a.kv.page_stride + int64_t(mine & page_mask) * a.kv.slot_stride;
              soff = int64_t(page) * args.s_page + int64_t(mine & page_mask) * args.s_slot;
            } else {
              atomicOr(a.status, kStatusBadIndex);
            }
          }
          cp_async_scales<Shape::kScaleBytes>(scale_to + stage, sbase + soff, off < 0 ? 0 : Shape::kScaleBytes);
          if constexpr (kHalves == 2) cp_async_scales<Shape::kScaleBytes>(scale_to + stage + kScaleV, sbase_v + soff, off < 0 ? 0 : Shape::kScaleBytes);
#pragma unroll
          for (int n = 0; n < kTimes; ++n) {
            const int64_t o = __shfl_sync(0xffffffffu, off, n * kRowsOnce + row0);
            cp_async16(dst_of(n) + stage, kbase + (o < 0 ? 0 : o), o < 0 ? 0 : 16);
            cp_async16(dst_of(n) + stage + Shape::kChunkBytes, vbase + (o < 0 ? 0 : o), o < 0 ? 0 : 16);
          }
        }
      }
      cp_commit();
    };
    int page[kStages];  // of the chunks that are filled next
#pragma unroll
    for (int i = 0; i < kStages; ++i) page[i] = page_of(i);
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
      fill(i, i * Shape::kStageBytes, page[i]);
      page[i] = page_of(i + kStages);
    }

    // Rows as the narrow operand: lane (g, c) loads dims 4c..4c+3 of each 16 of row g; afterwards it
    // holds scores of rows 2c and 2c+1, with these limits (keys the row may see) and scales.
    uint32_t qb[NT][kPieces][2];
    float row_scale[NT][2];
    int limit[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      int token, head;
      const bool live = row_of(a, cur, cur.m * kRows + t * 8 + g, token, head);
      const int sees = live ? keys_seen(cur.s, token - cur.s.first) : 0;
      const T* row = static_cast<const T*>(a.q) + (live ? token * a.q_token + head * a.q_head : 0) + c * 4;
      uint2 w[kPieces];
#pragma unroll
      for (int p = 0; p < kPieces; ++p) w[p] = live ? *reinterpret_cast<const uint2*>(row + p * 16) : make_uint2(0u, 0u);
      float scale = a.scale_log2;
      if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
        for (int p = 0; p < kPieces; ++p) qb[t][p][0] = __byte_perm(w[p].x, w[p].y, 0x5410), qb[t][p][1] = __byte_perm(w[p].x, w[p].y, 0x7632);
      } else {
        uint32_t top = 0;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) top = __vmaxu2(top, __vmaxu2(w[p].x & 0x7fff7fffu, w[p].y & 0x7fff7fffu));
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t e = min(max(top >> 7, 1u), 253u);  // the exponent's bits
        const float down = __uint_as_float((254u - e) << 23);
        scale = __fmul_rn(scale, __uint_as_float(e << 23));
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          float v[4];
          Elem<T>::unpack2(w[p].x, v[0], v[1]), Elem<T>::unpack2(w[p].y, v[2], v[3]);
          qb[t][p][0] = Elem<__half>::pack2(v[0] * down, v[2] * down);
          qb[t][p][1] = Elem<__half>::pack2(v[1] * down, v[3] * down);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        row_scale[t][e] = __shfl_sync(0xffffffffu, scale, (2 * c + e) * 4);
        limit[t][e] = __shfl_sync(0xffffffffu, sees, (2 * c + e) * 4);
      }
    }
    // o: dims 16 p + 2 g (0, 1) and + 1 (2, 3) of rows 2c (0, 2) and 2c + 1 (1, 3).  base: what weights are
    // relative to, the maximum in use of a visible key's score and its largest scale's logarithm.
    float o[NT][kPieces][4], base[NT][2], sum[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][p][e] = 0.f;
      base[t][0] = base[t][1] = -FLT_MAX, sum[t][0] = sum[t][1] = 0.f;
    }

    // matrices of ldmatrix: keys 0-7 and 8-15, of a block's two pieces
    const int r = (lane & 7) + (lane & 8), second = lane >> 4;
    uint32_t stage = 0;  // its offset
    uint32_t at_k[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) at_k[b] = ring + r * Shape::kRowBytes + (place(2 * b + second, r) << 4);
    const unsigned char* my_scales = my_ring + 2 * Shape::kChunkBytes + g * Shape::kScaleBytes;
    for (int i = 0; i < take; ++i) {
      cp_wait<kStages - 1>();
      __syncwarp();
      const unsigned char* scales = my_scales + stage;
      // s: keys g (0, 1) and g + 8 (2, 3) of each 16 by rows 2c (0, 2) and 2c + 1 (1, 3)
      float s[kHalves][NT][4];
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        uint32_t d0[kWords], d8[kWords];
        scales_of(scales + h * 16 * Shape::kScaleBytes, d0);
        scales_of(scales + (h * 16 + 8) * Shape::kScaleBytes, d8);
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          uint32_t w[4];
          ldsm4(at_k[b] + stage + h * 16 * Shape::kRowBytes, w);
          float part[NT][4];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint32_t k[4] = {quants(w[2 * p]), quants(w[2 * p + 1]), quants(w[2 * p] >> 8), quants(w[2 * p + 1] >> 8)};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              if (p == 0)
                mma_f16_new(part[t], k, qb[t][2 * b][0], qb[t][2 * b][1]);
              else
                mma_f16(part[t], k, qb[t][2 * b + 1][0], qb[t][2 * b + 1][1]);
            }
          }
          if (b % 2 == 0) d0[b / 2] = no_infinity(d0[b / 2]), d8[b / 2] = no_infinity(d8[b / 2]);
          float e0, e8, unused;
          if (b % 2 == 0)
            Elem<__half>::unpack2(d0[b / 2], e0, unused), Elem<__half>::unpack2(d8[b / 2], e8, unused);
          else
            Elem<__half>::unpack2(d0[b / 2], unused, e0), Elem<__half>::unpack2(d8[b / 2], unused, e8);
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              s[h][t][e] = b == 0 ? part[t][e] * (e < 2 ? e0 : e8) : __fmaf_rn(part[t][e], e < 2 ? e0 : e8, s[h][t][e]);
        }
      }
      uint32_t d0[kHalves][kWords], d8[kHalves][kWords];
      float up[kHalves][2];  // log2 of the largest scales of keys g and g + 8
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        scales_of(scales + kScaleV + h * 16 * Shape::kScaleBytes, d0[h]);
        scales_of(scales + kScaleV + (h * 16 + 8) * Shape::kScaleBytes, d8[h]);
        up[h][0] = log2_largest(d0[h]), up[h][1] = log2_largest(d8[h]);
      }
      // Scores to log2 units; keys a row may not see drop out by selection.
      const int j = j0 + i * kUnit + g;
      const bool partial_view = j - g + kChunk > of_all;
      bool grown = false;
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[h][t][e] *= row_scale[t][e & 1];
      if (partial_view) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (j + h * 16 + (e >> 1) * 8 >= limit[t][e & 1]) s[h][t][e] = -INFINITY;
      }
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) grown |= s[h][t][e] - base[t][e & 1] > kGrow8 - up[h][e >> 1];
      if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = fmaxf(s[0][t][e] + up[0][0], s[0][t][e + 2] + up[0][1]);
            if constexpr (kHalves == 2) m = fmaxf(m, fmaxf(s[kHalves - 1][t][e] + up[kHalves - 1][0], s[kHalves - 1][t][e + 2] + up[kHalves - 1][1]));
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            const float to = fmaxf(m, base[t][e]);
            f[e] = ex2(base[t][e] - to);
            base[t][e] = to;
            sum[t][e] *= f[e];
          }
#pragma unroll
          for (int p = 0; p < kPieces; ++p) o[t][p][0] *= f[0], o[t][p][1] *= f[1], o[t][p][2] *= f[0], o[t][p][3] *= f[1];
        }
      }
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[h][t][e] = ex2(s[h][t][e] - base[t][e & 1]);
            sum[t][e & 1] += s[h][t][e];
          }
      // A scale that is no number must not reach, as 0 * inf, the rows that may not see its key.
      bool careful = false;
      if (partial_view) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
          for (int k = 0; k < kWords; ++k)
            careful |= no_number<__half>(d0[h][k]) || no_number<__half>(d0[h][k] >> 16) || no_number<__half>(d8[h][k]) || no_number<__half>(d8[h][k] >> 16);
        careful = __any_sync(0xffffffffu, careful);
      }
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          uint32_t w[4];
          ldsm4t(at_k[b] + stage + Shape::kChunkBytes + h * 16 * Shape::kRowBytes, w);
          float e0, e8, unused;
          if (b % 2 == 0)
            Elem<__half>::unpack2(d0[h][b / 2], e0, unused), Elem<__half>::unpack2(d8[h][b / 2], e8, unused);
          else
            Elem<__half>::unpack2(d0[h][b / 2], unused, e0), Elem<__half>::unpack2(d8[h][b / 2], unused, e8);
          uint32_t pt[NT][2];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float p[4] = {s[h][t][0] * e0, s[h][t][1] * e0, s[h][t][2] * e8, s[h][t][3] * e8};
            if (careful) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (j + h * 16 + (e >> 1) * 8 >= limit[t][e & 1]) p[e] = 0.f;
            }
            pt[t][0] = transposed(Elem<__half>::pack2(p[0], p[1]));
            pt[t][1] = transposed(Elem<__half>::pack2(p[2], p[3]));
          }
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint32_t v[4] = {quants(w[2 * p]), quants(w[2 * p] >> 8), quants(w[2 * p + 1]), quants(w[2 * p + 1] >> 8)};
#pragma unroll
            for (int t = 0; t < NT; ++t) mma_f16(o[t][2 * b + p], v, pt[t][0], pt[t][1]);
          }
        }
      __syncwarp();
      fill(i + kStages, stage, page[0]);
      stage = stage == (kStages - 1) * Shape::kStageBytes ? 0 : stage + Shape::kStageBytes;
#pragma unroll
      for (int k = 0; k < kStages - 1; ++k) page[k] = page[k + 1];
      page[kStages - 1] = page_of(i + 2 * kStages);
    }
    cp_wait<0>();

    // Join the warps: their maxima and sums, then their outputs (f32 over the
    // ring, which is drained) scaled to the common maximum.
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) sum[t][e] += __shfl_xor_sync(0xffffffffu, sum[t][e], off);
        if (g == 0) ml[warp][t * 8 + 2 * c + e][0] = base[t][e], ml[warp][t * 8 + 2 * c + e][1] = sum[t][e];
      }
    __syncthreads();
    float* joined = reinterpret_cast<float*>(smem);  // [warp][kRows][D + 4]
    constexpr int kLd = D + 4;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = t * 8 + 2 * c + e;
        float m = ml[0][row][0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) m = fmaxf(m, ml[w][row][0]);
        const float f = ex2(base[t][e] - m);
#pragma unroll
        for (int p = 0; p < kPieces; ++p)
          *reinterpret_cast<float2*>(joined + (warp * kRows + row) * kLd + p * 16 + 2 * g) = make_float2(o[t][p][e] * f, o[t][p][e + 2] * f);
      }
    __syncthreads();
    const bool whole = cur.unit == 0 && take == cur.units;
    if (!kCluster && threadIdx.x == 0 && cur.unit == 0 && !whole) leave_join(a, cur, u, total, ctas);
    float* part = partial<kRows, D>(a, blockIdx.x, cur.unit == 0);
    for (int i = threadIdx.x; i < kRows * (D / 4); i += kWarps * 32) {
      const int row = i / (D / 4), col = i % (D / 4) * 4;
      int token, head;
      if (!row_of(a, cur, cur.m * kRows + row, token, head)) continue;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      float m = -FLT_MAX, l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 t = *reinterpret_cast<const float4*>(joined + (w * kRows + row) * kLd + col);
        v.x += t.x, v.y += t.y, v.z += t.z, v.w += t.w;
        m = fmaxf(m, ml[w][row][0]);
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (ml[w][row][1] != 0.f) l += ml[w][row][1] * ex2(ml[w][row][0] - m);
      if (kCluster) {  // in place: no other thread reads these
        *reinterpret_cast<float4*>(joined + row * kLd + col) = v;
        if (col == 0) own[row] = make_float2(m, l);
      } else if (whole) {
        const float inv = inverse(l, keys_seen(cur.s, token - cur.s.first));
        const uint2 w = make_uint2(Elem<T>::pack2(v.x * inv, v.y * inv), Elem<T>::pack2(v.z * inv, v.w * inv));
        *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + token * a.o_token + head * a.o_head + col) = w;
      } else {
        *reinterpret_cast<float4*>(part + row * D + col) = v;
        if (col == 0) part[kRows * D + row] = m, part[kRows * (D + 1) + row] = l;
      }
    }
    if constexpr (kCluster) {
      // Thread p of every ctas threads reads CTA p's part of four columns of a row.
      cg::cluster_group cluster = cg::this_cluster();
      cluster.sync();
      const int rows = min(kRows, cur.s.count * a.group - cur.m * kRows), values = rows * (D / 4);
      const int p = int(threadIdx.x) % ctas, per = kWarps * 32 / ctas;
      for (int e0 = int(blockIdx.x) % ctas * per; e0 < values; e0 += kWarps * 32) {
        const int e = e0 + int(threadIdx.x) / ctas, row = e / (D / 4), col = e % (D / 4) * 4;
        float2 his = make_float2(-FLT_MAX, 0.f);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (e < values) {
          his = *cluster.map_shared_rank(own + row, p);
          v = *reinterpret_cast<const float4*>(cluster.map_shared_rank(joined + row * kLd + col, p));
        }
        float m = his.x;
        for (int off = 1; off < ctas; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        const float f = his.y != 0.f ? ex2(his.x - m) : 0.f;  // a sum that is NaN counts
        float l = his.y * f;
        v.x *= f, v.y *= f, v.z *= f, v.w *= f;
        for (int off = 1; off < ctas; off <<= 1) {
          l += __shfl_xor_sync(0xffffffffu, l, off);
          v.x += __shfl_xor_sync(0xffffffffu, v.x, off), v.y += __shfl_xor_sync(0xffffffffu, v.y, off);
          v.z += __shfl_xor_sync(0xffffffffu, v.z, off), v.w += __shfl_xor_sync(0xffffffffu, v.w, off);
        }
        int token, head;
        if (p == 0 && e < values && row_of(a, cur, cur.m * kRows + row, token, head)) {
          const float inv = inverse(l, keys_seen(cur.s, token - cur.s.first));
          const uint2 w = make_uint2(Elem<T>::pack2(v.x * inv, v.y * inv), Elem<T>::pack2(v.z * inv, v.w * inv));
          *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + token * a.o_token + head * a.o_head + col) = w;
        }
      }
      cluster.sync();  // the parts have been read
      u += a.tiles;
    } else {
      __syncthreads();  // the ring and ml are free again
      u += take;
      if (u < u1) next_item<Tile>(a, cur);
    }
  }
  if (a.beside) pdl_wait();  // what follows waits for this launch, and with it for the one before
}

// Which kernel, from the rows a key head at most (new tokens times the group), where clusters do not take the call.
static bool many_rows8(int64_t max_new, int64_t group, bool one) { return max_new > (one ? 32 : 64) / group; }

// Where the work is split by shares of the axis, chunks are of 32 keys: two independent streams of
// instructions, and half the votes and waits (64 sequences of 16 heads over 8 of 64, 8000 keys at most: 61 us, 68 with 16;
// 16 x 64 heads over 8 of 128, 4000: 25.8 and 29.2; 64 x 32 over 8, 16384: 176 and 178; 16 x 12 tokens of 32 over 8, f16,
// 4000: 50 and 55).
template <int D, int NT>
using ShareShape = Shape8<D, NT, kWarps8, 2>;
template <int D>
static int64_t few_workspace8() {
  return std::max(attend_workspace(ShareShape<D, 1>::kCtas * num_sms(), 8, D), attend_workspace(ShareShape<D, 2>::kCtas * num_sms(), 16, D));
}
static int64_t few_workspace8(int dim) { return dim == 64 ? few_workspace8<64>() : few_workspace8<128>(); }

// The CTAs of a cluster for each sequence, key head and tile, which joins its
// own parts; 0: shares of the axis and a join, or the tensor-core kernel.  As in
// attend.cu: all clusters run at once, CTAs a cluster until each has two units at most, then as many as fit, up to
// ten units each (32 heads over 8 of 128, one token over 8191 keys: 11.8 us with clusters, 12.7
// by shares; over 16384: 18.3 and 15.7; 4 sequences of 4000: 13.0 and 14.5, of 8191: 17.0 and 16.9).
constexpr int kMostUnits8 = 10;
template <class T, int D, int NT>
static int attend8_cluster(Attend8Args& g, int64_t max_new, int dev, const char* who, int& ctas, int& warps) {
  AttendArgs& a = g.a;
  constexpr int kRows = 8 * NT;
  ctas = 0, warps = kWarps8;
  const int units = (a.kv.table_tokens + kKeys8 - 1) / kKeys8;
  a.tiles = int(std::min<int64_t>((max_new * a.group + kRows - 1) / kRows, 1024));
  const int64_t clusters = int64_t(a.kv.batch) * a.kv.kv_heads * a.tiles;
  if (units <= kWhole8 && !many_rows8(max_new, a.group, a.kv.batch == 1)) return Q1_OK;
  static int most[64][4] = {};  // clusters of 4, 8, 16 CTAs that run at once, and of 16 with twice the warps
  for (int i = 0; i < 4; ++i) {
    int once = dev >= 0 && dev < 64 ? most[dev][i] : 0;
    if (!once) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr = {};
      const int size = i < 3 ? 4 << i : 16;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = unsigned(size), attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.gridDim = dim3(unsigned(size)), cfg.blockDim = dim3((i < 3 ? 1 : 2) * kWarps8 * 32);
      cfg.dynamicSmemBytes = i < 3 ? Shape8<D, NT>::kSmem : Shape8<D, NT, 2 * kWarps8>::kSmem;
      cfg.attrs = &attr, cfg.numAttrs = 1;
      const cudaError_t e = i < 3 ? cudaOccupancyMaxActiveClusters(&once, k_attend_q8<T, D, NT, true>, &cfg)
                                  : cudaOccupancyMaxActiveClusters(&once, k_attend_q8<T, D, NT, true, 2 * kWarps8>, &cfg);
      if (int r = cuda_status(e, who)) return r;
      if (dev >= 0 && dev < 64) most[dev][i] = once;
    }
    if (clusters > once) break;
    if (i == 3) {
      warps = 2 * kWarps8;
      break;
    }
    ctas = 4 << i;
    if (units <= 2 * ctas) break;
  }
  if (units > kMostUnits8 * ctas * (warps / kWarps8)) ctas = 0;
  return Q1_OK;
}

template <class T, int D, int NT>
static int launch_attend8(Attend8Args& g, int64_t max_new, bool only_clusters, void* workspace, cudaStream_t s, bool& ran,
                          const AttendArgs* many) {
  using Shape = Shape8<D, NT>;
  using Wide = Shape8<D, NT, 2 * kWarps8>;
  using Share = ShareShape<D, NT>;
  const auto by_shares = k_attend_q8<T, D, NT, false, kWarps8, 2>;
  const char* who = "q1_paged_attention_q8 launch";
  AttendArgs& a = g.a;
  static bool set[64] = {};
  int dev = 0;
  if (int e = cuda_status(cudaGetDevice(&dev), who)) return e;
  if (dev < 0 || dev >= 64 || !set[dev]) {
    const auto most = cudaFuncAttributeMaxDynamicSharedMemorySize;
    if (int e = cuda_status(cudaFuncSetAttribute(by_shares, most, Share::kSmem), who)) return e;
    if (int e = cuda_status(cudaFuncSetAttribute(k_attend_q8<T, D, NT, true>, most, Shape::kSmem), who)) return e;
    if (int e = cuda_status(cudaFuncSetAttribute(k_attend_q8<T, D, NT, true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1), who))
      return e;
    if (int e = cuda_status(cudaFuncSetAttribute(k_attend_q8<T, D, NT, true, 2 * kWarps8>, most, Wide::kSmem), who)) return e;
    if (int e = cuda_status(cudaFuncSetAttribute(k_attend_q8<T, D, NT, true, 2 * kWarps8>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1), who))
      return e;
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  int ctas = 0, warps = kWarps8;
  if (only_clusters)
    if (int e = attend8_cluster<T, D, NT>(g, max_new, dev, who, ctas, warps)) return e;
  ran = ctas || !only_clusters;
  if (!ran) return Q1_OK;
  a.ctas = ctas;
  if (ctas) {
    const dim3 grid(unsigned(a.kv.batch * a.kv.kv_heads * a.tiles * ctas));
    if (warps > kWarps8)
      return launch_op<Attend8Args>(k_attend_q8<T, D, NT, true, 2 * kWarps8>, grid, 2 * kWarps8 * 32, Wide::kSmem, ctas, s, who, g);
    return launch_op<Attend8Args>(k_attend_q8<T, D, NT, true>, grid, kWarps8 * 32, Shape::kSmem, ctas, s, who, g);
  }
  a.ctas = Share::kCtas * num_sms();
  place_workspace(a, workspace);
  if (int e = launch_op<Attend8Args>(by_shares, dim3(unsigned(a.ctas)), kWarps8 * 32, Share::kSmem, 1, s, who, g)) return e;
  // No item has more units than stay whole: nothing to join.
  if (a.kv.table_tokens <= kWhole8 * kKeys8) return Q1_OK;
  if (many && many->ctas)
    return launch_op<JoinBoth>(k_attend_join_both<T, Shape::kRows, D>, dim3(unsigned(many->ctas * kTcJoinSlices + a.ctas * kJoinSlices)),
                               kJoinThreads, 0, 1, s, who, {*many, a});
  return launch_op(k_attend_join<T, Shape::kRows, D, false>, dim3(unsigned(a.ctas), kJoinSlices), kJoinThreads, 0, 1, s, who, a);
}

// The f16 copy of one sequence: pages of 128 tokens, keys and values in one or two parts, its
// table's entries, its factors and their making.
static int64_t copy_pages(int64_t table_tokens) { return (table_tokens + 127) / 128; }
static int copy_parts(int dtype) { return dtype == Q1_BF16 ? 1 : 2; }
static int64_t copy_bytes(int64_t pages, int64_t kv_heads, int64_t dim, int parts) {
  return pages * (2 * parts * kv_heads * 128 * dim * 2 + 16) + kv_heads * 2 * (4 + 4 * kTopSlices) + 16;
}

}  // namespace q1

using namespace q1;

extern "C" int64_t q1_paged_attention_q8_workspace(int64_t max_new, int64_t heads, int64_t kv_heads, int64_t dim,
                                                   int dtype, int64_t table_tokens, int64_t sequences) {
  if (dtype != Q1_BF16 && dtype != Q1_F16) return fail(Q1_ERR_ARG, "q1_paged_attention_q8_workspace: bad type %d", dtype);
  if (max_new < 1 || heads < 1 || kv_heads < 1 || heads > 4096 || heads % kv_heads || (dim != 64 && dim != 128) || table_tokens < 1 ||
      table_tokens > (int64_t(1) << 42) || sequences < 1 || sequences > (1 << 20))
    return fail(Q1_ERR_ARG, "q1_paged_attention_q8_workspace: bad shape max_new=%lld heads=%lld kv_heads=%lld dim=%lld table_tokens=%lld "
                            "sequences=%lld", (long long)max_new, (long long)heads, (long long)kv_heads, (long long)dim,
                (long long)table_tokens, (long long)sequences);
  const int64_t few = few_workspace8(int(dim));
  if (!many_rows8(max_new, heads / kv_heads, true)) return few;
  const int64_t pages = copy_pages(std::min<int64_t>(table_tokens, int64_t(1) << 30)), one = copy_bytes(pages, kv_heads, dim, copy_parts(dtype));
  if (one > (int64_t(1) << 62) / sequences)
    return fail(Q1_ERR_ARG, "q1_paged_attention_q8_workspace: bad shape, %lld sequences of %lld tokens are too much", (long long)sequences,
                (long long)table_tokens);
  return few + attend_tc_workspace(int(dim)) + sequences * one;  // a call may run both kernels
}

extern "C" int q1_paged_attention_q8(const void* q, int64_t q_token_stride, int64_t q_head_stride, int64_t heads, float scale,
                                     int dtype, const q1_paged_q8* kv, int64_t max_new, void* out, int64_t out_token_stride,
                                     int64_t out_head_stride, void* workspace, int64_t workspace_bytes, void* stream) {
  const char* who = "q1_paged_attention_q8";
  Paged8 p = {};
  if (int e = check_paged_q8(who, kv, p)) return e;
  if (dtype != Q1_BF16 && dtype != Q1_F16) return fail(Q1_ERR_ARG, "%s: bad type %d", who, dtype);
  if (heads < 1 || heads > 4096 || heads % kv->kv_heads)
    return fail(Q1_ERR_ARG, "%s: heads=%lld is no multiple of kv_heads=%lld up to 4096", who, (long long)heads,
                (long long)kv->kv_heads);
  if (int64_t(p.kv.total_new) * (heads / kv->kv_heads) >= (int64_t(1) << 31))
    return fail(Q1_ERR_ARG, "%s: %lld new tokens of %lld heads a key head are 2^31 rows or more", who, (long long)kv->total_new,
                (long long)(heads / kv->kv_heads));
  if (!q || !out || !workspace) return fail(Q1_ERR_ARG, "%s: null pointer", who);
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || q_token_stride % 8 || q_head_stride % 8 ||
      out_token_stride % 8 || out_head_stride % 8)
    return fail(Q1_ERR_ARG, "%s: buffers must be 16-byte aligned, strides multiples of 8", who);
  if (q_head_stride < kv->dim || q_token_stride < kv->dim || out_head_stride < kv->dim || out_token_stride < kv->dim)
    return fail(Q1_ERR_ARG, "%s: a stride is less than dim", who);
  if (!std::isfinite(scale * 1.4426950408889634f)) return fail(Q1_ERR_ARG, "%s: scale must be finite", who);
  if (max_new < 1) return fail(Q1_ERR_ARG, "%s: max_new must be positive", who);
  const int64_t table_tokens = kv->table_width * kv->page_size;
  const int64_t need = q1_paged_attention_q8_workspace(max_new, heads, kv->kv_heads, kv->dim, dtype, table_tokens, 1);
  if (need < 0) return int(need);
  if (workspace_bytes < need)
    return fail(Q1_ERR_ARG, "%s: the workspace holds %lld bytes, %lld are needed", who, (long long)workspace_bytes,
                (long long)need);
  Attend8Args g = {};
  AttendArgs& a = g.a;
  a.kv = p.kv;
  g.ks = p.ks, g.vs = p.vs, g.s_page = p.s_page, g.s_slot = p.s_slot, g.s_head = p.s_head;
  a.q = q, a.out = out, a.q_token = q_token_stride, a.q_head = q_head_stride;
  a.o_token = out_token_stride, a.o_head = out_head_stride;
  if (int e = ops_status_ptr(&a.status)) return e;
  const bool sized = many_rows8(max_new, heads / kv->kv_heads, true);  // the workspace has room for the copies
  max_new = std::min<int64_t>(max_new, a.kv.total_new);
  a.heads = int(heads), a.group = int(heads / kv->kv_heads);
  a.group_inverse = uint32_t((uint64_t(1) << 32) / uint64_t(a.group) + 1);
  a.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf = dtype == Q1_BF16;
  a.least_rows = 0, a.most_rows = INT_MAX;
  bool ran = false;
  const auto few = [&](bool only_clusters, bool narrow, const AttendArgs* many = nullptr) {
    const auto as = [&](auto type, auto dim) {
      using T = decltype(type);
      constexpr int D = decltype(dim)::value;
      return narrow ? launch_attend8<T, D, 1>(g, max_new, only_clusters, workspace, s, ran, many)
                    : launch_attend8<T, D, 2>(g, max_new, only_clusters, workspace, s, ran, many);
    };
    if (kv->dim == 128)
      return bf ? as(__nv_bfloat16(), std::integral_constant<int, 128>()) : as(__half(), std::integral_constant<int, 128>());
    return bf ? as(__nv_bfloat16(), std::integral_constant<int, 64>()) : as(__half(), std::integral_constant<int, 64>());
  };
  const bool narrow = max_new * a.group <= 8;
  if (int e = few(true, narrow)) return e;
  if (ran) return Q1_OK;
  if (!sized || !many_rows8(max_new, a.group, kv->batch == 1)) return few(false, narrow);

  // As many sequences at a time as the workspace has room for; those of one tile at most among
  // several go to the kernel for few rows, beside the last launch of the other.
  const int64_t pages = copy_pages(a.kv.table_tokens), one = copy_bytes(pages, kv->kv_heads, kv->dim, copy_parts(dtype));
  char* tc_space = static_cast<char*>(workspace) + few_workspace8(int(kv->dim));
  char* copies = tc_space + attend_tc_workspace(int(kv->dim));
  const int64_t fit = (workspace_bytes - (copies - static_cast<char*>(workspace))) / one;
  const int at_once = int(std::min<int64_t>({fit, kv->batch, 65535, (int64_t(1) << 30) / pages}));
  const int64_t tensor = int64_t(at_once) * pages * kv->kv_heads * 128 * kv->dim * copy_parts(dtype);  // values
  const bool both = kv->batch > 1;
  constexpr int kFewRows = 16;
  AttendArgs many = {};
  for (int b0 = 0; b0 < a.kv.batch; b0 += at_once) {
    const int count = std::min(at_once, a.kv.batch - b0);
    CopyQ8 c = {};
    c.p = p;
    c.p.kv.table += b0 * p.kv.table_stride, c.p.kv.kv_len += b0, c.p.kv.new_start += b0, c.p.kv.batch = count;
    c.k = reinterpret_cast<__half*>(copies), c.v = c.k + tensor;
    c.table = reinterpret_cast<int32_t*>(c.v + tensor);
    c.tops = reinterpret_cast<uint32_t*>(c.table + at_once * pages);
    c.factors = reinterpret_cast<float*>(c.tops + int64_t(at_once) * kv->kv_heads * 2 * kTopSlices);
    c.status = a.status, c.pages = int(pages), c.parts = copy_parts(dtype);
    c.dim = int(kv->dim), c.group = a.group, c.least_rows = both ? kFewRows + 1 : 1;
    if (int e = launch_copy_q8(c, s)) return e;
    AttendArgs t = a;
    t.kv = c.p.kv;
    t.kv.k = c.k, t.kv.v = c.v;
    t.kv.slot_stride = kv->dim, t.kv.head_stride = 128 * kv->dim, t.kv.page_stride = kv->kv_heads * 128 * kv->dim;
    t.kv.table = c.table, t.kv.table_stride = pages, t.kv.pages = int(pages * count), t.kv.page_shift = 7;
    if (both) t.least_rows = kFewRows + 1;
    const bool last = b0 + count == a.kv.batch;
    if (int e = launch_attend_tc(t, tc_space, bf, int(kv->dim), s, ran, both && last ? &many : nullptr, c.factors)) return e;
    if (!ran) return fail(Q1_ERR_CUDA, "%s: no tensor map for the workspace", who);
  }
  if (!both) return Q1_OK;
  a.most_rows = kFewRows, a.beside = true;
  return few(false, false, &many);
}
