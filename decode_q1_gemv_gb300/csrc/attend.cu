// attend.cu -- q1_paged_attention: new tokens attend to their sequence's paged
// cache, causal, grouped heads.  This file holds the kernel for few rows a key
// head (single tokens and short chunks) and the entry points.
//
// For row r at position p: o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m) over
// keys j <= p, s_j = scale log2(e) q.k_j, m the running maximum.  Keys and values
// are read once in one pass; with up to 16 rows that is 2 D bytes and at most
// 64 D operations a key and row tile, so bytes bound it: what counts is reads in
// flight and equal shares for the SMs.  Each warp takes chunks of 16 keys on
// its own: a private ring of kStages chunks in shared memory filled by 16-byte
// asynchronous copies, scores and p v by m16n8k16 MMAs (16-bit operands, f32
// sums), maximum, sum and output in registers, no barrier between warps until
// an item ends.  p is rounded to the cache's type for its product with v (off
// by 2^-8 or 2^-11 of a term at most, as the output's own rounding is, or, f16
// below 2^-14, by 2^-25 of the largest weight's); the sum of p is taken in f32
// before that.  The MMAs cut their sums, not round them: over 16384 keys, a
// thousand MMAs on one accumulator, by 2^-13 at most; equal values of one sign
// come out as they went in, in both types.
//
// Rows past 16 are further tiles (their keys come from L2) up to where the
// tensor-core kernel is faster, see attend_cluster and many_rows.  96 KB of ring a CTA (D = 128) and
// two CTAs an SM hold 29 MB of reads in flight.
//
// Measured (32 heads over 8 key heads of 128, bf16): one token of each of 64
// sequences, 2.04 GB of keys and values, 312 us: 6.5 TB/s, 0.98 of the copy
// bandwidth; one token over 8191 keys, 34 MB, 11.8 us with its join (5.0 at that
// bandwidth: finding the share, the pages and the join's launch are the rest).
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include <cooperative_groups.h>

#include "attend.cuh"

namespace q1 {

namespace cg = cooperative_groups;

constexpr int kRowsS = 16;   // rows of a tile
constexpr int kKeysS = 64;   // keys of a unit: 16 for each warp
constexpr int kWarpsS = 4;
// Units of an item that is not split (30 tokens over up to 909 keys: 7.2 us with
// 2, 8.0 with 4, 9.8 with 8; two short prompts 22.8, 23.6, 22.0).
constexpr int kWholeS = 2;
constexpr int kStagesS = 3;  // 2 x 96 KB of reads in flight an SM at D = 128

template <class T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

template <int D>
constexpr int attend_smem() {
  return kWarpsS * kStagesS * 2 * 16 * D * 2;
}

// kCluster: not shares of the axis but a cluster of a.ctas CTAs for each sequence,
// key head and tile (of a.tiles a key head; more are taken in turn), each with its share of the units, which joins its parts through
// distributed shared memory: no cursor to find, no second launch.
template <class T, int D, bool kCluster>
__global__ void __launch_bounds__(kWarpsS * 32) k_attend(AttendArgs a) {
  using Tile = Tiling<kRowsS, kKeysS>;
  constexpr int kRowBytes = D * 2, kChunkBytes = 16 * kRowBytes, kPieces = kRowBytes / 16;  // 16-byte pieces of a row
  constexpr int kSteps = D / 16;       // k16 steps of q.k, and pairs of n8 tiles of p v
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ LocateScratch scratch;
  __shared__ float ml[kWarpsS][16][2];
  __shared__ float2 own[kRowsS];  // kCluster: the CTA's maxima and sums
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    total = locate<Tile, kWholeS>(a, blockIdx.x, ctas, scratch, cur, u0, u1);
    if (threadIdx.x == 0) a.joins[blockIdx.x].parts = 0;
  }
  const uint32_t ring = smem_addr(smem) + warp * (kStagesS * 2 * kChunkBytes);
  const int page_mask = (1 << a.kv.page_shift) - 1;
  for (int64_t u = u0; u < u1;) {
    int take = 0;  // units of this item here
    if constexpr (kCluster) {
      const int c = int(blockIdx.x) % ctas;
      cur.m = int(u), cur.units = Tile::units(a, cur.s, cur.m);
      cur.unit = int(share(cur.units, c, ctas)), take = int(share(cur.units, c + 1, ctas)) - cur.unit;
    } else {
      take = int(min(int64_t(cur.units - cur.unit), u1 - u));
    }
    const int keys = Tile::keys(a, cur.s, cur.m), of_all = Tile::keys_of_all(a, cur.s, cur.m);
    const int32_t* table = a.kv.table + cur.b * a.kv.table_stride;
    const T* kbase = static_cast<const T*>(a.kv.k) + cur.h * a.kv.head_stride;
    const T* vbase = static_cast<const T*>(a.kv.v) + cur.h * a.kv.head_stride;

    // Chunk i of this warp: keys j0 + 64 i .. +15.  Lane l < 16 finds row l's
    // place (its page well before it is needed); the copies then run over
    // rows in pairs (or fours, D = 64).
    const int j0 = cur.unit * kKeysS + warp * 16;
    const auto page_of = [&](int i) {  // of this lane's row; -1 past the keys
      const int j = j0 + i * kKeysS + (lane & 15);
      return i < take && j < keys ? table[j >> a.kv.page_shift] : -1;
    };
    const auto fill = [&](int i, int page) {
      if (i < take) {
        const int j = j0 + i * kKeysS + (lane & 15);
        int64_t off = -1;
        if (j < keys) {
          if (page >= 0 && page < a.kv.pages)
            off = int64_t(page) * a.kv.page_stride + int64_t(j & page_mask) * a.kv.slot_stride;
          else
            atomicOr(a.status, kStatusBadIndex);
        }
        constexpr int kRowsOnce = 32 / kPieces;
        const int piece = lane % kPieces;
#pragma unroll
        for (int r0 = 0; r0 < 16; r0 += kRowsOnce) {
          const int r = r0 + lane / kPieces;
          const int64_t o = __shfl_sync(0xffffffffu, off, r);
          const uint32_t dst = ring + (i % kStagesS) * 2 * kChunkBytes + r * kRowBytes + ((piece ^ (r & 7)) << 4);
          const int64_t e = (o < 0 ? 0 : o) + piece * 8;  // rows that are not there read as zeros
          cp_async16(dst, kbase + e, o < 0 ? 0 : 16);
          cp_async16(dst + kChunkBytes, vbase + e, o < 0 ? 0 : 16);
        }
      }
      cp_commit();
    };
    int page[kStagesS];  // of the chunks that are filled next
#pragma unroll
    for (int i = 0; i < kStagesS; ++i) page[i] = page_of(i);
#pragma unroll
    for (int i = 0; i < kStagesS; ++i) {
      fill(i, page[i]);
      page[i] = page_of(i + kStagesS);
    }

    // Q of the tile as A fragments: rows lane/4 and lane/4 + 8.
    uint32_t qa[kSteps][4];
    int limit[2];  // keys each of the two rows may see
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      int token, head;
      const int r = cur.m * kRowsS + lane / 4 + half * 8;
      const bool live = row_of(a, cur, r, token, head);
      limit[half] = live ? cur.s.len - cur.s.count + (token - cur.s.first) + 1 : 0;
      const T* row = static_cast<const T*>(a.q) + (live ? token * a.q_token + head * a.q_head : 0) + (lane & 3) * 2;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        qa[k][half] = live ? *reinterpret_cast<const uint32_t*>(row + k * 16) : 0u;
        qa[k][half + 2] = live ? *reinterpret_cast<const uint32_t*>(row + k * 16 + 8) : 0u;
      }
    }
    float o[2 * kSteps][4], mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2 * kSteps; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;

    for (int i = 0; i < take; ++i) {
      cp_wait<kStagesS - 1>();
      __syncwarp();
      const uint32_t kt = ring + (i % kStagesS) * 2 * kChunkBytes, vt = kt + kChunkBytes;
      // Even and odd steps apart: chains of four (D = 64: of four as it is; 26 pairs over 3140
      // keys 15.4 -> 15.0 us, 54 x 6 over 7793 35.3 -> 34.2).
      constexpr bool kApart = D == 128;
      float s[2][4] = {}, odd[2][4] = {};
      {
        // matrices: keys 0-7 and 8-15, each with the step's two groups of 8 dims
        const int r = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t b[4];
          ldsm4(kt + r * kRowBytes + (((k * 2 + ((lane >> 3) & 1)) ^ (r & 7)) << 4), b);
          mma16816<T>(kApart && (k & 1) ? odd[0] : s[0], qa[k], b[0], b[1]);
          mma16816<T>(kApart && (k & 1) ? odd[1] : s[1], qa[k], b[2], b[3]);
        }
      }
      // Scores to log2 units; keys a row may not see drop out by selection.
      const int j = j0 + i * kKeysS + (lane & 3) * 2;
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (kApart) s[t][e] += odd[t][e];
          s[t][e] = j + t * 8 + (e & 1) < limit[e >> 1] ? s[t][e] * a.scale_log2 : -INFINITY;
          top[e >> 1] = fmaxf(top[e >> 1], s[t][e]);
        }
      float base[2];
      bool grown = false;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float m = fmaxf(mx[half], quad_max(top[half]));
        base[half] = m == -INFINITY ? 0.f : m;  // a row that sees nothing yet
        if (m > mx[half]) {
          grown = true;
          const float f = ex2(mx[half] - base[half]);
          sum[half] *= f;
          top[half] = f;
        } else {
          top[half] = 1.f;
        }
        mx[half] = m;
      }
      if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
        for (int n = 0; n < 2 * kSteps; ++n) o[n][0] *= top[0], o[n][1] *= top[0], o[n][2] *= top[1], o[n][3] *= top[1];
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[t][e] = ex2(s[t][e] - base[e >> 1]);
          sum[e >> 1] += s[t][e];
        }
      const uint32_t p[4] = {Elem<T>::pack2(s[0][0], s[0][1]), Elem<T>::pack2(s[0][2], s[0][3]),
                             Elem<T>::pack2(s[1][0], s[1][1]), Elem<T>::pack2(s[1][2], s[1][3])};
      if (min(j0 + i * kKeysS + 16, keys) > of_all) {  // some rows may not see all of these keys
        unsigned char* values = smem + (vt - smem_addr(smem));
        NoNumbers<T> none;
#pragma unroll
        for (int e = 0; e < 16 * kPieces; e += 32) none.look(reinterpret_cast<const uint4*>(values)[e + lane]);
        if (__any_sync(0xffffffffu, none.found())) {
#pragma unroll 1
          for (int r = 0; r < 16; ++r)
#pragma unroll
            for (int n = 0; n < 2 * kSteps; ++n) {
              const uint32_t v = *reinterpret_cast<const uint32_t*>(values + r * kRowBytes + ((n ^ (r & 7)) << 4) + (lane & 3) * 4);
#pragma unroll
              for (int half = 0; half < 2; ++half)
                if (j0 + i * kKeysS + r < limit[half]) add_no_numbers<T>(v, o[n][half * 2], o[n][half * 2 + 1]);
            }
          __syncwarp();
          for (int e = lane; e < 16 * kPieces; e += 32) {
            uint4& v = reinterpret_cast<uint4*>(values)[e];
            v = numbers<T>(v);
          }
        }
        __syncwarp();
      }
      const int r = lane & 15;
#pragma unroll
      for (int n = 0; n < kSteps; ++n) {
        uint32_t b[4];
        ldsm4t(vt + r * kRowBytes + (((n * 2 + (lane >> 4)) ^ (r & 7)) << 4), b);
        mma16816<T>(o[2 * n], p, b[0], b[1]);
        mma16816<T>(o[2 * n + 1], p, b[2], b[3]);
      }
      __syncwarp();
      fill(i + kStagesS, page[0]);
#pragma unroll
      for (int k = 0; k < kStagesS - 1; ++k) page[k] = page[k + 1];
      page[kStagesS - 1] = page_of(i + 2 * kStagesS);
    }
    cp_wait<0>();

    // Join the warps: their maxima and sums, then their outputs (f32 over the
    // ring, which is drained) scaled to the common maximum.
    sum[0] = quad_sum(sum[0]);
    sum[1] = quad_sum(sum[1]);
    if ((lane & 3) == 0) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        ml[warp][lane / 4 + half * 8][0] = mx[half];
        ml[warp][lane / 4 + half * 8][1] = sum[half];
      }
    }
    __syncthreads();
    float* joined = reinterpret_cast<float*>(smem);  // [warp][16][D + 4]
    constexpr int kLd = D + 4;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = lane / 4 + half * 8;
      float m = ml[0][r][0];
#pragma unroll
      for (int w = 1; w < kWarpsS; ++w) m = fmaxf(m, ml[w][r][0]);
      const float f = mx[half] == -INFINITY ? 0.f : ex2(mx[half] - m);
#pragma unroll
      for (int n = 0; n < 2 * kSteps; ++n) {
        float2 v = make_float2(o[n][half * 2] * f, o[n][half * 2 + 1] * f);
        *reinterpret_cast<float2*>(joined + (warp * 16 + r) * kLd + n * 8 + (lane & 3) * 2) = v;
      }
    }
    __syncthreads();
    const bool whole = cur.unit == 0 && take == cur.units;
    if (!kCluster && threadIdx.x == 0 && cur.unit == 0 && !whole) leave_join(a, cur, u, total, ctas);
    float* part = partial<kRowsS, D>(a, blockIdx.x, cur.unit == 0);
    for (int i = threadIdx.x; i < 16 * (D / 4); i += kWarpsS * 32) {
      const int r = i / (D / 4), col = i % (D / 4) * 4;
      int token, head;
      if (!row_of(a, cur, cur.m * kRowsS + r, token, head)) continue;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarpsS; ++w) {
        const float4 t = *reinterpret_cast<const float4*>(joined + (w * 16 + r) * kLd + col);
        v.x += t.x, v.y += t.y, v.z += t.z, v.w += t.w;
        m = fmaxf(m, ml[w][r][0]);
      }
#pragma unroll
      for (int w = 0; w < kWarpsS; ++w)
        if (ml[w][r][1] != 0.f) l += ml[w][r][1] * ex2(ml[w][r][0] - m);
      if (kCluster) {  // in place: no other thread reads these
        *reinterpret_cast<float4*>(joined + r * kLd + col) = v;
        if (col == 0) own[r] = make_float2(m, l);
      } else if (whole) {
        const float inv = inverse(l, keys_seen(cur.s, token - cur.s.first));
        const uint2 w = make_uint2(Elem<T>::pack2(v.x * inv, v.y * inv), Elem<T>::pack2(v.z * inv, v.w * inv));
        *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + token * a.o_token + head * a.o_head + col) = w;
      } else {
        *reinterpret_cast<float4*>(part + r * D + col) = v;
        if (col == 0) part[kRowsS * D + r] = m, part[kRowsS * (D + 1) + r] = l;
      }
    }
    if constexpr (kCluster) {
      // Thread p of every ctas threads reads CTA p's part of four columns of a row.
      cg::cluster_group cluster = cg::this_cluster();
      cluster.sync();
      const int rows = min(kRowsS, cur.s.count * a.group - cur.m * kRowsS), values = rows * (D / 4);
      const int p = int(threadIdx.x) % ctas, per = kWarpsS * 32 / ctas;
      for (int e0 = int(blockIdx.x) % ctas * per; e0 < values; e0 += kWarpsS * 32) {
        const int e = e0 + int(threadIdx.x) / ctas, r = e / (D / 4), col = e % (D / 4) * 4;
        float2 his = make_float2(-INFINITY, 0.f);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (e < values) {
          his = *cluster.map_shared_rank(own + r, p);
          v = *reinterpret_cast<const float4*>(cluster.map_shared_rank(joined + r * kLd + col, p));
        }
        float m = his.x;
        for (int off = 1; off < ctas; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        const float f = his.y != 0.f ? ex2(his.x - (m == -INFINITY ? 0.f : m)) : 0.f;  // a sum that is NaN counts
        float l = his.y * f;
        v.x *= f, v.y *= f, v.z *= f, v.w *= f;
        for (int off = 1; off < ctas; off <<= 1) {
          l += __shfl_xor_sync(0xffffffffu, l, off);
          v.x += __shfl_xor_sync(0xffffffffu, v.x, off), v.y += __shfl_xor_sync(0xffffffffu, v.y, off);
          v.z += __shfl_xor_sync(0xffffffffu, v.z, off), v.w += __shfl_xor_sync(0xffffffffu, v.w, off);
        }
        int token, head;
        if (p == 0 && e < values && row_of(a, cur, cur.m * kRowsS + r, token, head)) {
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

// Where clusters do not take the call (attend_cluster): which kernel, from the
// rows a key head at most (new tokens times the group).
// One sequence: this one up to 32 rows (32 over 4000 keys: 16.4 us against 17.3;
// 64 over 8000: 26.7 against 23.4).  Several: up to 64 (8 x 64 rows over 3000
// keys: 21.2 us against 35.6; 16 x 64, mixed lengths: 26.3 against 35.8), since sequences
// of up to 16 rows among others with more are this kernel's too, in a launch
// of their own: a tile of 128 rows costs the same however few are in use.
static bool many_rows(int64_t max_new, int64_t group, bool one) { return max_new > (one ? 32 : 64) / group; }

static int attend_ctas() { return 2 * num_sms(); }

// The CTAs of a cluster for each sequence, key head and tile, which joins its
// own parts; 0: shares of the axis and a join, or the tensor-core kernel.
// Clusters want all of them to run at once and a short table: CTAs a cluster
// until each has two units at most (32 heads over 8 of 128, one token over 200 keys: 4.9
// us with 4, 6.4 with 16, 7.1 by shares; over 500: 5.6, 6.4, 7.6), then as many as
// fit up to seven units each (4000 keys: 9.0 us with 16 against 9.8; 8191: 12.2
// against 11.9; 4 sequences of 2000: 8.6 us with 8 against 12.0, of 8191: 19.9
// against 18.8).  Further rows are further tiles as long as they fit (32 heads over 8,
// 16 tokens over 1000 keys: 9.9 us, 20.0 with the tensor-core kernel; 128 tokens of 8 heads: 11.0, 20.8).
// A table of one or two units wants no join by shares either (3 sequences: 4.9 us).
template <class T, int D>
static int attend_cluster(AttendArgs& a, int64_t max_new, int dev, const char* who, int& ctas) {
  ctas = 0;
  const int units = (a.kv.table_tokens + kKeysS - 1) / kKeysS;
  a.tiles = int(std::min<int64_t>((max_new * a.group + kRowsS - 1) / kRowsS, 1024));
  if (units > 7 * 16 || (units <= kWholeS && !many_rows(max_new, a.group, a.kv.batch == 1))) return Q1_OK;
  static int most[64][3] = {};  // clusters of 4, 8, 16 CTAs that run at once
  for (int i = 0; i < 3; ++i) {
    int once = dev >= 0 && dev < 64 ? most[dev][i] : 0;
    if (!once) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr = {};
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = unsigned(4 << i), attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.gridDim = dim3(unsigned(4 << i)), cfg.blockDim = dim3(kWarpsS * 32), cfg.dynamicSmemBytes = attend_smem<D>();
      cfg.attrs = &attr, cfg.numAttrs = 1;
      if (int e = cuda_status(cudaOccupancyMaxActiveClusters(&once, k_attend<T, D, true>, &cfg), who)) return e;
      if (dev >= 0 && dev < 64) most[dev][i] = once;
    }
    if (int64_t(a.kv.batch) * a.kv.kv_heads * a.tiles > once) break;
    ctas = 4 << i;
    if (units <= 2 * ctas) break;
  }
  if (units > 7 * ctas) ctas = 0;
  return Q1_OK;
}

template <class T, int D>
static int launch_attend(AttendArgs& a, int64_t max_new, bool only_clusters, void* workspace, cudaStream_t s, bool& ran,
                         const AttendArgs* many) {
  const char* who = "q1_paged_attention launch";
  static bool set[64] = {};
  int dev = 0;
  if (int e = cuda_status(cudaGetDevice(&dev), who)) return e;
  if (dev < 0 || dev >= 64 || !set[dev]) {
    if (int e = cuda_status(cudaFuncSetAttribute(k_attend<T, D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, attend_smem<D>()),
                            who))
      return e;
    if (int e = cuda_status(cudaFuncSetAttribute(k_attend<T, D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, attend_smem<D>()),
                            who))
      return e;
    if (int e = cuda_status(cudaFuncSetAttribute(k_attend<T, D, true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1), who))
      return e;
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  int ctas = 0;
  if (only_clusters)
    if (int e = attend_cluster<T, D>(a, max_new, dev, who, ctas)) return e;
  ran = ctas || !only_clusters;
  if (!ran) return Q1_OK;
  a.ctas = ctas;
  if (ctas)
    return launch_op(k_attend<T, D, true>, dim3(unsigned(a.kv.batch * a.kv.kv_heads * a.tiles * ctas)), kWarpsS * 32, attend_smem<D>(), ctas, s,
                     who, a);
  a.ctas = attend_ctas();
  place_workspace(a, workspace);
  if (int e = launch_op(k_attend<T, D, false>, dim3(unsigned(a.ctas)), kWarpsS * 32, attend_smem<D>(), 1, s, who, a)) return e;
  // No item has more units than stay whole: nothing to join.
  if (a.kv.table_tokens <= kWholeS * kKeysS) return Q1_OK;
  if (many && many->ctas)
    return launch_op<JoinBoth>(k_attend_join_both<T, kRowsS, D>, dim3(unsigned(many->ctas * kTcJoinSlices + a.ctas * kJoinSlices)), kJoinThreads, 0, 1, s,
                               who, {*many, a});
  return launch_op(k_attend_join<T, kRowsS, D, false>, dim3(unsigned(a.ctas), kJoinSlices), kJoinThreads, 0, 1, s, who, a);
}

}  // namespace q1

using namespace q1;

extern "C" int64_t q1_paged_attention_workspace(int64_t max_new, int64_t heads, int64_t kv_heads, int64_t dim) {
  if (max_new < 1 || heads < 1 || kv_heads < 1 || heads > 4096 || heads % kv_heads || (dim != 64 && dim != 128))
    return fail(Q1_ERR_ARG, "q1_paged_attention_workspace: bad shape max_new=%lld heads=%lld kv_heads=%lld dim=%lld",
                (long long)max_new, (long long)heads, (long long)kv_heads, (long long)dim);
  const int64_t few = attend_workspace(attend_ctas(), kRowsS, int(dim));
  if (!many_rows(max_new, heads / kv_heads, true)) return few;
  return few + attend_tc_workspace(int(dim));  // a call may run both kernels
}

extern "C" int q1_paged_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, int64_t heads, float scale,
                                  const q1_paged_kv* kv, int64_t max_new, void* out, int64_t out_token_stride,
                                  int64_t out_head_stride, void* workspace, int64_t workspace_bytes, void* stream) {
  const char* who = "q1_paged_attention";
  AttendArgs a = {};
  if (int e = check_paged(who, kv, a.kv)) return e;
  if (heads < 1 || heads > 4096 || heads % kv->kv_heads)
    return fail(Q1_ERR_ARG, "%s: heads=%lld is no multiple of kv_heads=%lld up to 4096", who, (long long)heads,
                (long long)kv->kv_heads);
  if (int64_t(a.kv.total_new) * (heads / kv->kv_heads) >= (int64_t(1) << 31))
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
  const int64_t need = q1_paged_attention_workspace(max_new, heads, kv->kv_heads, kv->dim);
  if (need < 0) return int(need);
  if (workspace_bytes < need)
    return fail(Q1_ERR_ARG, "%s: the workspace holds %lld bytes, %lld are needed", who, (long long)workspace_bytes,
                (long long)need);
  a.q = q, a.out = out, a.q_token = q_token_stride, a.q_head = q_head_stride;
  a.o_token = out_token_stride, a.o_head = out_head_stride;
  if (int e = ops_status_ptr(&a.status)) return e;
  max_new = std::min<int64_t>(max_new, a.kv.total_new);
  a.heads = int(heads), a.group = int(heads / kv->kv_heads);
  a.group_inverse = uint32_t((uint64_t(1) << 32) / uint64_t(a.group) + 1);
  a.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf = kv->dtype == Q1_BF16;
  a.least_rows = 0, a.most_rows = INT_MAX;
  bool ran = false;
  const auto few = [&](bool only_clusters, const AttendArgs* many = nullptr) {
    if (kv->dim == 128)
      return bf ? launch_attend<__nv_bfloat16, 128>(a, max_new, only_clusters, workspace, s, ran, many)
                : launch_attend<__half, 128>(a, max_new, only_clusters, workspace, s, ran, many);
    return bf ? launch_attend<__nv_bfloat16, 64>(a, max_new, only_clusters, workspace, s, ran, many)
              : launch_attend<__half, 64>(a, max_new, only_clusters, workspace, s, ran, many);
  };
  if (int e = few(true)) return e;
  if (ran) return Q1_OK;
  if (!many_rows(max_new, a.group, kv->batch == 1)) return few(false);
  // Several sequences: those of one tile at most go to the kernel for few rows.  It
  // starts where the tensor-core kernel's CTAs end, and one launch joins
  // both's items (a mixed batch: 66 us, 78 one after the other).
  const bool both = kv->batch > 1;
  if (both) a.least_rows = kRowsS + 1;
  AttendArgs many = {};
  void* second = static_cast<char*>(workspace) + attend_workspace(attend_ctas(), kRowsS, int(kv->dim));
  if (int e = launch_attend_tc(a, second, bf, int(kv->dim), s, ran, both ? &many : nullptr)) return e;
  a.least_rows = 0;
  if (!ran) return few(false);
  if (!both) return Q1_OK;
  a.most_rows = kRowsS, a.beside = true;
  return few(false, &many);
}
