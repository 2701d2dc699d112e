// lora.cu -- q1_lora_add: out_v = base_v + scale_a * B_a (A_a x_v) for the
// adapter a of each vector v, many adapters in one launch.
//
// Few vectors share an adapter, so each adapter's A (rank x n) and B (rows x
// rank) have to be read about once and take 2 operations a value and vector:
// bytes bound it, and for one vector the chain of dependent memory reads.
//
// Both products run in one launch: a cluster of CTAs takes one bucket (up to
// eight vectors of one adapter), each CTA a slice of n in the first product
// and a slice of the rows in the second; the rank values between them (at
// most 128 a vector) pass through distributed shared memory, so there is no
// workspace and no second launch.
//
// Weights come through a ring of asynchronous 16-byte copies that is private
// to each thread (a thread reads only what it copied: no barrier, and the
// second product's first chunks are under way before the first has ended).
// The products run on m16n8k8 MMAs with tf32 operands and f32 sums: 16 rank
// rows (output rows) by the bucket's eight vectors.  Weights of 8 or 11
// significant bits are exact in tf32; an f32 value x (t) is taken as hi + lo,
// x rounded to 11 bits and the exact rest rounded to 11, which is off by 2^-24
// of it at most, as f32's own roundings are.  One form
// serves one to eight vectors: with products on the FMA pipe the code for each
// count, unrolled, missed the instruction cache, and eight vectors were bound
// by instructions (1000 vectors of prompts: 107 us).  An MMA takes its k
// indices in any order as long as both operands agree, so a lane's 16 bytes,
// eight neighbouring k, serve four MMAs as they are.
//
// Measured: 64 vectors, most with an adapter of their own (f16, ranks 16 to 64, 4096
// to 14336), 63 MB, in 24.3 us: 2.6 TB/s, 0.38 of the copy bandwidth; 1000 vectors of
// prompts (bf16, rank 32, 14336 to 4096), 94 MB, in 63 us.  Neither DRAM (39 and 15 %) nor issue (38 %)
// bounds them but each bucket's chain: index, x, first product, exchange through the
// cluster, second product.  One vector of rank 16, 4096 x 4096: 5.0 us.
//
// Vectors are grouped on the device: in a window of 64 vectors, every
// eighth vector of an adapter leads a bucket of it and the next ones of that
// window.  A cluster whose vector leads no bucket has nothing to do.
#include <cooperative_groups.h>

#include "ops.cuh"

namespace q1 {

namespace cg = cooperative_groups;

struct LoraArgs {
  const float* x;
  const void *wa, *wb;     // [adapters][rank][n], [adapters][rows][rank]
  const int32_t* index;
  const int32_t* ranks;    // or null
  const float* scale;      // or null
  const float* base;
  float* out;
  unsigned* status;
  int64_t ldx, ldb, ldo;
  int nvec, n, rows, rank, adapters;
};

constexpr int kLoraTokens = 8;    // vectors of a bucket: an MMA's N
constexpr int kLoraWindow = 64;   // vectors among which buckets form
constexpr int kLoraThreads = 256, kLoraWarps = kLoraThreads / 32;
constexpr int kLoraMaxRank = 128;
constexpr int kLoraStages = 4;    // stages of four 16-byte pieces a thread: 64 KB a CTA, two CTAs an SM
constexpr int kLoraRing = kLoraStages * 4 * kLoraThreads * 16;
// x in shared memory: 8192 values of all vectors, each vector's part padded by
// four so that the lanes' 16-byte reads of two vectors fall into different banks.
constexpr int kLoraX = 8192, kLoraXBytes = (kLoraX + 4 * kLoraTokens) * 4;
constexpr int kLoraSmem = kLoraRing + kLoraXBytes;
static_assert(kLoraWarps * kLoraMaxRank * kLoraTokens * 4 <= kLoraXBytes, "the warps' sums take x's place");

struct LoraShared {
  float mine[kLoraMaxRank][kLoraTokens];               // this CTA's slice of n
  float t[2][kLoraTokens][kLoraMaxRank + 4];           // all slices, scaled, as hi and lo
  int token[kLoraTokens];
  int count;
};

__device__ __forceinline__ void lora_copy(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void lora_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

__device__ __forceinline__ void mma_tf32(float (&c)[4], const float a0, const float a1, const float a2, const float a3,
                                         const float b0, const float b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
                 "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}
// Eight f32 values as hi + lo, both rounded to 11 significant bits.
__device__ __forceinline__ float round_tf32(float v) {
  return __uint_as_float((__float_as_uint(v) + 0x1000u) & 0xffffe000u);
}
__device__ __forceinline__ void split_tf32(const float (&v)[8], float (&hi)[8], float (&lo)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi[i] = round_tf32(v[i]);
    lo[i] = round_tf32(__fsub_rn(v[i], hi[i]));
  }
}
// sum += 16 rows (row g of the lane's quad and g + 8) x 32 k, eight of them in
// the lane, by the eight vectors (vector g of the lane's quad in v).  The MMAs
// cut, not round, their sums, so each 32 k start from zero and are added with
// rounding (14336 values in one accumulator were off by 2e-6).
template <class T>
__device__ __forceinline__ void mma_pieces(float (&sum)[4], const uint4& row, const uint4& row8, const float (&hi)[8],
                                           const float (&lo)[8]) {
  float a[8], b[8], c[4] = {0.f, 0.f, 0.f, 0.f};
  Elem<T>::unpack(row, a);
  Elem<T>::unpack(row8, b);
#pragma unroll
  for (int s = 0; s < 8; s += 2) {
    mma_tf32(c, a[s], b[s], a[s + 1], b[s + 1], lo[s], lo[s + 1]);
    mma_tf32(c, a[s], b[s], a[s + 1], b[s + 1], hi[s], hi[s + 1]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) sum[i] = __fadd_rn(sum[i], c[i]);
}

// A CTA's part of a bucket.  In the first product warp w takes blocks of 32
// values of n: w, w + 8, ...; a stage is a block of two tiles of 16 rank rows,
// or (rank up to 16) two blocks of the one tile.  In the second, chunks of 256
// output rows, 32 a warp, a stage a chunk's next 32 rank values.
template <class T>
struct LoraPart {
  const LoraArgs& a;
  const T *A, *B;                // the adapter's, from this CTA's first value and first row on
  int rank, slice, rows;         // rank in use, values of n, rows of this CTA
  int tiles, pairs, ranks32;     // of 16 rank rows, of two of those (at least 1), of 32 rank values
  int warp, quad, piece;         // lane / 4 and lane % 4
  unsigned char* ring;
  // What the next copies are of: the place in the work, and the lane's first
  // piece there (moved on by addition: products of 64-bit strides for every
  // piece were a third of all instructions).
  int f_block, f_pair = 0, f_chunk = 0, f_k = 0, f_slot = 0;
  const T *f_a, *f_b;

  __device__ __forceinline__ LoraPart(const LoraArgs& args) : a(args) {}

  // After the members above `f_block` are set.
  __device__ __forceinline__ void start() {
    f_block = warp;
    f_a = A + int64_t(quad) * a.n + warp * 32 + piece * 8;
    f_b = B + int64_t(warp * 32 + quad * 2) * a.rank + piece * 8;
  }

  // The next stage's four pieces, in order; past everything an empty group.
  __device__ __forceinline__ void fetch() {
    const uint32_t dst = smem_addr(ring) + f_slot * (4 * kLoraThreads * 16) + threadIdx.x * 16;
    if (f_block * 32 < slice) {
      const int64_t down8 = int64_t(8) * a.n;
      // Pieces 2 and 3: the next tile of rank rows, or (one tile) the warp's next block.
      const int64_t second = tiles <= 1 ? 32 * kLoraWarps : 2 * down8;
      const int j = f_block * 32 + piece * 8, row = f_pair * 32 + quad;
      const int j2 = tiles <= 1 ? j + 32 * kLoraWarps : j, row2 = tiles <= 1 ? row : row + 16;
      const bool in0 = j < slice && row < rank, in1 = j < slice && row + 8 < rank;
      const bool in2 = j2 < slice && row2 < rank, in3 = j2 < slice && row2 + 8 < rank;
      lora_copy(dst, in0 ? f_a : A, in0);
      lora_copy(dst + kLoraThreads * 16, in1 ? f_a + down8 : A, in1);
      lora_copy(dst + 2 * kLoraThreads * 16, in2 ? f_a + second : A, in2);
      lora_copy(dst + 3 * kLoraThreads * 16, in3 ? f_a + second + down8 : A, in3);
      f_a += 4 * down8;
      if (++f_pair >= pairs) {
        f_pair = 0;
        f_a -= pairs * 4 * down8;
        const int blocks = tiles <= 1 ? 2 * kLoraWarps : kLoraWarps;
        f_block += blocks, f_a += blocks * 32;
      }
    } else if (f_chunk * 256 < rows) {
      const int row = f_chunk * 256 + warp * 32 + quad * 2;
      const bool k_in = f_k * 32 + piece * 8 < rank;
      const T* p = f_b;
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // rows row, row + 16, row + 1, row + 17
        const bool live = k_in && row + (i & 1) * 16 + (i >> 1) < rows;
        lora_copy(dst + i * (kLoraThreads * 16), live ? p + ((i & 1) * 16 + (i >> 1)) * a.rank : B, live);
      }
      f_b += 32;
      if (++f_k >= ranks32) {
        f_k = 0, ++f_chunk;
        f_b += 256 * int64_t(a.rank) - ranks32 * 32;
      }
    }
    lora_commit();
    f_slot = (f_slot + 1) % kLoraStages;
  }
  // Waits for the stage in `slot`.
  __device__ __forceinline__ void take(int slot, uint4 (&w)[4]) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLoraStages - 1) : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint4*>(ring + ((slot * 4 + i) * kLoraThreads + threadIdx.x) * 16);
  }
};

// The window of x from value `from` of the slice on: `count` vectors, each
// `window` values and four of padding apart.
__device__ __forceinline__ void lora_fetch_x(const LoraArgs& a, const LoraShared& sh, uint32_t xs, int j0, int window, int size) {
  for (int v = 0; v < sh.count; ++v) {
    const float* x = a.x + sh.token[v] * a.ldx + j0;
#pragma unroll 1
    for (int p = threadIdx.x; p < size / 4; p += kLoraThreads) lora_copy(xs + (v * (window + 4) + p * 4) * 4, x + p * 4, true);
  }
  lora_commit();
}

// One bucket.  VEC: base and out rows allow 8-byte accesses, rows is even.
template <class T, bool VEC>
__device__ __forceinline__ void lora_bucket(const LoraArgs& a, LoraShared& sh, LoraPart<T>& part, int j0, int r0, float scale,
                                            cg::cluster_group& cluster) {
  const int quad = part.quad, piece = part.piece, count = sh.count;
  float* xs = reinterpret_cast<float*>(part.ring + kLoraRing);
  const int window = kLoraX >> (count <= 1 ? 0 : count <= 2 ? 1 : count <= 4 ? 2 : 3);  // values of a vector
  lora_fetch_x(a, sh, smem_addr(xs), j0, window, min(window, part.slice));
#pragma unroll 1
  for (int i = 0; i < kLoraStages - 1; ++i) part.fetch();
  asm volatile("cp.async.wait_group %0;" ::"n"(kLoraStages - 1) : "memory");
  __syncthreads();  // the first window of x

  float acc[kLoraMaxRank / 16][4];
#pragma unroll
  for (int i = 0; i < kLoraMaxRank / 16; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  int slot = 0;
  const auto next_slot = [&]() { slot = (slot + 1) % kLoraStages; };
  const auto x_piece = [&](int block, float (&hi)[8], float (&lo)[8]) {
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (quad < count && block * 32 + piece * 8 < part.slice) {
      const float4* src = reinterpret_cast<const float4*>(xs + quad * (window + 4) + (block * 32) % window + piece * 8);
      const float4 p = src[0], q = src[1];
      v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w, v[4] = q.x, v[5] = q.y, v[6] = q.z, v[7] = q.w;
    }
    split_tf32(v, hi, lo);
  };
  const int step = part.tiles <= 1 ? 2 * kLoraWarps : kLoraWarps;  // a window is whole steps
  int in_window = 0;
#pragma unroll 1
  for (int b0 = 0; b0 * 32 < part.slice; b0 += step) {  // the whole CTA together; warp w's block is b0 + w
    if (in_window * 32 == window) {  // the next window of x
      in_window = 0;
      __syncthreads();
      lora_fetch_x(a, sh, smem_addr(xs), j0 + b0 * 32, window, min(window, part.slice - b0 * 32));
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();
    }
    in_window += step;
    const int block = b0 + part.warp;
    if (block * 32 >= part.slice) continue;  // as the copies: nothing is under way for it
    float hi[8], lo[8];
    uint4 w[4];
    if (part.tiles <= 1) {
      part.fetch();
      part.take(slot, w);
      next_slot();
      x_piece(block, hi, lo);
      mma_pieces<T>(acc[0], w[0], w[1], hi, lo);
      x_piece(block + kLoraWarps, hi, lo);
      mma_pieces<T>(acc[0], w[2], w[3], hi, lo);
    } else {
      x_piece(block, hi, lo);
#pragma unroll
      for (int p = 0; p < kLoraMaxRank / 32; ++p) {
        if (p >= part.pairs) break;
        part.fetch();
        part.take(slot, w);
        next_slot();
        mma_pieces<T>(acc[2 * p], w[0], w[1], hi, lo);
        mma_pieces<T>(acc[2 * p + 1], w[2], w[3], hi, lo);
      }
    }
  }
  // The warps' sums, over the place of x; then in order.
  __syncthreads();
  float* sums = xs + part.warp * (kLoraMaxRank * kLoraTokens);
#pragma unroll
  for (int i = 0; i < kLoraMaxRank / 16; ++i) {
    if (i >= part.tiles) break;
    float* dst = sums + (i * 16 + quad) * kLoraTokens + piece * 2;
    *reinterpret_cast<float2*>(dst) = make_float2(acc[i][0], acc[i][1]);
    *reinterpret_cast<float2*>(dst + 8 * kLoraTokens) = make_float2(acc[i][2], acc[i][3]);
  }
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i < part.rank * kLoraTokens; i += kLoraThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kLoraWarps; ++w) v = __fadd_rn(v, xs[w * (kLoraMaxRank * kLoraTokens) + i]);
    (&sh.mine[0][0])[i] = v;
  }
  cluster.sync();
#pragma unroll 1
  for (int i = threadIdx.x; i < part.rank * kLoraTokens; i += kLoraThreads) {
    float v = 0.f;
    for (int p = 0; p < int(cluster.num_blocks()); p += 4) {  // four reads at a time; a cluster has 4, 8 or 16 CTAs
      float s[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] = cluster.map_shared_rank(&sh.mine[0][0], p + k)[i];
#pragma unroll
      for (int k = 0; k < 4; ++k) v = __fadd_rn(v, s[k]);
    }
    v = __fmul_rn(v, scale);
    const float hi = round_tf32(v);
    sh.t[0][i % kLoraTokens][i / kLoraTokens] = hi;
    sh.t[1][i % kLoraTokens][i / kLoraTokens] = round_tf32(__fsub_rn(v, hi));
  }
  // Rank values past the adapter's, up to a multiple of 32, are zero.
  for (int i = part.rank + (threadIdx.x >> 4); i < part.ranks32 * 32; i += kLoraThreads / 16)
    sh.t[threadIdx.x >> 3 & 1][threadIdx.x & 7][i] = 0.f;
  cluster.sync();  // every CTA has read `mine`, and t is complete

  // Second product.  A lane's outputs: two neighbouring rows (and the same
  // eight pairs further on) of vectors 2 piece and 2 piece + 1; what they are
  // added to is read one chunk ahead.
  const int row_lane = part.warp * 32 + quad * 2;
  const float* in[2];
  float* out[2];
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const int64_t token = sh.token[2 * piece + v < count ? 2 * piece + v : 0];
    in[v] = a.base + token * a.ldb + r0 + row_lane;
    out[v] = a.out + token * a.ldo + r0 + row_lane;
  }
  float2 next[2][2];
  const auto fetch_base = [&](int row0) {
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = row0 + row_lane + h * 16;
        next[v][h] = make_float2(0.f, 0.f);
        if (2 * piece + v >= count || row >= part.rows) continue;
        const float* src = in[v] + row0 + h * 16;
        if constexpr (VEC) {
          next[v][h] = *reinterpret_cast<const float2*>(src);
        } else {
          next[v][h].x = src[0];
          if (row + 1 < part.rows) next[v][h].y = src[1];
        }
      }
  };
  fetch_base(0);
#pragma unroll 1
  for (int row0 = 0; row0 < part.rows; row0 += 256) {
    float2 base[2][2];
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
      for (int h = 0; h < 2; ++h) base[v][h] = next[v][h];
    fetch_base(row0 + 256);
    float c[2][4] = {};
#pragma unroll 1
    for (int k = 0; k < part.ranks32; ++k) {
      uint4 w[4];
      part.fetch();
      part.take(slot, w);
      next_slot();
      // Values past the adapter's rank may be anything: zero, like their t.
      const int inside = part.rank - k * 32 - piece * 8;
      if (inside > 0 && inside < 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t* word = reinterpret_cast<uint32_t*>(&w[i]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            word[e] = inside >= 2 * e + 2 ? word[e] : inside == 2 * e + 1 ? word[e] & 0xffffu : 0u;
        }
      }
      float hi[8], lo[8];
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const float4 h4 = *reinterpret_cast<const float4*>(&sh.t[0][quad][k * 32 + piece * 8 + e]);
        const float4 l4 = *reinterpret_cast<const float4*>(&sh.t[1][quad][k * 32 + piece * 8 + e]);
        hi[e] = h4.x, hi[e + 1] = h4.y, hi[e + 2] = h4.z, hi[e + 3] = h4.w;
        lo[e] = l4.x, lo[e + 1] = l4.y, lo[e + 2] = l4.z, lo[e + 3] = l4.w;
      }
      mma_pieces<T>(c[0], w[0], w[1], hi, lo);
      mma_pieces<T>(c[1], w[2], w[3], hi, lo);
    }
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = row0 + row_lane + h * 16;
        if (2 * piece + v >= count || row >= part.rows) continue;
        float* dst = out[v] + row0 + h * 16;
        const float2 r = make_float2(__fadd_rn(base[v][h].x, c[0][2 * h + v]), __fadd_rn(base[v][h].y, c[1][2 * h + v]));
        if constexpr (VEC) {
          *reinterpret_cast<float2*>(dst) = r;
        } else {
          dst[0] = r.x;
          if (row + 1 < part.rows) dst[1] = r.y;
        }
      }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <class T, bool VEC>
__global__ void __launch_bounds__(kLoraThreads, 2) k_lora_add(LoraArgs a) {
  __shared__ LoraShared sh;
  extern __shared__ __align__(16) unsigned char ring[];
  cg::cluster_group cluster = cg::this_cluster();
  pdl_launch_dependents();
  pdl_wait();
  const int C = int(cluster.num_blocks()), clusters = int(gridDim.x) / C, c = int(cluster.block_rank());
#pragma unroll 1
  for (int v = int(blockIdx.x) / C; v < a.nvec; v += clusters) {
    // Warp 0 looks at the window: which of its vectors have v's adapter.
    const int raw = a.index[v];
    const int adapter = raw >= 0 && raw < a.adapters ? raw : -1;
    const int w0 = v / kLoraWindow * kLoraWindow;
    if (threadIdx.x < 32) {
      uint64_t same = 0;
#pragma unroll
      for (int h = 0; h < kLoraWindow / 32; ++h) {
        const int u = w0 + h * 32 + int(threadIdx.x);
        int au = u < a.nvec ? a.index[u] : -2;
        if (u < a.nvec && (au < 0 || au >= a.adapters)) au = -1;
        same |= uint64_t(__ballot_sync(0xffffffffu, au == adapter)) << (32 * h);
      }
      const int before = __popcll(same & ((uint64_t(1) << (v - w0)) - 1));
      if (threadIdx.x == 0) {
        int count = 0;
        if (before % kLoraTokens == 0) {
#pragma unroll 1
          for (uint64_t rest = same >> (v - w0) << (v - w0); rest && count < kLoraTokens; rest &= rest - 1)
            sh.token[count++] = w0 + __ffsll(int64_t(rest)) - 1;
        }
        sh.count = count;
        if (raw < -1 || raw >= a.adapters) atomicOr(a.status, kStatusBadIndex);
      }
    }
    __syncthreads();
    const int count = sh.count;
    if (count && adapter < 0) {
      if (a.out != a.base) {
#pragma unroll 1
        for (int i = 0; i < count; ++i)
#pragma unroll 1
          for (int r = c * kLoraThreads + threadIdx.x; r < a.rows; r += C * kLoraThreads)
            a.out[sh.token[i] * a.ldo + r] = a.base[sh.token[i] * a.ldb + r];
      }
    } else if (count) {
      LoraPart<T> part(a);
      const int per_n = (a.n / 8 + C - 1) / C * 8, per_r = ((a.rows + 1) / 2 + C - 1) / C * 2;
      const int j0 = min(a.n, c * per_n), r0 = min(a.rows, c * per_r);
      part.rank = a.ranks ? max(0, min(a.ranks[adapter], a.rank)) : a.rank;
      part.A = static_cast<const T*>(a.wa) + int64_t(adapter) * a.rank * a.n + j0;
      part.B = static_cast<const T*>(a.wb) + (int64_t(adapter) * a.rows + r0) * a.rank;
      part.rows = min(a.rows, r0 + per_r) - r0;
      part.tiles = (part.rank + 15) / 16, part.pairs = max(1, (part.tiles + 1) / 2);
      part.slice = part.rank ? min(a.n, j0 + per_n) - j0 : 0;  // rank 0: no first product
      part.ranks32 = max(1, (part.rank + 31) / 32);
      part.warp = threadIdx.x >> 5, part.quad = (threadIdx.x & 31) >> 2, part.piece = threadIdx.x & 3;
      part.ring = ring;
      part.start();
      lora_bucket<T, VEC>(a, sh, part, j0, r0, a.scale ? a.scale[adapter] : 1.f, cluster);
    }
    __syncthreads();  // sh is free again
  }
}

template <class T, bool VEC>
static int launch_lora(const LoraArgs& g, cudaStream_t s) {
  const char* who = "q1_lora_add launch";
  static bool set[64] = {};
  int dev = 0;
  if (int e = cuda_status(cudaGetDevice(&dev), who)) return e;
  if (dev < 0 || dev >= 64 || !set[dev]) {
    if (int e = cuda_status(cudaFuncSetAttribute(k_lora_add<T, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, kLoraSmem), who))
      return e;
    if (int e = cuda_status(cudaFuncSetAttribute(k_lora_add<T, VEC>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1), who))
      return e;
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  // Clusters of 16 while all of them run at once (one vector of rank 16, 4096 x
  // 4096: 5.0 us against 6.2 with 8), of 8 up to 128 vectors (64 of rank 64: 27 us
  // against 39 with 4), of 4 beyond: fewer CTAs wait for each other (1000 vectors of
  // prompts: 66 us against 82, 163 of rank 48: 29 against 33).  Their number
  // is odd: the vectors that lead buckets are every eighth in a prompt, and a
  // cluster takes every so many-th vector.
  const int cluster = g.nvec * 16 <= 2 * num_sms() ? 16 : g.nvec <= 128 ? 8 : 4;
  const int64_t most = (num_sms() - 1) | 1;
  const dim3 grid(unsigned((g.nvec < most ? g.nvec : most) * cluster));
  return launch_op(k_lora_add<T, VEC>, grid, kLoraThreads, kLoraSmem, cluster, s, who, g);
}

}  // namespace q1

using namespace q1;

extern "C" int q1_lora_add(const float* x, int64_t ldx, int64_t nvec, int64_t n, int64_t rows, const void* a,
                           const void* b, int dtype, int64_t adapters, int64_t rank, const int32_t* index,
                           const int32_t* ranks, const float* scale, const float* base, int64_t ldb, float* out,
                           int64_t ldo, void* stream) {
  const char* who = "q1_lora_add";
  if (nvec < 1 || nvec > 65535 || n < 8 || n > (int64_t(1) << 24) || n % 8 || rows < 1 || rows > (int64_t(1) << 26) ||
      adapters < 1 || adapters > (1 << 20) || rank < 8 || rank > kLoraMaxRank || rank % 8)
    return fail(Q1_ERR_ARG, "%s: bad shape nvec=%lld n=%lld rows=%lld adapters=%lld rank=%lld (n and rank multiples of 8, "
                "rank in 8..128)", who, (long long)nvec, (long long)n, (long long)rows, (long long)adapters, (long long)rank);
  if (dtype != Q1_BF16 && dtype != Q1_F16) return fail(Q1_ERR_ARG, "%s: bad weight type %d", who, dtype);
  if (!x || !a || !b || !index || !base || !out) return fail(Q1_ERR_ARG, "%s: null pointer", who);
  if (!aligned16(x) || !aligned16(a) || !aligned16(b) || ldx % 4 || reinterpret_cast<uintptr_t>(base) % 4 ||
      reinterpret_cast<uintptr_t>(out) % 4)
    return fail(Q1_ERR_ARG, "%s: x, a and b must be 16-byte aligned, rows of x multiples of 4", who);
  if (ldx < n || ldb < rows || ldo < rows) return fail(Q1_ERR_ARG, "%s: a row stride is less than its row", who);
  if (base == out && ldb != ldo) return fail(Q1_ERR_ARG, "%s: in place, base and out need the same stride", who);
  LoraArgs g = {x, a, b, index, ranks, scale, base, out, nullptr, ldx, ldb, ldo, int(nvec), int(n), int(rows), int(rank),
                int(adapters)};
  if (int e = ops_status_ptr(&g.status)) return e;
  const bool vec = reinterpret_cast<uintptr_t>(base) % 8 == 0 && reinterpret_cast<uintptr_t>(out) % 8 == 0 && ldb % 2 == 0 &&
                   ldo % 2 == 0 && rows % 2 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == Q1_BF16) return vec ? launch_lora<__nv_bfloat16, true>(g, s) : launch_lora<__nv_bfloat16, false>(g, s);
  return vec ? launch_lora<__half, true>(g, s) : launch_lora<__half, false>(g, s);
}
