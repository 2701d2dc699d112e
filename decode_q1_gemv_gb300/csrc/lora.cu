// lora.cu -- q1_lora_add: out_v = base_v + scale_a * B_a (A_a x_v) for the
// adapter a of each vector v, many adapters in one launch.
//
// Few vectors share an adapter, so each adapter's A (rank x n) and B (rows x
// rank) have to be read about once and take 2 operations a value and vector:
// bytes bound it, and for one vector the chain of dependent memory reads.
//
// Both products run in one launch: a cluster of CTAs, or half of one, takes one
// bucket (up to eight or sixteen vectors of one adapter), each CTA a slice of n in the
// first product and a slice of the rows in the second; the rank values between them
// (at most 128 a vector) pass through distributed shared memory, so there is
// no workspace and no second launch.
//
// Weights, x and base come through a ring of asynchronous 16-byte copies that
// is private to each warp: no barrier in either product, and the second
// product's first chunks are under way before the first has ended.  (x in
// windows for the whole CTA, each waited for: 27,000 cycles of the first
// product of a bucket of prompts, against 15,000 now for as many vectors.)
//
// The products run on MMAs with 16-bit weights by parts of the f32 values that
// are exact in the MMA's type (see LoraMul).  One form serves one to eight
// vectors: with products on the FMA pipe the code for each count, unrolled,
// missed the instruction cache, and eight vectors were bound by instructions
// (1000 vectors of prompts: 107 us).  Instructions bound it still: ldmatrix puts
// the weights into the MMA's registers in their order (moving them there cost
// a tenth of all instructions), and a copy outside a matrix is left out, not
// redirected.
//
// Measured: 64 vectors, most with an adapter of their own (f16, ranks 16 to 64, 4096
// to 14336), 63 MB, in 20.4 us: 3.1 TB/s, 0.46 of the copy bandwidth; 1000 vectors of
// prompts (bf16, rank 32, 14336 to 4096), 94 MB, in 32 us: 3.0 TB/s.  One vector of
// rank 16, 4096 x 4096: 4.7 us.  Half of the issue slots are used in the
// products; the rest of a bucket's time is its chain: index, first product,
// exchange through the cluster, second product.
//
// Vectors are grouped on the device: in a window of 64 vectors, every
// eighth (sixteenth) vector of an adapter leads a bucket of it and the next
// ones of that window.  The device also counts the buckets, and gives each a
// cluster while all run at once, else half a cluster: what a call of up to 288 vectors
// takes depends on the adapters that its vectors name, not on how many there are.
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
  int nvec, n, rows, rank, adapters, log_cluster;
};

constexpr int kLoraWindow = 64;   // vectors among which buckets form
constexpr int kLoraThreads = 256, kLoraWarps = kLoraThreads / 32;
constexpr int kLoraRound = kLoraWarps * kLoraWindow;  // vectors whose buckets are counted at a time

// N: groups of eight vectors (an MMA's N) of a bucket.  A stage holds, for each
// thread, four 16-byte pieces of weights and 2 N of x or of base; 96 KB a CTA,
// two CTAs an SM.
template <int N>
struct LoraTile {
  static constexpr int kTokens = 8 * N, kMaxRank = N == 1 ? 128 : 64, kTiles = kMaxRank / 16;
  static constexpr int kPieces = 4 + 2 * N, kStages = N == 1 ? 4 : 3;
  static constexpr int kStage = kPieces * kLoraThreads * 16, kRing = kStages * kStage;
};

struct LoraShared {
  float mine[1024];                         // this CTA's slice of n: [tile][group][16 ranks][8]
  __align__(16) unsigned char t[9216];      // all slices, scaled, as parts (LoraMul)
  uint64_t leads[kLoraWarps];               // of a round's windows: the vectors that lead buckets
  int adapter[kLoraRound];                  // of a round's vectors
  const float *x[16], *base[16];            // the vectors' slices of the CTA
  float* out[16];
  int slot[kLoraWarps];                     // the ring's free stage, where a warp leaves its sums
  int count;                                // vectors of the bucket
  int log, step;                            // CTAs that share one (log2), the next one's distance
  bool halves;                              // of the cluster have buckets of their own, and meet at these:
  uint64_t ready, read;                     // everyone's `mine` is there; mine has been read by everyone
  uint32_t parity;                          // of the bucket's phase of both
  int total;                                // of this round and those before
};

// Dynamic shared memory: this, then the ring.
extern __shared__ __align__(128) unsigned char lora_smem[];
constexpr int kLoraRingAt = (sizeof(LoraShared) + 127) / 128 * 128;

__device__ __forceinline__ void lora_copy(uint32_t dst, const void* src, bool live) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %2, 0;\n@p cp.async.cg.shared.global [%0], [%1], 16;\n}" ::"r"(dst), "l"(src),
               "r"(int(live)) : "memory");
}
// The first `bytes` of 16, zeros after them.
__device__ __forceinline__ void lora_copy_part(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void lora_copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void lora_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ uint4 lora_read(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
  return v;
}

// Four 8 x 8 matrices of 16-bit values, a row of one at the address of each lane.
__device__ __forceinline__ void lora_matrix(uint32_t src, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(src) : "memory");
}

// Two tiles of 16 rows of weights by 32 k: [tile][16 k][operand register].
// A lane has values 8 c + 2 piece and the next one of each eight k, c = 0 to 3, of rows
// g (its quad) and g + 8; of x and t it has the same k of vector g.
using LoraWeights = uint32_t[2][2][4];

// How a lane's eight k of x, or of t, stand as parts that are exact in the
// MMA's operand type, and their product with two tiles of weights.  The MMAs cut, not round, their sums, so each 32 k
// start from zero, small parts first, and are added with rounding (14336
// values in one accumulator were off by 2e-6).  The chains of the tiles and
// vector groups take turns: one after another, each MMA would wait for the last.
template <class T>
struct LoraMul;
// Where t has rank value k: each 32 in the order of the lanes that read them.
__device__ __forceinline__ int lora_place(int k) { return (k & ~31) | (k & 6) << 2 | (k & 24) >> 2 | (k & 1); }

// bf16: three bf16 parts, 8 bits each, hold all of an f32; weights go into the MMA as they are.
template <>
struct LoraMul<__nv_bfloat16> {
  struct X {
    uint4 part[3];
  };
  static __device__ __forceinline__ uint32_t take(float& a, float& b) {  // a bf16 of each, which leaves the rest
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&h);
    a = __fsub_rn(a, __uint_as_float(u << 16));
    b = __fsub_rn(b, __uint_as_float(u & 0xffff0000u));
    return u;
  }
  static __device__ __forceinline__ void split(float (&v)[8], X& x) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      x.part[i].x = take(v[0], v[1]);
      x.part[i].y = take(v[2], v[3]);
      x.part[i].z = take(v[4], v[5]);
      x.part[i].w = take(v[6], v[7]);
    }
  }
  // t: [part][vector][kRank + 32 bf16], a lane's eight k together, so that two vectors' 64 bytes fall into different banks.
  template <int kTokens, int kRank>
  static __device__ __forceinline__ void store(unsigned char* t, int vec, int row, float v) {
    float none = 0.f;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      *reinterpret_cast<uint16_t*>(t + ((i * kTokens + vec) * (kRank + 32) + lora_place(row)) * 2) = uint16_t(take(v, none));
  }
  template <int kTokens, int kRank>
  static __device__ __forceinline__ void load(uint32_t t, int vec, int k, X& x) {
#pragma unroll
    for (int i = 0; i < 3; ++i) x.part[i] = lora_read(t + ((i * kTokens + vec) * (kRank + 32) + k) * 2);
  }
  template <int N>
  static __device__ __forceinline__ void multiply(float (&c)[2][N][4], const LoraWeights& w, const X (&x)[N]) {
#pragma unroll
    for (int i = 2; i >= 0; --i)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int g = 0; g < N; ++g)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t b0 = s ? x[g].part[i].z : x[g].part[i].x, b1 = s ? x[g].part[i].w : x[g].part[i].y;
            if (i == 2 && s == 0)
              asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                           : "=f"(c[h][g][0]), "=f"(c[h][g][1]), "=f"(c[h][g][2]), "=f"(c[h][g][3])
                           : "r"(w[h][s][0]), "r"(w[h][s][1]), "r"(w[h][s][2]), "r"(w[h][s][3]), "r"(b0), "r"(b1), "f"(0.f));
            else
              asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                           : "+f"(c[h][g][0]), "+f"(c[h][g][1]), "+f"(c[h][g][2]), "+f"(c[h][g][3])
                           : "r"(w[h][s][0]), "r"(w[h][s][1]), "r"(w[h][s][2]), "r"(w[h][s][3]), "r"(b0), "r"(b1));
          }
  }
};

// f16: two tf32 parts (x rounded to 11 bits, the exact rest cut to 11: of its 12 bits at most the last may go,
// 2^-23 of x, twice f32's own rounding; f16 has not x's range), the weights as tf32, which holds them.
// A NaN stays one: hi may lose it (0x7fffffff + 0x1000 is -0), the rest is arithmetic, and cut.
template <>
struct LoraMul<__half> {
  struct X {
    float hi[8], lo[8];
  };
  static __device__ __forceinline__ void take(float v, float& hi, float& lo) {
    hi = __uint_as_float((__float_as_uint(v) + 0x1000u) & 0xffffe000u);
    lo = __uint_as_float(__float_as_uint(__fsub_rn(v, hi)) & 0xffffe000u);
  }
  static __device__ __forceinline__ void split(float (&v)[8], X& x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) take(v[i], x.hi[i], x.lo[i]);
  }
  // t: [hi, lo][vector][kRank + 4 f32].
  template <int kTokens, int kRank>
  static __device__ __forceinline__ void store(unsigned char* t, int vec, int row, float v) {
    float* at = reinterpret_cast<float*>(t) + vec * (kRank + 4) + lora_place(row);
    take(v, at[0], at[kTokens * (kRank + 4)]);
  }
  template <int kTokens, int kRank>
  static __device__ __forceinline__ void load(uint32_t t, int vec, int k, X& x) {
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const uint4 h = lora_read(t + (vec * (kRank + 4) + k + e) * 4), l = lora_read(t + ((kTokens + vec) * (kRank + 4) + k + e) * 4);
      x.hi[e] = __uint_as_float(h.x), x.hi[e + 1] = __uint_as_float(h.y), x.hi[e + 2] = __uint_as_float(h.z), x.hi[e + 3] = __uint_as_float(h.w);
      x.lo[e] = __uint_as_float(l.x), x.lo[e + 1] = __uint_as_float(l.y), x.lo[e + 2] = __uint_as_float(l.z), x.lo[e + 3] = __uint_as_float(l.w);
    }
  }
  template <int N>
  static __device__ __forceinline__ void multiply(float (&c)[2][N][4], const LoraWeights& w, const X (&x)[N]) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      float a[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        Elem<__half>::unpack2(w[h][s / 2][s % 2 * 2], a[h][0], a[h][2]);
        Elem<__half>::unpack2(w[h][s / 2][s % 2 * 2 + 1], a[h][1], a[h][3]);
      }
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int g = 0; g < N; ++g)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float b0 = part ? x[g].hi[2 * s] : x[g].lo[2 * s], b1 = part ? x[g].hi[2 * s + 1] : x[g].lo[2 * s + 1];
            if (s == 0 && part == 0)
              asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                           : "=f"(c[h][g][0]), "=f"(c[h][g][1]), "=f"(c[h][g][2]), "=f"(c[h][g][3])
                           : "r"(__float_as_uint(a[h][0])), "r"(__float_as_uint(a[h][1])), "r"(__float_as_uint(a[h][2])),
                             "r"(__float_as_uint(a[h][3])), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)), "f"(0.f));
            else
              asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                           : "+f"(c[h][g][0]), "+f"(c[h][g][1]), "+f"(c[h][g][2]), "+f"(c[h][g][3])
                           : "r"(__float_as_uint(a[h][0])), "r"(__float_as_uint(a[h][1])), "r"(__float_as_uint(a[h][2])),
                             "r"(__float_as_uint(a[h][3])), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
          }
    }
  }
};

// sum += two tiles of rows by 32 k.
template <class T, int N>
__device__ __forceinline__ void lora_mma(float (&sum0)[N][4], float (&sum1)[N][4], const LoraWeights& w,
                                         const typename LoraMul<T>::X (&x)[N]) {
  float c[2][N][4];
  LoraMul<T>::template multiply<N>(c, w, x);
#pragma unroll
  for (int g = 0; g < N; ++g)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum0[g][i] = __fadd_rn(sum0[g][i], c[0][g][i]);
      sum1[g][i] = __fadd_rn(sum1[g][i], c[1][g][i]);
    }
}

// A CTA's part of a bucket.  In the first product warp w takes blocks of 32
// values of n: w, w + 8, ...; a stage is two tiles of 16 rank rows of a block,
// the block's first with its x.  In the second, chunks of 256 output rows, 32
// a warp; a stage is a chunk's next 32 rank values, the chunk's first with
// what its rows are added to.
template <class T, int N, bool VEC>
struct LoraPart {
  using S = LoraTile<N>;
  const LoraShared& sh;
  int rank, a_rank, slice, rows; // rank in use, row stride of B, values of n, rows of this CTA
  int tiles, pairs, ranks32;     // of 16 rank rows, of two of those (at least 1), of 32 rank values
  int count, warp, lane, quad, piece;  // vectors of the bucket, lane / 4 and lane % 4
  uint32_t ring;                 // its address in shared memory
  // What the next copies are of: the place in the work, and the lane's first
  // piece there (moved on by addition: products of 64-bit strides for every
  // piece were a third of all instructions).
  int f_block, f_pair = 0, f_chunk = 0, f_k = 0, f_slot = 0;  // f_slot: the stage's offset
  const T *f_a, *f_b;
  int64_t down8, next_block, next_chunk;  // in A: eight rows on, from past a block's rows to the next block; in B
  uint32_t to, from;                      // the lane's 16 bytes of a weight copy; its row for lora_matrix

  // After the members above `f_block` are set.
  __device__ __forceinline__ LoraPart(const LoraShared& shared) : sh(shared) {}
  __device__ __forceinline__ void start(const T* A, const T* B, int64_t n) {
    f_block = warp;
    f_a = A + quad * n + warp * 32 + piece * 8;
    f_b = B + int64_t(warp * 32 + quad * 2) * a_rank + piece * 8;
    down8 = 8 * n, next_block = kLoraWarps * 32 - (pairs - 1) * 4 * down8;
    next_chunk = 256 * int64_t(a_rank) - (ranks32 - 1) * 32;
    // A row's four 16-byte pieces are moved by half the row, so that eight rows' are in different banks.
    to = ring + warp * 512 + quad * 64 + ((piece ^ quad >> 1) & 3) * 16;
    const int r = lane & 7;
    from = ring + (lane >> 3 & 1) * (kLoraThreads * 16) + warp * 512 + r * 64 + ((lane >> 4 ^ r >> 1) & 3) * 16;
  }

  // The next stage's pieces, in order; past everything an empty group.  What
  // lies outside the matrices is not copied: the ring has old values there.
  __device__ __forceinline__ void fetch() {
    constexpr int kPiece = kLoraThreads * 16;
    const uint32_t stage = ring + f_slot, dst = to + f_slot;
    if (f_block * 32 < slice) {
      const int left = slice - f_block * 32, ranks = piece * 8 < left ? rank - f_pair * 32 - quad : 0;
      const T* p = f_a;
#pragma unroll
      for (int i = 0; i < 4; ++i, p += down8) lora_copy(dst + i * kPiece, p, ranks > 8 * i);
      if (f_pair == 0) {
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) {
          const int vec = i * 4 + lane / 8;
          lora_copy(stage + x_place(vec, lane % 8), sh.x[vec] + f_block * 32 + lane % 8 * 4,
                    lane % 8 * 4 < left && vec < count);
        }
      }
      const bool turn = f_pair + 1 >= pairs;
      f_a += turn ? next_block : 4 * down8;
      f_pair = turn ? 0 : f_pair + 1;
      f_block += turn ? kLoraWarps : 0;
    } else if (f_chunk * 256 < rows) {
      const int first = f_chunk * 256 + warp * 32;
      const int left = f_k * 32 + piece * 8 < rank ? rows - first - quad * 2 : 0;
      // Rows row, row + 16, row + 1, row + 17 of row = first + 2 quad.
      lora_copy(dst, f_b, left > 0);
      lora_copy(dst + kPiece, f_b + 16 * a_rank, left > 16);
      lora_copy(dst + 2 * kPiece, f_b + a_rank, left > 1);
      lora_copy(dst + 3 * kPiece, f_b + 17 * a_rank, left > 17);
      if (f_k == 0) {
        const int from = first + lane % 8 * 4;
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) {
          const int vec = i * 4 + lane / 8;
          if (vec >= count || from >= rows) continue;
          const uint32_t at = stage + base_place(vec, lane % 8);
          const float* src = sh.base[vec] + from;
          if constexpr (VEC) {
            lora_copy_part(at, src, min(16, (rows - from) * 4));
          } else {
#pragma unroll 1
            for (int e = 0; e < min(4, rows - from); ++e) lora_copy4(at + e * 4, src + e);
          }
        }
      }
      const bool turn = f_k + 1 >= ranks32;
      f_b += turn ? next_chunk : 32;
      f_k = turn ? 0 : f_k + 1;
      f_chunk += turn;
    }
    lora_commit();
    f_slot = after(f_slot);
  }
  static __device__ __forceinline__ int after(int slot) {
    return slot == (S::kStages - 1) * S::kStage ? 0 : slot + S::kStage;
  }
  // Waits for the stage at `slot`.
  __device__ __forceinline__ void take(int slot, LoraWeights& w) {
    asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 1) : "memory");
    __syncwarp();  // the warp's copies are for all its lanes
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t at = from + slot + h * (2 * kLoraThreads * 16);
      lora_matrix(at, w[h][0]);
      lora_matrix(at ^ 32, w[h][1]);
    }
  }
  // Where a stage has values 4 c to 4 c + 3 of a vector's 32, x or base: 128
  // bytes a vector, so that a copy takes whole lines, in an order in which the
  // lanes' reads, of four vectors at a time, fall into different banks.
  __device__ __forceinline__ uint32_t x_place(int vec, int c) const {
    return (4 + vec / 4) * (kLoraThreads * 16) + warp * 512 + vec % 4 * 128 + (c ^ (vec & 3) * 2) * 16;
  }
  __device__ __forceinline__ uint32_t base_place(int vec, int c) const {
    return (4 + vec / 4) * (kLoraThreads * 16) + warp * 512 + vec % 4 * 128 + (c ^ (vec & 6)) * 16;
  }
  // A warp's sums of a tile of 16 ranks by eight vectors, 512 bytes: in its part of the stage that
  // is free when its first product ends (stage `slot`), beyond that stage's pieces in t's place.
  __device__ __forceinline__ float* sums(LoraShared& s, unsigned char* pieces, int slot, int w, int tile) const {
    if (tile < S::kPieces) return reinterpret_cast<float*>(pieces + slot + tile * (kLoraThreads * 16) + w * 512);
    return reinterpret_cast<float*>(s.t) + (w * (S::kTiles * N - S::kPieces) + tile - S::kPieces) * 128;
  }
};
static_assert(kLoraWarps * (LoraTile<1>::kTiles - LoraTile<1>::kPieces) * 512 <= sizeof(LoraShared::t), "sums");
static_assert(LoraTile<2>::kTiles * 2 <= LoraTile<2>::kPieces, "sums");
static_assert(2 * 8 * (128 + 4) * 4 <= sizeof(LoraShared::t) && 3 * 8 * (128 + 32) * 2 <= sizeof(LoraShared::t), "t");
static_assert(2 * 16 * (64 + 4) * 4 <= sizeof(LoraShared::t) && 3 * 16 * (64 + 32) * 2 <= sizeof(LoraShared::t), "t");

// A barrier of the CTAs first .. first + count - 1 of the cluster: every CTA has one, each arrives
// at everyone's and waits at its own.  The CTA's threads are at one before they arrive.
__device__ __forceinline__ void half_arrive(uint64_t& bar, int first, int count) {
  if (int(threadIdx.x) < count)
    asm volatile("{\n.reg .b32 a;\nmapa.shared::cluster.u32 a, %0, %1;\nmbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n}" ::"r"(
                     smem_addr(&bar)), "r"(first + int(threadIdx.x)) : "memory");
}
// (Bounded; a wait that gives up is reported, and the launch's results are not to be used.)
__device__ __forceinline__ void half_wait(uint64_t& bar, uint32_t parity, unsigned* status) {
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(done) : "r"(smem_addr(&bar)), "r"(parity) : "memory");
    if (done) return;
    if (i == 0) t0 = globaltimer();
    if ((i & 63) == 63 && globaltimer() - t0 > 1000000000ull) break;
  }
  atomicOr(status, kStatusWaitTimeout);
}

// One bucket.  VEC: base and out rows start on 16 bytes, rows is even.
template <class T, int N, bool VEC>
__device__ __forceinline__ void lora_bucket(LoraShared& sh, unsigned char* pieces, LoraPart<T, N, VEC>& part, float scale,
                                            unsigned* status) {
  using S = LoraTile<N>;
  using M = LoraMul<T>;
  const int quad = part.quad, piece = part.piece, count = part.count;
#pragma unroll 1
  for (int i = 0; i < S::kStages - 1; ++i) part.fetch();

  float acc[S::kTiles][N][4];
#pragma unroll
  for (int i = 0; i < S::kTiles; ++i)
#pragma unroll
    for (int g = 0; g < N; ++g)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][g][j] = 0.f;
  int slot = 0;
#pragma unroll 1
  for (int block = part.warp; block * 32 < part.slice; block += kLoraWarps) {
    const int left = part.slice - block * 32;
    typename M::X x[N];
#pragma unroll 1
    for (int p = 0; p < part.pairs; ++p) {
      LoraWeights w;
      part.fetch();
      part.take(slot, w);
      if (left < 32) {  // both operands are zero past the slice, a multiple of 8
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t& v = w[i >> 1][c >> 1][(c & 1) * 2 + (i & 1)];
            v = c * 8 < left ? v : 0u;
          }
      }
      if (p == 0) {
#pragma unroll
        for (int g = 0; g < N; ++g) {
          float f[8];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float2 u = *reinterpret_cast<const float2*>(pieces + slot + part.x_place(g * 8 + quad, 2 * c + piece / 2) + piece % 2 * 8);
            f[2 * c] = c * 8 < left ? u.x : 0.f, f[2 * c + 1] = c * 8 < left ? u.y : 0.f;
          }
          M::split(f, x[g]);
        }
      }
      slot = part.after(slot);
      // The tiles' sums are registers, so each pair has its own code; the copies' has one place.
#pragma unroll
      for (int q = 0; q < S::kTiles / 2; ++q)
        if (p == q) lora_mma<T, N>(acc[2 * q], acc[2 * q + 1], w, x);
    }
  }
  // The warps' sums, then in order.
#pragma unroll
  for (int i = 0; i < S::kTiles; ++i) {
    if (i >= part.tiles) break;
#pragma unroll
    for (int g = 0; g < N; ++g) {
      float* dst = part.sums(sh, pieces, part.f_slot, part.warp, i * N + g) + quad * 8 + piece * 2;
      *reinterpret_cast<float2*>(dst) = make_float2(acc[i][g][0], acc[i][g][1]);
      *reinterpret_cast<float2*>(dst + 64) = make_float2(acc[i][g][2], acc[i][g][3]);
    }
  }
  if (part.lane == 0) sh.slot[part.warp] = part.f_slot;
  __syncthreads();
  const int sums = part.tiles * N * 128;
#pragma unroll 1
  for (int i = threadIdx.x; i < sums; i += kLoraThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kLoraWarps; ++w) v = __fadd_rn(v, part.sums(sh, pieces, sh.slot[w], w, i >> 7)[i & 127]);
    sh.mine[i] = v;
  }
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = 1 << sh.log, first = int(cluster.block_rank()) & -ctas;
  if (sh.halves) {
    __syncthreads();
    half_arrive(sh.ready, first, ctas);
    half_wait(sh.ready, sh.parity, status);
  } else {
    cluster.sync();
  }
#pragma unroll 1
  for (int i = threadIdx.x; i < sums; i += kLoraThreads) {
    const int row = i / (N * 128) * 16 + (i & 127) / 8, vec = (i >> 7) % N * 8 + (i & 7);
    float s[16], v = 0.f;  // up to 16 CTAs share a bucket: all reads at once, added in order
#pragma unroll
    for (int k = 0; k < 16; ++k) s[k] = vec < count && k < ctas ? cluster.map_shared_rank(sh.mine, first + k)[i] : 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) v = __fadd_rn(v, s[k]);
    v = row < part.rank ? __fmul_rn(v, scale) : 0.f;  // rows past the rank are old values' products
    M::template store<S::kTokens, S::kMaxRank>(sh.t, vec, row, v);
  }
  // Rank values past the last tile, up to a multiple of 32, are zero.
  if (part.tiles * 16 < part.ranks32 * 32) {
#pragma unroll 1
    for (int i = threadIdx.x; i < (part.ranks32 * 32 - part.tiles * 16) * S::kTokens; i += kLoraThreads)
      M::template store<S::kTokens, S::kMaxRank>(sh.t, i % S::kTokens, part.tiles * 16 + i / S::kTokens, 0.f);
  }
  // Others' `mine` has been read; own t is complete.  That this CTA's has been read is waited for at the end.
  __syncthreads();
  if (sh.halves)
    half_arrive(sh.read, first, ctas);
  else
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

  // Second product.  A lane's outputs: two neighbouring rows (and the same
  // sixteen rows further on) of vectors 2 piece and 2 piece + 1.
  const int row_lane = part.warp * 32 + quad * 2;
  const uint32_t t = smem_addr(sh.t);
#pragma unroll 1
  for (int row0 = 0; row0 < part.rows; row0 += 256) {
    float c[2][N][4] = {};
    float2 base[2 * N][2];
#pragma unroll 1
    for (int k = 0; k < part.ranks32; ++k) {
      LoraWeights w;
      part.fetch();
      part.take(slot, w);
      if (k == 0) {
#pragma unroll
        for (int u = 0; u < 2 * N; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            base[u][h] = *reinterpret_cast<const float2*>(pieces + slot + part.base_place((u >> 1) * 8 + piece * 2 + (u & 1), h * 4 + quad / 2) +
                                                          quad % 2 * 8);
      }
      slot = part.after(slot);
      // Values past the adapter's rank may be anything: zero, like their t.
      if (k * 32 + 32 > part.rank) {
        const int inside = part.rank - k * 32 - piece * 2;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t& v = w[i >> 1][c >> 1][(c & 1) * 2 + (i & 1)];
            v = inside >= c * 8 + 2 ? v : inside == c * 8 + 1 ? v & 0xffffu : 0u;
          }
      }
      typename M::X x[N];
#pragma unroll
      for (int g = 0; g < N; ++g) M::template load<S::kTokens, S::kMaxRank>(t, g * 8 + quad, k * 32 + piece * 8, x[g]);
      lora_mma<T, N>(c[0], c[1], w, x);
    }
#pragma unroll
    for (int u = 0; u < 2 * N; ++u) {
      const int vec = (u >> 1) * 8 + piece * 2 + (u & 1);
      if (vec >= count) continue;
      float* dst = sh.out[vec] + row0 + row_lane;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = row0 + row_lane + h * 16;
        if (row >= part.rows) continue;
        const float r = __fadd_rn(base[u][h].x, c[0][u >> 1][2 * h + (u & 1)]);
        const float r1 = __fadd_rn(base[u][h].y, c[1][u >> 1][2 * h + (u & 1)]);
        if constexpr (VEC) {
          *reinterpret_cast<float2*>(dst + h * 16) = make_float2(r, r1);
        } else {
          dst[h * 16] = r;
          if (row + 1 < part.rows) dst[h * 16 + 1] = r1;
        }
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  if (sh.halves)
    half_wait(sh.read, sh.parity, status);
  else
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// A bucket of sh.count vectors.
template <class T, int N, bool VEC>
__device__ __forceinline__ void lora_part(const T* A, const T* B, int n, int a_rank, int rank, int slice, int rows, float scale,
                                          unsigned* status) {
  LoraShared& sh = *reinterpret_cast<LoraShared*>(lora_smem);
  unsigned char* ring = lora_smem + kLoraRingAt;
  const int lane = threadIdx.x & 31;
  LoraPart<T, N, VEC> part(sh);
  part.rank = rank, part.a_rank = a_rank, part.count = sh.count;
  part.rows = rows, part.slice = slice;
  part.tiles = (rank + 15) / 16, part.pairs = max(1, (part.tiles + 1) / 2);
  part.ranks32 = max(1, (rank + 31) / 32);
  part.warp = __shfl_sync(0xffffffffu, int(threadIdx.x) >> 5, 0), part.lane = lane, part.quad = lane >> 2, part.piece = lane & 3;
  part.ring = smem_addr(ring);
  part.start(A, B, n);
  lora_bucket<T, N, VEC>(sh, ring, part, scale, status);
}
template <class T, int N, bool VEC>
__global__ void __launch_bounds__(kLoraThreads, 2) k_lora_add(LoraArgs a) {
  using S = LoraTile<N>;
  LoraShared& sh = *reinterpret_cast<LoraShared*>(lora_smem);
  pdl_launch_dependents();
  pdl_wait();
  const int clusters = int(gridDim.x) >> a.log_cluster, own = int(blockIdx.x) >> a.log_cluster;
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
  const auto adapter_of = [&](int u) {  // -1: none, -2: past the end
    if (u >= a.nvec) return -2;
    const int i = a.index[u];
    return i >= 0 && i < a.adapters ? i : -1;
  };
  // With a cluster for each vector a cluster looks at its own vector.  Else every
  // CTA counts the buckets, a window a warp, and (half) cluster i of m takes buckets i, i +
  // m, ... (looking at every so many-th vector cost 8000 cycles a bucket,
  // and some clusters found two buckets and others none).
  const bool few = a.nvec <= clusters;
  int next = 0, seen = 0;  // this CTA's next bucket, buckets of the rounds before
  if (few && threadIdx.x == 0) sh.log = a.log_cluster, sh.step = sh.total = 1, sh.halves = false;
#pragma unroll 1
  for (int from = 0; from < a.nvec; from += kLoraRound) {
    if (!few) {
      const int u = from + warp * kLoraWindow + lane;
      const int lo = adapter_of(u), hi = adapter_of(u + 32);
      int before = 0;  // vectors of hi's adapter among the window's first 32
#pragma unroll 8
      for (int i = 0; i < 32; ++i) before += __shfl_sync(0xffffffffu, lo, i) == hi;
      const uint32_t below = (1u << lane) - 1u;
      const int lo_nth = __popc(__match_any_sync(0xffffffffu, lo) & below);
      const int hi_nth = before + __popc(__match_any_sync(0xffffffffu, hi) & below);
      const uint32_t lo_leads = __ballot_sync(0xffffffffu, lo != -2 && lo_nth % S::kTokens == 0);
      const uint32_t hi_leads = __ballot_sync(0xffffffffu, hi != -2 && hi_nth % S::kTokens == 0);
      __syncthreads();  // the last round's are not needed any more
      if (lane == 0) sh.leads[warp] = uint64_t(hi_leads) << 32 | lo_leads;
      sh.adapter[warp * kLoraWindow + lane] = lo, sh.adapter[warp * kLoraWindow + 32 + lane] = hi;
      __syncthreads();
      if (threadIdx.x == 0) {
        int total = 0;
        for (int w = 0; w < kLoraWarps; ++w) total += __popcll(sh.leads[w]);
        sh.total = seen + total;
        if (from == 0) {
          // The first round's buckets tell how many there are: a cluster each where they run
          // at once (36 of eight CTAs do), else half a cluster each.  f16, rank 64, 4096 to
          // 14336: 64 vectors of 32 adapters 20.3 us with whole clusters, 32 with halves; of 64
          // adapters 38.8 and 33.1; 128 vectors of 64 (100 buckets) 64.8 and 59, 256 of 256 204 and 121.
          const int64_t buckets = a.nvec > kLoraRound ? int64_t(total) * a.nvec / kLoraRound : total;
          const int half = buckets > clusters ? 1 : 0;
          sh.log = a.log_cluster - half, sh.step = clusters << half, sh.halves = half;
          if (half) {
            mbar_init(smem_addr(&sh.ready), 1 << sh.log), mbar_init(smem_addr(&sh.read), 1 << sh.log);
            fence_barrier_init();
            sh.parity = 1;
          }
        }
      }
      __syncthreads();
      if (from == 0) {
        const int half = a.log_cluster - sh.log;
        next = own << half | (int(blockIdx.x) & ((1 << a.log_cluster) - 1)) >> sh.log;
        if (half) cg::this_cluster().sync();  // everyone's barriers are there
      }
    }
#pragma unroll 1
    for (; next < sh.total; next += sh.step) {
      int v = own;
      if (!few) {
        int w = 0, nth = next - seen;
        uint64_t leads;
        for (;; ++w) {
          leads = sh.leads[w];
          const int n = __popcll(leads);
          if (nth < n) break;
          nth -= n;
        }
#pragma unroll 1
        for (; nth > 0; --nth) leads &= leads - 1;
        v = from + w * kLoraWindow + __ffsll(int64_t(leads)) - 1;
      }
      const int w0 = v / kLoraWindow * kLoraWindow;
      int adapter, near[kLoraWindow / 32];
      if (few) {  // one round of loads
        adapter = a.index[v];
#pragma unroll
        for (int h = 0; h < kLoraWindow / 32; ++h) near[h] = a.index[min(w0 + h * 32 + lane, a.nvec - 1)];
        adapter = adapter >= 0 && adapter < a.adapters ? adapter : -1;
#pragma unroll
        for (int h = 0; h < kLoraWindow / 32; ++h)
          near[h] = w0 + h * 32 + lane >= a.nvec ? -2 : near[h] >= 0 && near[h] < a.adapters ? near[h] : -1;
      } else {
        adapter = sh.adapter[v - from];
#pragma unroll
        for (int h = 0; h < kLoraWindow / 32; ++h) near[h] = sh.adapter[w0 - from + h * 32 + lane];
      }
      const int log = few ? a.log_cluster : sh.log, c = int(blockIdx.x) & ((1 << log) - 1);
      const int per_n = ((a.n / 8 + (1 << log) - 1) >> log) * 8, per_r = (((a.rows + 3) / 4 + (1 << log) - 1) >> log) * 4;
      const int j0 = min(a.n, c * per_n), r0 = min(a.rows, c * per_r);
      const int ranks = adapter >= 0 && a.ranks ? a.ranks[adapter] : a.rank;
      const float scale = adapter >= 0 && a.scale ? a.scale[adapter] : 1.f;
      // Warp 0 looks at the window: which of its vectors have v's adapter.
      if (warp == 0) {
        uint64_t same = 0;
#pragma unroll
        for (int h = 0; h < kLoraWindow / 32; ++h) same |= uint64_t(__ballot_sync(0xffffffffu, near[h] == adapter)) << (32 * h);
        const int before = __popcll(same & ((uint64_t(1) << (v - w0)) - 1));
        const uint64_t rest = same >> (v - w0) << (v - w0);
        // The first kTokens of the rest, each by the lane of its place.
        const bool lead = before % S::kTokens == 0;
#pragma unroll
        for (int h = 0; h < kLoraWindow / 32; ++h) {
          const int at = h * 32 + lane, nth = __popcll(rest & ((uint64_t(1) << at) - 1));
          if (lead && (rest >> at & 1) && nth < S::kTokens) {
            const int64_t token = w0 + at;
            sh.x[nth] = a.x + token * a.ldx + j0;
            sh.base[nth] = a.base + token * a.ldb + r0;
            sh.out[nth] = a.out + token * a.ldo + r0;
            if (adapter < 0 && a.index[token] != -1) atomicOr(a.status, kStatusBadIndex);
          }
        }
        if (lane == 0) sh.count = lead ? min(S::kTokens, __popcll(rest)) : 0;
        if (lane == 0 && adapter >= 0) sh.parity ^= 1;
      }
      __syncthreads();
      const int count = sh.count, rows = min(a.rows, r0 + per_r) - r0;
      if (count && adapter < 0) {
        if (a.out != a.base) {
#pragma unroll 1
          for (int i = 0; i < count; ++i)
#pragma unroll 1
            for (int r = threadIdx.x; r < rows; r += kLoraThreads) sh.out[i][r] = sh.base[i][r];
        }
      } else if (count) {
        const int rank = max(0, min(ranks, a.rank));
        const T* A = static_cast<const T*>(a.wa) + int64_t(adapter) * a.rank * a.n + j0;
        const T* B = static_cast<const T*>(a.wb) + (int64_t(adapter) * a.rows + r0) * a.rank;
        const int slice = rank ? min(a.n, j0 + per_n) - j0 : 0;  // rank 0: no first product
        lora_part<T, N, VEC>(A, B, a.n, a.rank, rank, slice, rows, scale, a.status);
      }
      __syncthreads();  // sh is free again
    }
    if (few) return;
    seen = sh.total;
  }
  if (sh.halves) cg::this_cluster().sync();  // no one arrives at a CTA that has left
}

// Launches in clusters of 1 << log CTAs: how many of them run at once, and (`g`) the call, with a
// cluster for each vector where they do, else as many as do.
template <class T, int N, bool VEC>
static int launch_lora(int log, int& once, const LoraArgs* call, cudaStream_t s) {
  using S = LoraTile<N>;
  constexpr int kSmem = kLoraRingAt + S::kRing;
  const char* who = "q1_lora_add launch";
  const auto kernel = k_lora_add<T, N, VEC>;
  static bool set[64] = {};
  static int most[64][5] = {};
  int dev = 0;
  if (int e = cuda_status(cudaGetDevice(&dev), who)) return e;
  const bool known = dev >= 0 && dev < 64;
  if (!known || !set[dev]) {
    if (int e = cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem), who)) return e;
    if (int e = cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1), who)) return e;
    if (known) set[dev] = true;
  }
  once = known ? most[dev][log] : 0;
  if (!once) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1u << log, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(1u << log), cfg.blockDim = dim3(kLoraThreads), cfg.dynamicSmemBytes = kSmem;
    cfg.attrs = &attr, cfg.numAttrs = 1;
    if (int e = cuda_status(cudaOccupancyMaxActiveClusters(&once, kernel, &cfg), who)) return e;
    once = max(once, 1);
    if (known) most[dev][log] = once;
  }
  if (!call) return Q1_OK;
  LoraArgs g = *call;
  g.log_cluster = log;
  const dim3 grid(unsigned((g.nvec < once ? g.nvec : once) << log));
  return launch_op(kernel, grid, kLoraThreads, kSmem, 1 << log, s, who, g);
}

template <class T, bool VEC>
static int launch_lora(const LoraArgs& g, cudaStream_t s) {
  // Clusters of sixteen CTAs while halves of those that run at once are enough for every vector:
  // one vector of rank 16, 4096 x 4096, 4.8 us against 5.6 with eight; 20 of rank 64, 4096 to
  // 14336, of one adapter 10.9 against 14.3, of 20 19.0 against 18.9.
  int once;
  if (int e = launch_lora<T, 1, VEC>(4, once, nullptr, s)) return e;
  if (g.nvec <= 2 * once) return launch_lora<T, 1, VEC>(4, once, &g, s);
  if (int e = launch_lora<T, 1, VEC>(3, once, nullptr, s)) return e;
  // Buckets of sixteen vectors pay where those of eight are more than run at once even if all are
  // full, and if they fill: 1000 vectors of one adapter 52 us against 62 in eights, 384 29 against 32, but
  // 192 27.5 against 19.5; in runs of 16 tokens 78 against 63 (1000 of 62), of 12 in any order 70 against
  // 53 (300 of 18).  Runs of 32 break even.  How many adapters there are bounds those in use, and
  // is all that the host knows; of prompts of few adapters out of many it makes eights (in
  // one kernel that has both, which the device could choose from, either takes a third longer,
  // and a launch of each, one of which leaves, 2 to 6 us).
  if (g.nvec > 8 * once && g.nvec >= 32 * int64_t(g.adapters) && g.rank <= LoraTile<2>::kMaxRank)
    return launch_lora<T, 2, VEC>(3, once, &g, s);
  return launch_lora<T, 1, VEC>(3, once, &g, s);
}

}  // namespace q1

using namespace q1;

extern "C" int q1_lora_add(const float* x, int64_t ldx, int64_t nvec, int64_t n, int64_t rows, const void* a,
                           const void* b, int dtype, int64_t adapters, int64_t rank, const int32_t* index,
                           const int32_t* ranks, const float* scale, const float* base, int64_t ldb, float* out,
                           int64_t ldo, void* stream) {
  const char* who = "q1_lora_add";
  if (nvec < 1 || nvec > 65535 || n < 8 || n > (int64_t(1) << 24) || n % 8 || rows < 1 || rows > (int64_t(1) << 26) ||
      adapters < 1 || adapters > (1 << 20) || rank < 8 || rank > LoraTile<1>::kMaxRank || rank % 8)
    return fail(Q1_ERR_ARG, "%s: bad shape nvec=%lld n=%lld rows=%lld adapters=%lld rank=%lld (n and rank multiples of 8, "
                "rank in 8..128)", who, (long long)nvec, (long long)n, (long long)rows, (long long)adapters, (long long)rank);
  if (dtype != Q1_BF16 && dtype != Q1_F16) return fail(Q1_ERR_ARG, "%s: bad weight type %d", who, dtype);
  if (!x || !a || !b || !index || !base || !out) return fail(Q1_ERR_ARG, "%s: null pointer", who);
  if (!aligned16(x) || !aligned16(a) || !aligned16(b) || ldx % 4 || reinterpret_cast<uintptr_t>(base) % 4 ||
      reinterpret_cast<uintptr_t>(out) % 4)
    return fail(Q1_ERR_ARG, "%s: x, a and b must be 16-byte aligned, rows of x multiples of 4", who);
  if (!aligned4(index) || !aligned4(ranks) || !aligned4(scale))
    return fail(Q1_ERR_ARG, "%s: index, ranks and scale must be 4-byte aligned", who);
  if (ldx < n || ldb < rows || ldo < rows) return fail(Q1_ERR_ARG, "%s: a row stride is less than its row", who);
  if (base == out && ldb != ldo) return fail(Q1_ERR_ARG, "%s: in place, base and out need the same stride", who);
  LoraArgs g = {x, a, b, index, ranks, scale, base, out, nullptr, ldx, ldb, ldo, int(nvec), int(n), int(rows), int(rank),
                int(adapters), 0};
  if (int e = ops_status_ptr(&g.status)) return e;
  const bool vec = aligned16(base) && aligned16(out) && ldb % 4 == 0 && ldo % 4 == 0 && rows % 2 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == Q1_BF16) return vec ? launch_lora<__nv_bfloat16, true>(g, s) : launch_lora<__nv_bfloat16, false>(g, s);
  return vec ? launch_lora<__half, true>(g, s) : launch_lora<__half, false>(g, s);
}
