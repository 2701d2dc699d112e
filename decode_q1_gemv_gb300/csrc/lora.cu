// lora.cu -- q1_lora_add: out_v = base_v + scale_a * B_a (A_a x_v) for the
// adapter a of each vector v, many adapters in one launch.
//
// Few vectors share an adapter, so each adapter's A (rank x n) and B (rows x
// rank) have to be read about once and take 2 operations a value and vector:
// bytes bound it, and for one vector the chain of dependent memory reads.
// Both products run in one launch: a cluster of CTAs takes one bucket (up to
// kLoraTokens vectors of one adapter), each CTA a slice of n in the first
// product and a slice of the rows in the second; the rank values between them
// (at most 128 a vector) pass through distributed shared memory, so there is
// no workspace and no second launch.  Sums are f32 in a fixed order: the
// lanes' chains over a slice, the butterfly of a warp, the warps' parts, the
// cluster's slices.
//
// Vectors are grouped on the device: in a window of 64 vectors, every
// kLoraTokens-th vector of an adapter leads a bucket of it and the next ones
// of that window.  A cluster whose vector leads no bucket has nothing to do.
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

constexpr int kLoraTokens = 8;    // vectors of a bucket
constexpr int kLoraWindow = 64;   // vectors among which buckets form
constexpr int kLoraLogThreads = 8, kLoraThreads = 1 << kLoraLogThreads;
constexpr int kLoraMaxRank = 128;
constexpr int kLoraStages = 4;    // chunks of 16 KB in flight: 64 KB a CTA, two CTAs an SM
constexpr int kLoraRing = kLoraStages * 4 * kLoraThreads * 16;
constexpr int kLoraX = 8192;      // values of x in shared memory: of all vectors of the bucket
constexpr int kLoraSmem = kLoraRing + kLoraX * 4;

struct LoraShared {
  float part[kLoraThreads / 8][4 * kLoraTokens];       // (quad, warp of it): the sums of four rank rows
  float mine[kLoraMaxRank][kLoraTokens];               // this CTA's slice of n
  float t[kLoraMaxRank][kLoraTokens];                  // all slices, scaled
  int token[kLoraTokens];
  int count;
};

__device__ __forceinline__ void lora_copy(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

// Sums of v over the lanes of aligned groups of `width` lanes, where each
// halving step gives a lane half of the values it still has: afterwards lane
// i of a group holds `Keep` consecutive sums.
template <int N>
__device__ __forceinline__ void fold(float (&v)[N], int width, int lane) {
  if constexpr (N > 1) {
    if (width > 1) {
      const int half = width / 2;
      const bool up = lane & half;
      float r[N / 2];
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float send = up ? v[i] : v[i + N / 2], keep = up ? v[i + N / 2] : v[i];
        r[i] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, send, half));
      }
      fold<N / 2>(r, half, lane);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) v[i] = r[i];
    }
  } else {
    for (int half = width / 2; half > 0; half >>= 1) v[0] = __fadd_rn(v[0], __shfl_xor_sync(0xffffffffu, v[0], half));
  }
}

// What a CTA has to do for a bucket: a slice of n of the first product, then a
// slice of the rows of the second, both cut into chunks in which every thread
// has four 16-byte pieces of weights:
//   first:  four rank rows (quad) at one piece of n (part); parts * 8 values of
//           n a chunk, parts a power of two;
//   second: four rows at one piece of the rank; `width` (a power of two) lanes
//           share a row.
struct LoraSplit {
  int rank, r0, r1, slice;   // rank in use; rows; values of n
  int quads;                 // of four rank rows: a power of two, as are
  int parts, width;          // parts = 1 << lparts and width = 1 << lwidth
  int lparts, lwidth;
  int down, up;              // chunks of each product
  // The calling thread's place: in the first product its quad and part, in the
  // second the first row of a chunk and its piece.
  int quad, part, row, piece;
  const void* a0;            // its first piece in A (row quad * 4), chunks parts * 8 values apart
  const void* b0;            // its first piece in B (row r0 + row), chunks 4 * 256 / width rows apart
  int b_step;                // values of B from one chunk to the next
};

// The least k with 2^k >= v, v >= 0 (0 for 0 and 1).
__device__ __forceinline__ int log2_from(int v) { return v <= 1 ? 0 : 32 - __clz(v - 1); }

// Asynchronous copies of chunk c (of both products in turn) into the calling
// thread's own places of the ring; what lies past an end reads as zero.
template <class T>
__device__ __forceinline__ void lora_fetch(const LoraArgs& a, const LoraSplit& s, uint32_t ring, int c) {
  const uint32_t dst = ring + (c % kLoraStages) * (4 * kLoraThreads * 16) + threadIdx.x * 16;
  if (c < s.down) {
    const T* src = static_cast<const T*>(s.a0) + c * s.parts * 8;
    const bool inside = (c * s.parts + s.part) * 8 < s.slice;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const bool live = inside && s.quad * 4 + r < s.rank;
      lora_copy(dst + r * (kLoraThreads * 16), live ? src : static_cast<const T*>(a.wa), live);
      src += a.n;
    }
  } else if (c < s.down + s.up) {
    const int k = c - s.down, left = s.r1 - s.r0 - s.row - k * (4 * kLoraThreads >> s.lwidth);
    const T* src = static_cast<const T*>(s.b0) + int64_t(k) * s.b_step;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const bool live = r < left && s.piece * 8 < s.rank;
      lora_copy(dst + r * (kLoraThreads * 16), live ? src : static_cast<const T*>(a.wb), live);
      src += a.rank;
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// The thread's four pieces of chunk c, and the copies of the chunk that takes
// the place of the one before it.
template <class T>
__device__ __forceinline__ void lora_pieces(const LoraArgs& a, const LoraSplit& s, unsigned char* ring, int c, float (&w)[4][8]) {
  lora_fetch<T>(a, s, smem_addr(ring), c + kLoraStages - 1);
  asm volatile("cp.async.wait_group %0;" ::"n"(kLoraStages - 1) : "memory");
#pragma unroll
  for (int r = 0; r < 4; ++r)
    Elem<T>::unpack(*reinterpret_cast<const uint4*>(ring + (((c % kLoraStages) * 4 + r) * kLoraThreads + threadIdx.x) * 16), w[r]);
}

// Copies x from element j0 on (`count` of them, a multiple of 8) of the
// bucket's vectors into shared memory, 16-byte pieces of even and odd number
// apart ([vector][2][window / 8]), so that neighbouring lanes read
// neighbouring pieces.
template <int M>
__device__ __forceinline__ void lora_fetch_x(const LoraArgs& a, const LoraShared& sh, uint32_t xs, int j0, int count) {
  constexpr int kWindow = kLoraX / M;
#pragma unroll
  for (int i = 0; i < M; ++i) {
    const float* x = a.x + sh.token[i] * a.ldx + j0;
#pragma unroll 1
    for (int p = threadIdx.x; p < count / 4; p += kLoraThreads)
      lora_copy(xs + (i * (kWindow / 4) + (p & 1) * (kWindow / 8) + p / 2) * 16, x + p * 4, true);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// First product: mine[k][i] = sum over this CTA's slice of A[k] x_i, k < rank.
// The first window of x is under way (before the ring's first chunks).
template <class T, int M>
__device__ __forceinline__ void lora_down(const LoraArgs& a, LoraShared& sh, const LoraSplit& s, unsigned char* ring, int j0) {
  constexpr int kWindow = kLoraX / M;  // at least parts * 8: a window is whole chunks
  constexpr int kLog4M = M == 1 ? 2 : M == 2 ? 3 : M == 4 ? 4 : 5;
  static_assert(kLoraX / kLoraTokens >= 1024, "a chunk of rank 8 (parts * 8 = 1024) fits the smallest window");
  const int lane = threadIdx.x & 31;
  const float4* xs = reinterpret_cast<const float4*>(ring + kLoraRing);
  asm volatile("cp.async.wait_group %0;" ::"n"(kLoraStages - 1) : "memory");
  __syncthreads();
  float acc[4 * M];
#pragma unroll
  for (int i = 0; i < 4 * M; ++i) acc[i] = 0.f;
#pragma unroll 1
  for (int c = 0; c < s.down; ++c) {
    const int j = (c * s.parts + s.part) * 8;
    if (c > 0 && c * s.parts * 8 % kWindow == 0) {  // the next window of x
      __syncthreads();
      lora_fetch_x<M>(a, sh, smem_addr(xs), j0 + c * s.parts * 8, min(kWindow, s.slice - c * s.parts * 8));
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();
    }
    float w[4][8];
    lora_pieces<T>(a, s, ring, c, w);
    if (j >= s.slice) continue;
    const float4* xj = xs + j % kWindow / 8;
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const float4 lo = xj[i * (kWindow / 4)], hi = xj[i * (kWindow / 4) + kWindow / 8];
      const float xv[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r * M + i] = __fmaf_rn(w[r][e], xv[e], acc[r * M + i]);
    }
  }
  // Over the parts: the lanes of a quad, then (more than 32 parts) its warps.
  const int width = s.parts < 32 ? s.parts : 32, lwarps = s.parts < 32 ? 0 : s.lparts - 5;
  fold<4 * M>(acc, width, lane);
  // A lane holds 4 M / width sums, or one that width / (4 M) lanes share.
  const int at = lane & (width - 1), lshare = s.parts < 32 ? s.lparts - kLog4M : 5 - kLog4M;
  const int keep = lshare > 0 ? 1 : 1 << -lshare;
  if ((at & ((1 << (lshare > 0 ? lshare : 0)) - 1)) == 0) {
    float* dst = sh.part[(s.quad << lwarps) + s.part / 32] + (lshare > 0 ? at >> lshare : at << -lshare);
#pragma unroll
    for (int i = 0; i < 4 * M; ++i)
      if (i < keep) dst[i] = acc[i];
  }
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i < s.quads * 4 * M; i += kLoraThreads) {
    float v = 0.f;
#pragma unroll 1
    for (int p = 0; p < 1 << lwarps; ++p) v = __fadd_rn(v, sh.part[(i / (4 * M) << lwarps) + p][i % (4 * M)]);
    sh.mine[i / M][i % M] = v;
  }
}

// Second product: rows [r0, r1) of B t for the bucket's vectors.
template <class T, int M, bool VEC>
__device__ __forceinline__ void lora_up(const LoraArgs& a, const LoraShared& sh, const LoraSplit& s, unsigned char* ring) {
  const int lane = threadIdx.x & 31, piece = s.piece;
  // A row's lanes share out the vectors to write: `keep` each, from `first` on.
  constexpr int kLogM = M == 1 ? 0 : M == 2 ? 1 : M == 4 ? 2 : 3;
  const int lshare = s.lwidth - kLogM, keep = lshare > 0 ? 1 : 1 << -lshare;
  const int first = lshare > 0 ? piece >> lshare : piece << -lshare;
  const bool writes = (piece & ((1 << (lshare > 0 ? lshare : 0)) - 1)) == 0;
  float t[8][M];
#pragma unroll
  for (int e = 0; e < 8; ++e)
#pragma unroll
    for (int i = 0; i < M; ++i) t[e][i] = piece * 8 + e < s.rank ? sh.t[piece * 8 + e][i] : 0.f;
  // The values that the chunk's results are added to, read one chunk ahead.
  constexpr int kKeep = M > 1 ? M / 2 : 1;
  float4 next[kKeep];
  const int step = 4 * kLoraThreads >> s.lwidth;  // rows of a chunk
  const auto fetch_base = [&](int row) {
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      next[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!writes || i >= keep || first + i >= sh.count) continue;
      const float* in = a.base + sh.token[first + i] * a.ldb + row;
      if constexpr (VEC) {  // rows is a multiple of four
        if (row < s.r1) next[i] = *reinterpret_cast<const float4*>(in);
      } else {
        if (row < s.r1) next[i].x = in[0];
        if (row + 1 < s.r1) next[i].y = in[1];
        if (row + 2 < s.r1) next[i].z = in[2];
        if (row + 3 < s.r1) next[i].w = in[3];
      }
    }
  };
  int row = s.r0 + s.row;
  fetch_base(row);
#pragma unroll 1
  for (int c = 0; c < s.up; ++c, row += step) {  // whole warps stay together
    float4 base[kKeep];
#pragma unroll
    for (int i = 0; i < kKeep; ++i) base[i] = next[i];
    if (c + 1 < s.up) fetch_base(row + step);
    float w[4][8], f[4][M];
    lora_pieces<T>(a, s, ring, s.down + c, w);
    if (piece * 8 + 8 > s.rank) {  // values past the adapter's rank may be anything
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int r = 0; r < 4; ++r) w[r][e] = piece * 8 + e < s.rank ? w[r][e] : 0.f;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
      for (int i = 0; i < M; ++i) {
        f[r][i] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[r][i] = __fmaf_rn(w[r][e], t[e][i], f[r][i]);
      }
      fold<M>(f[r], s.width, lane);
    }
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      if (!writes || i >= keep || first + i >= sh.count) continue;
      float* out = a.out + sh.token[first + i] * a.ldo + row;
      const float4 v = make_float4(__fadd_rn(base[i].x, f[0][i]), __fadd_rn(base[i].y, f[1][i]), __fadd_rn(base[i].z, f[2][i]),
                                   __fadd_rn(base[i].w, f[3][i]));
      if constexpr (VEC) {
        if (row < s.r1) *reinterpret_cast<float4*>(out) = v;
      } else {
        if (row < s.r1) out[0] = v.x;
        if (row + 1 < s.r1) out[1] = v.y;
        if (row + 2 < s.r1) out[2] = v.z;
        if (row + 3 < s.r1) out[3] = v.w;
      }
    }
  }
}

template <class T, int M, bool VEC>
__device__ __forceinline__ void lora_bucket(const LoraArgs& a, LoraShared& sh, const LoraSplit& s, unsigned char* ring,
                                            int j0, float scale, cg::cluster_group& cluster) {
  const int C = int(cluster.num_blocks());
  lora_fetch_x<M>(a, sh, smem_addr(ring + kLoraRing), j0, min(kLoraX / M, s.slice));
#pragma unroll 1
  for (int i = 0; i < kLoraStages - 1; ++i) lora_fetch<T>(a, s, smem_addr(ring), i);
  lora_down<T, M>(a, sh, s, ring, j0);
  cluster.sync();
#pragma unroll 1
  for (int i = threadIdx.x; i < s.rank * M; i += kLoraThreads) {
    float v = 0.f;
    for (int p = 0; p < C; p += 4) {  // four reads at a time; a cluster has 4, 8 or 16 CTAs
      float part[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) part[k] = cluster.map_shared_rank(&sh.mine[0][0], p + k)[i / M * kLoraTokens + i % M];
#pragma unroll
      for (int k = 0; k < 4; ++k) v = __fadd_rn(v, part[k]);
    }
    sh.t[i / M][i % M] = __fmul_rn(v, scale);
  }
  cluster.sync();  // every CTA has read `mine`, and t is complete
  lora_up<T, M, VEC>(a, sh, s, ring);
}

// VEC: base and out rows allow 16-byte accesses, and rows is a multiple of 4.
template <class T, bool VEC>
__global__ void __launch_bounds__(kLoraThreads, 2) k_lora_add(LoraArgs a) {
  __shared__ LoraShared sh;
  extern __shared__ __align__(16) unsigned char ring[];
  cg::cluster_group cluster = cg::this_cluster();
  pdl_launch_dependents();
  pdl_wait();
  const int C = int(cluster.num_blocks()), clusters = int(gridDim.x) / C;
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
          for (uint64_t rest = same >> (v - w0) << (v - w0); rest && count < kLoraTokens; rest &= rest - 1)
            sh.token[count++] = w0 + __ffsll(int64_t(rest)) - 1;
          for (int i = count; i < kLoraTokens; ++i) sh.token[i] = sh.token[0];
        }
        sh.count = count;
        if (raw < -1 || raw >= a.adapters) atomicOr(a.status, kStatusBadIndex);
      }
    }
    __syncthreads();
    const int count = sh.count;
    if (count && adapter < 0) {
      if (a.out != a.base) {
        const int c = int(cluster.block_rank());
#pragma unroll 1
        for (int i = 0; i < count; ++i)
#pragma unroll 1
          for (int r = c * kLoraThreads + threadIdx.x; r < a.rows; r += C * kLoraThreads)
            a.out[sh.token[i] * a.ldo + r] = a.base[sh.token[i] * a.ldb + r];
      }
    } else if (count) {
      LoraSplit s;
      s.rank = a.ranks ? max(0, min(a.ranks[adapter], a.rank)) : a.rank;
      const int c = int(cluster.block_rank());
      const int per_n = (a.n / 8 + C - 1) / C * 8, per_r = ((a.rows + 3) / 4 + C - 1) / C * 4;
      const int j0 = min(a.n, c * per_n);
      s.slice = min(a.n, j0 + per_n) - j0;
      s.r0 = min(a.rows, c * per_r), s.r1 = min(a.rows, s.r0 + per_r);
      const int lquads = max(1, log2_from((s.rank + 3) / 4));
      s.quads = 1 << lquads, s.lparts = kLoraLogThreads - lquads, s.parts = 1 << s.lparts;
      s.lwidth = max(1, log2_from((s.rank + 7) / 8)), s.width = 1 << s.lwidth;
      s.down = s.rank ? (s.slice + s.parts * 8 - 1) >> (s.lparts + 3) : 0;
      s.up = (((s.r1 - s.r0) << s.lwidth) + 4 * kLoraThreads - 1) / (4 * kLoraThreads);
      s.quad = threadIdx.x >> s.lparts, s.part = threadIdx.x & (s.parts - 1);
      s.row = (threadIdx.x >> s.lwidth) * 4, s.piece = threadIdx.x & (s.width - 1);
      s.a0 = static_cast<const T*>(a.wa) + (int64_t(adapter) * a.rank + s.quad * 4) * a.n + j0 + s.part * 8;
      s.b0 = static_cast<const T*>(a.wb) + (int64_t(adapter) * a.rows + s.r0 + s.row) * a.rank + s.piece * 8;
      s.b_step = (4 * kLoraThreads >> s.lwidth) * a.rank;
      const float scale = a.scale ? a.scale[adapter] : 1.f;
      if (count == 1)
        lora_bucket<T, 1, VEC>(a, sh, s, ring, j0, scale, cluster);
      else if (count == 2)
        lora_bucket<T, 2, VEC>(a, sh, s, ring, j0, scale, cluster);
      else if (count <= 4)
        lora_bucket<T, 4, VEC>(a, sh, s, ring, j0, scale, cluster);
      else
        lora_bucket<T, 8, VEC>(a, sh, s, ring, j0, scale, cluster);
      asm volatile("cp.async.wait_group 0;" ::: "memory");
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
  // Clusters of 16 while all of them run at once (13 vectors of one adapter,
  // n 8120: 12.8 us against 15.5 with 8), of 8 beyond (64 vectors, rank 64: 28.7 us
  // against 47).  Their number is odd: the vectors that lead buckets are every
  // eighth in a prompt, and a cluster takes every so many-th vector.
  const int cluster = g.nvec * 16 <= 2 * num_sms() ? 16 : 8;
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
  const bool vec = aligned16(base) && aligned16(out) && ldb % 4 == 0 && ldo % 4 == 0 && rows % 4 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == Q1_BF16) return vec ? launch_lora<__nv_bfloat16, true>(g, s) : launch_lora<__nv_bfloat16, false>(g, s);
  return vec ? launch_lora<__half, true>(g, s) : launch_lora<__half, false>(g, s);
}
