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
  int vec_out;             // base and out rows allow 16-byte access
};

constexpr int kLoraTokens = 8;    // vectors of a bucket
constexpr int kLoraWindow = 64;   // vectors among which buckets form
constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraMaxRank = 128;
constexpr int kLoraRowsWarp = 4;  // rank rows a warp takes at a time

struct LoraShared {
  float part[kLoraWarps][kLoraRowsWarp][kLoraTokens];  // a warp's sums
  float mine[kLoraMaxRank][kLoraTokens];               // this CTA's slice of n
  float t[kLoraMaxRank][kLoraTokens];                  // all slices, scaled
  int token[kLoraTokens];
  int count;
};

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

// First product: mine[k][i] = sum over this CTA's slice of A[k] x_i, k < rank.
template <class T, int M>
__device__ __forceinline__ void lora_down(const LoraArgs& a, LoraShared& sh, const T* A, int rank, int j0, int j1) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float* x[M];
#pragma unroll
  for (int i = 0; i < M; ++i) x[i] = a.x + sh.token[i] * a.ldx;
  // Warps share out (rank rows in fours) x (parts of the slice).
  const int quads = (rank + kLoraRowsWarp - 1) / kLoraRowsWarp;
  if (quads == 0) return;  // an adapter of rank 0 (the whole cluster agrees)
  int parts = 1;
  while (parts * 2 * quads <= kLoraWarps) parts *= 2;
  const int step = kLoraWarps / parts;  // quads at a time
  for (int q0 = 0; q0 < quads; q0 += step) {
    const int quad = q0 + warp / parts, part = warp % parts;
    float acc[kLoraRowsWarp * M];
#pragma unroll
    for (int i = 0; i < kLoraRowsWarp * M; ++i) acc[i] = 0.f;
    if (quad < quads) {
      const T* row[kLoraRowsWarp];
#pragma unroll
      for (int r = 0; r < kLoraRowsWarp; ++r) row[r] = A + int64_t(min(quad * kLoraRowsWarp + r, rank - 1)) * a.n;
      for (int j = j0 + (part * 32 + lane) * 8; j < j1; j += parts * 256) {
        float w[kLoraRowsWarp][8];
#pragma unroll
        for (int r = 0; r < kLoraRowsWarp; ++r) Elem<T>::unpack(__ldg(reinterpret_cast<const uint4*>(row[r] + j)), w[r]);
#pragma unroll
        for (int i = 0; i < M; ++i) {
          const float4 lo = *reinterpret_cast<const float4*>(x[i] + j), hi = *reinterpret_cast<const float4*>(x[i] + j + 4);
          const float xv[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int r = 0; r < kLoraRowsWarp; ++r) acc[r * M + i] = __fmaf_rn(w[r][e], xv[e], acc[r * M + i]);
        }
      }
    }
    fold<kLoraRowsWarp * M>(acc, 32, lane);
    // A lane holds kLoraRowsWarp * M / 32 sums, or one that 32 / that many lanes share.
    constexpr int kSums = kLoraRowsWarp * M;
    static_assert(kSums <= 32, "one sum a lane at most");
    if (lane % (32 / kSums) == 0) (&sh.part[warp][0][0])[lane / (32 / kSums)] = acc[0];
    __syncthreads();
    for (int i = threadIdx.x; i < step * kSums; i += kLoraThreads) {
      const int qd = i / kSums, k = (q0 + qd) * kLoraRowsWarp + i % kSums / M;
      if (k < rank) {
        float s = 0.f;
        for (int p = 0; p < parts; ++p) s = __fadd_rn(s, (&sh.part[qd * parts + p][0][0])[i % kSums]);
        sh.mine[k][i % M] = s;
      }
    }
    __syncthreads();
  }
}

// Second product: rows [r0, r1) of B t for the bucket's vectors.  `width`
// neighbouring lanes take the 16-byte pieces of a row of B, four rows at a
// time.
template <class T, int M>
__device__ __forceinline__ void lora_up(const LoraArgs& a, const LoraShared& sh, const T* B, int rank, int r0, int r1) {
  const int pieces = (rank + 7) / 8;
  int width = 2;
  while (width < pieces) width *= 2;
  const int lane = threadIdx.x & 31, piece = lane & (width - 1);
  float t[8][M];
#pragma unroll
  for (int e = 0; e < 8; ++e)
#pragma unroll
    for (int i = 0; i < M; ++i) t[e][i] = piece * 8 + e < rank ? sh.t[piece * 8 + e][i] : 0.f;
  const int rows_pass = kLoraThreads / width * 4;
  for (int base = r0; base < r1; base += rows_pass) {  // whole warps stay together
    const int row = base + threadIdx.x / width * 4;
    float acc[M][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint4 raw = make_uint4(0u, 0u, 0u, 0u);
      if (piece < pieces && row + k < r1) raw = __ldg(reinterpret_cast<const uint4*>(B + int64_t(row + k) * a.rank) + piece);
      float w[8];
      Elem<T>::unpack(raw, w);
      if (piece * 8 + 8 > rank) {  // values past the adapter's rank may be anything
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = piece * 8 + e < rank ? w[e] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < M; ++i) {
        acc[i][k] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][k] = __fmaf_rn(w[e], t[e][i], acc[i][k]);
      }
    }
    // Fold over the lanes of a row; each lane ends with the vectors it writes.
    float f[4][M];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int i = 0; i < M; ++i) f[k][i] = acc[i][k];
      fold<M>(f[k], width, lane);
    }
    const int shared_by = width > M ? width / M : 1, keep = width > M ? 1 : M / width;
    if (piece % shared_by) continue;
    const int first = piece / shared_by * keep;
#pragma unroll
    for (int i = 0; i < M; ++i) {
      if (i >= keep || first + i >= sh.count) continue;
      const int64_t v = sh.token[first + i];
      const float* in = a.base + v * a.ldb + row;
      float* out = a.out + v * a.ldo + row;
      if (a.vec_out && row + 4 <= r1) {
        float4 b = *reinterpret_cast<const float4*>(in);
        b.x = __fadd_rn(b.x, f[0][i]), b.y = __fadd_rn(b.y, f[1][i]), b.z = __fadd_rn(b.z, f[2][i]), b.w = __fadd_rn(b.w, f[3][i]);
        *reinterpret_cast<float4*>(out) = b;
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (row + k < r1) out[k] = __fadd_rn(in[k], f[k][i]);
      }
    }
  }
}

template <class T, int M>
__device__ __forceinline__ void lora_bucket(const LoraArgs& a, LoraShared& sh, int adapter, cg::cluster_group& cluster) {
  const int c = int(cluster.block_rank()), C = int(cluster.num_blocks());
  const int rank = a.ranks ? max(0, min(a.ranks[adapter], a.rank)) : a.rank;
  const int per_n = (a.n / 8 + C - 1) / C * 8;
  lora_down<T, M>(a, sh, static_cast<const T*>(a.wa) + int64_t(adapter) * a.rank * a.n, rank, min(a.n, c * per_n),
                  min(a.n, (c + 1) * per_n));
  cluster.sync();
  const float scale = a.scale ? a.scale[adapter] : 1.f;
  for (int i = threadIdx.x; i < rank * M; i += kLoraThreads) {
    float s = 0.f;
    for (int p = 0; p < C; ++p) s = __fadd_rn(s, cluster.map_shared_rank(&sh.mine[0][0], p)[i / M * kLoraTokens + i % M]);
    sh.t[i / M][i % M] = __fmul_rn(s, scale);
  }
  cluster.sync();  // every CTA has read `mine`, and t is complete
  const int per_r = ((a.rows + 3) / 4 + C - 1) / C * 4;
  lora_up<T, M>(a, sh, static_cast<const T*>(a.wb) + int64_t(adapter) * a.rows * a.rank, rank, min(a.rows, c * per_r),
                min(a.rows, (c + 1) * per_r));
}

template <class T>
__global__ void __launch_bounds__(kLoraThreads) k_lora_add(LoraArgs a) {
  __shared__ LoraShared sh;
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
        for (int i = 0; i < count; ++i)
          for (int r = c * kLoraThreads + threadIdx.x; r < a.rows; r += C * kLoraThreads)
            a.out[sh.token[i] * a.ldo + r] = a.base[sh.token[i] * a.ldb + r];
      }
    } else if (count == 1) {
      lora_bucket<T, 1>(a, sh, adapter, cluster);
    } else if (count && count <= 4) {
      lora_bucket<T, 4>(a, sh, adapter, cluster);
    } else if (count) {
      lora_bucket<T, 8>(a, sh, adapter, cluster);
    }
    __syncthreads();  // sh is free again
  }
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
                int(adapters), 0};
  if (int e = ops_status_ptr(&g.status)) return e;
  g.vec_out = aligned16(base) && aligned16(out) && ldb % 4 == 0 && ldo % 4 == 0;
  const int cluster = 8;
  const int64_t most = int64_t(num_sms()) * 4 / cluster;
  const dim3 grid(unsigned((nvec < most ? nvec : most) * cluster));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == Q1_BF16) return launch_op(k_lora_add<__nv_bfloat16>, grid, kLoraThreads, 0, cluster, s, who, g);
  return launch_op(k_lora_add<__half>, grid, kLoraThreads, 0, cluster, s, who, g);
}
