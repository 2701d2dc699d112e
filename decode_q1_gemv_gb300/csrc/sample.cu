// sample.cu -- q1_sample: the next token of each row of logits, drawn with a
// given random number from the tokens that top-k, top-p and min-p leave.
//
// w_i = 2^((x_i - max) c), c = log2(e) / temperature.  What stays is a prefix of
// the tokens in falling order (by count: top-k; by sum: top-p) and above a weight
// (min-p), so no row is sorted: a threshold is enough, and the token is found by sums
// in the vocabulary's order.
//
// The result is a whole number that changes where a sum crosses a border, so
// weights are fixed-point numbers (44 bits behind the point, 2^-30 of themselves) and
// sums are 64-bit integers: exact, in any order, the same in every launch.  Sums of
// f32 weights in f32 would give another token in some percent of rows.
//   x - max in two floats, times c in two floats: the exponent's whole part n, a
//   512th part k (a table of 2^(k/512)) and a rest r below 2^-10, whose 2^r - 1 is
//   r (ln 2 + r ln^2(2) / 2) (what follows is below 2^-34).
//
// A row belongs to a cluster of up to 16 CTAs (as many as all rows leave room
// for), each with a slice of the vocabulary, each warp with a part of it:
//   1  the maximum, and whether all values are numbers;
//   2  (small top-k) a value that top-k tokens at least reach: of the threads' own
//      maxima the one with k / CTAs - 1 others above it in each CTA, the least of these;
//      what reaches it is listed: 4a;
//   3  (top-p, large top-k, or a list that is too long) a histogram over the exponent, 1024
//      bins, of counts and sums, joined through distributed shared memory: the
//      bin where the threshold lies.  The tokens down to that bin are listed if they are few: 4a;
//      else those of the bin alone are, for the threshold; else (many equal ones) it is found by
//      histograms of their bits, ten at a time: 4b;
//   4a one CTA sorts the list, cuts, and draws;
//   4b (and without top-k and top-p) sums by warp, whose one holds the token, and the
//      token in it.
// Bytes bound the largest calls, a few barriers of the cluster the smallest ones.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include <cooperative_groups.h>

#include "ops.cuh"

namespace q1 {

namespace cg = cooperative_groups;

constexpr int kSampleThreads = 512, kSampleWarps = kSampleThreads / 32;
constexpr int kBins = 1024;
constexpr int kListed = 1024;        // tokens that one CTA sorts
constexpr int kFewTopK = 256;        // top-k by the threads' maxima
constexpr int kSteps = 512;          // parts of an exponent
constexpr int kOne = 44;             // bits behind the point
constexpr float kLeast = -44.f;      // exponents from here down are weights of zero

struct Powers {
  uint32_t bits[kSteps];  // 2^(k/512) 2^31
};
constexpr Powers make_powers() {
  Powers t = {};
  // 2^(1/512) to 2^-53: its powers are off by some 2^-44
  const double root = 1.0013547198921082058;
  double up = 1.0;
  for (int k = 0; k < kSteps; ++k) t.bits[k] = uint32_t(up * 2147483648.0 + 0.5), up *= root;
  return t;
}
__device__ const Powers g_powers = make_powers();

struct SampleArgs {
  const void* logits;
  int64_t ld;
  const float* uniform;
  q1_sampling set;
  int32_t* out;
  int vocab, ctas;  // CTAs of a row
  int cached;       // 16-byte groups of a slice that fit shared memory: all or none
};

struct Weigh {
  float max, ch, cl;  // the row's maximum, log2(e) / temperature in two floats
  const uint32_t* powers;
};

// The exponent of x's weight, to f32: it only falls where x falls.
__device__ __forceinline__ float exponent_of(const Weigh& w, float x) { return __fmul_rn(__fsub_rn(x, w.max), w.ch); }

// The weight of x, 2^44 for the maximum.
__device__ __forceinline__ uint64_t weight_of(const Weigh& w, float x) {
  const float d = __fsub_rn(x, w.max), y = __fmul_rn(d, w.ch);
  if (!(y > kLeast)) return 0;  // -inf - max among them, and its product with a factor of zero
  const float back = __fsub_rn(d, x);
  const float lost = __fsub_rn(__fsub_rn(x, __fsub_rn(d, back)), __fadd_rn(w.max, back));  // x - max - d
  const float rest = __fmaf_rn(lost, w.ch, __fmaf_rn(d, w.cl, __fmaf_rn(d, w.ch, -y)));
  // y = n + k / 512 + r: rounded by adding 1.5 2^23 (|y| 512 < 2^22)
  const float z = __fmaf_rn(y, float(kSteps), kMagic);
  const int whole = int(__float_as_uint(z) - kMagicBits);
  const float r = __fadd_rn(__fmaf_rn(__fsub_rn(z, kMagic), -1.0f / kSteps, y), rest);
  const float p = __fmul_rn(r, __fmaf_rn(r, 0.24022651f, 0.69314718f));  // 2^r - 1
  const uint32_t t = w.powers[whole & (kSteps - 1)];
  // t p < 2^22, rounded by the same addition; t as a float (truncated) by its bits
  const float tf = __uint_as_float((t >> 8) + (157u << 23));
  const uint32_t bits = t + (__float_as_uint(__fmaf_rn(tf, p, kMagic)) - kMagicBits);
  return (uint64_t(bits) << 32) >> (32 + 31 - kOne - (whole >> 9));
}
static_assert(kSteps == 512, "the shift above");

__device__ __forceinline__ uint32_t order_of(float x) {  // rises with x; -0 as 0
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.f));
  return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_order(uint32_t o) { return __uint_as_float(o >> 31 ? o ^ 0x80000000u : ~o); }

__device__ __forceinline__ int bin_of(const Weigh& w, float x) {  // of a weight above zero
  return min(int(__fmul_rn(exponent_of(w, x), kBins / kLeast)), kBins - 1);
}

// f * v, f in [0, 1), rounded down or up.
__device__ __forceinline__ uint64_t part_of(float f, uint64_t v, bool up) {
  const uint32_t b = __float_as_uint(f);
  if (b == 0) return 0;
  const int e = int(b >> 23);
  const uint64_t m = e ? (b & 0x7fffffu) | 0x800000u : b;
  const int shift = 150 - (e ? e : 1);  // f = m 2^-shift, 24 at least
  const uint64_t hi = __umul64hi(m, v), lo = m * v;
  uint64_t r;
  bool rest;
  if (shift < 64) {
    r = (hi << (64 - shift)) | (lo >> shift), rest = (lo << (64 - shift)) != 0;
  } else {
    const int s = min(shift - 64, 63);
    r = hi >> s, rest = lo != 0 || (hi & ((uint64_t(1) << s) - 1)) != 0;
  }
  return r + (up && rest);
}

// What a histogram's search gives: the bin, what lies before it and in it.
struct Found {
  int bin;
  uint32_t above, in;
  uint64_t mass_above, mass_in;
};

struct SampleShared {
  uint32_t powers[kSteps];
  uint32_t count[kBins], low[kBins], high[kBins];        // of this CTA
  uint32_t all_count[kBins];                             // of the row
  union {
    uint64_t all_mass[kBins];
    uint64_t sorted[kListed];  // (once the bins have been searched)
  };
  uint64_t list[kListed];
  uint64_t warp_mass[kSampleWarps];
  uint32_t warp_count[kSampleWarps];
  Found found;
  float own_max;
  float own_reached;       // what at least its part of top-k tokens reach
  int own_bad, listed, token;
  uint64_t own_mass;
  uint32_t own_ties;
  uint32_t cut;            // of the leader: what a list's threshold is
  uint64_t cut_ties;
};

template <class T>
__device__ __forceinline__ uint32_t masked_bits();  // -inf, in each 16 bits of a word or in all of it
template <>
__device__ __forceinline__ uint32_t masked_bits<float>() { return 0xff800000u; }
template <>
__device__ __forceinline__ uint32_t masked_bits<__nv_bfloat16>() { return 0xff80ff80u; }
template <>
__device__ __forceinline__ uint32_t masked_bits<__half>() { return 0xfc00fc00u; }

template <class T>
struct Row {
  static constexpr int G = Elem<T>::kGroup;
  const T* row;
  int vocab, skew;   // skew: elements between a 16-byte boundary and the row's start
  int first, last;   // groups of this CTA's slice
  uint4* cache;      // null: read again
  // Group i (of 16 aligned bytes): elements i G - skew on; -inf where there are none.
  __device__ __forceinline__ uint4 load(int i) const {
    const int e = i * G - skew;
    if (e >= 0 && e + G <= vocab) return *reinterpret_cast<const uint4*>(row + e);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = masked_bits<T>();
#pragma unroll
    for (int k = 0; k < G; ++k) {
      if (e + k < 0 || e + k >= vocab) continue;
      if constexpr (G == 4)
        w[k] = reinterpret_cast<const uint32_t*>(row)[e + k];
      else
        w[k / 2] = (w[k / 2] & (k & 1 ? 0xffffu : 0xffff0000u)) | uint32_t(reinterpret_cast<const uint16_t*>(row)[e + k]) << (k & 1 ? 16 : 0);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // f(group's values, its first element) over groups [a, b) of a warp, lane by lane.
  template <bool kFirst, class F>
  __device__ __forceinline__ void each(int a, int b, F&& f) const {
    const int lane = threadIdx.x & 31;
    for (int i0 = a + lane; i0 < b; i0 += 128) {
      uint4 r[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + 32 * k;
        r[k] = make_uint4(masked_bits<T>(), masked_bits<T>(), masked_bits<T>(), masked_bits<T>());
        if (i < b) r[k] = kFirst || !cache ? load(i) : cache[i - first];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + 32 * k;
        if (kFirst && cache && i < b) cache[i - first] = r[k];
        float v[G];
        Elem<T>::unpack(r[k], v);
        f(v, i * G - skew);
      }
    }
  }
};

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ uint64_t warp_prefix(uint64_t v) {  // with its own
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint64_t t = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += t;
  }
  return v;
}

// The first bin up to which the counts reach `need` (by mass: the sums), after
// `above` and `mass_above` before the histogram; its last bin with anything in it
// where none does.  Every thread of the CTA calls and gets it.
__device__ __forceinline__ Found search(SampleShared& sh, bool by_mass, uint64_t need, uint32_t above, uint64_t mass_above) {
  constexpr int kEach = kBins / kSampleThreads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t n[kEach], ns = 0;
  uint64_t m[kEach], ms = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    n[i] = sh.all_count[threadIdx.x * kEach + i], m[i] = sh.all_mass[threadIdx.x * kEach + i];
    ns += n[i], ms += m[i];
  }
  const uint32_t nincl = uint32_t(warp_prefix(ns));
  const uint64_t mincl = warp_prefix(ms);
  if (lane == 31) sh.warp_count[warp] = nincl, sh.warp_mass[warp] = mincl;
  if (threadIdx.x == 0) sh.found.bin = -1;
  __syncthreads();
  uint32_t nb = above + nincl - ns;
  uint64_t mb = mass_above + mincl - ms;
  for (int w = 0; w < warp; ++w) nb += sh.warp_count[w], mb += sh.warp_mass[w];
  uint32_t last = 0;  // counts before and with the bins, for the one that is last of all
  uint32_t total = above;
  for (int w = 0; w < kSampleWarps; ++w) total += sh.warp_count[w];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint64_t before = by_mass ? mb : nb, after = by_mass ? mb + m[i] : uint64_t(nb) + n[i];
    last = nb + n[i];
    if (n[i] && ((before < need && after >= need) || (after < need && last == total)))
      sh.found = {int(threadIdx.x) * kEach + i, nb, n[i], mb, m[i]};
    nb += n[i], mb += m[i];
  }
  __syncthreads();
  return sh.found;
}

// Sorts the n (up to kListed) different entries of sh.sorted, rising; ~0 follows them up to a power of two.
// Every thread of the CTA calls.
constexpr int kByRank = 256;
__device__ __forceinline__ void sort(SampleShared& sh, int n) {
  uint64_t* v = sh.sorted;
  __syncthreads();
  if (n <= kByRank) {  // each entry goes where it belongs: two threads count the entries below it (two barriers, not 28 to 36)
    const int i = threadIdx.x >> 1, half = threadIdx.x & 1, mid = (n + 1) / 2;
    const uint64_t mine = i < n ? v[i] : 0;
    int below = 0;
    if (i < n)
#pragma unroll 4
      for (int k = half ? mid : 0; k < (half ? n : mid); ++k) below += v[k] < mine;
    below += __shfl_xor_sync(0xffffffffu, below, 1);
    __syncthreads();
    if (i < n && half == 0) v[below] = mine;
    __syncthreads();
    return;
  }
  int padded = 2;
  while (padded < n) padded <<= 1;
  for (int i = n + threadIdx.x; i < padded; i += kSampleThreads) v[i] = ~uint64_t(0);
  for (int size = 2; size <= padded; size <<= 1)
    for (int step = size >> 1; step > 0; step >>= 1) {
      __syncthreads();
      for (int i = threadIdx.x; i < padded / 2; i += kSampleThreads) {
        const int lo = 2 * i - (i & (step - 1)), hi = lo + step;
        const uint64_t a = v[lo], b = v[hi];
        if ((a > b) == ((lo & size) == 0)) v[lo] = b, v[hi] = a;
      }
    }
  __syncthreads();
}

// The sums of v over the CTA's threads up to each (its own among them), and of all.
__device__ __forceinline__ uint64_t block_prefix(SampleShared& sh, uint64_t v, uint64_t& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t p = warp_prefix(v);
  __syncthreads();
  if (lane == 31) sh.warp_mass[warp] = p;
  __syncthreads();
  const uint64_t warps = warp_prefix(lane < kSampleWarps ? sh.warp_mass[lane] : 0);
  all = __shfl_sync(0xffffffffu, warps, 31);
  return p + (warp ? __shfl_sync(0xffffffffu, warps, warp - 1) : 0);
}

template <class T>
__global__ void __launch_bounds__(kSampleThreads, 2) k_sample(const __grid_constant__ SampleArgs a) {
  constexpr int G = Elem<T>::kGroup;
  extern __shared__ __align__(16) unsigned char dynamic[];
  __shared__ SampleShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = int(blockIdx.x) / a.ctas, rank = int(blockIdx.x) - row * a.ctas;
  for (int i = threadIdx.x; i < kSteps; i += kSampleThreads) sh.powers[i] = g_powers.bits[i];
  pdl_launch_dependents();
  pdl_wait();
  const float temperature = a.set.temperature ? a.set.temperature[row] : a.set.temperature_all;
  const int top_k = a.set.top_k ? a.set.top_k[row] : a.set.top_k_all;
  const float top_p = a.set.top_p ? a.set.top_p[row] : a.set.top_p_all;
  const float min_p = a.set.min_p ? a.set.min_p[row] : a.set.min_p_all;
  const float uniform = a.uniform[row];

  Row<T> x;
  x.row = static_cast<const T*>(a.logits) + row * a.ld, x.vocab = a.vocab;
  x.skew = int(reinterpret_cast<uintptr_t>(x.row) % 16 / sizeof(T));
  const int groups = (a.vocab + x.skew + G - 1) / G, per = (groups + a.ctas - 1) / a.ctas;
  x.first = min(groups, rank * per), x.last = min(groups, x.first + per);
  x.cache = a.cached ? reinterpret_cast<uint4*>(dynamic) : nullptr;
  const int mine = x.last - x.first, from = x.first + int(int64_t(mine) * warp / kSampleWarps),
            to = x.first + int(int64_t(mine) * (warp + 1) / kSampleWarps);

  // 1. The maximum.
  const bool by_count = top_k > 0 && top_k < a.vocab, by_mass = top_p < 1.f;
  float top = -INFINITY;
  bool bad = false;
  x.template each<true>(from, to, [&](const float (&v)[G], int) {
#pragma unroll
    for (int i = 0; i < G; ++i) top = fmaxf(top, v[i]), bad |= !(v[i] <= FLT_MAX);
  });
  const float mine_top = top;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (threadIdx.x == 0) sh.listed = 0, sh.token = a.vocab;
  for (int i = threadIdx.x; i < kBins; i += kSampleThreads) sh.count[i] = 0, sh.low[i] = 0, sh.high[i] = 0;
  if (lane == 0) sh.warp_count[warp] = __float_as_uint(top);
  bad = __syncthreads_or(bad);
  // 2. A value that so many threads' maxima reach that all CTAs together have top-k of them, to a 2^-10th of their range.
  const bool few = by_count && top_k <= kFewTopK && temperature > 0.f;
  if (few) {
    float lo = mine_top == -INFINITY ? INFINITY : mine_top;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    if (lane == 0) sh.warp_mass[warp] = __float_as_uint(lo);
    const int want = (top_k + a.ctas - 1) / a.ctas;
    const bool enough = __syncthreads_count(mine_top > -INFINITY) >= want;
    lo = __uint_as_float(uint32_t(sh.warp_mass[lane % kSampleWarps]));
    float hi = __uint_as_float(sh.warp_count[lane % kSampleWarps]);
#pragma unroll
    for (int off = kSampleWarps / 2; off > 0; off >>= 1)
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off)), hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    if (enough)
      for (int i = 0; i < 10; ++i) {
        const float mid = 0.5f * lo + 0.5f * hi;
        (__syncthreads_count(mine_top >= mid) >= want ? lo : hi) = mid;
      }
    if (threadIdx.x == 0) sh.own_reached = enough ? lo : -FLT_MAX;
  }
  if (warp == 0) {
    float m = lane < kSampleWarps ? __uint_as_float(sh.warp_count[lane]) : -INFINITY;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (lane == 0) sh.own_max = m, sh.own_bad = bad;
  }
  cluster.sync();
  float reached = INFINITY;
  {
    const SampleShared* his = cluster.map_shared_rank(&sh, lane < a.ctas ? lane : 0);
    top = his->own_max, reached = his->own_reached, bad = his->own_bad != 0;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      reached = fminf(reached, __shfl_xor_sync(0xffffffffu, reached, off));
    }
    bad = __any_sync(0xffffffffu, bad);
  }
  bad |= top == -INFINITY || isnan(temperature) || isnan(top_p) || isnan(min_p) || isnan(uniform);
  if (bad) {
    if (rank == 0 && threadIdx.x == 0) a.out[row] = -1;
    cluster.sync();  // the maxima have been read
    return;
  }
  if (!(temperature > 0.f)) {
    int at = a.vocab;
    x.template each<false>(from, to, [&](const float (&v)[G], int e) {
#pragma unroll
      for (int i = G - 1; i >= 0; --i)
        if (v[i] == top) at = min(at, e + i);
    });
    atomicMin(&sh.token, at);
    cluster.sync();
    if (rank == 0 && threadIdx.x == 0) {
      for (int r = 0; r < a.ctas; ++r) at = min(at, cluster.map_shared_rank(&sh, r)->token);
      a.out[row] = at;
    }
    cluster.sync();
    return;
  }
  Weigh w;
  // log2(e) / temperature: the quotient, and what is left divided again.  (An infinite temperature makes
  // all weights one.)
  constexpr float kLog = 1.4426950216293335f, kLogRest = 1.9259629e-8f;
  const float t = fmaxf(temperature, 1e-37f);
  w.max = top, w.ch = __fdiv_rn(kLog, t), w.powers = sh.powers;
  w.cl = w.ch > 0.f ? __fdiv_rn(__fadd_rn(__fmaf_rn(-w.ch, t, kLog), kLogRest), t) : 0.f;
  const float u = fminf(fmaxf(uniform, 0.f), 0.99999994f);
  const uint64_t least = min_p >= 1.f ? uint64_t(1) << kOne : min_p > 0.f ? part_of(min_p, uint64_t(1) << kOne, true) : 1;
  // 4a. The first CTA collects all lists, up to kListed tokens in all, and sorts them by falling values,
  // equal ones by their place; returns how many (0 where there are more: all CTAs get it, one sorts).
  const auto collect = [&]() {
    cluster.sync();
    const uint32_t upto = uint32_t(warp_prefix(lane < a.ctas ? cluster.map_shared_rank(&sh, lane)->listed : 0));
    const int n = int(__shfl_sync(0xffffffffu, upto, 31));
    if (n > kListed || rank != 0) return n > kListed ? 0 : n;
    for (int i = threadIdx.x; i - lane < n; i += kSampleThreads) {
      int r = 0, first = 0;  // the CTA whose list holds entry i, and where that list begins
      for (int k = 0; k < a.ctas; ++k) {
        const int end = int(__shfl_sync(0xffffffffu, upto, k));
        if (i >= end) r = k + 1, first = end;
      }
      if (i < n) sh.sorted[i] = cluster.map_shared_rank(&sh, r)->list[i - first];
    }
    sort(sh, n);
    return n;
  };
  const auto list = [&](float v, int place) {
    const int i = atomicAdd(&sh.listed, 1);
    if (i < kListed) sh.list[i] = uint64_t(~order_of(v)) << 32 | uint32_t(place);
  };
  const auto entry_weight = [&](uint32_t upside_down) { return weight_of(w, of_order(~upside_down)); };
  constexpr int kEach = kListed / kSampleThreads;
  // The token, where all that may stay is among the n tokens sorted: the first `count` of them, then by mass
  // (need 0: top_p of their own).
  const auto finish = [&](int n, int count, uint64_t need) {
    uint64_t weight[kEach], sum = 0, all;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int i = threadIdx.x * kEach + k;
      weight[k] = i < min(n, count) ? entry_weight(uint32_t(sh.sorted[i] >> 32)) : 0;
      sum += weight[k];
    }
    uint64_t before = block_prefix(sh, sum, all) - sum;
    if (by_mass && need == 0) need = max(part_of(fmaxf(top_p, 0.f), all, true), uint64_t(1));
    uint64_t entry[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int i = threadIdx.x * kEach + k;
      const bool stays = weight[k] >= least && (!by_mass || before < need);
      before += weight[k];
      if (i < n) entry[k] = sh.sorted[i] << 32 | sh.sorted[i] >> 32 | (stays ? 0 : uint64_t(1) << 63);  // (the others behind)
    }
    // In the vocabulary's order: the sums of the weights there.
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      if (threadIdx.x * kEach + k < n) sh.sorted[threadIdx.x * kEach + k] = entry[k];
    sort(sh, n);
    sum = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int i = threadIdx.x * kEach + k;
      entry[k] = i < n ? sh.sorted[i] : 0;
      weight[k] = i < n && !(entry[k] >> 63) ? entry_weight(uint32_t(entry[k])) : 0;
      sum += weight[k];
    }
    before = block_prefix(sh, sum, all) - sum;
    const uint64_t drawn = part_of(u, all, false);
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      if (drawn >= before && drawn < before + weight[k]) a.out[row] = int32_t(entry[k] >> 32);
      before += weight[k];
    }
  };
  if (few) {
    x.template each<false>(from, to, [&](const float (&v)[G], int e) {
#pragma unroll
      for (int i = 0; i < G; ++i)
        if (v[i] >= reached) list(v[i], e + i);
    });
    if (const int n = collect()) {
      if (rank == 0) finish(n, top_k, 0);
      cluster.sync();  // the lists have been read
      return;
    }
    cluster.sync();
    if (threadIdx.x == 0) sh.listed = 0;
  }

  // The histogram of this CTA (`which`: its bin of a value, -1 for none) becomes the row's, in every CTA.
  const auto histogram = [&](auto&& which) {
    x.template each<false>(from, to, [&](const float (&v)[G], int) {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const uint64_t m = weight_of(w, v[i]);
        const int b = m ? which(v[i]) : -1;
        if (b < 0) continue;
        atomicAdd(&sh.count[b], 1u);
        const uint32_t old = atomicAdd(&sh.low[b], uint32_t(m));
        atomicAdd(&sh.high[b], uint32_t(m >> 32) + (old + uint32_t(m) < old));
      }
    });
    cluster.sync();
    if (a.ctas == 1) {
      for (int b = threadIdx.x; b < kBins; b += kSampleThreads)
        sh.all_count[b] = sh.count[b], sh.all_mass[b] = uint64_t(sh.high[b]) << 32 | sh.low[b];
    } else {
      // A CTA sums a share of the bins: ctas / 2 threads a bin take two CTAs each, join, and give the sum to those two.
      const int share = kBins / a.ctas, part = int(threadIdx.x) / share, b = rank * share + int(threadIdx.x) % share;
      SampleShared *one = cluster.map_shared_rank(&sh, 2 * part), *other = cluster.map_shared_rank(&sh, 2 * part + 1);
      uint32_t n = one->count[b] + other->count[b];
      uint64_t m = (uint64_t(one->high[b]) << 32 | one->low[b]) + (uint64_t(other->high[b]) << 32 | other->low[b]);
      sh.list[threadIdx.x] = m, sh.list[kSampleThreads + threadIdx.x] = n;
      __syncthreads();
      n = 0, m = 0;
      for (int i = int(threadIdx.x) % share; i < kSampleThreads; i += share) m += sh.list[i], n += uint32_t(sh.list[kSampleThreads + i]);
      one->all_count[b] = n, one->all_mass[b] = m;
      other->all_count[b] = n, other->all_mass[b] = m;
    }
    cluster.sync();
    for (int i = threadIdx.x; i < kBins; i += kSampleThreads) sh.count[i] = 0, sh.low[i] = 0, sh.high[i] = 0;
  };

  uint32_t limit = 0;            // tokens above it (in order_of) stay,
  uint64_t ties = 0;             // and as many of those at it, the first ones
  uint64_t tie_weight = 0, kept = 0;  // kept: the sum of what top-k leaves
  if (by_count || by_mass) {
    const auto whole_row = [&](float v) { return bin_of(w, v); };
    histogram(whole_row);
    uint64_t need = by_count ? uint64_t(top_k) : 0;
    if (!by_count) {
      uint64_t all = 0;
      (void)block_prefix(sh, sh.all_mass[threadIdx.x] + sh.all_mass[threadIdx.x + kSampleThreads], all);
      need = max(part_of(fmaxf(top_p, 0.f), all, true), uint64_t(1));
    }
    bool mass = !by_count;  // what is searched for
    Found f = search(sh, mass, need, 0, 0);
    for (bool first = true;; first = false) {
      const bool all_few = f.above + f.in <= kListed;
      if (f.in <= kListed) {
        // 4a. All tokens down to this bin, or those of this bin alone.  (From the second search on top-k was dealt with.)
        const int bin = f.bin;
        x.template each<false>(from, to, [&](const float (&v)[G], int e) {
#pragma unroll
          for (int i = 0; i < G; ++i) {
            if (!(exponent_of(w, v[i]) > kLeast)) continue;
            const int b = bin_of(w, v[i]);
            if ((b == bin || (all_few && b < bin)) && weight_of(w, v[i])) list(v[i], e + i);
          }
        });
        const int n = collect();
        if (all_few) {
          if (rank == 0) finish(n, by_count && first ? top_k : n, first && by_count ? 0 : need);
          cluster.sync();  // the lists have been read
          return;
        }
        // The threshold is the first entry at which the count or the sum is reached: it, and those of its value before it.
        if (rank == 0) {
          uint64_t weight[kEach], sum = 0, all;
#pragma unroll
          for (int k = 0; k < kEach; ++k) {
            const int i = threadIdx.x * kEach + k;
            weight[k] = i < n ? entry_weight(uint32_t(sh.sorted[i] >> 32)) : 0;
            sum += weight[k];
          }
          uint64_t before = f.mass_above + block_prefix(sh, sum, all) - sum;
#pragma unroll
          for (int k = 0; k < kEach; ++k) {
            const int i = threadIdx.x * kEach + k;
            const bool is = mass ? before < need && before + weight[k] >= need : uint64_t(f.above) + i + 1 == need;
            if (i < n && (is || (i == n - 1 && (mass ? before + weight[k] : uint64_t(f.above) + n) < need))) {
              const uint32_t value = uint32_t(sh.sorted[i] >> 32);
              int same = 1;
              while (i - same >= 0 && uint32_t(sh.sorted[i - same] >> 32) == value) ++same;
              sh.cut = ~value, sh.cut_ties = same;
              sh.own_mass = before + weight[k];  // of all that stays
            }
            before += weight[k];
          }
        }
        cluster.sync();
        const SampleShared* his = cluster.map_shared_rank(&sh, 0);
        limit = his->cut, ties = his->cut_ties, tie_weight = weight_of(w, of_order(limit));
        kept = his->own_mass;
        cluster.sync();
        if (threadIdx.x == 0) sh.listed = 0;
        __syncthreads();
      } else {
        // The threshold within the bin, ten bits of its values at a time (of 16-bit types the first 20 differ).
        const int bin = f.bin;
        uint32_t prefix = 0, known = 0;  // the bits found
        Found at = f;
#pragma unroll 1
        for (int shift = 22;; shift = max(0, shift - 10)) {
          const uint32_t width = known ? min(10, __ffs(int(known)) - 1 - shift) : 10;
          const uint32_t most = (1u << width) - 1;
          histogram([&](float v) {
            const uint32_t o = order_of(v);
            return bin_of(w, v) == bin && (o & known) == prefix ? int(most - ((o >> shift) & most)) : -1;
          });
          at = search(sh, mass, need, at.above, at.mass_above);
          prefix |= (most - uint32_t(at.bin)) << shift, known |= most << shift;
          if (shift == 0 || (G == 8 && shift <= 12)) break;
        }
        if (G == 8) prefix |= prefix >> 31 ? 0 : 0xfffu;  // the bits that 16-bit types do not have
        limit = prefix, tie_weight = at.mass_in / at.in;
        ties = mass ? (need - at.mass_above + tie_weight - 1) / tie_weight : need - at.above;
        ties = min(ties, uint64_t(at.in));
        kept = at.mass_above + ties * tie_weight;
      }
      if (mass || !by_mass) break;
      // top-p of what top-k left: the same histogram, made once more.
      mass = true;
      need = max(part_of(top_p > 0.f ? top_p : 0.f, kept, true), uint64_t(1));
      histogram(whole_row);
      f = search(sh, true, need, 0, 0);
    }
    if (tie_weight < least) ties = 0;
  }

  // 4. Sums of what stays, by warp: weights above the limit, and values at it.
  const float border = limit ? of_order(limit) : -INFINITY;
  const auto sums_of = [&](int a0, int b0, uint64_t& sum, uint32_t& at_limit) {
    sum = 0, at_limit = 0;
    x.template each<false>(a0, b0, [&](const float (&v)[G], int) {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        at_limit += v[i] == border;
        if (v[i] > border) {
          const uint64_t m = weight_of(w, v[i]);
          sum += m >= least ? m : 0;
        }
      }
    });
    sum = warp_sum(sum);
    at_limit = __reduce_add_sync(0xffffffffu, at_limit);
  };
  // Of `n` values at the limit after `before` others: the sum of those that stay.
  const auto tied = [&](uint64_t before, uint64_t n) { return (before >= ties ? 0 : min(n, ties - before)) * tie_weight; };
  uint64_t sum;
  uint32_t at_limit;
  sums_of(from, to, sum, at_limit);
  __syncthreads();
  if (lane == 0) sh.warp_mass[warp] = sum, sh.warp_count[warp] = at_limit;
  __syncthreads();
  if (threadIdx.x == 0) {
    uint64_t m = 0;
    uint32_t n = 0;
    for (int i = 0; i < kSampleWarps; ++i) m += sh.warp_mass[i], n += sh.warp_count[i];
    sh.own_mass = m, sh.own_ties = n;
  }
  cluster.sync();
  uint64_t before, before_ties, all;  // what stays in the row's CTAs before this one, the ties there, and what stays in all
  {
    const SampleShared* his = cluster.map_shared_rank(&sh, lane < a.ctas ? lane : 0);
    const uint64_t m = lane < a.ctas ? his->own_mass : 0, n = lane < a.ctas ? his->own_ties : 0;
    const uint64_t first = warp_prefix(n) - n, with = m + tied(first, n), upto = warp_prefix(with);
    before_ties = __shfl_sync(0xffffffffu, first, rank);
    before = __shfl_sync(0xffffffffu, upto - with, rank);
    all = __shfl_sync(0xffffffffu, upto, 31);
  }
  const uint64_t drawn = part_of(u, all, false);
  const uint64_t own = sh.own_mass + tied(before_ties, sh.own_ties);
  if (drawn >= before && drawn < before + own) {
    // The warp's part that holds the token, then its sixteenth, then the token.
    int a0 = x.first, b0 = x.last;
    for (int round = 0; round < 2; ++round) {
      if (round) {
        const int n = b0 - a0;
        uint64_t m;
        uint32_t t;
        sums_of(a0 + n * warp / kSampleWarps, a0 + n * (warp + 1) / kSampleWarps, m, t);
        __syncthreads();
        if (lane == 0) sh.warp_mass[warp] = m, sh.warp_count[warp] = t;
        __syncthreads();
      }
      int i = 0;
      for (; i < kSampleWarps - 1; ++i) {
        const uint64_t with = sh.warp_mass[i] + tied(before_ties, sh.warp_count[i]);
        if (drawn < before + with) break;
        before += with, before_ties += sh.warp_count[i];
      }
      const int64_t n = b0 - a0;
      b0 = a0 + int(n * (i + 1) / kSampleWarps), a0 += int(n * i / kSampleWarps);
    }
    if (warp == 0) {
      bool done = false;
      for (int i0 = a0; i0 < b0 && !done; i0 += 32) {
        const int i = i0 + lane;
        uint4 r = make_uint4(masked_bits<T>(), masked_bits<T>(), masked_bits<T>(), masked_bits<T>());
        if (i < b0) r = x.cache ? x.cache[i - x.first] : x.load(i);
        float v[G];
        Elem<T>::unpack(r, v);
        uint64_t m[G], lane_sum = 0;
        uint32_t lane_ties = 0;
#pragma unroll
        for (int k = 0; k < G; ++k) lane_ties += v[k] == border;
        uint64_t tie = before_ties + warp_prefix(lane_ties) - lane_ties;
        before_ties += __reduce_add_sync(0xffffffffu, lane_ties);
#pragma unroll
        for (int k = 0; k < G; ++k) {
          m[k] = 0;
          if (v[k] == border) {
            m[k] = tied(tie, 1), ++tie;
          } else if (v[k] > border) {
            m[k] = weight_of(w, v[k]);
            if (m[k] < least) m[k] = 0;
          }
          lane_sum += m[k];
        }
        uint64_t sums = before + warp_prefix(lane_sum) - lane_sum;
        before += warp_sum(lane_sum);
#pragma unroll
        for (int k = 0; k < G; ++k) {
          if (drawn >= sums && drawn < sums + m[k]) a.out[row] = i * G - x.skew + k;
          sums += m[k];
        }
        done = drawn < before;
      }
    }
  }
  cluster.sync();  // the sums have been read
}

template <class T>
static int launch_sample(SampleArgs& a, int64_t rows, cudaStream_t s) {
  const char* who = "q1_sample launch";
  static bool set[64] = {};
  constexpr int kCache = 76 * 1024;  // with 34 KB of its own, a CTA of two on an SM
  int dev = 0;
  if (int e = cuda_status(cudaGetDevice(&dev), who)) return e;
  if (dev < 0 || dev >= 64 || !set[dev]) {
    if (int e = cuda_status(cudaFuncSetAttribute(k_sample<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kCache), who)) return e;
    if (int e = cuda_status(cudaFuncSetAttribute(k_sample<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1), who)) return e;
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  // Two CTAs an SM; each with at least 2048 values.
  a.ctas = 1;
  while (a.ctas < 16 && rows * a.ctas * 2 <= 2 * num_sms() && a.vocab > 2048 * a.ctas) a.ctas *= 2;
  constexpr int G = Elem<T>::kGroup;
  const int groups = (a.vocab + 2 * G - 2) / G, slice = (groups + a.ctas - 1) / a.ctas * 16;
  a.cached = slice <= kCache;
  return launch_op<SampleArgs>(k_sample<T>, dim3(unsigned(rows * a.ctas)), kSampleThreads, a.cached ? size_t(slice) : 0, a.ctas, s, who, a);
}

}  // namespace q1

using namespace q1;

extern "C" int q1_sample(const void* logits, int64_t ld, int64_t rows, int64_t vocab, int dtype, const float* uniform,
                         const q1_sampling* settings, int32_t* out, void* stream) {
  const char* who = "q1_sample";
  if (rows < 1 || rows > 65535 || vocab < 1 || vocab > (int64_t(1) << 19))
    return fail(Q1_ERR_ARG, "%s: bad shape rows=%lld vocab=%lld", who, (long long)rows, (long long)vocab);
  if (dtype != Q1_F32 && dtype != Q1_BF16 && dtype != Q1_F16) return fail(Q1_ERR_ARG, "%s: bad type %d", who, dtype);
  if (!logits || !uniform || !settings || !out) return fail(Q1_ERR_ARG, "%s: null pointer", who);
  if (ld < vocab && ld != 0) return fail(Q1_ERR_ARG, "%s: a row stride is less than vocab", who);
  if (reinterpret_cast<uintptr_t>(logits) % (dtype == Q1_F32 ? 4 : 2) || !aligned4(uniform) || !aligned4(out) ||
      !aligned4(settings->temperature) || !aligned4(settings->top_k) || !aligned4(settings->top_p) || !aligned4(settings->min_p))
    return fail(Q1_ERR_ARG, "%s: a misaligned pointer", who);
  if ((!settings->temperature && std::isnan(settings->temperature_all)) || (!settings->top_p && std::isnan(settings->top_p_all)) ||
      (!settings->min_p && std::isnan(settings->min_p_all)))
    return fail(Q1_ERR_ARG, "%s: a setting for all rows is NaN", who);
  SampleArgs a = {logits, ld, uniform, *settings, out, int(vocab), 1, 0};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == Q1_F32) return launch_sample<float>(a, rows, s);
  if (dtype == Q1_BF16) return launch_sample<__nv_bfloat16>(a, rows, s);
  return launch_sample<__half>(a, rows, s);
}
