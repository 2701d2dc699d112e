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
// sums are 64-bit integers: exact, in any order, the same in every launch.  (In f32, 10^5
// weights' sums are off by as much as some of the weights.)
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
//   3  (top-p, large top-k, or a list that is too long) how many tokens there are in each of
//      2048 bins of the exponent, joined through distributed shared memory.  Counts
//      times the weights of bins' middles tell to some 10^-4 where the sum crosses its border:
//      a few bins around that are listed, while the weights of all tokens are summed;
//   4  one CTA sorts the list and draws, if it is all that can stay, or finds the last token
//      that stays (where it does not lie in the list after all, or there are too many equal tokens:
//      by exact histograms of the values' bits, ten at a time);
//   5  sums by warp, whose one holds the drawn token, and the token in it.
// Bytes would bound it (33 MB, 5 us, for 64 rows of 128256 f32 logits); what does is, for one row, the chain
// of steps between barriers (profiled: the first stall reason), and for many rows with a large nucleus the weights'
// instructions (256 rows: issued in 70 % of the cycles, the pipe of shifts and masks 54 % active).
// (The arithmetic two values an instruction is 3 % faster for 256 rows and up to 5 % slower else; histograms of
// exact sums instead of counts took 3 shared atomics a value: 404 us for 256 rows.)
//
// Measured: one row of 128256 f32 logits, top-k 50 and top-p 0.95, 10.7 us; 64 rows of those 16.5, greedy 10.8, without
// cuts 23, with settings of their own 54 to 81 (what the largest nucleus takes); 256 rows of
// 151937 bf16 logits, a nucleus of 0.9 over a flat distribution, 173 us.  Exact histograms, where the bins around the
// border hold more tokens than the list (a spread of 1 at temperature 1 and top-p 0.9 does): 64 rows of 128256 103 us, one
// row of 262144 56 (33 to 34 where the list suffices); where there are three different logits 190 (64 rows of 128256).
#include <algorithm>
#include <cfloat>
#include <cmath>

#include <cooperative_groups.h>

#include "ops.cuh"

namespace q1 {

namespace cg = cooperative_groups;

constexpr int kSampleThreads = 512, kSampleWarps = kSampleThreads / 32;
constexpr int kBins = 2048;          // of exponents
constexpr int kDigits = 1024;        // of ten bits of a value
constexpr int kListed = 1024;        // tokens that one CTA sorts
// Top-k by the threads' maxima, else by counts.  (64 rows of 128256 f32 logits: k = 20 15.9 us and 32.3, 256 20.5 and 38,
// 400 30.5 and 37.3; one row: 400 20.4 and 19.2, which the rule does not tell apart.  Larger k were not compared.)
constexpr int kFewTopK = 400;
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
  const float d = __fsub_rn(x, w.max);
  const float y = fmaxf(__fmul_rn(d, w.ch), kLeast - 16.f);  // far below: zero whatever the rest is (-inf times 0 too)
  const float back = __fsub_rn(d, x);
  const float lost = __fsub_rn(__fsub_rn(x, __fsub_rn(d, back)), __fadd_rn(w.max, back));  // x - max - d
  const float rest = __fmaf_rn(lost, w.ch, __fmaf_rn(d, w.cl, __fmaf_rn(d, w.ch, -y)));
  // y = n + k / 512 + r: rounded by adding 1.5 2^23 (|y| 512 < 2^22)
  const float z = __fmaf_rn(y, float(kSteps), kMagic);
  const uint32_t whole = __float_as_uint(z);  // n 512 + k, and kMagicBits
  const float r = __fadd_rn(__fmaf_rn(__fsub_rn(z, kMagic), -1.0f / kSteps, y), rest);
  const float p = __fmul_rn(r, __fmaf_rn(r, 0.24022651f, 0.69314718f));  // 2^r - 1
  const uint32_t t = w.powers[whole & (kSteps - 1)];
  // t p < 2^22, rounded by the same addition; t as a float (truncated) by its bits
  const float tf = __uint_as_float((t >> 8) + (157u << 23));
  const uint32_t bits = t + (__float_as_uint(__fmaf_rn(tf, p, kMagic)) - kMagicBits);
  // bits 2^(13 + n): 2^32 bits, moved right by 19 - n (up to 79; from 64 on nothing is left)
  const uint32_t by = 32 + 31 - kOne + (kMagicBits >> 9) - (whole >> 9);
  const uint32_t low = __funnelshift_rc(__funnelshift_rc(0u, bits, by), 0u, uint32_t(max(int(by) - 32, 0)));
  return uint64_t(__funnelshift_rc(bits, 0u, by)) << 32 | low;
}
static_assert(kSteps == 512, "the shift above");

__device__ __forceinline__ uint32_t order_of(float x) {  // rises with x; -0 as 0
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.f));
  return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_order(uint32_t o) { return __uint_as_float(o >> 31 ? o ^ 0x80000000u : ~o); }

// The bin of an exponent in (kLeast, 0], which rises where the exponent falls, and the exponent in its middle.
__device__ __forceinline__ int bin_of(float y) {
  return int(__float_as_uint(__fmaf_rn(y, (kBins - 1) / kLeast, kMagic)) - kMagicBits);
}
__device__ __forceinline__ float middle_of(int bin) { return float(bin) * (kLeast / (kBins - 1)); }
// What part of itself the sum by middles may be off by for the bins around a border to hold it.  f32 logits
// spread over the bins: it is off by some 10^-5; those of 16 bits lie anywhere in theirs.  (f32 copies of 16-bit logits
// may be further off and then take the exact histograms: 64 rows of 128256, top-p 0.9, 59 us, other f32 logits 60.)
template <class T>
constexpr uint64_t kMiddles = sizeof(T) == 4 ? 8192 : 2048;

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

// What a histogram's search gives: the digit, what lies before it and in it.
struct Found {
  int digit;
  uint32_t above, in;
  uint64_t mass_above, mass_in;
};

struct SampleShared {
  uint32_t powers[kSteps];
  // This CTA's bins and the row's; or the counts, low and high halves of the sums of this CTA's digits and the row's counts.
  uint32_t count[kBins], all_count[kBins];
  union {
    uint64_t all_mass[kDigits];
    uint64_t sorted[kListed];
  };
  uint64_t list[kListed];
  uint64_t warp_mass[kSampleWarps], warp_base[kSampleWarps], warp_above[kSampleWarps];
  uint32_t warp_count[kSampleWarps];
  Found found;
  float own_max;
  float own_reached;       // what at least its part of top-k tokens reach
  int own_bad, listed, token;
  uint64_t own_mass, own_base, own_above;
  int border[4];           // of the search of bins: see there
  uint32_t border_count[4];  // of the bin that top-k reaches into; of the bins to look at
  bool cut_found;          // of the leader: the last token that stays
  uint32_t cut_value;
  int cut_place;
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
    return e >= 0 && e + G <= vocab ? *reinterpret_cast<const uint4*>(row + e) : load_edge(row, e, vocab);
  }
  static __device__ __noinline__ uint4 load_edge(const T* row, int e, int vocab) {
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
  // f(group's values, its first element) over groups [a, b) of a warp, lane by lane; the first time (kFirst) they
  // come from global memory and go to the cache.
  // Light work: four groups loaded at a time.
  template <bool kFirst, class F>
  __device__ __forceinline__ void each(int a, int b, F&& f) const {
    for (int i0 = a + int(threadIdx.x & 31); i0 < b; i0 += 128) {
      uint4 r[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) r[k] = i0 + 32 * k < b ? kFirst || !cache ? load(i0 + 32 * k) : cache[i0 + 32 * k - first] : nothing();
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
  // Weights: a group at a time, three ahead under way.  (Fewer instructions to fetch: 256 rows 204 us, 211 with four at a
  // time; the maximum alone 29000 cycles this way and 17000 the other.)
  template <class F>
  __device__ __forceinline__ void each_heavy(int a, int b, F&& f) const {
    constexpr int kAhead = 3;
    const auto get = [&](int i) { return i >= b ? nothing() : cache ? cache[i - first] : load(i); };
    uint4 r[kAhead];
    int i = a + int(threadIdx.x & 31);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) r[k] = get(i + 32 * k);
#pragma unroll 1
    for (; i < b; i += 32) {
      const uint4 now = r[0];
#pragma unroll
      for (int k = 0; k + 1 < kAhead; ++k) r[k] = r[k + 1];
      r[kAhead - 1] = get(i + 32 * kAhead);
      float v[G];
      Elem<T>::unpack(now, v);
      f(v, i * G - skew);
    }
  }
  static __device__ __forceinline__ uint4 nothing() {
    return make_uint4(masked_bits<T>(), masked_bits<T>(), masked_bits<T>(), masked_bits<T>());
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

// The first digit up to which the counts reach `need` (by mass: the sums), after
// `above` and `mass_above` before the histogram; its last one with anything in it
// where none does.  Every thread of the CTA calls and gets it.
__device__ __forceinline__ Found search(SampleShared& sh, bool by_mass, uint64_t need, uint32_t above, uint64_t mass_above) {
  constexpr int kEach = kDigits / kSampleThreads;
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
  __syncthreads();
  uint32_t nb = above + nincl - ns;
  uint64_t mb = mass_above + mincl - ms;
  uint32_t total = above;
  for (int w = 0; w < kSampleWarps; ++w) {
    if (w < warp) nb += sh.warp_count[w], mb += sh.warp_mass[w];
    total += sh.warp_count[w];
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint64_t before = by_mass ? mb : nb, after = by_mass ? mb + m[i] : uint64_t(nb) + n[i];
    if (n[i] && ((before < need && after >= need) || (after < need && nb + n[i] == total)))
      sh.found = {int(threadIdx.x) * kEach + i, nb, n[i], mb, m[i]};
    nb += n[i], mb += m[i];
  }
  __syncthreads();
  return sh.found;
}

// Bitonic, kEach (1 or 2) entries a thread; exchanges within a warp's entries by shuffles.
template <int kEach>
__device__ __forceinline__ void sort_bitonic(uint64_t* v, int n) {
  const int lane = threadIdx.x & 31, first = int(threadIdx.x >> 5) * 32 * kEach + lane;
  uint64_t mine[kEach];  // entries first and (two of them) first + 32
#pragma unroll
  for (int k = 0; k < kEach; ++k) mine[k] = first + 32 * k < n ? v[first + 32 * k] : ~uint64_t(0);
  const auto keep = [&](uint64_t& x, uint64_t other, int at, int step, int size) {
    if ((other < x) == (((at & step) == 0) == ((at & size) == 0))) x = other;
  };
  for (int size = 2; size <= kSampleThreads * kEach; size <<= 1)
    for (int step = size >> 1; step > 0; step >>= 1) {
      if (step >= 32 * kEach) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) v[first + 32 * k] = mine[k];
        __syncthreads();
        uint64_t other[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) other[k] = v[(first + 32 * k) ^ step];
#pragma unroll
        for (int k = 0; k < kEach; ++k) keep(mine[k], other[k], first + 32 * k, step, size);
        __syncthreads();
      } else if (step == 32) {
        const uint64_t lo = min(mine[0], mine[kEach - 1]), hi = max(mine[0], mine[kEach - 1]);
        const bool rising = (first & size) == 0;
        mine[0] = rising ? lo : hi, mine[kEach - 1] = rising ? hi : lo;
      } else {
#pragma unroll
        for (int k = 0; k < kEach; ++k) keep(mine[k], __shfl_xor_sync(0xffffffffu, mine[k], step), first + 32 * k, step, size);
      }
    }
#pragma unroll
  for (int k = 0; k < kEach; ++k) v[first + 32 * k] = mine[k];
  __syncthreads();
}

// Sorts the n (up to kListed) different entries of sh.sorted, rising.
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
  static_assert(kListed == 2 * kSampleThreads, "");
  if (n <= kSampleThreads)
    sort_bitonic<1>(v, n);
  else
    sort_bitonic<2>(v, n);
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
  for (int i = threadIdx.x; i < kBins; i += kSampleThreads) sh.count[i] = 0;
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
  // 4. The first CTA collects all lists, up to kListed tokens in all, and sorts them by falling values,
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
  const auto enough_of = [&](uint64_t mass) { return max(part_of(fmaxf(top_p, 0.f), mass, true), uint64_t(1)); };
  constexpr int kEach = kListed / kSampleThreads;
  // The token, where all that may stay is among the n tokens sorted: the first `count` of them, then by mass.
  const auto finish = [&](int n, int count, uint64_t base) {  // base: the sum that top-p is of, 0 for that of those
    uint64_t weight[kEach], sum = 0, all;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int i = threadIdx.x * kEach + k;
      weight[k] = i < min(n, count) ? entry_weight(uint32_t(sh.sorted[i] >> 32)) : 0;
      sum += weight[k];
    }
    uint64_t before = block_prefix(sh, sum, all) - sum;
    const uint64_t need = by_mass ? enough_of(base ? base : all) : 0;
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

  // Of this CTA's slice, in the vocabulary's order, the token at which the sum of value(x, token) exceeds pick(sum of the row);
  // -1 in all CTAs but the one that has it.  `summed`: sh.warp_mass holds the warps' sums.
  const auto locate = [&](bool summed, auto&& value, auto&& pick) {
    const auto sum_of = [&](int a0, int b0) {
      uint64_t sum = 0;
      x.each_heavy(a0, b0, [&](const float (&v)[G], int e) {
#pragma unroll
        for (int i = 0; i < G; ++i) sum += value(v[i], e + i);
      });
      sum = warp_sum(sum);
      __syncthreads();
      if (lane == 0) sh.warp_mass[warp] = sum;
      __syncthreads();
    };
    if (!summed) sum_of(from, to);
    if (threadIdx.x == 0) {
      uint64_t m = 0;
      for (int i = 0; i < kSampleWarps; ++i) m += sh.warp_mass[i];
      sh.own_mass = m;
    }
    cluster.sync();
    const uint64_t own = lane < a.ctas ? cluster.map_shared_rank(&sh, lane)->own_mass : 0, upto = warp_prefix(own);
    const uint64_t target = pick(__shfl_sync(0xffffffffu, upto, 31));
    uint64_t before = __shfl_sync(0xffffffffu, upto - own, rank);
    if (target < before || target >= before + __shfl_sync(0xffffffffu, own, rank)) return -1;
    // The warp's part that holds it, then its sixteenth, then the token.
    int a0 = x.first, b0 = x.last;
    for (int round = 0; round < 2; ++round) {
      const int n = b0 - a0;
      if (round) sum_of(a0 + int(int64_t(n) * warp / kSampleWarps), a0 + int(int64_t(n) * (warp + 1) / kSampleWarps));
      const uint64_t m = lane < kSampleWarps ? sh.warp_mass[lane] : 0, to_here = before + warp_prefix(m);
      const int i = __ffs(int(__ballot_sync(0xffffffffu, lane < kSampleWarps && target < to_here))) - 1;  // (there is one)
      before = __shfl_sync(0xffffffffu, to_here - m, i);
      b0 = a0 + int(int64_t(n) * (i + 1) / kSampleWarps), a0 += int(int64_t(n) * i / kSampleWarps);
    }
    if (warp == 0) {
      for (int i0 = a0; i0 < b0; i0 += 32) {
        const int i = i0 + lane;
        uint4 r = make_uint4(masked_bits<T>(), masked_bits<T>(), masked_bits<T>(), masked_bits<T>());
        if (i < b0) r = x.cache ? x.cache[i - x.first] : x.load(i);
        float v[G];
        Elem<T>::unpack(r, v);
        uint64_t m[G], sum = 0;
#pragma unroll
        for (int k = 0; k < G; ++k) m[k] = value(v[k], i * G - x.skew + k), sum += m[k];
        uint64_t upto = before + warp_prefix(sum) - sum;
#pragma unroll
        for (int k = 0; k < G; ++k) {
          if (target >= upto && target < upto + m[k]) sh.token = i * G - x.skew + k;
          upto += m[k];
        }
        before = __shfl_sync(0xffffffffu, upto, 31);
        if (target < before) break;
      }
    }
    __syncthreads();
    return sh.token;
  };

  float border = -INFINITY;  // tokens above it stay, and those at it up to this place
  int place = -1;
  bool summed = false;       // the warps' sums of what stays are known
  const auto stays = [&](float v, int e) { return v > border || (v == border && e <= place); };
  const auto kept_weight = [&](float v, int e) -> uint64_t {
    if (!stays(v, e)) return 0;
    const uint64_t m = weight_of(w, v);
    return m >= least ? m : 0;
  };
  if (by_count || by_mass) {
    // 3. Counts by exponents.
    x.each_heavy(from, to, [&](const float (&v)[G], int) {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const float y = exponent_of(w, v[i]);
        if (y > kLeast) atomicAdd(&sh.count[bin_of(y)], 1u);
      }
    });
    cluster.sync();
    {
      const int share = kBins / a.ctas;
      if (a.ctas >= 4) {  // ctas / 4 threads a bin take four CTAs each, join, and give the sum to those four
        const int part = int(threadIdx.x) / share, b = rank * share + int(threadIdx.x) % share;
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) n += cluster.map_shared_rank(&sh, 4 * part + i)->count[b];
        sh.list[threadIdx.x] = n;
        __syncthreads();
        n = 0;
        for (int i = int(threadIdx.x) % share; i < kSampleThreads; i += share) n += uint32_t(sh.list[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) cluster.map_shared_rank(&sh, 4 * part + i)->all_count[b] = n;
      } else {
        for (int b = rank * share + int(threadIdx.x); b < (rank + 1) * share; b += kSampleThreads) {
          uint32_t n = 0;
          for (int r = 0; r < a.ctas; ++r) n += cluster.map_shared_rank(&sh, r)->count[b];
          for (int r = 0; r < a.ctas; ++r) cluster.map_shared_rank(&sh, r)->all_count[b] = n;
        }
      }
    }
    cluster.sync();
    // The bins to look at: [lo, hi] around top-p's border, `end` the last one that top-k reaches into (if it leaves
    // any out: `cut`), with counts before and in them.
    int lo, hi, end;
    bool cut;
    uint32_t before_lo, upto_hi, before_end = 0, in_end = 0;
    {
      constexpr int kBinsEach = kBins / kSampleThreads;
      const int b0 = int(threadIdx.x) * kBinsEach;
      uint32_t n[kBinsEach], ns = 0;
      uint64_t m[kBinsEach], ms = 0;
      constexpr float kNext = 0.98521119f;  // 2^(-44 / 2047)
      static_assert(kBins == 2048 && kLeast == -44.f, "");
      float middle = exp2f(middle_of(b0)) * float(uint64_t(1) << kOne);
#pragma unroll
      for (int i = 0; i < kBinsEach; ++i) {
        n[i] = sh.all_count[b0 + i];
        m[i] = n[i] * __float2ull_rn(middle);
        middle *= kNext;
        ns += n[i], ms += m[i];
      }
      uint64_t total, of;
      const uint32_t nb = uint32_t(block_prefix(sh, ns, total)) - ns;
      const uint64_t mb = block_prefix(sh, ms, of) - ms;
      if (threadIdx.x < 3) sh.border[threadIdx.x] = -1;
      __syncthreads();
      // f(bin, counts and sums before and with it) for this thread's bins.
      const auto bins = [&](auto&& f) {
        uint32_t count = nb;
        uint64_t mass = mb;
#pragma unroll
        for (int i = 0; i < kBinsEach; ++i) {
          f(b0 + i, count, count + n[i], mass, mass + m[i]);
          count += n[i], mass += m[i];
        }
      };
      cut = by_count && uint64_t(top_k) < total;
      if (cut) {
        bins([&](int b, uint32_t count, uint32_t with, uint64_t mass, uint64_t) {
          if (count >= uint32_t(top_k) || with < uint32_t(top_k)) return;
          sh.border[2] = b, sh.border_count[0] = count, sh.border_count[1] = with - count;
          sh.own_mass = mass + (uint32_t(top_k) - count) * __float2ull_rn(exp2f(middle_of(b)) * float(uint64_t(1) << kOne));
        });
        __syncthreads();
        before_end = sh.border_count[0], in_end = sh.border_count[1], of = sh.own_mass;
      }
      end = cut ? sh.border[2] : kBins - 1;
      lo = hi = end;
      if (by_mass) {
        const uint64_t border_sum = enough_of(of), least_sum = max(border_sum - border_sum / kMiddles<T>, uint64_t(1)),
                       most_sum = border_sum + border_sum / kMiddles<T>;
        bins([&](int b, uint32_t, uint32_t, uint64_t mass, uint64_t with) {
          if (mass < least_sum && with >= least_sum) sh.border[0] = b;
          if (mass < most_sum && with >= most_sum) sh.border[1] = b;
        });
        __syncthreads();
        if (sh.border[0] >= 0) lo = min(lo, sh.border[0]);
        if (sh.border[1] >= 0) hi = min(hi, sh.border[1]);
      }
      bins([&](int b, uint32_t count, uint32_t with, uint64_t, uint64_t) {
        // (not the words above: without top-p no barrier lies between their last reader and here)
        if (b == lo) sh.border_count[2] = count;
        if (b == hi) sh.border_count[3] = with;
      });
      __syncthreads();
      before_lo = sh.border_count[2], upto_hi = sh.border_count[3];
    }
    const bool whole = max(upto_hi, before_end + in_end) <= kListed;  // all that may stay can be listed
    const bool apart = cut && end > hi;
    bool found = !cut && !by_mass;  // nothing is left out
    if (!found && (whole || upto_hi - before_lo + (apart ? in_end : 0) <= kListed)) {
      // The sums: of all that top-p is of but for the bin `end` (base), of what lies before lo (above), of what stays of it (kept).
      const int list_from = whole ? 0 : lo, list_to = whole && cut ? end : hi;
      const bool weigh = !whole || (by_mass && !cut);
      uint64_t base = 0, above = 0, kept = 0;
      const int base_to = cut ? end : kBins + 1, apart_at = cut ? end : -1;
      const bool any_weight = least == 1;
      x.each_heavy(from, to, [&](const float (&v)[G], int e) {
#pragma unroll
        for (int i0 = 0; i0 < G; i0 += 4) {  // four side by side, what is rare behind them
          int b[4];
          bool some = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float y = exponent_of(w, v[i0 + i]);
            b[i] = y > kLeast ? bin_of(y) : kBins;
            some |= (b[i] >= list_from && b[i] <= list_to) || b[i] == apart_at;
          }
          if (weigh) {
            uint64_t m[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = weight_of(w, v[i0 + i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              base += b[i] < base_to ? m[i] : 0;
              above += b[i] < list_from ? m[i] : 0;
            }
            if (!any_weight) {
#pragma unroll
              for (int i = 0; i < 4; ++i) kept += b[i] < list_from && m[i] >= least ? m[i] : 0;
            }
          }
          if (some) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((b[i] >= list_from && b[i] <= list_to) || b[i] == apart_at) list(v[i0 + i], e + i0 + i);
          }
        }
      });
      if (any_weight) kept = above;
      base = warp_sum(base), above = warp_sum(above), kept = warp_sum(kept);
      if (lane == 0) sh.warp_base[warp] = base, sh.warp_above[warp] = above;
      __syncthreads();
      if (threadIdx.x == 0) {
        base = above = 0;
        for (int i = 0; i < kSampleWarps; ++i) base += sh.warp_base[i], above += sh.warp_above[i];
        sh.own_base = base, sh.own_above = above;
      }
      const int n = collect();  // (as many as the counts say: none are left out)
      if (rank == 0) {
        const SampleShared* his = cluster.map_shared_rank(&sh, lane < a.ctas ? lane : 0);
        base = warp_sum(lane < a.ctas ? his->own_base : 0), above = warp_sum(lane < a.ctas ? his->own_above : 0);
        uint64_t weight[kEach], sum = 0, all;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
          const int i = threadIdx.x * kEach + k;
          weight[k] = i < n ? entry_weight(uint32_t(sh.sorted[i] >> 32)) : 0;
          sum += weight[k];
        }
        const uint64_t first = block_prefix(sh, sum, all) - sum;
        const int left = cut ? n - int(in_end) + top_k - int(before_end) : n;  // entries that top-k leaves
        if (whole) {
          // (top-p's border lies beyond the list where the middles were too far off)
          const bool reaches = cut || !by_mass || all >= enough_of(base);
          if (threadIdx.x == 0) sh.cut_found = reaches;
          if (reaches) finish(n, left, cut ? 0 : base);
        } else {
          if (threadIdx.x == 0) sh.cut_found = false;
          __syncthreads();
          uint64_t before = above + first;
          uint64_t need = 0;
          if (by_mass) {
            if (cut) {  // and of the bin `end`, what top-k leaves
              sum = 0;
#pragma unroll
              for (int k = 0; k < kEach; ++k) {
                const int i = threadIdx.x * kEach + k;
                if (i >= n - int(in_end) && i < left) sum += weight[k];
              }
              (void)block_prefix(sh, sum, all);
              base += all;
            }
            need = enough_of(base);
          }
          const int together = apart ? n - int(in_end) : left;  // entries that follow what lies before lo without a gap
#pragma unroll
          for (int k = 0; k < kEach; ++k) {
            const int i = threadIdx.x * kEach + k;
            const bool is = by_mass ? i < together && before < need && before + weight[k] >= need : i == left - 1;
            if (is) sh.cut_found = true, sh.cut_value = ~uint32_t(sh.sorted[i] >> 32), sh.cut_place = int(uint32_t(sh.sorted[i]));
            before += weight[k];
          }
        }
      }
      cluster.sync();
      const SampleShared* his = cluster.map_shared_rank(&sh, 0);
      found = his->cut_found;
      if (found && !whole) {
        border = of_order(his->cut_value), place = his->cut_place;
        // What stays of this CTA's list joins its warps' sums.
        if (lane == 0) sh.warp_mass[warp] = kept;
        __syncthreads();
        for (int i = threadIdx.x; i < sh.listed; i += kSampleThreads) {
          const float v = of_order(~uint32_t(sh.list[i] >> 32));
          const int e = int(uint32_t(sh.list[i]));
          const uint64_t m = kept_weight(v, e);
          if (!m) continue;
          const int g = (e + x.skew) / G - x.first;
          int k = int(int64_t(g) * kSampleWarps / mine);
          while (k + 1 < kSampleWarps && g >= int(int64_t(mine) * (k + 1) / kSampleWarps)) ++k;
          atomicAdd(reinterpret_cast<unsigned long long*>(&sh.warp_mass[k]), static_cast<unsigned long long>(m));
        }
        summed = true;
      }
      cluster.sync();
      if (found && whole) return;
    }
    if (!found) {
      // Exact histograms of the values' bits: the token at which the count, then the sum is reached.
      uint64_t need = cut ? uint64_t(top_k) : 0, kept = 0;
      uint32_t *counts = sh.count, *low = sh.count + kDigits, *high = sh.all_count + kDigits;
      for (bool mass = !cut;; mass = true) {
        uint32_t prefix = 0, known = 0;  // the bits found
        Found at = {0, 0, 0, 0, 0};
#pragma unroll 1
        for (int shift = 22;; shift = max(0, shift - 10)) {
          const uint32_t width = known ? min(10, __ffs(int(known)) - 1 - shift) : 10;
          const uint32_t most = (1u << width) - 1;
          __syncthreads();
          for (int i = threadIdx.x; i < kDigits; i += kSampleThreads) counts[i] = low[i] = high[i] = 0;
          __syncthreads();
          x.each_heavy(from, to, [&](const float (&v)[G], int) {
#pragma unroll
            for (int i = 0; i < G; ++i) {
              const uint32_t o = order_of(v[i]);
              if ((o & known) != prefix) continue;
              const uint64_t m = weight_of(w, v[i]);
              if (!m) continue;
              const uint32_t b = most - ((o >> shift) & most);
              atomicAdd(&counts[b], 1u);
              const uint32_t old = atomicAdd(&low[b], uint32_t(m));
              atomicAdd(&high[b], uint32_t(m >> 32) + (old + uint32_t(m) < old));
            }
          });
          cluster.sync();
          const int share = kDigits / a.ctas;
          for (int b = rank * share + int(threadIdx.x); b < (rank + 1) * share; b += kSampleThreads) {
            uint32_t n = 0;
            uint64_t m = 0;
            for (int r = 0; r < a.ctas; ++r) {
              const SampleShared* his = cluster.map_shared_rank(&sh, r);
              n += his->count[b], m += uint64_t(his->all_count[kDigits + b]) << 32 | his->count[kDigits + b];
            }
            for (int r = 0; r < a.ctas; ++r) {
              SampleShared* his = cluster.map_shared_rank(&sh, r);
              his->all_count[b] = n, his->all_mass[b] = m;
            }
          }
          cluster.sync();
          if (mass && need == 0) {
            uint64_t all;
            (void)block_prefix(sh, sh.all_mass[threadIdx.x] + sh.all_mass[threadIdx.x + kSampleThreads], all);
            need = enough_of(cut ? kept : all);
          }
          at = search(sh, mass, need, at.above, at.mass_above);
          prefix |= (most - uint32_t(at.digit)) << shift, known |= most << shift;
          if (shift == 0 || (G == 8 && shift <= 12)) break;
        }
        if (G == 8) prefix |= prefix >> 31 ? 0 : 0xfffu;  // the bits that 16-bit types do not have
        // Of the tokens of this value as many as it takes, the first ones.
        const uint64_t each = at.mass_in / at.in;
        const uint64_t ties = min(mass ? (need - at.mass_above + each - 1) / each : need - at.above, uint64_t(at.in));
        border = of_order(prefix), kept = at.mass_above + ties * each;
        if (mass || !by_mass) {
          const int last = locate(false, [&](float v, int) { return uint64_t(v == border); }, [&](uint64_t) { return ties - 1; });
          if (last >= 0 && threadIdx.x < a.ctas) cluster.map_shared_rank(&sh, threadIdx.x)->cut_place = last;
          cluster.sync();
          place = sh.cut_place;
          break;
        }
        need = 0;
      }
    }
  }

  // 5. The token.
  const auto pick = [&](uint64_t all) { return part_of(u, all, false); };
  const int token = border == -INFINITY && least == 1 ? locate(false, [&](float v, int) { return weight_of(w, v); }, pick)
                                                      : locate(summed, kept_weight, pick);
  if (token >= 0 && threadIdx.x == 0) a.out[row] = token;
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
  // As many CTAs a row as run at once, two an SM, each with at least 2048 values.  (Twice as many, in two rounds: 64
  // rows of top-k 50 25.6 us, 16.5 this way; with settings of their own, some of which take much longer, 61 and 82.)
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
