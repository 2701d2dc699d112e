// attend.cuh -- what the two paged attention kernels share: their arguments,
// the split of the work into items and units, and the join of split items.
#pragma once

#include <type_traits>

#include "paged.cuh"

namespace q1 {

struct AttendArgs {
  Paged kv;
  const void* q;           // [total_new][heads][dim], strides below
  void* out;
  int64_t q_token, q_head, o_token, o_head;  // elements
  float* part;             // partial results: two slots a CTA, see Partial
  struct JoinItem* joins;  // [CTAs]
  unsigned* status;
  int heads, group;        // query heads, and of one key head
  uint32_t group_inverse;  // 2^32 / group + 1 (group > 1), see by_group
  float scale_log2;        // scale * log2(e)
  int ctas;                // CTAs the units are split over, or of a cluster
  int tiles;               // with clusters: of a key head, at once
  int least_rows, most_rows;  // of a sequence that this launch takes (its new tokens times the group)
  // The launch before is the same call's, of other sequences: no wait for it at the start.
  // All of this library's kernels wait for the one before them before they end, and k_attend_tc
  // before it lets the next start, so this holds also where another thread launches one of them
  // in between: it starts behind k_attend_tc's wait, and what follows waits for all of them.
  bool beside;
};

// n / group, 0 <= n < 2^31: n * (2^32 / group + 1) / 2^32 is the quotient or
// one more.  (A hardware division by a run-time value takes some forty instructions.)
__device__ __forceinline__ int by_group(const AttendArgs& a, int n) {
  if (a.group == 1) return n;  // (2^32 itself would not fit)
  const int q = int(__umulhi(uint32_t(n), a.group_inverse));
  return q - (q * a.group > n);
}

__device__ __forceinline__ float ex2(float x) {  // 2^x, 0 at -inf
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// The work.  Rows of (sequence b, key head h) are its new tokens times the
// group's heads, token-major; a tile is TM of them, an item a tile with all
// keys it may see, cut into units of TK keys (one unit at least).  Items lie on one axis,
// sequences first, then key heads, then tiles, and CTA c of N takes units
// [U c / N, U (c + 1) / N) of it: equal shares of keys whatever the lengths
// are.  An item that no CTA has to itself is joined by k_attend_join.
template <int TM, int TK>
struct Tiling {
  __device__ static int tiles(const AttendArgs& a, const SeqSpan& s) {
    const int rows = s.count * a.group;
    return rows >= a.least_rows && rows <= a.most_rows ? (rows + TM - 1) / TM : 0;
  }
  // Keys that tile m of s may see: those of its last row.
  __device__ static int keys(const AttendArgs& a, const SeqSpan& s, int m) {
    const int last = min(s.count - 1, by_group(a, m * TM + TM - 1));
    return max(0, s.len - s.count + last + 1);
  }
  // Keys that the first row of tile m of s sees: all its rows do.
  __device__ static int keys_of_all(const AttendArgs& a, const SeqSpan& s, int m) {
    return max(0, s.len - s.count + by_group(a, m * TM) + 1);
  }
  __device__ static int units(const AttendArgs& a, const SeqSpan& s, int m) { return max(1, (keys(a, s, m) + TK - 1) / TK); }
  __device__ static int64_t seq_units(const AttendArgs& a, const SeqSpan& s) {  // of one key head
    int64_t u = 0;
    for (int m = 0, n = tiles(a, s); m < n; ++m) u += units(a, s, m);
    return u;
  }
};

// Position on the axis: an item and the unit within it.
struct Cursor {
  int b, h, m;      // sequence, key head, tile
  int unit, units;  // of this item
  SeqSpan s;
};

// total * c / n, in 32 bits where that suffices (the usual case; a 64-bit
// division takes some hundred instructions).
__device__ __forceinline__ int64_t share(int64_t total, int c, int n) {
  if (total < (int64_t(1) << 31) / n) return uint32_t(total) * uint32_t(c) / uint32_t(n);
  return total * c / n;
}

struct LocateScratch {
  int64_t total, cut[2];
  Cursor at;
};

// Total units of the call, the number n of CTAs that have a share (n as given
// or the units, if fewer), CTA c's share [u0, u1) and the cursor at its start.
// A cut within an item of at most kWhole units moves to the item's start:
// splitting it would cost more than the balance gains.  Every thread of the
// CTA calls; the first warp looks, a run of consecutive sequences a lane.
template <class Tile, int kWhole>
__device__ __forceinline__ int64_t locate(const AttendArgs& a, int c, int& n, LocateScratch& sh, Cursor& cur, int64_t& u0,
                                          int64_t& u1) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, per = (a.kv.batch + 31) / 32;
    const int b0 = min(a.kv.batch, lane * per), b1 = min(a.kv.batch, b0 + per);
    SeqSpan first = {0, 0, 0};
    int64_t mine = 0, first_units = 0;
    for (int b = b0; b < b1; ++b) {
      bool bad;
      const SeqSpan s = seq_span(a.kv, b, &bad);
      const int64_t su = Tile::seq_units(a, s);
      if (b == b0) first = s, first_units = su;
      mine += su * a.kv.kv_heads;
      if (bad) atomicOr(a.status, kStatusBadIndex);
    }
    int64_t incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t t = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += t;
    }
    const int64_t total = __shfl_sync(0xffffffffu, incl, 31), lo = incl - mine;
    const int ctas = n < total ? n : int(total);  // so that no share between two others is empty
    if (lane == 0) sh.total = total;
#pragma unroll 1
    for (int end = 0; end < 2; ++end) {  // where the share begins, and where it ends
      const int64_t u = c + end < ctas ? share(total, c + end, ctas) : total;
      if (u == total) {
        if (lane == 0) sh.cut[end] = total;
      } else if (u >= lo && u < lo + mine) {  // the run that holds u: one lane's
        int64_t at = lo, su = first_units;
        SeqSpan s = first;
        int b = b0;
        while (u >= at + su * a.kv.kv_heads && b + 1 < b1) {
          at += su * a.kv.kv_heads;
          s = seq_span(a.kv, ++b);
          su = Tile::seq_units(a, s);
        }
        const bool small = u - at < (int64_t(1) << 31) && su < (int64_t(1) << 31);
        const int h = small ? int(uint32_t(u - at) / uint32_t(su)) : int((u - at) / su);
        int64_t start = at + h * su;  // of the item
        int m = 0, un;
        for (;; ++m) {
          un = Tile::units(a, s, m);
          if (u < start + un || u < start) break;
          start += un;
        }
        const int64_t cut = un <= kWhole ? start : u;
        sh.cut[end] = cut;
        if (end == 0) sh.at = {b, h, m, int(cut - start), un, s};
      }
    }
  }
  __syncthreads();
  if (n > sh.total) n = int(sh.total);
  u0 = sh.cut[0], u1 = sh.cut[1];
  cur = sh.at;
  return sh.total;
}

// The item after cur's (there is one).
template <class Tile>
__device__ __forceinline__ void next_item(const AttendArgs& a, Cursor& cur) {
  cur.unit = 0;
  if (++cur.m >= Tile::tiles(a, cur.s)) {
    cur.m = 0;
    if (++cur.h >= a.kv.kv_heads) {
      cur.h = 0;
      do cur.s = seq_span(a.kv, ++cur.b);
      while (Tile::tiles(a, cur.s) == 0 && cur.b + 1 < a.kv.batch);
    }
  }
  cur.units = Tile::units(a, cur.s, cur.m);
}

// Row r of a tile: its token and query head; false past the last row.
__device__ __forceinline__ bool row_of(const AttendArgs& a, const Cursor& cur, int r, int& token, int& head) {
  const int t = by_group(a, r);
  token = cur.s.first + t;
  head = cur.h * a.group + r - t * a.group;
  return t < cur.s.count;
}

// Keys that new token t (of the sequence's) sees.
__device__ __forceinline__ int keys_seen(const SeqSpan& s, int t) { return max(0, s.len - s.count + t + 1); }

// What a row's sums are multiplied with, l the sum of its weights: a row that
// sees no key is zero; one whose visible scores are all -inf is 0 / 0.
__device__ __forceinline__ float inverse(float l, int seen) {
  return l != 0.f ? __fdiv_rn(1.0f, l) : seen ? __int_as_float(0x7fc00000) : 0.f;
}

// Values of the cache that are no numbers.  A weight of zero does not keep them
// from a row that may not see them (0 * inf is NaN), so they are taken out of
// the products of keys that only some rows of a tile see, and added to the rows
// that do see them (as they are: the weight of a visible key is positive).
template <class T>
__device__ __forceinline__ bool no_number(uint32_t bits) {  // of a value's 16 bits
  constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  return (bits & e) == e;
}
template <class T>
__device__ __forceinline__ uint32_t numbers(uint32_t w) {  // of two values; zero for the others
  return (no_number<T>(w) ? 0u : w & 0xffffu) | (no_number<T>(w >> 16) ? 0u : w & 0xffff0000u);
}
template <class T>
__device__ __forceinline__ uint4 numbers(const uint4& v) {
  return make_uint4(numbers<T>(v.x), numbers<T>(v.y), numbers<T>(v.z), numbers<T>(v.w));
}
// Whether one of many values is none: the sums of their products with zero are then NaN.
template <class T>
struct NoNumbers {
  using Two = std::conditional_t<std::is_same<T, __half>::value, __half2, __nv_bfloat162>;
  uint32_t sum[2] = {0u, 0u};
  static __device__ __forceinline__ uint32_t add(uint32_t w, uint32_t sum) {
    const uint32_t zero = 0u;
    const Two r = __hfma2(reinterpret_cast<const Two&>(w), reinterpret_cast<const Two&>(zero), reinterpret_cast<const Two&>(sum));
    return reinterpret_cast<const uint32_t&>(r);
  }
  __device__ __forceinline__ void look(const uint4& v) {
    sum[0] = add(v.y, add(v.x, sum[0]));
    sum[1] = add(v.w, add(v.z, sum[1]));
  }
  __device__ __forceinline__ bool found() const {
    return no_number<T>(sum[0]) || no_number<T>(sum[0] >> 16) || no_number<T>(sum[1]) || no_number<T>(sum[1] >> 16);
  }
};
template <class T>
__device__ __forceinline__ void add_no_numbers(uint32_t w, float& lo, float& hi) {
  float x, y;
  Elem<T>::unpack2(w, x, y);
  if (no_number<T>(w)) lo += x;
  if (no_number<T>(w >> 16)) hi += y;
}

// An item that begins in a CTA and ends in a later one: what the join has to
// know of it, left by that CTA (parts = 0: none begins there).
struct JoinItem {
  int parts;              // CTAs with a part, from this one on
  int first, count;       // the sequence's new tokens
  int head, tile;         // key head and tile
  int len;                // the sequence's keys
  int pad[2];
};

// Left by one thread of every CTA: first with no item, then for the one item
// that it begins and does not end (its units begin at u, cut at u1).
__device__ __forceinline__ void leave_join(const AttendArgs& a, const Cursor& cur, int64_t u, int64_t total, int ctas) {
  // The first cut at or past the item's end: the least k with total * k / ctas >= end.
  const int64_t end = u + cur.units;
  const bool small = total < (int64_t(1) << 31) / ctas;
  const int k = small ? int((uint32_t(end) * uint32_t(ctas) + uint32_t(total) - 1) / uint32_t(total))
                      : int((end * ctas + total - 1) / total);
  a.joins[blockIdx.x] = {k - int(blockIdx.x), cur.s.first, cur.s.count, cur.h, cur.m, cur.s.len, {0, 0}};
}

// A partial result of TM rows: dim sums of p v relative to the row's maximum,
// row by row or (Turned) column by column with the rows side by side, then
// the maxima (log2 units), then the sums of p.  Slot 1 of a CTA holds the item
// that it begins, slot 0 the one that began before it.
template <int TM, int D>
__device__ __forceinline__ float* partial(const AttendArgs& a, int cta, int slot) {
  return a.part + int64_t(2 * cta + slot) * (TM * (D + 2));
}

constexpr int kJoinThreads = 256;
constexpr int kJoinSlices = 4;   // CTAs that join an item of few rows
constexpr int kJoinGroups = 8;   // threads that share a value's parts, at most

constexpr int kJoinHeld = 4;     // parts whose weights a thread holds

// The join of up to kJoinHeld column-by-column partials: a thread takes a row,
// the slices share out the columns in fours.
template <class T, int TM, int D>
__device__ __forceinline__ void join_rows(const AttendArgs& a, const JoinItem& it, int cta, int slice, int slices) {
  static_assert(TM == kJoinThreads, "a row a thread");
  const int r = threadIdx.x;
  if (r >= it.count * a.group - it.tile * TM) return;
  const float* part[kJoinHeld];
  float pm[kJoinHeld], pl[kJoinHeld];
#pragma unroll
  for (int p = 0; p < kJoinHeld; ++p) {
    part[p] = partial<TM, D>(a, cta + (p < it.parts ? p : 0), p == 0 || p >= it.parts) + r;
    pm[p] = p < it.parts ? part[p][TM * D] : -INFINITY;
    pl[p] = p < it.parts ? part[p][TM * (D + 1)] : 0.f;
  }
  const float m = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
  float l = 0.f, w[kJoinHeld];
#pragma unroll
  for (int p = 0; p < kJoinHeld; ++p) {
    w[p] = pl[p] != 0.f ? ex2(pm[p] - (m == -INFINITY ? 0.f : m)) : 0.f;
    l = __fmaf_rn(pl[p], w[p], l);
  }
  const int row = it.tile * TM + r, t = by_group(a, row), head = it.head * a.group + row - t * a.group;
  const int seen = keys_seen({it.first, it.count, it.len}, t);
  const float inv = inverse(l, seen);
  T* out = static_cast<T*>(a.out) + (it.first + t) * a.o_token + head * a.o_head;
  for (int col = slice * 4; col < D; col += slices * 4) {
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < kJoinHeld; ++p)
      if (p < it.parts)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = __fmaf_rn(part[p][(col + k) * TM], w[p], o[k]);
    uint2 v = make_uint2(0u, 0u);  // a row that sees nothing
    if (seen) v = make_uint2(Elem<T>::pack2(o[0] * inv, o[1] * inv), Elem<T>::pack2(o[2] * inv, o[3] * inv));
    *reinterpret_cast<uint2*>(out + col) = v;
  }
}

// Joins an item that was split: `cta` is where the item begins, the slices
// share its values.  A thread takes four columns of a row;
// up to eight of them share out the parts, so that a long row of parts (one
// token over a long cache) costs few dependent reads.  Parts are added in a fixed order.
template <class T, int TM, int D, bool Turned>
__device__ __forceinline__ void join_item(const AttendArgs& a, int cta, int slice, int slices, float (&sh)[kJoinThreads][6]) {
  const JoinItem it = a.joins[cta];
  if (it.parts == 0) return;
  if constexpr (Turned) {
    // Few parts of many rows (a chunk of 2048 tokens: 351 us this way, 360 the other;
    // 20 tokens over 30000 keys, 19 parts: 51 and 46).
    if (it.parts <= kJoinHeld) {
      join_rows<T, TM, D>(a, it, cta, slice, slices);
      return;
    }
  }
  int groups = 1;
  while (groups < kJoinGroups && groups * 2 <= it.parts) groups *= 2;
  const int width = kJoinThreads / groups, g = threadIdx.x / width;
  const int rows = min(TM, it.count * a.group - it.tile * TM), values = rows * (D / 4);
  for (int base = slice * width; base < values; base += slices * width) {
    const int e = base + threadIdx.x % width;
    const int r = Turned ? e % rows : e / (D / 4), col = (Turned ? e / rows : e % (D / 4)) * 4;
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    const auto add = [&](float pm, float pl, const float (&po)[4]) {
      if (pl == 0.f) return;  // a sum that is NaN counts
      const float mx = fmaxf(m, pm), f = ex2(m - mx), h = ex2(pm - mx);
      l = __fmaf_rn(l, f, pl * h);
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = __fmaf_rn(o[k], f, po[k] * h);
      m = mx;
    };
    if (e < values) {
      for (int p0 = g; p0 < it.parts; p0 += 4 * groups) {  // four parts' reads at a time
        float pm[4], pl[4], po[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int p = p0 + i * groups;
          pm[i] = -INFINITY, pl[i] = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) po[i][k] = 0.f;
          if (p < it.parts) {
            const float* src = partial<TM, D>(a, cta + p, p == 0);
            pm[i] = src[TM * D + r], pl[i] = src[TM * (D + 1) + r];
            if constexpr (Turned) {
#pragma unroll
              for (int k = 0; k < 4; ++k) po[i][k] = src[(col + k) * TM + r];
            } else {
              const float4 v = *reinterpret_cast<const float4*>(src + r * D + col);
              po[i][0] = v.x, po[i][1] = v.y, po[i][2] = v.z, po[i][3] = v.w;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) add(pm[i], pl[i], po[i]);
      }
    }
    if (groups > 1) {
      __syncthreads();
      float* mine = sh[threadIdx.x];
      mine[0] = m, mine[1] = l;
#pragma unroll
      for (int k = 0; k < 4; ++k) mine[2 + k] = o[k];
      __syncthreads();
      if (g == 0)
        for (int i = 1; i < groups; ++i) {
          const float* his = sh[threadIdx.x + i * width];
          const float po[4] = {his[2], his[3], his[4], his[5]};
          add(his[0], his[1], po);
        }
    }
    const int row = it.tile * TM + r, t = by_group(a, row);
    if (g == 0 && e < values) {
      const float inv = inverse(l, keys_seen({it.first, it.count, it.len}, t));
      const uint2 w = make_uint2(Elem<T>::pack2(o[0] * inv, o[1] * inv), Elem<T>::pack2(o[2] * inv, o[3] * inv));
      const int head = it.head * a.group + row - t * a.group;
      *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + (it.first + t) * a.o_token + head * a.o_head + col) = w;
    }
  }
}

template <class T, int TM, int D, bool Turned>
__global__ void __launch_bounds__(kJoinThreads) k_attend_join(AttendArgs a) {
  __shared__ float sh[kJoinThreads][6];
  pdl_launch_dependents();
  pdl_wait();
  join_item<T, TM, D, Turned>(a, blockIdx.x, blockIdx.y, gridDim.y, sh);
}

// Bytes of a launch's workspace: the join items, then two partials a CTA.
inline int64_t attend_workspace(int ctas, int tm, int dim) {
  return int64_t(ctas) * sizeof(JoinItem) + int64_t(2) * ctas * tm * (dim + 2) * 4;
}
inline void place_workspace(AttendArgs& a, void* workspace) {
  a.joins = static_cast<JoinItem*>(workspace);
  a.part = reinterpret_cast<float*>(a.joins + a.ctas);
}

// attend_tc.cu: the kernel for many rows, its workspace in bytes.
// Split items are joined by it, or (`joined` given and its CTAs not 0) by the caller, with those arguments.
constexpr int kTcRows = 256, kTcJoinSlices = 16;  // rows of an item; CTAs that join it
int64_t attend_tc_workspace(int dim);
// With `factors` keys and values are a copy from a q8_0 cache (cache8.cu): f16, divided by them, and in
// two parts where q is f16 (a.kv.pages: of one part).
int launch_attend_tc(const AttendArgs& a, void* workspace, bool bf16, int dim, cudaStream_t s, bool& ran, AttendArgs* joined,
                     const float* factors = nullptr);

// The joins of a call that ran both kernels, in one launch; `few` has tiles of TM rows.
struct JoinBoth {
  AttendArgs many, few;
};
template <class T, int TM, int D>
__global__ void __launch_bounds__(kJoinThreads) k_attend_join_both(const __grid_constant__ JoinBoth a) {
  __shared__ float sh[kJoinThreads][6];
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x, first = a.many.ctas * kTcJoinSlices;
  if (b < first)
    join_item<T, kTcRows, D, true>(a.many, b / kTcJoinSlices, b % kTcJoinSlices, kTcJoinSlices, sh);
  else
    join_item<T, TM, D, false>(a.few, (b - first) / kJoinSlices, (b - first) % kJoinSlices, kJoinSlices, sh);
}

}  // namespace q1
