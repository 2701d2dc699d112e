// attend.cuh -- what the two paged attention kernels share: their arguments,
// the split of the work into items and units, and the join of split items.
#pragma once

#include "paged.cuh"

namespace q1 {

struct AttendArgs {
  Paged kv;
  const void* q;           // [total_new][heads][dim], strides below
  void* out;
  int64_t q_token, q_head, o_token, o_head;  // elements
  float* part;             // partial results: [2 * CTAs][rows of a tile][dim + 2]
  unsigned* status;
  int heads, group;        // query heads, and of one key head
  float scale_log2;        // scale * log2(e)
  int ctas;                // CTAs the units are split over
};

__device__ __forceinline__ float ex2(float x) {  // 2^x, 0 at -inf
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The work.  Rows of (sequence b, key head h) are its new tokens times the
// group's heads, token-major; a tile is TM of them, an item a tile with all
// keys it may see, cut into units of TK keys (one unit at least).  Items lie on one axis,
// sequences first, then key heads, then tiles, and CTA c of N takes units
// [U c / N, U (c + 1) / N) of it: equal shares of keys whatever the lengths
// are.  An item that no CTA has to itself is joined by k_attend_join.
template <int TM, int TK>
struct Tiling {
  __device__ static int tiles(const SeqSpan& s, int group) { return (s.count * group + TM - 1) / TM; }
  // Keys that tile m of s may see: those of its last row.
  __device__ static int keys(const SeqSpan& s, int group, int m) {
    const int last = min(s.count - 1, (m * TM + TM - 1) / group);
    return max(0, s.len - s.count + last + 1);
  }
  __device__ static int units(const SeqSpan& s, int group, int m) { return max(1, (keys(s, group, m) + TK - 1) / TK); }
  __device__ static int64_t seq_units(const SeqSpan& s, int group) {  // of one key head
    int64_t u = 0;
    for (int m = 0, n = tiles(s, group); m < n; ++m) u += units(s, group, m);
    return u;
  }
};

// Position on the axis: an item and the unit within it.
struct Cursor {
  int b, h, m;      // sequence, key head, tile
  int unit, units;  // of this item
  SeqSpan s;
};

// Total units of the call, the number n of CTAs that have a share (n as given
// or the units, if fewer), CTA c's share [u0, u1) and the cursor at its start.
// Every thread of the CTA calls; `scratch` is 34 int64 in shared memory.
template <class Tile>
__device__ __forceinline__ int64_t locate(const AttendArgs& a, int c, int& n, int64_t* scratch, Cursor& cur, int64_t& u0,
                                          int64_t& u1) {
  const int threads = blockDim.x, warps = threads / 32, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // Each thread takes a run of consecutive sequences.
  const int per = (a.kv.batch + threads - 1) / threads;
  const int b0 = min(a.kv.batch, int(threadIdx.x) * per), b1 = min(a.kv.batch, b0 + per);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) {
    mine += Tile::seq_units(seq_span(a.kv, b), a.group) * a.kv.kv_heads;
    if (a.kv.kv_len[b] < 0 || a.kv.kv_len[b] > a.kv.table_tokens || a.kv.new_start[b] < 0 ||
        a.kv.new_start[b + 1] < a.kv.new_start[b] || a.kv.new_start[b + 1] > a.kv.total_new)
      atomicOr(a.status, kStatusBadIndex);
  }
  int64_t incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += t;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < warps; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  if (n > total) n = int(total);  // so that no share between two others is empty
  u0 = c < n ? total * c / n : total;
  u1 = c < n ? total * (c + 1) / n : total;
  const int64_t lo = before + incl - mine;
  __syncthreads();
  if (u0 >= lo && u0 < lo + mine) {  // the run that holds u0: one thread's
    int64_t at = lo, su;
    int b = b0;
    SeqSpan s;
    for (;; ++b) {
      s = seq_span(a.kv, b);
      su = Tile::seq_units(s, a.group);
      if (u0 < at + su * a.kv.kv_heads || b + 1 >= b1) break;
      at += su * a.kv.kv_heads;
    }
    const int h = int((u0 - at) / su);
    int64_t left = (u0 - at) - h * su;
    int m = 0, un;
    for (;; ++m) {
      un = Tile::units(s, a.group, m);
      if (left < un || left < 0) break;
      left -= un;
    }
    scratch[0] = b, scratch[1] = h, scratch[2] = m, scratch[3] = left, scratch[4] = un;
  }
  __syncthreads();
  if (u0 < u1) {
    cur.b = int(scratch[0]), cur.h = int(scratch[1]), cur.m = int(scratch[2]);
    cur.unit = int(scratch[3]), cur.units = int(scratch[4]);
    cur.s = seq_span(a.kv, cur.b);
  }
  __syncthreads();
  return total;
}

// The item after cur's (there is one).
template <class Tile>
__device__ __forceinline__ void next_item(const AttendArgs& a, Cursor& cur) {
  cur.unit = 0;
  if (++cur.m >= Tile::tiles(cur.s, a.group)) {
    cur.m = 0;
    if (++cur.h >= a.kv.kv_heads) {
      cur.h = 0;
      do cur.s = seq_span(a.kv, ++cur.b);
      while (cur.s.count == 0 && cur.b + 1 < a.kv.batch);
    }
  }
  cur.units = Tile::units(cur.s, a.group, cur.m);
}

// Row r of a tile: its token and query head; false past the last row.
__device__ __forceinline__ bool row_of(const Cursor& cur, int group, int r, int& token, int& head) {
  const int t = r / group;
  token = cur.s.first + t;
  head = cur.h * group + r - t * group;
  return t < cur.s.count;
}

// Joins the items that were split over several CTAs.  CTA c of the launch
// takes the item whose first unit is CTA c's and whose last is not: its
// partials lie in slot 1 of CTA c and slot 0 of the CTAs after it (a CTA's
// first item, when it began before, is in slot 0).  A partial is, per row,
// dim sums of p v relative to the row's maximum, then the maximum (in log2
// units) and the sum of p.  Parts are added in order.
// Partials lie row by row, or (Turned) column by column, rows side by side.
template <class T, int TM, int TK, int D, bool Turned>
__global__ void __launch_bounds__(256) k_attend_join(AttendArgs a) {
  using Tile = Tiling<TM, TK>;
  __shared__ int64_t scratch[34];
  pdl_launch_dependents();
  pdl_wait();
  Cursor cur = {};
  int64_t u0, u1;
  const int c = blockIdx.x;
  int ctas = a.ctas;
  const int64_t total = locate<Tile>(a, c, ctas, scratch, cur, u0, u1);
  if (u0 >= u1) return;
  // The last item of CTA c.
  int64_t at = u0 - cur.unit;
  while (at + cur.units < u1) {
    at += cur.units;
    next_item<Tile>(a, cur);
  }
  const int64_t end = at + cur.units;
  if (end == u1 || at < u0) return;  // not split after c, or begun before c
  int parts = 1;
  while (total * (c + parts) / ctas < end) ++parts;
  constexpr int kRow = D + 2, kLanes = D / 4;  // a thread takes four columns of a row
  const int rows = min(TM, cur.s.count * a.group - cur.m * TM);
  for (int i = threadIdx.x; i < rows * kLanes; i += 256) {
    const int r = Turned ? i % rows : i / kLanes, col = (Turned ? i / rows : i % kLanes) * 4;
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int p = 0; p < parts; ++p) {
      const float* row = a.part + int64_t(2 * (c + p) + (p == 0)) * TM * kRow + (Turned ? r : r * kRow);
      constexpr int kNext = Turned ? TM : 1;  // from one column to the next
      const float pm = row[D * kNext], pl = row[(D + 1) * kNext];
      const float mx = fmaxf(m, pm);
      if (pl != 0.f) {  // a sum that is NaN counts
        const float f = ex2(m - mx), g = ex2(pm - mx);
        l = __fmaf_rn(l, f, pl * g);
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = __fmaf_rn(o[k], f, row[(col + k) * kNext] * g);
        m = mx;
      }
    }
    int token, head;
    if (!row_of(cur, a.group, cur.m * TM + r, token, head)) continue;
    const float inv = l > 0.f ? __fdiv_rn(1.0f, l) : 0.f;
    uint2 w = make_uint2(Elem<T>::pack2(o[0] * inv, o[1] * inv), Elem<T>::pack2(o[2] * inv, o[3] * inv));
    *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + token * a.o_token + head * a.o_head + col) = w;
  }
}

// attend_tc.cu: the kernel for many rows, its workspace in bytes.
int64_t attend_tc_workspace(int dim);
int launch_attend_tc(const AttendArgs& a, bool bf16, int dim, cudaStream_t s, bool& ran);

}  // namespace q1
