// attend_tc.cu -- q1_paged_attention for many rows a key head: the tensor-core
// kernel.
//
// The same formula as attend.cu, 4 D operations a (row, key) pair: from some
// tens of rows on these bound it, so both products run on tcgen05 MMAs of 128
// rows x 128 keys and the softmax between them on sixteen warps.
//
// An item is 256 rows (two tiles of 128) of one key head; a row is a new token
// and one of the group's heads, so grouped heads share each key and value
// tile.  Roles of the CTA's warps:
//   warps 0-7, 8-15 softmax of tile 0 and 1; warps q and q + 4 of a tile share rows
//                   32q..32q+31 (tensor-memory lanes), one thread a row, the
//                   first with keys 0-63 of a unit and the second with 64-127:
//                   maximum, p = 2^(s - m), P back to tensor memory over its
//                   own part of S, the output at an item's end.  They also
//                   copy the rows of Q into shared memory.
//   warps 16, 18    issue the MMAs of tile 0 and 1: O_w += P_w V and the next
//                   S_w = Q_w K^T, in turns, so that one tile's softmax runs
//                   under the other's products.  (Left to themselves the tiles
//                   fall into step and the tensor core waits for both
//                   softmaxes; with one warp for both, its waits, 150 cycles
//                   each, lie bare.)
//   warp 17         TMA: one box a page and 64 dims, keys and values through one ring
//                   of 128-key stages (128-byte swizzle; V is read as the
//                   MN-major operand, so nothing is transposed).
// A unit's weights are taken relative to the maximum in use before it, and its
// own maximum, exchanged between a row's two threads meanwhile, is looked at
// before P is stored: it rarely has grown by 2^8, and then they are taken again.
// Tensor memory: S_0, S_1 (128 columns each, P in columns 0-31 and 64-95), O_0, O_1.
// MMAs of one thread execute in order, so S_w of the next tile may be issued
// behind the product that reads P_w, and S_w's completion implies that O_w holds
// still: the softmax warps rescale O_w themselves, and only when a row's maximum
// has grown by more than 2^8 (weights are then at most 2^8 relative to the
// maximum in use, which f32 sums and both 16-bit types hold).
//
// Where V of a unit is looked at (only where not all rows see all of its keys): by
// the issuing warps, which wait for P then.  2 % of a mixed batch; by the softmax
// warps 12 %, by a warp of its own 5 % (and 3 % of a long chunk: the kernel's
// registers come out worse).
//
// Measured (32 heads over 8 of 128, bf16): 2048 new tokens over 16001 keys, 0.503
// Tflop, in 351 us with the join: 1.43 Pflop/s, 0.73 of this card's matrix product
// rate (1.95); the tensor pipe is active 63 % of the cycles (profiled launch, 345 us).
// What is left: with D = 128 the two tiles fill tensor memory, so a tile's scores,
// softmax and product with V follow each other, and two tiles hide each other's only in
// part.  With D = 64 the softmax bounds it: its arithmetic alone takes 346 cycles a
// warp and 64 keys (exponentials 256 of them), four warps a scheduler.
//
// Keys and values that were copied from a q8_0 cache (cache8.cu) are f16 for q of
// either type, since bf16 would add 2^-9 of every key's value to the weights' own rounding:
// divided by a power of two a sequence and key head (kNormed), which the scale of
// the scores and the output take back, as rows of bf16 q are by one each (kept in
// shared memory from when they are loaded).  With f16 q they come in two parts, value
// and remainder, twice the products.
//
// Every wait is bounded; one that gives up raises the CTA's abort flag and the
// device status word, and every role winds down.
#include <cuda.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "attend.cuh"
#include "tc.cuh"

namespace q1 {

constexpr int kTcM = 128;            // rows of a tile
constexpr int kTcItem = 2 * kTcM;    // rows of an item
static_assert(kTcItem == kTcRows, "");
constexpr int kTcKeys = 128;         // keys of a unit
constexpr int kTcSoftWarps = 16;     // softmax warps: two a 32-row quarter of a tile
constexpr int kTcAThreads = (kTcSoftWarps + 4) * 32;
// Registers a thread: 96 at launch, then 64 for the last warpgroup and 104 for
// the four with the softmax, the same total.
constexpr int kTcRegsLess = 64, kTcRegsMore = 104;
static_assert(128 * kTcRegsLess + 32 * kTcSoftWarps * kTcRegsMore <= kTcAThreads * 96, "the block's registers at launch");
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
// Units of an item that is not split (a mixed batch: 66.4 us with 8, 71.4 with 4,
// 66.7 with 12; 16 sequences of up to 72 tokens: 36.8, 36.9, 43.5).
constexpr int kTcWhole = 8;
constexpr float kTcGrow = 8.f;       // log2 units a maximum may be behind

struct AttendTcArgs {
  AttendArgs a;
  CUtensorMap k, v;   // boxes of 64 dims x box_keys slots
  uint32_t q_sign;    // 0x80008000 where the scale is negative: -q and |scale| instead
  int box_keys;
  int axis_head, axis_slot, axis_page;  // positions (1..3) of the axes in the maps
  const float* factors;  // kNormed: what keys and values of [sequence][key head] were divided by
};

template <int D>
struct TcShape {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kTcKeys * D * 2;       // of K, V or a tile of Q
  static constexpr int kHalfBytes = kTcKeys * 128;         // 64 dims of it
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kOffKV = 2 * kTileBytes;
  static constexpr int kOffBars = kOffKV + kStages * kTileBytes;
  static constexpr int kNumBars = 2 * kStages + 18;
  static constexpr int kSmem = kOffBars + kNumBars * 8 + 16 + 1024;  // + alignment
  static_assert(kSmem <= 227 * 1024 && kSmem > 114 * 1024, "one CTA an SM: it takes all of tensor memory");
};

// K-major operand tile, 128-byte swizzle: 8-row groups of 1024 bytes.
__device__ __forceinline__ uint64_t desc_k_sw128(uint32_t saddr) {
  return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}
// MN-major operand tile, 128-byte swizzle: 8 rows of K are 1024 bytes, 64
// columns further on is `chunk` bytes.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t chunk) {
  return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t((chunk >> 4) & 0x3FFFu) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
template <class T>
__host__ __device__ constexpr uint32_t idesc_attend(int N, bool b_mn_major) {
  const uint32_t f = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | (b_mn_major ? 1u << 16 : 0u) | (uint32_t(N >> 3) << 17) |
         (uint32_t(kTcM >> 4) << 24);
}
// D[tmem] (+)= A[smem] x B[smem], issued by one elected lane of a converged warp.
__device__ __forceinline__ void mma_f16_ss_elect(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                 uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p, e;\nsetp.ne.b32 p, %4, 0;\nelect.sync _|e, 0xffffffff;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void tmem_st32(uint32_t t, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3,%4,%5,%6}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ uint64_t f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A ring position: stage and parity of its current pass.
struct RingPos {
  int stage = 0;
  uint32_t parity = 0;
  template <int N>
  __device__ __forceinline__ void next() {
    if (++stage == N) stage = 0, parity ^= 1;
  }
};

// T: the products' type; U: that of q and the output; kParts: of each key and
// value, the second one's pages behind the first one's.
template <class T, int D, class U = T, int kParts = 1>
__global__ void __launch_bounds__(kTcAThreads, 1) k_attend_tc(const __grid_constant__ AttendTcArgs g) {
  using Tile = Tiling<kTcItem, kTcKeys>;
  using Shape = TcShape<D>;
  constexpr int kStages = Shape::kStages;
  constexpr bool kTurned = !std::is_same<T, U>::value, kNormed = kTurned || kParts > 1;  // kTurned: q is made another type
  const AttendArgs& a = g.a;
  extern __shared__ unsigned char raw_smem[];
  __shared__ LocateScratch scratch;
  __shared__ float exchange[2][2][2][kTcM];  // [unit parity][tile][half][row]
  __shared__ float q_factor[kTurned ? 2 : 1][2][kTurned ? kTcM : 1];  // [item parity][tile][row]
  __shared__ uint32_t tmem_base_s;
  __shared__ volatile uint32_t abort_s, taken_out_s;  // taken_out_s: V had values that are no numbers
  unsigned char* smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
  const uint32_t s0 = smem_addr(smem);
  const uint32_t bars = s0 + Shape::kOffBars;
  const auto full = [&](int s) { return bars + s * 8; };
  const auto empty = [&](int s) { return bars + (kStages + s) * 8; };
  // Two of each (one a tile); pair: one for each two warps that share rows.
  const uint32_t qfull = bars + 2 * kStages * 8, sfull = qfull + 16, ofull = qfull + 32, turn = qfull + 48,
                 pfull = qfull + 64, pair = qfull + 80;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(full(s), 1), mbar_init(empty(s), 2);
    for (int w = 0; w < 2; ++w) {
      mbar_init(qfull + 8 * w, 2 * kTcM);
      mbar_init(sfull + 8 * w, 1);
      mbar_init(pfull + 8 * w, 2 * kTcM);
      mbar_init(ofull + 8 * w, 1);
      mbar_init(turn + 8 * w, 1);
    }
    for (int i = 0; i < 8; ++i) mbar_init(pair + 8 * i, 2);
    fence_barrier_init();
    abort_s = taken_out_s = 0;
  }
  if (warp == kTcSoftWarps) tmem_alloc(smem_addr(&tmem_base_s), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;
  // In this order: the next launch may go on without waiting for this one (`beside`), and
  // then relies on what was before it.
  pdl_wait();
  pdl_launch_dependents();

  Cursor cur = {};
  int64_t u0, u1;
  int ctas = a.ctas;
  const int64_t total = locate<Tile, kTcWhole>(a, blockIdx.x, ctas, scratch, cur, u0, u1);
  if (threadIdx.x == 0) a.joins[blockIdx.x].parts = 0;

  // Whole warps wait, and agree on whether they may go on.  (Written out here:
  // a call in the loops would keep the register split from taking effect.)
  const auto wait = [&](uint32_t bar, uint32_t parity) {
    bool done = mbar_try(bar, parity);
    if (!done && !abort_s) {
      const uint64_t t0 = globaltimer();
      for (uint32_t i = 1; !(done = mbar_try(bar, parity)); ++i)
        if ((i & 63) == 0 && (abort_s || globaltimer() - t0 > 1000000000ull)) break;
      if (!done) {
        abort_s = 1;
        atomicOr(a.status, kStatusWaitTimeout);
      }
    }
    return bool(__all_sync(0xffffffffu, done));
  };
  // Units of the current item that this CTA takes, and whether it has two tiles.
  const auto part_of = [&](int64_t u) { return int(min(int64_t(cur.units - cur.unit), u1 - u)); };
  const auto tiles_of = [&](const Cursor& it) { return it.s.count * a.group - it.m * kTcItem > kTcM ? 2 : 1; };

  if (warp >= kTcSoftWarps) {
    regs_down<kTcRegsLess>();
    if (warp == kTcSoftWarps + 1) {
      // ------------------------------------------------------------- TMA --
      RingPos pos;
      const int boxes_max = kTcKeys / g.box_keys, page_mask = (1 << a.kv.page_shift) - 1;
      bool ok = true;
      for (int64_t u = u0; u < u1 && ok;) {
        const int take = part_of(u), keys = Tile::keys(a, cur.s, cur.m);
        const int32_t* table = a.kv.table + cur.b * a.kv.table_stride;
        // The page of this lane's box, one unit ahead.
        const auto page_at = [&](int unit) {
          const int j = unit * kTcKeys + lane * g.box_keys;
          return lane < boxes_max && j < keys ? table[j >> a.kv.page_shift] : 0;
        };
        int page = keys ? page_at(cur.unit) : 0;
        for (int t = 0; t < take && keys && ok; ++t) {
          const int unit = cur.unit + t, j = unit * kTcKeys + lane * g.box_keys;
          const int boxes = min(boxes_max, (keys - unit * kTcKeys + g.box_keys - 1) / g.box_keys);
          const int next = t + 1 < take ? page_at(unit + 1) : 0;
          if (lane < boxes && (page < 0 || page >= a.kv.pages)) {
            atomicOr(a.status, kStatusBadIndex);
            page = kParts * a.kv.pages;  // past the map's end: the box reads as zeros
          }
          int c[3];
#pragma unroll
          for (int i = 0; i < 3; ++i)
            c[i] = g.axis_head == i + 1 ? cur.h : g.axis_slot == i + 1 ? (j & page_mask) : page;
#pragma unroll
          for (int kv = 0; kv < 2 * kParts; ++kv) {
            if constexpr (kParts > 1) {
              const int step = kv == 0 ? 0 : kv % 2 ? a.kv.pages : -a.kv.pages;  // to the second part, and back
#pragma unroll
              for (int i = 0; i < 3; ++i) c[i] += g.axis_page == i + 1 ? step : 0;
            }
            if (!wait(empty(pos.stage), pos.parity ^ 1)) {
              ok = false;
              break;
            }
            if (lane == 0) mbar_arrive_expect_tx(full(pos.stage), uint32_t(boxes) * g.box_keys * D * 2);
            __syncwarp();
            if (lane < boxes) {
              const uint32_t dst = s0 + Shape::kOffKV + pos.stage * Shape::kTileBytes + lane * g.box_keys * 128;
#pragma unroll
              for (int h = 0; h < Shape::kHalves; ++h)
                tma_box(dst + h * Shape::kHalfBytes, kv / kParts ? &g.v : &g.k, full(pos.stage), h * 64, c[0], c[1], c[2]);
            }
            __syncwarp();
            pos.next<kStages>();
          }
          page = next;
        }
        u += take;
        if (u < u1) next_item<Tile>(a, cur);
      }
    } else if (warp != kTcSoftWarps + 3) {
      // ------------------------------------------------------------- MMA --
      // With D = 64 the products are short beside the softmax, and turns only
      // cost (10 sequences of up to 585 tokens: 77.3 us without, 79.6 with them).
      constexpr bool kTurns = D == 128;
      constexpr uint32_t kIdS = idesc_attend<T>(kTcKeys, false), kIdO = idesc_attend<T>(D, true);
      const int w = (warp - kTcSoftWarps) >> 1;  // tile
      RingPos pos;                    // of the next K or V tile
      uint32_t qpar = 0, ppar = 0, turnpar = 0;
      bool ok = true, handed = false;
      const uint32_t ts = tmem + w * 128, to = tmem + 256 + w * D;
      const uint64_t qdesc = desc_k_sw128(s0 + w * Shape::kTileBytes);
      const auto tile_addr = [&](int stage) { return s0 + Shape::kOffKV + stage * Shape::kTileBytes; };
      const auto hand_on = [&](bool hand) {
        if (kTurns && hand && lane == 0) mbar_arrive(turn + 8 * (w ^ 1));
        __syncwarp();
      };
      const auto scores = [&](bool hand) {  // S_w = Q_w K^T, of the parts from pos on
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          const int stage = pos.stage;
          const uint64_t kdesc = desc_k_sw128(tile_addr(stage));
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            constexpr int kHalf = Shape::kHalfBytes;
            const int off = ((k / 4) * kHalf + (k % 4) * 32) >> 4;
            mma_f16_ss_elect(ts, qdesc + off, kdesc + off, kIdS, k > 0 || part > 0);
          }
          if (part == kParts - 1) mma_commit_elect(sfull + 8 * w);
          mma_commit_elect(empty(stage));
          pos.next<kStages>();
        }
        hand_on(hand);
      };
      const auto parts_full = [&]() {  // from pos on
        bool done = wait(full(pos.stage), pos.parity);
        if constexpr (kParts > 1) {
          RingPos at = pos;
          at.next<kStages>();
          done = done && wait(full(at.stage), at.parity);
        }
        return done;
      };
      for (int64_t u = u0; u < u1 && ok;) {
        const int take = part_of(u), keys = Tile::keys(a, cur.s, cur.m), nw = tiles_of(cur);
        const int of_all = Tile::keys_of_all(a, cur.s, cur.m);
        if (keys && w >= nw) {
          // No rows for this tile: its share of releasing the stages.
          for (int t = 0; t < 2 * kParts * take && ok; ++t) {
            ok = wait(full(pos.stage), pos.parity);
            if (ok && lane == 0) mbar_arrive(empty(pos.stage));
            pos.next<kStages>();
          }
        } else if (keys) {
          // This warp's turn: after the other tile's batch before, if there was one
          // (of this item or of the last one with two tiles: neither warp may be
          // two batches ahead, its barrier would pass two phases).
          const auto my_turn = [&]() {
            if (!kTurns || nw == 1 || (w == 0 && !handed)) return true;
            const bool done = wait(turn + 8 * w, turnpar);
            turnpar ^= 1;
            return done;
          };
          ok = wait(qfull + 8 * w, qpar) && parts_full() && my_turn();
          qpar ^= 1;
          handed |= nw == 2;
          if (ok) {
            tc_fence_after();
            scores(nw == 2);
          }
          for (int t = 0; t < take && ok; ++t) {
            int vstages[kParts];
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
              const int vstage = vstages[part] = pos.stage;
              // (No way out of the loop here: 2048 bf16 tokens over 16001 keys of a 16-bit cache take 359.5 us, 362.9 with one.)
              ok = (part == 0 || ok) && wait(full(vstage), pos.parity);
              // V is made ready while the softmax is under way.  (Both tiles' warps look at all of it
              // and may write the same zeros.)
              const int unit0 = (cur.unit + t) * kTcKeys, valid = keys - unit0;
              if (ok && (valid < kTcKeys || of_all < unit0 + kTcKeys)) {
                uint4* v = reinterpret_cast<uint4*>(smem + Shape::kOffKV + vstage * Shape::kTileBytes);
                constexpr int kHalf = Shape::kHalfBytes / 16;
                // Values that are no numbers, of keys that not all rows of the item see, are taken
                // out; the output adds them to the rows that see them.
                const int lo = max(0, of_all - unit0) * 8 + lane, hi = min(valid, kTcKeys) * 8;
                NoNumbers<T> none;
#pragma unroll 1
                for (int i = lo - lane; i < hi; i += 128) {  // (loads side by side: 22.8 us for two prompts of 400, 23.5 without)
                  uint4 x[4][Shape::kHalves];
#pragma unroll
                  for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int h = 0; h < Shape::kHalves; ++h) x[e][h] = v[h * kHalf + min(i + e * 32 + lane, hi - 1)];
#pragma unroll
                  for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int h = 0; h < Shape::kHalves; ++h) none.look(x[e][h]);
                }
                if (__any_sync(0xffffffffu, none.found())) {
                  taken_out_s = 1;
                  __threadfence_block();  // whoever finds them gone finds this
#pragma unroll 1
                  for (int i = lo; i < hi; i += 32)
                    for (int h = 0; h < Shape::kHalves; ++h) v[h * kHalf + i] = numbers<T>(v[h * kHalf + i]);
                }
                // Rows past the keys hold whatever lay there: a weight of zero times that must be zero.
                for (int i = valid * 8 + lane; i < kTcKeys * 8; i += 32)
#pragma unroll
                  for (int h = 0; h < Shape::kHalves; ++h) v[h * kHalf + i] = make_uint4(0u, 0u, 0u, 0u);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
              }
              pos.next<kStages>();
            }
            if (!ok) break;
            const bool more = t + 1 < take;
            if (more) ok = parts_full();
            ok = ok && my_turn() && wait(pfull + 8 * w, ppar);
            ppar ^= 1;
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
              const uint64_t vdesc = desc_mn_sw128(tile_addr(vstages[part]), Shape::kHalfBytes);
#pragma unroll
              for (int k = 0; k < 8; ++k)
                mma_f16_ts_elect(to, ts + k / 4 * 64 + k % 4 * 8, vdesc + k * (2048 >> 4), kIdO, t > 0 || k > 0 || part > 0);
              mma_commit_elect(empty(vstages[part]));
            }
            if (more) {
              scores(nw == 2);
            } else {
              mma_commit_elect(ofull + 8 * w);
              hand_on(nw == 2);
            }
          }
        }
        u += take;
        if (u < u1) next_item<Tile>(a, cur);
      }
    }
  } else {
    // --------------------------------------------------------- softmax --
    regs_up<kTcRegsMore>();
    const int w = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;  // tile, keys, rows
    const int row = quarter * 32 + lane;
    const uint32_t lanes = uint32_t(quarter) * 32 << 16;
    constexpr int kCols = D / 2;  // columns of O that this warp rescales and writes
    const uint32_t ts = tmem + lanes + w * 128 + half * 64, to = tmem + lanes + 256 + w * D + half * kCols;
    const uint32_t pair_bar = pair + 8 * (w * 4 + quarter);
    uint32_t spar = 0, opar = 0, xpar = 0;
    // The value of the thread that shares the row (of the exchange whose parity is xpar).
    const auto post = [&](float v) {
      exchange[xpar][w][half][row] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(pair_bar);
    };
    const auto fetch = [&](float& v) {
      const bool done = wait(pair_bar, xpar);
      v = exchange[xpar][w][half ^ 1][row];
      xpar ^= 1;
      return done;
    };
    bool ok = true;
    uint64_t scale2 = f32x2(a.scale_log2, a.scale_log2);
    uint32_t q_parity = 0;  // of the item whose Q is loaded (bit 0), and of the one at work (bit 1)
    const auto scale_of = [&]() {  // of this item's scores
      float x = a.scale_log2, y;
      if constexpr (kNormed) split2(scale2, x, y);
      return x;
    };
    const auto factors_of = [&](const Cursor& it) { return g.factors + 2 * (it.b * a.kv.kv_heads + it.h); };
    // Q of an item, if this tile has rows of it that see keys: this warp's 16
    // rows, 16 (8) lanes a row; rows past the last are zero.
    const auto load_q = [&](const Cursor& it) {
      if (w >= tiles_of(it) || Tile::keys(a, it.s, it.m) == 0) return;
      constexpr int kLanes = D / 8, kOnce = 32 / kLanes;
      const int piece = lane % kLanes;
      unsigned char* q = smem + w * Shape::kTileBytes + (piece / 8) * Shape::kHalfBytes;
#pragma unroll
      for (int r0 = 0; r0 < 16; r0 += kOnce) {
        const int r = (warp & 7) * 16 + r0 + lane / kLanes;
        int qt, qh;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (row_of(a, it, it.m * kTcItem + w * kTcM + r, qt, qh))
          v = *reinterpret_cast<const uint4*>(static_cast<const U*>(a.q) + qt * a.q_token + qh * a.q_head + piece * 8);
        v.x ^= g.q_sign, v.y ^= g.q_sign, v.z ^= g.q_sign, v.w ^= g.q_sign;
        if constexpr (kTurned) {
          // Divided by a power of two near the row's largest value, which f16's 11 bits
          // hold exactly down to 2^-14 of it.
          const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
          uint32_t top = max(m & 0xffffu, m >> 16);
#pragma unroll
          for (int off = 1; off < kLanes; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
          const uint32_t e = min(max(top >> 7, 1u), 253u);  // the exponent's bits
          float x[8];
          Elem<U>::unpack(v, x);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= __uint_as_float((254u - e) << 23);
          v = Elem<T>::pack(x);
          if (piece == 0) q_factor[q_parity & 1][w][r] = __uint_as_float(e << 23);
        }
        *reinterpret_cast<uint4*>(q + r * 128 + (((piece & 7) ^ (r & 7)) << 4)) = v;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(qfull + 8 * w);
      q_parity ^= 1;
    };
    if (u0 < u1) load_q(cur);
    for (int64_t u = u0; u < u1 && ok;) {
      const int take = part_of(u), keys = Tile::keys(a, cur.s, cur.m);
      Cursor next = cur;
      bool have_next = false;
      // The next item and its Q: its last reader here, the scores of this
      // item's last unit, is done, so they are under way during the output.
      const auto advance = [&]() {
        have_next = u + take < u1;
        if (have_next) {
          next_item<Tile>(a, next);
          load_q(next);
        }
      };
      if (w < tiles_of(cur)) {
        const int row0 = cur.m * kTcItem + w * kTcM;
        int token, head;
        const bool live = row_of(a, cur, row0 + row, token, head);
        // Keys of this half of the CTA's first unit that the row may see.
        int seen = (live ? cur.s.len - cur.s.count + (token - cur.s.first) + 1 : 0) - cur.unit * kTcKeys - half * 64;
        float used = -INFINITY, sum = 0.f;  // the maximum that weights are relative to
        if (keys) {
          uint64_t sum2 = 0, base2 = 0;  // two partial sums; minus the maximum in use, twice
          for (int t = 0; t < take; ++t) {
            ok = wait(sfull + 8 * w, spar);
            spar ^= 1;
            if (!ok) break;
            tc_fence_after();
            if constexpr (kNormed) {
              if (t == 0) {  // (the row's factor was written before its Q, which these scores come from)
                float scale = a.scale_log2 * factors_of(cur)[0];
                if constexpr (kTurned) scale *= q_factor[q_parity >> 1][w][row];
                q_parity ^= 2;
                scale = fminf(fmaxf(scale, FLT_MIN), FLT_MAX);
                scale2 = f32x2(scale, scale);
              }
            }
            uint32_t p[32];
            const auto scores = [&](uint32_t (&s)[2][32]) {
              tmem_ld32(ts, s[0]);
              tmem_ld32(ts + 32, s[1]);
              tmem_wait_ld32(s[0]);
              tmem_wait_ld32(s[1]);
              if (__any_sync(0xffffffffu, seen < 64)) {
#pragma unroll
                for (int i = 0; i < 64; ++i) s[i / 32][i % 32] = i < seen ? s[i / 32][i % 32] : 0xff800000u;
              }
            };
            const auto weights = [&](uint32_t (&s)[2][32]) {  // p, and their sums
              uint64_t sum_a = 0, sum_b = 0;
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const uint32_t(&v)[32] = s[j / 16];
                float x, y;
                split2(fma2(f32x2(__uint_as_float(v[j % 16 * 2]), __uint_as_float(v[j % 16 * 2 + 1])), scale2, base2), x, y);
                x = ex2(x), y = ex2(y);
                (j & 1 ? sum_b : sum_a) = add2(j & 1 ? sum_b : sum_a, f32x2(x, y));
                p[j] = Elem<T>::pack2(x, y);
              }
              return add2(sum_a, sum_b);
            };
            uint64_t part;
            float mine, other;
            {
              uint32_t s[2][32];
              scores(s);
              float m[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t(&v)[32] = s[i / 2];
                const int j0 = i % 2 * 16;
                m[i] = fmaxf(__uint_as_float(v[j0]), __uint_as_float(v[j0 + 1]));
#pragma unroll
                for (int j = 2; j < 16; j += 2) m[i] = max3(m[i], __uint_as_float(v[j0 + j]), __uint_as_float(v[j0 + j + 1]));
              }
              mine = fmaxf(max3(m[0], m[1], m[2]), m[3]);
              part = weights(s);
              post(mine);
            }
            ok = fetch(other);
            if (!ok) break;
            const float top = fmaxf(mine, other) * scale_of();
            const bool grown = top > used + kTcGrow || (used == -INFINITY && top > -INFINITY);
            if (__any_sync(0xffffffffu, grown)) {
              float f = 1.f;
              if (grown) {
                f = ex2(used - top);
                used = top;
                base2 = f32x2(-used, -used);
                sum2 = mul2(sum2, f32x2(f, f));
              }
              if (t > 0) {
#pragma unroll
                for (int c = 0; c < kCols; c += 16) {
                  uint32_t o[16];
                  tmem_ld16(to + c, o);
                  tmem_wait_ld16(o);
#pragma unroll
                  for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                  tmem_st16(to + c, o);
                }
              }
              uint32_t s[2][32];
              scores(s);
              part = weights(s);
            }
            tmem_st32(ts, p);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(pfull + 8 * w);
            sum2 = add2(sum2, part);
            seen -= kTcKeys;
          }
          if (!ok) break;
          advance();
          float sa, sb, other;
          split2(sum2, sa, sb);
          sa += sb;
          post(sa);
          ok = fetch(other) && wait(ofull + 8 * w, opar);
          opar ^= 1;
          if (!ok) break;
          sum = sa + other;
          tc_fence_after();
        } else {
          advance();
        }
        const bool whole = cur.unit == 0 && take == cur.units;
        const int sees = live ? keys_seen(cur.s, token - cur.s.first) : 0;
        const float v_factor = kNormed ? factors_of(cur)[1] : 1.f;
        const float inv = kNormed ? inverse(sum, sees) * v_factor : inverse(sum, sees);
        if (threadIdx.x == 0 && cur.unit == 0 && !whole) leave_join(a, cur, u, total, ctas);
        float* part = partial<kTcItem, D>(a, blockIdx.x, cur.unit == 0) + w * kTcM + row;
        U* out = static_cast<U*>(a.out) + (live ? token * a.o_token + head * a.o_head : 0) + half * kCols;
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          uint32_t o[16];
          if (keys) {
            tmem_ld16(to + c, o);
            tmem_wait_ld16(o);
          }
          if (whole) {
            if (live) {
#pragma unroll
              for (int j = 0; j < 16; j += 8) {
                uint32_t pk[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)  // a row that sees nothing is zero, whatever O holds
                  pk[e] = sees ? Elem<U>::pack2(__uint_as_float(o[j + 2 * e]) * inv, __uint_as_float(o[j + 2 * e + 1]) * inv)
                                     : 0u;
                *reinterpret_cast<uint4*>(out + c + j) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              part[(half * kCols + c + j) * kTcItem] = kNormed ? __uint_as_float(o[j]) * v_factor : __uint_as_float(o[j]);
          }
        }
        if (taken_out_s) {  // (rolled, on what has been written: the loops above have no registers for it)
          const int j1 = min(sees, (cur.unit + take) * kTcKeys);
#pragma unroll 1
          for (int j = max(Tile::keys_of_all(a, cur.s, cur.m), cur.unit * kTcKeys); j < j1; ++j) {
            const int page = a.kv.table[cur.b * a.kv.table_stride + (j >> a.kv.page_shift)];
            if (page < 0 || page >= a.kv.pages) continue;
            const T* v = static_cast<const T*>(a.kv.v) + page * a.kv.page_stride +
                         (j & ((1 << a.kv.page_shift) - 1)) * a.kv.slot_stride + cur.h * a.kv.head_stride + half * kCols;
#pragma unroll 1
            for (int c = 0; c < kCols; ++c) {
              const float x = Elem<T>::to(v[c]);
              if (fabsf(x) <= FLT_MAX) continue;
              if (whole)
                out[c] = Elem<U>::from(Elem<U>::to(out[c]) + x);
              else
                part[(half * kCols + c) * kTcItem] += x;
            }
          }
        }
        if (!whole && half == 0) {
          part[D * kTcItem] = used;
          part[(D + 1) * kTcItem] = sum;
        }
        tc_fence_before();  // the next item's first product overwrites O after this thread's next arrival
      } else {
        advance();
      }
      u += take;
      cur = next;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (abort_s) {
    // Copies and products may still be under way: let them end first.
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000ull) {
    }
  }
  __syncthreads();
  if (warp == kTcSoftWarps) tmem_free(tmem, 512);
}

static CUresult encode_map(CUtensorMap* m, bool bf16, const Paged& p, int parts, void* base, int dim, int box_keys, int (&axis)[3]) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static Encode fn = nullptr;
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess || !f) {
      (void)cudaGetLastError();
      return CUDA_ERROR_NOT_SUPPORTED;
    }
    fn = reinterpret_cast<Encode>(f);
  }
  // The axes head, slot, page in the order of their strides.
  const int64_t stride[3] = {p.head_stride, p.slot_stride, p.page_stride};
  const uint64_t size[3] = {uint64_t(p.kv_heads), uint64_t(1) << p.page_shift, uint64_t(p.pages) * uint64_t(parts)};
  int order[3] = {0, 1, 2};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (stride[order[j]] > stride[order[j + 1]]) {
        const int t = order[j];
        order[j] = order[j + 1], order[j + 1] = t;
      }
  cuuint64_t dims[4] = {cuuint64_t(dim)}, strides[3];
  cuuint32_t box[4] = {64}, ones[4] = {1, 1, 1, 1};
  for (int i = 0; i < 3; ++i) {
    dims[i + 1] = size[order[i]];
    strides[i] = cuuint64_t(stride[order[i]]) * 2;
    box[i + 1] = order[i] == 1 ? cuuint32_t(box_keys) : 1;
    axis[order[i]] = i + 1;
  }
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, base, dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

int64_t attend_tc_workspace(int dim) { return attend_workspace(num_sms(), kTcItem, dim); }

template <class T, int D, class U, int kParts>
static int launch_tc_kernel(AttendTcArgs& g, cudaStream_t s, AttendArgs* joined) {
  const char* who = "q1_paged_attention launch";
  static bool set[64] = {};
  int dev = 0;
  if (int e = cuda_status(cudaGetDevice(&dev), who)) return e;
  if (dev < 0 || dev >= 64 || !set[dev]) {
    if (int e = cuda_status(cudaFuncSetAttribute(k_attend_tc<T, D, U, kParts>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 TcShape<D>::kSmem), who))
      return e;
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  if (int e = launch_op<AttendTcArgs>(k_attend_tc<T, D, U, kParts>, dim3(unsigned(g.a.ctas)), kTcAThreads, TcShape<D>::kSmem, 1, s, who, g))
    return e;
  // No item has more units than stay whole: nothing to join.
  if (g.a.kv.table_tokens <= kTcWhole * kTcKeys) return Q1_OK;
  if (joined) {
    *joined = g.a;
    return Q1_OK;
  }
  return launch_op(k_attend_join<U, kTcItem, D, true>, dim3(unsigned(g.a.ctas), kTcJoinSlices), kJoinThreads, 0, 1, s, who,
                   g.a);
}

// False in `ran` where no tensor map can describe the cache's strides.
int launch_attend_tc(const AttendArgs& a, void* workspace, bool bf16, int dim, cudaStream_t s, bool& ran, AttendArgs* joined,
                     const float* factors) {
  AttendTcArgs g = {};
  g.a = a;
  g.a.ctas = num_sms();
  g.factors = factors;
  place_workspace(g.a, workspace);
  // The largest score comes from the largest q.k, and a masked one stays -inf
  // when scaled, where the scale is positive.
  g.q_sign = a.scale_log2 < 0.f ? 0x80008000u : 0u;
  g.a.scale_log2 = std::max(std::fabs(a.scale_log2), FLT_MIN);
  g.box_keys = a.kv.page_shift < 7 ? 1 << a.kv.page_shift : kTcKeys;
  int axis[3] = {};
  const bool as_bf16 = bf16 && !factors;  // the copies are f16
  const int parts = factors && !bf16 ? 2 : 1;
  ran = encode_map(&g.k, as_bf16, a.kv, parts, a.kv.k, dim, g.box_keys, axis) == CUDA_SUCCESS &&
        encode_map(&g.v, as_bf16, a.kv, parts, a.kv.v, dim, g.box_keys, axis) == CUDA_SUCCESS;
  if (!ran) return Q1_OK;
  g.axis_head = axis[0], g.axis_slot = axis[1], g.axis_page = axis[2];
  const auto with = [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (factors) return bf16 ? launch_tc_kernel<__half, D, __nv_bfloat16, 1>(g, s, joined) : launch_tc_kernel<__half, D, __half, 2>(g, s, joined);
    return bf16 ? launch_tc_kernel<__nv_bfloat16, D, __nv_bfloat16, 1>(g, s, joined) : launch_tc_kernel<__half, D, __half, 1>(g, s, joined);
  };
  return dim == 128 ? with(std::integral_constant<int, 128>()) : with(std::integral_constant<int, 64>());
}

}  // namespace q1
