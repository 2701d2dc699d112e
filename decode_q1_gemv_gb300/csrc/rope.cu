// rope.cu -- q1_rope_append: rotary position of q and k, and k and v into the
// paged cache; and the checks of the cache's descriptor.
//
// For a pair (a, b) of a head at position p: (a cos - b sin, b cos + a sin),
// one row of cos and sin a position.  Every value is read once (4 bytes) and
// written once (2 bytes) with a handful of operations: bytes bound it when
// there are many tokens, and the chain of small loads (which sequence, its
// length, its page) when there are few.  That chain is one step of all
// threads for the sequence, then two dependent loads.
//
// Measured: 5751 tokens of seven prompts (32 + 8 + 8 heads of 64, 107 MB) in
// 16.4 us (15.3 in a chain of launches, where a part stays in L2): the copy bandwidth.  64 single tokens (heads of 128):
// 2.5 us a launch; while there are fewer tokens than SMs, several CTAs share a token's units.
#include "paged.cuh"

namespace q1 {

struct RopeArgs {
  Paged kv;
  const float *q, *k, *v;
  int64_t ldq, ldk, ldv;
  const float* cs;     // [positions][rot]: rot/2 cosines, then rot/2 sines
  void* q_out;
  unsigned* status;
  int heads, dim, rot, positions, interleaved;
  int shift, units;  // units of 8 values: log2 of a head's, of a token's q, k and v
};

// 5751 tokens of 384 units: 16.4 us with 128 threads, 17.6 with 64, 16.5 with 96,
// 16.9 with 192, 17.8 with 256; loading a thread's first values before the
// token's place is known took 50 registers and 20.9.
constexpr int kRopeThreads = 128;

// One CTA takes a token (or a part of its units, blockIdx.y); a unit is 8
// values of one head: with half-split rotation 4 of the first and the same 4
// of the second half, else 8 consecutive ones.
template <class T>
__global__ void __launch_bounds__(kRopeThreads) k_rope_append(RopeArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const Paged& kv = a.kv;
  const int token = blockIdx.x;
  // The token's sequence: how many sequences end at or before it.
  int before = 0;
  for (int b0 = 0; b0 < kv.batch; b0 += kRopeThreads) {
    const int b = b0 + threadIdx.x;
    before += __syncthreads_count(b < kv.batch && kv.new_start[b + 1] <= token);
  }
  const bool owned = before < kv.batch && kv.new_start[before < kv.batch ? before : 0] <= token;
  int pos = -1, page = -1;
  if (owned) {
    pos = kv.kv_len[before] - kv.new_start[before + 1] + token;
    if (pos >= 0 && pos < a.positions && pos < kv.table_tokens)
      page = kv.table[before * kv.table_stride + (pos >> kv.page_shift)];
  }
  const bool good = page >= 0 && page < kv.pages;
  if (owned && !good && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(a.status, kStatusBadIndex);
  const int64_t slot = int64_t(page) * kv.page_stride + int64_t(pos & ((1 << kv.page_shift) - 1)) * kv.slot_stride;

  const int qunits = a.heads << a.shift, kunits = kv.kv_heads << a.shift;
  for (int u = blockIdx.y * kRopeThreads + threadIdx.x; u < a.units; u += gridDim.y * kRopeThreads) {
    const int part = u < qunits ? 0 : u < qunits + kunits ? 1 : 2;
    const int v = part == 0 ? u : part == 1 ? u - qunits : u - qunits - kunits;
    const int head = v >> a.shift, unit = v & ((1 << a.shift) - 1);
    const float* src = part == 0 ? a.q + token * a.ldq : part == 1 ? a.k + token * a.ldk : a.v + token * a.ldv;
    src += head * a.dim;
    T* dst;
    if (part == 0)
      dst = static_cast<T*>(a.q_out) + (int64_t(token) * a.heads + head) * a.dim;
    else
      dst = static_cast<T*>(part == 1 ? kv.k : kv.v) + slot + head * kv.head_stride;
    if (part != 0 && !good) continue;
    const bool turned = part != 2 && unit * 8 < a.rot;
    const bool split = turned && !a.interleaved;
    // element offsets of the unit's two groups of four
    const int e0 = split ? unit * 4 : unit * 8, e1 = split ? unit * 4 + a.rot / 2 : unit * 8 + 4;
    float4 x = *reinterpret_cast<const float4*>(src + e0), y = *reinterpret_cast<const float4*>(src + e1);
    if (turned && good) {
      const float* cs = a.cs + int64_t(pos) * a.rot + unit * 4;
      const float4 c = *reinterpret_cast<const float4*>(cs), s = *reinterpret_cast<const float4*>(cs + a.rot / 2);
      const auto turn = [](float& p, float& q, float co, float si) {
        const float t = __fmaf_rn(-q, si, __fmul_rn(p, co));
        q = __fmaf_rn(p, si, __fmul_rn(q, co));
        p = t;
      };
      if (split) {
        turn(x.x, y.x, c.x, s.x), turn(x.y, y.y, c.y, s.y), turn(x.z, y.z, c.z, s.z), turn(x.w, y.w, c.w, s.w);
      } else {
        turn(x.x, x.y, c.x, s.x), turn(x.z, x.w, c.y, s.y), turn(y.x, y.y, c.z, s.z), turn(y.z, y.w, c.w, s.w);
      }
    } else if (!good) {
      x = y = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const uint2 lo = make_uint2(Elem<T>::pack2(x.x, x.y), Elem<T>::pack2(x.z, x.w));
    const uint2 hi = make_uint2(Elem<T>::pack2(y.x, y.y), Elem<T>::pack2(y.z, y.w));
    if (split) {
      *reinterpret_cast<uint2*>(dst + e0) = lo;
      *reinterpret_cast<uint2*>(dst + e1) = hi;
    } else {
      *reinterpret_cast<uint4*>(dst + e0) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  }
}

int check_paged(const char* who, const q1_paged_kv* kv, Paged& p) {
  if (!kv) return fail(Q1_ERR_ARG, "%s: null descriptor", who);
  if (kv->dtype != Q1_BF16 && kv->dtype != Q1_F16) return fail(Q1_ERR_ARG, "%s: bad cache type %d", who, kv->dtype);
  if (kv->pages < 1 || kv->pages > (int64_t(1) << 30) || kv->kv_heads < 1 || kv->kv_heads > 1024 || kv->batch < 1 ||
      kv->batch > (1 << 20) || kv->total_new < 1 || kv->total_new > (int64_t(1) << 24) || kv->table_width < 1 ||
      kv->table_width > (int64_t(1) << 30))
    return fail(Q1_ERR_ARG, "%s: bad shape pages=%lld kv_heads=%lld batch=%lld new=%lld table_width=%lld", who,
                (long long)kv->pages, (long long)kv->kv_heads, (long long)kv->batch, (long long)kv->total_new,
                (long long)kv->table_width);
  if (kv->page_size < 8 || kv->page_size > 4096 || (kv->page_size & (kv->page_size - 1)))
    return fail(Q1_ERR_ARG, "%s: page_size=%lld is no power of two in 8..4096", who, (long long)kv->page_size);
  if (kv->dim != 64 && kv->dim != 128) return fail(Q1_ERR_ARG, "%s: dim=%lld is not 64 or 128", who, (long long)kv->dim);
  if (!kv->k || !kv->v || !kv->table || !kv->kv_len || !kv->new_start) return fail(Q1_ERR_ARG, "%s: null pointer", who);
  if (!aligned16(kv->k) || !aligned16(kv->v)) return fail(Q1_ERR_ARG, "%s: the cache must be 16-byte aligned", who);
  if (!aligned4(kv->table) || !aligned4(kv->kv_len) || !aligned4(kv->new_start))
    return fail(Q1_ERR_ARG, "%s: table, kv_len and new_start must be 4-byte aligned", who);
  if (kv->page_stride % 8 || kv->slot_stride % 8 || kv->head_stride % 8 || kv->page_stride < kv->dim ||
      kv->slot_stride < kv->dim || kv->head_stride < kv->dim || kv->page_stride >= (int64_t(1) << 38) ||
      kv->slot_stride >= (int64_t(1) << 38) || kv->head_stride >= (int64_t(1) << 38))
    return fail(Q1_ERR_ARG, "%s: the cache's strides must be multiples of 8 values, from dim to 2^38", who);
  if (kv->table_stride < kv->table_width) return fail(Q1_ERR_ARG, "%s: table_stride is less than table_width", who);
  p = {};
  p.k = kv->k, p.v = kv->v;
  p.page_stride = kv->page_stride, p.slot_stride = kv->slot_stride, p.head_stride = kv->head_stride;
  p.table = kv->table, p.table_stride = kv->table_stride;
  p.kv_len = kv->kv_len, p.new_start = kv->new_start;
  p.pages = int(kv->pages), p.kv_heads = int(kv->kv_heads), p.batch = int(kv->batch);
  while ((int64_t(1) << p.page_shift) < kv->page_size) ++p.page_shift;
  const int64_t tokens = kv->table_width << p.page_shift;
  p.table_tokens = int(tokens < (int64_t(1) << 30) ? tokens : (int64_t(1) << 30));
  p.total_new = int(kv->total_new);
  return Q1_OK;
}

}  // namespace q1

using namespace q1;

extern "C" int q1_rope_append(const float* q, int64_t ldq, const float* k, int64_t ldk, const float* v, int64_t ldv,
                              const float* cos_sin, int64_t positions, int64_t rot, int interleaved, int64_t heads,
                              void* q_out, const q1_paged_kv* kv, void* stream) {
  const char* who = "q1_rope_append";
  RopeArgs a = {};
  if (int e = check_paged(who, kv, a.kv)) return e;
  if (heads < 1 || heads > 4096) return fail(Q1_ERR_ARG, "%s: bad heads=%lld", who, (long long)heads);
  if (rot < 8 || rot > kv->dim || rot % 8 || positions < 1 || positions > (int64_t(1) << 30))
    return fail(Q1_ERR_ARG, "%s: rot=%lld must be a multiple of 8 in 8..dim, positions=%lld in 1..2^30", who,
                (long long)rot, (long long)positions);
  if (!q || !k || !v || !cos_sin || !q_out) return fail(Q1_ERR_ARG, "%s: null pointer", who);
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(cos_sin) || !aligned16(q_out) || ldq % 4 ||
      ldk % 4 || ldv % 4)
    return fail(Q1_ERR_ARG, "%s: buffers must be 16-byte aligned, row strides multiples of 4", who);
  if (ldq < heads * kv->dim || ldk < kv->kv_heads * kv->dim || ldv < kv->kv_heads * kv->dim)
    return fail(Q1_ERR_ARG, "%s: a row stride is less than its row", who);
  a.q = q, a.k = k, a.v = v, a.ldq = ldq, a.ldk = ldk, a.ldv = ldv;
  a.cs = cos_sin, a.q_out = q_out;
  if (int e = ops_status_ptr(&a.status)) return e;
  a.heads = int(heads), a.dim = int(kv->dim), a.rot = int(rot), a.positions = int(positions);
  a.interleaved = interleaved != 0;
  a.shift = a.dim == 64 ? 3 : 4;
  a.units = (a.heads + 2 * a.kv.kv_heads) << a.shift;
  const int per = (a.units + kRopeThreads - 1) / kRopeThreads;
  const dim3 grid(unsigned(a.kv.total_new), unsigned(a.kv.total_new < num_sms() ? per : 1));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (kv->dtype == Q1_BF16) return launch_op(k_rope_append<__nv_bfloat16>, grid, kRopeThreads, 0, 1, s, who, a);
  return launch_op(k_rope_append<__half>, grid, kRopeThreads, 0, 1, s, who, a);
}
