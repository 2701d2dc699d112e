/*
 * q1gemv.h -- C ABI of the GB300 Q1_0 (1-bit) GEMV library (libq1gemv.so).
 *
 * The library computes the row-parallel product of 1-bit Q1_0 weights with a
 * q8_0-quantized activation, as bankML's "docs/modules/gpu.md" defines it
 * ("kernels.rs -- the Q1_0 kernels", first bullet):
 *
 *   for every output row, lanes l = 0..7 keep an f32 accumulator a_l = +0;
 *   for every 128-weight block b (in order), with weight scale d0 (fp16):
 *     for every 32-element sub-block k = 0..3, with activation scale d1 (fp16):
 *       s = sum over the lane's 4 elements 32k+4l+i of (bit ? q : -q),
 *           an exact integer, where negating -128 gives -128;
 *       ab = d1*s (k = 0), ab = fma(d1, s, ab) (k = 1..3);
 *     a_l = fma(d0, ab, a_l);
 *   out = ((a0+a4) + (a2+a6)) + ((a1+a5) + (a3+a7)).
 *
 * Every output element equals, bit for bit, the plain CPU definition above on
 * any GPU, launch shape or batch size.
 *
 * Conventions for every call:
 *   - n (activation length) is a multiple of 128, 128 <= n <= 1<<24; rows >= 1,
 *     rows <= 1<<26.
 *   - Pointers are DEVICE pointers owned by the caller unless noted; the
 *     library keeps no reference to them after the call returns.  Buffers must
 *     be 16-byte aligned and must not overlap.  The activation and output
 *     pointers of the products (x, q, d, out) may instead point into pinned
 *     host memory (cudaHostAlloc / cudaHostRegister) where the device can
 *     address it (unified addressing; on a GB300 the kernels then read and
 *     write it over NVLink-C2C, so a host round trip needs no separate copy).
 *     Packed weights must be device memory.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Calls
 *     only enqueue work; nothing blocks the host unless noted.
 *   - Return value: Q1_OK (0) on success, a negative Q1_ERR_* code on a
 *     rejected argument or a CUDA error (nothing is enqueued after a rejected
 *     argument); q1_last_error() then names the call and the reason.
 *   - Activation scales must be finite.  With a non-finite activation scale
 *     the affected outputs are unspecified (never a fault).  Weight scales
 *     must be finite too: q1_0_pack and q2_0_pack reject a block whose fp16
 *     scale is Inf or NaN (Q1_ERR_ARG naming its row and block).
 */
#ifndef Q1GEMV_H
#define Q1GEMV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define Q1_OK 0
#define Q1_ERR_ARG (-1)     /* shape, pointer, alignment or size rejected   */
#define Q1_ERR_CUDA (-2)    /* a CUDA runtime call or launch failed         */
#define Q1_ERR_NOMEM (-3)   /* q1_0_verify could not allocate device memory */
#define Q1_MISMATCH 2       /* q1_0_verify: some output differs             */

/* Text of the last error on the calling thread ("" if none).  The pointer is
 * valid until the next library call on the same thread. */
const char *q1_last_error(void);

/* Bytes of the packed weight buffer q1_0_pack writes for a rows x n matrix
 * (18 bytes per 128 weights, rows padded to a multiple of 256 and blocks per
 * row to a multiple of 4).  Returns a negative Q1_ERR_ARG for a bad shape.
 * Host-only; touches no device. */
int64_t q1_0_packed_bytes(int64_t rows, int64_t n);

/* Repack Q1_0 weights once into the library's device layout
 * ("kernels.rs -- the Q1_0 kernels", pack_q1_0 bullet: repacked once, the
 * numbers unchanged, only aligned).
 *   blocks : device, rows*(n/128) consecutive 18-byte blocks, row-major; each
 *            block = fp16 scale d0 (little-endian) + 16 bytes of sign bits,
 *            element j in byte 2 + j/8, bit j%8, 1 = +d0, 0 = -d0.
 *            Only 2-byte alignment is required for this pointer.
 *   packed : device, q1_0_packed_bytes(rows, n) bytes, written entirely.
 * Synchronous: returns after `stream` has finished the packing (see q1_0_gemv).
 * Errors: Q1_ERR_ARG for a bad shape or pointer, or when some block's fp16
 * scale is Inf or NaN (the message names the first such row and block; the
 * packed buffer must then not be used); Q1_ERR_CUDA on a failed launch or
 * copy.  The check uses a few bytes of device memory allocated on `stream`
 * for this call alone, so concurrent calls on other streams or threads do not
 * interfere. */
int q1_0_pack(const uint8_t *blocks, int64_t rows, int64_t n, void *packed, void *stream);

/* Inverse of q1_0_pack: writes rows*(n/128) 18-byte blocks identical to the
 * ones that were packed.  Same pointer rules as q1_0_pack. */
int q1_0_unpack(const void *packed, int64_t rows, int64_t n, uint8_t *blocks, void *stream);

/* q8_0 activation quantization (the q8_0 activation of "kernels.rs", pack_act
 * bullet; scale = max|x| / 127).  For each vector v < nvec and each 32-value
 * block: amax = max|x|, d = amax/127 (f32), id = d ? 1/d : 0 (f32),
 * q = roundf(x*id) (half away from zero), scale stored as fp16 (round to
 * nearest even) of d.
 *   x : device f32 [nvec][n]; q : device int8 [nvec][n];
 *   d : device fp16 bits [nvec][n/32].  Each of the three may instead be
 *   pinned host memory, under the same rule as the products' activations
 *   (one launch then reads x over the host link, in full 512-byte requests).
 * n is a multiple of 32 here (128 for use with the products), 1 <= nvec <= 65535.
 * Inputs must be finite and max|x| <= 65504*127 for the scale to stay finite. */
int q8_quantize_act(const float *x, int64_t nvec, int64_t n, int8_t *q, uint16_t *d, void *stream);

/* Matrix-vector product ("kernels.rs -- the Q1_0 kernels", first and second
 * bullets: one exact dot product per output row; rows are independent).
 *   packed : device, from q1_0_pack(rows, n).
 *   q, d   : device q8_0 activation: int8 [n], fp16 bits [n/32] (any quants,
 *            including -128).
 *   out    : device f32 [rows].
 * Launch uses programmatic dependent launch: the kernel starts streaming
 * `packed` while the preceding kernel on `stream` is still running, and reads
 * q and d only after that kernel's writes are visible.  So `packed` must not be
 * written by the kernel immediately preceding this call on the stream
 * (q1_0_pack and host copies are always complete before it). */
int q1_0_gemv(const void *packed, int64_t rows, int64_t n, const int8_t *q, const uint16_t *d,
              float *out, void *stream);

/* One product of a multi-product call: out = the matrix-vector product of the
 * packed rows x n matrix with one activation vector. */
typedef struct q1_product {
  const void *packed;     /* device, from q1_0_pack(rows, n)                         */
  int64_t rows, n;        /* matrix shape                                            */
  const float *x;         /* device f32 [n]: activation, quantized inside the kernel
                             exactly as q8_quantize_act would; or NULL              */
  const int8_t *q;        /* used when x is NULL: device int8 [n] q8_0 quants        */
  const uint16_t *d;      /* used when x is NULL: device fp16 bits [n/32] scales    */
  float *out;             /* device f32 [rows]                                       */
} q1_product;

#define Q1_MAX_PRODUCTS 256

/* Several independent matrix-vector products in ONE launch (the pages' own
 * next step, "batched submissions ... one wait per group" in "Advantages and
 * efficiency"; e.g. the q/k/v or gate/up products of a layer, or a whole set of
 * independent products).  Each out_j is bit-identical to q8_quantize_act(x_j)
 * (when x_j is given) followed by q1_0_gemv.  Products may differ in shape.
 *   products : HOST array of `count` descriptors (1 <= count <= Q1_MAX_PRODUCTS),
 *              read during the call only.
 * Outputs must not overlap each other or any input.  Same launch behaviour as
 * q1_0_gemv (programmatic dependent launch; `packed` may be read before the
 * preceding kernel on `stream` has finished). */
int q1_0_gemv_multi(const q1_product *products, int count, void *stream);

/* A device byte range (for q1_0_gemv_multi_prefetch). */
typedef struct q1_range {
  const void *ptr;        /* device pointer, 16-byte aligned; NULL with 0 bytes   */
  int64_t bytes;          /* 0 <= bytes <= 2^40, rounded down to a multiple of 16 */
} q1_range;

#define Q1_MAX_PREFETCH_RANGES 4

/* q1_0_gemv_multi, and while the launch runs its CTAs also pull the given
 * device byte ranges into the L2 cache (one bulk prefetch a CTA and range,
 * issued before the kernel waits for the preceding one; nothing waits for
 * them and nothing of them is read into the SMs).  For a chain of dependent
 * launches (a decode step, where each product's activation is produced by the
 * kernels before it), the ranges are the packed weights of the launch that
 * follows (they do not depend on the chain) and its activation (in a decode
 * step the output of the kernel just before, already in L2; a chain that
 * reads stored activations gets the same effect by prefetching them).  That
 * launch then finds its inputs in L2 instead of HBM.  A prefetch never
 * changes what a kernel reads: L2 is where every write lands first.  No
 * counterpart in the pages; it serves their point that each matrix call pays
 * its own submit and wait ("Limitations").
 *   prefetch : HOST array of `nranges` ranges (0 <= nranges <=
 *              Q1_MAX_PREFETCH_RANGES; NULL with 0), read during the call
 *              only.  Each range must be memory the device may read; its
 *              contents do not matter and no byte outside it is touched.
 * Outputs are those of q1_0_gemv_multi, bit for bit.  Q1_ERR_ARG for a bad
 * range, as for the products. */
int q1_0_gemv_multi_prefetch(const q1_product *products, int count, const q1_range *prefetch, int nranges,
                             void *stream);

/* The work split of a q1_0_gemv_multi launch, as the call would make it.
 * Planning only: nothing is launched and no pointer in `products` is read
 * (only rows and n; the shapes are checked as q1_0_gemv_multi checks them).
 * A tile is rows_per_thread x 32 rows (x 2 panel slots when rows_per_thread
 * is 1 or 2) across all of n; its cost is the product's quad-padded blocks
 * per row.  The products' tiles are laid on one axis in list order; CTA b gets the
 * tiles whose first block falls in its contiguous range of that axis.  With
 * more than 8 products the host places the range boundaries so that the
 * largest range is as small as contiguous ranges allow (a binary search over
 * the bound, each step one greedy fill in list order); otherwise the axis is
 * split evenly.  No counterpart in the pages: it exposes the launcher's own
 * decision for inspection and testing.
 *   sms      : SMs to plan for (0 = the current device's count).
 *   plan     : HOST, receives rows per thread, grid, the total cost and the
 *              largest cost any CTA gets.
 *   cuts     : optional HOST int64 [max_cuts], receives the grid+1 range
 *              boundaries (as many as fit); may be NULL.
 * Returns Q1_OK or Q1_ERR_ARG. */
typedef struct q1_multi_plan {
  int rows_per_thread;    /* rows of a tile each consumer thread handles (1, 2 or 8) */
  int grid;               /* CTAs launched                                          */
  int64_t total_cost;     /* sum over products of tiles x padded blocks per row     */
  int64_t max_range_cost; /* largest tile cost owned by one CTA                     */
  int panel_warps;        /* 0: the streaming kernel above.  Else the call (up to
                             8 products of few rows in total) runs as one CTA per
                             panel_panels consecutive 32-row panels of a
                             product, whose panel_warps warps share out those
                             panels' blocks in units of panel_unit_blocks (grid
                             = ceil(panels / panel_panels) summed over the
                             products, rows_per_thread = 4, both costs 0, no
                             cuts) */
  int panel_unit_blocks;  /* 4 (quads) or 2 (half quads); 0 with the streaming kernel */
  int panel_panels;       /* panels a CTA takes: 1, or 2..8 when one CTA per panel
                             would put two or more panels on an SM (the CTA then
                             builds the activation table once for all of them);
                             0 with the streaming kernel */
} q1_multi_plan;

int q1_0_gemv_multi_plan(const q1_product *products, int count, int sms, q1_multi_plan *plan, int64_t *cuts,
                         int max_cuts);

/* Small-batch product ("kernels.rs -- the Q1_0 kernels", second bullet: each
 * lane's chain over the blocks is independent of every other chain, so one
 * stream of the weights serves several activation vectors, each vector's
 * chains kept apart): the matrix-vector product for each of nvec activation
 * vectors sharing one pass over the weights (1 <= nvec <= 64).
 *   q : device int8 [nvec][n]; d : device fp16 bits [nvec][n/32];
 *   out : device f32 [nvec][rows] (row-major per vector).
 * out[v][r] is bit-identical to q1_0_gemv on vector v. */
int q1_0_gemm_small(const void *packed, int64_t rows, int64_t n, int64_t nvec, const int8_t *q,
                    const uint16_t *d, float *out, void *stream);

/* Which kernel q1_0_gemm_small runs, for every call that follows in this
 * process (no counterpart in the pages: a tuning and testing knob).  Both
 * kernels give identical bits.
 *   choice : 0 = automatic (the default): from 8 vectors up, a cost model
 *            measured on a GB300 picks the faster of the two for the shape;
 *            1 = the dp4a kernel (CUDA cores) always;
 *            2 = the tensor-core kernel always (an f16 MMA gives each lane's
 *            sub-block chain in one exact f32 accumulator where an activation
 *            bound allows it, the dp4a chain elsewhere; it takes a per-call
 *            scratch of about 8 KB per 128 weights of n per 16 vectors from
 *            a pool the library keeps per device, and rejects shapes needing
 *            more than 64 MB).
 * Returns the previous choice, or Q1_ERR_ARG for another value. */
int q1_gemm_small_kernel(int choice);

/* Small-batch product that allocates no device memory.  The pages have no
 * counterpart: this is a service for callers, not part of the method.
 *
 * q1_0_gemm_small takes its tensor-core scratch from a memory pool at call
 * time.  Some callers cannot allow that: a serving loop that reserves all
 * device memory up front and forbids allocation on its decode path (an
 * allocation can stall behind other device work, and fails when a
 * framework's allocator already holds the memory), or a host whose memory
 * accounting must see every byte the process uses.  This call runs the
 * tensor-core kernel of q1_0_gemm_small with its scratch in one fixed array
 * of 8 MiB that the library holds in every device's memory from load to
 * process exit.  It calls no allocator.
 *   Arguments, layout and outputs: as q1_0_gemm_small (1 <= nvec <= 64);
 *   out[v][r] is bit-identical to q1_0_gemm_small's.
 *   Limit: the scratch needs 8 KB per 128 weights of n for each group of 16
 *   vectors, plus a few bytes; a larger n is rejected with Q1_ERR_ARG before
 *   anything is enqueued (for example n <= 32640 with 33..64 vectors,
 *   n <= 130944 with 1..16).
 *   First call on a device: it looks up the device address of the array on
 *   the current device (once per device); make that first call before any
 *   stream capture.
 *   Sharing: every call on a device uses the same array, and the array keeps
 *   the last call's contents (nothing in it needs to start at zero: each call
 *   writes what it reads).  Calls whose work overlaps on the GPU (on different
 *   streams, or from different host threads without ordering) race on it;
 *   order them, e.g. issue them on one stream.
 * Errors: Q1_ERR_ARG for a bad shape, pointer or a size beyond the limit;
 * Q1_ERR_CUDA for a failed lookup or launch. */
int q1_0_gemm_small_noalloc(const void *packed, int64_t rows, int64_t n, int64_t nvec, const int8_t *q,
                            const uint16_t *d, float *out, void *stream);

/* ---------------------------------------------------------------------------
 * Q2_0 (ternary) weights: the sibling format the pages name as the next GPU
 * kernel ("Advantages and efficiency", where optimization goes next;
 * "Limitations": no Q2_0 GPU kernel yet) without giving its layout or
 * arithmetic.  This library's reading:
 *   block (34 bytes) = fp16 scale d0 (little-endian), then 32 bytes of 2-bit
 *     codes: element j's code is (qs[j/4] >> 2*(j%4)) & 3, and codes 0, 1, 2
 *     mean the weights -d0, 0, +d0 (code 3 is not a weight);
 *   row product = the Q1_0 definition at the top of this file with the lane
 *     sum taken over ternary values: +1 contributes q, -1 the negation of q
 *     (-(-128) stays -128), 0 nothing.
 * Every output is bit-identical to that CPU definition.  Same conventions as
 * the Q1_0 calls.
 * ------------------------------------------------------------------------- */

/* Bytes of the packed Q2_0 buffer for a rows x n matrix (34 bytes per 128
 * weights, rows padded to a multiple of 256 and blocks per row to a multiple
 * of 4).  Host-only; negative Q1_ERR_ARG for a bad shape. */
int64_t q2_0_packed_bytes(int64_t rows, int64_t n);

/* Repack Q2_0 weights once into the library's device layout (two sign planes,
 * +1 and -1, in the Q1_0 bit order).
 *   blocks : device, rows*(n/128) consecutive 34-byte blocks, row-major, as
 *            above; only 2-byte alignment is required.
 *   packed : device, q2_0_packed_bytes(rows, n) bytes, written entirely.
 * Synchronous.  Returns Q1_ERR_ARG if any element holds the code 3 or any
 * block's fp16 scale is Inf or NaN (the message names the first such row and
 * block; the packed buffer must then not be used), or for a bad shape or
 * pointer.  Like q1_0_pack, the check uses device memory of this call alone. */
int q2_0_pack(const uint8_t *blocks, int64_t rows, int64_t n, void *packed, void *stream);

/* Inverse of q2_0_pack: writes rows*(n/128) 34-byte blocks identical to the
 * ones that were packed (codes 0..2). */
int q2_0_unpack(const void *packed, int64_t rows, int64_t n, uint8_t *blocks, void *stream);

/* Q2_0 matrix-vector product: as q1_0_gemv, with `packed` from q2_0_pack. */
int q2_0_gemv(const void *packed, int64_t rows, int64_t n, const int8_t *q, const uint16_t *d,
              float *out, void *stream);

/* Several independent Q2_0 products in one launch: as q1_0_gemv_multi, each
 * descriptor's `packed` from q2_0_pack(rows, n). */
int q2_0_gemv_multi(const q1_product *products, int count, void *stream);

/* q2_0_gemv_multi with the L2 prefetch of q1_0_gemv_multi_prefetch. */
int q2_0_gemv_multi_prefetch(const q1_product *products, int count, const q1_range *prefetch, int nranges,
                             void *stream);

/* The work split of a q2_0_gemv_multi launch: as q1_0_gemv_multi_plan.  The
 * kernel choice for a single product can differ from Q1_0's (the Q2_0 panel
 * kernel keeps more registers a thread, so fewer of its CTAs fit an SM). */
int q2_0_gemv_multi_plan(const q1_product *products, int count, int sms, q1_multi_plan *plan, int64_t *cuts,
                         int max_cuts);

/* Device status word of the library's kernels on the current device.  A
 * kernel whose bounded internal wait gives up (it never should: every wait is
 * for work the same kernel issued) sets bit 0 instead of hanging, and skips
 * its remaining output.  Bit 1 (2): an index on the device (an adapter, a
 * page, a position, a length) lay outside what its call was given, see the
 * operators below.  Synchronous: copies the word to the host.
 *   clear : nonzero resets the word to 0 after reading it.
 * Returns the status flags (0 = no event) or a negative Q1_ERR_CUDA. */
int q1_device_status(int clear);

/* On-card self-check ("How it is verified": verify_q1_0 compares every kernel
 * and shape with the CPU bits, including -128 quants and a layer-shaped regime
 * whose per-block scales make products inexact in f32; the Q2_0 product is
 * checked the same way).  Runs synchronously on
 * the current device with its own allocations, against a host-side reference
 * compiled into the library.
 *   flags  : 0 = default shape set (small products for the panel kernel, two
 *            with too many rows for it that take the streaming kernel, and
 *            the batched product through q1_0_gemm_small and, for its
 *            tensor-core kernel, q1_0_gemm_small_noalloc), preceded by an
 *            exhaustive check of the kernels' quantizer rounding (every
 *            float |t| < 2^22 against the device's roundf); bit 0 (1) =
 *            quick set (three small shapes, no
 *            rounding check);
 *            bit 1 (2) = negative control: in every one-vector case the
 *            packed scales of one row (nonzero reference output, about the
 *            middle row) are doubled after packing, so the check must report
 *            that row as the first differing one and return Q1_MISMATCH;
 *            bit 2 (4) = before the cases, run the library's bounded wait on an
 *            mbarrier nothing completes (20 ms limit): it must give up and let
 *            its kernel return, and the cases that follow show the device still
 *            works (the failure path of every product kernel's waits).
 *   report : host buffer receiving one line per kernel and shape, or the first
 *            differing row ("row i differs ..."); may be NULL.
 * Returns Q1_OK if every output is bit-identical, Q1_MISMATCH (2) if any
 * differs, or a negative error. */
int q1_0_verify(int flags, char *report, size_t report_len);

/* ---------------------------------------------------------------------------
 * The operators between a decoder layer's products.  The pages name none of
 * them; they are the formulas that any layer around the products computes:
 * residual and root-mean-square norm with the next product's q8_0 activation,
 * low-rank adapters beside a product, rotary positions with a paged cache of
 * keys and values, and attention over that cache.
 *
 * Conventions of the calls above, except where a call says otherwise: element
 * strides are given, and index arrays are read on the device.  An index that
 * lies outside its range is never followed: the call says what happens to its
 * rows, and q1_device_status bit 1 is set.  All sums, maxima and norms are f32.
 * Like the products these launches start while the preceding kernel on the
 * stream drains, and read nothing before it has finished.
 * ------------------------------------------------------------------------- */

/* Element types. */
#define Q1_F32 0
#define Q1_BF16 1
#define Q1_F16 2

/* Residual addition, root-mean-square norm and q8_0 quantization of nvec rows:
 *   h = x + residual (x where residual is NULL), in f32;
 *   residual_out = h rounded to the type;
 *   y = (h * (1 / sqrt(mean(h^2) + eps))) * weight;  q, d = the q8_0 form of
 *   y exactly as q8_quantize_act gives it (of y in f32, before any rounding).
 *   x, residual, residual_out, y : [nvec][n] of `dtype` (Q1_F32, Q1_BF16,
 *     Q1_F16), rows ldx, ldr, ldo, ldy elements apart; residual, residual_out
 *     and y may be NULL.  residual_out may be x or residual itself, and y may be x.
 *   weight : f32 [n].  q : int8 [nvec][n], d : fp16 bits [nvec][n/32], both or
 *     neither (NULL); with them n is a multiple of 32, else any n >= 1.
 * The sum of h^2 must be finite in f32 (|h| below 1e19 / sqrt(n) is enough).  A row
 * with a NaN is NaN in residual_out (there), in y and in the scales d (everywhere).
 * Alignment: q and d 16 bytes, the others their type's size (16-byte aligned
 * rows are faster).  1 <= nvec <= 2^24, n <= 2^24.  A row's outputs do not
 * depend on the number of rows, bit for bit. */
int q8_add_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const float *weight, float eps,
                    int64_t nvec, int64_t n, int dtype, void *residual_out, int64_t ldo, void *y, int64_t ldy,
                    int8_t *q, uint16_t *d, void *stream);

/* Low-rank adapters of many requests beside a product: for each vector v with
 * adapter i = index[v],
 *   out_v = base_v + scale[i] * (b_i (a_i x_v)),
 * and out_v = base_v where index[v] is -1.
 *   x : f32 [nvec][n], rows ldx apart, of magnitude below 2^127.  base, out : f32 [nvec][rows], rows ldb
 *     and ldo apart; base may be out (in place).  1 <= nvec <= 65535.
 *   a : [adapters][rank][n], b : [adapters][rows][rank] of `dtype` (Q1_BF16 or
 *     Q1_F16); n and rank multiples of 8, rank in 8..128.
 *   index : int32 [nvec].  ranks : int32 [adapters] or NULL: the ranks in use
 *     (0..rank) of each adapter; what lies past them is not used and may hold
 *     anything.  scale : f32 [adapters] or NULL (1).
 * A value of x, or of a weight within the rank, that is no number makes what
 * it goes into no number (an infinite one NaN or infinite), and nothing else.
 * x, a and b must be 16-byte aligned, ldx a multiple of 4, the other arrays 4-byte
 * aligned.  An index outside
 * -1..adapters-1 counts as -1 and sets the status bit. */
int q1_lora_add(const float *x, int64_t ldx, int64_t nvec, int64_t n, int64_t rows, const void *a, const void *b,
                int dtype, int64_t adapters, int64_t rank, const int32_t *index, const int32_t *ranks,
                const float *scale, const float *base, int64_t ldb, float *out, int64_t ldo, void *stream);

/* A paged cache of keys and values, and the sequences of one call.  Sequence b
 * has its tokens 0 .. kv_len[b]-1 in the cache, the last new_start[b+1] -
 * new_start[b] of them new in this call; token t lies in page
 * table[b][t / page_size], slot t % page_size.  The new tokens of all
 * sequences are packed: rows new_start[b] .. new_start[b+1]-1 of q, k, v, out. */
typedef struct q1_paged_kv {
  void *k, *v;              /* device [pages][page_size][kv_heads][dim] of dtype, in any
                               order of the first three axes, the same for both        */
  int64_t page_stride, slot_stride, head_stride; /* elements; multiples of 8, at least dim */
  const int32_t *table;     /* device [batch][table_width], rows table_stride apart;
                               entries past a sequence's length are not read           */
  int64_t table_width, table_stride;
  const int32_t *kv_len;    /* device [batch]: cached tokens, the new ones among them  */
  const int32_t *new_start; /* device [batch + 1]: not falling                         */
  int64_t pages, page_size; /* page_size a power of two in 8..4096                     */
  int64_t kv_heads, dim;    /* dim 64 or 128                                           */
  int64_t batch, total_new; /* total_new: rows of the packed tensors, >= new_start[batch];
                               rows past new_start[batch] belong to no sequence        */
  int dtype;                /* Q1_BF16 or Q1_F16                                       */
} q1_paged_kv;

/* Rotary positions and the cache's new entries, from the q, k and v products'
 * outputs: each pair (e, f) of a head's first `rot` values at position p
 * becomes (e cos - f sin, f cos + e sin); values past rot stay.  Row j of a
 * sequence's new tokens has position kv_len - (new tokens) + j.
 *   q : f32 [total_new][heads][dim], k, v : f32 [total_new][kv_heads][dim], rows
 *     ldq, ldk, ldv elements apart (multiples of 4).
 *   cos_sin : f32 [positions][rot]: rot/2 cosines, then rot/2 sines.  rot is a
 *     multiple of 8 up to dim.
 *   interleaved : 0 pairs value i with value i + rot/2, else 2i with 2i + 1.
 *   q_out : [total_new][heads][dim] of the cache's type.
 * k (turned) and v go to the cache.  Pointers 16-byte aligned.  A token whose
 * position or page is out of range goes nowhere, its q_out row is zero, and
 * the status bit is set; so is the q_out row of a token of no sequence
 * (without the bit). */
int q1_rope_append(const float *q, int64_t ldq, const float *k, int64_t ldk, const float *v, int64_t ldv,
                   const float *cos_sin, int64_t positions, int64_t rot, int interleaved, int64_t heads, void *q_out,
                   const q1_paged_kv *kv, void *stream);

/* Bytes of q1_paged_attention's workspace for sequences of up to max_new new
 * tokens, on the current device; negative Q1_ERR_ARG for a bad shape. */
int64_t q1_paged_attention_workspace(int64_t max_new, int64_t heads, int64_t kv_heads, int64_t dim);

/* Causal attention of the new tokens over their sequence's cache: for a token
 * at position p and query head h (key head h / (heads / kv_heads)),
 *   out = sum_j w_j v_j / sum_j w_j over j = 0..p, w_j = exp(scale * q.k_j).
 *   q, out : [total_new][heads][dim] of the cache's type, strides in elements
 *     (multiples of 8).  A row that sees no key (p < 0) is zero; rows of no
 *     sequence are left as they are.
 *   total_new * heads / kv_heads below 2^31.
 *   scale : finite, and so is scale * log2(e).
 *   max_new : the most new tokens any sequence has (with the batch and the
 *     length of the table it picks the kernel: a larger or smaller number costs
 *     time, not correctness).
 *   workspace : device, 16-byte aligned, q1_paged_attention_workspace bytes;
 *     needs no initial value; calls that may overlap need one each.
 * Slots past a sequence's length may hold anything.  A value of q, k or v that
 * is no number (NaN, infinite) reaches the rows that see it by the formula, and
 * no others: not those of earlier tokens of the call.  (A row whose visible scores
 * are all -inf is NaN.)  The weights w_j are rounded to the cache's type for their
 * product with v (their sum is not).  A page out of range reads as zeros and sets
 * the status bit, as does a kv_len outside the table (it is clamped). */
int q1_paged_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride, int64_t heads, float scale,
                       const q1_paged_kv *kv, int64_t max_new, void *out, int64_t out_token_stride,
                       int64_t out_head_stride, void *workspace, int64_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * The paged cache in q8_0: one byte a value and an f16 scale for 32 of them,
 * 0.53 of a 16-bit cache's bytes.  The conventions of the operators above.
 * ------------------------------------------------------------------------- */

/* As q1_paged_kv, with keys and values as q8_0 blocks of 32 along dim. */
typedef struct q1_paged_q8 {
  int8_t *k, *v;              /* device [pages][page_size][kv_heads][dim], in any order of the
                                 first three axes, the same for both                        */
  uint16_t *k_scale, *v_scale; /* device fp16 bits [pages][page_size][kv_heads][dim/32], in any
                                 order of the first three axes, the same for both; a head's
                                 slots side by side (as in [pages][kv_heads][page_size]
                                 [dim/32]) make the attention's reads whole sectors         */
  int64_t page_stride, slot_stride, head_stride; /* of k and v, in values: multiples of 16, at least dim */
  int64_t scale_page_stride, scale_slot_stride, scale_head_stride; /* in scales: multiples of dim/32 */
  const int32_t *table;       /* these as in q1_paged_kv */
  int64_t table_width, table_stride;
  const int32_t *kv_len;
  const int32_t *new_start;
  int64_t pages, page_size;
  int64_t kv_heads, dim;      /* dim 64 or 128 */
  int64_t batch, total_new;
} q1_paged_q8;

/* q1_rope_append into a q8_0 cache: k (turned, in f32) and v are quantized as
 * q8_quantize_act does each 32 values of a head.  q_out is of `dtype` (Q1_BF16
 * or Q1_F16).  A block with a value that is no number (NaN, infinite) gets the
 * scale NaN; |k| and |v| up to 65504 * 127 keep the scale finite. */
int q1_rope_append_q8(const float *q, int64_t ldq, const float *k, int64_t ldk, const float *v, int64_t ldv,
                      const float *cos_sin, int64_t positions, int64_t rot, int interleaved, int64_t heads,
                      void *q_out, int dtype, const q1_paged_q8 *kv, void *stream);

/* Reads keys and values back: rows new_start[b] .. new_start[b+1]-1 of k_out and
 * v_out, [total_new][kv_heads][dim] of `dtype` (Q1_F32, Q1_BF16, Q1_F16), are
 * the last tokens of sequence b (all of them where new_start counts whole
 * lengths), each value quant * scale rounded once.  Rows of no sequence, and
 * of tokens whose page is out of range (which sets the status bit), are zero.
 * Either output may be NULL.  16-byte aligned. */
int q1_cache_read_q8(const q1_paged_q8 *kv, int dtype, void *k_out, void *v_out, void *stream);

/* Bytes of q1_paged_attention_q8's workspace, on the current device, for
 * sequences of up to max_new new tokens.  Where max_new asks for the
 * tensor-core kernel that includes f16 copies of the keys and values (for f16 q
 * in two parts) of `sequences` sequences of up to table_tokens (the table's width
 * times the page size); else both are not looked at.  Negative Q1_ERR_ARG for a bad shape. */
int64_t q1_paged_attention_q8_workspace(int64_t max_new, int64_t heads, int64_t kv_heads, int64_t dim,
                                        int dtype, int64_t table_tokens, int64_t sequences);

/* q1_paged_attention over a q8_0 cache; q and out are of `dtype` (Q1_BF16 or
 * Q1_F16).  Up to some tens of rows a key head (new tokens times the group) the
 * quants are multiplied as they are, which is exact, and scales are applied to
 * sums (keys) and weights (values: a weight's product with the scale is rounded to f16, off
 * by 2^-11 of itself or by 2^-25 of the row's largest).  More rows take the tensor-core kernel
 * over a copy of the sequence that the call makes in the workspace: each value quant *
 * scale, divided by a power of two for its sequence and head (so its size does not
 * matter; values 2^-28 of the head's largest and below are off by 2^-39 of it), rounded
 * to f16, and with f16 q the remainder as a second f16.  As many sequences
 * are copied at a time as the workspace holds: at least q1_paged_attention_q8_workspace(...,
 * 1) bytes are needed, and more make fewer launches for several such sequences.  A copy has room for
 * the whole width of the table, whatever the lengths are; and for so many rows this cache costs time (a
 * chunk 1.1 to 2.2, a mixed batch 1.9 to 2.2 times what it takes over a 16-bit one): it saves memory.
 * All else as q1_paged_attention; a value is no number where its scale is none. */
int q1_paged_attention_q8(const void *q, int64_t q_token_stride, int64_t q_head_stride, int64_t heads, float scale,
                          int dtype, const q1_paged_q8 *kv, int64_t max_new, void *out, int64_t out_token_stride,
                          int64_t out_head_stride, void *workspace, int64_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * The gated activation between the up and the down product, and the choice of
 * the next token from the output product's logits.
 * ------------------------------------------------------------------------- */

#define Q1_ACT_SILU 0 /* x / (1 + e^-x)                                                          */
#define Q1_ACT_GELU 1 /* x (1 + tanh u) / 2 = x / (1 + e^-2u), u = sqrt(2/pi) (x + 0.044715 x^3) */

/* y = act(gate) * up in f32, and its q8_0 form exactly as q8_quantize_act gives
 * it (of y before any rounding).
 *   gate, up, y : [nvec][n] of `dtype` (Q1_F32, Q1_BF16, Q1_F16), rows ldg, ldu,
 *     ldy elements apart; y may be NULL, or gate or up itself.
 *   q : int8 [nvec][n], d : fp16 bits [nvec][n/32], both or neither (NULL); with
 *     them n is a multiple of 32, else any n >= 1.
 * A block with a value that is no number (NaN, infinite) has the scale NaN.
 * Alignment: q and d 16 bytes, the others their type's size (16-byte aligned
 * rows are faster).  1 <= nvec <= 2^24, n <= 2^24. */
int q8_gated_act(const void *gate, int64_t ldg, const void *up, int64_t ldu, int64_t nvec, int64_t n, int dtype,
                 int activation, void *y, int64_t ldy, int8_t *q, uint16_t *d, void *stream);

/* The settings of q1_sample: for each, an array of one value a row, or (NULL)
 * one value for all of them. */
typedef struct q1_sampling {
  const float *temperature; /* device f32 [rows], or NULL */
  const int32_t *top_k;     /* device int32 [rows], or NULL */
  const float *top_p;       /* device f32 [rows], or NULL */
  const float *min_p;       /* device f32 [rows], or NULL */
  float temperature_all;
  int32_t top_k_all;
  float top_p_all, min_p_all;
} q1_sampling;

/* The next token of each row, drawn with a given random number:
 *   w_i = exp((x_i - max x) / temperature);
 *   of the tokens in the order of falling logits (equal ones by rising index)
 *   the first top_k stay (0 and below: all), of these the fewest first ones whose w
 *   sum to at least top_p of theirs (1 and above: all; one token always stays), and
 *   of these the ones with w_i >= min_p (0 and below: all; the largest always stay);
 *   out = the first token, in the order of the vocabulary, at which the sum of the w that
 *   stayed exceeds uniform times all of it.
 * temperature 0 and below: the first token with the largest logit.
 *   logits : [rows][vocab] of `dtype` (Q1_F32, Q1_BF16, Q1_F16), rows ld apart
 *     (0: one row for all), aligned to the type's size.
 *   uniform : f32 [rows], in [0, 1) (held within it).
 *   out : int32 [rows].
 * The weights are fixed-point numbers of 44 bits behind the point, off by 2^-30 of
 * themselves or the last bit (below 2^-44 of the largest: zero); their sums are whole numbers, so a row's token
 * does not depend on the order of anything, nor on the other rows.  Where a border lies within that of a sum, they
 * decide: of two equal maxima and nothing else above 2^-44, top_p 0.5 keeps one.  -inf masks a token.  A row with a NaN or
 * +inf, one whose logits are all -inf, and one with a setting or a uniform that is NaN give -1.
 * 1 <= rows <= 65535, 1 <= vocab <= 2^19. */
int q1_sample(const void *logits, int64_t ld, int64_t rows, int64_t vocab, int dtype, const float *uniform,
              const q1_sampling *settings, int32_t *out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* Q1GEMV_H */
