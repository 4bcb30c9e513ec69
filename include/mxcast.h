/*
 * mxcast.h -- C ABI of libmxcast: block-scaled quantisation of bf16 tensors
 * on MI355X (gfx950).
 *
 * The operations are the cast kernels that the pages measure:
 *   - MXFP8 cast, row-wise, column-wise (into the transposed layout) or both
 *     in one pass, optionally fused with a GELU / dGELU pre-op and a dbias
 *     column sum ("[Common] Fix pointer arithmatic to generate correct
 *     LDS/STS instructions", TransformerEngine PR 3291: tables "MXFP8 generic
 *     quantize kernel" and "MXFP8 specialized cast-only kernel
 *     (bidimensional)"; torchao PR 12 "Multiply with inverse scale in loop
 *     inside of dividing to improve perf": the dim1 cast and its inverse-scale
 *     multiply);
 *   - gated MXFP8 cast of act(gate) * linear with SwiGLU or GeGLU (PR 3291,
 *     table "MXFP8 gated (swiglu / geglu) kernel"), and the backward casts
 *     the same tables name: dSiLU (generic kernel) and dSwiGLU / dGeGLU
 *     (gated kernel);
 *   - NVFP4 quantize-transpose with 16-element or 16 x 16 blocks (PR 3291,
 *     the NVFP4 quantize-transpose kernels under "Important Files Changed",
 *     "Patched but not measurable" and table "NVFP4 2D quantize-transpose
 *     kernel");
 *   - grouped (per-expert) MXFP8 and NVFP4 casts of tensors stacked along
 *     rows (PR 3291, the grouped NVFP4 quantize-transpose row);
 *   - format, layout and shape extensions of the MXFP8 casts: E5M2 elements,
 *     the round-up scale rule, GEMM-ready scale tiles, any row count and row
 *     length (partial edge blocks);
 *   - products of the casts' outputs: MXFP8 matrix products, dense and grouped
 *     by expert, with their gradients, and NVFP4 matrix-vector products;
 *   - what stands around them in a transformer layer: the root-mean-square norm
 *     whose output the casts take, the router whose experts the products go
 *     through, and the way of the tokens' rows to the experts and back, each
 *     with its gradients.
 *
 * Numerics (the pages name these formats but do not define their
 * arithmetic; these are the readings the library implements bit-exactly):
 *   MXFP8 block of 32: amax = max|y|; scale byte (E8M0) = floor(log2 amax) - 8
 *     + 127 clamped to [0, 254]; element = E4M3(y * 2^(127 - byte)), round
 *     to nearest, ties to even code, saturating at +-448, sign kept.  A block
 *     holding Inf/NaN gets scale 0xFF and elements 0x7F.  (E5M2 and the
 *     round-up rule: see MX_ELEM_E5M2 / MX_SCALE_ROUND_UP.)
 *   Fused pre-ops: evaluated in fp32 (tanh-form GELU through
 *     0.5(1+tanh u) = 1/(1+e^-2u), the library's own exp), rounded once to
 *     bf16; that bf16 tensor y is what is quantised and what dbias sums.
 *   NVFP4: S_g = fl32(amax / 2688) (1 if amax = 0); per block of 16:
 *     s = E4M3(fl32(fl32(b/6)/S_g)), inv = fl32(1/fl32(decode(s)*S_g)) (0 if
 *     the product is 0), element = E2M1(fl32(x*inv)), nearest, ties to even,
 *     saturating at +-6.
 *
 * Conventions for every call:
 *   - All tensor pointers are DEVICE pointers owned by the caller; the
 *     library never allocates, frees or synchronises.  Work is enqueued on
 *     `stream` (NULL = the default stream) and completes asynchronously.
 *     Scratch memory comes from the caller (a workspace argument), except
 *     for mx_quantize_noalloc, whose scratch is a static device array.
 *   - bf16 tensors are raw 16-bit patterns; E4M3, E8M0 and packed E2M1 are
 *     raw bytes.  Every tensor is row-major and contiguous.
 *   - Column-wise outputs are transposed: for x[M][K], q_col is [K][M] and
 *     s_col is [K][ceil(M/32)] (MXFP8, compact scales) or q_col
 *     [K][ceil(M/2)], s_col [K][ceil(M/16)] (NVFP4).
 *   - Every pointer must be 16-byte aligned (dbias: 4-byte).
 *   - Arguments are validated on the host before anything is enqueued; on a
 *     validation error nothing is written and a non-zero status returns.
 *     Launch failures return MX_ERR_HIP.  Device faults surface at the
 *     caller's next synchronisation.
 *   - Calls hold no state and are safe from several host threads (the one
 *     exception, mx_quantize_noalloc's shared scratch, is described there).
 */
#ifndef MXCAST_H
#define MXCAST_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MXCAST_ABI_VERSION 10

typedef enum mx_status {
    MX_OK = 0,
    MX_ERR_NULL = 1,        /* a required pointer is NULL                     */
    MX_ERR_ENUM = 2,        /* unknown axis mask, fusion or activation        */
    MX_ERR_SHAPE = 3,       /* non-positive or too large size                 */
    MX_ERR_ALIGN = 4,       /* a pointer is not 16-byte aligned               */
    MX_ERR_WORKSPACE = 5,   /* workspace missing or smaller than required     */
    MX_ERR_ALIAS = 6,       /* an output overlaps an input or another output  */
    MX_ERR_HIP = 7,         /* the HIP runtime reported a launch error        */
    MX_ERR_UNSUPPORTED = 8  /* valid request this version does not implement  */
} mx_status;

/* axis_mask bits */
#define MX_ROWWISE 1u       /* blocks along K: q_row[M][K] and its scales    */
#define MX_COLWISE 2u       /* blocks along M, transposed outputs             */

/*
 * Format flags, OR-ed into the axis_mask of the three MXFP8 casts
 * (mx_quantize, mx_quantize_gated, mx_quantize_dgated; not NVFP4).  The
 * pages name the MXFP8 cast without fixing its element format or scale rule
 * (TransformerEngine PR 3291, table "MXFP8 generic quantize kernel"); the
 * default is E4M3 elements with the floor rule, and these select the other
 * choices of the OCP MX format family:
 *   MX_ELEM_E5M2       E5M2 elements (bias 15, max 57344, round to nearest
 *                      even, saturating) instead of E4M3 (max 448); the
 *                      floor rule becomes byte = floor(log2 amax) - 15 + 127.
 *   MX_SCALE_ROUND_UP  byte = ceil(log2(amax / max_elem)) + 127, the smallest
 *                      power-of-two scale under which no element saturates,
 *                      instead of floor(log2 amax) - emax + 127.
 * Bytes clamp to [0, 254]; a block holding Inf or NaN gets scale 0xFF and
 * elements 0x7F under every choice.  Output layouts are unchanged.
 */
#define MX_ELEM_E5M2 4u
#define MX_SCALE_ROUND_UP 8u

/*
 * MX_SCALE_TILED, OR-ed into the axis_mask of the MXFP8 casts: the scale
 * tensors are written in a GEMM-ready layout instead of compact row-major.
 * The pages only hint at consumer-ready scale shapes (the "fix scale shapes"
 * step of the torchao PR 12 stack); the layout is the one a gfx950
 * block-scaled 32x32x64 MFMA (v_mfma_scale_f32_32x32x64_f8f6f4) reads: lane
 * L of a wave supplies the E8M0 scale of row L % 32 and 32-element K block
 * L / 32 of each 64-wide step (its operand bytes hold 16 K values of each of
 * the step's two blocks), from a byte of a 32-bit register that the
 * instruction's op_sel picks per step; a GPU test feeds the cast's outputs
 * to that instruction.  For a scale matrix S[R][C] (s_row: R = M rows,
 * C = K/32 blocks; s_col: R = K transposed rows, C = M/32 blocks):
 *   tile (rt, bt) = rows 32 rt .. 32 rt + 31, blocks 8 bt .. 8 bt + 7,
 *                   256 bytes at byte offset (bt * ceil(R/32) + rt) * 256;
 *   inside it, the 4-byte word of lane L holds in byte j (j = 0..3) the scale
 *                   of row 32 rt + L % 32, block 8 bt + 2j + L / 32, i.e. the
 *                   scale lane L uses in the j-th of four consecutive steps.
 * Blocks past C in the last block tile are 0.  Size: ceil(R/32) * ceil(C/8)
 * * 256 bytes (mx_scale_size).  Element tensors are unchanged.
 */
#define MX_SCALE_TILED 16u

/* fusion: a pre-op in the low bits, optionally OR-ed with MX_FUSE_DBIAS */
#define MX_FUSE_NONE 0
#define MX_FUSE_GELU 1      /* y = GELU(x)                                    */
#define MX_FUSE_DGELU 2     /* y = GELU'(x) * grad                            */
#define MX_FUSE_DSILU 3     /* y = SiLU'(x) * grad                            */
#define MX_FUSE_DBIAS 0x10  /* also write dbias[k] = sum_m y[m][k] (fp32)     */

/* gated activation */
#define MX_GATED_SWIGLU 1   /* y = silu(gate) * linear                        */
#define MX_GATED_GEGLU 2    /* y = gelu(gate) * linear                        */

/*
 * MXFP8 cast of x[M][K] (bf16), block size 32.  Element bytes are E4M3
 * unless axis_mask holds MX_ELEM_E5M2.  When 32 does not divide K (M), the
 * last block of each row (column) is partial: its scale and codes come from
 * its own elements, and the scale tensors have ceil(K/32) (ceil(M/32))
 * blocks per line.
 *   x        device, bf16 [M][K]
 *   grad     device, bf16 [M][K]; required for MX_FUSE_DGELU / DSILU, else
 *            ignored
 *   M, K     rows, columns: any M, K >= 1, each <= 2^23, M*K <= 2^40.  K a
 *            multiple of 8 (every row of x 16-byte aligned) takes the tiled
 *            kernel, for any M (with M not a multiple of 16 the rows of q_col
 *            start at any byte and it writes them through a two-tile stage,
 *            at a lower bandwidth); any other K takes a kernel for arbitrary
 *            row alignment (same results, lower bandwidth still)
 *   axis_mask  MX_ROWWISE, MX_COLWISE or both (one pass over x), optionally
 *            with the format flags MX_ELEM_E5M2 / MX_SCALE_ROUND_UP and the
 *            layout flag MX_SCALE_TILED (scale tensors then have
 *            mx_scale_size() bytes in the tile layout)
 *   fusion   MX_FUSE_NONE | GELU | DGELU | DSILU, optionally | MX_FUSE_DBIAS
 *   q_row, s_row  E4M3 [M][K] and E8M0 [M][ceil(K/32)]; required iff MX_ROWWISE
 *   q_col, s_col  E4M3 [K][M] and E8M0 [K][ceil(M/32)]; required iff MX_COLWISE
 *   dbias    fp32 [K]; required iff MX_FUSE_DBIAS
 *   workspace, workspace_bytes  device scratch of at least
 *            mx_quantize_workspace_size() bytes (0 unless MX_FUSE_DBIAS);
 *            its contents on entry are ignored and on exit are undefined
 *   stream   HIP stream
 * With MX_FUSE_DBIAS a second, small kernel reduces per-tile column partial
 * sums (fp32, fixed order) into dbias, so results are run-to-run identical.
 */
mx_status mx_quantize(const void *x, const void *grad, int64_t M, int64_t K,
                      unsigned axis_mask, int fusion,
                      uint8_t *q_row, uint8_t *s_row, uint8_t *q_col, uint8_t *s_col,
                      float *dbias, void *workspace, size_t workspace_bytes,
                      hipStream_t stream);

/* Bytes of workspace mx_quantize needs for these arguments (0 without dbias;
 * 0 also for invalid arguments). */
size_t mx_quantize_workspace_size(int64_t M, int64_t K, unsigned axis_mask, int fusion);

/*
 * mx_quantize for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc.  The
 * same cast with the same arguments, minus the workspace: with MX_FUSE_DBIAS
 * the per-tile column partial sums go to a static device array of the
 * library, MX_NOALLOC_SCRATCH_BYTES per GPU, which each GPU the library runs
 * on holds until the process ends.  Outputs are bit-identical to
 * mx_quantize's (the same kernels and the same fixed summation order).
 *   - No device memory is allocated or freed, by the library or a library it
 *     calls.  Without MX_FUSE_DBIAS the scratch is not used at all.
 *   - A dbias cast whose workspace (mx_quantize_workspace_size) exceeds
 *     MX_NOALLOC_SCRATCH_BYTES returns MX_ERR_WORKSPACE and writes nothing.
 *   - Every call on one GPU shares that GPU's scratch, which keeps the last
 *     call's contents (every byte a call reads it has written first): calls
 *     with MX_FUSE_DBIAS that overlap on one GPU (on different streams, or
 *     from several host threads without ordering) race and may give wrong
 *     dbias values.  Calls ordered on one stream are safe.
 *   - The first call on each device looks up the scratch address (no
 *     allocation); the stream's device is made current for that lookup.
 * Other errors as for mx_quantize.
 */
#define MX_NOALLOC_SCRATCH_BYTES ((size_t)4 << 20)
mx_status mx_quantize_noalloc(const void *x, const void *grad, int64_t M, int64_t K,
                              unsigned axis_mask, int fusion,
                              uint8_t *q_row, uint8_t *s_row, uint8_t *q_col, uint8_t *s_col,
                              float *dbias, hipStream_t stream);

/*
 * Bytes of one scale tensor of an MXFP8 cast: the scales of a quantised
 * [rows][cols] tensor blocked along cols (s_row: rows = M, cols = K; s_col:
 * rows = K, cols = M; for the gated casts the quantised tensor's own sizes).
 * rows * ceil(cols/32) for the compact layout, ceil(rows/32) *
 * ceil(ceil(cols/32)/8) * 256 with MX_SCALE_TILED in axis_mask.  0 for a
 * non-positive size, a size above 2^23 or an invalid axis_mask.
 */
size_t mx_scale_size(int64_t rows, int64_t cols, unsigned axis_mask);

/*
 * Grouped (per-expert) MXFP8 cast: G tensors stacked along rows, cast in one
 * launch, each exactly as mx_quantize would cast it on its own.  The pages
 * name a grouped quantize-transpose (TransformerEngine PR 3291, the
 * group_quantize_transpose_nvfp4 row of its "Important Files Changed"
 * table) whose non-Hadamard path was not ready; this is that operation for
 * MXFP8.
 *   x, grad      device, bf16 [M][K], M = sum of group_rows; group g owns rows
 *                r_g .. r_g + group_rows[g] - 1, r_g = sum_{h<g} group_rows[h]
 *   group_rows   HOST array of G row counts, each >= 0 (an empty group is
 *                allowed); 1 <= G <= 64, 0 < M <= 2^23.  K a multiple of 8
 *                takes the tiled kernel, for any counts (counts that are not
 *                multiples of 16: as for an M that is not, in mx_quantize),
 *                any other K the any-shape kernel (same results)
 *   axis_mask, fusion  as for mx_quantize (format and layout flags included)
 *   q_row        [M][K]: the groups' row-wise elements (the stacked tensor's)
 *   s_row        the groups' row scales one after the other, group g's
 *                mx_scale_size(group_rows[g], K) bytes each (for the compact
 *                layout this is [M][ceil(K/32)])
 *   q_col        the groups' transposed elements one after the other: group
 *                g's [K][group_rows[g]] at byte K * r_g
 *   s_col        the groups' column scales one after the other, group g's
 *                mx_scale_size(K, group_rows[g]) bytes each
 *   dbias        fp32 [G][K], group g's column sums (0 for an empty group)
 *   workspace    mx_quantize_grouped_workspace_size() bytes with dbias
 * Errors as for mx_quantize; MX_ERR_SHAPE also for G out of range or a bad
 * group size.
 */
mx_status mx_quantize_grouped(const void *x, const void *grad, int64_t K,
                              const int64_t *group_rows, int G, unsigned axis_mask, int fusion,
                              uint8_t *q_row, uint8_t *s_row, uint8_t *q_col, uint8_t *s_col,
                              float *dbias, void *workspace, size_t workspace_bytes,
                              hipStream_t stream);

/* Workspace bytes of mx_quantize_grouped (0 without dbias or for invalid
 * arguments). */
size_t mx_quantize_grouped_workspace_size(int64_t K, const int64_t *group_rows, int G,
                                          unsigned axis_mask, int fusion);

/* Total bytes of the row scales (colwise = 0) or column scales (colwise = 1)
 * of mx_quantize_grouped (0 for invalid arguments). */
size_t mx_grouped_scale_size(int64_t K, const int64_t *group_rows, int G, unsigned axis_mask,
                             int colwise);

/*
 * Gated MXFP8 cast.  x is bf16 [M][2N] holding [gate | linear] (gate =
 * columns 0..N-1); the quantised tensor is y[M][N] = act(gate) * linear,
 * block size 32 (partial at the edges as for mx_quantize), any M, N >= 1
 * with M <= 2^23, 2N <= 2^23, M * 2N <= 2^40 (N a multiple of 8 takes the
 * tiled kernel, for any M, as in mx_quantize).  axis_mask as for mx_quantize
 * (format flags included).
 *   q_row, s_row  E4M3 [M][N], E8M0 [M][ceil(N/32)]   (iff MX_ROWWISE)
 *   q_col, s_col  E4M3 [N][M], E8M0 [N][ceil(M/32)]   (iff MX_COLWISE)
 */
mx_status mx_quantize_gated(const void *x, int64_t M, int64_t N, unsigned axis_mask, int act,
                            uint8_t *q_row, uint8_t *s_row, uint8_t *q_col, uint8_t *s_col,
                            hipStream_t stream);

/*
 * Gated backward MXFP8 cast (the dswiglu / dgeglu rows of the gated table).
 * grad is bf16 [M][N] (the gradient of act(gate) * linear), x the forward
 * input bf16 [M][2N] = [gate | linear].  With a = act(gate), a' = act'(gate)
 * (act = SiLU for MX_GATED_SWIGLU, GELU for MX_GATED_GEGLU), the quantised
 * tensor is dx[M][2N] = [d_gate | d_linear]:
 *   d_gate   = fl32(fl32(a' * grad) * linear),   d_linear = fl32(a * grad),
 * each rounded once to bf16; block size 32 along 2N (row-wise) and M.
 * Any M, N >= 1 with M <= 2^23, 2N <= 2^23, M * 2N <= 2^40 (partial blocks
 * at the edges as for mx_quantize; N a multiple of 8 takes the tiled kernel,
 * for any M).  axis_mask as for mx_quantize (format flags included).
 *   q_row, s_row  E4M3 [M][2N], E8M0 [M][ceil(2N/32)]   (iff MX_ROWWISE)
 *   q_col, s_col  E4M3 [2N][M], E8M0 [2N][ceil(M/32)]   (iff MX_COLWISE)
 * Errors as for mx_quantize_gated.
 */
mx_status mx_quantize_dgated(const void *grad, const void *x, int64_t M, int64_t N,
                             unsigned axis_mask, int act, uint8_t *q_row, uint8_t *s_row,
                             uint8_t *q_col, uint8_t *s_col, hipStream_t stream);

/*
 * Grouped gated casts (an MoE layer's experts in one launch): x is bf16
 * [M][2N] = [gate | linear] with the groups' rows stacked as for
 * mx_quantize_grouped (HOST group_rows, any counts >= 0, empty groups
 * allowed, 1 <= G <= 64); each group is cast exactly as mx_quantize_gated
 * (forward: quantised tensor [rows][N], W = N) or mx_quantize_dgated
 * (backward, grad bf16 [M][N]: quantised tensor [rows][2N], W = 2N) casts
 * it on its own.  q_row is [M][W]; q_col holds group g's [W][rows] at byte
 * W * r_g; s_row and s_col hold the groups' scale tensors one after the
 * other, group g's mx_scale_size(rows, W) and mx_scale_size(W, rows) bytes
 * (mx_grouped_scale_size(W, ...) in total).  axis_mask as for mx_quantize.
 * Errors as for mx_quantize_gated; MX_ERR_SHAPE also for G out of range or a
 * bad group size.
 */
mx_status mx_quantize_gated_grouped(const void *x, int64_t N, const int64_t *group_rows, int G,
                                    unsigned axis_mask, int act, uint8_t *q_row, uint8_t *s_row,
                                    uint8_t *q_col, uint8_t *s_col, hipStream_t stream);
mx_status mx_quantize_dgated_grouped(const void *grad, const void *x, int64_t N,
                                     const int64_t *group_rows, int G, unsigned axis_mask, int act,
                                     uint8_t *q_row, uint8_t *s_row, uint8_t *q_col,
                                     uint8_t *s_col, hipStream_t stream);

/*
 * The fused elementwise values alone, as bf16: y = pre-op(x[, grad]) for
 * op = MX_FUSE_GELU / MX_FUSE_DGELU / MX_FUSE_DSILU (x, grad and y are
 * [M][K]), the gated value for op = 0x100 | MX_GATED_SWIGLU / MX_GATED_GEGLU
 * (x is [M][2K], y is [M][K]), or the gated backward for op = 0x200 |
 * MX_GATED_SWIGLU / MX_GATED_GEGLU (x is [M][2K], grad [M][K], y [M][2K]).
 * This is the exact tensor the fused casts quantise; it is exposed so that
 * the pre-op arithmetic can be checked on its own.  Any M, K >= 1, each
 * <= 2^23 (2K <= 2^23 for gated ops), M * K <= 2^40.
 */
#define MX_OP_GATED 0x100
#define MX_OP_DGATED 0x200
mx_status mx_fused_values(const void *x, const void *grad, int64_t M, int64_t K, int op,
                          void *y, hipStream_t stream);

/*
 * Tensor absmax for NVFP4: *amax = max |x_i| over n bf16 elements, as fp32
 * (exact); a NaN when an element is NaN, else +Inf when one is infinite.
 * amax is a device pointer to one float; it is first cleared and then
 * combined with integer atomic max, so the result does not depend on
 * scheduling.  n > 0, n <= 2^40, x 16-byte aligned.
 */
mx_status mx_absmax_bf16(const void *x, int64_t n, float *amax, hipStream_t stream);

/*
 * NVFP4 quantize-transpose of x[M][K] (bf16), block size 16, any M, K >= 1,
 * each <= 2^23, M*K <= 2^40.  When 16 does not divide K (M), the last block
 * of each row (column) is partial: its scale and codes come from its own
 * elements, and a line of n codes packs into ceil(n/2) bytes, the high nibble
 * of an odd line's last byte 0.  K a multiple of 16 takes the tiled kernel,
 * for any M (with the transpose and M not a multiple of 16, its rows start
 * at any byte and a variant of the kernel writes them through a two-pair
 * stage); other K a kernel for arbitrary row alignment (same results).
 *   amax     device, one fp32: the tensor absmax the global scale is built
 *            from, as mx_absmax_bf16 computes it (on the same stream).  With
 *            a NaN or infinite amax (a tensor holding a NaN or an Inf) there
 *            is no usable global scale: every scale byte is 0x7F (the E4M3
 *            NaN), every element code 0, and S_g = amax / 2688 stays NaN or
 *            Inf.  An amax other than the tensor's absmax is outside the
 *            contract.
 *   q_row, s_row  packed E2M1 [M][ceil(K/2)] (element 2j in the low nibble
 *            of byte j), E4M3 [M][ceil(K/16)]        (iff MX_ROWWISE)
 *   q_col, s_col  the same for the transpose: [K][ceil(M/2)],
 *            [K][ceil(M/16)]                        (iff MX_COLWISE)
 *   global_scale_out  device, one fp32 receiving S_g; may be NULL
 */
mx_status nvfp4_quantize_transpose(const void *x, int64_t M, int64_t K, const float *amax,
                                   unsigned axis_mask,
                                   uint8_t *q_row, uint8_t *s_row, uint8_t *q_col, uint8_t *s_col,
                                   float *global_scale_out, hipStream_t stream);

/*
 * NVFP4 quantize-transpose with 2D scaling (the "nvfp42d" rows of the
 * quantize-transpose table): one E4M3 scale per 16 x 16 block of x (partial
 * at the right and bottom edges), from the block's amax over its elements by
 * the same chain as above; every element is coded with its block's
 * multiplier.  Arguments, layouts and errors exactly as for
 * nvfp4_quantize_transpose: the block's scale is written for each of its
 * rows in s_row and for each of its columns in s_col, so a consumer of the
 * 1D layouts reads 2D-scaled data unchanged.
 */
mx_status nvfp4_quantize_transpose_2d(const void *x, int64_t M, int64_t K, const float *amax,
                                      unsigned axis_mask,
                                      uint8_t *q_row, uint8_t *s_row, uint8_t *q_col,
                                      uint8_t *s_col, float *global_scale_out, hipStream_t stream);

/*
 * Per-group tensor absmax for the grouped NVFP4 cast: amax[g] = max |x| over
 * the rows of group g (0 for an empty group), as fp32.  x, group_rows, G as
 * for nvfp4_quantize_transpose_grouped; amax is a device array of G floats.
 */
mx_status mx_absmax_bf16_grouped(const void *x, int64_t K, const int64_t *group_rows, int G,
                                 float *amax, hipStream_t stream);

/*
 * Grouped NVFP4 quantize-transpose: G tensors stacked along rows (the
 * operation of the group_quantize_transpose_nvfp4 row of TransformerEngine PR
 * 3291's "Important Files Changed" table, without the Hadamard transform),
 * each quantised in one launch exactly as nvfp4_quantize_transpose (or, with
 * scaling_2d = 1, nvfp4_quantize_transpose_2d) quantises a tensor of its own:
 * with its own tensor amax and global scale.
 *   x            device, bf16 [M][K], M = sum of group_rows; group g owns rows
 *                r_g .. r_g + group_rows[g] - 1
 *   group_rows   HOST array of G row counts, each >= 0; 1 <= G <= 64,
 *                0 < M <= 2^23; any K >= 1.  K a multiple of 16 takes the
 *                tiled kernel, for any counts (counts that are not multiples
 *                of 16: through its variant for transposed rows at any byte,
 *                as for nvfp4_quantize_transpose), any other K the any-shape
 *                kernel (same results)
 *   amax         device, fp32 [G]: each group's tensor amax (for example from
 *                mx_absmax_bf16_grouped)
 *   q_row, s_row [M][ceil(K/2)], [M][ceil(K/16)]: the groups' rows (the
 *                stacked layout)
 *   q_col, s_col group g's [K][ceil(rows/2)] and [K][ceil(rows/16)], the
 *                groups one after the other
 *   global_scale_out  device fp32 [G] or NULL: each group's global scale
 *                (1 for an empty group)
 * Errors as for nvfp4_quantize_transpose; MX_ERR_ENUM also for scaling_2d not
 * 0 or 1, MX_ERR_SHAPE for G out of range or a bad group size.
 */
mx_status nvfp4_quantize_transpose_grouped(const void *x, int64_t K, const int64_t *group_rows,
                                           int G, const float *amax, int scaling_2d,
                                           unsigned axis_mask, uint8_t *q_row, uint8_t *s_row,
                                           uint8_t *q_col, uint8_t *s_col,
                                           float *global_scale_out, hipStream_t stream);

/*
 * Products of MXFP8 operands: what the casts' outputs are for.  An operand
 * value is its element times 2^(scale byte - 127) of its block; products are
 * exact, summed in fp32 on the matrix cores in an order that the sizes and the
 * operands determine (results are run-to-run identical), and rounded once to
 * the output type.  For bf16 outputs the 8-bit matrix instruction adds 8
 * neighbouring k after aligning them, and drops of each product what is below
 * 2^-13 of the largest one's power of two: at most 2^-10 sum |a b| in all, on
 * random operands 100 times below the output's rounding, but more than it
 * where large products cancel.  fp32 outputs take the bf16 instruction, for
 * which elements times scales are exact, at half the rate; where 64 k of a
 * tile hold blocks with values outside bf16 (2^128 and more, or bits below
 * 2^-133), those k take the 8-bit instruction one of 8 at a time, at an eighth
 * of its rate.  Both drop nothing.  A NaN block (scale 0xFF) gives NaN in the
 * output rows and columns it enters.
 *
 * flags, for the three calls:
 *   MX_A_E5M2, MX_B_E5M2  the operand's elements are E5M2 (MX_ELEM_E5M2 casts)
 *                      instead of E4M3
 *   MX_SCALE_TILED     both scale tensors are in the tile layout
 *   MX_OUT_F32         the output is fp32 instead of bf16
 *   MX_OUT_ACCUMULATE  with MX_OUT_F32: the product is added to what the
 *                      output holds (one rounding of that sum to fp32)
 */
#define MX_A_E5M2 4u
#define MX_B_E5M2 32u
#define MX_OUT_F32 64u
#define MX_OUT_ACCUMULATE 128u

/*
 * y[M][N] = A B^T of A [M][K] and B [N][K], both quantised along K.  A layer
 * with weights W [N][K] computes its forward product with B = q_row / s_row
 * of W, its input gradient dX [M][K] = dY W with A = q_row / s_row of dY and
 * B = q_col / s_col of W (that is W^T [K][N], quantised along N), and its
 * weight gradient dW [N][K] = dY^T X with A = q_col / s_col of dY and
 * B = q_col / s_col of X.
 *   qa, sa   elements [M][K] and their scales (mx_scale_size(M, K) bytes)
 *   qb, sb   elements [N][K] and their scales
 *   M, N, K  any sizes >= 1, each <= 2^23, every pair's product <= 2^40, and
 *            ceil(M/256) * ceil(N/256) <= 2^24 - 4096 tiles (2^40 outputs are
 *            more)
 *   y        bf16 or fp32 [M][N]
 *   workspace, workspace_bytes  device scratch of at least
 *            mx_matmul_workspace_size() bytes (NULL and 0 where that is 0)
 * Errors: MX_ERR_ENUM for an unknown flag or MX_OUT_ACCUMULATE without
 * MX_OUT_F32; MX_ERR_NULL, MX_ERR_SHAPE, MX_ERR_ALIGN (16 bytes, every
 * pointer), MX_ERR_WORKSPACE, MX_ERR_ALIAS (y overlaps an operand or the
 * workspace) as for the casts.
 */
mx_status mx_matmul(const uint8_t *qa, const uint8_t *sa, const uint8_t *qb, const uint8_t *sb,
                    int64_t M, int64_t N, int64_t K, unsigned flags, void *y, void *workspace,
                    size_t workspace_bytes, hipStream_t stream);

/*
 * The same for G experts in one launch: group g's rows of A, stacked as for
 * mx_quantize_grouped, by the expert's own B_g [N][K].
 *   qa, sa      the stacked rows' elements [M][K] and the groups' scales one
 *               after the other (q_row, s_row of a grouped cast)
 *   qb, sb      the experts' elements [G][N][K] and scales, one after the other
 *               (q_row, s_row of the stacked weights' grouped cast; for the
 *               input gradient its q_col, s_col)
 *   group_rows  HOST array of G row counts >= 0 with a positive sum M;
 *               1 <= G <= 64.  M, N, K as for mx_matmul, G * N * K <= 2^40, and
 *               the tiles of all groups count together
 *   y           bf16 or fp32 [M][N]; an empty group has no rows in it
 */
mx_status mx_matmul_grouped(const uint8_t *qa, const uint8_t *sa, const uint8_t *qb,
                            const uint8_t *sb, int64_t N, int64_t K, const int64_t *group_rows,
                            int G, unsigned flags, void *y, void *workspace, size_t workspace_bytes,
                            hipStream_t stream);

/*
 * The experts' weight gradients in one launch: dW_g [N][K] = sum over group
 * g's rows m of dY[m][n] X[m][k].
 *   qa, sa      q_col, s_col of the grouped cast of dY [M][N] (group g's
 *               transposed [N][rows] and its scales, one group after the other)
 *   qb, sb      q_col, s_col of the grouped cast of X [M][K]
 *   dw          bf16 or fp32 [G][N][K]; an empty group's gradient is 0 (with
 *               MX_OUT_ACCUMULATE: unchanged)
 */
mx_status mx_matmul_wgrad_grouped(const uint8_t *qa, const uint8_t *sa, const uint8_t *qb,
                                  const uint8_t *sb, int64_t N, int64_t K,
                                  const int64_t *group_rows, int G, unsigned flags, void *dw,
                                  void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace the three products need (0 for most sizes, and for invalid
 * arguments): copies of operands whose rows do not all start at multiples of 16
 * bytes (K, or for weight gradients a group's rows, no multiple of 16), unless
 * the product is small.  Contents on entry are ignored and on exit undefined;
 * calls that may overlap in time need workspaces of their own. */
size_t mx_matmul_workspace_size(int64_t M, int64_t N, int64_t K, unsigned flags);
size_t mx_matmul_grouped_workspace_size(int64_t N, int64_t K, const int64_t *group_rows, int G,
                                        unsigned flags);
size_t mx_matmul_wgrad_grouped_workspace_size(int64_t N, int64_t K, const int64_t *group_rows, int G,
                                              unsigned flags);

/*
 * Matrix-vector products with NVFP4 weights (decoding): y[T][N] = x W^T, with
 * W [N][K] as nvfp4_quantize_transpose writes it (1D or 2D blocks):
 *   y[t][n] = S_g * sum_k x[t][k] E2M1(qw[n][k]) E4M3(sw[n][k / 16]),
 * summed in fp32 and rounded once to the output type; S_g multiplies the sum.
 *   x        device, bf16 [T][K]; T >= 1 (the weights are read once for up
 *            to 64 tokens)
 *   qw, sw   packed E2M1 [N][ceil(K/2)] and E4M3 [N][ceil(K/16)]: q_row, s_row
 *   sg       device, one fp32: the cast's global scale
 *   flags    0 or MX_OUT_F32
 *   y        bf16 or fp32 [T][N]
 * Any T, N, K >= 1, each <= 2^23, every pair's product <= 2^40.  Every pointer
 * is 16-byte aligned (sg: 4-byte).
 */
mx_status nvfp4_matvec(const void *x, int64_t T, const uint8_t *qw, const uint8_t *sw,
                       const float *sg, int64_t N, int64_t K, unsigned flags, void *y,
                       hipStream_t stream);

/*
 * The same through routed experts: y[t][j] = x[t] W_e^T, e = experts[t][j].
 *   experts  device, int32 [T][top], 1 <= top <= 64; any values, repeated ones
 *            too.  An index outside 0 .. G - 1 (a padded slot, an expert that
 *            another device holds) gives a row of zeros
 *   qw, sw   the experts' weights one after the other, as
 *            nvfp4_quantize_transpose_grouped writes G stacked [N][K] matrices;
 *            sg fp32 [G]; 1 <= G <= 1024, G * N * K <= 2^40
 *   y        bf16 or fp32 [T][top][N], T * top <= 2^23
 */
mx_status nvfp4_matvec_experts(const void *x, const int32_t *experts, int64_t T, int64_t top,
                               const uint8_t *qw, const uint8_t *sw, const float *sg, int G,
                               int64_t N, int64_t K, unsigned flags, void *y, hipStream_t stream);

/*
 * Root-mean-square norm of a residual stream, with the casts of its output:
 *   h[m][k]  = bf16(fl32(x + residual)); x itself without a residual
 *   rstd[m]  = (mean_k h[m][k]^2 + eps)^(-1/2), in 64 bits in a fixed order
 *   y[m][k]  = bf16(fl32(h weight rstd)), with the rstd of 64 bits
 * and the MXFP8 casts of y, exactly as mx_quantize casts that tensor.
 *   x, residual  device, bf16 [M][K]; residual may be NULL
 *   weight     device, bf16 [K]; NULL: ones
 *   M, K       as for mx_quantize.  Rows of up to 16384 are held in registers, longer
 *              ones read twice
 *   eps        finite and not negative (MX_ERR_ENUM otherwise)
 *   axis_mask  0 (no casts), or as for mx_quantize, flags included
 *   h          bf16 [M][K], required iff there is a residual
 *   y          bf16 [M][K] or NULL (not written: the casts do not need it)
 *   q_row, s_row, q_col, s_col  as for mx_quantize
 *   q_h, s_h   NULL, or an 8-bit copy of h for the backward: the row-wise MXFP8
 *              cast of h with E4M3 elements, MX_SCALE_ROUND_UP and compact
 *              scales, [M][K] and [M][ceil(K/32)], whatever axis_mask says.  It
 *              is the activation checkpoint of mx_rmsnorm_backward, at half of
 *              h's memory; one step of its elements is 2^-3 of their binade
 *   rstd       fp32 [M], rounded once
 *   workspace, workspace_bytes  device scratch of at least
 *              mx_rmsnorm_workspace_size() bytes (8 M with MX_COLWISE: rstd in
 *              more bits; otherwise 0: NULL and 0 then).  Calls that may overlap in time
 *              need workspaces of their own
 * A row that holds Inf or NaN gets what these formulas give (rstd 0 or NaN); where rstd
 * passes fp32 (rows of tiny numbers with eps 0) it is Inf, in y too.  Errors as for
 * mx_quantize, and MX_ERR_WORKSPACE.
 */
mx_status mx_rmsnorm(const void *x, const void *residual, const void *weight, int64_t M, int64_t K,
                     float eps, unsigned axis_mask, void *h, void *y, uint8_t *q_row,
                     uint8_t *s_row, uint8_t *q_col, uint8_t *s_col, uint8_t *q_h, uint8_t *s_h,
                     float *rstd, void *workspace, size_t workspace_bytes, hipStream_t stream);
size_t mx_rmsnorm_workspace_size(int64_t M, unsigned axis_mask);

/*
 * Gradients of mx_rmsnorm.  With xhat = h rstd, g = dy weight and
 * c[m] = mean_k(g xhat):
 *   dh[m][k]    = bf16(dres + rstd (g - xhat c))     the gradient of x, and the
 *                 same of the residual
 *   dweight[k]  = sum_m dy xhat
 * g, xhat and the sums in fp32, these in a fixed order (results are run-to-run
 * identical); a column's weight gradient in lines of at most ceil(M / 256) rows, of 64
 * where rows are longer than 16384.
 *   dy         device, bf16 [M][K]: the gradient of y
 *   h          bf16 [M][K], or NULL: then
 *   q_h, s_h   the forward's 8-bit copy is read in its place (NULL with h)
 *   rstd       fp32 [M], of the forward
 *   weight     bf16 [K] or NULL
 *   dres       bf16 [M][K], the gradient that arrives at h from the residual
 *              stream, or NULL
 *   dh         bf16 [M][K]
 *   dweight    fp32 [K], or NULL: not computed
 *   workspace, workspace_bytes  device scratch of at least
 *              mx_rmsnorm_backward_workspace_size() bytes with dweight
 *              (per-workgroup partial sums; NULL and 0 without).  Calls that may
 *              overlap in time need workspaces of their own
 * MX_ERR_NULL also for both or neither of h and q_h.
 */
mx_status mx_rmsnorm_backward(const void *dy, const void *h, const uint8_t *q_h, const uint8_t *s_h,
                              const float *rstd, const void *weight, const void *dres, int64_t M,
                              int64_t K, void *dh, float *dweight, void *workspace,
                              size_t workspace_bytes, hipStream_t stream);
size_t mx_rmsnorm_backward_workspace_size(int64_t M, int64_t K);

/*
 * A router: each token's experts and their weights, from its logits.
 *   p[t][e]   = softmax over e of logits[t], or with MX_ROUTE_SIGMOID the
 *               logistic function of each
 *   key[t][e] = p + bias[e] (bias NULL: 0).  An expert whose logit or bias is
 *               -Inf is masked: it is never chosen
 *   groups    the E experts are `groups` runs of E / groups; a group's score is
 *             its best key, or with MX_ROUTE_GROUP_PAIR the sum of its two best
 *             (of its one, where it has one); the top_groups best groups stay.
 *             groups = 1: all of them
 *   experts   the `top` best keys of these, best first; equal keys, and equal
 *             groups, the lowest index first.  Keys are compared in 64 bits;
 *             without a bias, and where no two are added, by the logits
 *             themselves, exactly
 *   weights   p of the chosen ones (without the bias), in fp32 (0 below 2^-150,
 *             and in steps of 2^-149 below 2^-126), with MX_ROUTE_RENORM divided
 *             by their sum (0 where that is 0), times scale
 * A slot that no expert is left for (fewer unmasked ones than `top`) gets expert
 * -1 and weight 0, which nvfp4_matvec_experts and moe_sort take as no expert.  A
 * token with a NaN among the keys of its unmasked experts gets experts -1 and
 * weights NaN; what stands in masked places does not matter.
 *   logits    device, [T][E]: bf16, or fp32 with MX_ROUTE_F32
 *   bias      device, fp32 [E] or NULL
 *   T, E      1 <= T <= 2^23, 1 <= E <= 1024, T * E <= 2^40
 *   top       1 <= top <= 64, top <= E; 1 <= groups <= 64 divides E,
 *             1 <= top_groups <= groups
 *   scale     finite
 *   experts   int32 [T][top];  weights  fp32 [T][top]
 *   scores    fp32 [T][E], p itself (for a balance loss), or NULL
 * Errors: MX_ERR_ENUM for an unknown flag or a scale that is not finite,
 * MX_ERR_SHAPE for a size outside these; the others as for the casts (logits,
 * experts, weights and scores 16-byte aligned, bias 4-byte).
 */
#define MX_ROUTE_SIGMOID 1u
#define MX_ROUTE_RENORM 2u
#define MX_ROUTE_GROUP_PAIR 4u
#define MX_ROUTE_F32 8u
mx_status moe_route(const void *logits, const float *bias, int64_t T, int64_t E, int64_t top,
                    int64_t groups, int64_t top_groups, float scale, unsigned flags,
                    int32_t *experts, float *weights, float *scores, hipStream_t stream);

/*
 * The gradient of a router's logits (the choice itself has none, nor has the
 * bias): from the gradients of the weights and, with dscores, of the scores.
 *   logits, T, E, top, scale, flags  as for moe_route (MX_ROUTE_GROUP_PAIR may
 *             be set and changes nothing)
 *   experts   int32 [T][top] as moe_route chose them; an index outside 0 .. E - 1
 *             is no expert, one named twice counts twice
 *   dweights  fp32 [T][top];  dscores  fp32 [T][E] or NULL
 *   dlogits   [T][E], of the logits' type
 * Where p is NaN so is the gradient; a masked logit (-Inf) has gradient 0, whatever
 * stands in its dscores.  With MX_ROUTE_RENORM the weights' part is exactly 0 where
 * one choice is live.
 */
mx_status moe_route_backward(const void *logits, const int32_t *experts, const float *dweights,
                             const float *dscores, int64_t T, int64_t E, int64_t top, float scale,
                             unsigned flags, void *dlogits, hipStream_t stream);

/*
 * The order of the tokens' rows by expert.  A slot is a (token, choice) pair, in
 * the order of experts[T][top]; each expert's rows are its slots in that order,
 * the experts one after the other, each from a multiple of `align` rows on (the
 * rows that mx_quantize_grouped and mx_matmul_grouped take, with group_rows[e] =
 * counts[e] rounded up to align).
 *   experts   device, int32 [T][top]; an index outside 0 .. E - 1 is no expert
 *   T, top    >= 1, top <= 64, T * top <= 2^23;  1 <= E <= 1024;  1 <= align <= 4096
 *   rows      rows the caller has room for: at least moe_sort_rows(T, top, E,
 *             align), at most 2^24
 *   counts    int32 [E]: the slots of each expert (padding not among them)
 *   pos       int32 [T][top]: each slot's row, -1 without an expert
 *   slots     int32 [rows]: each row's slot; -1 for padding and for rows behind
 *             the last expert's
 *   workspace, workspace_bytes  device scratch of at least
 *             moe_sort_workspace_size() bytes (0 for few slots: NULL and 0 then);
 *             calls that may overlap in time need workspaces of their own
 * Errors as for the products (every pointer 16-byte aligned).
 */
mx_status moe_sort(const int32_t *experts, int64_t T, int64_t top, int64_t E, int64_t align,
                   int64_t rows, int32_t *counts, int32_t *pos, int32_t *slots, void *workspace,
                   size_t workspace_bytes, hipStream_t stream);

/* The most rows that T * top slots of E experts can take, T * top +
 * min(E, T * top) * (align - 1), and moe_sort's workspace in bytes (each 0 for
 * invalid arguments). */
int64_t moe_sort_rows(int64_t T, int64_t top, int64_t E, int64_t align);
size_t moe_sort_workspace_size(int64_t T, int64_t top, int64_t E);

/*
 * The tokens' rows in that order: row r of out is row slots[r] / top of x, or
 * zeros where slots[r] is outside 0 .. T * top - 1.  Rows are bytes of any type
 * (bf16, or the codes and compact scales of a row-wise cast).
 *   x         device, [T] rows of row_bytes;  out  [rows] of them
 *   slots     device, int32 [rows], as moe_sort gives it; any values
 *   T, top    as for moe_sort; 1 <= rows <= 2^24; 1 <= row_bytes <= 2^24,
 *             row_bytes * max(rows, T) <= 2^41
 * Its gradient is moe_combine without weights.
 */
mx_status moe_gather(const void *x, int64_t T, int64_t top, const int32_t *slots, int64_t rows,
                     int64_t row_bytes, void *out, hipStream_t stream);

/*
 * The experts' rows back to their tokens:
 *   out[t][k] = bf16(sum_j weights[t][j] y[pos[t][j]][k]), summed in fp32 in the
 * order of j; a slot whose pos is outside 0 .. rows - 1 adds nothing.
 *   y         device, bf16 [rows][K]
 *   pos       int32 [T][top], as moe_sort gives it (any values), or NULL: slot i
 *             is row i, the layout of nvfp4_matvec_experts' output; rows = T * top
 *             then
 *   weights   fp32 [T][top] or NULL (ones)
 *   T, top, rows  as for moe_gather; K and the products T * K, rows * K as for
 *             mx_quantize
 *   out       bf16 [T][K]
 */
mx_status moe_combine(const void *y, int64_t rows, int64_t K, const int32_t *pos,
                      const float *weights, int64_t T, int64_t top, void *out, hipStream_t stream);

/*
 * Its gradients:
 *   dy[r][k]       = bf16(weights[s] dout[t][k]) for the row r of slot s = (t, j)
 *   dweights[t][j] = sum_k dout[t][k] y[r][k], in fp32; 0 for a slot without a row
 *   pos, slots  device, both as moe_sort gives them, or both NULL (slot i is row
 *             i, rows = T * top).  A row whose slot is outside 0 .. T * top - 1 gets
 *             zeros.  Row r is its slot's where pos[slots[r]] is r again; a row
 *             for which that is not so is left as it was (moe_sort gives none)
 *   weights   fp32 [T][top] or NULL (ones)
 *   dy        bf16 [rows][K]
 *   dweights  fp32 [T][top], or NULL: not computed
 */
mx_status moe_combine_backward(const void *dout, const void *y, int64_t rows, int64_t K,
                               const int32_t *pos, const int32_t *slots, const float *weights,
                               int64_t T, int64_t top, void *dy, float *dweights,
                               hipStream_t stream);

/* Static string naming a status code. */
const char *mx_status_str(int status);

/* MXCAST_ABI_VERSION of the built library. */
int mx_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MXCAST_H */
