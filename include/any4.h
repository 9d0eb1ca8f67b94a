/*
 * any4.h -- C ABI of libany4.so, the MI355X (gfx950) any4 dequantize-GEMM
 * (with plain int4, the any2 and any3 variants, the any4 quantiser, what
 * fine-tunes of such a layer need: low-rank adapters, activations in 8 bits
 * and the input's gradient, and feed-forward blocks of such layers, dense or of
 * experts).
 *
 * any4 (the 10100.com any4 explainer, section 二) stores each weight of a
 * row as a 4-bit index into that row's 16-entry bf16 lookup table; each
 * contiguous group of g weights of a row also has a scale alpha and an offset
 * beta (step 1, "分组缩放": g = 128 typical, accuracy holds to g = 1024).  A
 * weight is w = alpha * LUT_row[idx] + beta.  The matmul y = x * W^T runs at
 * the decode batch sizes M = 1..16 that the same page's section 三 targets.
 *
 * Conventions shared by every call
 *   - All data pointers are DEVICE pointers owned by the caller.  The library
 *     allocates nothing, keeps no global state and may be called from several
 *     host threads.  Buffers must stay alive until the work on `stream`
 *     completes.
 *   - bf16 values travel as uint16_t bit patterns.  Dense row-major arrays:
 *         idx     [N][K]    uint8, values 0..15 (only the low 4 bits are read)
 *         lut     [N][16]   bf16, lut[n][i] is the value of index i in row n
 *         alpha   [N][K/g]  bf16, scale of weights k in [j*g, (j+1)*g) of row n
 *         beta    [N][K/g]  bf16, offset of the same group
 *         x       [M][K]    bf16 activations
 *         y       [M][N]    bf16 output
 *         w       [N][K]    bf16 dequantised weights
 *   - packed: the indices, two per byte, in tiles of 16 rows x 128 k
 *     (any4_packed_bytes(N, K) bytes; the tile layout is the library's, made
 *     so that one tile is one 16-byte load per lane of a 64-lane wave):
 *         tile (b, c) covers rows 16b..16b+15 and k 128c..128c+127 and starts
 *         at byte (b * K/128 + c) * 1024;
 *         byte 16*l + i of a tile (lane l = 0..63, i = 0..15) holds, for row
 *         n = 16b + (l % 16) and k = 128c + 32*(l / 16) + 2i,
 *             idx[n][k] in bits 0..3 and idx[n][k+1] in bits 4..7;
 *         rows n >= N (the last block when N % 16 != 0) are zero bytes.
 *     Equivalently: take the row-major nibble packing P[n][j] = idx[n][2j] |
 *     idx[n][2j+1] << 4, pad N up to a multiple of 16 with zero rows, view it
 *     as [N/16][16][K/128][4][16] and store it transposed to
 *     [N/16][K/128][4][16][16].
 *   - Calls are asynchronous on `stream` (0 = the default stream).  They
 *     return before the GPU work finishes; device faults show up at the
 *     caller's next synchronisation.
 *   - Arguments are checked before anything is launched.  On any error
 *     nothing is launched and every output is left untouched.
 *   - Outputs must not overlap inputs.  They are fully overwritten (no
 *     accumulate mode).
 *   - K must be a multiple of 128.  Group size: g must be a positive multiple
 *     of 128 that divides K (g = 128 .. 1024 are the sizes tested).  Every
 *     buffer must be smaller than 2 GiB.
 *   - Alignment: x, idx, packed and w need 16-byte aligned base pointers;
 *     lut needs 16 bytes for any4_gemm and 2 for any4_dequant; alpha, beta and
 *     y need 2 bytes, except that any4_gemm reads alpha and beta with 16-byte
 *     loads and needs them 16-byte aligned.
 */
#ifndef ANY4_H
#define ANY4_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum any4_status {
    ANY4_OK = 0,
    ANY4_E_NULL = 1,      /* a required pointer is NULL                               */
    ANY4_E_SHAPE = 2,     /* a size is negative, K is not a multiple of 128, g is not a
                             positive multiple of 128, K % g != 0, K/g > 512 or M > 65535*64 (any4_gemm*),
                             or a buffer would be 2 GiB or larger                     */
    ANY4_E_ALIGN = 3,     /* a base pointer misses the alignment stated above          */
    ANY4_E_WORKSPACE = 4, /* workspace smaller than any4_gemm_workspace_size()         */
    ANY4_E_HIP = 5        /* the HIP runtime refused a query or a launch               */
} any4_status;

/*
 * any4_packed_bytes -- size in bytes of the packed tiles of an N x K weight
 * matrix: ceil(N/16) * 16 * K/2.  Returns 0 when N < 0, K < 0 or K % 128 != 0.
 */
size_t any4_packed_bytes(int64_t N, int64_t K);

/*
 * any4_pack -- pack 4-bit indices two per byte into the tile layout above.
 * The offline step before inference, the counterpart of the "weights laid out
 * ahead of time" that the explainer's section 三 describes for its kernel.
 *   idx     device, [N][K] uint8, read-only; bits 4..7 of each byte are ignored.
 *   packed  device, any4_packed_bytes(N, K) bytes, written (padding included).
 *   N, K    N >= 0, K >= 0, K % 128 == 0.  N*K == 0 is a no-op.
 * Errors: ANY4_E_SHAPE, ANY4_E_NULL, ANY4_E_ALIGN (idx or packed not 16-byte
 * aligned), ANY4_E_HIP.
 */
any4_status any4_pack(const uint8_t* idx, uint8_t* packed, int64_t N, int64_t K,
                      hipStream_t stream);

/*
 * any4_dequant -- materialise the bf16 weights (the explainer, section 二:
 * a lookup in the row's table; step 1: group scale and offset):
 *     w[n][k] = bf16_rne( fp32( alpha[n][k/g] * lut[n][idx[n][k]] + beta[n][k/g] ) )
 * The bf16 x bf16 product is exact in fp32, so the inner value is one fp32
 * rounding (nearest even) of the exact sum; the result is then rounded to bf16
 * (nearest even).  Bit-exact: there is one correct answer.
 *   packed, lut, alpha, beta  device, read-only, layouts above.
 *   w                         device, [N][K] bf16, written.
 *   N >= 0, K >= 0, g as above.  N*K == 0 is a no-op.
 * Errors: ANY4_E_SHAPE, ANY4_E_NULL, ANY4_E_ALIGN, ANY4_E_HIP.
 */
any4_status any4_dequant(const uint8_t* packed, const uint16_t* lut, const uint16_t* alpha,
                         const uint16_t* beta, uint16_t* w, int64_t N, int64_t K, int64_t g,
                         hipStream_t stream);

/*
 * any4_gemm_workspace_size -- bytes of device workspace with which any4_gemm
 * may split K over several workgroups for this shape, or 0 when it does not
 * split.  It splits when the weights give each CU one or two 16-row blocks
 * (N/16 between 256 and 512 on the 256 CUs of an MI355X), K is at least
 * 12288, and the x rows the kernel loads (M rounded up to 1, 2, 4, 8 or 16)
 * exceed four per block of a CU (M = 5..16 with one block, M = 9..16 with
 * two): then x, which every workgroup reads for its whole K, would cost more
 * than the weights.  The workspace then holds S*M*N fp32
 * partial sums (S = 4 / blocks per CU), added up in a fixed order.  For
 * M >= 128 (prefill) it is N*K*2 bytes: room for the dequantised layer (see
 * any4_gemm).  Other shapes, and invalid ones, give 0.
 */
size_t any4_gemm_workspace_size(int64_t M, int64_t N, int64_t K, int64_t g);

/*
 * any4_gemm -- y = x * W^T with W the any4 weights above.  Built for the
 * decode batches M = 1..16 of the explainer's section 三 (weights streamed
 * once, decoded in registers); larger M (prefill) also works: up to 48 rows
 * with the weights still streamed once (two or three 16-row slices of x per
 * decoded tile; for a few shapes, 16-row slices of x and y that each stream
 * the weights), beyond that a tiled matrix-core product over weight tiles
 * dequantised in on-chip memory.  From M = 128 on, given a workspace of
 * any4_gemm_workspace_size bytes, the layer is instead dequantised into the
 * workspace (the any4_dequant values exactly, w[n][k] at element n*K + k) and
 * y is one bf16 GEMM with fp32 accumulation from hipBLASLt (the library's
 * summation order; the bound below holds with its fp32 summation error);
 * should the library decline, the tiled kernel runs.  (That path uses the
 * library handle of the calling thread's current device: `stream` must belong
 * to it.)
 *     y[m][n] = bf16_rne( sum_k x[m][k] * w[n][k] )
 * Otherwise every weight is dequantised inside the kernel (the weights are
 * never written to memory) as bf16_rne(fp32(alpha * v + beta)), v the table value
 * as the kernel holds it: each table row is kept as f16 scaled by 2^-s, s
 * chosen so that the row's largest finite magnitude lies in [2^14, 2^15)
 * (and s >= -60).  A table value is therefore held exactly -- and w[n][k] is
 * exactly the any4_dequant value -- when it is 0, inf, NaN, or its binary
 * exponent is at least both (that of the row's largest finite magnitude) - 31
 * and -77.  Any other value v of the row (more than 2^31 below the row's
 * largest, or a bf16 subnormal) is rounded to the f16 grid of the scaled row,
 * an error of at most 2^(s-25) (values below that become 0).
 * The products are exact and the sum is fp32 (matrix-core accumulation), so,
 * for tables whose values are all held exactly, y differs from the fp64
 * product y_ref over the any4_dequant weights by the fp32 summation error and
 * y's own rounding to bf16 (at most 2^-8 * |y|); that is within
 *     |y - y_ref| <= 2e-3 * sum_k |x[m][k] * w[n][k]| + 1e-3
 * whenever |y| <= sum_k |x[m][k] * w[n][k]| / 2 (sums with cancellation, as
 * for activations and weights of both signs).  With values not held exactly,
 * each such weight adds at most |alpha| * 2^(s-25) to that error: negligible
 * where a row's small values are small in absolute terms (1.0 beside 2^-40 or
 * subnormals), not where a row's other values are needed beside a value
 * 2^39 times larger.  Runs are deterministic (same inputs, same bits): the
 * summation order depends only on the shape (on the prefill path, the
 * library GEMM's order, which this library does not control: its algorithm
 * is picked once per shape and process by timing the library's candidates
 * on the first eager call, so two processes may round differently;
 * environment ANY4_BLAS_TUNE=0 keeps the library's first choice).
 *   x                         device, [M][K] bf16, read-only.
 *   packed, lut, alpha, beta  device, read-only.
 *   y                         device, [M][N] bf16, written.
 *   M >= 0 (at most 65535*64), N >= 0, K >= 0 with K % g == 0 and K/g <= 512.
 *   M*N == 0 is a no-op; K == 0 writes y = 0 (x, packed, lut, alpha and beta
 *   may then be NULL).
 *   workspace, workspace_bytes  optional device scratch, 16-byte aligned,
 *       owned by the caller, contents need not be initialised.  With at least
 *       any4_gemm_workspace_size(M, N, K, g) bytes the call may split K over
 *       workgroups (a second kernel then adds the partial sums in split order,
 *       so results stay deterministic) or, for M >= 128, dequantise the layer
 *       into it; with NULL it uses kernels that need no scratch (same result
 *       bound, another summation order).  Calls that share one workspace
 *       must be ordered (e.g. one stream).
 * Errors: ANY4_E_SHAPE, ANY4_E_NULL, ANY4_E_ALIGN (also a misaligned
 * workspace), ANY4_E_WORKSPACE (a non-NULL workspace smaller than
 * any4_gemm_workspace_size), ANY4_E_HIP.
 */
any4_status any4_gemm(const uint16_t* x, const uint8_t* packed, const uint16_t* lut,
                      const uint16_t* alpha, const uint16_t* beta, uint16_t* y, int64_t M,
                      int64_t N, int64_t K, int64_t g, void* workspace, size_t workspace_bytes,
                      hipStream_t stream);

/*
 * any4_gemm_noalloc -- any4_gemm for callers that cannot allocate device
 * memory (code under HIP graph capture, serving loops that must not call the
 * allocator, harnesses that forbid it): the same arguments without the
 * workspace, the same kernels and the same result, bit for bit, as any4_gemm
 * given a workspace of any4_gemm_workspace_size(M, N, K, g) bytes for
 * M <= 16 (for larger M: as any4_gemm with no workspace).  Where that size
 * is not 0 (K split over workgroups), the partial sums go to a
 * 4 MiB array of device memory inside the library, one per GPU, held until
 * the process ends; its device address is looked up on the first such call
 * on each GPU (with that GPU current: `stream` must belong to the current
 * device).  Nothing is allocated per call and nothing needs clearing (every
 * partial sum is written before it is read).  Calls on one GPU that use the
 * array and can overlap in time (other streams, other threads) race on it:
 * order them, e.g. on one stream.
 * Errors: as any4_gemm; ANY4_E_WORKSPACE if the shape would need more than
 * the array's 4 MiB (the splitting shapes need at most 1 MiB); ANY4_E_HIP if
 * the array's address cannot be looked up.
 */
any4_status any4_gemm_noalloc(const uint16_t* x, const uint8_t* packed, const uint16_t* lut,
                              const uint16_t* alpha, const uint16_t* beta, uint16_t* y,
                              int64_t M, int64_t N, int64_t K, int64_t g, hipStream_t stream);

/*
 * any4_gemv_dot -- the M = 1 product (y = x * W^T with one row of x) computed
 * on the vector ALUs with v_dot2_f32_bf16 instead of the matrix cores: the
 * GEMV form of the decode-batch product (the explainer's section 三, batch
 * 1), kept beside any4_gemm to compare the two; any4_gemm is the faster and
 * is what any4_gemm uses at M = 1.  Same decode and dequantisation as
 * any4_gemm (so the same exactness condition and bound), x [1][K], y [1][N].
 * Shapes whose x does not fit the kernel's on-chip staging (2*K bytes above
 * 64 KiB with the weights' tables) return ANY4_E_SHAPE.
 * Errors: ANY4_E_SHAPE, ANY4_E_NULL, ANY4_E_ALIGN, ANY4_E_HIP.
 */
any4_status any4_gemv_dot(const uint16_t* x, const uint8_t* packed, const uint16_t* lut,
                          const uint16_t* alpha, const uint16_t* beta, uint16_t* y, int64_t N,
                          int64_t K, int64_t g, hipStream_t stream);

/*
 * any4_gemm_int4 -- the same product for plain asymmetric int4 weights, the
 * baseline the explainer compares any4 against (section 二: int4 is the fixed
 * table 0..15, with the group scale and offset of step 1):
 *     w[n][k] = bf16_rne( fp32( alpha[n][k/g] * q[n][k] + beta[n][k/g] ) )
 *     y[m][n] = bf16_rne( sum_k x[m][k] * w[n][k] )
 * q[n][k] is the 4-bit code in `packed` (same tile layout), read as 0..15.
 * The result is bit-identical to any4_gemm with every table row 0, 1, .., 15
 * and the same workspace (given or NULL), and carries the same error bound.
 * Arguments, sizes, alignment, workspace and errors as any4_gemm, without
 * lut.
 */
any4_status any4_gemm_int4(const uint16_t* x, const uint8_t* packed, const uint16_t* alpha,
                           const uint16_t* beta, uint16_t* y, int64_t M, int64_t N, int64_t K,
                           int64_t g, void* workspace, size_t workspace_bytes,
                           hipStream_t stream);

/*
 * any2 -- the 2-bit variant at 2 bits per stored weight (the paper's abstract
 * names any2): each weight is a 2-bit code into its row's table, of which
 * only entries 0..3 are read (a [N][16] bf16 table as everywhere else, e.g.
 * any4_quantize with bits = 2; entries 4..15 are ignored).  Codes are packed
 * four to a byte in tiles of 16 rows x 128 k (any2_packed_bytes(N, K)
 * bytes):
 *     tile (b, c) covers rows 16b..16b+15 and k 128c..128c+127 and starts at
 *     byte (b * K/128 + c) * 512;
 *     byte 8*l + i of a tile (lane l = 0..63, i = 0..7) holds, for row
 *     n = 16b + (l % 16) and k = 128c + 32*(l / 16) + 4i,
 *         code[n][k+s] in bits 2s..2s+1 (s = 0..3);
 *     rows n >= N are zero bytes.
 * Equivalently: row-major bytes P[n][j] = sum_s code[n][4j+s] << 2s, padded to
 * a multiple of 16 rows, viewed as [N/16][16][K/128][4][8] and stored as
 * [N/16][K/128][4][16][8].
 * any2_pack, any2_dequant and any2_gemm take the same arguments and follow
 * the same conventions, checks and errors as any4_pack, any4_dequant and
 * any4_gemm (the same optional workspace, sized by
 * any4_gemm_workspace_size), with idx read as codes 0..3 (bits above 1
 * ignored):
 *     w[n][k] = bf16_rne( fp32( alpha[n][k/g] * lut[n][code[n][k]] + beta[n][k/g] ) )
 *     y[m][n] = bf16_rne( sum_k x[m][k] * w[n][k] )   (same bound as any4_gemm)
 * Returns of any2_packed_bytes: ceil(N/16) * 16 * K/4, or 0 as any4_packed_bytes.
 */
size_t any2_packed_bytes(int64_t N, int64_t K);
any4_status any2_pack(const uint8_t* idx, uint8_t* packed, int64_t N, int64_t K,
                      hipStream_t stream);
any4_status any2_dequant(const uint8_t* packed, const uint16_t* lut, const uint16_t* alpha,
                         const uint16_t* beta, uint16_t* w, int64_t N, int64_t K, int64_t g,
                         hipStream_t stream);
any4_status any2_gemm(const uint16_t* x, const uint8_t* packed, const uint16_t* lut,
                      const uint16_t* alpha, const uint16_t* beta, uint16_t* y, int64_t M,
                      int64_t N, int64_t K, int64_t g, void* workspace, size_t workspace_bytes,
                      hipStream_t stream);

/*
 * any3 -- the 3-bit variant at 3 bits per stored weight (the paper's abstract
 * names any3): each weight is a 3-bit code into its row's table, of which
 * only entries 0..7 are read (entries 8..15 are ignored; any4_quantize with
 * bits = 3 writes such tables).  Codes are stored in tiles of 16 rows x 128 k
 * (any3_packed_bytes(N, K) bytes):
 *     tile (b, c) covers rows 16b..16b+15 and k 128c..128c+127 and starts at
 *     byte (b * K/128 + c) * 768;
 *     the 12 bytes 12*l .. 12*l+11 of a tile (lane l = 0..63) hold row
 *     n = 16b + (l % 16), k = 128c + 32*(l / 16) + 0..31, as 16 pair indices
 *         P_i = code[n][k+2i] | code[n][k+2i+1] << 3      (i = 0..15);
 *     byte j (j = 0..11) holds P_j in bits 0-5, and in bits 6-7 the two bits
 *     2*(j/4), 2*(j/4)+1 of P_{12 + j%4};
 *     rows n >= N are zero bytes.
 * (So dwords 0-2 of a lane's 12 bytes carry the pair indices of its first
 * three 32-k MFMA operands one per byte, and the fourth operand's are
 * gathered from the bytes' top bits: one load of 12 bytes per lane.)
 * any3_pack, any3_dequant and any3_gemm take the same arguments and follow
 * the same conventions, checks and errors as any2_pack, any2_dequant and
 * any2_gemm, with idx read as codes 0..7 (bits above 2 ignored):
 *     w[n][k] = bf16_rne( fp32( alpha[n][k/g] * lut[n][code[n][k]] + beta[n][k/g] ) )
 *     y[m][n] = bf16_rne( sum_k x[m][k] * w[n][k] )   (same bound as any4_gemm)
 * Returns of any3_packed_bytes: ceil(N/16) * 16 * 3K/8, or 0 as any4_packed_bytes.
 */
size_t any3_packed_bytes(int64_t N, int64_t K);
any4_status any3_pack(const uint8_t* idx, uint8_t* packed, int64_t N, int64_t K,
                      hipStream_t stream);
any4_status any3_dequant(const uint8_t* packed, const uint16_t* lut, const uint16_t* alpha,
                         const uint16_t* beta, uint16_t* w, int64_t N, int64_t K, int64_t g,
                         hipStream_t stream);
any4_status any3_gemm(const uint16_t* x, const uint8_t* packed, const uint16_t* lut,
                      const uint16_t* alpha, const uint16_t* beta, uint16_t* y, int64_t M,
                      int64_t N, int64_t K, int64_t g, void* workspace, size_t workspace_bytes,
                      hipStream_t stream);

/*
 * any4_quantize -- the any4 quantiser: turns weights into the idx, lut, alpha
 * and beta arrays above (the explainer, section 二: step 1, group scaling and
 * the calibration statistic E|x|; step 2, the E-step / M-step iteration that
 * learns each row's 16 table values, weighting each weight by alpha * E|x|).
 * bits = 3 or 2 gives any3 / any2 (the paper's abstract): Q = 8 or 4 table
 * values instead of Q = 16, stored in the first Q entries of the 16-entry
 * row (the rest zero), indices 0..Q-1, so such layers run through any4_pack,
 * any4_dequant and any4_gemm unchanged (at 4 bits per stored index).
 * Per row, in binary64 and in this order:
 *   1. per group of g weights: beta = bf16(min), alpha = bf16((max - min) /
 *      (Q - 1)) (the asymmetric range mapping that makes the start table
 *      0..Q-1 the plain uniform grid);
 *   2. ws = (w - beta) / alpha (0 where alpha == 0), wt = alpha * ex[k];
 *   3. L = 0, 1, .., Q-1, then `iters` rounds of: assign every weight to its
 *      nearest table value (ties: the lower index), then
 *      L[q] = sum(wt * ws) / sum(wt) over the members of q, summed in
 *      increasing k with products and sums rounded separately; a cluster
 *      without members keeps its value;
 *   4. lut = bf16(L), and idx = the nearest stored value for every weight.
 * The result is a deterministic function of the inputs.  One GPU thread
 * works through one row (the sums must run in k order), so this is an
 * offline step: milliseconds per layer.
 *   W      device, [N][K] fp32, read-only.
 *   ex     device, [K] fp32, E|x| of each input channel, read-only.
 *   idx    device, [N][K] uint8 (values 0..15), written; pack it with any4_pack.
 *   lut    device, [N][16] bf16, written.
 *   alpha, beta  device, [N][K/g] bf16, written.
 *   N >= 0, K >= 0, g > 0 with K % g == 0, iters >= 0, bits in 2..4,
 *   N*K < 2^31.  N*K == 0 is a no-op.
 * Errors: ANY4_E_SHAPE, ANY4_E_NULL, ANY4_E_ALIGN (W or ex not 4-byte aligned,
 * lut, alpha or beta not 2-byte aligned), ANY4_E_HIP.
 */
any4_status any4_quantize(const float* W, const float* ex, uint8_t* idx, uint16_t* lut,
                          uint16_t* alpha, uint16_t* beta, int64_t N, int64_t K, int64_t g,
                          int iters, int bits, hipStream_t stream);

/*
 * Low-rank adapters beside a layer, for many requests at once: row m of the
 * batch uses adapter a = ids[m] (a fine-tune of the frozen layer) on top of
 * the shared projection, whichever format that has:
 *     h[m]   = A_a x[m]                          (fp32, r values)
 *     out[m] = bf16_rne( y[m] + scale[a] * sum_j h[m][j] B_a[j] )
 *   x      [M][K] bf16            y, out  [M][N] bf16
 *   A      [L][r][K] bf16, B [L][r][N] bf16 (B rank-major: the transpose of the
 *          usual [N][r]); adapters of lower rank are padded with zero rows
 *   scale  [L] fp32               ids     [M] int32
 * A row whose id is not in 0..L-1 (-1, say) has no adapter: out[m] = y[m] bit
 * for bit, h[m] = 0.  Products are exact and sums fp32; the fp32 h enters the
 * second product unrounded, so out carries fp32 summation error and one
 * rounding.  Results are deterministic and a row's result depends on no other
 * row's values.  Infinities and NaN of x, y, dy, dx and scale give the h, out
 * and dx_out of the formulas, whatever r is.  A non-finite weight of an adapter
 * makes the outputs it reaches non-finite, and a non-finite row the gradients
 * of its adapter (which kind is not specified).
 * Sizes of all any4_lora* calls: 0 <= M <= 2^20, 0 <= N <= 2^24, K <= 2^24 a
 * positive multiple of 128, 1 <= r <= 128, 1 <= L <= 4096; x, y, A and B below
 * 2 GiB.
 * N, r and M need not be multiples of anything.
 */

/*
 * any4_lora_plan_bytes, any4_lora_plan -- the rows of a batch sorted by
 * adapter (stable), with the tables the kernels go by: `bytes` of device
 * memory at `plan`, 16-byte aligned.  The plan depends on ids alone, so a
 * program makes it once per batch and hands it to the calls of every layer;
 * calls without one make their own in the workspace (small batches, of at
 * most 64 rows, or 256 with few adapters in any4_lora, need none and ignore
 * it).  any4_lora_plan_bytes gives 0 for sizes out of range and M = 0.
 * M = 0 is a no-op.
 * Errors: ANY4_E_SHAPE, ANY4_E_NULL, ANY4_E_ALIGN, ANY4_E_WORKSPACE (bytes too
 * small), ANY4_E_HIP.
 */
size_t any4_lora_plan_bytes(int64_t M, int64_t L);
any4_status any4_lora_plan(const int32_t* ids, void* plan, size_t bytes, int64_t M, int64_t L,
                           hipStream_t stream);

/*
 * any4_lora -- out and, where asked for, what the backward pass needs.
 *   plan   device, of these ids, M and L; or NULL.  (A plan that any4_lora_plan
 *          made for another M > 0 or L leaves the outputs unwritten: its sizes
 *          are looked at before anything else of it is read.)
 *   out    device, written; may be y itself, else must not overlap an input.
 *   h      device, [M][r] fp32, written; or NULL.
 *   q, qs  device, x in 8 bits as any4_act8_save writes it, in the same pass
 *          over x (rows without an adapter too); or both NULL.
 *   workspace  device, 16-byte aligned, any4_lora_workspace_size(M, N, K, r, L)
 *          bytes, required where that is not 0 (it is 0 where the call needs
 *          none, for M = 0 and for sizes out of range); contents need not be
 *          initialised; calls that share one must be ordered.
 *   M = 0 is a no-op; N = 0 only writes h, q and qs (B, y, out may be NULL).
 *   x, A, plan, q and workspace need 16-byte alignment, the others that of
 *   their elements.
 * Errors: ANY4_E_SHAPE, ANY4_E_NULL, ANY4_E_ALIGN, ANY4_E_WORKSPACE, ANY4_E_HIP.
 */
size_t any4_lora_workspace_size(int64_t M, int64_t N, int64_t K, int64_t r, int64_t L);
any4_status any4_lora(const uint16_t* x, const uint16_t* A, const uint16_t* B, const float* scale,
                      const int32_t* ids, const void* plan, const uint16_t* y, uint16_t* out,
                      float* h, int8_t* q, float* qs, int64_t M, int64_t N, int64_t K, int64_t r,
                      int64_t L, void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * any4_lora_backward -- the gradients of any4_lora for dy = d loss / d out
 * (bf16 [M][N]):
 *     dh[m]     = scale[a] * B_a dy[m]                       (a = ids[m])
 *     dx_out[m] = bf16_rne( dx[m] + sum_j dh[m][j] A_a[j] )
 *     dA_a      = sum_{ids[m] = a} dh[m]^T x[m]              (fp32 [L][r][K])
 *     dB_a      = scale[a] * sum_{ids[m] = a} h[m]^T dy[m]   (fp32 [L][r][N])
 * with h as any4_lora wrote it.  The gradient of y is dy itself; dx is what
 * the shared projection's backward pass gave (any4_gemm_dx), NULL for zero.
 * dA and dB are written whole: an adapter without rows gets zeros.
 *   x      device, [M][K] bf16, or NULL with q, qs: x in 8 bits (its values
 *          q * qs enter dA unrounded).  x goes first where both are given.
 *   dx_out may be dx itself, else must not overlap an input.  dx_out, dA and
 *          dB may each be NULL: not wanted (x, q, qs are then not read without
 *          dA, h not without dB).
 *   plan, workspace  as for any4_lora, any4_lora_backward_workspace_size bytes.
 *   N >= 1; M = 0 writes dA = dB = 0 (the other pointers may be NULL).
 *   x, A, q, dx, dx_out, plan and workspace need 16-byte alignment, the others
 *   that of their elements.
 * Errors: as any4_lora.
 */
size_t any4_lora_backward_workspace_size(int64_t M, int64_t N, int64_t K, int64_t r, int64_t L);
any4_status any4_lora_backward(const uint16_t* dy, const uint16_t* x, const int8_t* q,
                               const float* qs, const float* h, const uint16_t* A,
                               const uint16_t* B, const float* scale, const int32_t* ids,
                               const void* plan, const uint16_t* dx, uint16_t* dx_out, float* dA,
                               float* dB, int64_t M, int64_t N, int64_t K, int64_t r, int64_t L,
                               void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * any4_act8_save, any4_act8_load -- an activation kept in 8 bits between the
 * forward and the backward pass, and read back: one fp32 scale per 128
 * channels of a row,
 *     amax = max |x|,  qs = fp32(amax / 127),  q = rint( fp32( x * fp32(127 / amax) ) )
 *     x'   = bf16_rne( fp32( q * qs ) )
 * (rint: nearest, ties to even).  Bit-exact: there is one correct answer.  A
 * group whose amax is below 2^-100 is kept as zeros (qs = 0); a group with an
 * infinity or NaN has a non-finite qs and reads back as non-finite values.
 *   x  device, [M][K] bf16    q  device, [M][K] int8    qs  device, [M][K/128] fp32
 *   0 <= M <= 65535*64, K >= 0 a multiple of 128, x below 2 GiB.  M*K == 0 is a
 *   no-op.  x and q need 16-byte alignment, qs 4.
 * Errors: ANY4_E_SHAPE, ANY4_E_NULL, ANY4_E_ALIGN, ANY4_E_HIP.
 */
any4_status any4_act8_save(const uint16_t* x, int8_t* q, float* qs, int64_t M, int64_t K,
                           hipStream_t stream);
any4_status any4_act8_load(const int8_t* q, const float* qs, uint16_t* x, int64_t M, int64_t K,
                           hipStream_t stream);

/*
 * any4_gemm_dx, any4_gemm_int4_dx, any2_gemm_dx, any3_gemm_dx -- the gradient
 * of a quantised layer's input (the layer itself is frozen):
 *     dx[m][k] = bf16_rne( sum_n dy[m][n] * w[n][k] )
 * with w the values of any4_dequant (any2_dequant, any3_dequant; plain int4 as
 * any4_gemm_int4 reads it), exact products and fp32 sums.  Deterministic: the
 * order of a sum depends only on the shape.
 *   dy     device, [M][N] bf16    dx  device, [M][K] bf16, written whole
 *   packed, lut, alpha, beta  as for the format's dequantisation.
 *   workspace  device, 16-byte aligned, any4_gemm_dx_workspace_size(M, N, K, g)
 *          bytes (any format; 0 for sizes out of range and empty ones),
 *          required; contents need not be initialised; calls that share one
 *          must be ordered.
 *   0 <= M <= 65535*64, 0 <= N <= 2^21, K >= 0 and g as for any4_gemm (K/g is not
 *   limited).  Every buffer but the workspace below 2 GiB.  M*K == 0 is a
 *   no-op; N = 0 writes dx = 0 (the other pointers may be NULL).
 *   dx, packed and workspace need 16-byte alignment, the others 2 (dy with 16
 *   and N a multiple of 64 is read in place, else through a padded copy).
 * Errors: ANY4_E_SHAPE, ANY4_E_NULL, ANY4_E_ALIGN, ANY4_E_WORKSPACE, ANY4_E_HIP.
 */
size_t any4_gemm_dx_workspace_size(int64_t M, int64_t N, int64_t K, int64_t g);
any4_status any4_gemm_dx(const uint16_t* dy, const uint8_t* packed, const uint16_t* lut,
                         const uint16_t* alpha, const uint16_t* beta, uint16_t* dx, int64_t M,
                         int64_t N, int64_t K, int64_t g, void* workspace, size_t workspace_bytes,
                         hipStream_t stream);
any4_status any4_gemm_int4_dx(const uint16_t* dy, const uint8_t* packed, const uint16_t* alpha,
                              const uint16_t* beta, uint16_t* dx, int64_t M, int64_t N, int64_t K,
                              int64_t g, void* workspace, size_t workspace_bytes,
                              hipStream_t stream);
any4_status any2_gemm_dx(const uint16_t* dy, const uint8_t* packed, const uint16_t* lut,
                         const uint16_t* alpha, const uint16_t* beta, uint16_t* dx, int64_t M,
                         int64_t N, int64_t K, int64_t g, void* workspace, size_t workspace_bytes,
                         hipStream_t stream);
any4_status any3_gemm_dx(const uint16_t* dy, const uint8_t* packed, const uint16_t* lut,
                         const uint16_t* alpha, const uint16_t* beta, uint16_t* dx, int64_t M,
                         int64_t N, int64_t K, int64_t g, void* workspace, size_t workspace_bytes,
                         hipStream_t stream);

/*
 * The feed-forward block around a quantised layer, dense or of many experts:
 * bias, activation, gate and residual in the product's epilogue, a router, the
 * experts' products and the sum that the router weights.  What lies between two of
 * these calls (z, an output that any4_combine or any4_act_backward reads, an input's
 * gradient) is bf16, or where the argument behind it (z_f32, out_f32, ..) is not 0 fp32, in
 * the same shape and with an alignment of 4: then it is not rounded in between.
 * Rows that enter a matrix product are bf16.  So that they need not be rounded to
 * 8 bits either, the outputs and inputs that say so may be in two bf16 parts (the
 * argument behind them ANY4_PARTS, which no truth value is): a tensor [2][..] of the hi
 * parts, each value cut to bf16, and the lo parts, bf16_rne(value - hi); hi + lo is
 * the value but for 2^-16 of it at most.  An infinity has a lo of 0.  A product takes both
 * parts of a row, for twice the matrix work.
 */
enum { ANY4_PARTS = -1 };
typedef enum any4_format {
    ANY4_FORMAT_ANY4 = 0, /* any4_pack, lut of 16 entries              */
    ANY4_FORMAT_INT4 = 1, /* any4_pack, plain codes 0..15, lut not read */
    ANY4_FORMAT_ANY2 = 2, /* any2_pack, lut entries 0..3               */
    ANY4_FORMAT_ANY3 = 3  /* any3_pack, lut entries 0..7               */
} any4_format;

typedef enum any4_activation {
    ANY4_ACT_NONE = 0,     /* z                                              */
    ANY4_ACT_RELU = 1,     /* max(z, 0)                                      */
    ANY4_ACT_SILU = 2,     /* z / (1 + e^-z)                                 */
    ANY4_ACT_GELU = 3,     /* z (1 + erf(z / sqrt 2)) / 2                    */
    ANY4_ACT_GELU_TANH = 4 /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
} any4_activation;

/*
 * any4_gemm_act -- a layer's product with what surrounds it:
 *     zf[m][n] = sum_k x[m][k] w[n][k] + bias[n]          (fp32, w the any4_dequant values)
 *     out[m][n] = bf16_rne( act(zf[m][n]) + residual[m][n] )
 * or with gate != 0, the layer's N rows being [gate; up] of N/2 each:
 *     out[m][n] = bf16_rne( act(zf[m][n]) * zf[m][N/2 + n] + residual[m][n] ),  n < N/2
 * The weights are exactly the any4_dequant values, products are exact and sums
 * fp32, nothing is rounded in between.  z, where asked for, is bf16_rne(zf) (or zf itself):
 * what any4_act_backward needs.  Non-finite z give what the formulas give (act(-inf)
 * may be NaN).  Deterministic; a row's result depends on no other row's values.
 *   x         device, [M][K] bf16      bias  device, [N] bf16, or NULL
 *   residual  device, [M][No] bf16, or NULL; may be out itself where that is bf16 (No = N, gated N/2)
 *   z         device, [M][N] bf16 or fp32, written; or NULL
 *   out       device, [M][No] bf16 or fp32, written
 *   packed, lut, alpha, beta  as for the format's dequantisation.
 *   0 <= M <= 2^20, N >= 0 (even with a gate), K a positive multiple of 128, g as for
 *   any4_gemm (K/g is not limited); M*N and M*K below 2^30, N*K (N rounded up to a
 *   multiple of 16) below 2^32.
 *   M*N == 0 is a no-op.
 *   workspace  device, 16-byte aligned, any4_gemm_act_workspace_size(M, N, K, g)
 *          bytes, required where that is not 0; contents need not be
 *          initialised; calls that share one must be ordered.
 *   x, packed and workspace need 16-byte alignment, the others 2.
 * Errors: ANY4_E_SHAPE (also an unknown format or activation), ANY4_E_NULL,
 * ANY4_E_ALIGN, ANY4_E_WORKSPACE, ANY4_E_HIP.
 */
size_t any4_gemm_act_workspace_size(int64_t M, int64_t N, int64_t K, int64_t g);
any4_status any4_gemm_act(any4_format format, const uint16_t* x, const uint8_t* packed, const uint16_t* lut,
                          const uint16_t* alpha, const uint16_t* beta, const uint16_t* bias,
                          const uint16_t* residual, void* z, int z_f32, void* out, int out_f32,
                          any4_activation act, int gate, int64_t M, int64_t N, int64_t K, int64_t g, void* workspace,
                          size_t workspace_bytes, hipStream_t stream);

/*
 * any4_act_backward -- the gradients of an epilogue for dy = d loss / d out,
 * from z as any4_gemm_act or any4_experts_gemm kept it:
 *     dz[m][n] = bf16_rne( dy[m][n] act'(z[m][n]) ), or with a gate
 *     dz[m][n] = bf16_rne( dy[m][n] z[m][N/2 + n] act'(z[m][n]) ),
 *     dz[m][N/2 + n] = bf16_rne( dy[m][n] act(z[m][n]) ),      n < N/2
 *     dbias[n] = sum_m of the same values before their rounding     (fp32)
 * (all rows' sum: the bias that many experts have of their own has its gradient from
 * any4_experts_bias_backward).  act' of ANY4_ACT_RELU is 0 at 0.  The gradient of x is any4_gemm_dx of dz, that of the
 * residual dy itself.
 *   dy  device, [M][No] bf16 or fp32    z  device, [M][N] bf16 or fp32
 *   dz  device, [M][N] bf16, written (may be z itself where that is bf16)
 *   dbias  device, [N] fp32, or NULL (workspace is then not used)
 *   0 <= M <= 2^20, 0 <= N <= 2^29, M*N below 2^30.  M = 0 writes dbias = 0.
 *   workspace  device, 16-byte aligned, any4_act_backward_workspace_size(M, N, gate)
 *          bytes, required with dbias where that is not 0.
 *   dy, z and dz need 2-byte alignment, dbias 4.
 * any4_act_backward_parts writes dz in two bf16 parts, [2][M][N] (not z itself), as
 * any4_experts_gemm_dx_parts takes it; all else is the same.
 * Errors: as any4_gemm_act.
 */
size_t any4_act_backward_workspace_size(int64_t M, int64_t N, int gate);
any4_status any4_act_backward(const void* dy, int dy_f32, const void* z, int z_f32, uint16_t* dz,
                              float* dbias, any4_activation act, int gate, int64_t M, int64_t N, void* workspace,
                              size_t workspace_bytes, hipStream_t stream);
any4_status any4_act_backward_parts(const void* dy, int dy_f32, const void* z, int z_f32, uint16_t* dz,
                                    float* dbias, any4_activation act, int gate, int64_t M, int64_t N, void* workspace,
                                    size_t workspace_bytes, hipStream_t stream);

/*
 * any4_route -- the experts of each token and their weights, from the router's
 * logits:
 *     s[t] = softmax(logits[t]) or sigmoid(logits[t])
 *     c[t] = s[t] + bias                        (a bias for balance: it chooses, it does not weight)
 *     of `groups` groups of E / groups experts, the top_groups stay whose two
 *     largest c have the largest sum (one-expert groups: whose c is largest; an
 *     expert that is out counts as -inf, a sum without a value too)
 *     ids[t] = the k experts of largest c among those that stay, largest first
 *     w[t][j] = scale * s[t][ids[t][j]], with renorm != 0 divided by the sum of the k
 * Experts are compared by c in 64 bits, without a bias by the logits themselves (the same
 * order); ties go to the lowest index.  An expert whose logit is -inf or NaN has a score of 0
 * and is never chosen, nor is one whose c is NaN or -inf (its score counts in the softmax's
 * sum all the same); where fewer than k are left, the remaining ids are -1 with weights of 0.  A logit of +inf counts as the largest
 * finite fp32 value.  With renorm, weights whose scores are all 0 are 0.
 *   logits  device, [T][E], fp32 or (logits_bf16 != 0) bf16
 *   bias    device, [E] fp32, or NULL
 *   w       device, [T][k] fp32, written       ids  device, [T][k] int32, written
 *   0 <= T <= 2^20, 1 <= E <= 1024, 1 <= k <= 64, groups in 1..64 that divide E,
 *   1 <= top_groups <= groups, k <= top_groups * E / groups, T*k <= 2^20.  T = 0 is a no-op.
 *   Alignment: that of the elements.
 * Errors: ANY4_E_SHAPE (also an unknown score), ANY4_E_NULL, ANY4_E_ALIGN, ANY4_E_HIP.
 */
typedef enum any4_score { ANY4_SCORE_SOFTMAX = 0, ANY4_SCORE_SIGMOID = 1 } any4_score;
any4_status any4_route(const void* logits, int logits_bf16, const float* bias, float* w, int32_t* ids,
                       any4_score score, int renorm, float scale, int64_t T, int64_t E, int64_t k,
                       int64_t groups, int64_t top_groups, hipStream_t stream);

/*
 * any4_route_backward -- dlogits (of the logits' type) from dw = d loss / d w, the
 * choice being constant: the derivative of w[t][j] above.  ids as any4_route
 * wrote them (outside 0..E-1: no expert; dw there is not used).
 *   dw  device, [T][k] fp32    dlogits  device, [T][E], written whole
 * Sizes and errors as any4_route.
 */
any4_status any4_route_backward(const float* dw, const void* logits, int logits_bf16, const int32_t* ids,
                                void* dlogits, any4_score score, int renorm, float scale, int64_t T,
                                int64_t E, int64_t k, hipStream_t stream);

/*
 * any4_experts_gemm -- any4_gemm_act through stacked layers: pair p = t*k + j goes
 * through expert e = ids[t][j],
 *     zf[p] = W_e x[per_pair ? p : t] + bias[e],   out[p] = bf16_rne( act(zf[p]) ) or gated
 * A pair whose id is not in 0..E-1 gives zeros (out and z).
 *   x       device, [T][K] bf16, or with per_pair != 0 [T*k][K]; then also, x_f32 being
 *           ANY4_PARTS, [2][T*k][K], the results of another such product in two parts; for
 *           up to 64 pairs, with any other x_f32 but 0, fp32, split into such parts here
 *   packed  device, the experts' packed layers one after another (each of
 *           any4_packed_bytes(N, K), or the format's)
 *   lut [E][N][16], alpha, beta [E][N][K/g], bias [E][N] bf16 (or NULL)
 *   ids     device, [T][k] int32
 *   plan    device, any4_lora_plan(ids, ..., T*k, E), which a program makes once for the
 *           products of a block; or NULL (made in the workspace; up to 64 pairs
 *           need none and ignore it).  A plan that any4_lora_plan made for other sizes
 *           leaves the outputs unwritten.
 *   z       device, [T*k][N] bf16 or fp32, written; or NULL
 *   out     device, [T*k][No] bf16 or fp32, or (out_f32 ANY4_PARTS) [2][T*k][No], written
 *   0 <= T*k <= 2^20, 1 <= E <= 1024, the other sizes as any4_gemm_act for M = T*k, or in M*K
 *   for the rows that x has (T without per_pair); the stacked arrays may be of any size.
 *   T = 0 and N = 0 are no-ops.
 *   workspace  as for any4_gemm_act, any4_experts_workspace_size(T, k, E, N, K, g) bytes
 *          (where the call makes its own plan or splits K), for an x in parts
 *          any4_experts_parts_workspace_size.
 *   x, packed, plan and workspace need 16-byte alignment, ids 4, the others 2.
 * Errors: as any4_gemm_act.
 */
size_t any4_experts_workspace_size(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K, int64_t g);
size_t any4_experts_parts_workspace_size(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K, int64_t g);
any4_status any4_experts_gemm(any4_format format, const void* x, int x_f32, int per_pair,
                              const uint8_t* packed, const uint16_t* lut, const uint16_t* alpha, const uint16_t* beta,
                              const uint16_t* bias, const int32_t* ids, const void* plan, void* z,
                              int z_f32, void* out, int out_f32, any4_activation act, int gate, int64_t T, int64_t k,
                              int64_t E, int64_t N, int64_t K, int64_t g, void* workspace,
                              size_t workspace_bytes, hipStream_t stream);

/*
 * any4_experts_bias_backward -- the gradient of any4_experts_gemm's bias:
 *     dbias[e][n] = sum of dz[p][n] over the pairs p with ids[p] = e     (fp32)
 * dz being any4_act_backward's values before their rounding, of the same dy, z, act and
 * gate.  Experts without a pair get zeros, pairs without an expert are left out.
 * Sums are fp32, in an order that the ids alone decide.
 *   dy  device, [T*k][No] bf16 or fp32    z  device, [T*k][N] bf16 or fp32, as kept
 *   dbias  device, [E][N] fp32, written whole      ids, plan  as any4_experts_gemm
 *   0 <= T*k <= 2^20, k >= 1, 1 <= E <= 1024, 0 <= N <= 2^28, T*k*N below 2^30.  T = 0 writes zeros.
 *   workspace  device, 16-byte aligned, any4_experts_bias_workspace_size(T, k, E, N) bytes,
 *          with a plan less by any4_lora_plan_bytes(T*k, E): none for up to 512 pairs.
 *   dy and z need 2-byte (fp32: 4-byte) alignment, ids and dbias 4, plan 16.
 * Errors: as any4_gemm_act.
 */
size_t any4_experts_bias_workspace_size(int64_t T, int64_t k, int64_t E, int64_t N);
any4_status any4_experts_bias_backward(const void* dy, int dy_f32, const void* z, int z_f32, const int32_t* ids,
                                       const void* plan, float* dbias, any4_activation act, int gate, int64_t T,
                                       int64_t k, int64_t E, int64_t N, void* workspace, size_t workspace_bytes,
                                       hipStream_t stream);

/*
 * any4_experts_gemm_dx -- the gradient of the rows that went through the experts:
 *     dx[p][k] = bf16_rne( sum_n dy[p][n] w_e[n][k] ),   e = ids[p]
 * A pair whose id is not in 0..E-1 gives zeros.  (The gradient of an x that k
 * pairs share is the sum of theirs: any4_combine without weights.)
 *   dy  device, [T*k][N] bf16 (read in place if 16-byte aligned and N % 8 == 0, else
 *       through a padded copy)      dx  device, [T*k][K] bf16 or fp32, written
 *   N >= 1; sizes, ids, plan and errors as any4_experts_gemm (here N is taken
 *   rounded up to a multiple of 8).
 *   workspace  device, any4_experts_dx_workspace_size(T, k, E, N, K, g) bytes, required.
 * any4_experts_gemm_dx_parts takes dy in two bf16 parts, [2][T*k][N], for twice the matrix work,
 * and any4_experts_dx_parts_workspace_size bytes; all else is the same.
 */
size_t any4_experts_dx_workspace_size(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K, int64_t g);
any4_status any4_experts_gemm_dx(any4_format format, const uint16_t* dy, const uint8_t* packed,
                                 const uint16_t* lut, const uint16_t* alpha, const uint16_t* beta,
                                 const int32_t* ids, const void* plan, void* dx, int dx_f32, int64_t T,
                                 int64_t k, int64_t E, int64_t N, int64_t K, int64_t g, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream);
size_t any4_experts_dx_parts_workspace_size(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K, int64_t g);
any4_status any4_experts_gemm_dx_parts(any4_format format, const uint16_t* dy, const uint8_t* packed,
                                       const uint16_t* lut, const uint16_t* alpha, const uint16_t* beta,
                                       const int32_t* ids, const void* plan, void* dx, int dx_f32, int64_t T,
                                       int64_t k, int64_t E, int64_t N, int64_t K, int64_t g, void* workspace,
                                       size_t workspace_bytes, hipStream_t stream);

/*
 * any4_combine, any4_combine_backward -- the experts' outputs as the router
 * weights them, and the gradients:
 *     out[t]   = bf16_rne( residual[t] + sum_j w[t][j] y[t][j] )
 *     dy[t][j] = bf16_rne( w[t][j] dout[t] ),   dw[t][j] = sum_n dout[t][n] y[t][j][n]
 * Sums are fp32, in the order of j.
 *   y   device, [T][k][N] bf16 or fp32       dy  device, [T][k][N] bf16
 *   w, dw  device, [T][k] fp32 (w NULL in any4_combine:
 *   weights of 1)     residual  device, [T][N] bf16, or NULL; may be out itself
 *   out, dout  device, [T][N] bf16.   dy or dw NULL: not wanted.  dy may be y itself where that is bf16.
 *   0 <= T <= 2^20, k >= 1, T*k <= 2^20, N >= 0, T*k*N below 2^30.  T*N == 0 is a no-op
 *   (with N = 0 dw gets zeros).  Alignment: that of the elements.
 * Errors: ANY4_E_SHAPE, ANY4_E_NULL, ANY4_E_ALIGN, ANY4_E_HIP.
 */
any4_status any4_combine(const void* y, int y_f32, const float* w, const uint16_t* residual,
                         uint16_t* out, int64_t T, int64_t k, int64_t N, hipStream_t stream);
any4_status any4_combine_backward(const uint16_t* dout, const void* y, int y_f32, const float* w,
                                  uint16_t* dy, float* dw, int64_t T, int64_t k, int64_t N, hipStream_t stream);

/*
 * any4_ffn_form -- a measurement aid, not part of the method: which kernel the products of
 * these sizes run, for tests that mean to reach one.  E = 0: any4_gemm_act of P rows; else
 * the experts' products of P pairs, back != 0 the input's gradient, parts != 0 of rows in two
 * parts.  Touches no GPU.
 *   form  host, 4 words: rows of a tile (0: the few-row kernel), waves of a workgroup, splits of
 *         the sum, 1 where the layer is laid out as bf16 first
 * Errors: ANY4_E_SHAPE, ANY4_E_NULL.
 */
any4_status any4_ffn_form(int64_t P, int64_t E, int64_t N, int64_t K, int back, int parts, int32_t* form);

/*
 * any4_read_probe -- a measurement aid, not part of the method: reads `bytes`
 * of device memory at `buf` once, with the GEMM kernels' loads (16 bytes per
 * lane, 1 KB per wave, non-temporal), one workgroup of 16 waves per CU, each
 * wave issuing its ceil(bytes / 4 MiB) loads (at most 16 at a time) at once,
 * and writes at most one word to `out`.  Its duration is the streaming-read
 * ceiling that the GEMM's bandwidth is compared with.  bytes: a multiple of
 * 1024, below 2 GiB (0: no-op).
 * Errors: ANY4_E_SHAPE, ANY4_E_NULL, ANY4_E_ALIGN (buf not 16-byte or out
 * not 4-byte aligned), ANY4_E_HIP.
 */
any4_status any4_read_probe(const void* buf, size_t bytes, uint32_t* out, hipStream_t stream);

/* A static, human-readable name for a status code (never NULL). */
const char* any4_status_string(any4_status s);

#ifdef __cplusplus
}
#endif

#endif /* ANY4_H */
