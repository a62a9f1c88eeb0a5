/*
 * lvq.h - C ABI of the MI355X (gfx950) Leech-lattice dequantize-plus-matvec
 * library, liblvq.so.
 *
 * What is computed.  Batch-1 (up to 4) decode-phase y = W x, where W is stored
 * as 2-bit-class weight codes.  The main format follows arXiv 2609.02652,
 * "Unfolding the Leech Lattice: Fused Multi-Shell Decoding and VRAM Layouts
 * for 2-Bit LLM Weights" (section 1, contributions C1 and C2): every block of
 * 24 weights of a row is a point of the Leech lattice Lambda24 from the ball of
 * shells m <= 12 (301 coordinate-permutation classes), one scale per row,
 * unfolded offline into a divergence-free bit-plane layout plus a small shared
 * class table, and read by a fused kernel with shifts, masks and one table
 * lookup per block.  Two comparison arms and a dense control come with it:
 * the BPDQ bit-plane format (model card "Qwen3-8B - 2-bit BPDQ (packed)",
 * sections Format and Kernels), a bitshift trellis (blog "Qwen3.8-27B on a 12
 * GB card", section "A trellis is a codebook you walk"), and an fp16 matvec.
 * Next to them stand the other operators of a decoder block: 4-bit weights with
 * group scales for the projections that do not stand two bits (fp16 or 8-bit x),
 * the root-mean-square norm of a residual stream and the gated activation, with
 * fp16 or 8-bit outputs that the 4-bit arm reads; the key/value cache in 4 bits and
 * the attention over it; a mixture-of-experts layer in the 4-bit weights.
 *
 * Conventions shared by every function.
 *   - Return value: LVQ_OK (0) or a negative LVQ_E_* code.  No exception or
 *     abort crosses the ABI.  lvq_strerror() names a code.
 *   - Ownership: the caller owns every buffer; the library never allocates,
 *     frees or keeps a pointer past the call.
 *   - Device functions take device pointers and a HIP stream (hipStream_t
 *     passed as void*; NULL is the null stream).  They validate every argument
 *     on the host first and enqueue nothing on failure; on success the work is
 *     enqueued asynchronously on that stream and the call returns without
 *     synchronizing.  A failed launch returns LVQ_E_HIP.
 *   - Activations x are fp16 (IEEE binary16 bit patterns as uint16_t),
 *     row-major [batch][cols]; outputs y are fp32, row-major [batch][rows];
 *     1 <= batch <= 4.  Accumulation is fp32.
 *   - Device pointers must be 16-byte aligned (LVQ_E_ALIGN otherwise).
 *   - rows >= 0 and cols >= 0; a zero dimension is legal and enqueues nothing
 *     except writing zeros to y when rows > 0.
 *   - Inputs are assumed finite; non-finite x or weights give IEEE results.
 */
#ifndef LVQ_H
#define LVQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  LVQ_OK = 0,
  LVQ_E_NULL = -1,      /* a required pointer is NULL */
  LVQ_E_SHAPE = -2,     /* rows/cols negative, not a required multiple, or too large */
  LVQ_E_ALIGN = -3,     /* a device pointer is not 16-byte aligned */
  LVQ_E_NOT_LEECH = -4, /* lvq_expand: a block is not a Leech lattice point */
  LVQ_E_NORM = -5,      /* lvq_expand: a lattice block lies beyond shell 12 */
  LVQ_E_BATCH = -6,     /* batch outside 1..4 */
  LVQ_E_HIP = -7,       /* a HIP call or kernel launch failed */
  LVQ_E_LAYOUT = -8     /* a block's class cannot be stored in the requested layout */
};

/* Element types of the arguments that say so. */
enum {
  LVQ_F32 = 0,  /* IEEE binary32 */
  LVQ_F16 = 1,  /* IEEE binary16 */
  LVQ_BF16 = 2, /* bfloat16 */
  LVQ_I8 = 3,   /* int8, -127..127, largest magnitude 127 */
  LVQ_E4M3 = 4  /* 8-bit float, 4 exponent and 3 mantissa bits, no infinities, largest 448 */
};

#define LVQ_NUM_CLASSES 302 /* 301 classes on shells 2..12 plus the origin */
#define LVQ_MAX_BATCH 4

/* Static, thread-safe description of a status code ("unknown status" for
 * values that are not LVQ codes). */
const char* lvq_strerror(int code);

/* After lvq_expand returned LVQ_E_NOT_LEECH or LVQ_E_NORM on this thread:
 * the row and block index of the first offending block.  Returns LVQ_E_NULL
 * for NULL pointers; (-1, -1) when the last call on this thread succeeded. */
int lvq_last_error_index(int* row, int* block);

/* ---------------------------------------------------------------------------
 * Leech format: class table, layout and the offline expander (host only).
 *
 * Coordinates.  A block is 24 integers in the sqrt(8)-scaled frame where
 * shell m holds the vectors of squared norm 16 m; the Leech lattice there is
 *   even type: all x_i even, {i : x_i = 2 mod 4} a Golay codeword, sum = 0 mod 8
 *   odd type:  all x_i odd,  {i : x_i = 3 mod 4} a Golay codeword, sum = 4 mod 8
 * with the extended Golay code generated by the cyclic code of
 * g(x) = 1 + x^2 + x^4 + x^5 + x^6 + x^10 + x^11 plus an overall parity bit
 * (coordinate 23).  The dequantized weight of coordinate j of block k in row r
 * is  w[r][24k + j] = scale[r] * x_j ; the last cols % 24 columns of a row are
 * an unquantized fp16 tail added without the scale (the row scale is applied,
 * then the unquantized tail is added: arXiv 2609.35465, section 5.1).
 *
 * Class.  The multiset of |x_j| (a coordinate-permutation class: 301 of them
 * on shells 2..12, paper section 1).  Class ids follow the canonical order:
 * id 0 is the origin, the others ascend by (m, |x| sorted descending).
 * A class has at most 5 distinct magnitudes, each <= 13.
 * ------------------------------------------------------------------------- */

/* The 302-entry class table, one little-endian uint64 per class id:
 * bytes 0..4 the ascending distinct magnitudes (padded with 0), bytes 5..6
 * zero, byte 7 = m | (parity << 7).  The same table is the first section of
 * every blob.  Returns LVQ_E_NULL for a NULL out. */
int lvq_class_table(uint64_t out[LVQ_NUM_CLASSES]);

/* Bytes of the packed blob for a rows x cols matrix, or 0 when rows or cols
 * is negative.  Blob layout (every section starts at a multiple of 256 bytes;
 * nb = cols / 24 blocks per row, tau = cols % 24 tail columns):
 *   table  uint64 [302]        the class table above
 *   codes  uint32 [rows][nb][3] code word w of block (r, k) holds coordinates
 *                               8w..8w+7 in 8 nibble "slots" n = 0..7; slot n
 *                               holds coordinate j = 8w + 2(n%4) + n/4, so the
 *                               two coordinates of slots v and v+4 are adjacent
 *                               columns:
 *            bits 4n..4n+2        table slot = rank + 1 (1..5), where rank is
 *                                 the index of |x_j| in the class's ascending
 *                                 distinct magnitudes
 *            bit (4n + 11) mod 32 1 if x_j >= 0, 0 if x_j < 0
 *   cls    uint16 [rows][nb]   class id of each block
 *   scale  fp16   [rows]
 *   tail   fp16   [rows][tau]
 * Logically a block is 112 bits (class, a sign plane and three rank planes of
 * 24 bits each); the layout above is that record, transposed. */
size_t lvq_layout_bytes(int rows, int cols);

/* Expand integer lattice blocks into the packed blob (CPU, deterministic,
 * no HIP call).
 *   coords  int8 [rows][cols/24][24] lattice coordinates
 *   scale   fp16 [rows] row scales
 *   tail    fp16 [rows][cols%24], may be NULL when cols % 24 == 0
 *   blob_out host buffer of lvq_layout_bytes(rows, cols) bytes
 * Errors: LVQ_E_NULL, LVQ_E_SHAPE, LVQ_E_NOT_LEECH (a block breaks the
 * membership rules), LVQ_E_NORM (a lattice block beyond shell 12); the first
 * offending block is reported by lvq_last_error_index().  On error the content
 * of blob_out is unspecified. */
int lvq_expand(const int8_t* coords, const uint16_t* scale, const uint16_t* tail,
               int rows, int cols, void* blob_out);

/* LP2 layout: two rank planes and the class inside the code record, for
 * blocks whose class has at most four distinct magnitudes and an id below 256
 * (every class of shells m <= 8).  The paper measures smaller in-VRAM layouts
 * than its served record (section 1, contribution C2: 5.51, 4.80, 4.34 and
 * 3.59 bits per weight); this packing is the library's.  Blob sections (each
 * at a multiple of 256 bytes): the class table u64 [302]; codes u32
 * [rows][nb][3] (12 bytes per block, no class section); scale fp16 [rows];
 * tail fp16 [rows][tau].  In code word w, coordinate j = 8w + 2v + h
 * (v = 0..3, h = 0, 1) has its rank (0..3, the index of |x_j| among the
 * class's ascending distinct magnitudes) at bits 2v+16h .. 2v+16h+1 and a
 * non-negative flag at bit 8+2v+16h; word 0's odd bits carry the class id:
 * id bit 2i at bit 9+2i and id bit 2i+1 at bit 25+2i (i < 4).  lvq_expand_lp2
 * returns LVQ_E_LAYOUT for a block outside that set (the first one is
 * reported by lvq_last_error_index); other errors as lvq_expand. */
size_t lvq_layout_bytes_lp2(int rows, int cols);
int lvq_expand_lp2(const int8_t* coords, const uint16_t* scale, const uint16_t* tail, int rows,
                   int cols, void* blob_out);

/* LP2X: LP2 for the whole ball.  The blocks LP2 cannot hold (a class with
 * five distinct magnitudes or an id of 256 or more: shells m >= 9, about
 * 0.1 % of blocks when P(m) ~ 2^-m) keep a zero LP2 record and go to an
 * exception side channel appended to the LP2 blob (the paper's sparse overlay,
 * contribution C2: where the exception stream enters, the rate curve turns):
 *   exc_off u32 [rows + 1]  first entry of each row (256-byte aligned section)
 *   exc     16-byte entries {block index | class id << 16, LP3 code words
 *           0..2 of the block as lvq_expand writes them}, rows in order,
 *           blocks ascending inside a row.
 * lvq_lp2x_exceptions counts those blocks (host; membership errors as
 * lvq_expand), lvq_layout_bytes_lp2x sizes the blob, lvq_expand_lp2x writes
 * it (LVQ_E_SHAPE if n_exceptions is not the count). */
int lvq_lp2x_exceptions(const int8_t* coords, int rows, int cols, size_t* n_exceptions);
size_t lvq_layout_bytes_lp2x(int rows, int cols, size_t n_exceptions);
int lvq_expand_lp2x(const int8_t* coords, const uint16_t* scale, const uint16_t* tail, int rows,
                    int cols, size_t n_exceptions, void* blob_out);

/* Direct layout: no class table and no class stream.  Every coordinate of a
 * Lambda24 point has the parity p of the block (all even or all odd), so
 * |x_j| = 2 e_j + p with e_j = 0..6 for the ball (|x_j| <= 13); the record
 * holds p, three bits of e_j and a sign per coordinate, and a coordinate pair
 * decodes into an fp16 pair with one rotate, one AND-OR and no lookup.  The
 * paper measures its layouts by their in-VRAM rate (section 1, contribution
 * C2); this 5.33-bit packing is the library's, the rate cost of a decode
 * without the predicated table.  Blob sections (each at a multiple of 256
 * bytes): codes u32 [rows][nb][4] (16 bytes per block) at offset 0; scale
 * fp16 [rows]; tail fp16 [rows][tau].  In a block record, p is bit 0 of word 0;
 * coordinate j (pair P = j/2, half h = j%2) lives in word P/3, view v = P%3:
 * bit f of e_j (f = 0..2) at bit (1 + f + 16h + 5v) mod 32 and the sign
 * (1 = negative) at bit (15 + 16h + 5v) mod 32; every other bit is zero.
 * lvq_expand_direct validates blocks and reports errors as lvq_expand. */
size_t lvq_layout_bytes_direct(int rows, int cols);
int lvq_expand_direct(const int8_t* coords, const uint16_t* scale, const uint16_t* tail, int rows,
                      int cols, void* blob_out);

/* One-hot layout: the rank of each coordinate as indicator masks instead of
 * binary rank planes.  The paper times a one-hot-mask layout beside its bit
 * planes and finds the planes smaller and faster at the same bandwidth
 * (section 1, contribution C2: 5.51 against 4.80 bits per weight); it prints
 * no bit format, so this packing is the library's.  Blob sections (each at a
 * multiple of 256 bytes): the class table u64 [302]; codes u32 [rows][nb][4]
 * (16 bytes per block); class ids u16 [rows][nb]; scale fp16 [rows]; tail
 * fp16 [rows][tau] (18 bytes per block, 6.0 bits per weight).  Word i
 * (0..3) of a block is the indicator mask of rank i + 1 (rank 0, the
 * smallest magnitude of the class, has no bit): coordinate 2P at bit P,
 * coordinate 2P + 1 at bit 16 + P (P = 0..11).  The spare bits 12..14 and
 * 28..30 of word i carry the signs (1 = negative) of pairs P = 3i .. 3i + 2:
 * coordinate 2P at bit 12 + P - 3i, coordinate 2P + 1 at bit 28 + P - 3i.
 * Bits 15 and 31 are zero.  Errors as lvq_expand. */
size_t lvq_layout_bytes_onehot(int rows, int cols);
int lvq_expand_onehot(const int8_t* coords, const uint16_t* scale, const uint16_t* tail, int rows,
                      int cols, void* blob_out);

/* Shape-gain variant of lvq_expand: gain_bits uint8 [rows][cols/24] (0 or 1;
 * LVQ_E_SHAPE otherwise) is stored in bit 15 of each block's class id.  Read
 * such a blob with lvq_gemv_gain only.  gain_bits may be NULL when there are
 * no blocks. */
int lvq_expand_gain(const int8_t* coords, const uint8_t* gain_bits, const uint16_t* scale,
                    const uint16_t* tail, int rows, int cols, void* blob_out);

/* ---------------------------------------------------------------------------
 * 48-bit block words (arXiv 2609.02652: the source method stores each
 * 24-weight block as a 47-bit index into the m <= 12 ball plus one gain bit,
 * and the paper unfolds these words into its GPU layouts at load time; quality
 * protocol, published results and validity envelope paragraphs).
 *
 * Word: bits 0..46 the index, bit 47 the gain bit, bits 48..63 zero.
 * Index order (this library's; the pages give none): a ball point is
 * x = r + 4z with r = 2c (even type) or r = 1 + 2c (odd type), c an extended
 * Golay codeword (bit i of the mask = coordinate i) and sum(z) even (even type)
 * or odd (odd type); points are ordered by type (even first), then by the
 * codeword's 12-bit message (generator rows x^i g(x) extended by parity, row i
 * for message bit i), then lexicographically by (x_0, ..., x_23).  Indices run
 * from 0 to 111,043,117,458,000 (the ball size).
 * ------------------------------------------------------------------------- */

/* Index of each block (host): coords int8 [nblocks][24] -> index_out uint64
 * [nblocks].  LVQ_E_NOT_LEECH / LVQ_E_NORM for a block that is not a ball
 * point (the block is not reported); LVQ_E_NULL for NULL pointers. */
int lvq_rank(const int8_t* coords, size_t nblocks, uint64_t* index_out);

/* ---------------------------------------------------------------------------
 * Device entry points (HIP, gfx950).
 * ------------------------------------------------------------------------- */

/* y[b][r] = sum_c w[r][c] * x[b][c] over a Leech blob (device copy of what
 * lvq_expand wrote for the same rows, cols).  The kernel stages x and the
 * class table in LDS, streams the code words once, decodes each coordinate
 * with the same shift/mask/byte-permute sequence whatever its class, and
 * accumulates in fp32.  The order in which a row is summed is fixed by its
 * columns alone, not by the launch geometry, so a row's result is the same bit
 * for bit whatever the row count or device size.  Limit: batch * cols <= 65536
 * (LVQ_E_SHAPE). */
int lvq_gemv(const void* blob, int rows, int cols, const uint16_t* x, float* y,
             int batch, void* stream);

/* Several Leech GEMVs over one x in one launch: the fusion of the q, k, v
 * projections, and of gate and up, that arXiv 2609.02652 measures (section 1,
 * contribution C4, and the conclusion): 144 launches per token of the 8B stack
 * instead of 252.
 *   n        number of matrices, 1..4 (LVQ_E_SHAPE otherwise)
 *   blobs    host array of n device blob pointers (lvq_expand output)
 *   rows     host array of n row counts, each >= 0, sum < 2^31
 *   cols     shared by all n matrices
 *   x        fp16 [batch][cols], shared
 *   y        host array of n device pointers, y[m] fp32 [batch][rows[m]]
 * The results are those of n separate lvq_gemv calls, bit for bit: every row
 * is summed in the same order.  The host arrays are read during the call
 * only.  LVQ_E_NULL for a NULL array or a NULL entry, LVQ_E_ALIGN for a
 * misaligned device pointer; other limits as lvq_gemv. */
#define LVQ_MAX_FUSED 4
int lvq_gemv_fused(int n, const void* const* blobs, const int* rows, int cols,
                   const uint16_t* x, float* const* y, int batch, void* stream);

/* No-weights control (arXiv 2609.02652, section 1 contribution C4 and the
 * related-work paragraph on performance models): the launch lvq_gemv makes
 * for this shape (same grid, workgroup size, x and class table staging,
 * instructions, waits and reduction) with every weight load (code words,
 * class ids, tail, row scale) issued against an empty buffer range: out of
 * range, each returns 0 without a memory request, so no weight byte is read.
 * Its time prices the launch geometry and the decode.  The zeros decode as
 * class 0 with scale 0 and tail 0, so y is +0.0 exactly for finite x.  With
 * cols < 24 (no whole block, only the tail) y is filled with zeros by a
 * plain fill kernel.  blob must still point at a device copy of the class
 * table (the first section of any blob); other arguments and errors as
 * lvq_gemv. */
int lvq_gemv_noweights(const void* blob, int rows, int cols, const uint16_t* x, float* y,
                       int batch, void* stream);

/* lvq_gemv over an LP2 blob (lvq_expand_lp2): the same kernel and launch
 * rule, the class read from the code record, one rank bit fewer per
 * coordinate; 12 bytes per block instead of 14.  Limits and errors as
 * lvq_gemv. */
int lvq_gemv_lp2(const void* blob, int rows, int cols, const uint16_t* x, float* y, int batch,
                 void* stream);

/* lvq_gemv over a direct-layout blob (lvq_expand_direct): the same kernel
 * and launch rule; one 16-byte load per block, no class table staged in LDS,
 * three VALU operations per coordinate pair before the dot product.  Limits
 * and errors as lvq_gemv. */
int lvq_gemv_direct(const void* blob, int rows, int cols, const uint16_t* x, float* y, int batch,
                    void* stream);

/* lvq_gemv over a one-hot blob (lvq_expand_onehot): the same kernel and
 * launch rule; a coordinate pair is the class's smallest magnitude plus, for
 * each rank mask, its indicator bits times that rank's step, then the signs:
 * about 15 VALU operations per pair against the bit planes' four.  Limits
 * and errors as lvq_gemv. */
int lvq_gemv_onehot(const void* blob, int rows, int cols, const uint16_t* x, float* y, int batch,
                    void* stream);

/* lvq_gemv over an LP2X blob, one launch: the LP2 kernel, whose waves also
 * decode their row's side-channel blocks (the LP3 code words of each entry,
 * lanes taking the entries in turn) into their accumulators before the
 * row's reduction.  n_exceptions is the count the blob was written with
 * (with 0 the blob reads as plain LP2).  Limits and errors as lvq_gemv. */
int lvq_gemv_lp2x(const void* blob, int rows, int cols, size_t n_exceptions, const uint16_t* x,
                  float* y, int batch, void* stream);

/* Shape-gain GEMV: lvq_gemv over a blob from lvq_expand_gain, each block's
 * weights multiplied by gain0 or gain1 as its gain bit says:
 *   w[r][24k + j] = scale[r] * gain[g(r, k)] * x_j   (the tail unscaled).
 * The pages give no gain levels; the caller supplies them (fp32).  Each code
 * word's partial sum is multiplied by its block's gain before it is added, so
 * results do not depend on the launch geometry either.  Limits as lvq_gemv. */
int lvq_gemv_gain(const void* blob, int rows, int cols, float gain0, float gain1,
                  const uint16_t* x, float* y, int batch, void* stream);

/* Load-time unfolding: words uint64 [nblocks] (device) -> coords_out int8
 * [nblocks][24] (device) and gain_out uint8 [nblocks] (device): the gain bit,
 * or 0xFF (with zero coordinates) for a word whose index is past the ball or
 * whose bits 48..63 are not zero.  One thread per word.  The first call on a
 * device uploads the index tables (about 1 MB, into device globals of the
 * library; no allocation) and waits for that copy; later calls are
 * asynchronous on `stream`. */
int lvq_unfold(const uint64_t* words, size_t nblocks, int8_t* coords_out, uint8_t* gain_out,
               void* stream);

/* Decode a Leech blob back to its integer coordinates, int8 [rows][cols/24][24]
 * (device, 16-byte aligned; blob as lvq_gemv): the inverse of lvq_expand on the
 * code section, through the same pair decode as the GEMV.  It is the check of
 * arXiv 2609.02652's quality protocol (the paragraph with Table 5): the
 * transcoding is a bijection of decoded content, checked on every block, so
 * decode followed by lvq_expand must give the blob back bit for bit.  One
 * thread per block, asynchronous on `stream`; LVQ_E_NULL, LVQ_E_ALIGN,
 * LVQ_E_SHAPE (negative sizes) before any launch. */
int lvq_decode(const void* blob, int rows, int cols, int8_t* coords_out, void* stream);

/* BPDQ arm (model card, section Format, "Elsewhere" layout):
 *   codes  uint32 [cols/16][rows]: column c of row r is the 2-bit code at bits
 *          2*(c%16)..2*(c%16)+1 of codes[c/16][r]; bit_i is bit i of that code
 *   coeffs fp16 [cols/256][3][rows]: (c0, c1, c2) of group c/256 and row r
 *   w[r][c] = c0 * bit_0 + c1 * bit_1 + c2
 * cols must be a multiple of 256, batch * cols <= 65536, the codes at most
 * 2 GiB (rows * cols / 4 bytes) and the staged x must fit one workgroup's LDS
 * (160 KiB on gfx950: at batch 1 up to 63,488 columns; at batch 2-4 the
 * batch * cols bound comes first); LVQ_E_SHAPE otherwise, before any launch. */
int bpdq_gemv(const uint32_t* codes, const uint16_t* coeffs, int rows, int cols,
              const uint16_t* x, float* y, int batch, void* stream);

/* Bitshift-trellis arm (blog, section "A trellis is a codebook you walk"; L=16
 * state bits, T=2 bits shifted in per weight, one weight per step):
 *   bits   uint32 [rows][cols/16]: 2-bit symbols read MSB-first, symbol k of a
 *          row at bits 31-2(k%16) .. 30-2(k%16) of word k/16
 *   table  fp16 [65536], scale fp16 [rows]
 * Every 256 columns (512 bits) form a tail-biting packet; the state of
 * symbol k is the 16-bit window of the packet's last 8 symbols ending at k
 * (newest symbol in the low bits, wrapping to the packet's end for k < 7), and
 * w[r][c] = scale[r] * table[state].  cols must be a multiple of 256 and
 * batch * cols <= 12288 (the table fills most of LDS). */
int trellis_gemv(const uint32_t* bits, const uint16_t* table, const uint16_t* scale,
                 int rows, int cols, const uint16_t* x, float* y, int batch,
                 void* stream);

/* Dense control, the FP16 matvec the quantized kernels are measured against
 * (arXiv 2609.02652, section 1, contribution C2: the served layout runs at
 * 2.15x an FP16 matvec; the FP16 arm's measured bandwidth is the paper's byte
 * bound): y = W x with W fp16 [rows][cols] row-major, fp32 accumulation.
 * cols must be a multiple of 8 and batch * cols <= 65536. */
int fp16_gemv(const uint16_t* W, int rows, int cols, const uint16_t* x, float* y,
              int batch, void* stream);

/* 4-bit weights with group scales: the arm for the projections that do not
 * stand two bits.  y[b][r] = sum_c w[r][c] * x[b][c] with
 *   w[r][c] = scale[r][c/group] * (q[r][c] - zero[r][c/group])
 *   codes  uint8 [rows][16 * ceil(cols/32)], two columns per byte: q of column
 *          c is bits 4*(c%2)..4*(c%2)+3 of byte c/2 of its row, 0..15 (read as
 *          32-bit words, column c is bits 4*(c%8)..+3 of word c/8).  Rows are
 *          padded to whole 16-byte units; the padding's content is ignored.
 *   scale  fp16 [rows][G], G = ceil(cols/group)
 *   zero   fp16 [rows][G], any finite value; NULL for 8 everywhere
 *   group  columns per scale: 32, 64, 128, 256, or 0 for one scale per row
 *          (G = 1); the last group of a row may be short
 * cols is any number with batch * cols <= 65536.  LVQ_E_SHAPE for any other
 * size or group, and when y overlaps an input.  The products of a group are
 * summed with the codes as they are and the zero is applied to the sum of x, so
 * an infinity in x gives NaN; other batch rows, and the other rows' results
 * where a scale or zero is not finite, are not touched by it.  A row's result is
 * the same from run to run and whatever the batch; the order of its sum depends
 * on the matrix's shape and the device. */
int q4_gemv(const uint8_t* codes, const uint16_t* scale, const uint16_t* zero, int group, int rows,
            int cols, const uint16_t* x, float* y, int batch, void* stream);

/* q4_gemv with x in 8 bits, as lvq_rms_norm and lvq_silu_mul write it:
 *   x        int8 or e4m3 [batch][cols], x_type LVQ_I8 or LVQ_E4M3
 *   x_scale  fp32 [batch][H], H = ceil(cols/x_group): the value of column c is
 *            x_scale[b][c/x_group] * x[b][c]
 *   x_group  32, 64, 128, 256, or 0 for one scale per batch row (H = 1)
 * int8 products are summed in 32-bit integers over 32 columns, then in fp32.
 * LVQ_E_SHAPE for any other x_type or x_group; otherwise as q4_gemv. */
int q4_gemv_q8(const uint8_t* codes, const uint16_t* scale, const uint16_t* zero, int group,
               int rows, int cols, const void* x, int x_type, const float* x_scale, int x_group,
               float* y, int batch, void* stream);

/* Mixture-of-experts layer of a few tokens in 4-bit weights:
 *   l = router x;  the `top` largest l are chosen, equal ones by the lower index
 *   w = exp(l) / sum exp(l), the sum over all experts, or with renormalize 1 over the chosen
 *   y = sum over the chosen e of w_e down_e (silu(gate_e x) * (up_e x))
 *   x            fp16 [tokens][hidden], tokens 0..LVQ_MAX_MOE_TOKENS, tokens * hidden <= 65536
 *   router       fp32, fp16 or bf16 (router_type) [experts][hidden], experts 1..512
 *   top          1..LVQ_MAX_MOE_TOP, at most experts
 *   gu_*         codes, scale, zero (or NULL) and group of [experts][2 inner][hidden] matrices
 *                as q4_gemv reads them, an expert's behind the other's; rows 0..inner - 1 are
 *                the gate's, the others up's
 *   down_*       the same of [experts][hidden][inner] matrices
 *   hidden, inner  1..65536, any numbers
 *   y            fp32 [tokens][hidden]
 *   ids_out, weights_out  int32 and fp32 [tokens][top], largest first; either may be NULL
 *   workspace    device, q4_moe_workspace bytes, its content of no account before and after;
 *                calls that may run at the same time need one each
 * Logits are summed in fp64 and compared as two fp32, the rounded value and the rest; sums
 * and weights are fp32, the weights from the rounded logits.  An activation is kept as two
 * fp16, the rounded value and the rest (22 bits), so one past 65504 makes its token's y NaN
 * (lvq_silu_mul's fp16 output is infinite there, and q4_gemv's y of it NaN), and one below
 * 2^-14 is off by 2^-36.  A NaN among a token's logits makes its weights NaN.  An
 * infinity in x gives NaN in its token.  Tokens do not affect each other's values, and the
 * result is the same from run to run; the order of its sums depends on the sizes, the
 * device and, for the sum over the experts, on which are chosen by the tokens together.
 * LVQ_E_SHAPE for any other size, a short workspace, or an output over an input or another
 * output; all pointers 16-byte aligned. */
#define LVQ_MAX_MOE_TOKENS 16
#define LVQ_MAX_MOE_TOP 16
size_t q4_moe_workspace(int tokens, int hidden, int inner, int experts, int top);
int q4_moe(const uint16_t* x, int tokens, int hidden, const void* router, int router_type,
           int experts, int top, int renormalize, const uint8_t* gu_codes,
           const uint16_t* gu_scale, const uint16_t* gu_zero, int gu_group,
           const uint8_t* down_codes, const uint16_t* down_scale, const uint16_t* down_zero,
           int down_group, int inner, float* y, int32_t* ids_out, float* weights_out,
           void* workspace, size_t workspace_bytes, void* stream);

/* Root-mean-square norm of a residual stream, between two projections:
 *   h = x + residual                       (fp32; h = x when residual is NULL)
 *   residual_out = h                       (rounded once; skipped when NULL)
 *   out = h * (mean_c(h^2) + eps)^-1/2 * weight
 *   x            fp32, fp16 or bf16 (x_type) [rows] rows of cols values,
 *                x_stride values from one row's start to the next's
 *                (x_stride >= cols)
 *   residual     [rows][cols] of residual_type (fp32, fp16 or bf16), or NULL
 *   residual_out [rows][cols] of residual_type, or NULL; may be residual itself
 *   weight       [cols] of weight_type (fp32, fp16 or bf16), or NULL for ones
 *   out          [rows][cols] of out_type: fp16 (rounded once from fp32), or 8
 *                bits, LVQ_I8 or LVQ_E4M3, with
 *   out_scale    fp32 [rows][H], H = ceil(cols/out_group), out_group 32, 64,
 *                128, 256 or 0 for one scale per row: with a the largest
 *                magnitude of the group's fp32 results and M the type's largest
 *                value (127 or 448), out_scale = a / M and the codes are the
 *                results times M / a, rounded to the nearest (ties to even).  A
 *                group whose a is below 2^-100 gets scale 0 and zero codes, one
 *                that holds a NaN or an infinity zero codes and a scale that is
 *                not finite.  NULL and out_group 0 for fp16.
 * The statistics and the results before the rounding are fp32, so a row with
 * values above about 1.8e19 has an infinite mean square and zeros as results, and
 * one whose values are all below about 1e-19 needs an eps above 0.  The
 * order of a row's sum of squares depends on cols, rows and the device: a row may
 * differ in the last bits of its fp32 results between calls of few and of many
 * rows, and is the same from run to run.  rows is any number >= 0, cols <= 32768;
 * with rows or cols 0 nothing is written, neither out_scale.  x needs the alignment
 * of its type only (it may be a slice of a wider buffer); every other pointer 16
 * bytes.  No output may overlap an input or another output, residual_out ==
 * residual excepted (LVQ_E_SHAPE). */
int lvq_rms_norm(const void* x, int x_type, int64_t x_stride, const void* residual,
                 int residual_type, void* residual_out, const void* weight, int weight_type,
                 float eps, int rows, int cols, void* out, int out_type, float* out_scale,
                 int out_group, void* stream);

/* Gated activation between the gate/up projections and the down projection:
 *   out = gate / (1 + exp(-gate)) * up        (fp32, rounded once; exp(-gate) is
 *         off by up to 2^-23 |gate| of it, and out is 0 for gates below -88.72,
 *         where it leaves the fp32 range)
 *   gate, up   fp32, fp16 or bf16 (in_type) rows of cols values, in_stride
 *              values apart (gate and up may be the halves of one matrix's
 *              output, in_stride = 2 * cols); in_stride >= cols
 *   out, out_type, out_scale, out_group as lvq_rms_norm
 * cols <= 65536, with one scale per row cols <= 32768; otherwise limits,
 * alignment (gate and up as x there) and errors as lvq_rms_norm. */
int lvq_silu_mul(const void* gate, const void* up, int in_type, int64_t in_stride, int rows,
                 int cols, void* out, int out_type, float* out_scale, int out_group,
                 void* stream);

/* ---------------------------------------------------------------------------
 * Key/value cache in 4 bits, in pages, and the attention that reads it: the other half
 * of a decoder layer, between the q/k/v projections and the output projection.
 *
 * The cache is described by a struct that is read during the call only; the buffers it
 * points at are the caller's.  Position p of sequence s lies in page table[s][p / page],
 * at p % page.  A page holds its tokens head by head, each head's in blocks of 16 tokens;
 * with g = dim / group groups of channels (1 for group 0), a block is
 *   uint8 [16][dim/2]  keys, token by token: channel 32 a + 8 b + i (b < 4, i < 8) is bits
 *                      4 f..4 f + 3, f = i / 2 + 4 (i % 2), of the 32-bit word a of
 *                      quarter b of the token's dim / 2 bytes
 *   uint8 [dim/2][16]  values: channels 32 a + p (low half) and 32 a + 16 + p (high half)
 *                      of token t are byte [16 a + p][t]
 *   fp16 [g][16][2]    scale and low end of the keys of each group and token
 *   fp16 [g][16][2]    of the values
 * The value of a code c is scale * c + low.
 * ------------------------------------------------------------------------- */
typedef struct {
  void* pool;           /* device, [pages] pages of lvq_kv_page_bytes bytes */
  const int32_t* table; /* device, [seqs][max_pages] page numbers */
  int pages, seqs, max_pages; /* >= 0; max_pages * page <= 2^30 */
  int kv_heads;         /* 1..1024 */
  int dim;              /* channels of a head: 64, 128 or 256 */
  int page;             /* tokens of a page: 16, 32, 64, 128, 256, 512 or 1024 */
  int group;            /* channels per scale: 32, 64, 128 or 256, at most dim; 0 for dim */
} lvq_kv_cache;

/* Bytes of a page, 0 for sizes that no cache has. */
size_t lvq_kv_page_bytes(int kv_heads, int dim, int page, int group);

/* Stores `tokens` tokens and rotates their queries.  Token i belongs to position pos[i] of
 * sequence seq[i] (seq NULL: of sequence i, one token of each).  The first rot channels of
 * every head of k and q are turned, in pairs (j, j + rot/2), j < rot/2, or with interleaved
 * 1 (2 j, 2 j + 1), by the angle whose cosine and sine are cos[pos][j] and sin[pos][j]:
 *   a' = a cos - b sin,  b' = b cos + a sin
 * (fp32, each product rounded before the sum).  Then keys and values are rounded to 4 bits,
 * per token, head and group of channels:
 *   scale = fp16((max - min) * fp32(1/15)),  low = fp16(min),
 *   code = (v - low) * (1 / scale) rounded to the nearest (ties to even), within 0..15,
 *   0 where the scale is 0
 * A group that holds an infinity or a NaN gets an infinite scale and reads as NaN, and one with
 * magnitudes past fp16's range an infinite scale or low end (NaN or infinities).
 *   k, v       fp32, fp16 or bf16 (type), [tokens] rows of kv_heads * dim values, k_stride
 *              and v_stride values from one row's start to the next's (< 2^31)
 *   seq, pos   device, int32 [tokens]
 *   cos, sin   device, fp32 [positions][rot/2]; rot a multiple of 16, at most dim, 0 for
 *              no rotation (NULL will do where rot or positions is 0)
 *   q, q_out   heads (0..1024; 0 for none) heads of dim channels per token: rows of `type`,
 *              q_stride apart, and fp16, bf16 or fp32 (q_out_type) [tokens][heads * dim]
 * A token whose sequence, position (negative, past the table of pages, or past `positions`
 * where there is a rotation) or page is out of range is left out: nothing of it is stored
 * and its row of q_out stays as it is.  No two tokens of a call may have the same place
 * (what it then holds is unspecified).  Nothing else in the pool changes.  k, v and q need the
 * alignment of their type, seq and pos of theirs, every other pointer 16 bytes.  The pool and
 * q_out may overlap no input and not each other (LVQ_E_SHAPE). */
int lvq_kv_append(const lvq_kv_cache* cache, const void* k, int64_t k_stride, const void* v,
                  int64_t v_stride, int type, const int32_t* seq, const int32_t* pos, int tokens,
                  const float* cos, const float* sin, int rot, int positions, int interleaved,
                  const void* q, int64_t q_stride, int heads, void* q_out, int q_out_type,
                  void* stream);

/* Reads `tokens` tokens back: k_out, v_out (either may be NULL) [tokens][kv_heads * dim] of
 * out_type (fp32, fp16 or bf16), the value of each code computed in fp32 and rounded once.
 * seq and pos as in lvq_kv_append; a token out of range reads as zeros. */
int lvq_kv_read(const lvq_kv_cache* cache, const int32_t* seq, const int32_t* pos, int tokens,
                void* k_out, void* v_out, int out_type, void* stream);

/* Causal attention of the last `queries` tokens of every sequence over the cache:
 *   out[s][i][h] = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale * q[s][i][h] . k_t)
 * over the positions t <= lens[s] - queries + i of sequence s (with window > 0 only the last
 * `window` of them), k and v those of key/value head h / (heads / kv_heads).
 *   q          fp16 or bf16 (q_type), rows of heads * dim values, q_stride apart, row
 *              s * queries + i for query i of sequence s
 *              (bf16: a head's values times a power of two are taken as fp16, so those below
 *              2^-17 of its largest are off by up to 2^-25 of it)
 *   heads      a multiple of kv_heads, at most 1024; queries 1..LVQ_MAX_QUERIES
 *   lens       device, int32 [seqs]: tokens of each sequence, the queries' own included
 *              (a length past the table counts as the table's end, a negative one as 0)
 *   scale      above 0, finite; times a query's magnitudes below 2^100 (past it, NaN)
 *   out        fp32, fp16 or bf16 (out_type) [seqs * queries][heads * dim]
 *   workspace  device, lvq_attend_workspace bytes, its content of no account before and
 *              after; calls that may run at the same time need one each
 * A query that sees nothing (a length of 0, or fewer tokens than queries before it) gets
 * zeros.  Tokens on pages outside the pool are not seen.  What no query of a sequence sees
 * has no effect on it, whatever it holds, nor has a NaN or an infinity that only its other queries
 * see; one that a query sees (in the query, or as a scale or low end of a token's keys or values,
 * in any of its groups) gives NaN in every channel.  Sums and weights are fp32, the weights times the
 * values' scales in two fp16 (22 bits, in a unit that goes by the largest scale so far, of
 * any query's tokens).  The result is the same from run to run; how a sequence is split, and
 * so the order of its sums, depends on its length, the cache's sizes, the window and the
 * device.  cache->seqs <= 65535. */
#define LVQ_MAX_QUERIES 16
size_t lvq_attend_workspace(const lvq_kv_cache* cache, int heads, int queries);
int lvq_attend(const lvq_kv_cache* cache, const void* q, int q_type, int64_t q_stride, int heads,
               int queries, const int32_t* lens, float scale, int window, void* out, int out_type,
               void* workspace, size_t workspace_bytes, void* stream);

/* Activation rotation before a GEMV whose weights are stored in a rotated
 * basis.  arXiv 2609.02652 (the incoherence-rotated basis; the paragraph on
 * the rotated basis and the shared-memory wall) fixes a Walsh-Hadamard
 * transform of each projection's whole input, held in one workgroup's shared
 * memory: the case m = 1 with no signs.  For widths that are not powers of two
 * the form is borrowed from another system, Mirai S, whose runtime rotation
 * the blog post "Qwen3.8-27B on a 12 GB card" gives in its section "What the
 * kernel does per token":
 *   y = (H kron Q)(S x),  n = K * m, K a power of two, 1 <= m <= 32,
 *   y[a*m + b] = K^-1/2 sum_c H[a][c] sum_d Q[b][d] s_(c*m+d) x_(c*m+d),
 *   H[a][c] = (-1)^popcount(a & c)  (the Sylvester Walsh-Hadamard matrix).
 *   x          fp16 [batch][n]; y fp16 [batch][n] (round to nearest even of
 *              the fp32 result); y may be x (in place) when m = 1, and must
 *              not overlap x when m > 1 (LVQ_E_SHAPE)
 *   sign_words uint32 [ceil(n/32)], device: bit j%32 of word j/32 set means
 *              coordinate j is negated; NULL for no signs
 *   q          fp32 [m][m] row-major, device; NULL for the identity (then m
 *              interleaved K-point transforms)
 * Arithmetic is fp32 in LDS: one workgroup per (batch row, b) transforms its
 * K-point sequence (for K >= 16 and m <= 8 reading its groups straight from
 * x; otherwise staging the row of x first), so 4 K bytes (+ 2 n + 64 for
 * the staged row) must fit in a CU's LDS.
 * LVQ_E_SHAPE if n < 0, m outside 1..32, n % m != 0, n / m not a power of two
 * or the row does not fit in LDS; LVQ_E_NULL for a NULL x or y when n > 0;
 * LVQ_E_ALIGN for a device pointer not 16-byte aligned; batch 1..4. */
int lvq_rotate(const uint16_t* x, const uint32_t* sign_words, const float* q, int n, int m,
               uint16_t* y, int batch, void* stream);

/* Rotation and GEMV in one launch: y = W (H kron Q)(S x), with the rotation
 * of lvq_rotate (same arguments, same arithmetic) computed by every workgroup
 * on its staged copy of x in LDS (the f32 buffer of the transform next to
 * it), while the first weight loads are in flight; then lvq_gemv's decode and
 * accumulation.  The result equals lvq_gemv(blob, ..., lvq_rotate(x), ...)
 * bit for bit.  cols = K m as in lvq_rotate and cols >= 24; LDS must hold
 * the class table, batch rows of x and 4 cols (+ 4 m^2 with Q) bytes
 * (LVQ_E_SHAPE otherwise: e.g. cols 25600 fits at batch 1).  Other
 * arguments and errors as lvq_gemv and lvq_rotate. */
int lvq_gemv_rotated(const void* blob, int rows, int cols, const uint32_t* sign_words,
                     const float* q, int m, const uint16_t* x, float* y, int batch, void* stream);

/* Introspection, not part of the method: the launch a Leech GEMV entry point
 * makes for a shape, without making it.  kind: 0 lvq_gemv, 1
 * lvq_gemv_rotated (with m as there), 2 lvq_gemv_direct, 3 lvq_gemv_onehot, 4
 * lvq_gemv_lp2, 5 lvq_gemv_gain, 6 lvq_gemv_noweights.  info_out (host, 5
 * ints): threads per workgroup, workgroups in the grid, blocks per lane per
 * item, register sets in the item ring, LDS bytes per workgroup.  The grid
 * comes from the occupancy of that kernel on the current device.  Returns 0,
 * LVQ_E_NULL, or the error the entry point would return for that shape
 * (LVQ_E_SHAPE also for rows < 1, cols < 24 or an unknown kind).  Enqueues
 * nothing and touches no device memory. */
int lvq_gemv_launch_info(int kind, int rows, int cols, int batch, int m, int* info_out);

/* Measurement hook, not part of the method: reads all `bytes` of `buf`
 * (device, 16-byte aligned, bytes a multiple of 4) once with the loads a
 * weight stream uses.  Each workgroup stores the XOR of the words it read
 * into its own word of sink (device, 4-byte aligned, LVQ_STREAM_SINK_WORDS
 * words the caller clears first), so the XOR of all sink words is the XOR of
 * all words of the buffer.  Its duration is the achievable read bandwidth a
 * GEMV over a blob of the same size is compared with.  Asynchronous on
 * `stream`; LVQ_E_NULL / LVQ_E_ALIGN on bad arguments, no launch then. */
#define LVQ_STREAM_SINK_WORDS 4096
int lvq_stream_read(const void* buf, size_t bytes, uint32_t* sink, void* stream);

/* Measurement hook, not part of the method: the read of lvq_stream_read with
 * the launch shape chosen by the caller, for a sweep that finds the fastest
 * plain read of a given byte count (the ceiling a GEMV is compared with).
 * threads: workgroup size, 256, 512 or 1024.  wgs_per_cu: 1..8 workgroups per
 * compute unit, grid-strided; 0 = enough workgroups for one trip per thread.
 * unroll: 16-byte loads in flight per thread per trip, 1, 2, 4 or 8.
 * nontemporal: 1 = non-temporal loads (as the weight streams), 0 = ordinary.
 * sink: device, 4-byte aligned, LVQ_STREAM_GEOM_SINK_WORDS words cleared by
 * the caller; the XOR of its words is the XOR of the buffer's words.  Other
 * arguments as lvq_stream_read.  LVQ_E_SHAPE for any other threads, unroll or
 * wgs_per_cu, or when the grid would need more workgroups than sink words;
 * nothing is launched then. */
#define LVQ_STREAM_GEOM_SINK_WORDS 65536
int lvq_stream_read_geom(const void* buf, size_t bytes, uint32_t* sink, int threads,
                         int wgs_per_cu, int unroll, int nontemporal, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LVQ_H */
