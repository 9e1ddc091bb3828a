/*
 * fa.h -- C ABI of the GB300 (sm_103a) exact-attention forward library.
 *
 * The operation is the FlashAttention-2 forward pass: for every batch b,
 * head h and query row i,
 *
 *     O[b,h,i,:] = sum_j softmax_j(scale * Q[b,h,i,:] . K[b,h,j,:]) * V[b,h,j,:]
 *     LSE[b,h,i] = ln sum_j exp(scale * Q[b,h,i,:] . K[b,h,j,:])
 *
 * over the allowed keys j (j < Sk; with causal, also j <= i).  Sources:
 *   - "FlashAttention-2 相比 FlashAttention-1，到底改了什么" (source walk-through),
 *     section "第二处源码差异：kernel 主循环怎么组织": the online-softmax loop
 *     with O = acc / l and the epilogue that writes O and LSE;
 *     section "第一处源码差异：launch grid 怎么铺": the problem parameters
 *     (batch, heads, query length) and the stream passed at launch;
 *   - "FlashAttention-2 — L3 Cross-Paper Synthesis", §3 item 4: causal
 *     masking with whole-block skipping above the diagonal.
 *
 * Conventions shared by every entry point:
 *   - Tensors are row-major and contiguous, [B, H, S, D] for Q, K, V and O,
 *     [B, H, Sq] for LSE.  bf16 means IEEE bfloat16 bit patterns.
 *   - Every pointer is a DEVICE pointer on the current CUDA device, owned and
 *     allocated by the caller, 16-byte aligned.  The library allocates no
 *     device memory, performs no host<->device copy and no synchronisation:
 *     each call enqueues its kernel on `stream` (a cudaStream_t; NULL means
 *     the legacy default stream) and returns.  The outputs are complete when
 *     the stream reaches the end of that kernel.
 *   - Arguments are checked before anything is launched; a bad argument
 *     returns its negative code and launches nothing.  A launch failure
 *     returns FA_ERR_CUDA (fa_strerror gives the CUDA text of the last one).
 *   - Calls are thread-safe; per-device lazily initialised state (the
 *     driver's tensor-map encoder, kernel attributes) is guarded.
 */
#ifndef FA_GB300_FA_H
#define FA_GB300_FA_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FA_OK = 0,
    FA_ERR_NULLPTR = -1,            /* a required pointer is NULL                    */
    FA_ERR_BAD_SHAPE = -2,          /* B, H, Sq or Sk < 1, or a size out of range    */
    FA_ERR_UNSUPPORTED_D = -3,      /* head dim other than 64 or 128                 */
    FA_ERR_UNSUPPORTED_CAUSAL = -4, /* causal with Sq != Sk, or causal not 0/1       */
    FA_ERR_MISALIGNED = -5,         /* a pointer is not 16-byte aligned              */
    FA_ERR_BAD_SCALE = -6,          /* scale not finite or not > 0                   */
    FA_ERR_CUDA = -7,               /* CUDA runtime / driver error                   */
    FA_ERR_TIMEOUT = -8,            /* a bounded on-chip wait gave up (status word)  */
    FA_ERR_ALIAS = -9,              /* an output overlaps an input or the other one */
    FA_ERR_BAD_WINDOW = -10,        /* window bound below -1, or band with Sq != Sk  */
    FA_ERR_WORKSPACE = -11,         /* workspace missing, misaligned or too small    */
    FA_ERR_SCRATCH_LIMIT = -12,     /* more scratch than the built-in buffer holds   */
    FA_ERR_BAD_MASK = -13,          /* mask heads not 1 or B * H, or pair stride < 1 */
    FA_ERR_BAD_PAGE = -14           /* page size not 16/32/64/128, or (status word) a
                                       page or position outside the cache             */
} fa_status;

/*
 * fa_fwd -- attention forward, O = softmax(scale * Q K^T [+ causal mask]) V,
 * plus LSE (natural log).  Walk-through "FlashAttention-2 相比
 * FlashAttention-1，到底改了什么", section "第二处源码差异：kernel 主循环怎么组织".
 *
 *   q       bf16 [B, H, Sq, D]   device, read only
 *   k, v    bf16 [B, H, Sk, D]   device, read only
 *   o       bf16 [B, H, Sq, D]   device, written (rows < Sq only)
 *   lse     fp32 [B, H, Sq]      device, written: ln sum_j exp(scale q.k_j)
 *   B, H    batch and heads, >= 1
 *   Sq, Sk  query and key lengths, >= 1; causal requires Sq == Sk
 *   D       head dimension, 64 or 128
 *   scale   softmax temperature applied to Q.K before max/exp; finite, > 0
 *   causal  0: every key; 1: key j allowed for query i iff j <= i
 *   stream  cudaStream_t to launch on (NULL = default stream)
 *
 * Errors: FA_ERR_NULLPTR, FA_ERR_MISALIGNED, FA_ERR_BAD_SHAPE,
 * FA_ERR_UNSUPPORTED_D, FA_ERR_UNSUPPORTED_CAUSAL, FA_ERR_BAD_SCALE,
 * FA_ERR_ALIAS before launch; FA_ERR_CUDA if the launch fails.
 * Accumulation is fp32; P is rounded to bf16 before P*V; O is rounded to
 * bf16 (round-to-nearest-even).  No atomics: results are bitwise
 * deterministic for a given input.
 */
int fa_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H,
           int Sq, int Sk, int D, float scale, int causal, void *stream);

/*
 * fa_fwd_window -- attention forward restricted to a band of keys around each
 * query: key j is allowed for query i iff  i - window_left <= j <= i + window_right.
 * A bound of -1 means unbounded on that side; window_right = 0 is causal, and
 * (window_left = W, window_right = 0) is causal sliding-window attention.
 * This is the sliding-window generalisation of causal block skipping named in
 * "FlashAttention-2 — L3 Cross-Paper Synthesis", §5 item 4: key tiles outside
 * every row's band are skipped whole, tiles crossing a band edge are masked.
 *
 * Arguments, layout, ownership and outputs are those of fa_fwd (O and LSE
 * over the allowed keys only).  A bounded window (either bound >= 0) needs
 * Sq == Sk, so every query row sees at least its own key.
 * Errors: those of fa_fwd, plus FA_ERR_BAD_WINDOW for a bound below -1 or a
 * bounded window with Sq != Sk.  fa_fwd(..., causal, ...) equals
 * fa_fwd_window(..., -1, causal ? 0 : -1, ...).
 */
int fa_fwd_window(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H,
                  int Sq, int Sk, int D, float scale, int window_left, int window_right,
                  void *stream);

/*
 * fa_fwd_blockmask -- attention forward over the key blocks a block mask keeps:
 * the "unified sparse-block-skip mechanism" into which "FlashAttention-2 — L3
 * Cross-Paper Synthesis", §5 item 4, generalises causal block skipping (the
 * sliding window and dilated patterns being instances).  Key j is allowed for
 * query i iff j < Sk, the band keeps it (i - window_left <= j <= i +
 * window_right, as in fa_fwd_window: -1 unbounded, (-1, 0) causal) and
 *     block_mask[m][i / FA_BLOCK_M][j / FA_BLOCK_N] != 0,
 * where m = 0 when mask_heads = 1 (one pattern for every head) and m = b*H + h
 * when mask_heads = B * H.  Key blocks a query block does not keep are never
 * loaded or multiplied.
 *
 *   block_mask  uint8 [mask_heads, ceil(Sq / FA_BLOCK_M), ceil(Sk / FA_BLOCK_N)]
 *               DEVICE pointer, read by the kernel (must stay valid until the
 *               stream passes it), any alignment, must not overlap O or LSE
 *   mask_heads  1 or B * H
 *   pair_stride >= 1, a scheduling hint that does not change the result: query
 *               blocks a and a + pair_stride are computed together (in groups
 *               of 2 * pair_stride blocks; the last blocks with their
 *               neighbours) and share the loads of the key blocks either keeps.
 *               1 suits masks whose neighbouring block rows keep like blocks
 *               (bands, local patterns); a dilated pattern with stride r wants r.
 * Other arguments, layout, ownership and outputs are those of fa_fwd_window.
 * A query row with no allowed key (its block row keeps nothing, or the band
 * leaves nothing of what it keeps) gets O = 0 and LSE = -inf.
 * Errors: those of fa_fwd_window, plus FA_ERR_NULLPTR for a null mask,
 * FA_ERR_BAD_MASK for mask_heads other than 1 or B * H or pair_stride < 1, and FA_ERR_ALIAS when
 * the mask overlaps O or LSE.  With every block kept it equals fa_fwd_window.
 */
#define FA_BLOCK_M 128
#define FA_BLOCK_N 128
int fa_fwd_blockmask(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H,
                     int Sq, int Sk, int D, float scale, int window_left, int window_right,
                     const unsigned char *block_mask, int mask_heads, int pair_stride, void *stream);

/*
 * fa_fwd_fp8 -- attention forward with 8-bit (e4m3) Q, K, V and per-tensor
 * scaling: the FP8 tensor-core path that "Architectural Innovations in
 * FlashAttention-2 and FlashAttention-3" names as FA3's throughput lever
 * (section 三, FA3 item (3)), with the loss of precision held in check by
 * scaling and mixed precision (section 四, item ③).
 *
 * Each of q, k, v is an e4m3 tensor (1 byte per element: sign, 4 exponent
 * bits with bias 7, 3 mantissa bits; 0x7F and 0xFF are NaN) whose real value
 * is code * descale_x; layouts are fa_fwd's ([B, H, S, D] row-major, device
 * memory, 16-byte aligned).  The call computes, for the dequantised inputs,
 *   O   = softmax(scale * Q K^T [+ causal mask]) V   (bf16 [B, H, Sq, D])
 *   LSE = natural-log row log-sum-exp of scale * Q K^T  (fp32 [B, H, Sq])
 * S accumulates in fp32; P is rounded to e4m3 (times a power of two) for the
 * P V product, which accumulates in fp32; O is rounded to bf16 once.
 * D must be 128.  causal as in fa_fwd (needs Sq == Sk).  Ownership and
 * launch semantics are fa_fwd's.
 * Errors: those of fa_fwd; FA_ERR_UNSUPPORTED_D for D != 128;
 * FA_ERR_BAD_SCALE when scale or a descale is not finite and > 0 (or their
 * product underflows or overflows fp32).
 */
int fa_fwd_fp8(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H,
               int Sq, int Sk, int D, float scale, int causal, float descale_q, float descale_k,
               float descale_v, void *stream);

/*
 * fa_fwd_splitkv -- attention for decode: a few query rows per head against a
 * long key/value sequence, with the keys of each head split across CTAs.
 * "FlashAttention-2 — L3 Cross-Paper Synthesis", §5 item 5 (decode needs
 * parallelism over the key/value sequence); the split-and-merge of v1's
 * num_splits in "FlashAttention-2 相比 FlashAttention-1，到底改了什么", section
 * "第一处源码差异：launch grid 怎么铺".  Each split s of a head produces
 * lse_s = ln sum_{j in s} exp(scale q.k_j) and the normalised partial o_s;
 * the merge is lse = ln sum_s exp(lse_s), o = sum_s exp(lse_s - lse) o_s.
 * Every query row sees every key (no mask).
 *
 *   q, k, v, o, lse, B, H, Sk, D, scale, stream: as fa_fwd
 *   Sq            1 .. 8 query rows per head
 *   num_splits    key ranges per head, 1 .. 256; <= 0 picks a count from the
 *                 problem size and the SM count (fa_splitkv_num_splits);
 *                 each range holds a multiple of 64 keys, so fewer ranges
 *                 may be used when Sk is short
 *   workspace     caller-owned DEVICE scratch of at least
 *                 fa_fwd_splitkv_workspace_bytes(...) bytes, 16-byte aligned,
 *                 not overlapping any other argument; it holds fp32 partial
 *                 results between the two kernels this call enqueues, and
 *                 must not be used by another call until the stream has run
 *                 past this one
 *   B * H         at most 65535
 *
 * Errors: those of fa_fwd (causal does not apply), FA_ERR_BAD_SHAPE for
 * Sq > 8, B*H > 65535 or num_splits > 256, FA_ERR_WORKSPACE for a missing,
 * misaligned or short workspace.  Deterministic; no atomics.  If an on-chip
 * wait gives up (fa_device_status then returns FA_ERR_TIMEOUT), the affected
 * partials are marked invalid and the merged O and LSE of their rows are NaN.
 */
int fa_fwd_splitkv(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H,
                   int Sq, int Sk, int D, float scale, int num_splits, void *workspace,
                   size_t workspace_bytes, void *stream);

/*
 * fa_fwd_splitkv_workspace_bytes -- bytes of workspace fa_fwd_splitkv needs for
 * these sizes and num_splits (<= 0: the automatic count); 0 for unsupported sizes.
 */
size_t fa_fwd_splitkv_workspace_bytes(int B, int H, int Sq, int Sk, int D, int num_splits);

/* fa_splitkv_num_splits -- the split count fa_fwd_splitkv picks automatically
 * for these sizes on the current device (or FA_ERR_BAD_SHAPE). */
int fa_splitkv_num_splits(int B, int H, int Sq, int Sk, int D);

/*
 * fa_fwd_splitkv_noalloc -- fa_fwd_splitkv for callers that cannot allocate
 * device memory.  The pages have no counterpart to this call: it exists for
 * callers such as a process whose device memory is all reserved up front by
 * another allocator (a cudaMalloc there fails or fragments that pool), or a
 * latency-critical path that must not take the implicit synchronisation and
 * driver locks that cudaMalloc/cudaFree can take.  It allocates nothing: the
 * scratch lives in a 16 MiB array inside this library's device image (every
 * GPU that loads the library holds it until the process exits).
 *
 * Arguments and results are those of fa_fwd_splitkv without the workspace;
 * the caller still provides q, k, v, o and lse.  Every call looks up the
 * array's device address in the current device's context
 * (cudaGetSymbolAddress); the first call on a device also loads the library's
 * module there, so make that first call before any stream capture.  All
 * calls on a device share the one array and it keeps the last call's bytes;
 * nothing in it needs to start at zero (each call's partial kernel writes
 * every partial result before its merge kernel reads it; after a wait that
 * gave up, the partials it could not finish are marked invalid, as for
 * fa_fwd_splitkv).  Calls whose kernels overlap on the GPU (two streams, or
 * two host threads) race on the array: serialise them.
 * Errors: those of fa_fwd_splitkv, plus FA_ERR_SCRATCH_LIMIT when the sizes
 * need more than 16 MiB of scratch (fa_fwd_splitkv_workspace_bytes tells the
 * need; pass a workspace to fa_fwd_splitkv for larger problems).
 */
int fa_fwd_splitkv_noalloc(const void *q, const void *k, const void *v, void *o, float *lse, int B,
                           int H, int Sq, int Sk, int D, float scale, int num_splits, void *stream);

/*
 * fa_bwd -- gradients of fa_fwd: given dO = dL/dO for the forward's O,
 *   P = exp(scale Q K^T - LSE),  Delta_i = dO_i . O_i,  dS = P (dO V^T - Delta),
 *   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO.
 * "FlashAttention-2 — L3 Cross-Paper Synthesis", §3 items 1-2 (the backward
 * pass; FA2's atomic dQ accumulation is non-deterministic) and §5 item 2 (a
 * deterministic two-pass backward).  Two kernels run on `stream`: one CTA per
 * query tile writes dQ and Delta, then one CTA per key tile writes dK and dV.
 * No atomics: results are bitwise deterministic.
 *
 *   q, k, v, B, H, Sq, Sk, D, scale, causal   as passed to fa_fwd
 *   o, lse        the forward's outputs (bf16 [B,H,Sq,D], fp32 [B,H,Sq])
 *   dout          bf16 [B,H,Sq,D]
 *   dq            bf16 [B,H,Sq,D] written;  dk, dv  bf16 [B,H,Sk,D] written
 *   delta         fp32 [B,H,Sq] caller-owned scratch, written with Delta
 * All device pointers, 16-byte aligned; outputs may not overlap inputs or one
 * another.  Errors: those of fa_fwd (full and causal attention only).
 */
int fa_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
           const void *dout, void *dq, void *dk, void *dv, float *delta, int B, int H, int Sq,
           int Sk, int D, float scale, int causal, void *stream);

/*
 * fa_rope_phases -- the frequencies of rotary positions, for fa_rope, fa_rope_bwd and
 * fa_kv_append_rope.  A HOST call: it writes host memory and needs no GPU.
 *
 * Pair i of rot_dim / 2 turns by the angle position * f_i.  Its phase is f_i in units of
 * 2^-64 turns, modulo a turn (the low 64 bits of position * phase are the angle, exactly,
 * for any position and for negative ones):
 *   f_i = frequencies[i], in radians, or, where frequencies is NULL, base^(-2 i / rot_dim);
 *   FA_ROPE_PLAIN   as they are
 *   FA_ROPE_LINEAR  f_i / factor
 *   FA_ROPE_NTK     from base * factor^(rot_dim / (rot_dim - 2))
 *   FA_ROPE_YARN    f_i (1 - r_i) + f_i / factor r_i, with a ramp r_i from 0 at the pair that
 *                   makes `fast` turns in `span` positions to 1 at the one that makes
 *                   `slow`, and amplitude 0.1 ln(factor) + 1
 * The phases are then copied to the device by the caller; *amplitude (1 but for
 * FA_ROPE_YARN) is passed to the calls.
 *   rot_dim  a multiple of 16, 16 .. 128
 * span, fast and slow (usually 32 and 1) are read for FA_ROPE_YARN only, factor (>= 1) for all
 * but FA_ROPE_PLAIN.  frequencies go with FA_ROPE_PLAIN and FA_ROPE_LINEAR.
 * Errors: FA_ERR_NULLPTR; FA_ERR_BAD_SHAPE for rot_dim, scaling, or frequencies with another
 * scaling; FA_ERR_BAD_SCALE for numbers that are not finite or out of range.
 */
#define FA_ROPE_PLAIN 0
#define FA_ROPE_LINEAR 1
#define FA_ROPE_NTK 2
#define FA_ROPE_YARN 3
int fa_rope_phases(unsigned long long *phases, float *amplitude, int rot_dim, double base, int scaling,
                   double factor, double span, double fast, double slow, const double *frequencies);

/*
 * fa_rope -- rotary positions: turns pairs of each head's elements by angles that
 * grow with the token's position,
 *   (y1, y2) = amplitude (x1 cos t - x2 sin t, x1 sin t + x2 cos t),  t = position * f_i,
 * in fp32, rounded once to bf16.
 *
 *   q, k          bf16 [B, H, S, D] with any strides: queries (Hq heads) and keys (Hk heads),
 *                 read; k and k_out are NULL with Hk = 0
 *   q_out, k_out  the same shapes, written; each may be its input itself (same pointer and
 *                 strides), and may be columns of one fused tensor with others: otherwise
 *                 outputs overlap nothing
 *   positions     int32 [B, S] with positions_stride between sequences (0: all alike), or NULL:
 *                 0 .. S - 1 in each
 *   phases        64-bit [rot_dim / 2] on the device, 8-byte aligned (fa_rope_phases)
 *   rot_dim       elements of a head that are rotated, a multiple of 16, 16 .. D; those behind
 *                 them are copied
 *   strides       HOST array of 12 strides in elements, read during the call: of q, k, q_out and
 *                 k_out, each between sequences, tokens and heads; multiples of 8, >= 0; an
 *                 output's must keep its elements apart
 *   interleaved   0: elements i and i + rot_dim / 2 are a pair; 1: 2 i and 2 i + 1
 *   amplitude     finite, > 0
 *   B * S <= 2^30, Hq and Hk <= 65535, D 64 or 128
 * Packed tokens [T, H, D] are B = 1, S = T.  Deterministic.
 * Errors: FA_ERR_NULLPTR, FA_ERR_MISALIGNED, FA_ERR_UNSUPPORTED_D, FA_ERR_BAD_SHAPE,
 * FA_ERR_BAD_SCALE, FA_ERR_ALIAS; FA_ERR_CUDA if the launch fails.
 */
int fa_rope(const void *q, const void *k, void *q_out, void *k_out, const int *positions,
            const unsigned long long *phases, int B, int S, int Hq, int Hk, int D, int rot_dim,
            const long long *strides, long long positions_stride, int interleaved, float amplitude,
            void *stream);

/*
 * fa_rope_bwd -- the gradients of fa_rope: dq and dk from dq_out and dk_out, by the transposed
 * rotation, amplitude (g1 cos t + g2 sin t, -g1 sin t + g2 cos t).  Arguments and errors are
 * fa_rope's, with the gradients of its outputs in the place of its inputs (strides in the same
 * order: dq_out, dk_out, dq, dk).
 */
int fa_rope_bwd(const void *dq_out, const void *dk_out, void *dq, void *dk, const int *positions,
                const unsigned long long *phases, int B, int S, int Hq, int Hk, int D, int rot_dim,
                const long long *strides, long long positions_stride, int interleaved, float amplitude,
                void *stream);

/*
 * ---------------------------------------------------------------------------
 * The paged 8-bit key/value cache: decode serving, and prompts in chunks.
 *
 * A cache holds num_pages pages of page_size tokens (16, 32, 64 or 128) for
 * each key/value head, in e4m3 codes with one fp32 scale per page and head:
 *
 *   k_pages, v_pages   e4m3 [num_pages, Hkv, page_size, D]   value = code * scale
 *   k_scale, v_scale   fp32 [num_pages, Hkv], finite and > 0; v_scale of 2^-100 to
 *                      2^120 (as fa_kv_append gives it), those of one sequence's pages
 *                      within a factor of 2^100 of one another
 *   k_mean             int8 [num_pages, Hkv, D]  and
 *   k_mean_scale       fp32 [num_pages, Hkv]: the page's mean key, m * scale
 *                      (only fa_page_select reads them)
 *
 * Token t of sequence b is row t % page_size of page block_table[b][t / page_size]
 * (int32 [B, max_pages]; entries past a sequence's last page are never read).
 * The step's tokens of all sequences are packed: q [T, Hq, D], o [T, Hq, D],
 * lse [T, Hq]; those of sequence b are rows cu_q[b] .. cu_q[b+1]-1 (int32
 * [B+1], ascending from 0) and are its last tokens: with L = seq_lens[b] (int32
 * [B], this step's tokens included) and n = cu_q[b+1] - cu_q[b], row i of them
 * is at position L - n + i and sees the keys 0 .. L - n + i.  Rows from cu_q[B]
 * on (padding) are left as they were.  Query head h reads key/value head
 * h / (Hq / Hkv).
 *
 * One step:  fa_kv_plan -> fa_kv_append -> [fa_page_select ->] fa_fwd_paged, or, where rotary
 * positions are applied on the way, fa_kv_plan_positions -> fa_kv_append_rope -> ...; with many
 * new tokens a sequence (prompts, chunks of them) fa_fwd_paged_chunk in the place of fa_fwd_paged.
 *
 * Lengths and tables are read on the device, so that a step can be captured in
 * a graph and replayed with other lengths.  What they hold is checked there:
 * lengths are clamped to what the table and T hold; a page or position outside
 * the cache is never read or written, sets FA_ERR_BAD_PAGE in the status word
 * (fa_device_status), and the rows that would have read it come out NaN.  Where
 * cu_q does not ascend, so that its tokens exceed what T says, fa_fwd_paged writes
 * nothing and sets FA_ERR_BAD_SHAPE there, or rows are written more than once.
 * None of what a call reads may change while it runs, lengths and tables above all.
 * D is 64 or 128; q, k and v may be strided over tokens (strides in elements,
 * multiples of 8, each token's heads contiguous).  Tensors of codes and bf16 are
 * 16-byte aligned, int32 and fp32 arrays 4-byte aligned (FA_ERR_MISALIGNED).
 * num_pages * page_size, max_pages * page_size and num_pages * Hkv < 2^31, num_pages * Hkv *
 * page_size < 2^32, strides < 2^40, B <= 8192, T <= 2^30, Hkv <= 1024, Hq <= 65535 and a multiple
 * of Hkv.
 * These operations have no counterpart in the pages.
 */

/*
 * fa_kv_plan -- block tables and slot maps from request lengths: gives the
 * pages that a step's new tokens need, first come, first served.
 *
 *   cached_lens, new_lens  int32 [B]: tokens in the cache, and of this step
 *   free_pages             int32 [num_free] page numbers, of which the first
 *   free_count             int32 [1] are free; pages are taken from the end:
 *                          the i-th one taken is free_pages[free_count - 1 - i]
 *   block_table            int32 [B, max_pages], read and written: row b holds
 *                          ceil(cached/page_size) pages; the new ones are added
 *   cu_q                   int32 [B+1] written: 0, and the running sums of
 *                          new_lens (at most T)
 *   seq_lens               int32 [B] written: cached + new
 *   slot_map               int32 [T] written: page * page_size + row of each new
 *                          token; -1 behind the last token
 *   free_left              int32 [1] written: pages still free
 *
 * Request b is served when its lengths are >= 0, cached + new fits in max_pages
 * pages, and it needs no page or the pages that requests 0 .. b need are free
 * (a request that does not fit thus keeps later ones from taking pages).  One
 * that is not served keeps its row of block_table, gets slots of -1 and
 * seq_lens[b] = 0 (attention writes O = 0, LSE = -inf for its rows); its rows of
 * q, k and v stay counted in cu_q.  Where the new tokens are more than T, those behind
 * T get no slot, though seq_lens counts them: give T at least their sum.  A slot whose page is outside the cache is -1.
 * Outputs may not overlap inputs or one another (free_left is not free_count).
 * Errors: FA_ERR_NULLPTR, FA_ERR_MISALIGNED, FA_ERR_BAD_SHAPE (B, T, max_pages,
 * num_free or num_pages < 1, or out of range: num_free <= 2^30), FA_ERR_BAD_PAGE, FA_ERR_ALIAS.
 */
int fa_kv_plan(const int *cached_lens, const int *new_lens, const int *free_pages, const int *free_count,
               int *block_table, int *cu_q, int *seq_lens, int *slot_map, int *free_left, int B, int T,
               int max_pages, int num_free, int num_pages, int page_size, void *stream);

/*
 * fa_kv_plan_positions -- fa_kv_plan, which also writes each token's position:
 *   positions   int32 [T] written: max(cached, 0) + i for the i-th new token of a request, served or
 *               not; -1 behind the last token
 * as fa_rope and fa_kv_append_rope take it.  Errors: those of fa_kv_plan.
 */
int fa_kv_plan_positions(const int *cached_lens, const int *new_lens, const int *free_pages,
                         const int *free_count, int *block_table, int *cu_q, int *seq_lens, int *slot_map,
                         int *positions, int *free_left, int B, int T, int max_pages, int num_free,
                         int num_pages, int page_size, void *stream);

/*
 * fa_kv_append -- rounds a step's keys and values into the cache.
 *
 *   k, v        bf16 [T, Hkv, D], token strides k_stride, v_stride
 *   slot_map    int32 [T]; tokens with a negative slot are skipped
 *   k_pages .. v_scale, k_mean, k_mean_scale   the cache, read and written
 *               (k_mean and k_mean_scale both NULL: no means are kept)
 *
 * Consecutive tokens with consecutive slots in one page are a run.  For each run
 * and head, with amax = max |x| over its finite values,
 *   scale = 2^ceil(log2(amax / 448))   (1 for amax = 0; exponent in [-100, 120]),
 * and, where the run does not begin at row 0 of its page, at least the page's
 * scale; the rows before it are then rounded again, to code * old / scale.  Codes
 * are x / scale rounded to nearest even; +-inf become +-448, NaN stays NaN.
 * The mean is over the page's rows up to the run's last one:
 *   S_d = sum of codes (NaN as 0), A = max_d |S_d|,
 *   k_mean_d = rint(S_d * (127 / A)),  k_mean_scale = A * scale / (127 * rows)
 * (left to right in fp32: infinite where A * scale is).
 * Rows behind the run are left as they were.  A page may be in one run of a call
 * only; with more, what it holds afterwards is undefined.  A slot past the cache
 * is skipped and sets FA_ERR_BAD_PAGE in the status word.
 * Errors: FA_ERR_NULLPTR, FA_ERR_MISALIGNED, FA_ERR_BAD_SHAPE,
 * FA_ERR_UNSUPPORTED_D, FA_ERR_BAD_PAGE, FA_ERR_ALIAS.
 */
int fa_kv_append(const void *k, const void *v, const int *slot_map, void *k_pages, void *v_pages,
                 float *k_scale, float *v_scale, signed char *k_mean, float *k_mean_scale, int T, int Hkv,
                 int D, long long k_stride, long long v_stride, int num_pages, int page_size, void *stream);

/*
 * fa_kv_append_rope -- fa_kv_append with the keys rotated on the way, as fa_rope rotates them, but
 * kept in fp32 until they are rounded to codes (scales come from the rotated keys); and, where
 * q is given, the step's queries rotated beside, as fa_rope does it.
 *
 *   positions   int32 [T]: the tokens' positions (fa_kv_plan_positions)
 *   phases, rot_dim, interleaved, amplitude   as in fa_rope
 *   q, q_out    bf16 [T, Hq, D], token strides q_stride and q_out_stride: queries, and where they
 *               go (all T rows, whatever their slots); q_out may be q itself, and columns of
 *               the fused tensor that k and v are columns of.  Both NULL: no queries (Hq is not read)
 * Other arguments, and what a call leaves undefined, are fa_kv_append's.
 * Errors: those of fa_kv_append and, for the rotation, of fa_rope.
 */
int fa_kv_append_rope(const void *k, const void *v, const int *positions, const unsigned long long *phases,
                      const int *slot_map, void *k_pages, void *v_pages, float *k_scale, float *v_scale,
                      signed char *k_mean, float *k_mean_scale, const void *q, void *q_out, int T, int Hkv,
                      int Hq, int D, int rot_dim, int interleaved, float amplitude, long long k_stride,
                      long long v_stride, long long q_stride, long long q_out_stride, int num_pages,
                      int page_size, void *stream);

/*
 * fa_page_select -- the pages that a sequence's queries attend to: the top_k
 * that an 8-bit score puts first, per sequence and key/value head.
 *
 *   q, cu_q, seq_lens, block_table, k_mean, k_mean_scale   as above
 *   sel        int32 [B, Hkv, top_k] written: positions in the block table,
 *              ascending; -1 behind the last one
 *   sel_count  int32 [B, Hkv] written: how many; 0 for a sequence without queries
 *
 * Each query row is rounded to 8 bits, q8 = rint(q * (127 / max|q|)) over its
 * finite values (others count as 0), and
 *   score(page) = max over the sequence's rows r of the head's query heads of
 *                 (sum_d q8_rd * k_mean_d) * (max|q_r| / 127) * k_mean_scale,
 * the sum in integers, so that it is the same whatever its order.  The first
 * keep_first and the last keep_last pages come before all others, then higher
 * scores, and the lower position among equals; pages outside the cache last.
 * 1 <= top_k <= 2^30, keep_first, keep_last >= 0, keep_first + keep_last <= top_k.
 * max_pages <= 49152, T * Hq < 2^31.
 * Errors: FA_ERR_NULLPTR, FA_ERR_MISALIGNED, FA_ERR_BAD_SHAPE,
 * FA_ERR_UNSUPPORTED_D, FA_ERR_BAD_PAGE, FA_ERR_ALIAS.
 */
int fa_page_select(const void *q, const int *cu_q, const int *seq_lens, const int *block_table,
                   const signed char *k_mean, const float *k_mean_scale, int *sel, int *sel_count, int B,
                   int T, int Hq, int Hkv, int D, long long q_stride, int max_pages, int num_pages,
                   int page_size, int top_k, int keep_first, int keep_last, void *stream);

/*
 * fa_fwd_paged -- attention of a step's query tokens over the cache:
 *   O = softmax(scale q K^T) V,  LSE = ln sum exp(scale q.k_j)  over the keys that
 * the row sees (above), or those among them in the selected pages.
 *
 *   sel, sel_count  both NULL: every page; else int32 [B, Hkv, sel_width] and
 *                   [B, Hkv], as fa_page_select writes them (any order; a
 *                   position that is there twice counts twice)
 *   o               bf16 [T, Hq, D] contiguous, written
 *   lse             fp32 [T, Hq] contiguous, written
 *   workspace       caller-owned DEVICE scratch of at least
 *                   fa_fwd_paged_workspace_bytes(...) bytes, 16-byte aligned; it
 *                   holds partial results within the call, needs no
 *                   initialisation, and must not be used by another call until
 *                   the stream has run past this one
 *
 * A row that sees no key gets O = 0, LSE = -inf.  Keys a row does not see never
 * touch it, whatever their codes are (NaN included).  Scores and sums are fp32;
 * q and K enter the products exactly (q as bf16 scaled by a power of two to fp16:
 * elements below 2^-17 of their row's largest are rounded, to steps of 2^-24 of it),
 * the softmax weights are rounded to fp16 (each by at most 2^-11 of itself, or 2^-29 of
 * the row's largest), O once to bf16.  Any number of query
 * tokens a sequence is taken; the kernel is made for a few (decode, drafts): 8 to 32
 * rows (query tokens times heads of the group) share a pass over the keys.
 * How many is told from T / B, so T much above the tokens that there are, or one long
 * run of tokens beside many single ones, costs time (a call for each kind is faster).
 * T * Hq < 2^31, and so is, at most, (T * Hq / Hkv / 8 + B) * Hkv times the 32-key
 * tiles of a full table row, plus 3 (FA_ERR_BAD_SHAPE).  Deterministic; no atomics on
 * results.
 * Errors: FA_ERR_NULLPTR, FA_ERR_MISALIGNED, FA_ERR_BAD_SHAPE,
 * FA_ERR_UNSUPPORTED_D, FA_ERR_BAD_PAGE, FA_ERR_BAD_SCALE, FA_ERR_WORKSPACE,
 * FA_ERR_ALIAS; FA_ERR_CUDA if a launch fails.
 */
int fa_fwd_paged(const void *q, const int *cu_q, const int *seq_lens, const int *block_table,
                 const void *k_pages, const void *v_pages, const float *k_scale, const float *v_scale,
                 const int *sel, const int *sel_count, void *o, float *lse, int B, int T, int Hq, int Hkv,
                 int D, float scale, long long q_stride, int max_pages, int num_pages, int page_size,
                 int sel_width, void *workspace, size_t workspace_bytes, void *stream);

/* fa_fwd_paged_workspace_bytes -- bytes of workspace fa_fwd_paged needs on the
 * current device for these sizes (the same for all lengths); 0 for unsupported sizes. */
size_t fa_fwd_paged_workspace_bytes(int B, int T, int Hq, int Hkv, int D);

/*
 * fa_fwd_paged_chunk -- fa_fwd_paged (over all pages) made for many query tokens a sequence:
 * prompts, or chunks of them behind what is cached, beside sequences with a single token.  The
 * rows of a sequence and key/value head (query tokens times heads of the group) are taken 256 at
 * a time, on the tensor cores; where these are few, keys are split over the chip and joined.
 *
 * Arguments, layout, checks of what tables hold, and outputs are fa_fwd_paged's.  Scores and sums
 * are fp32.  q and K enter the products exactly (q as bf16 scaled by a power of two to fp16: elements below
 * 2^-17 of their row's largest are rounded, to steps of 2^-24 of it).  Softmax weights are rounded to fp16
 * (each by at most 2^-11 of itself, or 2^-29 of the largest among those that the row sees first, from its
 * end; where a v_scale is no power of two, the weight times what it is beside one), but weights times v_scale
 * are rounded to bf16 (2^-8 of each) for 128 keys among which a v_scale is not within 2^-15 to 2^7 of the
 * largest that the pass began with (or met since, more than 2^40 above it).  O is rounded once to bf16.  A
 * scale that is not finite makes the rows that see its keys NaN or infinite, and no others.
 * T * Hq < 2^31, max_pages * page_size < 2^31 - 1023.  Deterministic; no atomics on results.
 *   workspace   at least fa_fwd_paged_chunk_workspace_bytes(...) bytes, as for fa_fwd_paged
 * Errors: those of fa_fwd_paged.  An on-chip wait that gives up sets FA_ERR_TIMEOUT in the status word
 * (fa_device_status); O and LSE are then undefined.
 */
int fa_fwd_paged_chunk(const void *q, const int *cu_q, const int *seq_lens, const int *block_table,
                       const void *k_pages, const void *v_pages, const float *k_scale, const float *v_scale,
                       void *o, float *lse, int B, int T, int Hq, int Hkv, int D, float scale,
                       long long q_stride, int max_pages, int num_pages, int page_size, void *workspace,
                       size_t workspace_bytes, void *stream);

/* fa_fwd_paged_chunk_workspace_bytes -- bytes of workspace fa_fwd_paged_chunk needs on the current
 * device for these sizes (the same for all lengths); 0 for unsupported sizes. */
size_t fa_fwd_paged_chunk_workspace_bytes(int B, int T, int Hq, int Hkv, int D);

/*
 * fa_strerror -- static English text for a status code.  For FA_ERR_CUDA
 * the text of the most recent CUDA error seen by this thread is appended.
 * The returned pointer stays valid until the next call on the same thread.
 */
const char *fa_strerror(int status);

/*
 * fa_device_status -- the kernels' on-device status word, then clears it.
 * Every on-chip wait of every kernel in this library is bounded in time;
 * a wait that gives up records FA_ERR_TIMEOUT there (instead of hanging or
 * trapping) and the kernel winds down.  This call synchronises `stream`,
 * reads and resets the word on the current device, and returns FA_OK,
 * FA_ERR_TIMEOUT, FA_ERR_BAD_PAGE or FA_ERR_BAD_SHAPE (the paged cache's calls:
 * contents of tables that they could not use), or FA_ERR_CUDA.  Meant for tests and debugging; it is the
 * only call here that synchronises.
 */
int fa_device_status(void *stream);

/*
 * fa_selftest_bounded_wait -- launches one CTA that waits on an on-chip
 * barrier that nothing ever arrives on, with a wait limit of `timeout_us`
 * microseconds (1 .. 1000000), using the same bounded-wait routine as the
 * attention kernels.  The wait must give up and record FA_ERR_TIMEOUT in the
 * status word, which fa_device_status then returns.  No fault, trap or hang
 * is involved: this exists so tests can show the give-up path works.
 */
int fa_selftest_bounded_wait(int timeout_us, void *stream);

/*
 * fa_selftest_fwd_timeout -- fa_fwd with every on-chip wait of the forward
 * kernel bounded by `timeout_ns` (0 .. 2e9) instead of the 2 s that fa_fwd
 * uses.  With a limit shorter than a tile load (0 gives up at the first wait
 * that is not already satisfied), the kernel's own give-up path runs: the
 * wait raises the CTA's abort flag and records FA_ERR_TIMEOUT in the status
 * word, the other roles stop at their next wait, the producer waits (bounded,
 * 20 ms) for the copies it issued, the MMA issuer for its MMAs, TMEM is freed
 * and the CTA returns -- no trap, fault or hang.  O and LSE are then
 * undefined.  Arguments, checks and errors are fa_fwd's, plus
 * FA_ERR_BAD_SHAPE for timeout_ns above 2e9.  The surveyed pages have no
 * counterpart: it exists so tests can show the forward kernel winds down
 * cleanly and leaves the context usable.
 */
int fa_selftest_fwd_timeout(const void *q, const void *k, const void *v, void *o, float *lse,
                            int B, int H, int Sq, int Sk, int D, float scale, int causal,
                            unsigned long long timeout_ns, void *stream);

/*
 * fa_selftest_bwd_timeout -- fa_bwd with every on-chip wait of both backward
 * kernels bounded by `timeout_ns` (0 .. 2e9) instead of the 2 s that fa_bwd
 * uses.  With a limit shorter than a tile load the kernels' own give-up path
 * runs, as for fa_selftest_fwd_timeout: the CTA's abort flag is raised and
 * FA_ERR_TIMEOUT recorded in the status word, the other roles stop at their
 * next wait, copies and MMAs in flight are waited for (bounded), TMEM is freed
 * and the CTA returns.  dQ, dK, dV and delta are then undefined.  Arguments,
 * checks and errors are fa_bwd's, plus FA_ERR_BAD_SHAPE for timeout_ns above
 * 2e9.  The surveyed pages have no counterpart: it exists so tests can show
 * the backward kernels wind down cleanly and leave the context usable.
 */
int fa_selftest_bwd_timeout(const void *q, const void *k, const void *v, const void *o, const float *lse,
                            const void *dout, void *dq, void *dk, void *dv, float *delta, int B, int H,
                            int Sq, int Sk, int D, float scale, int causal, unsigned long long timeout_ns,
                            void *stream);

/*
 * fa_selftest_splitkv_timeout -- fa_fwd_splitkv with every on-chip wait of the
 * partial kernel bounded by `timeout_ns` (0 .. 2e9) instead of 2 s.  With a
 * limit shorter than a tile load the kernel gives up as the forward kernel
 * does (abort flag, FA_ERR_TIMEOUT in the status word, copies in flight
 * waited for, no trap); a CTA that gave up writes NaN as its partial
 * log-sum-exp, so the merged O and LSE of its rows come out NaN instead of
 * plausible stale values.  Arguments, checks and errors are fa_fwd_splitkv's,
 * plus FA_ERR_BAD_SHAPE for timeout_ns above 2e9.  The surveyed pages have no
 * counterpart: it exists so tests can show the decode kernels wind down
 * cleanly and leave the context usable.
 */
int fa_selftest_splitkv_timeout(const void *q, const void *k, const void *v, void *o, float *lse, int B,
                                int H, int Sq, int Sk, int D, float scale, int num_splits, void *workspace,
                                size_t workspace_bytes, unsigned long long timeout_ns, void *stream);

/*
 * fa_selftest_paged_chunk_timeout -- fa_fwd_paged_chunk with every on-chip wait bounded by `timeout_ns`
 * (0 .. 2e9, counted in microseconds) instead of 2 s.  With a limit shorter than the first tile's way
 * through the kernel, and always with 0, its own give-up path runs, as for fa_selftest_fwd_timeout: the block's abort flag is
 * raised and FA_ERR_TIMEOUT recorded in the status word, the other roles stop at their next wait, MMAs in
 * flight are waited for (bounded), TMEM is freed and the block returns.  O and LSE are then undefined.
 * Arguments, checks and errors are fa_fwd_paged_chunk's, plus FA_ERR_BAD_SHAPE for timeout_ns above 2e9.
 */
int fa_selftest_paged_chunk_timeout(const void *q, const int *cu_q, const int *seq_lens, const int *block_table,
                                    const void *k_pages, const void *v_pages, const float *k_scale,
                                    const float *v_scale, void *o, float *lse, int B, int T, int Hq, int Hkv, int D,
                                    float scale, long long q_stride, int max_pages, int num_pages, int page_size,
                                    void *workspace, size_t workspace_bytes, unsigned long long timeout_ns,
                                    void *stream);

/* fa_version -- library version, major*10000 + minor*100 + patch. */
int fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_FA_H */
