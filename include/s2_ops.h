/*
 * s2_ops.h -- per-kernel C ABI of libs2.so, for kernel-level parity tests
 * and for callers that drive the Dual-AR layers themselves.
 *
 * Every pointer argument is DEVICE memory owned by the caller; nothing is
 * allocated.  Work is enqueued on ``stream`` (a cudaStream_t, NULL = legacy
 * default stream).  Returns S2_OK (0) or a negative S2_E* status from s2.h:
 * S2_EINVAL for shapes the kernels do not support (stated per call), S2_ECUDA
 * when the launch fails.  Matrices are row-major; "ld" is a row pitch in
 * elements.
 */
#ifndef S2_OPS_H_
#define S2_OPS_H_

#include <stddef.h>
#include <stdint.h>

#include "s2.h"

#ifdef __cplusplus
extern "C" {
#endif

/* K1 -- weight-streaming GEMV on CUDA cores.
 *   Y[b, n] (op)= sum_k W[n, k] * a[b, k],  b < B (1..8), n < N
 * with a = RMSNorm(X[b]) * gain (eps) when gain != NULL, else a = X[b]
 * ("s2pro-native", Where it stands: at batch 1 a frame is bound by reading
 * every weight once; "SGLang Day-0 ...", Architecture: Qwen3-style blocks,
 * whose projections are preceded by RMSNorm).
 *   W: [N, K] bf16 (w_bf16 = 1) or fp32; K % 8 == 0, rows 16-byte aligned.
 *   X: fp32 [B, ldx]; Y: fp32.
 *   mode 0: Y[b, n] = y;  1: Y[b, n] += y (residual);
 *   mode 2: rows (2i, 2i+1) hold (gate_i, up_i): Y[b, i] = silu(gate) * up
 *   (SwiGLU MLP), N even.
 *   grid_ctas: CTAs to launch (0 = one per SM). */
int s2op_gemv(const void* W, int w_bf16, int N, int K, const float* X, int ldx, int B,
              const float* gain, float eps, float* Y, int ldy, int mode, int grid_ctas,
              void* stream);

/* K6 -- constrained greedy head: codes[b] = argmax_n sum_k W[n, k] a[b, k]
 * (a as in s2op_gemv), ties to the lowest n ("SGLang Day-0 ...",
 * Background: constrained decoding restricts the head to the legal ids; the
 * caller passes only those rows).  logits (optional, fp32 [B, N]) receives
 * the scores.  workspace: at least s2op_argmax_workspace_bytes(B) bytes of
 * zero-initialised device memory; it is left zeroed again on exit. */
size_t s2op_argmax_workspace_bytes(int B);
int s2op_gemv_argmax(const void* W, int w_bf16, int N, int K, const float* X, int ldx, int B,
                     const float* gain, float eps, int32_t* codes, float* logits,
                     void* workspace, void* stream);

/* K2 -- tcgen05 tensor-core GEMM (bf16 in, fp32 accumulate):
 *   Y[t, n] (op)= sum_k A[n, k] * Bm[t, k],  t < T, n < N
 *   A: bf16 [N, K] (weights), Bm: bf16 [T, ldb] (activations), both
 *   16-byte aligned; N % 128 == 0, K % 64 == 0, ldb % 8 == 0.
 *   epi 0: Y = y;  1: Y += y;  2: SwiGLU of interleaved (gate, up) rows into
 *   bf16 Y16[t, n/2] (the MLP of the S2 blocks).
 *   split_k: 0 = automatic; otherwise the number of K splits (at most K/64;
 *   split s covers 64-wide k-tiles [s*kt/S, (s+1)*kt/S) of the kt = K/64,
 *   summed in split order).  With more than one split, workspace (fp32, at least
 *   s2op_tc_gemm_workspace_bytes) and tickets (zeroed, at least
 *   s2op_tc_gemm_tickets) are required; tickets are zero again on exit. */
size_t s2op_tc_gemm_workspace_bytes(int N, int K, int T, int split_k);
size_t s2op_tc_gemm_tickets(int N, int T);
int s2op_tc_gemm(const void* A, int N, int K, const void* Bm, int T, int ldb, float* Y, int ldy,
                 void* Y16, int ldy16, int epi, int split_k, float* workspace, uint32_t* tickets,
                 void* stream);

/* K2, two-plane operand: as s2op_tc_gemm but the activations arrive as a bf16
 * pair (Bhi, Blo) with x ~= Bhi + Blo (Blo = bf16(x - Bhi)), and the kernel
 * accumulates A*Bhi + A*Blo -- ~16 mantissa bits of the activations at twice
 * the tensor work and the same weight traffic.  For epi 2 the bf16 output is
 * written the same way: Y16 (hi) and, when non-NULL, Y16lo (remainder).
 * Token tiles are at most 128 wide in this mode; workspace and tickets as
 * given by the *_2 size queries. */
size_t s2op_tc_gemm2_workspace_bytes(int N, int K, int T, int split_k);
size_t s2op_tc_gemm2_tickets(int N, int T);
int s2op_tc_gemm2(const void* A, int N, int K, const void* Bhi, const void* Blo, int T, int ldb,
                  float* Y, int ldy, void* Y16, void* Y16lo, int ldy16, int epi, int split_k,
                  float* workspace, uint32_t* tickets, void* stream);

/* K2 phase trace (diagnostics): every later K2 launch of the process has
 * each CTA c write six globaltimer stamps (ns, uint64) to buf[6c .. 6c+5]:
 * kernel entry, setup done (barriers, tensor memory, programmatic-launch
 * wait), first operand stage landed, last MMA issued, accumulator complete,
 * epilogue done.  buf: device memory of max_ctas * 48 bytes; CTAs with a
 * linear index >= max_ctas write nothing.  max_ctas = 0 turns it off.
 * S2_EINVAL for a NULL buf with max_ctas > 0. */
int s2op_tc_set_trace(void* buf, int max_ctas);

/* K3 + K4 -- decode attention over a paged KV cache for B sequences with m
 * (1 or 2) new rows each ("SGLang Day-0 ...", Optimizations: paged KV cache;
 * Engineering Appendix: bf16-rounded RoPE table).  For row i of sequence b at
 * position p = pos[b] + i:
 *   q_h, k, v from qkv[(b*m + i), :] = [q (H*hd) | k (Hkv*hd) | v (Hkv*hd)];
 *   q_h, k <- RMSNorm per head (gains q_gain, k_gain [hd]) then rotate-half
 *   RoPE with rope_cos/rope_sin [positions][hd/2];
 *   k, v are written to slot p % 16 of page table[b*table_ld + p/16];
 *   o[b*m+i, h] = softmax_j(q_h . k_j / sqrt(hd)) v_j over keys j <= p of kv
 *   head h / (H/Hkv).
 * kv: one layer's pool, pages of [2][Hkv][16][hd] (kv_bf16 = 1: bf16, else
 * fp32).  Supported: (hd, H/Hkv) = (128, 4) or (64, 2).  nsplit >= 1 splits
 * the keys across CTAs (32-key chunks); the splits are merged in fixed order.
 * A sequence with at most 64 keys (p + 1 for its last row) is attended by one
 * split whatever nsplit is, so its rows round as with nsplit = 1.  workspace:
 * s2op_attn_decode_workspace_bytes(...) bytes, zero-initialised (zero again
 * on exit); may be NULL when nsplit == 1.  o: fp32 [B*m, o_ld]. */
size_t s2op_attn_decode_workspace_bytes(int B, int m, int H, int Hkv, int hd, int nsplit);
/* The key-split count the model path takes for B sequences on this device:
 * within one wave of resident CTAs, enough CTAs for twice the SMs and up to
 * as many as the wave holds; past one wave, the fewest splits (at most 16)
 * whose waves are at least 90% full.  A negative status for bad sizes. */
int s2op_attn_decode_pick_split(int B, int H, int Hkv, int hd, int kv_bf16);
int s2op_attn_decode(const float* qkv, int qkv_ld, int B, int m, int H, int Hkv, int hd,
                     const float* q_gain, const float* k_gain, float eps, const float* rope_cos,
                     const float* rope_sin, const int32_t* pos, void* kv, int kv_bf16,
                     const int32_t* table, int table_ld, float* o, int o_ld, int nsplit,
                     void* workspace, void* stream);

/* K11 + K3/K4 -- decode attention (m = 1 new row per sequence) for B
 * sequences whose page tables share their first ``shared_len`` keys (whole
 * 16-token pages: one radix-cached prompt prefix, "SGLang Day-0 ...",
 * Optimizations with SGLang Omni: radix prefix caching).  The same result as
 * s2op_attn_decode: the keys from shared_len on (each sequence's own, with
 * the appended new key) by the split-KV decode attention, which leaves its
 * partials; the keys below shared_len on the tcgen05 tensor cores, once per
 * kv head for all B x 4 query rows (128-row tiles; products of bf16 hi/lo
 * operand planes, fp32 accumulation), in thread-block clusters of 8 CTAs
 * that merge their partials with the split-KV ones (in key order) into o.
 * Supported: hd 128, H = 4 Hkv.  max_keys bounds every context (sizes the
 * workspace); shared_len a multiple of 16, at most max_keys.
 *
 * workspace: s2op_attn_decode_prefix_workspace_bytes zero-initialised bytes
 * (its tickets are zero again on exit).  Its first part holds the shared
 * keys as the MMAs' operand images: s2op_attn_prefix_planes writes them
 * from the pages (table row 0 must hold the shared pages), and
 * s2op_attn_decode_shared_prefix reads them, so call s2op_attn_prefix_planes
 * (same kv, kv_bf16, table, Hkv, hd, shared_len, max_keys, workspace) first,
 * and again whenever those pages change.  s2op_attn_decode_shared_prefix
 * synchronises ``stream`` once (it uploads shared_len).  S2_EINVAL for
 * unsupported shapes or a shared_len that is not a multiple of 16 (below 16
 * for s2op_attn_prefix_planes). */
size_t s2op_attn_decode_prefix_workspace_bytes(int B, int H, int Hkv, int hd, int nsplit, int max_keys);
int s2op_attn_prefix_planes(const void* kv, int kv_bf16, const int32_t* table, int Hkv, int hd, int shared_len,
                            int max_keys, void* workspace, void* stream);
int s2op_attn_decode_shared_prefix(const float* qkv, int qkv_ld, int B, int H, int Hkv, int hd,
                                   const float* q_gain, const float* k_gain, float eps,
                                   const float* rope_cos, const float* rope_sin, const int32_t* pos,
                                   void* kv, int kv_bf16, const int32_t* table, int table_ld,
                                   int shared_len, int max_keys, float* o, int o_ld, int nsplit,
                                   void* workspace, void* stream);

/* Phase trace of the shared-prefix tensor-core kernel (measurement only):
 * while on, each launch's CTA i < max_ctas (i = (tile * Hkv + kv head) * 8 +
 * cluster rank) writes 16 uint64 globaltimer stamps (ns) to device memory
 * ``buf`` + 16 i: entry, after setup, after the wait on the previous launch,
 * after issuing the query tile's copy, operands of its first chunk landed,
 * after S = Q K^T, after the softmax, after O = P V, after its last chunk,
 * after the first cluster barrier, after the merge, at exit (slots 12-15
 * unused; stamps of phases a CTA skips stay as they were).  max_ctas 0 turns
 * it off.  S2_EINVAL for max_ctas < 0 or a NULL buf with max_ctas > 0. */
int s2op_attn_prefix_set_trace(void* buf, int max_ctas);

/* K9 -- prefill attention for T new rows of one sequence at positions
 * pos0 .. pos0+T-1 whose q/k/v are in qkv (layout as above): q/k norm +
 * RoPE, K/V appended to the sequence's pages, then causal attention over all
 * keys 0 .. pos0+T-1 (keys before pos0 come from cached -- e.g. radix-shared
 * -- pages and are not recomputed).  q_scratch: fp32 [T, H*hd].  o: fp32
 * [T, o_ld]. */
int s2op_attn_prefill(const float* qkv, int qkv_ld, int T, int pos0, int H, int Hkv, int hd,
                      const float* q_gain, const float* k_gain, float eps, const float* rope_cos,
                      const float* rope_sin, void* kv, int kv_bf16, const int32_t* table,
                      float* q_scratch, float* o, int o_ld, void* stream);

/* RoPE table of the S2 blocks: cos/sin of p * theta^(-2i/hd) for p < n_pos,
 * i < hd/2, rounded to float then to bf16 (ties to even), stored as fp32
 * ("SGLang Day-0 ...", Engineering Appendix: BF16 RoPE Precision Mismatch).
 * Host buffers of n_pos*hd/2 floats each. */
int s2op_rope_table(int n_pos, int hd, float theta, float* cos_out, float* sin_out);

/* HBM read-bandwidth calibration: streams n_ops device buffers (bufs[i],
 * bytes[i] bytes, 16-byte aligned, bytes % 16 == 0; bufs and bytes are HOST
 * arrays of n_ops entries, read during the call) reps times over and
 * discards the data ("s2pro-native", Where it stands: a decode frame is
 * bound by how fast the weights can be read, so this is the stream to
 * compare the weight-streaming kernels against).
 *   mode 0: one launch per buffer, each thread eight 16-byte loads in flight;
 *   mode 1: one persistent launch (one CTA per SM): a producer thread copies
 *     the CTA's contiguous share of each buffer into a ring of ``stages``
 *     shared-memory chunks of ``chunk_bytes`` (bulk copies by the TMA engine,
 *     chunk_bytes * stages <= 200 KB), consumer warps read and release them;
 *     barrier != 0 puts a grid barrier before each buffer on the consumer
 *     side only (a dependent chain of operations), the producer streams on.
 * scratch: device memory of s2op_stream_read_scratch_bytes(n_ops) bytes,
 * owned by the caller.  err_out (host, may be NULL): receives the kernel's
 * error word (0 = ok, nonzero = a bounded wait gave up); reading it
 * synchronises the stream.  Returns S2_EINVAL for bad sizes, S2_ECUDA when a
 * launch fails. */
size_t s2op_stream_read_scratch_bytes(int n_ops);
int s2op_stream_read(const void* const* bufs, const unsigned long long* bytes, int n_ops, int reps,
                     int mode, int chunk_bytes, int stages, int barrier, void* scratch,
                     int* err_out, void* stream);

/* Decode attention without any allocation -- no counterpart on the pages;
 * an addition of this library.  Same arguments and results as
 * s2op_attn_decode, minus the workspace.  It is meant for callers that
 * cannot allocate device memory themselves: a real-time audio thread, where
 * cudaMalloc/cudaFree may block on the driver or synchronise the device in
 * the middle of a frame, or a host whose device memory is owned by another
 * allocator (a framework's caching pool, a fixed per-plugin budget).
 *   Scratch: the split-KV partials and tickets live in a file-scope device
 *   array of S2_NOALLOC_SCRATCH_BYTES (8 MiB) that every GPU loading the
 *   library holds until the process exits.  A call needing more --
 *   B*m*H*nsplit*(hd+2)*4 bytes of partials plus B*Hkv*4 bytes of tickets,
 *   the tickets on a 256-byte boundary -- returns S2_EINVAL
 *   (s2op_attn_decode_noalloc_max_bytes() reports the limit).
 *   Set-up: the first call on a device looks up the array's device address
 *   (cudaGetSymbolAddress, with that device current); make that first call
 *   before any stream capture.  The address is kept per device index and is
 *   valid only within the device's current primary context: after
 *   cudaDeviceReset (or anything else that destroys that context) the kept
 *   address is stale, so do not call this entry point again in that process.
 *   Sharing: every call uses the same array, which keeps the previous
 *   call's contents; each call clears its tickets itself (a memset on
 *   ``stream``).  Calls whose work overlaps on the GPU -- e.g. on two
 *   streams -- race on the array and must be serialised by the caller.
 *   No cudaMalloc, cudaFree or allocating library routine is called. */
#define S2_NOALLOC_SCRATCH_BYTES (8u << 20)
size_t s2op_attn_decode_noalloc_max_bytes(void);
int s2op_attn_decode_noalloc(const float* qkv, int qkv_ld, int B, int m, int H, int Hkv, int hd,
                             const float* q_gain, const float* k_gain, float eps,
                             const float* rope_cos, const float* rope_sin, const int32_t* pos,
                             void* kv, int kv_bf16, const int32_t* table, int table_ld, float* o,
                             int o_ld, int nsplit, void* stream);

/* ------------------------------------------------------------------------
 * 8-bit KV cache.  The cache's bytes bound decode attention at large batches
 * and long contexts; these calls keep keys and values in e4m3.
 *
 * Pool: n_pages pages of 16 tokens, kv8 [n_pages][2 (K, V)][Hkv][16][hd] e4m3
 * bytes (16-byte aligned) and kv_scale fp32 [n_pages][2][Hkv]; a cached value
 * is byte value * scale.  A block (the 16 rows of one page, K or V, head) has
 * the scale 2^e with the smallest e in [-32, 32] whose 448 * 2^e covers the
 * block's largest magnitude (NaN does not count and is stored as NaN; values
 * beyond 448 * 2^32, infinities among them, saturate).  Rounding is to nearest
 * even, on keys that are normed and rotated to about 2^-44, so the bytes of a
 * token depend neither on the batch nor on whether a prompt or a single step
 * appended it, with one exception.  New rows in a block with older ones take the
 * larger of both scales; where it grows, the older rows are rescaled, which is
 * exact but for values that become e4m3 subnormals: these are rounded a second
 * time, and may differ by one rounding from what one call with all the rows
 * would have stored.  Scales are powers of two as these calls write
 * them: in place of another value the power of two next to it is taken.
 *
 * hd is 64 or 128, H / Hkv 1..8, B 1..1024.  qkv rows as in s2op_attn_decode:
 * [q (H*hd) | k (Hkv*hd) | v (Hkv*hd)], fp32, qkv_ld >= (H + 2 Hkv) hd;
 * rope_cos / rope_sin [n_pos][hd/2]; sequence b's page j is table[b *
 * table_ld + j].  o: rows of H*hd values, pitch o_ld, fp32 (o_bf16 = 0) or
 * bf16 (1).  Softmax statistics and sums are fp32 (a row of q or k has to have a
 * sum of squares that fp32 holds); the products run on the tensor cores, e4m3
 * values being exact in f16, with q and the probabilities as f16 pairs (hi + lo,
 * 22 bits).  A probability times its block's scale 2^e is held against the largest
 * of these in its row: single tokens round it by 2^-31 of the largest among blocks
 * of up to 2^10 times its scale, prompts by 2^-22 (2^-18 with a bf16 output) of the
 * largest probability among blocks of up to 2^14 times its scale, at its scale; a
 * block of larger values counts only as far as its weight.  Prompt attention with a
 * bf16 output takes q and the probabilities as single f16 (11 bits): the
 * probabilities' rounding is an eighth of the output's, q's moves a score by up to
 * 2^-11 sum |q_i k_i| / sqrt(hd), which grows with the scores (with gains of 0.5 to
 * 1.5 the error is 1.02 times that of the output's rounding alone, with query gains
 * of 20 times that 1.29 times); an fp32 output has pairs.
 *
 * A sequence whose new positions do not lie in [0, min(n_pos, 16 table_ld))
 * (pos[b] = -1, for instance: a padded batch) is left out: nothing is stored
 * for it and its rows of o are zero.  A table entry outside [0, n_pages) is
 * not followed: its keys count as masked and its new rows are not stored (a
 * row without any key is zero).  Sequences of a call may read a page together,
 * but one that a sequence appends to must not be among another's pages.
 * Pages' rows behind the last appended one keep their bytes.  workspace
 * (16-byte aligned): zero-initialised, zero where it has to be again on exit.
 * One of the largest size serves calls of both kinds and of any sizes one after
 * the other; calls that may overlap in time need one each. */

/* Decode attention for B sequences with m new rows each, row b*m + i at
 * position pos[b] + i: q and k normed and rotated, k and v stored, then
 * attention over all keys up to the row's position.  m * H / Hkv <= 8, B * Hkv *
 * table_ld < 2^31.  The workspace's size depends on m, H, Hkv and hd and grows
 * with m. */
size_t s2op_attn_decode_kv8_workspace_bytes(int B, int m, int H, int Hkv, int hd);
int s2op_attn_decode_kv8(const float* qkv, int qkv_ld, int B, int m, int H, int Hkv, int hd,
                         const float* q_gain, const float* k_gain, float eps, const float* rope_cos,
                         const float* rope_sin, int n_pos, const int32_t* pos, void* kv8,
                         float* kv_scale, int n_pages, const int32_t* table, int table_ld, void* o,
                         int o_bf16, int o_ld, void* workspace, void* stream);

/* Prompt attention of B sequences in one call: sequence b has the rows
 * row0[b] .. row0[b+1] - 1 (row0: B + 1 non-decreasing entries on the device;
 * none is fine) at positions pos0[b], pos0[b] + 1, ..., behind pos0[b] cached
 * tokens.  T (at most 2^24) bounds row0[B]; rows in no sequence are left as they
 * are.  Positions at or beyond 2^20 count as outside the table.  The workspace's size
 * depends on hd alone. */
size_t s2op_attn_prefill_kv8_workspace_bytes(int T, int B, int H, int Hkv, int hd);
int s2op_attn_prefill_kv8(const float* qkv, int qkv_ld, int T, int B, const int32_t* row0,
                          const int32_t* pos0, int H, int Hkv, int hd, const float* q_gain,
                          const float* k_gain, float eps, const float* rope_cos,
                          const float* rope_sin, int n_pos, void* kv8, float* kv_scale, int n_pages,
                          const int32_t* table, int table_ld, void* o, int o_bf16, int o_ld,
                          void* workspace, void* stream);

/* Page src[i] of an fp32 (kv_bf16 = 0) or bf16 pool [n_src][2][Hkv][16][hd]
 * into page dst[i] of an 8-bit pool, i < n (src, dst, fill: device arrays).
 * fill (NULL: 16 each): rows of the page that are in use; the others become
 * zero and do not count for the scales.  A pair with an index outside its
 * pool is left out; no two pairs may have the same dst.  Pools 16-byte
 * aligned.  Pages of several layers go through one call when the layers'
 * pools lie one after the other (page p of layer l is page l * n_pages + p). */
int s2op_kv8_pack_pages(const void* kv, int kv_bf16, int n_src, const int32_t* src,
                        const int32_t* fill, void* kv8, float* kv_scale, int n_dst,
                        const int32_t* dst, int n, int Hkv, int hd, void* stream);
/* The reverse: byte value * scale, exact in fp32 and in bf16. */
int s2op_kv8_unpack_pages(const void* kv8, const float* kv_scale, int n_src, const int32_t* src,
                          void* kv, int kv_bf16, int n_dst, const int32_t* dst, int n, int Hkv,
                          int hd, void* stream);

/* Copy pages within a pool of any cache type (the forking of a sequence's
 * last, partly filled page; the moving of pages when a pool is compacted):
 * page src[i] -> dst[i] in each of ``layers`` layers, page p of layer l at
 * kv + (l * n_pages + p) * page_bytes; with scale != NULL its scale_bytes too.
 * src and dst are HOST arrays, read during the call (a captured call keeps
 * these pairs).  A page may be the source of several pairs; S2_EINVAL for an
 * index outside the pool, a destination named twice or one that is also a
 * source, page_bytes not a multiple of 16 or kv not 16-byte aligned,
 * scale_bytes not a multiple of 4. */
int s2op_kv_copy_pages(void* kv, size_t page_bytes, void* scale, size_t scale_bytes, int n_pages,
                       int layers, const int32_t* src, const int32_t* dst, int n, void* stream);
/* Entries of a device page table [rows][cols], pitch table_ld, that equal
 * src[i] become dst[i] (HOST arrays; S2_EINVAL for a source named twice or one
 * that is also a destination); all others stay. */
int s2op_kv_remap_pages(int32_t* table, int rows, int cols, int table_ld, const int32_t* src,
                        const int32_t* dst, int n, void* stream);

/* ------------------------------------------------------------------------
 * 4-bit weights and 8-bit rows.  A decode step of few sequences is bound by
 * reading the weights once; these calls keep them in 4 bits, a quarter of the
 * bf16 matrices' bytes, and the rows that meet them in 8.
 *
 * A row of K values is held in groups of 32 with a power of two 2^e each (the
 * OCP microscaling formats MXFP4 and MXFP8).  e is the smallest of [-126, 120]
 * with largest magnitude <= top * 2^e; the values divided by 2^e are rounded to
 * nearest, ties to even: no finite value but weights beyond 6 * 2^120 saturates.
 *   weights, e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and negatives; top 6): codes
 *   [N][Kp/2] bytes, value 2i in the low and 2i+1 in the high four bits of
 *   byte i, Kp = K rounded up to a multiple of 128, padded with zeros; 32-byte
 *   aligned, s2op_w4_code_bytes(N, K) in all.
 *   rows, e4m3 (top 448): [T][ld8] bytes, 16-byte aligned, ld8 a multiple of
 *   16, ld8 >= K.  Bytes from K on are neither read nor written.
 *   scales: bytes e + 127 (255: NaN) of row r, group g at
 *     ((r / 128) * ceil(K / 128) + g / 4) * 512 + r % 32 * 16 + r / 32 % 4 * 4 + g % 4,
 *   tiles of 128 rows x 4 groups; 16-byte aligned, s2op_mx_scale_bytes(rows, K)
 *   in all.  Groups beyond K hold 2^0 in rows that exist; the bytes of rows that
 *   do not exist are neither written nor used.
 * Sizes: any N, T in [0, 2^24] (none: nothing is done) and K in [1, 2^20].
 * Plain matrices are fp32 or bf16 (*_bf16 = 1) with a row pitch ld* of at least
 * their columns, aligned to their elements (16-byte aligned rows are read and
 * written fastest).  Operands of a call do not overlap unless it says so.  S2_EINVAL
 * for a NULL or misaligned pointer, a pitch or a size out of range. */
size_t s2op_w4_code_bytes(int N, int K);
size_t s2op_mx_scale_bytes(int rows, int K);

/* Weights W [N][K] into codes and scales.  A group that holds a NaN or an
 * infinity becomes NaN as a whole. */
int s2op_w4_pack(const void* W, int w_bf16, int N, int K, int ldw, void* codes, void* scale,
                 void* stream);
/* The reverse: code * 2^e, exact in fp32 and in bf16. */
int s2op_w4_unpack(const void* codes, const void* scale, int N, int K, void* W, int w_bf16, int ldw,
                   void* stream);

/* Rows X [T][K] to 8 bits with scales.  NaN and infinities are stored as NaN
 * and do not count for the scales. */
int s2op_mx8_pack(const void* X, int x_bf16, int ldx, int T, int K, void* y8, int ld8,
                  void* y_scale, void* stream);

/* h = x + r (r NULL: x), rounded to x's type and stored to H, then
 *   y = h / sqrt(mean_k h^2 + eps) * gain,  to 8 bits with scales
 * as in s2op_mx8_pack.  y is computed to about 2^-44 of itself and 2^-120 of the
 * gain before it is rounded, so its codes do not depend on the order of the sum.
 * gain: fp32 [K]; eps >= 0 and finite.
 * H: of x's type; may be X itself (then ldh = ldx) and, without r, NULL; R may
 * be H (of the same type and pitch).  A row with a NaN or an
 * infinity in h, or without a square above zero and eps = 0, is NaN in y8. */
int s2op_add_rmsnorm_mx8(const void* X, int x_bf16, int ldx, const void* R, int r_bf16, int ldr,
                         int T, int K, const float* gain, float eps, void* H, int ldh, void* y8,
                         int ld8, void* y_scale, void* stream);

/* Products with 4-bit weights:
 *   Y[t, n] (op)= sum_k X[t, k] W[n, k],   n < N
 *   mode 0: Y = y;  1: Y += y (residual);  2: rows (2i, 2i+1) of W hold
 *   (gate_i, up_i): Y[t, i] = silu(gate) * up, N even.
 * Y: fp32 or bf16 (y_bf16 = 1), apart from the other operands; sums are fp32,
 * rounded to Y's type once, as they are stored.  They are added up on the tensor
 * cores, which cut towards zero, by about 2^-24 of the sum so far for each 32 k, and
 * go to sums rounded to nearest every 896 k or sooner; where Y is bf16 and T above
 * 64, every 16,384 k or sooner (about 2^-15 of sum |x w| at most, which an output
 * of much smaller size shows).  Rows and weights that are NaN make NaN of their
 * own row or column of Y alone.  Every operand, the weights among them, is read in
 * the stream's order: a product may follow the call that writes it directly.
 * s2op_w4_gemv: B = 1..8 plain rows X; infinities in them count as NaN.  A value is
 * taken whole where it lies within 2^13 (fp32; bf16: 2^17) of the largest of its
 * group of 32, and to 2^-37 (2^-25) of that one where it is smaller; of all values
 * 2^-136 may be missing, which groups below 2^-98 (2^-110) notice.  Their 8-bit parts
 * are summed apart, so that sums are finite where sum |x w| < 2^127.  workspace:
 * at least s2op_w4_gemv_workspace_bytes(K, B) bytes, 16-byte aligned, of any content
 * (0 bytes for sizes that are refused).  Calls that may overlap in time need one
 * each.
 * s2op_w4_gemm: T rows of 8 bits with scales, from s2op_mx8_pack or
 * s2op_add_rmsnorm_mx8. */
size_t s2op_w4_gemv_workspace_bytes(int K, int B);
int s2op_w4_gemv(const void* codes, const void* scale, int N, int K, const void* X, int x_bf16,
                 int ldx, int B, void* Y, int y_bf16, int ldy, int mode, void* workspace,
                 void* stream);
int s2op_w4_gemm(const void* codes, const void* scale, int N, int K, const void* X8, int ld8,
                 const void* x_scale, int T, void* Y, int y_bf16, int ldy, int mode, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* S2_OPS_H_ */
