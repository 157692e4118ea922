/*
 * pa.h -- C ABI of the paged-KV-cache attention library (libpa.so), sm_103a.
 *
 * The operations follow the statement of the problem on three web pages:
 *   [P1] "Basics of LLM Inference and vLLM Internals: KV Cache, PagedAttention,
 *        and Scheduler" -- s.2 "KV Cache and Sizing Formulas", s.4 "PagedAttention
 *        and Block Management", s.6 "Chunked Prefill, Scheduler, and Preemption";
 *   [P2] drpranayjha.com (Red Hat AI Inference Server part) -- "How PagedAttention
 *        pages the KV cache";
 *   [P3] "The Memory Trick Behind Fast LLM Serving" -- "PagedAttention changes
 *        the shape of the problem", "Batching does not merge the conversations".
 *
 * Conventions shared by every call
 * --------------------------------
 * Memory.   Every pointer argument named as "device" is caller-owned GPU memory
 *           of the current device; the library allocates no memory, keeps no
 *           state besides per-device attribute caches, and never synchronises
 *           the stream (except pa_read_device_status, which says so).
 * Streams.  Work is enqueued asynchronously on `stream` (NULL = legacy default
 *           stream).  pa_stream_t is the same handle as cudaStream_t.
 * Errors.   Host-checkable problems are reported before anything is launched:
 *           PA_ERR_INVALID_ARG (null pointer, negative count, misaligned buffer,
 *           H_q not a multiple of H_kv, ...; the per-sequence or per-token arrays
 *           of an empty batch may be null: such a call does nothing and returns
 *           PA_OK), PA_ERR_UNSUPPORTED (head_dim != 128,
 *           block_size not 8, 16 or 32, dtype pair not listed), PA_ERR_WORKSPACE (workspace
 *           too small).  A failed launch returns PA_ERR_CUDA.  Problems only the
 *           device can see (a block-table entry outside the pool, a bounded wait
 *           that ran out) are recorded in the workspace's status word and
 *           returned by pa_read_device_status; kernels never trap.
 * Shapes.   head_dim d = 128; block_size bs = 8, 16 (the default the pages
 *           use) or 32: larger blocks waste more of a sequence's last block,
 *           smaller ones cut the kernels' contiguous runs [P1 s.11, question 3].
 *           Cache layout is [num_blocks][num_kv_heads][bs][128] for both K and V,
 *           so one (block, KV head) tile is bs x 128 contiguous elements (4 KiB
 *           in bf16/fp16 and 2 KiB in FP8 at bs = 16).  A slot number is
 *           physical_block * bs + offset.
 * GQA.      Query head h reads KV head h / (num_q_heads / num_kv_heads):
 *           consecutive query heads form a group [P1 s.2].
 * FP8.      FP8-E4M3 ("fn": bias 7, max 448, no inf, NaN = S.1111.111) with
 *           float32 scales, separate for K and V, one per tensor (PA_FP8_E4M3) or
 *           one per KV head (PA_FP8_E4M3_PER_HEAD), read from device memory so
 *           that calls can be captured in CUDA graphs.
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define PA_API __attribute__((visibility("default")))
#else
#define PA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* pa_stream_t;

typedef enum {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = 1,
    PA_ERR_UNSUPPORTED = 2,
    PA_ERR_CUDA = 3,
    PA_ERR_TIMEOUT = 4,        /* device: a bounded wait gave up */
    PA_ERR_OUT_OF_RANGE = 5,   /* device: a block-table entry outside [0, num_blocks) */
    PA_ERR_WORKSPACE = 6
} pa_status;

/*
 * Element types.  PA_FP8_E4M3 caches carry one float32 scale per tensor (k_scale,
 * v_scale point to one float each); PA_FP8_E4M3_PER_HEAD caches hold the same
 * e4m3 codes with one scale per KV head (k_scale, v_scale point to
 * num_kv_heads floats, head h's elements dequantised with scale[h]).  The pages
 * mention an FP8 KV cache [P1 s.7 "--kv-cache-dtype fp8"] but not its scaling;
 * per-head scales are this library's variant of it.
 */
typedef enum { PA_BF16 = 0, PA_FP16 = 1, PA_FP8_E4M3 = 2, PA_FP8_E4M3_PER_HEAD = 3 } pa_dtype;

/* Static description of a status code.  Never NULL. */
PA_API const char* pa_status_string(int status);

/* Library ABI version (major * 100 + minor). */
PA_API int pa_version(void);

/* Kernels this library has enqueued in this process (every entry point counts the
 * launches it makes; a launch into a stream being captured counts once, at
 * capture).  A caller can read it before and after a call to see how many kernels
 * the call launches. */
PA_API unsigned long long pa_kernel_launches(void);

/* Text of the last CUDA failure seen by a call of this thread that returned
 * PA_ERR_CUDA (which CUDA call failed and its error string); "" if none.  The
 * buffer is thread-local and valid until the next failing call. */
PA_API const char* pa_last_error(void);

/*
 * Slot write ("reshape_and_cache") [P1 s.4 block table; P3 "PagedAttention
 * changes the shape of the problem"].
 *
 * For every new token t in [0, num_tokens) with slot = slot_mapping[t] >= 0,
 * stores k[t][h][:] into k_cache[slot / bs][h][slot % bs][:] and v[t][h][:]
 * into v_cache at the same place, for every KV head h.  A negative slot is
 * padding and writes nothing.  A slot >= num_blocks * block_size is skipped (nothing is
 * written).  Two tokens with the same slot in one call: undefined which wins.
 *
 *   k, v           device, [num_tokens][num_kv_heads][128] of src_dtype (bf16|fp16)
 *   k_cache,v_cache device, [num_blocks][num_kv_heads][16][128] of cache_dtype,
 *                  16-byte aligned
 *   slot_mapping   device, int64 [num_tokens]
 *   cache_dtype    == src_dtype (bits copied unchanged), or PA_FP8_E4M3:
 *                  code = e4m3(fl32(x) / scale), the quotient rounded once to
 *                  binary32 (IEEE division), then round-to-nearest-even to E4M3 with
 *                  magnitudes above 448 clamped to 448; a NaN quotient ->
 *                  S.1111.111 with S the sign bit of the source element x; a zero
 *                  result keeps the quotient's sign [P1 s.2, s.7 "--kv-cache-dtype fp8"];
 *                  or PA_FP8_E4M3_PER_HEAD: the same with head h's scale[h].
 *   k_scale,v_scale device float32: one each (PA_FP8_E4M3) or num_kv_heads each
 *                  (PA_FP8_E4M3_PER_HEAD); required (non-NULL) iff FP8.
 * Bytes outside the written slots are never touched.
 */
PA_API pa_status pa_reshape_and_cache(const void* k, const void* v, void* k_cache, void* v_cache,
                               const int64_t* slot_mapping, int num_tokens, int num_kv_heads,
                               int head_dim, int block_size, int num_blocks, pa_dtype src_dtype,
                               pa_dtype cache_dtype, const float* k_scale, const float* v_scale,
                               pa_stream_t stream);

/*
 * Rotary positions (no counterpart on the pages, which take q and k as already
 * positioned): a head's first rot_dim components are turned in pairs by angles that
 * grow with the token's position p,
 *   u = a cos(p f_i) - b sin(p f_i),  v = b cos(p f_i) + a sin(p f_i),
 * with the pairs (i, i + rot_dim / 2) or (2i, 2i + 1), i < rot_dim / 2.
 *
 * pa_rope_frequencies: the f_i, on the host (no GPU work).
 *   PA_ROPE_UNSCALED  f_i = base^(-2 i / rot_dim)
 *   PA_ROPE_LINEAR    f_i / factor: positions interpolated into the trained range
 *   PA_ROPE_BY_PARTS  f_i blended with f_i / factor by the turns t = trained f_i / 2 pi
 *                     it makes over the trained length: kept for t >= high_turns, divided
 *                     for t <= low_turns, keep = (t - low_turns) / (high_turns - low_turns)
 *                     between: the ramp in turns of the paper "YaRN: Efficient
 *                     Context Window Extension of Large Language Models", s.3.2.
 *                     NOT what most checkpoints released as YaRN were trained with:
 *                     those blend linearly over the component i, between two bounds
 *                     rounded to whole components, and differ from this by up to 1.7
 *                     times (base 10^6, trained 32768, factor 4) or 4.3 times (10^4,
 *                     4096, 40) between the ends of the ramp.  Compute such
 *                     frequencies by the checkpoint's own rule and pass them to
 *                     pa_rope_table, which takes any
 *   freqs             host, [rot_dim / 2]
 *   rot_dim           a multiple of 16, 16 .. 128
 *   base, factor      > 0 and finite; factor is read by the scaled forms
 *   trained, low_turns, high_turns
 *                     read by PA_ROPE_BY_PARTS: trained > 0, high_turns > low_turns >= 0
 * Arguments whose frequencies are not all finite are PA_ERR_INVALID_ARG (freqs is left as
 * it was).
 */
typedef enum { PA_ROPE_UNSCALED = 0, PA_ROPE_LINEAR = 1, PA_ROPE_BY_PARTS = 2 } pa_rope_scaling;

PA_API pa_status pa_rope_frequencies(double* freqs, int rot_dim, double base, pa_rope_scaling scaling, double factor,
                                     double trained, double low_turns, double high_turns);

/*
 * The table of a set of frequencies: for p < max_positions and i < rot_dim / 2
 *   cos_sin[p][i] = attention cos(p f_i),  cos_sin[p][rot_dim / 2 + i] = attention sin(p f_i)
 * each entry to within 3.5 x 2^-24 of itself (two to three units in the last place of
 * float32 at most, small sines included), but for what the angle itself is off by: it is
 * held modulo one turn in 64-bit fixed point, up to 2^-54 + p 2^-61 + p |f_i| 2^-52 radians.
 * Built once; any table of this layout serves pa_rope_and_cache.
 *   cos_sin    device, float32 [max_positions][rot_dim], 16-byte aligned
 *   freqs      host, [rot_dim / 2], finite (read during the call)
 *   attention  factor on both (YaRN's scaling of the logits; 1 for none)
 * max_positions == 0 does nothing.
 */
PA_API pa_status pa_rope_table(float* cos_sin, int max_positions, int rot_dim, const double* freqs, float attention,
                               pa_stream_t stream);

/*
 * Rotation of a step's queries and keys with the slot write in one pass: q_out[t] =
 * q[t] turned by positions[t], and k[t] turned likewise and v[t] as it is stored at
 * slot_mapping[t] as pa_reshape_and_cache stores them.  Positions and slots are
 * separate: after pa_evict a token's place in the cache is no longer its position.
 *
 * Each product and sum of the rotation is rounded to float32, its result once to the
 * type stored (for an FP8 cache: divided by the scale in float32, then rounded; a NaN
 * there becomes 0.1111.111).  Components from rot_dim on are copied.
 *
 *   q_out          device, [num_tokens][num_q_heads][128] of src_dtype; may be q itself
 *                  (same pointer and stride), otherwise must not overlap the inputs
 *   q, k, v        device, [num_tokens][heads][128] of src_dtype
 *   *_stride       elements from one token to the next (a multiple of 8; the heads of a
 *                  token are contiguous), so that q, k and v can be parts of one
 *                  [num_tokens][num_q_heads + 2 num_kv_heads][128] projection; an output
 *                  stride is at least num_q_heads * 128
 *   positions      device, int64 [num_tokens]; a negative position is padding (nothing of
 *                  the token is written); a position >= max_positions is recorded as
 *                  PA_ERR_OUT_OF_RANGE and nothing of the token is written
 *   slot_mapping   device, int64 [num_tokens]; a negative slot writes no K or V (q is
 *                  turned all the same); a slot beyond the pool is recorded as
 *                  PA_ERR_OUT_OF_RANGE and not written
 *   cos_sin        device, float32 [max_positions][rot_dim], 16-byte aligned (pa_rope_table)
 *   rot_dim        a multiple of 16, 16 .. 128 (others: PA_ERR_UNSUPPORTED)
 *   workspace      NULL (nothing is recorded), or a workspace whose status word records errors
 * Other arguments as pa_reshape_and_cache.
 */
typedef enum { PA_ROPE_HALF = 0, PA_ROPE_INTERLEAVED = 1 } pa_rope_layout;

PA_API pa_status pa_rope_and_cache(void* q_out, long long q_out_stride, const void* q, long long q_stride,
                                   const void* k, long long k_stride, const void* v, long long v_stride,
                                   void* k_cache, void* v_cache, const int64_t* slot_mapping,
                                   const int64_t* positions, const float* cos_sin, int max_positions, int rot_dim,
                                   pa_rope_layout layout, int num_tokens, int num_q_heads, int num_kv_heads,
                                   int head_dim, int block_size, int num_blocks, pa_dtype src_dtype,
                                   pa_dtype cache_dtype, const float* k_scale, const float* v_scale, void* workspace,
                                   pa_stream_t stream);

/*
 * pa_rope_and_cache of heads that are normed first, with positions of several axes: each
 * query and key head x becomes
 *   y_i = x_i / sqrt(sum_k x_k^2 / 128 + eps) * (weight_offset + weight_i)
 * (an RMS norm over the head), then its pairs are turned, pair i by
 *   cos_sin[positions[axis_of_pair[i]][t]][i] and [rot_dim / 2 + i],
 * and k and v are stored at slot_mapping[t].  With several axes a token of a picture or a
 * video has a time, a row and a column, and every pair of a head follows one of them.
 *
 * Norm and rotation are in float32, rounded once to the type stored (the FP8 slot-write
 * rule as in pa_rope_and_cache); v is stored as it is.
 *
 *   q_weight, k_weight  device, [128] of src_dtype, 16-byte aligned; NULL: those heads are
 *                  not normed
 *   eps            >= 0 and finite (the sum of squares is float32: with eps == 0 a head whose
 *                  squares vanish there becomes NaN, and one whose squares pass its range,
 *                  components of 1e18 and more, zeros)
 *   weight_offset  added to the weights (1 for checkpoints that store weight - 1)
 *   positions      device, int64 [num_axes][num_tokens]; a token any of whose positions is
 *                  negative is padding (nothing of it is written); one with a position >=
 *                  max_positions is recorded as PA_ERR_OUT_OF_RANGE and not written
 *   num_axes       1 .. 4
 *   axis_of_pair   host, [rot_dim / 2], each in [0, num_axes) (read during the call); NULL:
 *                  every pair follows axis 0
 * Other arguments as pa_rope_and_cache.
 */
PA_API pa_status pa_norm_rope_and_cache(void* q_out, long long q_out_stride, const void* q, long long q_stride,
                                        const void* k, long long k_stride, const void* v, long long v_stride,
                                        const void* q_weight, const void* k_weight, float eps, float weight_offset,
                                        void* k_cache, void* v_cache, const int64_t* slot_mapping,
                                        const int64_t* positions, int num_axes, const uint8_t* axis_of_pair,
                                        const float* cos_sin, int max_positions, int rot_dim, pa_rope_layout layout,
                                        int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                        int block_size, int num_blocks, pa_dtype src_dtype, pa_dtype cache_dtype,
                                        const float* k_scale, const float* v_scale, void* workspace,
                                        pa_stream_t stream);

/*
 * Bytes of workspace pa_decode / pa_mixed need on the CURRENT device for
 * num_seqs sequences (the default worker count depends on the device's SM
 * count).  The workspace is caller-owned device memory, 256-byte aligned.  Its
 * first 256 bytes must be zero before the first call: they hold the device
 * status word (the first word, see pa_read_device_status) and the counter from
 * which decode warps claim the last pieces of work, which every call leaves
 * ready for the next.  The rest is scratch each call overwrites before reading
 * and needs no initialisation.  One workspace must not be used by two calls
 * that may overlap on the GPU.  Returns 0 for invalid arguments.
 */
PA_API size_t pa_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim);

/*
 * Bytes of workspace with which pa_decode_shared_prefix can cut the shared
 * prefix into as many key segments as it wants (up to 16 partials per query
 * row: num_seqs * num_q_heads * 520 bytes each beyond pa_workspace_size).
 * Same rules as pa_workspace_size.  Returns 0 for invalid arguments.
 */
PA_API size_t pa_workspace_size_shared_prefix(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim);

/*
 * Bytes of workspace for pa_decode_weights: pa_workspace_size and the scores of up to
 * max_tokens cached tokens (the sum over the batch of each sequence's length rounded up
 * to 16), 4 bytes per token, KV head and query head of its group (a group counted up to
 * an even number, groups of more than 8 up to a multiple of 8).  Same rules as
 * pa_workspace_size.  Returns 0 for invalid arguments.
 */
PA_API size_t pa_workspace_size_weights(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                                        long long max_tokens);

/* Default number of decode workers (warps) on the current device for a 16-bit
 * cache: two 4-warp CTAs per SM.  An FP8 cache defaults to twice as many (four
 * CTAs per SM: its warps are bound by the latency of the work on each block, not
 * by HBM); the 16-bit decode rows of pa_mixed and the private suffixes of
 * pa_decode_shared_prefix run three CTAs per SM (shorter rings: those grids run
 * beside another grid).  Explicit worker counts run from 1 to this value. */
PA_API int pa_default_workers(void);

/*
 * Decode attention over the paged cache [P1 s.2 "attention revisits the keys
 * and values of all preceding tokens", s.4 block table; P2 "How PagedAttention
 * pages the KV cache"].
 *
 * For every sequence s and query head h (KV head kh = h / G, G = H_q / H_kv):
 *   out[s][h][:] = softmax_t( scale * q[s][h] . K_s[t] ) . V_s[t],  t < seq_lens[s]
 * where token t of sequence s lives in physical block block_tables[s][t / 16],
 * offset t % 16, KV head kh.  seq_lens[s] counts every cached token, including
 * this step's own (write it with pa_reshape_and_cache first).  seq_lens[s] == 0
 * gives zeros.  Entries of block_tables past ceil(seq_lens[s] / 16) are never
 * read.  An entry that is read and lies outside [0, num_blocks) is replaced by
 * block 0 and recorded as PA_ERR_OUT_OF_RANGE in the workspace status word.
 *
 *   out            device, [num_seqs][num_q_heads][128] of q_dtype
 *   q              device, [num_seqs][num_q_heads][128], q_dtype bf16|fp16, 16-byte aligned
 *   k_cache,v_cache device, layout above; cache_dtype == q_dtype, PA_FP8_E4M3 or
 *                  PA_FP8_E4M3_PER_HEAD
 *   block_tables   device, int32 [num_seqs][max_blocks_per_seq]; a table's width in tokens
 *                  (block_size * max_blocks_per_seq) at most 2^31 - 1024, else
 *                  PA_ERR_UNSUPPORTED
 *   seq_lens       device, int32 [num_seqs]; each <= block_size * max_blocks_per_seq
 *   scale          softmax scale (e.g. 1/sqrt(128))
 *   k_scale,v_scale device float32 scalars, required iff cache is FP8 (dequant
 *                  is code * scale)
 *   workspace      see pa_workspace_size
 * Scores, the softmax and the sums over keys are float32; the probabilities are
 * rounded to the cache's 16-bit type (fp16 for an FP8 cache) for the product
 * with V, and with an FP8 cache the query to fp16 (a bf16 query's components
 * beyond 65504 become infinite).
 * num_seqs <= 8192.  The work is split evenly over the workers by cached
 * blocks; a sequence split across workers is merged by a log-sum-exp combine
 * launched behind the decode kernel on the same stream.  The result does not
 * depend on where blocks live.
 */
PA_API pa_status pa_decode(void* out, const void* q, const void* k_cache, const void* v_cache,
                    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                    int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                    int num_blocks, float scale, pa_dtype q_dtype, pa_dtype cache_dtype,
                    const float* k_scale, const float* v_scale, void* workspace,
                    size_t workspace_bytes, pa_stream_t stream);

/*
 * One decode step in one pass: pa_reshape_and_cache of each sequence's new token
 * followed by pa_decode, with the same results (the cache bytes bit for bit, the
 * outputs exactly) [P1 s.3: each step appends one token per running request and
 * attends over all of them; s.4 slot mapping].  The warps that read a sequence's
 * last 16 keys store its new token into the cache slot first, so the slot write
 * costs no separate launch.
 *
 *   k_new, v_new   device, [num_seqs][num_kv_heads][128] of q_dtype, 16-byte aligned
 *   slot_mapping   device, int64 [num_seqs]: slot_mapping[s] must be the slot of
 *                  position seq_lens[s] - 1 of sequence s (block
 *                  block_tables[s][(seq_lens[s] - 1) / block_size], offset
 *                  (seq_lens[s] - 1) % block_size), or negative (padding: nothing is
 *                  written).  Another slot, or a non-negative slot for an empty
 *                  sequence, is recorded as PA_ERR_OUT_OF_RANGE and not written.
 *   k_cache, v_cache written at those slots (FP8 with the pa_reshape_and_cache rule)
 * The block holding a new token must belong to its sequence alone (copy it first
 * when it is shared, see pa_pool_copy_on_write).  Other arguments as pa_decode.
 */
PA_API pa_status pa_decode_append(void* out, const void* q, const void* k_new, const void* v_new,
                                  const int64_t* slot_mapping, void* k_cache, void* v_cache,
                                  const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                                  int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                  int num_blocks, float scale, pa_dtype q_dtype, pa_dtype cache_dtype,
                                  const float* k_scale, const float* v_scale, void* workspace,
                                  size_t workspace_bytes, pa_stream_t stream);

/* pa_decode_append with an explicit worker count (1 .. pa_default_workers(); 0 =
 * the default), as pa_decode_ex is to pa_decode.  The cache bytes it writes do not
 * depend on the worker count; outputs agree with pa_decode_append to rounding.
 * With long ranges per worker (>= 48 16-key units, 16-bit cache, at most 4
 * query heads per KV head) the last ~10% of the work is handed out at run time
 * in pieces, so a small worker count is how a small batch reaches that path. */
PA_API pa_status pa_decode_append_ex(void* out, const void* q, const void* k_new, const void* v_new,
                                     const int64_t* slot_mapping, void* k_cache, void* v_cache,
                                     const int32_t* block_tables, int max_blocks_per_seq,
                                     const int32_t* seq_lens, int num_seqs, int num_q_heads, int num_kv_heads,
                                     int head_dim, int block_size, int num_blocks, float scale,
                                     pa_dtype q_dtype, pa_dtype cache_dtype, const float* k_scale,
                                     const float* v_scale, void* workspace, size_t workspace_bytes,
                                     int num_workers, pa_stream_t stream);

/* pa_decode with an explicit worker count (1 .. pa_default_workers(); 0 = the
 * default).  Fewer workers means longer ranges per worker and fewer split
 * points; results agree with pa_decode to rounding. */
PA_API pa_status pa_decode_ex(void* out, const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_tables, int max_blocks_per_seq,
                       const int32_t* seq_lens, int num_seqs, int num_q_heads, int num_kv_heads,
                       int head_dim, int block_size, int num_blocks, float scale,
                       pa_dtype q_dtype, pa_dtype cache_dtype, const float* k_scale,
                       const float* v_scale, void* workspace, size_t workspace_bytes,
                       int num_workers, pa_stream_t stream);

/*
 * pa_decode that also adds up how much each cached token is attended to (no counterpart on
 * the pages; pa_evict chooses by these sums): out as pa_decode, and for every sequence s,
 * KV head h and token t < seq_lens[s]
 *   weights_out[s][h][t] = weights_in[s][h][t] + sum over the query heads of h's group of
 *                          their softmax weight of token t, in float32.
 * Entries of weights_out from seq_lens[s] on are left as they were.
 *
 *   weights_in     device, float32 [num_seqs][num_kv_heads][weight_stride], or NULL for
 *                  zeros (weights_out is then this step's weights alone)
 *   weights_out    device, the same layout; may be weights_in, otherwise must not overlap it
 *   weight_stride  at least max_blocks_per_seq * block_size
 *   workspace      pa_workspace_size_weights bytes.  A batch with more tokens than the
 *                  workspace holds scores for is recorded as PA_ERR_WORKSPACE in its status
 *                  word: out is computed, weights_out is left as it was
 * Other arguments as pa_decode; out agrees with pa_decode's exactly, its 16-bit
 * probabilities included (the weights are of the unrounded ones).  The last queries of a
 * prompt can be observed the same way before an eviction: one row for each, all with the
 * prompt's block table, seq_lens = its position + 1, and a row of weights_out of its own
 * (added up afterwards).
 */
PA_API pa_status pa_decode_weights(void* out, float* weights_out, const float* weights_in, long long weight_stride,
                                   const void* q, const void* k_cache, const void* v_cache,
                                   const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
                                   int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                   int num_blocks, float scale, pa_dtype q_dtype, pa_dtype cache_dtype,
                                   const float* k_scale, const float* v_scale, void* workspace,
                                   size_t workspace_bytes, pa_stream_t stream);

/*
 * Decode for a batch whose block tables share their leading blocks: the same
 * result as pa_decode, computed in cascade.  The pages describe requests that
 * start with the same prompt reusing the same full KV blocks, so that their
 * block tables point at the same physical blocks [P3 "Prefix caching is the
 * second win"; P1 s.4 block table, s.5 prefix caching]; they give no kernel for
 * it (the cascade split below is this library's).
 *
 * Precondition: for every sequence s, block_tables[s][j] == block_tables[0][j]
 * for j < prefix_blocks, and seq_lens[s] >= block_size * prefix_blocks.  A batch
 * that violates it is recorded as PA_ERR_OUT_OF_RANGE in the workspace status
 * word (its outputs are then unspecified).  The split between the shared part
 * and the private parts falls on a multiple of 16 keys: with 8-token blocks and
 * an odd prefix_blocks the last shared block is read with each sequence's
 * private blocks (and is not checked against the precondition).
 *
 * The prefix keys are read once for the whole batch: every decode row of every
 * sequence is contracted against them on the tensor cores as one dense tile
 * grid (one CTA per 256 query rows of a KV head and key segment), leaving an
 * unnormalised partial per row and segment; the private blocks after the
 * prefix stream through the decode kernel; the combine kernel merges all of
 * them by log-sum-exp.  The prefix is cut into key segments of whole 128-key
 * steps until its grid has about one CTA per SM, as far as the workspace
 * holds the extra partials; a prefix grid under half the SMs runs beside the
 * decode grid (which then takes the other SMs), a larger one runs first.
 * prefix_blocks == 0 reduces to pa_decode with every row merged by the
 * combine.
 *
 *   prefix_blocks  host, 0 <= prefix_blocks <= max_blocks_per_seq
 *   workspace      at least pa_workspace_size(num_seqs, num_q_heads,
 *                  num_kv_heads, head_dim) bytes (then the prefix is one
 *                  segment); pa_workspace_size_shared_prefix bytes allow
 *                  every split
 * Other arguments as pa_decode; results agree with pa_decode to rounding.
 */
PA_API pa_status pa_decode_shared_prefix(void* out, const void* q, const void* k_cache, const void* v_cache,
                                  const int32_t* block_tables, int max_blocks_per_seq,
                                  const int32_t* seq_lens, int num_seqs, int prefix_blocks,
                                  int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                  int num_blocks, float scale, pa_dtype q_dtype, pa_dtype cache_dtype,
                                  const float* k_scale, const float* v_scale, void* workspace,
                                  size_t workspace_bytes, pa_stream_t stream);

/*
 * Mixed batch: decode rows and prefill chunks in one flattened query array
 * [P3 "Batching does not merge the conversations"; P1 s.6 chunked prefill].
 *
 * Sequence s owns query rows query_start_loc[s] .. query_start_loc[s+1]-1
 * (q_len_s rows).  seq_lens[s] counts the cached tokens including this step's
 * q_len_s new ones, so row j of sequence s sits at position
 * pos = seq_lens[s] - q_len_s + j and attends causally to tokens 0 .. pos of its
 * own sequence only.  q_len_s == 1 is a decode row; q_len_s == 0 contributes
 * nothing.
 *
 *   out, q          device, [total_q][num_q_heads][128] of q_dtype
 *   query_start_loc device, int32 [num_seqs + 1], non-decreasing,
 *                   query_start_loc[0] == 0, query_start_loc[num_seqs] == total_q
 *   max_q_len       host upper bound of q_len_s (0 or 1: no prefill chunks, the
 *                   prefill kernel is not launched)
 * Other arguments as pa_decode.
 */
PA_API pa_status pa_mixed(void* out, const void* q, const int32_t* query_start_loc, const void* k_cache,
                   const void* v_cache, const int32_t* block_tables, int max_blocks_per_seq,
                   const int32_t* seq_lens, int num_seqs, int total_q, int max_q_len,
                   int num_q_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                   float scale, pa_dtype q_dtype, pa_dtype cache_dtype, const float* k_scale,
                   const float* v_scale, void* workspace, size_t workspace_bytes,
                   pa_stream_t stream);

/*
 * Bytes of workspace pa_mixed_scored and pa_tree need on the CURRENT device (they leave the
 * partial results of sequences that several SMs share in it; the size does not depend on the
 * batch's lengths).  Same rules as pa_workspace_size, only the status word must start at zero.
 * Returns 0 for invalid arguments.
 */
PA_API size_t pa_workspace_size_scored(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim);

/*
 * Mixed batch whose scores are capped, biased by distance, windowed or open over a prefix
 * (no counterpart on the pages, whose attention is plain and causal): rows, lengths and
 * positions as pa_mixed.  Row j of sequence s, at position pos = seq_lens[s] - q_len_s + j,
 * sees token t if
 *   (t <= pos or t < prefix_lens[s])  and  (window == 0 or pos - t < window)  and  t < seq_lens[s],
 * with the score, x = scale * q . K_s[t],
 *   cap tanh(x / cap) (cap > 0) or x (cap == 0),  less slopes[query head] * |pos - t|,
 * and out is the softmax over the tokens it sees times V.  A row that sees nothing is zeros;
 * rows of out that no sequence owns are left as they were.
 *
 *   prefix_lens    device, int32 [num_seqs]: the sequence's first tokens that all its rows
 *                  see, those behind them too; NULL: none
 *   slopes         device, float32 [num_q_heads]; NULL: no bias
 *   cap            0, or from 1e-6 to 1e6 with scale / cap finite
 *   window         >= 0; 0: none.  Table entries of blocks that no row of a call sees through
 *                  the window need not name a block (they are not read)
 *   workspace      pa_workspace_size_scored bytes
 * A sequence whose lengths do not fit (rows outside q, more rows than tokens, more tokens than
 * the table) is recorded as PA_ERR_OUT_OF_RANGE and its rows are left as they were.  What a
 * token that no row of its sequence sees holds does not matter (it may be NaN); one that some
 * of its rows see must be finite for the others.  Other arguments, and the precision, as
 * pa_mixed (over fp16 and FP8 caches a key that weighs less than 2^-31 of its row's largest
 * adds nothing beside V); at most 128 query heads per KV head.
 */
PA_API pa_status pa_mixed_scored(void* out, const void* q, const int32_t* query_start_loc, const void* k_cache,
                                 const void* v_cache, const int32_t* block_tables, int max_blocks_per_seq,
                                 const int32_t* seq_lens, const int32_t* prefix_lens, const float* slopes, float cap,
                                 int window, int num_seqs, int total_q, int num_q_heads, int num_kv_heads, int head_dim,
                                 int block_size, int num_blocks, float scale, pa_dtype q_dtype, pa_dtype cache_dtype,
                                 const float* k_scale, const float* v_scale, void* workspace, size_t workspace_bytes,
                                 pa_stream_t stream);

/*
 * Attention for a tree of drafted tokens over the cache (no counterpart on the pages): the
 * last q_len_s = query_start_loc[s + 1] - query_start_loc[s] cached tokens of sequence s are
 * the nodes of a tree, written at places seq_lens[s] - q_len_s + i (i < q_len_s), and row j
 * of the sequence is node j's query.  It sees every token before the tree and node i if bit
 * i % 64 of masks[row][i / 64] is set: the nodes on its path from the root, its own among
 * them (a bit has to be set for the row to see itself; bits from q_len_s on are ignored).
 *
 *   masks          device, 64-bit words [total_q][mask_words], 8-byte aligned; q_len_s <=
 *                  64 * mask_words, else the sequence is recorded as PA_ERR_OUT_OF_RANGE and
 *                  its rows are left as they were
 *   cap            as pa_mixed_scored
 *   window         0: none; else of the tokens before the tree row j sees those with
 *                  pos - t < window, pos being the place of the first node plus the number of
 *                  nodes that it sees (one at least), less one: its depth.  Table entries of
 *                  blocks wholly before place first node - window + 1 are not read; tokens from
 *                  there on must be finite
 * A row that sees nothing (no token before the tree and an empty mask) is zeros.  Other
 * arguments, and what tokens that no row sees may hold, as pa_mixed_scored.
 */
PA_API pa_status pa_tree(void* out, const void* q, const int32_t* query_start_loc, const void* k_cache,
                         const void* v_cache, const int32_t* block_tables, int max_blocks_per_seq,
                         const int32_t* seq_lens, const uint64_t* masks, int mask_words, float cap, int window,
                         int num_seqs, int total_q, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                         int num_blocks, float scale, pa_dtype q_dtype, pa_dtype cache_dtype, const float* k_scale,
                         const float* v_scale, void* workspace, size_t workspace_bytes, pa_stream_t stream);

/*
 * Commit of the accepted paths of verified trees, in the caches of several layers at once:
 * node paths[s][i] of sequence s (i < path_lens[s]) moves to the place behind the tokens
 * before the tree and the i nodes accepted before it, i.e. the K and V rows at place
 * seq_lens[s] - q_len_s + paths[s][i] are copied to place seq_lens[s] - q_len_s + i, and
 *   seq_lens_out[s] = seq_lens[s] - q_len_s + path_lens[s].
 * Rows behind the accepted ones keep what they hold.
 *
 *   seq_lens_out   device, int32 [num_seqs]; shares no memory with the arrays below
 *   num_layers     0: nothing is done (the lengths are not written either)
 *   k_caches, v_caches
 *                  host, num_layers pointers each to a cache (layout as pa_decode); all
 *                  distinct.  Read during the call
 *   paths          device, int32 [num_seqs][max_path]: ascending, each in [0, q_len_s);
 *                  entries from path_lens[s] on are never read
 *   path_lens      device, int32 [num_seqs]: 0 .. min(max_path, q_len_s)
 *   query_start_loc, block_tables, seq_lens   as the pa_tree call had them
 *   workspace      NULL, or a workspace whose status word records errors
 * A sequence with a path that is none, with lengths that do not fit or with a block outside
 * the pool among those that its path needs is recorded as PA_ERR_OUT_OF_RANGE; nothing of it
 * moves and its seq_lens_out is left as it was.  Blocks of a tree must not be shared between
 * sequences.
 */
PA_API pa_status pa_tree_commit(int32_t* seq_lens_out, void* const* k_caches, void* const* v_caches, int num_layers,
                                const int32_t* paths, const int32_t* path_lens, int max_path,
                                const int32_t* query_start_loc, const int32_t* block_tables, int max_blocks_per_seq,
                                const int32_t* seq_lens, int num_seqs, int num_kv_heads, int head_dim, int block_size,
                                int num_blocks, pa_dtype cache_dtype, void* workspace, pa_stream_t stream);

/*
 * Decode without a caller-provided workspace (no counterpart on the pages; the
 * pages do not discuss memory ownership of the kernels).
 *
 * Same computation and arguments as pa_decode, minus the workspace.  It is for
 * callers that cannot allocate device memory themselves: a plugin or host
 * framework that hands over only input and output buffers, or a latency-critical
 * path where cudaMalloc / cudaFree (which may synchronise the device) are not
 * allowed.  The scratch lives in one static 16 MiB device array inside libpa.so;
 * every GPU that loads the library holds it until the process exits.  This call
 * allocates nothing and calls no allocating routine.
 *
 *  - Limit: the batch must fit the 16 MiB scratch.  With S = num_seqs,
 *    G = num_q_heads / num_kv_heads, W = pa_default_workers() (1216 on a 152-SM
 *    GB300), N = S * num_kv_heads * ceil(G / 8) + 2 W partial slots and R(x) = x
 *    rounded up to a multiple of 256, a call needs
 *        256 + R(4 (S + 1)) + R(512 S num_q_heads) + R(8 S num_q_heads)
 *            + R(64 N) + 4096 N
 *    bytes; the 2 W slots alone take about 10.1 MB on a 152-SM GB300.  There
 *    that allows at most 100 sequences with 64 query and 8 KV heads, 133 with
 *    32 and 8, 177 with 8 and 8, 457 with 12 and 2, 533 with 8 and 2.  Larger
 *    batches return PA_ERR_WORKSPACE with the sizes in pa_last_error().
 *  - The first call on a device looks up the array's device address
 *    (cudaGetSymbolAddress) with that device current and caches it; make that
 *    first call before any stream capture.
 *  - All calls share the one array, which keeps the previous call's contents;
 *    each call clears the part that must start at zero (the status word and
 *    the work counter at its head) on its stream.  Calls that may overlap on the GPU (other streams, other threads)
 *    race on the array and give undefined results: serialise them.
 *  - Device-side reports (PA_ERR_OUT_OF_RANGE for a bad block-table entry,
 *    PA_ERR_TIMEOUT) stay in the static array, where no caller can read them,
 *    and the next call clears them: this call cannot report them.  A caller
 *    that needs those checks must use pa_decode with a workspace and read it
 *    with pa_read_device_status.
 */
PA_API pa_status pa_decode_noalloc(void* out, const void* q, const void* k_cache, const void* v_cache,
                                   const int32_t* block_tables, int max_blocks_per_seq,
                                   const int32_t* seq_lens, int num_seqs, int num_q_heads,
                                   int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                   float scale, pa_dtype q_dtype, pa_dtype cache_dtype,
                                   const float* k_scale, const float* v_scale, pa_stream_t stream);

/*
 * Block copies for copy-on-write [P1 s.4: a physical block shared by several
 * block tables carries a reference count; a sequence about to write into a
 * shared block needs its own copy first].
 *
 * For i < num_pairs: block dst[i] <- block src[i], every KV head, in both
 * caches (layout as pa_decode).  The dst blocks must be distinct and none may be
 * a src block of the same call (the result is otherwise unspecified).  An id
 * outside [0, num_blocks) skips its pair and, when workspace is not NULL, is
 * recorded as PA_ERR_OUT_OF_RANGE in its status word.
 *
 *   src, dst        device, int32 [num_pairs]
 *   workspace       NULL, or a workspace whose status word records errors
 */
PA_API pa_status pa_copy_blocks(void* k_cache, void* v_cache, const int32_t* src, const int32_t* dst,
                                int num_pairs, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                pa_dtype cache_dtype, void* workspace, pa_stream_t stream);

/*
 * Eviction: brings every sequence to at most `budget` cached tokens, keeping for each KV
 * head the tokens that were attended to most (no counterpart on the pages, whose cache
 * only grows until a request is preempted [P1 s.6]; P1 s.2's sizing is what it bounds).
 *
 * For sequence s with n = seq_lens[s] tokens and KV head h:
 *   n <= budget: every token stays;
 *   n >  budget: tokens t < sinks and t >= n - recent stay, and of the others the
 *     budget - sinks - recent with the largest weights[s][h][t]; of equal weights the lower t;
 *     -0 counts as 0, a NaN as less than everything.
 * Each head keeps tokens of its own, all the same number left = min(n, budget) of them, in
 * their order.  The j-th kept token of head h moves to place j of the new table: its K and
 * V rows are copied to block new_tables[s][j / block_size], offset j % block_size, and
 *   kept[s][h][j] = its place t before (j < left), -1 (left <= j < budget)
 *   weights_out[s][h][j] = weights[s][h][t] (j < left; -0 becomes 0, a NaN some NaN),
 *                          0 (left <= j < n), else as it was
 *   seq_lens_out[s] = left.
 * The source blocks are only read (they may be shared with other sequences); the caller
 * frees the old table afterwards.  The copied keys keep the rotation of the positions they
 * were written with; the next token's position goes on counting all tokens ever written.
 *
 *   weights        device, float32 [num_seqs][num_kv_heads][weight_stride] (pa_decode_weights
 *                  adds to it), 16-byte aligned; weight_stride a multiple of 4 and at least
 *                  max_blocks_per_seq * block_size
 *   weights_out    the same layout; may be weights itself (up to 393216 tokens of table:
 *                  beyond that PA_ERR_UNSUPPORTED), otherwise must not overlap it
 *   kept           device, int32 [num_seqs][num_kv_heads][budget]
 *   seq_lens_out   device, int32 [num_seqs]; shares no memory with the arrays below
 *   new_tables     device, int32 [num_seqs][max_new_blocks_per_seq], not block_tables itself, with
 *                  max_new_blocks_per_seq * block_size >= min(budget, max_blocks_per_seq *
 *                  block_size); entries past ceil(left / block_size) are never read.  Its
 *                  blocks must be distinct and none may be read by the call (the result is
 *                  otherwise unspecified).
 *   budget         1 .. 2^30 - 1; sinks, recent >= 0 and sinks + recent <= budget
 *   workspace      NULL, or a workspace whose status word records PA_ERR_OUT_OF_RANGE: a
 *                  length beyond the table (cut to it), a source block outside the pool (block 0
 *                  is read instead), a new block outside it (its rows are not copied)
 * Cache layout and types as pa_decode (the FP8 scales do not change).  The call's shape goes
 * by the table's width, the lengths being on the device: a table much wider than its longest
 * sequence costs time; a copy of it cut to the blocks that the longest needs does not.
 */
PA_API pa_status pa_evict(int32_t* kept, int32_t* seq_lens_out, float* weights_out, const float* weights,
                          long long weight_stride, void* k_cache, void* v_cache, const int32_t* block_tables,
                          int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* new_tables,
                          int max_new_blocks_per_seq, int num_seqs, int budget, int sinks, int recent,
                          int num_kv_heads, int head_dim, int block_size, int num_blocks, pa_dtype cache_dtype,
                          void* workspace, pa_stream_t stream);

/*
 * Block pool (host memory, no GPU work) [P1 s.4 "PagedAttention and Block
 * Management", s.5 "Prefix Caching"; P3 "The block pool", "Prefix caching is the
 * second win"].
 *
 * A pool of num_blocks physical blocks of block_size tokens.  Block 0 is the
 * null block and is never handed out, so num_blocks - 1 are usable.  Free blocks
 * wait in one queue; allocation takes them from the front.  A block in use has
 * a reference count (one per block table holding it).  A full block of a prompt
 * is registered under a chained hash (the previous block's hash, its own
 * tokens, and extra_key at the root of the chain); when its count drops to zero
 * it keeps that content and goes to the back of the queue (a request's last
 * blocks ahead of its earlier ones), so later prompts with the same prefix can
 * reuse it until the front of the queue reaches it.  A block without registered
 * content goes to the front.  Hits are checked against the stored tokens.
 *
 * Functions return PA_ERR_INVALID_ARG for bad arguments (NULL pool, an id that
 * is not in use where one must be), PA_ERR_OUT_OF_RANGE when the queue holds
 * too few blocks (then nothing changes).  A pool serialises its own calls.
 */
typedef struct pa_block_pool pa_block_pool;

/* NULL for num_blocks < 2, block_size < 1 or no memory. */
PA_API pa_block_pool* pa_pool_create(int num_blocks, int block_size);
PA_API void pa_pool_destroy(pa_block_pool* pool);
/* Blocks in the free queue (with or without reusable content). */
PA_API int pa_pool_num_free(pa_block_pool* pool);
/* Blocks holding registered prompt content (in use or free). */
PA_API int pa_pool_num_cached(pa_block_pool* pool);
/* Reference count of a block (0 when free), -1 for an id outside the pool. */
PA_API int pa_pool_ref_count(pa_block_pool* pool, int block);
/* n blocks for new content (count 1; any content they held is dropped). */
PA_API pa_status pa_pool_allocate(pa_block_pool* pool, int n, int32_t* blocks);
/* One more reference to each block (another table aliases it). */
PA_API pa_status pa_pool_share(pa_block_pool* pool, const int32_t* blocks, int n);
/* One reference less to each block, given in table order; blocks reaching zero
 * enter the free queue as described above. */
PA_API pa_status pa_pool_free(pa_block_pool* pool, const int32_t* blocks, int n);
/* Blocks for a prompt of num_tokens tokens: ceil(num_tokens / block_size)
 * entries in `blocks`.  The longest run of leading full blocks whose content is
 * registered is reused (one more reference each), never including the block
 * that holds the last token; the rest are allocated, and their full blocks
 * registered.  *hit_tokens = block_size * reused blocks. */
PA_API pa_status pa_pool_allocate_prompt(pa_block_pool* pool, const int32_t* tokens, int num_tokens,
                                         uint64_t extra_key, int32_t* blocks, int* hit_tokens);
/* Copy-on-write: every blocks[i] with more than one reference is replaced by a
 * newly allocated block (the shared one loses a reference); the (old, new) pairs
 * go to src/dst (n entries each at most) for pa_copy_blocks, *num_copies of
 * them. */
PA_API pa_status pa_pool_copy_on_write(pa_block_pool* pool, int32_t* blocks, int n, int32_t* src, int32_t* dst,
                                       int* num_copies);

/*
 * Reads (and clears) the device-side status word of a workspace.  Synchronises
 * `stream`.  Returns PA_OK, PA_ERR_TIMEOUT, PA_ERR_OUT_OF_RANGE or PA_ERR_WORKSPACE
 * (of several recorded the first in this order), or PA_ERR_CUDA if the copy failed.
 */
PA_API pa_status pa_read_device_status(void* workspace, pa_stream_t stream);

/*
 * Self-test of the bounded waits: launches one warp that waits on a barrier
 * nothing will ever complete, with a limit of timeout_us microseconds; the wait
 * must give up and record PA_ERR_TIMEOUT in the workspace status word (read it
 * with pa_read_device_status).  Touches only the status word.
 */
PA_API pa_status pa_selftest_wait_timeout(void* workspace, size_t workspace_bytes, unsigned timeout_us,
                                   pa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
