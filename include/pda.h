/*
 * pda.h -- fp8 paged decode attention for NVIDIA GB300 (sm_103a), C ABI.
 *
 * One call computes single-query ("decode") attention for a batch of
 * sequences whose keys and values sit in a paged fp8 cache:
 *
 *   out[s][h][:] = softmax_t( scale * q[s][h] . k_t ) . v_t ,  t < seq_lens[s]
 *
 * with k_t, v_t the e4m3 cache bytes of token t times k_scale / v_scale,
 * gathered page by page through block_tables, and query head h reading kv
 * head h / (num_heads / num_kv_heads).
 *
 * Sources. What the call computes and its argument roles follow the vLLM API
 * page "vllm.v1.attention.backends.rocm_aiter_unified_attn"
 * (RocmAiterUnifiedAttentionImpl.forward: q, k, v, out, seqused_k,
 * softmax_scale, block_table, k_descale, v_descale). The cache layout follows
 * vLLM pull request lishuoshuo-amd/vllm#3 ("Details", item "Layout"): for an
 * fp8 cache, K as [blocks, kv_heads, head_size/16, 16, 16] and V as
 * [blocks, kv_heads, head_size, 16] with 16-token blocks, pages addressed by
 * a dense page stride. The K intra-page order (token-major inside each
 * 16-dimension chunk) is the one the API page's _shuffle_kv_views gives
 * (K viewed as (nb, nkv, hd//x, bs, x), x = 16 bytes). Per-tensor scales
 * follow the pull request's "Scale tables" item (a table filled with the
 * per-tensor scale); block sizes that are multiples of 16 follow the API
 * page's supports_block_size / customize_spec; GQA ratios up to 8 follow the
 * pull request's "Claims" and "Cut and precision" items.
 *
 * Around that call: the cache write (pda_reshape_and_cache), rotary positions
 * alone or with it (pda_rope, pda_rope_and_cache), attention of chunks of new
 * tokens over the same cache (pda_extend), and the bookkeeping of its pages
 * (pda_grow_pages and the calls beside it).
 *
 * Threading and ordering. Every entry point is thread-safe. pda_decode is
 * stream-ordered: it validates on the host, enqueues its kernels on `stream`
 * and returns without synchronising the host, reading device memory from the
 * host, or allocating (once the workspace is large enough), so it can be
 * captured in a CUDA graph. Errors detected on the host return before any
 * launch; nothing is written to `out` then.
 */
#ifndef PDA_H_
#define PDA_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same opaque handle types as the CUDA runtime's (identical typedefs). */
typedef struct CUstream_st* cudaStream_t;
typedef struct CUevent_st* cudaEvent_t;

typedef enum pda_status {
  PDA_OK = 0,
  PDA_ERR_INVALID_ARG = 1,     /* null / misaligned pointer, negative size, H % Hk != 0 */
  PDA_ERR_UNSUPPORTED = 2,     /* valid but outside the supported set (see pda_decode) */
  PDA_ERR_WORKSPACE = 3,       /* workspace must grow while the stream is being captured */
  PDA_ERR_CUDA = 4,            /* a CUDA runtime call or kernel launch failed */
  PDA_ERR_DEVICE_TIMEOUT = 5,  /* a kernel reported a device-side error (pda_query_device_status) */
  PDA_ERR_NOALLOC_CAPACITY = 6 /* pda_decode_noalloc: the call needs more scratch than its static buffer */
} pda_status;

/*
 * pda_decode -- decode attention over a paged fp8 KV cache.
 *
 * Device pointers (all on the device that is current for the calling thread
 * and that owns `stream`; each 16-byte aligned; row-major, unpadded):
 *   out           bf16  [num_seqs][num_heads][head_size]          written
 *   q             bf16  [num_seqs][num_heads][head_size]          read
 *   k_cache       e4m3  [num_blocks][num_kv_heads][head_size/16][block_size][16]  read
 *   v_cache       e4m3  [num_blocks][num_kv_heads][head_size][block_size]          read
 *   block_tables  int32 [num_seqs][max_num_blocks_per_seq]        read
 *   seq_lens      int32 [num_seqs]                                read
 * e4m3 is OCP FP8 E4M3 (torch.float8_e4m3fn). Sequence s reads the first
 * ceil(seq_lens[s] / block_size) entries of its table row and, in its last
 * page, only the slots below seq_lens[s]; other slots and entries may hold
 * anything. A sequence with seq_lens[s] == 0 gets a zero output row.
 *
 * Scalars: scale is the softmax scale (1/sqrt(head_size) for plain
 * attention); k_scale and v_scale multiply the e4m3 values on dequantisation
 * (value = e4m3 * scale), i.e. the k/v "descale" of the API page.
 *
 * Value range: q may hold any finite bf16 values (the whole bf16 range, not
 * only f16's): each query row is scaled by a power of two before it enters
 * the f16 tensor-core products and the logit scale by its inverse, which is
 * exact. The logits scale * k_scale * q . k_t must stay finite in binary32
 * (|logit| < 2^126 suffices), and they carry binary32's relative precision:
 * with logits of magnitude X, tokens whose logits differ by less than about
 * X * 2^-22 are weighted only that precisely (at X ~ 1e5, a few tenths of a
 * percent). NaN or infinite inputs give undefined output.
 * Arithmetic: e4m3 -> f16 is exact, and so is the shifted bf16 q -> f16 for
 * every value within 2^24 of its row's largest (smaller ones round to f16's
 * subnormal grid); scores, softmax and accumulation are fp32; the
 * probabilities enter the PV product as two f16 parts (f16(p) and
 * f16(p - f16(p))), about 2^-22 relative.
 *
 * max_num_blocks_per_seq is the row stride of block_tables. It is not in the
 * argument list the method states; it is required to index a [S, MB] table
 * and gives the host an upper bound on context length without reading
 * seq_lens back from the device (which would synchronise).
 *
 * Supported set: head_size == 128; block_size a multiple of 16, 16..128;
 * num_heads % num_kv_heads == 0 with a ratio of 1..8; num_seqs >= 0
 * (0 returns PDA_OK with no launch); seq_lens[s] <= max_num_blocks_per_seq *
 * block_size and every used block id in [0, num_blocks) are the caller's
 * contract (the kernel never reads past a table row and clamps lengths to
 * the row's capacity; it does not know num_blocks). pda_set_block_check
 * makes the kernels check block ids against a given pool size;
 * pda_decode_host checks the table on the host.
 *
 * Ownership: the caller owns every buffer. The library owns an internal
 * per-(device, stream) workspace: the persistent kernel's work-queue words
 * and unit order, and the split partials. It grows with cudaMallocAsync on
 * `stream` when a call needs more and the stream is not capturing. If it is
 * capturing, a call that needs split partials returns PDA_ERR_WORKSPACE
 * (size the workspace first with pda_reserve), and a one-split call runs the
 * per-unit kernel, which needs none. Calls on one stream run in stream order
 * and share its workspace; calls on different streams have their own.
 * A CUDA graph that captured a call keeps that call's workspace address: when
 * a later, larger call grows the workspace, the old buffer is kept allocated
 * (not reused) until pda_release, so replaying the graph stays valid.
 * pda_release frees every workspace, old ones included, and so invalidates
 * every graph that captured a pda_decode* call; re-capture after it. Two
 * replays of graphs that captured calls on one stream share that stream's
 * workspace and must not run at the same time.
 *
 * Determinism: for fixed inputs and a fixed split count the result is
 * bitwise reproducible. Which CTA computes a work unit, and when, changes
 * from call to call (the persistent kernel hands units out from a queue) but
 * never changes the unit's result. The split count depends on
 * num_seqs * num_kv_heads and max_num_blocks_per_seq, so a sequence's result
 * may change in the last bits with the batch it shares a call with.
 *
 * Returns PDA_OK, PDA_ERR_INVALID_ARG, PDA_ERR_UNSUPPORTED,
 * PDA_ERR_WORKSPACE or PDA_ERR_CUDA (launch failure).
 */
pda_status pda_decode(void* out, const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                      int num_heads, int num_kv_heads, int head_size, int block_size,
                      int max_num_blocks_per_seq, float scale, float k_scale, float v_scale,
                      cudaStream_t stream);

/*
 * KV cache layouts (pda_decode_ex, pda_reshape_and_cache). K is always
 * [num_blocks][num_kv_heads][head_size/16][block_size][16].
 *   PDA_KV_NATIVE      V [num_blocks][num_kv_heads][head_size][block_size]
 *   PDA_KV_SHUFFLED_V  V [num_blocks][num_kv_heads][block_size/16][head_size][16]
 * The shuffled V is AITER's layout; at block_size 16 the two are the same
 * bytes (vLLM pull request lishuoshuo-amd/vllm#3, "Details", item "Layout";
 * the API page's _shuffle_kv_views views V as (nb, nkv, bs//x, hd, x)).
 */
typedef enum pda_kv_layout {
  PDA_KV_NATIVE = 0,
  PDA_KV_SHUFFLED_V = 1
} pda_kv_layout;

/* Output element type of pda_decode_ex. */
typedef enum pda_out_dtype {
  PDA_OUT_BF16 = 0,  /* bf16 [num_seqs][num_heads][head_size] */
  PDA_OUT_E4M3 = 1   /* e4m3 bytes [num_seqs][num_heads][head_size]: E4M3(o / output_scale) */
} pda_out_dtype;

/*
 * pda_decode_ex -- pda_decode with attention sinks and fused fp8 output.
 *
 * Source: the vLLM API page "vllm.v1.attention.backends.rocm_aiter_unified_attn"
 * passes sinks= and output_scale= to the attention call (its backend reports
 * supports_sink, and fused output quantisation for kFp8StaticTensorSym, one
 * static symmetric per-tensor scale). The page does not print either
 * computation; this library takes the plain reading of each:
 *
 *   sinks        fp32 [num_heads] on the device, or NULL. sinks[h] is a
 *                logit of query head h in the units of scale * q . k that
 *                joins the softmax normaliser and carries no value:
 *                out = sum_t e^(z_t) v_t / (sum_t e^(z_t) + e^(sinks[h])).
 *                A zero-length sequence still gives zeros.
 *   out_dtype    PDA_OUT_BF16 (as pda_decode) or PDA_OUT_E4M3: out holds
 *                e4m3 bytes E4M3(o / output_scale), the binary32 quotient
 *                rounded to the nearest e4m3 value (ties to even),
 *                saturating at +-448.
 *   output_scale finite and > 0 when out_dtype is PDA_OUT_E4M3 (ignored
 *                otherwise).
 *
 *   kv_layout    PDA_KV_NATIVE (pda_decode's layout) or PDA_KV_SHUFFLED_V.
 *
 * Everything else is pda_decode's. Returns PDA_ERR_INVALID_ARG for an
 * unknown kv_layout or out_dtype, a bad output_scale or a misaligned sinks
 * pointer.
 */
pda_status pda_decode_ex(void* out, const void* q, const void* k_cache, const void* v_cache,
                         const int32_t* block_tables, const int32_t* seq_lens, int num_seqs, int num_heads,
                         int num_kv_heads, int head_size, int block_size, int max_num_blocks_per_seq, float scale,
                         float k_scale, float v_scale, int kv_layout, const float* sinks, int out_dtype,
                         float output_scale, cudaStream_t stream);

/*
 * pda_decode_strided -- pda_decode on token-major ("flash" / NHD family)
 * caches given by byte strides.
 *
 * Source: the vLLM API page "vllm.v1.attention.backends.rocm_aiter_unified_attn":
 * the backend's kv_cache is documented as [num_blocks, 2, block_size,
 * num_kv_heads, head_size], its _split_kv_cache turns a (blocks, heads,
 * tokens, 2*head_size) tensor into K and V views of shape (blocks, tokens,
 * heads, head_size) ("keep K and V packed in the content dim"), and it
 * supports the LBHNC and LHBNC layouts. In all of these the head_size bytes
 * of one (block, token, kv head) are contiguous and everything else is a
 * stride, so one entry point covers them:
 *
 *   K row of (block b, token t, kv head h) = k_cache + b*k_block_stride
 *                                           + t*k_token_stride + h*k_head_stride
 *   (V likewise with v_cache and the v_* strides), head_size = 128 bytes, e4m3.
 *
 * Examples (bytes; D = 128):
 *   [NB, bs, Hk, D] for K and for V:  block bs*Hk*D, token Hk*D, head D
 *   [NB, 2, bs, Hk, D]:               K = base, V = base + bs*Hk*D;
 *                                     block 2*bs*Hk*D, token Hk*D, head D
 *   [NB, Hk, bs, 2*D] (K|V packed):   K = base, V = base + D;
 *                                     block Hk*bs*2*D, token 2*D, head bs*2*D
 *
 * num_blocks bounds the block index (pages are read through TMA tensor maps
 * built from these strides; a block id outside [0, num_blocks) reads zeros).
 * Strides must be positive multiples of 16 that nest without overlap once
 * sorted (smallest >= 128), and K and V must sort in the same order; else
 * PDA_ERR_UNSUPPORTED. Everything else is pda_decode's.
 */
pda_status pda_decode_strided(void* out, const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* block_tables, const int32_t* seq_lens, int num_seqs, int num_heads,
                              int num_kv_heads, int head_size, int block_size, int max_num_blocks_per_seq,
                              long long num_blocks, long long k_block_stride, long long k_token_stride,
                              long long k_head_stride, long long v_block_stride, long long v_token_stride,
                              long long v_head_stride, float scale, float k_scale, float v_scale,
                              cudaStream_t stream);

/*
 * pda_decode_slot_scales -- pda_decode with per-slot dequantisation scales.
 *
 * Source: vLLM pull request lishuoshuo-amd/vllm#3, "Details", item "Scale
 * tables": the asm kernel reads per-slot [blocks, kv_heads, block_size]
 * scales (filled there with the per-tensor scale).
 *
 *   k_scales, v_scales  fp32 [num_blocks][num_kv_heads][block_size]  read,
 *                       16-byte aligned, on the current device
 *
 * The token in slot o of block b, kv head k, dequantises as e4m3 *
 * k_scales[b][k][o] (V: v_scales[b][k][o]). Every other argument, the
 * supported set and the error behaviour are pda_decode's; tables filled with
 * one value give pda_decode's result for that per-tensor scale (up to fp32
 * rounding order). Entries of slots past a sequence's length are never used
 * (they may hold anything). Within one KV split, the largest ratio between
 * two V scales must stay below 2^15 (each probability, times its slot's V
 * scale relative to the split's first one, enters the PV product in f16
 * parts, whose range ends at 65504); the tests cover ratios of 2^14.
 * Multi-wave calls of GQA groups of at most 6 heads (4 at 128-token blocks)
 * run on the persistent kernel, whose tail pieces each take their own first
 * slot as the reference (a subset of the split: the same bound holds);
 * pda_plan_slot_scales tells which kernel a call takes.
 */
pda_status pda_decode_slot_scales(void* out, const void* q, const void* k_cache, const void* v_cache,
                                  const float* k_scales, const float* v_scales, const int32_t* block_tables,
                                  const int32_t* seq_lens, int num_seqs, int num_heads, int num_kv_heads,
                                  int head_size, int block_size, int max_num_blocks_per_seq, float scale,
                                  cudaStream_t stream);

/*
 * pda_reshape_and_cache -- KV-cache write: quantise new keys and values to
 * e4m3 with the per-tensor scales and scatter them into the paged cache.
 *
 * Source: vLLM API page "vllm.v1.attention.backends.rocm_aiter_unified_attn",
 * RocmAiterUnifiedAttentionImpl.do_kv_cache_update, which hands key, value,
 * key_cache, value_cache, slot_mapping, k_scale and v_scale to the cache
 * writer before attention runs; the page layout is pda_decode's.
 *
 *   key, value    bf16  [num_tokens][num_kv_heads][head_size]   read
 *   k_cache       e4m3  [num_blocks][num_kv_heads][head_size/16][block_size][16]  written
 *   v_cache       e4m3  as kv_layout says (PDA_KV_NATIVE: [num_blocks][num_kv_heads]
 *                 [head_size][block_size]; PDA_KV_SHUFFLED_V: [num_blocks]
 *                 [num_kv_heads][block_size/16][head_size][16])           written
 *   slot_mapping  int64 [num_tokens]: slot = block * block_size + offset;
 *                 negative = padding (skipped)
 *
 * Token t goes to block slot/block_size, offset slot%block_size; byte d of
 * kv head k is E4M3(float(x) / scale), the IEEE binary32 quotient rounded to
 * the nearest e4m3 value (ties to even), saturating at +-448 (infinities
 * included), NaN kept. Slots >= num_blocks * block_size are not written and
 * set a code in the device status word (see pda_query_device_status).
 * Slots must be distinct (two tokens writing one slot leave either value).
 * Pointers 16-byte aligned (slot_mapping 8-byte), all on the current device.
 * Supported: head_size 128, block_size a multiple of 16 up to 128. Scales
 * must be finite and nonzero. Stream-ordered, no host sync, capturable.
 */
pda_status pda_reshape_and_cache(const void* key, const void* value, void* k_cache, void* v_cache,
                                 const int64_t* slot_mapping, int num_tokens, int num_kv_heads, int head_size,
                                 int block_size, long long num_blocks, float k_scale, float v_scale, int kv_layout,
                                 cudaStream_t stream);

/*
 * pda_decode_noalloc -- pda_decode for callers that cannot allocate device
 * memory. No counterpart on the pages: this is an interface convenience of
 * this library.
 *
 * pda_decode keeps its split partials in a workspace it grows with
 * cudaMallocAsync. Some callers cannot allow that: a serving process that
 * reserved all device memory for its own pool at start-up, code that must
 * not add to the device's allocation (for example under a strict memory
 * budget or an allocator that must see every byte), or a caller whose first
 * use of a shape would otherwise trigger an allocation at a bad moment. This
 * entry point computes what pda_decode computes, with the same per-unit
 * arithmetic, but always on the per-unit decode kernel with 3 CTAs per SM
 * and the split count pda_choose_splits gives for that residency; its
 * partials live in a fixed 16 MiB array compiled into the library: every
 * GPU that loads the library holds that array until the process exits. It
 * calls no cudaMalloc, cudaFree or other allocating routine. Where
 * pda_decode plans the same split count (every batch that does not fit one
 * wave of 4 CTAs per SM) the results are bitwise equal; otherwise they
 * agree to rounding.
 *
 * Arguments, layouts, supported set and ordering are pda_decode's. Limit:
 * num_seqs * num_heads * splits * 520 bytes must fit in 16 MiB (splits is
 * the split count above; a call that needs one split uses no scratch at
 * all); larger calls return PDA_ERR_NOALLOC_CAPACITY before
 * launching anything. The first call on each device (and the first after
 * pda_release) also looks up the array's device address and the device's
 * properties (no allocation); make that call outside any stream capture. All calls on a device share
 * the one array: nothing in it needs to start at zero (each call writes the
 * partials it reads), but two calls whose kernels can run at the same time
 * on the GPU (on two streams with no ordering between them, from two host
 * threads, or from two libraries' copies in one process sharing a stream
 * order they do not control) race on it and give wrong results; order them
 * on one stream or with events. Profiling events
 * (pda_set_profile_events) are not recorded by this entry point.
 */
pda_status pda_decode_noalloc(void* out, const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* block_tables, const int32_t* seq_lens, int num_seqs, int num_heads,
                              int num_kv_heads, int head_size, int block_size, int max_num_blocks_per_seq,
                              float scale, float k_scale, float v_scale, cudaStream_t stream);

/*
 * pda_decode_host -- pda_decode on inputs and output in host memory. No
 * counterpart on the pages (whose decode call reads device tensors): an
 * interface convenience for callers whose batch lives on the host, and the
 * end-to-end path the benchmark times.
 *
 * Host pointers (layouts as pda_decode's; none needs 16-byte alignment):
 *   out           bf16  [num_seqs][num_heads][head_size]          written
 *   q             bf16  [num_seqs][num_heads][head_size]          read
 *   k_cache       e4m3  [num_blocks][num_kv_heads][head_size/16][block_size][16]  read
 *   v_cache       e4m3  [num_blocks][num_kv_heads][head_size][block_size]          read
 *   block_tables  int32 [num_seqs][max_num_blocks_per_seq]        read
 *   seq_lens      int32 [num_seqs]                                read
 * num_blocks is the number of blocks in the cache arrays (their extent,
 * which the call copies whole).
 *
 * Before anything is enqueued the host checks every table entry a sequence
 * reads (the first ceil(seq_lens[s] / block_size) of row s) against
 * [0, num_blocks) and every length against [0, max_num_blocks_per_seq *
 * block_size]; a bad entry or length returns PDA_ERR_INVALID_ARG and nothing
 * runs. Then, on `stream`: one cudaMemcpyAsync host -> device per input into
 * a staging buffer the library keeps per (device, stream), pda_decode on the
 * staged copies, and one cudaMemcpyAsync device -> host of the output. The
 * call returns without synchronising: the caller synchronises `stream`
 * before reading `out` and keeps every input unchanged and alive until then.
 * Pinned host memory (cudaHostAlloc / cudaHostRegister) makes the copies
 * asynchronous; with pageable memory they may block the calling thread.
 *
 * The staging buffer grows with cudaMallocAsync outside stream capture;
 * growing it during capture returns PDA_ERR_WORKSPACE (make one call of the
 * largest shape first). pda_release frees it. Other errors and the supported
 * set are pda_decode's.
 */
pda_status pda_decode_host(void* out, const void* q, const void* k_cache, const void* v_cache,
                           const int32_t* block_tables, const int32_t* seq_lens, int num_seqs, int num_heads,
                           int num_kv_heads, int head_size, int block_size, int max_num_blocks_per_seq,
                           long long num_blocks, float scale, float k_scale, float v_scale, cudaStream_t stream);

/*
 * pda_rope -- rotary positions of query and key heads.
 *
 * For pair i < rot_dim/2 of every head of token t, with the angle
 * positions[t] * inv_freq[i] (radians):
 *
 *   (a, b) -> magnitude * (a cos - b sin, a sin + b cos)
 *
 * where (a, b) is (x[i], x[i + rot_dim/2]) (interleaved == 0, the "half"
 * layout) or (x[2i], x[2i+1]) (interleaved != 0). Dims from rot_dim on are
 * copied unchanged (not scaled by magnitude).
 *
 *   q, k         head arrays (see pda_rope_heads); k may be NULL (or have 0
 *                heads): queries only
 *   positions    int64 [num_tokens] on the device; any value, negative ones
 *                turn backwards (so -p undoes p, up to magnitude)
 *   inv_freq     double [rot_dim/2] in HOST memory, read before the call
 *                returns: radians per position, each in [-pi, pi). Long
 *                contexts are reached by scaling these
 *                (pda_rope_frequencies)
 *   magnitude    finite factor of the rotated dims
 *
 * The angle is reduced modulo a turn in 64-bit integers, so it is as
 * accurate at position 10^6 as at 1 (about 1e-7 rad); the rotation is fp32
 * and rounds once, to bf16. out may be in (in place) when the strides agree;
 * otherwise the two must not overlap. Supported: head_size 128, rot_dim
 * even, 0..128. Heads on the 16-byte grid (base, strides) with rot_dim a
 * multiple of 16 run the wide-access kernel; anything else runs a slower one
 * of 2-byte accesses. Stream-ordered, no workspace, capturable.
 */
typedef struct pda_rope_heads {
  const void* in;               /* bf16: head h of token t at in + t*in_token_stride + h*in_head_stride */
  void* out;                    /* bf16, likewise with the out strides (ignored where nothing is written) */
  long long in_token_stride;    /* strides in elements; the head's 128 dims are contiguous */
  long long in_head_stride;
  long long out_token_stride;
  long long out_head_stride;
  int num_heads;
} pda_rope_heads;

pda_status pda_rope(const pda_rope_heads* q, const pda_rope_heads* k, const int64_t* positions, int num_tokens,
                    int head_size, const double* inv_freq, int rot_dim, int interleaved, float magnitude,
                    cudaStream_t stream);

/*
 * pda_rope_and_cache -- pda_rope and pda_reshape_and_cache in one pass:
 * rotates q into q->out, and writes the rotated keys and the values into the
 * paged cache as e4m3.
 *
 * A key is rotated in fp32 and quantised from there, so it rounds once (the
 * two calls in a row round twice, by way of bf16, and can differ from this
 * one by an e4m3 step). v->in is not rotated; k->out and v->out are ignored.
 * slot_mapping, the caches, scales, kv_layout, padding (negative slots write
 * nothing to the cache; their q is rotated all the same) and slots past the
 * pool are as for pda_reshape_and_cache, rotary arguments as for pda_rope. A
 * slot that a call names twice ends with bytes of either token, not
 * necessarily all of one. 16 consecutive tokens (counted from the call's
 * first) whose slots are consecutive from a multiple of 16 on are written
 * fastest.
 * q->out must not overlap k->in or v->in.
 */
pda_status pda_rope_and_cache(const pda_rope_heads* q, const pda_rope_heads* k, const pda_rope_heads* v,
                              const int64_t* positions, const int64_t* slot_mapping, int num_tokens, int head_size,
                              const double* inv_freq, int rot_dim, int interleaved, float magnitude, void* k_cache,
                              void* v_cache, int block_size, long long num_blocks, float k_scale, float v_scale,
                              int kv_layout, cudaStream_t stream);

/*
 * pda_rope_frequencies -- inv_freq and magnitude for pda_rope (host only,
 * pure). Plain: inv_freq[i] = base^(-2i/rot_dim), magnitude 1. The scalings
 * stretch a context by `factor` >= 1:
 *   PDA_ROPE_LINEAR  every frequency divided by factor
 *   PDA_ROPE_BASE    base raised to base * factor^(rot_dim/(rot_dim-2)): the
 *                    fastest pair kept, the slowest divided by factor
 *   PDA_ROPE_RAMP    pairs that make more than `high` turns over
 *                    original_length kept, those below `low` divided by
 *                    factor, a linear ramp over the pair index between (its
 *                    ends rounded outwards to whole indices); magnitude
 *                    0.1 ln(factor) + 1 (the YaRN paper, arXiv 2309.00071;
 *                    it uses low 1, high 32)
 *   PDA_ROPE_BANDS   the same two bands by turns over original_length, with
 *                    a blend linear in the turns between (usual: low 1,
 *                    high 4); magnitude 1
 * original_length, low and high are read by RAMP and BANDS only (all > 0,
 * high > low). magnitude may be NULL.
 */
typedef enum pda_rope_scaling {
  PDA_ROPE_PLAIN = 0,
  PDA_ROPE_LINEAR = 1,
  PDA_ROPE_BASE = 2,
  PDA_ROPE_RAMP = 3,
  PDA_ROPE_BANDS = 4
} pda_rope_scaling;

pda_status pda_rope_frequencies(double* inv_freq, double* magnitude, int rot_dim, double base, int scaling,
                                double factor, double original_length, double low, double high);

/*
 * pda_extend -- causal attention of new tokens over the paged cache: a chunk
 * of a prompt, drafted tokens to check, or a batch that mixes chunks with
 * single tokens.
 *
 *   out, q        [num_tokens][num_heads][head_size], the new tokens of all
 *                 sequences packed one after the other
 *   query_starts  int32 [num_seqs + 1]: sequence s owns rows
 *                 [query_starts[s], query_starts[s+1]) (nondecreasing, within
 *                 [0, num_tokens]; a sequence may own none). Rows that
 *                 belong to no sequence (in front of the first, behind the
 *                 last) are left as they were
 *   seq_lens      int32 [num_seqs]: tokens in the cache, the new ones (whose
 *                 K and V must already be written) included
 *
 * With n the rows of sequence s, its row i stands at position
 * p = seq_lens[s] - n + i and attends to tokens max(0, p - window + 1) .. p
 * (window > 0) or 0 .. p (window == 0: no limit); a row with p < 0 (fewer
 * tokens in the cache than rows) gets zeros. The probabilities enter the
 * second product as one f16 each, half a step (2^-11) off relative to
 * themselves, where pda_decode takes two f16 parts (2^-22): at most 2^-11 of
 * the weighted mean of |v| in an output, and probabilities below about 2^-31 of
 * the row's largest may vanish. The normaliser sums them in fp32, unrounded.
 * Everything else (cache, table, scales, sinks, out_dtype, output_scale,
 * kv_layout, supported set, value range, logits' precision,
 * pda_set_block_check) is as for pda_decode / pda_decode_ex; the
 * first row's position and the window also bound which table entries are
 * read: those of pages that hold a token some row attends to. A NaN among the
 * tokens below seq_lens[s] gives undefined output in the sequence's rows.
 *
 * Limits: as pda_decode, and num_tokens * num_heads < 2^31. A call whose
 * tiles do not fill the GPU splits the KV range and needs a workspace per
 * (device, stream) for the partials, grown, kept and shared as pda_decode's
 * is; captured without one (pda_reserve_extend, or an earlier call of the same
 * sizes on that stream) it runs unsplit. The result may differ in the last bits
 * with the split; for one split count it is bitwise reproducible.
 */
pda_status pda_extend(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                      const int32_t* seq_lens, const int32_t* query_starts, int num_tokens, int num_seqs,
                      int num_heads, int num_kv_heads, int head_size, int block_size, int max_num_blocks_per_seq,
                      float scale, float k_scale, float v_scale, int window, int kv_layout, const float* sinks,
                      int out_dtype, float output_scale, cudaStream_t stream);

/* pda_reserve_extend -- size the workspace of (current device, stream) for
 * pda_extend calls of up to num_tokens, num_seqs and max_num_blocks_per_seq,
 * with these heads and this block size. It is the page calls' workspace too. */
pda_status pda_reserve_extend(int num_tokens, int num_seqs, int num_heads, int num_kv_heads,
                              int max_num_blocks_per_seq, int block_size, cudaStream_t stream);

/*
 * Pages. The calls below keep a block table, its lengths and a reference
 * count per page on the device, so that a captured step can grow, fork and
 * free sequences without the host.
 *
 *   ref_counts    int32 [num_blocks]: table entries that hold the page; a
 *                 page with count 0 is free. A caller that holds a page
 *                 itself (a prefix kept for later) adds 1
 *   block_tables  int32 [num_rows][max_num_blocks_per_seq]
 *   seq_lens      int32 [num_rows]: row r holds its first
 *                 ceil(seq_lens[r] / block_size) entries; others are unused
 *                 and left as they are
 *
 * All on the current device, updated in place in stream order. New pages are
 * the lowest free ids in the order of the requests: the outcome is a function
 * of the state alone. Requests are lists of row numbers on the device;
 * negative rows are padding. A request that cannot be served (a row out of
 * range, a row that an earlier request of the call already named, a length
 * past the table row, too few free pages: request i is short when requests
 * 0..i together need more pages than are free) changes nothing and sets bit 128 of the
 * device status word (pda_query_device_status); table entries outside
 * [0, num_blocks) are skipped and set bit 64.
 *
 * The calls share one workspace per (device, stream), grown like
 * pda_decode's (PDA_ERR_WORKSPACE when it must grow during capture: size it
 * with pda_reserve_pages) and freed by pda_release; calls on one stream run
 * in its order, and those of several threads follow each other whole (no
 * kernel of one call falls between two of another's). block_size a multiple
 * of 16 up to 128.
 */
typedef struct pda_page_table {
  int32_t* ref_counts;
  int32_t* block_tables;
  int32_t* seq_lens;
  long long num_blocks;
  int num_rows;
  int max_num_blocks_per_seq;
  int block_size;
} pda_page_table;

/* One array of pages: a layer's K cache, V cache or scale table. The page of
 * block b is the bytes_per_block bytes at base + b * bytes_per_block; base
 * 16-byte aligned, bytes_per_block a multiple of 16. Arrays of one call must
 * not overlap. */
typedef struct pda_page_array {
  void* base;
  long long bytes_per_block;
} pda_page_array;

/* pda_copy_pages -- pages src[i] -> dst[i] in every array. src, dst int32
 * [num_pairs] on the device; pairs with a negative entry, or src == dst, are
 * skipped, ids past num_blocks are skipped and set bit 64. Targets must be
 * distinct and no source of the call. arrays is host memory. */
pda_status pda_copy_pages(const pda_page_array* arrays, int num_arrays, const int32_t* src, const int32_t* dst,
                          int num_pairs, long long num_blocks, cudaStream_t stream);

/* pda_grow_pages -- row rows[i] takes add[i] >= 0 more tokens: its length
 * grows, and it gets fresh pages where its last page does not hold them. */
pda_status pda_grow_pages(const pda_page_table* table, const int32_t* rows, const int32_t* add, int n,
                          cudaStream_t stream);

/* pda_fork_pages -- row children[i], which must be empty, becomes a copy of
 * row parents[i]: the parent's full pages are shared (their counts grow),
 * a last page that is partly filled is copied, in every array, to a fresh
 * page of the child's own, so that both rows can grow. A row that is a child
 * of the call cannot be a parent in it. arrays (host memory) may be empty: the
 * bookkeeping alone. A child's row stays empty until its entries and its page
 * are in place. */
pda_status pda_fork_pages(const pda_page_table* table, const int32_t* parents, const int32_t* children, int n,
                          const pda_page_array* arrays, int num_arrays, cudaStream_t stream);

/* pda_free_pages -- rows rows[i] become empty and give their pages up (a row
 * named twice is freed once). */
pda_status pda_free_pages(const pda_page_table* table, const int32_t* rows, int n, cudaStream_t stream);

/* pda_compact_pages -- moves pages so that the L held pages are ids 0..L-1:
 * the k-th free id below L takes the k-th held page at or above L, in every
 * array; counts move along, and every table entry in use follows (one that
 * names a free page stays as it is and sets bit 128). new_ids
 * (int32 [num_blocks] on the device, or NULL) receives each page's id after
 * the call, for holders outside the table. */
pda_status pda_compact_pages(const pda_page_table* table, const pda_page_array* arrays, int num_arrays,
                             int32_t* new_ids, cudaStream_t stream);

/* pda_reserve_pages -- size the page calls' workspace of (current device,
 * stream) for pools and tables up to these sizes and calls of up to
 * max_requests requests. */
pda_status pda_reserve_pages(long long num_blocks, int num_rows, int max_requests, cudaStream_t stream);

/* Static text for a status code; never NULL. */
const char* pda_status_string(int status);

/*
 * pda_choose_splits -- the split-count heuristic (pure, host only).
 *
 * Returns how many KV splits each (sequence, kv head) work unit is cut into
 * for a batch of num_seqs * num_kv_heads units with at most
 * max_num_blocks_per_seq pages of block_size tokens, on a device with
 * sm_count SMs that hold ctas_per_sm decode CTAs each. Like the pull
 * request's dispatch rule ("Claims": work units compared with the
 * compute-unit count), it compares work units with the resident CTA slots:
 * a unit is split when its K/V bytes (at max_num_blocks_per_seq pages)
 * exceed 1 MiB, or when the units fill less than one wave of slots (then up
 * to one wave), never below 256 tokens per split. Result in
 * [1, max(1, max_num_blocks_per_seq)]. Invalid arguments return 1.
 */
int pda_choose_splits(int num_seqs, int num_kv_heads, int max_num_blocks_per_seq, int block_size,
                      int sm_count, int ctas_per_sm);

/*
 * pda_plan_splits -- the split count pda_decode would use on the current
 * device for these sizes (heuristic or override). Returns < 1 on error.
 */
int pda_plan_splits(int num_seqs, int num_heads, int num_kv_heads, int max_num_blocks_per_seq,
                    int block_size);

/* Decode kernel instances (pda_plan_kernel). */
typedef enum {
  PDA_KERNEL_PER_UNIT = 0,       /* one CTA per work unit, 3 CTAs per SM, 64 KiB page ring */
  PDA_KERNEL_PER_UNIT_DENSE = 1, /* one CTA per work unit, 4 CTAs per SM, 48 KiB page ring */
  PDA_KERNEL_PERSISTENT = 2      /* one CTA per resident slot working through a queue of units */
} pda_kernel;

/*
 * pda_plan_kernel -- the decode kernel instance pda_decode (and pda_decode_ex,
 * and pda_decode_strided with token-major pages) would launch on the current
 * device for these sizes: the dense per-unit
 * instance when the planned grid fits one wave of 4 CTAs per SM, else the
 * persistent kernel. A call captured into a CUDA graph without a prior
 * pda_reserve (so with no workspace for the persistent kernel's queue) runs
 * the 3-CTA per-unit instance instead. Diagnostic; returns < 0 on error.
 */
int pda_plan_kernel(int num_seqs, int num_heads, int num_kv_heads, int max_num_blocks_per_seq, int block_size);

/*
 * pda_choose_kernel -- the planner's choice for a pda_decode call (pure,
 * host only, no device needed): for a batch of num_seqs * num_kv_heads
 * units with at most max_num_blocks_per_seq pages of block_size tokens, on a
 * device with sm_count SMs holding ctas_per_sm per-unit / persistent CTAs
 * or ctas_per_sm_dense dense per-unit CTAs each. Returns the PDA_KERNEL_*
 * instance and, when the pointers are non-NULL, stores the split count and
 * the kernels launched per call. The dense per-unit instance is chosen when
 * its grid fits one wave, else the persistent kernel (the 3-CTA per-unit
 * kernel past 2^31 units). The split count follows pda_choose_splits with
 * the chosen residency; the split override is not applied. Invalid
 * arguments return -1. pda_plan_kernel / pda_plan_splits / pda_plan_launches
 * give the same answers for the current device.
 */
int pda_choose_kernel(int num_seqs, int num_kv_heads, int max_num_blocks_per_seq, int block_size, int sm_count,
                      int ctas_per_sm, int ctas_per_sm_dense, int* num_splits, int* launches);

/*
 * pda_plan_launches -- kernels one pda_decode call launches for these sizes
 * on the current device: the decode kernel, plus the unit-order kernel when
 * the persistent kernel has more units than resident CTAs (up to 16384
 * units), plus the tail merge kernel when those units leave a partial last
 * round (units modulo resident CTAs > 0; it runs even when no unit of that
 * round is long enough to cut), plus the merge kernel when the call splits
 * (with pda_set_tail_split(0): no tail merge kernel). A one-wave per-unit
 * call of 2 to 16 splits has no merge launch: the splits of each (sequence,
 * kv head) run as one thread-block cluster and combine their results
 * through distributed shared memory. 0 for num_seqs == 0;
 * < 0 on error. Diagnostic (counts graph nodes, profiler launches).
 */
int pda_plan_launches(int num_seqs, int num_heads, int num_kv_heads, int max_num_blocks_per_seq, int block_size);

/*
 * pda_tail_pieces -- the tail-piece cut the persistent kernel makes (host
 * only; no device is needed). A call whose units overrun the resident CTAs
 * (`ctas`) by a partial last round of `tail_units` units (0 < tail_units <
 * ctas) cuts each of those units of `pages` pages (of its split) into
 * pieces: at least 256 tokens each, units under 1024 tokens whole, pieces
 * that shrink toward the end of the hand-out when tail_units >= ctas / 3,
 * else equal ones. Writes the first min(pieces, max_sizes) piece sizes in
 * pages to `sizes` (in hand-out order within the unit) and returns the
 * piece count; -1 for invalid arguments. Diagnostic (tests, tuning); no
 * counterpart in the pages (a scheduling choice, not part of what the
 * operation computes).
 */
int pda_tail_pieces(int pages, int tail_units, int ctas, int block_size, int* sizes, int max_sizes);

/*
 * pda_plan_slot_scales -- the plan pda_decode_slot_scales makes for these
 * sizes on the current device. *kernel receives PDA_KERNEL_PERSISTENT when
 * the grid is past one wave of 3 CTAs per SM and the GQA group's query rows
 * leave room for a stage's scale rows in the persistent kernel's side
 * entries (g <= 6 at 16- to 64-token blocks, g <= 4 at 128), else
 * PDA_KERNEL_PER_UNIT; *num_splits the split count; *launches the kernels
 * one call launches (the unit-order, tail merge and merge kernels as for
 * pda_decode). Any out pointer may be NULL. Returns 0, or -1 for invalid
 * sizes or a CUDA error. Diagnostic.
 */
int pda_plan_slot_scales(int num_seqs, int num_heads, int num_kv_heads, int max_num_blocks_per_seq, int block_size,
                         int* kernel, int* num_splits, int* launches);

/*
 * pda_set_split_override -- force the split count of later pda_decode calls
 * (process-wide; 0 restores the heuristic). For tests and measurements.
 * Values above the table row length are clamped at call time.
 */
void pda_set_split_override(int num_splits);

/*
 * pda_set_tail_split -- tail pieces of the persistent kernel (process-wide;
 * on by default). When a multi-wave batch hands out its units in
 * longest-first order, the units of the last, partial round (units modulo
 * resident CTAs, at most 1024) that hold at least 1024 tokens are cut into
 * pieces of at least 256 tokens, at most 8 per unit, that the CTAs done with
 * their whole units share. A tail merge kernel, launched as the decode
 * kernel's programmatic dependent, folds the pieces' (O, m, l) in piece
 * order and stores the unit's result (or the split's partial, which the
 * merge kernel then folds), so the result of such a unit is not bitwise
 * the whole unit's (it is the same softmax, within rounding). 0 turns the
 * pieces off for later calls (tests that compare kernels bit for bit,
 * measurements).
 */
void pda_set_tail_split(int enable);

/*
 * pda_set_tma_gather -- four-row TMA gathers (process-wide; on by default).
 * With 16-token blocks the persistent decode kernel copies a stage's four
 * K pages and four V pages as one tile::gather4 copy per cache, and the
 * per-slot-scale entry point (pda_decode_slot_scales) a stage's four K and
 * four V scale rows as one gather per table (larger blocks: one bulk copy
 * per scale row). 0 copies pages one bulk copy each and scale rows as
 * 16-byte cp.async pieces, for later calls. The same bytes arrive either
 * way, so results are bitwise equal; for tests and measurements. No
 * counterpart in the pages (a copy strategy, not part of what the
 * operation computes).
 */
void pda_set_tma_gather(int enable);

/*
 * pda_set_block_check -- device-side check of block ids for later decode
 * calls (process-wide). pda_decode, pda_decode_ex, pda_decode_slot_scales
 * and pda_decode_noalloc are not given the pool size, so a table entry
 * outside the pool would make them read outside k_cache / v_cache (the
 * caller's error, see pda_decode). With num_blocks > 0 their kernels check
 * every block id they read against [0, num_blocks): an id outside it sets
 * bit 64 of the device status word (pda_query_device_status) and its page is
 * read from block 0 instead, so that call's output is wrong but no read
 * leaves the pool. 0 (the default) turns the check off. pda_decode_strided
 * and pda_decode_host, which are given the pool size, bound their reads
 * themselves. For debugging and for callers that cannot vouch for their
 * tables; the check adds a compare per block id in the producer warp.
 */
void pda_set_block_check(long long num_blocks);

/*
 * pda_reserve -- size the workspace of (current device, stream) for calls up
 * to these sizes (any entry point's plan: queue words, unit order, split
 * partials), so later calls (for example under stream capture) need no
 * allocation. Stream-ordered; returns PDA_OK or PDA_ERR_CUDA.
 */
pda_status pda_reserve(int num_seqs, int num_heads, int num_kv_heads, int max_num_blocks_per_seq,
                       int block_size, cudaStream_t stream);

/*
 * pda_release -- free every workspace and staging buffer the library holds,
 * the ones that growth retired included (synchronises each device used),
 * and forget the per-device set-up (SM counts, kernel attributes, the
 * pda_decode_noalloc array's address), which the next call takes again.
 * Graphs that captured a pda_decode*, pda_decode_host, pda_extend or page call
 * refer to freed memory afterwards and must not be replayed. A cudaDeviceReset destroys
 * everything the library set up on that device: call pda_release before
 * resetting a device the library has used.
 */
pda_status pda_release(void);

/*
 * pda_workspace_info -- the decode workspace of (current device, stream; the
 * one that pda_extend and the page calls share is apart): *bytes
 * receives its current size (0 when it has none) and *retired the number of
 * smaller buffers it replaced that are still allocated for graphs that
 * captured them. Diagnostic; host only, no synchronisation.
 */
pda_status pda_workspace_info(cudaStream_t stream, long long* bytes, int* retired);

/*
 * pda_query_device_status -- synchronise `stream`, then read and clear the
 * device status word of the current device. *code receives 0 when every
 * kernel since the last query finished normally, or a nonzero code when a
 * kernel gave up on a bounded wait, or skipped or redirected an access
 * outside the pool (a cache-write slot past the pool: bit 16; with
 * pda_set_block_check, or in the page calls, a block id outside the pool: bit
 * 64), or refused a page request (bit 128, which changes nothing); the output
 * of that call is then undefined but for what the call says of it. Returns PDA_ERR_DEVICE_TIMEOUT when
 * *code != 0. Test / debug call: it blocks.
 */
pda_status pda_query_device_status(cudaStream_t stream, int* code);

/*
 * pda_set_profile_events -- when both events are non-NULL, later pda_decode
 * calls record `before` immediately before and `after` immediately after the
 * split-KV decode kernel on their stream (capturable); with the persistent
 * kernel's unit-order kernel, `before` precedes that one too (the two run
 * overlapped), and with its tail merge kernel, `after` follows that one too
 * (a programmatic dependent of the decode kernel). The split merge kernel
 * stays outside. NULL, NULL turns it off. Process-wide; for measurement only.
 */
void pda_set_profile_events(cudaEvent_t before, cudaEvent_t after);

/*
 * pda_test_bounded_wait -- launch one CTA that waits on a barrier nothing
 * will complete, with a limit of timeout_us microseconds, on `stream`. The
 * kernel gives up, records PDA timeout code in the device status word and
 * returns (no trap, no fault); pda_query_device_status then reports it.
 * Exercises the bounded-wait error path of the decode kernel's barriers.
 * timeout_us must be in [1, 2000000].
 */
pda_status pda_test_bounded_wait(int timeout_us, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PDA_H_ */
