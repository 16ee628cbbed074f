/*
 * nf4.h - C ABI of the NF4 weight-only linear layer library (libnf4.so, NVIDIA GB300 / sm_103a).
 *
 * Format (deep-fold README, wertick01/deep-fold, format paragraph): weights are stored in groups of
 * 64 consecutive in-features of one output row; each group holds 64 four-bit NF4 codes and one
 * FP16 scale.  NF4 is the 16-value NormalFloat table introduced with QLoRA (deep-fold README,
 * method paragraph; values published by Dettmers et al., 2023).  The library fixes what the pages
 * leave open:
 *   - codes[N][K/2] (uint8): weight (n, 2j) in the low nibble of byte (n, j), weight (n, 2j+1) in
 *     the high nibble;
 *   - scales[N][K/64] (IEEE binary16 bits): scale of group g of row n = fp16 round-to-nearest-even
 *     of s = max |w[n][64g .. 64g+63]| computed in fp32;
 *   - code of w = the index i minimising the fp32 distance |fp32(w / s) - T[i]|, ties to the lower
 *     index; an all-zero group (s = 0) gets code 7 (T[7] = 0);
 *   - dequantized weight w_hat = bf16_rn(fp32(T[code] * float(scale)));
 *   - y[m][n] = bf16_rn(sum_k x[m][k] * w_hat[n][k]) with at least fp32 accumulation.  Accepted
 *     results satisfy |y - y64| <= 2^-8 |y64| + 2^-12 sum_k |x[m][k] w_hat[n][k]|, y64 being the
 *     same sum in exact products and double-precision addition.
 *
 * Common rules for every entry point:
 *   - Pointers are device pointers owned by the caller, row-major and contiguous, each aligned to
 *     16 bytes where nothing else is said.  bf16 and fp16 values travel as their 16-bit patterns (uint16_t).
 *   - Calls are asynchronous on `stream` (0 = the legacy default stream).  No call synchronises
 *     the device, allocates memory or keeps state beyond a per-device capability check, except the
 *     ring calls of the overflow-streaming section, which own explicitly created state.  (The
 *     attention keeps counters in the workspace that its caller passes.)
 *   - Arguments are checked on the host before anything is launched; on an error nothing is
 *     launched and no output is written.  A failed launch returns NF4_ERR_CUDA and leaves the CUDA
 *     error state cleared.
 *   - Shapes: N and M may be 0 (nothing is launched, NF4_OK); K must be a positive multiple of 64;
 *     M, N and K must each be at most 2^31 - 1.
 *   - Non-finite inputs are outside the contract: results are unspecified, but no call faults.
 *   - The same inputs give the same output bytes on every call (fixed reduction order; atomics only
 *     hand out the attention's work, add integers, and list candidates whose order is then settled).
 *   - Every call may be captured into a CUDA graph (the kernels build their constant tables in
 *     shared memory at launch; no call needs one-time device work), except the first call of
 *     nf4_linear_host_noalloc on a device (see there).
 *   - Every pipeline wait inside the kernels is bounded (one second of wall-clock time per wait by
 *     default).  A wait that runs out records a code in the device error word, and the kernel
 *     drains and exits instead of hanging; the call itself has already returned NF4_OK and the
 *     outputs of that launch are then unspecified.  Callers that need to know read the word with
 *     nf4_check_device_error (the tests and the benchmark do after every timed region).
 *   - Every entry point except the ring calls (see their section) may be called from several host
 *     threads at once, on the same or different streams: the only shared state is the per-device
 *     capability cache (atomic) and one-time kernel attributes (std::call_once).
 */
#ifndef NF4_H
#define NF4_H

#include <stdint.h>

#include <cuda_runtime_api.h> /* cudaStream_t */

#ifdef __cplusplus
extern "C" {
#endif

#define NF4_GROUP_SIZE 64
#define NF4_ABI_VERSION 3

typedef enum nf4_status {
    NF4_OK = 0,
    NF4_ERR_NULL = 1,               /* a required pointer is NULL */
    NF4_ERR_SHAPE = 2,              /* negative size, K not a positive multiple of 64, or > 2^31-1 */
    NF4_ERR_ALIGN = 3,              /* a pointer is not aligned as its call asks (16 bytes) */
    NF4_ERR_ALIAS = 4,              /* an output range overlaps an input range */
    NF4_ERR_UNSUPPORTED_DEVICE = 5, /* the current device is not compute capability 10.3 (sm_103) */
    NF4_ERR_CUDA = 6,               /* a CUDA runtime call or kernel launch failed */
    NF4_ERR_MEMORY = 7,             /* memory of the wrong kind: a host pointer that is not page-locked,
                                       or a ring used on a device other than its own */
    NF4_ERR_CAPTURE = 8             /* the first nf4_linear_host_noalloc call on a device was made while
                                       `stream` is being captured into a CUDA graph: its one-time set-up
                                       cannot run inside a capture */
} nf4_status;

/*
 * nf4_quantize - pack fp32 weights into NF4 codes and fp16 group scales.
 * Defines: the format paragraph of the deep-fold README (64-weight groups, 4-bit NF4 codes, one
 * FP16 scale); the pages do this offline in their compressor, here it is a device kernel.
 *   w       in   float [N][K]
 *   codes   out  uint8 [N][K/2]   low nibble first
 *   scales  out  fp16 bits [N][K/64]
 * codes and scales must not overlap w or each other.
 */
nf4_status nf4_quantize(const float* w, int64_t N, int64_t K, uint8_t* codes, uint16_t* scales,
                        cudaStream_t stream);

/*
 * nf4_dequant - expand packed weights to a dense bf16 matrix (a test and inspection entry point:
 * the linear layer below never writes this matrix, as the execution-path table of the deep-fold
 * README requires).
 *   codes   in   uint8 [N][K/2]
 *   scales  in   fp16 bits [N][K/64]
 *   w_hat   out  bf16 bits [N][K], w_hat = bf16_rn(fp32(T[code] * float(scale)))
 */
nf4_status nf4_dequant(const uint8_t* codes, const uint16_t* scales, int64_t N, int64_t K,
                       uint16_t* w_hat, cudaStream_t stream);

/*
 * nf4_linear - y = x * w_hat^T with the weights streamed in packed form and dequantized tile by
 * tile on chip (deep-fold README, execution-path table: N=1 decode GEMV, prefill GEMM of up to 32
 * positions; larger M is this library's extension).  M <= 3 runs a CUDA-core GEMV (K up to 32768
 * for M = 1, 16384 for M = 2..3); M <= 32, and M <= 3 with a longer K, run a weight-streaming
 * kernel that dequantizes on the CUDA cores into tensor memory and multiplies on the tcgen05 tensor
 * cores (one CTA per SM, K split into slices when a CTA has few rows); larger M runs a tcgen05 GEMM
 * over 128-row weight tiles.  The kernel depends on M and K; the K split on M, N and the SM count.
 *   x       in   bf16 bits [M][K]
 *   codes   in   uint8 [N][K/2]
 *   scales  in   fp16 bits [N][K/64]
 *   y       out  bf16 bits [M][N]; must not overlap x, codes or scales
 */
nf4_status nf4_linear(const uint16_t* x, const uint8_t* codes, const uint16_t* scales, uint16_t* y,
                      int64_t M, int64_t N, int64_t K, cudaStream_t stream);

/*
 * nf4_linear_grouped - several linears that read the same x, y_i = x * w_hat_i^T for i < count
 * (for instance the q, k and v projections, or the gate and up projections, of one decoder layer;
 * the deep-fold README's execution-path table runs decode as GEMVs over such linears).  For M <= 32
 * the linears share one launch over their rows; for larger M they run one GEMM after another on
 * `stream`.  Each y_i meets the nf4_linear bound and repeated calls give the
 * same bytes; the K split can differ from a separate nf4_linear call, so low-order bits may too.
 *   x        in   bf16 bits [M][K], shared by all linears
 *   count    1 .. 8
 *   codes    host array of count device pointers; codes[i]: uint8 [Ns[i]][K/2]
 *   scales   host array of count device pointers; scales[i]: fp16 bits [Ns[i]][K/64]
 *   ys       host array of count device pointers; ys[i]: bf16 bits [M][Ns[i]]; no y may overlap x,
 *            any codes or scales, or another y
 *   Ns       host array of count row counts (each >= 0, sum <= 2^31 - 1); empty linears are skipped
 * The host arrays are read before the call returns.  Errors as for nf4_linear (count outside
 * 1..8 gives NF4_ERR_SHAPE).
 */
nf4_status nf4_linear_grouped(const uint16_t* x, int64_t M, int64_t K, int count, const uint8_t* const* codes,
                              const uint16_t* const* scales, uint16_t* const* ys, const int64_t* Ns,
                              cudaStream_t stream);

/*
 * nf4_embed - rows of a packed embedding table, dequantized on request (deep-fold README, overview
 * paragraph: embeddings reconstruct only the rows that are asked for; the 20B run of its results
 * uses these packed embedding rows).  The table has the same format as a linear's weights: V rows
 * of K dimensions, groups of 64 along K with one FP16 scale each.
 *   ids     in   int32 [n_ids]; each should be in [0, V)
 *   codes   in   uint8 [V][K/2]
 *   scales  in   fp16 bits [V][K/64]
 *   out     out  bf16 bits [n_ids][K], out[i][k] = bf16_rn(fp32(T[code] * float(scale))) of row ids[i]
 *            (bit for bit the rows nf4_dequant would write); must not overlap ids, codes or scales
 * An id outside [0, V) gives a row of zeros and records code 41 in the device error word (see
 * nf4_check_device_error); nothing is read for it.  n_ids = 0 is a no-op.  Other errors as for
 * nf4_dequant.
 */
nf4_status nf4_embed(const int32_t* ids, int64_t n_ids, const uint8_t* codes, const uint16_t* scales, int64_t V,
                     int64_t K, uint16_t* out, cudaStream_t stream);

/*
 * Overflow streaming (deep-fold README, overview and execution-path table: a model larger than the
 * card keeps part of its packed weights in pinned host memory and copies them through two reusable
 * device slots, overlapped with the same GEMV / GEMM; the 32B row of its results runs this way).
 *
 * A ring is the one stateful object of the library: two device slots, a copy stream and events,
 * created on the current device.  nf4_ring_run walks a list of linears whose packed weights live in
 * page-locked host memory.  Linear i is copied into slot i mod 2 on the ring's copy stream (after
 * the linear that last read that slot has finished) and then runs as nf4_linear on `stream`, so
 * the copy of linear i + 1 overlaps the compute of linear i.  The linears run in list order on
 * `stream`, so the y of one may be the x of a later one.  Results are bit for bit those of
 * nf4_linear on device-resident copies of the same weights.
 */
typedef struct nf4_ring nf4_ring;

/* One linear of a streamed list. */
typedef struct nf4_host_linear {
    const uint16_t* x;      /* device, bf16 bits [M][K] */
    const uint8_t* codes;   /* page-locked host, uint8 [N][K/2] */
    const uint16_t* scales; /* page-locked host, fp16 bits [N][K/64] */
    uint16_t* y;            /* device, bf16 bits [M][N]; must not overlap x */
    int64_t M, N, K;        /* as for nf4_linear; M = 0 or N = 0 skips the entry */
} nf4_host_linear;

/*
 * nf4_ring_create - allocate a ring whose two slots hold up to `slot_bytes` of packed weights each:
 * a linear fits when N*K/2 rounded up to 256, plus N*(K/64)*2, is at most slot_bytes.
 *   slot_bytes  > 0
 *   ring        out: the new ring (NULL on error)
 * Errors: NF4_ERR_NULL, NF4_ERR_SHAPE (slot_bytes <= 0), NF4_ERR_UNSUPPORTED_DEVICE, NF4_ERR_CUDA
 * (allocation failed; nothing is left allocated).
 */
nf4_status nf4_ring_create(int64_t slot_bytes, nf4_ring** ring);

/*
 * nf4_ring_run - stream `count` linears through the ring, asynchronously on `stream`.
 *   ring    from nf4_ring_create, used on its own device
 *   ops     host array of count entries (read before the call returns)
 *   count   >= 0 (0 is a no-op)
 * Every entry is checked before anything is enqueued: shapes and alignment as for nf4_linear,
 * NF4_ERR_SHAPE when an entry does not fit a slot, NF4_ERR_MEMORY when codes or scales are not
 * page-locked host memory (first and last byte checked) or the current device is not the ring's.
 * The host buffers must stay unchanged until the work enqueued by the call has finished.  A ring
 * may be captured into a CUDA graph: a captured run orders its copies after the work already on
 * `stream`, and so do the ring's eager runs from then on; a graph and eager runs that share a ring
 * must therefore be issued on one stream (or be ordered by the caller).  Calls on one ring must not run concurrently from several host threads; runs on
 * different streams are ordered through the ring's events.  A CUDA failure part way returns
 * NF4_ERR_CUDA with the earlier entries enqueued.
 */
nf4_status nf4_ring_run(nf4_ring* ring, const nf4_host_linear* ops, int64_t count, cudaStream_t stream);

/* nf4_ring_destroy - wait for the ring's outstanding work and free it.  NULL is a no-op. */
nf4_status nf4_ring_destroy(nf4_ring* ring);

/*
 * nf4_linear_host_noalloc - one linear whose packed weights live in page-locked host memory, staged
 * through a device buffer that is part of the library itself, so that nothing is allocated.  The
 * pages have no counterpart: it is an addition of this library.
 *
 * Who needs it: a caller that cannot allocate device memory when it runs the layer.  Examples: a
 * host application whose own pool allocator has already reserved the GPU's memory (a cudaMalloc
 * from the library would fail or fragment that pool), or a decode loop that cannot afford
 * cudaMalloc / cudaFree, which may synchronise the whole device.  nf4_ring_create allocates its
 * slots with cudaMalloc; this call uses one static device array of NF4_NOALLOC_SLOT_BYTES instead.
 * Every device on which the library runs holds that array until the process exits.
 *
 *   x       in   device, bf16 bits [M][K]
 *   codes   in   page-locked host, uint8 [N][K/2]
 *   scales  in   page-locked host, fp16 bits [N][K/64]
 *   y       out  device, bf16 bits [M][N]; must not overlap x
 *
 * On `stream` the call copies codes and scales into the array and then runs nf4_linear on that copy;
 * y is bit for bit what nf4_linear gives on device-resident weights.  It calls no cudaMalloc,
 * cudaFree or other allocating routine.
 * Limit: N*K/2 rounded up to 256, plus N*(K/64)*2, must not exceed NF4_NOALLOC_SLOT_BYTES (16 MiB,
 * e.g. 11008 x 2048 fits); a larger linear returns NF4_ERR_SHAPE and nothing is enqueued.  Host
 * buffers that are not page-locked give NF4_ERR_MEMORY.  Other errors as for nf4_linear.  The host
 * buffers must stay unchanged until the call's work on `stream` has finished.
 * Sharing: all calls on a device use the same array, which keeps the weights of the last call (each
 * call rewrites every byte the kernels read, so nothing needs clearing).  Calls on one stream are
 * ordered and safe; calls whose work may overlap on the GPU (different streams with no ordering
 * between them) race on the array and give wrong results.
 * Set-up: the first call on a device looks up the array's device address; make that first call
 * before any stream capture.
 * A first call made while `stream` is capturing returns NF4_ERR_CAPTURE and leaves the capture
 * untouched.
 */
#define NF4_NOALLOC_SLOT_BYTES (16 * 1024 * 1024)
nf4_status nf4_linear_host_noalloc(const uint16_t* x, const uint8_t* codes, const uint16_t* scales, uint16_t* y,
                                   int64_t M, int64_t N, int64_t K, cudaStream_t stream);

/*
 * Operators around the linears of a decoder layer: rotary positions, a paged key-value cache that
 * quantises what it is given, the attention of one new token over it, and the residual norm.  With
 * nf4_linear_grouped (q|k|v, gate|up) and nf4_linear (o, down) they make one decode step of a
 * layer: norm, q|k|v, rope, append, attention, o, norm, gate|up, down.  The pages describe such a
 * layer's linears only; the formulas below define the rest.  The common rules above hold.
 */

/*
 * nf4_kv_cache - a paged key-value cache in the caller's memory (a description passed by pointer and
 * read before the call returns; the library keeps nothing of it).  K and V are each
 * [pages][kv_heads][page_size] vectors of head_dim values; place `slot` = page * page_size + offset
 * holds one token's vectors of every kv head.  Formats, x being a vector of head_dim bf16 values:
 *   NF4_KV_BF16  the values (2 head_dim bytes); no scales
 *   NF4_KV_FP8   e4m3 codes (head_dim bytes), code = e4m3_rn(fp32(x / s)) saturated at +-448, and one
 *                fp32 scale s = fp32(max |x| / 448) a vector; value = code * s; s = 0: code 0
 *   NF4_KV_NF4   the library's NF4 format along head_dim: head_dim/2 bytes of codes and head_dim/64
 *                fp16 scales, bit for bit what nf4_quantize gives for the same values
 */
typedef enum nf4_kv_format { NF4_KV_BF16 = 0, NF4_KV_FP8 = 1, NF4_KV_NF4 = 2 } nf4_kv_format;

typedef struct nf4_kv_cache {
    void* k;        /* device, [pages][kv_heads][page_size][bytes of a vector] */
    void* v;        /* the same for the values */
    void* k_scales; /* device: NULL (BF16), float [pages][kv_heads][page_size] (FP8) or
                       fp16 bits [pages][kv_heads][page_size][head_dim/64] (NF4) */
    void* v_scales;
    int64_t pages;     /* 0 .. 2^31-1, and pages * kv_heads * page_size at most 2^40 */
    int32_t kv_heads;  /* 1 .. 65535 */
    int32_t page_size; /* tokens a page: a multiple of 16, up to 65536 */
    int32_t head_dim;  /* 64, 128 or 256 */
    int32_t format;    /* an nf4_kv_format */
} nf4_kv_cache;

/*
 * nf4_kv_append - write T tokens' keys and values into the cache, quantised to its format.
 *   cache  k, v and the scales are written at the given places only
 *   k, v   in   bf16 bits [T][kv_heads][head_dim]
 *   slots  in   int64 [T]: the place of each token; a negative slot skips its token (a padded row of
 *               a batch); a slot >= pages * page_size is skipped and records code 42 in the device
 *               error word.  The slots that are not skipped must be distinct: two tokens written to
 *               one place leave an unspecified mix.
 * Errors: NF4_ERR_SHAPE also for a format, head_dim, page_size or kv_heads outside the lists above.
 */
nf4_status nf4_kv_append(const nf4_kv_cache* cache, const uint16_t* k, const uint16_t* v, const int64_t* slots,
                         int64_t T, cudaStream_t stream);

/*
 * nf4_kv_read - read T tokens' keys and values back as bf16, bf16_rn(fp32(code value * scale)).
 *   slots  in   int64 [T], in any order, repeats allowed; a negative slot gives zeros; a slot
 *               >= pages * page_size gives zeros and records code 42
 *   k, v   out  bf16 bits [T][kv_heads][head_dim]; either may be NULL (not read then)
 */
nf4_status nf4_kv_read(const nf4_kv_cache* cache, const int64_t* slots, int64_t T, uint16_t* k, uint16_t* v,
                       cudaStream_t stream);

/*
 * nf4_attention_decode - attention of one new token a sequence over the cache:
 *   out[b][h] = sum_j p_j v_j,  p = softmax_j(scale * q[b][h] . k_j),
 * j over places max(0, lengths[b] - window) .. lengths[b] - 1 of sequence b (window = 0: from 0),
 * k_j and v_j the cache's values (not rounded to bf16; see below) of kv head h / (q_heads / kv_heads); place j
 * is in page page_table[b][j / page_size].  A sequence with nothing to attend to gives zeros.  The
 * new token's own key and value are in the cache before the call.
 *   q           in   bf16 bits [B][q_heads][head_dim]; q_heads a multiple of kv_heads
 *   page_table  in   int32 [B][max_pages]; entries past a sequence's length do not matter
 *                    (page_table and lengths need the alignment of an int32 only: a batch may be cut)
 *   lengths     in   int32 [B]; a negative length counts as 0.  A length past max_pages * page_size is
 *                    cut there, and a needed page outside [0, pages) is left out of the sum; both
 *                    record code 43 in the device error word.
 *   out         out  bf16 bits [B][q_heads][head_dim]
 *   workspace   nf4_attention_workspace_bytes(cache, B, q_heads) bytes on the device, for the partial
 *               results of sequences that are split.  It must be zero before its first use; every
 *               call leaves it fit for the next one.  Calls that may overlap on the GPU need a
 *               workspace each; one workspace serves calls of different sizes as long as it is large
 *               enough for each.
 * Scores, softmax statistics and sums are fp32.  Rounded to fewer bits on the way:
 *   bf16  p, to the sum of two bf16 numbers (2^-16 of it)
 *   fp8   p * scale of V, to fp16 (2^-11 of it, or 2^-31 of the largest scale of V met, if that is more)
 *   NF4   the same; and the 16 table values, of K and of V, to fp16: each within 6.4e-4 of its value,
 *         rounded so that the errors cancel in a mean over values alike on both sides of zero (below 2.5e-6
 *         of their mean size; up to 1.8e-4 of it for values all on one side, 6e-5 for skewed ones around
 *         zero: nf4_kv_read has the values without that)
 *   q, with fp8 and NF4: elements below 2^-28 of their head's largest
 * Values in places that are not attended to (past a length, before the window) do not matter, NaN
 * and infinities included.  NF4_ERR_SHAPE also for B > 65535, q_heads > 65535, B * q_heads > 2^30,
 * max_pages * page_size >= 2^31, B * max_pages * page_size > 2^35 and for a workspace_bytes below the
 * need.  nf4_attention_workspace_bytes gives -1 for a cache, B or q_heads that the call refuses so.
 */
int64_t nf4_attention_workspace_bytes(const nf4_kv_cache* cache, int64_t B, int64_t q_heads);
nf4_status nf4_attention_decode(const nf4_kv_cache* cache, const uint16_t* q, const int32_t* page_table,
                                int64_t max_pages, const int32_t* lengths, int64_t B, int64_t q_heads, float scale,
                                int64_t window, uint16_t* out, void* workspace, int64_t workspace_bytes,
                                cudaStream_t stream);

/*
 * nf4_rope - rotary positions with up to four axes (one for text; time, height and width for images
 * and video) on q and k in one launch.  Pair i < rotary_dim / 2 of a head is elements (i, i +
 * rotary_dim/2), or (2i, 2i + 1) when `interleaved`; its angle is positions[a][t] * inv_freq[i] as a
 * real product (reduced exactly, at any position), a being the axis of the run of `sections` that
 * i falls in.  (x, y) becomes (x cos - y sin, y cos + x sin) * magnitude in fp32, rounded once to
 * bf16; elements past rotary_dim are copied.
 *   q, k           in   bf16 bits [T][q_heads][head_dim], [T][k_heads][head_dim]; either head count may
 *                       be 0 (its pointers are not used)
 *   positions      in   int32 [axes][T] (aligned to an int32)
 *   sections       in   host array of `axes` (1..4) counts of pairs, each >= 0, sum rotary_dim / 2
 *   inv_freq       in   float [rotary_dim / 2], any finite values
 *   rotary_dim     a multiple of 16, at most head_dim and 256; head_dim a multiple of 16, and
 *                  (q_heads + k_heads) * head_dim at most 2^24
 *   q_out, k_out   out  the same shapes; each may be its own input (in place), no other overlap
 */
nf4_status nf4_rope(const uint16_t* q, int64_t q_heads, const uint16_t* k, int64_t k_heads, int64_t T, int64_t head_dim,
                    const int32_t* positions, int axes, const int32_t* sections, const float* inv_freq,
                    int64_t rotary_dim, int interleaved, float magnitude, uint16_t* q_out, uint16_t* k_out,
                    cudaStream_t stream);

/*
 * nf4_rmsnorm - root-mean-square norm with the residual's addition: h = x + residual in fp32 (h = x
 * without one), residual_out = bf16_rn(h), y = h * rsqrt(mean(h^2) + eps) * weight in fp32, written as
 * bf16 (y, what nf4_linear reads) and / or in 8 bits: y8 = e4m3_rn(y / s) saturated at +-448 with one
 * fp32 scale s = max |y| / 448 a row.  An all-zero row gives zeros, s = 0 and codes 0, for eps = 0 too.
 * The squares are summed in fp32 and max |y| is found as max |h * weight| times the row's factor, so rows
 * with |h| past 2^63 / sqrt(H), or with |h * weight| past fp32's range, are outside the contract.  (The 8-bit
 * output is for a caller's own 8-bit product: nf4_linear reads bf16.)
 *   x, residual    in   bf16 bits [T][H], H a positive multiple of 8; residual may be NULL
 *   weight         in   bf16 bits [H]
 *   residual_out   out  bf16 bits [T][H] or NULL; may be residual or x itself
 *   y              out  bf16 bits [T][H] or NULL; may be x itself
 *   y8, y8_scales  out  e4m3 codes [T][H] and float [T], or both NULL; y or y8 must be given
 */
nf4_status nf4_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int64_t T, int64_t H,
                       float eps, uint16_t* residual_out, uint16_t* y, uint8_t* y8, float* y8_scales,
                       cudaStream_t stream);

/*
 * Operators of a server that decodes for many requests at once: the indices of a step, made on the GPU from
 * the requests' lengths; the requests' own low-rank adapters beside the packed projections; the choice of the
 * next token.  With nf4_embed, the layers above and nf4_linear for the output head they close the loop:
 * plan, embed, layers, head, sample, and the sampled tokens are the next step's ids.  The common rules hold.
 */

/*
 * nf4_plan_step - the indices of a step: pages handed out and taken back, and the place, position and
 * sequence of every new token.  Sequence b holds lengths[b] tokens in ceil(lengths[b] / page_size) pages and
 * brings new_tokens[b] more: 1 when it decodes, a piece of its prompt, 0 when it waits; a negative number
 * says that it is finished: its pages go back and its length becomes 0.  The new tokens are rows of the step's
 * batch in the order of the sequences, starts[b] being the first of sequence b.
 * Free pages are a ring of `pages` entries, free_in[0] the first one and free_in[1] how many there are.  Pages
 * given back go to the ring's end, in order, and may be handed out in the same step; new pages come from its
 * beginning, in the order of the sequences.  A sequence is refused (its length stays, its new tokens get no
 * place) if its tokens pass row T, if its pages pass max_pages, or if it needs new pages and the ring does not
 * hold all that it and the sequences before it need.
 *   lengths      in   int32 [B]; a negative one counts as 0
 *   new_tokens   in   int32 [B]
 *   page_size    16 .. 65536, a multiple of 16 (nf4_kv_cache)
 *   pages        entries of the ring and pages of the cache, 0 .. 2^31-2
 *   page_table   in/out int32 [B][max_pages]: entries of new pages are written, no others; those of a
 *                finished sequence stay as they are
 *   free_pages   in/out int32 [pages]: entries behind the ring's end are written
 *   free_in      in   int64 [2]
 *   free_out     out  int64 [2]; may be free_in
 *   lengths_out  out  int32 [B]; may be lengths
 *   starts       out  int32 [B + 1]; starts[B] is the number of new tokens (sums stop at 2^31-1, which counts as past row T)
 *   slots        out  int64 [T], what nf4_kv_append takes: page * page_size + offset; -1 for the tokens of a
 *                     refused sequence and for rows from starts[B] on
 *   positions    out  int32 [T], lengths[b] + i for token i of sequence b; 0 from row starts[B] on
 *   sequences    out  int32 [T], b; -1 from row starts[B] on
 * All of them are aligned to their elements at least (not to 16 bytes).  B at most 8192, T at most 2^31 - 1, B *
 * max_pages at most 2^40.  A page outside [0, pages) where a token goes gives the place -1, a ring's state outside
 * the ring is cut to it, pages that the ring has no room for are lost: each records code 45 in the device error word.
 */
nf4_status nf4_plan_step(const int32_t* lengths, const int32_t* new_tokens, int64_t B, int64_t page_size, int64_t pages,
                         int32_t* page_table, int64_t max_pages, int32_t* free_pages, const int64_t* free_in,
                         int64_t* free_out, int32_t* lengths_out, int32_t* starts, int64_t T, int64_t* slots,
                         int32_t* positions, int32_t* sequences, cudaStream_t stream);

/*
 * nf4_lora_plan - the tokens of a step, listed adapter by adapter.  Made once for all nf4_lora calls with the same
 * tokens (every projection of every layer).
 *   ids        in   int32 [T], the adapter of each token; negative: none.  With `sequences`: int32 [S], the
 *                   adapter of each sequence
 *   sequences  in   NULL, or int32 [T], the sequence of each token (as nf4_plan_step gives it); negative: no
 *                   adapter
 *   T          0 .. 2^24;  adapters  0 .. 8192 that are loaded
 *   plan       out  nf4_lora_plan_bytes(T, adapters) bytes on the device, 16-byte aligned
 * An id >= adapters, or a sequence >= S, counts as none and records code 46 in the device error word.
 * nf4_lora_plan_bytes gives -1 for sizes that are refused.
 */
int64_t nf4_lora_plan_bytes(int64_t T, int64_t adapters);
nf4_status nf4_lora_plan(const int32_t* ids, const int32_t* sequences, int64_t S, int64_t T, int64_t adapters, void* plan,
                         int64_t plan_bytes, cudaStream_t stream);

/*
 * nf4_lora - low-rank adapters of many requests beside up to 8 projections that share their input:
 *   ys[i][t] = bf16_rn(bases[i][t] + scales[a] * sum_r b[i][a][:, r] h_r),  h_r = sum_k a[i][a][r, k] x[t, k]
 * for a token t with adapter a; without one, ys[i][t] = bases[i][t] (rows that are in place are not touched).
 *   x          in   bf16 bits [T][K], K a positive multiple of 64
 *   plan       in   from nf4_lora_plan with the same T and adapters
 *   rank       of all adapters: a multiple of 8, 8 .. 128 (pad a smaller one with zeros)
 *   scales     in   float [adapters]
 *   count      1 .. 8
 *   a          host array of count device pointers; a[i]: bf16 bits [adapters][rank][K]
 *   b          host array; b[i]: bf16 bits [adapters][Ns[i]][rank]
 *   bases      host array; bases[i]: bf16 bits [T][Ns[i]] (what nf4_linear_grouped gave); NULL: ys
 *   ys         host array; ys[i]: bf16 bits [T][Ns[i]]; may be its own base, no other overlap
 *   workspace  nf4_lora_workspace_bytes(T, adapters, rank, count) bytes on the device; needs no set-up.  Calls that
 *              may overlap on the GPU need one each
 * Sums are fp32; scales[a] * h_r goes into the second product as the sum of two bf16 numbers (2^-16 of it; past bf16's range,
 * 3.39e38, as an infinity).  The order of the sums follows from the call's sizes and from how its tokens share the adapters:
 * the same call gives the same bytes, a token beside other tokens the same within rounding.  The host arrays are read before
 * the call returns.  A plan of other sizes records code 47, and nothing is computed.
 */
int64_t nf4_lora_workspace_bytes(int64_t T, int64_t adapters, int64_t rank, int64_t count);
nf4_status nf4_lora(const uint16_t* x, int64_t T, int64_t K, const void* plan, int64_t plan_bytes, int64_t adapters,
                    int64_t rank, const float* scales, int count, const uint16_t* const* a, const uint16_t* const* b,
                    const uint16_t* const* bases, uint16_t* const* ys, const int64_t* Ns, void* workspace,
                    int64_t workspace_bytes, cudaStream_t stream);

/*
 * nf4_sample - the next token of every row of logits, from a given random number.  With l the row's logits and T
 * its temperature, token i has the weight w_i = exp((l_i - max l) / T).  Tokens are ordered by l, equal ones by
 * index.  Of that order are kept: the first top_k; of these the smallest number whose weights reach top_p of
 * theirs; of these the ones with w_i >= min_p; the first token always.  The token drawn is the first i, in order of
 * index, for which the kept weights up to i pass random * (their sum).  T = 0 (or below 2^-100): the first of
 * the largest logits.
 *   logits       in   [B][stride], the first V of a row used; bf16 bits (logits_bf16 != 0; what nf4_linear gives) or
 *                     float
 *   temperature  in   float [B], NULL: 1
 *   top_k        in   int32 [B]; 0 or less, V or more: all.  NULL: all
 *   top_p        in   float [B]; 1 or more: all.  NULL: all
 *   min_p        in   float [B]; 0 or less: all.  NULL: all
 *   random       in   float [B] in [0, 1)
 *   tokens       out  int32 [B]
 *   logprobs     out  float [B] or NULL: log softmax(l) of the token, before temperature and cuts, its sum in fp32 by the
 *                     hardware's exp2: off by 2^-17 + 2^-22 of its size at most, by some 4e-8 on a model's logits
 * V in 1 .. 262144, stride >= V, B at most 2^24; everything is aligned to its elements (rows may start anywhere).
 * Logits of -inf (masked) and NaN have no weight; a row with nothing else gives token -1 and logprob -inf, one with
 * +inf the first of n such and logprob -log n.  Weights are whole multiples of 2^-40 (each within 1.1 * 2^-30 of its size,
 * or half a multiple), so sums are exact and the drawn token does not depend on their order; what weighs less than half a
 * multiple is never drawn.  So the borders between tokens lie within 2^-30 of the whole of where the formula has them, plus
 * V * 2^-41 where many tokens weigh only a few multiples.
 */
nf4_status nf4_sample(const void* logits, int logits_bf16, int64_t B, int64_t V, int64_t stride, const float* temperature,
                      const int32_t* top_k, const float* top_p, const float* min_p, const float* random, int32_t* tokens,
                      float* logprobs, cudaStream_t stream);

/*
 * nf4_check_device_error - diagnostics: read and clear the device-side error words of the current
 * device.  The linear kernels bound every pipeline wait (one second of wall-clock time per wait,
 * see nf4_diag_set_wait_limit); a wait that runs out records a nonzero code (1..39; 39 is
 * nf4_diag_bounded_wait's), and the kernel drains and exits instead of hanging, leaving its outputs
 * unspecified.  nf4_embed records 41 for an id outside the table, the cache calls 42 for a slot
 * outside the cache, nf4_attention_decode 43 for a page or length outside its bounds (44: a
 * shared-memory layout that its kernel does not know; nothing is computed then), nf4_plan_step 45,
 * nf4_lora_plan 46 and nf4_lora 47 (see there).  *code receives the first recorded code (0 = none).  This call waits for the device (it is not meant for the hot path).
 */
nf4_status nf4_check_device_error(int* code);

/*
 * nf4_diag_bounded_wait - diagnostics, no counterpart in the pages: checks that a pipeline wait
 * which runs out reports instead of hanging.  Launches one thread on `stream` that waits on an
 * mbarrier nothing ever arrives on, through the same bounded wait and error word as the linear
 * kernels; after `ns` nanoseconds of wall-clock time it gives up and records code 39, which
 * nf4_check_device_error then returns.  The device stays usable.  ns must be in [1, 2^31] (about
 * 2.1 s), else NF4_ERR_SHAPE.
 */
nf4_status nf4_diag_bounded_wait(int64_t ns, cudaStream_t stream);

/*
 * nf4_diag_set_wait_limit - diagnostics, no counterpart in the pages: sets the wall-clock limit of
 * each pipeline wait of the linear kernels on the current device to `ns` nanoseconds, or restores
 * the default of one second when ns = 0.  The limit applies to every wait separately (it restarts
 * at each wait), so a kernel that runs far longer than the limit is unaffected as long as each of
 * its waits is shorter.  Stream-ordered on `stream`.  ns must be in [0, 2^36] (about 69 s), else
 * NF4_ERR_SHAPE.
 */
nf4_status nf4_diag_set_wait_limit(int64_t ns, cudaStream_t stream);

/* Static, human-readable name of a status code (never NULL). */
const char* nf4_status_str(nf4_status status);

/* NF4_ABI_VERSION of the built library. */
int nf4_abi_version(void);

/* NF4_NOALLOC_SLOT_BYTES of the built library (the size of nf4_linear_host_noalloc's array). */
int64_t nf4_noalloc_slot_bytes(void);

/* Name of the last CUDA error (for instance "cudaErrorInvalidValue") behind an NF4_ERR_CUDA returned
 * to the calling host thread, or "cudaSuccess" if there was none.  Static string, never NULL. */
const char* nf4_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* NF4_H */
