// Launchers shared between the C-ABI layer and the kernel translation units (host side).
#pragma once

#include <cstdint>
#include <cuda_runtime_api.h>

namespace nf4 {

// Each launcher enqueues its kernels on `stream` and returns the result of cudaGetLastError()
// (cudaSuccess when nothing was launched).  Arguments are validated by the caller.
cudaError_t launch_quantize(const float* w, int64_t N, int64_t K, uint8_t* codes, uint16_t* scales,
                            int num_sms, cudaStream_t stream);
cudaError_t launch_dequant(const uint8_t* codes, const uint16_t* scales, int64_t N, int64_t K,
                           uint16_t* w_hat, int num_sms, cudaStream_t stream);
// CUDA-core GEMV family: y[M, N] for 1 <= M <= kGemvMaxTokens (measured on the 14B-shaped decode
// pass: at M = 4 the tensor-core small-M kernel is faster, 1354 against 1204 GB/s).
constexpr int kGemvMaxTokens = 3;
cudaError_t launch_gemv(const uint16_t* x, const uint8_t* codes, const uint16_t* scales, uint16_t* y,
                        int64_t M, int64_t N, int64_t K, int num_sms, cudaStream_t stream);

// The same for up to kMaxGroupedLinears linears sharing x and K (concatenated rows, one launch).
constexpr int kMaxGroupedLinears = 8;
cudaError_t launch_gemv_grouped(const uint16_t* x, int count, const uint8_t* const* codes,
                                const uint16_t* const* scales, uint16_t* const* ys, const int64_t* Ns, int64_t M,
                                int64_t K, int num_sms, cudaStream_t stream);

// tcgen05 weight streaming (dequantized tiles in tensor memory) for every M the GEMV does not take:
// y_i[M, N_i] for up to kMaxGroupedLinears linears that share x and K, one launch.
cudaError_t launch_stream(const uint16_t* x, int count, const uint8_t* const* codes, const uint16_t* const* scales,
                          uint16_t* const* ys, const int64_t* Ns, int64_t M, int64_t K, int num_sms,
                          cudaStream_t stream);
// Device error word of the linear kernels (nonzero after a bounded pipeline wait timed out).
cudaError_t read_and_clear_error(int* code);
cudaError_t launch_diag_wait(int64_t ns, cudaStream_t stream);
// Per-wait wall-clock limit of the pipeline waits on the current device (0 = the default, 1 s).
cudaError_t set_wait_limit(int64_t ns, cudaStream_t stream);

// Packed embedding rows (out-of-range ids write zeros and set the embed error word to 41).
cudaError_t launch_embed(const int32_t* ids, int64_t n_ids, const uint8_t* codes, const uint16_t* scales, int64_t V,
                         int64_t K, uint16_t* out, int num_sms, cudaStream_t stream);
cudaError_t read_and_clear_embed_error(int* code);

// Key-value cache formats (nf4_kv_format) and the checked description of a cache.
constexpr int kKvBf16 = 0, kKvFp8 = 1, kKvNf4 = 2;
struct KvCache {
    uint8_t *k, *v;              // [pages][kv_heads][page_size] vectors
    uint8_t *k_scales, *v_scales;
    int64_t pages;
    int kv_heads, page_size, head_dim, format;
};
cudaError_t launch_kv_append(const KvCache& c, const uint16_t* k, const uint16_t* v, const int64_t* slots, int64_t T,
                             int num_sms, cudaStream_t stream);
cudaError_t launch_kv_read(const KvCache& c, const int64_t* slots, int64_t T, uint16_t* k, uint16_t* v, int num_sms,
                           cudaStream_t stream);
// Error word of the cache calls (42: a slot outside the cache) and of the attention (43: a page or a
// length outside its bounds).
cudaError_t read_and_clear_kv_error(int* code);
cudaError_t read_and_clear_attention_error(int* code);

// One new token a sequence over the cache; the workspace is described in nf4_attn.cu.
int64_t attention_workspace_bytes(int kv_heads, int head_dim, int64_t B, int64_t q_heads);
cudaError_t launch_attention(const KvCache& c, const uint16_t* q, const int32_t* page_table, int64_t max_pages,
                             const int32_t* lengths, int64_t B, int64_t q_heads, float scale, int64_t window,
                             uint16_t* out, void* workspace, int num_sms, cudaStream_t stream);

struct RopeArgs {
    const uint16_t *q, *k;
    uint16_t *q_out, *k_out;
    const int32_t* positions;  // [axes][T]
    const float* inv_freq;
    int64_t T;
    int q_heads, k_heads, head_dim, rotary_dim, axes, interleaved;
    int section_end[4];  // first pair past axis a's run
    float magnitude;
};
cudaError_t launch_rope(const RopeArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int64_t T, int64_t H,
                           float eps, uint16_t* residual_out, uint16_t* y, uint8_t* y8, float* y8_scales, int num_sms,
                           cudaStream_t stream);

// A step's indices (nf4_plan_step); every CTA keeps five words a sequence in shared memory.
constexpr int kPlanMaxBatch = 8192, kPlanThreads = 1024;
struct PlanArgs {
    const int32_t *lengths, *new_tokens;
    int32_t* page_table;
    int32_t* free_pages;
    const int64_t* free_in;
    int64_t* free_out;
    int32_t *lengths_out, *starts;
    int64_t* slots;
    int32_t *positions, *sequences;
    int64_t T, max_pages, pages;
    int B;
    uint32_t page_size;
    bool in_place;  // an output is its own input
};
cudaError_t launch_plan(const PlanArgs& a, int num_sms, cudaStream_t stream);
// Error words: 45, a page or a ring's state outside the pool; 46, an adapter or a row outside its list; 47, a plan
// of other sizes.
cudaError_t read_and_clear_plan_error(int* code);

// Low-rank adapters of many requests.
constexpr int64_t kLoraMaxAdapters = 8192, kLoraMaxTokens = 1 << 24;
int64_t lora_plan_bytes(int64_t T, int64_t adapters);
int64_t lora_workspace_bytes(int64_t T, int64_t adapters, int64_t rank, int64_t count);
cudaError_t launch_lora_plan(const int32_t* ids, const int32_t* sequences, int64_t S, int64_t T, int64_t adapters,
                             void* plan, cudaStream_t stream);
struct LoraArgs {
    const uint16_t* x;
    const int32_t* plan;
    const float* scales;
    float* h;  // the workspace
    const uint16_t *a[kMaxGroupedLinears], *b[kMaxGroupedLinears], *base[kMaxGroupedLinears];
    uint16_t* y[kMaxGroupedLinears];
    int64_t N[kMaxGroupedLinears];
    int64_t T, K, adapters;
    int rank, count;
};
cudaError_t launch_lora(const LoraArgs& a, int num_sms, cudaStream_t stream);
cudaError_t read_and_clear_lora_error(int* code);

// The next token of every row.
struct SampleArgs {
    const void* logits;
    const float *temperature, *top_p, *min_p, *random;
    const int32_t* top_k;
    int32_t* tokens;
    float* logprobs;
    int64_t B, V, stride;
    int bf16;
};
constexpr int64_t kSampleMaxVocab = 262144;
cudaError_t launch_sample(const SampleArgs& a, int num_sms, cudaStream_t stream);

// The C-ABI layer's device check (an nf4_status value): the current device and its SM count.
int abi_current_device(int* device, int* sms);
// Records a CUDA error for nf4_last_cuda_error (no-op for cudaSuccess).
void note_cuda_error(cudaError_t e);

}  // namespace nf4
