// Attention of one new token a sequence over the paged key-value cache.
//
// The plainest form: one CTA of four warps for each (sequence, query head); a warp takes every
// fourth key, its lanes a slice of head_dim each, with the running maximum and sum of a softmax;
// the warps' results are joined in shared memory.
#include "nf4_kv.cuh"

namespace nf4 {
namespace {

__device__ int g_attention_error;

template <int FMT, int D>
__device__ __forceinline__ void load_values(const uint8_t* base, const uint8_t* scales, int64_t at, int lane,
                                            float (&x)[D / 32]) {
    constexpr int E = D / 32;
#pragma unroll
    for (int e = 0; e < E; e++) {
        const int d = lane * E + e;
        if (FMT == kKvBf16) {
            x[e] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base)[at * D + d]);
        } else if (FMT == kKvFp8) {
            const uint32_t h = e4m3x2_to_f16x2(base[at * D + d]);
            x[e] = __half2float(__ushort_as_half(static_cast<uint16_t>(h & 0xFFFFu))) *
                   reinterpret_cast<const float*>(scales)[at];
        } else {
            const uint32_t b = base[at * (D / 2) + d / 2];
            x[e] = kNF4[(d & 1) ? b >> 4 : b & 15u] *
                   __half2float(__ushort_as_half(reinterpret_cast<const uint16_t*>(scales)[at * (D / 64) + d / 64]));
        }
    }
}

template <int FMT, int D>
__global__ void __launch_bounds__(128) attention_kernel(KvCache c, const uint16_t* __restrict__ q,
                                                        const int32_t* __restrict__ page_table, int64_t max_pages,
                                                        const int32_t* __restrict__ lengths, int q_heads, float scale,
                                                        int64_t window, uint16_t* __restrict__ out) {
    constexpr int E = D / 32;
    __shared__ float part[4][D + 2];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int h = blockIdx.x, kv = h / (q_heads / c.kv_heads);
    const int64_t b = blockIdx.y;
    pdl_launch_dependents();
    pdl_wait();
    int64_t n = lengths[b];
    if (n < 0) n = 0;
    if (n > max_pages * c.page_size) {
        n = max_pages * c.page_size;
        if (threadIdx.x == 0) atomicCAS(&g_attention_error, 0, 43);
    }
    const int64_t first = window > 0 && n > window ? n - window : 0;
    float qs[E], acc[E];
#pragma unroll
    for (int e = 0; e < E; e++) {
        qs[e] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(q)[(b * q_heads + h) * D + lane * E + e]) * scale;
        acc[e] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    for (int64_t j = first + warp; j < n; j += 4) {
        const int64_t page = page_table[b * max_pages + j / c.page_size];
        if (page < 0 || page >= c.pages) {
            if (lane == 0) atomicCAS(&g_attention_error, 0, 43);
            continue;
        }
        const int64_t at = (page * c.kv_heads + kv) * c.page_size + j % c.page_size;
        float x[E], s = 0.0f;
        load_values<FMT, D>(c.k, c.k_scales, at, lane, x);
#pragma unroll
        for (int e = 0; e < E; e++) s = fmaf(qs[e], x[e], s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        const float top = fmaxf(m, s), f = expf(m - top), p = expf(s - top);
        m = top;
        l = l * f + p;
        load_values<FMT, D>(c.v, c.v_scales, at, lane, x);
#pragma unroll
        for (int e = 0; e < E; e++) acc[e] = fmaf(p, x[e], acc[e] * f);
    }
#pragma unroll
    for (int e = 0; e < E; e++) part[warp][lane * E + e] = acc[e];
    if (lane == 0) part[warp][D] = m, part[warp][D + 1] = l;
    __syncthreads();
    float top = -INFINITY, sum = 0.0f;
    for (int w = 0; w < 4; w++) top = fmaxf(top, part[w][D]);
    float f[4];
    for (int w = 0; w < 4; w++) {
        f[w] = top == -INFINITY ? 0.0f : expf(part[w][D] - top);
        sum += f[w] * part[w][D + 1];
    }
    for (int d = threadIdx.x; d < D; d += 128) {
        float o = 0.0f;
        for (int w = 0; w < 4; w++) o += f[w] * part[w][d];
        out[(b * q_heads + h) * D + d] = bf16_bits(sum > 0.0f ? o / sum : 0.0f);
    }
}

template <int FMT, int D>
cudaError_t attend(const KvCache& c, const uint16_t* q, const int32_t* page_table, int64_t max_pages,
                   const int32_t* lengths, int64_t B, int64_t q_heads, float scale, int64_t window, uint16_t* out,
                   cudaStream_t stream) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(q_heads), static_cast<unsigned>(B));
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attention_kernel<FMT, D>, c, q, page_table, max_pages, lengths,
                              static_cast<int>(q_heads), scale, window, out);
}

}  // namespace

int64_t attention_workspace_bytes(int, int, int64_t, int64_t) { return 16; }

cudaError_t launch_attention(const KvCache& c, const uint16_t* q, const int32_t* page_table, int64_t max_pages,
                             const int32_t* lengths, int64_t B, int64_t q_heads, float scale, int64_t window,
                             uint16_t* out, void*, int, cudaStream_t stream) {
#define NF4_CALL(F, D) attend<F, D>(c, q, page_table, max_pages, lengths, B, q_heads, scale, window, out, stream)
    if (c.format == kKvBf16)
        return c.head_dim == 64 ? NF4_CALL(kKvBf16, 64) : c.head_dim == 128 ? NF4_CALL(kKvBf16, 128) : NF4_CALL(kKvBf16, 256);
    if (c.format == kKvFp8)
        return c.head_dim == 64 ? NF4_CALL(kKvFp8, 64) : c.head_dim == 128 ? NF4_CALL(kKvFp8, 128) : NF4_CALL(kKvFp8, 256);
    return c.head_dim == 64 ? NF4_CALL(kKvNf4, 64) : c.head_dim == 128 ? NF4_CALL(kKvNf4, 128) : NF4_CALL(kKvNf4, 256);
#undef NF4_CALL
}

cudaError_t read_and_clear_attention_error(int* code) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_attention_error, sizeof(int));
    if (e != cudaSuccess) return e;
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_attention_error, &zero, sizeof(int));
    *code = v;
    return e;
}

}  // namespace nf4
