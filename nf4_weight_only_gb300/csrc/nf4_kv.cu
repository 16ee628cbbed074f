// Writing the paged key-value cache (with the quantization of its format) and reading it back.
//
// Both are streaming kernels: a vector of D values (one token, one kv head, K or V) is handled by D/8
// lanes, eight values (16 bytes of bf16) a lane, so that the bf16 side moves in whole 16-byte pieces
// and the absmax of a vector or of a 64-value group takes three to five shuffles.
#include "nf4_kv.cuh"

namespace nf4 {
namespace {

// Error word of the cache calls (42: a slot outside the cache).
__device__ int g_kv_error;

// The decision thresholds of the NF4 code: t[i] is the smallest binary32 r in [T[i], T[i+1]] that is
// strictly closer, in fp32 distance, to T[i+1] than to T[i], so that the nearest-code rule (ties to
// the lower index) is code(r) = number of thresholds <= r.  nf4_quantize finds them by bisection in
// every CTA; a call here may write a single token, so the compiler finds them, by the same predicate.
struct Thresholds {
    float t[15];
};
constexpr float distance(float a, float b) { return a < b ? b - a : a - b; }
constexpr float next_up(float x) {
    float step = 0x1p-60f, up = x;
    for (; up == x; step *= 2.0f) up = x + step;
    return up;
}
constexpr Thresholds nf4_thresholds() {
    constexpr float table[16] = {-1.0f, -0.6961928009986877f, -0.5250730514526367f, -0.39491748809814453f,
                                 -0.28444138169288635f, -0.18477343022823334f, -0.09105003625154495f, 0.0f,
                                 0.07958029955625534f, 0.16093020141124725f, 0.24611230194568634f,
                                 0.33791524171829224f, 0.44070982933044434f, 0.5626170039176941f,
                                 0.7229568362236023f, 1.0f};
    Thresholds r{};
    for (int i = 0; i < 15; i++) {
        const float lo = table[i], hi = table[i + 1];
        float at = lo;  // nearest to lo throughout
        for (float step = 0.25f; step > 0x1p-40f; step *= 0.5f) {
            const float c = at + step;
            if (c > at && c < hi && !(distance(c, hi) < distance(c, lo))) at = c;
        }
        for (float c = next_up(at); !(distance(c, hi) < distance(c, lo)); c = next_up(at)) at = c;  // sums were rounded
        r.t[i] = next_up(at);
    }
    return r;
}
__device__ __constant__ const Thresholds kThresholds = nf4_thresholds();

__device__ __forceinline__ uint32_t nf4_code(float r, const float* thr) {
    uint32_t c = r >= thr[7] ? 8u : 0u;
    c += r >= thr[c + 3] ? 4u : 0u;
    c += r >= thr[c + 1] ? 2u : 0u;
    c += r >= thr[c] ? 1u : 0u;
    return c;
}

// The vector index of place `slot` for kv head h: ((page * kv_heads + h) * page_size + offset.
__device__ __forceinline__ int64_t place_index(int64_t slot, int h, int kv_heads, int page_size) {
    int64_t page;
    int off;
    if ((slot >> 32) == 0) {
        page = static_cast<uint32_t>(slot) / static_cast<uint32_t>(page_size);
        off = static_cast<int>(static_cast<uint32_t>(slot) - static_cast<uint32_t>(page) * static_cast<uint32_t>(page_size));
    } else {
        page = slot / page_size;
        off = static_cast<int>(slot - page * page_size);
    }
    return (page * kv_heads + h) * page_size + off;
}

// Item i of a launch (one token and kv head) -> token and head, in 32 bits where the count allows.
__device__ __forceinline__ void split_item(int64_t i, int64_t items, int heads, int64_t& t, int& h) {
    if (items <= 0xFFFFFFFFll) {
        t = static_cast<uint32_t>(i) / static_cast<uint32_t>(heads);
    } else {
        t = i / heads;
    }
    h = static_cast<int>(i - t * heads);
}

template <int FMT, int D>
__global__ void __launch_bounds__(256) append_kernel(KvCache c, const uint16_t* __restrict__ k_in,
                                                     const uint16_t* __restrict__ v_in,
                                                     const int64_t* __restrict__ slots, int64_t T) {
    constexpr int L = D / 8;  // lanes a vector
    __shared__ float thr[16];
    if (FMT == kKvNf4) {
        if (threadIdx.x < 15) thr[threadIdx.x] = kThresholds.t[threadIdx.x];
        __syncthreads();
    }
    pdl_launch_dependents();
    pdl_wait();
    const uint16_t* src = blockIdx.y ? v_in : k_in;
    uint8_t* dst = blockIdx.y ? c.v : c.k;
    uint8_t* dst_scales = blockIdx.y ? c.v_scales : c.k_scales;
    const int l = threadIdx.x % L;
    const int64_t items = T * c.kv_heads, capacity = c.pages * c.page_size;
    const int64_t per_grid = static_cast<int64_t>(gridDim.x) * (256 / L);
    // whole warps stay in the loop: the shuffles below take all 32 lanes
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * (256 / L); base < items; base += per_grid) {
        const int64_t i = base + threadIdx.x / L;
        int64_t t = 0, slot = -1;
        int h = 0;
        if (i < items) {
            split_item(i, items, c.kv_heads, t, h);
            slot = slots[t];
        }
        if (slot >= capacity) {
            if (l == 0) atomicCAS(&g_kv_error, 0, 42);
            slot = -1;
        }
        uint4 w = make_uint4(0, 0, 0, 0);
        if (slot >= 0) w = __ldcs(reinterpret_cast<const uint4*>(src) + i * L + l);
        const int64_t at = slot >= 0 ? place_index(slot, h, c.kv_heads, c.page_size) : 0;
        if (FMT == kKvBf16) {
            if (slot >= 0) reinterpret_cast<uint4*>(dst)[at * L + l] = w;
            continue;
        }
        float x[8];
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float2 p = bf16x2_to_f32x2(ws[j]);
            x[2 * j] = p.x, x[2 * j + 1] = p.y;
        }
        float s = fabsf(x[0]);
#pragma unroll
        for (int j = 1; j < 8; j++) s = fmaxf(s, fabsf(x[j]));
#pragma unroll
        for (int o = 1; o < (FMT == kKvNf4 ? 8 : L); o <<= 1) s = fmaxf(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
        if (FMT == kKvFp8) {
            s = __fdiv_rn(s, kFp8Max);
            uint2 out = make_uint2(0, 0);
            if (s > 0.0f) {
#pragma unroll
                for (int j = 0; j < 8; j++) x[j] = __fdiv_rn(x[j], s);
                out.x = f32x2_to_e4m3x2(x[0], x[1]) | (f32x2_to_e4m3x2(x[2], x[3]) << 16);
                out.y = f32x2_to_e4m3x2(x[4], x[5]) | (f32x2_to_e4m3x2(x[6], x[7]) << 16);
            }
            if (slot >= 0) {
                reinterpret_cast<uint2*>(dst)[at * L + l] = out;
                if (l == 0) reinterpret_cast<float*>(dst_scales)[at] = s;
            }
        } else if (FMT == kKvNf4) {
            const float d = s != 0.0f ? s : 1.0f;  // an all-zero group divides by 1: r = +-0, code 7
            uint32_t word = 0;
#pragma unroll
            for (int j = 0; j < 8; j++) word |= nf4_code(__fdiv_rn(x[j], d), thr) << (4 * j);
            if (slot >= 0) {
                reinterpret_cast<uint32_t*>(dst)[at * L + l] = word;
                if (l % 8 == 0)
                    reinterpret_cast<uint16_t*>(dst_scales)[at * (D / 64) + l / 8] = __half_as_ushort(__float2half_rn(s));
            }
        }
    }
}

// Read back: the inverse, eight values a lane; bf16_rn(fp32(code value * scale)).
template <int FMT, int D>
__global__ void __launch_bounds__(256) read_kernel(KvCache c, const int64_t* __restrict__ slots, int64_t T,
                                                   uint16_t* __restrict__ k_out, uint16_t* __restrict__ v_out) {
    constexpr int L = D / 8;
    __shared__ float table[16];
    if (FMT == kKvNf4) {
        if (threadIdx.x < 16) table[threadIdx.x] = kNF4[threadIdx.x];
        __syncthreads();
    }
    pdl_launch_dependents();
    pdl_wait();
    uint16_t* out = blockIdx.y ? v_out : k_out;
    const uint8_t* src = blockIdx.y ? c.v : c.k;
    const uint8_t* scales = blockIdx.y ? c.v_scales : c.k_scales;
    if (!out) return;
    const int l = threadIdx.x % L;
    const int64_t items = T * c.kv_heads, capacity = c.pages * c.page_size;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * (256 / L) + threadIdx.x / L; i < items;
         i += static_cast<int64_t>(gridDim.x) * (256 / L)) {
        int64_t t;
        int h;
        split_item(i, items, c.kv_heads, t, h);
        int64_t slot = slots[t];
        if (slot >= capacity) {
            if (l == 0) atomicCAS(&g_kv_error, 0, 42);
            slot = -1;
        }
        uint4 o = make_uint4(0, 0, 0, 0);
        if (slot >= 0) {
            const int64_t at = place_index(slot, h, c.kv_heads, c.page_size);
            if (FMT == kKvBf16) {
                o = __ldcs(reinterpret_cast<const uint4*>(src) + at * L + l);
            } else if (FMT == kKvFp8) {
                const uint2 w = __ldcs(reinterpret_cast<const uint2*>(src) + at * L + l);
                const float s = reinterpret_cast<const float*>(scales)[at];
                const uint32_t hs[4] = {e4m3x2_to_f16x2(w.x & 0xFFFFu), e4m3x2_to_f16x2(w.x >> 16),
                                        e4m3x2_to_f16x2(w.y & 0xFFFFu), e4m3x2_to_f16x2(w.y >> 16)};
                uint32_t r[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hs[j]));
                    r[j] = f32x2_to_bf16x2(__fmul_rn(f.x, s), __fmul_rn(f.y, s));
                }
                o = make_uint4(r[0], r[1], r[2], r[3]);
            } else {
                const uint32_t w = __ldcs(reinterpret_cast<const uint32_t*>(src) + at * L + l);
                const float s = __half2float(
                    __ushort_as_half(reinterpret_cast<const uint16_t*>(scales)[at * (D / 64) + l / 8]));
                uint32_t r[4];
#pragma unroll
                for (int j = 0; j < 4; j++)
                    r[j] = f32x2_to_bf16x2(__fmul_rn(table[(w >> (8 * j)) & 15u], s),
                                           __fmul_rn(table[(w >> (8 * j + 4)) & 15u], s));
                o = make_uint4(r[0], r[1], r[2], r[3]);
            }
        }
        __stcs(reinterpret_cast<uint4*>(out) + i * L + l, o);
    }
}

cudaLaunchConfig_t pdl_config(dim3 grid, int threads, cudaStream_t stream, cudaLaunchAttribute* attr) {
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

dim3 vector_grid(int64_t items, int D, int num_sms) {
    const int64_t per = 256 / (D / 8), cap = static_cast<int64_t>(num_sms) * 8;
    int64_t blocks = (items + per - 1) / per;
    if (blocks > cap) blocks = cap;
    return dim3(static_cast<unsigned>(blocks), 2);
}

template <int FMT, int D>
cudaError_t append(const KvCache& c, const uint16_t* k, const uint16_t* v, const int64_t* slots, int64_t T,
                   int num_sms, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = pdl_config(vector_grid(T * c.kv_heads, D, num_sms), 256, stream, &attr);
    return cudaLaunchKernelEx(&cfg, append_kernel<FMT, D>, c, k, v, slots, T);
}

template <int FMT, int D>
cudaError_t read(const KvCache& c, const int64_t* slots, int64_t T, uint16_t* k, uint16_t* v, int num_sms,
                 cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = pdl_config(vector_grid(T * c.kv_heads, D, num_sms), 256, stream, &attr);
    return cudaLaunchKernelEx(&cfg, read_kernel<FMT, D>, c, slots, T, k, v);
}

}  // namespace

#define NF4_KV_DISPATCH(CALL)                                          \
    do {                                                               \
        if (c.format == kKvBf16) {                                     \
            if (c.head_dim == 64) return CALL(kKvBf16, 64);            \
            if (c.head_dim == 128) return CALL(kKvBf16, 128);          \
            return CALL(kKvBf16, 256);                                 \
        }                                                              \
        if (c.format == kKvFp8) {                                      \
            if (c.head_dim == 64) return CALL(kKvFp8, 64);             \
            if (c.head_dim == 128) return CALL(kKvFp8, 128);           \
            return CALL(kKvFp8, 256);                                  \
        }                                                              \
        if (c.head_dim == 64) return CALL(kKvNf4, 64);                 \
        if (c.head_dim == 128) return CALL(kKvNf4, 128);               \
        return CALL(kKvNf4, 256);                                      \
    } while (0)

cudaError_t launch_kv_append(const KvCache& c, const uint16_t* k, const uint16_t* v, const int64_t* slots, int64_t T,
                             int num_sms, cudaStream_t stream) {
#define NF4_CALL(F, D) append<F, D>(c, k, v, slots, T, num_sms, stream)
    NF4_KV_DISPATCH(NF4_CALL);
#undef NF4_CALL
}

cudaError_t launch_kv_read(const KvCache& c, const int64_t* slots, int64_t T, uint16_t* k, uint16_t* v, int num_sms,
                           cudaStream_t stream) {
#define NF4_CALL(F, D) read<F, D>(c, slots, T, k, v, num_sms, stream)
    NF4_KV_DISPATCH(NF4_CALL);
#undef NF4_CALL
}

cudaError_t read_and_clear_kv_error(int* code) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_kv_error, sizeof(int));
    if (e != cudaSuccess) return e;
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_kv_error, &zero, sizeof(int));
    *code = v;
    return e;
}

}  // namespace nf4
