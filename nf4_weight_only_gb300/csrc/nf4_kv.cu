// Writing the paged key-value cache (with the quantization of its format) and reading it back.
//
// Both are streaming kernels: a vector of D values (one token, one kv head, K or V) is handled by D/8
// lanes, eight values (16 bytes of bf16) a lane, so that the bf16 side moves in whole 16-byte pieces
// and the absmax of a vector or of a 64-value group takes three to five shuffles.
#include <numeric>

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
    constexpr float table[16] = NF4_TABLE_VALUES;
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

// Code of r by a table of 65 intervals: interval j holds the r with round(32 r + 32) = j, so it is 1/32 wide
// and at most one threshold (they are 0.08 apart) lies in it; its entry is the code below that threshold
// and the threshold (2 if there is none).  Entries are replicated for 16 lanes side by side, so that
// a half-warp's 64-bit loads do not conflict.  (A four-step search over the thresholds: 48 us for 16384
// tokens of 8 heads; this: 27, where the bytes take 12.6.)
struct Interval {
    uint32_t code;
    float threshold;
};
struct Intervals {
    Interval e[65];
};
constexpr Intervals nf4_intervals() {
    const Thresholds thr = nf4_thresholds();
    Intervals r{};
    for (int j = 0; j < 65; j++) {
        // the ends of an interval belong to one neighbour or the other: both take a threshold that is there
        const float lo = (j - 0.5f) / 32.0f - 1.0f, hi = (j + 0.5f) / 32.0f - 1.0f;
        uint32_t c = 0;
        while (c < 15 && thr.t[c] < lo) c++;
        r.e[j].code = c;
        r.e[j].threshold = c < 15 && thr.t[c] <= hi ? thr.t[c] : 2.0f;  // r <= 1
    }
    return r;
}
__device__ __constant__ const Intervals kIntervals = nf4_intervals();
constexpr int kIntervalCopies = 16;

__device__ __forceinline__ uint32_t nf4_code(float r, uint32_t column) {
    // 2^23 + 32 + 32 r rounds to the interval's number in its low bits (r is in [-1, 1]; a non-finite r is
    // outside the contract and only has to stay inside the table)
    const uint32_t j = min(static_cast<uint32_t>(__float_as_int(__fmaf_rn(r, 32.0f, 8388640.0f)) - 0x4B000000), 64u);
    const float2 e = lds_f2(column + j * (kIntervalCopies * 8));
    return __float_as_uint(e.x) + (r >= e.y ? 1u : 0u);
}

// An item is one token and kv head, K and V; a thread walks items a grid's width apart.  The width is a
// multiple of the heads wherever there is a second step, so a thread keeps its head and only its token moves:
// the division of items by heads is done once (with the one of slots by page size it was half of the
// instructions of reading a long prefix back in 4 bits, and that is bound by them).
struct Walk {
    int64_t items;
    uint32_t width, tokens;  // items, and tokens, between a thread's items
    uint64_t page_magic;     // ceil(2^64 / page_size)
};

// The vector index of place `slot` for kv head h: (page * kv_heads + h) * page_size + offset; -1 for a slot that
// is skipped.  `reader`: the one lane that reports a slot outside the cache.
__device__ __forceinline__ int64_t place_of(const KvCache& c, uint64_t page_magic, int64_t slot, int h, bool reader) {
    if (slot < 0) return -1;
    if (slot >= c.pages * c.page_size) {
        if (reader) atomicCAS(&g_kv_error, 0, 42);
        return -1;
    }
    // exact below 2^32: the magic number is off by less than page_size <= 2^16 in 2^64
    const int64_t page = (slot >> 32) == 0 ? static_cast<int64_t>(__umul64hi(slot, page_magic)) : slot / c.page_size;
    return slot + (page * (c.kv_heads - 1) + h) * c.page_size;
}

// x / s for the many x of one divisor, correctly rounded: q = x r with r = RN(1 / s) is within an ulp of the
// quotient, and q + r (x - q s), with the remainder exact in one fma, rounds to RN(x / s) (Markstein's
// theorem) as long as nothing leaves the normal range: that is asked of s, and a quotient too small for it
// is far below the smallest code step of either format.  Other divisors take the division itself.
__device__ __forceinline__ void divide8(float (&x)[8], float s) {
    if (s > 0x1p-60f && s < 0x1p60f) {
        const float r = __frcp_rn(s);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const float q = __fmul_rn(x[j], r);
            x[j] = __fmaf_rn(__fmaf_rn(-s, q, x[j]), r, q);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) x[j] = __fdiv_rn(x[j], s);
    }
}

// One lane's eight values, quantised together with the other lanes of their vector; all 32 lanes call it.
// out: its 4, 8 or 16 bytes; scale: of the vector (fp8) or of the lane's group (NF4).
template <int FMT, int D>
__device__ __forceinline__ void quantise8(const uint4& w, uint32_t column, uint32_t (&out)[4], float& scale) {
    if (FMT == kKvBf16) {
        out[0] = w.x, out[1] = w.y, out[2] = w.z, out[3] = w.w;
        return;
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
    for (int o = 1; o < (FMT == kKvNf4 ? 8 : D / 8); o <<= 1) s = fmaxf(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
    if (FMT == kKvFp8) {
        scale = s = __fdiv_rn(s, kFp8Max);
        // A scale of 0: every code is 0.  (Divided by, it would take the slow path of the division, in lanes without an
        // item, too: one token 3.3 us, so 1.8; 4099 tokens of 8 heads 7.8 and 6.7.)
        const uint32_t keep = s > 0.0f ? 0xFFFFFFFFu : 0u;
        divide8(x, s > 0.0f ? s : 1.0f);
        out[0] = (f32x2_to_e4m3x2(x[0], x[1]) | (f32x2_to_e4m3x2(x[2], x[3]) << 16)) & keep;
        out[1] = (f32x2_to_e4m3x2(x[4], x[5]) | (f32x2_to_e4m3x2(x[6], x[7]) << 16)) & keep;
    } else {
        scale = s;
        divide8(x, s != 0.0f ? s : 1.0f);  // an all-zero group divides by 1: r = +-0, code 7
        uint32_t word = 0;
#pragma unroll
        for (int j = 0; j < 8; j++) word |= nf4_code(x[j], column) << (4 * j);
        out[0] = word;
    }
}

// Eight values of a lane from its bytes.
template <int FMT>
__device__ __forceinline__ uint4 dequantise8(const uint4& w, float s, const float* table) {
    if (FMT == kKvBf16) return w;
    uint32_t r[4];
    if (FMT == kKvFp8) {
        const uint32_t hs[4] = {e4m3x2_to_f16x2(w.x & 0xFFFFu), e4m3x2_to_f16x2(w.x >> 16),
                                e4m3x2_to_f16x2(w.y & 0xFFFFu), e4m3x2_to_f16x2(w.y >> 16)};
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hs[j]));
            r[j] = f32x2_to_bf16x2(__fmul_rn(f.x, s), __fmul_rn(f.y, s));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++)
            r[j] = f32x2_to_bf16x2(__fmul_rn(table[(w.x >> (8 * j)) & 15u], s),
                                   __fmul_rn(table[(w.x >> (8 * j + 4)) & 15u], s));
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// A lane's bytes of a stored vector: B (4, 8 or 16) of them at p.
template <int B>
__device__ __forceinline__ uint4 load_bytes(const uint8_t* p) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (B == 16) {
        v = __ldcs(reinterpret_cast<const uint4*>(p));
    } else if (B == 8) {
        const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
        v.x = u.x, v.y = u.y;
    } else {
        v.x = __ldcs(reinterpret_cast<const uint32_t*>(p));
    }
    return v;
}
template <int B>
__device__ __forceinline__ void store_bytes(uint8_t* p, const uint32_t (&v)[4]) {
    if (B == 16)
        *reinterpret_cast<uint4*>(p) = make_uint4(v[0], v[1], v[2], v[3]);
    else if (B == 8)
        *reinterpret_cast<uint2*>(p) = make_uint2(v[0], v[1]);
    else
        *reinterpret_cast<uint32_t*>(p) = v[0];
}

template <int FMT, int D>
__global__ void __launch_bounds__(256) append_kernel(KvCache c, const uint16_t* __restrict__ k_in,
                                                     const uint16_t* __restrict__ v_in,
                                                     const int64_t* __restrict__ slots, const Walk walk) {
    constexpr int L = D / 8;  // lanes a vector
    constexpr int B = kv_vector_bytes(FMT, D) / L;
    __shared__ float2 intervals[FMT == kKvNf4 ? 65 * kIntervalCopies : 1];
    if (FMT == kKvNf4) {
        for (int i = threadIdx.x; i < 65 * kIntervalCopies; i += 256) {
            const Interval e = kIntervals.e[i / kIntervalCopies];
            intervals[i] = make_float2(__uint_as_float(e.code), e.threshold);
        }
        __syncthreads();
    }
    const uint32_t column = smem_u32(intervals) + threadIdx.x % kIntervalCopies * 8;
    pdl_launch_dependents();
    pdl_wait();
    const int l = threadIdx.x % L;
    const uint32_t i0 = blockIdx.x * (256 / L) + threadIdx.x / L;  // (a grid is at most 2^26 items wide)
    uint32_t t = i0 / c.kv_heads;
    const int h = static_cast<int>(i0 - t * c.kv_heads);
    // whole warps stay in the loop: the shuffles take all 32 lanes
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * (256 / L); base < walk.items;
         base += walk.width, t += walk.tokens) {
        const int64_t i = base + threadIdx.x / L;
        uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        int64_t at = -1;
        if (i < walk.items) {
            w[0] = __ldcs(reinterpret_cast<const uint4*>(k_in) + i * L + l);
            w[1] = __ldcs(reinterpret_cast<const uint4*>(v_in) + i * L + l);
            at = place_of(c, walk.page_magic, slots[t], h, l == 0);
        }
#pragma unroll
        for (int side = 0; side < 2; side++) {
            uint32_t out[4] = {0, 0, 0, 0};
            float s = 0.0f;
            quantise8<FMT, D>(w[side], column, out, s);
            if (at < 0) continue;
            store_bytes<B>((side ? c.v : c.k) + (at * L + l) * B, out);
            uint8_t* scales = side ? c.v_scales : c.k_scales;
            if (FMT == kKvFp8 && l == 0) reinterpret_cast<float*>(scales)[at] = s;
            if (FMT == kKvNf4 && l % 8 == 0)
                reinterpret_cast<uint16_t*>(scales)[at * (D / 64) + l / 8] = __half_as_ushort(__float2half_rn(s));
        }
    }
}

// Read back: the inverse; bf16_rn(fp32(code value * scale)).
template <int FMT, int D>
__global__ void __launch_bounds__(256) read_kernel(KvCache c, const int64_t* __restrict__ slots, const Walk walk,
                                                   uint16_t* __restrict__ k_out, uint16_t* __restrict__ v_out) {
    constexpr int L = D / 8;
    constexpr int B = kv_vector_bytes(FMT, D) / L;
    __shared__ float table[16];
    if (FMT == kKvNf4) {
        if (threadIdx.x < 16) table[threadIdx.x] = kNF4[threadIdx.x];
        __syncthreads();
    }
    pdl_launch_dependents();
    pdl_wait();
    const int l = threadIdx.x % L;
    const uint32_t i0 = blockIdx.x * (256 / L) + threadIdx.x / L;
    uint32_t t = i0 / c.kv_heads;
    const int h = static_cast<int>(i0 - t * c.kv_heads);
    for (int64_t i = i0; i < walk.items; i += walk.width, t += walk.tokens) {
        const int64_t at = place_of(c, walk.page_magic, slots[t], h, l == 0);
        uint4 w[2];
        float s[2];
#pragma unroll
        for (int side = 0; side < 2; side++) {
            w[side] = make_uint4(0, 0, 0, 0);
            s[side] = 0.0f;
            if (at < 0 || !(side ? v_out : k_out)) continue;
            w[side] = load_bytes<B>((side ? c.v : c.k) + (at * L + l) * B);
            const uint8_t* scales = side ? c.v_scales : c.k_scales;
            if (FMT == kKvFp8) s[side] = reinterpret_cast<const float*>(scales)[at];
            if (FMT == kKvNf4)
                s[side] = __half2float(
                    __ushort_as_half(reinterpret_cast<const uint16_t*>(scales)[at * (D / 64) + l / 8]));
        }
#pragma unroll
        for (int side = 0; side < 2; side++) {
            uint16_t* out = side ? v_out : k_out;
            if (!out) continue;
            uint4 o = make_uint4(0, 0, 0, 0);  // a skipped item reads as zeros
            if (at >= 0) o = dequantise8<FMT>(w[side], s[side], table);
            __stcs(reinterpret_cast<uint4*>(out) + i * L + l, o);
        }
    }
}

// Up to 8 CTAs an SM; more than one step only with a width that the heads divide.  (Reading takes 32 registers, so 8 fit
// at once; writing 41 to 47, so 5, and the rest are a second wave.)
Walk item_walk(const KvCache& c, int64_t T, int D, int num_sms, dim3* grid) {
    Walk w;
    const int64_t per = 256 / (D / 8), cap = static_cast<int64_t>(num_sms) * 8;
    w.items = T * c.kv_heads;
    int64_t blocks = (w.items + per - 1) / per;
    if (blocks > cap) {
        const int64_t unit = c.kv_heads / std::gcd(static_cast<int64_t>(c.kv_heads), per);
        blocks = (cap + unit - 1) / unit * unit;
    }
    w.width = static_cast<uint32_t>(blocks * per);
    w.tokens = w.width / c.kv_heads;
    w.page_magic = ~uint64_t{0} / c.page_size + 1;
    *grid = dim3(static_cast<unsigned>(blocks));
    return w;
}

template <int FMT, int D>
cudaError_t append(const KvCache& c, const uint16_t* k, const uint16_t* v, const int64_t* slots, int64_t T,
                   int num_sms, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    dim3 grid;
    const Walk walk = item_walk(c, T, D, num_sms, &grid);
    const cudaLaunchConfig_t cfg = pdl_config(grid, 256, stream, &attr);
    return cudaLaunchKernelEx(&cfg, append_kernel<FMT, D>, c, k, v, slots, walk);
}

template <int FMT, int D>
cudaError_t read(const KvCache& c, const int64_t* slots, int64_t T, uint16_t* k, uint16_t* v, int num_sms,
                 cudaStream_t stream) {
    cudaLaunchAttribute attr;
    dim3 grid;
    const Walk walk = item_walk(c, T, D, num_sms, &grid);
    const cudaLaunchConfig_t cfg = pdl_config(grid, 256, stream, &attr);
    return cudaLaunchKernelEx(&cfg, read_kernel<FMT, D>, c, slots, walk, k, v);
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
