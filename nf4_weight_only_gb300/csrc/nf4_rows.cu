// Rotary positions and the residual RMS norm: elementwise work over rows of activations, bound by the
// bytes of their rows (long calls) or by the latency of one launch (decode).
#include <cmath>
#include <mutex>

#include "nf4_kv.cuh"

namespace nf4 {
namespace {

// ---------------------------------------------------------------------------------------------
// Rotary positions
// ---------------------------------------------------------------------------------------------
// A thread owns eight pairs of one token (16 values a head, two 16-byte pieces) and walks some of the
// token's q and k heads with them, so the angles are computed once for all of these heads.
//
// Angle of a pair: positions * inv_freq radians, a real product, needed modulo 2 pi.  inv_freq / (2 pi) is
// held as a 64-bit binary fraction F of a turn; F * position modulo 2^64 is then the fraction of the product,
// exactly, by integer wrap-around.  With inv_freq = m 2^e (m of 24 bits) F is the product of m and 2^64 / (2 pi),
// shifted by e, all in integers (double precision here runs at a sixty-fourth of the single rate and took
// half of the kernel's time); F's error, 2^-63 below inv_freq = 1 (2^-55 below 256, 2^-64 above), times the position
// is below 2^-31 turn (2^-24).  The upper 32 bits of F * position, as a signed number, are an angle in [-pi, pi),
// where the hardware sine and cosine have an absolute error near 2^-21, far below the 2^-8 of the bf16 result.
constexpr int kRopeThreads = 256;

struct Turn {
    float c[8], s[8];
};

// 1 / (2 pi) in binary, 32 bits a word, behind a word of zeros.
__device__ __constant__ const uint32_t kInverseTwoPi[8] = {0x00000000u, 0x28BE60DBu, 0x9391054Au, 0x7F09D5F4u,
                                                           0x7D4D3770u, 0x36D8A566u, 0x4F10E410u, 0x7F9458EAu};

// |f| = m 2^e from 256 on, e in [-15, 104] (the reduction of Payne and Hanek, 1983): of 1 / (2 pi), the bits before
// 2^-e give whole turns, and the 96 bits from there, times m, the fraction to 2^-64.
// (Kept out of line: inlined, the compiler computes it for every pair and selects.)
__device__ __noinline__ uint64_t turn_fraction_large(uint32_t m, int e) {
    const int word = (e + 32) >> 5, bit = (e + 32) & 31;
    uint32_t g[3];
#pragma unroll
    for (int i = 0; i < 3; i++) g[i] = __funnelshift_l(kInverseTwoPi[word + i + 1], kInverseTwoPi[word + i], bit);
    return m * ((static_cast<uint64_t>(g[0]) << 32) | g[1]) + ((static_cast<uint64_t>(m) * g[2]) >> 32);
}

// The fraction of a turn, times 2^64, that one position moves a pair of angular frequency f.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
    const uint32_t bits = __float_as_uint(f) & 0x7FFFFFFFu;
    const int e = max(static_cast<int>(bits >> 23), 1) - 150;  // |f| = m 2^e
    const uint64_t m = (bits & 0x7FFFFFu) | (bits >= 0x800000u ? 0x800000u : 0u);
    uint64_t frac;
    if (e <= -16) {  // |f| < 256
        const uint64_t high = __umul64hi(2935890503282001226ull, m << 40);  // m 2^64 / (2 pi) / 2^24
        const int shift = e + 24;
        frac = shift >= 0 ? high << shift : shift > -64 ? high >> -shift : 0;
    } else {
        frac = turn_fraction_large(static_cast<uint32_t>(m), e);
    }
    return f < 0.0f ? 0 - frac : frac;
}

// AHEAD: heads whose loads are in flight together.
template <int AHEAD>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a, int heads_step) {
    pdl_launch_dependents();
    const int chunks = a.head_dim / 16, rot = a.rotary_dim / 16;
    const int per_token = chunks * heads_step;
    int64_t t;
    int id;
    if (per_token <= kRopeThreads) {
        const int per_block = kRopeThreads / per_token;
        t = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x / per_token;
        id = threadIdx.x % per_token;
        if (threadIdx.x / per_token >= per_block) t = a.T;
    } else {
        t = blockIdx.x;
        id = blockIdx.y * kRopeThreads + threadIdx.x;
    }
    if (t >= a.T || id >= per_token) {
        pdl_wait();
        return;
    }
    const int c = id % chunks, h0 = id / chunks;
    pdl_wait();
    const bool turn = c < rot;
    // elements of this thread's two pieces inside a head
    const int e0 = turn && !a.interleaved ? 8 * c : 16 * c;
    const int e1 = turn && !a.interleaved ? 8 * c + a.rotary_dim / 2 : 16 * c + 8;
    const int heads = a.q_heads + a.k_heads;
    uint4 u[AHEAD], v[AHEAD];
    uint16_t* dst[AHEAD];
    auto load = [&](int h) {
#pragma unroll
        for (int n = 0; n < AHEAD; n++) {
            const int hn = h + n * heads_step;
            dst[n] = nullptr;
            if (hn < heads) {
                const bool is_q = hn < a.q_heads;
                const int64_t row = (is_q ? t * a.q_heads + hn : t * a.k_heads + (hn - a.q_heads)) * a.head_dim;
                const uint16_t* src = (is_q ? a.q : a.k) + row;
                dst[n] = (is_q ? a.q_out : a.k_out) + row;
                u[n] = __ldcs(reinterpret_cast<const uint4*>(src + e0));
                v[n] = __ldcs(reinterpret_cast<const uint4*>(src + e1));
            }
        }
    };
    load(h0);  // in flight while the angles are worked out
    Turn r;
    if (turn) {
        int32_t pos[4];
#pragma unroll
        for (int x = 0; x < 4; x++) pos[x] = x < a.axes ? a.positions[x * a.T + t] : 0;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int i = 8 * c + j;
            const int32_t p = i < a.section_end[0]   ? pos[0]
                              : i < a.section_end[1] ? pos[1]
                              : i < a.section_end[2] ? pos[2]
                                                     : pos[3];
            const uint64_t at = turn_fraction(a.inv_freq[i]) * static_cast<uint64_t>(static_cast<int64_t>(p));
            constexpr float kTurn = 1.4629180792671596e-9f;  // 2 pi / 2^32
            const float angle = static_cast<float>(static_cast<int32_t>(at >> 32)) * kTurn;
            r.s[j] = __sinf(angle) * a.magnitude;
            r.c[j] = __cosf(angle) * a.magnitude;
        }
    }
    for (int h = h0; h < heads;) {
#pragma unroll
        for (int n = 0; n < AHEAD; n++) {
            if (!dst[n]) continue;
            if (turn) {
                const uint32_t in0[4] = {u[n].x, u[n].y, u[n].z, u[n].w}, in1[4] = {v[n].x, v[n].y, v[n].z, v[n].w};
                uint32_t o0[4], o1[4];
                if (a.interleaved) {
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const float2 p = bf16x2_to_f32x2(j < 4 ? in0[j & 3] : in1[j & 3]);
                        const uint32_t w = f32x2_to_bf16x2(p.x * r.c[j] - p.y * r.s[j], p.y * r.c[j] + p.x * r.s[j]);
                        (j < 4 ? o0 : o1)[j & 3] = w;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const float2 p = bf16x2_to_f32x2(in0[j]), q = bf16x2_to_f32x2(in1[j]);
                        const float c0 = r.c[2 * j], c1 = r.c[2 * j + 1], s0 = r.s[2 * j], s1 = r.s[2 * j + 1];
                        o0[j] = f32x2_to_bf16x2(p.x * c0 - q.x * s0, p.y * c1 - q.y * s1);
                        o1[j] = f32x2_to_bf16x2(q.x * c0 + p.x * s0, q.y * c1 + p.y * s1);
                    }
                }
                u[n] = make_uint4(o0[0], o0[1], o0[2], o0[3]);
                v[n] = make_uint4(o1[0], o1[1], o1[2], o1[3]);
            }
            __stcs(reinterpret_cast<uint4*>(dst[n] + e0), u[n]);
            __stcs(reinterpret_cast<uint4*>(dst[n] + e1), v[n]);
        }
        h += AHEAD * heads_step;
        if (h < heads) load(h);
    }
}

// ---------------------------------------------------------------------------------------------
// Residual RMS norm
// ---------------------------------------------------------------------------------------------
// Two forms.  rmsnorm_kernel, for few rows, narrow or very wide ones: one CTA a row.  h = x + residual stays in
// registers (CH pieces of eight values a thread; CH = 0, for rows past 32768 values, reads the row again), one
// block reduction gives sum(h^2) and max |h w| at once: max |y| = rsqrt(...) * max |h w|, so the 8-bit scale
// needs no second one.  With many rows its CTAs spend their time waiting for their loads (8192 x 5120, 8 bits
// out: 58 us, 75% of the measured copy rate; 2048 x 16384, which stays with it: to bf16 55 us, 73%).
// rmsnorm_ring_kernel, for those: persistent CTAs whose next two rows are on their way into shared memory;
// each thread copies what it will read itself, so the ring needs no barrier.
__device__ __forceinline__ float2 block_sum_max(float2 v, float2* part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
        v.y = fmaxf(v.y, __shfl_xor_sync(0xFFFFFFFFu, v.y, o));
    }
    const int warps = blockDim.x / 32;
    if (warps == 1) return v;
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    float2 r = part[0];
    for (int w = 1; w < warps; w++) {
        const float2 p = part[w];
        r.x += p.x;
        r.y = fmaxf(r.y, p.y);
    }
    return r;
}

// 1 / sqrt(mean square + eps); 0 for a zero row without an eps, so that it gives zeros and not 0 * inf.
__device__ __forceinline__ float row_rstd(float square_sum, float inv_h, float eps) {
    const float v = square_sum * inv_h + eps;
    return v == 0.0f ? 0.0f : 1.0f / sqrtf(v);
}

struct NormArgs {
    const uint4 *x, *residual, *weight;
    uint4 *residual_out, *y;
    uint2* y8;
    float* y8_scales;
    int vecs;  // 16-byte pieces a row
    float inv_h, eps;
};

__device__ __forceinline__ void unpack(const uint4& x, float (&h)[8]) {
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const float2 f = bf16x2_to_f32x2(xs[j]);
        h[2 * j] = f.x, h[2 * j + 1] = f.y;
    }
}

// x + residual of a piece.
__device__ __forceinline__ void load_h(const NormArgs& a, int64_t at, float (&h)[8]) {
    unpack(a.x[at], h);
    if (a.residual) {
        float r[8];
        unpack(a.residual[at], r);
#pragma unroll
        for (int j = 0; j < 8; j++) h[j] += r[j];
    }
}

__device__ __forceinline__ uint4 pack_bf16(const float (&v)[8]) {
    return make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]),
                      f32x2_to_bf16x2(v[6], v[7]));
}

// The row's 8-bit scale: codes of y / scale, as y * inv where the reciprocal is a normal number (its ulp is as much as
// y's own rounding to fp32; a correctly rounded quotient made 8192 x 5120 4% slower), else by the division itself.
struct RowScale {
    float scale, inv;  // inv = 0: divide
    __device__ __forceinline__ explicit RowScale(float s) : scale(s), inv(s >= 0x1p-126f ? 1.0f / s : 0.0f) {}
};

__device__ __forceinline__ void store_out(const NormArgs& a, int64_t at, const float (&h)[8], const float (&w)[8],
                                          float rstd, const RowScale& s) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; j++) y[j] = h[j] * rstd * w[j];
    if (a.residual_out) a.residual_out[at] = pack_bf16(h);
    if (a.y) a.y[at] = pack_bf16(y);
    if (a.y8) {
        if (s.inv != 0.0f) {
#pragma unroll
            for (int j = 0; j < 8; j++) y[j] *= s.inv;
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) y[j] = s.scale > 0.0f ? __fdiv_rn(y[j], s.scale) : 0.0f;
        }
        a.y8[at] = make_uint2(f32x2_to_e4m3x2(y[0], y[1]) | (f32x2_to_e4m3x2(y[2], y[3]) << 16),
                              f32x2_to_e4m3x2(y[4], y[5]) | (f32x2_to_e4m3x2(y[6], y[7]) << 16));
    }
}

template <int CH>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const NormArgs a) {
    __shared__ float2 part[32];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * a.vecs;
    constexpr int N = CH ? CH : 1;
    float h[N][8];
    float2 acc = make_float2(0.0f, 0.0f);
    auto add = [&](const float (&v)[8], int i) {
        float w[8];
        if (a.y8) unpack(a.weight[i], w);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            acc.x = fmaf(v[j], v[j], acc.x);
            if (a.y8) acc.y = fmaxf(acc.y, fabsf(v[j] * w[j]));
        }
    };
    if (CH) {
#pragma unroll
        for (int c = 0; c < N; c++) {
            const int i = threadIdx.x + c * blockDim.x;
            if (i < a.vecs) load_h(a, row + i, h[c]);
        }
#pragma unroll
        for (int c = 0; c < N; c++) {
            const int i = threadIdx.x + c * blockDim.x;
            if (i < a.vecs) add(h[c], i);
        }
    } else {
        for (int i = threadIdx.x; i < a.vecs; i += blockDim.x) {
            load_h(a, row + i, h[0]);
            add(h[0], i);
        }
    }
    acc = block_sum_max(acc, part);
    const float rstd = row_rstd(acc.x, a.inv_h, a.eps);
    const RowScale scale(a.y8 ? acc.y * rstd / kFp8Max : 0.0f);
    if (a.y8 && threadIdx.x == 0) a.y8_scales[blockIdx.x] = scale.scale;
    if (CH) {
#pragma unroll
        for (int c = 0; c < N; c++) {
            const int i = threadIdx.x + c * blockDim.x;
            if (i < a.vecs) {
                float w[8];
                unpack(a.weight[i], w);
                store_out(a, row + i, h[c], w, rstd, scale);
            }
        }
    } else {
        for (int i = threadIdx.x; i < a.vecs; i += blockDim.x) {
            float w[8];
            load_h(a, row + i, h[0]);
            unpack(a.weight[i], w);
            store_out(a, row + i, h[0], w, rstd, scale);
        }
    }
}

constexpr int kNormStages = 3;

constexpr int kNormPieces = 2;  // 16-byte pieces of a row a thread

__global__ void __launch_bounds__(512, 2) rmsnorm_ring_kernel(const NormArgs a, int rows) {
    extern __shared__ __align__(16) uint4 ring[];  // [kNormStages][x, residual][vecs]
    __shared__ float2 part[2][32];
    pdl_launch_dependents();
    pdl_wait();
    const int sides = a.residual ? 2 : 1;
    uint4 w[kNormPieces];
#pragma unroll
    for (int c = 0; c < kNormPieces; c++) {
        const int i = threadIdx.x + c * blockDim.x;
        w[c] = i < a.vecs ? a.weight[i] : make_uint4(0, 0, 0, 0);
    }
    int stage_in = 0, stage = 0;
    auto issue = [&](int64_t row) {
        if (row < rows) {
            uint4* to = ring + stage_in * sides * a.vecs;
#pragma unroll
            for (int c = 0; c < kNormPieces; c++) {
                const int i = threadIdx.x + c * blockDim.x;
                if (i < a.vecs) {
                    cp_async16(to + i, a.x + row * a.vecs + i);
                    if (a.residual) cp_async16(to + a.vecs + i, a.residual + row * a.vecs + i);
                }
            }
            stage_in = stage_in + 1 == kNormStages ? 0 : stage_in + 1;
        }
        cp_async_commit();
    };
    for (int k = 0; k < kNormStages - 1; k++) issue(blockIdx.x + static_cast<int64_t>(k) * gridDim.x);
    int flip = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, flip ^= 1) {
        cp_async_wait<kNormStages - 2>();
        const uint4* from = ring + stage * sides * a.vecs;
        stage = stage + 1 == kNormStages ? 0 : stage + 1;
        float h[kNormPieces][8];
        float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int c = 0; c < kNormPieces; c++) {
            const int i = threadIdx.x + c * blockDim.x;
            if (i >= a.vecs) continue;
            unpack(from[i], h[c]);
            float v[8];
            if (a.residual) {
                unpack(from[a.vecs + i], v);
#pragma unroll
                for (int j = 0; j < 8; j++) h[c][j] += v[j];
            }
            unpack(w[c], v);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                acc.x = fmaf(h[c][j], h[c][j], acc.x);
                if (a.y8) acc.y = fmaxf(acc.y, fabsf(h[c][j] * v[j]));
            }
        }
        issue(row + static_cast<int64_t>(kNormStages - 1) * gridDim.x);
        acc = block_sum_max(acc, part[flip]);
        const float rstd = row_rstd(acc.x, a.inv_h, a.eps);
        const RowScale scale(a.y8 ? acc.y * rstd / kFp8Max : 0.0f);
        if (a.y8 && threadIdx.x == 0) a.y8_scales[row] = scale.scale;
#pragma unroll
        for (int c = 0; c < kNormPieces; c++) {
            const int i = threadIdx.x + c * blockDim.x;
            if (i >= a.vecs) continue;
            float v[8];
            unpack(w[c], v);
            store_out(a, row * a.vecs + i, h[c], v, rstd, scale);
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int num_sms, cudaStream_t stream) {
    const int heads = a.q_heads + a.k_heads, chunks = a.head_dim / 16;
    // Heads a thread walks: as many (up to eight) as leave every SM a thousand threads.
    const int64_t threads = a.T * heads * chunks;
    int64_t walk = threads / (static_cast<int64_t>(num_sms) * 1024);
    if (walk > 8) walk = 8;
    if (walk < 1) walk = 1;
    const int step = static_cast<int>((heads + walk - 1) / walk), per_token = chunks * step;
    dim3 grid(static_cast<unsigned>(a.T), (per_token + kRopeThreads - 1) / kRopeThreads);
    if (per_token <= kRopeThreads) {
        const int per_block = kRopeThreads / per_token;
        grid = dim3(static_cast<unsigned>((a.T + per_block - 1) / per_block));
    }
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = pdl_config(grid, kRopeThreads, stream, &attr);
    return walk > 1 ? cudaLaunchKernelEx(&cfg, rope_kernel<4>, a, step)
                    : cudaLaunchKernelEx(&cfg, rope_kernel<1>, a, step);
}

cudaError_t launch_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int64_t T, int64_t H,
                           float eps, uint16_t* residual_out, uint16_t* y, uint8_t* y8, float* y8_scales, int num_sms,
                           cudaStream_t stream) {
    NormArgs a{};
    a.x = reinterpret_cast<const uint4*>(x);
    a.residual = reinterpret_cast<const uint4*>(residual);
    a.weight = reinterpret_cast<const uint4*>(weight);
    a.residual_out = reinterpret_cast<uint4*>(residual_out);
    a.y = reinterpret_cast<uint4*>(y);
    a.y8 = reinterpret_cast<uint2*>(y8);
    a.y8_scales = y8_scales;
    a.vecs = static_cast<int>(H / 8);
    a.inv_h = static_cast<float>(1.0 / static_cast<double>(H));
    a.eps = eps;
    // Many rows of 2048 to 8192 values: the ring (8192 x 5120, 8 bits out: 48 us, without it 58; 4096 x 6144: 35
    // and 40; narrower rows gain nothing, 32768 x 1024: 46 and 40).
    if (T > 4 * num_sms && a.vecs > 256 && a.vecs <= 512 * kNormPieces) {
        static std::once_flag attr_once[64];  // once per device
        int dev = 0;
        cudaGetDevice(&dev);
        cudaError_t attr_err = cudaSuccess;
        std::call_once(attr_once[dev & 63], [&] {
            attr_err = cudaFuncSetAttribute(rmsnorm_ring_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            kNormStages * 2 * 512 * kNormPieces * 16);
        });
        if (attr_err != cudaSuccess) return attr_err;
        const int ring_bytes = kNormStages * (residual ? 2 : 1) * a.vecs * 16;
        const int threads = ((a.vecs + kNormPieces - 1) / kNormPieces + 31) / 32 * 32;
        int per_sm = 224 * 1024 / (ring_bytes + 2048);
        if (per_sm > 1024 / threads) per_sm = 1024 / threads;  // 64 registers a thread
        int64_t grid = static_cast<int64_t>(num_sms) * per_sm;
        if (grid > T) grid = T;
        cudaLaunchAttribute attr;
        cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(grid)), threads, stream, &attr);
        cfg.dynamicSmemBytes = ring_bytes;
        return cudaLaunchKernelEx(&cfg, rmsnorm_ring_kernel, a, static_cast<int>(T));
    }
    // Few rows: as many threads as the row has pieces.  Many rows: up to four pieces a thread, which
    // leaves room for more rows an SM.
    const int want = T <= 2 * num_sms ? 1024 : 256;
    const int64_t pieces = (a.vecs + want - 1) / want;
    const int ch = pieces <= 1 ? 1 : pieces <= 2 ? 2 : 4;
    int64_t threads = ((a.vecs + ch - 1) / ch + 31) / 32 * 32;
    const bool wide = threads > 1024;
    if (wide) threads = 1024;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg =
        pdl_config(dim3(static_cast<unsigned>(T)), static_cast<int>(threads), stream, &attr);
    if (wide) return cudaLaunchKernelEx(&cfg, rmsnorm_kernel<0>, a);
    switch (ch) {
        case 1: return cudaLaunchKernelEx(&cfg, rmsnorm_kernel<1>, a);
        case 2: return cudaLaunchKernelEx(&cfg, rmsnorm_kernel<2>, a);
        default: return cudaLaunchKernelEx(&cfg, rmsnorm_kernel<4>, a);
    }
}

}  // namespace nf4
