// Low-rank adapters of many requests beside projections that share their input:
//   y[t] = base[t] + s[a] * B[a] (A[a] x[t]),  a the adapter of token t.
//
// Tokens are first listed adapter by adapter (lora_plan_kernel, once for all calls of a step), in chunks of up to
// 64 tokens of one adapter, so that an adapter's matrices are read once a chunk.  Two kernels follow:
//   shrink  h = A x for a chunk, the rank columns of all projections side by side; the long axis K is split over
//           warps and CTAs, and a slice's sums go to the workspace in fp32
//   expand  adds the slices in order, scales, and adds B h to the base
// Both use mma.sync m16n8k16 with tokens as the 16 rows and weights as the 8 columns.  A product's k axis may
// be permuted at will if both operands are permuted alike: a lane takes eight consecutive k (16 bytes) of its
// row or column, which is two k steps of the instruction, and needs neither shared memory nor shuffles.
#include <mutex>

#include "nf4_kv.cuh"

namespace nf4 {
namespace {

constexpr int kChunk = 64;      // tokens of a chunk at most
constexpr int kHeader = 8;      // int32 before the chunks: T, adapters, chunks, tokens with an adapter
constexpr int kThreads = 256;
constexpr int kSliceUnits = 304;  // chunks * slices of K, two CTAs for each of 152 SMs
constexpr int kMaxSlices = 32;

__device__ int g_lora_error;  // 46: an adapter or a row outside its list; 47: a plan of other sizes

__host__ __device__ inline int64_t max_chunks(int64_t T, int64_t adapters) {
    const int64_t n = T / kChunk + (adapters < T ? adapters : T);
    return n < T ? n : T;
}

// ---------------------------------------------------------------------------------------------
// Plan
// ---------------------------------------------------------------------------------------------
// A counting sort in one CTA that keeps the tokens of an adapter in order.
__global__ void __launch_bounds__(1024) lora_plan_kernel(const int32_t* __restrict__ ids,
                                                         const int32_t* __restrict__ sequences, int64_t S, int64_t T,
                                                         int adapters, int32_t* __restrict__ plan) {
    extern __shared__ int32_t counts[];  // [adapters + 1] tokens, then places; [adapters + 1] first chunks
    int32_t* chunk_at = counts + adapters + 1;
    __shared__ int32_t part[2][32];
    __shared__ int2 groups[32][32];  // of a round, for each warp: the lists that its tokens belong to, and how many each
    __shared__ int32_t n_groups[32];
    pdl_launch_dependents();
    for (int a = threadIdx.x; a <= adapters; a += blockDim.x) counts[a] = 0;
    __syncthreads();
    pdl_wait();
    bool bad = false;
    // the list that token t belongs to: its adapter's, or the last one's for none
    auto list_of = [&](int64_t t) {
        int64_t row = t;
        if (sequences) {
            row = sequences[t];
            if (row < 0) return adapters;
            if (row >= S) {
                bad = true;
                return adapters;
            }
        }
        const int32_t id = ids[row];
        if (id >= adapters) bad = true;
        return id < 0 || id >= adapters ? adapters : id;
    };
    const int64_t rounds = (T + blockDim.x - 1) / blockDim.x;
    const int lane = threadIdx.x % 32;
    for (int64_t i = 0; i < rounds; i++) {
        const int64_t t = i * blockDim.x + threadIdx.x;
        const int list = t < T ? list_of(t) : -1;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, list);
        if (list >= 0 && lane == __ffs(same) - 1) atomicAdd(&counts[list], __popc(same));
    }
    __syncthreads();
    // exclusive sums of tokens and of chunks; each thread takes a run of lists
    const int per = (adapters + 1 + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
    const int a0 = min(adapters + 1, static_cast<int>(threadIdx.x) * per), a1 = min(adapters + 1, a0 + per);
    int32_t n = 0, c = 0;
    for (int a = a0; a < a1; a++) {
        n += counts[a];
        c += a < adapters ? (counts[a] + kChunk - 1) / kChunk : 0;
    }
    int32_t sn = n, sc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t un = __shfl_up_sync(0xFFFFFFFFu, sn, o), uc = __shfl_up_sync(0xFFFFFFFFu, sc, o);
        if (lane >= o) sn += un, sc += uc;
    }
    if (lane == 31) part[0][threadIdx.x / 32] = sn, part[1][threadIdx.x / 32] = sc;
    __syncthreads();
    int32_t bn = 0, bc = 0, chunks = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x) / 32; w++) {
        if (w == static_cast<int>(threadIdx.x) / 32) bn += sn - n, bc = chunks + sc - c;
        if (w < static_cast<int>(threadIdx.x) / 32) bn += part[0][w];
        chunks += part[1][w];
    }
    int4* out = reinterpret_cast<int4*>(plan + kHeader);
    int32_t* order = plan + kHeader + 4 * max_chunks(T, adapters);
    for (int a = a0; a < a1; a++) {
        const int32_t tokens = counts[a];
        counts[a] = bn;
        chunk_at[a] = bc;
        bn += tokens;
        bc += a < adapters ? (tokens + kChunk - 1) / kChunk : 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < chunks; i += blockDim.x) {
        int lo = 0, hi = adapters;  // the last list whose first chunk is at most i (lists without chunks come before)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (chunk_at[mid] <= i)
                lo = mid;
            else
                hi = mid;
        }
        const int32_t first = counts[lo] + (i - chunk_at[lo]) * kChunk;
        out[i] = make_int4(lo, first, min(kChunk, counts[lo + 1] - first), 0);
    }
    if (threadIdx.x == 1) *reinterpret_cast<int4*>(plan + 4) = make_int4(0, 0, 0, 0);
    if (threadIdx.x == 0)
        *reinterpret_cast<int4*>(plan) = make_int4(static_cast<int32_t>(T), adapters, chunks, counts[adapters]);
    __syncthreads();
    for (int64_t i = 0; i < rounds; i++) {
        const int64_t t = i * blockDim.x + threadIdx.x;
        const int list = t < T ? list_of(t) : -1;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, list);
        const bool leads = list >= 0 && lane == __ffs(same) - 1;
        const uint32_t leaders = __ballot_sync(0xFFFFFFFFu, leads);
        const int warp = threadIdx.x / 32;
        if (leads) groups[warp][__popc(leaders & ((1u << lane) - 1))] = make_int2(list, __popc(same));
        if (lane == 0) n_groups[warp] = __popc(leaders);
        __syncthreads();
        int32_t at = 0;
        if (leads) {
            at = counts[list];
            for (int w = 0; w < warp; w++)
                for (int j = 0; j < n_groups[w]; j++) {
                    const int2 group = groups[w][j];
                    at += group.x == list ? group.y : 0;
                }
        }
        __syncthreads();
        if (leads) atomicAdd(&counts[list], __popc(same));  // a sum: any order
        at = __shfl_sync(0xFFFFFFFFu, at, __ffs(same) - 1) + __popc(same & ((1u << lane) - 1));
        if (list >= 0) order[at] = static_cast<int32_t>(t);
        __syncthreads();
    }
    if (bad) atomicCAS(&g_lora_error, 0, 46);
}

// ---------------------------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two k steps: rows g and g + 8 of 16 tokens against column g of 8 weights, eight k a lane.
__device__ __forceinline__ void mma_k32(float (&d)[4], const uint4& x0, const uint4& x1, const uint4& w) {
    mma_bf16(d, x0.x, x1.x, x0.y, x1.y, w.x, w.y);
    mma_bf16(d, x0.z, x1.z, x0.w, x1.w, w.z, w.w);
}

// The plan as both kernels read it.
struct Plan {
    const int4* chunks;
    const int32_t* order;
    int n_chunks, n_tokens;
};
// False (and 47 recorded) if the plan was made for other sizes.
__device__ __forceinline__ bool read_plan(const LoraArgs& a, Plan* p) {
    const int4 h = *reinterpret_cast<const int4*>(a.plan);
    const int64_t most = max_chunks(a.T, a.adapters);
    p->chunks = reinterpret_cast<const int4*>(a.plan + kHeader);
    p->order = a.plan + kHeader + 4 * most;
    p->n_chunks = h.z, p->n_tokens = h.w;
    if (h.x != a.T || h.y != a.adapters || h.z < 0 || h.z > most || h.w < 0 || h.w > a.T ||
        h.w > static_cast<int64_t>(h.z) * kChunk) {
        if (threadIdx.x == 0) atomicCAS(&g_lora_error, 0, 47);
        return false;
    }
    return true;
}
__device__ __forceinline__ bool chunk_ok(const LoraArgs& a, const Plan& p, const int4& c) {
    return c.x >= 0 && c.x < a.adapters && c.y >= 0 && c.z > 0 && c.z <= kChunk && c.y + c.z <= p.n_tokens;
}
__device__ __forceinline__ int64_t token_at(const LoraArgs& a, const Plan& p, int at) {
    return min(static_cast<uint32_t>(p.order[at]), static_cast<uint32_t>(a.T - 1));
}
// Slices of K: as many as fill the GPU, each with at least one step of 32 for every warp.
__device__ __forceinline__ int slices(const LoraArgs& a, const Plan& p) {
    const int steps = static_cast<int>(a.K / 32 / (kThreads / 32));
    return max(1, min(min(kMaxSlices, steps), kSliceUnits / max(1, p.n_chunks)));
}

// One slice of one chunk and up to NT * 8 rank columns; MT tiles of 16 tokens.
template <int MT, int NT>
__device__ __forceinline__ void shrink_unit(const LoraArgs& a, const Plan& p, const int4& chunk, int slice, int n_slices,
                                            int tile0, float* sums) {
    constexpr int kCols = NT * 8, kStride = kCols + 4;  // (a warp's 64-bit stores: 8 rows, 4 columns apart)
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int per = a.rank / 8, tiles = min(NT, a.count * per - tile0);
    const uint16_t* xp[MT][2];
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
        for (int h = 0; h < 2; h++)  // a row past the chunk's end repeats the last
            xp[m][h] = a.x + token_at(a, p, chunk.y + min(m * 16 + h * 8 + g, chunk.z - 1)) * a.K + 8 * t;
    const uint16_t* wp[NT];
#pragma unroll
    for (int j = 0; j < NT; j++) {
        const int tile = tile0 + min(j, tiles - 1), i = tile / per;
        wp[j] = a.a[i] + (static_cast<int64_t>(chunk.x) * a.rank + (tile - i * per) * 8 + g) * a.K + 8 * t;
    }
    float acc[MT][NT][4] = {};
    const int64_t steps = a.K / 32, k0 = steps * slice / n_slices, k1 = steps * (slice + 1) / n_slices;
    uint4 x[MT][2], w[NT];
    auto load = [&](int64_t k) {
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int h = 0; h < 2; h++) x[m][h] = *reinterpret_cast<const uint4*>(xp[m][h] + 32 * k);
#pragma unroll
        for (int j = 0; j < NT; j++)
            if (j < tiles) w[j] = __ldg(reinterpret_cast<const uint4*>(wp[j] + 32 * k));
    };
    for (int64_t k = k0 + warp; k < k1; k += kThreads / 32) {
        load(k);
#pragma unroll
        for (int j = 0; j < NT; j++)
            if (j < tiles)
#pragma unroll
                for (int m = 0; m < MT; m++) mma_k32(acc[m][j], x[m][0], x[m][1], w[j]);
    }
    // the warps' sums: four of them write, the others add, then all add the four, always in this order
    float* own = sums + (warp % 4) * (MT * 16 * kStride);
    __syncthreads();  // the last unit's sums are read
#pragma unroll
    for (int round = 0; round < 2; round++) {
        if (warp / 4 == round)
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int j = 0; j < NT; j++)
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        float2* at = reinterpret_cast<float2*>(own + (m * 16 + h * 8 + g) * kStride + j * 8 + 2 * t);
                        float2 v = make_float2(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
                        if (round) {
                            const float2 o = *at;
                            v.x += o.x, v.y += o.y;
                        }
                        *at = v;
                    }
        __syncthreads();
    }
    const int R = a.count * a.rank;
    float* out = a.h + (static_cast<int64_t>(slice) * p.n_tokens + chunk.y) * R + tile0 * 8;
    for (int e = threadIdx.x; e < chunk.z * kCols; e += kThreads) {
        const int row = e / kCols, col = e % kCols;
        if (col >= tiles * 8) continue;
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < 4; q++) v += sums[q * (MT * 16 * kStride) + row * kStride + col];
        out[static_cast<int64_t>(row) * R + col] = v;
    }
}

constexpr int kShrinkTiles = 4;  // rank columns of a unit, in eights
constexpr int kShrinkSmem = 4 * kChunk * (kShrinkTiles * 8 + 4) * 4;

__global__ void __launch_bounds__(kThreads, 2) shrink_kernel(const LoraArgs a) {
    __shared__ __align__(16) float sums[kShrinkSmem / 4];
    pdl_launch_dependents();
    pdl_wait();
    Plan p;
    if (!read_plan(a, &p)) return;
    const int n_slices = slices(a, p), groups = (a.count * a.rank / 8 + kShrinkTiles - 1) / kShrinkTiles;
    const int64_t units = static_cast<int64_t>(p.n_chunks) * n_slices * groups;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t cs = u / groups;
        const int4 chunk = p.chunks[cs / n_slices];
        if (!chunk_ok(a, p, chunk)) continue;
        const int slice = static_cast<int>(cs % n_slices), tile0 = static_cast<int>(u % groups) * kShrinkTiles;
        if (chunk.z <= 16)
            shrink_unit<1, kShrinkTiles>(a, p, chunk, slice, n_slices, tile0, sums);
        else if (chunk.z <= 32)
            shrink_unit<2, kShrinkTiles>(a, p, chunk, slice, n_slices, tile0, sums);
        else
            shrink_unit<4, kShrinkTiles>(a, p, chunk, slice, n_slices, tile0, sums);
    }
}

// KB: steps of 32 that hold the rank.  A unit is a chunk and 256 rows of one projection, 32 a warp; column g of
// a warp's tile j is row 8 (g / 2) + 2 j + g % 2, so that a lane's results are eight consecutive values of y.
template <int KB>
__global__ void __launch_bounds__(kThreads) expand_kernel(const LoraArgs a, int blocks, bool copy) {
    constexpr int kStride = KB * 32 + 8;
    __shared__ __align__(16) uint16_t hi[kChunk * kStride], lo[kChunk * kStride];
    __shared__ int32_t rows[kChunk];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    pdl_launch_dependents();
    pdl_wait();
    Plan p;
    if (!read_plan(a, &p)) return;
    const int n_slices = slices(a, p), R = a.count * a.rank;
    // rows without an adapter are copied where the output is not the base itself
    const int idle = copy ? static_cast<int>((a.T - p.n_tokens + kChunk - 1) / kChunk) : 0;
    const int64_t units = static_cast<int64_t>(p.n_chunks + idle) * blocks;
    const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
    int held = -1;  // the chunk and projection in shared memory
    for (int64_t u = u0; u < u1; u++) {
        const int c = static_cast<int>(u / blocks);
        int block = static_cast<int>(u % blocks), i = 0;
        for (; i < a.count; i++) {
            const int n = static_cast<int>((a.N[i] + 255) / 256);
            if (block < n) break;
            block -= n;
        }
        const int64_t N = a.N[i], n0 = static_cast<int64_t>(block) * 256 + warp * 32;
        const bool vec = N % 8 == 0;
        if (c >= p.n_chunks) {
            if (a.base[i] == a.y[i]) continue;
            const int first = p.n_tokens + (c - p.n_chunks) * kChunk, n = min(kChunk, static_cast<int>(a.T) - first);
            for (int r = g; r < n; r += 8) {
                const int64_t at = token_at(a, p, first + r) * N + n0 + 8 * t;
                if (vec) {
                    if (n0 + 8 * t < N)
                        *reinterpret_cast<uint4*>(a.y[i] + at) = *reinterpret_cast<const uint4*>(a.base[i] + at);
                } else {
                    for (int j = 0; j < 8; j++)
                        if (n0 + 8 * t + j < N) a.y[i][at + j] = a.base[i][at + j];
                }
            }
            continue;
        }
        const int4 chunk = p.chunks[c];
        if (!chunk_ok(a, p, chunk)) continue;
        if (held != c * a.count + i) {
            held = c * a.count + i;
            __syncthreads();
            const float s = a.scales[chunk.x];
            for (int e = threadIdx.x; e < kChunk * KB * 32; e += kThreads) {
                const int row = e / (KB * 32), col = e % (KB * 32);
                float v = 0.0f;
                if (row < chunk.z && col < a.rank) {
                    const float* h = a.h + (static_cast<int64_t>(chunk.y) + row) * R + i * a.rank + col;
                    for (int q = 0; q < n_slices; q++) v += h[static_cast<int64_t>(q) * p.n_tokens * R];
                    v *= s;
                }
                // to the sum of two bf16 numbers (2^-16 of it)
                const uint16_t h16 = bf16_bits(v);
                hi[row * kStride + col] = h16;
                lo[row * kStride + col] = bf16_bits(v - __uint_as_float(static_cast<uint32_t>(h16) << 16));
            }
            if (threadIdx.x < kChunk)
                rows[threadIdx.x] =
                    static_cast<int32_t>(token_at(a, p, chunk.y + min(static_cast<int>(threadIdx.x), chunk.z - 1)));
            __syncthreads();
        }
        if (n0 >= N) continue;
        uint4 w[4][KB];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int64_t n = n0 + 8 * (g / 2) + 2 * j + g % 2;
#pragma unroll
            for (int k = 0; k < KB; k++) {
                w[j][k] = make_uint4(0, 0, 0, 0);
                if (n < N && k * 32 + 8 * t < a.rank)
                    w[j][k] = __ldg(reinterpret_cast<const uint4*>(
                        a.b[i] + (static_cast<int64_t>(chunk.x) * N + n) * a.rank + k * 32 + 8 * t));
            }
        }
        for (int m = 0; m * 16 < chunk.z; m++) {
            float acc[4][4] = {};
#pragma unroll
            for (int k = 0; k < KB; k++) {
                const int at = (m * 16 + g) * kStride + k * 32 + 8 * t;
                const uint4 h0 = lds128(hi + at), h1 = lds128(hi + at + 8 * kStride);
                const uint4 l0 = lds128(lo + at), l1 = lds128(lo + at + 8 * kStride);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    mma_k32(acc[j], l0, l1, w[j][k]);
                    mma_k32(acc[j], h0, h1, w[j][k]);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int r = m * 16 + h * 8 + g;
                if (r >= chunk.z) continue;
                const int64_t at = rows[r] * N + n0 + 8 * t;
                if (vec) {
                    if (n0 + 8 * t >= N) continue;
                    const uint4 v = *reinterpret_cast<const uint4*>(a.base[i] + at);
                    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
                    uint32_t out[4];
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const float2 f = bf16x2_to_f32x2(in[j]);
                        out[j] = f32x2_to_bf16x2(f.x + acc[j][2 * h], f.y + acc[j][2 * h + 1]);
                    }
                    *reinterpret_cast<uint4*>(a.y[i] + at) = make_uint4(out[0], out[1], out[2], out[3]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        if (n0 + 8 * t + j < N) {
                            const float f = __uint_as_float(static_cast<uint32_t>(a.base[i][at + j]) << 16);
                            a.y[i][at + j] = bf16_bits(f + acc[j / 2][2 * h + j % 2]);
                        }
                }
            }
        }
    }
}

template <int KB>
cudaError_t expand(const LoraArgs& a, int blocks, bool copy, int64_t most, int num_sms, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const int64_t cap = static_cast<int64_t>(num_sms) * 2;
    const cudaLaunchConfig_t cfg =
        pdl_config(dim3(static_cast<unsigned>(most < cap ? most : cap)), kThreads, stream, &attr);
    return cudaLaunchKernelEx(&cfg, expand_kernel<KB>, a, blocks, copy);
}

}  // namespace

int64_t lora_plan_bytes(int64_t T, int64_t adapters) {
    return (kHeader + 4 * max_chunks(T, adapters) + T) * static_cast<int64_t>(sizeof(int32_t));
}

int64_t lora_workspace_bytes(int64_t T, int64_t adapters, int64_t rank, int64_t count) {
    (void)adapters;
    // tokens * slices: at most kMaxSlices each, and a chunk's 64 tokens kSliceUnits times in all
    int64_t rows = T > kChunk * kSliceUnits ? T : int64_t{kChunk} * kSliceUnits;
    if (rows > T * kMaxSlices) rows = T * kMaxSlices;
    return rows * rank * count * static_cast<int64_t>(sizeof(float));
}

cudaError_t launch_lora_plan(const int32_t* ids, const int32_t* sequences, int64_t S, int64_t T, int64_t adapters,
                             void* plan, cudaStream_t stream) {
    static std::once_flag once[64];
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    std::call_once(once[device & 63], [&] {
        e = cudaFuncSetAttribute(lora_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 2 * (kLoraMaxAdapters + 1) * static_cast<int>(sizeof(int32_t)));
    });
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    const int threads = T <= 256 && adapters < 256 ? 256 : 1024;
    cudaLaunchConfig_t cfg = pdl_config(dim3(1), threads, stream, &attr);
    cfg.dynamicSmemBytes = 2 * (adapters + 1) * sizeof(int32_t);
    return cudaLaunchKernelEx(&cfg, lora_plan_kernel, ids, sequences, S, T, static_cast<int>(adapters),
                              static_cast<int32_t*>(plan));
}

cudaError_t launch_lora(const LoraArgs& a, int num_sms, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const int64_t chunks = max_chunks(a.T, a.adapters), cap = static_cast<int64_t>(num_sms) * 2;
    int blocks = 0;
    bool copy = false;
    for (int i = 0; i < a.count; i++) {
        blocks += static_cast<int>((a.N[i] + 255) / 256);
        copy |= a.base[i] != a.y[i];
    }
    const int64_t groups = (a.count * a.rank / 8 + kShrinkTiles - 1) / kShrinkTiles;
    const int64_t units = chunks * groups * kMaxSlices;
    if (units > 0) {
        const cudaLaunchConfig_t cfg =
            pdl_config(dim3(static_cast<unsigned>(units < cap ? units : cap)), kThreads, stream, &attr);
        const cudaError_t e = cudaLaunchKernelEx(&cfg, shrink_kernel, a);
        if (e != cudaSuccess) return e;
    }
    const int64_t most = (chunks + (copy ? (a.T + kChunk - 1) / kChunk : 0)) * blocks;
    if (most == 0) return cudaSuccess;  // no adapters, and in place
    if (a.rank <= 32) return expand<1>(a, blocks, copy, most, num_sms, stream);
    if (a.rank <= 64) return expand<2>(a, blocks, copy, most, num_sms, stream);
    return expand<4>(a, blocks, copy, most, num_sms, stream);
}

cudaError_t read_and_clear_lora_error(int* code) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_lora_error, sizeof(int));
    if (e != cudaSuccess) return e;
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_lora_error, &zero, sizeof(int));
    *code = v;
    return e;
}

}  // namespace nf4
