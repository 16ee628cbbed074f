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
// A counting sort in one CTA that keeps the tokens of an adapter in order: every warp counts a run of the tokens, list by
// list (a list: the tokens of one adapter, or of none); sums over the lists and, inside a list, over the warps give
// each warp the places of its tokens, and it walks its run again.  With many lists fewer warps share the work, as
// their counts have to fit in shared memory.
constexpr int kPlanWarps = 32;
constexpr int kPlanCounts = 200 * 1024 / 4 - 2 * (static_cast<int>(kLoraMaxAdapters) + 1);

__host__ __device__ inline int plan_warps(int64_t T, int64_t adapters) {
    const int64_t room = kPlanCounts / (adapters + 1), need = (T + 31) / 32;
    const int64_t n = room < need ? room : need;
    return static_cast<int>(n < 1 ? 1 : n < kPlanWarps ? n : kPlanWarps);
}

__global__ void __launch_bounds__(1024) lora_plan_kernel(const int32_t* __restrict__ ids,
                                                         const int32_t* __restrict__ sequences, int64_t S, int64_t T,
                                                         int adapters, int32_t* __restrict__ plan, int warps) {
    extern __shared__ int32_t first_of[];  // [adapters + 1] tokens before a list; the same of chunks; counts
    const int lists = adapters + 1;
    int32_t* chunk_at = first_of + lists;
    int32_t* counts = chunk_at + lists;  // [warps][lists]
    __shared__ int32_t part[2][32];
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < warps * lists; i += blockDim.x) counts[i] = 0;
    __syncthreads();
    pdl_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    bool bad = false;
    // the list that token t belongs to; -1 past the end
    auto list_of = [&](int64_t t) {
        if (t >= T) return -1;
        int64_t row = t;
        if (sequences) {
            row = sequences[t];
            if (row < 0 || row >= S) {
                bad |= row >= S;
                return adapters;
            }
        }
        const int32_t id = ids[row];
        bad |= id >= adapters;
        return id < 0 || id >= adapters ? adapters : id;
    };
    // a run of whole warps' widths each
    const int64_t steps = (T + 31) / 32, run0 = warp < warps ? steps * warp / warps : 0;
    const int64_t run1 = warp < warps ? steps * (warp + 1) / warps : 0;
    constexpr int kAhead = 8;  // loads in flight
    int32_t* own = counts + warp * lists;
    auto walk = [&](auto what) {
        for (int64_t i = run0; i < run1; i += kAhead) {
            int list[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; j++) list[j] = i + j < run1 ? list_of((i + j) * 32 + lane) : -1;
#pragma unroll
            for (int j = 0; j < kAhead; j++) {
                if (i + j >= run1) break;
                const uint32_t same = __match_any_sync(0xFFFFFFFFu, list[j]);
                what((i + j) * 32 + lane, list[j], same);
                __syncwarp();
            }
        }
    };
    walk([&](int64_t, int list, uint32_t same) {
        if (list >= 0 && lane == __ffs(same) - 1) own[list] += __popc(same);
    });
    __syncthreads();
    // each thread a run of lists: what the warps before a warp have, the list's tokens; sums over the lists
    const int per = (lists + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
    const int a0 = min(lists, static_cast<int>(threadIdx.x) * per), a1 = min(lists, a0 + per);
    int32_t n = 0, c = 0;
    for (int a = a0; a < a1; a++) {
        int32_t all = 0;
        for (int w = 0; w < warps; w++) {
            const int32_t of_warp = counts[w * lists + a];
            counts[w * lists + a] = all;
            all += of_warp;
        }
        first_of[a] = all;
        n += all;
        c += a < adapters ? (all + kChunk - 1) / kChunk : 0;
    }
    int32_t sn = n, sc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t un = __shfl_up_sync(0xFFFFFFFFu, sn, o), uc = __shfl_up_sync(0xFFFFFFFFu, sc, o);
        if (lane >= o) sn += un, sc += uc;
    }
    if (lane == 31) part[0][warp] = sn, part[1][warp] = sc;
    __syncthreads();
    int32_t bn = sn - n, bc = sc - c, chunks = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x) / 32; w++) {
        if (w < warp) bn += part[0][w], bc += part[1][w];
        chunks += part[1][w];
    }
    for (int a = a0; a < a1; a++) {
        const int32_t tokens = first_of[a];
        first_of[a] = bn;
        chunk_at[a] = bc;
        for (int w = 0; w < warps; w++) counts[w * lists + a] += bn;
        bn += tokens;
        bc += a < adapters ? (tokens + kChunk - 1) / kChunk : 0;
    }
    __syncthreads();
    int4* out = reinterpret_cast<int4*>(plan + kHeader);
    int32_t* order = plan + kHeader + 4 * max_chunks(T, adapters);
    for (int i = threadIdx.x; i < chunks; i += blockDim.x) {
        int lo = 0, hi = adapters;  // the last list whose first chunk is at most i (lists without chunks come before)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (chunk_at[mid] <= i)
                lo = mid;
            else
                hi = mid;
        }
        const int32_t first = first_of[lo] + (i - chunk_at[lo]) * kChunk;
        out[i] = make_int4(lo, first, min(kChunk, first_of[lo + 1] - first), 0);
    }
    if (threadIdx.x == 0) {
        reinterpret_cast<int4*>(plan)[0] = make_int4(static_cast<int32_t>(T), adapters, chunks, first_of[adapters]);
        reinterpret_cast<int4*>(plan)[1] = make_int4(0, 0, 0, 0);
    }
    walk([&](int64_t t, int list, uint32_t same) {
        const int leader = __ffs(same) - 1;
        int32_t at = 0;
        if (list >= 0 && lane == leader) {
            at = own[list];
            own[list] = at + __popc(same);
        }
        at = __shfl_sync(0xFFFFFFFFu, at, leader) + __popc(same & ((1u << lane) - 1));
        if (list >= 0) order[at] = static_cast<int32_t>(t);
    });
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
// Slices of K (in units of 64): as many as fill the GPU, each with at least one step of 32 for every warp.
__device__ __forceinline__ int slices(const LoraArgs& a, const Plan& p) {
    const int steps = static_cast<int>(a.K / 32 / (kThreads / 32));
    return max(1, min(min(kMaxSlices, steps), kSliceUnits / max(1, p.n_chunks)));
}

// The sums of a unit (a chunk, a slice of K, some rank columns): parts [part][64][cols] in shared memory, added in
// order, go to the workspace.  All threads have written theirs.
__device__ __forceinline__ void write_sums(const LoraArgs& a, const Plan& p, const int4& chunk, int slice, int tile0,
                                           int tiles, const float* sums, int parts, int stride, int part_stride) {
    const int R = a.count * a.rank, cols = tiles * 8;
    float* out = a.h + (static_cast<int64_t>(slice) * p.n_tokens + chunk.y) * R + tile0 * 8;
    for (int e = threadIdx.x; e < chunk.z * cols / 4; e += kThreads) {
        const int row = e / (cols / 4), col = e % (cols / 4) * 4;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int q = 0; q < parts; q++) {
            const float4 u = *reinterpret_cast<const float4*>(sums + q * part_stride + row * stride + col);
            v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
        *reinterpret_cast<float4*>(out + static_cast<int64_t>(row) * R + col) = v;
    }
}

// The address of row `row` (0 .. 7 of a tile) of rank column tile `tile` of all projections.
__device__ __forceinline__ const uint16_t* column_of(const LoraArgs& a, int adapter, int tile, int row) {
    const int per = a.rank / 8, i = tile / per;
    return a.a[i] + (static_cast<int64_t>(adapter) * a.rank + (tile - i * per) * 8 + row) * a.K;
}

// A unit with few tokens: bound by the latency of reading A, so U steps of a warp are on their way at once, and the
// operands go straight to registers.  MT tiles of 16 tokens, up to NT * 8 columns.
template <int MT, int NT, int U>
__device__ __forceinline__ void shrink_few(const LoraArgs& a, const Plan& p, const int4& chunk, int slice, int n_slices,
                                           int tile0, float* sums) {
    constexpr int kStride = NT * 8 + 4;  // (a warp's 64-bit stores: 8 rows, 4 columns apart)
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int tiles = min(NT, a.count * a.rank / 8 - tile0);
    const uint16_t* xp[MT][2];
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
        for (int h = 0; h < 2; h++)  // a row past the chunk's end repeats the last
            xp[m][h] = a.x + token_at(a, p, chunk.y + min(m * 16 + h * 8 + g, chunk.z - 1)) * a.K + 8 * t;
    const uint16_t* wp[NT];
#pragma unroll
    for (int j = 0; j < NT; j++) wp[j] = column_of(a, chunk.x, tile0 + min(j, tiles - 1), g) + 8 * t;
    float acc[MT][NT][4] = {};
    const int64_t steps = a.K / 64, k0 = 2 * (steps * slice / n_slices), k1 = 2 * (steps * (slice + 1) / n_slices);
    constexpr int kWarps = kThreads / 32;
    for (int64_t k = k0 + warp; k < k1; k += kWarps * U) {
        uint4 x[U][MT][2], w[U][NT];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const bool in = k + u * kWarps < k1;
            const int64_t at = 32 * (k + u * kWarps);
#pragma unroll
            for (int j = 0; j < NT; j++) {
                w[u][j] = make_uint4(0, 0, 0, 0);
                if (in && j < tiles) w[u][j] = __ldg(reinterpret_cast<const uint4*>(wp[j] + at));
            }
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    x[u][m][h] = make_uint4(0, 0, 0, 0);
                    if (in) x[u][m][h] = *reinterpret_cast<const uint4*>(xp[m][h] + at);
                }
        }
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int j = 0; j < NT; j++)
                if (j < tiles)
#pragma unroll
                    for (int m = 0; m < MT; m++) mma_k32(acc[m][j], x[u][m][0], x[u][m][1], w[u][j]);
    }
    // four of the warps write, the others add, then all add the four
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
    write_sums(a, p, chunk, slice, tile0, tiles, sums, 4, kStride, MT * 16 * kStride);
}

// A unit with many tokens, up to 64 by 128 columns: bound by the bytes of x, so x is read once for all columns.  Stages
// of 128 k, of x and of A, are copied into shared memory while the last one is multiplied; a row is 16 pieces of 16
// bytes, and the odd rows' pieces change places by four, so that the eight lanes of a 128-bit read (two rows) hit
// all banks.  Eight warps: two halves of the tokens, and column groups of up to four tiles; with few columns the
// warps of a half share out the stage's k instead.
constexpr int kStageK = 128, kStageRows = kChunk + 128, kStageBytes = kStageRows * kStageK * 2;

__device__ __forceinline__ uint32_t piece_at(int row, int piece) {
    return row * (kStageK * 2) + ((piece ^ ((row & 1) << 2)) << 4);
}

__device__ __forceinline__ void shrink_many(const LoraArgs& a, const Plan& p, const int4& chunk, int slice, int n_slices,
                                            int tile0, uint8_t* ring) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int tiles = min(16, a.count * a.rank / 8 - tile0);
    const int col_groups = tiles > 8 ? 4 : tiles > 4 ? 2 : 1, k_groups = 4 / col_groups;
    const int half = warp % 2, col_group = warp / 2 % col_groups, k_group = warp / 2 / col_groups;
    const int each = (tiles + col_groups - 1) / col_groups, first_tile = col_group * each;
    const int own_tiles = max(0, min(each, tiles - first_tile));
    const int64_t steps = a.K / 64, k0 = 64 * (steps * slice / n_slices), k1 = 64 * (steps * (slice + 1) / n_slices);
    // what this thread copies: piece `piece` of rows row0, row0 + 16, ...
    const int piece = threadIdx.x % 16, row0 = threadIdx.x / 16;
    const uint16_t* src[12];
#pragma unroll
    for (int i = 0; i < 4; i++)
        src[i] = a.x + token_at(a, p, chunk.y + min(row0 + 16 * i, chunk.z - 1)) * a.K + piece * 8;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int col = min(row0 + 16 * i, tiles * 8 - 1);
        src[4 + i] = column_of(a, chunk.x, tile0 + col / 8, col % 8) + piece * 8;
    }
    auto copy = [&](int64_t k, uint8_t* stage) {
        const uint32_t bytes = k + piece * 8 < k1 ? 16u : 0u;  // zeros past the slice
        const int64_t at = bytes ? k : 0;
#pragma unroll
        for (int i = 0; i < 12; i++) {
            const int row = row0 + 16 * i;  // rows of x, then of A
            if (i >= 4 && row - kChunk >= tiles * 8) continue;
            cp_async16(stage + piece_at(row, piece), src[i] + at, bytes);
        }
        cp_async_commit();
    };
    float acc[2][4][4] = {};
    __syncthreads();  // the last unit's sums are read
    copy(k0, ring);
    int at = 0;
    for (int64_t k = k0; k < k1; k += kStageK, at ^= 1) {
        if (k + kStageK < k1)
            copy(k + kStageK, ring + (at ^ 1) * kStageBytes);
        else
            cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();
        const uint8_t* stage = ring + at * kStageBytes;
#pragma unroll
        for (int s = 0; s < kStageK / 32; s++) {
            if (s % k_groups != k_group) continue;
            uint4 x[2][2];
#pragma unroll
            for (int m = 0; m < 2; m++)
#pragma unroll
                for (int h = 0; h < 2; h++)
                    x[m][h] = lds128(stage + piece_at(half * 32 + m * 16 + h * 8 + g, 4 * s + t));
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (j >= own_tiles) continue;
                const uint4 w = lds128(stage + piece_at(kChunk + (first_tile + j) * 8 + g, 4 * s + t));
#pragma unroll
                for (int m = 0; m < 2; m++) mma_k32(acc[m][j], x[m][0], x[m][1], w);
            }
        }
        __syncthreads();
    }
    float* sums = reinterpret_cast<float*>(ring);
    const int stride = tiles * 8 + 4, part = kChunk * stride;
#pragma unroll
    for (int m = 0; m < 2; m++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if (j >= own_tiles) continue;
#pragma unroll
            for (int h = 0; h < 2; h++)
                *reinterpret_cast<float2*>(sums + k_group * part + (half * 32 + m * 16 + h * 8 + g) * stride +
                                           (first_tile + j) * 8 + 2 * t) =
                    make_float2(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
        }
    __syncthreads();
    write_sums(a, p, chunk, slice, tile0, tiles, sums, k_groups, stride, part);
}

constexpr int kFewTiles = 4;     // rank columns of a unit with few tokens, in eights
constexpr int kFewTokens = 32;

__global__ void __launch_bounds__(kThreads, 2) shrink_kernel(const LoraArgs a) {
    extern __shared__ __align__(16) uint8_t ring[];
    pdl_launch_dependents();
    pdl_wait();
    Plan p;
    if (!read_plan(a, &p)) return;
    const int n_slices = slices(a, p), tiles = a.count * a.rank / 8;
    const int64_t pairs = static_cast<int64_t>(p.n_chunks) * n_slices;
    const int64_t units = pairs * ((tiles + kFewTiles - 1) / kFewTiles);
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t cs = u % pairs;
        const int group = static_cast<int>(u / pairs);
        const int4 chunk = p.chunks[cs / n_slices];
        if (!chunk_ok(a, p, chunk)) continue;
        const int slice = static_cast<int>(cs % n_slices);
        if (chunk.z > kFewTokens) {
            if (group * 16 < tiles) shrink_many(a, p, chunk, slice, n_slices, group * 16, ring);
        } else if (chunk.z > 16) {
            shrink_few<2, kFewTiles, 2>(a, p, chunk, slice, n_slices, group * kFewTiles, reinterpret_cast<float*>(ring));
        } else {
            shrink_few<1, kFewTiles, 3>(a, p, chunk, slice, n_slices, group * kFewTiles, reinterpret_cast<float*>(ring));
        }
    }
}

// Where a lane's results stand: column g of a warp's tile j is row 8 (g / 2) + 2 j + g % 2 of 32, so that its eight
// results for a token are eight consecutive values of y.
// W: 16-byte words of a lane that hold a row of B; 0: half of one (rank 16 or less), and a step of 16 instead of two.
template <int W>
struct Weights {
    uint4 w[4][W];
    __device__ __forceinline__ void load(const uint16_t* b, int64_t n0, int64_t N, int rank, int g, int t) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int64_t n = n0 + 8 * (g / 2) + 2 * j + g % 2;
#pragma unroll
            for (int k = 0; k < W; k++) {
                w[j][k] = make_uint4(0, 0, 0, 0);
                if (n < N && k * 32 + 8 * t < rank)
                    w[j][k] = __ldg(reinterpret_cast<const uint4*>(b + n * rank + k * 32 + 8 * t));
            }
        }
    }
    __device__ __forceinline__ void multiply(float (&acc)[4][4], const uint16_t* hi, const uint16_t* lo, int row, int stride,
                                             int t) const {
#pragma unroll
        for (int k = 0; k < W; k++) {
            const int at = row * stride + k * 32 + 8 * t;
            const uint4 l0 = lds128(lo + at), l1 = lds128(lo + at + 8 * stride);
            const uint4 h0 = lds128(hi + at), h1 = lds128(hi + at + 8 * stride);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                mma_k32(acc[j], l0, l1, w[j][k]);
                mma_k32(acc[j], h0, h1, w[j][k]);
            }
        }
    }
};
template <>
struct Weights<0> {
    uint2 w[4];
    __device__ __forceinline__ void load(const uint16_t* b, int64_t n0, int64_t N, int rank, int g, int t) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int64_t n = n0 + 8 * (g / 2) + 2 * j + g % 2;
            w[j] = make_uint2(0, 0);
            if (n < N && 4 * t < rank) w[j] = __ldg(reinterpret_cast<const uint2*>(b + n * rank + 4 * t));
        }
    }
    __device__ __forceinline__ void multiply(float (&acc)[4][4], const uint16_t* hi, const uint16_t* lo, int row, int stride,
                                             int t) const {
        const int at = row * stride + 4 * t;
        const uint2 l0 = *reinterpret_cast<const uint2*>(lo + at), l1 = *reinterpret_cast<const uint2*>(lo + at + 8 * stride);
        const uint2 h0 = *reinterpret_cast<const uint2*>(hi + at), h1 = *reinterpret_cast<const uint2*>(hi + at + 8 * stride);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            mma_bf16(acc[j], l0.x, l1.x, l0.y, l1.y, w[j].x, w[j].y);
            mma_bf16(acc[j], h0.x, h1.x, h0.y, h1.y, w[j].x, w[j].y);
        }
    }
};

// A unit is a chunk and 256 rows of one projection, 32 a warp.  Bound by the bytes of y (many tokens) or of B (few), so
// all that a warp needs is on its way before anything is multiplied: B's rows and the base of D units with few
// tokens, or those of one unit and up to 64 tokens.
template <int W, int D>
__global__ void __launch_bounds__(kThreads, 2) expand_kernel(const LoraArgs a, int blocks, bool copy) {
    constexpr int kCols = W ? W * 32 : 16, kStride = kCols + 8;
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
    int held = -1, batch = 0;  // the chunk and projection in shared memory
    int c = static_cast<int>(u0 / blocks), at_block = static_cast<int>(u0 % blocks);
    for (int64_t u = u0; u < u1; u += batch, at_block += batch) {
        if (at_block >= blocks) at_block -= blocks, c++;  // (a batch ends with its projection)
        int block = at_block, i = 0, last = 0;
        for (; i < a.count; i++) {
            last = static_cast<int>((a.N[i] + 255) / 256);
            if (block < last) break;
            block -= last;
        }
        const int64_t N = a.N[i], n0 = static_cast<int64_t>(block) * 256 + warp * 32;
        const uint16_t* base = a.base[i];
        uint16_t* y = a.y[i];
        const bool vec = N % 8 == 0;
        batch = 1;
        if (c >= p.n_chunks) {
            if (base == y) continue;
            const int first = p.n_tokens + (c - p.n_chunks) * kChunk, n = min(kChunk, static_cast<int>(a.T) - first);
            const int rounds = (n + 7) / 8;  // of eight rows a warp
            batch = static_cast<int>(min(static_cast<int64_t>(min(8 / rounds, last - block)), u1 - u));
            uint4 v[8];
            if (vec) {
#pragma unroll
                for (int q = 0; q < 8; q++) {
                    const int r = q % rounds * 8 + g;
                    const int64_t col = n0 + q / rounds * 256 + 8 * t;
                    if (q < batch * rounds && r < n && col < N)
                        v[q] = *reinterpret_cast<const uint4*>(base + token_at(a, p, first + r) * N + col);
                }
#pragma unroll
                for (int q = 0; q < 8; q++) {
                    const int r = q % rounds * 8 + g;
                    const int64_t col = n0 + q / rounds * 256 + 8 * t;
                    if (q < batch * rounds && r < n && col < N)
                        *reinterpret_cast<uint4*>(y + token_at(a, p, first + r) * N + col) = v[q];
                }
            } else {
                for (int q = 0; q < batch; q++)
                    for (int r = 0; r < n; r++) {
                        const int64_t col = n0 + q * 256 + lane, at = token_at(a, p, first + r) * N + col;
                        if (col < N) y[at] = base[at];
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
            // four columns of a row each, up to 4 at a time; the slices in order
            const int items = (chunk.z + 15) / 16 * 16 * (kCols / 4);
            for (int e0 = threadIdx.x; e0 < items; e0 += 4 * kThreads) {
                float4 v[4];
                int at[4];  // in the chunk's part of a slice
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int e = e0 + j * kThreads, row = e / (kCols / 4), col = e % (kCols / 4) * 4;
                    v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    at[j] = row < chunk.z && col < a.rank ? row * R + i * a.rank + col : -1;
                }
                const float* h = a.h + static_cast<int64_t>(chunk.y) * R;
#pragma unroll 2
                for (int q = 0; q < n_slices; q++, h += static_cast<int64_t>(p.n_tokens) * R)
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        if (at[j] >= 0) {
                            const float4 o = *reinterpret_cast<const float4*>(h + at[j]);
                            v[j].x += o.x, v[j].y += o.y, v[j].z += o.z, v[j].w += o.w;
                        }
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int e = e0 + j * kThreads, row = e / (kCols / 4), col = e % (kCols / 4) * 4;
                    if (e >= items) continue;
                    // to the sum of two bf16 numbers (2^-16 of it)
                    const float f[4] = {v[j].x * s, v[j].y * s, v[j].z * s, v[j].w * s};
                    const uint32_t h01 = f32x2_to_bf16x2(f[0], f[1]), h23 = f32x2_to_bf16x2(f[2], f[3]);
                    const float2 r01 = bf16x2_to_f32x2(h01), r23 = bf16x2_to_f32x2(h23);
                    *reinterpret_cast<uint2*>(hi + row * kStride + col) = make_uint2(h01, h23);
                    *reinterpret_cast<uint2*>(lo + row * kStride + col) = make_uint2(
                        f32x2_to_bf16x2(f[0] - r01.x, f[1] - r01.y), f32x2_to_bf16x2(f[2] - r23.x, f[3] - r23.y));
                }
            }
            if (threadIdx.x < kChunk)
                rows[threadIdx.x] =
                    static_cast<int32_t>(token_at(a, p, chunk.y + min(static_cast<int>(threadIdx.x), chunk.z - 1)));
            __syncthreads();
        }
        const uint16_t* b = a.b[i] + static_cast<int64_t>(chunk.x) * N * a.rank;
        // token r's eight values from column n on: base in, y out
        auto fetch = [&](int r, int64_t n) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (vec && r < chunk.z && n < N) v = *reinterpret_cast<const uint4*>(base + rows[r] * N + n);
            return v;
        };
        auto store = [&](int r, int64_t n, const uint4& v, const float (&acc)[4][4], int h) {
            if (r >= chunk.z) return;
            const int64_t at = rows[r] * N + n;
            if (vec) {
                if (n >= N) return;
                const uint32_t in[4] = {v.x, v.y, v.z, v.w};
                uint32_t out[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const float2 f = bf16x2_to_f32x2(in[j]);
                    out[j] = f32x2_to_bf16x2(f.x + acc[j][2 * h], f.y + acc[j][2 * h + 1]);
                }
                *reinterpret_cast<uint4*>(y + at) = make_uint4(out[0], out[1], out[2], out[3]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (n + j < N)
                        y[at + j] = bf16_bits(__uint_as_float(static_cast<uint32_t>(base[at + j]) << 16) +
                                              acc[j / 2][2 * h + j % 2]);
            }
        };
        if (chunk.z <= 16) {
            batch = static_cast<int>(min(static_cast<int64_t>(min(D, last - block)), u1 - u));
            Weights<W> w[D];
            uint4 in[D][2];
#pragma unroll
            for (int d = 0; d < D; d++) {
                const int64_t n = n0 + 256 * d, edge = d < batch ? N : 0;
                w[d].load(b, n, edge, a.rank, g, t);
                in[d][0] = in[d][1] = make_uint4(0, 0, 0, 0);
                if (d < batch) in[d][0] = fetch(g, n + 8 * t), in[d][1] = fetch(g + 8, n + 8 * t);
            }
#pragma unroll
            for (int d = 0; d < D; d++) {
                if (d >= batch) continue;
                float acc[4][4] = {};
                w[d].multiply(acc, hi, lo, g, kStride, t);
                store(g, n0 + 256 * d + 8 * t, in[d][0], acc, 0);
                store(g + 8, n0 + 256 * d + 8 * t, in[d][1], acc, 1);
            }
        } else if (n0 < N) {
            constexpr int kTiles = W >= 4 ? 2 : 4;  // tiles of 16 tokens whose base is on its way
            Weights<W> w;
            w.load(b, n0, N, a.rank, g, t);
            for (int m0 = 0; m0 * 16 < chunk.z; m0 += kTiles) {
                uint4 in[kTiles][2];
#pragma unroll
                for (int m = 0; m < kTiles; m++)
#pragma unroll
                    for (int h = 0; h < 2; h++) in[m][h] = fetch((m0 + m) * 16 + h * 8 + g, n0 + 8 * t);
#pragma unroll
                for (int m = 0; m < kTiles; m++) {
                    if ((m0 + m) * 16 >= chunk.z) continue;
                    float acc[4][4] = {};
                    w.multiply(acc, hi, lo, (m0 + m) * 16 + g, kStride, t);
#pragma unroll
                    for (int h = 0; h < 2; h++) store((m0 + m) * 16 + h * 8 + g, n0 + 8 * t, in[m][h], acc, h);
                }
            }
        }
    }
}

template <int W, int D>
cudaError_t expand(const LoraArgs& a, int blocks, bool copy, int64_t most, int num_sms, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const int64_t cap = static_cast<int64_t>(num_sms) * 2;
    const cudaLaunchConfig_t cfg =
        pdl_config(dim3(static_cast<unsigned>(most < cap ? most : cap)), kThreads, stream, &attr);
    return cudaLaunchKernelEx(&cfg, expand_kernel<W, D>, a, blocks, copy);
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
        e = cudaFuncSetAttribute(lora_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    const int warps = plan_warps(T, adapters);
    const int threads = warps <= 8 && adapters < 256 ? 256 : 1024;
    cudaLaunchConfig_t cfg = pdl_config(dim3(1), threads, stream, &attr);
    cfg.dynamicSmemBytes = (2 + warps) * (adapters + 1) * sizeof(int32_t);
    return cudaLaunchKernelEx(&cfg, lora_plan_kernel, ids, sequences, S, T, static_cast<int>(adapters),
                              static_cast<int32_t*>(plan), warps);
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
    const int64_t groups = (a.count * a.rank / 8 + kFewTiles - 1) / kFewTiles;
    const int64_t units = chunks * groups * kMaxSlices;
    if (units > 0) {
        static std::once_flag once[64];
        int device = 0;
        cudaError_t e = cudaGetDevice(&device);
        if (e != cudaSuccess) return e;
        std::call_once(once[device & 63], [&] {
            e = cudaFuncSetAttribute(shrink_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * kStageBytes);
        });
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg =
            pdl_config(dim3(static_cast<unsigned>(units < cap ? units : cap)), kThreads, stream, &attr);
        cfg.dynamicSmemBytes = 2 * kStageBytes;
        e = cudaLaunchKernelEx(&cfg, shrink_kernel, a);
        if (e != cudaSuccess) return e;
    }
    const int64_t most = (chunks + (copy ? (a.T + kChunk - 1) / kChunk : 0)) * blocks;
    if (most == 0) return cudaSuccess;  // no adapters, and in place
    if (a.rank <= 16) return expand<0, 4>(a, blocks, copy, most, num_sms, stream);
    if (a.rank <= 32) return expand<1, 3>(a, blocks, copy, most, num_sms, stream);
    if (a.rank <= 64) return expand<2, 2>(a, blocks, copy, most, num_sms, stream);
    return expand<4, 1>(a, blocks, copy, most, num_sms, stream);
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
