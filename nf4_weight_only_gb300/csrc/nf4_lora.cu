// Low-rank adapters of many requests beside projections that share their input:
//   y[t] = base[t] + s[a] * B[a] (A[a] x[t]),  a the adapter of token t.
//
// Tokens are first listed adapter by adapter (lora_plan_kernel, once for all calls of a step), in chunks of up to
// 64 tokens of one adapter, so that an adapter's matrices are read once a chunk.  Chunks of few tokens, up to 16, stand
// behind the others: their products are bound by reading A and B, the others' by x and y.  Two kernels follow:
//   shrink  h = A x for a chunk, the rank columns of all projections side by side; the long axis K is split over
//           warps and CTAs, and a slice's sums go to the workspace in fp32
//   expand  adds the slices in order, scales, and adds B h to the base
// Both use mma.sync m16n8k16 with tokens as the 16 rows and weights as the 8 columns.  A product's k axis may
// be permuted at will if both operands are permuted alike: a lane takes eight consecutive k (16 bytes) of its
// row or column, which is two k steps of the instruction, and needs neither shared memory nor shuffles.
//
// Times with the plan, calls queued, and those of the bytes alone at the measured copy rate (us): q|k|v of one token, rank
// 16: 11.0 / 0.04; gate|up of 64 tokens with 48 adapters: 28.9 / 9.9; q|k|v of 256 tokens, rank 64: 41.5 / 11.8; down of
// 5, rank 128: 21.5 / 6.4; o of 8191, rank 16: 75 / 37; gate|up of 4099, rank 64: 194 / 91.  Few tokens are bound by three
// launches and the chains of loads inside them, many by the latency of the base's loads at 16 warps an SM (second kernel:
// issue slots 34-36%, L1 53-56%, tensor pipe 11-33%, long-scoreboard stalls 3.9 an issue).
#include <mutex>

#include "nf4_kv.cuh"
#include "nf4_lora_index.h"

namespace nf4 {
namespace {

constexpr int kChunk = 64;      // tokens of a chunk at most
constexpr int kFew = 16;        // of a chunk of few (8: q|k|v of 256 tokens 42 -> 45 us, o of 8191 76 -> 74)
constexpr int kHeader = 8;      // int32 before the chunks: T, adapters, chunks of many, of few, tokens with an adapter
constexpr int kThreads = 256;
// Of the first product: two CTAs for each of 152 SMs.  (152: down of 5 tokens 23 -> 26 us, o of 8191 85 -> 95, q|k|v of 256
// 43 -> 41; 608: 26, 87 and 44.)
constexpr int kUnits = 304;
constexpr int kMaxSlices = 32;

__device__ int g_lora_error;  // 46: an adapter or a row outside its list; 47: a plan of other sizes

__host__ __device__ inline int64_t max_many(int64_t T) { return T / (kFew + 1); }
__host__ __device__ inline int64_t max_few(int64_t T, int64_t adapters) { return adapters < T ? adapters : T; }
__host__ __device__ inline int64_t max_chunks(int64_t T, int64_t adapters) {
    const int64_t n = max_many(T) + max_few(T, adapters);
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
constexpr int kPlanCounts = 200 * 1024 / 4 - 3 * (static_cast<int>(kLoraMaxAdapters) + 1);

__host__ __device__ inline int plan_warps(int64_t T, int64_t adapters) {
    const int64_t room = kPlanCounts / (adapters + 1), need = (T + 31) / 32;
    const int64_t n = room < need ? room : need;
    return static_cast<int>(n < 1 ? 1 : n < kPlanWarps ? n : kPlanWarps);
}

__global__ void __launch_bounds__(1024) lora_plan_kernel(const int32_t* __restrict__ ids,
                                                         const int32_t* __restrict__ sequences, int64_t S, int64_t T,
                                                         int adapters, int32_t* __restrict__ plan, int warps) {
    extern __shared__ int32_t first_of[];  // [adapters + 1] tokens before a list; chunks of many, of few; counts
    const int lists = adapters + 1;
    int32_t *many_at = first_of + lists, *few_at = many_at + lists;
    int32_t* counts = few_at + lists;  // [warps][lists]
    __shared__ int32_t part[3][32];
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
    constexpr int kAhead = 8;  // steps whose loads are in flight; a run of no more keeps what it found
    int32_t* own = counts + warp * lists;
    int list[kAhead];
    uint32_t same[kAhead];  // the lanes with the same list
    auto walk = [&](bool again, auto what) {
#pragma unroll 1
        for (int64_t i = run0; i < run1; i += kAhead) {
            if (!again || run1 - run0 > kAhead) {
#pragma unroll
                for (int j = 0; j < kAhead; j++) list[j] = i + j < run1 ? list_of((i + j) * 32 + lane) : -1;
#pragma unroll
                for (int j = 0; j < kAhead; j++) same[j] = __match_any_sync(0xFFFFFFFFu, list[j]);
            }
#pragma unroll
            for (int j = 0; j < kAhead; j++) {
                if (i + j < run1) what((i + j) * 32 + lane, list[j], same[j]);
                __syncwarp();
            }
        }
    };
    walk(false, [&](int64_t, int in, uint32_t with) {
        if (in >= 0 && lane == __ffs(with) - 1) own[in] += __popc(with);
    });
    __syncthreads();
    // what the warps before a warp have of a list, and the list's tokens: a warp a list, or, for few warps, a thread
    if (warps > 8) {
        for (int a = warp; a < lists; a += static_cast<int>(blockDim.x) / 32) {
            const int32_t of_warp = lane < warps ? counts[lane * lists + a] : 0;
            int32_t upto = of_warp;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                if (lane >= o) upto += v;
            }
            if (lane < warps) counts[lane * lists + a] = upto - of_warp;
            if (lane == 31) first_of[a] = upto;
        }
    } else {
        for (int a = threadIdx.x; a < lists; a += blockDim.x) {
            int32_t all = 0;
            for (int w = 0; w < warps; w++) {
                const int32_t of_warp = counts[w * lists + a];
                counts[w * lists + a] = all;
                all += of_warp;
            }
            first_of[a] = all;
        }
    }
    __syncthreads();
    // sums over the lists, a run of them a thread
    const int per = (lists + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
    const int a0 = min(lists, static_cast<int>(threadIdx.x) * per), a1 = min(lists, a0 + per);
    auto many_of = [&](int a, int32_t tokens) {
        return a < adapters ? tokens / kChunk + (tokens % kChunk > kFew ? 1 : 0) : 0;
    };
    auto few_of = [&](int a, int32_t tokens) {
        return a < adapters && tokens % kChunk != 0 && tokens % kChunk <= kFew ? 1 : 0;
    };
    int32_t n[3] = {0, 0, 0}, upto[3];  // tokens, chunks of many, chunks of few
    for (int a = a0; a < a1; a++) {
        const int32_t all = first_of[a];
        n[0] += all, n[1] += many_of(a, all), n[2] += few_of(a, all);
    }
#pragma unroll
    for (int i = 0; i < 3; i++) {
        upto[i] = n[i];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t v = __shfl_up_sync(0xFFFFFFFFu, upto[i], o);
            if (lane >= o) upto[i] += v;
        }
        if (lane == 31) part[i][warp] = upto[i];
        upto[i] -= n[i];
    }
    __syncthreads();
    int32_t many = 0, few = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x) / 32; w++) {
        if (w < warp) upto[0] += part[0][w], upto[1] += part[1][w], upto[2] += part[2][w];
        many += part[1][w], few += part[2][w];
    }
    int4* out = reinterpret_cast<int4*>(plan + kHeader);
    int32_t* order = plan + kHeader + 4 * max_chunks(T, adapters);
    for (int a = a0; a < a1; a++) {
        const int32_t tokens = first_of[a];
        first_of[a] = upto[0];
        many_at[a] = upto[1];
        if (few_of(a, tokens))
            out[many + upto[2]] = make_int4(a, upto[0] + tokens / kChunk * kChunk, tokens % kChunk, 0);
        upto[0] += tokens, upto[1] += many_of(a, tokens), upto[2] += few_of(a, tokens);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < many; i += blockDim.x) {
        int lo = 0, hi = adapters;  // the last list whose first chunk is at most i (lists without chunks come before)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (many_at[mid] <= i)
                lo = mid;
            else
                hi = mid;
        }
        const int32_t first = first_of[lo] + (i - many_at[lo]) * kChunk;
        out[i] = make_int4(lo, first, min(kChunk, first_of[lo + 1] - first), 0);
    }
    if (threadIdx.x == 0) {
        reinterpret_cast<int4*>(plan)[0] = make_int4(static_cast<int32_t>(T), adapters, many, few);
        reinterpret_cast<int4*>(plan)[1] = make_int4(first_of[adapters], 0, 0, 0);
    }
    walk(true, [&](int64_t t, int in, uint32_t with) {
        const int leader = __ffs(with) - 1;
        int32_t at = 0;
        if (in >= 0 && lane == leader) {
            at = own[in];
            own[in] = at + __popc(with);
            at += first_of[in];
        }
        at = __shfl_sync(0xFFFFFFFFu, at, leader) + __popc(with & ((1u << lane) - 1));
        if (in >= 0) order[at] = static_cast<int32_t>(t);
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
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// Two k steps: rows g and g + 8 of 16 tokens against column g of 8 weights, eight k a lane.
__device__ __forceinline__ void mma_k32(float (&d)[4], const uint4& x0, const uint4& x1, const uint4& w) {
    mma_bf16(d, x0.x, x1.x, x0.y, x1.y, w.x, w.y);
    mma_bf16(d, x0.z, x1.z, x0.w, x1.w, w.z, w.w);
}

// The plan as both kernels read it.
struct Plan {
    const int4* chunks;  // adapter, first place in `order`, tokens
    const int32_t* order;
    int n_many, n_few, n_tokens;
};
// False (and 47 recorded) if the plan was made for other sizes.
__device__ __forceinline__ bool read_plan(const LoraArgs& a, Plan* p) {
    const int4 h = reinterpret_cast<const int4*>(a.plan)[0];
    p->chunks = reinterpret_cast<const int4*>(a.plan + kHeader);
    p->order = a.plan + kHeader + 4 * max_chunks(a.T, a.adapters);
    p->n_many = h.z, p->n_few = h.w, p->n_tokens = a.plan[4];
    if (h.x != a.T || h.y != a.adapters || h.z < 0 || h.z > max_many(a.T) || h.w < 0 || h.w > max_few(a.T, a.adapters) ||
        h.z + h.w > max_chunks(a.T, a.adapters) || p->n_tokens < 0 || p->n_tokens > a.T) {
        if (threadIdx.x == 0) atomicCAS(&g_lora_error, 0, 47);
        return false;
    }
    return true;
}
__device__ __forceinline__ bool chunk_ok(const LoraArgs& a, const Plan& p, const int4& c, int most) {
    return chunk_in_lists(c.x, c.y, c.z, most, a.adapters, p.n_tokens);
}
__device__ __forceinline__ int64_t token_at(const LoraArgs& a, const Plan& p, int at) {
    return min(static_cast<uint32_t>(p.order[at]), static_cast<uint32_t>(a.T - 1));
}
// Rank columns of a unit with few tokens, in eights (4 make fewer, longer units: down of 5 tokens 22 -> 23 us, gate|up of 64
// 29 -> 30), and with many (all that the stage and the accumulators hold, so that x is read once).
constexpr int kFewTiles = 2, kManyTiles = 16;

// How the first product is cut: rank-column groups, slices of K (in units of 64), and the rows of the workspace that a
// chunk's slice takes (64 or 16, the chunks of many first).  As many slices as fill the GPU in one round, each with at
// least one step of 32 for every warp; but with many tokens, whose sums the second product waits for, no more than eight
// (q|k|v of 256 tokens: 43.3 us; 44.6 with four, 46.6 with sixteen) or slices of 512 (649 tokens, K 16064, rank 64: 66 us
// with eight, 56 with 23).
struct Cut {
    int many_groups, few_groups, many_slices, few_slices;
    __device__ __forceinline__ int64_t many_row(int chunk, int slice) const {
        return (static_cast<int64_t>(chunk) * many_slices + slice) * kChunk;
    }
    __device__ __forceinline__ int64_t few_row(int many, int chunk, int slice) const {
        return many_row(many, 0) + (static_cast<int64_t>(chunk) * few_slices + slice) * kFew;
    }
};
__device__ __forceinline__ Cut cut_of(const LoraArgs& a, const Plan& p) {
    const int tiles = a.count * a.rank / 8, K = static_cast<int>(a.K), most = max(1, min(kMaxSlices, K / 256));
    Cut c;
    c.many_groups = (tiles + kManyTiles - 1) / kManyTiles;
    c.few_groups = (tiles + kFewTiles - 1) / kFewTiles;
    const int many = max(1, p.n_many * c.many_groups), few = max(1, p.n_few * c.few_groups);
    c.many_slices = max(1, min(min(most, max(8, K / 512)), kUnits / many));
    c.few_slices = max(1, min(most, kUnits / few));
    return c;
}

// The sums of a unit (a chunk, a slice of K, some rank columns): parts [part][64][cols] in shared memory, added in
// order, go to the workspace.  All threads have written theirs.
__device__ __forceinline__ void write_sums(const LoraArgs& a, int64_t row0, int rows, int tile0, int tiles,
                                           const float* sums, int parts, int stride, int part_stride) {
    const int R = a.count * a.rank, cols = tiles * 8;
    float* out = a.h + row0 * R + tile0 * 8;
    for (int e = threadIdx.x; e < rows * cols / 4; e += kThreads) {
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

// A unit with few tokens, up to ROWS (8 or 16), and up to NT * 8 columns: bound by the latency of reading A, so U steps of
// a warp are on their way at once, and the operands go straight to registers.
template <int ROWS, int NT, int U>
__device__ __forceinline__ void shrink_few(const LoraArgs& a, const Plan& p, const int4& chunk, int slice, int n_slices,
                                           int tile0, int64_t row0, float* sums) {
    constexpr int kStride = NT * 8 + 4;  // (a warp's 64-bit stores: 8 rows, 4 columns apart)
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int tiles = min(NT, a.count * a.rank / 8 - tile0);
    constexpr int H = ROWS / 8;
    const uint16_t* xp[H];
#pragma unroll
    for (int h = 0; h < H; h++)  // a row past the chunk's end repeats the last
        xp[h] = a.x + token_at(a, p, chunk.y + min(h * 8 + g, chunk.z - 1)) * a.K + 8 * t;
    const uint16_t* wp[NT];
#pragma unroll
    for (int j = 0; j < NT; j++) wp[j] = column_of(a, chunk.x, tile0 + min(j, tiles - 1), g) + 8 * t;
    float acc[NT][4] = {};
    const int64_t steps = a.K / 64, k0 = 2 * (steps * slice / n_slices), k1 = 2 * (steps * (slice + 1) / n_slices);
    constexpr int kWarps = kThreads / 32;
    for (int64_t k = k0 + warp; k < k1; k += kWarps * U) {
        uint4 x[U][2], w[U][NT];
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
            for (int h = 0; h < 2; h++) {
                x[u][h] = make_uint4(0, 0, 0, 0);
                if (in && h < H) x[u][h] = *reinterpret_cast<const uint4*>(xp[h % H] + at);
            }
        }
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int j = 0; j < NT; j++)
                if (j < tiles) mma_k32(acc[j], x[u][0], x[u][1], w[u][j]);
    }
    // four of the warps write, the others add, then all add the four
    float* own = sums + (warp % 4) * (ROWS * kStride);
    __syncthreads();  // the last unit's sums are read
#pragma unroll
    for (int round = 0; round < 2; round++) {
        if (warp / 4 == round)
#pragma unroll
            for (int j = 0; j < NT; j++)
#pragma unroll
                for (int h = 0; h < H; h++) {
                    float2* at = reinterpret_cast<float2*>(own + (h * 8 + g) * kStride + j * 8 + 2 * t);
                    float2 v = make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
                    if (round) {
                        const float2 o = *at;
                        v.x += o.x, v.y += o.y;
                    }
                    *at = v;
                }
        __syncthreads();
    }
    write_sums(a, row0, chunk.z, tile0, tiles, sums, 4, kStride, ROWS * kStride);
}

// A unit with many tokens, up to 64 by 128 columns: bound by the bytes of x, so x is read once for all columns.  Stages
// of 128 k, of x and of A, are copied into shared memory while one is multiplied, two of 128 columns or up to four of
// fewer (o of 8191 tokens, rank 16: 76.3 -> 74.8 us); a row is 16 pieces of 16
// bytes, and the odd rows' pieces change places by four, so that the eight lanes of a 128-bit read (two rows) hit
// all banks.  Eight warps: two halves of the tokens, and column groups of up to four tiles; with few columns the
// warps of a half share out the stage's k instead.
constexpr int kStageK = 128, kStageRows = kChunk + 128, kStageBytes = kStageRows * kStageK * 2;

__device__ __forceinline__ uint32_t piece_at(int row, int piece) {
    return row * (kStageK * 2) + ((piece ^ ((row & 1) << 2)) << 4);
}

__device__ __forceinline__ void shrink_many(const LoraArgs& a, const Plan& p, const int4& chunk, int slice, int n_slices,
                                            int tile0, int64_t row0, uint8_t* ring) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int tiles = min(kManyTiles, a.count * a.rank / 8 - tile0);
    const int col_groups = tiles > 8 ? 4 : tiles > 4 ? 2 : 1, k_groups = 4 / col_groups;
    const int half = warp % 2, col_group = warp / 2 % col_groups, k_group = warp / 2 / col_groups;
    const int each = (tiles + col_groups - 1) / col_groups, first_tile = col_group * each;
    const int own_tiles = max(0, min(each, tiles - first_tile));
    const int64_t steps = a.K / 64, k0 = 64 * (steps * slice / n_slices), k1 = 64 * (steps * (slice + 1) / n_slices);
    const int stage_bytes = (kChunk + tiles * 8) * kStageK * 2, stages = min(4, 2 * kStageBytes / stage_bytes);
    // what this thread copies: piece `piece` of rows first, first + 16, ...
    const int piece = threadIdx.x % 16, first = threadIdx.x / 16;
    const uint16_t* src[12];
#pragma unroll
    for (int i = 0; i < 4; i++)
        src[i] = a.x + token_at(a, p, chunk.y + min(first + 16 * i, chunk.z - 1)) * a.K + piece * 8;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int col = min(first + 16 * i, tiles * 8 - 1);
        src[4 + i] = column_of(a, chunk.x, tile0 + col / 8, col % 8) + piece * 8;
    }
    auto copy = [&](int64_t k, uint8_t* stage) {
        const uint32_t bytes = k + piece * 8 < k1 ? 16u : 0u;  // zeros past the slice
        const int64_t at = bytes ? k : 0;
#pragma unroll
        for (int i = 0; i < 12; i++) {
            const int row = first + 16 * i;  // rows of x, then of A
            if (i >= 4 && row - kChunk >= tiles * 8) continue;
            cp_async16(stage + piece_at(row, piece), src[i] + at, bytes);
        }
        cp_async_commit();
    };
    float acc[2][4][4] = {};
    __syncthreads();  // the last unit's sums are read
    for (int i = 0; i < stages - 1; i++) {
        if (k0 + i * kStageK < k1)
            copy(k0 + i * kStageK, ring + i * stage_bytes);
        else
            cp_async_commit();
    }
    int at = 0;
    for (int64_t k = k0; k < k1; k += kStageK, at = at + 1 == stages ? 0 : at + 1) {
        if (k + (stages - 1) * kStageK < k1)
            copy(k + (stages - 1) * kStageK, ring + (at ? at - 1 : stages - 1) * stage_bytes);
        else
            cp_async_commit();
        if (stages == 2)
            cp_async_wait<1>();
        else if (stages == 3)
            cp_async_wait<2>();
        else
            cp_async_wait<3>();
        __syncthreads();
        const uint8_t* stage = ring + at * stage_bytes;
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
    write_sums(a, row0, chunk.z, tile0, tiles, sums, k_groups, stride, part);
}

__global__ void __launch_bounds__(kThreads, 2) shrink_kernel(const __grid_constant__ LoraArgs a) {
    extern __shared__ __align__(16) uint8_t ring[];
    pdl_launch_dependents();
    pdl_wait();
    Plan p;
    if (!read_plan(a, &p)) return;
    const Cut cut = cut_of(a, p);
    const int64_t many = static_cast<int64_t>(p.n_many) * cut.many_slices * cut.many_groups;
    const int64_t units = many + static_cast<int64_t>(p.n_few) * cut.few_slices * cut.few_groups;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        // (a chunk's units are neighbours: they read the same x or the same A)
        if (u < many) {
            const int group = static_cast<int>(u) % cut.many_groups, rest = static_cast<int>(u) / cut.many_groups;
            const int slice = rest % cut.many_slices, c = rest / cut.many_slices;
            const int4 chunk = p.chunks[c];
            if (chunk_ok(a, p, chunk, kChunk))
                shrink_many(a, p, chunk, slice, cut.many_slices, group * kManyTiles, cut.many_row(c, slice), ring);
        } else {
            const int v = static_cast<int>(u - many), group = v % cut.few_groups, rest = v / cut.few_groups;
            const int slice = rest % cut.few_slices, c = rest / cut.few_slices;
            const int4 chunk = p.chunks[p.n_many + c];
            if (!chunk_ok(a, p, chunk, kFew)) continue;
            float* sums = reinterpret_cast<float*>(ring);
            const int64_t row0 = cut.few_row(p.n_many, c, slice);
            if (chunk.z <= 8)
                shrink_few<8, kFewTiles, 4>(a, p, chunk, slice, cut.few_slices, group * kFewTiles, row0, sums);
            else
                shrink_few<16, kFewTiles, 3>(a, p, chunk, slice, cut.few_slices, group * kFewTiles, row0, sums);
        }
    }
}

// Where a lane's results stand: column g of a warp's tile j is row 8 (g / 2) + 2 j + g % 2 of 32, so that its eight
// results for a token are eight consecutive values of y.
// W: 16-byte words of a lane that hold a row of B; 0: half of one (rank 16 or less), and a step of 16 instead of two.
template <int W>
struct Weights {
    uint4 w[4][W];
    static constexpr int kLane = 8, kCols = W * 32;  // values of a row that a lane takes at a time, that fit
    // of h's rows in shared memory, so that the eight lanes of a 128-bit read (two rows) hit all banks
    static constexpr int kStride = W == 1 ? kCols : kCols + 32;
    // Rows `from`, from + 2, ... behind p, all there and of kCols values: every address is a constant away.
    __device__ __forceinline__ void load_whole(const uint16_t* p, int from) {
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int k = 0; k < W; k++)
                w[j][k] = __ldg(reinterpret_cast<const uint4*>(p + (from + 2 * j) * kCols + k * 32));
    }
    // Any: a row past `last` reads that instead (its results are not stored), columns from the rank on are zeros.
    __device__ __forceinline__ void load(const uint16_t* p, int from, int last, int rank, int t) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint16_t* row = p + static_cast<int64_t>(min(from + 2 * j, last)) * rank;
#pragma unroll
            for (int k = 0; k < W; k++) {
                w[j][k] = make_uint4(0, 0, 0, 0);
                if (k * 32 + 8 * t < rank) w[j][k] = __ldg(reinterpret_cast<const uint4*>(row + k * 32));
            }
        }
    }
    // acc: the product of 16 tokens, rows row .. of hi + lo, and these 32 rows of B
    __device__ __forceinline__ void multiply(float (&acc)[4][4], const uint16_t* hi, const uint16_t* lo, int row, int stride,
                                             int t) const {
#pragma unroll
        for (int k = 0; k < W; k++) {
            const int at = row * stride + k * 32 + 8 * t;
            const uint4 l0 = lds128(lo + at), l1 = lds128(lo + at + 8 * stride);
            const uint4 h0 = lds128(hi + at), h1 = lds128(hi + at + 8 * stride);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (k == 0)
                    mma_bf16_first(acc[j], l0.x, l1.x, l0.y, l1.y, w[j][k].x, w[j][k].y);
                else
                    mma_bf16(acc[j], l0.x, l1.x, l0.y, l1.y, w[j][k].x, w[j][k].y);
                mma_bf16(acc[j], l0.z, l1.z, l0.w, l1.w, w[j][k].z, w[j][k].w);
                mma_k32(acc[j], h0, h1, w[j][k]);
            }
        }
    }
};
template <>
struct Weights<0> {
    uint2 w[4];
    static constexpr int kLane = 4, kCols = 16, kStride = 16;  // (sixteen lanes, four rows)
    __device__ __forceinline__ void load_whole(const uint16_t* p, int from) {
#pragma unroll
        for (int j = 0; j < 4; j++) w[j] = __ldg(reinterpret_cast<const uint2*>(p + (from + 2 * j) * kCols));
    }
    __device__ __forceinline__ void load(const uint16_t* p, int from, int last, int rank, int t) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            w[j] = make_uint2(0, 0);
            if (4 * t < rank)
                w[j] = __ldg(reinterpret_cast<const uint2*>(p + static_cast<int64_t>(min(from + 2 * j, last)) * rank));
        }
    }
    __device__ __forceinline__ void multiply(float (&acc)[4][4], const uint16_t* hi, const uint16_t* lo, int row, int stride,
                                             int t) const {
        const int at = row * stride + 4 * t;
        const uint2 l0 = *reinterpret_cast<const uint2*>(lo + at), l1 = *reinterpret_cast<const uint2*>(lo + at + 8 * stride);
        const uint2 h0 = *reinterpret_cast<const uint2*>(hi + at), h1 = *reinterpret_cast<const uint2*>(hi + at + 8 * stride);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            mma_bf16_first(acc[j], l0.x, l1.x, l0.y, l1.y, w[j].x, w[j].y);
            mma_bf16(acc[j], h0.x, h1.x, h0.y, h1.y, w[j].x, w[j].y);
        }
    }
};

// Which 256 rows of which projection a unit has.
struct Block {
    int i, first, left;  // the projection, its first row, and how many blocks from here on it has
};
__device__ __forceinline__ Block block_of(const LoraArgs& a, int block) {
    Block r{0, 0, 0};
    for (;; r.i++) {
        r.left = static_cast<int>((a.N[r.i] + 255) / 256) - block;
        if (r.left > 0 || r.i + 1 == a.count) break;
        block -= static_cast<int>((a.N[r.i] + 255) / 256);
    }
    r.first = block * 256;
    return r;
}

// v * s as the sum of two bf16 numbers each; an infinity as itself and zero, so that it stays one.
__device__ __forceinline__ float rest_of(float f, float hi) { return fabsf(hi) == INFINITY ? 0.0f : f - hi; }
__device__ __forceinline__ void split_h(const float4& v, float s, uint16_t* hi, uint16_t* lo) {
    const float f[4] = {v.x * s, v.y * s, v.z * s, v.w * s};
    const uint32_t h01 = f32x2_to_bf16x2(f[0], f[1]), h23 = f32x2_to_bf16x2(f[2], f[3]);
    const float2 r01 = bf16x2_to_f32x2(h01), r23 = bf16x2_to_f32x2(h23);
    *reinterpret_cast<uint2*>(hi) = make_uint2(h01, h23);
    *reinterpret_cast<uint2*>(lo) = make_uint2(f32x2_to_bf16x2(rest_of(f[0], r01.x), rest_of(f[1], r01.y)),
                                               f32x2_to_bf16x2(rest_of(f[2], r23.x), rest_of(f[3], r23.y)));
}

// h of a chunk for one projection: its slices from `h` on, `step` floats apart, summed in order, times s, as the sum of
// two bf16 numbers (2^-16 of it), rows of kStride; zeros up to whole tiles.  A thread takes four columns of a row, and
// four slices at a time.
// (The thread's number is hidden from the compiler: it would work the places out ahead of the loop that stages now and
// then, and keep them in registers that the loop needs.)
template <int kCols, int kStride>
__device__ __forceinline__ void stage_h(const float* h, int R, int rank, int tokens, int n_slices, int step, float s,
                                        uint16_t* hi, uint16_t* lo) {
    constexpr int kAhead = 4;
    const int items = (tokens + 15) / 16 * 16 * (kCols / 4);
    int thread = threadIdx.x;
    asm volatile("" : "+r"(thread));
    for (int e = thread; e < items; e += kThreads) {
        const int row = e / (kCols / 4), col = e % (kCols / 4) * 4;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (row < tokens && col < rank) {
            const float* from = h + row * R + col;
#pragma unroll 1
            for (int q0 = 0; q0 < n_slices; q0 += kAhead) {
                float4 o[kAhead];
#pragma unroll
                for (int q = 0; q < kAhead; q++)
                    if (q0 + q < n_slices) o[q] = *reinterpret_cast<const float4*>(from + (q0 + q) * step);
#pragma unroll
                for (int q = 0; q < kAhead; q++)
                    if (q0 + q < n_slices) v.x += o[q].x, v.y += o[q].y, v.z += o[q].z, v.w += o[q].w;
            }
        }
        split_h(v, s, hi + row * kStride + col, lo + row * kStride + col);
    }
}

// Eight values of the base from column col on, in rows that begin anywhere: read one by one, and before anything is
// stored (a load stays behind a store that may be to its place: one by one, 778 tokens beside 328 + 73 columns took 32 us,
// not 22).
__device__ __forceinline__ uint4 odd_row(const uint16_t* base, int col, int N) {
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = col + j < N ? base[j] : 0;
    return make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
}

// Adds a lane's eight results (row h * 8 + g of a tile) to the base `v`, to `y`: columns col .. col + 7 of N.
__device__ __forceinline__ void add_row(uint16_t* y, const uint4& v, const float (&acc)[4][4], int h, bool vec, int col,
                                        int N) {
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const float2 f = bf16x2_to_f32x2(in[j]);
        out[j] = f32x2_to_bf16x2(f.x + acc[j][2 * h], f.y + acc[j][2 * h + 1]);
    }
    if (vec) {
        *reinterpret_cast<uint4*>(y) = make_uint4(out[0], out[1], out[2], out[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (col + j < N) y[j] = static_cast<uint16_t>(out[j / 2] >> (16 * (j % 2)));
    }
}

// A unit is a chunk and 256 rows of one projection, 32 a warp.  Units u0 .. u1 of the chunks of many: bound by the base and
// y, so the base of several tiles is on its way at once.
template <int W, bool EXACT>
__device__ __forceinline__ void expand_many(const LoraArgs& a, const Plan& p, const Cut& cut, int blocks, int64_t u0,
                                            int64_t u1, uint16_t* hi, uint16_t* lo, int32_t* rows) {
    constexpr int kCols = Weights<W>::kCols, kStride = Weights<W>::kStride;
    // tiles of 16 tokens whose base is on its way (gate|up of 4099 tokens, rank 64: 194 us; 207 with one, 210 with four)
    constexpr int kTiles = W >= 4 ? 1 : W >= 1 ? 2 : 4;
    const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4, warp_row = threadIdx.x / 32 * 32;
    const int rank = EXACT ? kCols : a.rank, R = a.count * rank;
    int held = -1, c = static_cast<int>(u0 / blocks), at_block = static_cast<int>(u0 % blocks);
#pragma unroll 1
    for (int64_t u = u0; u < u1; u++, at_block++) {
        if (at_block == blocks) at_block = 0, c++;
        const Block block = block_of(a, at_block);
        const int i = block.i, N = static_cast<int>(a.N[i]), n0 = block.first + warp_row, n = n0 + 8 * t;
        const int4 chunk = p.chunks[c];
        if (!chunk_ok(a, p, chunk, kChunk)) continue;
        if (held != c * a.count + i) {
            held = c * a.count + i;
            __syncthreads();
            stage_h<kCols, kStride>(a.h + cut.many_row(c, 0) * R + i * rank, R, rank, chunk.z, cut.many_slices,
                                    kChunk * R, a.scales[chunk.x], hi, lo);
            if (threadIdx.x < kChunk)
                rows[threadIdx.x] =
                    static_cast<int32_t>(token_at(a, p, chunk.y + min(static_cast<int>(threadIdx.x), chunk.z - 1)));
            __syncthreads();
        }
        if (n0 >= N) continue;
        const bool vec = N % 8 == 0, in_row = n < N;
        const int first_row = n0 + 8 * (g / 2) + g % 2;
        const uint16_t* base = a.base[i] + n;
        uint16_t* y = a.y[i] + n;
        const uint16_t* b = a.b[i] + (static_cast<int64_t>(chunk.x) * N + first_row) * rank + Weights<W>::kLane * t;
        Weights<W> w;
        if (EXACT && whole_blocks(block.first, N, 1))
            w.load_whole(b, 0);
        else
            w.load(b, 0, N - 1 - first_row, rank, t);
#pragma unroll 1
        for (int r0 = 0; r0 < chunk.z; r0 += 16 * kTiles) {
            uint4 in[2 * kTiles];
#pragma unroll
            for (int m = 0; m < 2 * kTiles; m++) {
                const int r = r0 + g + 8 * m;
                if (vec && in_row && r < chunk.z)
                    in[m] = *reinterpret_cast<const uint4*>(base + static_cast<int64_t>(rows[r]) * N);
            }
#pragma unroll
            for (int m = 0; m < 2 * kTiles; m += 2) {
                if (r0 + 8 * m >= chunk.z) continue;
                if (!vec)
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const int r = r0 + g + 8 * (m + h);
                        if (r < chunk.z) in[m + h] = odd_row(base + static_cast<int64_t>(rows[r]) * N, n, N);
                    }
                float acc[4][4];
                w.multiply(acc, hi, lo, r0 + g + 8 * m, kStride, t);
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int r = r0 + g + 8 * (m + h);
                    if (r >= chunk.z || !in_row) continue;
                    const int64_t at = static_cast<int64_t>(rows[r]) * N;
                    add_row(y + at, in[m + h], acc, h, vec, n, N);
                }
            }
        }
    }
}

// Rows without an adapter, where the output is not the base itself: copied, 64 tokens and 256 columns a unit.
// A warp's eight loads, of eight rows each, may be of several units.
__device__ __forceinline__ void copy_idle(const LoraArgs& a, const Plan& p, int blocks, int64_t u0, int64_t u1) {
    const int lane = threadIdx.x % 32, g = lane / 4, warp_row = threadIdx.x / 32 * 32;
    int batch = 0;
#pragma unroll 1
    for (int64_t u = u0; u < u1; u += batch) {
        const Block block = block_of(a, static_cast<int>(u % blocks));
        const int first = p.n_tokens + static_cast<int>(u / blocks) * kChunk;
        const int tokens = min(kChunk, static_cast<int>(a.T) - first), rounds = (tokens + 7) / 8;
        const int N = static_cast<int>(a.N[block.i]), n0 = block.first + warp_row, n = n0 + 8 * (lane % 4);
        batch = min(8 / rounds, static_cast<int>(min(static_cast<int64_t>(block.left), u1 - u)));
        const uint16_t* base = a.base[block.i];
        uint16_t* y = a.y[block.i];
        if (base == y) continue;
        if (N % 8 == 0) {
            uint4 v[8];
            int64_t at[8];
#pragma unroll
            for (int q = 0; q < 8; q++) {
                const int r = q % rounds * 8 + g, more = q / rounds * 256;
                at[q] = q < batch * rounds && r < tokens && column_there(n, more, N)
                            ? token_at(a, p, first + r) * N + n + more
                            : -1;
                if (at[q] >= 0) v[q] = *reinterpret_cast<const uint4*>(base + at[q]);
            }
#pragma unroll
            for (int q = 0; q < 8; q++)
                if (at[q] >= 0) *reinterpret_cast<uint4*>(y + at[q]) = v[q];
        } else {
            for (int more = 0; more < batch * 256 && column_there(n0 + lane, more, N); more += 256)
                for (int r = 0; r < tokens; r += 8) {  // loads before stores, which may not pass each other
                    uint16_t v[8];
                    int64_t at[8];
#pragma unroll
                    for (int q = 0; q < 8; q++) {
                        at[q] = token_at(a, p, first + min(r + q, tokens - 1)) * N + n0 + lane + more;
                        v[q] = base[at[q]];
                    }
#pragma unroll
                    for (int q = 0; q < 8; q++) y[at[q]] = v[q];  // (the last row may be written twice, alike)
                }
        }
    }
}

// Units u0 .. u1 of the chunks of few: bound by the bytes of B, so the rows and the base of D units are on their way at
// once.
template <int W, int D, bool EXACT>
__device__ __forceinline__ void expand_few(const LoraArgs& a, const Plan& p, const Cut& cut, int blocks, int64_t u0,
                                           int64_t u1, uint16_t* hi, uint16_t* lo) {
    constexpr int kCols = Weights<W>::kCols, kStride = Weights<W>::kStride;
    const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4, warp_row = threadIdx.x / 32 * 32;
    const int rank = EXACT ? kCols : a.rank, R = a.count * rank;
    int held = -1, held_chunk = -1, batch = 0, c = static_cast<int>(u0 / blocks), at_block = static_cast<int>(u0 % blocks);
    int4 chunk = make_int4(0, 0, 0, 0);
    int32_t token[2] = {0, 0};  // of rows g and g + 8
#pragma unroll 1
    for (int64_t u = u0; u < u1; u += batch, at_block += batch) {
        if (at_block >= blocks) at_block -= blocks, c++;  // (a batch ends with its projection)
        const Block block = block_of(a, at_block);
        const int i = block.i, N = static_cast<int>(a.N[i]), n0 = block.first + warp_row, n = n0 + 8 * t;
        const int left = static_cast<int>(min(static_cast<int64_t>(block.left), u1 - u));
        const bool vec = N % 8 == 0;
        const uint16_t* base = a.base[i] + n;
        uint16_t* y = a.y[i] + n;
        if (held_chunk != c) {
            held_chunk = c;
            chunk = p.chunks[p.n_many + c];
            if (!chunk_ok(a, p, chunk, kFew)) chunk.z = 0;
#pragma unroll
            for (int h = 0; h < 2; h++)
                if (8 * h + g < chunk.z) token[h] = static_cast<int32_t>(token_at(a, p, chunk.y + 8 * h + g));
        }
        batch = min(D, left);
        if (chunk.z == 0) continue;
        const int first_row = n0 + 8 * (g / 2) + g % 2, last_row = N - 1 - first_row;
        const uint16_t* b = a.b[i] + (static_cast<int64_t>(chunk.x) * N + first_row) * rank + Weights<W>::kLane * t;
        if (held != c * a.count + i) {
            held = c * a.count + i;
            // B starts on its way to L2 meanwhile
            if (lane_in_row(Weights<W>::kLane, t, rank)) {
#pragma unroll
                for (int j = 0; j < 4 * D; j++) {
                    const int row = min(j / 4 * 256 + j % 4 * 2, last_row);
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(b + static_cast<int64_t>(row) * rank));
                }
            }
            __syncthreads();
            stage_h<kCols, kStride>(a.h + cut.few_row(p.n_many, c, 0) * R + i * rank, R, rank, chunk.z, cut.few_slices,
                                    kFew * R, a.scales[chunk.x], hi, lo);
            __syncthreads();
        }
        const bool real[2] = {g < chunk.z, g + 8 < chunk.z}, both = chunk.z > 8;
        const int64_t at[2] = {static_cast<int64_t>(token[0]) * N, static_cast<int64_t>(token[1]) * N};
        Weights<W> w[D];
        uint4 in[D][2];
        if (EXACT && vec && whole_blocks(block.first, N, D) && left >= D) {
#pragma unroll
            for (int d = 0; d < D; d++) w[d].load_whole(b, 256 * d);
#pragma unroll
            for (int h = 0; h < 2; h++)
                if (real[h])
#pragma unroll
                    for (int d = 0; d < D; d++) in[d][h] = *reinterpret_cast<const uint4*>(base + at[h] + 256 * d);
        } else {
#pragma unroll
            for (int d = 0; d < D; d++) {
                if (d >= batch) continue;
                w[d].load(b, 256 * d, last_row, rank, t);
#pragma unroll
                for (int h = 0; h < 2; h++)
                    if (vec && real[h] && n + 256 * d < N)
                        in[d][h] = *reinterpret_cast<const uint4*>(base + at[h] + 256 * d);
            }
        }
#pragma unroll
        for (int d = 0; d < D; d++) {
            if (d >= batch) continue;
            if (!vec)
#pragma unroll
                for (int h = 0; h < 2; h++)
                    if (real[h]) in[d][h] = odd_row(base + at[h] + 256 * d, n + 256 * d, N);
            float acc[4][4];
            w[d].multiply(acc, hi, lo, g, kStride, t);
            if (n + 256 * d >= N) continue;
            const int64_t more = 256 * d;
            if (real[0]) add_row(y + at[0] + more, in[d][0], acc, 0, vec, n + 256 * d, N);
            if (both && real[1]) add_row(y + at[1] + more, in[d][1], acc, 1, vec, n + 256 * d, N);
        }
    }
}

// The units of all kinds on one line, each as long as it weighs (what it moves, roughly), cut into equal parts for the
// CTAs: a unit belongs to the one in whose part it begins.  (All weights 1: q|k|v of 256 tokens 42 -> 50 us; many against
// few 4 : 1 or 2 instead of 2 : 1: 44.)
template <int W, int D, bool EXACT>
__global__ void __launch_bounds__(kThreads, 2) expand_kernel(const LoraArgs a, int blocks, bool copy) {
    constexpr int kStride = Weights<W>::kStride;
    __shared__ __align__(16) uint16_t hi[kChunk * kStride], lo[kChunk * kStride];
    __shared__ int32_t rows[kChunk];
    pdl_launch_dependents();
    pdl_wait();
    Plan p;
    if (!read_plan(a, &p)) return;
    const Cut cut = cut_of(a, p);
    constexpr int kMany = 2, kFewWeight = 1;
    const int64_t idle = copy ? (a.T - p.n_tokens + kChunk - 1) / kChunk * blocks : 0;
    const int idle_weight = a.T - p.n_tokens >= kChunk ? kMany : 1;
    const int64_t to_few = static_cast<int64_t>(p.n_many) * blocks * kMany;
    const int64_t to_idle = to_few + static_cast<int64_t>(p.n_few) * blocks * kFewWeight;
    const int64_t end = to_idle + idle * idle_weight;
    const int64_t from = end * blockIdx.x / gridDim.x, to = end * (blockIdx.x + 1) / gridDim.x;
    // the first unit, of those of `weight` from `first` up to `last`, that begins at `at` or later
    auto unit = [](int64_t at, int64_t first, int64_t last, int weight) {
        return (max(min(at, last), first) - first + weight - 1) / weight;
    };
    if (from < to_few)
        expand_many<W, EXACT>(a, p, cut, blocks, unit(from, 0, to_few, kMany), unit(to, 0, to_few, kMany), hi, lo, rows);
    if (from < to_idle && to > to_few)
        expand_few<W, D, EXACT>(a, p, cut, blocks, unit(from, to_few, to_idle, kFewWeight),
                                unit(to, to_few, to_idle, kFewWeight), hi, lo);
    if (to > to_idle) copy_idle(a, p, blocks, unit(from, to_idle, end, idle_weight), unit(to, to_idle, end, idle_weight));
}

template <int W, int D, bool EXACT>
cudaError_t expand(const LoraArgs& a, int num_sms, cudaStream_t stream) {
    int blocks = 0;
    bool copy = false;
    for (int i = 0; i < a.count; i++) {
        blocks += static_cast<int>((a.N[i] + 255) / 256);
        copy |= a.base[i] != a.y[i];
    }
    cudaLaunchAttribute attr;
    const int64_t cap = static_cast<int64_t>(num_sms) * 2;
    const int64_t units = (max_chunks(a.T, a.adapters) + (copy ? (a.T + kChunk - 1) / kChunk : 0)) * blocks;
    if (units == 0) return cudaSuccess;  // no adapters, and in place
    const cudaLaunchConfig_t cfg =
        pdl_config(dim3(static_cast<unsigned>(units < cap ? units : cap)), kThreads, stream, &attr);
    return cudaLaunchKernelEx(&cfg, expand_kernel<W, D, EXACT>, a, blocks, copy);
}

}  // namespace

int64_t lora_plan_bytes(int64_t T, int64_t adapters) {
    return (kHeader + 4 * max_chunks(T, adapters) + T) * static_cast<int64_t>(sizeof(int32_t));
}

int64_t lora_workspace_bytes(int64_t T, int64_t adapters, int64_t rank, int64_t count) {
    // chunks * slices: kMaxSlices each at most, and so many in all as the slices' rule allows
    auto rows_of = [](int64_t chunks, int64_t units, int64_t each) {
        const int64_t most = chunks > units ? chunks : units;
        return each * (chunks * kMaxSlices < most ? chunks * kMaxSlices : most);
    };
    const int64_t rows = rows_of(max_many(T), kUnits, kChunk) + rows_of(max_few(T, adapters), kUnits, kFew);
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
    cfg.dynamicSmemBytes = (3 + warps) * (adapters + 1) * sizeof(int32_t);
    return cudaLaunchKernelEx(&cfg, lora_plan_kernel, ids, sequences, S, T, static_cast<int>(adapters),
                              static_cast<int32_t*>(plan), warps);
}

cudaError_t launch_lora(const LoraArgs& a, int num_sms, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    const int64_t chunks = max_chunks(a.T, a.adapters), cap = static_cast<int64_t>(num_sms) * 2;
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
    // Ranks of exactly 16, 32, 64 and 128 have constants for addresses (o of 8191 tokens 89 -> 85 us).  D is what registers
    // allow (rank 16, gate|up of 64 tokens: 30.3 us with 2, 34 with 1, 32 with 4, which spills).  At two CTAs an SM the higher
    // ranks spill all the same: 32 bytes at 32, 12 at 64, 204 to 224 at 128.
#define NF4_EXPAND(W, D) \
    return a.rank == Weights<W>::kCols ? expand<W, D, true>(a, num_sms, stream) : expand<W, D, false>(a, num_sms, stream)
    if (a.rank <= 16) NF4_EXPAND(0, 2);
    if (a.rank <= 32) NF4_EXPAND(1, 2);
    if (a.rank <= 64) NF4_EXPAND(2, 1);
    NF4_EXPAND(4, 1);
#undef NF4_EXPAND
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
