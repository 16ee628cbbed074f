// The indices of a step: pages handed out and taken back, and the place of every new token.
//
// Sequence b holds lengths[b] tokens, so ceil(length / page_size) pages, and brings n = new_tokens[b] more.  A
// prefix sum over n gives the rows of its tokens, one over the pages that it lacks the entries of the ring
// of free pages that it takes; both are integers, so every order of addition gives the same.
//
// What bounds it: the latency of one launch, of two dependent reads and of two block scans (8 sequences of one
// token: 3.4 us replayed in a graph, 5.1 us a call, the host's), and for long prompts the search for a token's sequence
// and page (32768 tokens of 512 sequences: 5.7 us, 0.08 of it their 16 bytes each).  Every CTA reads all B counts and
// scans them for itself (a few kilobytes from L2), which spares a second launch; the rows are shared out among the CTAs.
// Where `lengths` or the ring's state are updated in place, the CTAs are one cluster: its barrier stands between the
// last read and the first write.
#include <mutex>

#include "nf4_kv.cuh"

namespace nf4 {
namespace {

__device__ int g_plan_error;  // 45: a page or a ring state outside the pool

constexpr uint32_t kMost = 0x7FFFFFFFu;  // sums stop here: no row and no page has that number

// Sums that stop at kMost; both at most kMost.
__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) { return min(a + b, kMost); }

struct Sums {
    uint32_t a, b;
};

// Exclusive sums over the threads of the block, and the totals.
__device__ __forceinline__ Sums block_scan(Sums v, Sums* part, Sums* total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    auto scan = [&](Sums s) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t a = __shfl_up_sync(0xFFFFFFFFu, s.a, o), b = __shfl_up_sync(0xFFFFFFFFu, s.b, o);
            if (lane >= o) s.a = add(s.a, a), s.b = add(s.b, b);
        }
        return s;
    };
    auto before = [&](const Sums& s) {  // of the lane before
        const uint32_t a = __shfl_up_sync(0xFFFFFFFFu, s.a, 1), b = __shfl_up_sync(0xFFFFFFFFu, s.b, 1);
        return lane ? Sums{a, b} : Sums{0, 0};
    };
    const Sums own = scan(v);
    if (lane == 31) part[warp] = own;
    __syncthreads();
    const Sums all = scan(lane < warps ? part[lane] : Sums{0, 0});  // every warp for itself
    *total = {__shfl_sync(0xFFFFFFFFu, all.a, 31), __shfl_sync(0xFFFFFFFFu, all.b, 31)};
    const Sums warps_before = before(all), lanes_before = before(own);
    return {add(__shfl_sync(0xFFFFFFFFu, warps_before.a, warp), lanes_before.a),
            add(__shfl_sync(0xFFFFFFFFu, warps_before.b, warp), lanes_before.b)};
}

// The last index i in [0, n) with at[i] <= x (at[0] <= x); half: the largest power of two below n, or 1.
__device__ __forceinline__ int last_at_most(const uint32_t* at, int n, int half, uint32_t x) {
    int i = 0;
    for (int o = half; o > 0; o >>= 1)
        if (i + o < n && at[i + o] <= x) i += o;
    return i;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a, uint64_t page_magic, int half) {
    extern __shared__ uint32_t tables[];
    __shared__ Sums part[2][32];
    __shared__ uint32_t taken_s;
    const int B = a.B, per = (B + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
    // of a sequence: its first row; the pages that are new, that go back, before its own; its length (~length: refused); the
    // pages that it holds
    uint32_t *start = tables, *fresh = start + B + 1, *back = fresh + B + 1, *held = back + B + 1;
    int32_t* length = reinterpret_cast<int32_t*>(held + B + 1);
    if (threadIdx.x == 0) taken_s = 0;
    pdl_launch_dependents();
    pdl_wait();
    // the ring, kept inside its bounds whatever its state says
    int64_t first_in = a.free_in[0], count_in = a.free_in[1];
    const uint32_t pages = static_cast<uint32_t>(a.pages);
    bool bad = false;
    if (first_in < 0 || (first_in >= a.pages && first_in > 0) || count_in < 0 || count_in > a.pages) {
        bad = true;
        first_in = a.pages > 0 && first_in > 0 ? first_in % a.pages : 0;
        count_in = min(max(count_in, int64_t{0}), a.pages);
    }
    const uint32_t first = static_cast<uint32_t>(first_in), count = static_cast<uint32_t>(count_in);
    // exact below 2^32: the magic number is off by less than page_size <= 2^16 in 2^64
    auto page_of = [&](uint32_t place) { return static_cast<uint32_t>(__umul64hi(place, page_magic)); };
    auto pages_of = [&](uint32_t tokens) { return tokens ? page_of(tokens - 1) + 1 : 0; };  // (up to 2^32 - 1 tokens)

    const int b0 = min(B, static_cast<int>(threadIdx.x) * per), b1 = min(B, b0 + per);
    const uint32_t wide = static_cast<uint32_t>(a.max_pages);
    Sums sum{0, 0}, total;
    for (int b = b0; b < b1; b++) {
        const int32_t n = a.new_tokens[b], len = max(a.lengths[b], 0);
        const uint32_t has = pages_of(len);
        length[b] = len;
        fresh[b] = static_cast<uint32_t>(n);
        held[b] = has;
        bad |= n < 0 && has > wide;
        sum.a = add(sum.a, max(n, 0));
        sum.b = add(sum.b, n < 0 ? min(has, wide) : 0);
    }
    Sums at = block_scan(sum, part[0], &total);
    const uint32_t tokens = total.a, returned = min(total.b, pages - count);
    bad |= total.b > returned;
    sum = {0, 0};
    for (int b = b0; b < b1; b++) {
        const int32_t n = static_cast<int32_t>(fresh[b]);
        start[b] = at.a;
        back[b] = min(at.b, returned);
        uint32_t need = kMost;  // cannot be served
        if (n < 0) {
            need = 0;
            at.b = add(at.b, min(held[b], wide));
            length[b] = 0;
        } else {
            const uint32_t after = pages_of(static_cast<uint32_t>(length[b]) + n), end = add(at.a, n);
            if (after <= wide && static_cast<uint32_t>(length[b]) + n <= kMost && end < kMost &&
                end <= static_cast<uint64_t>(a.T))
                need = after - held[b];
            at.a = end;
        }
        fresh[b] = need;
        if (need != kMost) sum.a = add(sum.a, need);
    }
    at = block_scan(sum, part[1], &total);
    const uint32_t available = count + returned;
    uint32_t taken = 0;
    for (int b = b0; b < b1; b++) {
        const uint32_t need = fresh[b];
        fresh[b] = min(at.a, available);
        if (need != kMost && need > 0) {
            at.a = add(at.a, need);
            if (at.a <= available) taken = at.a;
        }
        if (need == kMost || (need > 0 && at.a > available)) length[b] = ~length[b];
    }
    taken = __reduce_max_sync(0xFFFFFFFFu, taken);
    if (taken > 0 && threadIdx.x % 32 == 0) atomicMax(&taken_s, taken);  // a maximum: any order
    if (threadIdx.x == 0) start[B] = tokens, back[B] = returned;
    __syncthreads();
    taken = taken_s;
    // a served sequence's new pages are the taken ones fresh[b], fresh[b] + 1, ...
    const uint32_t id = blockIdx.x * blockDim.x + threadIdx.x, step = gridDim.x * blockDim.x;
    auto in_ring = [&](uint32_t i) { return i < pages ? i : i - pages; };
    // The page that is given back as the j-th; that is taken as the k-th: from the ring, then from those given back.
    auto given_back = [&](uint32_t j) {
        const int b = last_at_most(back, B, half, j);
        return a.page_table[static_cast<int64_t>(b) * a.max_pages + (j - back[b])];
    };
    auto page_at = [&](uint32_t k) { return k < count ? a.free_pages[in_ring(first + k)] : given_back(k - count); };
    if (a.in_place && gridDim.x > 1) {  // every CTA has read the lengths and the ring's state: they may be written now
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    for (uint32_t b = id; b < static_cast<uint32_t>(B); b += step) {
        const int32_t len = length[b];
        a.lengths_out[b] = len < 0 ? ~len : len + static_cast<int32_t>(start[b + 1] - start[b]);
        a.starts[b] = static_cast<int32_t>(start[b]);
    }
    if (id == 0) {
        a.starts[B] = static_cast<int32_t>(tokens);
        a.free_out[0] = pages > 0 ? (first + taken) % pages : 0;
        a.free_out[1] = available - taken;
    }
    for (uint32_t j = id; j < returned; j += step) a.free_pages[in_ring(in_ring(first + count) + j)] = given_back(j);
    for (uint32_t k = id; k < taken; k += step) {
        const int b = last_at_most(fresh, B, half, k);
        a.page_table[static_cast<int64_t>(b) * a.max_pages + held[b] + (k - fresh[b])] = page_at(k);
    }
    for (uint32_t i = id; i < a.T; i += step) {
        int64_t slot = -1;
        uint32_t pos = 0;
        int seq = -1;
        if (i < tokens) {
            seq = last_at_most(start, B, half, i);
            const int32_t len = length[seq];
            pos = (len < 0 ? ~len : len) + (i - start[seq]);
            if (len >= 0) {
                const uint32_t p = page_of(pos), has = held[seq];
                const int32_t page = p >= has ? page_at(fresh[seq] + (p - has))
                                              : a.page_table[static_cast<int64_t>(seq) * a.max_pages + p];
                if (page >= 0 && static_cast<uint32_t>(page) < pages)
                    slot = static_cast<int64_t>(page) * a.page_size + (pos - p * a.page_size);
                else
                    bad = true;
            }
        }
        a.slots[i] = slot;
        a.positions[i] = static_cast<int32_t>(pos);
        a.sequences[i] = seq;
    }
    if (bad) atomicCAS(&g_plan_error, 0, 45);
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& a, int num_sms, cudaStream_t stream) {
    // A row or two a thread; in place no more CTAs than a cluster has (32768 tokens: 6.5 us with 32 CTAs, 8.3 with 8, 33
    // with one).  Small CTAs start sooner (5.7 us with 64 of 256 threads); large ones scan many sequences, or share out the
    // rows of a cluster.
    const int64_t rows = a.T > a.B ? a.T : a.B;
    const int threads = rows <= 256 || (!a.in_place && a.B <= 1024) ? 256 : kPlanThreads;
    int ctas = 1;
    while (ctas < (a.in_place ? 8 : num_sms / 2) && rows > 2 * threads * ctas) ctas *= 2;
    const int bytes = 5 * (a.B + 1) * static_cast<int>(sizeof(int32_t));
    static std::once_flag once[64];
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    std::call_once(once[device & 63], [&] {
        e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 5 * (kPlanMaxBatch + 1) * static_cast<int>(sizeof(int32_t)));
    });
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = pdl_config(dim3(ctas), threads, stream, attr);
    cfg.dynamicSmemBytes = bytes;
    if (a.in_place && ctas > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
        cfg.numAttrs = 2;
    }
    int half = 1;
    while (half * 2 < a.B) half *= 2;
    return cudaLaunchKernelEx(&cfg, plan_kernel, a, ~uint64_t{0} / a.page_size + 1, half);
}

cudaError_t read_and_clear_plan_error(int* code) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_plan_error, sizeof(int));
    if (e != cudaSuccess) return e;
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_plan_error, &zero, sizeof(int));
    *code = v;
    return e;
}

}  // namespace nf4
