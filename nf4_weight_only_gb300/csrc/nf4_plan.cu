// The indices of a step: pages handed out and taken back, and the place of every new token.
//
// Sequence b holds lengths[b] tokens, so ceil(length / page_size) pages, and brings n = new_tokens[b] more.  A
// prefix sum over n gives the rows of its tokens, one over the pages that it lacks the entries of the ring
// of free pages that it takes; both are integers, so every order of addition gives the same.
//
// What bounds it: the latency of one launch, of two dependent reads and of two block scans (8 sequences of one
// token), and for long prompts the 16 bytes that a token's place, position and sequence take.  Every CTA reads all
// B counts and scans them for itself (a few kilobytes from L2), which spares a second launch; the rows are
// shared out among the CTAs of one cluster.  A cluster, because `lengths` and the ring's state may be updated in
// place: its barrier stands between the last read and the first write.
#include <mutex>

#include "nf4_kv.cuh"

namespace nf4 {
namespace {

__device__ int g_plan_error;  // 45: a page or a ring state outside the pool

struct Sums {
    int64_t a, b;
};

// Exclusive sums over the threads of the block, and the totals; `part` holds 33 entries.
__device__ __forceinline__ Sums block_scan(Sums v, Sums* part, Sums* total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    Sums s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t a = __shfl_up_sync(0xFFFFFFFFu, s.a, o), b = __shfl_up_sync(0xFFFFFFFFu, s.b, o);
        if (lane >= o) s.a += a, s.b += b;
    }
    __syncthreads();  // the last use of `part`
    if (lane == 31) part[warp] = s;
    __syncthreads();
    if (warp == 0) {
        Sums w = lane < warps ? part[lane] : Sums{0, 0};
        const Sums own = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t a = __shfl_up_sync(0xFFFFFFFFu, w.a, o), b = __shfl_up_sync(0xFFFFFFFFu, w.b, o);
            if (lane >= o) w.a += a, w.b += b;
        }
        if (lane == 31) part[32] = w;
        if (lane < warps) part[lane] = {w.a - own.a, w.b - own.b};
    }
    __syncthreads();
    *total = part[32];
    return {part[warp].a + s.a - v.a, part[warp].b + s.b - v.b};
}

// The last index i in [0, n) with at[i] <= x (at[0] <= x).
__device__ __forceinline__ int last_at_most(const int32_t* at, int n, int32_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// A sequence as the tables in shared memory hold it.
struct Tables {
    int32_t *start, *length, *fresh, *back;  // rows; length (~length: refused); new pages; pages given back
};

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
    extern __shared__ int32_t tables[];
    __shared__ Sums part[33];
    __shared__ unsigned long long taken_s;
    const int B = a.B, per = (B + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
    const Tables s = {tables, tables + (B + 1), tables + 2 * (B + 1), tables + 3 * (B + 1)};
    if (threadIdx.x == 0) taken_s = 0;
    pdl_launch_dependents();
    pdl_wait();
    // the ring, kept inside its bounds whatever its state says
    int64_t first = a.free_in[0], count = a.free_in[1];
    bool bad = first < 0 || (first >= a.pages && first > 0) || count < 0 || count > a.pages;
    first = a.pages > 0 && first > 0 ? first % a.pages : 0;
    count = min(max(count, int64_t{0}), a.pages);

    auto pages_of = [&](int64_t tokens) {
        return tokens < (int64_t{1} << 32) - a.page_size
                   ? static_cast<int64_t>((static_cast<uint32_t>(tokens) + a.page_size - 1) / a.page_size)
                   : (tokens + a.page_size - 1) / a.page_size;
    };
    const int b0 = min(B, static_cast<int>(threadIdx.x) * per), b1 = min(B, b0 + per);
    Sums sum{0, 0}, total;
    for (int b = b0; b < b1; b++) {
        const int32_t n = a.new_tokens[b], len = max(a.lengths[b], 0);
        s.length[b] = len;
        s.fresh[b] = n;
        int64_t back = n < 0 ? pages_of(len) : 0;
        if (back > a.max_pages) back = a.max_pages, bad = true;
        sum.a += max(n, 0);
        sum.b += back;
    }
    Sums at = block_scan(sum, part, &total);
    const int64_t tokens = total.a, returned = min(total.b, a.pages - count);
    bad |= total.b > returned;
    sum = {0, 0};
    for (int b = b0; b < b1; b++) {
        const int32_t n = s.fresh[b], len = s.length[b];
        s.start[b] = static_cast<int32_t>(min(at.a, int64_t{0x7FFFFFFF}));
        s.back[b] = static_cast<int32_t>(min(at.b, returned));
        int32_t need = 0;  // -1: cannot be served
        if (n < 0) {
            at.b += min(pages_of(len), a.max_pages);
            s.length[b] = 0;
        } else {
            const int64_t after = pages_of(static_cast<int64_t>(len) + n);
            need = after <= a.max_pages && at.a + n <= a.T ? static_cast<int32_t>(after - pages_of(len)) : -1;
            at.a += n;
        }
        s.fresh[b] = need;
        sum.a += max(need, 0);
    }
    at = block_scan(sum, part, &total);
    const int64_t available = count + returned;
    int64_t taken = 0;
    for (int b = b0; b < b1; b++) {
        const int32_t need = s.fresh[b];
        s.fresh[b] = static_cast<int32_t>(min(at.a, available));
        if (need > 0) {
            at.a += need;
            if (at.a <= available) taken = at.a;
        }
        if (need < 0 || (need > 0 && at.a > available)) s.length[b] = ~s.length[b];
    }
    if (taken > 0) atomicMax(&taken_s, static_cast<unsigned long long>(taken));  // a maximum: any order
    if (threadIdx.x == 0) {
        s.start[B] = static_cast<int32_t>(min(tokens, int64_t{0x7FFFFFFF}));
        s.back[B] = static_cast<int32_t>(returned);
    }
    __syncthreads();
    taken = static_cast<int64_t>(taken_s);
    // a served sequence's new pages are the taken ones fresh[b], fresh[b] + 1, ...
    const uint32_t rank = blockIdx.x, ranks = gridDim.x;
    const uint32_t id = rank * blockDim.x + threadIdx.x, step = ranks * blockDim.x;
    // The page that is taken as the k-th: from the ring, then from those given back in this step.
    auto given_back = [&](int32_t j) {
        const int b = last_at_most(s.back, B, j);
        return a.page_table[static_cast<int64_t>(b) * a.max_pages + (j - s.back[b])];
    };
    auto page_at = [&](int64_t k) {
        if (k >= count) return given_back(static_cast<int32_t>(k - count));
        const int64_t i = first + k;
        return a.free_pages[i < a.pages ? i : i - a.pages];
    };
    // every CTA has read the lengths and the ring's state: from here on they may be written
    if (ranks > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    for (uint32_t b = id; b < static_cast<uint32_t>(B); b += step) {
        const int32_t len = s.length[b];
        a.lengths_out[b] = len < 0 ? ~len : len + (s.start[b + 1] - s.start[b]);
        a.starts[b] = s.start[b];
    }
    if (id == 0) {
        a.starts[B] = s.start[B];
        const int64_t i = a.pages > 0 ? (first + taken) % a.pages : 0;
        a.free_out[0] = i;
        a.free_out[1] = count + returned - taken;
    }
    for (int64_t j = id; j < returned; j += step) {
        const int64_t i = first + count + j;
        a.free_pages[i < a.pages ? i : i - a.pages] = given_back(static_cast<int32_t>(j));
    }
    for (int64_t k = id; k < taken; k += step) {
        const int b = last_at_most(s.fresh, B, static_cast<int32_t>(k));
        const int64_t p = pages_of(s.length[b]) + (k - s.fresh[b]);
        a.page_table[static_cast<int64_t>(b) * a.max_pages + p] = page_at(k);
    }
    for (int64_t i = id; i < a.T; i += step) {
        int64_t slot = -1;
        int32_t pos = 0, seq = -1;
        if (i < tokens) {
            seq = last_at_most(s.start, B, static_cast<int32_t>(i));
            const int32_t len = s.length[seq];
            pos = (len < 0 ? ~len : len) + (static_cast<int32_t>(i) - s.start[seq]);
            if (len >= 0) {
                const int64_t p = static_cast<uint32_t>(pos) / a.page_size, held = pages_of(len);
                const int32_t page = p >= held ? page_at(s.fresh[seq] + (p - held))
                                               : a.page_table[static_cast<int64_t>(seq) * a.max_pages + p];
                if (page >= 0 && page < a.pages)
                    slot = static_cast<int64_t>(page) * a.page_size + static_cast<uint32_t>(pos) % a.page_size;
                else
                    bad = true;
            }
        }
        a.slots[i] = slot;
        a.positions[i] = pos;
        a.sequences[i] = seq;
    }
    if (bad) atomicCAS(&g_plan_error, 0, 45);
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t stream) {
    const int64_t rows = a.T > 4 * a.B ? a.T : 4 * a.B;
    int ctas = 1;
    while (ctas < 8 && rows > 2048 * ctas) ctas *= 2;
    const int threads = a.B <= 256 && rows <= 512 ? 256 : kPlanThreads;
    const int bytes = 4 * (a.B + 1) * static_cast<int>(sizeof(int32_t));
    static std::once_flag once[64];
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    std::call_once(once[device & 63], [&] {
        e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 4 * (kPlanMaxBatch + 1) * static_cast<int>(sizeof(int32_t)));
    });
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = pdl_config(dim3(ctas), threads, stream, attr);
    cfg.dynamicSmemBytes = bytes;
    if (ctas > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, plan_kernel, a);
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
