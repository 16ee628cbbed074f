// The next token of every row of logits.
//
// With z_i = (l_i - max l) / T, the weight of token i is w_i = exp(z_i).  Top-k, top-p and min-p each keep a
// beginning of the tokens ordered by logit (ties: the lower index first); the token drawn is the first index i, in
// index order, at which the sum of the kept weights up to i passes u times their whole sum.
//
// Sums are exact: a weight is a whole number of 2^-40 (its error a few of them), and sums of up to 2^18 of them
// fit 64 bits.  So no order of addition, number of CTAs or atomic changes a result, and the border between two
// tokens is within 2^-36 or so of where the formula has it; sums in fp32 would move the borders of a flat
// distribution over 150,000 tokens by some hundredths of a token.
//
// A row is held by the CTAs of one cluster, a slice of it in the shared memory of each, so the logits are read once
// from memory; what a row needs next (its maximum, where the order is cut, which slice the token is in)
// is exchanged through distributed shared memory.
#include <cooperative_groups.h>

#include <mutex>

#include "nf4_kv.cuh"

namespace cg = cooperative_groups;

namespace nf4 {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kMaxCluster = 8;
constexpr int kOne = 40;           // a weight of 1 is 2^40
constexpr float kFarthest = 41.0f; // in powers of 2: what lies further from the top has no weight
constexpr float kColdest = 0x1p-100f;  // a temperature below counts as 0

// 2^(40 - j / 1024), rounded.  exp by its series, in double precision at compile time.
struct PowerTable {
    unsigned long long e[1024];
};
constexpr PowerTable power_table() {
    PowerTable r{};
    for (int j = 0; j < 1024; j++) {
        const double x = -0.69314718055994530942 * j / 1024;
        double term = 1.0, sum = 1.0;
        for (int n = 1; n < 24; n++) {
            term *= x / n;
            sum += term;
        }
        r.e[j] = static_cast<unsigned long long>(sum * 1099511627776.0 + 0.5);
    }
    return r;
}
__device__ const PowerTable kPowers = power_table();

// What a row asks for, and its maximum.
struct Row {
    float top;           // the largest logit
    float c_hi, c_lo;    // log2(e) / T, as two floats
    float to_bin;        // bins per unit of distance from the top
};

// 2^40 exp((l - top) / T), to a few units.  log2(e) (top - l) / T = k / 1024 + r in two floats; 2^-k/1024 is a table's
// entry and a shift, 2^-r = 1 - q with q = p - p^2 / 2 + p^3 / 6, p = r ln 2 < 2^-11, in units of 2^-40.
__device__ __forceinline__ uint64_t weight_of(float l, const Row& row, const unsigned long long* table) {
    const float s = row.top - l, b = s - row.top;
    const float err = (row.top - (s - b)) - (l + b);  // top - l = s + err exactly
    const float y = s * row.c_hi;
    if (!(y < kFarthest)) return 0;
    const float y_lo = fmaf(s, row.c_hi, -y) + fmaf(s, row.c_lo, err * row.c_hi);
    const float z = fmaf(y, 1024.0f, 12582912.0f);  // 1.5 * 2^23: the sum's last bits are a whole number
    const int k = __float_as_int(z) - 0x4B400000;
    const float r = fmaf(z - 12582912.0f, -1.0f / 1024, y);  // exact
    const int ri = __float2int_rn(r * 0x1p41f) + __float2int_rn(y_lo * 0x1p41f);
    const int p = __mulhi(ri, 1488522236);                   // ln 2 * 2^31: units of 2^-40
    const int p2 = __mulhi(p, p);                            // p^2 in 2^-48
    const int q = p - (p2 >> 9) + ((__mulhi(p2, p) >> 16) / 6);
    const unsigned long long t = table[k & 1023];
    const uint64_t w = t - ((static_cast<int64_t>(static_cast<int>(t >> 10)) * q) >> 30);
    const int n = k >> 10;
    return n > 0 ? (w + (uint64_t{1} << (n - 1))) >> n : w;
}

// Unsigned keys in the order of the logits (-0 and 0 alike); NaN below everything.
__device__ __forceinline__ uint32_t key_of(float l) {
    const uint32_t u = __float_as_uint(l + 0.0f);
    return l != l ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// floor (or ceil) of f * s for f in [0, 1]; what is outside counts as the nearer end
__device__ __forceinline__ uint64_t fraction_of(float f, uint64_t s, bool up) {
    if (!(f > 0.0f)) return 0;
    f = fminf(f, 1.0f);
    const uint32_t bits = __float_as_uint(f);
    const int e = max(static_cast<int>(bits >> 23), 1);
    const uint64_t m = (bits & 0x7FFFFFu) | (bits >= 0x800000u ? 0x800000u : 0u);  // f = m 2^(e - 150)
    const int shift = 150 - e;                                                     // 23 or more
    const uint64_t lo = m * s, hi = __umul64hi(m, s);
    uint64_t whole, rest;
    if (shift < 64) {
        whole = (hi << (64 - shift)) | (lo >> shift);
        rest = lo << (64 - shift);
    } else if (shift < 128) {
        whole = shift == 64 ? hi : hi >> (shift - 64);
        rest = lo | (shift == 64 ? 0 : hi << (128 - shift));
    } else {
        whole = 0;
        rest = 1;
    }
    return whole + (up && rest ? 1 : 0);
}

struct Slot {
    unsigned long long a, b;
};

struct Shared {
    unsigned long long table[1024];
    unsigned long long weights[2][kBins];  // of the bins, one for each of two rounds that follow one another
    uint32_t counts[2][kBins];
    Slot slot[2];          // what this CTA tells the others
    Slot part[kWarps];
    unsigned long long found[4];
    Row row;
};

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max(v, static_cast<uint64_t>(__shfl_xor_sync(0xFFFFFFFFu, v, o)));
    return v;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

template <bool BF16>
__device__ __forceinline__ float value_at(const void* values, int i) {
    if (BF16) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(values)[i]) << 16);
    return static_cast<const float*>(values)[i];
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a, int per) {
    extern __shared__ __align__(16) uint8_t slice[];
    __shared__ Shared sh;
    constexpr int E = BF16 ? 2 : 4, VEC = 16 / E;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int64_t b = blockIdx.x / ranks;
    for (int i = tid; i < 1024; i += kThreads) sh.table[i] = kPowers.e[i];
    pdl_launch_dependents();
    pdl_wait();

    // the slice: elements e0 .. e1 of the row, behind `off` places so that 16-byte pieces stay aligned
    const int e0 = static_cast<int>(min(a.V, static_cast<int64_t>(rank) * per));
    const int e1 = static_cast<int>(min(a.V, static_cast<int64_t>(e0) + per));
    const uint8_t* src = static_cast<const uint8_t*>(a.logits) + (b * a.stride + e0) * E;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15) / E;
    const int places = e1 > e0 ? (off + (e1 - e0) + VEC - 1) / VEC * VEC : 0;
    uint64_t best = 0;  // the largest key, and the lowest index that has it
    for (int v = tid; v < places / VEC; v += kThreads) {
        const int p0 = v * VEC;
        union {
            uint4 u;
            uint16_t h[8];
            float f[4];
        } x;
        if (p0 >= off && p0 + VEC <= off + (e1 - e0)) {
            x.u = __ldcs(reinterpret_cast<const uint4*>(src + (p0 - off) * E));
        } else {
#pragma unroll
            for (int j = 0; j < VEC; j++) {
                const int i = p0 + j - off;
                const bool in = i >= 0 && i < e1 - e0;
                if (BF16)
                    x.h[j] = in ? reinterpret_cast<const uint16_t*>(src)[i] : 0xFF80u;
                else
                    x.f[j] = in ? reinterpret_cast<const float*>(src)[i] : __uint_as_float(0xFF800000u);
            }
        }
        reinterpret_cast<uint4*>(slice)[v] = x.u;
#pragma unroll
        for (int j = 0; j < VEC; j++) {
            const float l = BF16 ? __uint_as_float(static_cast<uint32_t>(x.h[j]) << 16) : x.f[j];
            const uint64_t at = (static_cast<uint64_t>(key_of(l)) << 32) | (0xFFFFFFFFu - (e0 + p0 + j - off));
            best = max(best, at);
        }
    }
    // sums over the row: every CTA's in two buffers by turns, one barrier each
    int turn = 0;
    auto reduce = [&](uint64_t x, uint64_t y, bool maximum, uint64_t* total_x, uint64_t* total_y) {
        x = maximum ? warp_max(x) : warp_sum(x);
        y = maximum ? warp_max(y) : warp_sum(y);
        if (lane == 0) sh.part[warp] = {x, y};
        __syncthreads();
        if (warp == 0) {
            Slot s = lane < kWarps ? sh.part[lane] : Slot{0, 0};
            const uint64_t sx = maximum ? warp_max(s.a) : warp_sum(s.a), sy = maximum ? warp_max(s.b) : warp_sum(s.b);
            if (lane == 0) sh.slot[turn] = {sx, sy};
        }
        cluster.sync();
        uint64_t rx = 0, ry = 0;
        for (int r = 0; r < ranks; r++) {
            const Slot s = *cluster.map_shared_rank(&sh.slot[turn], r);
            rx = maximum ? max(rx, static_cast<uint64_t>(s.a)) : rx + s.a;
            ry = maximum ? max(ry, static_cast<uint64_t>(s.b)) : ry + s.b;
        }
        turn ^= 1;
        *total_x = rx;
        if (total_y) *total_y = ry;
    };
    uint64_t top, unused;
    reduce(best, 0, true, &top, &unused);
    const uint32_t top_key = static_cast<uint32_t>(top >> 32);
    const int top_at = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(top));
    const float top_l = __uint_as_float((top_key & 0x80000000u) ? top_key ^ 0x80000000u : ~top_key);
    const float heat = a.temperature ? a.temperature[b] : 1.0f;
    // no logit above -inf: no token; +inf, or no heat: the first of the largest
    const bool none = top_key <= 0x007FFFFFu, greedy = !(heat >= kColdest) || top_l > 3.4028235e38f;
    int token = none ? -1 : top_at;
    float log_sum = 0.0f;
    if (a.logprobs && !none) {
        float sum = 0.0f;
        for (int i = tid; i < places; i += kThreads) sum += exp2f(fmaxf(value_at<BF16>(slice, i) - top_l, -1e30f) * 1.4426950408889634f);
        uint64_t total;
        reduce(static_cast<uint64_t>(static_cast<double>(sum) * 0x1p44), 0, false, &total, nullptr);
        log_sum = logf(static_cast<float>(static_cast<double>(total) * 0x1p-44));
    }
    if (!none && !greedy) {
        if (tid == 0) {
            const double c = 1.4426950408889634 / static_cast<double>(heat);
            sh.row.top = top_l;
            sh.row.c_hi = static_cast<float>(c);
            sh.row.c_lo = static_cast<float>(c - static_cast<double>(sh.row.c_hi));
            sh.row.to_bin = static_cast<float>(c) * (kBins / kFarthest);
        }
        __syncthreads();
        const Row row = sh.row;
        // the distance bin of a logit; logits without weight are past the last
        auto bin_of = [&](float l) {
            const float x = (row.top - l) * row.to_bin;
            return x < static_cast<float>(kBins) ? static_cast<int>(x) : kBins;
        };
        int round = 0;
        // One round: counts (and weights) of the elements that `in` puts into a bin, then the bin in which the sum
        // passes `want`, and the sum before it.  Every CTA adds the same numbers.  False: not passed at all.
        auto histogram = [&](auto in, bool weighted, uint64_t want, int* bin, uint64_t* before) {
            uint32_t* counts = sh.counts[round];
            unsigned long long* weights = sh.weights[round];
            for (int i = tid; i < kBins; i += kThreads) counts[i] = 0, weights[i] = 0;
            __syncthreads();
            for (int i = tid; i < places; i += kThreads) {
                const float l = value_at<BF16>(slice, i);
                const int at = in(l);
                if (at < 0 || at >= kBins) continue;
                if (weighted)
                    atomicAdd(&weights[at], static_cast<unsigned long long>(weight_of(l, row, sh.table)));
                else
                    atomicAdd(&counts[at], 1u);
            }
            cluster.sync();
            // two bins a thread, in order
            uint64_t v[2] = {0, 0};
            for (int r = 0; r < ranks; r++)
#pragma unroll
                for (int j = 0; j < 2; j++)
                    v[j] += weighted ? cluster.map_shared_rank(weights, r)[2 * tid + j]
                                     : cluster.map_shared_rank(counts, r)[2 * tid + j];
            const uint64_t mine = v[0] + v[1], upto = warp_scan(mine, lane);
            if (lane == 31) sh.part[warp].a = upto;
            if (tid == 0) sh.found[0] = kBins;
            __syncthreads();
            uint64_t ahead = upto - mine;
            for (int w = 0; w < warp; w++) ahead += sh.part[w].a;
            if (ahead < want && ahead + mine >= want) {
                const int j = ahead + v[0] >= want ? 0 : 1;
                sh.found[0] = 2 * tid + j;
                sh.found[1] = ahead + (j ? v[0] : 0);
            }
            __syncthreads();
            *bin = static_cast<int>(sh.found[0]);
            *before = sh.found[1];
            __syncthreads();
            round ^= 1;
            return *bin < kBins;
        };
        // The key at which the sum over the ordered elements with lowest < key passes `want`, and the sum above it.
        // False: it never does.
        auto select = [&](bool weighted, uint64_t want, uint32_t lowest, uint32_t* key, uint64_t* before) {
            int first = 0;
            uint64_t sum = 0, more = 0;
            if (!histogram([&](float l) { return key_of(l) > lowest ? bin_of(l) : -1; }, weighted, want, &first, &sum))
                return false;
            // the keys of that bin, then ever narrower ranges of keys
            uint64_t hi = 0, lo = 0;
            for (int i = tid; i < places; i += kThreads) {
                const float l = value_at<BF16>(slice, i);
                if (key_of(l) > lowest && bin_of(l) == first) {
                    hi = max(hi, static_cast<uint64_t>(key_of(l)));
                    lo = max(lo, static_cast<uint64_t>(0xFFFFFFFFu - key_of(l)));
                }
            }
            reduce(hi, lo, true, &hi, &lo);
            uint32_t high = static_cast<uint32_t>(hi), low = 0xFFFFFFFFu - static_cast<uint32_t>(lo);
            while (low < high) {
                const int bits = 32 - __clz(high - low), shift = bits > 10 ? bits - 10 : 0;
                int at = 0;
                histogram(
                    [&](float l) {
                        const uint32_t k = key_of(l);
                        return k >= low && k <= high ? static_cast<int>((high - k) >> shift) : -1;
                    },
                    weighted, want - sum, &at, &more);
                sum += more;
                high -= static_cast<uint32_t>(at) << shift;
                low = shift == 0 ? high : max(low, high - ((1u << shift) - 1));
            }
            *key = high;
            *before = sum;
            return true;
        };
        uint32_t cut = 0;                   // elements with larger keys are kept
        uint64_t ties = ~uint64_t{0};       // and so many of those with this key
        auto logit_of = [](uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k); };
        // -inf and NaN have no weight: they are never kept
        constexpr uint32_t kNothing = 0x007FFFFFu;
        cut = kNothing, ties = 0;
        const int k = a.top_k ? a.top_k[b] : 0;
        if (k > 0 && k < a.V) {
            uint32_t key;
            uint64_t before;
            if (select(false, static_cast<uint64_t>(k), kNothing, &key, &before)) cut = key, ties = k - before;
        }
        const float p = a.top_p ? a.top_p[b] : 1.0f;
        if (p < 1.0f) {
            uint64_t above = 0, at = 0;
            for (int i = tid; i < places; i += kThreads) {
                const float l = value_at<BF16>(slice, i);
                if (key_of(l) > cut) above += weight_of(l, row, sh.table);
            }
            reduce(above, 0, false, &above, &at);
            const uint64_t of_tie = ties ? weight_of(logit_of(cut), row, sh.table) : 0;
            const uint64_t all = above + ties * of_tie;
            const uint64_t want = max(fraction_of(p, all, true), uint64_t{1});
            if (want > above) {  // of the tied ones, those with less than `want` before them
                if (of_tie) ties = min(ties, (want - above + of_tie - 1) / of_tie);
            } else {
                uint32_t key;
                uint64_t before;
                select(true, want, cut, &key, &before);
                const uint64_t w = weight_of(logit_of(key), row, sh.table);
                cut = key;
                ties = w ? (want - before + w - 1) / w : 1;
            }
        }
        const float least_p = a.min_p ? a.min_p[b] : 0.0f;
        // at least the largest stays
        const uint64_t least =
            least_p >= 1.0f ? uint64_t{1} << kOne : max(fraction_of(least_p, uint64_t{1} << kOne, true), uint64_t{1});
        // Each warp takes a run of the slice; a run's sum is that of what lies above the cut, and of as many tied
        // elements as the runs before it leave.
        const int run = ((places + kWarps - 1) / kWarps + 31) / 32 * 32;
        const int r0 = min(places, warp * run), r1 = min(places, r0 + run);
        uint64_t sum = 0, tied = 0;
        const uint64_t of_tie = ties ? weight_of(logit_of(cut), row, sh.table) : 0;
        const bool tie_counts = of_tie >= least;
        for (int i = r0 + lane; i < r1; i += 32) {
            const float l = value_at<BF16>(slice, i);
            const uint32_t key = key_of(l);
            if (key > cut) {
                const uint64_t w = weight_of(l, row, sh.table);
                sum += w >= least ? w : 0;
            } else if (key == cut) {
                tied++;
            }
        }
        sum = warp_sum(sum);
        tied = warp_sum(tied);
        if (lane == 0) sh.part[warp] = {sum, tied};
        __syncthreads();
        if (tid == 0) {
            Slot s{0, 0};
            for (int w = 0; w < kWarps; w++) s.a += sh.part[w].a, s.b += sh.part[w].b;
            sh.slot[turn] = s;
        }
        cluster.sync();
        uint64_t ahead = 0, tied_ahead = 0, total = 0;
        {
            uint64_t seen = 0;
            for (int r = 0; r < ranks; r++) {
                const Slot s = *cluster.map_shared_rank(&sh.slot[turn], r);
                if (r == rank) ahead = total, tied_ahead = seen;
                const uint64_t kept = tie_counts ? min(static_cast<uint64_t>(s.b), ties - min(ties, seen)) : 0;
                total += s.a + kept * of_tie;
                seen += s.b;
            }
            turn ^= 1;
        }
        const uint64_t goal = min(fraction_of(a.random[b], total, false), total - 1);
        for (int w = 0; w < warp; w++) {
            const Slot s = sh.part[w];
            const uint64_t kept = tie_counts ? min(static_cast<uint64_t>(s.b), ties - min(ties, tied_ahead)) : 0;
            ahead += s.a + kept * of_tie;
            tied_ahead += s.b;
        }
        const uint64_t kept = tie_counts ? min(tied, ties - min(ties, tied_ahead)) : 0;
        if (tid == 0) sh.found[0] = ~0ull;
        __syncthreads();
        if (goal >= ahead && goal < ahead + sum + kept * of_tie) {  // this warp's run has the token
            for (int i0 = r0; i0 < r1; i0 += 32) {
                const int i = i0 + lane;
                uint64_t w = 0;
                const float l = i < r1 ? value_at<BF16>(slice, i) : __uint_as_float(0xFF800000u);
                const uint32_t key = key_of(l);
                const uint32_t equal = __ballot_sync(0xFFFFFFFFu, i < r1 && key == cut);
                if (i < r1 && key > cut) {
                    w = weight_of(l, row, sh.table);
                    if (w < least) w = 0;
                } else if (i < r1 && key == cut && tie_counts &&
                           tied_ahead + __popc(equal & ((1u << lane) - 1)) < ties) {
                    w = of_tie;
                }
                const uint64_t upto = ahead + warp_scan(w, lane);
                const uint32_t passed = __ballot_sync(0xFFFFFFFFu, upto > goal);
                if (passed) {
                    if (lane == __ffs(passed) - 1) sh.found[0] = static_cast<unsigned long long>(e0 + i - off);
                    break;
                }
                ahead = __shfl_sync(0xFFFFFFFFu, upto, 31);
                tied_ahead += __popc(equal);
            }
        }
        __syncthreads();
        if (tid == 0 && sh.found[0] != ~0ull) {
            const int i = static_cast<int>(sh.found[0]);
            a.tokens[b] = i;
            if (a.logprobs) a.logprobs[b] = (value_at<BF16>(slice, i - e0 + off) - top_l) - log_sum;
        }
    } else if (rank == 0 && tid == 0) {
        a.tokens[b] = token;
        if (a.logprobs) a.logprobs[b] = none ? __uint_as_float(0xFF800000u) : 0.0f - log_sum;
    }
    cluster.sync();  // no CTA leaves while another may read from it
}

template <bool BF16>
cudaError_t sample(const SampleArgs& a, int num_sms, cudaStream_t stream) {
    constexpr int E = BF16 ? 2 : 4;
    static std::once_flag once[64];
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    constexpr int kMost = static_cast<int>(kSampleMaxVocab / kMaxCluster * E + 32);
    std::call_once(once[device & 63], [&] {
        e = cudaFuncSetAttribute(sample_kernel<BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    });
    if (e != cudaSuccess) return e;
    int ranks = 1;
    while (ranks < kMaxCluster && a.V > 4096 * ranks) ranks *= 2;
    const int per = static_cast<int>(((a.V + ranks - 1) / ranks + 7) / 8 * 8);
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(a.B * ranks)), kThreads, stream, attr);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(ranks), 1, 1};
    cfg.numAttrs = 2;
    cfg.dynamicSmemBytes = static_cast<size_t>(per) * E + 32;
    (void)num_sms;
    return cudaLaunchKernelEx(&cfg, sample_kernel<BF16>, a, per);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, int num_sms, cudaStream_t stream) {
    return a.bf16 ? sample<true>(a, num_sms, stream) : sample<false>(a, num_sms, stream);
}

}  // namespace nf4
