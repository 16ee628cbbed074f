// The next token of every row of logits.
//
// With z_i = (l_i - max l) / T, the weight of token i is w_i = exp(z_i).  Top-k, top-p and min-p each keep a
// beginning of the tokens ordered by logit (ties: the lower index first); the token drawn is the first index i, in
// index order, at which the sum of the kept weights up to i passes u times their whole sum.
//
// Sums are exact: a weight is a whole number of 2^-40 (within 1.1 * 2^-30 of its own size of the exponential, or half
// a unit), and sums of up to 2^18 of them fit 64 bits.  So no order of addition, number of CTAs or atomic changes a
// result, and since the weights' errors do not add up (each is rounded by itself), the border between two of 150,000
// equal tokens is within some 10^-5 of a token of where the formula has it; sums in fp32 move it by hundredths.
//
// A row is held by the CTAs of one cluster, a slice of it in the shared memory of each, so the logits are read once
// from memory; what a row needs next (its maximum, where the order is cut, which slice the token is in)
// is exchanged through distributed shared memory.
//
// What bounds it: for few rows the chain of steps between barriers (one row of 151936 bf16 logits, top-k 50: 9.9 us, 0.05 of
// it the bytes); for many the instructions of the passes over a slice and those steps, of two CTAs an SM (256 such rows
// 55.8 us, 11.7 of it the bytes: issue slots 36%; 128 rows in fp32 without cuts, a weight and an exponential for each of
// their 19 million logits, 89 us: 83 instructions a logit, which fill half of the issue slots, and the CTAs' waits for one
// another; 81 without logprobs).
#include <cooperative_groups.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "nf4_kv.cuh"

namespace cg = cooperative_groups;

namespace nf4 {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1024;  // two a thread
constexpr int kMaxCluster = 8;
constexpr int kList = 2048;            // candidates that a row's cut is found among
constexpr int kFewBins = 256;          // eight a lane
constexpr int kFewest = 128;           // top_k up to this may take the short way (256 rows of top-k 50: 198 -> 56 us)
constexpr int kSliceBytes = 80 * 1024; // of a slice, for two CTAs an SM
constexpr int kOne = 40;               // a weight of 1 is 2^40
constexpr float kFarthest = 41.0f;     // in powers of 2: what lies further from the top has no weight
constexpr float kColdest = 0x1p-100f;  // a temperature below counts as 0

// 2^(31 - j / 1024), rounded.  exp by its series, in double precision at compile time.
struct alignas(16) PowerTable {
    uint32_t e[1024];
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
        r.e[j] = static_cast<uint32_t>(sum * 2147483648.0 + 0.5);
    }
    return r;
}
__device__ const PowerTable kPowers = power_table();

// Two floats in one register pair, for the instructions that work on both.
struct Pair {
    unsigned long long v;
    __device__ __forceinline__ Pair(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ explicit Pair(float a) : Pair(a, a) {}
    __device__ __forceinline__ float2 get() const {
        float2 f;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
        return f;
    }
};
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(a.v) : "l"(a.v), "l"(b.v));
    return a;
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(a.v) : "l"(a.v), "l"(b.v));
    return a;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(a.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return a;
}

// What a row asks for, and its maximum.
struct Row {
    float top;         // the largest logit
    float c_hi, c_lo;  // log2(e) / T, as two floats
    float to_bin;      // bins per unit of distance from the top
};

// 2^40 exp((l - top) / T) of two logits.  y = log2(e) (top - l) / T, in two floats, is k / 1024 + r; 2^(-k / 1024)
// is a table's entry and a shift, 2^-r = 1 - p + p^2 / 2 with p = r ln 2 < 2^-11.5 (the next term is below 2^-37).  The
// entry and the correction are rounded to 31 bits, half of 2^-30 each, and fp32 adds a tenth: 1.1 * 2^-30.
__device__ __forceinline__ void weights_of(float l0, float l1, const Row& row, const uint32_t* table, uint64_t (&w)[2]) {
    const Pair l(l0, l1), top(row.top), minus(-1.0f), c_hi(row.c_hi);
    const Pair s = fma2(l, minus, top), b = s + Pair(-row.top);
    const Pair err = fma2(l + b, minus, fma2(fma2(b, minus, s), minus, top));  // top - l = s + err exactly
    const Pair y = s * c_hi;
    const Pair y_lo = fma2(err, c_hi, fma2(s, Pair(row.c_lo), fma2(s, c_hi, s * Pair(-row.c_hi))));
    const Pair z = fma2(y, Pair(1024.0f), Pair(12582912.0f));  // 1.5 * 2^23: the sum's last bits are k
    const Pair r = fma2(z + Pair(-12582912.0f), Pair(-1.0f / 1024), y) + y_lo;
    const Pair p = r * Pair(0.6931471805599453f * 0x1p41f);
    const float2 q = fma2(p, p * Pair(-0x1p-42f), p).get(), zs = z.get(), ys = y.get();
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const uint32_t k = __float_as_uint(j ? zs.y : zs.x), n = (k >> 10) & 63u;  // (1.5 * 2^23 adds no bit to either)
        const uint32_t t = table[k & 1023u];
        // (rounded: cut, the weights were too large by 0.35 * 2^-30 on average, and by up to 1.5 * 2^-30)
        const uint32_t m = t - ((__mulhi(static_cast<int>(t >> 1), __float2int_rn(j ? q.y : q.x)) + 128) >> 8);
        uint64_t v;
        if (n >= 10)
            v = (static_cast<uint64_t>(m) * (1u << ((41u - n) & 31u)) + 0x80000000u) >> 32;
        else
            v = ((static_cast<uint64_t>(m) << 10 >> n) + 1) >> 1;
        w[j] = (j ? ys.y : ys.x) < kFarthest ? v : 0;  // (false for -inf, too)
    }
}
__device__ __forceinline__ uint64_t weight_of(float l, const Row& row, const uint32_t* table) {
    uint64_t w[2];
    weights_of(l, l, row, table, w);
    return w[0];
}

// Unsigned keys in the order of the logits (-0 and 0 alike).
__device__ __forceinline__ uint32_t key_of(float l) {
    const uint32_t u = __float_as_uint(l + 0.0f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
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

// What a CTA tells the others: its largest logit, how many have it, the sum of exp(l - that) over the rest, an index or
// a line that top_k of its logits reach, and how many reach that.
struct alignas(16) Note {
    float top, sum;
    int32_t at, count, tops;
};
struct alignas(16) Shared {  // the slice follows, in 16-byte pieces
    uint32_t table[1024];
    uint32_t low[kBins], high[kBins];  // of the bins: counts, or weights in two words
    unsigned long long list[kList];    // candidates: key and index, or keys; sums before candidates
    Note notes[2][kMaxCluster];
    unsigned long long sums[kMaxCluster][2];
    unsigned long long part[kWarps][2];
    float fpart[kWarps][2];
    int32_t tops[kWarps];
    unsigned long long found[2];
    uint32_t count, line;
    float log_sum;
};

static_assert(sizeof(Shared) % 16 == 0, "the slice's pieces are aligned");

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
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
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

constexpr uint32_t kNothing = 0x007FFFFFu;  // the key of -inf
__device__ __forceinline__ float minus_inf() { return __uint_as_float(0xFF800000u); }

// Slices hold no NaN (loading makes them -inf).
template <bool BF16>
__device__ __forceinline__ float value_at(const void* values, int i) {
    if (BF16) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(values)[i]) << 16);
    return static_cast<const float*>(values)[i];
}

// 16 bytes of logits: without NaN, their maximum, and each as a float.
template <bool BF16>
struct Piece {
    uint32_t w[4];
    __device__ __forceinline__ explicit Piece(const uint4& u) : w{u.x, u.y, u.z, u.w} {}
    __device__ __forceinline__ static uint32_t larger(uint32_t a, uint32_t b) {
        uint32_t r;
        if (BF16)
            asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        else
            asm("max.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static constexpr uint32_t kLeast = BF16 ? 0xFF80FF80u : 0xFF800000u;
    __device__ __forceinline__ void clean() {
#pragma unroll
        for (int j = 0; j < 4; j++) w[j] = larger(w[j], kLeast);
    }
    __device__ __forceinline__ uint32_t top() const { return larger(larger(w[0], w[1]), larger(w[2], w[3])); }
    __device__ __forceinline__ static float single(uint32_t m) {
        return BF16 ? fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u)) : __uint_as_float(m);
    }
    __device__ __forceinline__ float operator[](int j) const {
        if (!BF16) return __uint_as_float(w[j]);
        return __uint_as_float((j & 1) ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
    }
};

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a, int per) {
    extern __shared__ __align__(16) uint8_t memory[];
    Shared& sh = *reinterpret_cast<Shared*>(memory);
    uint8_t* slice = memory + sizeof(Shared);
    constexpr int E = BF16 ? 2 : 4, VEC = 16 / E;
    using P = Piece<BF16>;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int64_t b = blockIdx.x / ranks;
    for (int i = tid; i < kBins; i += kThreads) sh.low[i] = 0;
    reinterpret_cast<uint2*>(sh.table)[tid] = reinterpret_cast<const uint2*>(kPowers.e)[tid];
    if (tid == 0) sh.count = 0;
    cluster.barrier_arrive();  // no CTA writes to another before that one has begun
    pdl_launch_dependents();
    pdl_wait();

    // the slice: elements e0 .. e1 of the row, behind `off` places so that 16-byte pieces stay aligned
    const int e0 = static_cast<int>(min(a.V, static_cast<int64_t>(rank) * per));
    const int e1 = static_cast<int>(min(a.V, static_cast<int64_t>(e0) + per));
    const uint8_t* src = static_cast<const uint8_t*>(a.logits) + (b * a.stride + e0) * E;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15) / E;
    const int places = e1 > e0 ? (off + (e1 - e0) + VEC - 1) / VEC * VEC : 0, pieces = places / VEC;
    const float heat = a.temperature ? a.temperature[b] : 1.0f, top_p = a.top_p ? a.top_p[b] : 1.0f;
    const float min_p = a.min_p ? a.min_p[b] : 0.0f, random = a.random[b];
    const int k = a.top_k ? a.top_k[b] : 0;
    float mine;  // the largest of this thread's pieces: tid, tid + kThreads, ...
    {
        uint32_t best = P::kLeast;
        auto keep = [&](int v, const uint4& u) {
            P p(u);
            p.clean();
            best = P::larger(best, p.top());
            reinterpret_cast<uint4*>(slice)[v] = make_uint4(p.w[0], p.w[1], p.w[2], p.w[3]);
        };
        const int v0 = off ? 1 : 0, v1 = (off + (e1 - e0)) / VEC;  // whole pieces
        const uint4* whole = reinterpret_cast<const uint4*>(src - off * E);
        int v = tid < v0 ? tid + kThreads : tid;
        for (; v + 3 * kThreads < v1; v += 4 * kThreads) {
            uint4 u[4];
#pragma unroll
            for (int j = 0; j < 4; j++) u[j] = __ldcs(whole + v + j * kThreads);
#pragma unroll
            for (int j = 0; j < 4; j++) keep(v + j * kThreads, u[j]);
        }
        for (; v < v1; v += kThreads) keep(v, __ldcs(whole + v));
        // the pieces at the ends, where the row begins or ends inside one
        for (int end = 0; end < 2; end++) {
            const int at = end ? v1 : 0;
            if (tid != at % kThreads || at >= pieces || (at >= v0 && at < v1) || (end && at == 0)) continue;
            uint32_t w[4] = {P::kLeast, P::kLeast, P::kLeast, P::kLeast};
#pragma unroll
            for (int j = 0; j < VEC; j++) {
                const int i = at * VEC + j - off;
                if (i < 0 || i >= e1 - e0) continue;
                if (BF16)
                    w[j / 2] = (w[j / 2] & (j & 1 ? 0x0000FFFFu : 0xFFFF0000u)) |
                               (static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(src)[i]) << (16 * (j & 1)));
                else
                    w[j] = reinterpret_cast<const uint32_t*>(src)[i];
            }
            keep(at, make_uint4(w[0], w[1], w[2], w[3]));
        }
        mine = P::single(best);
    }
    auto block_ends = [&](float hi, float lo, float* out_hi, float* out_lo) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
            lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
        }
        if (lane == 0) sh.fpart[warp][0] = hi, sh.fpart[warp][1] = lo;
        __syncthreads();
        hi = sh.fpart[lane % kWarps][0], lo = sh.fpart[lane % kWarps][1];
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1) {
            hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
            lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
        }
        *out_hi = hi, *out_lo = lo;
        __syncthreads();
    };
    // Short way, for small top_k: a line that at least k logits of the slice reach, and few more do.  It is the k-th of
    // the largest logits of single threads, as far as the m largest of every warp's tell (m twice the mean number
    // of the first k that a warp has, or more).  Where fewer than k threads of a slice have a logit that is not masked, every
    // place reaches the line and the row goes the long way (256 rows of top-k 50: 56 us, 199 with 100 tokens allowed).
    const bool cold = !(heat >= kColdest);
    const bool few = !cold && k > 0 && k <= kFewest && k < a.V;
    const int m = k <= 64 ? 8 : 16, known = m * kWarps;
    if (few) {
        uint32_t key = key_of(mine);
        for (int i = 0; i < m; i++) {
            const uint32_t largest = __reduce_max_sync(0xFFFFFFFFu, key);
            if (lane == 0) sh.high[warp * m + i] = largest;
            if (key == largest) key = 0;  // (equal ones fall together: more reach the line)
        }
        if (tid == 0) sh.line = 0xFFFFFFFFu;
    }
    float top_here, unused_end;  // the slice's largest logit
    block_ends(mine, 0.0f, &top_here, &unused_end);
    float line = cold ? top_here : __uint_as_float(0x7F800000u);
    if (few) {
        const int parts = kThreads / known, part = tid % parts;
        const uint32_t own = sh.high[tid / parts];
        int larger = 0;
#pragma unroll 8
        for (int j = part; j < known / 4; j += parts) {
            const uint4 o = reinterpret_cast<const uint4*>(sh.high)[j];
            larger += (o.x > own) + (o.y > own) + (o.z > own) + (o.w > own);
        }
        for (int o = 1; o < parts; o *= 2) larger += __shfl_xor_sync(0xFFFFFFFFu, larger, o);
        // the least value with fewer than k larger ones
        const uint32_t lowest_own = __reduce_min_sync(0xFFFFFFFFu, larger < k ? own : 0xFFFFFFFFu);
        if (lane == 0 && lowest_own != 0xFFFFFFFFu) atomicMin(&sh.line, lowest_own);
        __syncthreads();
        line = sh.line <= kNothing ? minus_inf() : logit_of(sh.line);
    }
    cluster.barrier_wait();
    const int room_log = 31 - __clz(kList / ranks), room = 1 << room_log;  // of the list, for each CTA
    float sum = 0.0f;
    int first = 0x7FFFFFFF, tops = 0;
    if (top_here > minus_inf() && (a.logprobs || few || cold)) {
        unsigned long long* list = cluster.map_shared_rank(sh.list, 0) + rank * room;
        const Pair minus_top(-top_here), log2e(1.4426950408889634f);
        Pair sums(0.0f);
        auto power = [&](const P& p, int j) {
            float2 e = ((Pair(p[j], p[j + 1]) + minus_top) * log2e).get();
            asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
            asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
            return e;
        };
        for (int v = tid; v < pieces; v += kThreads) {
            const P p(reinterpret_cast<const uint4*>(slice)[v]);
            const float most = P::single(p.top());
            if (a.logprobs) {
                if (most < top_here) {
#pragma unroll
                    for (int j = 0; j < VEC; j += 2) {
                        const float2 e = power(p, j);
                        sums = sums + Pair(e.x, e.y);
                    }
                } else {
                    // The largest logits are counted, not added: next to their 1 a small rest would lose its last
                    // bits, and with them the logarithm of a probability near 1.
#pragma unroll
                    for (int j = 0; j < VEC; j += 2) {
                        const float2 e = power(p, j);
                        tops += (p[j] == top_here) + (p[j + 1] == top_here);
                        sum += (p[j] == top_here ? 0.0f : e.x) + (p[j + 1] == top_here ? 0.0f : e.y);
                    }
                }
            }
            if (!(most >= line)) continue;
            const int i0 = e0 + v * VEC - off;
            uint32_t reach = 0;
#pragma unroll
            for (int j = 0; j < VEC; j++) reach |= (p[j] >= line ? 1u : 0u) << j;
            if (cold) {
                first = min(first, i0 + __ffs(reach) - 1);
                continue;
            }
            uint32_t at = atomicAdd(&sh.count, __popc(reach));
            for (; reach; reach &= reach - 1, at++) {
                const int j = __ffs(reach) - 1;
                const uint32_t low_word = j & (VEC / 4) ? p.w[1] : p.w[0], high_word = j & (VEC / 4) ? p.w[3] : p.w[2];
                const uint32_t word = j & (VEC / 2) ? high_word : low_word;
                const float l = __uint_as_float(!BF16 ? word : j & 1 ? word & 0xFFFF0000u : word << 16);
                if (at < static_cast<uint32_t>(room))
                    list[at] = (static_cast<unsigned long long>(key_of(l)) << 32) | (0xFFFFFFFFu - (i0 + j));
            }
        }
        sum += sums.get().x + sums.get().y;
    }
    {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        first = __reduce_min_sync(0xFFFFFFFFu, first);
        tops = __reduce_add_sync(0xFFFFFFFFu, tops);
        if (lane == 0) sh.fpart[warp][0] = sum, sh.fpart[warp][1] = __int_as_float(first), sh.tops[warp] = tops;
        __syncthreads();
        if (warp == 0) {
            sum = lane < kWarps ? sh.fpart[lane][0] : 0.0f;
            first = __reduce_min_sync(0xFFFFFFFFu, __float_as_int(sh.fpart[lane % kWarps][1]));
            tops = __reduce_add_sync(0xFFFFFFFFu, lane < kWarps ? sh.tops[lane] : 0);
#pragma unroll
            for (int o = kWarps / 2; o > 0; o >>= 1) sum += __shfl_down_sync(0xFFFFFFFFu, sum, o);
            sum = __shfl_sync(0xFFFFFFFFu, sum, 0);
            if (lane < ranks)
                cluster.map_shared_rank(&sh, lane)->notes[0][rank] = {top_here, sum, few ? __float_as_int(line) : first,
                                                                      static_cast<int32_t>(sh.count), tops};
        }
    }
    cluster.sync();
    float top = minus_inf(), lowest = minus_inf();  // of the row; at least k of its logits reach `lowest`
    bool fits = true;
    int arg = 0x7FFFFFFF;
    for (int r = 0; r < ranks; r++) {
        const Note n = sh.notes[0][r];
        if (n.top > top) top = n.top, arg = n.at;
        fits &= n.count <= room;
        lowest = fmaxf(lowest, __int_as_float(n.at));  // (of use where they are lines)
    }
    auto log_of_sum = [&] {
        float rest = 0.0f, ones = 0.0f;
        for (int r = 0; r < ranks; r++) {
            const Note n = sh.notes[0][r];
            const float tops = static_cast<float>(n.tops);
            if (n.top == top)
                ones += tops, rest += n.sum;
            else if (n.top > minus_inf())
                rest += (tops + n.sum) * exp2f((n.top - top) * 1.4426950408889634f);
        }
        return log1pf(rest / ones) + logf(ones);
    };
    // one thread; the others have seen sh.log_sum written
    auto finish = [&](int token, float logit) {
        a.tokens[b] = token;
        if (a.logprobs) a.logprobs[b] = token < 0 ? minus_inf() : (logit == top ? 0.0f : logit - top) - sh.log_sum;
    };
    if (top == minus_inf() || cold) {  // no token, or the first of the largest
        if (rank == 0 && tid == 0) {
            if (a.logprobs) sh.log_sum = log_of_sum();
            finish(top == minus_inf() ? -1 : arg, top);
        }
        return;
    }
    if (top == __uint_as_float(0x7F800000u)) {  // the first of the infinite ones
        int at = 0x7FFFFFFF;
        for (int i = tid; i < places; i += kThreads)
            if (value_at<BF16>(slice, i) == top) at = min(at, e0 + i - off);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) at = min(at, __shfl_xor_sync(0xFFFFFFFFu, at, o));
        if (lane == 0) sh.fpart[warp][0] = __int_as_float(at);
        __syncthreads();
        if (tid < ranks) {
            for (int w = 0; w < kWarps; w++) at = min(at, __float_as_int(sh.fpart[w][0]));
            cluster.map_shared_rank(&sh, tid)->notes[1][rank].at = at;
        }
        cluster.sync();
        if (rank == 0 && tid == 0) {
            for (int r = 0; r < ranks; r++) at = min(at, sh.notes[1][r].at);
            if (a.logprobs) sh.log_sum = log_of_sum();
            finish(at, top);
        }
        return;
    }
    const bool listed = few && fits;
    if (listed && rank != 0) return;
    if (a.logprobs && tid == kThreads - 1) sh.log_sum = log_of_sum();  // barriers follow before it is used
    // The bin in which the counts (or weights) of the bins, two a thread, pass `want`, and their sum before it; kBins if
    // they do not.
    auto passed = [&](uint64_t v0, uint64_t v1, uint64_t want, uint64_t* before) {
        const uint64_t both = v0 + v1, upto = warp_scan(both, lane);
        if (lane == 31) sh.part[warp][0] = upto;
        if (tid == 0) sh.found[0] = kBins, sh.found[1] = 0;
        __syncthreads();
        uint64_t ahead = upto - both;
        for (int w = 0; w < warp; w++) ahead += sh.part[w][0];
        if (ahead < want && ahead + both >= want) {
            const int j = ahead + v0 >= want ? 0 : 1;
            sh.found[0] = 2 * tid + j;
            sh.found[1] = ahead + (j ? v0 : 0);
        }
        __syncthreads();
        *before = sh.found[1];
        const int bin = static_cast<int>(sh.found[0]);
        __syncthreads();
        return bin;
    };
    // log2(e) / T in two floats: the quotient, and what its remainder gives
    Row row;
    row.top = top;
    row.c_hi = __fdiv_rn(1.4426950216293335f, heat);
    const float rest = fmaf(-row.c_hi, heat, 1.4426950216293335f) + 1.9259629911266175e-8f;
    row.c_lo = row.c_hi > 0.0f ? __fdividef(rest, heat) : 0.0f;
    row.to_bin = row.c_hi * (kBins / kFarthest);
    const uint64_t least =
        min_p >= 1.0f ? uint64_t{1} << kOne : max(fraction_of(min_p, uint64_t{1} << kOne, true), uint64_t{1});
    auto block_sum = [&](uint64_t x) {
        x = warp_sum(x);
        if (lane == 0) sh.part[warp][0] = x;
        __syncthreads();
        uint64_t s = 0;
        for (int w = 0; w < kWarps; w++) s += sh.part[w][0];
        __syncthreads();
        return s;
    };
    if (listed) {
        // Of the candidates, those in the bins that hold the first k; then all pairs of these, eight threads each.
        unsigned long long* names = reinterpret_cast<unsigned long long*>(slice);
        unsigned long long* weights = names + kList;
        // (a name: key and index, so that larger names stand first)
        auto listed_at = [&](int e) {
            const bool in = (e & (room - 1)) < sh.notes[0][e >> room_log].count;
            const unsigned long long name = in ? sh.list[e] : 0;
            return static_cast<uint32_t>(name >> 32) >= max(key_of(lowest), kNothing + 1) ? name : 0ull;
        };
        if (lowest == minus_inf()) {  // all the CTAs have fewer logits than lines ask for
            float least_one = top, ignored;
            for (int e = tid; e < kList; e += kThreads) {
                const unsigned long long name = listed_at(e);
                if (name) least_one = fminf(least_one, logit_of(static_cast<uint32_t>(name >> 32)));
            }
            block_ends(0.0f, least_one, &ignored, &lowest);
        }
        if (tid == 0) sh.count = 0;
        const float to_bin = (kFewBins - 0.5f) / fmaxf(top - lowest, 1e-30f);
        auto bin_of = [&](unsigned long long name) {
            return min(kFewBins - 1, static_cast<int>((top - logit_of(static_cast<uint32_t>(name >> 32))) * to_bin));
        };
#pragma unroll
        for (int e = 0; e < kList; e += kThreads) {
            const unsigned long long name = listed_at(e + tid);
            if (name) atomicAdd(&sh.low[bin_of(name)], 1u);
        }
        __syncthreads();
        // every warp for itself: the bin that the first k reach
        int last;
        {
            uint32_t in_bins[8], all = 0;
#pragma unroll
            for (int j = 0; j < 8; j++) all += in_bins[j] = sh.low[8 * lane + j];
            uint32_t upto = all;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                if (lane >= o) upto += u;
            }
            upto -= all;
            int bin = kFewBins - 1;
#pragma unroll
            for (int j = 7; j >= 0; j--) {
                all -= in_bins[j];
                if (upto + all < static_cast<uint32_t>(k) && upto + all + in_bins[j] >= static_cast<uint32_t>(k))
                    bin = 8 * lane + j;
            }
            last = __reduce_min_sync(0xFFFFFFFFu, bin);
        }
#pragma unroll 1
        for (int e = tid; e < kList; e += kThreads) {
            const unsigned long long name = listed_at(e);
            if (!name || bin_of(name) > last) continue;
            const uint32_t at = atomicAdd(&sh.count, 1u);
            names[at] = name;
            weights[at] = weight_of(logit_of(static_cast<uint32_t>(name >> 32)), row, sh.table);
        }
        __syncthreads();
        const int n = static_cast<int>(sh.count), sub = tid % 8;
        // what stands before each; the sum of the first k
        unsigned long long* before = sh.list;  // (no longer needed)
        for (int i = tid / 8; i < (n + 63) / 64 * 64; i += kThreads / 8) {
            const unsigned long long name = i < n ? names[i] : ~0ull;
            int place = 0;
            uint64_t weight = 0;
            for (int j = sub; j < n; j += 8)
                if (names[j] > name) place++, weight += weights[j];
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) {
                place += __shfl_xor_sync(0xFFFFFFFFu, place, o);
                weight += __shfl_xor_sync(0xFFFFFFFFu, weight, o);
            }
            if (i < n && sub == 0) {
                before[i] = place < k ? weight : ~0ull;
                if (place == min(k, n) - 1) sh.found[0] = weight + weights[i];
            }
        }
        __syncthreads();
        const uint64_t want =
            top_p < 1.0f ? max(fraction_of(top_p, sh.found[0], true), uint64_t{1}) : ~uint64_t{0};
        uint64_t kept = 0;
        for (int i = sub == 0 ? tid / 8 : n; i < n; i += kThreads / 8) {
            const uint64_t w = before[i] >= want || weights[i] < least ? 0 : weights[i];
            weights[i] = w;
            kept += w;
        }
        kept += __shfl_xor_sync(0xFFFFFFFFu, kept, 8);
        kept += __shfl_xor_sync(0xFFFFFFFFu, kept, 16);
        if (lane == 0) sh.part[warp][0] = kept;
        __syncthreads();
        kept = 0;
#pragma unroll
        for (int w = 0; w < kWarps; w++) kept += sh.part[w][0];
        const uint64_t goal = min(fraction_of(random, kept, false), kept - 1);
        for (int i = tid / 8; i < (n + 63) / 64 * 64; i += kThreads / 8) {
            // (the lower half of a name falls as the index rises)
            const uint32_t name = i < n ? static_cast<uint32_t>(names[i]) : 0;
            uint64_t ahead = 0;
            for (int j = sub; j < n; j += 8)
                if (static_cast<uint32_t>(names[j]) > name) ahead += weights[j];
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) ahead += __shfl_xor_sync(0xFFFFFFFFu, ahead, o);
            if (i < n && sub == 0 && ahead <= goal && goal < ahead + weights[i])
                finish(static_cast<int>(0xFFFFFFFFu - name), logit_of(static_cast<uint32_t>(names[i] >> 32)));
        }
        return;
    }
    // Long way, any size: bins of the distance from the top over the whole row, then what shares the bin in which the
    // sum passes its goal.
    auto bin_of = [&](float l) {  // logits without weight are past the last
        const float x = (row.top - l) * row.to_bin;
        return x < static_cast<float>(kBins) ? static_cast<int>(x) : kBins;
    };
    uint32_t cut = kNothing;  // elements with larger keys are kept
    uint64_t ties = 0;        // and so many of those with this key
    // First by number (top_k), then, of these, by weight (top_p): the key at which the sum over the elements above
    // the cut, in falling order, reaches `want`, and the sum before it.
#pragma unroll 1
    for (int weighted = 0; weighted < 2; weighted++) {
        if (weighted ? !(top_p < 1.0f) : !(k > 0 && k < a.V)) continue;
        const uint64_t of_tie = ties ? weight_of(logit_of(cut), row, sh.table) : 0;
        uint64_t want = static_cast<uint64_t>(k), before = 0, above = 0;
        uint32_t high = 0, low = 0;  // the range of keys that it is reached in, once that is known
        int bin = 0;
        bool reached = true;
#pragma unroll 1
        for (bool ranged = false;; ranged = true) {
            // bins, of the distance from the top, then of keys
            const int bits = 32 - __clz(high - low), shift = bits > 10 ? bits - 10 : 0;
            for (int i = tid; i < kBins; i += kThreads) sh.low[i] = 0, sh.high[i] = 0;
            if (tid == 0) sh.count = 0;
            __syncthreads();
            for (int v = tid; v < pieces; v += kThreads) {
                const P p(reinterpret_cast<const uint4*>(slice)[v]);
#pragma unroll
                for (int j = 0; j < VEC; j += 2) {
                    int at[2];
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const uint32_t key = key_of(p[j + i]);
                        at[i] = ranged ? (key >= low && key <= high ? static_cast<int>((high - key) >> shift) : kBins)
                                       : (key > cut ? bin_of(p[j + i]) : kBins);
                    }
                    if (at[0] >= kBins && at[1] >= kBins) continue;
                    uint64_t w[2] = {1, 1};
                    if (weighted) weights_of(p[j], p[j + 1], row, sh.table, w);
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        if (at[i] >= kBins) continue;
                        const uint32_t lo = static_cast<uint32_t>(w[i]), old = atomicAdd(&sh.low[at[i]], lo);
                        const uint32_t hi = static_cast<uint32_t>(w[i] >> 32) + (old + lo < old ? 1 : 0);
                        if (hi) atomicAdd(&sh.high[at[i]], hi);
                    }
                }
            }
            cluster.sync();
            uint64_t in_bin[2] = {0, 0};
            for (int r = 0; r < ranks; r++) {
                const uint2 lo = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(sh.low, r) + 2 * tid);
                const uint2 hi = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(sh.high, r) + 2 * tid);
                in_bin[0] += (static_cast<uint64_t>(hi.x) << 32) + lo.x;
                in_bin[1] += (static_cast<uint64_t>(hi.y) << 32) + lo.y;
            }
            if (weighted && !ranged) {
                above = block_sum(in_bin[0] + in_bin[1]);
                want = max(fraction_of(top_p, above + ties * of_tie, true), uint64_t{1});
            }
            uint64_t more = 0;
            const int found = passed(in_bin[0], in_bin[1], want - before, &more);
            if (found == kBins) {  // only in the first round: the elements above the cut do not reach it
                reached = false;
                break;
            }
            before += more;
            if (ranged) {
                high -= static_cast<uint32_t>(found) << shift;
                low = shift == 0 ? high : max(low, high - ((1u << shift) - 1));
            } else {
                bin = found;
            }
            if (ranged && low == high) break;
            // what is in that bin goes to every CTA's list
            uint32_t* list = reinterpret_cast<uint32_t*>(sh.list);
            const int room_each = 2 * kList / ranks;
            float most = minus_inf(), fewest = __uint_as_float(0x7F800000u);
            for (int v = tid; v < pieces; v += kThreads) {
                const P p(reinterpret_cast<const uint4*>(slice)[v]);
#pragma unroll
                for (int j = 0; j < VEC; j++) {
                    const uint32_t key = key_of(p[j]);
                    if (ranged ? key > high || key < low : key <= cut || bin_of(p[j]) != bin) continue;
                    most = fmaxf(most, p[j]), fewest = fminf(fewest, p[j]);
                    const uint32_t at = atomicAdd(&sh.count, 1u);
                    if (at < static_cast<uint32_t>(room_each))
                        for (int r = 0; r < ranks; r++) cluster.map_shared_rank(list, r)[rank * room_each + at] = key;
                }
            }
            block_ends(most, fewest, &most, &fewest);
            if (tid < ranks)
                cluster.map_shared_rank(&sh, tid)->notes[1][rank] = {most, fewest, 0, static_cast<int32_t>(sh.count), 0};
            cluster.sync();
            int n = 0, mine_at = tid;
            uint32_t own = 0;
            bool whole = true;
            for (int r = 0; r < ranks; r++) {
                const Note note = sh.notes[1][r];
                if (mine_at >= 0 && mine_at < note.count && note.count <= room_each) own = list[r * room_each + mine_at];
                mine_at -= note.count;
                n += note.count;
                whole &= note.count <= room_each;
                if (note.count > 0) most = fmaxf(most, note.top), fewest = fminf(fewest, note.sum);
            }
            if (whole && n <= kThreads) {
                // each thread has one of them, and compares it with all
                uint64_t* weights = reinterpret_cast<uint64_t*>(sh.low);
                uint32_t* keys = sh.high;
                keys[tid] = own;
                weights[tid] = !weighted ? 1 : weight_of(logit_of(own), row, sh.table);
                __syncthreads();
                uint64_t larger = 0, equal = 0;
                if (tid < n)
                    for (int j = 0; j < n; j++) {
                        larger += keys[j] > own ? weights[j] : 0;
                        equal += keys[j] == own ? weights[j] : 0;
                    }
                if (tid < n && before + larger < want && want <= before + larger + equal) {
                    sh.found[0] = own;  // the same from every thread that has this key
                    sh.found[1] = before + larger;
                }
                __syncthreads();
                high = low = static_cast<uint32_t>(sh.found[0]);
                before = sh.found[1];
                break;
            }
            if (!ranged) high = key_of(most), low = key_of(fewest);
            if (low == high) break;
        }
        if (reached) {
            const uint64_t w = weighted ? weight_of(logit_of(high), row, sh.table) : 1;
            cut = high;
            ties = (want - before + w - 1) / w;
        } else if (weighted && of_tie) {  // among the tied ones: those with less than `want` before them
            ties = min(ties, (want - above + of_tie - 1) / of_tie);
        }
        __syncthreads();
        cluster.sync();  // all have read the bins, the lists and the notes
    }
    // Every thread takes a run of the slice's pieces; a run's sum is that of what lies above the cut, and of as many
    // tied elements as the runs before it leave.
    const int run = ((pieces + kThreads - 1) / kThreads) | 1;  // odd: a warp's reads spread over the banks
    const int r0 = min(pieces, tid * run), r1 = min(pieces, r0 + run);
    const uint64_t of_tie = ties ? weight_of(logit_of(cut), row, sh.table) : 0;
    const bool tie_counts = of_tie >= least;
    uint64_t above = 0, tied = 0;
    const float cut_at = logit_of(cut);
    if (cut == kNothing && least == 1) {  // nothing is cut off
        for (int v = r0; v < r1; v++) {
            const P p(reinterpret_cast<const uint4*>(slice)[v]);
#pragma unroll
            for (int j = 0; j < VEC; j += 2) {
                uint64_t w[2];
                weights_of(p[j], p[j + 1], row, sh.table, w);
                above += w[0] + w[1];
            }
        }
    } else {
        for (int v = r0; v < r1; v++) {
            const P p(reinterpret_cast<const uint4*>(slice)[v]);
            if (P::single(p.top()) < cut_at) continue;
#pragma unroll
            for (int j = 0; j < VEC; j += 2) {
                if (!(fmaxf(p[j], p[j + 1]) > cut_at)) continue;
                uint64_t w[2];
                weights_of(p[j], p[j + 1], row, sh.table, w);
#pragma unroll
                for (int i = 0; i < 2; i++) above += p[j + i] > cut_at && w[i] >= least ? w[i] : 0;
            }
            if (ties)
#pragma unroll
                for (int j = 0; j < VEC; j++) tied += p[j] == cut_at;
        }
    }
    const uint64_t scan_a = warp_scan(above, lane), scan_t = ties ? warp_scan(tied, lane) : 0;
    if (lane == 31) sh.part[warp][0] = scan_a, sh.part[warp][1] = scan_t;
    if (tid == 0) sh.found[0] = kThreads;
    __syncthreads();
    uint64_t ahead = scan_a - above, tied_ahead = scan_t - tied, here = 0, tied_here = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
        const uint64_t x = sh.part[w][0], y = sh.part[w][1];
        if (w < warp) ahead += x, tied_ahead += y;
        here += x, tied_here += y;
    }
    if (tid < ranks) {
        Shared* other = cluster.map_shared_rank(&sh, tid);
        other->sums[rank][0] = here;
        other->sums[rank][1] = tied_here;
    }
    cluster.sync();
    // of n tied elements behind `seen` others
    auto kept_of = [&](uint64_t n, uint64_t seen) { return tie_counts ? min(n, ties - min(ties, seen)) * of_tie : 0; };
    uint64_t total = 0, seen = 0, before_slice = 0, seen_before = 0;
    for (int r = 0; r < ranks; r++) {
        if (r == rank) before_slice = total, seen_before = seen;
        total += sh.sums[r][0];
        seen += sh.sums[r][1];
    }
    total += kept_of(seen, 0);
    tied_ahead += seen_before;
    // (all that lies before a run: what is above the cut there, and the first of its tied elements)
    const uint64_t goal = min(fraction_of(random, total, false), total - 1);
    ahead += before_slice + kept_of(tied_ahead, 0);
    if (goal >= ahead && goal < ahead + above + kept_of(tied, tied_ahead)) {
        sh.found[0] = tid;
        sh.part[0][0] = ahead;
        sh.part[0][1] = tied_ahead;
    }
    __syncthreads();
    const int at = static_cast<int>(sh.found[0]);
    if (at == kThreads || warp != 0) return;
    ahead = sh.part[0][0], tied_ahead = sh.part[0][1];
    const int end = min(places, (at + 1) * run * VEC);
    for (int i0 = at * run * VEC; i0 < end; i0 += 32) {
        const int i = i0 + lane;
        const float l = i < end ? value_at<BF16>(slice, i) : minus_inf();
        const uint32_t equal = __ballot_sync(0xFFFFFFFFu, i < end && l == cut_at);
        uint64_t w = 0;
        if (i < end && l > cut_at) {
            w = weight_of(l, row, sh.table);
            if (w < least) w = 0;
        } else if (i < end && l == cut_at && tie_counts && tied_ahead + __popc(equal & ((1u << lane) - 1)) < ties) {
            w = of_tie;
        }
        const uint64_t upto = ahead + warp_scan(w, lane);
        const uint32_t over = __ballot_sync(0xFFFFFFFFu, upto > goal);
        if (over) {
            if (lane == __ffs(over) - 1) finish(e0 + i - off, l);
            break;
        }
        ahead = __shfl_sync(0xFFFFFFFFu, upto, 31);
        tied_ahead += __popc(equal);
    }
}

template <bool BF16>
cudaError_t sample(const SampleArgs& a, int num_sms, cudaStream_t stream) {
    constexpr int E = BF16 ? 2 : 4;
    static std::once_flag once[64];
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    auto bytes = [](int64_t per) {  // the slice also holds a list's names and weights
        return static_cast<int>(sizeof(Shared)) + std::max(static_cast<int>(per) * E + 32, 2 * kList * 8);
    };
    const int kMost = bytes(std::max<int64_t>(kSampleMaxVocab / kMaxCluster, kSliceBytes / E + 8));
    std::call_once(once[device & 63], [&] {
        e = cudaFuncSetAttribute(sample_kernel<BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    });
    if (e != cudaSuccess) return e;
    // Eight CTAs a row for a few rows, where the row's own steps count (one row of 151936 bf16 logits, top-k 50: 9.9 us
    // with 8, 10.9 with 4; 16 rows of 50001: 32.4 with 8, 44 with 2); for many rows as few as leave an SM room for two CTAs,
    // since each has the same overhead whatever its slice (256 rows of 151936: 76 us with 8, 56 with 4).
    int ranks = 1;
    while (ranks < kMaxCluster && a.V > 4096 * ranks &&
           (a.B * ranks < num_sms || (a.V + ranks - 1) / ranks * E > kSliceBytes))
        ranks *= 2;
    const int per = static_cast<int>(((a.V + ranks - 1) / ranks + 7) / 8 * 8);
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(a.B * ranks)), kThreads, stream, attr);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(ranks), 1, 1};
    cfg.numAttrs = 2;
    cfg.dynamicSmemBytes = bytes(per);
    return cudaLaunchKernelEx(&cfg, sample_kernel<BF16>, a, per);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, int num_sms, cudaStream_t stream) {
    return a.bf16 ? sample<true>(a, num_sms, stream) : sample<false>(a, num_sms, stream);
}

}  // namespace nf4
