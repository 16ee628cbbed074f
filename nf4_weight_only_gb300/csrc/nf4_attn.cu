// Attention of one new token a sequence over the paged key-value cache.
//
// Mathematics.  For one sequence and kv head, the G query heads that share it give
//   S = K q^T [keys x heads],  p = 2^(S c - m),  O^T = V^T p^T [dims x heads],  l = sum p,
// one pass over the cache with a running maximum m a head (c = scale log2 e); O / l at the end.  Both
// products go through mma.sync m16n8k16 with the cache as the 16-row operand and the heads as the
// eight columns: 512 bytes of bf16 cache feed one instruction, so the tensor work is far below what
// the cache's bytes cost, and the fragments are read in an order that needs no rearrangement of the
// cache: the dims of a product's k axis may be permuted at will (q is permuted alike), and so may the
// keys.  tcgen05 takes 64 or 128 rows from shared or tensor memory in canonical tiles; here the rows are in
// pages of 16 and more, quantised, a tile would be used once, for eight columns, and the tensor pipe is busy
// for 14 to 20% of the time as it is.
//
// What bounds it, measured on GB300 (DRAM copy rate 6774 GB/s; 8 kv heads of 5 query heads, head_dim 128):
//   bf16   the memory (64 sequences up to 8192: 183 us, 98% of that rate; one of 131071: 85 us, 93%)
//   fp8    the same for many sequences (99 us, 94%), the latency of a ring of two stages for one (48 us, 86%)
//   NF4    the latency of decoding, no pipe being full (LSU 60%, issue 54%, ALU 42%, tensor 20%): 340 instructions
//          for 16 keys, 81 of them shared-memory reads, in a chain lookup, product, softmax, lookup, product, with three
//          warps a scheduler to cover it (32 sequences up to 16384: 74 us, 63%; one of 131071: 39 us, 55%)
//   short  one sequence of 517 tokens and 2 kv heads, bf16, 7.8 us: its segments are not cut, so two SMs read 265 KB
//          each (2 us at 64 bytes a clock) in four rounds of their rings, after lengths and page table; 8
//          sequences of up to 4095 in fp8 12 us: the longest one's pieces and their join
// More than eight query heads a kv head (NT = 2) take 249 to 255 registers, so eight warps of fp8 and NF4 in place of
// twelve: the 32 sequences with 12 heads take 114 us in NF4 (5 heads: 74), 107 in fp8 (96), 184 in bf16 (178).  With
// head_dim 256 they also spill 248 to 304 bytes: 274 us (5 heads: 149), 222 (190), 372 (348).  The main fp8 form spills 8.
//
// Quantised formats stay codes until they are fragments.  fp8 codes convert to fp16 exactly; an NF4 byte (two
// codes) indexes a table of fp16 pairs in shared memory (see kTableF16).  The scales are applied in fp32: K's to
// S, V's to p.  q in fp16 is scaled by a power of two a head (exact except for elements below 2^-28 of the
// head's largest); p * scale is rounded to fp16, times a power of two a warp that follows the largest scale of V
// it has met (the error is 2^-11 of the product or 2^-31 of that scale, whichever is larger).  With a bf16 cache
// p goes in as the sum of two bf16 numbers (one alone, 2^-8, would cost as much as the output's own rounding).
// S, m, l and O are fp32 throughout.
//
// Work.  A unit is 16 or 32 keys of one sequence and kv head (or of one group of at most 16 of its query
// heads): a segment.  Segments are cut into pieces by a rule on the lengths alone (make_plan), which the
// kernel works out for itself (no plan from the host), so ragged batches, one long sequence and thousands
// of short ones load the SMs alike.  A worker is a group of warps, two to a CTA and SM, so that one
// streams while the other starts or joins a piece.  Inside a piece its warps take units in turn, each with
// its own ring of cp.async stages and no barrier; their results are joined in shared memory.  The pieces
// of a segment leave partial results in the workspace; the worker that finishes the last of them joins
// them in their order (24 at a time, then the joined ones), so results do not depend on timing.
#include <algorithm>
#include <mutex>

#include "nf4_kv.cuh"

namespace nf4 {
namespace {

// Error word of the attention (43: a page or a length outside its bounds).
__device__ int g_attention_error;

constexpr int kMaxWorkers = 320;      // of W / 2 warps
constexpr int kRounds = 4;            // pieces a worker gets where workers are few warps
constexpr int kLongUnits = 32;        // units a warp to do, from which a few segments, too, are cut by line
constexpr int kStartRounds = 3;       // units a warp: what a segment's start and join count for in a line
constexpr int kFanIn = 24;            // partial results joined at a time
constexpr int kSlots = 2 * kMaxWorkers * kRounds + 2;  // partial results (see slot0)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazy = 8.0f;         // p may reach 2^8 before the running maximum moves

struct AttnArgs {
    KvCache c;
    const uint16_t* q;
    const int32_t* page_table;
    const int32_t* lengths;
    uint16_t* out;
    uint32_t* tickets;  // [0] pieces handed out, [1] workers done
    uint32_t* joins;    // [2][kSlots] partial results of a batch, batches of a segment
    float* partials;    // [kSlots][slot_floats]
    int64_t max_pages, window;
    uint64_t page_magic;  // ceil(2^64 / (page_size / 16))
    int B, q_heads, group;
    int chunks, chunk_heads;  // query heads of a kv head: `chunks` groups of at most chunk_heads
    int slot_floats;          // floats of one partial result
    float scale;
};

// ---------------------------------------------------------------------------------------------
// Fragments
// ---------------------------------------------------------------------------------------------
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8x8 transpose of 16-bit elements across the warp: lane (g, t) gives row g, columns 2t and 2t + 1, and
// gets rows 2t and 2t + 1 of column g.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 lds128a(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
// The table is never written after the first barrier: its loads may move.
__device__ __forceinline__ uint32_t lds_table(uint32_t a) {
    uint32_t v;
    asm("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// B bytes (4, 8 or 16) global -> shared; B source bytes are read, or none and zeros written.
// policy: of the L2 lines that 16-byte copies bring.
template <int B>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool live, uint64_t policy) {
    const uint32_t n = live ? B : 0;
    if (B == 16)
        asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(n),
                     "l"(policy)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(n), "n"(B) : "memory");
}

// What a long call reads of the cache is read once and leaves the L2 (129 MB) first: partial results, page tables
// and the next kernels' data stay (NF4, 64 sequences up to 2000: 48.0 -> 46.3 us; fp8, one of 131071: 49.8 -> 47.2).  A
// short call's may stay: it may still be there when the layer comes round again (8 ragged sequences, fp8, 23 MB:
// 12.3 -> 12.0 us).
constexpr int64_t kStreamBytes = 32 << 20;
__device__ __forceinline__ uint64_t l2_policy(bool stream) {
    uint64_t first, normal;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
    asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(normal));
    return stream ? first : normal;
}

// The NF4 table in fp16, times kTableUnit.  A table rounded entry by entry has a mean error of up to
// 6e-5 of the values' size (the table is not symmetric), which an average over 10^5 values near zero
// mean shows: 1% of the result at 131071 keys.  The unit and the direction of each entry's rounding are
// therefore chosen together (enumerated over all fp16 units and all 2^13 directions) so that the mean error
// is below 2.5e-6 of the values' size for normal, Laplace and uniform values of any width against their
// group's maximum; each entry stays within one fp16 step (6.4e-4 relative), 2.8e-4 in the mean square.  For values
// all on one side of zero it is up to 1.8e-4, for skewed ones around zero 6e-5 (exponential less its mean).
constexpr float kTableUnit = 1307.0f / 2048.0f;
__device__ __constant__ const float kTableF16[16] = {
    -0.63818359375f,   -0.4443359375f,    -0.335205078125f,  -0.251953125f,   -0.181640625f,  -0.117919921875f,
    -0.058135986328125f, 0.0f,            0.050811767578125f, 0.10272216796875f, 0.1571044921875f, 0.2156982421875f,
    0.28125f,          0.359130859375f,   0.46142578125f,    0.63818359375f};

// The four e4m3 codes of a word -> two fp16 pairs (bytes 0, 1 and bytes 2, 3), exact.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Shared memory of a CTA.  NF4 keeps its pair table at shared address 64 KB, entry v (a code byte) at
// 256 v and lane l's copy 4 l into it, so one byte permute of a code word and the lane's constant is a
// lookup's whole address and the 32 lanes never conflict.  The warps' rings lie on both sides of it.
constexpr uint32_t kTableAt = 65536, kTableEnd = 131072;

template <int FMT, int D, int NT>
struct Shape {
    static constexpr bool kBf = FMT == kKvBf16;
    static constexpr int VB = kv_vector_bytes(FMT, D);           // bytes of a vector
    static constexpr int SB = 16 * kv_scale_bytes(FMT, D);       // bytes of 16 keys' scales of one side
    static constexpr int GR = FMT == kKvNf4 ? D / 64 : 1;        // scale groups of a vector
    // Blocks of 16 keys in a unit: two give the decoding formats two independent chains and halve the
    // bookkeeping, where registers and shared memory allow it.
    static constexpr int KS = FMT != kKvBf16 && NT == 1 && D <= 128 ? 2 : 1;
    static constexpr int kBlock = 32 * VB + 2 * SB;              // 16 keys, K and V
    static constexpr int kStage = KS * kBlock;
    // Warps and stages.  bf16: 8 warps with 8 KB stages are 128 KB in flight an SM.  Decoding wants more warps, and
    // registers: 12 warps at 168 (NF4, 32 sequences up to 16384: 75 us; 16 at 128 work the addresses out again
    // for every unit: 79; 8: 81), except where a warp's state alone takes more (8 warps: NT = 2 uses 254; in 12
    // warps it was 18% slower).
    static constexpr int W = FMT == kKvBf16 ? (D == 256 ? 4 : 8) : D == 256 || NT == 2 ? 8 : 12;
    static constexpr int kRingMost = FMT == kKvNf4 ? (W == 12 ? 8704 : 20480) : 230400 / W / 16 * 16;
    static constexpr int kStagesFit = kRingMost / kStage;
    static constexpr int NST = kStagesFit > 10 ? 10 : kStagesFit;
    static constexpr int kRing = NST * kStage;
    static constexpr int kResult = NT * 8 * (D + 2) * 4;         // bytes of a warp's result
    static constexpr int kSmem = 225 * 1024;                     // dynamic; with 2 KB of static, all there is
    static constexpr int kArea = kRing > kResult ? kRing : kResult;
    static_assert(kArea >= (kSlots / 2 / kFanIn + 2) * 2 * NT * 8 * 4, "an area holds the maxima and sums of a join");
    // dynamic shared memory starts 2 to 4 KB into the window
    static constexpr int kBelow = FMT == kKvNf4 ? static_cast<int>(kTableAt - 4096) / kArea : W;
    static_assert(NST >= 2, "a ring has at least two stages");
    static_assert(FMT == kKvNf4 ? (W - kBelow) * kArea <= kSmem + 2048 - static_cast<int>(kTableEnd)
                                : W * kArea <= kSmem, "the areas fit");
};

// Dynamic shared memory cut into areas of `bytes`, the NF4 table left out: address of area w.  Used for
// the warps' rings and, once these are drained, for their results.
template <int FMT>
__device__ __forceinline__ uint32_t area_of(uint32_t base, int w, uint32_t bytes) {
    if (FMT != kKvNf4) return base + w * bytes;
    const int below = (kTableAt - base) / bytes;
    return w < below ? base + w * bytes : kTableEnd + (w - below) * bytes;
}

// Key of fragment row r (0..7; row r + 8 holds the key 8 later).  Rows r = 0..3 and 4..7, and rows 2t (or
// 2t + 1) over t, are distinct modulo 4, and rows 2i and 2i + 1 differ in bit 2: the bank groups below.
__device__ __forceinline__ int key_of_row(int r) { return (r & 1) ? 4 + (((r >> 1) + 2) & 3) : r >> 1; }

// Offset of 16-byte piece p of key row `row` inside a block's K or V.  The global side reads a block in order,
// 512 contiguous bytes a warp instruction (segments of 64 or 128 bytes of several rows reach 5.4 TB/s in a
// bare copy ring of this shape, whole lines in order 7.2); the pieces are permuted so that the fragment
// reads do not conflict:
//   16 bytes a lane, K: rows 2i, 2i + 1 by four pieces, told apart by bit 2 of the row
//   16 bytes a lane, V: rows of four t by two pieces, told apart by the row modulo 4
//   NF4 (8 bytes of a group, K; 4, V): four rows of 32 bytes, told apart by the row modulo 4
template <int FMT, int D, bool IS_V>
__device__ __forceinline__ uint32_t piece_at(int row, int p) {
    constexpr int VB = kv_vector_bytes(FMT, D);
    if (FMT == kKvNf4) {
        if (D == 64) return row * 32 + p * 16;
        if (D == 128) return row * 64 + (p ^ (((row >> 1) & 1) << 1)) * 16;
        return row * 128 + (p ^ ((row & 3) << 1)) * 16;
    }
    if (VB == 64) {  // two rows a 128-byte line
        if (IS_V) return row * 64 + (p ^ (((row >> 1) & 1) << 1)) * 16;
        return ((row * 4 + p) ^ (((row >> 2) & 1) << 2)) * 16;
    }
    return row * VB + (IS_V ? p ^ ((row & 3) << 1) : p ^ (((row >> 2) & 1) << 2)) * 16;
}

// ---------------------------------------------------------------------------------------------
// One block of 16 keys into its part of a stage
// ---------------------------------------------------------------------------------------------
// place: vector index of the block's first key.  lo and hi: its live keys (ALL: every one);
// dead ones are filled with zeros so that nothing non-finite meets a weight of 0.
template <int FMT, int D, int NT, bool ALL>
__device__ __forceinline__ void copy_block(const KvCache& c, uint32_t buf, int64_t place, int lo, int hi, int lane,
                                           uint64_t policy) {
    using S = Shape<FMT, D, NT>;
    const uint32_t kb = buf, vb = buf + 16 * S::VB, sb = buf + 32 * S::VB;
    const uint8_t* k = c.k + place * S::VB;
    const uint8_t* v = c.v + place * S::VB;
    auto live = [&](int key) { return ALL || (key >= lo && key < hi); };
    constexpr int P = S::VB / 16;  // 16-byte pieces of a vector
#pragma unroll
    for (int j = 0; j < P / 2; j++) {
        const int n = j * 32 + lane, key = n / P, p = n % P;
        cp_async<16>(kb + piece_at<FMT, D, false>(key, p), k + n * 16, live(key), policy);
        cp_async<16>(vb + piece_at<FMT, D, true>(key, p), v + n * 16, live(key), policy);
    }
    if (S::SB) {
        constexpr int SK = S::SB ? S::SB / 16 : 1;  // scale bytes of a key
        const uint8_t* ks = c.k_scales + place * SK;
        const uint8_t* vs = c.v_scales + place * SK;
#pragma unroll
        for (int i = 0; i < 2 * S::SB; i += 128) {
            const int o = i + lane * 4;
            if (o < 2 * S::SB) {
                const int at = o < S::SB ? o : o - S::SB;
                const bool on = live(at / SK) || live((at + 3) / SK);
                cp_async<4>(sb + o, (o < S::SB ? ks : vs) + at, on, policy);
            }
        }
    }
}

// A block that may have nothing to read (place < 0: zeros) or dead keys.
template <int FMT, int D, int NT>
__device__ __forceinline__ void copy_edge_block(const KvCache& c, uint32_t buf, int64_t place, int lo, int hi, int lane,
                                                uint64_t policy) {
    if (place < 0) {
        for (int i = lane * 4; i < Shape<FMT, D, NT>::kBlock; i += 128)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(buf + i), "r"(0) : "memory");
    } else {
        copy_block<FMT, D, NT, false>(c, buf, place, lo, hi, lane, policy);
    }
}

// ---------------------------------------------------------------------------------------------
// The running softmax and output of a warp
// ---------------------------------------------------------------------------------------------
template <int FMT, int D, int NT>
struct WarpState {
    uint32_t q[NT][D / 16][2];  // fragments of q^T
    float mul[NT][2];           // S -> base-2 logit, heads 2t and 2t + 1
    float m[NT][2], l[NT][2];
    float o[NT][D / 16][4];
    float vn, vlim;             // V scales are multiplied by vn; they stay below vlim
};

// First dim of a lane's run of consecutive dims: K side (t) and V side (g).
template <int FMT, int D>
__device__ __forceinline__ int k_dim(int i, int t) {  // i-th run of the lane; runs of 8 (bf16) or 16
    if (FMT == kKvBf16) return (i * 4 + t) * 8;
    return (i * 4 + t) * 16;
}
template <int FMT, int D>
__device__ __forceinline__ constexpr int v_run() {  // dims of a run on the V side
    return FMT == kKvFp8 ? (D / 8 < 16 ? D / 8 : 16) : 8;
}

template <int FMT, int D, int NT>
__device__ __forceinline__ void load_q(const AttnArgs& a, WarpState<FMT, D, NT>& s, const uint16_t* q, int heads,
                                       int lane) {
    const int g = lane >> 2, t = lane & 3;
    constexpr int RUN = FMT == kKvBf16 ? 8 : 16;  // consecutive dims of a lane
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
        const int h = nt * 8 + g;
        uint32_t w[D / 8];
#pragma unroll
        for (int i = 0; i < D / 4 / RUN; i++)
#pragma unroll
            for (int j = 0; j < RUN / 8; j++) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (h < heads) x = *reinterpret_cast<const uint4*>(q + h * D + k_dim<FMT, D>(i, t) + 8 * j);
                const int at = (i * RUN + 8 * j) / 2;
                w[at] = x.x, w[at + 1] = x.y, w[at + 2] = x.z, w[at + 3] = x.w;
            }
        float mul = a.scale * (FMT == kKvNf4 ? kLog2e / kTableUnit : kLog2e);
        if (FMT != kKvBf16) {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < D / 8; i++) {
                const float2 f = bf16x2_to_f32x2(w[i]);
                top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            // the head's largest element to [2^14, 2^15)
            const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 15), 254);
            const float up = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);
            mul *= __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
#pragma unroll
            for (int i = 0; i < D / 8; i++) {
                const float2 f = bf16x2_to_f32x2(w[i]);
                w[i] = pack_f16(f.x * up, f.y * up);
            }
        }
#pragma unroll
        for (int i = 0; i < D / 16; i++) s.q[nt][i][0] = w[2 * i], s.q[nt][i][1] = w[2 * i + 1];
        s.mul[nt][0] = __shfl_sync(0xFFFFFFFFu, mul, 8 * t);
        s.mul[nt][1] = __shfl_sync(0xFFFFFFFFu, mul, 8 * t + 4);
        s.m[nt][0] = s.m[nt][1] = -3e38f;
        s.l[nt][0] = s.l[nt][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 16; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) s.o[nt][i][j] = 0.0f;
    }
    s.vn = 1.0f;
    s.vlim = -1.0f;
}

// One unit from its stage.  full: every key is live; otherwise [lo, hi) are, without the blocks whose bit
// is set in `bad`.
template <int FMT, int D, int NT>
__device__ __forceinline__ void attend_unit(WarpState<FMT, D, NT>& s, uint32_t buf, bool full, int lo, int hi,
                                            uint32_t bad, int lane) {
    using S = Shape<FMT, D, NT>;
    constexpr bool BF = S::kBf;
    constexpr int GR = S::GR, KS = S::KS;
    constexpr uint32_t VOFF = 16 * S::VB, SOFF = 32 * S::VB;  // of a block's V and scales
    const int g = lane >> 2, t = lane & 3, key = key_of_row(g);
    // the lane's constant in a table lookup's address: 64 KB and 4 * lane around the code byte
    const uint32_t column = (kTableAt >> 8) | static_cast<uint32_t>(4 * lane);
    auto pair_of = [&](uint32_t word, int byte) {  // fp16 pair of byte `byte` of a code word
        return lds_table(prmt(word, column, 0x6504u + 16u * static_cast<uint32_t>(byte)));
    };

    // S = K q^T: two chains a block (a chain for each scale group with NF4)
    constexpr int CH = FMT == kKvNf4 ? GR : 2;
    float sc[KS][NT][CH][4];
#pragma unroll
    for (int b = 0; b < KS; b++) {
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int c = 0; c < CH; c++)
#pragma unroll
                for (int j = 0; j < 4; j++) sc[b][nt][c][j] = 0.0f;
        const uint32_t kb = buf + b * S::kBlock;
        if (FMT == kKvNf4) {
#pragma unroll
            for (int r = 0; r < GR; r++) {
                const uint32_t at = kb + piece_at<FMT, D, false>(key, 2 * r) + t * 8;
                const uint2 u = lds64(at), w = lds64(at + 8 * S::VB);
#pragma unroll
                for (int i = 0; i < 4; i++) {  // four dims a row each
                    const uint32_t x = i < 2 ? u.x : u.y, y = i < 2 ? w.x : w.y;
                    const int n = 2 * (i & 1);
                    const uint32_t f[4] = {pair_of(x, n), pair_of(y, n), pair_of(x, n + 1), pair_of(y, n + 1)};
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
                        mma16816<false>(sc[b][nt][r], f, s.q[nt][r * 4 + i][0], s.q[nt][r * 4 + i][1]);
                }
            }
        } else {
            constexpr int CK = S::VB / 4 < 16 ? S::VB / 4 : 16, NK = S::VB / 4 / CK, WK = CK / 4;
#pragma unroll
            for (int i = 0; i < NK; i++) {
                uint32_t x[WK], y[WK];
                const uint32_t at = kb + piece_at<FMT, D, false>(key, i * 4 + t);
                const uint4 u = lds128a(at), w = lds128a(at + 8 * S::VB);
                x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
                y[0] = w.x, y[1] = w.y, y[2] = w.z, y[3] = w.w;
                if (BF) {
#pragma unroll
                    for (int j = 0; j < WK / 2; j++) {
                        const uint32_t f[4] = {x[2 * j], y[2 * j], x[2 * j + 1], y[2 * j + 1]};
#pragma unroll
                        for (int nt = 0; nt < NT; nt++)
                            mma16816<true>(sc[b][nt][j & 1], f, s.q[nt][i * 2 + j][0], s.q[nt][i * 2 + j][1]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < WK; j++) {
                        uint32_t f[4];
                        e4m3x4_to_f16x4(x[j], f[0], f[2]);
                        e4m3x4_to_f16x4(y[j], f[1], f[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; nt++)
                            mma16816<false>(sc[b][nt][j & 1], f, s.q[nt][i * 4 + j][0], s.q[nt][i * 4 + j][1]);
                    }
                }
            }
        }
    }

    // scales of keys `key` (row g) and key + 8 of each block
    float ks[KS][2][GR], vs[KS][2][GR];
    auto on = [&](int b, int r) {
        const int k = 16 * b + 8 * r + key;
        return k >= lo && k < hi && !((bad >> b) & 1);
    };
    if (FMT != kKvBf16) {
#pragma unroll
        for (int b = 0; b < KS; b++)
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const uint32_t at = buf + b * S::kBlock + SOFF + key * (S::SB / 16) + r * (S::SB / 2);
                if (FMT == kKvFp8) {
                    ks[b][r][0] = __uint_as_float(lds32(at));
                    vs[b][r][0] = __uint_as_float(lds32(at + S::SB));
                } else if (GR == 1) {
                    ks[b][r][0] = __half2float(__ushort_as_half(lds_u16(at)));
                    vs[b][r][0] = __half2float(__ushort_as_half(lds_u16(at + S::SB)));
                } else {
#pragma unroll
                    for (int p = 0; p < GR / 2; p++) {
                        const uint32_t kw = lds32(at + 4 * p), vw = lds32(at + S::SB + 4 * p);
                        const float2 kf = __half22float2(*reinterpret_cast<const __half2*>(&kw));
                        const float2 vf = __half22float2(*reinterpret_cast<const __half2*>(&vw));
                        ks[b][r][2 * p] = kf.x, ks[b][r][2 * p + (GR > 1)] = kf.y;
                        vs[b][r][2 * p] = vf.x, vs[b][r][2 * p + (GR > 1)] = vf.y;
                    }
                }
            }
    }

    // y: S with K's scales; x = y mul - m: base-2 logits of keys (row g: j = 0, 1; row g + 8: 2, 3) and heads
    // 2t, 2t + 1, from the running maximum
    float y[KS][NT][4], x[KS][NT][4];
    float most = -INFINITY;
#pragma unroll
    for (int b = 0; b < KS; b++)
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int r = j >> 1;
                float v;
                if (FMT == kKvNf4) {
                    v = sc[b][nt][0][j] * ks[b][r][0];
#pragma unroll
                    for (int c = 1; c < GR; c++) v = fmaf(sc[b][nt][c][j], ks[b][r][c], v);
                } else {
                    v = sc[b][nt][0][j] + sc[b][nt][CH > 1][j];
                    if (FMT == kKvFp8) v *= ks[b][r][0];
                }
                y[b][nt][j] = v;
                x[b][nt][j] = fmaf(v, s.mul[nt][j & 1], -s.m[nt][j & 1]);
            }
    if (!full) {
#pragma unroll
        for (int b = 0; b < KS; b++)
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int j = 0; j < 4; j++)
                    if (!on(b, j >> 1)) x[b][nt][j] = -INFINITY;
#pragma unroll
        for (int b = 0; b < KS; b++)
#pragma unroll
            for (int r = 0; r < 2; r++)
#pragma unroll
                for (int c = 0; c < GR; c++)
                    if (!on(b, r)) vs[b][r][c] = 0.0f;
    }
    float widest = 0.0f;  // the largest V scale
    if (FMT != kKvBf16) {
#pragma unroll
        for (int b = 0; b < KS; b++)
#pragma unroll
            for (int r = 0; r < 2; r++)
#pragma unroll
                for (int c = 0; c < GR; c++) widest = fmaxf(widest, vs[b][r][c]);
    }
#pragma unroll
    for (int b = 0; b < KS; b++)
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int j = 0; j < 4; j++) most = fmaxf(most, x[b][nt][j]);
    // rare, and one vote for both (two: 1.5% slower with NF4): V's scales leave the fp16 range (the largest times vn
    // stays below 2^7), or the maxima move
    if (__any_sync(0xFFFFFFFFu, (FMT != kKvBf16 && widest > s.vlim) || most > kLazy)) {
        if (FMT != kKvBf16 && __any_sync(0xFFFFFFFFu, widest > s.vlim)) {
            widest = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(widest)));
            const int e = min(max(static_cast<int>(__float_as_uint(widest) >> 23), 7), 254);
            const float vn = __uint_as_float(static_cast<uint32_t>(260 - e) << 23), f = vn / s.vn;
            s.vn = vn;
            s.vlim = __uint_as_float(static_cast<uint32_t>(min(e + 1, 254)) << 23);
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int i = 0; i < D / 16; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++) s.o[nt][i][j] *= f;
        }
        if (__any_sync(0xFFFFFFFFu, most > kLazy)) {
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    float top = s.m[nt][j];
#pragma unroll
                    for (int b = 0; b < KS; b++)
#pragma unroll
                        for (int r = 0; r < 2; r++) {
                            float& z = x[b][nt][j + 2 * r];
                            z = z == -INFINITY ? z : y[b][nt][j + 2 * r] * s.mul[nt][j];
                            top = fmaxf(top, z);
                        }
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                    const float f = exp2_approx(s.m[nt][j] - top);
                    s.m[nt][j] = top;
                    s.l[nt][j] *= f;
#pragma unroll
                    for (int i = 0; i < D / 16; i++) s.o[nt][i][j] *= f, s.o[nt][i][j + 2] *= f;
#pragma unroll
                    for (int b = 0; b < KS; b++) x[b][nt][j] -= top, x[b][nt][j + 2] -= top;
                }
        }
    }
    // weights, and p^T fragments
    constexpr int PB = FMT == kKvBf16 ? 2 : GR;  // bf16: p's high and low part; else one for each scale group
    uint32_t pb[KS][NT][PB][2];
#pragma unroll
    for (int b = 0; b < KS; b++)
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            float p[4];
#pragma unroll
            for (int j = 0; j < 4; j++) p[j] = exp2_approx(x[b][nt][j]);
            s.l[nt][0] += p[0] + p[2];
            s.l[nt][1] += p[1] + p[3];
            if (FMT == kKvBf16) {
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    const uint32_t hi16 = f32x2_to_bf16x2(p[2 * r], p[2 * r + 1]);
                    const float2 f = bf16x2_to_f32x2(hi16);
                    pb[b][nt][0][r] = transpose8x8(hi16);
                    pb[b][nt][PB - 1][r] = transpose8x8(f32x2_to_bf16x2(p[2 * r] - f.x, p[2 * r + 1] - f.y));
                }
            } else {
#pragma unroll
                for (int c = 0; c < GR; c++) {
                    const float v0 = vs[b][0][c] * s.vn, v1 = vs[b][1][c] * s.vn;
                    pb[b][nt][c][0] = transpose8x8(pack_f16(p[0] * v0, p[1] * v0));
                    pb[b][nt][c][1] = transpose8x8(pack_f16(p[2] * v1, p[3] * v1));
                }
            }
        }

    // O^T += V^T p^T: fragment column pairs are keys of rows (2t, 2t + 1) and (2t + 8, 2t + 9)
#pragma unroll
    for (int b = 0; b < KS; b++) {
        const uint32_t vb = buf + b * S::kBlock + VOFF;
        if (FMT == kKvNf4) {
            const int ka = key_of_row(2 * t), kc = key_of_row(2 * t + 1);
#pragma unroll
            for (int r = 0; r < GR; r++) {
                const uint32_t at_a = vb + piece_at<FMT, D, true>(ka, 2 * r) + g * 4;
                const uint32_t at_c = vb + piece_at<FMT, D, true>(kc, 2 * r) + g * 4;
                const uint32_t wa = lds32(at_a), wb = lds32(at_c);
                const uint32_t wc = lds32(at_a + 8 * S::VB), wd = lds32(at_c + 8 * S::VB);
                // code bytes (first key low, second key high) of the even and of the odd dims
                const uint32_t lo4 = 0x0F0F0F0Fu;
                const uint32_t e0 = (wa & lo4) | ((wb << 4) & ~lo4), o0 = ((wa >> 4) & lo4) | (wb & ~lo4);
                const uint32_t e1 = (wc & lo4) | ((wd << 4) & ~lo4), o1 = ((wc >> 4) & lo4) | (wd & ~lo4);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint32_t f[4] = {pair_of(e0, i), pair_of(o0, i), pair_of(e1, i), pair_of(o1, i)};
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
                        mma16816<false>(s.o[nt][r * 4 + i], f, pb[b][nt][r][0], pb[b][nt][r][1]);
                }
            }
        } else {
            constexpr int CV = S::VB / 8 < 16 ? S::VB / 8 : 16, NV = S::VB / 8 / CV, WV = CV / 4;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                uint32_t w[4][4];
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const int row = key_of_row(2 * t + (r & 1));
                    const uint32_t at = vb + (r >> 1) * 8 * S::VB +
                                        (CV == 16 ? piece_at<FMT, D, true>(row, i * 8 + g)
                                                  : piece_at<FMT, D, true>(row, g / 2) + (g & 1) * 8);
                    if (CV == 16) {
                        const uint4 u = lds128a(at);
                        w[r][0] = u.x, w[r][1] = u.y, w[r][2] = u.z, w[r][3] = u.w;
                    } else {
                        const uint2 u = lds64(at);
                        w[r][0] = u.x, w[r][1] = u.y;
                    }
                }
#pragma unroll
                for (int j = 0; j < WV; j++) {
                    if (BF) {
                        const uint32_t f[4] = {prmt(w[0][j], w[1][j], 0x5410), prmt(w[0][j], w[1][j], 0x7632),
                                               prmt(w[2][j], w[3][j], 0x5410), prmt(w[2][j], w[3][j], 0x7632)};
#pragma unroll
                        for (int nt = 0; nt < NT; nt++) {
                            mma16816<true>(s.o[nt][i * WV + j], f, pb[b][nt][0][0], pb[b][nt][0][1]);
                            mma16816<true>(s.o[nt][i * WV + j], f, pb[b][nt][PB - 1][0], pb[b][nt][PB - 1][1]);
                        }
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; h++) {  // dims 0, 1 and 2, 3 of the word
                            uint32_t f[4];
                            e4m3x4_to_f16x4(prmt(w[0][j], w[1][j], h ? 0x7362 : 0x5140), f[0], f[1]);
                            e4m3x4_to_f16x4(prmt(w[2][j], w[3][j], h ? 0x7362 : 0x5140), f[2], f[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; nt++)
                                mma16816<false>(s.o[nt][(i * WV + j) * 2 + h], f, pb[b][nt][0][0], pb[b][nt][0][1]);
                        }
                    }
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------
// Lengths and runs
// ---------------------------------------------------------------------------------------------
struct Span {
    int start, end;  // keys [start, end) of a sequence
    template <int KEYS>
    __device__ int units() const {  // of KEYS keys each, aligned (`end` may be within KEYS of 2^31)
        return end > start ? static_cast<int>((static_cast<uint32_t>(end) + (KEYS - 1)) / KEYS) - start / KEYS : 0;
    }
};

__device__ __forceinline__ Span span_of(const AttnArgs& a, int b) {
    const int64_t most = a.max_pages * a.c.page_size;
    const int64_t n0 = a.lengths[b];
    const int n = static_cast<int>(n0 < 0 ? 0 : n0 > most ? most : n0);
    Span s;
    s.end = n;
    s.start = a.window > 0 && n > a.window ? n - static_cast<int>(a.window) : 0;
    return s;
}

// Four dims (column i) of one head, joined over `n` results in their order: part(j) is result j, [heads][D]
// sums of weighted values, then [heads] maxima and [heads] sums of weights at ml(j).
struct Joined {
    float4 o;
    float top, l;
};
template <int N>
__device__ __forceinline__ void join_some(Joined& r, const float4 (&v)[N], const float (&m)[N], const float (&l)[N]) {
    float top = r.top;
#pragma unroll
    for (int j = 0; j < N; j++) top = fmaxf(top, m[j]);
    const float f0 = exp2_approx(r.top - top);
    r.top = top;
    r.l *= f0, r.o.x *= f0, r.o.y *= f0, r.o.z *= f0, r.o.w *= f0;
#pragma unroll
    for (int j = 0; j < N; j++) {
        const float f = exp2_approx(m[j] - top);
        r.l = fmaf(f, l[j], r.l);
        r.o.x = fmaf(f, v[j].x, r.o.x), r.o.y = fmaf(f, v[j].y, r.o.y);
        r.o.z = fmaf(f, v[j].z, r.o.z), r.o.w = fmaf(f, v[j].w, r.o.w);
    }
}
// N results are loaded at a time.  R_SHARED, M_SHARED: the results, and their maxima and sums, are in shared
// memory.
template <int D, int N, bool R_SHARED, bool M_SHARED, typename Part, typename Ml>
__device__ __forceinline__ Joined join(const Part& part, const Ml& ml, int n, int heads, int i) {
    const int h = i / (D / 4);
    Joined r{make_float4(0.0f, 0.0f, 0.0f, 0.0f), -3e38f, 0.0f};
#pragma unroll 1
    for (int j0 = 0; j0 < n; j0 += N) {
        float4 v[N];
        float m[N], l[N];
#pragma unroll
        for (int j = 0; j < N; j++) {
            v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f), m[j] = -3e38f, l[j] = 0.0f;
            if (j0 + j < n) {
                const float4* p = reinterpret_cast<const float4*>(part(j0 + j)) + i;
                const float* q = ml(j0 + j) + h;
                v[j] = R_SHARED ? *p : __ldcg(p);
                m[j] = M_SHARED ? *q : __ldcg(q);
                l[j] = M_SHARED ? q[heads] : __ldcg(q + heads);
            }
        }
        join_some(r, v, m, l);
    }
    return r;
}
__device__ __forceinline__ uint2 normalised(const Joined& r) {
    const float f = r.l > 0.0f ? 1.0f / r.l : 0.0f;
    return make_uint2(f32x2_to_bf16x2(r.o.x * f, r.o.y * f), f32x2_to_bf16x2(r.o.z * f, r.o.w * f));
}
template <int D>
__device__ __forceinline__ void store_partial(float* slot, const Joined& r, int heads, int i) {
    __stcg(reinterpret_cast<float4*>(slot) + i, r.o);
    if (i % (D / 4) == 0) {
        __stcg(slot + heads * D + i / (D / 4), r.top);
        __stcg(slot + heads * D + heads + i / (D / 4), r.l);
    }
}

// Counts up to `last` and wraps to 0; the old count.  Releases what this thread has seen (the worker's stores, by
// the barrier before) and acquires what the others released.
__device__ __forceinline__ uint32_t ticket_inc(uint32_t* at, uint32_t last) {
    uint32_t old;
    asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(old) : "l"(at), "r"(last) : "memory");
    return old;
}

// Barrier of a worker's warps (barrier 0 is the CTA's).
__device__ __forceinline__ void worker_barrier(int group, int warps) {
    if (warps == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(warps * 32) : "memory");
}

// How the work is cut.  By segment: every segment into pieces of at most `cut` units, as equal as they come.
// By line (cut = 0): the units of all segments end to end, each segment's behind `start` units that stand for the
// time its start and join take, into one cell of `cell` units a worker; a cell's part of a segment is a piece.
struct Plan {
    uint32_t warps, workers;  // warps of a worker; workers of the grid
    uint32_t count;           // pieces, or cells
    uint32_t cut, cell, start;
    uint64_t total;           // units (by line: with the starts)
};

// (a 64-bit division takes longer than what follows it)
__device__ __forceinline__ uint32_t quotient(uint64_t a, uint32_t d) {
    return a < (uint64_t{1} << 32) ? static_cast<uint32_t>(a) / d : static_cast<uint32_t>(a / d);
}

__device__ __forceinline__ uint32_t divide_up(uint64_t a, uint32_t d) {  // at most 2^30
    if (a < (uint64_t{1} << 31)) return (static_cast<uint32_t>(a) + d - 1) / d;
    const uint64_t q = (a + d - 1) / d;
    return static_cast<uint32_t>(q < (1u << 30) ? q : (1u << 30));
}

// units(b): of sequence b, asked by lane b % 32.  The whole warp calls it.
template <typename Units>
__device__ __forceinline__ uint32_t count_pieces(const Units& units, int B, uint32_t segs, uint32_t cut, int lane) {
    uint32_t p = 0;
    for (int b = lane; b < B; b += 32) p += (units(b) + cut - 1) / cut;
    return __reduce_add_sync(0xFFFFFFFFu, p) * segs;
}

// A rule on the lengths alone, the same in every CTA (one warp works it out).  W warps a CTA; a worker is
// W / 2 of them, so that a CTA has one that streams while the other starts or joins a piece, except
//  - all W, when there is at most a segment for each CTA and little to do (no second piece to overlap with), or
//    a segment for eight CTAs (half as many partial results to join; one bf16 sequence of 131071 keys and 8
//    heads: 84 us, 87 with halves);
//  - fewer, when there are many segments too short to keep W / 2 warps busy.
// Then, the figures being of bf16, fp8 and NF4 caches with 8 kv heads:
//  - Sequences of up to 8 units a warp (4, where there are more segments than workers, so that a worker's pieces even
//    out) are not cut: the join of partial results costs 3 us, about what these units do.
//  - Many segments, and long ones, are cut by line: every worker does the same, whatever the lengths.  A segment's
//    start and join (and units that do not fill a round of the worker's warps) take as long as about three units a
//    warp, so the line counts that many more for each (64 sequences of 200 to 4000 tokens: 88, 50, 47 us; without it
//    97, 71, 70; cut by segment into up to four pieces a worker: 94, 61, 61.  One of 131071: 85, 47, 39; by
//    segment 93, 47, 40).
//  - The rest, a few segments with little to do, by segment: the pieces of each are as equal as they come and their
//    count fits the workers, so `cut` grows until it does.  So are many segments too short for W / 2 warps, into
//    up to kRounds pieces a worker, taken by ticket.
template <int W, typename Units>
__device__ __forceinline__ Plan make_plan(const Units& units, int B, uint32_t segs, int lane) {
    uint32_t sum = 0, live = 0, longest = 0;
    for (int b = lane; b < B; b += 32) {
        const uint32_t n = units(b);
        sum += n;
        live += n > 0;
        longest = max(longest, n);
    }
    sum = __reduce_add_sync(0xFFFFFFFFu, sum);
    live = __reduce_add_sync(0xFFFFFFFFu, live);
    longest = __reduce_max_sync(0xFFFFFFFFu, longest);
    const uint64_t segments = static_cast<uint64_t>(live) * segs, total = static_cast<uint64_t>(sum) * segs;
    Plan p;
    p.total = total, p.start = 0;
    p.warps = W / 2;
    if (segments * 8 <= gridDim.x || (segments <= gridDim.x && total <= static_cast<uint64_t>(8 * W) * gridDim.x))
        p.warps = W;
    while (p.warps > 1 && segments >= 2 * gridDim.x * (W / p.warps) && total < 4 * p.warps * segments) p.warps /= 2;
    p.workers = gridDim.x * (W / p.warps);
    const uint32_t uncut = (p.warps >= W / 2 && segments > p.workers ? 4 : 8) * p.warps;
    if (longest <= uncut) {
        p.cut = uncut;
        p.count = static_cast<uint32_t>(segments);
        return p;
    }
    const uint32_t share = divide_up(total, p.workers);
    if (p.warps >= W / 2 && (segments > p.workers / 2 || share >= kLongUnits * p.warps) && share < (1u << 29)) {
        p.cut = 0;
        p.start = kStartRounds * p.warps;
        p.total = total + segments * p.start;
        p.cell = divide_up(p.total, p.workers);
        p.count = p.workers;
        return p;
    }
    const uint32_t rounds = segments > p.workers / 2 ? kRounds : 1;
    // (the second bound keeps the workspace's slots enough when workers of few warps are many)
    uint32_t low = max(divide_up(total, rounds * p.workers), divide_up(total, kRounds * gridDim.x * 2));
    low = max(low, 2 * p.warps);
    const uint32_t most = rounds * p.workers;
    if (segments <= most / 2 && B <= 32) {
        // lane i tries low + i low / 31; the last one fits: total / cut + segments <= most
        // (ceilings in floating point: a cut that is off by one costs nothing but balance)
        const uint32_t tried = low + (low * lane + 30) / 31, mine = lane < B ? units(lane) : 0;
        const float inverse = 1.0f / static_cast<float>(tried);
        float pieces = 0.0f;
        for (int b = 0; b < B; b++)
            pieces += ceilf(static_cast<float>(__shfl_sync(0xFFFFFFFFu, mine, b)) * inverse);
        const uint32_t fits = __ballot_sync(0xFFFFFFFFu, pieces * segs <= static_cast<float>(most));
        low = __shfl_sync(0xFFFFFFFFu, tried, fits ? __ffs(fits) - 1 : 31);
    } else if (segments <= most / 2 && count_pieces(units, B, segs, low, lane) > most) {
        uint32_t high = 2 * low + 1;  // fits
        while (high - low > 1 + (low >> 5)) {
            const uint32_t mid = low + (high - low) / 2;
            if (count_pieces(units, B, segs, mid, lane) > most)
                low = mid;
            else
                high = mid;
        }
        low = high;
    }
    p.cut = low;
    p.count = count_pieces(units, B, segs, low, lane);
    return p;
}

// By line: the first unit of a cell.
__device__ __forceinline__ uint64_t cell_start(const volatile Plan& p, uint32_t cell) {
    const uint64_t x = static_cast<uint64_t>(cell) * p.cell;
    return x < p.total ? x : p.total;
}

// A sequence among the others, and what precedes it.
struct Place {
    int b;
    uint32_t units_before;   // units of the sequences before it (one segment each)
    uint32_t pieces_before;  // by segment: pieces of those sequences (one segment each)
};

// What precedes each 32nd sequence (units and pieces of one segment each), for as many as kBlocks of them.
constexpr int kBlocks = 64;
struct Before {
    uint32_t units, pieces;
};
constexpr int kUnitsKept = 4096;  // sequences whose units are kept while the plan is made

// The whole warp calls it.
template <typename Units>
__device__ __forceinline__ void make_blocks(const Units& units, int B, uint32_t cut, uint32_t start, int lane,
                                            Before* blocks) {
    Before sum{0, 0};
    for (int i = 0; i * 32 < B; i++) {
        if (lane == 0) blocks[i] = sum;
        const int b = i * 32 + lane;
        const uint32_t n = b < B ? units(b) : 0;
        sum.units += __reduce_add_sync(0xFFFFFFFFu, n ? n + start : 0);
        sum.pieces += __reduce_add_sync(0xFFFFFFFFu, cut ? (n + cut - 1) / cut : 0);
    }
}

// The sequence in which number `id` falls (there is one): of the pieces of one segment of each sequence,
// ceil(n / cut) for n units, or (cut = 0) of its units with its start.  Searched from its block of 32 on, or, with more
// sequences than the blocks cover, from the last place found.  The whole warp calls it.
template <typename Units>
__device__ __forceinline__ Place locate(const Units& units_of, int B, Place at, const Before* blocks, uint32_t id,
                                        uint32_t cut, uint32_t start, int lane) {
    if (B == 1) return at;
    if (B > 32 && B <= 32 * kBlocks) {
        int block = -1;  // the last one that nothing past `id` precedes
#pragma unroll
        for (int i = 0; i < kBlocks; i += 32) {
            const bool reached = (i + lane) * 32 < B && (cut ? blocks[i + lane].pieces : blocks[i + lane].units) <= id;
            block += __popc(__ballot_sync(0xFFFFFFFFu, reached));
        }
        at = Place{block * 32, blocks[block].units, blocks[block].pieces};
    }
    for (;;) {
        const int b = at.b + lane;
        const uint32_t n = b < B ? units_of(b) : 0, p = cut ? (n + cut - 1) / cut : 0;
        const uint32_t line = n ? n + start : 0;
        uint32_t sum = p, units = line;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, sum, o), up_units = __shfl_up_sync(0xFFFFFFFFu, units, o);
            if (lane >= o) sum += up, units += up_units;
        }
        const uint32_t past =
            __ballot_sync(0xFFFFFFFFu, cut ? at.pieces_before + sum > id : at.units_before + units > id);
        if (past) {
            const int f = __ffs(past) - 1;
            at.b += f;
            at.units_before += __shfl_sync(0xFFFFFFFFu, units - line, f);
            at.pieces_before += __shfl_sync(0xFFFFFFFFu, sum - p, f);
            return at;
        }
        at.b += 32;
        at.units_before += __shfl_sync(0xFFFFFFFFu, units, 31);
        at.pieces_before += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
}

template <int FMT, int D, int NT>
__global__ void __launch_bounds__(Shape<FMT, D, NT>::W * 32, 1) attention_kernel(const AttnArgs a) {
    using S = Shape<FMT, D, NT>;
    constexpr int NST = S::NST, KS = S::KS, KEYS = 16 * KS;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint32_t s_word[S::W][2];            // a worker's next piece; whether it joins
    __shared__ float s_ml[S::W * 2 * NT * 8];       // the maxima and sums of the warps
    __shared__ Plan s_plan;
    __shared__ Before s_blocks[kBlocks];
    const int lane = threadIdx.x % 32;
    const uint32_t base = smem_u32(smem);
    // the table, by all warps but the one that plans, and before the previous kernel has finished
    if (FMT == kKvNf4 && threadIdx.x >= 32) {
        for (int i = threadIdx.x - 32; i < 256 * 32; i += S::W * 32 - 32) {
            const int v = i >> 5;
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(kTableAt + v * 256 + (i & 31) * 4),
                         "r"(pack_f16(kTableF16[v & 15], kTableF16[v >> 4]))
                         : "memory");
        }
    }
    pdl_launch_dependents();
    pdl_wait();
    if (base > 4096) {  // not where the areas were laid out for: nothing is computed, and that is reported
        if (threadIdx.x == 0) atomicCAS(&g_attention_error, 0, 44);
        return;
    }

    const uint32_t segs = a.c.kv_heads * a.chunks;  // segments of a sequence
    auto units_of = [&](int b) { return static_cast<uint32_t>(span_of(a, b).units<KEYS>()); };
    // the lengths are read once: one a lane of the planning warp, or by everyone into what will be the rings
    uint32_t* s_units = reinterpret_cast<uint32_t*>(smem);
    if (a.B > 32) {
        for (int b = threadIdx.x; b < a.B && b < kUnitsKept; b += S::W * 32) s_units[b] = units_of(b);
        __syncthreads();
    }
    if (threadIdx.x < 32) {
        const uint32_t mine = a.B <= 32 && lane < a.B ? units_of(lane) : 0;
        auto kept = [&](int b) { return a.B <= 32 ? mine : b < kUnitsKept ? s_units[b] : units_of(b); };
        const Plan p = make_plan<S::W>(kept, a.B, segs, lane);
        if (lane == 0) s_plan = p;
        if (a.B > 32 && a.B <= 32 * kBlocks) make_blocks(kept, a.B, p.cut, p.start, lane, s_blocks);
    }
    __syncthreads();
    // (the plan is read where it is needed: it does not live in registers)
    const volatile Plan& plan = s_plan;
    const uint64_t policy = l2_policy(plan.total > kStreamBytes / static_cast<uint64_t>(S::kStage));
    const int wg = plan.warps, threads = wg * 32;
    const int group = threadIdx.x / threads, tid = threadIdx.x - group * threads, warp = tid / 32;

    const uint32_t ring = area_of<FMT>(base, threadIdx.x / 32, S::kArea);
    auto area = [&](int w) {  // of warp w of this worker, once its ring is drained
        return reinterpret_cast<float*>(smem + (area_of<FMT>(base, group * wg + w, S::kArea) - base));
    };
    const int blocks_per_page = a.c.page_size >> 4;
    WarpState<FMT, D, NT> s;
    Place at{0, 0, 0};
    uint32_t id = blockIdx.x * (S::W / wg) + group, next = 0;
    uint64_t x = 0, stop = 0;  // by line: what is left of the cell
    while (id < plan.count) {
        const uint32_t cut = plan.cut;
        const bool by_line = cut == 0;
        if (x == stop) {
            if (by_line) {
                x = cell_start(plan, id), stop = cell_start(plan, id + 1);
                if (x == stop) break;
                at = locate(units_of, a.B, at, s_blocks, quotient(x, segs), 0, plan.start, lane);
            } else {
                at = locate(units_of, a.B, at, s_blocks, id / segs, cut, 0, lane);
            }
            if (tid == 0) next = plan.count > plan.workers ? atomicAdd(a.tickets, 1u) + plan.workers : 0xFFFFFFFFu;
        }
        // the piece: units [u0, u1) of the n of segment `seg`
        const Span span = span_of(a, at.b);
        const uint32_t n = span.units<KEYS>();
        uint32_t parts = 1, part = 0;  // by segment: of how many it is which
        int seg, u0, u1;
        if (!by_line) {
            parts = (n + cut - 1) / cut;
            const uint32_t in_seq = id - at.pieces_before * segs, len = parts == 1 ? n : (n + parts - 1) / parts;
            seg = static_cast<int>(parts == 1 ? in_seq : in_seq / parts);
            part = in_seq - seg * parts;
            u0 = static_cast<int>(part * len), u1 = static_cast<int>(min(n, part * len + len));
        } else {
            const uint32_t start = plan.start, line = n ? n + start : 0;
            const uint64_t in_seq = x - static_cast<uint64_t>(at.units_before) * segs;
            if (in_seq >= static_cast<uint64_t>(line) * segs) {  // on to the next sequence
                at.units_before += line;
                at.b++;
                continue;
            }
            seg = static_cast<int>(quotient(in_seq, line));
            uint32_t from = static_cast<uint32_t>(in_seq - static_cast<uint64_t>(seg) * line);
            if (from < start) {
                x += start - from, from = start;
                if (x >= stop) break;  // (a worker has one cell)
            }
            const uint64_t left = stop - x;
            u0 = static_cast<int>(from - start);
            u1 = static_cast<int>(left < n - u0 ? u0 + left : n);
            x += u1 - u0;
        }
        const int kv = seg / a.chunks, head0 = (seg - kv * a.chunks) * a.chunk_heads;
        const int heads = min(a.chunk_heads, a.group - head0);
        const int64_t row0 = static_cast<int64_t>(at.b) * a.q_heads + static_cast<int64_t>(kv) * a.group + head0;

        // this warp's units: u0 + warp + WG j, j < mine; lane i holds where block 32 * batch + i of them lies
        const int mine = u1 - u0 > warp ? (u1 - u0 - warp + wg - 1) / wg : 0;
        const int first = span.start / KEYS + u0 + warp;
        auto place_of = [&](int i) -> int64_t {
            const uint32_t block = (first + i / KS * wg) * KS + i % KS;
            // past the warp's units, or nothing live in it: its page is not looked up
            if (i >= mine * KS || block * 16 >= static_cast<uint32_t>(span.end) ||
                block * 16 + 16 <= static_cast<uint32_t>(span.start))
                return -2;
            const uint32_t p = blocks_per_page == 1 ? block : static_cast<uint32_t>(__umul64hi(block, a.page_magic));
            const int64_t page = a.page_table[at.b * a.max_pages + p];
            if (page < 0 || page >= a.c.pages) {
                atomicCAS(&g_attention_error, 0, 43);
                return -1;
            }
            return (page * a.c.kv_heads + kv) * a.c.page_size + (block - p * blocks_per_page) * 16;
        };
        int64_t places = place_of(lane), next_places = mine * KS > 32 ? place_of(32 + lane) : -2;

        uint32_t bad = 0;  // bits of the blocks issued last (the newest lowest): no page
        uint32_t in_buf = ring, out_buf = ring;
        auto issue = [&](int ahead) {
            bad <<= KS;
            if (ahead < mine) {
                if (ahead > 0 && (ahead * KS & 31) == 0) {
                    places = next_places;
                    next_places = place_of(ahead * KS + 32 + lane);
                }
                const int key0 = (first + ahead * wg) * KEYS;
                const int lo = span.start - key0, hi = span.end - key0;
                int64_t place[KS];
                bool fast = lo <= 0 && hi >= KEYS;
#pragma unroll
                for (int b = 0; b < KS; b++) {
                    place[b] = __shfl_sync(0xFFFFFFFFu, places, (ahead * KS + b) & 31);
                    fast = fast && place[b] >= 0;
                }
                if (fast) {
#pragma unroll
                    for (int b = 0; b < KS; b++)
                        copy_block<FMT, D, NT, true>(a.c, in_buf + b * S::kBlock, place[b], 0, 16, lane, policy);
                } else {
#pragma unroll 1
                    for (int b = 0; b < KS; b++) {
                        const int64_t at_b = KS > 1 && b ? place[KS - 1] : place[0];
                        bad |= at_b == -1 ? 1u << b : 0u;
                        copy_edge_block<FMT, D, NT>(a.c, in_buf + b * S::kBlock, at_b, lo - 16 * b, hi - 16 * b, lane,
                                                    policy);
                    }
                }
                in_buf = in_buf + S::kStage == ring + S::kRing ? ring : in_buf + S::kStage;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll 1
        for (int j = 0; j < NST - 1; j++) issue(j);
        load_q<FMT, D, NT>(a, s, a.q + row0 * D, heads, lane);  // while the first stages arrive
#pragma unroll 1
        for (int j = 0; j < mine; j++) {
            cp_async_wait<NST - 2>();
            __syncwarp();  // the stage is complete for every lane, and the one before it is free
            issue(j + NST - 1);
            const int key0 = (first + j * wg) * KEYS, lo = span.start - key0, hi = span.end - key0;
            const uint32_t gone = (bad >> (KS * (NST - 1))) & ((1u << KS) - 1);
            attend_unit<FMT, D, NT>(s, out_buf, lo <= 0 && hi >= KEYS && gone == 0, lo, hi, gone, lane);
            out_buf = out_buf + S::kStage == ring + S::kRing ? ring : out_buf + S::kStage;
        }
        cp_async_wait<0>();
        __syncwarp();  // the warp's ring is drained: its memory takes the warp's result

        const int joiners = min(wg, u1 - u0);  // warps that had a unit
        const bool whole = u0 == 0 && u1 == static_cast<int>(n);
        const bool alone = whole && joiners == 1;  // nothing to join: the warp writes the output
        if (alone && warp == 0) {
            const int g = lane >> 2, t = lane & 3;
            constexpr int RUN = v_run<FMT, D>();
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const int h = nt * 8 + 2 * t + j;
                    float l = s.l[nt][j];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
                    const float back = FMT == kKvBf16 ? 1.0f : (FMT == kKvNf4 ? 1.0f / kTableUnit : 1.0f) / s.vn;
                    const float f = l > 0.0f ? back / l : 0.0f;
                    if (h < heads) {
#pragma unroll
                        for (int i = 0; i < D / 16; i++) {
                            const int dim = (2 * i) / RUN * (8 * RUN) + g * RUN + (2 * i) % RUN;
                            *reinterpret_cast<uint32_t*>(a.out + (row0 + h) * D + dim) =
                                f32x2_to_bf16x2(s.o[nt][i][j] * f, s.o[nt][i][j + 2] * f);
                        }
                    }
                }
        } else if (warp < joiners) {
            float* dst = area(warp);
            const int g = lane >> 2, t = lane & 3;
            const float back = FMT == kKvBf16 ? 1.0f : (FMT == kKvNf4 ? 1.0f / kTableUnit : 1.0f) / s.vn;
            constexpr int RUN = v_run<FMT, D>();
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const int h = nt * 8 + 2 * t + j;
                    float l = s.l[nt][j];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
                    if (h < heads) {
#pragma unroll
                        for (int i = 0; i < D / 16; i++) {
                            const int dim = (2 * i) / RUN * (8 * RUN) + g * RUN + (2 * i) % RUN;
                            *reinterpret_cast<float2*>(dst + h * D + dim) =
                                make_float2(s.o[nt][i][j] * back, s.o[nt][i][j + 2] * back);
                        }
                        if (g == 0) {
                            float* ml = s_ml + (threadIdx.x / 32) * (2 * NT * 8);
                            ml[h] = s.m[nt][j];
                            ml[heads + h] = l;
                        }
                    }
                }
        }
        if (tid == 0) s_word[group][0] = next;
        worker_barrier(group, wg);
        uint2* out = reinterpret_cast<uint2*>(a.out + row0 * D);
        const int columns = heads * (D / 4);
        // The slots of a segment's pieces, one after the other.  By segment: those that are cut have more than `cut`
        // units, so the runs of slots from twice their first unit's quotient are disjoint.  By line: from twice the
        // cell they begin in, since the next one that is cut begins in the cell where this one ends, or later.
        int slot0 = 0;
        if (!whole) {
            const uint64_t before = static_cast<uint64_t>(at.units_before) * segs;
            if (!by_line) {
                slot0 = 2 * static_cast<int>(quotient(before + static_cast<uint64_t>(seg) * n, cut));
            } else {
                const uint32_t start = plan.start, size = plan.cell;
                const uint64_t first_unit = before + static_cast<uint64_t>(seg) * (n + start) + start;
                const uint32_t first_cell = quotient(first_unit, size);
                slot0 = 2 * static_cast<int>(first_cell);
                parts = quotient(first_unit + n - 1, size) - first_cell + 1;
                part = id - first_cell;
            }
        }
        auto slot = [&](int i) { return a.partials + static_cast<int64_t>(slot0 + i) * a.slot_floats; };
        for (int i = alone ? columns : tid; i < columns; i += threads) {
            const Joined r = join<D, 4, true, true>(
                area, [&](int w) { return s_ml + (group * wg + w) * (2 * NT * 8); }, joiners, heads, i);
            if (whole)
                out[i] = normalised(r);
            else
                store_partial<D>(slot(part), r, heads, i);
        }
        // joins `count` slots, `step` apart, once `tickets` says that all of them are there; whether it did
        auto join_slots = [&](uint32_t* ticket, int from, int step, int count, bool last) {
            worker_barrier(group, wg);  // every thread's stores come before the ticket, and its loads after it
            if (tid == 0) s_word[group][1] = ticket_inc(ticket, count - 1) == static_cast<uint32_t>(count - 1);
            worker_barrier(group, wg);
            if (!s_word[group][1]) return false;
            auto piece = [&](int j) { return slot(from + j * step); };
            if (last && count <= 8) {  // everything in one round of loads
                for (int i = tid; i < columns; i += threads)
                    out[i] = normalised(join<D, 8, false, false>(
                        piece, [&](int j) { return piece(j) + heads * D; }, count, heads, i));
                return true;
            }
            // the maxima and sums to shared memory first: one round for all of them, not one for each eight
            float* ml = area(0);
            for (int i = tid; i < count * 2 * heads; i += threads) {
                const int j = i / (2 * heads);
                ml[i] = __ldcg(piece(j) + heads * D + (i - j * 2 * heads));
            }
            worker_barrier(group, wg);
            for (int i = tid; i < columns; i += threads) {
                const Joined r =
                    join<D, 8, false, true>(piece, [&](int j) { return ml + j * 2 * heads; }, count, heads, i);
                if (last)
                    out[i] = normalised(r);
                else  // (into the first of them: nobody but this thread reads its column, nor the sums again)
                    store_partial<D>(slot(from), r, heads, i);
            }
            return true;
        };
        if (!whole) {
            const int from = static_cast<int>(part) / kFanIn * kFanIn, batches = (parts + kFanIn - 1) / kFanIn;
            const int count = min(kFanIn, static_cast<int>(parts) - from);
            if (join_slots(a.joins + slot0 + from, from, 1, count, batches == 1) && batches > 1)
                join_slots(a.joins + kSlots + slot0, 0, kFanIn, batches, true);
        }
        if (x == stop) id = s_word[group][0];
        worker_barrier(group, wg);  // the areas become rings again
    }

    // sequences with nothing to attend to, and lengths past their tables
    for (int b = blockIdx.x * S::W + threadIdx.x / 32; b < a.B; b += gridDim.x * S::W) {
        if (lane == 0 && a.lengths[b] > a.max_pages * a.c.page_size) atomicCAS(&g_attention_error, 0, 43);
        if (span_of(a, b).units<KEYS>() == 0)
            for (int i = lane; i < a.q_heads * (D / 8); i += 32)
                reinterpret_cast<uint4*>(a.out)[static_cast<int64_t>(b) * (a.q_heads * (D / 8)) + i] =
                    make_uint4(0, 0, 0, 0);
    }
    // the last worker leaves the tickets as it found them
    if (tid == 0 && plan.count > plan.workers) {
        const uint32_t last = plan.workers - 1;
        if (ticket_inc(a.tickets + 1, last) == last) a.tickets[0] = 0;
    }
}

int slot_floats(int chunk_heads, int D) { return (chunk_heads * (D + 2) + 3) / 4 * 4; }

template <int FMT, int D, int NT>
cudaError_t launch(const AttnArgs& a, int num_sms, cudaStream_t stream) {
    using S = Shape<FMT, D, NT>;
    static std::once_flag attr_once[64];  // once per device
    int dev = 0;
    cudaGetDevice(&dev);
    cudaError_t attr_err = cudaSuccess;
    std::call_once(attr_once[dev & 63], [&] {
        attr_err = cudaFuncSetAttribute(attention_kernel<FMT, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        S::kSmem);
    });
    if (attr_err != cudaSuccess) return attr_err;
    // as many CTAs as SMs, or fewer where there are fewer segments and the longest possible sequences leave less to do
    const int64_t segments = static_cast<int64_t>(a.B) * a.c.kv_heads * a.chunks;
    const int64_t units = segments * ((a.max_pages * a.c.page_size + 16 * S::KS - 1) / (16 * S::KS));
    const int64_t useful = std::max(segments, (units + S::W - 1) / S::W);
    int64_t grid = std::min(num_sms, kMaxWorkers / 2);
    if (grid > useful) grid = useful;
    if (grid < 1) grid = 1;
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(grid)), S::W * 32, stream, &attr);
    cfg.dynamicSmemBytes = S::kSmem;
    return cudaLaunchKernelEx(&cfg, attention_kernel<FMT, D, NT>, a);
}

// Query heads of a kv head in groups of at most 16, as even as they come.
void head_chunks(int group, int* chunks, int* chunk_heads) {
    *chunks = (group + 15) / 16;
    *chunk_heads = (group + *chunks - 1) / *chunks;
}

template <int FMT, int D>
cudaError_t launch_nt(const AttnArgs& a, int num_sms, cudaStream_t stream) {
    return a.chunk_heads > 8 ? launch<FMT, D, 2>(a, num_sms, stream) : launch<FMT, D, 1>(a, num_sms, stream);
}

template <int FMT>
cudaError_t launch_d(const AttnArgs& a, int num_sms, cudaStream_t stream) {
    return a.c.head_dim == 64    ? launch_nt<FMT, 64>(a, num_sms, stream)
           : a.c.head_dim == 128 ? launch_nt<FMT, 128>(a, num_sms, stream)
                                 : launch_nt<FMT, 256>(a, num_sms, stream);
}

}  // namespace

// Workspace: the tickets (zero before the first use, and again after each call), then the partial results.
constexpr int kControlBytes = (16 + 2 * kSlots * 4 + 255) / 256 * 256;
int64_t attention_workspace_bytes(int kv_heads, int head_dim, int64_t, int64_t q_heads) {
    int chunks, chunk_heads;
    head_chunks(static_cast<int>(q_heads / kv_heads), &chunks, &chunk_heads);
    return kControlBytes + static_cast<int64_t>(kSlots) * slot_floats(chunk_heads, head_dim) * 4;
}

cudaError_t launch_attention(const KvCache& c, const uint16_t* q, const int32_t* page_table, int64_t max_pages,
                             const int32_t* lengths, int64_t B, int64_t q_heads, float scale, int64_t window,
                             uint16_t* out, void* workspace, int num_sms, cudaStream_t stream) {
    AttnArgs a{};
    a.c = c;
    a.q = q, a.page_table = page_table, a.lengths = lengths, a.out = out;
    a.tickets = static_cast<uint32_t*>(workspace);
    a.joins = a.tickets + 4;
    a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kControlBytes);
    a.max_pages = max_pages, a.window = window;
    const uint64_t upp = static_cast<uint64_t>(c.page_size / 16);
    a.page_magic = upp > 1 ? ~uint64_t{0} / upp + 1 : 0;
    a.B = static_cast<int>(B), a.q_heads = static_cast<int>(q_heads);
    a.group = static_cast<int>(q_heads / c.kv_heads);
    head_chunks(a.group, &a.chunks, &a.chunk_heads);
    a.slot_floats = slot_floats(a.chunk_heads, c.head_dim);
    a.scale = scale;
    switch (c.format) {
        case kKvBf16: return launch_d<kKvBf16>(a, num_sms, stream);
        case kKvFp8: return launch_d<kKvFp8>(a, num_sms, stream);
        default: return launch_d<kKvNf4>(a, num_sms, stream);
    }
}

cudaError_t read_and_clear_attention_error(int* code) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_attention_error, sizeof(int));
    if (e != cudaSuccess) return e;
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_attention_error, &zero, sizeof(int));
    *code = v;
    return e;
}

}  // namespace nf4
