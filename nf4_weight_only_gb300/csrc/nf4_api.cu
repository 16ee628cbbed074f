// C ABI of libnf4.so: argument checks, the per-device capability check and the M-based dispatch.
#include <atomic>
#include <cstdint>

#include <cuda_runtime_api.h>

#include "../../include/nf4.h"
#include "nf4_internal.h"

namespace nf4 {
int64_t gemv_max_k(int64_t M);
}

namespace {

constexpr int kMaxDevices = 64;

// The last CUDA error this host thread saw inside the library (read by nf4_last_cuda_error).
thread_local cudaError_t g_last_cuda_error = cudaSuccess;
constexpr int64_t kMaxDim = 0x7FFFFFFF;
constexpr int64_t kMaxVectors = int64_t{1} << 40;  // of one side of a cache

// Per-device cache: 0 = unknown, -1 = unsupported, otherwise the SM count of a 10.3 device.
std::atomic<int> g_device_sms[kMaxDevices];

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a_bytes > 0 && b_bytes > 0 && a0 < b0 + static_cast<uintptr_t>(b_bytes) &&
           b0 < a0 + static_cast<uintptr_t>(a_bytes);
}

nf4_status check_k(int64_t K) {
    if (K <= 0 || K % NF4_GROUP_SIZE != 0 || K > kMaxDim) return NF4_ERR_SHAPE;
    return NF4_OK;
}

// Current device must be compute capability 10.3; returns its SM count through `sms`.
nf4_status current_device(int* device, int* sms) {
    if (cudaGetDevice(device) != cudaSuccess) {
        g_last_cuda_error = cudaGetLastError();
        return NF4_ERR_CUDA;
    }
    if (*device < 0 || *device >= kMaxDevices) return NF4_ERR_UNSUPPORTED_DEVICE;
    int cached = g_device_sms[*device].load(std::memory_order_relaxed);
    if (cached == 0) {
        int major = 0, minor = 0, count = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *device) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *device) != cudaSuccess ||
            cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, *device) != cudaSuccess) {
            g_last_cuda_error = cudaGetLastError();
            return NF4_ERR_CUDA;
        }
        cached = (major == 10 && minor == 3 && count > 0) ? count : -1;
        g_device_sms[*device].store(cached, std::memory_order_relaxed);
    }
    if (cached < 0) return NF4_ERR_UNSUPPORTED_DEVICE;
    *sms = cached;
    return NF4_OK;
}

nf4_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return NF4_OK;
    g_last_cuda_error = e;
    cudaGetLastError();
    return NF4_ERR_CUDA;
}

// A cache description: sizes first, then (for a cache that holds anything) its pointers.
nf4_status check_cache(const nf4_kv_cache* c) {
    if (!c) return NF4_ERR_NULL;
    if (c->format < NF4_KV_BF16 || c->format > NF4_KV_NF4) return NF4_ERR_SHAPE;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return NF4_ERR_SHAPE;
    if (c->page_size < 16 || c->page_size > 65536 || c->page_size % 16 != 0) return NF4_ERR_SHAPE;
    if (c->kv_heads < 1 || c->kv_heads > 65535 || c->pages < 0 || c->pages > kMaxDim) return NF4_ERR_SHAPE;
    // (at 32 bytes a vector or more no memory holds that many; the byte counts below fit 64 bits)
    if (c->pages > kMaxVectors / (static_cast<int64_t>(c->kv_heads) * c->page_size)) return NF4_ERR_SHAPE;
    if (c->pages == 0) return NF4_OK;
    const bool scaled = c->format != NF4_KV_BF16;
    if (!c->k || !c->v || (scaled && (!c->k_scales || !c->v_scales))) return NF4_ERR_NULL;
    if (!aligned16(c->k) || !aligned16(c->v)) return NF4_ERR_ALIGN;
    if (scaled && (!aligned16(c->k_scales) || !aligned16(c->v_scales))) return NF4_ERR_ALIGN;
    return NF4_OK;
}

// The byte ranges of a cache: k, v, k_scales, v_scales (unused ones empty).
struct Ranges {
    const void* p[4];
    int64_t n[4];
};
Ranges cache_ranges(const nf4_kv_cache* c) {
    const int64_t places = c->pages * c->kv_heads * c->page_size;
    const int64_t vec = c->format == NF4_KV_BF16 ? 2 * c->head_dim : c->format == NF4_KV_FP8 ? c->head_dim : c->head_dim / 2;
    const int64_t sc = c->format == NF4_KV_BF16 ? 0 : c->format == NF4_KV_FP8 ? 4 : c->head_dim / NF4_GROUP_SIZE * 2;
    return {{c->k, c->v, c->k_scales, c->v_scales}, {places * vec, places * vec, places * sc, places * sc}};
}
bool overlaps_cache(const Ranges& r, const void* p, int64_t bytes) {
    for (int i = 0; i < 4; i++)
        if (overlap(r.p[i], r.n[i], p, bytes)) return true;
    return false;
}

bool attention_sizes_ok(const nf4_kv_cache* c, int64_t B, int64_t q_heads) {
    return B >= 0 && B <= 65535 && q_heads >= 1 && q_heads <= 65535 && q_heads % c->kv_heads == 0 &&
           B * q_heads <= (int64_t{1} << 30);
}

nf4::KvCache device_cache(const nf4_kv_cache* c) {
    return {static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), static_cast<uint8_t*>(c->k_scales),
            static_cast<uint8_t*>(c->v_scales), c->pages, c->kv_heads, c->page_size, c->head_dim, c->format};
}

}  // namespace

namespace nf4 {
int abi_current_device(int* device, int* sms) { return current_device(device, sms); }
void note_cuda_error(cudaError_t e) {
    if (e != cudaSuccess) g_last_cuda_error = e;
}
}  // namespace nf4

extern "C" {

const char* nf4_status_str(nf4_status status) {
    switch (status) {
        case NF4_OK: return "NF4_OK";
        case NF4_ERR_NULL: return "NF4_ERR_NULL: a required pointer is NULL";
        case NF4_ERR_SHAPE: return "NF4_ERR_SHAPE: bad size (K must be a positive multiple of 64; sizes <= 2^31-1)";
        case NF4_ERR_ALIGN: return "NF4_ERR_ALIGN: a pointer is not 16-byte aligned";
        case NF4_ERR_ALIAS: return "NF4_ERR_ALIAS: an output overlaps an input";
        case NF4_ERR_UNSUPPORTED_DEVICE: return "NF4_ERR_UNSUPPORTED_DEVICE: current device is not sm_103";
        case NF4_ERR_CUDA: return "NF4_ERR_CUDA: a CUDA call or launch failed";
        case NF4_ERR_MEMORY: return "NF4_ERR_MEMORY: host memory not page-locked, or a ring used on another device";
        case NF4_ERR_CAPTURE:
            return "NF4_ERR_CAPTURE: first nf4_linear_host_noalloc call on this device made under stream capture (make one call outside capture first)";
    }
    return "NF4 status: unknown code";
}

int nf4_abi_version(void) { return NF4_ABI_VERSION; }

const char* nf4_last_cuda_error(void) { return cudaGetErrorName(g_last_cuda_error); }

nf4_status nf4_linear_grouped(const uint16_t* x, int64_t M, int64_t K, int count, const uint8_t* const* codes,
                              const uint16_t* const* scales, uint16_t* const* ys, const int64_t* Ns,
                              cudaStream_t stream) {
    if (count < 1 || count > nf4::kMaxGroupedLinears) return NF4_ERR_SHAPE;
    if (!codes || !scales || !ys || !Ns) return NF4_ERR_NULL;
    if (M < 0 || M > kMaxDim) return NF4_ERR_SHAPE;
    nf4_status st = check_k(K);
    if (st != NF4_OK) return st;
    int64_t rows = 0;
    for (int i = 0; i < count; i++) {
        if (Ns[i] < 0 || Ns[i] > kMaxDim) return NF4_ERR_SHAPE;
        rows += Ns[i];
    }
    if (rows > kMaxDim) return NF4_ERR_SHAPE;
    if (M == 0 || rows == 0) return NF4_OK;
    if (!x) return NF4_ERR_NULL;
    if (!aligned16(x)) return NF4_ERR_ALIGN;
    const int64_t xb = M * K * 2;
    for (int i = 0; i < count; i++) {
        if (Ns[i] == 0) continue;
        if (!codes[i] || !scales[i] || !ys[i]) return NF4_ERR_NULL;
        if (!aligned16(codes[i]) || !aligned16(scales[i]) || !aligned16(ys[i])) return NF4_ERR_ALIGN;
    }
    for (int i = 0; i < count; i++) {
        if (Ns[i] == 0) continue;
        const int64_t yb = M * Ns[i] * 2;
        if (overlap(ys[i], yb, x, xb)) return NF4_ERR_ALIAS;
        for (int j = 0; j < count; j++) {
            if (Ns[j] == 0) continue;
            const int64_t cb = Ns[j] * K / 2, sb = Ns[j] * (K / NF4_GROUP_SIZE) * 2;
            if (overlap(ys[i], yb, codes[j], cb) || overlap(ys[i], yb, scales[j], sb)) return NF4_ERR_ALIAS;
            if (j != i && overlap(ys[i], yb, ys[j], M * Ns[j] * 2)) return NF4_ERR_ALIAS;
        }
    }
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms)) != NF4_OK) return st;
    // drop empty problems, keep the order
    const uint8_t* c[nf4::kMaxGroupedLinears];
    const uint16_t* sc[nf4::kMaxGroupedLinears];
    uint16_t* yy[nf4::kMaxGroupedLinears];
    int64_t nn[nf4::kMaxGroupedLinears];
    int k = 0;
    for (int i = 0; i < count; i++)
        if (Ns[i] > 0) {
            c[k] = codes[i];
            sc[k] = scales[i];
            yy[k] = ys[i];
            nn[k] = Ns[i];
            k++;
        }
    if (M <= nf4::kGemvMaxTokens && K <= nf4::gemv_max_k(M))
        return from_cuda(nf4::launch_gemv_grouped(x, k, c, sc, yy, nn, M, K, sms, stream));
    return from_cuda(nf4::launch_stream(x, k, c, sc, yy, nn, M, K, sms, stream));
}

nf4_status nf4_check_device_error(int* code) {
    if (!code) return NF4_ERR_NULL;
    *code = 0;
    int dev = 0, sms = 0;
    nf4_status st = current_device(&dev, &sms);
    if (st != NF4_OK) return st;
    int linear = 0, embed = 0, kv = 0, attention = 0;
    if ((st = from_cuda(nf4::read_and_clear_error(&linear))) != NF4_OK) return st;
    if ((st = from_cuda(nf4::read_and_clear_embed_error(&embed))) != NF4_OK) return st;
    if ((st = from_cuda(nf4::read_and_clear_kv_error(&kv))) != NF4_OK) return st;
    if ((st = from_cuda(nf4::read_and_clear_attention_error(&attention))) != NF4_OK) return st;
    *code = linear ? linear : embed ? embed : kv ? kv : attention;
    return NF4_OK;
}

nf4_status nf4_diag_bounded_wait(int64_t ns, cudaStream_t stream) {
    if (ns <= 0 || ns > (int64_t{1} << 31)) return NF4_ERR_SHAPE;
    int dev = 0, sms = 0;
    nf4_status st = current_device(&dev, &sms);
    if (st != NF4_OK) return st;
    return from_cuda(nf4::launch_diag_wait(ns, stream));
}

nf4_status nf4_diag_set_wait_limit(int64_t ns, cudaStream_t stream) {
    if (ns < 0 || ns > (int64_t{1} << 36)) return NF4_ERR_SHAPE;
    int dev = 0, sms = 0;
    nf4_status st = current_device(&dev, &sms);
    if (st != NF4_OK) return st;
    return from_cuda(nf4::set_wait_limit(ns, stream));
}

nf4_status nf4_embed(const int32_t* ids, int64_t n_ids, const uint8_t* codes, const uint16_t* scales, int64_t V,
                     int64_t K, uint16_t* out, cudaStream_t stream) {
    if (n_ids < 0 || V < 0 || n_ids > kMaxDim || V > kMaxDim) return NF4_ERR_SHAPE;
    nf4_status st = check_k(K);
    if (st != NF4_OK) return st;
    if (n_ids == 0) return NF4_OK;
    if (!ids || !out || (V > 0 && (!codes || !scales))) return NF4_ERR_NULL;
    if (!aligned16(ids) || !aligned16(out) || (V > 0 && (!aligned16(codes) || !aligned16(scales))))
        return NF4_ERR_ALIGN;
    const int64_t ob = n_ids * K * 2, ib = n_ids * 4, cb = V * K / 2, sb = V * (K / NF4_GROUP_SIZE) * 2;
    if (overlap(out, ob, ids, ib) || overlap(out, ob, codes, cb) || overlap(out, ob, scales, sb)) return NF4_ERR_ALIAS;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms)) != NF4_OK) return st;
    return from_cuda(nf4::launch_embed(ids, n_ids, codes, scales, V, K, out, sms, stream));
}

nf4_status nf4_quantize(const float* w, int64_t N, int64_t K, uint8_t* codes, uint16_t* scales,
                        cudaStream_t stream) {
    if (N < 0 || N > kMaxDim) return NF4_ERR_SHAPE;
    nf4_status st = check_k(K);
    if (st != NF4_OK) return st;
    if (N == 0) return NF4_OK;
    if (!w || !codes || !scales) return NF4_ERR_NULL;
    if (!aligned16(w) || !aligned16(codes) || !aligned16(scales)) return NF4_ERR_ALIGN;
    const int64_t wb = N * K * 4, cb = N * K / 2, sb = N * (K / NF4_GROUP_SIZE) * 2;
    if (overlap(codes, cb, w, wb) || overlap(scales, sb, w, wb) || overlap(codes, cb, scales, sb))
        return NF4_ERR_ALIAS;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms)) != NF4_OK) return st;
    return from_cuda(nf4::launch_quantize(w, N, K, codes, scales, sms, stream));
}

nf4_status nf4_dequant(const uint8_t* codes, const uint16_t* scales, int64_t N, int64_t K, uint16_t* w_hat,
                       cudaStream_t stream) {
    if (N < 0 || N > kMaxDim) return NF4_ERR_SHAPE;
    nf4_status st = check_k(K);
    if (st != NF4_OK) return st;
    if (N == 0) return NF4_OK;
    if (!codes || !scales || !w_hat) return NF4_ERR_NULL;
    if (!aligned16(codes) || !aligned16(scales) || !aligned16(w_hat)) return NF4_ERR_ALIGN;
    const int64_t ob = N * K * 2, cb = N * K / 2, sb = N * (K / NF4_GROUP_SIZE) * 2;
    if (overlap(w_hat, ob, codes, cb) || overlap(w_hat, ob, scales, sb)) return NF4_ERR_ALIAS;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms)) != NF4_OK) return st;
    return from_cuda(nf4::launch_dequant(codes, scales, N, K, w_hat, sms, stream));
}

nf4_status nf4_linear(const uint16_t* x, const uint8_t* codes, const uint16_t* scales, uint16_t* y, int64_t M,
                      int64_t N, int64_t K, cudaStream_t stream) {
    if (M < 0 || N < 0 || M > kMaxDim || N > kMaxDim) return NF4_ERR_SHAPE;
    nf4_status st = check_k(K);
    if (st != NF4_OK) return st;
    if (M == 0 || N == 0) return NF4_OK;
    if (!x || !codes || !scales || !y) return NF4_ERR_NULL;
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scales) || !aligned16(y)) return NF4_ERR_ALIGN;
    const int64_t yb = M * N * 2, xb = M * K * 2, cb = N * K / 2, sb = N * (K / NF4_GROUP_SIZE) * 2;
    if (overlap(y, yb, x, xb) || overlap(y, yb, codes, cb) || overlap(y, yb, scales, sb)) return NF4_ERR_ALIAS;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms)) != NF4_OK) return st;
    if (M <= nf4::kGemvMaxTokens && K <= nf4::gemv_max_k(M))
        return from_cuda(nf4::launch_gemv(x, codes, scales, y, M, N, K, sms, stream));
    return from_cuda(nf4::launch_stream(x, 1, &codes, &scales, &y, &N, M, K, sms, stream));
}

nf4_status nf4_kv_append(const nf4_kv_cache* cache, const uint16_t* k, const uint16_t* v, const int64_t* slots,
                         int64_t T, cudaStream_t stream) {
    nf4_status st = check_cache(cache);
    if (st != NF4_OK) return st;
    if (T < 0 || T > kMaxDim) return NF4_ERR_SHAPE;
    if (T == 0) return NF4_OK;
    if (!k || !v || !slots) return NF4_ERR_NULL;
    if (!aligned16(k) || !aligned16(v) || !aligned16(slots)) return NF4_ERR_ALIGN;
    const Ranges r = cache_ranges(cache);
    const int64_t in = T * cache->kv_heads * cache->head_dim * 2;
    if (overlaps_cache(r, k, in) || overlaps_cache(r, v, in) || overlaps_cache(r, slots, T * 8)) return NF4_ERR_ALIAS;
    for (int i = 0; i < 4; i++)
        for (int j = i + 1; j < 4; j++)
            if (overlap(r.p[i], r.n[i], r.p[j], r.n[j])) return NF4_ERR_ALIAS;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms)) != NF4_OK) return st;
    return from_cuda(nf4::launch_kv_append(device_cache(cache), k, v, slots, T, sms, stream));
}

nf4_status nf4_kv_read(const nf4_kv_cache* cache, const int64_t* slots, int64_t T, uint16_t* k, uint16_t* v,
                       cudaStream_t stream) {
    nf4_status st = check_cache(cache);
    if (st != NF4_OK) return st;
    if (T < 0 || T > kMaxDim) return NF4_ERR_SHAPE;
    if (T == 0 || (!k && !v)) return NF4_OK;
    if (!slots) return NF4_ERR_NULL;
    if (!aligned16(k) || !aligned16(v) || !aligned16(slots)) return NF4_ERR_ALIGN;
    const Ranges r = cache_ranges(cache);
    const int64_t ob = T * cache->kv_heads * cache->head_dim * 2;
    if ((k && (overlaps_cache(r, k, ob) || overlap(k, ob, slots, T * 8))) ||
        (v && (overlaps_cache(r, v, ob) || overlap(v, ob, slots, T * 8))) || (k && v && overlap(k, ob, v, ob)))
        return NF4_ERR_ALIAS;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms)) != NF4_OK) return st;
    return from_cuda(nf4::launch_kv_read(device_cache(cache), slots, T, k, v, sms, stream));
}

int64_t nf4_attention_workspace_bytes(const nf4_kv_cache* cache, int64_t B, int64_t q_heads) {
    if (!cache || check_cache(cache) == NF4_ERR_SHAPE || !attention_sizes_ok(cache, B, q_heads)) return -1;
    return nf4::attention_workspace_bytes(cache->kv_heads, cache->head_dim, B, q_heads);
}

nf4_status nf4_attention_decode(const nf4_kv_cache* cache, const uint16_t* q, const int32_t* page_table,
                                int64_t max_pages, const int32_t* lengths, int64_t B, int64_t q_heads, float scale,
                                int64_t window, uint16_t* out, void* workspace, int64_t workspace_bytes,
                                cudaStream_t stream) {
    nf4_status st = check_cache(cache);
    if (st != NF4_OK) return st;
    if (!attention_sizes_ok(cache, B, q_heads)) return NF4_ERR_SHAPE;
    if (max_pages < 0 || max_pages > kMaxDim || max_pages * cache->page_size > kMaxDim || window < 0) return NF4_ERR_SHAPE;
    if (max_pages > 0 && B > (int64_t{1} << 35) / (max_pages * cache->page_size)) return NF4_ERR_SHAPE;
    if (B == 0) return NF4_OK;
    if (!q || !lengths || !out || !workspace || (max_pages > 0 && !page_table)) return NF4_ERR_NULL;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace)) return NF4_ERR_ALIGN;
    if (!aligned4(lengths) || !aligned4(page_table)) return NF4_ERR_ALIGN;
    const int64_t need = nf4::attention_workspace_bytes(cache->kv_heads, cache->head_dim, B, q_heads);
    if (workspace_bytes < need) return NF4_ERR_SHAPE;
    const Ranges r = cache_ranges(cache);
    const int64_t qb = B * q_heads * cache->head_dim * 2, tb = B * max_pages * 4;
    const void* outs[2] = {out, workspace};
    const int64_t ons[2] = {qb, need};
    for (int i = 0; i < 2; i++)
        if (overlaps_cache(r, outs[i], ons[i]) || overlap(outs[i], ons[i], q, qb) ||
            overlap(outs[i], ons[i], page_table, tb) || overlap(outs[i], ons[i], lengths, B * 4))
            return NF4_ERR_ALIAS;
    if (overlap(out, qb, workspace, need)) return NF4_ERR_ALIAS;
    int dev = 0, sms = 0;
    if ((st = current_device(&dev, &sms)) != NF4_OK) return st;
    return from_cuda(nf4::launch_attention(device_cache(cache), q, page_table, max_pages, lengths, B, q_heads, scale,
                                           window, out, workspace, sms, stream));
}

nf4_status nf4_rope(const uint16_t* q, int64_t q_heads, const uint16_t* k, int64_t k_heads, int64_t T, int64_t head_dim,
                    const int32_t* positions, int axes, const int32_t* sections, const float* inv_freq,
                    int64_t rotary_dim, int interleaved, float magnitude, uint16_t* q_out, uint16_t* k_out,
                    cudaStream_t stream) {
    if (T < 0 || T > kMaxDim || q_heads < 0 || q_heads > 65535 || k_heads < 0 || k_heads > 65535) return NF4_ERR_SHAPE;
    if (head_dim < 16 || head_dim % 16 != 0 || head_dim > (1 << 24) || (q_heads + k_heads) * head_dim > (1 << 24))
        return NF4_ERR_SHAPE;
    if (rotary_dim < 16 || rotary_dim > head_dim || rotary_dim > 256 || rotary_dim % 16 != 0) return NF4_ERR_SHAPE;
    if (axes < 1 || axes > 4) return NF4_ERR_SHAPE;
    if (!sections) return NF4_ERR_NULL;
    nf4::RopeArgs a{};
    int64_t pairs = 0;
    for (int i = 0; i < 4; i++) {
        if (i < axes) {
            if (sections[i] < 0) return NF4_ERR_SHAPE;
            pairs += sections[i];
        }
        a.section_end[i] = static_cast<int>(pairs > kMaxDim ? kMaxDim : pairs);
    }
    if (pairs != rotary_dim / 2) return NF4_ERR_SHAPE;
    if (T == 0 || q_heads + k_heads == 0) return NF4_OK;
    if (!positions || !inv_freq || (q_heads && (!q || !q_out)) || (k_heads && (!k || !k_out))) return NF4_ERR_NULL;
    const void* ins[4] = {positions, inv_freq, q_heads ? q : nullptr, k_heads ? k : nullptr};
    const void* outs[2] = {q_heads ? q_out : nullptr, k_heads ? k_out : nullptr};
    const int64_t in_bytes[4] = {axes * T * 4, rotary_dim * 2, T * q_heads * head_dim * 2, T * k_heads * head_dim * 2};
    if (!aligned4(positions)) return NF4_ERR_ALIGN;
    for (int i = 1; i < 4; i++)
        if (!aligned16(ins[i])) return NF4_ERR_ALIGN;
    for (const void* p : outs)
        if (!aligned16(p)) return NF4_ERR_ALIGN;
    for (int o = 0; o < 2; o++)
        for (int i = 0; i < 4; i++)
            if (!(i == o + 2 && outs[o] == ins[i]) && overlap(outs[o], in_bytes[o + 2], ins[i], in_bytes[i]))
                return NF4_ERR_ALIAS;
    if (overlap(outs[0], in_bytes[2], outs[1], in_bytes[3])) return NF4_ERR_ALIAS;
    int dev = 0, sms = 0;
    nf4_status st = current_device(&dev, &sms);
    if (st != NF4_OK) return st;
    a.q = q, a.k = k, a.q_out = q_out, a.k_out = k_out, a.positions = positions, a.inv_freq = inv_freq;
    a.T = T, a.q_heads = static_cast<int>(q_heads), a.k_heads = static_cast<int>(k_heads);
    a.head_dim = static_cast<int>(head_dim), a.rotary_dim = static_cast<int>(rotary_dim), a.axes = axes;
    a.interleaved = interleaved != 0, a.magnitude = magnitude;
    return from_cuda(nf4::launch_rope(a, sms, stream));
}

nf4_status nf4_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int64_t T, int64_t H,
                       float eps, uint16_t* residual_out, uint16_t* y, uint8_t* y8, float* y8_scales,
                       cudaStream_t stream) {
    if (T < 0 || T > kMaxDim || H <= 0 || H > kMaxDim || H % 8 != 0) return NF4_ERR_SHAPE;
    if (T == 0) return NF4_OK;
    if (!x || !weight || (!y && !y8) || (y8 != nullptr) != (y8_scales != nullptr)) return NF4_ERR_NULL;
    const void* all[7] = {x, residual, weight, residual_out, y, y8, y8_scales};
    const int64_t n[7] = {T * H * 2, T * H * 2, H * 2, T * H * 2, T * H * 2, T * H, T * 4};
    for (const void* p : all)
        if (!aligned16(p)) return NF4_ERR_ALIGN;
    for (int o = 3; o < 7; o++)
        for (int i = 0; i < 7; i++) {
            if (i == o || !all[o] || !all[i]) continue;
            const bool same = all[o] == all[i] && ((o == 3 && i <= 1) || (o == 4 && i == 0));  // in place
            if (!same && overlap(all[o], n[o], all[i], n[i])) return NF4_ERR_ALIAS;
        }
    int dev = 0, sms = 0;
    nf4_status st = current_device(&dev, &sms);
    if (st != NF4_OK) return st;
    return from_cuda(nf4::launch_rmsnorm(x, residual, weight, T, H, eps, residual_out, y, y8, y8_scales, sms, stream));
}

}  // extern "C"
