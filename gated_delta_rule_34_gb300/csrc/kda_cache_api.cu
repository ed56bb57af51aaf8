// kda_cache_api.cu -- the C ABI of the global-attention operators: rotary positions,
// the paged 8-bit cache and the attention over it.
//
// Every check happens on the host before anything is launched; nothing here
// reads device memory.
#include <cmath>
#include <cstdint>

#include "kda_cache_internal.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

kda_status ok() { return kda::report(KDA_OK, "%s", ""); }

kda_status launched(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return ok();
    return kda::report(KDA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
    return sms > 0 ? sms : 148;
}

#define KDA_REQUIRE(cond, status, ...)                        \
    do {                                                      \
        if (!(cond)) return kda::report(status, __VA_ARGS__); \
    } while (0)

#define KDA_POINTER(p, bytes)                                                                   \
    do {                                                                                        \
        KDA_REQUIRE((p) != nullptr, KDA_ERR_INVALID_ARG, "%s is NULL", #p);                     \
        KDA_REQUIRE(aligned(p, bytes), KDA_ERR_INVALID_ARG, "%s is not %d-byte aligned", #p,    \
                    (int)(bytes));                                                              \
    } while (0)

bool valid_dtype(kda_dtype d) { return d == KDA_DTYPE_F32 || d == KDA_DTYPE_BF16; }
int element_size(kda_dtype d) { return d == KDA_DTYPE_BF16 ? 2 : 4; }

// A stride between tokens whose rows are H * d dense elements and start on 16 bytes.
kda_status check_stride(const char* name, int64_t stride, int64_t row, kda_dtype dtype) {
    KDA_REQUIRE(stride >= row, KDA_ERR_INVALID_ARG, "%s = %lld is less than a row of %lld elements",
                name, (long long)stride, (long long)row);
    KDA_REQUIRE(stride * element_size(dtype) % 16 == 0, KDA_ERR_INVALID_ARG,
                "%s = %lld: rows must start on 16-byte boundaries", name, (long long)stride);
    return KDA_OK;
}
#define KDA_STRIDE(s, row)                                                     \
    do {                                                                       \
        const kda_status st_ = check_stride(#s, s, row, dtype);                \
        if (st_ != KDA_OK) return st_;                                         \
    } while (0)

kda_status check_pool(int H_kv, int d, int64_t n_pages, int page, int table_pages) {
    KDA_REQUIRE(H_kv > 0 && d > 0 && n_pages >= 0 && table_pages >= 0, KDA_ERR_INVALID_ARG,
                "bad sizes H_kv=%d d=%d n_pages=%lld table_pages=%d", H_kv, d, (long long)n_pages,
                table_pages);
    KDA_REQUIRE(d % 16 == 0 && d <= 128, KDA_ERR_UNSUPPORTED,
                "the cache takes d a multiple of 16 up to 128 (d=%d)", d);
    KDA_REQUIRE(page >= 16 && page <= 256 && (page & (page - 1)) == 0, KDA_ERR_UNSUPPORTED,
                "a page is 16, 32, 64, 128 or 256 tokens (%d)", page);
    KDA_REQUIRE(H_kv <= 65535, KDA_ERR_UNSUPPORTED, "H_kv must be <= 65535 (%d)", H_kv);
    KDA_REQUIRE(n_pages <= INT32_MAX, KDA_ERR_UNSUPPORTED, "n_pages must be below 2^31");
    return KDA_OK;
}

int log2_of(int n) {
    int s = 0;
    while ((1 << s) < n) ++s;
    return s;
}

kda_status make_span(kda::CacheSpan& w, bool packed, int n_seqs, int64_t T, int H_kv, int d,
                     int64_t n_pages, int page, int table_pages) {
    KDA_REQUIRE(n_seqs >= 0 && T >= 0, KDA_ERR_INVALID_ARG, "bad sizes n_seqs=%d T=%lld", n_seqs,
                (long long)T);
    const kda_status st = check_pool(H_kv, d, n_pages, page, table_pages);
    if (st != KDA_OK) return st;
    // positions are 32-bit: no sequence brings more tokens than they count
    KDA_REQUIRE(T <= INT32_MAX, KDA_ERR_UNSUPPORTED, "T must be below 2^31 (%lld)", (long long)T);
    w.n_seqs = n_seqs;
    w.H = H_kv;
    w.d = d;
    w.page_shift = log2_of(page);
    w.n_pages = n_pages;
    w.table_pages = table_pages;
    w.T = packed ? 0 : T;
    w.rows = packed ? T : T * n_seqs;
    w.slots_per_seq = packed ? 0 : (T + 2 * page - 2) / page;
    KDA_REQUIRE(kda::cache_slots(w, packed) <= INT32_MAX / (2 * (int64_t)H_kv), KDA_ERR_UNSUPPORTED,
                "too many pages and heads for one call (%d sequences, %lld tokens, %d heads)", n_seqs,
                (long long)w.rows, H_kv);
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_rotary(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int H_q,
                      const void* k, int64_t k_stride, void* k_out, int64_t k_out_stride, int H_k,
                      const int32_t* positions, const double* freq, float amplitude,
                      int64_t n_tokens, int d, int rot, kda_rotary_layout layout, kda_dtype dtype,
                      cudaStream_t stream) {
    KDA_REQUIRE(valid_dtype(dtype), KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    KDA_REQUIRE(layout == KDA_ROTARY_HALF || layout == KDA_ROTARY_INTERLEAVED, KDA_ERR_INVALID_ARG,
                "unknown layout %d", (int)layout);
    KDA_REQUIRE(n_tokens >= 0 && H_q > 0 && H_k >= 0 && d > 0, KDA_ERR_INVALID_ARG,
                "bad sizes n_tokens=%lld H_q=%d H_k=%d d=%d", (long long)n_tokens, H_q, H_k, d);
    KDA_REQUIRE(rot >= 2 && rot <= d && rot % 2 == 0, KDA_ERR_INVALID_ARG,
                "rot must be even, from 2 to d (rot=%d d=%d)", rot, d);
    KDA_REQUIRE(d <= 256 && d * element_size(dtype) % 16 == 0, KDA_ERR_UNSUPPORTED,
                "heads must be whole 16-byte vectors of at most 256 channels (d=%d)", d);
    KDA_REQUIRE(H_q <= 65535 && H_k <= 65535, KDA_ERR_UNSUPPORTED, "H_q and H_k must be <= 65535");
    KDA_REQUIRE(n_tokens <= INT32_MAX, KDA_ERR_UNSUPPORTED, "n_tokens must be below 2^31");
    KDA_STRIDE(q_stride, (int64_t)H_q * d);
    KDA_STRIDE(q_out_stride, (int64_t)H_q * d);
    if (H_k > 0) {
        KDA_STRIDE(k_stride, (int64_t)H_k * d);
        KDA_STRIDE(k_out_stride, (int64_t)H_k * d);
    }
    if (n_tokens == 0) return ok();
    KDA_POINTER(q, 16);
    KDA_POINTER(q_out, 16);
    if (H_k > 0) {
        KDA_POINTER(k, 16);
        KDA_POINTER(k_out, 16);
    }
    KDA_POINTER(positions, 4);
    KDA_POINTER(freq, 8);
    return launched(kda::run_rotary(q, q_stride, q_out, q_out_stride, H_q, k, k_stride, k_out,
                                    k_out_stride, H_k, positions, freq, amplitude, n_tokens, d, rot,
                                    layout == KDA_ROTARY_HALF, dtype == KDA_DTYPE_BF16, stream,
                                    sm_count()),
                    "kda_rotary launch");
}

kda_status kda_cache_write(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           void* k_codes, void* v_codes, float* k_scale, float* v_scale,
                           const int32_t* block_table, int table_pages, const int32_t* start,
                           const int32_t* cu_seqlens, int n_seqs, int64_t T, int H_kv, int d,
                           int64_t n_pages, int page, kda_dtype dtype, cudaStream_t stream) {
    KDA_REQUIRE(valid_dtype(dtype), KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    kda::CacheSpan w;
    const kda_status st = make_span(w, cu_seqlens != nullptr, n_seqs, T, H_kv, d, n_pages, page,
                                    table_pages);
    if (st != KDA_OK) return st;
    KDA_STRIDE(k_stride, (int64_t)H_kv * d);
    KDA_STRIDE(v_stride, (int64_t)H_kv * d);
    if (w.rows == 0 || n_seqs == 0 || n_pages == 0 || table_pages == 0) return ok();
    KDA_POINTER(k, 16);
    KDA_POINTER(v, 16);
    KDA_POINTER(k_codes, 16);
    KDA_POINTER(v_codes, 16);
    KDA_POINTER(k_scale, 4);
    KDA_POINTER(v_scale, 4);
    KDA_POINTER(block_table, 4);
    KDA_POINTER(start, 4);
    KDA_REQUIRE(aligned(cu_seqlens, 4), KDA_ERR_INVALID_ARG, "cu_seqlens is not 4-byte aligned");
    return launched(kda::run_cache_write(w, k, k_stride, v, v_stride, k_codes, v_codes, k_scale,
                                         v_scale, block_table, start, cu_seqlens,
                                         dtype == KDA_DTYPE_BF16, stream),
                    "kda_cache_write launch");
}

kda_status kda_cache_read(const void* k_codes, const void* v_codes, const float* k_scale,
                          const float* v_scale, const int32_t* block_table, int table_pages,
                          const int32_t* start, const int32_t* cu_seqlens, int n_seqs, int64_t T,
                          int H_kv, int d, int64_t n_pages, int page, void* k, void* v,
                          kda_dtype dtype, cudaStream_t stream) {
    KDA_REQUIRE(valid_dtype(dtype), KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    kda::CacheSpan w;
    const kda_status st = make_span(w, cu_seqlens != nullptr, n_seqs, T, H_kv, d, n_pages, page,
                                    table_pages);
    if (st != KDA_OK) return st;
    if (w.rows == 0 || n_seqs == 0) return ok();
    KDA_POINTER(k, 16);
    KDA_POINTER(v, 16);
    KDA_POINTER(start, 4);
    if (n_pages > 0) {
        KDA_POINTER(k_codes, 16);
        KDA_POINTER(v_codes, 16);
        KDA_POINTER(k_scale, 4);
        KDA_POINTER(v_scale, 4);
    }
    if (table_pages > 0) KDA_POINTER(block_table, 4);
    KDA_REQUIRE(aligned(cu_seqlens, 4), KDA_ERR_INVALID_ARG, "cu_seqlens is not 4-byte aligned");
    return launched(kda::run_cache_read(w, k_codes, v_codes, k_scale, v_scale, block_table, start,
                                        cu_seqlens, k, v, dtype == KDA_DTYPE_BF16, stream),
                    "kda_cache_read launch");
}

static kda_status attention_sizes(kda::CacheAttention& a, int B, int T_q, int H_q, int H_kv, int d,
                                  int64_t n_pages, int page, int table_pages) {
    KDA_REQUIRE(B >= 0 && T_q >= 0 && H_q > 0, KDA_ERR_INVALID_ARG, "bad sizes B=%d T_q=%d H_q=%d", B,
                T_q, H_q);
    const kda_status st = check_pool(H_kv, d, n_pages, page, table_pages);
    if (st != KDA_OK) return st;
    KDA_REQUIRE(H_q % H_kv == 0, KDA_ERR_INVALID_ARG, "H_q must be a multiple of H_kv (%d, %d)", H_q,
                H_kv);
    KDA_REQUIRE(H_q <= 65535 && B <= 65535, KDA_ERR_UNSUPPORTED, "B and H_q must be <= 65535");
    // (less than a tile below 2^31, so that counts of row tiles do not overflow)
    KDA_REQUIRE((int64_t)B * T_q * H_q <= INT32_MAX - 255, KDA_ERR_UNSUPPORTED,
                "B * T_q * H_q must be at most 2^31 - 256");
    KDA_REQUIRE((int64_t)table_pages * page <= INT32_MAX, KDA_ERR_UNSUPPORTED,
                "table_pages * page must be below 2^31");
    a.B = B;
    a.T_q = T_q;
    a.H_q = H_q;
    a.H_kv = H_kv;
    a.d = d;
    a.n_pages = n_pages;
    a.page_shift = log2_of(page);
    a.table_pages = table_pages;
    return KDA_OK;
}

size_t kda_cache_attention_workspace_size(int B, int T_q, int H_q, int H_kv, int d, int page,
                                          int table_pages) {
    kda::CacheAttention a = {};
    if (attention_sizes(a, B, T_q, H_q, H_kv, d, 0, page, table_pages) != KDA_OK) return 0;
    return kda::cache_attention_workspace_bytes(a, sm_count());
}

kda_status kda_cache_attention(const void* q, int64_t q_stride, const void* k_codes,
                               const void* v_codes, const float* k_scale, const float* v_scale,
                               const int32_t* block_table, int table_pages, const int32_t* lengths,
                               void* o, float* lse, int B, int T_q, int H_q, int H_kv, int d,
                               int64_t n_pages, int page, float scale, int64_t window, int sinks,
                               kda_dtype dtype, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream) {
    KDA_REQUIRE(valid_dtype(dtype), KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    kda::CacheAttention a = {};
    const kda_status st = attention_sizes(a, B, T_q, H_q, H_kv, d, n_pages, page, table_pages);
    if (st != KDA_OK) return st;
    KDA_REQUIRE(window >= 0 && sinks >= 0, KDA_ERR_INVALID_ARG,
                "window and sinks must not be negative (%lld, %d)", (long long)window, sinks);
    KDA_REQUIRE(std::isfinite(scale), KDA_ERR_INVALID_ARG, "scale is not finite");
    KDA_STRIDE(q_stride, (int64_t)H_q * d);
    if (B == 0 || T_q == 0) return ok();
    KDA_POINTER(q, 16);
    KDA_POINTER(o, 16);
    KDA_POINTER(lengths, 4);
    KDA_REQUIRE(aligned(lse, 4), KDA_ERR_INVALID_ARG, "lse is not 4-byte aligned");
    if (n_pages > 0) {
        KDA_POINTER(k_codes, 16);
        KDA_POINTER(v_codes, 16);
        KDA_POINTER(k_scale, 4);
        KDA_POINTER(v_scale, 4);
    }
    if (table_pages > 0) KDA_POINTER(block_table, 4);
    a.q = q;
    a.q_stride = q_stride;
    // (a pool without pages is not read, but its address goes into empty copies)
    a.k_codes = static_cast<const uint8_t*>(n_pages > 0 ? k_codes : q);
    a.v_codes = static_cast<const uint8_t*>(n_pages > 0 ? v_codes : q);
    a.k_scale = n_pages > 0 ? k_scale : static_cast<const float*>(q);
    a.v_scale = n_pages > 0 ? v_scale : static_cast<const float*>(q);
    a.table = block_table;
    a.lengths = lengths;
    a.o = o;
    a.lse = lse;
    a.scale = scale;
    // (positions are below 2^31: a wider window is none, and differences with it stay in range)
    a.window = window > INT32_MAX ? 0 : window;
    a.sinks = sinks;
    const int sms = sm_count();
    const size_t need = kda::cache_attention_workspace_bytes(a, sms);
    if (need > 0) {
        KDA_REQUIRE(workspace != nullptr && workspace_bytes >= need, KDA_ERR_WORKSPACE,
                    "workspace of %zu bytes required, got %zu at %p", need, workspace_bytes, workspace);
        KDA_REQUIRE(aligned(workspace, 256), KDA_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
    }
    return launched(kda::run_cache_attention(a, dtype == KDA_DTYPE_BF16, workspace, stream, sms),
                    "kda_cache_attention launch");
}

}  // extern "C"
