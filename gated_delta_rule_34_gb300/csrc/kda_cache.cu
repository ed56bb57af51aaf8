// kda_cache.cu -- keys and values into the paged 8-bit cache, and back.
//
//   write  s <- max(s of the page's older tokens, s(max |x| of the new ones)),
//          code = e4m3(x / s); where s grew, the older codes are rounded again
//   read   x = code * s
//
// Both are bound by memory: every new element is read once and written once.
//
// The split.  An item is one (sequence, page, head, k or v): all the new rows
// that a call brings to that page and head, whose one scale needs all of them.
// GROUP warps take an item, hold up to kHeld units of 16 elements a thread in
// registers between finding the maximum and rounding (a page of 64 tokens of
// 128 bf16 channels fits), and read what is beyond that again.  Four warps
// an item where a sequence brings many tokens; one warp an item where it
// brings few, as in a decode step, whose rows are a few hundred bytes.
//
// Pages are dealt out without a look at the lengths on the host: sequence n,
// whose first packed row is r, owns the slots from floor((r + n (2 P - 2)) / P);
// the next sequence's start is at least floor((len + 2 P - 2) / P) further, which
// no run of len tokens, wherever it starts in a page, needs more of.
//
// Measured with heads of 128 channels and pages of 64 tokens, bf16: 64 packed sequences of up to 4096 tokens, 16 heads,
// written in 255 us, 6.4 TB/s; 16 of up to 16384 tokens, 8 heads, read in 132 us, 6.5 TB/s; one token of each of 256
// sequences, 8 heads, written in 5.6 us packed and 3.6 us as a batch, most of it loads that wait for one another.  That is
// the size these numbers of threads suit.  Smaller items leave threads idle and pay each item's search, offsets, table and
// barrier for less: the same bytes in pages of 16 tokens take 2.5 times as long to write and 1.8 times to read, with heads of
// 16 channels 4.8 and 2.9 times; pages of 128 tokens, more than is held, 1.3 times to write.
#include "kda_cache.cuh"
#include "kda_cache_internal.h"
#include "kda_chained.cuh"

namespace kda {

constexpr int kCacheThreads = 128;
constexpr int kHeld = 4;

struct PageRun {
    int64_t row;      // first packed row of the run
    int64_t at;       // position of the run's first token
    int n;            // tokens of the run, 0: none
    int32_t page;     // page id, or -1: not held
};

__device__ __forceinline__ int64_t first_slot(int64_t row, int64_t n, int page_shift) {
    return (row + n * ((2LL << page_shift) - 2)) >> page_shift;
}

// The run of tokens of slot `slot`: which sequence owns it (fixed length T, or
// by a 32-way search of cu, all lanes of a warp together) and what part of the
// sequence's new tokens lies on the slot's page.
__device__ __forceinline__ PageRun page_run(int64_t slot, const CacheSpan& w, const int32_t* cu,
                                            const int32_t* start, const int32_t* table) {
    PageRun r{0, 0, 0, -1};
    int n;
    int64_t ordinal, len;
    if (cu) {
        int lo = 0, hi = w.n_seqs;            // the owner is in [lo, hi)
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32;
            const int probe = lo + (int)(threadIdx.x & 31) * step;
            bool owns = false;
            if (probe < hi) {
                int64_t row = cu[probe];
                row = row < 0 ? 0 : (row > w.rows ? w.rows : row);
                owns = first_slot(row, probe, w.page_shift) <= slot;
            }
            const uint32_t yes = __ballot_sync(0xffffffffu, owns);
            const int last = yes ? 31 - __clz(yes) : 0;
            lo += last * step;
            hi = lo + step < hi ? lo + step : hi;
        }
        n = lo;
        int64_t bos, eos;
        seq_bounds(cu, n, 0, w.rows, bos, eos);
        r.row = bos;
        len = eos - bos;
        ordinal = slot - first_slot(bos, n, w.page_shift);
    } else {
        n = (int)(slot / w.slots_per_seq);
        ordinal = slot - (int64_t)n * w.slots_per_seq;
        r.row = (int64_t)n * w.T;
        len = w.T;
    }
    int64_t s = start[n];
    s = s < 0 ? 0 : s;
    const int64_t p = (s >> w.page_shift) + ordinal;
    const int64_t b = p << w.page_shift, e = b + (1LL << w.page_shift);
    const int64_t from = s > b ? s : b, to = s + len < e ? s + len : e;
    if (ordinal < 0 || from >= to) return r;
    r.row += from - s;
    r.at = from;
    r.n = (int)(to - from);
    if (p < w.table_pages) {
        const int32_t id = table[(int64_t)n * w.table_pages + p];
        r.page = id >= 0 && id < w.n_pages ? id : -1;
    }
    return r;
}

// Sixteen elements as floats.
template <typename T>
__device__ __forceinline__ void unpack_unit(const uint4 (&raw)[sizeof(T)], float (&f)[16]) {
    const T* e = reinterpret_cast<const T*>(raw);
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = to_f32(e[i]);
}
template <typename T>
__device__ __forceinline__ void load_unit(const T* p, uint4 (&raw)[sizeof(T)]) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) raw[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
}
// The largest |x| of a unit and m, an infinity among them; NaN does not count.
template <typename T>
__device__ __forceinline__ float unit_amax(const uint4 (&raw)[sizeof(T)], float m) {
    if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162* e = reinterpret_cast<const __nv_bfloat162*>(raw);
        __nv_bfloat162 top = __habs2(e[0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) top = __hmax2(top, __habs2(e[i]));
        return fmaxf(m, fmaxf(__low2float(top), __high2float(top)));
    } else {
        const float* e = reinterpret_cast<const float*>(raw);
#pragma unroll
        for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(e[i]));
        return m;
    }
}
// The same of its finite values alone.
template <typename T>
__device__ __forceinline__ float unit_finite_amax(const uint4 (&raw)[sizeof(T)], float m) {
    float f[16];
    unpack_unit<T>(raw, f);
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, finite_abs(f[i]));
    return m;
}
// u / per_row for u < 2048 and per_row <= 8, from the reciprocal 65536 / per_row
// rounded up: its excess below 1 adds less than 2048 / 65536 < 1 / 8.
__device__ __forceinline__ int row_of(int u, int reciprocal) { return u * reciprocal >> 16; }
template <typename T>
__device__ __forceinline__ void round_unit(const uint4 (&raw)[sizeof(T)], float inv, uint8_t* to) {
    float f[16];
    unpack_unit<T>(raw, f);
    uint4 c;
    c.x = to_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
    c.y = to_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
    c.z = to_e4m3x4(f[8] * inv, f[9] * inv, f[10] * inv, f[11] * inv);
    c.w = to_e4m3x4(f[12] * inv, f[13] * inv, f[14] * inv, f[15] * inv);
    *reinterpret_cast<uint4*>(to) = c;
}

// (Eight CTAs a SM with bf16 rows: 64 sequences of up to 4096 tokens, 16 heads of 128 channels in 254 us,
// 6.4 TB/s; 258 us with seven.)
template <typename T, int GROUP>
__global__ void __launch_bounds__(kCacheThreads, sizeof(T) == 2 ? 8 : 5)
cache_write_kernel(CacheSpan w, const T* k, int64_t k_stride, const T* v,
                   int64_t v_stride, uint8_t* k_codes, uint8_t* v_codes,
                   float* k_scale, float* v_scale,
                   const int32_t* table, const int32_t* start,
                   const int32_t* cu) {
    constexpr int ITEMS = kCacheThreads / 32 / GROUP;      // of one CTA, all of one slot
    constexpr int THREADS = 32 * GROUP;
    __shared__ float warp_max[kCacheThreads / 32];
    after_the_kernel_before();
    const int chunks = (2 * w.H + ITEMS - 1) / ITEMS;
    const int64_t slot = blockIdx.x / chunks;
    const int item = (int)(blockIdx.x - slot * chunks) * ITEMS + threadIdx.x / THREADS;
    const int tid = threadIdx.x % THREADS;
    const PageRun run = page_run(slot, w, cu, start, table);
    // The whole CTA has one run; only whole warps leave beyond this point.
    if (run.n == 0 || run.page < 0) return;
    const bool mine = item < 2 * w.H;
    if (GROUP == 1 && !mine) return;
    const bool is_v = item >= w.H;
    const int h = is_v ? item - w.H : item;
    const int64_t stride = is_v ? v_stride : k_stride;
    const T* x = (is_v ? v : k) + run.row * stride + (int64_t)h * w.d;
    const int64_t block = (int64_t)run.page * w.H + h;
    float* scale = (is_v ? v_scale : k_scale) + block;
    const int offset = (int)(run.at & ((1 << w.page_shift) - 1));
    uint8_t* codes = (is_v ? v_codes : k_codes) + (block << w.page_shift) * w.d;
    uint8_t* fresh = codes + offset * w.d;
    const float old = offset > 0 ? valid_scale(*scale) : 0.0f;

    const int per_row = w.d / 16, units = run.n * per_row, reciprocal = (65536 + per_row - 1) / per_row;
    auto unit = [&](int u) {
        const int r = row_of(u, reciprocal);
        return x + r * stride + (u - r * per_row) * 16;
    };
    uint4 held[kHeld][sizeof(T)];
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int u = tid + j * THREADS;
        if (u < units) load_unit(unit(u), held[j]);
    }
    auto over_all = [&](auto of_unit) {
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if (tid + j * THREADS < units) amax = of_unit(held[j], amax);
        for (int u = tid + kHeld * THREADS; u < units; u += THREADS) {
            uint4 raw[sizeof(T)];
            load_unit(unit(u), raw);
            amax = of_unit(raw, amax);
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
        if constexpr (GROUP > 1) {
            if (threadIdx.x % 32 == 0) warp_max[threadIdx.x / 32] = amax;
            __syncthreads();                               // also: `old` is read before it is written
            amax = warp_max[0];
#pragma unroll
            for (int i = 1; i < GROUP; ++i) amax = fmaxf(amax, warp_max[i]);
        } else {
            __syncwarp();
        }
        return amax;
    };
    float amax = over_all([](const uint4 (&raw)[sizeof(T)], float m) { return unit_amax<T>(raw, m); });
    if (amax > 3.402823466e38f) {                          // an infinity: once more without it
        if constexpr (GROUP > 1) __syncthreads();
        amax = over_all([](const uint4 (&raw)[sizeof(T)], float m) { return unit_finite_amax<T>(raw, m); });
    }
    const float s = fmaxf(page_scale(amax), pow2_ceil(old));   // (old may be a caller's own, no power of two)
    const float inv = pow2_inverse(s);
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int u = tid + j * THREADS;
        if (u < units) round_unit<T>(held[j], inv, fresh + u * 16);
    }
    for (int u = tid + kHeld * THREADS; u < units; u += THREADS) {
        uint4 raw[sizeof(T)];
        load_unit(unit(u), raw);
        round_unit<T>(raw, inv, fresh + u * 16);
    }
    if (old > 0.0f && s > old) {
        const float ratio = old * inv;
        for (int u = tid; u < offset * per_row; u += THREADS) {
            uint4 c = *reinterpret_cast<uint4*>(codes + u * 16);
            uint32_t* word = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float f[4];
                from_e4m3x4(word[i], f);
                word[i] = to_e4m3x4(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
            }
            *reinterpret_cast<uint4*>(codes + u * 16) = c;
        }
    }
    if (tid == 0) *scale = s;
}

template <typename T>
__global__ void __launch_bounds__(kCacheThreads)
cache_read_kernel(CacheSpan w, const uint8_t* k_codes,
                  const uint8_t* v_codes, const float* k_scale,
                  const float* v_scale, const int32_t* table,
                  const int32_t* start, const int32_t* cu,
                  T* k, T* v) {
    after_the_kernel_before();
    const int64_t slot = blockIdx.x / (2 * w.H);
    const int item = (int)(blockIdx.x - slot * (2 * w.H));
    const PageRun run = page_run(slot, w, cu, start, table);
    if (run.n == 0) return;
    const bool is_v = item >= w.H;
    const int h = is_v ? item - w.H : item;
    T* y = (is_v ? v : k) + (run.row * w.H + h) * w.d;
    const bool is_held = run.page >= 0;
    const int64_t block = (int64_t)(is_held ? run.page : 0) * w.H + h;
    const float s = is_held ? (is_v ? v_scale : k_scale)[block] : 0.0f;
    const uint8_t* codes = (is_v ? v_codes : k_codes) +
                           ((block << w.page_shift) + (run.at & ((1 << w.page_shift) - 1))) * w.d;
    const int per_row = w.d / 16, units = run.n * per_row, reciprocal = (65536 + per_row - 1) / per_row;
    const int64_t row_stride = (int64_t)w.H * w.d;
    for (int u0 = threadIdx.x; u0 < units; u0 += kHeld * kCacheThreads) {
        uint4 c[kHeld];
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            const int u = u0 + j * kCacheThreads;
            c[j] = make_uint4(0, 0, 0, 0);
            if (u < units && is_held) c[j] = __ldcs(reinterpret_cast<const uint4*>(codes + u * 16));
        }
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            const int u = u0 + j * kCacheThreads;
            if (u >= units) break;
            float f[16];
            from_e4m3x4(c[j].x, f);
            from_e4m3x4(c[j].y, f + 4);
            from_e4m3x4(c[j].z, f + 8);
            from_e4m3x4(c[j].w, f + 12);
            uint4 out[sizeof(T)];
            T* e = reinterpret_cast<T*>(out);
#pragma unroll
            for (int i = 0; i < 16; ++i) e[i] = from_f32<T>(f[i] * s);
            const int r = row_of(u, reciprocal);
            uint4* to = reinterpret_cast<uint4*>(y + r * row_stride + (u - r * per_row) * 16);
#pragma unroll
            for (int i = 0; i < (int)sizeof(T); ++i) __stcs(to + i, out[i]);
        }
    }
}

int64_t cache_slots(const CacheSpan& w, bool packed) {
    const int64_t P = 1LL << w.page_shift;
    if (packed) return (w.rows + (int64_t)w.n_seqs * (2 * P - 2)) >> w.page_shift;
    return (int64_t)w.n_seqs * w.slots_per_seq;
}

template <typename T>
static cudaError_t launch_write(const CacheSpan& w, const void* k, int64_t ks, const void* v,
                                int64_t vs, void* kc, void* vc, float* k_scale, float* v_scale,
                                const int32_t* table, const int32_t* start, const int32_t* cu,
                                cudaStream_t stream) {
    const int64_t slots = cache_slots(w, cu != nullptr);
    // One warp an item up to an average of 8 rows a sequence, four above.
    if (w.rows <= 8LL * w.n_seqs) {
        const int64_t grid = slots * ((2 * w.H + 3) / 4);
        return launch_chained(
            cache_write_kernel<T, 1>, (unsigned)grid, kCacheThreads, 0, stream,
            w, static_cast<const T*>(k), ks, static_cast<const T*>(v), vs, static_cast<uint8_t*>(kc),
            static_cast<uint8_t*>(vc), k_scale, v_scale, table, start, cu);
    } else {
        const int64_t grid = slots * 2 * w.H;
        return launch_chained(
            cache_write_kernel<T, 4>, (unsigned)grid, kCacheThreads, 0, stream,
            w, static_cast<const T*>(k), ks, static_cast<const T*>(v), vs, static_cast<uint8_t*>(kc),
            static_cast<uint8_t*>(vc), k_scale, v_scale, table, start, cu);
    }
}

cudaError_t run_cache_write(const CacheSpan& w, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, void* k_codes, void* v_codes, float* k_scale,
                            float* v_scale, const int32_t* table, const int32_t* start,
                            const int32_t* cu, bool bf16, cudaStream_t stream) {
    if (bf16)
        return launch_write<__nv_bfloat16>(w, k, k_stride, v, v_stride, k_codes, v_codes, k_scale,
                                           v_scale, table, start, cu, stream);
    return launch_write<float>(w, k, k_stride, v, v_stride, k_codes, v_codes, k_scale, v_scale, table,
                               start, cu, stream);
}

cudaError_t run_cache_read(const CacheSpan& w, const void* k_codes, const void* v_codes,
                           const float* k_scale, const float* v_scale, const int32_t* table,
                           const int32_t* start, const int32_t* cu, void* k, void* v, bool bf16,
                           cudaStream_t stream) {
    const int64_t grid = cache_slots(w, cu != nullptr) * 2 * w.H;
    const uint8_t* kc = static_cast<const uint8_t*>(k_codes);
    const uint8_t* vc = static_cast<const uint8_t*>(v_codes);
    if (bf16)
        return launch_chained(
            cache_read_kernel<__nv_bfloat16>, (unsigned)grid, kCacheThreads, 0, stream, w, kc, vc, k_scale, v_scale, table, start, cu, static_cast<__nv_bfloat16*>(k),
            static_cast<__nv_bfloat16*>(v));
    return launch_chained(
        cache_read_kernel<float>, (unsigned)grid, kCacheThreads, 0, stream, w, kc, vc, k_scale, v_scale, table, start, cu,
        static_cast<float*>(k), static_cast<float*>(v));
}

}  // namespace kda
