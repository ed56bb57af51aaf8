// kda_rotary.cu -- rotary positions on the queries and keys of a step.
//
//   a = p f_i,   (x, y) <- A (x cos a - y sin a, y cos a + x sin a)
//
// for the pairs (i, i + rot / 2) or (2 i, 2 i + 1) of the first rot channels
// of every head; the other channels are copied.
//
// The angle.  p f_i in 32 bits has lost the turn's fraction by p = 2^20, so the
// angle is kept as a fraction of a turn in 64-bit fixed point: f_i / 2 pi (its
// whole part dropped) becomes a multiple of 2^-64, the product with p wraps
// modulo one turn by itself, and the top 32 bits go to sincospif.  One 64-bit
// multiply an angle and three 64-bit float operations; the angle is off by at
// most 2^-32 turns plus p 2^-53.
//
// The split.  Bound by memory: every element is read and written once.  A CTA
// takes a few tokens with all their heads, works out their rot / 2 angles once
// into shared memory, and then gives every thread one (head, 16-byte vector)
// place for all its tokens, so that the place is worked out once and the
// loads of four tokens are in flight together.
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {

struct RotarySide {
    const void* x;
    void* y;
    int64_t xs, ys;   // elements between tokens
    int heads;
};

constexpr int kRotaryThreads = 256;
constexpr int kRotaryBatch = 4;               // tokens whose loads a thread has in flight
constexpr int kRotaryRowBytes = 16 * 1024;    // of one pass of the ragged kernel (twice in shared memory)

__device__ __forceinline__ float2 rotary_angle(double turns_per_position, int32_t position) {
    const double frac = turns_per_position - floor(turns_per_position);
    const uint64_t fixed = __double2ull_rz(frac * 18446744073709551616.0);
    const uint64_t phase = fixed * (uint64_t)(int64_t)position;
    float s, c;
    sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31
    return make_float2(c, s);
}

template <typename T>
__device__ __forceinline__ void unpack16(const uint4& raw, float* f) {
    const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < (int)(16 / sizeof(T)); ++i) f[i] = to_f32(e[i]);
}
template <typename T>
__device__ __forceinline__ uint4 pack16(const float* f) {
    uint4 raw;
    T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int i = 0; i < (int)(16 / sizeof(T)); ++i) e[i] = from_f32<T>(f[i]);
    return raw;
}

// cos and sin of the CTA's tokens, [tokens][rot / 2].
__device__ __forceinline__ void rotary_table(float2* cs, const int32_t* positions,
                                             const double* freq, float amplitude, int64_t t0, int nt,
                                             int half) {
    for (int i = threadIdx.x; i < nt * half; i += kRotaryThreads) {
        const int t = i / half;
        const float2 a = rotary_angle(freq[i - t * half] * 0.15915494309189535,   // 1 / 2 pi
                                      positions[t0 + t]);
        cs[i] = make_float2(a.x * amplitude, a.y * amplitude);
    }
    __syncthreads();
}

// Whole 16-byte vectors of pairs: in the half layout rot / 2 is a multiple of
// the vector, in the interleaved one rot is.  A unit is the vector (or, in the
// half layout, the two) that one thread turns; the last units of a head are
// vectors past rot, copied.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kRotaryThreads)
rotary_kernel(RotarySide q, RotarySide k, const int32_t* __restrict__ positions,
              const double* __restrict__ freq, float amplitude, int64_t n_tokens, int d, int rot,
              int tile) {
    constexpr int V = 16 / sizeof(T);
    extern __shared__ __align__(16) float2 cs[];
    const int half = rot / 2;
    const int64_t t0 = (int64_t)blockIdx.x * tile;
    const int nt = (int)(n_tokens - t0 < tile ? n_tokens - t0 : tile);
    rotary_table(cs, positions, freq, amplitude, t0, nt, half);

    const int turned = HALF ? half / V : rot / V;
    const int units = turned + (d - rot) / V;
    const int places = (q.heads + k.heads) * units;
    for (int place = threadIdx.x; place < places; place += kRotaryThreads) {
        const int row = place / units, u = place - row * units;
        const bool is_q = row < q.heads;
        const int h = is_q ? row : row - q.heads;
        const int64_t xs = is_q ? q.xs : k.xs, ys = is_q ? q.ys : k.ys;
        const bool copied = u >= turned;
        const int64_t e0 = (int64_t)h * d + (copied ? rot + (u - turned) * V : u * V);
        const T* x = static_cast<const T*>(is_q ? q.x : k.x) + t0 * xs + e0;
        T* y = static_cast<T*>(is_q ? q.y : k.y) + t0 * ys + e0;
        const bool pair = HALF && !copied;
        for (int t = 0; t < nt; t += kRotaryBatch) {
            uint4 a[kRotaryBatch], b[kRotaryBatch];
#pragma unroll
            for (int j = 0; j < kRotaryBatch; ++j)
                if (t + j < nt) {
                    a[j] = __ldcs(reinterpret_cast<const uint4*>(x + (t + j) * xs));
                    if (pair) b[j] = __ldcs(reinterpret_cast<const uint4*>(x + (t + j) * xs + half));
                }
#pragma unroll
            for (int j = 0; j < kRotaryBatch; ++j)
                if (t + j < nt) {
                    uint4 out = a[j];
                    if (!copied) {
                        const float2* c = cs + (t + j) * half;
                        float f[V];
                        unpack16<T>(a[j], f);
                        if constexpr (HALF) {
                            float g[V];
                            unpack16<T>(b[j], g);
#pragma unroll
                            for (int i = 0; i < V; ++i) {
                                const float2 w = c[u * V + i];
                                const float fx = f[i], gx = g[i];
                                f[i] = fx * w.x - gx * w.y;
                                g[i] = gx * w.x + fx * w.y;
                            }
                            __stcs(reinterpret_cast<uint4*>(y + (t + j) * ys + half), pack16<T>(g));
                        } else {
#pragma unroll
                            for (int i = 0; i < V; i += 2) {
                                const float2 w = c[(u * V + i) / 2];
                                const float fx = f[i], gx = f[i + 1];
                                f[i] = fx * w.x - gx * w.y;
                                f[i + 1] = gx * w.x + fx * w.y;
                            }
                        }
                        out = pack16<T>(f);
                    }
                    __stcs(reinterpret_cast<uint4*>(y + (t + j) * ys), out);
                }
        }
    }
}

// Any even rot: rows pass through shared memory a group of heads at a time
// (read whole, then written from the copy, so the output may be the input),
// and a thread makes the 16-byte vectors of the output element by element.
// Two buffers: a group is read into one while the other's readers finish.
template <typename T>
__global__ void __launch_bounds__(kRotaryThreads)
rotary_ragged_kernel(RotarySide q, RotarySide k, const int32_t* __restrict__ positions,
                     const double* __restrict__ freq, float amplitude, int64_t n_tokens, int d,
                     int rot, bool half_layout, int tile, int group) {
    constexpr int V = 16 / sizeof(T);
    extern __shared__ __align__(16) float2 cs[];
    const int half = rot / 2;
    const int64_t t0 = (int64_t)blockIdx.x * tile;
    const int nt = (int)(n_tokens - t0 < tile ? n_tokens - t0 : tile);
    uint4* rows = reinterpret_cast<uint4*>(cs + ((tile * half + 1) & ~1));   // 2 x [group][units]
    const T* elems = reinterpret_cast<const T*>(rows);
    rotary_table(cs, positions, freq, amplitude, t0, nt, half);

    const int units = d / V, heads = q.heads + k.heads;
    int buf = 0;
    for (int t = 0; t < nt; ++t) {
        const float2* c = cs + t * half;
        for (int h0 = 0; h0 < heads; h0 += group) {
            const int places = (heads - h0 < group ? heads - h0 : group) * units;
            for (int place = threadIdx.x; place < places; place += kRotaryThreads) {
                const int at = h0 * units + place;
                const bool is_q = at < q.heads * units;
                const int off = is_q ? at : at - q.heads * units;
                const T* x = static_cast<const T*>(is_q ? q.x : k.x) + (t0 + t) * (is_q ? q.xs : k.xs);
                rows[buf + place] = __ldcs(reinterpret_cast<const uint4*>(x) + off);
            }
            __syncthreads();
            for (int place = threadIdx.x; place < places; place += kRotaryThreads) {
                const int at = h0 * units + place;
                const bool is_q = at < q.heads * units;
                const int off = is_q ? at : at - q.heads * units;
                const int row = place / units, e0 = (place - row * units) * V;
                float f[V];
                unpack16<T>(rows[buf + place], f);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = e0 + i;
                    if (e < rot) {
                        const bool first = half_layout ? e < half : (e & 1) == 0;
                        const int mate = half_layout ? (first ? e + half : e - half) : e ^ 1;
                        const float2 w = c[half_layout ? (first ? e : mate) : e >> 1];
                        const float g = to_f32(elems[buf * V + row * d + mate]);
                        f[i] = first ? f[i] * w.x - g * w.y : f[i] * w.x + g * w.y;
                    }
                }
                T* y = static_cast<T*>(is_q ? q.y : k.y) + (t0 + t) * (is_q ? q.ys : k.ys);
                __stcs(reinterpret_cast<uint4*>(y) + off, pack16<T>(f));
            }
            buf = buf ? 0 : group * units;
        }
    }
}

template <typename T>
static cudaError_t launch_rotary(const RotarySide& q, const RotarySide& k, const int32_t* positions,
                                 const double* freq, float amplitude, int64_t n_tokens, int d,
                                 int rot, bool half_layout, cudaStream_t stream, int num_sms) {
    constexpr int V = 16 / sizeof(T);
    // Tokens a CTA takes: enough that the angles are shared out and four tokens'
    // loads are in flight, but no more while there are SMs without a CTA.
    int tile = 8;
    while (tile > 1 && (n_tokens + tile - 1) / tile < 2 * num_sms) tile /= 2;
    const unsigned grid = (unsigned)((n_tokens + tile - 1) / tile);
    const size_t table = (size_t)((tile * (rot / 2) + 1) & ~1) * sizeof(float2);
    if (half_layout && rot / 2 % V == 0) {
        rotary_kernel<T, true><<<grid, kRotaryThreads, table, stream>>>(
            q, k, positions, freq, amplitude, n_tokens, d, rot, tile);
    } else if (!half_layout && rot % V == 0) {
        rotary_kernel<T, false><<<grid, kRotaryThreads, table, stream>>>(
            q, k, positions, freq, amplitude, n_tokens, d, rot, tile);
    } else {
        int group = kRotaryRowBytes / (d * (int)sizeof(T));   // d <= 256: at least 16 heads
        if (group > q.heads + k.heads) group = q.heads + k.heads;
        const size_t smem = table + 2 * (size_t)group * d * sizeof(T);
        rotary_ragged_kernel<T><<<grid, kRotaryThreads, smem, stream>>>(
            q, k, positions, freq, amplitude, n_tokens, d, rot, half_layout, tile, group);
    }
    return cudaGetLastError();
}

cudaError_t run_rotary(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int H_q,
                       const void* k, int64_t k_stride, void* k_out, int64_t k_out_stride, int H_k,
                       const int32_t* positions, const double* freq, float amplitude,
                       int64_t n_tokens, int d, int rot, bool half_layout, bool bf16,
                       cudaStream_t stream, int num_sms) {
    const RotarySide qs{q, q_out, q_stride, q_out_stride, H_q};
    const RotarySide ks{k, k_out, k_stride, k_out_stride, H_k};
    if (bf16)
        return launch_rotary<__nv_bfloat16>(qs, ks, positions, freq, amplitude, n_tokens, d, rot,
                                            half_layout, stream, num_sms);
    return launch_rotary<float>(qs, ks, positions, freq, amplitude, n_tokens, d, rot, half_layout,
                                stream, num_sms);
}

}  // namespace kda
