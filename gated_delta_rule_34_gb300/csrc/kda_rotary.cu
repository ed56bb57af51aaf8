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
// modulo one turn by itself.  The nearest quarter is taken from the top 32 bits, of what remains (an eighth of a turn at
// most) cos and sin are taken at its first 24 bits and corrected by the others: (c - s x, s + c x).  One 64-bit
// multiply an angle and three 64-bit float operations; the angle is off by at
// most 2^-32 turns plus p 2^-53, times f above 1.  (The top 32 bits as one fp32 number: off by up to 2^-26 turns near half a turn.)
//
// The split.  Bound by memory: every element is read and written once.  A CTA
// takes a few tokens with all their heads and works out their rot / 2 angles once
// into shared memory, in the order in which a warp's lanes read them together.  A thread
// then has one vector's place in the head, of up to four heads of a token: their
// loads are in flight together, and the angles are read once for the four.  (One head
// and four tokens a thread: 70% of the copy rate at 40 heads of 128 channels, all
// turned, 16384 tokens; 80% so.)  The vector is 16 bytes where rot allows it (rot / 2 whole
// vectors in the half layout, rot in the interleaved one), else 8, 4 or 2.
// Measured: 65536 tokens of 32 + 8 heads of 128 channels, 64 turned, bf16: 202 us, 6.6 TB/s;
// 4097 tokens of 16 + 16 heads of 64 channels, fp32: 10.5 us, 6.4 TB/s; one token: 2.4 us.
#include "kda_cache_internal.h"
#include "kda_chained.cuh"
#include "kda_common.cuh"

namespace kda {

struct RotarySide {
    const void* x;
    void* y;
    int64_t xs, ys;   // elements between tokens
    int heads;
};

constexpr int kRotaryThreads = 256;
// Heads of one thread: four, or more of the interleaved layout's narrower
// vectors (40 heads of 128 channels, 50 of them turned: 110 us with 4, 84 us with 16; in the half
// layout, with two vectors a head, more than four gained nothing).
constexpr int rotary_heads(bool half, int bytes) { return half || bytes > 8 ? 4 : 64 / bytes; }

__device__ __forceinline__ float2 rotary_angle(double turns_per_position, int32_t position) {
    const double frac = turns_per_position - floor(turns_per_position);
    const uint64_t fixed = __double2ull_rz(frac * 18446744073709551616.0);
    const uint64_t phase = fixed * (uint64_t)(int64_t)position;
    const uint32_t top = (uint32_t)(phase >> 32), quarter = (top + 0x20000000u) >> 30;
    const int32_t rest = (int32_t)(top - (quarter << 30));                 // of 2^-32 turns, within 2^29
    const float first = (float)rest;
    const float more = (float)(rest - (int32_t)first) * 1.4629180792671596e-9f;   // 2 pi 2^-32
    float s, c;
    sincospif(first * 4.656612873077393e-10f, &s, &c);                     // 2^-31
    const float cx = fmaf(-s, more, c), sx = fmaf(c, more, s);
    const float x = quarter & 1 ? sx : cx, y = quarter & 1 ? cx : sx;
    return make_float2(quarter + 1 & 2 ? -x : x, quarter & 2 ? -y : y);
}

// A vector of N elements of T as one load or store.
template <int BYTES>
struct RawOf;
template <>
struct RawOf<16> { using type = uint4; };
template <>
struct RawOf<8> { using type = uint2; };
template <>
struct RawOf<4> { using type = uint32_t; };
template <>
struct RawOf<2> { using type = unsigned short; };

template <typename T, int V>
__device__ __forceinline__ void unpack_raw(const typename RawOf<V * sizeof(T)>::type& raw, float (&f)[V]) {
    const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f32(e[i]);
}
template <typename T, int V>
__device__ __forceinline__ typename RawOf<V * sizeof(T)>::type pack_raw(const float (&f)[V]) {
    typename RawOf<V * sizeof(T)>::type raw;
    T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = from_f32<T>(f[i]);
    return raw;
}

// A unit is the vector (or, in the half layout, the two) that one thread turns.
// A head's last units, past rot, are copied.  Where vectors are single bf16 values,
// those from the next 16 bytes on are copied apart, 16 bytes at a time, and not at
// all where the output is the input (50 of 128 channels turned: 174 us without, 117 us
// so; wider vectors lose by it, as two passes then write the same sectors).
template <typename T, bool HALF, int V>
__global__ void __launch_bounds__(kRotaryThreads)
rotary_kernel(RotarySide q, RotarySide k, const int32_t* positions,
              const double* freq, float amplitude, int64_t n_tokens, int d, int rot,
              int tile) {
    using Raw = typename RawOf<V * sizeof(T)>::type;
    constexpr int A = HALF ? V : V / 2;                    // angles of a unit
    constexpr int H = rotary_heads(HALF, V * sizeof(T));
    extern __shared__ __align__(16) float2 cs[];           // [tokens][A][turned]
    after_the_kernel_before();
    const int half = rot / 2, turned = half / A;
    const int64_t t0 = (int64_t)blockIdx.x * tile;
    const int nt = (int)(n_tokens - t0 < tile ? n_tokens - t0 : tile);
    for (int i = threadIdx.x; i < nt * half; i += kRotaryThreads) {
        const int t = i / half, angle = i - t * half;
        const float2 w = rotary_angle(freq[angle] * 0.15915494309189535, positions[t0 + t]);   // 1 / 2 pi
        cs[t * half + angle % A * turned + angle / A] = make_float2(w.x * amplitude, w.y * amplitude);
    }
    __syncthreads();

    constexpr int W = 16 / sizeof(T);
    constexpr bool APART = V * sizeof(T) == 2;
    const int wide0 = APART ? (rot + W - 1) / W * W : d;   // where 16-byte copies begin
    const int units = turned + (wide0 - rot) / V;
    const int heads = q.heads + k.heads, lanes = (heads + H - 1) / H;
    const int each = lanes * units;
    for (int i = threadIdx.x; i < nt * each; i += kRotaryThreads) {
        const int t = i / each, rest = i - t * each;
        const int h0 = rest / units, u = rest - h0 * units;
        const bool copied = u >= turned;
        const int e0 = copied ? rot + (u - turned) * V : u * V;
        const T* qx = static_cast<const T*>(q.x) + (t0 + t) * q.xs + e0;
        const T* kx = static_cast<const T*>(k.x) + (t0 + t) * k.xs + e0;
        Raw a[H], b[H];
#pragma unroll
        for (int j = 0; j < H; ++j) {
            const int h = h0 + j * lanes;
            if (h < heads) {
                const T* x = h < q.heads ? qx + h * d : kx + (h - q.heads) * d;
                a[j] = __ldcs(reinterpret_cast<const Raw*>(x));
                if (HALF && !copied) b[j] = __ldcs(reinterpret_cast<const Raw*>(x + half));
            }
        }
        float2 w[A];
        if (!copied) {
#pragma unroll
            for (int c = 0; c < A; ++c) w[c] = cs[t * half + c * turned + u];
        }
        T* qy = static_cast<T*>(q.y) + (t0 + t) * q.ys + e0;
        T* ky = static_cast<T*>(k.y) + (t0 + t) * k.ys + e0;
#pragma unroll
        for (int j = 0; j < H; ++j) {
            const int h = h0 + j * lanes;
            if (h >= heads) break;
            T* y = h < q.heads ? qy + h * d : ky + (h - q.heads) * d;
            if (!copied) {
                float f[V];
                unpack_raw<T, V>(a[j], f);
                if constexpr (HALF) {
                    float g[V];
                    unpack_raw<T, V>(b[j], g);
#pragma unroll
                    for (int c = 0; c < V; ++c) {
                        const float fx = f[c], gx = g[c];
                        f[c] = fx * w[c].x - gx * w[c].y;
                        g[c] = gx * w[c].x + fx * w[c].y;
                    }
                    __stcs(reinterpret_cast<Raw*>(y + half), pack_raw<T, V>(g));
                } else {
#pragma unroll
                    for (int c = 0; c < A; ++c) {
                        const float fx = f[2 * c], gx = f[2 * c + 1];
                        f[2 * c] = fx * w[c].x - gx * w[c].y;
                        f[2 * c + 1] = gx * w[c].x + fx * w[c].y;
                    }
                }
                a[j] = pack_raw<T, V>(f);
            }
            __stcs(reinterpret_cast<Raw*>(y), a[j]);
        }
    }

    if constexpr (!APART) return;
    const bool q_apart = q.x != q.y || q.xs != q.ys, k_apart = k.x != k.y || k.xs != k.ys;
    const int wide = lanes * ((d - wide0) / W);
    if (wide == 0 || !(q_apart || k_apart)) return;
    for (int i = threadIdx.x; i < nt * wide; i += kRotaryThreads) {
        const int t = i / wide, rest = i - t * wide;
        const int h0 = rest / (wide / lanes), e0 = wide0 + (rest - h0 * (wide / lanes)) * W;
        const T* qx = static_cast<const T*>(q.x) + (t0 + t) * q.xs + e0;
        const T* kx = static_cast<const T*>(k.x) + (t0 + t) * k.xs + e0;
        T* qy = static_cast<T*>(q.y) + (t0 + t) * q.ys + e0;
        T* ky = static_cast<T*>(k.y) + (t0 + t) * k.ys + e0;
        uint4 a[H];
#pragma unroll
        for (int j = 0; j < H; ++j) {
            const int h = h0 + j * lanes;
            if (h < heads)
                a[j] = __ldcs(reinterpret_cast<const uint4*>(h < q.heads ? qx + h * d : kx + (h - q.heads) * d));
        }
#pragma unroll
        for (int j = 0; j < H; ++j) {
            const int h = h0 + j * lanes;
            if (h < heads)
                __stcs(reinterpret_cast<uint4*>(h < q.heads ? qy + h * d : ky + (h - q.heads) * d), a[j]);
        }
    }
}

template <typename T, bool HALF, int V>
static cudaError_t launch_rotary(const RotarySide& q, const RotarySide& k, const int32_t* positions,
                                 const double* freq, float amplitude, int64_t n_tokens, int d,
                                 int rot, cudaStream_t stream, int num_sms) {
    // Tokens a CTA takes: enough to keep its threads busy for some rounds, but no
    // more while there are SMs without a CTA.
    int tile = 16;
    while (tile > 1 && (n_tokens + tile - 1) / tile < 4 * num_sms) tile /= 2;
    const unsigned grid = (unsigned)((n_tokens + tile - 1) / tile);
    return launch_chained(rotary_kernel<T, HALF, V>, grid, kRotaryThreads, (size_t)tile * (rot / 2) * sizeof(float2), stream,
                          q, k, positions, freq, amplitude, n_tokens, d, rot, tile);
}

// The widest vector that rot allows; d is whole 16-byte vectors.
template <typename T>
static cudaError_t by_vector(const RotarySide& q, const RotarySide& k, const int32_t* positions,
                             const double* freq, float amplitude, int64_t n_tokens, int d, int rot,
                             bool half_layout, cudaStream_t stream, int num_sms) {
    constexpr int W = 16 / sizeof(T);
#define KDA_ROTARY(HALF, V) \
    launch_rotary<T, HALF, V>(q, k, positions, freq, amplitude, n_tokens, d, rot, stream, num_sms)
    if (half_layout) {
        const int n = rot / 2;
        if (n % W == 0) return KDA_ROTARY(true, W);
        if (n % (W / 2) == 0) return KDA_ROTARY(true, W / 2);
        if constexpr (W == 8)
            if (n % 2 == 0) return KDA_ROTARY(true, 2);
        return KDA_ROTARY(true, 1);
    }
    if (rot % W == 0) return KDA_ROTARY(false, W);
    if constexpr (W == 8)
        if (rot % 4 == 0) return KDA_ROTARY(false, 4);
    return KDA_ROTARY(false, 2);
#undef KDA_ROTARY
}

cudaError_t run_rotary(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int H_q,
                       const void* k, int64_t k_stride, void* k_out, int64_t k_out_stride, int H_k,
                       const int32_t* positions, const double* freq, float amplitude,
                       int64_t n_tokens, int d, int rot, bool half_layout, bool bf16,
                       cudaStream_t stream, int num_sms) {
    const RotarySide qs{q, q_out, q_stride, q_out_stride, H_q};
    const RotarySide ks{k, k_out, k_stride, k_out_stride, H_k};
    return bf16 ? by_vector<__nv_bfloat16>(qs, ks, positions, freq, amplitude, n_tokens, d, rot,
                                           half_layout, stream, num_sms)
                : by_vector<float>(qs, ks, positions, freq, amplitude, n_tokens, d, rot, half_layout,
                                   stream, num_sms);
}

}  // namespace kda
