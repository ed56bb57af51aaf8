// kda_cache_attention.cu -- attention of a sequence's newest tokens over the paged 8-bit cache.
//
// Row (b, i, h) is query head h of the i-th of T_q newest tokens; its position is
// p = lengths[b] - T_q + i and its keys are those of head h / (H_q / H_kv).  It sees
// token t if t <= p, t < sinks or t > p - window, and t's page is held:
//
//   s_t = scale q.k_t,   o = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m),   m = max_t s_t
//
// one pass over the tokens with the running maximum and sum.  A row that sees
// nothing, or whose scores are all -inf, gives zeros and lse = -inf.
#include "kda_cache.cuh"
#include "kda_internal.h"

namespace kda {

constexpr int kSimpleWarps = 4;

template <typename T>
__global__ void __launch_bounds__(32 * kSimpleWarps) simple_attention_kernel(CacheAttention a) {
    __shared__ float q_s[128];
    __shared__ float part[kSimpleWarps][130];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x;                       // (b, i, h)
    const int h = (int)(row % a.H_q);
    const int64_t bi = row / a.H_q;
    const int i = (int)(bi % a.T_q), b = (int)(bi / a.T_q);
    const int hk = h / (a.H_q / a.H_kv);
    for (int c = threadIdx.x; c < a.d; c += blockDim.x)
        q_s[c] = to_f32(static_cast<const T*>(a.q)[bi * a.q_stride + (int64_t)h * a.d + c]);
    __syncthreads();
    const int64_t cap = (int64_t)a.table_pages << a.page_shift;
    const int64_t len = a.lengths[b] < 0 ? 0 : (a.lengths[b] > cap ? cap : a.lengths[b]);
    const int64_t p = len - a.T_q + i;
    const int64_t lo = a.window > 0 && p - a.window + 1 > 0 ? p - a.window + 1 : 0;
    float m = -INFINITY, l = 0.0f, acc[4] = {0, 0, 0, 0};
    for (int64_t t0 = 32 * warp; t0 <= p; t0 += 32 * kSimpleWarps) {
        if (t0 + 32 <= lo && t0 >= a.sinks) continue;
        const int64_t t = t0 + lane;
        float s = -INFINITY;
        int64_t at = -1;                                  // (page, head) of this lane's token
        if (t <= p && (t >= lo || t < a.sinks)) {
            const int32_t id = a.table[(int64_t)b * a.table_pages + (t >> a.page_shift)];
            if (id >= 0 && id < a.n_pages) at = (int64_t)id * a.H_kv + hk;
        }
        const int64_t slot = t & ((1 << a.page_shift) - 1);
        if (at >= 0) {
            const uint8_t* kr = a.k_codes + ((at << a.page_shift) + slot) * a.d;
            float dot = 0.0f;
            for (int c = 0; c < a.d; c += 4) {
                float f[4];
                from_e4m3x4(*reinterpret_cast<const uint32_t*>(kr + c), f);
                dot += q_s[c] * f[0] + q_s[c + 1] * f[1] + q_s[c + 2] * f[2] + q_s[c + 3] * f[3];
            }
            s = dot * a.k_scale[at] * a.scale;
        }
        float mx = s;
        for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float m_new = fmaxf(m, mx);
        const float ref = m_new == -INFINITY ? 0.0f : m_new;
        const float keep = expf(m - ref), pr = at >= 0 ? expf(s - ref) : 0.0f;
        l = l * keep + warp_sum(pr);
        m = m_new;
        for (int j = 0; j < 4; ++j) acc[j] *= keep;
        for (int j = 0; j < 32; ++j) {
            const int64_t at_j = __shfl_sync(0xffffffffu, at, j);
            const float p_j = __shfl_sync(0xffffffffu, pr, j);
            if (at_j < 0 || lane * 4 >= a.d) continue;
            const int64_t slot_j = (t0 + j) & ((1 << a.page_shift) - 1);
            float f[4];
            from_e4m3x4(*reinterpret_cast<const uint32_t*>(
                            a.v_codes + ((at_j << a.page_shift) + slot_j) * a.d + lane * 4), f);
            const float w = p_j * a.v_scale[at_j];
            for (int c = 0; c < 4; ++c) acc[c] += w * f[c];
        }
    }
    part[warp][128] = m;
    part[warp][129] = l;
    for (int c = 0; c < 4; ++c) part[warp][lane * 4 + c] = acc[c];
    __syncthreads();
    if (warp) return;
    float top = -INFINITY, sum = 0.0f, out[4] = {0, 0, 0, 0};
    for (int w = 0; w < kSimpleWarps; ++w) top = fmaxf(top, part[w][128]);
    const float ref = top == -INFINITY ? 0.0f : top;
    for (int w = 0; w < kSimpleWarps; ++w) {
        const float f = expf(part[w][128] - ref);
        sum += f * part[w][129];
        for (int c = 0; c < 4; ++c) out[c] += f * part[w][lane * 4 + c];
    }
    for (int c = 0; c < 4; ++c)
        if (lane * 4 + c < a.d)
            static_cast<T*>(a.o)[row * a.d + lane * 4 + c] = from_f32<T>(sum == 0.0f ? 0.0f : out[c] / sum);
    if (a.lse && lane == 0) a.lse[row] = sum == 0.0f ? -INFINITY : logf(sum) + top;
}

size_t cache_attention_workspace_bytes(const CacheAttention&, int) { return 0; }

cudaError_t run_cache_attention(const CacheAttention& a, bool bf16, void*, cudaStream_t stream, int) {
    const unsigned grid = (unsigned)((int64_t)a.B * a.T_q * a.H_q);
    if (bf16)
        simple_attention_kernel<__nv_bfloat16><<<grid, 32 * kSimpleWarps, 0, stream>>>(a);
    else
        simple_attention_kernel<float><<<grid, 32 * kSimpleWarps, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
