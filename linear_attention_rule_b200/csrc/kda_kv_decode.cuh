// Softmax attention of the newest tokens over the paged cache.
//
// Per query row, in one pass over its visible keys with the running maximum m, the sum l and
// the weighted values acc:  m' = max(m, s_j);  l' = l e^{m - m'} + e^{s_j - m'};
// acc' = acc e^{m - m'} + e^{s_j - m'} v_j.  Two such triples join the same way.
#pragma once

#include "kda_kv_cache.cuh"

namespace kda {
namespace attend {

struct Params {
    const void* q;
    int64_t q_stride;
    const int32_t* cu;
    int32_t num_seqs, Hq, max_q, window;
    int64_t total;
    float scale, softcap;
    const float* slopes;
    const int32_t* kv_start;
    void* out;
    float* lse;
    kv::Cache c;
};

constexpr int kWarps = 4;

// One CTA per (sequence, new token, query head); its warps take every fourth key.
template <int D, typename T, typename TC>
__global__ void __launch_bounds__(32 * kWarps) attend_kernel(const Params P) {
    constexpr int E = D / 32;   // channels per lane
    __shared__ float sm[kWarps], sl[kWarps], sacc[kWarps][D];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int n = blockIdx.x / P.max_q, i = blockIdx.x % P.max_q, h = blockIdx.y;
    int64_t t0, t1;
    if (!kv::seq_tokens(P.cu, n, P.total, t0, t1)) return;
    if (t1 - t0 > P.max_q) {
        kda_set_status(KDA_ERR_BAD_SEQLENS);
        return;
    }
    if (i >= t1 - t0) return;
    const int64_t t = t0 + i;
    const int hkv = h / (P.Hq / P.c.Hkv);
    const int64_t pos = (int64_t)P.c.seq_lens[n] - (t1 - t0) + i;
    const int64_t held = (int64_t)P.c.max_pages << P.c.page_shift, last = min(pos, held - 1);
    if (pos >= held) kda_set_status(KDA_ERR_BAD_PAGE);
    int64_t first = P.kv_start ? max(P.kv_start[n], 0) : 0;
    if (P.window > 0) first = max(first, pos - P.window + 1);
    float q[E], acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = to_f32(static_cast<const T*>(P.q)[t * P.q_stride + h * D + lane + 32 * e]);
        acc[e] = 0.f;
    }
    const float ks = P.c.k_scale ? P.c.k_scale[hkv] : 1.f, vs = P.c.v_scale ? P.c.v_scale[hkv] : 1.f;
    float m = -INFINITY, l = 0.f;
    for (int64_t j = first + w; j <= last; j += kWarps) {
        const int64_t row = kv::row_offset(P.c, n, j, hkv);
        if (row < 0) {
            kda_set_status(KDA_ERR_BAD_PAGE);
            continue;
        }
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s += q[e] * to_f32(static_cast<const TC*>(P.c.k)[row + lane + 32 * e]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= P.scale * ks;
        if (P.softcap > 0.f) s = P.softcap * tanhf(s / P.softcap);
        if (P.slopes) s += P.slopes[h] * (float)(j - pos);
        const float m2 = fmaxf(m, s);
        const float keep = m2 == -INFINITY ? 1.f : expf(m - m2), p = m2 == -INFINITY ? 0.f : expf(s - m2);
        l = l * keep + p;
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = acc[e] * keep + p * to_f32(static_cast<const TC*>(P.c.v)[row + lane + 32 * e]);
        m = m2;
    }
    if (lane == 0) { sm[w] = m; sl[w] = l; }
#pragma unroll
    for (int e = 0; e < E; ++e) sacc[w][lane + 32 * e] = acc[e];
    __syncthreads();
    float mt = -INFINITY, lt = 0.f;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) mt = fmaxf(mt, sm[x]);
    float f[kWarps];
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
        f[x] = mt == -INFINITY ? 0.f : expf(sm[x] - mt);
        lt += sl[x] * f[x];
    }
    for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
        float o = 0.f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) o += sacc[x][d] * f[x];
        static_cast<T*>(P.out)[(t * P.Hq + h) * D + d] = from_f32<T>(lt == 0.f ? 0.f : o * vs / lt);
    }
    if (threadIdx.x == 0 && P.lse) P.lse[t * P.Hq + h] = lt == 0.f ? -INFINITY : mt + logf(lt);
}

template <int D, typename T, typename TC>
cudaError_t launch(const Params& P, cudaStream_t stream) {
    const dim3 grid((unsigned)P.num_seqs * (unsigned)P.max_q, (unsigned)P.Hq);
    attend_kernel<D, T, TC><<<grid, 32 * kWarps, 0, stream>>>(P);
    return cudaGetLastError();
}

}  // namespace attend
}  // namespace kda
