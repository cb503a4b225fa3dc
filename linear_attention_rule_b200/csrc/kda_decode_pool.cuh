// The gated delta rule's recurrent form over a pool of states: one or several tokens per
// sequence, the state read from one slot of the pool and stored to others.
//
// With the state S[key][value] of one head, one token is
//   S' = Diag(e^g) S;  p = S'^T k;  r = S'^T q;  u = beta (v - p)
//   o  = r + u (k . q);   S = S' + k u^T
// The value channels (columns of S) never meet, so a warp owns 32 columns and keeps its
// D x 32 slice in registers over all tokens of the sequence: no block-wide barrier stands
// between two tokens, and the slice is read once and written once per stored state.
#pragma once

#include "kda_common.cuh"

namespace kda {
namespace pool {

struct Params {
    const void *q, *k, *v;
    const float *g, *beta;
    int64_t q_stride, k_stride, v_stride;
    float* state;
    const int32_t *slots_in, *slots_out, *cu;
    int32_t num_slots, num_seqs, Hk, Hv;
    int64_t total;
    void* out;
    uint32_t in_flags;
};

constexpr int kTokens = 4;   // tokens whose q, k, decay, v are staged at a time

// One CTA of D threads per (sequence, value head).  Lane (rg, cg) = (lane / 8, lane % 8) of
// warp w holds rows rg * D/4 .. + D/4 - 1 of columns 32 w + 4 cg .. + 3: a warp's load
// covers four rows of 128 bytes, and a column's sum takes two shuffles.
template <int D, typename T>
__global__ void __launch_bounds__(D) decode_pool_kernel(const Params P) {
    constexpr int R = D / 4;           // rows per lane
    constexpr int PAD = R + 4;         // the four row groups fall into different banks
    constexpr int W = D / 32;
    __shared__ __align__(16) float sk[kTokens][4 * PAD], sq[kTokens][4 * PAD], sa[kTokens][4 * PAD];
    __shared__ __align__(16) float sv[kTokens][D];
    __shared__ float sred[kTokens][3][W];   // k.q, k.k, q.q by warp

    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int rg = lane >> 3, cg = lane & 7;
    const int n = blockIdx.x / P.Hv, h = blockIdx.x - n * P.Hv;
    kda_grid_wait();
    int64_t t0 = n, t1 = n + 1;
    if (P.cu) {
        t0 = P.cu[n];
        t1 = P.cu[n + 1];
        if (t0 < 0 || t1 < t0 || t1 > P.total || (n == 0 && t0 != 0)) {
            if (tid == 0) kda_set_status(KDA_ERR_BAD_SEQLENS);
            return;
        }
    }
    if (t1 == t0) return;
    const int32_t slot = P.slots_in[n];
    if (slot < -1 || slot >= P.num_slots) {
        if (tid == 0) kda_set_status(KDA_ERR_BAD_SLOT);
        return;
    }
    const size_t slot_stride = (size_t)P.Hv * D * D;
    // this lane's corner of a head's state: row rg * R, column 32 w + 4 cg
    const size_t corner = (size_t)h * D * D + (size_t)(rg * R) * D + 32 * w + 4 * cg;
    float4 s[R];
    if (slot >= 0) {
        const float* src = P.state + (size_t)slot * slot_stride + corner;
#pragma unroll
        for (int i = 0; i < R; ++i) s[i] = __ldcs(reinterpret_cast<const float4*>(src + (size_t)i * D));
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }

    const int hk = h / (P.Hv / P.Hk);
    const bool scalar = P.in_flags & kInGScalar, logits = P.in_flags & kInGLogits;
    const bool norm = P.in_flags & kInNormQK;
    const int pos = (tid / R) * PAD + tid % R;   // channel tid in the padded arrays

    for (int64_t tb = t0; tb < t1; tb += kTokens) {
        const int nt = (int)min((int64_t)kTokens, t1 - tb);
        if (tb != t0) __syncthreads();   // the staged tokens before these are used up
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
            if (j >= nt) break;
            const int64_t t = tb + j;
            const float kk = to_f32(static_cast<const T*>(P.k)[t * P.k_stride + hk * D + tid]);
            const float qq = to_f32(static_cast<const T*>(P.q)[t * P.q_stride + hk * D + tid]);
            const float gx = scalar ? P.g[t * P.Hv + h] : P.g[(t * P.Hv + h) * D + tid];
            sk[j][pos] = kk;
            sq[j][pos] = qq;
            // with gate logits x the decay is e^{logsigmoid(x)} = sigmoid(x)
            sa[j][pos] = logits ? kda_sigmoid(gx) : expf(gx);
            sv[j][tid] = to_f32(static_cast<const T*>(P.v)[t * P.v_stride + h * D + tid]);
            float kq = kk * qq, k2 = kk * kk, q2 = qq * qq;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                kq += __shfl_xor_sync(0xffffffffu, kq, o);
                if (norm) {
                    k2 += __shfl_xor_sync(0xffffffffu, k2, o);
                    q2 += __shfl_xor_sync(0xffffffffu, q2, o);
                }
            }
            if (lane == 0) {
                sred[j][0][w] = kq;
                sred[j][1][w] = k2;
                sred[j][2][w] = q2;
            }
        }
        __syncthreads();

        for (int j = 0; j < nt; ++j) {
            const int64_t t = tb + j;
            float kq = 0.f, ik = 1.f, iq = 1.f;
#pragma unroll
            for (int x = 0; x < W; ++x) kq += sred[j][0][x];
            if (norm) {   // k and q enter unnormalised; their norms scale p, r, u and k . q
                float k2 = 0.f, q2 = 0.f;
#pragma unroll
                for (int x = 0; x < W; ++x) { k2 += sred[j][1][x]; q2 += sred[j][2][x]; }
                ik = kda_inv_norm(k2);
                iq = kda_inv_norm(q2);
                kq *= ik * iq;
            }
            float b = P.beta[t * P.Hv + h];
            if (P.in_flags & kInBetaLogits) b = kda_sigmoid(b);

            const float4* k4 = reinterpret_cast<const float4*>(&sk[j][rg * PAD]);
            const float4* q4 = reinterpret_cast<const float4*>(&sq[j][rg * PAD]);
            const float4* a4 = reinterpret_cast<const float4*>(&sa[j][rg * PAD]);
            float p[4] = {0.f, 0.f, 0.f, 0.f}, r[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < R; i += 4) {
                const float4 kv = k4[i / 4], qv = q4[i / 4], av = a4[i / 4];
                const float kr[4] = {kv.x, kv.y, kv.z, kv.w}, qr[4] = {qv.x, qv.y, qv.z, qv.w};
                const float ar[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float4& x = s[i + e];
                    x.x *= ar[e]; x.y *= ar[e]; x.z *= ar[e]; x.w *= ar[e];
                    p[0] += x.x * kr[e]; p[1] += x.y * kr[e]; p[2] += x.z * kr[e]; p[3] += x.w * kr[e];
                    r[0] += x.x * qr[e]; r[1] += x.y * qr[e]; r[2] += x.z * qr[e]; r[3] += x.w * qr[e];
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                p[c] += __shfl_xor_sync(0xffffffffu, p[c], 8);
                p[c] += __shfl_xor_sync(0xffffffffu, p[c], 16);
                r[c] += __shfl_xor_sync(0xffffffffu, r[c], 8);
                r[c] += __shfl_xor_sync(0xffffffffu, r[c], 16);
            }
            const float4 vv = *reinterpret_cast<const float4*>(&sv[j][32 * w + 4 * cg]);
            const float v4[4] = {vv.x, vv.y, vv.z, vv.w};
            float u[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) u[c] = b * (v4[c] - ik * p[c]);
            // each of the four row groups writes one of the lane's four columns
            const float rsel = rg == 0 ? r[0] : rg == 1 ? r[1] : rg == 2 ? r[2] : r[3];
            const float usel = rg == 0 ? u[0] : rg == 1 ? u[1] : rg == 2 ? u[2] : u[3];
            static_cast<T*>(P.out)[(t * P.Hv + h) * D + 32 * w + 4 * cg + rg] =
                from_f32<T>(iq * rsel + usel * kq);
#pragma unroll
            for (int c = 0; c < 4; ++c) u[c] *= ik;
#pragma unroll
            for (int i = 0; i < R; i += 4) {
                const float4 kv = k4[i / 4];
                const float kr[4] = {kv.x, kv.y, kv.z, kv.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float4& x = s[i + e];
                    x.x += kr[e] * u[0]; x.y += kr[e] * u[1]; x.z += kr[e] * u[2]; x.w += kr[e] * u[3];
                }
            }
            const int32_t to = P.slots_out[t];
            if (to >= 0 && to < P.num_slots) {
                float* dst = P.state + (size_t)to * slot_stride + corner;
#pragma unroll
                for (int i = 0; i < R; ++i) __stcs(reinterpret_cast<float4*>(dst + (size_t)i * D), s[i]);
            } else if (to != -1 && tid == 0) {
                kda_set_status(KDA_ERR_BAD_SLOT);
            }
        }
    }
}

template <int D, typename T>
cudaError_t launch(const Params& P, cudaStream_t stream) {
    return kda_launch_chained(decode_pool_kernel<D, T>, dim3((unsigned)P.num_seqs * (unsigned)P.Hv), D, 0, stream, P);
}

}  // namespace pool
}  // namespace kda
