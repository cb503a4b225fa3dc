// The gated delta rule's recurrent form over a pool of states: one or several tokens per
// sequence, the state read from one slot of the pool and stored to others.
//
// With the state S[key][value] of one head, one token is
//   S' = Diag(e^g) S;  p = S'^T k;  r = S'^T q;  u = beta (v - p)
//   o  = r + u (k . q);   S = S' + k u^T
// The value channels (columns of S) never meet, so a warp owns 16 columns and keeps its D x 16
// slice in registers over all tokens of the sequence, D / 8 rows of 4 columns a lane: no barrier stands
// between two tokens, and the slice is read once and written once per stored state.  Bound by the
// states' bytes.  With 32 columns a warp, 206 registers left 8 warps an SM: 256 x 32 states of 128 x 128
// took 196 us, now 181 to 189 (5.8 TB/s of reads and writes; slots in order 8 us less), and 16 tokens of 33 x 12
// states of 64 x 64 17.5 us, now 11.7.  A prefetch of the next CTA's state to L2 cost 7 us, warps with runs of
// 128 bytes instead of 64 and a sum over two warps 3 us.
#pragma once

#include "kda_launch.cuh"

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

// One CTA of 2 D threads per (sequence, value head).  Lane (rg, cg) = (lane / 4, lane % 4) of warp w holds
// rows rg * D/8 .. + D/8 - 1 of columns 16 w + 4 cg .. + 3.
template <int D, typename T>
__global__ void __launch_bounds__(2 * D, 256 / D) decode_pool_kernel(const __grid_constant__ Params P) {
    constexpr int R = D / 8;           // rows per lane
    constexpr int PAD = R + 4;         // the eight row groups fall into different banks
    constexpr int W = D / 32;          // warps of the channels of a token
    struct Stage {
        float k[kTokens][8 * PAD], q[kTokens][8 * PAD], a[kTokens][8 * PAD];
        float v[kTokens][D];
        float dot[kTokens][3][W];      // k.q, k.k, q.q by warp
        float beta[kTokens];
        int32_t to[kTokens];
    };
    __shared__ __align__(16) Stage stages[2];

    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int rg = lane >> 2, cg = lane & 3;
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

    const int hk = h / (P.Hv / P.Hk);
    const bool scalar = P.in_flags & kInGScalar, logits = P.in_flags & kInGLogits;
    const bool norm = P.in_flags & kInNormQK;
    // Staging: channel ch of tokens part and part + 2 of a group of four; the next group's are on their
    // way while one is computed.
    const int ch = tid % D, part = tid / D;
    const int pos = (ch / R) * PAD + ch % R;   // in the padded arrays
    float fk[2], fq[2], fg[2], fv[2], fb = 0.f;
    int32_t fto = -1;
    auto fetch = [&](int64_t tb) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int64_t t = tb + part + 2 * x;
            fk[x] = fq[x] = fg[x] = fv[x] = 0.f;
            if (t < t1) {
                fk[x] = to_f32(static_cast<const T*>(P.k)[t * P.k_stride + hk * D + ch]);
                fq[x] = to_f32(static_cast<const T*>(P.q)[t * P.q_stride + hk * D + ch]);
                fg[x] = scalar ? P.g[t * P.Hv + h] : P.g[(t * P.Hv + h) * D + ch];
                fv[x] = to_f32(static_cast<const T*>(P.v)[t * P.v_stride + h * D + ch]);
            }
        }
        if (tid < kTokens && tb + tid < t1) {
            fb = P.beta[(tb + tid) * P.Hv + h];
            fto = P.slots_out[tb + tid];
        }
    };
    auto stage = [&](Stage& st) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int j = part + 2 * x;
            st.k[j][pos] = fk[x];
            st.q[j][pos] = fq[x];
            // with gate logits x the decay is e^{logsigmoid(x)} = sigmoid(x)
            st.a[j][pos] = logits ? kda_sigmoid(fg[x]) : expf(fg[x]);
            st.v[j][ch] = fv[x];
            float kq = fk[x] * fq[x], k2 = fk[x] * fk[x], q2 = fq[x] * fq[x];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                kq += __shfl_xor_sync(0xffffffffu, kq, o);
                if (norm) {
                    k2 += __shfl_xor_sync(0xffffffffu, k2, o);
                    q2 += __shfl_xor_sync(0xffffffffu, q2, o);
                }
            }
            if (lane == 0) {
                st.dot[j][0][w % W] = kq;
                st.dot[j][1][w % W] = k2;
                st.dot[j][2][w % W] = q2;
            }
        }
        if (tid < kTokens) {
            st.beta[tid] = P.in_flags & kInBetaLogits ? kda_sigmoid(fb) : fb;
            st.to[tid] = fto;
        }
    };

    fetch(t0);
    if (slot < -1 || slot >= P.num_slots) {
        if (tid == 0) kda_set_status(KDA_ERR_BAD_SLOT);
        return;
    }
    const size_t slot_stride = (size_t)P.Hv * D * D;
    // this lane's corner of a head's state
    const size_t corner = (size_t)h * D * D + (size_t)(rg * R) * D + 16 * w + 4 * cg;
    float4 s[R];
    if (slot >= 0) {
        const float* src = P.state + (size_t)slot * slot_stride + corner;
#pragma unroll
        for (int i = 0; i < R; ++i) s[i] = __ldcs(reinterpret_cast<const float4*>(src + (size_t)i * D));
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    stage(stages[0]);
    __syncthreads();

    int buf = 0;
    for (int64_t tb = t0; tb < t1; tb += kTokens, buf ^= 1) {
        const int nt = (int)min((int64_t)kTokens, t1 - tb);
        const bool more = tb + kTokens < t1;
        if (more) fetch(tb + kTokens);
        const Stage& st = stages[buf];
        for (int j = 0; j < nt; ++j) {
            const int64_t t = tb + j;
            float kq = 0.f, ik = 1.f, iq = 1.f;
#pragma unroll
            for (int x = 0; x < W; ++x) kq += st.dot[j][0][x];
            if (norm) {   // k and q enter unnormalised; their norms scale p, r, u and k . q
                float k2 = 0.f, q2 = 0.f;
#pragma unroll
                for (int x = 0; x < W; ++x) { k2 += st.dot[j][1][x]; q2 += st.dot[j][2][x]; }
                ik = kda_inv_norm(k2);
                iq = kda_inv_norm(q2);
                kq *= ik * iq;
            }
            const float4* k4 = reinterpret_cast<const float4*>(&st.k[j][rg * PAD]);
            const float4* q4 = reinterpret_cast<const float4*>(&st.q[j][rg * PAD]);
            const float4* a4 = reinterpret_cast<const float4*>(&st.a[j][rg * PAD]);
            float p[8] = {};   // S'^T k of the four columns, then S'^T q
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
                    p[4] += x.x * qr[e]; p[5] += x.y * qr[e]; p[6] += x.z * qr[e]; p[7] += x.w * qr[e];
                }
            }
            // sums over the row groups: each step halves the values that a lane goes on with, so that row
            // group rg ends with value rg
#pragma unroll
            for (int o = 4; o > 0; o >>= 1)
#pragma unroll
                for (int i = 0; i < o; ++i) {
                    const bool hi = rg & o;
                    const float give = hi ? p[i] : p[i + o], keep = hi ? p[i + o] : p[i];
                    p[i] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * o);
                }
            // row groups 0 .. 3 have p of column rg and form u, 4 .. 7 have r of column rg - 4 and the output
            const float u1 = st.beta[j] * (st.v[j][16 * w + 4 * cg + (rg & 3)] - ik * p[0]);
            const float mine = __shfl_xor_sync(0xffffffffu, u1, 16);
            if (rg >= 4)
                static_cast<T*>(P.out)[(t * P.Hv + h) * D + 16 * w + 4 * cg + rg - 4] = from_f32<T>(iq * p[0] + mine * kq);
            float u[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) u[c] = ik * __shfl_sync(0xffffffffu, u1, 4 * c + cg);
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
            const int32_t to = st.to[j];
            if (to >= 0 && to < P.num_slots) {
                float* dst = P.state + (size_t)to * slot_stride + corner;
#pragma unroll
                for (int i = 0; i < R; ++i) __stcs(reinterpret_cast<float4*>(dst + (size_t)i * D), s[i]);
            } else if (to != -1 && tid == 0) {
                kda_set_status(KDA_ERR_BAD_SLOT);
            }
        }
        if (more) {
            stage(stages[buf ^ 1]);
            __syncthreads();
        }
    }
}

template <int D, typename T>
cudaError_t launch(const Params& P, cudaStream_t stream) {
    return kda_launch_chained(decode_pool_kernel<D, T>, dim3((unsigned)P.num_seqs * (unsigned)P.Hv), 2 * D, 0, stream, P);
}

}  // namespace pool
}  // namespace kda
