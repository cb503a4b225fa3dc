// Appending new keys and values to the paged cache, with the rotary rotation of the keys
// and queries on the way.
//
// Pair i of a head turns by angle = position * inv_freq[i]:
//   y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin.
// Positions reach 2^31 and an fp32 angle of 2^20 is off by up to 2^-5, so the angle is
// formed in fp64, in turns, and only its fraction of a turn is rounded to fp32.  The kernel is
// bound by memory: every element is read once and written once, and a token's sines are
// computed once for all of its heads.
#pragma once

#include "kda_kv_cache.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace append {

struct Params {
    const void *k, *v, *q;
    int64_t k_stride, v_stride, q_stride;
    const int32_t* cu;
    int32_t num_seqs, Hq;
    int64_t total;
    void* q_out;
    const float* inv_freq;
    const int32_t* positions;
    int32_t rot, axis_end[4], adjacent;
    kv::Cache c;
};

constexpr int kThreads = 128;

template <typename T> struct Vec8;   // 8 consecutive elements
template <> struct Vec8<float> {
    static __device__ __forceinline__ void load(const float* p, float* x) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    static __device__ __forceinline__ void store(float* p, const float* x) {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};
template <> struct Vec8<__nv_bfloat16> {
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* x) {
        sm100::unpack_bf16x8(*reinterpret_cast<const uint4*>(p), x);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* x) {
        *reinterpret_cast<uint4*>(p) = sm100::pack_bf16x8(x);
    }
};
template <> struct Vec8<__nv_fp8_e4m3> {
    // rounded to nearest even, finite values held at +-448
    static __device__ __forceinline__ void store(__nv_fp8_e4m3* p, const float* x) {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
            w[i] = lo | (hi << 16);
        }
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
};

// The sequence of token t: the last n with cu[n] <= t, found by the 32 lanes of a warp
// together (each step keeps one of 32 parts).  -1 for padding, or where cu is inconsistent
// around t (reported).
__device__ __forceinline__ int find_sequence(const Params& P, int64_t t, int lane) {
    if (!P.cu) return (int)t;
    int lo = 0, hi = P.num_seqs;   // cu[lo] <= t; the answer lies in [lo, hi]
    while (hi - lo > 0) {
        const int step = (hi - lo + 31) / 32;
        const int at = min(lo + (lane + 1) * step, hi);
        const unsigned m = __ballot_sync(0xffffffffu, P.cu[at] <= t);
        // entries rise, so the lanes that vote yes come first
        const int c = __popc(m);
        const int nlo = c == 0 ? lo : min(lo + c * step, hi);
        const int nhi = c == 32 ? hi : min(lo + (c + 1) * step, hi) - 1;
        lo = nlo;
        hi = max(nhi, nlo);
        if (c == 32) { lo = hi; }
    }
    if (lo >= P.num_seqs) return -1;   // behind the last sequence
    const int64_t a = P.cu[lo], b = P.cu[lo + 1];
    if (a < 0 || t < a || t >= b || b > P.total || (lo == 0 && a != 0)) {
        if (lane == 0) kda_set_status(KDA_ERR_BAD_SEQLENS);
        return -1;
    }
    return lo;
}

// One CTA per token.
template <int D, typename T, typename TC>
__global__ void __launch_bounds__(kThreads) append_kernel(const Params P) {
    __shared__ float scos[D / 2], ssin[D / 2];
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t t = blockIdx.x;
    kda_grid_wait();
    const int n = find_sequence(P, t, lane);
    if (n < 0) return;
    const int64_t t0 = P.cu ? P.cu[n] : n, t1 = P.cu ? P.cu[n + 1] : n + 1;
    const int64_t pos = (int64_t)P.c.seq_lens[n] - (t1 - t0) + (t - t0);
    const int64_t row = kv::row_offset(P.c, n, pos, 0);
    if (row < 0 && tid == 0) kda_set_status(KDA_ERR_BAD_PAGE);
    const int half = P.rot / 2;
    for (int i = tid; i < half; i += kThreads) {
        int axis = 0;
        while (axis < 3 && i >= P.axis_end[axis]) ++axis;
        const double x = P.positions ? (double)P.positions[axis * P.total + t] : (double)pos;
        double turns = x * (double)P.inv_freq[i] * 0.15915494309189533577;   // 1 / (2 pi)
        turns -= rint(turns);
        sincospif(2.f * (float)turns, &ssin[i], &scos[i]);
    }
    __syncthreads();

    // units of work: 8 channels, or 8 and their partners half a rotation on
    const int paired = P.adjacent ? 0 : half / 8;             // units of two vectors per head
    const int per_rot = paired + (D - (P.adjacent ? 0 : P.rot)) / 8;
    const int rows_rot = P.Hq + P.c.Hkv;
    const int units = rows_rot * per_rot + P.c.Hkv * (D / 8);
    for (int u = tid; u < units; u += kThreads) {
        float x[8], y[8];
        if (u >= rows_rot * per_rot) {   // values: a copy
            const int e = u - rows_rot * per_rot, h = e / (D / 8), i = e % (D / 8);
            if (row < 0) continue;
            Vec8<T>::load(static_cast<const T*>(P.v) + t * P.v_stride + h * D + 8 * i, x);
            if constexpr (sizeof(TC) == 1) {
                const float sc = P.c.v_scale ? P.c.v_scale[h] : 1.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] /= sc;
            }
            Vec8<TC>::store(static_cast<TC*>(P.c.v) + row + h * P.c.head_stride + 8 * i, x);
            continue;
        }
        const int hr = u / per_rot, i = u % per_rot;
        const bool is_q = hr < P.Hq;
        const int h = is_q ? hr : hr - P.Hq;
        if (!is_q && row < 0) continue;
        const T* src = is_q ? static_cast<const T*>(P.q) + t * P.q_stride + h * D
                            : static_cast<const T*>(P.k) + t * P.k_stride + h * D;
        const bool two = i < paired;
        const int c0 = two ? 8 * i : (P.adjacent ? 8 * i : P.rot + 8 * (i - paired));
        Vec8<T>::load(src + c0, x);
        if (two) {
            float z[8];
            Vec8<T>::load(src + c0 + half, z);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float c = scos[c0 + j], s = ssin[c0 + j];
                y[j] = z[j] * c + x[j] * s;
                x[j] = x[j] * c - z[j] * s;
            }
        } else if (P.adjacent && c0 < P.rot) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float c = scos[c0 / 2 + j], s = ssin[c0 / 2 + j];
                const float a = x[2 * j], b = x[2 * j + 1];
                x[2 * j] = a * c - b * s;
                x[2 * j + 1] = b * c + a * s;
            }
        }
        if (is_q) {
            T* dst = static_cast<T*>(P.q_out) + (t * P.Hq + h) * D + c0;
            Vec8<T>::store(dst, x);
            if (two) Vec8<T>::store(dst + half, y);
        } else {
            if constexpr (sizeof(TC) == 1) {
                const float sc = P.c.k_scale ? P.c.k_scale[h] : 1.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) { x[j] /= sc; y[j] /= sc; }
            }
            TC* dst = static_cast<TC*>(P.c.k) + row + h * P.c.head_stride + c0;
            Vec8<TC>::store(dst, x);
            if (two) Vec8<TC>::store(dst + half, y);
        }
    }
}

template <int D, typename T, typename TC>
cudaError_t launch(const Params& P, cudaStream_t stream) {
    return kda_launch_chained(append_kernel<D, T, TC>, dim3((unsigned)P.total), kThreads, 0, stream, P);
}

}  // namespace append
}  // namespace kda
