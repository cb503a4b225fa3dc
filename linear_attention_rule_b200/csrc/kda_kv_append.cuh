// Appending new keys and values to the paged cache, with the rotary rotation of the keys
// and queries on the way.
//
// Pair i of a head turns by angle = position * inv_freq[i]:
//   y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin.
// Positions reach 2^31 and an fp32 angle of 2^20 is off by up to 2^-5, so the angle is formed in
// fp64, in turns; its fraction of a turn goes to fp32 in two parts, the second of which turns
// the first part's sine and cosine to first order.  The kernel is bound by memory: every element is read
// once and written once.
//
// A warp has one token, or every 2nd or 4th part of one where there are few tokens.  Its lanes hold the
// same channels of several heads, so that a lane's sines and cosines stay in registers; the first
// loads are on their way before the token's sequence, page and angles are known.  With a CTA per token,
// a table of sines in shared memory and the loads behind it, 9,221 tokens of 16 + 2 x 4 heads took 48 us, now 26.3;
// 34,953 of 32 + 2 x 8 heads took 164 us, now 140 (6.15 TB/s).  Keys and values brought to L2 ahead by a
// prefetch made the latter 155.
#pragma once

#include <cfloat>

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
    int32_t rot, axis_end[4], adjacent, parts;   // parts: warps of a token
    uint32_t blocks;                                // CTAs of the tokens
    kv::Cache c;
};

constexpr int kWarps = 4;

template <typename T> struct Vec8;   // 8 consecutive elements
template <> struct Vec8<float> {
    typedef struct { float4 a, b; } Raw;
    static __device__ __forceinline__ Raw fetch(const float* p) {
        return {reinterpret_cast<const float4*>(p)[0], reinterpret_cast<const float4*>(p)[1]};
    }
    static __device__ __forceinline__ void unpack(const Raw& r, float* x) {
        x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
        x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
    }
    static __device__ __forceinline__ void store(float* p, const float* x) {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};
template <> struct Vec8<__nv_bfloat16> {
    typedef uint4 Raw;
    static __device__ __forceinline__ Raw fetch(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }
    static __device__ __forceinline__ void unpack(const Raw& r, float* x) { sm100::unpack_bf16x8(r, x); }
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

// Whether the entries of sequence n are consistent; whether it has token t and they are.
__device__ __forceinline__ bool consistent(const Params& P, int n, int a, int b) {
    return a >= 0 && b >= a && b <= P.total && (n > 0 || a == 0);
}
__device__ __forceinline__ bool has_token(const Params& P, int n, int t) {
    const int a = P.cu[n], b = P.cu[n + 1];
    return a <= t && t < b && consistent(P, n, a, b);
}
// A sequence that has token t, -1 for none, by the 32 lanes of a warp together.  Entries that rise are searched: the
// first n with cu[n + 1] > t (each step keeps one of 32 parts).  Where that is no sequence of the token's, it is padding
// or an inconsistent entry misled the search, and all are looked at (up to 32 the search has seen them all, and
// only one that it ends at can mislead it).
__device__ __forceinline__ int find_sequence(const Params& P, int64_t t, int lane) {
    if (!P.cu) return (int)t;
    int lo = 0, hi = P.num_seqs;   // the answer lies in [lo, hi]
    while (hi - lo > 0) {
        const int step = (hi - lo + 31) / 32;
        const int at = min(lo + (lane + 1) * step, hi);
        const unsigned m = __ballot_sync(0xffffffffu, P.cu[at] <= t);
        // the lanes that vote yes before the first that does not; entries that fall have others behind it
        const int c = __clz(__brev(~m));
        const int nlo = c == 0 ? lo : min(lo + c * step, hi);
        const int nhi = c == 32 ? hi : min(lo + (c + 1) * step, hi) - 1;
        lo = nlo;
        hi = max(nhi, nlo);
        if (c == 32) { lo = hi; }
    }
    if (lo < P.num_seqs ? has_token(P, lo, (int)t) : P.num_seqs <= 32) return lo < P.num_seqs ? lo : -1;
#pragma unroll 1
    for (int n = lane; n - lane < P.num_seqs; n += 32) {
        const unsigned m = __ballot_sync(0xffffffffu, n < P.num_seqs && has_token(P, n, (int)t));
        if (m) return n - lane + __ffs(m) - 1;
    }
    return -1;
}

// x / d for the quotients that are rounded to 8 bits, r = 1 / d rounded to nearest: the product's
// remainder is exact in one fma, and with it the quotient is the correctly rounded one (Markstein 1990).
__device__ __forceinline__ float quotient(float x, float d, float r) {
    const float q = x * r, better = fmaf(fmaf(-q, d, x), r, q);
    return fabsf(q) <= 3.4e38f ? better : q;   // infinities and NaN as they are
}

template <int D, typename T, typename TC>
struct Token {
    typedef typename Vec8<T>::Raw Raw;
    static constexpr bool F8 = sizeof(TC) == 1;

    const Params& P;
    int64_t t;
    int lane, part;
    // A unit is 8 channels, or 8 and their partners half a rotation on; `width` lanes have a head's.
    int half, units, width;
    bool mine, two;            // this lane has a unit, and it has partners
    int c0;                    // its first channel
    int first, step;           // this lane's heads
    float c[8], s[8];          // cosines and sines of its pairs

    __device__ __forceinline__ Token(const Params& p, int64_t token, int ln, int pt) : P(p), t(token), lane(ln), part(pt) {
        half = P.rot / 2;
        const int paired = P.adjacent ? 0 : half / 8;
        units = paired + (D - (P.adjacent ? 0 : P.rot)) / 8;
        width = units <= 8 ? 8 : 16;
        const int u = lane % width;
        mine = u < units;
        two = u < paired;
        c0 = two || P.adjacent ? 8 * u : P.rot + 8 * (u - paired);
        step = 32 / width * P.parts;
        first = part * (32 / width) + lane / width;
    }
    // Two heads, `first` and `step` behind it, of `heads`.
    __device__ __forceinline__ void fetch(const T* src, int h, int heads, Raw (&a)[2], Raw (&b)[2]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (mine && h + i * step < heads) {
                const T* at = src + (int64_t)(h + i * step) * D;
                a[i] = Vec8<T>::fetch(at);
                if (two) b[i] = Vec8<T>::fetch(at + half);
            }
    }
    // Sines and cosines of the token: each lane forms those of pairs lane and lane + 32, then takes its own.
    __device__ __forceinline__ void angles(int64_t pos) {
        float cc[2] = {1.f, 1.f}, ss[2] = {0.f, 0.f};
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
            const int i = lane + 32 * x;
            if (i < half) {
                const int axis = (i >= P.axis_end[0]) + (i >= P.axis_end[1]) + (i >= P.axis_end[2]);
                const double where = P.positions ? (double)P.positions[axis * P.total + t] : (double)pos;
                double turns = where * (double)P.inv_freq[i] * 0.15915494309189533577;   // 1 / (2 pi)
                turns -= rint(turns);
                const float hi = (float)turns, lo = (float)(turns - (double)hi) * 6.2831853f;
                float sn, cs;
                sincospif(2.f * hi, &sn, &cs);
                ss[x] = sn + cs * lo;
                cc[x] = cs - sn * lo;
            }
        }
        const int p0 = P.adjacent ? c0 / 2 : c0, n = P.adjacent ? 4 : 8;   // this lane's pairs
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j >= n) break;
            const int i = p0 + j;
            const float c_lo = __shfl_sync(0xffffffffu, cc[0], i & 31), s_lo = __shfl_sync(0xffffffffu, ss[0], i & 31);
            c[j] = c_lo;
            s[j] = s_lo;
            if (D > 64) {
                const float c_hi = __shfl_sync(0xffffffffu, cc[1], i & 31), s_hi = __shfl_sync(0xffffffffu, ss[1], i & 31);
                if (i >= 32) { c[j] = c_hi; s[j] = s_hi; }
            }
        }
    }
    __device__ __forceinline__ void turn(const Raw& a, const Raw& b, float (&x)[8], float (&y)[8]) const {
        Vec8<T>::unpack(a, x);
        if (two) {
            float z[8];
            Vec8<T>::unpack(b, z);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y[j] = z[j] * c[j] + x[j] * s[j];
                x[j] = x[j] * c[j] - z[j] * s[j];
            }
        } else if (P.adjacent && c0 < P.rot) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = x[2 * j], o = x[2 * j + 1];
                x[2 * j] = e * c[j] - o * s[j];
                x[2 * j + 1] = o * c[j] + e * s[j];
            }
        }
    }
    static __device__ __forceinline__ void put(TC* dst, float (&x)[8], const float* scales, int h) {
        if constexpr (F8) {
            if (scales) {
                // finite also for a subnormal d, so that 0 stays 0
                const float d = scales[h], r = fminf(__frcp_rn(d), FLT_MAX);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = quotient(x[j], d, r);
            }
        }
        Vec8<TC>::store(dst, x);
    }
    // The next heads are on their way while two are turned: two more with AHEAD, else each head's as soon as
    // its registers are free.
    template <bool AHEAD>
    __device__ __forceinline__ void queries(Raw (&a)[2], Raw (&b)[2]) const {
        const T* src = static_cast<const T*>(P.q) + t * P.q_stride + c0;
        T* dst = static_cast<T*>(P.q_out) + t * P.Hq * D + c0;
        if constexpr (AHEAD) {
            for (int h = first; h < P.Hq; h += 2 * step) {
                Raw na[2], nb[2];
                fetch(src, h + 2 * step, P.Hq, na, nb);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x[8], y[8];
                    if (!mine || h + i * step >= P.Hq) continue;
                    turn(a[i], b[i], x, y);
                    T* at = dst + (int64_t)(h + i * step) * D;
                    Vec8<T>::store(at, x);
                    if (two) Vec8<T>::store(at + half, y);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) { a[i] = na[i]; b[i] = nb[i]; }
            }
        } else {
            for (int h = first; h < P.Hq; h += 2 * step) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x[8], y[8];
                    const int now = h + i * step, next = now + 2 * step;
                    if (!mine || now >= P.Hq) continue;
                    turn(a[i], b[i], x, y);
                    if (next < P.Hq) {
                        const T* from = src + (int64_t)next * D;
                        a[i] = Vec8<T>::fetch(from);
                        if (two) b[i] = Vec8<T>::fetch(from + half);
                    }
                    T* at = dst + (int64_t)now * D;
                    Vec8<T>::store(at, x);
                    if (two) Vec8<T>::store(at + half, y);
                }
            }
        }
    }
    __device__ __forceinline__ void keys(int64_t row) const {
        const T* src = static_cast<const T*>(P.k) + t * P.k_stride + c0;
        TC* dst = static_cast<TC*>(P.c.k) + row + c0;
        for (int h = first; h < P.c.Hkv; h += 2 * step) {
            Raw a[2], b[2];
            fetch(src, h, P.c.Hkv, a, b);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x[8], y[8];
                const int hi = h + i * step;
                if (!mine || hi >= P.c.Hkv) continue;
                turn(a[i], b[i], x, y);
                put(dst + hi * P.c.head_stride, x, P.c.k_scale, hi);
                if (two) put(dst + hi * P.c.head_stride + half, y, P.c.k_scale, hi);
            }
        }
    }
    __device__ __forceinline__ void values(int64_t row) const {   // a copy
        constexpr int U = D / 8;
        const T* src = static_cast<const T*>(P.v) + t * P.v_stride;
        TC* dst = static_cast<TC*>(P.c.v) + row;
        const int n = P.c.Hkv * U;
        for (int e = 32 * part + lane; e < n; e += 64 * P.parts) {
            Raw a[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (e + i * 32 * P.parts < n) a[i] = Vec8<T>::fetch(src + (int64_t)(e + i * 32 * P.parts) * 8);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at = e + i * 32 * P.parts, h = at / U;
                if (at >= n) continue;
                float x[8];
                Vec8<T>::unpack(a[i], x);
                put(dst + h * P.c.head_stride + 8 * (at % U), x, P.c.v_scale, h);
            }
        }
    }
};

template <int D, typename T, typename TC, bool AHEAD>
__global__ void __launch_bounds__(32 * kWarps, sizeof(T) == 2 ? 8 : 6) append_kernel(const __grid_constant__ Params P) {
    typedef Token<D, T, TC> Tok;
    const int lane = threadIdx.x & 31;
    const int64_t id = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t t = id / P.parts;
    const int part = (int)(id - t * P.parts);
    kda_grid_wait();
    if (blockIdx.x >= P.blocks) {   // the CTAs behind the tokens' look at the entries of a sequence a thread
        const int64_t n = (int64_t)(blockIdx.x - P.blocks) * (32 * kWarps) + threadIdx.x;
        if (n < P.num_seqs && !consistent(P, (int)n, P.cu[n], P.cu[n + 1])) kda_set_status(KDA_ERR_BAD_SEQLENS);
        return;
    }
    if (t >= P.total) return;
    Tok k(P, t, lane, part);
    typename Tok::Raw a[2], b[2];
    if (P.q) k.fetch(static_cast<const T*>(P.q) + t * P.q_stride + k.c0, k.first, P.Hq, a, b);
    const int n = find_sequence(P, t, lane);
    if (n < 0) return;
    const int64_t t0 = P.cu ? P.cu[n] : n, t1 = P.cu ? P.cu[n + 1] : n + 1;
    const int64_t pos = (int64_t)P.c.seq_lens[n] - (t1 - t0) + (t - t0);
    const int64_t row = kv::row_offset(P.c, n, pos, 0);
    if (row < 0 && lane == 0) kda_set_status(KDA_ERR_BAD_PAGE);
    if (P.rot) k.angles(pos);
    if (P.q) k.template queries<AHEAD>(a, b);
    if (row < 0) return;
    k.keys(row);
    k.values(row);
}

template <int D, typename T, typename TC>
cudaError_t launch(Params& P, cudaStream_t stream) {
    // Few tokens are shared by several warps each, so that the heads of one do not queue behind each other (a
    // call by itself): 64 tokens take 14.3 us by one warp each, 10.2 by four, 600 tokens 16.4 and 12.3; 1,500
    // tokens take 18.4 by one, 16.4 by two, 18.4 by four; prompts of 34,953 145 by one, 158 by four.
    P.parts = P.total >= 148 * 16 ? 1 : P.total >= 148 * 8 ? 2 : 4;
    P.blocks = (uint32_t)((P.total * P.parts + kWarps - 1) / kWarps);
    const dim3 grid(P.blocks + (P.cu ? ((uint32_t)P.num_seqs + 32 * kWarps - 1) / (32 * kWarps) : 0));
    // Two heads further ahead where a bf16 token's heads are all one warp's: 34,953 tokens of 32 + 2 x 8 heads with
    // neighbours paired take 147 us instead of 174, over e4m3 133 instead of 140.  It spills 52 to 60 bytes of
    // stores (28 to 40 without), which costs where the loop is short (1,500 tokens 7.6 us instead of 7.3) or a head takes twice
    // the registers (fp32, 4 prompts: 192 us instead of 176).
    if constexpr (sizeof(T) == 2)
        if (P.parts == 1)
            return kda_launch_chained(append_kernel<D, T, TC, true>, grid, 32 * kWarps, 0, stream, P);
    return kda_launch_chained(append_kernel<D, T, TC, false>, grid, 32 * kWarps, 0, stream, P);
}

}  // namespace append
}  // namespace kda
