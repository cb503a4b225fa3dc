// The paged attention in fp32, on CUDA cores: no tensor-core type holds the products, and one
// product in three tf32 parts would need every key and value split on the way.  With up to 8
// query rows a CTA's 36 TFMA/s / 148 keep up with its share of the memory bandwidth.
//
// A tile is 32 KB of keys and values.  The 8 consumer warps take it together, in three steps
// between barriers: scores (a thread has 16 channels of one key, summed up over 4 or 8 lanes),
// weights (warp r has row r), values (a thread has one channel and 16 keys).
#pragma once

#include "kda_kv_decode.cuh"

namespace kda {
namespace attend {

template <int D_, int R>
struct Simt {
    static constexpr int D = D_;
    static constexpr int TOK = 32 * 128 / D, CW = 8, THREADS = 32 * (CW + 2);
    static constexpr int ROWB = 4 * D, RAW = TOK * ROWB, STAGE = 2 * RAW;
    // for Fetch: blocks of 32 channels, 128-byte rows
    static constexpr bool QSWIZZLED = false;
    static constexpr int BLKS = D / 32, BROWB = 128, BLOCK = TOK * 128, QBLKS = 1, QROWB = ROWB, QBLOCK = 0;
    static constexpr int STG = 6, QS = STG, MD = STG + 2;
    static constexpr int PARTS = 32 * CW / TOK, KPW = 32 / PARTS;    // lanes of a key, keys of a warp
    static constexpr int GROUPS = 32 * CW / D;                       // threads of a channel, 16 keys each
    static constexpr int QB = R * D * 4;
    static constexpr int Q = STG * STAGE, SC = Q + QS * QB, RED = SC + 2 * R * TOK * 4;
    static constexpr int META = RED + R * D * 4, OKM = META + MD * 64, FROW = OKM + MD * 16, ML = FROW + 2 * R * 4, FULL = ML + 2 * R * 4,
                         EMPTY = FULL + 8 * STG, MFULL = EMPTY + 8 * STG, ABORT = MFULL + 8 * MD, BYTES = ABORT + 16;
    static_assert(BYTES <= kMaxSmem && META % 16 == 0 && FULL % 8 == 0, "shared memory of a CTA");
};

template <int D, int R>
struct SimtKernel {
    typedef Simt<D, R> C;
    typedef Walk<C::TOK, R> W;
    static constexpr int TOK = C::TOK;

    const Params& P;
    uint8_t* sm;
    uint32_t sb;

    __device__ __forceinline__ Meta* meta(int t) const { return reinterpret_cast<Meta*>(sm + C::META) + t % C::MD; }
    __device__ __forceinline__ void fail() const {
        kda_set_status(KDA_ERR_TIMEOUT);
        *reinterpret_cast<volatile uint32_t*>(sm + C::ABORT) = 1;
    }
    __device__ __forceinline__ bool aborted() const { return *reinterpret_cast<volatile uint32_t*>(sm + C::ABORT) != 0; }

    __device__ __forceinline__ void fetcher(Fetch<C, R>& f, W& w) {
        int puts = 0;
        const bool ok = f.run(
            w,
            [&](int t) {
                return !aborted() && (t < C::STG || wait_warp(sb + C::EMPTY + 8 * (t % C::STG), (t / C::STG - 1) & 1));
            },
            [&](int t) {
                f.put(w, sb + (t % C::STG) * C::STAGE, sb + C::Q + (w.item % C::QS) * C::QB, sb + C::FULL + 8 * (t % C::STG),
                      sb + C::FULL + 8 * (t % C::STG), sb + C::MFULL + 8 * (t % C::MD), meta(t),
                      reinterpret_cast<uint32_t*>(sm + C::OKM + (t % C::MD) * 16), nullptr);
                puts = t + 1;
            });
        if (!ok) {   // copies still in flight are waited for
            fail();
            for (int t = max(puts - C::STG, 0); t < puts; ++t) wait_warp(sb + C::FULL + 8 * (t % C::STG), (t / C::STG) & 1);
        }
    }

    // byte offset of 16-byte chunk ch of a key's row
    static __device__ __forceinline__ int chunk(int key, int ch) { return (ch >> 3) * C::BLOCK + (int)sm100::sw128_off(key, ch & 7); }

    __device__ __forceinline__ void consumer(int w, int lane) {
        constexpr uint32_t NT = 32 * C::CW;
        const int tid = 32 * w + lane;
        const int part = lane % C::PARTS, gr = lane / C::PARTS;
        // eight lanes read 128 bytes without a bank twice: with 4 lanes a key, of keys 4 apart
        const int key = w * C::KPW + (C::PARTS == 4 ? (gr >> 1) | ((gr & 1) << 2) : gr);
        const int d = tid % D, kg = tid / D;
        float acc[R], m = -INFINITY, l = 0.f;   // m, l: of row w
        bool bad = false;
        for (int t = 0;; ++t) {
            bad |= !wait_warp(sb + C::FULL + 8 * (t % C::STG), (t / C::STG) & 1);
            if (bar_any(1, bad || aborted(), NT)) break;
            const Meta mt = *meta(t);
            const uint32_t* okm = reinterpret_cast<const uint32_t*>(sm + C::OKM + (t % C::MD) * 16);
            bool all = true;   // all keys there
#pragma unroll
            for (int i = 0; i < TOK / 32; ++i) all = all && okm[i] == 0xffffffffu;
            const bool edge = (mt.flags & kEdge) || !all;
            const uint8_t* k = sm + (t % C::STG) * C::STAGE;
            const uint8_t* v = k + C::RAW;
            const float* q = reinterpret_cast<const float*>(sm + C::Q + (mt.item % C::QS) * C::QB);
            float* sc = reinterpret_cast<float*>(sm + C::SC) + (t & 1) * R * TOK;
            float* frow = reinterpret_cast<float*>(sm + C::FROW) + (t & 1) * R;
            if (mt.flags & kFirst) {
#pragma unroll
                for (int r = 0; r < R; ++r) acc[r] = 0.f;
                m = -INFINITY;
                l = 0.f;
            }
            {   // scores, in units of log 2; -infinity where the row does not see the key
                float4 kk[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    kk[i] = *reinterpret_cast<const float4*>(k + chunk(key, i * C::PARTS + part));
                const int j = mt.j0 + key;
                const bool ok = (okm[key >> 5] >> (key & 31)) & 1;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (r >= mt.rows) break;
                    float x = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 a = *reinterpret_cast<const float4*>(q + r * D + (i * C::PARTS + part) * 4);
                        x += a.x * kk[i].x + a.y * kk[i].y + a.z * kk[i].z + a.w * kk[i].w;
                    }
#pragma unroll
                    for (int o = 1; o < C::PARTS; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                    if (part == r % C::PARTS) {
                        const int ir = mt.block * R + r, tok = ir / P.group, p = mt.pos0 + tok;
                        x *= P.scale;
                        if (P.softcap > 0.f) x = P.softcap * tanhf(x / P.softcap);
                        x *= kLog2e;
                        if (P.slopes) x += P.slopes[mt.h * P.group + (ir - tok * P.group)] * kLog2e * (float)(j - p);
                        if (!ok || (edge && (j > p || j < first_key(P, mt.start, p)))) x = -INFINITY;
                        sc[r * TOK + key] = x;
                    }
                }
            }
            bar_all(1, NT);
            if (w < mt.rows) {
                float x[TOK / 32], top = -INFINITY;
#pragma unroll
                for (int i = 0; i < TOK / 32; ++i) {
                    x[i] = sc[w * TOK + 32 * i + lane];
                    top = fmaxf(top, x[i]);
                }
                top = fmaxf(m, warp_max(top));
                const float f = m == -INFINITY ? 0.f : ex2(m - top), ms = top == -INFINITY ? 0.f : top;
                m = top;
                l *= f;
#pragma unroll
                for (int i = 0; i < TOK / 32; ++i) {
                    const float p = ex2(x[i] - ms);
                    l += p;
                    sc[w * TOK + 32 * i + lane] = x[i] == -INFINITY ? -0.f : p;   // -0: takes nothing of the value
                }
                if (lane == 0) frow[w] = f;
            }
            bar_all(1, NT);
            {
                float vv[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int kx = kg * 16 + i;
                    vv[i] = *reinterpret_cast<const float*>(v + chunk(kx, d >> 2) + (d & 3) * 4);
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (r >= mt.rows) break;
                    float a = acc[r] * frow[r];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 p = *reinterpret_cast<const float4*>(sc + r * TOK + kg * 16 + 4 * i);
                        const float pp[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            // a row that does not see the key takes nothing of its value, be it NaN
                            if (!edge || __float_as_uint(pp[e]) != 0x80000000u) a += pp[e] * vv[4 * i + e];
                        }
                    }
                    acc[r] = a;
                }
            }
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(sb + C::EMPTY + 8 * (t % C::STG));
            if (mt.flags & kLast) {
                float* red = reinterpret_cast<float*>(sm + C::RED);
                float* ml = reinterpret_cast<float*>(sm + C::ML);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                if (w < R && lane == 0) { ml[w] = m; ml[R + w] = l; }
#pragma unroll
                for (int g = 0; g < C::GROUPS; ++g) {   // the groups add up their keys in turn
                    if (kg == g) {
#pragma unroll
                        for (int r = 0; r < R; ++r) red[r * D + d] = g == 0 ? acc[r] : red[r * D + d] + acc[r];
                    }
                    bar_all(1, NT);
                }
                float* to = P.partial + (int64_t)mt.part * (R * (D + 2));
                for (int x = tid; x < mt.rows * D; x += NT) {
                    const int r = x / D, c = x % D;
                    const float a = red[r * D + c];
                    const float sum = ml[R + r];
                    if (mt.part < 0) {
                        const int ir = mt.block * R + r, tok = ir / P.group;
                        const int64_t at = (mt.t0 + tok) * P.Hq + mt.h * P.group + (ir - tok * P.group);
                        static_cast<float*>(P.out)[at * D + c] = sum == 0.f ? 0.f : a / sum;
                        if (P.lse && c == 0) P.lse[at] = sum == 0.f ? -INFINITY : ml[r] * kLn2 + logf(sum);
                    } else {
                        to[2 * R + x] = a;
                        if (c == 0) { to[r] = ml[r]; to[R + r] = sum; }
                    }
                }
                if (mt.flags & kEnd) break;
            }
        }
        if (bad) fail();
    }

    __device__ __forceinline__ void run() {
        const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
        if (tid == 0) { prefetch_map(&P.k_map); prefetch_map(&P.v_map); prefetch_map(&P.q_map); }
        kda_grid_wait();
        W w(P);
        w.template find<C::THREADS>(reinterpret_cast<int64_t*>(sm));
        kda_grid_launch_next();
        Fetch<C, R> f{P, lane, warp == C::CW, {}};
        if (warp >= C::CW) {
            if (f.keys && lane == 0) {
                for (int i = 0; i < C::STG; ++i) {
                    sm100::mbar_init(sb + C::FULL + 8 * i, 1);
                    sm100::mbar_init(sb + C::EMPTY + 8 * i, C::CW);
                }
                for (int i = 0; i < C::MD; ++i) sm100::mbar_init(sb + C::MFULL + 8 * i, 1);
                sm100::fence_mbar_init();
            }
            const bool any = f.begin(w);
            if (f.keys && lane == 0) *reinterpret_cast<volatile uint32_t*>(sm + C::ABORT) = 0;
            if (f.keys && lane == 0) *reinterpret_cast<volatile uint32_t*>(sm + C::ABORT + 4) = any;
        }
        __syncthreads();
        if (!*reinterpret_cast<volatile uint32_t*>(sm + C::ABORT + 4)) return;
        if (warp < C::CW) consumer(warp, lane);
        else fetcher(f, w);
    }
};

template <int D, int R>
__global__ void __launch_bounds__(Simt<D, R>::THREADS, 1) attend_simt_kernel(const __grid_constant__ Params P) {
    extern __shared__ __align__(1024) uint8_t smem[];
    SimtKernel<D, R> k{P, smem, sm100::smem_u32(smem)};
    k.run();
}

}  // namespace attend
}  // namespace kda
