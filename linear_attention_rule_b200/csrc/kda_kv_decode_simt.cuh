// The paged attention in fp32, on CUDA cores: no tensor-core type holds the products, and one
// product in three tf32 parts would need every key and value split on the way.  With up to 8
// query rows a CTA's 36 TFMA/s / 148 keep up with its share of the memory bandwidth.
//
// A tile is 32 KB of keys and values.  The 8 consumer warps take it together, with one barrier: scores
// (a thread has 16 channels of one key, summed up over 4 or 8 lanes) before it, values (a thread has one
// channel and 16 keys) behind it.  The weights in between are formed by every warp for itself: with
// a warp per row and another barrier a tile took half as long again.
//
// 16 x 4,096 keys, 8 heads of 128, 537 MB: 89 us with one row a head (6.0 TB/s), 112 with two, 154 with four, 242
// with eight; 16 rows, two blocks that read the cache each, 464.  One row is bound by memory, several by the
// latency of shared memory and of the sums with 8 warps an SM (8 rows: 37% of the issue slots, 51% of the load/store pipe).  Four channels of four keys
// a thread, a quarter of the weights' loads, changed nothing per tile and made item ends dearer.
#pragma once

#include <type_traits>

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
    static constexpr int STG = R <= 2 ? 6 : 5, QS = STG, MD = STG + 2;
    static constexpr int PARTS = 32 * CW / TOK, KPW = 32 / PARTS;    // lanes of a key, keys of a warp
    static constexpr int GROUPS = 32 * CW / D;                       // threads of a channel, 16 keys each
    static constexpr int QB = R * D * 4;
    static constexpr int Q = STG * STAGE, SC = Q + QS * QB, PW = SC + 2 * R * TOK * 4, RED = PW + CW * R * TOK * 4, META = RED + R * D * 4,
                         OKM = META + MD * 64, FULL = OKM + MD * 16, EMPTY = FULL + 8 * STG, MFULL = EMPTY + 8 * STG,
                         ABORT = MFULL + 8 * MD, BYTES = ABORT + 16;
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
        float* pw = reinterpret_cast<float*>(sm + C::PW) + w * R * TOK;   // the warp's copy of the weights
        // Rows go by groups of G without a branch between them, so that their chains overlap; those of a
        // group behind the block's last row are zeros and go nowhere.  After the sums a lane
        // has the score of row part % G of each group.
        constexpr int G = R < 4 ? R : 4, GS = R / G;
        const int mine = part & (G - 1);
        float acc[R], m[R], l[R], slope[GS];   // l: this lane's keys
        int tok[GS];
        bool bad = false;
        for (int t = 0;; ++t) {
            bad |= !wait_warp(sb + C::FULL + 8 * (t % C::STG), (t / C::STG) & 1);
            if (bad) {   // nothing of the tile is known: the vote below, and all stop
                bar_any(1, true, NT);
                break;
            }
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
            if (mt.flags & kFirst) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    acc[r] = 0.f;
                    m[r] = -INFINITY;
                    l[r] = 0.f;
                }
#pragma unroll
                for (int g = 0; g < GS; ++g) {
                    const int r = g * G + mine;
                    slope[g] = P.slopes && r < mt.rows ? P.slopes[mt.h * P.group + (mt.block * R + r) % P.group] * kLog2e : 0.f;
                    tok[g] = mt.tok0 + (r < mt.left0 ? 0 : 1 + (r - mt.left0) / P.group);
                }
            }
            {   // scores, in units of log 2; -infinity where the row does not see the key
                float4 kk[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) kk[i] = *reinterpret_cast<const float4*>(k + chunk(key, i * C::PARTS + part));
                const int j = mt.j0 + key;
                const bool ok = (okm[key >> 5] >> (key & 31)) & 1;
#pragma unroll
                for (int g = 0; g < GS; ++g) {
                    if (g * G >= mt.rows) break;
                    float y[G];
#pragma unroll
                    for (int r = 0; r < G; ++r) {
                        float x[4];   // four short chains
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 a = *reinterpret_cast<const float4*>(q + (g * G + r) * D + (i * C::PARTS + part) * 4);
                            x[i] = a.x * kk[i].x + a.y * kk[i].y + a.z * kk[i].z + a.w * kk[i].w;
                        }
                        y[r] = (x[0] + x[1]) + (x[2] + x[3]);
                    }
                    // lanes that differ in a bit exchange the halves of their rows, then sum up what is left
                    int o = 1;
#pragma unroll
                    for (int n = G; n > 1; n >>= 1, o <<= 1) {
                        const bool odd = part & o;
#pragma unroll
                        for (int r = 0; r < n / 2; ++r) {
                            const float keep = odd ? y[2 * r + 1] : y[2 * r], give = odd ? y[2 * r] : y[2 * r + 1];
                            y[r] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                        }
                    }
#pragma unroll
                    for (; o < C::PARTS; o <<= 1) y[0] += __shfl_xor_sync(0xffffffffu, y[0], o);
                    if (part < G) {
                        const int pos = mt.pos0 + tok[g];
                        float z = y[0] * P.scale;
                        if (P.softcap > 0.f) z = P.softcap * tanhf(z / P.softcap);
                        z = z * kLog2e + slope[g] * (float)(j - pos);
                        if (!ok || (edge && (j > pos || j < first_key(P, mt.start, pos)))) z = -INFINITY;
                        sc[(g * G + mine) * TOK + key] = z;
                    }
                }
            }
            if (bar_any(1, bad || aborted(), NT)) break;
            float f[R];
#pragma unroll
            for (int g = 0; g < GS; ++g) {
                if (g * G >= mt.rows) break;
#pragma unroll
                for (int r = g * G; r < g * G + G; ++r) {
                    float x[TOK / 32], top = -INFINITY;
#pragma unroll
                    for (int i = 0; i < TOK / 32; ++i) {
                        x[i] = sc[r * TOK + 32 * i + lane];
                        top = fmaxf(top, x[i]);
                    }
                    top = fmaxf(m[r], warp_max(top));
                    f[r] = m[r] == -INFINITY ? 0.f : ex2(m[r] - top);
                    const float ms = top == -INFINITY ? 0.f : top;
                    m[r] = top;
                    l[r] *= f[r];
#pragma unroll
                    for (int i = 0; i < TOK / 32; ++i) {
                        const float p = ex2(x[i] - ms);
                        l[r] += p;
                        pw[r * TOK + 32 * i + lane] = x[i] == -INFINITY ? -0.f : p;   // -0: takes nothing of the value
                    }
                }
            }
            __syncwarp();
            {
                float vv[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) vv[i] = *reinterpret_cast<const float*>(v + chunk(kg * 16 + i, d >> 2) + (d & 3) * 4);
                const auto values = [&](auto some) {   // some: of rows that may not see a key
#pragma unroll
                    for (int g = 0; g < GS; ++g) {
                        if (g * G >= mt.rows) break;
#pragma unroll
                        for (int r = g * G; r < g * G + G; ++r) {
                            float a[4] = {acc[r] * f[r], 0.f, 0.f, 0.f};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float4 p = *reinterpret_cast<const float4*>(pw + r * TOK + kg * 16 + 4 * i);
                                const float pp[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    // a row that does not see the key takes nothing of its value, be it NaN
                                    const float with = fmaf(pp[e], vv[4 * i + e], a[i]);
                                    a[i] = decltype(some)::value && __float_as_uint(pp[e]) == 0x80000000u ? a[i] : with;
                                }
                            }
                            acc[r] = (a[0] + a[1]) + (a[2] + a[3]);
                        }
                    }
                };
                if (edge) values(std::true_type());
                else values(std::false_type());
            }
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(sb + C::EMPTY + 8 * (t % C::STG));
            if (mt.flags & kLast) {
                float* red = reinterpret_cast<float*>(sm + C::RED);
#pragma unroll
                for (int g = 0; g < C::GROUPS; ++g) {   // the groups add up their keys in turn
                    if (kg == g) {
#pragma unroll
                        for (int r = 0; r < R; ++r) red[r * D + d] = g == 0 ? acc[r] : red[r * D + d] + acc[r];
                    }
                    bar_all(1, NT);
                }
                // a warp writes a row, and knows its statistics itself
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (r >= mt.rows || w != r) continue;
                    float sum = l[r];
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (mt.part < 0) {
                        const int ir = mt.block * R + r, tok = ir / P.group;
                        const int64_t at = (mt.t0 + tok) * P.Hq + mt.h * P.group + (ir - tok * P.group);
                        const float inv = sum == 0.f ? 0.f : 1.f / sum;
                        for (int c = lane; c < D; c += 32) static_cast<float*>(P.out)[at * D + c] = red[r * D + c] * inv;
                        if (P.lse && lane == 0) P.lse[at] = sum == 0.f ? -INFINITY : m[r] * kLn2 + logf(sum);
                    } else {
                        float* to = P.partial + (int64_t)mt.part * (R * (D + 2));
                        for (int c = lane; c < D; c += 32) to[2 * R + r * D + c] = red[r * D + c];
                        if (lane == 0) { to[r] = m[r]; to[R + r] = sum; }
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
        if (!w.few()) w.template find<C::THREADS>(reinterpret_cast<int64_t*>(sm));
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
