// Softmax attention of the newest tokens over the paged cache.
//
// Per query row, in one pass over its visible keys with the running maximum m, the sum l and
// the weighted values acc (scores in units of log 2, so that e^x is one ex2):
//   m' = max(m, s_j);  l' = l 2^{m - m'} + 2^{s_j - m'};  acc' = acc 2^{m - m'} + 2^{s_j - m'} v_j.
// Two such triples over different keys join the same way, which is how a sequence is split.
//
// Bound by the cache's bytes: a key and a value row serve the G = Hq / Hkv query heads of
// their group and the sequence's new tokens (G x tokens rows), 4 D flops per row for 2 D
// elements.  So the work is cut by bytes alone.  All (sequence, kv head, row block) items are
// laid end to end in tiles of kTok keys, and each of 148 x 8 warps takes one equal stretch of that
// line, whatever the lengths.  A warp streams its tiles through its own ring of shared-memory
// stages with cp.async and never waits for another warp.  Items that lie within one stretch are
// finished there; the others leave a partial triple per stretch, which the join kernel adds up.
#pragma once

#include <cuda_fp16.h>

#include "kda_kv_cache.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace attend {

struct Params {
    const void* q;
    int64_t q_stride;
    const int32_t* cu;
    int32_t num_seqs, Hq, group, max_q, window;
    int64_t total;
    float scale, softcap;
    const float* slopes;
    const int32_t* kv_start;
    void* out;
    float* lse;
    kv::Cache c;
    int64_t* first;    // workspace: num_seqs + 1 places where the sequences' work begins, then
    float* partial;    // kWorkers x 2 partial triples
};

constexpr int kCtas = 148, kWarps = 8, kWorkers = kCtas * kWarps;
constexpr int kGroups = 1024;      // entries of the table of work in shared memory
constexpr int kMinTiles = 2;       // the least that a warp takes
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// The running maximum follows the scores only when they exceed it by 2^8: until then weights are
// up to 2^8, which fp32 sums, bf16 and fp16 weights hold as well, and acc is not rescaled.
constexpr float kSlack = 8.f;

// Keys per tile: 8 KB of keys and values where that is at most 32 keys.
template <int D, typename TC> constexpr int tile_tokens() {
    return 4096 / (D * (int)sizeof(TC)) > 32 ? 32 : 4096 / (D * (int)sizeof(TC));
}
template <int D, typename TC> constexpr int stage_bytes() { return 2 * tile_tokens<D, TC>() * D * (int)sizeof(TC); }
template <int D, typename TC> constexpr int stages() { return 3 * 8192 / stage_bytes<D, TC>(); }
template <int D, typename TC> constexpr int smem_bytes() {
    return kWarps * stages<D, TC>() * stage_bytes<D, TC>() + (kGroups + 1) * 8 + kWarps * 8 + kWarps * stages<D, TC>() * 4;
}

// One sequence's share: its new tokens, the keys [lo, hi) that any of them sees, and its tiles.
struct Seq {
    int64_t t0;
    int nq, pos0;        // new tokens, position of the first
    int start, lo, hi;   // kv_start, first and behind the last visible key
    int tile0, tiles, blocks;
};

template <int TOK>
__device__ __forceinline__ Seq seq_info(const Params& P, int n, int rows) {
    Seq s = {};
    int64_t t1;
    if (!kv::seq_tokens(P.cu, n, P.total, s.t0, t1)) return s;
    const int64_t nq = t1 - s.t0;
    if (nq > P.max_q) {
        kda_set_status(KDA_ERR_BAD_SEQLENS);
        return s;
    }
    s.nq = (int)nq;
    // positions are ints, with room for a tile behind the last one
    const int64_t held = min((int64_t)P.c.max_pages << P.c.page_shift, (int64_t)INT32_MAX - 64);
    const int len = max(P.c.seq_lens[n], 0);
    s.pos0 = len - s.nq;
    s.hi = (int)min((int64_t)len, held);
    s.start = P.kv_start ? max(P.kv_start[n], 0) : 0;
    s.lo = P.window > 0 ? max(s.start, (int)max((int64_t)s.pos0 - P.window + 1, (int64_t)0)) : s.start;
    if (s.nq == 0) return s;
    if (len > held) kda_set_status(KDA_ERR_BAD_PAGE);
    s.blocks = (s.nq * P.group + rows - 1) / rows;
    s.tiles = 1;   // a sequence that sees nothing still has its rows written
    if (s.hi > s.lo) {
        s.tile0 = s.lo / TOK;
        s.tiles = (s.hi - 1) / TOK - s.tile0 + 1;
    }
    return s;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
    // a row that is not to be read is filled with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// d (16 x 8, fp32) += a (16 x 16) b (16 x 8), in bf16 or fp16
template <bool kHalf>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kHalf)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t lo16) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)lo16, __NV_E4M3);
    return (uint32_t)h.x | ((uint32_t)h.y << 16);
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// What a warp knows of the item that it works on.
template <int NR>
struct Rows {
    int pos[NR], lo[NR];   // a row's position and first visible key
    float factor[NR];      // scale of the raw products
    float slope[NR];
};

// Raw product -> score in units of log 2.
__device__ __forceinline__ float score(const Params& P, float x, float factor, float slope, int gap) {
    x *= factor;
    if (P.softcap > 0.f) x = P.softcap * tanhf(x / P.softcap);
    x *= kLog2e;
    if (P.slopes) x += slope * (float)gap;   // the slope carries log2 e
    return x;
}

// A warp's position in its ring of stages, and the loads.
template <int D, typename TC>
struct Loader {
    static constexpr int TOK = tile_tokens<D, TC>(), STG = stages<D, TC>(), BYTES = stage_bytes<D, TC>();
    static constexpr int ROWB = D * (int)sizeof(TC), CPR = ROWB / 16, ITER = TOK * CPR / 32;
    static constexpr int SW = CPR < 8 ? CPR - 1 : 7;

    const Params& P;
    uint32_t smem;
    uint32_t* okm;
    const char *kb, *vb;
    const int32_t* table;
    int lane, lo, hi, tile0, ntiles, page;   // page: of this lane's token in the tile that is issued next

    __device__ __forceinline__ void fetch(int i) {
        const int j = (tile0 + i) * TOK + lane;
        page = -1;
        if (i < ntiles && lane < TOK && j >= lo && j < hi) page = __ldg(table + (j >> P.c.page_shift));
    }
    __device__ __forceinline__ void begin(const Seq& s, int n, int h, int first_tile, int tiles) {
        const int64_t off = h * P.c.head_stride;
        kb = static_cast<const char*>(P.c.k) + off * (int64_t)sizeof(TC);
        vb = static_cast<const char*>(P.c.v) + off * (int64_t)sizeof(TC);
        table = P.c.table + n * P.c.table_stride;
        lo = s.lo;
        hi = s.hi;
        tile0 = s.tile0 + first_tile;
        ntiles = tiles;
        fetch(0);
    }
    // Starts the loads of tile i and looks up the pages of the next one.
    __device__ __forceinline__ void issue(int i) {
        if (i < ntiles) {
            const int j = (tile0 + i) * TOK + lane;
            const bool wanted = lane < TOK && j >= lo && j < hi;
            const bool ok = wanted && page >= 0 && page < P.c.num_pages;
            if (wanted && !ok) kda_set_status(KDA_ERR_BAD_PAGE);
            const uint32_t m = __ballot_sync(0xffffffffu, ok);
            const int64_t off = ok ? (page * P.c.page_stride + (j & ((1 << P.c.page_shift) - 1)) * P.c.row_stride) *
                                         (int64_t)sizeof(TC)
                                   : 0;
            const int st = i % STG;
            if (lane == 0) okm[st] = m;
            const uint32_t dst = smem + st * BYTES;
#pragma unroll
            for (int it = 0; it < ITER; ++it) {
                const int idx = lane + 32 * it, r = idx / CPR, ch = idx % CPR;
                const int64_t o = __shfl_sync(0xffffffffu, off, r) + ch * 16;
                const bool rok = (m >> r) & 1;
                const uint32_t d = dst + r * ROWB + ((ch ^ (r & SW)) << 4);
                cp_async16(d, rok ? kb + o : static_cast<const char*>(P.q), rok);
                cp_async16(d + TOK * ROWB, rok ? vb + o : static_cast<const char*>(P.q), rok);
            }
            fetch(i + 1);
        }
        cp_async_commit();
    }
};

// bf16 queries over a bf16 or e4m3 cache: mma.sync tiles of 16 x MT query rows (lane / 4 and
// + 8 of each block) against TOK keys.  e4m3 keys and values are exact in fp16, so that cache
// multiplies in fp16: weights round to 2^-11, and each query row is scaled by a power of two to a
// largest element in [1, 2), which loses nothing that an fp32 sum of its products would hold.
template <int D, typename TC, int MT>
struct MmaEngine {
    static constexpr bool F8 = sizeof(TC) == 1;
    static constexpr int TOK = tile_tokens<D, TC>(), NT = TOK / 8, KS = D / 16, ROWS = 16 * MT, NR = 2 * MT;
    static constexpr int ROWB = D * (int)sizeof(TC), SW = ROWB / 16 < 8 ? ROWB / 16 - 1 : 7;
    typedef __nv_bfloat16 T;

    uint32_t q[MT][KS][4];
    float acc[MT][D / 8][4], m[NR], l[NR];
    Rows<NR> row;
    int lane;

    // row index within the block of this lane's i-th row
    __device__ __forceinline__ int local(int i) const { return 16 * (i >> 1) + (lane >> 2) + 8 * (i & 1); }

    __device__ __forceinline__ void begin(const Params& P, const Seq& s, int h, int block) {
        const float ks = F8 && P.c.k_scale ? P.c.k_scale[h] : 1.f;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int r = block * ROWS + local(i), tok = r / P.group, g = r - tok * P.group;
            const bool ok = tok < s.nq;
            row.pos[i] = s.pos0 + tok;
            row.lo[i] = P.window > 0 ? max(s.start, (int)max((int64_t)row.pos[i] - P.window + 1, (int64_t)0)) : s.start;
            row.slope[i] = P.slopes && ok ? P.slopes[h * P.group + g] * kLog2e : 0.f;
            m[i] = -INFINITY;
            l[i] = 0.f;
            const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(P.q) + (s.t0 + (ok ? tok : 0)) * P.q_stride +
                                       (h * P.group + g) * D;
            const int c = lane & 3;
            float f = P.scale * ks;
            if constexpr (!F8) {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    q[i >> 1][k][i & 1] = ok ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * c) : 0u;
                    q[i >> 1][k][2 + (i & 1)] = ok ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * c + 8) : 0u;
                }
            } else {
                uint2 raw[KS];
                float top = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    raw[k] = ok ? *reinterpret_cast<const uint2*>(src + 16 * k + 4 * c) : make_uint2(0u, 0u);
                    top = fmaxf(top, fmaxf(fmaxf(fabsf(__uint_as_float(raw[k].x << 16)), fabsf(__uint_as_float(raw[k].x & 0xffff0000u))),
                                           fmaxf(fabsf(__uint_as_float(raw[k].y << 16)), fabsf(__uint_as_float(raw[k].y & 0xffff0000u)))));
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = (int)((__float_as_uint(top) >> 23) & 255u);
                const int x = e == 0 || e == 255 ? 0 : e - 127;   // zeros, and infinities, stay as they are
                const float down = scalbnf(1.f, -x);
                f = scalbnf(f, x);
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    q[i >> 1][k][i & 1] = pack_half2(__uint_as_float(raw[k].x << 16) * down, __uint_as_float(raw[k].x & 0xffff0000u) * down);
                    q[i >> 1][k][2 + (i & 1)] = pack_half2(__uint_as_float(raw[k].y << 16) * down, __uint_as_float(raw[k].y & 0xffff0000u) * down);
                }
            }
            row.factor[i] = f;
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int d = 0; d < D / 8; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[t][d][e] = 0.f;
    }

    // One tile: keys j0 .. j0 + TOK - 1 at smem, their values behind them.  `ok`: rows that were
    // read; [all_lo, all_hi]: keys that every row sees.
    __device__ __forceinline__ void tile(const Params& P, uint32_t smem, int j0, uint32_t ok, int all_lo, int all_hi) {
        const int c = lane & 3, mi = lane >> 3, mr = lane & 7;
        float s[MT][NT][4];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[t][n][e] = 0.f;
        if constexpr (!F8) {
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    uint32_t b[4];   // channels 16 k .. + 7 and + 8 .. 15 of keys 8 n .. + 7, then of the next 8
                    const int r = 8 * n + mr + 8 * (mi >> 1), ch = 2 * k + (mi & 1);
                    ldsm4(b, smem + r * ROWB + ((ch ^ (r & SW)) << 4));
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        mma<false>(s[t][n], q[t][k], b[0], b[1]);
                        mma<false>(s[t][n + 1], q[t][k], b[2], b[3]);
                    }
                }
        } else {
            // a 16-byte chunk holds the 16 channels of one product step: lane c gets channels 4 c .. + 3,
            // which stand for the fragment's k = 2 c, 2 c + 1, 2 c + 8, 2 c + 9 on both sides
#pragma unroll
            for (int k = 0; k < KS; k += 2)
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    uint32_t b[4];
                    const int r = 8 * n + mr + 8 * (mi >> 1), ch = k + (mi & 1);
                    ldsm4(b, smem + r * ROWB + ((ch ^ (r & SW)) << 4));
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t b0 = e4m3x2_to_half2(b[x] & 0xffffu), b1 = e4m3x2_to_half2(b[x] >> 16);
#pragma unroll
                        for (int t = 0; t < MT; ++t) mma<true>(s[t][n + (x >> 1)], q[t][k + (x & 1)], b0, b1);
                    }
                }
        }
        constexpr uint32_t FULL = TOK == 32 ? 0xffffffffu : (1u << TOK) - 1u;
        const bool inside = ok == FULL && j0 >= all_lo && j0 + TOK - 1 <= all_hi;
        // keys that all rows see go through the value product; keys that only some see (NaN times a weight
        // of zero would reach the others) are added row by row below
        uint32_t all = FULL;
        if (!inside) {
            const int a = max(all_lo - j0, 0), b = min(all_hi - j0, TOK - 1);   // bits a .. b
            all = ok & (a <= b ? (0xffffffffu >> (31 - b)) & (0xffffffffu << a) : 0u);
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int t = i >> 1, e = 2 * (i & 1);
            float top = -INFINITY;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int j = 8 * n + 2 * c + x;
                    float v = score(P, s[t][n][e + x], row.factor[i], row.slope[i], j0 + j - row.pos[i]);
                    if (!inside && !(((ok >> j) & 1) && j0 + j <= row.pos[i] && j0 + j >= row.lo[i])) v = -INFINITY;
                    s[t][n][e + x] = v;
                    top = fmaxf(top, v);
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const bool up = top > m[i] + kSlack;   // also the first visible key: m = -inf
            if (__any_sync(0xffffffffu, up)) {
                const float f = up ? ex2(m[i] - top) : 1.f;
                if (up) m[i] = top;
                l[i] *= f;
#pragma unroll
                for (int d = 0; d < D / 8; ++d) { acc[t][d][e] *= f; acc[t][d][e + 1] *= f; }
            }
            const float ms = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float p = ex2(s[t][n][e + x] - ms);
                    s[t][n][e + x] = p;
                    l[i] += p;
                }
        }
        const uint32_t vs = smem + TOK * ROWB;
#pragma unroll
        for (int k = 0; k < NT / 2; ++k) {   // 16 keys
            uint32_t a[MT][4];
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float lo = s[t][2 * k + (e >> 1)][2 * (e & 1)], hi = s[t][2 * k + (e >> 1)][2 * (e & 1) + 1];
                    a[t][e] = F8 ? pack_half2(lo, hi) : sm100::pack_bf16x2(lo, hi);
                }
            // values that do not go through the product are cleared: two keys a register
            const uint32_t bits = all >> (16 * k + 2 * c);
            const uint32_t keep0 = (bits & 1 ? 0xffffu : 0u) | (bits & 2 ? 0xffff0000u : 0u);
            const uint32_t keep1 = (bits & 256 ? 0xffffu : 0u) | (bits & 512 ? 0xffff0000u : 0u);
#pragma unroll
            for (int d = 0; d < ROWB / 16; d += 2) {
                uint32_t b[4];   // keys 0 .. 7 and 8 .. 15 of chunk d, then of chunk d + 1
                const int r = 16 * k + mr + 8 * (mi & 1), ch = d + (mi >> 1);
                ldsm4_t(b, vs + r * ROWB + ((ch ^ (r & SW)) << 4));
                if constexpr (!F8) {
                    if (!inside) { b[0] &= keep0; b[1] &= keep1; b[2] &= keep0; b[3] &= keep1; }
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        mma<false>(acc[t][d], a[t], b[0], b[1]);
                        mma<false>(acc[t][d + 1], a[t], b[2], b[3]);
                    }
                } else {
                    // a register holds channels 2 g, 2 g + 1 (g = lane / 4) of two keys: the even channels
                    // make one fragment, the odd ones another
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t y0 = __byte_perm(b[2 * x], 0, 0x3120), y1 = __byte_perm(b[2 * x + 1], 0, 0x3120);
                        uint32_t e0 = e4m3x2_to_half2(y0 & 0xffffu), o0 = e4m3x2_to_half2(y0 >> 16);
                        uint32_t e1 = e4m3x2_to_half2(y1 & 0xffffu), o1 = e4m3x2_to_half2(y1 >> 16);
                        if (!inside) { e0 &= keep0; o0 &= keep0; e1 &= keep1; o1 &= keep1; }
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            mma<true>(acc[t][2 * (d + x)], a[t], e0, e1);
                            mma<true>(acc[t][2 * (d + x) + 1], a[t], o0, o1);
                        }
                    }
                }
            }
        }
        if (!inside) {
            uint32_t some = ok & ~all;
            while (some) {
                const int j = __ffs(some) - 1;
                some &= some - 1;
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const int t = i >> 1, e = 2 * (i & 1);
                    float p = 0.f;   // the weight of key j, held by lane (j / 2) % 4 of this row's four
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        if (n == j >> 3) p = j & 1 ? s[t][n][e + 1] : s[t][n][e];
                    p = __shfl_sync(0xffffffffu, p, (lane & ~3) | ((j >> 1) & 3));
                    if (j0 + j > row.pos[i] || j0 + j < row.lo[i]) continue;
#pragma unroll
                    for (int d = 0; d < D / 8; ++d)
#pragma unroll
                        for (int x = 0; x < 2; ++x) acc[t][d][e + x] += p * value(vs, j, channel(d, x));
                }
            }
        }
    }
    // the channel of acc[..][d][x] and [x + 2]
    __device__ __forceinline__ int channel(int d, int x) const {
        const int c = lane & 3;
        return F8 ? 16 * (d >> 1) + 4 * c + 2 * x + (d & 1) : 8 * d + 2 * c + x;
    }
    static __device__ __forceinline__ float value(uint32_t vs, int j, int ch) {
        const uint32_t a = vs + j * ROWB + ((((ch * (int)sizeof(TC)) >> 4) ^ (j & SW)) << 4) + ((ch * (int)sizeof(TC)) & 15);
        if constexpr (F8) {
            uint32_t b;
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(b) : "r"(a));
            return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3)));
        } else {
            uint16_t b;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b) : "r"(a));
            return __uint_as_float((uint32_t)b << 16);
        }
    }

    __device__ __forceinline__ void sums() {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        }
    }
    __device__ __forceinline__ void finish(const Params& P, const Seq& s, int h, int block) {
        sums();
        const float vs = F8 && P.c.v_scale ? P.c.v_scale[h] : 1.f;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int r = block * ROWS + local(i), tok = r / P.group, g = r - tok * P.group, t = i >> 1, e = 2 * (i & 1);
            if (tok >= s.nq) continue;
            const int64_t at = (s.t0 + tok) * P.Hq + h * P.group + g;
            const float f = l[i] == 0.f ? 0.f : vs / l[i];
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(P.out) + at * D;
            if constexpr (!F8) {
#pragma unroll
                for (int d = 0; d < D / 8; ++d)
                    *reinterpret_cast<uint32_t*>(dst + channel(d, 0)) = sm100::pack_bf16x2(acc[t][d][e] * f, acc[t][d][e + 1] * f);
            } else {
#pragma unroll
                for (int d = 0; d < D / 8; d += 2)
                    *reinterpret_cast<uint2*>(dst + channel(d, 0)) =
                        make_uint2(sm100::pack_bf16x2(acc[t][d][e] * f, acc[t][d + 1][e] * f),
                                   sm100::pack_bf16x2(acc[t][d][e + 1] * f, acc[t][d + 1][e + 1] * f));
            }
            if (P.lse && (lane & 3) == 0) P.lse[at] = l[i] == 0.f ? -INFINITY : m[i] * kLn2 + logf(l[i]);
        }
    }
    __device__ __forceinline__ void leave(const Params& P, const Seq& s, int h, int block, float* to) {
        sums();
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int lr = local(i), r = block * ROWS + lr, t = i >> 1, e = 2 * (i & 1);
            if (r >= s.nq * P.group) continue;
            if ((lane & 3) == 0) { to[lr] = m[i]; to[ROWS + lr] = l[i]; }
            float* dst = to + 2 * ROWS + lr * D;
            if constexpr (!F8) {
#pragma unroll
                for (int d = 0; d < D / 8; ++d)
                    *reinterpret_cast<float2*>(dst + channel(d, 0)) = make_float2(acc[t][d][e], acc[t][d][e + 1]);
            } else {
#pragma unroll
                for (int d = 0; d < D / 8; d += 2)
                    *reinterpret_cast<float4*>(dst + channel(d, 0)) =
                        make_float4(acc[t][d][e], acc[t][d + 1][e], acc[t][d][e + 1], acc[t][d + 1][e + 1]);
            }
        }
    }
};

// fp32: no tensor-core type holds the products, so CUDA cores compute them.  A lane owns D / 32
// channels of every row; the score of a key is a sum over the warp.
template <int D, int R>
struct SimtEngine {
    static constexpr int TOK = tile_tokens<D, float>(), E = D / 32, ROWS = R, ROWB = 4 * D, SW = 7;
    typedef float T;

    float q[R][E], acc[R][E], m[R], l[R];
    Rows<R> row;
    int lane, rows;

    static __device__ __forceinline__ void load(float (&x)[E], uint32_t base, int j, int lane) {
        const int b = lane * E * 4;   // this lane's bytes of the row
        const uint32_t a = base + j * ROWB + (((b >> 4) ^ (j & SW)) << 4) + (b & 15);
        if constexpr (E == 4)
            asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(a) : "memory");
        else
            asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(x[0]), "=f"(x[1]) : "r"(a) : "memory");
    }
    __device__ __forceinline__ void begin(const Params& P, const Seq& s, int h, int block) {
        rows = min(R, s.nq * P.group - block * R);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = block * R + i, tok = r / P.group, g = r - tok * P.group;
            const bool ok = i < rows;
            row.pos[i] = s.pos0 + tok;
            row.lo[i] = P.window > 0 ? max(s.start, (int)max((int64_t)row.pos[i] - P.window + 1, (int64_t)0)) : s.start;
            row.slope[i] = P.slopes && ok ? P.slopes[h * P.group + g] * kLog2e : 0.f;
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                q[i][e] = ok ? static_cast<const float*>(P.q)[(s.t0 + tok) * P.q_stride + (h * P.group + g) * D + lane * E + e] : 0.f;
                acc[i][e] = 0.f;
            }
        }
    }
    __device__ __forceinline__ void tile(const Params& P, uint32_t smem, int j0, uint32_t ok, int all_lo, int all_hi) {
        constexpr uint32_t FULL = (1u << TOK) - 1u;
        const bool inside = ok == FULL && j0 >= all_lo && j0 + TOK - 1 <= all_hi;
        float s[R][TOK];
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
            float k[E];
            load(k, smem, j, lane);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float x = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) x += q[i][e] * k[e];
                s[i][j] = x;
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (i >= rows) break;
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < TOK; ++j) {
                float x = s[i][j];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                x = score(P, x, P.scale, row.slope[i], j0 + j - row.pos[i]);
                if (!inside && !(((ok >> j) & 1) && j0 + j <= row.pos[i] && j0 + j >= row.lo[i])) x = -INFINITY;
                s[i][j] = x;
                top = fmaxf(top, x);
            }
            if (top > m[i] + kSlack) {
                const float f = ex2(m[i] - top);
                m[i] = top;
                l[i] *= f;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[i][e] *= f;
            }
            const float ms = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
            for (int j = 0; j < TOK; ++j) {
                s[i][j] = ex2(s[i][j] - ms);
                l[i] += s[i][j];
            }
        }
#pragma unroll
        for (int j = 0; j < TOK; ++j) {
            float v[E];
            load(v, smem + TOK * ROWB, j, lane);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (i >= rows) break;
                // a row that does not see key j takes nothing of its value, be it NaN
                if (inside || (((ok >> j) & 1) && j0 + j <= row.pos[i] && j0 + j >= row.lo[i])) {
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[i][e] += s[i][j] * v[e];
                }
            }
        }
    }
    __device__ __forceinline__ void finish(const Params& P, const Seq& s, int h, int block) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (i >= rows) break;
            const int r = block * R + i, tok = r / P.group, g = r - tok * P.group;
            const int64_t at = (s.t0 + tok) * P.Hq + h * P.group + g;
            const float f = l[i] == 0.f ? 0.f : 1.f / l[i];
            float* dst = static_cast<float*>(P.out) + at * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; ++e) dst[e] = acc[i][e] * f;
            if (P.lse && lane == 0) P.lse[at] = l[i] == 0.f ? -INFINITY : m[i] * kLn2 + logf(l[i]);
        }
    }
    __device__ __forceinline__ void leave(const Params&, const Seq&, int, int, float* to) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (i >= rows) break;
            if (lane == 0) { to[i] = m[i]; to[ROWS + i] = l[i]; }
#pragma unroll
            for (int e = 0; e < E; ++e) to[2 * ROWS + i * D + lane * E + e] = acc[i][e];
        }
    }
};

// Tiles of a warp's stretch when `total` tiles are shared out.
__device__ __forceinline__ int64_t stretch(int64_t total) {
    return max((total + kWorkers - 1) / kWorkers, (int64_t)kMinTiles);
}

template <int D, typename TC, typename Engine>
__global__ void __launch_bounds__(32 * kWarps, 1) attend_kernel(const __grid_constant__ Params P) {
    typedef Loader<D, TC> L;
    constexpr int TOK = L::TOK, ROWS = Engine::ROWS;
    extern __shared__ __align__(128) uint8_t smem[];
    int64_t* work = reinterpret_cast<int64_t*>(smem + kWarps * L::STG * L::BYTES);   // kGroups + 1
    int64_t* wsum = work + kGroups + 1;                                              // kWarps
    uint32_t* okm = reinterpret_cast<uint32_t*>(wsum + kWarps);                      // kWarps x STG
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int N = P.num_seqs, per_group = (N + kGroups - 1) / kGroups, groups = (N + per_group - 1) / per_group;

    // where each group of sequences begins on the line of tiles
    constexpr int SLICE = kGroups / (32 * kWarps);
    const int slice = (groups + 32 * kWarps - 1) / (32 * kWarps);   // groups of one thread, up to SLICE
    int64_t mine[SLICE], sum = 0;
#pragma unroll
    for (int i = 0; i < SLICE; ++i) {
        const int gr = tid * slice + i;
        mine[i] = 0;
        if (i < slice && gr < groups)
            for (int n = gr * per_group; n < min(N, (gr + 1) * per_group); ++n) {
                const Seq s = seq_info<TOK>(P, n, ROWS);
                mine[i] += (int64_t)s.tiles * s.blocks * P.c.Hkv;
            }
        sum += mine[i];
    }
    int64_t before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += x;
    }
    if (lane == 31) wsum[w] = before;
    __syncthreads();
    before -= sum;
    for (int x = 0; x < w; ++x) before += wsum[x];
#pragma unroll
    for (int i = 0; i < SLICE; ++i) {
        const int gr = tid * slice + i;
        if (i < slice && gr <= groups) work[gr] = before;
        if (i < slice && blockIdx.x == 0 && gr < groups) {   // for the join
            int64_t at = before;
            for (int n = gr * per_group; n < min(N, (gr + 1) * per_group); ++n) {
                P.first[n] = at;
                if (per_group > 1) {
                    const Seq s = seq_info<TOK>(P, n, ROWS);
                    at += (int64_t)s.tiles * s.blocks * P.c.Hkv;
                }
            }
        }
        before += mine[i];
    }
    if (tid == 32 * kWarps - 1) {
        if (groups == 32 * kWarps * slice) work[groups] = before;
        if (blockIdx.x == 0) P.first[N] = before;
    }
    __syncthreads();
    kda_grid_launch_next();

    const int64_t total = work[groups], per = stretch(total);
    const int64_t worker = (int64_t)blockIdx.x * kWarps + w;
    int64_t at = worker * per;
    const int64_t begin = at, end = min(at + per, total);
    if (at >= end) return;
    int gr = 0;   // the group that holds `at`: the last with work[gr] <= at
    for (int lo = 0, hi = groups - 1; lo <= hi;) {
        const int mid = (lo + hi) >> 1;
        if (work[mid] <= at) { gr = mid; lo = mid + 1; } else hi = mid - 1;
    }
    int n = gr * per_group;
    int64_t base = work[gr];   // where sequence n begins
    Seq s = seq_info<TOK>(P, n, ROWS);
    L load{P, sm100::smem_u32(smem) + w * L::STG * L::BYTES, okm + w * L::STG};
    load.lane = lane;
    Engine e;
    e.lane = lane;
    while (at < end) {
        int64_t items = (int64_t)s.blocks * P.c.Hkv;
        while (at - base >= items * s.tiles) {
            base += items * s.tiles;
            ++n;
            s = seq_info<TOK>(P, n, ROWS);
            items = (int64_t)s.blocks * P.c.Hkv;
        }
        const int item = (int)((at - base) / s.tiles), h = item / s.blocks, block = item - h * s.blocks;
        const int64_t a = base + (int64_t)item * s.tiles, b = a + s.tiles;   // the item's tiles
        const int first = (int)(at - a), tiles = (int)(min(b, end) - at);
        load.begin(s, n, h, first, tiles);
        e.begin(P, s, h, block);
        const int last = s.pos0 + s.nq - 1;
        const int all_lo = P.window > 0 ? max(s.start, (int)max((int64_t)last - P.window + 1, (int64_t)0)) : s.start;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < L::STG - 1; ++i) load.issue(i);
        for (int i = 0; i < tiles; ++i) {
            cp_async_wait<L::STG - 2>();
            __syncwarp();   // the tile is there for all lanes, and the stage before it is used up
            load.issue(i + L::STG - 1);
            const int st = i % L::STG;
            e.tile(P, load.smem + st * L::BYTES, (load.tile0 + i) * TOK, load.okm[st], all_lo, s.pos0);
        }
        cp_async_wait<0>();
        if (at == a && at + tiles == b) {
            e.finish(P, s, h, block);
        } else {
            // a stretch has at most one item that began before it and one that goes on behind it
            e.leave(P, s, h, block, P.partial + (2 * worker + (a < begin ? 0 : 1)) * (int64_t)(ROWS * (D + 2)));
        }
        at += tiles;
    }
}

constexpr int kJoinWarps = 4;

// Adds up the partial triples of the items that lie across stretches: one CTA per output row.
template <int D, typename T, typename TC, int ROWS>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ Params P) {
    constexpr int TOK = tile_tokens<D, TC>(), E = D / 32;
    __shared__ float sm[kJoinWarps], sl[kJoinWarps], sacc[kJoinWarps][D];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int n = blockIdx.x / P.max_q, tok = blockIdx.x % P.max_q, hq = blockIdx.y;
    const Seq s = seq_info<TOK>(P, n, ROWS);
    kda_grid_wait();
    if (tok >= s.nq || s.tiles == 0) return;
    const int h = hq / P.group, r = tok * P.group + (hq - h * P.group), block = r / ROWS, lr = r - block * ROWS;
    const int64_t a = P.first[n] + ((int64_t)h * s.blocks + block) * s.tiles, b = a + s.tiles;
    const int64_t per = stretch(P.first[P.num_seqs]), w0 = a / per, w1 = (b - 1) / per;
    if (w0 == w1) return;   // finished where it was computed
    float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int64_t x = w0 + w; x <= w1; x += kJoinWarps) {
        const float* from = P.partial + (2 * x + (a < x * per ? 0 : 1)) * (int64_t)(ROWS * (D + 2));
        const float m2 = from[lr], l2 = from[ROWS + lr];
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = from[2 * ROWS + lr * D + lane * E + e];
        const float mt = fmaxf(m, m2);
        const float f1 = m == -INFINITY ? 0.f : ex2(m - mt), f2 = m2 == -INFINITY ? 0.f : ex2(m2 - mt);
        l = l * f1 + l2 * f2;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * f1 + v[e] * f2;
        m = mt;
    }
    if (lane == 0) { sm[w] = m; sl[w] = l; }
#pragma unroll
    for (int e = 0; e < E; ++e) sacc[w][lane * E + e] = acc[e];
    __syncthreads();
    float mt = -INFINITY, lt = 0.f, f[kJoinWarps];
#pragma unroll
    for (int x = 0; x < kJoinWarps; ++x) mt = fmaxf(mt, sm[x]);
#pragma unroll
    for (int x = 0; x < kJoinWarps; ++x) {
        f[x] = sm[x] == -INFINITY ? 0.f : ex2(sm[x] - mt);
        lt += sl[x] * f[x];
    }
    const int64_t at = (s.t0 + tok) * P.Hq + hq;
    const float vs = (sizeof(TC) == 1 && P.c.v_scale ? P.c.v_scale[h] : 1.f);
    const float inv = lt == 0.f ? 0.f : vs / lt;
    for (int d = threadIdx.x; d < D; d += 32 * kJoinWarps) {
        float o = 0.f;
#pragma unroll
        for (int x = 0; x < kJoinWarps; ++x) o += sacc[x][d] * f[x];
        static_cast<T*>(P.out)[at * D + d] = from_f32<T>(o * inv);
    }
    if (threadIdx.x == 0 && P.lse) P.lse[at] = lt == 0.f ? -INFINITY : mt * kLn2 + logf(lt);
}

// Query rows that one warp takes at a time.
inline int block_rows(bool f32, int rows) { return f32 ? (rows <= 2 ? 2 : 8) : (rows <= 16 ? 16 : 32); }

inline size_t header_bytes(int num_seqs) { return (((size_t)num_seqs + 1) * 8 + 255) & ~(size_t)255; }
inline size_t workspace_bytes(int num_seqs, int D, int rows) {
    return header_bytes(num_seqs) + (size_t)kWorkers * 2 * block_rows(false, rows) * (D + 2) * 4;
}

template <int D, typename T, typename TC, typename Engine>
cudaError_t launch_engine(const Params& P, cudaStream_t stream) {
    auto kern = attend_kernel<D, TC, Engine>;
    constexpr int bytes = smem_bytes<D, TC>();
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err != cudaSuccess) return err;
    kern<<<kCtas, 32 * kWarps, bytes, stream>>>(P);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)P.num_seqs * (unsigned)P.max_q, (unsigned)P.Hq);
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<D, T, TC, Engine::ROWS>, P);
}

template <int D, typename T, typename TC>
cudaError_t launch(const Params& P, cudaStream_t stream) {
    const int rows = block_rows(sizeof(T) == 4, P.group * P.max_q);
    if constexpr (sizeof(T) == 4)
        return rows == 2 ? launch_engine<D, T, TC, SimtEngine<D, 2>>(P, stream)
                         : launch_engine<D, T, TC, SimtEngine<D, 8>>(P, stream);
    else
        return rows == 16 ? launch_engine<D, T, TC, MmaEngine<D, TC, 1>>(P, stream)
                          : launch_engine<D, T, TC, MmaEngine<D, TC, 2>>(P, stream);
}

}  // namespace attend
}  // namespace kda
