// The paged attention on tcgen05: bf16 queries over a bf16 or e4m3 cache.
//
// A tile is 128 keys.  Both products have the long side as M, so the few query rows (N = 16, 32
// or 64) waste nothing of the tensor pipe's 128 lanes:
//   S^T [keys x N]     = K [keys x D] (K-major, as it lies in the cache) * Q [N x D]
//   O^T [D x N]       += V^T (MN-major, again as it lies in the cache) * P [keys x N]
// Keys are TMEM lanes, so a softmax thread owns one key: it masks, scales and exponentiates the
// rows' scores without a shuffle, keeps its own share of every row's sum, and writes its weights
// as one 16-byte chunk per 8 rows (P MN-major without swizzle, free of bank conflicts).  Only the
// running maximum is shared, and the tile that raises it by more than 2^8 is rare (SLACK).
//
// Warps: 4 for softmax and epilogue (TMEM lanes 32 w ..) for every 8 rows (16 of 64), which share
// nothing but keys and values; then two that fetch tiles, one that issues the products, and
// with an e4m3 cache four that split queries.  S and O are double-buffered in TMEM, so the product
// of the next tile runs during the softmax of this one and the next item starts during the epilogue
// of the last.  Tiles land in the operand images directly: TMA's swizzle is the images'.
//
// bf16: a weight rounded to 8 bits would be the largest error by far (0.0023 of an output's size where the
// rounding of the output alone is 0.0017).  So it goes into the product in two bf16 parts side by side in N,
// 2^-16 of it, whose columns are summed up at an item's end.  With the scores' arithmetic two rows at a time it
// takes about the time that one part took: 185 us for 64 sequences of 512 to 16,384 keys (186), 170 for 32 of
// 8,192 with 16 rows a kv head (171), 180 with 32 (180), 264 to 272 with 64 (262), 112 with one row of 64 channels (107).
//
// e4m3: tcgen05 multiplies 8-bit with 8-bit operands only, and queries or weights rounded to 8 bits
// would lose what the scores need.  So they are split into e4m3 parts that sum up to them, side by
// side in N, which costs nothing while the long operand bounds the product:
//   a query row is scaled by a power of two to a largest element in [2^7, 2^8); q = q1 + q2 / 16
//     holds bf16's 8 bits, down to 2^-22 of the row's largest;
//   a weight is p1 + p2 / 16 + p3 / 256, down to 2^-25 of the row's largest, to 2^-13 of itself: of a weight in [1, 2) p1
//     leaves 2^-4 at most, p2 2^-9 and p3 2^-14, and the first remainder, rounded to fp16 so that the others take
//     half the instructions, is off by 2^-16.  With the weight itself in fp16 (2^-11) drafts took 77 us instead of 79,
//     and an output was off by 0.0002 of its size beside its own rounding, now by 0.00002.
// The products are exact and summed in fp32: 2^-25 of the sum of magnitudes over 128 products.  The
// other way, turning the cache's tiles into fp16 images, took eight warps 1,900 cycles an operand and
// four times the shared-memory traffic: 151 us for 75,800 keys of 8 heads, now 79.
//
// A product with M = 128 takes 124 cycles whatever its type, its operands' order and N up to 48 (measured), 16 of
// them a bf16 tile of 128 channels: 1,980 of the 2,780 cycles in which an SM's share of the memory brings it.  A
// softmax warp's way through a tile takes about 1,900.  So bf16 is bound by memory (6.1 to 6.4 TB/s over long
// sequences), e4m3 by that way, at 2,150 cycles a tile where the memory would need 1,390 (4.3 TB/s).  64 rows take
// 4.0 TB/s over bf16 (two tiles in flight, 16 softmax warps) and 1.7 over e4m3, whose instance has 80 registers a
// thread and spills 92 bytes of stores and 152 to 160 of loads.
#pragma once

#include "kda_kv_decode.cuh"
#include "kda_kv_decode_simt.cuh"

namespace kda {
namespace attend {

template <int D_, typename TC, int N>
struct Tc {
    static constexpr int D = D_;
    static constexpr bool F8 = sizeof(TC) == 1;
    static constexpr int TOK = 128;
    static constexpr int RW = N == 64 ? 16 : 8, SW = 4 * N / RW;              // rows of four softmax warps, softmax warps
    static constexpr int LW = F8 ? 4 : 0;                                     // splitting warps
    static constexpr int THREADS = 32 * (SW + 3 + LW);
    static constexpr int QP = F8 ? 2 : 1, PP = F8 ? 3 : 2;                    // parts of queries and weights
    // The running maximum follows the scores only when they exceed it by SLACK (in units of log 2):
    // until then acc is not rescaled.  Weights are 2^(s - m + BASE): up to 2^8, which fp32 sums and bf16
    // parts hold as well as 1; with e4m3 parts from 2^7 (the smallest parts then lie far below the
    // largest weight) to 2^8.75 (e4m3 ends at 448).
    static constexpr float BASE = F8 ? 7.f : 0.f, SLACK = F8 ? 1.75f : 8.f;
    static constexpr int ROWB = D * (int)sizeof(TC);                   // a cache row
    // an operand image: BLKS blocks of rows of BROWB bytes, swizzled over those
    static constexpr int BROWB = ROWB < 128 ? ROWB : 128, BLKS = ROWB / BROWB, BLOCK = TOK * BROWB, RAW = TOK * ROWB;
    static constexpr int KSTEP = F8 ? 32 : 16;                         // of one tcgen05.mma
    static constexpr uint32_t SWZ = BROWB == 64 ? sm100::kSwizzle64 : sm100::kSwizzle128;
    static constexpr int STAGE = 2 * RAW;
    // queries: D bf16 in blocks of 128-byte rows; split, QP N rows of the cache's form in the same place
    static constexpr bool QSWIZZLED = true;
    static constexpr int QBLKS = D / 64, QROWB = 128, QBLOCK = N * 128, QB = N * D * 2;
    static constexpr int PG = 16 / (F8 ? 1 : 2);                       // rows of a 16-byte chunk of weights
    static constexpr int PB = PP * N * TOK * (F8 ? 1 : 2);
    static constexpr int OB = 2 * (QP + PP) * N <= 512 ? 2 : 1;        // O buffers that Tensor Memory has room for
    static constexpr int COLS = (2 * QP + OB * PP) * N;
    static constexpr int TCOLS = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    // A stage is free when its tile is done; queries need one slot per stage, meta is read a little longer.
    // Where that leaves two stages and two slots would leave three (32 bf16 rows of 128 channels: 180 us instead of 232),
    // queries get two, and wait for the scores of the item before the last (for its tiles to be done, items of one to
    // four tiles took 120 us instead of 110).
    static constexpr int metas(int stg) { return stg + 2; }
    static constexpr int misc(int stg) {
        return metas(stg) * 64 + metas(stg) * 16 + stg * N * 4 + N * 8 + N * 8 + 4 * N * 4 + N * 4 + 8 * (4 * stg + metas(stg) + 13) + 16 + 4 * SW + stg * 4;
    }
    static constexpr int total(int stg, int qs) { return stg * STAGE + qs * QB + PB + misc(stg); }
    static constexpr int most(int stg) { return stg > 2 && total(stg, stg) > kMaxSmem ? most(stg - 1) : stg; }
    static constexpr bool FEWQ = most(6) == 2 && total(3, 2) <= kMaxSmem;
    static_assert(!(FEWQ && F8), "queries are free when the scores are there");
    static constexpr int STG = FEWQ ? 3 : most(6), QS = FEWQ ? 2 : STG, MD = metas(STG);
    static constexpr int BYTES = total(STG, QS);
    static_assert(BYTES <= kMaxSmem, "shared memory of a CTA");
    static_assert((kGroups + 1) * 8 + 32 * 8 <= STG * STAGE, "the table of work lies where the ring comes");
    // offsets
    static constexpr int RING = 0, Q = RING + STG * STAGE, PM = Q + QS * QB, META = PM + PB, OKM = META + MD * 64,
                         QF = OKM + MD * 16, RINFO = QF + QS * N * 4, MROW = RINFO + N * 8, WRED = MROW + N * 8,
                         FROW = WRED + 4 * N * 4, BAR = FROW + N * 4;
    static_assert(META % 16 == 0 && OKM % 16 == 0 && RINFO % 16 == 0 && BAR % 8 == 0, "alignment");
    // barriers
    static constexpr int FULL = BAR, EMPTY = FULL + 8 * STG, QRAW = EMPTY + 8 * STG, QFULL = QRAW + 8 * QS, MFULL = QFULL + 8 * QS,
                         SFULL = MFULL + 8 * MD, SFREE = SFULL + 16, PFULL = SFREE + 16, PVDONE = PFULL + 8, OFREE = PVDONE + 16,
                         FIN = OFREE + 16, LOOKED = FIN + 8, TMEM = LOOKED + 8, ABORT = TMEM + 4, ANY = ABORT + 4, BITS = ANY + 4,
                         QLAST = BITS + 4 * SW;
    static_assert(QLAST + QS * 4 <= BYTES, "misc");
    // byte offset of 16-byte chunk ch of a row of an image
    static __device__ __forceinline__ uint32_t chunk(uint32_t row, uint32_t ch) {
        return BROWB == 64 ? sm100::sw64_off(row, ch) : (ch >> 3) * BLOCK + sm100::sw128_off(row, ch & 7);
    }
};

// Instruction descriptor: bf16 (kind::f16) or e4m3 (kind::f8f6f4) operands, fp32 accumulate.
__host__ __device__ constexpr uint32_t idesc(bool bf16, int M, int N, bool a_mn, bool b_mn) {
    const uint32_t f = bf16 ? 1u : 0u;
    return (1u << 4) | (f << 7) | (f << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a), "l"(b), "r"(id), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}

// true in one lane of the warp, the same each time
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
// Two fp32 operations in one.
__device__ __forceinline__ uint64_t bits2(float2 x) { return (uint64_t)__float_as_uint(x.y) << 32 | __float_as_uint(x.x); }
__device__ __forceinline__ float2 of_bits2(uint64_t x) { return make_float2(__uint_as_float((uint32_t)x), __uint_as_float((uint32_t)(x >> 32))); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return of_bits2(r);
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return of_bits2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return of_bits2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return of_bits2(r);
}
__device__ __forceinline__ void load8(const float* from, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        const float4 u = *reinterpret_cast<const float4*>(from + i);
        x[i] = u.x; x[i + 1] = u.y; x[i + 2] = u.z; x[i + 3] = u.w;
    }
}
// A weight over a bf16 cache is its upper half and the rest, rounded to bf16.  The rest is taken 2^-19 of the weight
// larger, so that it is positive where the weight is (an infinite value times a rest of 0 would be NaN).
constexpr float kAbove1 = 1.f + 1.f / (1 << 19);
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) { return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3); }
__device__ __forceinline__ uint32_t e4m3x2(__half2 x) { return __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3); }
__device__ __forceinline__ __half2 half2_of(uint32_t e4m3x2) { return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)e4m3x2, __NV_E4M3)); }
template <int D, typename TC, int N>
struct TcKernel {
    typedef Tc<D, TC, N> C;
    typedef Walk<C::TOK, N> W;
    static constexpr bool F8 = C::F8;
    static constexpr int TOK = C::TOK;
    // named barriers: 1 .. of the groups of softmax warps, then of the splitting warps
    static constexpr uint32_t kSplitBar = 1 + C::SW / 4;

    const Params& P;
    uint8_t* sm;
    uint32_t sb;

    __device__ __forceinline__ Meta* meta(int t) const { return reinterpret_cast<Meta*>(sm + C::META) + t % C::MD; }
    __device__ __forceinline__ void fail() const {
        kda_set_status(KDA_ERR_TIMEOUT);
        *reinterpret_cast<volatile uint32_t*>(sm + C::ABORT) = 1;
    }
    __device__ __forceinline__ bool aborted() const { return *reinterpret_cast<volatile uint32_t*>(sm + C::ABORT) != 0; }

    // ------------------------------------------------------------------ fetching
    __device__ __forceinline__ void put(Fetch<C, N>& f, const W& w, int t) {
        f.put(w, sb + C::RING + (t % C::STG) * C::STAGE, sb + C::Q + (w.item % C::QS) * C::QB, sb + C::FULL + 8 * (t % C::STG),
              F8 ? sb + C::QRAW + 8 * (w.item % C::QS) : sb + C::FULL + 8 * (t % C::STG), sb + C::MFULL + 8 * (t % C::MD), meta(t),
              reinterpret_cast<uint32_t*>(sm + C::OKM + (t % C::MD) * 16), reinterpret_cast<uint32_t*>(sm + C::QLAST) + w.item % C::QS);
    }
    __device__ __forceinline__ void fetcher(Fetch<C, N>& f, W& w) {
        int puts = 0;
        const bool ok = f.run(
            w,
            [&](int t) {
                if (aborted() || (t >= C::STG && !wait_warp(sb + C::EMPTY + 8 * (t % C::STG), (t / C::STG - 1) & 1))) return false;
                // Queries into the slot of the item before the last: the scores of its tiles, up to t - 2 at most, are
                // there.  (Those of t - 4 are, by the wait above, and those of t cannot be: the phase is meant.)
                return !C::FEWQ || f.keys || w.i > 0 || w.item < C::QS || wait_warp(sb + C::SFULL + 8 * (t & 1), ((t - 2) >> 1) & 1);
            },
            [&](int t) {
                put(f, w, t);
                puts = t + 1;
            });
        if (!ok) {   // copies still in flight are waited for
            fail();
            for (int t = max(puts - C::STG, 0); t < puts; ++t) wait_warp(sb + C::FULL + 8 * (t % C::STG), (t / C::STG) & 1);
        }
    }

    // ------------------------------------------------------------------ queries in two e4m3 parts
    // bf16 rows of an item -> QP N rows of e4m3, in the same place: everything is read before anything
    // is written.  What undoes the scaling goes to qf.
    __device__ __forceinline__ void split_queries(int slot, int lw, int lane) {
        constexpr int LANES = D / 4, RPI = 32 / LANES;          // lanes of a row, rows of a warp at a time
        constexpr int ITER = N / (C::LW * RPI);
        uint8_t* q = sm + C::Q + slot * C::QB;
        const int sub = lane % LANES, byte = sub * 8;
        uint32_t one[ITER], two[ITER];
#pragma unroll
        for (int it = 0; it < ITER; ++it) {
            const int r = (it * C::LW + lw) * RPI + lane / LANES;
            const uint2 u = *reinterpret_cast<const uint2*>(q + (byte >> 7) * C::QBLOCK + sm100::sw128_off(r, (byte & 127) >> 4) + (byte & 15));
            float x[4] = {__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                          __uint_as_float(u.y & 0xffff0000u)};
            float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const int ex = (int)((__float_as_uint(top) >> 23) & 255u);
            const int sh = ex == 0 || ex == 255 ? 0 : max(ex - 127 - 7, -126);
            const float down = __uint_as_float((uint32_t)(127 - sh) << 23);   // 2^-sh, exact
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = ex == 255 ? x[e] - x[e] : x[e] * down;   // a row with an infinity scores NaN
            uint32_t a = 0, b = 0;
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const uint32_t hi = e4m3x2(x[e], x[e + 1]);
                const float2 h = __half22float2(half2_of(hi));
                a |= hi << (8 * e);
                b |= e4m3x2((x[e] - h.x) * 16.f, (x[e + 1] - h.y) * 16.f) << (8 * e);
            }
            one[it] = a;
            two[it] = b;
            if (sub == 0) reinterpret_cast<float*>(sm + C::QF)[slot * N + r] = __uint_as_float((uint32_t)(127 + sh) << 23);
        }
        bar_all(kSplitBar, 32 * C::LW);
#pragma unroll
        for (int it = 0; it < ITER; ++it) {
            const int r = (it * C::LW + lw) * RPI + lane / LANES;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const uint32_t row = y * N + r;
                const uint32_t at = (C::BROWB == 64 ? sm100::sw64_off(row, sub >> 2) : sm100::sw128_off(row, sub >> 2)) + (sub & 3) * 4;
                *reinterpret_cast<uint32_t*>(q + at) = y ? two[it] : one[it];
            }
        }
    }
    __device__ __forceinline__ void splitter(int lw, int lane) {
        bool ok = true;
        for (int item = 0;; ++item) {
            const int slot = item % C::QS;
            ok = wait_warp(sb + C::QRAW + 8 * slot, (item / C::QS) & 1);
            if (bar_any(kSplitBar, !ok || aborted(), 32 * C::LW)) break;
            const bool last = reinterpret_cast<const uint32_t*>(sm + C::QLAST)[slot];
            split_queries(slot, lw, lane);
            sm100::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(sb + C::QFULL + 8 * slot);
            if (last) break;
        }
        if (!ok) fail();
    }

    // ------------------------------------------------------------------ products
    __device__ __forceinline__ uint8_t* v_image(int t) const { return sm + C::RING + (t % C::STG) * C::STAGE + C::RAW; }
    __device__ __forceinline__ bool wait_full(int t) const { return wait_warp(sb + C::FULL + 8 * (t % C::STG), (t / C::STG) & 1); }
    static __device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
        if constexpr (F8) umma_f8(d, a, b, id, accumulate);
        else sm100::umma_bf16(d, a, b, id, accumulate);
    }

    // Scores of tile s, values of tile p, in whatever order the operands come.  The whole warp walks
    // through (its decisions are votes, so that descriptors stay in uniform registers), one lane issues.
    __device__ __forceinline__ void issuer(uint32_t tmem) {
        using namespace sm100;
        constexpr uint32_t id_s = idesc(!F8, 128, C::QP * N, false, false), id_o = idesc(!F8, D, C::PP * N, true, true);
        constexpr uint32_t SBO = 8 * C::BROWB;
        // queries, split or not, are rows of BROWB bytes as the keys are
        const uint64_t k0 = smem_desc(sb + C::RING, 16, SBO, C::SWZ), q0 = smem_desc(sb + C::Q, 16, SBO, C::SWZ);
        const uint64_t v0 = smem_desc(sb + C::RING + C::RAW, C::BLOCK, SBO, C::SWZ);
        const uint64_t p0 = smem_desc(sb + C::PM, 128, TOK * 16, 0);
        constexpr int KPB = C::BROWB / 32;   // products along a block of channels, 32 bytes each
        int s = 0, p = 0, ss = 0, ps = 0;    // tiles, and their stages
        uint32_t sp = 0;                     // phase of tile s's stage
        int qitem = -1, qslot = -1, item = -1;   // of tile s, of tile p
        long long t0 = 0;
        bool ok = true, more = true, done = false;   // more scores to come, all done
        for (uint32_t idle = 0; !done;) {
            bool go = more && s < p + 2 && mbar_test(sb + C::FULL + 8 * ss, sp) &&
                      (s < 2 || mbar_test(sb + C::SFREE + 8 * (s & 1), ((s >> 1) - 1) & 1));
            if (__all_sync(0xffffffffu, go)) {
                const bool first = __any_sync(0xffffffffu, meta(s)->flags & kFirst);
                const int it = qitem + (first ? 1 : 0), slot = !first ? qslot : qslot + 1 == C::QS ? 0 : qslot + 1;
                go = !F8 || !first || mbar_test(sb + C::QFULL + 8 * slot, (it / C::QS) & 1);
                if (__all_sync(0xffffffffu, go)) {
                    qitem = it;
                    qslot = slot;
                    tc_fence_after();
                    const uint64_t k = k0 + ((uint32_t)(ss * C::STAGE) >> 4), q = q0 + ((uint32_t)(qslot * C::QB) >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int x = 0; x < C::BLKS * KPB; ++x)
                            product(tmem + C::QP * N * (s & 1), k + ((x / KPB * C::BLOCK + x % KPB * 32) >> 4),
                                    q + ((x / KPB * C::QBLOCK + x % KPB * 32) >> 4), id_s, x > 0);
                        umma_commit(sb + C::SFULL + 8 * (s & 1));
                    }
                    __syncwarp();
                    more = !__any_sync(0xffffffffu, meta(s)->flags & kEnd);
                    ++s;
                    if (++ss == C::STG) { ss = 0; sp ^= 1; }
                    idle = 0;
                    continue;
                }
            }
            go = p < s && mbar_test(sb + C::PFULL, p & 1);
            if (__all_sync(0xffffffffu, go)) {
                const bool first = __any_sync(0xffffffffu, meta(p)->flags & kFirst);
                const int it = item + (first ? 1 : 0);
                go = !first || it < C::OB || mbar_test(sb + C::OFREE + 8 * (it % C::OB), (it / C::OB - 1) & 1);
                if (__all_sync(0xffffffffu, go)) {
                    item = it;
                    tc_fence_after();
                    const uint64_t v = v0 + ((uint32_t)(ps * C::STAGE) >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int x = 0; x < TOK / C::KSTEP; ++x)
                            product(tmem + 2 * C::QP * N + C::PP * N * (it % C::OB), v + (x * C::KSTEP * C::BROWB >> 4),
                                    p0 + (x * C::KSTEP * 16 >> 4), id_o, x > 0 || !first);
                        umma_commit(sb + C::PVDONE + 8 * (p & 1));
                        umma_commit(sb + C::EMPTY + 8 * ps);
                    }
                    __syncwarp();
                    done = __any_sync(0xffffffffu, meta(p)->flags & kEnd);
                    ++p;
                    if (++ps == C::STG) ps = 0;
                    idle = 0;
                    continue;
                }
            }
            if (idle++ == 0) t0 = clock64();
            if ((idle & 255u) == 0 && __any_sync(0xffffffffu, aborted() || clock64() - t0 > 4000000000ll)) { ok = false; break; }
        }
        if (!ok) fail();
        // nothing may still run on the tensor pipe when Tensor Memory is released
        if (elect_one()) umma_commit(sb + C::FIN);
        __syncwarp();
        wait_warp(sb + C::FIN, 0);
    }

    // ------------------------------------------------------------------ softmax
    // Four warps have RW rows: wq is the warp among them, row0 the first row, bar their barrier.
    // This thread's channel of O^T: TMEM lanes are channels, with D = 64 the first 16 of each 32; -1: none.
    static __device__ __forceinline__ int channel(int wq, int lane) { return D == 128 ? 32 * wq + lane : lane < 16 ? 16 * wq + lane : -1; }
    typedef typename std::conditional<F8, uint8_t, uint16_t>::type Bits;   // of a value
    static __device__ __forceinline__ bool finite(uint32_t x) { return F8 ? (x & 0x7fu) != 0x7fu : (x & 0x7f80u) != 0x7f80u; }
    __device__ __forceinline__ bool sees(const Meta& mt, int j, int p) const {
        return (j <= p) & (j >= mt.start) & ((P.window <= 0) | (p - j < P.window));
    }

    // Keys that some tokens see and some do not take part in the product for all (with weight 0
    // for those that do not see them), which a NaN or infinity among their values would break: such
    // elements are taken out of the image, and the channel's rows that see them noted in pos / neg.
    // Each group of four warps looks for itself; the first takes the elements out when all have looked.
    // False when that wait ran out.
    __device__ __forceinline__ bool sanitize(const Meta& mt, int t, bool ok, int w, int lane, uint32_t& events, uint32_t& pos, uint32_t& neg) {
        const int wq = w & 3, row0 = (w >> 2) * C::RW;
        const uint32_t bar = 1 + (w >> 2);
        uint8_t* v = v_image(t);
        const int key = 32 * wq + lane, j = mt.j0 + key;
        uint32_t bad = 0;
        if (ok && (j > mt.pos0 || j < mt.all_lo)) {
#pragma unroll
            for (int ch = 0; ch < C::ROWB / 16; ++ch) {
                const uint4 u = *reinterpret_cast<const uint4*>(v + C::chunk(key, ch));
                const uint32_t a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int x = 0; x < 4; ++x)   // all ones in a field carry out of it
                    bad |= F8 ? ((a[x] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u : ((a[x] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
            }
        }
        if (!bar_any(bar, bad != 0, 128)) return true;
        volatile uint32_t* bits = reinterpret_cast<volatile uint32_t*>(sm + C::BITS) + (w & ~3);
        const uint32_t mine = __ballot_sync(0xffffffffu, bad != 0);
        if (lane == 0) bits[wq] = mine;
        bar_all(bar, 128);
        const int d = channel(wq, lane);
        auto element = [&](int k) {
            const int byte = d * (int)sizeof(Bits);
            return reinterpret_cast<Bits*>(v + C::chunk(k, byte >> 4) + (byte & 15));
        };
        if (d >= 0)
            for (int x = 0; x < 4; ++x)
                for (uint32_t m = bits[x]; m; m &= m - 1) {
                    const int k = 32 * x + __ffs(m) - 1;
                    const uint32_t val = *element(k);
                    if (finite(val)) continue;
                    const bool nan = F8 || (val & 0x7fu) != 0, minus = val & 0x8000u;   // e4m3 has no infinities
                    for (int r = 0; r < C::RW && row0 + r < mt.rows; ++r) {
                        if (!sees(mt, mt.j0 + k, mt.pos0 + (mt.block * N + row0 + r) / P.group)) continue;
                        if (nan || !minus) pos |= 1u << r;
                        if (nan || minus) neg |= 1u << r;
                    }
                }
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(sb + C::LOOKED);
        const uint32_t phase = events++ & 1;
        if (row0) return true;
        if (!wait_warp(sb + C::LOOKED, phase)) return false;
        if (d >= 0)
            for (int x = 0; x < 4; ++x)
                for (uint32_t m = bits[x]; m; m &= m - 1) {
                    Bits* e = element(32 * x + __ffs(m) - 1);
                    if (!finite(*e)) *e = 0;
                }
        return true;
    }

    // 8 rows of O^T, the parts summed up
    static __device__ __forceinline__ void load_out(uint32_t t, float (&o)[8]) {
        tmem_ld8(t, o);
        float b[8];
        tmem_ld8(t + N, b);
        if constexpr (F8) {
            float c[8];
            tmem_ld8(t + 2 * N, c);
            sm100::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] += (b[i] + c[i] * (1.f / 16)) * (1.f / 16);
        } else {
            sm100::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] += b[i];
        }
    }

    __device__ __forceinline__ void softmax(uint32_t tmem, int w, int lane) {
        using namespace sm100;
        constexpr int RW = C::RW;
        const int wq = w & 3, row0 = (w >> 2) * RW, tid = 32 * wq + lane, key = tid;
        const uint32_t bar = 1 + (w >> 2), tl = tmem + ((uint32_t)(32 * wq) << 16);
        float* limit = reinterpret_cast<float*>(sm + C::MROW) + row0;   // maximum + slack
        float* base = limit + N;                                        // what a score's exponent counts from: maximum - BASE, or 0
        float* unit = reinterpret_cast<float*>(sm + C::RINFO) + row0;   // scale of the raw products
        float* slope = unit + N;                                        // bias per key
        float* wred = reinterpret_cast<float*>(sm + C::WRED) + row0;
        float* frow = reinterpret_cast<float*>(sm + C::FROW) + row0;
        const float cap2 = P.softcap * kLog2e, scale = P.scale * (P.softcap > 0.f ? 1.f / P.softcap : kLog2e);
        float l[RW];
        uint32_t pos = 0, neg = 0, events = 0;
        bool bad = false;
        for (int t = 0;; ++t) {
            bad |= !wait_warp(sb + C::MFULL + 8 * (t % C::MD), (t / C::MD) & 1);
            const Meta mt = *meta(t);
            // After a wait that ran out nothing of the tile is known.  No barrier of the group stands before the
            // votes below, so a warp can go to them at once, and the group stops together.
            if (bad) {
                bar_any(bar, true, 128);
                bar_any(bar, true, 128);
                break;
            }
            const bool first = mt.flags & kFirst, edge = mt.flags & kEdge;
            const int rows = min(mt.rows - row0, RW);   // of these warps; maybe none
            if (first) {
                if constexpr (F8) bad |= !wait_warp(sb + C::QFULL + 8 * (mt.item % C::QS), (mt.item / C::QS) & 1);
                if (lane < RW) {   // every warp writes the same, so that no barrier stands before the vote
                    limit[lane] = -INFINITY;
                    base[lane] = 0.f;
                    float f = scale;
                    if (F8) f *= (P.c.k_scale ? P.c.k_scale[mt.h] : 1.f) * reinterpret_cast<const float*>(sm + C::QF)[(mt.item % C::QS) * N + row0 + lane];
                    unit[lane] = f;
                    slope[lane] = P.slopes && lane < rows ? P.slopes[mt.h * P.group + (mt.block * N + row0 + lane) % P.group] * kLog2e : 0.f;
                }
                __syncwarp();
#pragma unroll
                for (int r = 0; r < RW; ++r) l[r] = 0.f;
                pos = neg = 0;
            }
            bad |= !wait_warp(sb + C::SFULL + 8 * (t & 1), (t >> 1) & 1);
            tc_fence_after();
            const bool ok = (reinterpret_cast<const uint32_t*>(sm + C::OKM + (t % C::MD) * 16)[wq] >> lane) & 1;
            const bool mask = edge || !__all_sync(0xffffffffu, ok);
            const uint32_t tS = tl + C::QP * N * (t & 1) + row0, tO = tl + 2 * C::QP * N + C::PP * N * (mt.item % C::OB) + row0;
            const int j = mt.j0 + key;
            float s[RW];
            if (rows > 0) {
                if constexpr (RW == 16) tmem_ld16(tS, s);
                else tmem_ld8(tS, s);
                tmem_wait_ld();
            }
            uint32_t up = 0;   // counted without branches
            int tok = mt.tok0, left = mt.left0;
            if ((P.slopes || mask) && row0) {
                tok = (mt.block * N + row0) / P.group;
                left = (tok + 1) * P.group - (mt.block * N + row0);
            }
#pragma unroll
            for (int c = 0; c < RW; c += 8) {
                if (c >= rows) break;
                if constexpr (F8) {   // the product with the queries' second part
                    float s2[8];
                    tmem_ld8(tS + N + c, s2);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[c + i] += s2[i] * (1.f / 16);
                }
                float f[8], top[8];
                load8(unit + c, f);   // the same for all lanes
                load8(limit + c, top);
                if (P.softcap > 0.f) {
                    // tanh y by its Taylor series up to y^9 where |y| <= 1/4 (the next term is below 2^-26 of it: most
                    // scores lie far below their cap, and no ex2 or rcp is spent on them), 1 - 2 / (1 + e^{2 y}) beyond
                    float big = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float y = s[c + i] * f[i], z = y * y;
                        const float tail = z * (-1.f / 3 + z * (2.f / 15 + z * (-17.f / 315 + z * (62.f / 2835))));
                        big = fmaxf(big, fabsf(y));
                        s[c + i] = fabsf(y) > 0.25f ? y : cap2 * (y + y * tail);
                        f[i] = y;
                    }
                    if (__any_sync(0xffffffffu, big > 0.25f)) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float y = f[i];
                            if (fabsf(y) > 0.25f) s[c + i] = cap2 - 2.f * cap2 * rcp(1.f + ex2(y * (2.f * kLog2e)));
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float2 x = mul2(make_float2(s[c + i], s[c + i + 1]), make_float2(f[i], f[i + 1]));
                        s[c + i] = x.x;
                        s[c + i + 1] = x.y;
                    }
                }
                if (P.slopes || mask) {
                    float a[8];
                    load8(slope + c, a);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int p = mt.pos0 + tok;
                        s[c + i] += a[i] * (float)(j - p);   // no bias: a slope of 0
                        s[c + i] = ok & sees(mt, j, p) ? s[c + i] : -INFINITY;
                        const bool over = --left == 0;
                        tok += over;
                        left = over ? P.group : left;
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) up |= s[c + i] > top[i];
            }
            // the weights of the tile before, and O, are free
            if (t > 0) bad |= !wait_warp(sb + C::PVDONE + 8 * ((t - 1) & 1), ((t - 1) >> 1) & 1);
            if (bar_any(bar, up != 0 || bad, 128)) {
                if (bar_any(bar, bad, 128)) break;   // a wait ran out: all stop here
                // some row's maximum rises: the new one, and what the sums so far are worth in it
                tc_fence_after();
                float mine = -INFINITY;
#pragma unroll
                for (int c = 0; c < RW; c += 8) {
                    if (c >= rows) break;
#pragma unroll
                    for (int i = c; i < c + 8; ++i) {
                        const float x = warp_max(s[i]);
                        if (lane == i) mine = x;
                    }
                }
                if (lane < RW) wred[wq * N + lane] = mine;
                bar_all(bar, 128);
                if (tid < RW) {
                    const float top = fmaxf(fmaxf(wred[tid], wred[N + tid]), fmaxf(wred[2 * N + tid], wred[3 * N + tid]));
                    const float old = limit[tid];
                    float f = 1.f;
                    if (top > old) {
                        f = old == -INFINITY ? 0.f : ex2(base[tid] + C::BASE - top);
                        limit[tid] = top + C::SLACK;
                        base[tid] = top - C::BASE;
                    }
                    frow[tid] = f;
                }
                bar_all(bar, 128);
                if (!first) {
#pragma unroll
                    for (int c = 0; c < RW; c += 8) {
                        if (c >= rows) break;
#pragma unroll
                        for (int i = 0; i < 8; ++i) l[c + i] *= frow[c + i];
#pragma unroll
                        for (int y = 0; y < C::PP; ++y) {
                            float o[8];
                            tmem_ld8(tO + y * N + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] *= frow[c + i];
                            tmem_st8(tO + y * N + c, o);
                        }
                    }
                    tmem_wait_st();
                }
            }
#pragma unroll
            for (int c = 0; c < RW; c += 8) {
                if (c >= rows) break;
                uint32_t pk[2][4], part[3][2] = {};
                float m[8];
                load8(base + c, m);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float2 x = sub2(make_float2(s[c + i], s[c + i + 1]), make_float2(m[i], m[i + 1]));
                    const float a = ex2(x.x), b = ex2(x.y);
                    const float2 sum = add2(make_float2(l[c + i], l[c + i + 1]), make_float2(a, b));
                    l[c + i] = sum.x;
                    l[c + i + 1] = sum.y;
                    if constexpr (F8) {   // remainders are exact, but that the first is rounded to fp16
                        const __half2 k16 = __float2half2_rn(16.f);
                        const uint32_t e = e4m3x2(a, b);
                        const float2 h = __half22float2(half2_of(e));
                        const float2 rest = fma2(h, make_float2(-16.f, -16.f), mul2(make_float2(a, b), make_float2(16.f, 16.f)));
                        __half2 r = __floats2half2_rn(rest.x, rest.y);
                        part[0][i / 4] |= e << (16 * (i / 2 % 2));
#pragma unroll
                        for (int y = 1; y < 3; ++y) {
                            const uint32_t e = e4m3x2(r);
                            part[y][i / 4] |= e << (16 * (i / 2 % 2));
                            if (y < 2) r = __hmul2(__hsub2(r, half2_of(e)), k16);
                        }
                    } else {
                        const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
                        pk[0][i / 2] = __byte_perm(ua, ub, 0x7632);
                        const float2 rest = fma2(make_float2(a, b), make_float2(kAbove1, kAbove1),
                                                 make_float2(-__uint_as_float(ua & 0xffff0000u), -__uint_as_float(ub & 0xffff0000u)));
                        pk[1][i / 2] = pack_bf16x2(rest.x, rest.y);
                    }
                }
                uint8_t* at = sm + C::PM + (row0 + c) / C::PG * (TOK * 16) + key * 16;
                if constexpr (F8) {
#pragma unroll
                    for (int y = 0; y < 3; ++y)
                        *reinterpret_cast<uint2*>(at + y * (N / 16) * (TOK * 16) + (row0 + c) % 16) = make_uint2(part[y][0], part[y][1]);
                } else {
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        *reinterpret_cast<uint4*>(at + y * (N / 8) * (TOK * 16)) = make_uint4(pk[y][0], pk[y][1], pk[y][2], pk[y][3]);
                }
            }
            if (row0 == 0 && !__all_sync(0xffffffffu, ok)) {   // a value row that was not fetched, or that no token sees
                bad |= !wait_full(t);
                if (!ok)
#pragma unroll
                    for (int ch = 0; ch < C::ROWB / 16; ++ch) *reinterpret_cast<uint4*>(v_image(t) + C::chunk(key, ch)) = make_uint4(0u, 0u, 0u, 0u);
                __syncwarp();
            }
            if (edge && mt.nq > 1) {
                bad |= !wait_full(t);
                bad |= !sanitize(mt, t, ok, w, lane, events, pos, neg);
            }
            tc_fence_before();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(sb + C::SFREE + 8 * (t & 1));
                mbar_arrive(sb + C::PFULL);
            }
            if (!(mt.flags & kLast)) continue;

            // the item's end here: the sums while the last product runs, then the outputs
            float* to = P.partial + (int64_t)mt.part * (N * (D + 2)) + row0;   // of a split item
            // sums over the warp's keys: lane i of the first RW ends with row i
            if (rows > 0) {
                float v[RW];
#pragma unroll
                for (int i = 0; i < RW; ++i) {
                    v[i] = l[i] + __shfl_xor_sync(0xffffffffu, l[i], 16);
                    if (RW == 8) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 8);
                }
#pragma unroll
                for (int o = RW / 2; o > 0; o >>= 1)
#pragma unroll
                    for (int i = 0; i < o; ++i) {
                        const bool hi = lane & o;
                        const float give = hi ? v[i] : v[i + o], keep = hi ? v[i + o] : v[i];
                        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                    }
                if (lane < RW) wred[wq * N + lane] = v[0];
            }
            bar_all(bar, 128);
            float sum = 0.f, top = 0.f;
            if (tid < rows) {
                sum = wred[tid] + wred[N + tid] + wred[2 * N + tid] + wred[3 * N + tid];
                top = limit[tid] == -INFINITY ? -INFINITY : base[tid];
                const float vs = F8 && P.c.v_scale ? P.c.v_scale[mt.h] : 1.f;
                frow[tid] = mt.part >= 0 ? 1.f : sum == 0.f ? 0.f : vs / sum;
            }
            bar_all(bar, 128);
            bad |= !wait_warp(sb + C::PVDONE + 8 * (t & 1), (t >> 1) & 1);
            tc_fence_after();
            const int d = channel(wq, lane);
            tok = mt.tok0;
            left = mt.left0;
            if (row0) {
                tok = (mt.block * N + row0) / P.group;
                left = (tok + 1) * P.group - (mt.block * N + row0);
            }
            const int64_t at0 = (mt.t0 + tok) * P.Hq + mt.h * P.group + (P.group - left);   // output row
            if (mt.part < 0) {
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(P.out) + at0 * D + d;
                const int64_t step = (int64_t)(P.Hq - P.group + 1) * D;   // to the next token's first row
#pragma unroll
                for (int c = 0; c < RW; c += 8) {
                    if (c >= rows) break;
                    float o[8];
                    load_out(tO + c, o);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float x = o[i];
                        x += (pos >> (c + i)) & 1 ? INFINITY : 0.f;   // what sanitize has noted
                        x -= (neg >> (c + i)) & 1 ? INFINITY : 0.f;
                        if ((c + i < rows) & (d >= 0)) *dst = __float2bfloat16_rn(x * frow[c + i]);
                        const bool over = --left == 0;
                        dst += over ? step : D;
                        left = over ? P.group : left;
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < RW; c += 8) {
                    if (c >= rows) break;
                    float o[8];
                    load_out(tO + c, o);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float x = o[i];
                        x += (pos >> (c + i)) & 1 ? INFINITY : 0.f;
                        x -= (neg >> (c + i)) & 1 ? INFINITY : 0.f;
                        if ((c + i < rows) & (d >= 0)) to[2 * N + row0 * (D - 1) + (c + i) * D + d] = x;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sb + C::OFREE + 8 * (mt.item % C::OB));
            if (tid < rows) {
                if (mt.part >= 0) {
                    to[tid] = top;
                    to[N + tid] = sum;
                } else if (P.lse) {
                    const int ir = mt.block * N + row0 + tid, tk = ir / P.group;
                    P.lse[(mt.t0 + tk) * P.Hq + mt.h * P.group + (ir - tk * P.group)] = sum == 0.f ? -INFINITY : top * kLn2 + logf(sum);
                }
            }
            if (mt.flags & kEnd) break;
        }
        if (bad) fail();
    }

    __device__ __forceinline__ void run() {
        const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
        if (tid == 0) { prefetch_map(&P.k_map); prefetch_map(&P.v_map); prefetch_map(&P.q_map); }
        kda_grid_wait();
        W w(P);
        if (!w.few()) w.template find<C::THREADS>(reinterpret_cast<int64_t*>(sm + C::RING));
        kda_grid_launch_next();
        Fetch<C, N> f{P, lane, warp == C::SW, {}};
        if (warp == 0) sm100::tmem_alloc(sb + C::TMEM, C::TCOLS);
        if (warp == C::SW || warp == C::SW + 1) {
            if (f.keys && lane == 0) {
                for (int i = 0; i < C::STG; ++i) {
                    sm100::mbar_init(sb + C::FULL + 8 * i, 1);
                    sm100::mbar_init(sb + C::EMPTY + 8 * i, 1);
                    sm100::mbar_init(sb + C::QRAW + 8 * i, 1);
                    sm100::mbar_init(sb + C::QFULL + 8 * i, F8 ? C::LW : 1);
                }
                for (int i = 0; i < C::MD; ++i) sm100::mbar_init(sb + C::MFULL + 8 * i, 1);
                for (int i = 0; i < 2; ++i) {
                    sm100::mbar_init(sb + C::SFULL + 8 * i, 1);
                    sm100::mbar_init(sb + C::SFREE + 8 * i, C::SW);
                    sm100::mbar_init(sb + C::PVDONE + 8 * i, 1);
                    sm100::mbar_init(sb + C::OFREE + 8 * i, C::SW);
                }
                sm100::mbar_init(sb + C::PFULL, C::SW);
                sm100::mbar_init(sb + C::FIN, 1);
                sm100::mbar_init(sb + C::LOOKED, C::SW);
                sm100::fence_mbar_init();
            }
            const bool any = f.begin(w);
            if (f.keys && lane == 0) *reinterpret_cast<volatile uint32_t*>(sm + C::ABORT) = 0;
            if (f.keys && lane == 0) *reinterpret_cast<volatile uint32_t*>(sm + C::ANY) = any;
        }
        sm100::tc_fence_before();
        __syncthreads();
        sm100::tc_fence_after();
        const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + C::TMEM);
        if (!*reinterpret_cast<volatile uint32_t*>(sm + C::ANY)) {
            // nothing to do here
        } else if (warp < C::SW) {
            softmax(tmem, warp, lane);
        } else if (warp <= C::SW + 1) {
            fetcher(f, w);
        } else if (warp == C::SW + 2) {
            issuer(tmem);
        } else {
            if constexpr (F8) splitter(warp - C::SW - 3, lane);
        }
        sm100::tc_fence_before();
        __syncthreads();
        sm100::tc_fence_after();
        __syncwarp();
        if (warp == 0) sm100::tmem_dealloc(tmem, C::TCOLS);
    }
};

template <int D, typename TC, int N>
__global__ void __launch_bounds__(Tc<D, TC, N>::THREADS, 1) attend_tc_kernel(const __grid_constant__ Params P) {
    extern __shared__ __align__(1024) uint8_t smem[];
    TcKernel<D, TC, N> k{P, smem, sm100::smem_u32(smem)};
    k.run();
}

template <int D, typename TC, int N>
cudaError_t launch_tc(Params& P, cudaStream_t stream) {
    typedef Tc<D, TC, N> C;
    if (!make_maps<C>(P, D, (int)sizeof(TC), sizeof(TC) == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                      CU_TENSOR_MAP_DATA_TYPE_BFLOAT16))
        return cudaErrorNotSupported;
    return launch_pair<D, __nv_bfloat16, TC, N>(attend_tc_kernel<D, TC, N>, C::THREADS, C::BYTES, P, stream);
}
template <int D, int R>
cudaError_t launch_simt(Params& P, cudaStream_t stream) {
    typedef Simt<D, R> C;
    if (!make_maps<C>(P, D, 4, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, CU_TENSOR_MAP_DATA_TYPE_FLOAT32)) return cudaErrorNotSupported;
    return launch_pair<D, float, float, R>(attend_simt_kernel<D, R>, C::THREADS, C::BYTES, P, stream);
}
template <int D, typename T, typename TC>
cudaError_t launch(Params& P, cudaStream_t stream) {
    const int rows = block_rows(sizeof(T) == 4, P.group * P.max_q);
    if constexpr (sizeof(T) == 4)
        return rows == 1 ? launch_simt<D, 1>(P, stream) : rows == 2 ? launch_simt<D, 2>(P, stream) : launch_simt<D, 8>(P, stream);
    else
        return rows == 16 ? launch_tc<D, TC, 16>(P, stream) : rows == 32 ? launch_tc<D, TC, 32>(P, stream) : launch_tc<D, TC, 64>(P, stream);
}

}  // namespace attend
}  // namespace kda
