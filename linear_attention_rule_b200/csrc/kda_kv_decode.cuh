// Softmax attention of the newest tokens over the paged cache: what the kernels share.
//
// Per query row, in one pass over its visible keys with the running maximum m, the sum l and
// the weighted values acc (scores in units of log 2, so that e^x is one ex2):
//   m' = max(m, s_j);  l' = l 2^{m - m'} + 2^{s_j - m'};  acc' = acc 2^{m - m'} + 2^{s_j - m'} v_j.
// Two such triples over different keys join the same way, which is how a sequence is split.
//
// A key and a value row serve the G = Hq / Hkv query heads of their group and the sequence's new
// tokens (G x tokens rows), 4 D flops per row for 2 D elements.  As long as these rows are one block (up to 64
// rows, in fp32 8) the cache is read once, and its bytes bound the kernel up to 32 rows (fp32: one); each
// further block reads it again.  So the work is cut by bytes alone: all (sequence, kv head, row block) items are laid
// end to end in tiles of keys, and each of 148 CTAs (one per SM) takes one equal stretch of that
// line, whatever the lengths.  Its tiles go through a ring of shared-memory stages.  Items that lie within one stretch are
// finished there; the others leave a partial triple per stretch, which the join kernel adds up.
//
// Two warps of a CTA walk its stretch and fetch the tiles with TMA (a load takes about 40 issue cycles, and
// pages of 16 rows make 32 of a 64 KB tile): one the keys, one the values and queries.  A box is the part of a page
// in the tile (page_size rows, or the tile), so pages may end anywhere in a tile; boxes without a
// visible key are not fetched.  The first version fetched rows with 16-byte cp.async from four warps:
// it kept the load/store pipe so busy (1,750 of the 3,850 cycles of a 64 KB tile) that the
// softmax's own shared-memory loads queued behind it.
#pragma once

#include <algorithm>

#include <cuda.h>
#include <cuda_fp16.h>

#include "kda_kv_cache.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace attend {

// An item that starts in a worker's stretch and goes on behind it (for the join).
struct Split {
    int64_t t0;               // first new token of the sequence
    int32_t h, block, nq;     // kv head, row block, new tokens
    int32_t last;             // the worker that holds the item's last tile; -1: no such item
};

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
    Split* split;      // workspace: one per worker, then
    int32_t box_shift;   // rows of a TMA box: 1 << box_shift
    CUtensorMap k_map, v_map, q_map;
    float* partial;    // two partial triples per worker: of the item that began before it, and of the one that goes on
};

constexpr int kWorkers = 148;      // one CTA per SM
constexpr int kGroups = 1024;      // entries of the table of work in shared memory
constexpr int kMaxSmem = 232448;   // dynamic shared memory of a CTA
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// One sequence's share: its new tokens, the keys [lo, hi) that any of them sees, and its tiles.
struct Seq {
    int64_t t0;
    int nq, pos0;        // new tokens, position of the first
    int start, lo, hi;   // kv_start, first and behind the last visible key
    int tile0, tiles, blocks;
};

// First key that a token at position pos sees.
__device__ __forceinline__ int first_key(const Params& P, int start, int pos) {
    return P.window > 0 ? max(start, (int)max((int64_t)pos - P.window + 1, (int64_t)0)) : start;
}

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
    const int64_t held = min((int64_t)P.c.max_pages << P.c.page_shift, (int64_t)INT32_MAX - 2 * TOK);
    const int len = max(P.c.seq_lens[n], 0);
    s.pos0 = len - s.nq;
    s.hi = (int)min((int64_t)len, held);
    s.start = P.kv_start ? max(P.kv_start[n], 0) : 0;
    s.lo = first_key(P, s.start, s.pos0);
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
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// largest of the warp's values; NaN only if all are
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
// Bounded wait of a whole warp for an mbarrier phase (about a second); false when it ran out.  The lanes leave
// it together: what follows (tcgen05.ld, barriers) wants them so.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, sm100::mbar_try_wait(bar, parity))) return true;
    const long long t0 = clock64();
    while (true) {
        if (__all_sync(0xffffffffu, sm100::mbar_try_wait(bar, parity))) return true;
        if (__any_sync(0xffffffffu, clock64() - t0 > 2000000000ll)) return false;
    }
}
// TMA box loads; all boxes start at a multiple of 16 bytes of the innermost axis.
__device__ __forceinline__ void tma4(uint32_t dst, const CUtensorMap* map, int x, int row, int head, int page, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(map), "r"(x), "r"(row), "r"(head), "r"(page), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma3(uint32_t dst, const CUtensorMap* map, int x, int head, int token, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(x), "r"(head), "r"(token), "r"(bar) : "memory");
}
// Barrier `id` of `count` threads that tells all of them whether `p` holds for any.
__device__ __forceinline__ bool bar_any(uint32_t id, bool p, uint32_t count) {
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred a, b;\n\t"
        "setp.ne.u32 a, %1, 0;\n\t"
        "barrier.cta.red.or.pred b, %2, %3, a;\n\t"
        "selp.u32 %0, 1, 0, b;\n\t}"
        : "=r"(r) : "r"((uint32_t)p), "r"(id), "r"(count) : "memory");
    __syncwarp();
    return r != 0;
}

// Barrier `id` of `count` threads.
__device__ __forceinline__ void bar_all(uint32_t id, uint32_t count) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
    __syncwarp();
}

// What the fetching warp tells the other warps of a tile.
struct Meta {
    int64_t t0;
    int32_t j0;          // first key
    int32_t flags;       // kFirst ..
    int32_t h, block, rows, nq, pos0, start;
    int32_t all_lo;      // keys all_lo .. pos0 are seen by every token
    int32_t item;        // count of items in this stretch
    int32_t part;        // where the item's triple goes: -1 (finished here) or a slot of P.partial
    int32_t tok0, left0; // token of the block's first row, and how many rows of the block are of that token
    int32_t pad;
};
static_assert(sizeof(Meta) == 64, "laid out in shared memory");
enum : int32_t { kFirst = 1, kLast = 2, kEdge = 4, kEnd = 8 };   // first, last tile of the item here; not all keys seen by all; last tile of all

// The stretch of this worker, and the walk along its tiles.  An item takes a unit of the line for each of
// its tiles and, before them, kItemCost for its beginning and end (queries, the first maximum, the
// outputs).  64 sequences of 512 to 16,384 bf16 keys and 48 of 64 to 16,384 e4m3 keys with drafts took 237
// and 126 us at a cost of 0, 204 and 99 at 1, 204 and 87 at 2, 208 and 93 at 4 (a call by itself).
constexpr int kItemCost = 2;

template <int TOK, int ROWS>
struct Walk {
    const Params& P;
    int64_t begin, end, at, per;
    int64_t base;       // where sequence n begins
    int n, item;
    Seq s;
    int h, block, tile, tiles, i;   // the item here: its tiles [tile, tile + tiles), the i-th of them is next
    bool starts, ends;              // whether it begins and ends in this stretch
    bool more;                      // whether another item has tiles here

    __device__ __forceinline__ explicit Walk(const Params& p) : P(p) {}

    // Finds the stretch: a table of the work of groups of sequences, summed up by all threads of
    // the CTA in `work` (kGroups + 1 entries and one per warp), which is free again afterwards.
    template <int THREADS>
    __device__ __forceinline__ void find(int64_t* work) {
        constexpr int SLICE = (kGroups + THREADS - 1) / THREADS;
        int64_t* wsum = work + kGroups + 1;
        const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
        const int N = P.num_seqs, per_group = (N + kGroups - 1) / kGroups, groups = (N + per_group - 1) / per_group;
        const int slice = (groups + THREADS - 1) / THREADS;   // groups of one thread, up to SLICE
        int64_t mine[SLICE], sum = 0;
#pragma unroll
        for (int x = 0; x < SLICE; ++x) {
            const int gr = tid * slice + x;
            mine[x] = 0;
            if (x < slice && gr < groups)
                for (int m = gr * per_group; m < min(N, (gr + 1) * per_group); ++m) {
                    const Seq q = seq_info<TOK>(P, m, ROWS);
                    mine[x] += units(q) * q.blocks * P.c.Hkv;
                }
            sum += mine[x];
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
        for (int x = 0; x < SLICE; ++x) {
            const int gr = tid * slice + x;
            if (x < slice && gr < groups) work[gr] = before;
            before += mine[x];
        }
        if (tid == THREADS - 1) work[groups] = before;
        __syncthreads();
        place(work[groups]);
        int gr = 0;   // the group that holds `at`: the last with work[gr] <= at
        for (int lo = 0, hi = groups - 1; lo <= hi;) {
            const int mid = (lo + hi) >> 1;
            if (work[mid] <= at) { gr = mid; lo = mid + 1; } else hi = mid - 1;
        }
        n = gr * per_group;
        base = work[gr];
        // TMA writes there next, through another proxy than these loads and stores, which a barrier alone does not order
        sm100::fence_proxy_async_smem();
        __syncthreads();
    }
    // With up to 32 sequences each warp that walks knows them all, a lane each: no barrier, no table, and
    // no loads when the walk comes to the next one.  8 sequences of up to 300 keys took 11.5 us with the
    // table, 10.4 us so.
    static constexpr int kFew = 32;
    Seq lanes;
    __device__ __forceinline__ bool few() const { return P.num_seqs <= kFew; }
    __device__ __forceinline__ void find_few(int lane) {
        lanes = {};
        if (lane < P.num_seqs) lanes = seq_info<TOK>(P, lane, ROWS);
        const int64_t mine = units(lanes) * lanes.blocks * P.c.Hkv;
        int64_t behind = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, behind, o);
            if (lane >= o) behind += x;
        }
        place(__shfl_sync(0xffffffffu, behind, 31));
        const unsigned m = __ballot_sync(0xffffffffu, behind - mine <= at && lane < P.num_seqs);
        n = 31 - __clz(m);   // lane 0 holds place 0
        base = __shfl_sync(0xffffffffu, behind - mine, n);
    }
    // This worker's stretch of `total` units.
    __device__ __forceinline__ void place(int64_t total) {
        per = max((total + kWorkers - 1) / kWorkers, (int64_t)1);
        begin = min((int64_t)blockIdx.x * per, total);
        end = min(begin + per, total);
        at = begin;
        item = -1;
    }
    // Sequence n, by all lanes.
    __device__ __forceinline__ Seq sequence() const {
        if (!few()) return seq_info<TOK>(P, n, ROWS);
        Seq q;
        q.t0 = __shfl_sync(0xffffffffu, lanes.t0, n);
        q.nq = __shfl_sync(0xffffffffu, lanes.nq, n);
        q.pos0 = __shfl_sync(0xffffffffu, lanes.pos0, n);
        q.start = __shfl_sync(0xffffffffu, lanes.start, n);
        q.lo = __shfl_sync(0xffffffffu, lanes.lo, n);
        q.hi = __shfl_sync(0xffffffffu, lanes.hi, n);
        q.tile0 = __shfl_sync(0xffffffffu, lanes.tile0, n);
        q.tiles = __shfl_sync(0xffffffffu, lanes.tiles, n);
        q.blocks = __shfl_sync(0xffffffffu, lanes.blocks, n);
        return q;
    }

    // Units of an item of a sequence.
    static __device__ __forceinline__ int64_t units(const Seq& q) { return q.tiles + kItemCost; }
    // The item that holds `at`; false if nothing of its tiles lies in the stretch.
    __device__ __forceinline__ bool seek() {
        if (at >= end) return false;
        int64_t items = (int64_t)s.blocks * P.c.Hkv;
        while (at - base >= items * units(s)) {
            base += items * units(s);
            ++n;
            s = sequence();
            items = (int64_t)s.blocks * P.c.Hkv;
        }
        const int x = quotient(at - base, units(s));
        const int64_t a = base + x * units(s) + kItemCost, b = a + s.tiles;   // its tiles
        at = max(at, a);
        if (at >= end) return false;
        h = x / s.blocks;
        block = x - h * s.blocks;
        rows = min(ROWS, s.nq * P.group - block * ROWS);
        tok0 = block * ROWS / P.group;
        all_lo = first_key(P, s.start, s.pos0 + s.nq - 1);
        tile = s.tile0 + (int)(at - a);
        tiles = (int)(min(b, end) - at);
        starts = at == a;
        ends = b <= end;
        more = end - b > kItemCost;
        last_worker = quotient(b - 1, per);
        i = 0;
        ++item;
        return true;
    }
    int last_worker, rows, tok0, all_lo;

    // a / b < 2^31; 64-bit division takes four times as long as 32-bit
    static __device__ __forceinline__ int quotient(int64_t a, int64_t b) {
        return ((a | b) >> 32) == 0 ? (int)((uint32_t)a / (uint32_t)b) : (int)(a / b);
    }

    __device__ __forceinline__ int j0() const { return (tile + i) * TOK; }
    __device__ __forceinline__ bool next() {
        ++at;
        return ++i < tiles || seek();
    }
    __device__ __forceinline__ void fill(Meta* m) const {
        const int j = j0();
        const bool inside = j >= all_lo && j + TOK - 1 <= min(s.pos0, s.hi - 1);
        m->t0 = s.t0;
        m->j0 = j;
        m->flags = (i == 0 ? kFirst : 0) | (i == tiles - 1 ? kLast | (more ? 0 : kEnd) : 0) | (inside ? 0 : kEdge);
        m->h = h;
        m->block = block;
        m->rows = rows;
        m->nq = s.nq;
        m->pos0 = s.pos0;
        m->start = s.start;
        m->all_lo = all_lo;
        m->item = item;
        m->tok0 = tok0;
        m->left0 = (tok0 + 1) * P.group - block * ROWS;
        m->part = starts && ends ? -1 : 2 * (int)blockIdx.x + (starts ? 1 : 0);
    }
    __device__ __forceinline__ void tell_join(Split* to) const {
        if (starts && !ends) *to = {s.t0, h, block, s.nq, last_worker};
    }
};

// A fetching warp.  C: the kernel's layout: TOK keys a tile; operands in blocks of BLK channels,
// each a run of rows of BROWB bytes; values lie RAW bytes behind the keys.
template <typename C, int ROWS>
struct Fetch {
    static constexpr int RPL = C::TOK / 32;   // rows of a lane
    typedef Walk<C::TOK, ROWS> W;

    const Params& P;
    int lane;
    bool keys;       // keys and what the others need to know of a tile, or values and queries
    int page[RPL];   // of the lane's rows in the tile that is fetched next, -1 where none is needed

    // The lane's row x lies in a box with a visible key.
    __device__ __forceinline__ bool needed(const W& w, int x) const {
        const int r = (lane * RPL + x) >> P.box_shift << P.box_shift, j = w.j0() + r;
        return j + (1 << P.box_shift) > w.s.lo && j < w.s.hi && w.s.hi > w.s.lo;
    }
    __device__ __forceinline__ void look(const W& w) {
        const int32_t* table = P.c.table + w.n * P.c.table_stride;
#pragma unroll
        for (int x = 0; x < RPL; ++x) {
            page[x] = -1;
            if (needed(w, x)) page[x] = __ldg(table + ((w.j0() + lane * RPL + x) >> P.c.page_shift));
        }
    }
    // Fetches the tile that the walk stands at (and, with an item's first, its queries at q) and
    // fills in what the others need to know of it.
    // Queries with a barrier of their own come with *last: whether it is the stretch's last item.
    __device__ __forceinline__ void put(const W& w, uint32_t stage, uint32_t q, uint32_t bar, uint32_t qbar, uint32_t meta_bar, Meta* meta,
                                        uint32_t* okm, uint32_t* last) {
        const int j0 = w.j0(), box = 1 << P.box_shift;
        uint32_t bits = 0, boxes = 0;
        bool wrong = false;
#pragma unroll
        for (int x = 0; x < RPL; ++x) {
            const int r = lane * RPL + x, j = j0 + r;
            const bool need = needed(w, x), ok = need && page[x] >= 0 && page[x] < P.c.num_pages;
            wrong = wrong || (need && !ok);
            if (ok && j >= w.s.lo && j < w.s.hi) bits |= 1u << x;
            if (ok && (r & (box - 1)) == 0) ++boxes;
            if (!ok) page[x] = -1;
        }
        if (wrong && keys) kda_set_status(KDA_ERR_BAD_PAGE);
        if (keys) {
            bits <<= (lane * RPL) & 31;
#pragma unroll
            for (int o = 1; o < 32 / RPL; o <<= 1) bits |= __shfl_xor_sync(0xffffffffu, bits, o);
            if (lane % (32 / RPL) == 0) okm[lane * RPL / 32] = bits;
            boxes = __reduce_add_sync(0xffffffffu, boxes);
            if (lane == 0) w.fill(meta);
            __syncwarp();
            if (lane == 0) {
                sm100::mbar_arrive(meta_bar);
                const uint32_t queries = w.i == 0 ? C::QB : 0;
                sm100::mbar_arrive_expect_tx(bar, boxes * (uint32_t)(2 * box * C::ROWB) + (qbar == bar ? queries : 0));
                if (qbar != bar && queries) *last = !w.more;
                if (qbar != bar && queries) sm100::mbar_arrive_expect_tx(qbar, queries);
            }
            __syncwarp();
        } else if (w.i == 0) {
            for (int r = lane; r < ROWS; r += 32) {
                const int ir = w.block * ROWS + r, tok = ir / P.group, g = ir - tok * P.group;
                // rows behind the item's: a token behind the last one, which TMA fills with zeros
                const int head = r < w.rows ? w.h * P.group + g : 0, token = r < w.rows ? (int)w.s.t0 + tok : (int)P.total;
#pragma unroll
                for (int b = 0; b < C::QBLKS; ++b)
                    tma3(q + b * C::QBLOCK + r * C::QROWB, &P.q_map, b * (C::D / C::QBLKS), head, token, qbar);
            }
        }
        const CUtensorMap* map = keys ? &P.k_map : &P.v_map;
#pragma unroll
        for (int x = 0; x < RPL; ++x) {
            const int r = lane * RPL + x;
            if (page[x] < 0 || (r & (box - 1)) != 0) continue;
            const int row = (j0 + r) & ((1 << P.c.page_shift) - 1);
            const uint32_t dst = stage + (keys ? 0 : C::RAW) + r * C::BROWB;
#pragma unroll
            for (int b = 0; b < C::BLKS; ++b) {
                tma4(dst + b * C::BLOCK, map, b * (C::D / C::BLKS), row, w.h, page[x], bar);
            }
        }
    }
    // Finds the first tile; false if the stretch has none.
    __device__ __forceinline__ bool begin(W& w) {
        if (keys && lane == 0) P.split[blockIdx.x].last = -1;
        if (w.few()) w.find_few(lane);
        w.s = w.sequence();
        if (!w.seek()) return false;
        if (keys && lane == 0) w.tell_join(P.split + blockIdx.x);
        look(w);
        return true;
    }
    // Tiles from the one that the walk stands at.  free(t): waits until stage, queries and meta of tile t
    // may be overwritten; at(t): puts it there.
    template <typename Free, typename Put>
    __device__ __forceinline__ bool run(W& w, Free free, Put at) {
        for (int t = 0;; ++t) {
            if (!free(t)) return false;
            at(t);
            if (!w.next()) return true;
            if (keys && w.i == 0 && lane == 0) w.tell_join(P.split + blockIdx.x);
            look(w);
        }
    }
};

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Adds up the partial triples of the items that lie across stretches.  CTA (w, y): rows 8 y .. + 7 of the
// item that starts in worker w's stretch and goes on.  A warp has one row and, with fewer than 8 rows,
// every 8 / rows-th part of it.
constexpr int kJoinWarps = 8;

template <int D, typename T, typename TC, int ROWS>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ Params P) {
    constexpr int E = D / 32;
    __shared__ float sm[kJoinWarps], sl[kJoinWarps], sacc[kJoinWarps][D];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, w0 = blockIdx.x;
    kda_grid_wait();
    const Split s = P.split[w0];
    const int here = min(s.nq * P.group - s.block * ROWS, ROWS) - kJoinWarps * (int)blockIdx.y;   // rows from this CTA's first on
    if (s.last < 0 || here <= 0) return;
    const int rows = min(here, kJoinWarps), slices = kJoinWarps / rows, row = w % rows, slice = w / rows;
    const int lr = kJoinWarps * blockIdx.y + row, parts = s.last - w0 + 1;
    const size_t size = (size_t)ROWS * (D + 2);
    // part x: the second slot of worker w0, then the first slots of the workers behind it
    auto part = [&](int x) { return P.partial + (x == 0 ? 2 * w0 + 1 : 2 * (w0 + x)) * size; };
    float m = -INFINITY, l = 0.f, acc[E] = {};
    if (slice < slices) {
        for (int x0 = slice; x0 < parts; x0 += 32 * slices) {   // 32 parts at a time: a lane looks at one's statistics
            const int x = x0 + lane * slices;
            const float mx = x < parts ? part(x)[lr] : -INFINITY, lx = x < parts ? part(x)[ROWS + lr] : 0.f;
            const float top = fmaxf(m, warp_max(mx)), f = m == -INFINITY ? 0.f : ex2(m - top);
            const float wt = mx == -INFINITY ? 0.f : ex2(mx - top);
            float sum = lx * wt;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l = l * f + sum;
            m = top;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] *= f;
            const int n = min(32, (parts - x0 + slices - 1) / slices);
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const float wi = __shfl_sync(0xffffffffu, wt, i);
                const float* from = part(x0 + i * slices) + 2 * ROWS + lr * D + lane * E;
                float v[E];
                if constexpr (E == 4) {
                    const float2 a = reinterpret_cast<const float2*>(from)[0], c = reinterpret_cast<const float2*>(from)[1];
                    v[0] = a.x; v[1] = a.y; v[2] = c.x; v[3] = c.y;
                } else {
                    const float2 a = *reinterpret_cast<const float2*>(from);
                    v[0] = a.x; v[1] = a.y;
                }
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += wi * v[e];
            }
        }
        if (lane == 0) { sm[w] = m; sl[w] = l; }
#pragma unroll
        for (int e = 0; e < E; ++e) sacc[w][lane * E + e] = acc[e];
    }
    __syncthreads();
    if (slice > 0) return;
    for (int x = 1; x < slices; ++x) {
        const int o = x * rows + row;
        const float top = fmaxf(m, sm[o]), f1 = m == -INFINITY ? 0.f : ex2(m - top), f2 = sm[o] == -INFINITY ? 0.f : ex2(sm[o] - top);
        l = l * f1 + sl[o] * f2;
        m = top;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * f1 + sacc[o][lane * E + e] * f2;
    }
    const int r = s.block * ROWS + lr, tok = r / P.group;
    const int64_t at = (s.t0 + tok) * P.Hq + s.h * P.group + (r - tok * P.group);
    const float vs = sizeof(TC) == 1 && P.c.v_scale ? P.c.v_scale[s.h] : 1.f;
    const float f = l == 0.f ? 0.f : vs / l;
#pragma unroll
    for (int e = 0; e < E; ++e) static_cast<T*>(P.out)[at * D + lane * E + e] = from_f32<T>(acc[e] * f);
    if (lane == 0 && P.lse) P.lse[at] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
}

// Query rows that a CTA takes at a time: the least instance that holds all that a kv head may have by max_q, so that
// keys and values are read once; 64 (8 in fp32) where none does, and then once for every block.  4 rows as 32 took
// 17.4 us instead of 15.2 over 8 short sequences, 64 rows in two blocks of 32 152 us instead of 119; one row of fp32 as
// two (16 x 4,096 keys, 8 heads of 128) 112 us instead of 89.  Above the instances (32 x 8,192 bf16 keys): 64 rows 264 us,
// 128 rows 511; fp32 (16 x 4,096 keys): 8 rows 242 us, 16 rows 464, 64 rows 1,810.  The call's lengths are on the
// device, so a max_q above them costs: 8 heads a group with one new token 168 us with max_q = 1, 231 with 16.
inline int block_rows(bool f32, int rows) {
    return f32 ? (rows == 1 ? 1 : rows == 2 ? 2 : 8) : (rows <= 16 ? 16 : rows <= 32 ? 32 : 64);
}
inline size_t header_bytes() { return (sizeof(Split) * kWorkers + 255) & ~(size_t)255; }
inline size_t workspace_bytes(int D, int rows) {
    return header_bytes() + (size_t)kWorkers * 2 * block_rows(false, rows) * (D + 2) * 4;
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// cuTensorMapEncodeTiled through the runtime's driver entry point (no link against libcuda).
inline EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess && q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeFn>(p);
        return static_cast<EncodeFn>(nullptr);
    }();
    return fn;
}

// The maps of the caches (channels, rows of a page, heads, pages) and of the queries (channels,
// heads, tokens) for a kernel of layout C.
template <typename C>
bool make_maps(Params& P, int64_t D, int esz, CUtensorMapDataType type, CUtensorMapDataType qtype) {
    const EncodeFn encode = encode_fn();
    if (!encode) return false;
    int box = P.c.page_shift;
    while ((1 << box) > C::TOK) --box;
    P.box_shift = box;
    const cuuint64_t one = (cuuint64_t)D * esz;   // a stride that no coordinate uses
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)1 << P.c.page_shift, (cuuint64_t)P.c.Hkv, (cuuint64_t)std::max(P.c.num_pages, 1)};
    const cuuint64_t strides[3] = {dims[1] > 1 ? (cuuint64_t)P.c.row_stride * esz : one, dims[2] > 1 ? (cuuint64_t)P.c.head_stride * esz : one,
                                   dims[3] > 1 ? (cuuint64_t)P.c.page_stride * esz : one};
    const cuuint32_t boxes[4] = {(cuuint32_t)(D / C::BLKS), 1u << box, 1, 1}, ones[4] = {1, 1, 1, 1};
    const CUtensorMapSwizzle swizzle = C::BROWB == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    if (C::BROWB << box < 128) return false;   // a box lands at a multiple of 128 bytes
    for (int x = 0; x < 2; ++x)
        // without pages nothing is read
        if (encode(x ? &P.v_map : &P.k_map, type, 4, P.c.num_pages == 0 ? const_cast<void*>(P.q) : x ? P.c.v : P.c.k, dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    const int qsz = qtype == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2;
    const cuuint64_t qdims[3] = {(cuuint64_t)D, (cuuint64_t)P.Hq, (cuuint64_t)P.total};
    const cuuint64_t qstrides[2] = {(cuuint64_t)D * qsz, (cuuint64_t)(P.total > 1 ? P.q_stride : P.Hq * D) * qsz};
    const cuuint32_t qbox[3] = {(cuuint32_t)(D / C::QBLKS), 1, 1};
    return encode(&P.q_map, qtype, 3, const_cast<void*>(P.q), qdims, qstrides, qbox, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  C::QSWIZZLED ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The attention kernel (one CTA per worker), then the join.
template <int D, typename T, typename TC, int ROWS, typename Kernel>
cudaError_t launch_pair(Kernel kern, int threads, int bytes, const Params& P, cudaStream_t stream) {
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err != cudaSuccess) return err;
    err = kda_launch_chained(kern, dim3(kWorkers), (unsigned)threads, (size_t)bytes, stream, P);
    if (err != cudaSuccess) return err;
    const dim3 grid(kWorkers, (unsigned)(std::min(P.group * P.max_q, ROWS) + kJoinWarps - 1) / kJoinWarps);
    return kda_launch_chained(join_kernel<D, T, TC, ROWS>, grid, 32 * kJoinWarps, (size_t)0, stream, P);
}

}  // namespace attend
}  // namespace kda
