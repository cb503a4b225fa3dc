// Softmax attention of the newest tokens over the paged cache: what the kernels share.
//
// Per query row, in one pass over its visible keys with the running maximum m, the sum l and
// the weighted values acc (scores in units of log 2, so that e^x is one ex2):
//   m' = max(m, s_j);  l' = l 2^{m - m'} + 2^{s_j - m'};  acc' = acc 2^{m - m'} + 2^{s_j - m'} v_j.
// Two such triples over different keys join the same way, which is how a sequence is split.
//
// Bound by the cache's bytes: a key and a value row serve the G = Hq / Hkv query heads of
// their group and the sequence's new tokens (G x tokens rows), 4 D flops per row for 2 D
// elements.  So the work is cut by bytes alone: all (sequence, kv head, row block) items are laid
// end to end in tiles of keys, and each of 148 CTAs (one per SM) takes one equal stretch of that
// line, whatever the lengths.  A CTA's loader warps walk the stretch and stream its tiles through
// a ring of shared-memory stages; the other warps follow.  Items that lie within one stretch are
// finished there; the others leave a partial triple per stretch, which the join kernel adds up.
//
// The rows of a tile are fetched with 16-byte cp.async, not with TMA boxes: a page may hold one
// row only and end anywhere in a tile, rows that no token sees are not read at all (they are
// filled with zeros, so that what the cache holds there cannot reach a product), and e4m3 rows
// have to pass through registers anyway.  It costs about 650 issue slots of the 10,800 in which
// an SM's share of the memory bandwidth brings a tile.
#pragma once

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
    float* partial;    // two partial triples per worker: of the item that began before it, and of the one that goes on
};

constexpr int kWorkers = 148;      // one CTA per SM
constexpr int kGroups = 1024;      // entries of the table of work in shared memory
constexpr int kMaxSmem = 232448;   // dynamic shared memory of a CTA
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// The running maximum follows the scores only when they exceed it by 2^8: until then weights are
// up to 2^8, which fp32 sums, bf16 and fp16 weights hold as well, and acc is not rescaled.
constexpr float kSlack = 8.f;

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
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
    // a row that is not to be read is filled with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Barrier ID of `count` threads that tells all of them whether `p` holds for any.
template <int ID> __device__ __forceinline__ bool bar_any(bool p, uint32_t count) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred a, b;\n\t"
        "setp.ne.u32 a, %1, 0;\n\t"
        "barrier.cta.red.or.pred b, %2, %3, a;\n\t"
        "selp.u32 %0, 1, 0, b;\n\t}"
        : "=r"(r) : "r"((uint32_t)p), "n"(ID), "r"(count) : "memory");
    return r != 0;
}

// What the loaders tell the other warps of a tile.
struct Meta {
    int64_t t0;
    int32_t j0;          // first key
    int32_t flags;       // kFirst ..
    int32_t h, block, rows, nq, pos0, start;
    int32_t all_lo;      // keys all_lo .. pos0 are seen by every token
    int32_t item;        // count of items in this stretch
    int32_t part;        // where the item's triple goes: -1 (finished here) or a slot of P.partial
    int32_t pad[3];
};
static_assert(sizeof(Meta) == 64, "laid out in shared memory");
enum : int32_t { kFirst = 1, kLast = 2, kEdge = 4 };   // first, last tile of the item here; not all keys seen by all

// The stretch of tiles of this worker, and the walk along it.
template <int TOK, int ROWS>
struct Walk {
    const Params& P;
    int64_t begin, end, at, per;
    int64_t base;       // where sequence n begins
    int n, item;
    Seq s;
    int h, block, tile, tiles, i;   // the item here: its tiles [tile, tile + tiles), the i-th of them is next
    bool starts, ends;              // whether it begins and ends in this stretch

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
                    mine[x] += (int64_t)q.tiles * q.blocks * P.c.Hkv;
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
        const int64_t total = work[groups];
        per = max((total + kWorkers - 1) / kWorkers, (int64_t)1);
        begin = min((int64_t)blockIdx.x * per, total);
        end = min(begin + per, total);
        at = begin;
        int gr = 0;   // the group that holds `at`: the last with work[gr] <= at
        for (int lo = 0, hi = groups - 1; lo <= hi;) {
            const int mid = (lo + hi) >> 1;
            if (work[mid] <= at) { gr = mid; lo = mid + 1; } else hi = mid - 1;
        }
        n = gr * per_group;
        base = work[gr];
        item = -1;
        __syncthreads();
    }
    // The item that holds `at` < end.
    __device__ __forceinline__ void seek() {
        int64_t items = (int64_t)s.blocks * P.c.Hkv;
        while (at - base >= items * s.tiles) {
            base += items * s.tiles;
            ++n;
            s = seq_info<TOK>(P, n, ROWS);
            items = (int64_t)s.blocks * P.c.Hkv;
        }
        const int64_t a = base + (at - base) / s.tiles * s.tiles, b = a + s.tiles;
        const int x = (int)((at - base) / s.tiles);
        h = x / s.blocks;
        block = x - h * s.blocks;
        tile = s.tile0 + (int)(at - a);
        tiles = (int)(min(b, end) - at);
        starts = a >= begin;
        ends = b <= end;
        last_worker = (int)((b - 1) / per);
        i = 0;
        ++item;
    }
    int last_worker;

    __device__ __forceinline__ int j0() const { return (tile + i) * TOK; }
    __device__ __forceinline__ void next() {
        ++at;
        if (++i == tiles && at < end) seek();
    }
    __device__ __forceinline__ void fill(Meta* m) const {
        const int j = j0(), all_lo = first_key(P, s.start, s.pos0 + s.nq - 1);
        const bool inside = j >= all_lo && j + TOK - 1 <= min(s.pos0, s.hi - 1);
        m->t0 = s.t0;
        m->j0 = j;
        m->flags = (i == 0 ? kFirst : 0) | (i == tiles - 1 ? kLast : 0) | (inside ? 0 : kEdge);
        m->h = h;
        m->block = block;
        m->rows = min(ROWS, s.nq * P.group - block * ROWS);
        m->nq = s.nq;
        m->pos0 = s.pos0;
        m->start = s.start;
        m->all_lo = all_lo;
        m->item = item;
        m->part = starts && ends ? -1 : 2 * (int)blockIdx.x + (starts ? 1 : 0);
    }
    __device__ __forceinline__ void tell_join(Split* to) const {
        if (starts && !ends) *to = {s.t0, h, block, s.nq, last_worker};
    }
};

// A loader lane's place in the cache for the tile that is issued next.
struct Place {
    const char *kb, *vb;
    const int32_t* table;
    int page;

    template <typename W>
    __device__ __forceinline__ void item(const Params& P, const W& w, int esz) {
        const int64_t off = w.h * P.c.head_stride * esz;
        kb = static_cast<const char*>(P.c.k) + off;
        vb = static_cast<const char*>(P.c.v) + off;
        table = P.c.table + w.n * P.c.table_stride;
    }
    template <typename W>
    __device__ __forceinline__ void look(const Params& P, const W& w, int row, bool has) {
        const int j = w.j0() + row;
        page = -1;
        if (has && j >= w.s.lo && j < w.s.hi) page = __ldg(table + (j >> P.c.page_shift));
    }
    // The lane's row: whether it is read, and its byte offset.
    template <typename W>
    __device__ __forceinline__ bool row(const Params& P, const W& w, int row, bool has, int esz, int64_t& off) const {
        const int j = w.j0() + row;
        const bool wanted = has && j >= w.s.lo && j < w.s.hi;
        const bool ok = wanted && page >= 0 && page < P.c.num_pages;
        if (wanted && !ok) kda_set_status(KDA_ERR_BAD_PAGE);
        off = ok ? (page * P.c.page_stride + (j & ((1 << P.c.page_shift) - 1)) * P.c.row_stride) * esz : 0;
        return ok;
    }
};

// Adds up the partial triples of the items that lie across stretches.  CTA (w, row): the item
// that starts in worker w's stretch and goes on; groups of D threads share its parts.
constexpr int kJoinThreads = 256;

template <int D, typename T, typename TC, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Params P) {
    constexpr int GROUPS = kJoinThreads / D;
    __shared__ float wt[kWorkers], sacc[GROUPS][D], red[kJoinThreads / 32], tot[2];
    const int tid = threadIdx.x, lane = tid & 31, lr = blockIdx.y, w0 = blockIdx.x;
    kda_grid_wait();
    const Split s = P.split[w0];
    const int r = s.block * ROWS + lr, parts = s.last - w0 + 1;
    if (s.last < 0 || r >= s.nq * P.group) return;
    const size_t size = (size_t)ROWS * (D + 2);
    // part x: the second slot of worker w0, then the first slots of the workers behind it
    auto part = [&](int x) { return P.partial + (x == 0 ? 2 * w0 + 1 : 2 * (w0 + x)) * size; };
    float m = -INFINITY, l = 0.f;
    if (tid < parts) { m = part(tid)[lr]; l = part(tid)[ROWS + lr]; }   // parts <= kWorkers < kJoinThreads
    float top = warp_max(m);
    if (lane == 0) red[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kJoinThreads / 32; ++x) top = x == 0 ? red[0] : fmaxf(top, red[x]);
    const float f = m == -INFINITY ? 0.f : ex2(m - top);
    if (tid < parts) wt[tid] = f;
    float sum = l * f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if (lane == 0) red[tid >> 5] = sum;
    __syncthreads();
    if (tid == 0) {
        float t = 0.f;
        for (int x = 0; x < kJoinThreads / 32; ++x) t += red[x];
        tot[0] = t;
    }
    const int d = tid % D, g = tid / D;
    float acc = 0.f;
#pragma unroll 8
    for (int x = g; x < parts; x += GROUPS) acc += wt[x] * part(x)[2 * ROWS + lr * D + d];
    sacc[g][d] = acc;
    __syncthreads();
    const float lt = tot[0];
    const int tok = r / P.group;
    const int64_t at = (s.t0 + tok) * P.Hq + s.h * P.group + (r - tok * P.group);
    if (g == 0) {
#pragma unroll
        for (int x = 1; x < GROUPS; ++x) acc += sacc[x][d];
        const float vs = sizeof(TC) == 1 && P.c.v_scale ? P.c.v_scale[s.h] : 1.f;
        static_cast<T*>(P.out)[at * D + d] = from_f32<T>(acc * (lt == 0.f ? 0.f : vs / lt));
    }
    if (tid == 0 && P.lse) P.lse[at] = lt == 0.f ? -INFINITY : top * kLn2 + logf(lt);
}

// Query rows that a CTA takes at a time.
inline int block_rows(bool f32, int rows) {
    return f32 ? (rows <= 2 ? 2 : 8) : (rows <= 16 ? 16 : rows <= 32 ? 32 : 64);
}
inline size_t header_bytes() { return (sizeof(Split) * kWorkers + 255) & ~(size_t)255; }
inline size_t workspace_bytes(int D, int rows) {
    return header_bytes() + (size_t)kWorkers * 2 * block_rows(false, rows) * (D + 2) * 4;
}

// The attention kernel (one CTA per worker), then the join.
template <int D, typename T, typename TC, int ROWS, typename Kernel>
cudaError_t launch_pair(Kernel kern, int threads, int bytes, const Params& P, cudaStream_t stream) {
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err != cudaSuccess) return err;
    kern<<<kWorkers, threads, bytes, stream>>>(P);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kWorkers, (unsigned)(P.group * P.max_q < ROWS ? P.group * P.max_q : ROWS));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<D, T, TC, ROWS>, P);
}

}  // namespace attend
}  // namespace kda
