// libkda C-ABI: argument checking, workspace sizing and dispatch to the kernels.
// Everything here is host code; the kernels live in the included .cuh files so the
// whole library is one translation unit (one device status word, no relocatable code).
#include <stdint.h>
#include <string.h>

#include <mutex>

#include "libkda.h"
#include "kda_common.cuh"
#include "kda_decode.cuh"
#include "kda_decode_pool.cuh"
#include "kda_kv_append.cuh"
#include "kda_kv_decode_tc.cuh"
#include "kda_prefill_simt.cuh"
#include "kda_prefill_tc.cuh"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool supported_dim(int32_t dk, int32_t dv) { return dk == dv && (dk == 64 || dk == 128); }

// bf16 runs on the tensor cores (d = 64 as the first 64 channels of a 128-channel problem);
// fp32 on CUDA cores.
bool tensor_core_path(kda_dtype dt, int32_t dk) { return dt == KDA_BF16 && (dk == 128 || dk == 64); }

bool valid_chunk(kda_dtype dt, int32_t C) {
    if (dt == KDA_BF16) return C == 64;
    return C == 16 || C == 32 || C == 64;
}

template <typename T>
cudaError_t dispatch_simt(int32_t dk, int32_t C, const void* q, const void* k, const void* v,
                          const float* g, const float* beta, const float* s0, const int32_t* cu,
                          int num_seqs, int64_t total, int H, void* out, float* sf,
                          cudaStream_t st, uint32_t in_flags) {
#define KDA_SIMT_CASE(D, CC)                                                                  \
    if (dk == D && C == CC)                                                                   \
        return kda::launch_prefill_simt<T, D, CC>(q, k, v, g, beta, s0, cu, num_seqs, total, H, \
                                                  out, sf, st, in_flags);
    KDA_SIMT_CASE(64, 16) KDA_SIMT_CASE(64, 32) KDA_SIMT_CASE(64, 64)
    KDA_SIMT_CASE(128, 16) KDA_SIMT_CASE(128, 32) KDA_SIMT_CASE(128, 64)
#undef KDA_SIMT_CASE
    return cudaErrorInvalidValue;
}

}  // namespace

extern "C" {

int32_t kda_abi_version(void) { return 8; }

const char* kda_status_string(kda_status s) {
    switch (s) {
        case KDA_OK: return "ok";
        case KDA_ERR_INVALID_ARG: return "invalid argument";
        case KDA_ERR_UNSUPPORTED: return "unsupported problem size or chunk size";
        case KDA_ERR_CUDA: return "CUDA runtime error";
        case KDA_ERR_TIMEOUT: return "a bounded device wait expired";
        case KDA_ERR_BAD_SEQLENS: return "cu_seqlens inconsistent with total_tokens";
        case KDA_ERR_BAD_EMIT_POS: return "an emission position is not a chunk boundary of a sequence";
        case KDA_ERR_BAD_PAGE: return "a cache position outside the block table, or a page outside the cache";
        case KDA_ERR_BAD_SLOT: return "a state slot outside the pool";
    }
    return "unknown status";
}

size_t kda_prefill_workspace_size(int64_t total_tokens, int32_t num_seqs, int32_t H, int32_t dk,
                                  int32_t dv, int32_t C, kda_dtype dt) {
    if (total_tokens < 0 || num_seqs < 0 || H <= 0 || !supported_dim(dk, dv) ||
        !valid_chunk(dt, C))
        return 0;
    if (!tensor_core_path(dt, dk)) return 0;
    size_t bytes = 0;
    return kda::tc::workspace_bytes_checked(total_tokens, num_seqs, H, &bytes) ? bytes : 0;
}

size_t kda_prefill_workspace_size_min(int64_t total_tokens, int32_t num_seqs, int32_t H, int32_t dk,
                                      int32_t dv, int32_t C, kda_dtype dt) {
    if (kda_prefill_workspace_size(total_tokens, num_seqs, H, dk, dv, C, dt) == 0) return 0;
    return kda::tc::workspace_bytes_min(total_tokens, num_seqs, H);
}

int64_t kda_prefill_windows(int64_t total_tokens, int32_t num_seqs, int32_t H, int32_t dk, int32_t dv,
                            int32_t C, kda_dtype dt, size_t ws_bytes) {
    if (total_tokens < 0 || num_seqs < 0 || H <= 0 || !supported_dim(dk, dv) || !valid_chunk(dt, C))
        return -1;
    if (!tensor_core_path(dt, dk) || num_seqs == 0) return 1;
    if (kda_prefill_workspace_size(total_tokens, num_seqs, H, dk, dv, C, dt) == 0) return -1;
    const int64_t w = kda::tc::window_chunks(total_tokens, num_seqs, H, ws_bytes);
    if (w <= 0) return -1;
    const int64_t mc = kda::tc::max_chunks(total_tokens, num_seqs);
    return w >= mc ? 1 : (mc + w - 1) / w;
}

int32_t kda_prefill_launches(int64_t total_tokens, int32_t num_seqs, int32_t H, int32_t dk,
                             int32_t dv, int32_t C, kda_dtype dt, uint32_t in_flags, int32_t num_emit) {
    if (total_tokens < 0 || num_seqs < 0 || H <= 0 || !supported_dim(dk, dv) || !valid_chunk(dt, C))
        return -1;
    if (num_seqs == 0) return 0;
    if (!tensor_core_path(dt, dk)) return 1;
    // chunk table, [recurrence order of several sequences], [emission slots], preparation,
    // strongly decayed chunks, recurrence
    int32_t n = 1 + (num_seqs > 1 ? 1 : 0) + (num_emit > 0 ? 1 : 0) + (total_tokens > 0 ? 2 : 0) + 1;
    if (!(in_flags & KDA_IN_SERIAL_CHAINS) && kda::tc::scan_segment_chunks(total_tokens, num_seqs, H) > 0)
        n += 3;   // segment table, segment transitions, starting states
    return n;
}

// A tensor-core problem whose workspace or launch grids cannot be addressed (see
// workspace_bytes_checked) is rejected before anything is launched.
static bool tc_problem_fits(int64_t total_tokens, int32_t num_seqs, int32_t H) {
    size_t bytes = 0;
    return kda::tc::workspace_bytes_checked(total_tokens, num_seqs, H, &bytes);
}

static kda_status prefill_common(const void* q, const void* k, const void* v, const float* g,
                                 const float* beta, const float* initial_state,
                                 const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                                 int32_t H, int32_t dk, int32_t dv, kda_dtype dt, void* out,
                                 float* final_state, int32_t C, const int64_t* emit_pos,
                                 int32_t num_emit, float* emit_states, void* workspace,
                                 size_t ws_bytes, kda_stream_t stream, uint32_t in_flags) {
    if (num_seqs < 0 || total_tokens < 0 || H <= 0 || dk <= 0 || dv <= 0 || num_emit < 0)
        return KDA_ERR_INVALID_ARG;
    if (in_flags & ~(uint32_t)(KDA_IN_NORMALIZE_QK | KDA_IN_G_LOGITS | KDA_IN_BETA_LOGITS |
                               KDA_IN_G_SCALAR | KDA_IN_STRONG_DECAY | KDA_IN_SERIAL_CHAINS))
        return KDA_ERR_INVALID_ARG;
    if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (total_tokens > INT32_MAX) return KDA_ERR_UNSUPPORTED;  // cu_seqlens is int32
    if (!supported_dim(dk, dv) || !valid_chunk(dt, C)) return KDA_ERR_UNSUPPORTED;
    if (num_emit > 0) {
        if (!emit_pos || !emit_states || (reinterpret_cast<uintptr_t>(emit_pos) & 7u) != 0 ||
            !aligned16(emit_states) || num_seqs == 0)
            return KDA_ERR_INVALID_ARG;
        if (!tensor_core_path(dt, dk)) return KDA_ERR_UNSUPPORTED;
    }
    if (tensor_core_path(dt, dk) && !tc_problem_fits(total_tokens, num_seqs, H)) return KDA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return KDA_OK;
    if (!cu_seqlens) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!q || !k || !v || !g || !beta || !out)) return KDA_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, g, beta, out, initial_state, final_state};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0) return KDA_ERR_INVALID_ARG;
    // A workspace below the full size runs the chunks in windows (window_chunks), down to
    // kda_prefill_workspace_size_min.
    const size_t need = kda_prefill_workspace_size_min(total_tokens, num_seqs, H, dk, dv, C, dt);
    if (ws_bytes < need || (need > 0 && (!workspace ||
                                         (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)))
        return KDA_ERR_INVALID_ARG;
    int64_t window = INT64_MAX;
    if (tensor_core_path(dt, dk) && need > 0) {
        window = kda::tc::window_chunks(total_tokens, num_seqs, H, ws_bytes);
        if (window <= 0) return KDA_ERR_INVALID_ARG;
    }

    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t err;
    if (tensor_core_path(dt, dk))
        err = kda::tc::launch_prefill(q, k, v, g, beta, initial_state, cu_seqlens, num_seqs,
                                      total_tokens, H, out, final_state, workspace, st, emit_pos,
                                      num_emit, emit_states, in_flags, window, dk);
    else if (dt == KDA_F32)
        err = dispatch_simt<float>(dk, C, q, k, v, g, beta, initial_state, cu_seqlens, num_seqs,
                                   total_tokens, H, out, final_state, st, in_flags);
    else
        return KDA_ERR_UNSUPPORTED;   // unreachable: every bf16 problem takes the tensor cores
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_prefill(const void* q, const void* k, const void* v, const float* g,
                       const float* beta, const float* initial_state, const int32_t* cu_seqlens,
                       int32_t num_seqs, int64_t total_tokens, int32_t H, int32_t dk, int32_t dv,
                       kda_dtype dt, void* out, float* final_state, int32_t C, void* workspace,
                       size_t ws_bytes, kda_stream_t stream) {
    return prefill_common(q, k, v, g, beta, initial_state, cu_seqlens, num_seqs, total_tokens, H, dk,
                          dv, dt, out, final_state, C, nullptr, 0, nullptr, workspace, ws_bytes, stream,
                          0u);
}

kda_status kda_prefill_gdn(const void* q, const void* k, const void* v, const float* g,
                           const float* beta, const float* initial_state, const int32_t* cu_seqlens,
                           int32_t num_seqs, int64_t total_tokens, int32_t H, int32_t dk, int32_t dv,
                           kda_dtype dt, void* out, float* final_state, int32_t C, void* workspace,
                           size_t ws_bytes, kda_stream_t stream) {
    return prefill_common(q, k, v, g, beta, initial_state, cu_seqlens, num_seqs, total_tokens, H, dk,
                          dv, dt, out, final_state, C, nullptr, 0, nullptr, workspace, ws_bytes, stream,
                          (uint32_t)KDA_IN_G_SCALAR);
}

kda_status kda_prefill_ex(const void* q, const void* k, const void* v, const float* g,
                          const float* beta, const float* initial_state, const int32_t* cu_seqlens,
                          int32_t num_seqs, int64_t total_tokens, int32_t H, int32_t dk, int32_t dv,
                          kda_dtype dt, void* out, float* final_state, int32_t C, uint32_t in_flags,
                          const int64_t* emit_pos, int32_t num_emit, float* emit_states,
                          void* workspace, size_t ws_bytes, kda_stream_t stream) {
    return prefill_common(q, k, v, g, beta, initial_state, cu_seqlens, num_seqs, total_tokens, H, dk,
                          dv, dt, out, final_state, C, emit_pos, num_emit, emit_states, workspace,
                          ws_bytes, stream, in_flags);
}

kda_status kda_prefill_emit(const void* q, const void* k, const void* v, const float* g,
                            const float* beta, const float* initial_state,
                            const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                            int32_t H, int32_t dk, int32_t dv, kda_dtype dt, void* out,
                            float* final_state, int32_t C, const int64_t* emit_pos,
                            int32_t num_emit, float* emit_states, void* workspace,
                            size_t ws_bytes, kda_stream_t stream) {
    return prefill_common(q, k, v, g, beta, initial_state, cu_seqlens, num_seqs, total_tokens, H, dk,
                          dv, dt, out, final_state, C, emit_pos, num_emit, emit_states, workspace,
                          ws_bytes, stream, 0u);
}

// Checks shared by the staged tensor-core entry points.
static kda_status check_staged(const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                               int32_t H, int32_t dk, int32_t dv, kda_dtype dt, int32_t C,
                               const void* workspace, size_t ws_bytes) {
    if (num_seqs < 0 || total_tokens < 0 || H <= 0 || dk <= 0 || dv <= 0) return KDA_ERR_INVALID_ARG;
    if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (total_tokens > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (!tensor_core_path(dt, dk) || !supported_dim(dk, dv) || !valid_chunk(dt, C))
        return KDA_ERR_UNSUPPORTED;
    if (!tc_problem_fits(total_tokens, num_seqs, H)) return KDA_ERR_UNSUPPORTED;
    if (num_seqs > 0 && (!cu_seqlens || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0))
        return KDA_ERR_INVALID_ARG;
    const size_t need = kda_prefill_workspace_size(total_tokens, num_seqs, H, dk, dv, C, dt);
    if (ws_bytes < need || !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

kda_status kda_prefill_prepare(const void* q, const void* k, const void* v, const float* g,
                               const float* beta, const int32_t* cu_seqlens, int32_t num_seqs,
                               int64_t total_tokens, int32_t H, int32_t dk, int32_t dv,
                               kda_dtype dt, int32_t C, void* workspace, size_t ws_bytes,
                               kda_stream_t stream) {
    kda_status st = check_staged(cu_seqlens, num_seqs, total_tokens, H, dk, dv, dt, C, workspace, ws_bytes);
    if (st != KDA_OK || num_seqs == 0) return st;
    if (total_tokens > 0 && (!q || !k || !v || !g || !beta)) return KDA_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, g, beta};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_INVALID_ARG;
    return kda::tc::launch_prepare(q, k, v, g, beta, cu_seqlens, num_seqs, total_tokens, H, workspace,
                                   reinterpret_cast<cudaStream_t>(stream), nullptr, 0, 0u, dk) == cudaSuccess
               ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_prefill_scan(const float* initial_state, float* final_state, void* out,
                            const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                            int32_t H, int32_t dk, int32_t dv, kda_dtype dt, int32_t C,
                            void* workspace, size_t ws_bytes, kda_stream_t stream) {
    kda_status st = check_staged(cu_seqlens, num_seqs, total_tokens, H, dk, dv, dt, C, workspace, ws_bytes);
    if (st != KDA_OK || num_seqs == 0) return st;
    if ((initial_state && !aligned16(initial_state)) || (final_state && !aligned16(final_state)))
        return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!out || !aligned16(out))) return KDA_ERR_INVALID_ARG;
    return kda::tc::launch_scan(initial_state, final_state, out, num_seqs, total_tokens, H,
                                workspace, reinterpret_cast<cudaStream_t>(stream), nullptr, 0u, dk) == cudaSuccess
               ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_selftest_bounded_wait(uint64_t limit_ns, kda_stream_t stream) {
    if (limit_ns < 1000ull || limit_ns > 2000000000ull) return KDA_ERR_INVALID_ARG;
    kda::tc::selftest_wait_kernel<<<1, 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(limit_ns);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

static kda_status decode_common(const void* q, const void* k, const void* v, const float* g,
                                const float* beta, float* state_inout, void* out, int32_t N, int32_t H,
                                int32_t dk, int32_t dv, kda_dtype dt, kda_stream_t stream, uint32_t in_flags) {
    if (N < 0 || H <= 0 || dk <= 0 || dv <= 0) return KDA_ERR_INVALID_ARG;
    if (in_flags & ~(uint32_t)(KDA_IN_NORMALIZE_QK | KDA_IN_G_LOGITS | KDA_IN_BETA_LOGITS |
                               KDA_IN_G_SCALAR | KDA_IN_STRONG_DECAY | KDA_IN_SERIAL_CHAINS))
        return KDA_ERR_INVALID_ARG;
    in_flags &= ~(uint32_t)(KDA_IN_STRONG_DECAY | KDA_IN_SERIAL_CHAINS);   // no effect on one token
    if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (!supported_dim(dk, dv)) return KDA_ERR_UNSUPPORTED;
    if (N == 0) return KDA_OK;
    if ((int64_t)N * H > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (!q || !k || !v || !g || !beta || !state_inout || !out) return KDA_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, g, beta, state_inout, out};
    for (const void* p : ptrs)
        if (!aligned16(p)) return KDA_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t err;
    if (dt == KDA_F32)
        err = dk == 64 ? kda::launch_decode<64, float>(q, k, v, g, beta, state_inout, out, N, H, st, in_flags)
                       : kda::launch_decode<128, float>(q, k, v, g, beta, state_inout, out, N, H, st, in_flags);
    else
        err = dk == 64 ? kda::launch_decode<64, __nv_bfloat16>(q, k, v, g, beta, state_inout, out, N, H, st,
                                                               in_flags)
                       : kda::launch_decode<128, __nv_bfloat16>(q, k, v, g, beta, state_inout, out, N, H,
                                                                st, in_flags);
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_decode(const void* q, const void* k, const void* v, const float* g,
                      const float* beta, float* state_inout, void* out, int32_t N, int32_t H,
                      int32_t dk, int32_t dv, kda_dtype dt, kda_stream_t stream) {
    return decode_common(q, k, v, g, beta, state_inout, out, N, H, dk, dv, dt, stream, 0u);
}

kda_status kda_decode_gdn(const void* q, const void* k, const void* v, const float* g,
                          const float* beta, float* state_inout, void* out, int32_t N, int32_t H,
                          int32_t dk, int32_t dv, kda_dtype dt, kda_stream_t stream) {
    return decode_common(q, k, v, g, beta, state_inout, out, N, H, dk, dv, dt, stream,
                         (uint32_t)KDA_IN_G_SCALAR);
}

kda_status kda_decode_ex(const void* q, const void* k, const void* v, const float* g,
                         const float* beta, float* state_inout, void* out, int32_t N, int32_t H,
                         int32_t dk, int32_t dv, kda_dtype dt, uint32_t in_flags, kda_stream_t stream) {
    return decode_common(q, k, v, g, beta, state_inout, out, N, H, dk, dv, dt, stream, in_flags);
}

// ------------------------------------------------------------------------------------------
// The hybrid stack's decode step: the recurrence over a pool of states, the paged cache and
// the attention over it.
namespace {

constexpr int32_t kMaxQ = 16;           // new tokens of a sequence that kda_kv_decode takes
constexpr int32_t kMaxPageSize = 4096;

// A token stride in elements of `elem` bytes: whole 16-byte units, at least the dense size.
bool valid_stride(int64_t stride, int64_t dense, int64_t elem) {
    return stride >= dense && stride <= INT64_MAX / 64 && (stride * elem) % 16 == 0;
}

// What kda_kv_append and kda_kv_decode check alike.
kda_status check_cache(const kda_kv_cache* c, kda_dtype dt, int32_t num_seqs, int64_t total_tokens,
                       const int32_t* cu_seqlens, kda::kv::Cache* out) {
    if (!c || num_seqs < 0 || total_tokens < 0 || c->num_pages < 0 || c->max_pages < 0 || c->Hkv <= 0 ||
        c->D <= 0 || c->page_size <= 0)
        return KDA_ERR_INVALID_ARG;
    if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (c->dt != KDA_F32 && c->dt != KDA_BF16 && c->dt != KDA_E4M3) return KDA_ERR_INVALID_ARG;
    if (total_tokens > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if ((c->D != 64 && c->D != 128) || (c->page_size & (c->page_size - 1)) != 0 || c->page_size > kMaxPageSize)
        return KDA_ERR_UNSUPPORTED;
    if ((dt == KDA_F32) != (c->dt == KDA_F32)) return KDA_ERR_UNSUPPORTED;
    if (!cu_seqlens && num_seqs != total_tokens) return KDA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0) return KDA_ERR_INVALID_ARG;
    if (num_seqs == 0 || total_tokens == 0) return KDA_OK;   // nothing is looked at
    if (!c->seq_lens || (c->max_pages > 0 && !c->block_table) || (c->num_pages > 0 && (!c->k || !c->v)))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(c->k) || !aligned16(c->v)) return KDA_ERR_INVALID_ARG;
    const uintptr_t words[] = {reinterpret_cast<uintptr_t>(c->seq_lens), reinterpret_cast<uintptr_t>(c->block_table),
                               reinterpret_cast<uintptr_t>(c->k_scale), reinterpret_cast<uintptr_t>(c->v_scale)};
    for (uintptr_t p : words)
        if ((p & 3u) != 0) return KDA_ERR_INVALID_ARG;
    if ((c->k_scale || c->v_scale) && c->dt != KDA_E4M3) return KDA_ERR_INVALID_ARG;
    const int64_t elem = c->dt == KDA_F32 ? 4 : c->dt == KDA_BF16 ? 2 : 1;
    if (!valid_stride(c->page_stride, c->D, elem) || !valid_stride(c->head_stride, c->D, elem) ||
        !valid_stride(c->row_stride, c->D, elem) || c->table_stride < c->max_pages)
        return KDA_ERR_INVALID_ARG;
    int shift = 0;
    while ((1 << shift) < c->page_size) ++shift;
    *out = {c->k, c->v, c->k_scale, c->v_scale, c->block_table, c->seq_lens, c->page_stride, c->head_stride,
            c->row_stride, c->table_stride, c->num_pages, shift, c->max_pages, c->Hkv};
    return KDA_OK;
}

// The kernel instance for head size D, the type of q, k, v and the cache's type.
#define KDA_KV_DISPATCH(launch, D, dt, cdt, ...)                                                        \
    (dt == KDA_F32 ? (D == 64 ? launch<64, float, float>(__VA_ARGS__) : launch<128, float, float>(__VA_ARGS__)) \
     : cdt == KDA_BF16                                                                                  \
         ? (D == 64 ? launch<64, __nv_bfloat16, __nv_bfloat16>(__VA_ARGS__)                             \
                    : launch<128, __nv_bfloat16, __nv_bfloat16>(__VA_ARGS__))                           \
         : (D == 64 ? launch<64, __nv_bfloat16, __nv_fp8_e4m3>(__VA_ARGS__)                             \
                    : launch<128, __nv_bfloat16, __nv_fp8_e4m3>(__VA_ARGS__)))

}  // namespace

kda_status kda_decode_pool(const void* q, const void* k, const void* v, const float* g, const float* beta,
                           int64_t q_stride, int64_t k_stride, int64_t v_stride, float* state_pool,
                           int32_t num_slots, const int32_t* slots_in, const int32_t* slots_out,
                           const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens, int32_t Hk,
                           int32_t Hv, int32_t dk, int32_t dv, kda_dtype dt, void* out, uint32_t in_flags,
                           kda_stream_t stream) {
    if (num_seqs < 0 || total_tokens < 0 || num_slots < 0 || Hk <= 0 || Hv <= 0 || dk <= 0 || dv <= 0)
        return KDA_ERR_INVALID_ARG;
    if (in_flags & ~(uint32_t)(KDA_IN_NORMALIZE_QK | KDA_IN_G_LOGITS | KDA_IN_BETA_LOGITS | KDA_IN_G_SCALAR |
                               KDA_IN_STRONG_DECAY | KDA_IN_SERIAL_CHAINS))
        return KDA_ERR_INVALID_ARG;
    if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (Hv % Hk != 0 || (!cu_seqlens && num_seqs != total_tokens)) return KDA_ERR_INVALID_ARG;
    if (!supported_dim(dk, dv) || total_tokens > INT32_MAX || (int64_t)num_seqs * Hv > INT32_MAX)
        return KDA_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0) return KDA_ERR_INVALID_ARG;
    if (num_seqs == 0 || total_tokens == 0) return KDA_OK;
    if (!q || !k || !v || !g || !beta || !slots_in || !slots_out || !out || (num_slots > 0 && !state_pool))
        return KDA_ERR_INVALID_ARG;
    const void* ptrs[] = {q, k, v, state_pool, out};
    for (const void* p : ptrs)
        if (!aligned16(p)) return KDA_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(slots_in) | reinterpret_cast<uintptr_t>(slots_out) |
          reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(beta)) & 3u) != 0)
        return KDA_ERR_INVALID_ARG;
    const int64_t elem = dt == KDA_F32 ? 4 : 2;
    if (!valid_stride(q_stride, (int64_t)Hk * dk, elem) || !valid_stride(k_stride, (int64_t)Hk * dk, elem) ||
        !valid_stride(v_stride, (int64_t)Hv * dv, elem))
        return KDA_ERR_INVALID_ARG;
    const kda::pool::Params P = {q, k, v, g, beta, q_stride, k_stride, v_stride, state_pool, slots_in, slots_out,
                                 cu_seqlens, num_slots, num_seqs, Hk, Hv, total_tokens, out, in_flags};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t err =
        dt == KDA_F32 ? (dk == 64 ? kda::pool::launch<64, float>(P, st) : kda::pool::launch<128, float>(P, st))
                      : (dk == 64 ? kda::pool::launch<64, __nv_bfloat16>(P, st)
                                  : kda::pool::launch<128, __nv_bfloat16>(P, st));
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_kv_append(const void* k, const void* v, const void* q, int64_t k_stride, int64_t v_stride,
                         int64_t q_stride, kda_dtype dt, const kda_kv_cache* cache, const int32_t* cu_seqlens,
                         int32_t num_seqs, int64_t total_tokens, int32_t Hq, const kda_rope* rope, void* q_out,
                         kda_stream_t stream) {
    kda::append::Params P = {};
    const kda_status cs = check_cache(cache, dt, num_seqs, total_tokens, cu_seqlens, &P.c);
    if (cs != KDA_OK) return cs;
    if (Hq < 0) return KDA_ERR_INVALID_ARG;
    if (rope) {
        if (rope->rot_dim <= 0 || rope->rot_dim > cache->D || rope->rot_dim % 16 != 0 || rope->num_axes < 1 ||
            rope->num_axes > 4)
            return KDA_ERR_INVALID_ARG;
        int64_t pairs = 0;
        for (int a = 0; a < 4; ++a) {
            if (a < rope->num_axes && rope->axis_pairs[a] < 0) return KDA_ERR_INVALID_ARG;
            pairs += a < rope->num_axes ? rope->axis_pairs[a] : 0;
            if (pairs > rope->rot_dim / 2) return KDA_ERR_INVALID_ARG;
            P.axis_end[a] = (int32_t)pairs;
        }
        if (pairs != rope->rot_dim / 2) return KDA_ERR_INVALID_ARG;
        P.rot = rope->rot_dim;
        P.adjacent = rope->adjacent != 0;
        P.inv_freq = rope->inv_freq;
        P.positions = rope->positions;
    }
    if (num_seqs == 0 || total_tokens == 0) return KDA_OK;   // empty arrays may have no address
    if (!k || !v || (Hq > 0) != (q != nullptr) || (q && !q_out)) return KDA_ERR_INVALID_ARG;
    if (rope && (!rope->inv_freq || (rope->num_axes > 1 && !rope->positions))) return KDA_ERR_INVALID_ARG;
    const void* ptrs[] = {k, v, q, q_out};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(P.inv_freq) | reinterpret_cast<uintptr_t>(P.positions)) & 3u) != 0)
        return KDA_ERR_INVALID_ARG;
    const int64_t elem = dt == KDA_F32 ? 4 : 2, D = cache->D;
    if (!valid_stride(k_stride, cache->Hkv * D, elem) || !valid_stride(v_stride, cache->Hkv * D, elem) ||
        (q && !valid_stride(q_stride, Hq * D, elem)))
        return KDA_ERR_INVALID_ARG;
    // units of work of one token are counted in 32 bits
    if ((int64_t)(Hq + (int64_t)2 * cache->Hkv) * D > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (q == q_out && q && q_stride != Hq * D) return KDA_ERR_INVALID_ARG;   // in place only when dense
    P.k = k; P.v = v; P.q = q;
    P.k_stride = k_stride; P.v_stride = v_stride; P.q_stride = q_stride;
    P.cu = cu_seqlens; P.num_seqs = num_seqs; P.Hq = Hq; P.total = total_tokens; P.q_out = q_out;
    const cudaError_t err = KDA_KV_DISPATCH(kda::append::launch, cache->D, dt, cache->dt, P,
                                            reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_kv_decode_workspace_size(int32_t num_seqs, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_q) {
    if (num_seqs < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || (D != 64 && D != 128) || max_q < 1 || max_q > kMaxQ)
        return 0;
    return kda::attend::workspace_bytes(D, (Hq / Hkv) * max_q);
}

kda_status kda_kv_decode(const void* q, int64_t q_stride, kda_dtype dt, const kda_kv_cache* cache,
                         const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens, int32_t max_q,
                         int32_t Hq, float scale, float softcap, int32_t window, const float* alibi_slopes,
                         const int32_t* kv_start, void* out, float* lse, void* workspace, size_t ws_bytes,
                         kda_stream_t stream) {
    kda::attend::Params P = {};
    const kda_status cs = check_cache(cache, dt, num_seqs, total_tokens, cu_seqlens, &P.c);
    if (cs != KDA_OK) return cs;
    if (Hq <= 0 || Hq % cache->Hkv != 0 || max_q < 1 || window < 0 || !(softcap >= 0.f) || !(scale - scale == 0.f) ||
        !(softcap - softcap == 0.f))
        return KDA_ERR_INVALID_ARG;
    // scale / softcap has to keep its bits: subnormal ones cost a score up to 2^-150 |q . k| softcap
    if (softcap > 0.f && (softcap < 0x1p-100f || softcap > 0x1p100f)) return KDA_ERR_UNSUPPORTED;
    if (max_q > kMaxQ || Hq > 65535 || (int64_t)num_seqs * max_q > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (cache->dt == KDA_E4M3 && cache->D == 64 && cache->page_size == 1) return KDA_ERR_UNSUPPORTED;   // boxes of 64 bytes
    if (num_seqs == 0 || total_tokens == 0) return KDA_OK;
    if (!q || !out || !aligned16(q) || !aligned16(out)) return KDA_ERR_INVALID_ARG;
    const uintptr_t words[] = {reinterpret_cast<uintptr_t>(alibi_slopes), reinterpret_cast<uintptr_t>(kv_start),
                               reinterpret_cast<uintptr_t>(lse)};
    for (uintptr_t p : words)
        if ((p & 3u) != 0) return KDA_ERR_INVALID_ARG;
    if (!valid_stride(q_stride, (int64_t)Hq * cache->D, dt == KDA_F32 ? 4 : 2)) return KDA_ERR_INVALID_ARG;
    if (ws_bytes < kda_kv_decode_workspace_size(num_seqs, Hq, cache->Hkv, cache->D, max_q) || !workspace ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return KDA_ERR_INVALID_ARG;
    P.q = q; P.q_stride = q_stride; P.cu = cu_seqlens; P.num_seqs = num_seqs; P.Hq = Hq; P.max_q = max_q;
    P.window = window; P.total = total_tokens; P.scale = scale; P.softcap = softcap; P.slopes = alibi_slopes;
    P.kv_start = kv_start; P.out = out; P.lse = lse; P.group = Hq / cache->Hkv;
    P.split = static_cast<kda::attend::Split*>(workspace);
    P.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + kda::attend::header_bytes());
    const cudaError_t err = KDA_KV_DISPATCH(kda::attend::launch, cache->D, dt, cache->dt, P,
                                            reinterpret_cast<cudaStream_t>(stream));
    // strides beyond 2^40 bytes have no TMA map
    return err == cudaSuccess ? KDA_OK : err == cudaErrorNotSupported ? KDA_ERR_UNSUPPORTED : KDA_ERR_CUDA;
}

#ifdef KDA_TRACE
// Trace builds only: copy the first n clock stamps to host memory.
int kda_debug_read_trace(unsigned long long* host, int n) {
    if (n > kTraceSlots) n = kTraceSlots;
    return cudaMemcpyFromSymbol(host, g_kda_trace, sizeof(unsigned long long) * n) == cudaSuccess ? n : -1;
}
#endif

kda_status kda_get_device_status(kda_stream_t stream) {
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(st) != cudaSuccess) return KDA_ERR_CUDA;
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_kda_status, sizeof(int)) != cudaSuccess) return KDA_ERR_CUDA;
    if (v != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_kda_status, &zero, sizeof(int)) != cudaSuccess) return KDA_ERR_CUDA;
    }
    return static_cast<kda_status>(v);
}

}  // extern "C"

// ------------------------------------------------------------------------------------------
// Allocation-free prefill: the tensor-core prefill with its workspace taken from a static
// device array inside this library instead of from the caller (for callers that cannot
// allocate device memory where they run).  Every GPU that loads the library holds the
// array until the process exits; all calls on a device share it.
static __device__ __align__(256) uint8_t g_kda_noalloc_scratch[KDA_NOALLOC_SCRATCH_BYTES];

namespace {
typedef CUresult (*CtxGetCurrentFn)(CUcontext*);

// cuCtxGetCurrent through the runtime's driver entry point (no link against libcuda).
CtxGetCurrentFn ctx_get_current() {
    static const CtxGetCurrentFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<CtxGetCurrentFn>(p);
        return static_cast<CtxGetCurrentFn>(nullptr);
    }();
    return fn;
}

// Last looked-up scratch address per CUDA context.  The array's name is only a host-side
// stand-in; the kernels must get the device address, which belongs to the context that
// loaded the module: a new primary context after cudaDeviceReset, or another context made
// current, has its own.
struct ScratchEntry {
    CUcontext ctx;
    void* ptr;
};
constexpr int kMaxContexts = 64;
std::mutex g_noalloc_mutex;
ScratchEntry g_noalloc_cache[kMaxContexts] = {};

// Device address of the scratch array in the current context.  Outside stream capture the
// address is looked up on every call (cudaGetSymbolAddress, a host-side query once the
// module is loaded) and the cache refreshed; while `stream` is capturing only the cache
// of this context is used, so the first call in a context must come before any capture.
cudaError_t noalloc_scratch(cudaStream_t stream, void** ptr) {
    CtxGetCurrentFn get = ctx_get_current();
    if (!get) return cudaErrorNotSupported;
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    cudaError_t err = cudaStreamIsCapturing(stream, &cap);
    if (err != cudaSuccess) return err;
    void* p = nullptr;
    if (cap == cudaStreamCaptureStatusNone) {
        // also makes the device's primary context current if nothing was yet
        err = cudaGetSymbolAddress(&p, g_kda_noalloc_scratch);
        if (err != cudaSuccess) return err;
    }
    CUcontext ctx = nullptr;
    if (get(&ctx) != CUDA_SUCCESS || ctx == nullptr) return cudaErrorDeviceUninitialized;
    std::lock_guard<std::mutex> lock(g_noalloc_mutex);
    int slot = -1;
    for (int i = 0; i < kMaxContexts; ++i)
        if (g_noalloc_cache[i].ctx == ctx) { slot = i; break; }
    if (cap != cudaStreamCaptureStatusNone) {
        if (slot < 0) return cudaErrorStreamCaptureUnsupported;
        *ptr = g_noalloc_cache[slot].ptr;
        return cudaSuccess;
    }
    if (slot < 0) {
        for (int i = 0; i < kMaxContexts && slot < 0; ++i)
            if (g_noalloc_cache[i].ctx == nullptr) slot = i;
        if (slot < 0) slot = 0;   // table full: reuse the first entry
    }
    g_noalloc_cache[slot] = {ctx, p};
    *ptr = p;
    return cudaSuccess;
}
}  // namespace

extern "C" kda_status kda_prefill_noalloc(const void* q, const void* k, const void* v,
                                          const float* g, const float* beta,
                                          const float* initial_state, const int32_t* cu_seqlens,
                                          int32_t num_seqs, int64_t total_tokens, int32_t H,
                                          int32_t dk, int32_t dv, kda_dtype dt, void* out,
                                          float* final_state, int32_t C, kda_stream_t stream) {
    if (num_seqs < 0 || total_tokens < 0 || H <= 0) return KDA_ERR_INVALID_ARG;
    if (dt != KDA_F32 && dt != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if (dt != KDA_BF16 || !tensor_core_path(dt, dk) || dv != dk || C != 64) return KDA_ERR_UNSUPPORTED;
    if (total_tokens > INT32_MAX || !tc_problem_fits(total_tokens, num_seqs, H)) return KDA_ERR_UNSUPPORTED;
    const size_t need = kda_prefill_workspace_size_min(total_tokens, num_seqs, H, dk, dv, C, dt);
    if (need == 0 || need > KDA_NOALLOC_SCRATCH_BYTES) return KDA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return KDA_OK;
    void* scratch = nullptr;
    if (noalloc_scratch(reinterpret_cast<cudaStream_t>(stream), &scratch) != cudaSuccess)
        return KDA_ERR_CUDA;
    return kda_prefill(q, k, v, g, beta, initial_state, cu_seqlens, num_seqs, total_tokens, H,
                       dk, dv, dt, out, final_state, C, scratch, KDA_NOALLOC_SCRATCH_BYTES, stream);
}
