// dt_abi_target.cu -- C ABI of the target-side calls: the paged caches, tree
// attention, head norms and token log-probabilities (include/dtree.h).  Argument checks only.
#include <atomic>
#include <cmath>

#include <cuda_runtime.h>

#include "dt_launch.h"
#include "dtree.h"

namespace {

dt_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return DT_OK;
    (void)cudaGetLastError();
    return DT_ERR_CUDA;
}

// Rows per key head up to which attention streams the cache through registers: two
// groups of 8, which an MMA's side takes.  At 16 rows, 64 requests over 1000 to 16000 take
// 264 us there and 364 on 128-row tiles, 16 requests of 16 heads of 64 38 and 61; with
// more rows the streaming kernel's sums would leave its registers.
constexpr long long kStreamRows = 16;

// SMs of the current device, asked for once per device.
int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    const bool here = cudaGetDevice(&dev) == cudaSuccess;
    if (here && dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (!here || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        return 152;
    }
    n = n < 512 ? n : 512;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

dt_status check_cache(const dt_kv_cache* c, int32_t batch) {
    if (!c || batch < 1) return DT_ERR_INVALID_ARG;
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return DT_ERR_INVALID_ARG;
    if (c->n_pages < 1 || c->max_pages < 1 || c->Hkv < 1) return DT_ERR_INVALID_ARG;
    if (c->D < 1) return DT_ERR_INVALID_ARG;
    if (c->D != 64 && c->D != 128) return DT_ERR_UNSUPPORTED;
    if (c->Hkv > 65535 || batch > 65535) return DT_ERR_UNSUPPORTED;
    if ((long long)c->max_pages * c->page > 0x7fff0000ll) return DT_ERR_UNSUPPORTED;  // token numbers are int32
    if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->table || !c->len) return DT_ERR_INVALID_ARG;
    if (!aligned16(c->k) || !aligned16(c->v)) return DT_ERR_INVALID_ARG;
    return DT_OK;
}

dt_status check_cache(const dt_kv_cache4* c, int32_t batch) {
    if (!c) return DT_ERR_INVALID_ARG;
    const dt_kv_cache f = dt_cache_of(*c);
    const dt_status s = check_cache(&f, batch);
    if (s != DT_OK) return s;
    return aligned16(c->k_scale) && aligned16(c->v_scale) ? DT_OK : DT_ERR_INVALID_ARG;
}

dt_status check_rope(const dt_rope* r, int32_t D) {
    if (!r) return DT_OK;
    if (r->rot < 16 || r->rot > D || (r->rot & 15) || r->max_pos < 1) return DT_ERR_INVALID_ARG;
    if (r->interleaved != 0 && r->interleaved != 1) return DT_ERR_INVALID_ARG;
    if (!r->cos || !r->sin || !aligned16(r->cos) || !aligned16(r->sin)) return DT_ERR_INVALID_ARG;
    return DT_OK;
}

bool rows_ok(const dt_rows* r, int esize) {
    if (!r || !r->ptr || !aligned16(r->ptr)) return false;
    const int64_t all[3] = {r->stride_b, r->stride_n, r->stride_h};
    for (int64_t s : all)
        if (s < 0 || (s * esize) % 16 != 0) return false;
    return true;
}

// Rows that a call writes: heads of D elements that lie apart.
bool rows_apart(const dt_rows* r, int esize, int64_t batch, int64_t n, int64_t heads, int D) {
    return rows_ok(r, esize) && (batch < 2 || r->stride_b >= D) && (n < 2 || r->stride_n >= D) && (heads < 2 || r->stride_h >= D);
}

const dt_rope kNoRope = {nullptr, nullptr, 0, 0, 0};

template <typename C, typename F>
dt_status append(const C* c, F launch, const dt_rope* rope, int32_t batch, int32_t M, int32_t dtype, const dt_rows* k,
                 const dt_rows* v, const int32_t* rows, int32_t N, const int32_t* count, int32_t count_add,
                 int32_t* len_out, int32_t* status, dt_stream_t stream) {
    dt_status s = check_cache(c, batch);
    if (s != DT_OK) return s;
    if ((s = check_rope(rope, c->D)) != DT_OK) return s;
    if (dtype != DT_BF16 && dtype != DT_F32) return DT_ERR_INVALID_ARG;
    const int esize = dtype == DT_BF16 ? 2 : 4;
    if (M < 1 || N < 1 || (!rows && N > M) || !rows_ok(k, esize) || !rows_ok(v, esize)) return DT_ERR_INVALID_ARG;
    if (N > (1 << 30)) return DT_ERR_UNSUPPORTED;
    if (count && (count_add < -(1 << 30) || count_add > (1 << 30))) return DT_ERR_INVALID_ARG;
    if (!status || len_out == c->len) return DT_ERR_INVALID_ARG;
    return cuda_status(launch(*c, rope ? *rope : kNoRope, batch, M, dtype, *k, *v, rows, N, count, count_add, len_out,
                              status, (cudaStream_t)stream));
}

dt_status attend(const dt_kv_cache& c, int bits, const dt_rope* rope, int32_t batch, int32_t M, int32_t Hq,
                 const dt_rows* q, const dt_rows* k, const dt_rows* v, const uint32_t* mask, const int32_t* pos,
                 const int32_t* n_nodes, float scale, void* out, void* workspace, size_t workspace_bytes, int32_t* status,
                 dt_stream_t stream) {
    const dt_status s = check_rope(rope, c.D);
    if (s != DT_OK) return s;
    if (M < 1 || Hq < 1 || Hq % c.Hkv != 0) return DT_ERR_INVALID_ARG;
    if (Hq / c.Hkv > 128 || Hq > 65535 || M > (1 << 20)) return DT_ERR_UNSUPPORTED;
    // the work division counts in 32 bits: a unit's tiles and its start, at the weights of AtPlan
    const long long rows = (long long)M * (Hq / c.Hkv);
    const double tiles = (double)c.max_pages * c.page / 128 + M / 128 + 2;
    const double unit = rows <= kStreamRows ? tiles + 6 : bits == 4 ? tiles * 6 + 30 : tiles * 5 + 20;
    if ((double)batch * c.Hkv * (rows / 256 + 1) * unit > 4.2e9) return DT_ERR_UNSUPPORTED;
    if (!rows_ok(q, 2) || !rows_ok(k, 2) || !rows_ok(v, 2)) return DT_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return DT_ERR_INVALID_ARG;
    if (!out || !aligned16(out) || !status) return DT_ERR_INVALID_ARG;
    const size_t need = dt_kn12_workspace(c.D, sm_count());
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace))) return DT_ERR_INVALID_ARG;
    const DtAttend a{c, rope ? *rope : kNoRope, batch, M, Hq, Hq / c.Hkv, *q, *k, *v, mask, pos, n_nodes, scale, out, status};
    if (rows <= kStreamRows) return cuda_status(dt_kn11_launch(a, bits, workspace, 2 * sm_count(), (cudaStream_t)stream));
    return cuda_status(dt_kn12_launch(a, bits, workspace, sm_count(), (cudaStream_t)stream));
}

dt_status read(const dt_kv_cache& c, int bits, int32_t batch, const int32_t* rows, int32_t N, const int32_t* start,
               const int32_t* count, int32_t count_add, int32_t dtype, const dt_rows* k, const dt_rows* v,
               int32_t* status, dt_stream_t stream) {
    if (dtype != DT_BF16 && dtype != DT_F32) return DT_ERR_INVALID_ARG;
    const int esize = dtype == DT_BF16 ? 2 : 4;
    if (N < 1 || (rows && start) || !status) return DT_ERR_INVALID_ARG;
    if (!rows_apart(k, esize, batch, N, c.Hkv, c.D) || !rows_apart(v, esize, batch, N, c.Hkv, c.D)) return DT_ERR_INVALID_ARG;
    if (k->ptr == v->ptr) return DT_ERR_INVALID_ARG;
    if (N > (1 << 30) || c.Hkv > 32767) return DT_ERR_UNSUPPORTED;
    if (count && (count_add < -(1 << 30) || count_add > (1 << 30))) return DT_ERR_INVALID_ARG;
    return cuda_status(dt_kn15_launch(c, bits, batch, rows, N, start, count, count_add, dtype, *k, *v, status,
                                      (cudaStream_t)stream));
}

}  // namespace

extern "C" {

dt_status dt_kv_append(const dt_kv_cache* c, const dt_rope* rope, int32_t batch, int32_t M, int32_t dtype,
                       const dt_rows* k, const dt_rows* v, const int32_t* rows, int32_t N, const int32_t* count,
                       int32_t count_add, int32_t* len_out, int32_t* status, dt_stream_t stream) {
    return append(c, dt_kn10_launch, rope, batch, M, dtype, k, v, rows, N, count, count_add, len_out, status, stream);
}

dt_status dt_kv_append4(const dt_kv_cache4* c, const dt_rope* rope, int32_t batch, int32_t M, int32_t dtype,
                        const dt_rows* k, const dt_rows* v, const int32_t* rows, int32_t N, const int32_t* count,
                        int32_t count_add, int32_t* len_out, int32_t* status, dt_stream_t stream) {
    if (c && c->Hkv > 32767) return DT_ERR_UNSUPPORTED;
    return append(c, dt_kn14_launch, rope, batch, M, dtype, k, v, rows, N, count, count_add, len_out, status, stream);
}

dt_status dt_kv_read(const dt_kv_cache* c, int32_t batch, const int32_t* rows, int32_t N, const int32_t* start,
                     const int32_t* count, int32_t count_add, int32_t dtype, const dt_rows* k, const dt_rows* v,
                     int32_t* status, dt_stream_t stream) {
    const dt_status s = check_cache(c, batch);
    return s != DT_OK ? s : read(*c, 8, batch, rows, N, start, count, count_add, dtype, k, v, status, stream);
}

dt_status dt_kv_read4(const dt_kv_cache4* c, int32_t batch, const int32_t* rows, int32_t N, const int32_t* start,
                      const int32_t* count, int32_t count_add, int32_t dtype, const dt_rows* k, const dt_rows* v,
                      int32_t* status, dt_stream_t stream) {
    const dt_status s = check_cache(c, batch);
    return s != DT_OK ? s : read(dt_cache_of(*c), 4, batch, rows, N, start, count, count_add, dtype, k, v, status, stream);
}

size_t dt_tree_attention_workspace(const dt_kv_cache* c, int32_t batch, int32_t M, int32_t Hq) {
    if (check_cache(c, batch) != DT_OK || M < 1 || Hq < 1) return 0;
    return dt_kn12_workspace(c->D, sm_count());
}

size_t dt_tree_attention4_workspace(const dt_kv_cache4* c, int32_t batch, int32_t M, int32_t Hq) {
    if (check_cache(c, batch) != DT_OK || M < 1 || Hq < 1) return 0;
    return dt_kn12_workspace(c->D, sm_count());
}

dt_status dt_tree_attention(const dt_kv_cache* c, const dt_rope* rope, int32_t batch, int32_t M, int32_t Hq,
                            const dt_rows* q, const dt_rows* k, const dt_rows* v, const uint32_t* mask,
                            const int32_t* pos, const int32_t* n_nodes, float scale, void* out, void* workspace,
                            size_t workspace_bytes, int32_t* status, dt_stream_t stream) {
    const dt_status s = check_cache(c, batch);
    if (s != DT_OK) return s;
    return attend(*c, 8, rope, batch, M, Hq, q, k, v, mask, pos, n_nodes, scale, out, workspace, workspace_bytes, status,
                  stream);
}

dt_status dt_tree_attention4(const dt_kv_cache4* c, const dt_rope* rope, int32_t batch, int32_t M, int32_t Hq,
                             const dt_rows* q, const dt_rows* k, const dt_rows* v, const uint32_t* mask,
                             const int32_t* pos, const int32_t* n_nodes, float scale, void* out, void* workspace,
                             size_t workspace_bytes, int32_t* status, dt_stream_t stream) {
    const dt_status s = check_cache(c, batch);
    if (s != DT_OK) return s;
    return attend(dt_cache_of(*c), 4, rope, batch, M, Hq, q, k, v, mask, pos, n_nodes, scale, out, workspace,
                  workspace_bytes, status, stream);
}

dt_status dt_qk_norm(int32_t batch, int32_t M, int32_t Hq, int32_t Hk, int32_t D, int32_t dtype, const dt_rows* q,
                     const dt_rows* k, const float* q_weight, int32_t q_weight_stride, const float* k_weight,
                     int32_t k_weight_stride, float eps, const dt_rope* rope, const int32_t* len, const int32_t* pos,
                     const int32_t* n_nodes, const dt_rows* q_out, const dt_rows* k_out, int32_t* status,
                     dt_stream_t stream) {
    if (batch < 1 || M < 1 || Hq < 0 || Hk < 0 || Hq + (long long)Hk < 1 || D < 1) return DT_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return DT_ERR_UNSUPPORTED;
    if (batch > 65535 || M > (1 << 20) || Hq > 65535 || Hk > 65535) return DT_ERR_UNSUPPORTED;
    if ((long long)batch * M > 0x7fffffffll) return DT_ERR_UNSUPPORTED;
    if (dtype != DT_BF16 && dtype != DT_F32) return DT_ERR_INVALID_ARG;
    const int esize = dtype == DT_BF16 ? 2 : 4;
    if (Hq > 0 && (!rows_ok(q, esize) || !rows_apart(q_out, esize, batch, M, Hq, D))) return DT_ERR_INVALID_ARG;
    if (Hk > 0 && (!rows_ok(k, esize) || !rows_apart(k_out, esize, batch, M, Hk, D))) return DT_ERR_INVALID_ARG;
    if (Hq > 0 && Hk > 0 && q_out->ptr == k_out->ptr) return DT_ERR_INVALID_ARG;
    if (!aligned16(q_weight) || !aligned16(k_weight)) return DT_ERR_INVALID_ARG;
    if ((q_weight_stride != 0 && q_weight_stride != D) || (k_weight_stride != 0 && k_weight_stride != D)) return DT_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !std::isfinite(eps) || !status) return DT_ERR_INVALID_ARG;
    const dt_status s = check_rope(rope, D);
    if (s != DT_OK) return s;
    const dt_rows none = {nullptr, 0, 0, 0};
    const DtNorm a{rope ? *rope : kNoRope, batch, M, Hq, Hk, D, dtype, Hq ? *q : none, Hk ? *k : none,
                   Hq ? *q_out : none, Hk ? *k_out : none, q_weight, k_weight, q_weight_stride, k_weight_stride, eps,
                   len, pos, n_nodes, status, 0, 0, 0, 0};
    return cuda_status(dt_kn16_launch(a, sm_count(), (cudaStream_t)stream));
}

dt_status dt_token_logprobs(const void* logits, int32_t dtype, int32_t batch, int32_t M, int32_t V, int64_t stride_b,
                            int64_t stride, const int32_t* rows, const int32_t* tokens, int32_t N, int32_t top,
                            float* logprob, float* entropy, int32_t* rank, int32_t* top_id, float* top_logprob,
                            dt_stream_t stream) {
    if (!logits || !tokens || batch < 1 || M < 1 || V < 1 || stride < V || stride_b < 0 || N < 1) return DT_ERR_INVALID_ARG;
    if (dtype != DT_BF16 && dtype != DT_F32) return DT_ERR_INVALID_ARG;
    if ((uintptr_t)logits % (dtype == DT_BF16 ? 2 : 4)) return DT_ERR_INVALID_ARG;
    if (V > DT_MAX_V || (long long)batch * N > 0x0fffffffll) return DT_ERR_UNSUPPORTED;
    if (!rows && N > M) return DT_ERR_INVALID_ARG;
    if (top < 0 || top > DT_MAX_TOP || top > V) return DT_ERR_INVALID_ARG;
    if (top > 0 && (!top_id || !top_logprob)) return DT_ERR_INVALID_ARG;
    const DtLogprobs a{logits, dtype, batch, M, V, stride_b, stride, rows, tokens, N, top, logprob, entropy, rank, top_id,
                       top_logprob};
    return cuda_status(dt_kn13_launch(a, (cudaStream_t)stream));
}

}  // extern "C"
