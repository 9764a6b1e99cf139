// paged_api.cu -- the C ABI of the paged cache and of draft verification (include/sgd.h): argument
// checks, the workspace, the launches.  As in api.cu nothing here allocates, frees or synchronises.
#include <math.h>

#include <algorithm>

#include "internal.h"
#include "paged.h"

namespace sgd {

namespace {

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_paged(const sgd_paged_kv *kv, bool upkeep) {
    if (!kv || !kv->k || !kv->v || !kv->page_table || !kv->lens) return SGD_ERR_NULL;
    if (upkeep && (!kv->held || !kv->ref_count)) return SGD_ERR_NULL;
    if (kv->B < 1 || kv->Hkv < 1 || kv->n_pages < 1 || kv->max_pages < 1) return SGD_ERR_SHAPE;
    if (kv->D != 64 && kv->D != 128) return SGD_ERR_SHAPE;
    if ((int64_t)kv->n_pages * kv->Hkv >= (int64_t(1) << 31) / SGD_PAGE) return SGD_ERR_SHAPE;
    if (kv->max_pages >= (1 << 24) || (int64_t)kv->B * kv->Hkv >= (int64_t(1) << 24)) return SGD_ERR_SHAPE;
    if (kv->Hkv > 65535) return SGD_ERR_SHAPE;
    if (kv->dtype != SGD_BF16 && kv->dtype != SGD_I8) return SGD_ERR_DTYPE;
    if (kv->dtype == SGD_I8 && (!kv->k_scale || !kv->v_scale)) return SGD_ERR_NULL;
    if (!aligned(kv->k, 16) || !aligned(kv->v, 16) || !aligned(kv->page_table, 4) || !aligned(kv->lens, 4))
        return SGD_ERR_ALIGN;
    if (upkeep && (!aligned(kv->held, 4) || !aligned(kv->ref_count, 16))) return SGD_ERR_ALIGN;
    if (kv->dtype == SGD_I8 && (!aligned(kv->k_scale, 4) || !aligned(kv->v_scale, 4))) return SGD_ERR_ALIGN;
    return SGD_OK;
}

PagedView view(const sgd_paged_kv *kv) {
    PagedView v;
    v.k = kv->k, v.v = kv->v;
    v.k_scale = kv->k_scale, v.v_scale = kv->v_scale;
    v.table = kv->page_table, v.lens = kv->lens, v.held = kv->held, v.ref = kv->ref_count;
    v.B = kv->B, v.Hkv = kv->Hkv, v.D = kv->D, v.es = kv->dtype == SGD_I8 ? 1 : 2;
    v.n_pages = kv->n_pages, v.max_pages = kv->max_pages;
    return v;
}

// the upkeep calls: a word per page and three per row behind the header
size_t upkeep_bytes(const sgd_paged_kv *kv) {
    return sizeof(WsHeader) + (((size_t)kv->n_pages + 3 * (size_t)kv->B + 64) * 4 + 255) / 256 * 256;
}

// SMs of a B200; the partial results of the attention are sized for them whatever the device
constexpr int kMaxSms = 148;

size_t workspace_bytes_of(const sgd_paged_kv *kv, int G, int M) {
    if (M == 0) return upkeep_bytes(kv);
    return std::max(upkeep_bytes(kv), sizeof(WsHeader) + paged_attn_scratch(kv->B, kv->Hkv, kv->D, G, M, kMaxSms));
}

// Checks the workspace and the device, and zeroes the status word unless the call's first kernel
// writes it.
int begin(void *ws, size_t have, size_t need, bool zero, cudaStream_t s, int *sms) {
    if (!ws) return SGD_ERR_NULL;
    if (!aligned(ws, 16)) return SGD_ERR_ALIGN;
    if (have < need) return SGD_ERR_WORKSPACE;
    const int rc = device_sms(sms);
    if (rc != SGD_OK) return rc;
    if (zero && cudaMemsetAsync(ws, 0, sizeof(int32_t), s) != cudaSuccess) return SGD_ERR_CUDA;
    return SGD_OK;
}

int32_t *status_of(void *ws) { return static_cast<int32_t *>(ws); }
int32_t *scratch_of(void *ws) { return reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) + sizeof(WsHeader)); }

}  // namespace

}  // namespace sgd

using namespace sgd;

extern "C" {

size_t sgd_paged_workspace_size(const sgd_paged_kv *kv, int G, int M) {
    if (check_paged(kv, false) != SGD_OK || M < 0 || M > SGD_MAX_NODES || (M > 0 && (G < 1 || G > 16))) return 0;
    return workspace_bytes_of(kv, G, M);
}

int sgd_paged_attn(const void *q, int G, int M, const sgd_paged_kv *kv, const int32_t *parent,
                   const int32_t *n_nodes, int window, int sinks, void *out, float *lse, void *workspace,
                   size_t workspace_bytes, void *stream) {
    int rc = check_paged(kv, false);
    if (rc != SGD_OK) return rc;
    if (!q || !out || !lse) return SGD_ERR_NULL;
    if (G < 1 || G > 16 || M < 1 || M > SGD_MAX_NODES) return SGD_ERR_SHAPE;
    if ((int64_t)kv->B * M * kv->Hkv * G >= (int64_t(1) << 31)) return SGD_ERR_SHAPE;
    if (window < 0 || sinks < 0) return SGD_ERR_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(parent, 4) || !aligned(n_nodes, 4))
        return SGD_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    PagedAttnArgs a = {};
    rc = begin(workspace, workspace_bytes, workspace_bytes_of(kv, G, M), false, s, &a.sms);
    if (rc != SGD_OK) return rc;
    a.q = q, a.parent = parent, a.n_nodes = n_nodes, a.out = out, a.lse = lse;
    // no position reaches 2^30 (max_pages < 2^24): larger values mean the same
    a.G = G, a.M = M, a.window = std::min(window, 1 << 30), a.sinks = window ? std::min(sinks, 1 << 30) : 0;
    a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)kv->D));
    a.ws = reinterpret_cast<uint8_t *>(scratch_of(workspace));
    a.status = status_of(workspace);
    a.sms = std::min(a.sms, kMaxSms);
    paged_test_hooks(&a.wait_limit, &a.idle_producer);
    return launch_paged_attn(view(kv), a, s);
}

int sgd_verify_tree(const void *p, sgd_dtype p_dtype, const void *q, int B, int M, int64_t V, const int32_t *tokens,
                    const int32_t *parent, const int32_t *n_nodes, const float *u_accept, const float *u_sample,
                    int32_t *n_path, int32_t *path, int32_t *next_token, void *workspace, size_t workspace_bytes,
                    void *stream) {
    if (!p || !tokens || !parent || !u_accept || !u_sample || !n_path || !path || !next_token) return SGD_ERR_NULL;
    if (B < 1 || B >= (1 << 24) || M < 1 || M > SGD_MAX_NODES || V < 1 || V >= (int64_t(1) << 31)) return SGD_ERR_SHAPE;
    if (p_dtype != SGD_F32 && p_dtype != SGD_BF16) return SGD_ERR_DTYPE;
    if (!aligned(p, 16) || !aligned(q, 16) || !aligned(tokens, 4) || !aligned(parent, 4) || !aligned(n_nodes, 4) ||
        !aligned(u_accept, 4) || !aligned(u_sample, 4) || !aligned(n_path, 4) || !aligned(path, 4) ||
        !aligned(next_token, 4))
        return SGD_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int sms;
    const int rc = begin(workspace, workspace_bytes, sizeof(WsHeader), true, s, &sms);
    if (rc != SGD_OK) return rc;
    VerifyArgs a = {};
    a.p = p, a.q = q, a.tokens = tokens, a.parent = parent, a.n_nodes = n_nodes;
    a.u_accept = u_accept, a.u_sample = u_sample;
    a.n_path = n_path, a.path = path, a.next = next_token;
    a.status = status_of(workspace);
    a.B = B, a.M = M, a.V = V, a.f32 = p_dtype == SGD_F32;
    return launch_verify(a, sms, s);
}

int sgd_pages_reserve(const sgd_paged_kv *kv, const int32_t *add, int32_t *new_lens, void *workspace,
                      size_t workspace_bytes, void *stream) {
    int rc = check_paged(kv, true);
    if (rc != SGD_OK) return rc;
    if (!add || !new_lens) return SGD_ERR_NULL;
    if (!aligned(add, 4) || !aligned(new_lens, 4)) return SGD_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int sms;
    rc = begin(workspace, workspace_bytes, upkeep_bytes(kv), false, s, &sms);
    if (rc != SGD_OK) return rc;
    return launch_pages_reserve(view(kv), add, new_lens, scratch_of(workspace), status_of(workspace), s);
}

int sgd_pages_append(const sgd_paged_kv *kv, const void *k_new, const void *v_new, const int32_t *cu_new,
                     int64_t T_new, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_paged(kv, false);
    if (rc != SGD_OK) return rc;
    if (!cu_new || (T_new > 0 && (!k_new || !v_new))) return SGD_ERR_NULL;
    if (T_new < 0 || T_new >= (int64_t(1) << 31) || T_new * kv->Hkv >= (int64_t(1) << 31)) return SGD_ERR_SHAPE;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(cu_new, 4) || !aligned(kv->held, 4) ||
        !aligned(kv->ref_count, 4))
        return SGD_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int sms;
    rc = begin(workspace, workspace_bytes, sizeof(WsHeader), true, s, &sms);
    if (rc != SGD_OK) return rc;
    return launch_pages_append(view(kv), k_new, v_new, cu_new, T_new, status_of(workspace), s);
}

int sgd_pages_fork(const sgd_paged_kv *kv, const int32_t *src, const int32_t *dst, int n, void *workspace,
                   size_t workspace_bytes, void *stream) {
    int rc = check_paged(kv, true);
    if (rc != SGD_OK) return rc;
    if (!src || !dst) return SGD_ERR_NULL;
    if (n < 1 || n >= kv->B) return SGD_ERR_SHAPE;  // every dst once and at least one src beside them
    if (!aligned(src, 4) || !aligned(dst, 4)) return SGD_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int sms;
    rc = begin(workspace, workspace_bytes, upkeep_bytes(kv), false, s, &sms);
    if (rc != SGD_OK) return rc;
    return launch_pages_fork(view(kv), src, dst, n, scratch_of(workspace), status_of(workspace), s);
}

int sgd_pages_release(const sgd_paged_kv *kv, const int32_t *keep, void *workspace, size_t workspace_bytes,
                      void *stream) {
    int rc = check_paged(kv, true);
    if (rc != SGD_OK) return rc;
    if (!keep) return SGD_ERR_NULL;
    if (!aligned(keep, 4)) return SGD_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int sms;
    rc = begin(workspace, workspace_bytes, sizeof(WsHeader), true, s, &sms);
    if (rc != SGD_OK) return rc;
    return launch_pages_release(view(kv), keep, status_of(workspace), s);
}

int sgd_pages_accept(const sgd_paged_kv *kv, const int32_t *path, const int32_t *n_path, const int32_t *n_nodes,
                     int M, int32_t *new_lens, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_paged(kv, false);
    if (rc != SGD_OK) return rc;
    if (!path || !n_path || !n_nodes || !new_lens || !kv->ref_count) return SGD_ERR_NULL;
    if (M < 1 || M > SGD_MAX_NODES) return SGD_ERR_SHAPE;
    if (new_lens == kv->lens) return SGD_ERR_ARG;
    if (!aligned(path, 4) || !aligned(n_path, 4) || !aligned(n_nodes, 4) || !aligned(new_lens, 4) ||
        !aligned(kv->ref_count, 4) || !aligned(kv->held, 4))
        return SGD_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int sms;
    rc = begin(workspace, workspace_bytes, sizeof(WsHeader), true, s, &sms);
    if (rc != SGD_OK) return rc;
    CompactArgs a = {};
    a.path = path, a.n_path = n_path, a.n_nodes = n_nodes, a.M = M;
    a.new_lens = new_lens, a.status = status_of(workspace);
    return launch_pages_compact(view(kv), a, true, s);
}

int sgd_pages_keep(const sgd_paged_kv *kv, const int32_t *idx, const int32_t *cu_kept, int64_t kept_total,
                   int32_t *new_lens, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_paged(kv, false);
    if (rc != SGD_OK) return rc;
    if (!idx || !cu_kept || !new_lens || !kv->ref_count) return SGD_ERR_NULL;
    if (kept_total < 1 || kept_total >= (int64_t(1) << 31)) return SGD_ERR_SHAPE;
    if (new_lens == kv->lens) return SGD_ERR_ARG;
    if (!aligned(idx, 4) || !aligned(cu_kept, 4) || !aligned(new_lens, 4) || !aligned(kv->ref_count, 4) ||
        !aligned(kv->held, 4))
        return SGD_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int sms;
    rc = begin(workspace, workspace_bytes, sizeof(WsHeader), true, s, &sms);
    if (rc != SGD_OK) return rc;
    CompactArgs a = {};
    a.idx = idx, a.cu_kept = cu_kept, a.kept_total = kept_total;
    a.new_lens = new_lens, a.status = status_of(workspace);
    return launch_pages_compact(view(kv), a, false, s);
}

}  // extern "C"
