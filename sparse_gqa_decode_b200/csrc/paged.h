// paged.h -- host-side interface between the paged entry points (paged_api.cu) and their kernels.
#pragma once

#include <atomic>

#include "common.cuh"

namespace sgd {

// A kernel's permission to use more shared memory than 48 KB, asked for once per device (the call costs a microsecond).
struct SmemOptIn {
    std::atomic<uint64_t> done{0};  // a bit per device; devices from 64 on ask every time
    bool set(const void *kern, int bytes) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return false;
        const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
        if (done.load(std::memory_order_relaxed) & bit) return true;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
        done.fetch_or(bit, std::memory_order_relaxed);
        return true;
    }
};

// An sgd_paged_kv as the kernels take it (device pointers).
struct PagedView {
    void *k, *v;          // [n_pages, Hkv, 64, D]
    const float *k_scale, *v_scale;
    int32_t *table;       // [B, max_pages]
    int32_t *lens, *held, *ref;
    int B, Hkv, D, es;    // es: bytes of an element (2 bf16, 1 INT8 codes)
    int n_pages, max_pages;
};

struct CompactArgs {
    // accept
    const int32_t *path, *n_path, *n_nodes;
    int M;
    // keep
    const int32_t *idx, *cu_kept;
    int64_t kept_total;
    int32_t *new_lens;
    int32_t *status;
};

int launch_pages_reserve(const PagedView &kv, const int32_t *add, int32_t *new_lens, int32_t *scratch,
                         int32_t *status, cudaStream_t s);
int launch_pages_fork(const PagedView &kv, const int32_t *src, const int32_t *dst, int n, int32_t *scratch,
                      int32_t *status, cudaStream_t s);
int launch_pages_release(const PagedView &kv, const int32_t *keep, int32_t *status, cudaStream_t s);
int launch_pages_append(const PagedView &kv, const void *k_new, const void *v_new, const int32_t *cu, int64_t T_new,
                        int32_t *status, cudaStream_t s);
int launch_pages_compact(const PagedView &kv, const CompactArgs &a, bool accept, cudaStream_t s);

// sgd_verify_tree
struct VerifyArgs {
    const void *p, *q;
    const int32_t *tokens, *parent, *n_nodes;
    const float *u_accept, *u_sample;
    int32_t *n_path, *path, *next;
    int32_t *status;
    int B, M;
    int64_t V;
    bool f32;
};
int launch_verify(const VerifyArgs &a, int sms, cudaStream_t s);

// sgd_paged_attn
struct PagedAttnArgs {
    const void *q;            // [B, M, Hq, D] bf16
    const int32_t *parent;    // [B, M] or NULL
    const int32_t *n_nodes;   // [B] or NULL
    void *out;                // [B, M, Hq, D] bf16
    float *lse;               // [B, M, Hq]
    int G, M, window, sinks;
    float scale_log2;         // log2(e) / sqrt(D)
    uint8_t *ws;              // behind the header
    int32_t *status;
    int sms;
    long long wait_limit;
    int idle_producer;
};
size_t paged_attn_scratch(int B, int Hkv, int D, int G, int M, int sms);
int launch_paged_attn(const PagedView &kv, const PagedAttnArgs &a, cudaStream_t s);

}  // namespace sgd
