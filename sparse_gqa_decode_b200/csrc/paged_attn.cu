// paged_attn.cu -- attention of a step's query tokens over the paged cache (sgd_paged_attn in
// include/sgd.h).
//
// One CTA per (sequence, query token, head): its warps walk the entries that the query sees, a lane
// holds D / 32 channels, each warp keeps a running maximum, sum and output, and the four are merged
// at the end:  m' = max(m, z),  l' = l e^(m - m') + e^(z - m'),  o' = o e^(m - m') + e^(z - m') v.
#include <math.h>

#include "paged.h"
#include "quant.cuh"

namespace sgd {

namespace {

template <bool I8, int D>
__global__ void __launch_bounds__(128) paged_attn_kernel(PagedView kv, PagedAttnArgs a) {
    constexpr int E = D / 32;
    const int Hq = kv.Hkv * a.G, h = blockIdx.x % Hq, m = blockIdx.x / Hq % a.M, b = blockIdx.x / Hq / a.M;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int bad = 0, n = a.M, L = kv.lens[b];
    const int room = (int)min((int64_t)kv.max_pages * SGD_PAGE, (int64_t)INT32_MAX);
    if (L < 0 || L > room) bad |= SGD_STATUS_SIZE_MISMATCH;
    L = min(max(L, 0), room);
    if (a.n_nodes) {
        n = a.n_nodes[b];
        if (n < 0 || n > a.M) bad |= SGD_STATUS_BAD_INDEX;
        n = min(max(n, 0), a.M);
    }
    const int base = L - n;
    const int32_t *par = a.parent ? a.parent + (int64_t)b * a.M : nullptr;
    auto parent = [&](int i) {
        if (!par) return i - 1;
        const int p = par[i];
        if (p < -1 || p >= i) {
            bad |= SGD_STATUS_BAD_INDEX;
            return -1;
        }
        return p;
    };
    auto depth = [&](int i) {
        int d = 0;
        for (int j = parent(i); j >= 0; j = parent(j)) ++d;
        return d;
    };
    __shared__ uint64_t anc_s;
    const int pos = base + depth(m);
    if (threadIdx.x == 0) {
        uint64_t anc = 0;
        for (int j = m; j >= 0; j = parent(j)) {
            const int at = base + depth(j);
            if (base + j >= 0 && (a.window == 0 || pos - at < a.window || at < a.sinks)) anc |= 1ull << j;
        }
        anc_s = m < n ? anc : 0;
    }
    __syncthreads();
    const uint64_t anc = anc_s;
    float q[E], o[E];
    const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(a.q) + (((int64_t)b * a.M + m) * Hq + h) * D + lane * E;
    for (int e = 0; e < E; ++e) q[e] = __bfloat162float(qp[e]) * a.scale_log2, o[e] = 0.f;
    float ks = 1.f, vs = 1.f;
    if constexpr (I8) {
        ks = calibrated_scale(kv.k_scale, a.status, threadIdx.x == 0);
        vs = calibrated_scale(kv.v_scale, a.status, threadIdx.x == 0);
    }
    float mx = -INFINITY, l = 0.f;
    for (int t = warp; t < L && m < n; t += 4) {
        const bool see = t < base ? a.window == 0 || pos - t < a.window || t < a.sinks : (anc >> (t - base)) & 1;
        if (!see) continue;
        int p = kv.table[(int64_t)b * kv.max_pages + t / SGD_PAGE];
        if (p < 0 || p >= kv.n_pages) bad |= SGD_STATUS_BAD_INDEX, p = 0;
        const int64_t at = (((int64_t)p * kv.Hkv + h / a.G) * SGD_PAGE + t % SGD_PAGE) * D + lane * E;
        float z = 0.f, v[E];
        for (int e = 0; e < E; ++e) {
            float k;
            if constexpr (I8) {
                k = ks * (float)static_cast<const int8_t *>(kv.k)[at + e];
                v[e] = vs * (float)static_cast<const int8_t *>(kv.v)[at + e];
            } else {
                k = __bfloat162float(static_cast<const __nv_bfloat16 *>(kv.k)[at + e]);
                v[e] = __bfloat162float(static_cast<const __nv_bfloat16 *>(kv.v)[at + e]);
            }
            z += q[e] * k;
        }
        z = warp_sum(z);
        const float m2 = fmaxf(mx, z), r = exp2f(mx - m2), w = exp2f(z - m2);
        l = l * r + w;
        for (int e = 0; e < E; ++e) o[e] = o[e] * r + w * v[e];
        mx = m2;
    }
    if (bad) atomicOr(a.status, bad);
    __shared__ float sm[4], sl[4], so[4][D];
    if (lane == 0) sm[warp] = mx, sl[warp] = l;
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
    __syncthreads();
    const float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float z = 0.f, w[4];
    for (int i = 0; i < 4; ++i) {
        w[i] = sl[i] > 0.f ? exp2f(sm[i] - top) : 0.f;
        z += w[i] * sl[i];
    }
    const int64_t row = ((int64_t)b * a.M + m) * Hq + h;
    if (threadIdx.x < D) {
        float x = 0.f;
        for (int i = 0; i < 4; ++i) x += w[i] * so[i][threadIdx.x];
        static_cast<__nv_bfloat16 *>(a.out)[row * D + threadIdx.x] = __float2bfloat16(z > 0.f ? x / z : 0.f);
    }
    if (threadIdx.x == 0) a.lse[row] = z > 0.f ? (top + log2f(z)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

size_t paged_attn_scratch(int, int, int, int, int, int) { return 0; }

int launch_paged_attn(const PagedView &kv, const PagedAttnArgs &a, cudaStream_t s) {
    const dim3 grid(kv.B * a.M * kv.Hkv * a.G);
    auto k = kv.es == 1 ? (kv.D == 128 ? paged_attn_kernel<true, 128> : paged_attn_kernel<true, 64>)
                        : (kv.D == 128 ? paged_attn_kernel<false, 128> : paged_attn_kernel<false, 64>);
    const cudaError_t e = launch_k(k, grid, dim3(128), 0, s, 1, kv, a);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? SGD_OK : SGD_ERR_CUDA;
}

}  // namespace sgd
