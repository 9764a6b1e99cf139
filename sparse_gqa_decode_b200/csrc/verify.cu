// verify.cu -- verification of drafted tokens (sgd_verify_tree in include/sgd.h).
//
// A refused draft replaces the weights w by max(w / Z - q, 0).  Starting from w = p, every such step
// keeps the form w = max(c p - d q, 0) with two numbers c and d: where the inner value is negative
// the next step's is too, and otherwise (c p - d q) / Z - q = (c / Z) p - (d / Z + 1) q.  So after any
// number of refusals a weight is one multiply-add of p and q, and nothing of a vocabulary's size is kept.
//
// What has to be read is one row of p (and of q) per sum, and the tested tokens' two probabilities.
// The latter are fetched for all nodes at once before the walk, so that the walk itself touches only
// shared memory until a sum over the vocabulary is due.
#include <cooperative_groups.h>

#include "paged.h"

namespace cg = cooperative_groups;

namespace sgd {

namespace {

constexpr int kVerifyThreads = 512, kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyCluster = 8;  // CTAs of one sequence over a large vocabulary

__device__ __forceinline__ double as_double(float x) { return (double)x; }
__device__ __forceinline__ double as_double(__nv_bfloat16 x) { return (double)__bfloat162float(x); }

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct Shared {
    double px[SGD_MAX_NODES], qx[SGD_MAX_NODES];  // p and q of each node's token after its parent
    float u[SGD_MAX_NODES];
    int32_t tok[SGD_MAX_NODES], parent[SGD_MAX_NODES];
    int32_t gone[SGD_MAX_NODES];                  // chosen drafts refused at this node (q == NULL)
    double part[kVerifyCluster];                  // every CTA's part of the sum
    double wsum[kVerifyWarps];                    // this CTA's warps' parts
    int32_t found;
};

// One cluster per sequence; CTA r holds tokens [r * per, (r + 1) * per), its warps equal consecutive
// parts of them.  Every CTA makes the same walk from the same sums, so none has to be told the way.
template <typename T, bool DRAWN>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(VerifyArgs a, int ncta) {
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int b = blockIdx.x / ncta, rank = blockIdx.x % ncta;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t V = a.V;
    const T *P = static_cast<const T *>(a.p) + (int64_t)b * a.M * V;
    const T *Q = DRAWN ? static_cast<const T *>(a.q) + (int64_t)b * a.M * V : nullptr;
    int bad = 0;
    int n = a.M;
    if (a.n_nodes) {
        n = min(max(a.n_nodes[b], 0), a.M);
        if (n != a.n_nodes[b]) bad = SGD_STATUS_BAD_INDEX;
    }
    if (tid < n) {
        const int m = tid;
        const int par = a.parent[(int64_t)b * a.M + m], x = a.tokens[(int64_t)b * a.M + m];
        const bool fit = par >= 0 && par < m && x >= 0 && x < V;
        if (m > 0 && !fit && par != -1) bad = SGD_STATUS_BAD_INDEX;
        if (m > 0 && (x < 0 || x >= V)) bad = SGD_STATUS_BAD_INDEX;
        if (m == 0 && par != -1) bad = SGD_STATUS_BAD_INDEX;
        sh.tok[m] = x;
        sh.parent[m] = fit ? par : -1;  // never walked to
        sh.u[m] = a.u_accept[(int64_t)b * a.M + m];
        if (m > 0 && fit) {
            sh.px[m] = as_double(P[par * V + x]);
            sh.qx[m] = DRAWN ? as_double(Q[par * V + x]) : 1.0;
        }
    }
    if (rank == 0 && bad) atomicOr(a.status, bad);
    if (tid == 0) sh.found = -1;
    cluster.sync();  // the shared arrays, and every CTA of the cluster is there
    if (n == 0) {
        if (rank == 0) {
            if (tid < a.M) a.path[(int64_t)b * a.M + tid] = -1;
            if (tid == 0) {
                a.n_path[b] = 0;
                a.next[b] = -1;
            }
        }
        return;
    }

    // warp's tokens
    const int64_t per_warp = (V + (int64_t)ncta * kVerifyWarps - 1) / ((int64_t)ncta * kVerifyWarps);
    const int64_t lo = min(((int64_t)rank * kVerifyWarps + warp) * per_warp, V), hi = min(lo + per_warp, V);

    int cur = 0, n_gone = 0;
    double c = 1.0, d = 0.0;
    auto weight = [&](int64_t y) -> double {
        double w = as_double(P[cur * V + y]);
        if constexpr (DRAWN) {
            if (d != 0.0) w = fmax(c * w - d * as_double(Q[cur * V + y]), 0.0);
        } else {
            for (int j = 0; j < n_gone; ++j)
                if (sh.gone[j] == y) w = 0.0;
        }
        return w;
    };
    // The sum of all weights, the same bits in every CTA; sh.part and sh.wsum keep its parts.
    auto sum_all = [&]() -> double {
        double s = 0.0;
        constexpr int U = 8;
        for (int64_t y0 = lo + lane; y0 < hi; y0 += 32 * U) {
            double w[U];
#pragma unroll
            for (int u = 0; u < U; ++u) w[u] = y0 + 32 * u < hi ? weight(y0 + 32 * u) : 0.0;
#pragma unroll
            for (int u = 0; u < U; ++u) s += w[u];
        }
        s = warp_sum_d(s);
        cluster.sync();  // the last sum's parts have been read everywhere
        if (lane == 0) sh.wsum[warp] = s;
        __syncthreads();
        if (tid < ncta) {
            double t = 0.0;
            for (int w = 0; w < kVerifyWarps; ++w) t += sh.wsum[w];
            cluster.map_shared_rank(&sh, tid)->part[rank] = t;
        }
        cluster.sync();
        double t = 0.0;
        for (int r = 0; r < ncta; ++r) t += sh.part[r];
        return t;
    };

    int n_path = 1;
    if (rank == 0 && tid < a.M) a.path[(int64_t)b * a.M + tid] = tid == 0 ? 0 : -1;
    __syncthreads();  // the -1s before the walk's entries
    double Z = 1.0;
    bool have = false;  // sh.part is the sum of the present weights
    double total = 0.0;
    for (int m = 1; m < n; ++m) {
        if (sh.parent[m] != cur) continue;
        double w = sh.px[m];
        if constexpr (DRAWN) {
            if (d != 0.0) w = fmax(c * w - d * sh.qx[m], 0.0);
        } else {
            for (int j = 0; j < n_gone; ++j)
                if (sh.gone[j] == sh.tok[m]) w = 0.0;
        }
        if ((double)sh.u[m] * sh.qx[m] * Z < w) {
            cur = m;
            c = 1.0, d = 0.0, Z = 1.0, n_gone = 0;
            have = false;
            if (rank == 0 && tid == 0) a.path[(int64_t)b * a.M + n_path] = m;
            ++n_path;
            continue;
        }
        const double c0 = c, d0 = d;
        if constexpr (DRAWN) {
            c = c / Z;
            d = d / Z + 1.0;
        } else {
            __syncthreads();
            if (tid == 0) sh.gone[n_gone] = sh.tok[m];
            __syncthreads();
            ++n_gone;
        }
        total = sum_all();
        have = total > 0.0;
        if (have) {
            Z = total;
        } else {  // nothing is left but rounding: as it was
            c = c0, d = d0;
            if constexpr (!DRAWN) --n_gone;
        }
    }
    if (!have) total = sum_all();

    // the CTA, then the warp, in whose tokens the running sum passes u * total
    const double thr = (double)a.u_sample[b] * total;
    double before = 0.0;
    int at = -1, last = -1;
    double at_before = 0.0, last_before = 0.0;
    for (int r = 0; r < ncta; ++r) {
        const double s = sh.part[r];
        if (s > 0.0) last = r, last_before = before;
        if (at < 0 && before + s > thr) at = r, at_before = before;
        before += s;
    }
    if (at < 0) at = last, at_before = last_before;  // rounding at the very end, or nothing positive
    if (at == rank) {
        double wb = at_before;
        int wat = -1, wlast = -1;
        double wat_before = 0.0, wlast_before = 0.0;
        for (int w = 0; w < kVerifyWarps; ++w) {
            const double s = sh.wsum[w];
            if (s > 0.0) wlast = w, wlast_before = wb;
            if (wat < 0 && wb + s > thr) wat = w, wat_before = wb;
            wb += s;
        }
        if (wat < 0) wat = wlast, wat_before = wlast_before;
        if (warp == wat) {
            int64_t pick = -1, high = -1;  // high: the last token with a positive weight
            double run = wat_before;
            for (int64_t y0 = lo; y0 < hi && pick < 0; y0 += 32) {
                const double w = y0 + lane < hi ? weight(y0 + lane) : 0.0;
                double inc = w;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double up = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += up;
                }
                const unsigned over = __ballot_sync(0xffffffffu, w > 0.0 && run + inc > thr);
                const unsigned pos = __ballot_sync(0xffffffffu, w > 0.0);
                if (over) pick = y0 + __ffs(over) - 1;
                if (pos) high = y0 + 31 - __clz(pos);
                run += __shfl_sync(0xffffffffu, inc, 31);
            }
            if (lane == 0) a.next[b] = (int32_t)(pick >= 0 ? pick : high);
        }
    }
    if (rank == 0 && tid == 0) {
        a.n_path[b] = n_path;
        if (at < 0) {
            a.next[b] = 0;
            atomicOr(a.status, SGD_STATUS_BAD_PROBS);
        }
    }
    cluster.sync();  // no CTA leaves while another may still write its parts
}

template <typename T, bool DRAWN>
int launch(const VerifyArgs &a, cudaStream_t s) {
    // one CTA walks a vocabulary of up to 8192 tokens, 16 to a thread; a cluster's barriers cost more
    const int ncta = a.V > 8192 ? kVerifyCluster : 1;
    const cudaError_t e =
        launch_k(verify_kernel<T, DRAWN>, dim3(a.B * ncta), dim3(kVerifyThreads), 0, s, ncta, a, ncta);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? SGD_OK : SGD_ERR_CUDA;
}

}  // namespace

int launch_verify(const VerifyArgs &a, cudaStream_t s) {
    if (a.f32) return a.q ? launch<float, true>(a, s) : launch<float, false>(a, s);
    return a.q ? launch<__nv_bfloat16, true>(a, s) : launch<__nv_bfloat16, false>(a, s);
}

}  // namespace sgd
