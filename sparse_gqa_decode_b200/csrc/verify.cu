// verify.cu -- verification of drafted tokens (sgd_verify_tree in include/sgd.h).
//
// A refused draft replaces the weights w by max(w / Z - q, 0).  Starting from w = p, every such step
// keeps the form w = max(c p - d q, 0) with two numbers c and d: where the inner value is negative
// the next step's is too, and otherwise (c p - d q) / Z - q = (c / Z) p - (d / Z + 1) q.  So after several
// refusals a weight is one multiply-add of p and q, and nothing of a vocabulary's size is kept.  Its rounding is up to
// 2^-52 c p, where c is 1 over the product of the node's Z, and d loses its 1 from c = 2^53 on: refusals that a draft
// probability below 2^-40 alone allows leave rounding in w, which the definition step by step would not.
//
// What has to be read is one row of p (and of q) per sum, and the tested tokens' two probabilities.
// The latter are fetched for all nodes at once before the walk, so that the walk itself touches only
// shared memory until a sum over the vocabulary is due.
//
// Measured: 64 trees of 24 nodes 64 us (54 us where p and q lie in L2 already).  Trees with several refusals end last:
// their passes over the vocabulary wait for one another on four CTAs each while other SMs have none (active cycles 0 to 104
// thousand, 60 on average), and in a pass the warps wait for their loads (long scoreboard 5.2 warps an issue, barriers 3.4,
// the 64-bit pipe 8% busy, DRAM 12%).
#include <cooperative_groups.h>

#include "paged.h"

namespace cg = cooperative_groups;

namespace sgd {

namespace {

constexpr int kVerifyThreads = 512, kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyCluster = 8;  // CTAs of one sequence over a large vocabulary

// The same value in 64 bits.  The conversion instruction yields 16 results a cycle and SM, which would bound a pass
// over rows in L2; a positive normal number's bits are moved instead (exponent bias 1023 - 127 = 896 more).
__device__ __forceinline__ double as_double(float x) {
    const uint32_t b = __float_as_uint(x);
    if (b - 0x00800000u < 0x7f000000u) return __hiloint2double((b >> 3) + 0x38000000u, b << 29);
    return b == 0 ? 0.0 : (double)x;  // zero, subnormal, negative, infinite, NaN
}
__device__ __forceinline__ double as_double(__nv_bfloat16 x) { return as_double(__bfloat162float(x)); }

// max(x, 0) by the sign bit (a NaN passes)
__device__ __forceinline__ double positive(double x) { return __double2hiint(x) < 0 ? 0.0 : x; }

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
    double part[2][kVerifyCluster];               // every CTA's part of the sum, of this and the last one
    double wsum[kVerifyWarps];                    // this CTA's warps' parts
};

// N consecutive values, one load where N > 1
template <typename T, int N>
struct alignas(N * sizeof(T)) Chunk {
    T v[N];
};

// One cluster per sequence; each of its CTAs holds an equal part of the tokens, its warps equal consecutive parts of
// that.  Every CTA makes the same walk from the same sums, so none has to be told the way.
// VEC: tokens a lane loads at once, 4 where every row starts on such a boundary, else 1.
template <typename T, bool DRAWN, int VEC>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_kernel(VerifyArgs a, int ncta) {
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

    // the warp's tokens: whole vectors
    const int64_t parts = (int64_t)ncta * kVerifyWarps, n_vec = (V + VEC - 1) / VEC, per = (n_vec + parts - 1) / parts;
    const int64_t lo = min(((int64_t)rank * kVerifyWarps + warp) * per, n_vec) * VEC, hi = min(lo + per * VEC, V);

    int cur = 0, n_gone = 0, sums = 0;
    double c = 1.0, d = 0.0;
    constexpr int U = VEC == 1 ? 4 : DRAWN ? 1 : 2;  // loads of p in flight per lane, as many of q, twice
    constexpr int STEP = 32 * VEC;                  // tokens of a warp's load
    // A lane's part of the weights' sum over tokens [y0, y1) of a warp: tokens y0 + STEP u + VEC lane + e, the next
    // U loads on their way while these are summed, VEC sums side by side (a 64-bit addition's latency is long).
    auto sum_range = [&](int64_t y0, int64_t y1) -> double {
        const T *pr = P + cur * V, *qr = DRAWN ? Q + cur * V : nullptr;
        const bool resid = DRAWN && d != 0.0;
        struct Buf {
            Chunk<T, VEC> x[U], z[U];
        };
        double s[VEC] = {};
        auto load = [&](Buf &f, int64_t y0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t y = y0 + STEP * u + VEC * lane;
                if (y < y1) {
                    f.x[u] = *reinterpret_cast<const Chunk<T, VEC> *>(pr + y);
                    if (resid) f.z[u] = *reinterpret_cast<const Chunk<T, VEC> *>(qr + y);
                }
            }
        };
        auto add = [&](const Buf &f, int64_t y0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t y = y0 + STEP * u + VEC * lane;
                if (y < y1) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        double t = as_double(f.x[u].v[e]);
                        if constexpr (DRAWN) {
                            if (resid) t = positive(c * t - d * as_double(f.z[u].v[e]));
                        } else {
                            for (int j = 0; j < n_gone; ++j)
                                if (sh.gone[j] == y + e) t = 0.0;
                        }
                        s[e] += t;
                    }
                }
            }
        };
        Buf f[2];
        load(f[0], y0);
#pragma unroll 1
        for (; y0 < y1; y0 += 2 * STEP * U) {
            load(f[1], y0 + STEP * U);
            add(f[0], y0);
            load(f[0], y0 + 2 * STEP * U);
            add(f[1], y0 + STEP * U);
        }
        double t = s[0];
#pragma unroll
        for (int e = 1; e < VEC; ++e) t += s[e];
        return warp_sum_d(t);
    };
    auto weight_of = [&](int64_t y) {
        double t = as_double(P[cur * V + y]);
        if constexpr (DRAWN) {
            if (d != 0.0) t = positive(c * t - d * as_double(Q[cur * V + y]));
        } else {
            for (int j = 0; j < n_gone; ++j)
                if (sh.gone[j] == y) t = 0.0;
        }
        return t;
    };
    // The sum of all weights, the same bits in every CTA; sh.part[sums & 1] and sh.wsum keep its parts.
    auto sum_all = [&]() -> double {
        const double s = sum_range(lo, hi);
        __syncthreads();  // sh.wsum has been read
        if (lane == 0) sh.wsum[warp] = s;
        __syncthreads();
        ++sums;
        if (tid < ncta) {
            double t = 0.0;
            for (int w = 0; w < kVerifyWarps; ++w) t += sh.wsum[w];
            cluster.map_shared_rank(&sh, tid)->part[sums & 1][rank] = t;
        }
        cluster.sync();  // one is enough: the other buffer's readers are past it when it is written again
        double t = 0.0;
        for (int r = 0; r < ncta; ++r) t += sh.part[sums & 1][r];
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
            if (d != 0.0) w = positive(c * w - d * sh.qx[m]);
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
        const double s = sh.part[sums & 1][r];
        if (s > 0.0) last = r, last_before = before;
        if (at < 0 && before + s > thr) at = r, at_before = before;
        before += s;
    }
    if (at < 0) at = last, at_before = last_before;  // rounding at the very end, or nothing positive
    if (at == rank) {
        // of n parts with these sums, the one in which the sum from `base` on passes thr; base moves to its start
        auto locate = [&](const double *part, int n, double &base) {
            int in = -1, last = -1;
            double run = base, in_base = base, last_base = base;
            for (int i = 0; i < n; ++i) {
                const double s = part[i];
                if (s > 0.0) last = i, last_base = run;
                if (in < 0 && run + s > thr) in = i, in_base = run;
                run += s;
            }
            base = in >= 0 ? in_base : last_base;
            return in >= 0 ? in : last;
        };
        double base = at_before;
        const int wat = max(locate(sh.wsum, kVerifyWarps, base), 0);
        // that warp's tokens again, a sixteenth for each warp
        const int64_t from = min(((int64_t)rank * kVerifyWarps + wat) * per, n_vec) * VEC, to = min(from + per * VEC, V);
        const int64_t sub = (per + kVerifyWarps - 1) / kVerifyWarps * VEC;
        const int64_t s_lo = min(from + warp * sub, to), s_hi = min(s_lo + sub, to);
        const double s = sum_range(s_lo, s_hi);
        __syncthreads();
        if (lane == 0) sh.wsum[warp] = s;
        __syncthreads();
        if (warp == max(locate(sh.wsum, kVerifyWarps, base), 0)) {
            int64_t pick = -1, high = -1;  // high: the last token with a positive weight
            double run = base;
            for (int64_t y0 = s_lo; y0 < s_hi && pick < 0; y0 += STEP) {
                const int64_t y = y0 + VEC * lane;
                double w[VEC], mine = 0.0;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    w[e] = y + e < s_hi ? weight_of(y + e) : 0.0;
                    mine += w[e];
                }
                double inc = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double up = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += up;
                }
                int first = VEC, top = -1;  // the lane's first token that passes thr, its last positive one
                double acc = run + (inc - mine);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    acc += w[e];
                    if (w[e] > 0.0) {
                        top = e;
                        if (acc > thr && first == VEC) first = e;
                    }
                }
                const unsigned over = __ballot_sync(0xffffffffu, first < VEC), pos = __ballot_sync(0xffffffffu, top >= 0);
                if (pos) {
                    const int l = 31 - __clz(pos);
                    high = y0 + VEC * l + __shfl_sync(0xffffffffu, top, l);
                }
                if (over) {
                    const int l = __ffs(over) - 1;
                    pick = y0 + VEC * l + __shfl_sync(0xffffffffu, first, l);
                }
                run += __shfl_sync(0xffffffffu, inc, 31);
            }
            if (lane == 0) a.next[b] = (int32_t)max(pick >= 0 ? pick : high, (int64_t)0);
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
int launch(const VerifyArgs &a, int sms, cudaStream_t s) {
    // A vocabulary of up to 8192 tokens is one CTA's (16 to a thread; a cluster's barriers cost more).  Larger ones take
    // as many CTAs, up to 8, as keep the batch resident at two CTAs per SM: the passes of a sequence depend on each
    // other, so a second wave would double the time.
    int ncta = 1;
    while (a.V > 8192 && ncta < kVerifyCluster && 2 * ncta * a.B <= 2 * sms) ncta *= 2;
    constexpr int VEC = 4;
    auto k = a.V % VEC == 0 ? verify_kernel<T, DRAWN, VEC> : verify_kernel<T, DRAWN, 1>;
    const cudaError_t e = launch_k(k, dim3(a.B * ncta), dim3(kVerifyThreads), 0, s, ncta, a, ncta);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? SGD_OK : SGD_ERR_CUDA;
}

}  // namespace

int launch_verify(const VerifyArgs &a, int sms, cudaStream_t s) {
    if (a.f32) return a.q ? launch<float, true>(a, sms, s) : launch<float, false>(a, sms, s);
    return a.q ? launch<__nv_bfloat16, true>(a, sms, s) : launch<__nv_bfloat16, false>(a, sms, s);
}

}  // namespace sgd
