// paged_attn.cu -- attention of a step's query tokens over the paged cache (sgd_paged_attn in
// include/sgd.h).
//
// The M query tokens and G heads of a KV head are the rows of a matrix product with the cache:
// S = Q K^T over tiles of 128 tokens (two pages), P = exp2(S scale - m) under the row's mask, O += P V, with
// the running maximum m and sum l of each row.  Both products run on the tensor cores with their
// accumulators in tensor memory: a row of S, P and O is one of its 128 lanes, so a softmax thread
// owns a whole row and needs no exchange with another.  P (bf16) replaces S in tensor memory and is the
// second product's A operand from there; V is its B operand as it lies in the page (MN-major).
//
// Up to 128 rows (M * G): one row tile a CTA, its KV tiles taken in turn by two softmax warpgroups,
// each with its own S and O, merged at the end of the segment; so one computes its softmax while the
// tensor cores work for the other.  More rows: two row tiles a CTA over the same KV tiles, and ranges
// of ceil(rows / 256) CTAs side by side that read the same tiles at the same time (from L2 but the
// first).  Either way the warpgroups g = 0, 1 alternate on the tensor cores:
//   QK_0 QK_1 | PV_0 QK_0 PV_1 QK_1 | PV_0 QK_0 ...
//
// The work is cut without the host: every CTA sums the rows' tile counts itself (a window leaves the
// tiles of the first tokens and of the window only), takes an equal range of the stream of all (row,
// KV head) items' tiles, and walks it segment by segment.  A segment that is its whole item writes the
// result, others leave normalised partial rows, which paged_merge_kernel joins.
//
// The running maximum is a reference only: it follows the true one when it is passed by more than 8 in
// log2 (p then stays below 2^8, exact in range), which happens a few times in a long row, and
// O is rescaled in tensor memory only then.  S, m, l and O are float32; P is rounded to bf16 (2^-8
// relative), as is the output; l sums the unrounded p.
#include <math.h>
#include <string.h>

#include <algorithm>

#include <cudaTypedefs.h>

#include "paged.h"
#include "quant.cuh"
#include "scan.cuh"
#include "tc.cuh"

namespace sgd {

namespace {

constexpr int kTile = 128;       // tokens of a KV tile, rows of a row tile
constexpr int kItemCharge = 2;   // tiles of work charged to an item beside its own (start, epilogue)
constexpr float kSlack = 8.f;    // log2 by which the true maximum may pass the reference
constexpr int kWarpProducer = 0, kWarpMma = 1, kWarpSoftmax = 4;  // softmax: warps 4..11

// What a launch needs beside the cache and the arguments.
struct AttnPlan {
    int Mt;        // query tokens of a row tile: 128 / G
    int RT;        // CTAs per range: ceil(row tiles / 2) with two row tiles a CTA, else 1
    int n_ranges;  // grid / RT
    float *o_part;     // [grid * 2, rows of a CTA, D] partial outputs, normalised
    float *lse_part;   // [grid * 2, rows of a CTA], log2 units
    int2 *item;        // [B * Hkv] first and last range of each item
};

// A row of the page table in a launch.
struct Seq {
    int L, n, base;  // tokens, nodes, entries before the nodes
    int sink_tiles;  // tiles of the first tokens that do not belong to the window
    int first;       // the window's first tile
    int tiles;       // >= 1
};

__device__ __forceinline__ Seq seq_of(const PagedView &kv, const PagedAttnArgs &a, int b, int &bad) {
    Seq s;
    const int room = kv.max_pages * SGD_PAGE;
    const int L = kv.lens[b];
    s.L = min(max(L, 0), room);
    if (s.L != L) bad |= SGD_STATUS_SIZE_MISMATCH;
    s.n = a.M;
    if (a.n_nodes) {
        const int n = a.n_nodes[b];
        s.n = min(max(n, 0), a.M);
        if (s.n != n) bad |= SGD_STATUS_BAD_INDEX;
    }
    s.base = s.L - s.n;
    const int all = (s.L + kTile - 1) / kTile;
    s.sink_tiles = s.first = 0;
    if (a.window) {
        s.first = max(s.base + 1 - a.window, 0) / kTile;
        s.sink_tiles = min((int)(((int64_t)a.sinks + kTile - 1) / kTile), s.first);
    }
    s.tiles = s.n == 0 ? 1 : max(1, s.sink_tiles + all - s.first);
    return s;
}

__device__ __forceinline__ int tile_of(const Seq &s, int v) { return v < s.sink_tiles ? v : v - s.sink_tiles + s.first; }

// bits i of 0..31 with from <= i < to
__device__ __forceinline__ uint32_t bits(int from, int to) {
    from = max(from, 0);
    to = min(to, 32);
    if (from >= to) return 0;
    return (to == 32 ? 0xffffffffu : (1u << to) - 1u) & ~((1u << from) - 1u);
}

template <int D_, bool I8_, bool TWO_>
struct Cfg {
    static constexpr int D = D_;
    static constexpr bool I8 = I8_, TWO = TWO_;
    static constexpr int HALVES = D / 64;                 // 64-channel halves, 16 KB each of a tile
    static constexpr int TILE_BYTES = kTile * D * 2;
    static constexpr int Q_BUFS = 2;                      // TWO: the two row tiles; else two segments'
    static constexpr int Q_STAGES = TWO ? 1 : 2;
    static constexpr int SLOTS = I8 ? (D == 128 ? 3 : 4) : (D == 128 ? 5 : 8);  // bf16 tiles of K or V
    static constexpr int RAW = I8 ? (D == 128 ? 4 : 8) : 0;                     // code tiles in flight
    static constexpr int RAW_BYTES = kTile * D;
    static constexpr int THREADS = I8 ? 512 : 384;
    static constexpr int ROWS = TWO ? 256 : 128;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_SLOT = Q_BUFS * TILE_BYTES;
    static constexpr int OFF_RAW = OFF_SLOT + SLOTS * TILE_BYTES;
    static constexpr int OFF_ML = OFF_RAW + RAW * RAW_BYTES;  // [2][128] (m, l) of the warpgroups
    static constexpr int OFF_BAR = OFF_ML + 2 * 128 * 8;
    static constexpr int SMEM = OFF_BAR + 512;
    static_assert(SMEM <= 232448, "fits a CTA's shared memory");
};

struct Bars {
    uint64_t full[8], empty[8];          // ring of bf16 K / V tiles, in the order the products take them
    uint64_t raw_full[8], raw_empty[8];  // I8: ring of code tiles
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t o_free, ml_full, drained;
    uint32_t tmem;
    int32_t abort;
    int32_t start_b, start_pos;          // the range's first row and its stream position
    int32_t sm[33];
};
static_assert(sizeof(Bars) <= 512, "barriers fit their space");

// Ring position of K and V of the j-th of T tiles of a segment, counted from the segment's first: the
// order in which the products take them.
template <bool TWO>
__device__ __forceinline__ int pos_k(int j) {
    return TWO ? 2 * j : (j < 2 ? j : 2 * j - 1);
}
template <bool TWO>
__device__ __forceinline__ int pos_v(int j, int T) {
    return TWO ? 2 * j + 1 : min(2 * j + 2, 2 * T - 1);
}

// Walks a CTA's range: the same sequence of segments in every role.
struct Walk {
    int b, h, start, x0, x1;  // item (b, h) starts at stream position `start`
    Seq s;
    bool fresh;               // b changed with the present segment
    int lo, hi;               // tiles of the present segment
    __device__ __forceinline__ void init(const PagedView &kv, const PagedAttnArgs &a, int b0, int pos0, int from, int to) {
        x0 = from, x1 = to;
        b = b0, start = pos0;
        h = -1;
        fresh = true;
        if (b < kv.B) {
            int bad = 0;
            s = seq_of(kv, a, b, bad);
            const int len = s.tiles + kItemCharge;
            h = (x0 - start) / len;
            start += h * len;
            --h;
            start -= len;  // next() steps onto it
        }
    }
    // to the next segment with tiles; false at the end of the range
    __device__ __forceinline__ bool next(const PagedView &kv, const PagedAttnArgs &a) {
        while (b < kv.B) {
            start += s.tiles + kItemCharge;
            if (++h == kv.Hkv) {
                h = 0;
                if (++b == kv.B) return false;
                int bad = 0;
                s = seq_of(kv, a, b, bad);
                fresh = true;
            }
            if (start >= x1) return false;
            lo = max(x0, start) - start;
            hi = min(x1 - start, s.tiles);
            if (lo < hi) return true;
        }
        return false;
    }
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    paged_attn_kernel(PagedView kv, PagedAttnArgs a, AttnPlan plan, const __grid_constant__ CUtensorMap map_q,
                      const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars &bar = *reinterpret_cast<Bars *>(smem + C::OFF_BAR);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int range = blockIdx.x / plan.RT, rt = blockIdx.x % plan.RT;
    constexpr int D = C::D;

    // rows of the CTA's row tiles, and the softmax warps that have any
    int rows[2], warps[2];
    for (int g = 0; g < 2; ++g) {
        const int m0 = (C::TWO ? rt * 2 + g : 0) * plan.Mt;
        rows[g] = max(0, min(plan.Mt, a.M - m0)) * a.G;
        warps[g] = max(1, (rows[g] + 31) / 32);
    }

    if (tid == 0) {
        for (int i = 0; i < C::SLOTS; ++i) {
            mbar_init(&bar.full[i], C::I8 ? 4 : 1);
            mbar_init(&bar.empty[i], 1);
        }
        for (int i = 0; i < C::RAW; ++i) {
            mbar_init(&bar.raw_full[i], 1);
            mbar_init(&bar.raw_empty[i], 4);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(&bar.q_full[g], 1);
            mbar_init(&bar.q_empty[g], 1);
            mbar_init(&bar.s_full[g], 1);
            mbar_init(&bar.p_full[g], warps[g]);
            mbar_init(&bar.o_full[g], 1);
        }
        mbar_init(&bar.o_free, warps[0] + warps[1]);
        mbar_init(&bar.ml_full, warps[0] + warps[1]);
        mbar_init(&bar.drained, 1);
        bar.abort = 0;
        bar.start_b = kv.B;
        bar.start_pos = 0;
        fence_barrier_init();
        prefetch_tensormap(&map_q);
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
    }
    if (warp == kWarpMma) tmem_alloc(&bar.tmem, 512);

    // the stream's length, this range of it, and the row it starts in: thread t sums consecutive rows
    int x0, x1;
    {
        const int per = (kv.B + C::THREADS - 1) / C::THREADS;
        const int b0 = min(tid * per, kv.B), b1 = min(b0 + per, kv.B);
        int sum = 0, bad = 0;
        for (int b = b0; b < b1; ++b) sum += (seq_of(kv, a, b, bad).tiles + kItemCharge) * kv.Hkv;
        if (bad && blockIdx.x == 0) atomicOr(a.status, bad);
        int total;
        int pos = block_exclusive_scan(sum, total, bar.sm);
        const int S = (total + plan.n_ranges - 1) / plan.n_ranges;
        x0 = min((int64_t)range * S, (int64_t)total);
        x1 = min(x0 + S, total);
        if (x0 < x1 && pos <= x0 && x0 < pos + sum) {
            for (int b = b0; b < b1; ++b) {
                const int len = (seq_of(kv, a, b, bad).tiles + kItemCharge) * kv.Hkv;
                if (x0 < pos + len) {
                    bar.start_b = b;
                    bar.start_pos = pos;
                    break;
                }
                pos += len;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    volatile int32_t *abort = &bar.abort;
    auto wait = [&](uint64_t *m, uint32_t parity) { return mbar_wait(m, parity, a.status, abort, a.wait_limit); };
    // the same answer in every lane, so that the warp stays together
    auto wait_warp = [&](uint64_t *m, uint32_t parity) { return (bool)__all_sync(0xffffffffu, wait(m, parity)); };
    Walk w;
    w.init(kv, a, bar.start_b, bar.start_pos, x0, x1);

    if (warp == kWarpProducer) {
        // ------------------------------------------------------------------ loads
        if (lane == 0 && !a.idle_producer) {
            const uint64_t policy = l2_evict_first_policy();
            constexpr int N = C::I8 ? C::RAW : C::SLOTS;
            uint64_t *full = C::I8 ? bar.raw_full : bar.full, *empty = C::I8 ? bar.raw_empty : bar.empty;
            uint32_t at = 0;   // ring position
            uint32_t seg = 0;  // segment of this CTA
            bool go = true;
            int bad = 0;
            auto load = [&](const CUtensorMap &map, int tile) {
                const int slot = at % N;
                if (at >= N && !wait(&empty[slot], (at / N - 1) & 1)) return go = false;
                const int32_t *row = kv.table + (int64_t)w.b * kv.max_pages;
                const int p0 = tile * 2, have = (w.s.L + SGD_PAGE - 1) / SGD_PAGE - p0;  // pages of this tile
                const int np = min(max(have, 0), 2);
                uint8_t *dst = smem + (C::I8 ? C::OFF_RAW + slot * C::RAW_BYTES : C::OFF_SLOT + slot * C::TILE_BYTES);
                if (np) mbar_arrive_expect_tx(&full[slot], np * SGD_PAGE * D * (C::I8 ? 1 : 2));
                else mbar_arrive(&full[slot]);  // a row without tokens: nothing of the tile is used
                for (int i = 0; i < np; ++i) {
                    int p = row[p0 + i];
                    if (p < 0 || p >= kv.n_pages) {
                        bad = SGD_STATUS_BAD_INDEX;
                        p = 0;
                    }
                    const int y = (p * kv.Hkv + w.h) * SGD_PAGE;
                    if constexpr (C::I8) {
                        tma_load_2d(dst + i * SGD_PAGE * D, &map, &full[slot], 0, y, policy);
                    } else {
                        for (int e = 0; e < C::HALVES; ++e)
                            tma_load_2d(dst + e * kTile * 128 + i * SGD_PAGE * 128, &map, &full[slot], e * 64, y, policy);
                    }
                }
                ++at;
                return true;
            };
            while (go && w.next(kv, a)) {
                const int qs = seg % C::Q_STAGES;
                if (seg >= C::Q_STAGES && !wait(&bar.q_empty[qs], (seg / C::Q_STAGES - 1) & 1)) break;
                const int mb = min(plan.Mt, a.M);  // query tokens of the box
                const int n_tiles = C::TWO && rows[1] > 0 ? 2 : 1;
                mbar_arrive_expect_tx(&bar.q_full[qs], n_tiles * mb * a.G * D * 2);
                for (int g = 0; g < n_tiles; ++g)
                    for (int e = 0; e < C::HALVES; ++e)
                        tma_load_4d(smem + C::OFF_Q + (C::TWO ? g : qs) * C::TILE_BYTES + e * kTile * 128, &map_q,
                                    &bar.q_full[qs], e * 64, w.h * a.G, (C::TWO ? rt * 2 + g : 0) * plan.Mt, w.b);
                ++seg;
                const int T = w.hi - w.lo;
                if constexpr (C::TWO) {
                    for (int j = 0; go && j < T; ++j) {
                        const int tile = tile_of(w.s, w.lo + j);
                        go = load(map_k, tile) && load(map_v, tile);
                    }
                } else {
                    for (int j = 0; go && j < min(T, 2); ++j) go = load(map_k, tile_of(w.s, w.lo + j));
                    for (int j = 0; go && j < T; ++j) {
                        go = load(map_v, tile_of(w.s, w.lo + j));
                        if (go && j + 2 < T) go = load(map_k, tile_of(w.s, w.lo + j + 2));
                    }
                }
            }
            if (bad) atomicOr(a.status, bad);
            if (*abort) {  // no copy may still be writing when the CTA ends
                for (uint32_t i = at > N ? at - N : 0; i < at; ++i) mbar_drain(&full[i % N], (i / N) & 1, a.wait_limit);
                for (uint32_t i = seg > C::Q_STAGES ? seg - C::Q_STAGES : 0; i < seg; ++i)
                    mbar_drain(&bar.q_full[i % C::Q_STAGES], (i / C::Q_STAGES) & 1, a.wait_limit);
            }
        }
    } else if (warp == kWarpMma) {
        // ------------------------------------------------------------------ products
        if (lane == 0) {
            constexpr uint32_t ID_QK = tc_idesc_bf16(128, kTile, false), ID_PV = tc_idesc_bf16(128, D, true);
            const uint32_t sq = smem_u32(smem + C::OFF_Q), ss = smem_u32(smem + C::OFF_SLOT);
            uint32_t at = 0, seg = 0, np[2] = {0, 0};
            bool go = true;
            auto full = [&](uint32_t pos) {
                if (go) go = wait(&bar.full[pos % C::SLOTS], (pos / C::SLOTS) & 1);
                return go;
            };
            auto qk = [&](int g, uint32_t q, uint32_t pos) {  // S_g = Q K^T
                const uint32_t k = ss + (pos % C::SLOTS) * C::TILE_BYTES;
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    const uint32_t off = (j / 4) * (kTile * 128) + (j % 4) * 32;
                    mma_ss(tmem + g * 128, desc_k_major(q + off), desc_k_major(k + off), ID_QK, j > 0);
                }
            };
            auto pv = [&](int g, uint32_t pos, bool acc) {  // O_g (+)= P_g V
                const uint32_t v = ss + (pos % C::SLOTS) * C::TILE_BYTES;
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < kTile / 16; ++j)
                    mma_ts(tmem + 256 + g * 128, tmem + g * 128 + j * 8, desc_mn_major(v + j * 2048, kTile * 128), ID_PV,
                           acc || j > 0);
            };
            auto release = [&](uint32_t pos) { tc_commit(&bar.empty[pos % C::SLOTS]); };
            auto p_ready = [&](int g) {
                if (go) go = wait(&bar.p_full[g], np[g]++ & 1);
                return go;
            };
            while (go && w.next(kv, a)) {
                const int T = w.hi - w.lo, qs = seg % C::Q_STAGES;
                if (!wait(&bar.q_full[qs], (seg / C::Q_STAGES) & 1)) break;
                const uint32_t q0 = sq + (C::TWO ? 0 : qs) * C::TILE_BYTES;
                auto o_free = [&](int j, int first) {  // before a segment's first PV: the last one's O was read
                    if (j == first && seg > 0 && go) go = wait(&bar.o_free, (seg - 1) & 1);
                    return go;
                };
                if constexpr (C::TWO) {
                    if (!full(at)) break;
                    for (int g = 0; g < 2; ++g) {
                        qk(g, q0 + g * C::TILE_BYTES, at);
                        tc_commit(&bar.s_full[g]);
                    }
                    release(at);
                    if (T == 1) tc_commit(&bar.q_empty[qs]);
                    for (int j = 0; j < T; ++j) {
                        const uint32_t pv_at = at + pos_v<true>(j, T), k_at = at + pos_k<true>(j + 1);
                        for (int g = 0; g < 2; ++g) {
                            if (!o_free(j, 0) || !p_ready(g) || !full(pv_at)) break;
                            pv(g, pv_at, j > 0);
                            if (j + 1 < T) {
                                if (!full(k_at)) break;
                                qk(g, q0 + g * C::TILE_BYTES, k_at);
                                tc_commit(&bar.s_full[g]);
                            } else {
                                tc_commit(&bar.o_full[g]);
                            }
                        }
                        if (!go) break;
                        release(pv_at);
                        if (j + 1 < T) release(k_at);
                        if (j + 2 == T) tc_commit(&bar.q_empty[qs]);
                    }
                } else {
                    for (int g = 0; g < min(T, 2); ++g) {
                        if (!full(at + g)) break;
                        qk(g, q0, at + g);
                        release(at + g);
                        tc_commit(&bar.s_full[g]);
                    }
                    if (T <= 2) tc_commit(&bar.q_empty[qs]);
                    for (int j = 0; go && j < T; ++j) {
                        const int g = j & 1;
                        const uint32_t pv_at = at + pos_v<false>(j, T), k_at = at + pos_k<false>(j + 2);
                        if (!o_free(j, 0) || !p_ready(g) || !full(pv_at)) break;
                        pv(g, pv_at, j > 1);
                        release(pv_at);
                        if (j + 2 < T) {
                            if (!full(k_at)) break;
                            qk(g, q0, k_at);
                            release(k_at);
                            tc_commit(&bar.s_full[g]);
                            if (j + 3 == T) tc_commit(&bar.q_empty[qs]);
                        } else {
                            tc_commit(&bar.o_full[g]);
                        }
                    }
                }
                at += 2 * T;
                ++seg;
            }
            // no product may still be reading, and no arrival be due, when the CTA ends
            tc_commit(&bar.drained);
            mbar_drain(&bar.drained, 0, a.wait_limit);
        }
    } else if (warp >= kWarpSoftmax && warp < kWarpSoftmax + 8) {
        // ------------------------------------------------------------------ softmax
        const int g = (warp - kWarpSoftmax) >> 2, wq = warp & 3;
        const int r = wq * 32 + lane;             // row of the tile = lane of tensor memory
        const int na = warps[g];                  // softmax warps of this group at work
        if (wq < na) {
            const bool valid = r < rows[g];
            const int m = (C::TWO ? rt * 2 + g : 0) * plan.Mt + r / a.G, gh = r % a.G;
            const uint32_t lane_at = tmem + ((uint32_t)(wq * 32) << 16);
            const uint32_t ts = lane_at + g * 128, to = lane_at + 256 + g * 128;
            float scale = a.scale_log2, vs = 1.f;
            if constexpr (C::I8) {
                const bool report = blockIdx.x == 0 && g == 0 && r == 0;
                scale *= calibrated_scale(kv.k_scale, a.status, report);
                vs = calibrated_scale(kv.v_scale, a.status, report);
            }
            uint32_t at = 0, seg = 0, ns = 0, no[2] = {0, 0};
            float2 *ml = reinterpret_cast<float2 *>(smem + C::OFF_ML);
            int lo = 0;          // the first entry of the row's window
            uint64_t sees = 0;   // the nodes that the row sees
            bool go = true;
            while (go && w.next(kv, a)) {
                const int T = w.hi - w.lo;
                const Seq &s = w.s;
                if (w.fresh) {  // the row's mask in this sequence: a walk up to its root
                    w.fresh = false;
                    sees = 0;
                    lo = a.window ? s.L : 0;
                    if (valid && m < s.n) {
                        const int32_t *par = a.parent ? a.parent + (int64_t)w.b * a.M : nullptr;
                        int bad = 0;
                        auto up = [&](int j) {
                            if (!par) return j - 1;
                            const int p = par[j];
                            if (p >= -1 && p < j) return p;
                            bad = SGD_STATUS_BAD_INDEX;
                            return -1;
                        };
                        int depth = 0;
                        for (int j = m; j >= 0; j = up(j)) {
                            // `depth` steps above m: in the window if depth < window
                            if (s.base + j >= 0 && (!a.window || depth < a.window)) sees |= 1ull << j;
                            ++depth;
                        }
                        const int pos = s.base + depth - 1;  // the row's position
                        if (a.window) {
                            lo = max(pos + 1 - a.window, 0);
                            if (s.base < a.sinks) {  // ancestors among the first tokens
                                int d = depth - 1;
                                for (int j = m; j >= 0; j = up(j), --d)
                                    if (s.base + j >= 0 && s.base + d < a.sinks) sees |= 1ull << j;
                            }
                        }
                        if (bad) atomicOr(a.status, bad);
                    }
                }
                const bool query = valid && m < s.n;
                const int prefix = query && s.base > 0 ? s.base : 0;  // entries before the nodes that the row may see
                const int sink = min(a.sinks, prefix);
                const int v_lo = s.base + 1 - a.window;               // no row sees an entry of [sinks, v_lo)
                float mx = -INFINITY, l = 0.f;
                for (int j = C::TWO ? 0 : g; j < T; j += C::TWO ? 1 : 2) {
                    const int t0 = tile_of(s, w.lo + j) * kTile;
                    // entries that no row sees may hold anything: their V rows become 0
                    const bool clean = t0 + kTile > s.L || (a.window && t0 < v_lo && t0 + kTile > a.sinks);
                    if (clean) {
                        const uint32_t pos = at + pos_v<C::TWO>(j, T);
                        if (!(go = wait_warp(&bar.full[pos % C::SLOTS], (pos / C::SLOTS) & 1))) break;
                        uint8_t *v = smem + C::OFF_SLOT + (pos % C::SLOTS) * C::TILE_BYTES;
                        for (int i = wq; i < kTile; i += na) {
                            const int t = t0 + i;
                            if ((t >= s.L || (a.window && t >= a.sinks && t < v_lo)) && lane < D / 8)
                                *reinterpret_cast<uint4 *>(v + (lane / 8) * kTile * 128 + i * 128 + (lane % 8) * 16) =
                                    make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_shared();
                    }
                    if (!(go = wait_warp(&bar.s_full[g], ns & 1))) break;
                    ++ns;
                    tc_fence_after();
                    const bool masked = __any_sync(
                        0xffffffffu, t0 + kTile > prefix || (lo > t0 && t0 + kTile > sink));
                    auto mask_of = [&](int c) {  // the row's entries among the 32 from t0 + 32 c
                        const int tw = t0 + c * 32, off = s.base - tw;
                        uint32_t k = bits(lo - tw, prefix - tw) | bits(-tw, sink - tw);
                        if (off >= 0) {
                            if (off < 32) k |= (uint32_t)(sees << off);
                        } else if (off > -64) {
                            k |= (uint32_t)(sees >> -off);
                        }
                        return k;
                    };
                    // the row's maximum
                    float top = -INFINITY;
                    if (masked) {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t x[32];
                            tmem_ld32(x, ts + c * 32);
                            tmem_wait_ld();
                            const uint32_t k = mask_of(c);
#pragma unroll
                            for (int i = 0; i < 32; ++i) top = fmaxf(top, k >> i & 1 ? __uint_as_float(x[i]) : -INFINITY);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t x[32];
                            tmem_ld32(x, ts + c * 32);
                            tmem_wait_ld();
                            float t4[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                            for (int i = 0; i < 32; ++i) t4[i & 3] = fmaxf(t4[i & 3], __uint_as_float(x[i]));
                            top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
                        }
                    }
                    const float mt = top == -INFINITY ? -INFINITY : top * scale;
                    const bool first = j < 2 && (C::TWO ? j == 0 : true);
                    if (__any_sync(0xffffffffu, mt > mx + kSlack)) {
                        const float m2 = fmaxf(mx, mt), f = mx == -INFINITY ? 0.f : ex2(mx - m2);
                        mx = m2;
                        l *= f;
                        if (!first) {
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t x[32];
                                tmem_ld32(x, to + c * 32);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                                tmem_st32(to + c * 32, x);
                            }
                        }
                    }
                    const float ref = mx == -INFINITY ? 0.f : mx;
                    // p, its sum, and P in the place of S (a chunk's columns of P lie among those of S read before)
                    float l4[4] = {0.f, 0.f, 0.f, 0.f};
                    if (masked) {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t x[32], y[16];
                            tmem_ld32(x, ts + c * 32);
                            tmem_wait_ld();
                            const uint32_t k = mask_of(c);
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                const float p0 = k >> i & 1 ? ex2(fmaf(__uint_as_float(x[i]), scale, -ref)) : 0.f;
                                const float p1 = k >> (i + 1) & 1 ? ex2(fmaf(__uint_as_float(x[i + 1]), scale, -ref)) : 0.f;
                                l4[i & 2] += p0;
                                l4[(i & 2) + 1] += p1;
                                y[i / 2] = pack_bf16(p0, p1);
                            }
                            tmem_st16(ts + c * 16, y);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t x[32], y[16];
                            tmem_ld32(x, ts + c * 32);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                const float p0 = ex2(fmaf(__uint_as_float(x[i]), scale, -ref));
                                const float p1 = ex2(fmaf(__uint_as_float(x[i + 1]), scale, -ref));
                                l4[i & 2] += p0;
                                l4[(i & 2) + 1] += p1;
                                y[i / 2] = pack_bf16(p0, p1);
                            }
                            tmem_st16(ts + c * 16, y);
                        }
                    }
                    l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.p_full[g]);
                }
                if (!go) break;

                // the segment's result
                const bool whole = w.lo == 0 && w.hi == s.tiles;
                const int64_t out_row = (((int64_t)w.b * a.M + m) * kv.Hkv + w.h) * a.G + gh;
                const int64_t part_row =
                    ((int64_t)blockIdx.x * 2 + (w.lo == 0)) * C::ROWS + (C::TWO ? g * 128 : 0) + r;
                float f0, f1 = 0.f, sum, ref;  // O_0 f0 + O_1 f1 is the normalised row
                constexpr int NO = C::TWO ? 1 : 2;
                if constexpr (C::TWO) {
                    sum = l, ref = mx;
                    f0 = sum > 0.f ? vs / sum : 0.f;
                } else {
                    // every warp has read the last segment's pair
                    if (seg > 0 && !(go = wait_warp(&bar.o_free, (seg - 1) & 1))) break;
                    ml[g * 128 + r] = make_float2(mx, l);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.ml_full);
                    if (!(go = wait_warp(&bar.ml_full, seg & 1))) break;
                    const float2 u = ml[r], v = ml[128 + r];
                    ref = fmaxf(u.x, v.x);
                    const float e0 = u.y > 0.f ? ex2(u.x - ref) : 0.f, e1 = v.y > 0.f ? ex2(v.x - ref) : 0.f;
                    sum = e0 * u.y + e1 * v.y;
                    f0 = sum > 0.f ? vs * e0 / sum : 0.f;
                    f1 = sum > 0.f ? vs * e1 / sum : 0.f;
                }
                for (int i = 0; i < 2; ++i) {
                    if (C::TWO ? i != g : i >= T) continue;
                    if (!(go = wait_warp(&bar.o_full[i], no[i]++ & 1))) break;
                }
                if (!go) break;
                tc_fence_after();
                // TWO: the row's D channels; else this group's half of them, from both accumulators
                constexpr int NC = C::TWO ? D / 32 : D / 64;
#pragma unroll 1
                for (int c = 0; c < NC; ++c) {
                    const int col = C::TWO ? c * 32 : g * (D / 2) + c * 32;
                    uint32_t x[32];
                    float o[32];
                    tmem_ld32(x, lane_at + 256 + (C::TWO ? g * 128 : 0) + col);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = f0 != 0.f ? f0 * __uint_as_float(x[i]) : 0.f;
                    if constexpr (NO == 2) {
                        if (T > 1) {
                            tmem_ld32(x, lane_at + 256 + 128 + col);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] += f1 != 0.f ? f1 * __uint_as_float(x[i]) : 0.f;
                        }
                    }
                    if (valid && whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + out_row * D + col);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            dst[i] = make_uint4(pack_bf16(o[8 * i], o[8 * i + 1]), pack_bf16(o[8 * i + 2], o[8 * i + 3]),
                                                pack_bf16(o[8 * i + 4], o[8 * i + 5]), pack_bf16(o[8 * i + 6], o[8 * i + 7]));
                    } else if (valid) {
                        float4 *dst = reinterpret_cast<float4 *>(plan.o_part + part_row * D + col);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                    __syncwarp();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.o_free);
                if (valid && (C::TWO || g == 0)) {
                    const float lse2 = sum > 0.f ? ref + log2f(sum) : -INFINITY;
                    if (whole) a.lse[out_row] = lse2 * 0.69314718055994531f;
                    else plan.lse_part[part_row] = lse2;
                }
                if (w.lo == 0 && rt == 0 && g == 0 && r == 0) {  // ranges of S tiles: the one that holds its last tile
                    const int S = x1 - x0;  // exact: an item that goes on is not in the last range
                    plan.item[w.b * kv.Hkv + w.h] = make_int2(range, whole ? range : (w.start + s.tiles - 1) / S);
                }
                at += 2 * T;
                ++seg;
            }
        }
    } else if (C::I8 && warp >= 12) {
        // ------------------------------------------------------------------ codes to bf16
        // u = 0x4300 | byte is the bf16 number 128 + (byte & 127) with the sign bit where 256's
        // exponent differs from 128's: (u without bit 7) - (u without bits 0-6) = byte as a signed number,
        // exactly
        const int ct = tid - 12 * 32;
        uint32_t at = 0;
        bool go = true;
        while (go && w.next(kv, a)) {
            const int T = w.hi - w.lo;
            for (int i = 0; i < 2 * T; ++i, ++at) {
                constexpr int RAW = C::RAW > 0 ? C::RAW : 1;
                const int rs = at % RAW, bs = at % C::SLOTS;
                if (!(go = wait_warp(&bar.raw_full[rs], (at / RAW) & 1))) break;
                if (at >= C::SLOTS && !(go = wait_warp(&bar.empty[bs], (at / C::SLOTS - 1) & 1))) break;
                const uint8_t *src = smem + C::OFF_RAW + rs * C::RAW_BYTES;
                uint8_t *dst = smem + C::OFF_SLOT + bs * C::TILE_BYTES;
                constexpr int UNITS = kTile * D / 16;  // 16 codes each
#pragma unroll 2
                for (int u = ct; u < UNITS; u += 128) {
                    const int row = u / (D / 16), cb = u % (D / 16);
                    const uint4 x = *reinterpret_cast<const uint4 *>(src + u * 16);
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                    uint32_t y[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t e = __byte_perm(xs[k / 2], 0x43434343u, k & 1 ? 0x4342 : 0x4140);
                        const uint32_t hi = e & 0xff7fff7fu, lo = e & 0xff80ff80u;
                        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&hi),
                                                         *reinterpret_cast<const __nv_bfloat162 *>(&lo));
                        y[k] = *reinterpret_cast<const uint32_t *>(&d);
                    }
                    // two 16-byte pieces of the swizzled row; the second half's threads start with the odd one, so
                    // that a quarter warp's stores cover all banks
                    uint8_t *base = dst + (cb / 4) * (kTile * 128) + row * 128;
                    const int ch = (cb % 4) * 2, odd = cb / 4 & 1;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int e = k ^ odd;
                        *reinterpret_cast<uint4 *>(base + (((ch + e) ^ (row & 7)) * 16)) =
                            e ? make_uint4(y[4], y[5], y[6], y[7]) : make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bar.full[bs]);
                    mbar_arrive(&bar.raw_empty[rs]);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the partial rows of an item that several ranges share: one CTA per output row, its warps take
// the ranges in turn.  lse = log2 sum_c 2^lse_c, out = sum_c 2^(lse_c - lse) o_c.
template <int D>
__global__ void __launch_bounds__(128) paged_merge_kernel(PagedView kv, PagedAttnArgs a, AttnPlan plan, int two) {
    __shared__ float so[4][D], sl[4], sm[4];
    const int Hq = kv.Hkv * a.G;
    const int64_t out_row = blockIdx.x;
    const int hq = (int)(out_row % Hq), m = (int)(out_row / Hq % a.M), b = (int)(out_row / Hq / a.M);
    const int2 it = plan.item[b * kv.Hkv + hq / a.G];
    if (it.x == it.y || it.x < 0 || it.y >= plan.n_ranges || it.x > it.y) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mt = m / plan.Mt, rt = two ? mt / 2 : 0, rows = two ? 256 : 128;
    const int r = (two ? mt % 2 * 128 : 0) + (m % plan.Mt) * a.G + hq % a.G;
    constexpr int E = D / 32;
    float mx = -INFINITY, l = 0.f, o[E] = {};
    constexpr int U = 4;
    for (int c0 = it.x + warp; c0 <= it.y; c0 += 4 * U) {
        float z[U], x[U][E];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + 4 * u;
            z[u] = -INFINITY;
            if (c <= it.y) {
                const int64_t row = (((int64_t)c * plan.RT + rt) * 2 + (c == it.x)) * rows + r;
                z[u] = plan.lse_part[row];
                if constexpr (E == 4) {
                    const float4 y = *reinterpret_cast<const float4 *>(plan.o_part + row * D + lane * E);
                    x[u][0] = y.x, x[u][1] = y.y, x[u][2] = y.z, x[u][3] = y.w;
                } else {
                    const float2 y = *reinterpret_cast<const float2 *>(plan.o_part + row * D + lane * E);
                    x[u][0] = y.x, x[u][1] = y.y;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (z[u] == -INFINITY) continue;
            const float m2 = fmaxf(mx, z[u]), f = mx == -INFINITY ? 0.f : ex2(mx - m2), e = ex2(z[u] - m2);
            mx = m2;
            l = l * f + e;
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] = o[i] * f + e * x[u][i];
        }
    }
    if (lane == 0) sm[warp] = mx, sl[warp] = l;
#pragma unroll
    for (int i = 0; i < E; ++i) so[warp][lane * E + i] = o[i];
    __syncthreads();
    const float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float f[4], sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i] = sl[i] > 0.f ? ex2(sm[i] - top) : 0.f;
        sum += f[i] * sl[i];
    }
    if (threadIdx.x < D) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) x += f[i] * so[i][threadIdx.x];
        static_cast<__nv_bfloat16 *>(a.out)[out_row * D + threadIdx.x] = __float2bfloat16(sum > 0.f ? x / sum : 0.f);
    }
    if (threadIdx.x == 0) a.lse[out_row] = sum > 0.f ? (top + log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

// ------------------------------------------------------------------------------------------ host
struct Shape {
    int Mt, tiles, RT;
    bool two;
    Shape(int G, int M) {
        Mt = kTile / G;
        tiles = (M + Mt - 1) / Mt;
        two = tiles > 1;
        RT = two ? (tiles + 1) / 2 : 1;
    }
    int rows() const { return two ? 256 : 128; }
    int ranges(int sms) const { return std::max(1, sms / RT); }
};

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
    }();
    return fn;
}

// the pool as [n_pages * Hkv * 64, D]; boxes of one page and KV head, 64 channels of bf16 (swizzled for the
// tensor cores) or all D codes
bool map_pool(CUtensorMap *map, const void *base, const PagedView &kv) {
    const bool i8 = kv.es == 1;
    cuuint64_t dims[2] = {(cuuint64_t)kv.D, (cuuint64_t)kv.n_pages * kv.Hkv * SGD_PAGE};
    cuuint64_t strides[1] = {(cuuint64_t)kv.D * kv.es};
    cuuint32_t box[2] = {(cuuint32_t)(i8 ? kv.D : 64), SGD_PAGE}, step[2] = {1, 1};
    return encode_fn()(map, i8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                       const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       i8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q as [B, M, Hq, D]; boxes of 64 channels, the G heads of a KV head and a row tile's query tokens
bool map_query(CUtensorMap *map, const PagedView &kv, const PagedAttnArgs &a, int Mt) {
    const cuuint64_t Hq = (cuuint64_t)kv.Hkv * a.G, row = (cuuint64_t)kv.D * 2;
    cuuint64_t dims[4] = {(cuuint64_t)kv.D, Hq, (cuuint64_t)a.M, (cuuint64_t)kv.B};
    cuuint64_t strides[3] = {row, Hq * row, Hq * row * a.M};
    cuuint32_t box[4] = {64, (cuuint32_t)a.G, (cuuint32_t)std::min(Mt, a.M), 1}, step[4] = {1, 1, 1, 1};
    return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(a.q), dims, strides, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

template <class C>
int launch(const PagedView &kv, const PagedAttnArgs &a, const AttnPlan &plan, cudaStream_t s) {
    CUtensorMap mq, mk, mv;
    if (!encode_fn() || !map_query(&mq, kv, a, plan.Mt) || !map_pool(&mk, kv.k, kv) || !map_pool(&mv, kv.v, kv))
        return SGD_ERR_CUDA;
    auto kern = paged_attn_kernel<C>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
        return SGD_ERR_CUDA;
    const cudaError_t e = launch_k(kern, dim3(plan.n_ranges * plan.RT), dim3(C::THREADS), C::SMEM, s, 1, kv, a, plan,
                                   mq, mk, mv);
    if (e != cudaSuccess) return SGD_ERR_CUDA;
    launch_k(paged_merge_kernel<C::D>, dim3(kv.B * a.M * kv.Hkv * a.G), dim3(128), 0, s, 1, kv, a, plan, (int)C::TWO);
    return cudaGetLastError() == cudaSuccess ? SGD_OK : SGD_ERR_CUDA;
}

}  // namespace

size_t paged_attn_scratch(int B, int Hkv, int D, int G, int M, int sms) {
    const Shape sh(G, M);
    const size_t slots = (size_t)sh.ranges(sms) * sh.RT * 2 * sh.rows();
    return up256(slots * D * 4) + up256(slots * 4) + up256((size_t)B * Hkv * 8);
}

int launch_paged_attn(const PagedView &kv, const PagedAttnArgs &a, cudaStream_t s) {
    const Shape sh(a.G, a.M);
    // an upper bound of the stream's length, which the kernel counts in 32 bits
    int64_t most = (int64_t)kv.max_pages * SGD_PAGE / kTile + 1;
    if (a.window) most = std::min(most, ((int64_t)a.window + a.M) / kTile + ((int64_t)a.sinks) / kTile + 4);
    most = (most + kItemCharge) * kv.Hkv * kv.B;
    if (most >= (int64_t(1) << 31)) return SGD_ERR_SHAPE;
    AttnPlan plan;
    plan.Mt = sh.Mt;
    plan.RT = sh.RT;
    plan.n_ranges = (int)std::min<int64_t>(sh.ranges(a.sms), most);
    const size_t slots = (size_t)plan.n_ranges * plan.RT * 2 * sh.rows();
    plan.o_part = reinterpret_cast<float *>(a.ws);
    plan.lse_part = reinterpret_cast<float *>(a.ws + up256(slots * kv.D * 4));
    plan.item = reinterpret_cast<int2 *>(a.ws + up256(slots * kv.D * 4) + up256(slots * 4));
    if (kv.es == 1) {
        if (kv.D == 128) return sh.two ? launch<Cfg<128, true, true>>(kv, a, plan, s) : launch<Cfg<128, true, false>>(kv, a, plan, s);
        return sh.two ? launch<Cfg<64, true, true>>(kv, a, plan, s) : launch<Cfg<64, true, false>>(kv, a, plan, s);
    }
    if (kv.D == 128) return sh.two ? launch<Cfg<128, false, true>>(kv, a, plan, s) : launch<Cfg<128, false, false>>(kv, a, plan, s);
    return sh.two ? launch<Cfg<64, false, true>>(kv, a, plan, s) : launch<Cfg<64, false, false>>(kv, a, plan, s);
}

}  // namespace sgd
