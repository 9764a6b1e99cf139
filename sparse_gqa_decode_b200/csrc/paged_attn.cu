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
// first).  Either way the groups g = 0, 1 take turns on the tensor cores:
//   QK_0 QK_1 | PV_0 QK_0 PV_1 QK_1 | PV_0 QK_0 ...   with the softmax of g between its QK and its PV.
//
// The work is cut without the host: every CTA sums the rows' tile counts itself (a window leaves the
// tiles of the first tokens and of the window only), takes an equal range of the stream of all (row,
// KV head) items' tiles, and walks it segment by segment.  A segment that is its whole item writes the
// result, others leave normalised partial rows, which paged_merge_kernel joins.
//
// The running maximum is a reference only: it follows the true one when it is passed by more than 8 in
// log2 (p then stays below 2^8, exact in range), which happens a few times in a long row, and
// O is rescaled in tensor memory only then.  S, m, l and O are float32; P is rounded to bf16 (2^-8
// relative), as is the output, since a product takes both operands in one type and V is bf16: the error against 64 bits
// is 1.4 times what the output's rounding alone gives (relative rms 0.0023 and 0.0017); l sums the unrounded p.
//
// INT8 codes are widened to f16 (exactly) in shared memory by warps of their own, a third fewer
// instructions than to bf16.  So Q and P are f16 there: a row of Q is scaled by a power of two to a
// maximum in [2^13, 2^14), which loses nothing but bits below 2^-38 of that maximum; P carries 2^7, so that
// f16's smallest step, 2^-24, is 2^-31 of the largest p and what 2^17 tokens could lose stays below 2^-14.
//
// Measured (D = 128, SM clock 1965 MHz; long runs meet the power cap and take 10 to 15% more):
//   bf16, 8 rows of up to 32K tokens, 16 nodes   137 us, 5.8 TB/s: HBM's rate inside a segment
//   bf16, 4 rows of up to 32K tokens, 64 nodes   249 to 257 us, 1.05 PFLOP/s: softmax, products and hand-overs in turn
//                                                (tensor pipe 43%, exponentials 43%, issue slots 36%: a latency chain)
//   INT8, 8 rows of up to 128K tokens, 4 nodes   463 us, 3.4 TB/s: no counter above 39% (DRAM 38%, tensor pipe 37%, issue
//                                                39%); 224 KB a tile pass through shared memory, codes twice, Q's 128 rows again
//   bf16, 64 windows of 4096 tokens, 1 node      129 us, 5.9 TB/s
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
// Tiles of work charged to an item beside its own (start, epilogue).  With 1, 2, 3, 4, 6, cold L2: 64 windows of 4096 tokens
// 160, 146, 144, 142, 147 us; 64 INT8 rows of 200 to 8000 tokens 92, 84, 73, 71, 77; 256 rows of 100 to 2000 74, 59, 57, 56, 59;
// 16 rows of 300 to 9000, 16 nodes, 52, 50, 46, 46, 46; 128 rows of 1000 114, whatever the charge
constexpr int kItemCharge = 3;
constexpr float kSlack = 8.f;    // log2 by which the true maximum may pass the reference
constexpr int kWarpProducer = 0, kWarpMma = 1, kWarpSoftmax = 4, kWarpConvert = 12;  // softmax: 4..11

// What a launch needs beside the cache and the arguments.
struct AttnPlan {
    int Mt;        // query tokens of a row tile: 128 / G
    int RT;        // CTAs per range: ceil(row tiles / 2) with two row tiles a CTA, else 1
    int n_ranges;  // grid / RT
    float *o_part;     // [grid * 2, rows of a CTA, D] partial outputs, normalised
    float *lse_part;   // [grid * 2, rows of a CTA], log2 units
    int2 *item;        // [B * Hkv] first and last range of each item
    int32_t *status;   // [grid] the CTAs' status bits
    int n_cta;         // grid
};

// A row of the page table in a launch.
struct Seq {
    int L, n, base;  // tokens, nodes, entries before the nodes
    int sink_tiles;  // tiles of the first tokens that do not belong to the window
    int first;       // the window's first tile
    int win;         // the first entry of any window, 0 without one
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
    s.sink_tiles = s.first = s.win = 0;
    if (a.window) {
        s.win = max(s.base + 1 - a.window, 0);
        s.first = s.win / kTile;
        s.sink_tiles = min((int)(((int64_t)a.sinks + kTile - 1) / kTile), s.first);
    }
    s.tiles = s.n == 0 ? 1 : max(1, s.sink_tiles + all - s.first);
    return s;
}

// The tile at t0 may have entries that no query of the sequence sees: behind its end, or between the first tokens and the
// windows.  They may hold anything.  The second product runs over the 16-token steps [from, to) that hold
// every seen entry; where those hold unseen ones too, their V rows have to become 0 before it.
struct Steps {
    int from, to;
    bool unseen;
};
__device__ __forceinline__ bool all_seen(const Seq &s, int t0) { return t0 + kTile <= s.L && t0 >= s.win; }
__device__ __forceinline__ Steps steps_of(const Seq &s, const PagedAttnArgs &a, int t0) {
    if (all_seen(s, t0)) return {0, kTile / 16, false};
    int lo = 0, hi = min(max(s.L - t0, 0), kTile);
    bool gap = false;
    if (a.window) {
        const int w = s.base + 1 - a.window - t0, f = a.sinks - t0;  // the windows' first entry, the end of the first tokens
        if (w > 0 && w > f) {
            if (f <= 0) lo = min(w, hi);
            else if (w >= hi) hi = min(hi, f);
            else gap = true;
        }
    }
    Steps r;
    r.to = max((hi + 15) / 16, 1);
    r.from = min(lo / 16, r.to - 1);
    r.unseen = gap || hi < r.to * 16 || lo > r.from * 16;
    return r;
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
    // Q: the two row tiles, or two segments'; one segment's with codes, whose tiles in flight need the space
    static constexpr int Q_STAGES = TWO || I8 ? 1 : 2, Q_BUFS = TWO ? 2 : Q_STAGES;
    static constexpr int SLOTS = I8 ? (D == 128 ? 3 : 4) : (D == 128 ? 5 : 8);  // 16-bit tiles of K or V
    static constexpr int RAW = !I8 ? 0 : D == 128 ? (TWO ? 4 : 6) : (TWO ? 8 : 12);  // code tiles in flight
    static constexpr int RAW_BYTES = kTile * D;
    static constexpr int CONVERT = I8 ? 128 : 0;         // threads that widen codes
    static constexpr int THREADS = 384 + CONVERT;
    static constexpr int ROWS = TWO ? 256 : 128;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_SLOT = Q_BUFS * TILE_BYTES;
    static constexpr int OFF_RAW = OFF_SLOT + SLOTS * TILE_BYTES;
    static constexpr int OFF_ML = OFF_RAW + RAW * RAW_BYTES;  // [2][128] (m, l) of the warpgroups
    static constexpr int OFF_QE = OFF_ML + 2 * 128 * 8;       // I8, one row tile: [128] the rows' powers of two
    static constexpr int OFF_BAR = OFF_QE + 128 * 4;
    static constexpr int SMEM = OFF_BAR + 512;
    static constexpr float SHIFT = I8 ? 7.f : 0.f;            // log2 that P carries
    static_assert(SMEM <= 232448, "fits a CTA's shared memory");
};

struct Bars {
    uint64_t full[8], empty[8];          // ring of bf16 K / V tiles, in the order the products take them
    uint64_t raw_full[12], raw_empty[12];  // I8: ring of code tiles
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], v_here[2], p_full[2], o_full[2];
    uint64_t q_ready, o_free, ml_full, drained;
    uint32_t tmem;
    int32_t abort;
    int32_t start_b, start_pos;          // the range's first row and its stream position
    int32_t status;                      // the CTA's SGD_STATUS_* bits
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

// Row r of a row tile of Q from bf16 to f16 in place, scaled by a power of two to a maximum in [2^13, 2^14); returns
// its inverse.  A thread has its row to itself; eight threads' 16-byte pieces lie in different banks.
template <class C>
__device__ __forceinline__ float q_to_f16(uint8_t *q, int r) {
    constexpr int N = C::D / 8;
    auto piece = [&](int c) { return reinterpret_cast<uint4 *>(q + c / 8 * kTile * 128 + r * 128 + ((c % 8) ^ (r & 7)) * 16); };
    uint32_t m = 0;
#pragma unroll 4
    for (int c = 0; c < N; ++c) {
        const uint4 x = *piece(c);
        m = bf16x2_absmax(bf16x2_absmax(bf16x2_absmax(bf16x2_absmax(m, x.x), x.y), x.z), x.w);
    }
    const float top = bf16x2_fold_max(m);
    // exponent of the maximum, 2^e <= top < 2^(e + 1); a zero, subnormal or infinite maximum takes the nearest normal
    const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 126);
    const float f = __uint_as_float((uint32_t)(127 + 13 - e) << 23);  // 2^(13 - e): 13 - e in [-113, 113]
#pragma unroll 4
    for (int c = 0; c < N; ++c) {
        uint4 x = *piece(c);
        auto half2 = [&](uint32_t w) { return pack_f16(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f); };
        x.x = half2(x.x), x.y = half2(x.y), x.z = half2(x.z), x.w = half2(x.w);
        *piece(c) = x;
    }
    return __uint_as_float((uint32_t)(127 - 13 + e) << 23);
}

// The polls after a wait's first one, out of line: two dozen copies of the loop would crowd the instruction cache.
__device__ __noinline__ bool wait_on(uint64_t *m, uint32_t parity, int32_t *status, volatile int32_t *abort,
                                     long long limit) {
    return mbar_wait(m, parity, status, abort, limit);
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
            mbar_init(&bar.full[i], C::I8 ? C::CONVERT / 32 : 1);
            mbar_init(&bar.empty[i], 1);
        }
        for (int i = 0; i < C::RAW; ++i) {
            mbar_init(&bar.raw_full[i], 1);
            mbar_init(&bar.raw_empty[i], C::CONVERT / 32);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(&bar.q_full[g], 1);
            mbar_init(&bar.q_empty[g], 1);
            mbar_init(&bar.s_full[g], 1);
            mbar_init(&bar.v_here[g], 1);
            mbar_init(&bar.p_full[g], warps[g]);
            mbar_init(&bar.o_full[g], 1);
        }
        mbar_init(&bar.q_ready, warps[0] + (C::TWO ? warps[1] : 0));
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
    if (tid == 64) bar.status = 0;
    // Rows of Q's tiles that no load fills stay 0, and so do theirs of S and P.  Multiplying zeros takes less power, which
    // caps the clock of a long run: with 32 rows of 128 (8 x 128K tokens of INT8, repeated for a second) 522 -> 511 us
    if (rows[0] < 128 || (C::TWO && rows[1] < 128)) {
        for (int i = tid; i < C::Q_BUFS * C::TILE_BYTES / 16; i += C::THREADS)
            *reinterpret_cast<uint4 *>(smem + C::OFF_Q + i * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_shared();
    }
    if (warp == kWarpMma) tmem_alloc(&bar.tmem, 512);
    grid_dependency_wait();  // nothing of the call's data was touched so far
    __syncthreads();

    // the stream's length, this range of it, and the row it starts in: thread t sums consecutive rows
    int x0, x1;
    {
        const int per = (kv.B + C::THREADS - 1) / C::THREADS;
        const int b0 = min(tid * per, kv.B), b1 = min(b0 + per, kv.B);
        int sum = 0, bad = 0;
        for (int b = b0; b < b1; ++b) sum += (seq_of(kv, a, b, bad).tiles + kItemCharge) * kv.Hkv;
        if (bad && blockIdx.x == 0) atomicOr(&bar.status, bad);
        int total;
        int pos = block_exclusive_scan(sum, total, reinterpret_cast<int32_t *>(smem + C::OFF_ML));
        const int S = total / plan.n_ranges + (total % plan.n_ranges != 0);  // total may be close to 2^31
        x0 = (int)min((int64_t)range * S, (int64_t)total);
        x1 = (int)min((int64_t)x0 + S, (int64_t)total);
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
    // the first poll looks at nothing but the barrier: while the tensor cores read their operands a shared-memory
    // access takes a few hundred cycles, and the abort flag would double that
    auto wait = [&](uint64_t *m, uint32_t parity) {
        return mbar_try_wait(m, parity) || wait_on(m, parity, &bar.status, abort, a.wait_limit);
    };
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
                        // an error where a query sees an entry of the page; one between the first tokens and the windows may
                        // have been given back
                        const int t = (p0 + i) * SGD_PAGE;
                        if (w.s.n > 0 && !(a.window && t >= a.sinks && t + SGD_PAGE <= w.s.win)) bad = SGD_STATUS_BAD_INDEX;
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
            if (bad) atomicOr(&bar.status, bad);
            if (*abort) {  // no copy may still be writing when the CTA ends
                for (uint32_t i = at > N ? at - N : 0; i < at; ++i) mbar_drain(&full[i % N], (i / N) & 1, a.wait_limit);
                for (uint32_t i = seg > C::Q_STAGES ? seg - C::Q_STAGES : 0; i < seg; ++i)
                    mbar_drain(&bar.q_full[i % C::Q_STAGES], (i / C::Q_STAGES) & 1, a.wait_limit);
            }
        }
    } else if (warp == kWarpMma) {
        // ------------------------------------------------------------------ products
        // One thread issues all products, from code that the whole warp runs (the operands then stay in uniform
        // registers; from a branch of one lane a product took 60 cycles to issue).  The warp waits for every KV tile, in
        // ring order: a parity tells a barrier's phases apart only for who misses none.  A tile's V, and with two row
        // tiles the next K, is waited for before its P, while the softmax is at work: 318 -> 264 us for 512 rows and
        // 4 x 31K tokens.  An issuing warp for each group instead took 320 us.
        constexpr uint32_t ID_QK = tc_idesc(C::I8, 128, kTile, false), ID_PV = tc_idesc(C::I8, 128, D, true);
        const uint32_t sq = smem_u32(smem + C::OFF_Q), ss = smem_u32(smem + C::OFF_SLOT);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        uint32_t at = 0, seg = 0, np[2] = {0, 0};
        bool go = true;
        auto slot = [&](uint32_t pos) { return ss + (pos % C::SLOTS) * C::TILE_BYTES; };
        auto full = [&](uint32_t pos) { return go && (go = wait_warp(&bar.full[pos % C::SLOTS], (pos / C::SLOTS) & 1)); };
        auto commit = [&](uint64_t *m) {
            if (elect_one()) tc_commit(m);
        };
        auto release = [&](uint32_t pos) { commit(&bar.empty[pos % C::SLOTS]); };
        auto qk = [&](int g, uint32_t q, uint32_t pos) {  // S_g = Q K^T
            tc_fence_after();
            const uint64_t dq = desc_k_major(q), dk = desc_k_major(slot(pos));
            if (elect_one()) {
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    const uint32_t off = ((j / 4) * (kTile * 128) + (j % 4) * 32) >> 4;  // in the descriptors' 16 bytes
                    mma_ss(tm + g * 128, dq + off, dk + off, ID_QK, j > 0);
                }
                tc_commit(&bar.s_full[g]);
            }
        };
        auto pv = [&](int g, uint32_t pos, const Steps &st, bool acc) {  // O_g (+)= P_g V
            if (!go || !(go = wait_warp(&bar.p_full[g], np[g]++ & 1))) return false;
            tc_fence_after();
            const uint64_t dv = desc_mn_major(slot(pos), kTile * 128);
            if (elect_one()) {  // rolled: the unrolled loop, or two of them, cost the INT8 case 2 to 10% in instruction fetches
#pragma unroll 1
                for (int j = st.from; j < st.to; ++j)
                    mma_ts(tm + 256 + g * 128, tm + g * 128 + j * 8, dv + j * (2048 >> 4), ID_PV, acc || j > st.from);
            }
            return true;
        };
        while (go && w.next(kv, a)) {
            const int T = __shfl_sync(0xffffffffu, w.hi - w.lo, 0), qs = seg % C::Q_STAGES;
            go = C::I8 ? wait_warp(&bar.q_ready, seg & 1) : wait_warp(&bar.q_full[qs], (seg / C::Q_STAGES) & 1);
            if (!go) break;
            const uint32_t q0 = sq + (C::TWO ? 0 : qs) * C::TILE_BYTES;
            if constexpr (C::TWO) {
                if (!full(at)) break;
                for (int g = 0; g < 2; ++g) qk(g, q0 + g * C::TILE_BYTES, at);
                release(at);
                if (T == 1) commit(&bar.q_empty[qs]);  // the last product that reads Q was issued
            } else {
                for (int g = 0; g < min(T, 2); ++g) {
                    if (!full(at + g)) break;
                    qk(g, q0, at + g);
                    release(at + g);
                }
                if (!go) break;
                if (T <= 2) commit(&bar.q_empty[qs]);
            }
            if (seg > 0 && !(go = wait_warp(&bar.o_free, (seg - 1) & 1))) break;  // the last segment's O was read
            for (int j = 0; j < T; ++j) {
                const uint32_t v_at = at + pos_v<C::TWO>(j, T), k_at = at + pos_k<C::TWO>(C::TWO ? j + 1 : j + 2);
                const int t0 = tile_of(w.s, w.lo + j) * kTile;
                Steps st = {0, kTile / 16, false};
                if (__any_sync(0xffffffffu, !all_seen(w.s, t0))) {
                    st = steps_of(w.s, a, t0);
                    st.from = __shfl_sync(0xffffffffu, st.from, 0), st.to = __shfl_sync(0xffffffffu, st.to, 0);
                }
                if (!full(v_at)) break;
                if (lane == 0 && st.unseen) {  // its rows may be cleared
                    mbar_arrive(&bar.v_here[C::TWO ? 0 : j & 1]);
                    if (C::TWO) mbar_arrive(&bar.v_here[1]);
                }
                __syncwarp();
                if constexpr (C::TWO) {
                    const bool more = j + 1 < T;
                    if (more && !full(k_at)) break;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        if (!pv(g, v_at, st, j > 0)) break;
                        if (more) qk(g, q0 + g * C::TILE_BYTES, k_at);
                        else commit(&bar.o_full[g]);
                    }
                    if (!go) break;
                    release(v_at);
                    if (more) release(k_at);
                    if (j + 2 == T) commit(&bar.q_empty[qs]);
                } else {
                    const int g = j & 1;
                    if (!pv(g, v_at, st, j > 1)) break;
                    if (j + 2 >= T) commit(&bar.o_full[g]);
                    release(v_at);
                    if (j + 2 < T) {
                        if (!full(k_at)) break;
                        qk(g, q0, k_at);
                        release(k_at);
                        if (j + 3 == T) commit(&bar.q_empty[qs]);
                    }
                }
            }
            at += 2 * T;
            ++seg;
        }
        // no product may still be reading, and no arrival be due, when the CTA ends
        commit(&bar.drained);
        if (lane == 0) mbar_drain(&bar.drained, 0, a.wait_limit);
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
            float scale = a.scale_log2, vs = 1.f, scale_k = scale;
            if constexpr (C::I8) {
                const bool report = blockIdx.x == 0 && g == 0 && r == 0;
                scale_k *= checked_scale(*kv.k_scale, &bar.status, report);
                vs = checked_scale(*kv.v_scale, &bar.status, report);
            }
            uint32_t at = 0, seg = 0, ns = 0, nv = 0, no[2] = {0, 0};
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
                        if (bad) atomicOr(&bar.status, bad);
                    }
                }
                if constexpr (C::I8) {  // the row of Q as f16, scaled by 2^-e
                    const int qs = seg % C::Q_STAGES;
                    float *qe = reinterpret_cast<float *>(smem + C::OFF_QE);
                    if (C::TWO || g == 0) {
                        if (!(go = wait_warp(&bar.q_full[qs], (seg / C::Q_STAGES) & 1))) break;
                        if (valid) {
                            const float f = q_to_f16<C>(smem + C::OFF_Q + (C::TWO ? g : qs) * C::TILE_BYTES, r);
                            scale = scale_k * f;
                            if constexpr (!C::TWO) qe[r] = f;
                        }
                        fence_proxy_async_shared();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar.q_ready);
                    } else {
                        if (!(go = wait_warp(&bar.q_ready, seg & 1))) break;
                        if (valid) scale = scale_k * qe[r];
                    }
                }
                const bool query = valid && m < s.n;
                const int prefix = query && s.base > 0 ? s.base : 0;  // entries before the nodes that the row may see
                const int sink = min(a.sinks, prefix);
                const int v_lo = s.base + 1 - a.window;               // no row sees an entry of [sinks, v_lo)
                float mx = query ? -INFINITY : INFINITY, l = 0.f;     // p of a row that asks nothing is 0
                for (int j = C::TWO ? 0 : g; j < T; j += C::TWO ? 1 : 2) {
                    const int t0 = tile_of(s, w.lo + j) * kTile;
                    if (!(go = wait_warp(&bar.s_full[g], ns & 1))) break;
                    ++ns;
                    tc_fence_after();
                    // rows that ask nothing do not count: whatever they gather is dropped at the end
                    const bool masked = __any_sync(
                        0xffffffffu, query && (t0 + kTile > prefix || (lo > t0 && t0 + kTile > sink)));
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
                    if (!masked) {
#pragma unroll 1
                        for (int c = 0; c < 4; c += 2) {
                            uint32_t x[32], y[32];
                            tmem_ld32(x, ts + c * 32);
                            tmem_ld32(y, ts + c * 32 + 32);
                            tmem_wait_ld(x);
                            tmem_wait_ld(y);
                            float t4[4] = {top, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                t4[i & 3] = max3(t4[i & 3], __uint_as_float(x[i]), __uint_as_float(y[i]));
                            top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
                        }
                    } else {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t x[32];
                            tmem_ld32(x, ts + c * 32);
                            tmem_wait_ld(x);
                            const uint32_t k = mask_of(c);
#pragma unroll
                            for (int i = 0; i < 32; ++i) top = fmaxf(top, k >> i & 1 ? __uint_as_float(x[i]) : -INFINITY);
                        }
                    }
                    const float mt = top == -INFINITY ? -INFINITY : top * scale;
                    const bool first = j < 2 && (C::TWO ? j == 0 : true);
                    if (__any_sync(0xffffffffu, query && mt > mx + kSlack)) {
                        const float m2 = fmaxf(mx, mt), f = mx == -INFINITY ? 0.f : ex2(mx - m2);
                        mx = m2;
                        l *= f;
                        if (!first) {
#pragma unroll 1
                            for (int c = 0; c < D / 8; ++c) {  // 8 at a time: a row of S is held meanwhile
                                uint32_t y[8];
                                tmem_ld8(y, to + c * 8);
                                tmem_wait_ld(y);
#pragma unroll
                                for (int i = 0; i < 8; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
                                tmem_st8(to + c * 8, y);
                            }
                        }
                    }
                    const float ref = (mx == -INFINITY ? 0.f : mx) - C::SHIFT;
                    // p, its sum, and P in the place of S (a chunk's columns of P lie among those of S read before)
                    auto pack = [](float p0, float p1) { return C::I8 ? pack_f16(p0, p1) : pack_bf16(p0, p1); };
                    if (masked) {
                        float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t x[32], y[16];
                            tmem_ld32(x, ts + c * 32);
                            tmem_wait_ld(x);
                            const uint32_t k = mask_of(c);
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                const float p0 = k >> i & 1 ? ex2(fmaf(__uint_as_float(x[i]), scale, -ref)) : 0.f;
                                const float p1 = k >> (i + 1) & 1 ? ex2(fmaf(__uint_as_float(x[i + 1]), scale, -ref)) : 0.f;
                                l4[i & 2] += p0;
                                l4[(i & 2) + 1] += p1;
                                y[i / 2] = pack(p0, p1);
                            }
                            tmem_st16(ts + c * 16, y);
                        }
                        l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
                    } else {
                        float l4[4] = {0.f, 0.f, 0.f, 0.f};
                        auto chunk = [&](const uint32_t (&x)[32], int c) {
                            uint32_t y[16];
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                const float p0 = ex2(fmaf(__uint_as_float(x[i]), scale, -ref));
                                const float p1 = ex2(fmaf(__uint_as_float(x[i + 1]), scale, -ref));
                                l4[i & 2] += p0;
                                l4[(i & 2) + 1] += p1;
                                y[i / 2] = pack(p0, p1);
                            }
                            tmem_st16(ts + c * 16, y);
                        };
                        // the next chunk's load runs beside this one's exponentials
                        uint32_t x0[32], x1[32];
                        tmem_ld32(x0, ts);
                        tmem_wait_ld(x0);
#pragma unroll 1
                        for (int c = 0; c < 4; c += 2) {
                            tmem_ld32(x1, ts + c * 32 + 32);
                            chunk(x0, c);
                            tmem_wait_ld(x1);
                            if (c == 0) tmem_ld32(x0, ts + 64);
                            chunk(x1, c + 1);
                            if (c == 0) tmem_wait_ld(x0);
                        }
                        l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
                    }
                    if (!all_seen(s, t0)) {
                        const Steps st = steps_of(s, a, t0);
                        if (st.unseen) {  // clear V's rows once they are here
                            if (!(go = wait_warp(&bar.v_here[g], nv++ & 1))) break;
                            const uint32_t pos = at + pos_v<C::TWO>(j, T);
                            uint8_t *v = smem + C::OFF_SLOT + (pos % C::SLOTS) * C::TILE_BYTES;
                            auto zero = [&](int from, int to) {  // rows of the tile, 16 bytes a lane
                                constexpr int PER = D / 8;
                                // both ends first: a window or a row may lie 2^30 entries away
                                from = min(max(from, st.from * 16), st.to * 16), to = min(max(to, 0), st.to * 16);
#pragma unroll 1
                                for (int u = from * PER + wq * 32 + lane; u < to * PER; u += na * 32)
                                    *reinterpret_cast<uint4 *>(v + (u % PER) / 8 * kTile * 128 + u / PER * 128 + u % 8 * 16) =
                                        make_uint4(0, 0, 0, 0);
                            };
                            zero(s.L - t0, kTile);
                            if (a.window) zero(a.sinks - t0, v_lo - t0);
                            fence_proxy_async_shared();
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.p_full[g]);
                }
                if (!go) break;

                if (!query) l = 0.f;

                // The segment's result.  A row that sees nothing has sum 0 exactly; a NaN (from its query) stays one.
                const bool whole = w.lo == 0 && w.hi == s.tiles;
                const int64_t out_row = (((int64_t)w.b * a.M + m) * kv.Hkv + w.h) * a.G + gh;
                const int64_t part_row =
                    ((int64_t)blockIdx.x * 2 + (w.lo == 0)) * C::ROWS + (C::TWO ? g * 128 : 0) + r;
                float f0, f1 = 0.f, sum, ref;  // O_0 f0 + O_1 f1 is the normalised row
                if constexpr (C::TWO) {
                    sum = l, ref = mx;
                    f0 = sum != 0.f ? vs / sum : 0.f;
                } else {
                    // every warp has read the last segment's pair
                    if (seg > 0 && !(go = wait_warp(&bar.o_free, (seg - 1) & 1))) break;
                    ml[g * 128 + r] = make_float2(mx, l);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.ml_full);
                    if (!(go = wait_warp(&bar.ml_full, seg & 1))) break;
                    const float2 u = ml[r], v = ml[128 + r];
                    ref = fmaxf(u.x, v.x);
                    const float e0 = u.y != 0.f ? ex2(u.x - ref) : 0.f, e1 = v.y != 0.f ? ex2(v.x - ref) : 0.f;
                    sum = e0 * u.y + e1 * v.y;
                    f0 = sum != 0.f ? vs * e0 / sum : 0.f;
                    f1 = sum != 0.f ? vs * e1 / sum : 0.f;
                }
                for (int i = 0; i < 2; ++i) {
                    if (C::TWO ? i != g : i >= T) continue;
                    if (!(go = wait_warp(&bar.o_full[i], no[i]++ & 1))) break;
                }
                if (!go) break;
                tc_fence_after();
                // TWO: the row's D channels; else this group's half of them, from both accumulators
                constexpr int NC = (C::TWO ? D : D / 2) / 16;
#pragma unroll 1
                for (int c = 0; c < NC; ++c) {
                    const int col = (C::TWO ? 0 : g * (D / 2)) + c * 16;
                    uint32_t x[16];
                    float o[16];
                    tmem_ld16(x, lane_at + 256 + (C::TWO ? g * 128 : 0) + col);
                    tmem_wait_ld(x);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = f0 != 0.f ? f0 * __uint_as_float(x[i]) : 0.f;
                    if (!C::TWO && T > 1) {
                        tmem_ld16(x, lane_at + 256 + 128 + col);
                        tmem_wait_ld(x);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] += f1 != 0.f ? f1 * __uint_as_float(x[i]) : 0.f;
                    }
                    if (valid && whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + out_row * D + col);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            dst[i] = make_uint4(pack_bf16(o[8 * i], o[8 * i + 1]), pack_bf16(o[8 * i + 2], o[8 * i + 3]),
                                                pack_bf16(o[8 * i + 4], o[8 * i + 5]), pack_bf16(o[8 * i + 6], o[8 * i + 7]));
                    } else if (valid) {
                        float4 *dst = reinterpret_cast<float4 *>(plan.o_part + part_row * D + col);
#pragma unroll
                        for (int i = 0; i < 4; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                    __syncwarp();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.o_free);
                if (valid && (C::TWO || g == 0)) {
                    const float lse2 = sum != 0.f ? ref - C::SHIFT + log2f(sum) : -INFINITY;
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
    } else if (C::I8 && warp >= kWarpConvert) {
        // ------------------------------------------------------------------ codes to f16
        constexpr int UNITS = kTile * D / 16, U = UNITS / 128, RAW = C::RAW > 0 ? C::RAW : 1;  // 16 codes each
        const int ct = tid - kWarpConvert * 32;
        uint32_t at = 0, rd = 0, end = 0;  // ring positions written, read, known so far
        bool go = true;
        auto known = [&](uint32_t pos) {  // whether the CTA's range has this position
            while (pos >= end && w.next(kv, a)) end += 2 * (w.hi - w.lo);
            return pos < end;
        };
        auto read = [&](uint4 (&x)[U]) {
            if (!go || !known(rd)) return;
            const int rs = rd % RAW;
            if (!(go = wait_warp(&bar.raw_full[rs], (rd / RAW) & 1))) return;
            const uint8_t *src = smem + C::OFF_RAW + rs * C::RAW_BYTES;
#pragma unroll
            for (int i = 0; i < U; ++i) x[i] = lds128(smem_u32(src + (ct + 128 * i) * 16));
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.raw_empty[rs]);
            ++rd;
        };
        auto write = [&](const uint4 (&x)[U]) {
            const int bs = at % C::SLOTS;
            if (at >= C::SLOTS && !(go = wait_warp(&bar.empty[bs], (at / C::SLOTS - 1) & 1))) return;
            uint8_t *dst = smem + C::OFF_SLOT + bs * C::TILE_BYTES;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int u = ct + 128 * i, row = u / (D / 16), cb = u % (D / 16);
                uint32_t y[8];
                s8x4_to_f16x2x2(x[i].x, y[0], y[1]);
                s8x4_to_f16x2x2(x[i].y, y[2], y[3]);
                s8x4_to_f16x2x2(x[i].z, y[4], y[5]);
                s8x4_to_f16x2x2(x[i].w, y[6], y[7]);
                // two 16-byte pieces of the swizzled row; the second half's threads start with the odd one, so that a
                // quarter warp's stores cover all banks
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
            if (lane == 0) mbar_arrive(&bar.full[bs]);
            ++at;
        };
        uint4 x[U];
        for (read(x); go && at < end; read(x)) write(x);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) plan.status[blockIdx.x] = bar.status;
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the partial rows of an item that several ranges share: WARPS warps per output row take its
// ranges in turn, four at a time.  lse = log2 sum_c 2^lse_c, out = sum_c 2^(lse_c - lse) o_c.
constexpr int kMergeThreads = 256;

template <int D, int WARPS>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(PagedView kv, PagedAttnArgs a, AttnPlan plan,
                                                                    int two, int64_t n_rows) {
    constexpr int ROWS = kMergeThreads / 32 / WARPS;  // output rows of a CTA
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wr = warp % WARPS;
    const int Hq = kv.Hkv * a.G;
    grid_dependency_wait();
    if (blockIdx.x == 0 && warp == 0) {  // the call's status
        int bits = 0;
        for (int c = lane; c < plan.n_cta; c += 32) bits |= plan.status[c];
        bits = __reduce_or_sync(0xffffffffu, (unsigned)bits);
        if (lane == 0) *a.status = bits;
    }
    const int64_t out_row = (int64_t)blockIdx.x * ROWS + warp / WARPS;
    if (out_row >= n_rows) return;  // WARPS > 1: ROWS is 1, the CTA leaves as a whole
    const int hq = (int)(out_row % Hq), m = (int)(out_row / Hq % a.M), b = (int)(out_row / Hq / a.M);
    const int2 it = plan.item[b * kv.Hkv + hq / a.G];
    if (it.x >= it.y || it.x < 0 || it.y >= plan.n_ranges) return;  // written by its only range
    const int mt = m / plan.Mt, rt = two ? mt / 2 : 0, rows = two ? 256 : 128;
    const int r = (two ? mt % 2 * 128 : 0) + (m % plan.Mt) * a.G + hq % a.G;
    constexpr int E = D / 32;
    float mx = -INFINITY, l = 0.f, o[E] = {};
    constexpr int U = 4;
    for (int c0 = it.x + wr; c0 <= it.y; c0 += WARPS * U) {
        float z[U], x[U][E];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + WARPS * u;
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
    if constexpr (WARPS > 1) {
        __shared__ float so[WARPS][D], sl[WARPS], sm[WARPS];
        if (lane == 0) sm[warp] = mx, sl[warp] = l;
#pragma unroll
        for (int i = 0; i < E; ++i) so[warp][lane * E + i] = o[i];
        __syncthreads();
        if (warp != 0) return;
        mx = -INFINITY;
        for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, sm[w]);
        l = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = 0.f;
        for (int w = 0; w < WARPS; ++w) {
            const float f = sl[w] != 0.f ? ex2(sm[w] - mx) : 0.f;
            l += f * sl[w];
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] += f * so[w][lane * E + i];
        }
    }
    const float f = l != 0.f ? 1.f / l : 0.f;
    uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.out) + out_row * D) + lane * (E / 2);
    if constexpr (E == 4)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(o[0] * f, o[1] * f), pack_bf16(o[2] * f, o[3] * f));
    else
        *dst = pack_bf16(o[0] * f, o[1] * f);
    if (lane == 0) a.lse[out_row] = l != 0.f ? (mx + log2f(l)) * 0.69314718055994531f : -INFINITY;
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
    static SmemOptIn opt_in;
    if (!opt_in.set(reinterpret_cast<const void *>(kern), C::SMEM)) return SGD_ERR_CUDA;
    const cudaError_t e =
        launch_k_early(kern, dim3(plan.n_ranges * plan.RT), dim3(C::THREADS), C::SMEM, s, kv, a, plan, mq, mk, mv);
    if (e != cudaSuccess) return SGD_ERR_CUDA;
    // Few rows may have many ranges each (up to all of them): then a CTA per row, else a warp.  Whole call, CTA against warp
    // per row, cold L2: 64 rows of 128K tokens 103 and 106 us, 512 rows of 16K 29.7 and 31.7; 1024 rows of 512 to 32K 105 and
    // 103, 2048 INT8 rows of 16K to 32K 140 and 136, 4096 rows of 1K to 16K 58 and 50
    const int64_t n_rows = (int64_t)kv.B * a.M * kv.Hkv * a.G;
    constexpr int W = kMergeThreads / 32;
    if (n_rows <= 512)
        launch_k_early(paged_merge_kernel<C::D, W>, dim3((unsigned)n_rows), dim3(kMergeThreads), 0, s, kv, a, plan, (int)C::TWO, n_rows);
    else
        launch_k_early(paged_merge_kernel<C::D, 1>, dim3((unsigned)((n_rows + W - 1) / W)), dim3(kMergeThreads), 0, s, kv, a, plan,
                 (int)C::TWO, n_rows);
    return cudaGetLastError() == cudaSuccess ? SGD_OK : SGD_ERR_CUDA;
}

}  // namespace

size_t paged_attn_scratch(int B, int Hkv, int D, int G, int M, int sms) {
    const Shape sh(G, M);
    // as many CTAs as SMs, though RT may not divide them: a smaller step's RT may, and takes the same workspace
    const size_t slots = (size_t)std::max(sms, sh.RT) * 2 * sh.rows();
    return up256(slots * D * 4) + up256(slots * 4) + up256((size_t)B * Hkv * 8) + up256((size_t)sms * 4);
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
    plan.status = reinterpret_cast<int32_t *>(reinterpret_cast<uint8_t *>(plan.item) + up256((size_t)kv.B * kv.Hkv * 8));
    plan.n_cta = plan.n_ranges * plan.RT;
    if (kv.es == 1) {
        if (kv.D == 128) return sh.two ? launch<Cfg<128, true, true>>(kv, a, plan, s) : launch<Cfg<128, true, false>>(kv, a, plan, s);
        return sh.two ? launch<Cfg<64, true, true>>(kv, a, plan, s) : launch<Cfg<64, true, false>>(kv, a, plan, s);
    }
    if (kv.D == 128) return sh.two ? launch<Cfg<128, false, true>>(kv, a, plan, s) : launch<Cfg<128, false, false>>(kv, a, plan, s);
    return sh.two ? launch<Cfg<64, false, true>>(kv, a, plan, s) : launch<Cfg<64, false, false>>(kv, a, plan, s);
}

}  // namespace sgd
