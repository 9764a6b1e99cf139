// pages.cu -- upkeep of the paged cache: reserving, appending, forking, releasing and compacting
// pages (sgd_pages_* in include/sgd.h).
//
// The pool's whole allocation state is ref_count: a page is free when its count is 0, and the
// lowest free page is taken first.  So the calls keep no list whose order could depend on how threads
// ran: equal states give equal pages, and releasing what was just taken restores the state exactly.
#include <algorithm>

#include "paged.h"
#include "quant.cuh"
#include "scan.cuh"

namespace sgd {

namespace {

constexpr int kAllocThreads = 1024;

__device__ __forceinline__ int ceil_pages(int tokens) { return (tokens + SGD_PAGE - 1) / SGD_PAGE; }

// The `want` lowest free pages, ascending, into list[]; returns how many there are (<= want).
// Called by every thread of the block.  One pass over ref_count, 4 entries per thread and round,
// that ends as soon as enough are found: 16 KB a round, about a microsecond each (the CTA waits for
// one round of loads and one block scan).
__device__ int find_free(const int32_t *ref, int n_pages, int want, int32_t *list, int32_t *sm) {
    int found = 0;
    for (int at = 0; at < n_pages && found < want; at += kAllocThreads * 4) {
        const int p0 = at + threadIdx.x * 4;
        int free4 = 0;  // bit j: page p0 + j is free
        if (p0 + 3 < n_pages) {
            const int4 r = *reinterpret_cast<const int4 *>(ref + p0);
            free4 = (r.x == 0) | (r.y == 0) << 1 | (r.z == 0) << 2 | (r.w == 0) << 3;
        } else {
            for (int j = 0; j < 4; ++j)
                if (p0 + j < n_pages && ref[p0 + j] == 0) free4 |= 1 << j;
        }
        int total;
        int rank = found + block_exclusive_scan(__popc(free4), total, sm);
        for (int j = 0; j < 4; ++j)
            if (free4 >> j & 1) {
                if (rank < want) list[rank] = p0 + j;
                ++rank;
            }
        found += total;
    }
    __syncthreads();  // list[] is read by other threads
    return min(found, want);
}

// The OR of every thread's bits (sm: 33 words as in the scans).
__device__ __forceinline__ int block_or(int v, int32_t *sm) {
    v = __reduce_or_sync(0xffffffffu, (unsigned)v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) v |= sm[w];
    __syncthreads();
    return v;
}

// largest b < n with off[b] <= r (off ascending, off[0] = 0)
__device__ __forceinline__ int owner(const int32_t *off, int n, int r) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (off[mid] <= r) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// One CTA: needs, checks, the free pages, then the new state.  Everything is decided before
// anything is written.
__global__ void __launch_bounds__(kAllocThreads) reserve_kernel(PagedView kv, const int32_t *add,
                                                                int32_t *new_lens, int32_t *off, int32_t *list,
                                                                int32_t *status) {
    __shared__ int32_t sm[33];
    __shared__ unsigned long long wanted;
    grid_dependency_wait();
    const int per = (kv.B + kAllocThreads - 1) / kAllocThreads;
    const int b0 = min((int)threadIdx.x * per, kv.B), b1 = min(b0 + per, kv.B);
    int bad = 0;
    long long sum = 0;
    auto need = [&](int b) { return max(0, ceil_pages(kv.lens[b] + add[b]) - kv.held[b]); };
    for (int b = b0; b < b1; ++b) {
        const int L = kv.lens[b], a = add[b], h = kv.held[b];
        const long long room = (long long)kv.max_pages * SGD_PAGE;
        if (L < 0 || a < 0 || h < 0 || h > kv.max_pages || L > (long long)h * SGD_PAGE || (long long)L + a > room) {
            bad |= SGD_STATUS_SIZE_MISMATCH;
            continue;
        }
        // the held pages that it grows in: the part-filled last one, and any behind the last token
        for (int j = L / SGD_PAGE; a > 0 && j < min(h, ceil_pages(L + a)); ++j) {
            const int p = kv.table[(int64_t)b * kv.max_pages + j];
            if (p < 0 || p >= kv.n_pages) bad |= SGD_STATUS_BAD_INDEX;
            else if (kv.ref[p] > 1) bad |= SGD_STATUS_SHARED_PAGE;
        }
        sum += need(b);
    }
    if (threadIdx.x == 0) wanted = 0;
    bad = block_or(bad, sm);
    if (!bad && sum) atomicAdd(&wanted, (unsigned long long)sum);  // in 64 bits: it may pass 2^31
    __syncthreads();
    int total = 0;
    if (!bad) {
        if (wanted > (unsigned long long)kv.n_pages) {
            bad = SGD_STATUS_NO_PAGES;
        } else {
            int o = block_exclusive_scan((int)sum, total, sm);
            for (int b = b0; b < b1; ++b) {
                off[b] = o;
                o += need(b);
            }
            if (find_free(kv.ref, kv.n_pages, total, list, sm) < total) bad = SGD_STATUS_NO_PAGES;
        }
    }
    if (threadIdx.x == 0) *status = bad;
    if (!bad)
        for (int r = threadIdx.x; r < total; r += kAllocThreads) {
            const int b = owner(off, kv.B, r), p = list[r];
            kv.table[(int64_t)b * kv.max_pages + kv.held[b] + r - off[b]] = p;
            kv.ref[p] = 1;
        }
    __syncthreads();  // held and lens are read above
    for (int b = b0; b < b1; ++b) {
        const int L = kv.lens[b];
        if (!bad) kv.held[b] += need(b);
        new_lens[b] = bad ? L : L + add[b];
    }
}

// One CTA: checks the rows of a fork and takes the pages for part-filled last pages.
// fresh[i]: the new page of fork i, -1 where none is needed; *go = 1 where the fork goes ahead.
__global__ void __launch_bounds__(kAllocThreads) fork_plan_kernel(PagedView kv, const int32_t *src,
                                                                  const int32_t *dst, int n,
                                                                  int32_t *mark, int32_t *fresh, int32_t *list,
                                                                  int32_t *go, int32_t *status) {
    __shared__ int32_t sm[33];
    grid_dependency_wait();
    for (int b = threadIdx.x; b < kv.B; b += kAllocThreads) mark[b] = 0;
    __syncthreads();
    const int per = (n + kAllocThreads - 1) / kAllocThreads;
    const int i0 = min((int)threadIdx.x * per, n), i1 = min(i0 + per, n);
    int bad = 0, sum = 0;
    for (int i = i0; i < i1; ++i) {
        const int s = src[i], d = dst[i];
        if (s < 0 || s >= kv.B || d < 0 || d >= kv.B || kv.held[d] != 0 || atomicAdd(&mark[d], 1) != 0) {
            bad |= SGD_STATUS_BAD_INDEX;
            continue;
        }
        const int L = kv.lens[s], h = kv.held[s];
        if (L < 0 || h < 0 || h > kv.max_pages || L > (long long)h * SGD_PAGE) {
            bad |= SGD_STATUS_SIZE_MISMATCH;
            continue;
        }
        if (L % SGD_PAGE != 0) {
            const int p = kv.table[(int64_t)s * kv.max_pages + L / SGD_PAGE];
            if (p < 0 || p >= kv.n_pages) bad |= SGD_STATUS_BAD_INDEX;
            ++sum;
        }
    }
    __syncthreads();
    for (int i = i0; i < i1; ++i) {
        const int s = src[i];
        if (s >= 0 && s < kv.B && mark[s] != 0) bad |= SGD_STATUS_BAD_INDEX;
    }
    bad = block_or(bad, sm);
    if (!bad) {
        int total;
        int o = block_exclusive_scan(sum, total, sm);
        if (find_free(kv.ref, kv.n_pages, total, list, sm) < total) {
            bad = SGD_STATUS_NO_PAGES;
        } else {
            for (int i = i0; i < i1; ++i) fresh[i] = kv.lens[src[i]] % SGD_PAGE != 0 ? list[o++] : -1;
        }
    }
    if (threadIdx.x == 0) {
        *status = bad;
        *go = bad == 0;
    }
}

// CTA (i, h, K or V): the valid tokens of fork i's part-filled page, one KV head of K or V (one
// contiguous run of at most 16 KB); the CTA of h = 0, K also writes the new row's state.  A release and a fork of
// 64 rows to 7 each: 24 us, of which the plan takes 8 and the copies 16.
__global__ void __launch_bounds__(128) fork_copy_kernel(PagedView kv, const int32_t *src, const int32_t *dst,
                                                        const int32_t *fresh, const int32_t *go, int32_t *status) {
    grid_dependency_wait();
    if (*go == 0) return;
    const int i = blockIdx.x, h = blockIdx.y, s = src[i], d = dst[i];
    const int L = kv.lens[s], full = L / SGD_PAGE, to = fresh[i];
    const int32_t *from_row = kv.table + (int64_t)s * kv.max_pages;
    if (to >= 0) {
        const int64_t row = (int64_t)kv.D * kv.es, page = (int64_t)kv.Hkv * SGD_PAGE * row;
        uint8_t *pool = static_cast<uint8_t *>(blockIdx.z ? kv.v : kv.k);
        const int64_t head = (int64_t)h * SGD_PAGE * row;
        const uint4 *a = reinterpret_cast<const uint4 *>(pool + from_row[full] * page + head);
        uint4 *b = reinterpret_cast<uint4 *>(pool + to * page + head);
        const int nv = (int)((L % SGD_PAGE) * row / 16);
        uint4 x[8];  // 128 threads x 8 x 16 bytes: the whole run in flight at once
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (threadIdx.x + 128 * u < nv) x[u] = __ldcs(a + threadIdx.x + 128 * u);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (threadIdx.x + 128 * u < nv) b[threadIdx.x + 128 * u] = x[u];
    }
    if (h == 0 && blockIdx.z == 0) {
        int32_t *to_row = kv.table + (int64_t)d * kv.max_pages;
        for (int j = threadIdx.x; j < full; j += 128) {
            const int p = from_row[j];
            to_row[j] = p;
            if (p >= 0 && p < kv.n_pages) atomicAdd(&kv.ref[p], 1);
            else atomicOr(status, SGD_STATUS_BAD_INDEX);
        }
        if (threadIdx.x == 0) {
            if (to >= 0) {
                to_row[full] = to;
                kv.ref[to] = 1;
            }
            kv.held[d] = full + (to >= 0);
            kv.lens[d] = L;
        }
    }
}

// CTA b: the entries behind keep[b] lose a reference.
__global__ void __launch_bounds__(128) release_kernel(PagedView kv, const int32_t *__restrict__ keep,
                                                      int32_t *status) {
    const int b = blockIdx.x;
    int h = kv.held[b], k = keep[b], bad = 0;
    if (h < 0 || h > kv.max_pages || k < 0) bad = SGD_STATUS_SIZE_MISMATCH;
    h = min(max(h, 0), kv.max_pages);
    k = max(k, 0);
    const int stay = k / SGD_PAGE + (k % SGD_PAGE != 0);
    for (int j = stay + threadIdx.x; j < h; j += 128) {
        const int p = kv.table[(int64_t)b * kv.max_pages + j];
        if (p < 0 || p >= kv.n_pages) {
            bad |= SGD_STATUS_BAD_INDEX;
        } else if (atomicSub(&kv.ref[p], 1) <= 0) {  // was free already: put the count back
            atomicAdd(&kv.ref[p], 1);
            bad |= SGD_STATUS_BAD_INDEX;
        }
    }
    if (bad) atomicOr(status, bad);
    __syncthreads();
    if (threadIdx.x == 0) kv.held[b] = min(h, stay);
}

// CTA (32 new tokens, KV head): the first 32 threads find each token's slot, then all threads move
// the tokens' K and V rows, 16 bytes of the source at a time: 5.4 TB/s (43 us for 8 rows of 1000 to 8192).
constexpr int kAppendTokens = 32;

template <bool I8>
__global__ void __launch_bounds__(256) append_kernel(PagedView kv, const __nv_bfloat16 *__restrict__ k_new,
                                                     const __nv_bfloat16 *__restrict__ v_new,
                                                     const int32_t *__restrict__ cu, int64_t T_new, int32_t *status) {
    __shared__ int64_t slot[kAppendTokens];  // row of the pool seen as [n_pages * Hkv * 64, D], -1: not written
    const int h = blockIdx.y;
    const int64_t i0 = (int64_t)blockIdx.x * kAppendTokens;
    if (threadIdx.x < kAppendTokens) {
        const int64_t i = i0 + threadIdx.x;
        int64_t row = -1;
        int bad = 0;
        if (i < T_new) {
            int lo = 0, hi = kv.B - 1;  // the last b with cu[b] <= i
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (cu[mid] <= i) lo = mid;
                else hi = mid - 1;
            }
            const int64_t t = (int64_t)kv.lens[lo] - cu[lo + 1] + i;
            if (i < cu[lo] || i >= cu[lo + 1] || t < 0 || t >= (int64_t)kv.max_pages * SGD_PAGE) {
                bad = SGD_STATUS_SIZE_MISMATCH;
            } else {
                const int p = kv.table[(int64_t)lo * kv.max_pages + t / SGD_PAGE];
                const int held = kv.held ? kv.held[lo] : kv.max_pages;
                // a page of the row's own: lens may be that of a refused reserve, or of a row that has ended
                const int owners = p < 0 || p >= kv.n_pages ? 0 : kv.ref ? kv.ref[p] : 1;
                if (t >= (int64_t)held * SGD_PAGE) bad = SGD_STATUS_SIZE_MISMATCH;
                else if (owners == 1) row = ((int64_t)p * kv.Hkv + h) * SGD_PAGE + t % SGD_PAGE;
                else bad = owners < 1 ? SGD_STATUS_BAD_INDEX : SGD_STATUS_SHARED_PAGE;
            }
        }
        if (blockIdx.x == 0 && threadIdx.x == 0 && (cu[0] != 0 || cu[kv.B] != T_new)) bad |= SGD_STATUS_SIZE_MISMATCH;
        if (bad) atomicOr(status, bad);
        slot[threadIdx.x] = row;
    }
    float ks = 0.f, vs = 0.f;
    if constexpr (I8) {
        const bool report = blockIdx.x == 0 && h == 0 && threadIdx.x == 0;
        ks = calibrated_scale(kv.k_scale, status, report);
        vs = calibrated_scale(kv.v_scale, status, report);
    }
    __syncthreads();
    const int shift = kv.D == 128 ? 4 : 3;  // 16-byte vectors of a source row
    const int n = (int)min((int64_t)kAppendTokens, T_new - i0) << shift;
    const int64_t first = ((int64_t)h * T_new + i0) * kv.D;
#pragma unroll 2
    for (int e = threadIdx.x; e < n; e += 256) {
        const int64_t row = slot[e >> shift];
        if (row < 0) continue;
        const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(k_new + first) + e);
        const uint4 c = __ldcs(reinterpret_cast<const uint4 *>(v_new + first) + e);
        const int64_t at = row * kv.D + (e & ((1 << shift) - 1)) * 8;  // element of the pool
        if constexpr (I8) {
            float x[8];
            Vec<__nv_bfloat16>::unpack(a, x);
            store_codes<8, true>(static_cast<int8_t *>(kv.k) + at, x, ks, ks != 0.f ? __frcp_rn(ks) : 0.f, 127.f * ks);
            Vec<__nv_bfloat16>::unpack(c, x);
            store_codes<8, true>(static_cast<int8_t *>(kv.v) + at, x, vs, vs != 0.f ? __frcp_rn(vs) : 0.f, 127.f * vs);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(kv.k) + at) = a;
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(kv.v) + at) = c;
        }
    }
}

// Compaction in place: of one row and KV head, entry base + list[i] moves to base + i, i < n.
// list ascends strictly from >= 0, so list[i] >= i, and the row that entry i overwrites can only be the
// source of entries up to i: steps of rows are written in order, each after a barrier behind which all
// sources up to its own were read.  Reading ahead is always safe (a source is never a row that a smaller
// entry overwrote), so the steps' sources stream through a ring of asynchronous copies, two steps of 32 KB
// ahead, and their list entries as far ahead of those.  A step has a row for every thread, which finds where it
// comes from and goes to; with fewer rows a step, or pieces looked up one by one, the lookups bound the kernel
// (8 x 32K tokens kept to an eighth: 94 us piece by piece, 79 us with 64 rows a step, 52 us with 256).  What is left:
// page table entries looked up in global memory between a step's two barriers (long scoreboard 3.1 warps an issue, short 1.8,
// DRAM 28%), and unequal CTAs (active cycles of an SM 18 to 43 thousand).
// CTA (row, KV head; K or V; slice of the row's bytes); LANES threads of 16 bytes to a slice.
constexpr int kCompactThreads = 256, kRing = 3;

template <int LANES>
struct CompactShared {
    uint4 ring[kRing][LANES][kCompactThreads];  // a thread's pieces are its own
    int32_t ids[kRing + 2][kCompactThreads];    // list entries of the steps ahead
    int2 move[kRing + 1][kCompactThreads];      // their (from, to) as rows of the pool; from < 0: stays
};

// The first of n entries that moves in any of a row's `heads` lists, `stride` apart: one that names itself stays, and as
// a list ascends strictly those are its first ones.  `least` is shared memory.  Out of line: it is for rows with
// shared pages alone, and its code beside the copies' cost the others 2 of 52 us (8 x 32K tokens kept to an eighth).
__device__ __noinline__ int first_move(const int32_t *lists, int heads, int64_t stride, int n, int32_t *least) {
    if (threadIdx.x == 0) *least = n;
    __syncthreads();
    for (int g = threadIdx.x; g < heads; g += kCompactThreads) {
        const int32_t *list = lists + g * stride;
        int lo = 0, hi = n;
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (list[mid] == mid) lo = mid + 1;
            else hi = mid;
        }
        atomicMin(least, lo);
    }
    __syncthreads();
    const int first = *least;
    __syncthreads();  // before the memory serves another purpose
    return first;
}

template <bool ACCEPT, int LANES>
__global__ void __launch_bounds__(kCompactThreads, 2) compact_kernel(PagedView kv, CompactArgs a) {
    const int b = blockIdx.x / kv.Hkv, h = blockIdx.x % kv.Hkv;
    int L = kv.lens[b], bad = 0, n, base = 0, limit;
    const int held = kv.held ? kv.held[b] : kv.max_pages;
    const int32_t *list;
    auto leave = [&](int why) {  // the row stays as it is, and a release that follows takes nothing from it
        if (threadIdx.x != 0) return;
        atomicOr(a.status, why);
        if (h == 0 && blockIdx.y == 0 && blockIdx.z == 0) a.new_lens[b] = L;
    };
    if (L < 0 || L > (int64_t)kv.max_pages * SGD_PAGE) bad = SGD_STATUS_SIZE_MISMATCH;
    const int len = min(max(L, 0), kv.max_pages * SGD_PAGE);
    if constexpr (ACCEPT) {
        const int nodes = min(max(a.n_nodes[b], 0), min(len, a.M));
        n = min(max(a.n_path[b], 0), nodes);
        if (nodes != a.n_nodes[b] || n != a.n_path[b]) bad |= SGD_STATUS_SIZE_MISMATCH;
        base = len - nodes;
        limit = nodes;
        list = a.path + (int64_t)b * a.M;
    } else {
        const int64_t c0 = a.cu_kept[b], c1 = a.cu_kept[b + 1];
        if (bad || c0 < 0 || c1 < c0 || c1 > a.kept_total || c1 - c0 > len) return leave(SGD_STATUS_SIZE_MISMATCH);
        n = (int)(c1 - c0);
        limit = len;
        list = a.idx + (int64_t)h * a.kept_total + c0;
    }
    const int32_t *row = kv.table + (int64_t)b * kv.max_pages;
    // a row that was released but still has its old length lists pages that are free, or another row's by now
    if (len > (int64_t)held * SGD_PAGE) return leave(SGD_STATUS_SIZE_MISMATCH);
    // the pages of the entries that the list names: base / 64 .. (base + n - 1) / 64
    int shared = 0, vacant = 0;
    for (int j = base / SGD_PAGE + threadIdx.x; j < ceil_pages(base + n) && n > 0; j += kCompactThreads) {
        const int p = row[j];
        if (p < 0 || p >= kv.n_pages) {
            bad |= SGD_STATUS_BAD_INDEX;
        } else {
            const int owners = kv.ref[p];
            shared |= owners > 1;
            vacant |= owners < 1;
        }
    }
    extern __shared__ __align__(16) uint8_t smem[];
    auto &sh = *reinterpret_cast<CompactShared<LANES> *>(smem);
    int first = 0;  // entries before this one stay where they are
    if (__syncthreads_or(shared | vacant)) {
        if (__syncthreads_or(vacant)) return leave(SGD_STATUS_BAD_INDEX);
        first = first_move(ACCEPT ? list : list - (int64_t)h * a.kept_total, ACCEPT ? 1 : kv.Hkv, a.kept_total, n, &sh.ids[0][0]);
        shared = 0;
        for (int j = (base + first) / SGD_PAGE + threadIdx.x; j < ceil_pages(base + n) && first < n; j += kCompactThreads) {
            const int p = row[j];
            if (p >= 0 && p < kv.n_pages && kv.ref[p] > 1) shared = 1;
        }
        if (__syncthreads_or(shared)) return leave(SGD_STATUS_SHARED_PAGE);
    }
    if (threadIdx.x == 0 && h == 0 && blockIdx.y == 0 && blockIdx.z == 0) a.new_lens[b] = base + n;

    constexpr int ROWS = kCompactThreads;  // of a step
    const int row_bytes = kv.D * kv.es, tid = threadIdx.x;
    uint8_t *pool = static_cast<uint8_t *>(blockIdx.y ? kv.v : kv.k) + (int64_t)blockIdx.z * LANES * 16 + tid % LANES * 16;
    auto row_of = [&](int u) { return u * (ROWS / LANES) + tid / LANES; };  // the step's row of the thread's piece u
    auto load_ids = [&](int step) {
        const int i = step * ROWS + tid;
        if (i < n) cp_async_4(&sh.ids[step % (kRing + 2)][tid], list + i);
    };
    auto pool_row = [&](int t) {  // entry t, -1 for a page outside the pool
        const int p = row[t / SGD_PAGE];
        if (p >= 0 && p < kv.n_pages) return (p * kv.Hkv + h) * SGD_PAGE + t % SGD_PAGE;
        bad |= SGD_STATUS_BAD_INDEX;
        return -1;
    };
    auto resolve = [&](int step) {  // thread k: the step's row k
        const int i = step * ROWS + tid;
        if (i >= n) return;
        const int id = sh.ids[step % (kRing + 2)][tid];
        const int prev = i == 0 ? -1 : tid > 0 ? sh.ids[step % (kRing + 2)][tid - 1] : sh.ids[(step - 1) % (kRing + 2)][ROWS - 1];
        const int from = min(max(id, i), limit - 1);  // a bad list stays within [i, limit)
        if (from != id || prev >= id) bad |= SGD_STATUS_BAD_INDEX;
        int2 m = make_int2(-1, -1);
        if (from != i && i >= first) {
            m = make_int2(pool_row(base + from), pool_row(base + i));
            if (m.y < 0) m.x = -1;
        }
        sh.move[step % (kRing + 1)][tid] = m;
    };
    auto load = [&](int step) {
#pragma unroll
        for (int u = 0; u < LANES; ++u) {
            if (step * ROWS + row_of(u) >= n) continue;
            const int from = sh.move[step % (kRing + 1)][row_of(u)].x;
            if (from >= 0) cp_async_16(&sh.ring[step % kRing][u][tid], pool + (int64_t)from * row_bytes);
        }
    };
    auto store = [&](int step) {
#pragma unroll
        for (int u = 0; u < LANES; ++u) {
            if (step * ROWS + row_of(u) >= n) continue;
            const int2 m = sh.move[step % (kRing + 1)][row_of(u)];
            if (m.x >= 0) *reinterpret_cast<uint4 *>(pool + (int64_t)m.y * row_bytes) = sh.ring[step % kRing][u][tid];
        }
    };
    constexpr int AHEAD = ACCEPT ? 1 : kRing;  // an accepted path is one step
    for (int s = 0; s < AHEAD; ++s) load_ids(s);
    cp_async_wait_all();
    __syncthreads();
    for (int s = 0; s < AHEAD; ++s) resolve(s);
    __syncthreads();
    if constexpr (ACCEPT) {
        load(0);
        cp_async_wait_all();
        __syncthreads();
        store(0);
    } else {
        const int steps = (n + ROWS - 1) / ROWS;
        for (int s = 0; s < kRing - 1; ++s) {  // group s: the sources of step s, the list of step s + kRing
            load(s);
            load_ids(s + kRing);
            cp_async_commit();
        }
        for (int s = 0; s < steps; ++s) {
            cp_async_wait_group<kRing - 2>();  // groups up to s
            __syncthreads();
            store(s);
            load(s + kRing - 1);
            load_ids(s + 2 * kRing - 1);
            cp_async_commit();
            resolve(s + kRing);
        }
        cp_async_wait_all();
    }
    if (bad) atomicOr(a.status, bad);
}

template <bool ACCEPT, int LANES>
int launch_compact(const PagedView &kv, const CompactArgs &a, cudaStream_t s) {
    auto k = compact_kernel<ACCEPT, LANES>;
    constexpr int smem = sizeof(CompactShared<LANES>);
    static SmemOptIn opt_in;
    if (!opt_in.set(reinterpret_cast<const void *>(k), smem)) return SGD_ERR_CUDA;
    const dim3 grid(kv.B * kv.Hkv, 2, kv.D * kv.es / (LANES * 16));
    const cudaError_t e = launch_k(k, grid, dim3(kCompactThreads), smem, s, 1, kv, a);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? SGD_OK : SGD_ERR_CUDA;
}

bool ok() { return cudaGetLastError() == cudaSuccess; }

}  // namespace

int launch_pages_reserve(const PagedView &kv, const int32_t *add, int32_t *new_lens, int32_t *scratch,
                         int32_t *status, cudaStream_t s) {
    launch_k_early(reserve_kernel, dim3(1), dim3(kAllocThreads), 0, s, kv, add, new_lens, scratch, scratch + kv.B, status);
    return ok() ? SGD_OK : SGD_ERR_CUDA;
}

int launch_pages_fork(const PagedView &kv, const int32_t *src, const int32_t *dst, int n, int32_t *scratch,
                      int32_t *status, cudaStream_t s) {
    int32_t *mark = scratch, *fresh = mark + kv.B, *go = fresh + kv.B, *list = go + 1;
    launch_k_early(fork_plan_kernel, dim3(1), dim3(kAllocThreads), 0, s, kv, src, dst, n, mark, fresh, list, go, status);
    launch_k_early(fork_copy_kernel, dim3(n, kv.Hkv, 2), dim3(128), 0, s, kv, src, dst, fresh, go, status);
    return ok() ? SGD_OK : SGD_ERR_CUDA;
}

int launch_pages_release(const PagedView &kv, const int32_t *keep, int32_t *status, cudaStream_t s) {
    launch_k(release_kernel, dim3(kv.B), dim3(128), 0, s, 1, kv, keep, status);
    return ok() ? SGD_OK : SGD_ERR_CUDA;
}

int launch_pages_append(const PagedView &kv, const void *k_new, const void *v_new, const int32_t *cu, int64_t T_new,
                        int32_t *status, cudaStream_t s) {
    // without tokens one CTA still checks cu_new
    const dim3 grid((unsigned)std::max<int64_t>((T_new + kAppendTokens - 1) / kAppendTokens, 1), kv.Hkv);
    auto k = kv.es == 1 ? append_kernel<true> : append_kernel<false>;
    launch_k(k, grid, dim3(256), 0, s, 1, kv, static_cast<const __nv_bfloat16 *>(k_new),
             static_cast<const __nv_bfloat16 *>(v_new), cu, T_new, status);
    return ok() ? SGD_OK : SGD_ERR_CUDA;
}

int launch_pages_compact(const PagedView &kv, const CompactArgs &a, bool accept, cudaStream_t s) {
    if (kv.D * kv.es < 128) return accept ? launch_compact<true, 4>(kv, a, s) : launch_compact<false, 4>(kv, a, s);
    return accept ? launch_compact<true, 8>(kv, a, s) : launch_compact<false, 8>(kv, a, s);
}

}  // namespace sgd
