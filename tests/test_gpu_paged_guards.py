"""Calls on a paged cache whose counts, lengths or owners are not what the call needs: rows that cannot be
served stay as they are, nothing of another row is written, and the status says so."""
import numpy as np
import pytest
import torch

from test_gpu_paged import PAGE, Case, ints, same_state, sgd  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------------------
# compaction
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("cu,wrong", [([0, 2, 1, 5], 1), ([0, 2, 4, 90], 2), ([-1, 2, 4, 5], 0), ([0, 2, 4, 35], 2), ([0, 2, 4, 5], None)])
def test_keep_leaves_rows_with_wrong_counts(sgd, cu, wrong):
    """cu_kept that descends, leaves the list or asks for more tokens than the row has: the row keeps all of its tokens,
    and the release that follows a keep takes no page from it.  (None: a length that no row can have.)"""
    case = Case((100, 70, 30), seed=4)
    if wrong is None:
        case.lens[1], wrong = 10 ** 6, 1
    cache, st = case.gpu(sgd), case.host()
    idx = np.tile(np.arange(40), (2, 1))
    idx[:, :5] = (3, 9, 5, 29, 29)
    if cu[2] == 1:
        idx[:, :5] = (0, 2, 9, 11, 29)
    new, ws = sgd.pages_keep(cache, ints(idx), ints(cu))
    assert sgd.workspace_status(ws) == 0x4
    want = np.diff(cu)
    want[wrong] = case.lens[wrong]
    assert new.tolist() == want.tolist()
    for b in range(3):
        for h in range(2):
            if b != wrong:
                st._compact(b, h, 0, idx[h, cu[b]:cu[b + 1]])
    same_state(cache, st)
    sgd.pages_release(cache, new)
    held = [-(-int(n) // PAGE) for n in want]
    held[wrong] = int(case.held[wrong])
    assert cache.held.tolist() == held and int(cache.ref_count.sum()) == sum(held)


@pytest.mark.parametrize("call", ["keep", "accept"])
@pytest.mark.parametrize("taken", [True, False])
def test_compaction_of_an_ended_row_writes_nothing(sgd, call, taken):
    """A row that was released but still has its old length: its table lists pages that are free, or another row's."""
    case = Case((200, 64, 130), seed=11, max_pages=8)
    cache = case.gpu(sgd)
    for t in (cache.k, cache.v):
        t.nan_to_num_(0.0)
    sgd.pages_release(cache, ints([0, 64, 130]))
    if taken:  # row 1 takes the pages
        new, ws = sgd.pages_reserve(cache.with_lens(ints([0, 64, 130])), ints([0, 200, 0]))
        assert sgd.workspace_status(ws) == 0 and new.tolist() == [0, 264, 130]
        cache.lens[1] = 264
        assert set(cache.page_table[1, 1:5].tolist()) & set(cache.page_table[0, :4].tolist())
    k, v, L = cache.k.clone(), cache.v.clone(), cache.lens.tolist()

    def go(held):
        c = sgd.PagedKv(cache.k, cache.v, cache.page_table, cache.lens, cache.held if held else None, cache.ref_count)
        if call == "keep":  # rows 1 and 2 keep everything
            parts = [np.arange(1, 150), np.arange(L[1]), np.arange(L[2])]
            cu = np.concatenate([[0], np.cumsum([len(p) for p in parts])])
            return sgd.pages_keep(c, ints(np.tile(np.concatenate(parts), (2, 1))), ints(cu))
        return sgd.pages_accept(c, ints([[3, 5, 6, -1, -1, -1, -1], [0, 1, 2, 3, 4, 5, 6], [0, 1, 2, 3, 4, 5, 6]]), ints([3, 7, 7]),
                                ints([7, 7, 7]))

    new, ws = go(True)
    assert sgd.workspace_status(ws) == 0x4 and new.tolist() == L
    assert torch.equal(cache.k, k) and torch.equal(cache.v, v)
    if not taken:  # without held the free pages themselves tell
        new, ws = go(False)
        assert sgd.workspace_status(ws) == 0x8 and new.tolist() == L
        assert torch.equal(cache.k, k) and torch.equal(cache.v, v)


def forked(sgd, L, seed):
    """Row 0 of L tokens, row 1 its fork, row 2 with 300 tokens of its own; finite everywhere."""
    case = Case((L, 0, 300), seed=seed, spare=4, max_pages=-(-L // PAGE) + 1)
    case.k.nan_to_num_(0.0)
    case.v.nan_to_num_(0.0)
    cache, st = case.gpu(sgd), case.host()
    sgd.pages_fork(cache, ints([0]), ints([1]))
    assert st.fork(np.array([0]), np.array([1])) == 0
    return cache, st


def lists(per_row):
    """per_row[b][h] -> (idx [Hkv, kept], cu)."""
    cu = np.concatenate([[0], np.cumsum([len(r[0]) for r in per_row])]).astype(np.int32)
    return np.stack([np.concatenate([r[h] for r in per_row]) for h in range(2)]).astype(np.int32), cu


@pytest.mark.parametrize("L", [200, 5010, 192])
def test_keep_of_shared_pages_that_are_not_written(sgd, L):
    """Tokens that stay where they are in pages of a fork are no write: the row may drop others behind them."""
    full = L // PAGE * PAGE
    some = np.array([1, 5, 64, 130, 299])
    cut = np.arange(100)                                                  # cut inside a shared page
    own = [np.concatenate([np.arange(full), t]) for t in ([full + 1, full + 7], [full, full + 4])] if L > full else \
        [np.arange(L)] * 2                                                # moves in the own last page alone
    cache, st = forked(sgd, L, L)
    idx, cu = lists([[cut, cut], own, [some, some + 0]])
    new, ws = sgd.pages_keep(cache, ints(idx), ints(cu))
    assert sgd.workspace_status(ws) == 0 and np.array_equal(new.cpu().numpy(), st.keep(idx, cu))
    same_state(cache, st)
    # one head would write a shared page: the row stays as it is, with all of its heads
    cache, st = forked(sgd, L, L)
    drop = np.delete(np.arange(len(own[0]) + 1), 70)
    drop = drop[:len(own[0])] if drop[len(own[0]) - 1] < L else np.delete(np.arange(L), 70)
    keep = [own[0][:len(drop)], drop]
    idx, cu = lists([[cut, cut], keep, [some, some]])
    new, ws = sgd.pages_keep(cache, ints(idx), ints(cu))
    assert sgd.workspace_status(ws) == 0x40 and new.tolist() == [100, L, 5]
    for h in range(2):
        st._compact(2, h, 0, some)
    same_state(cache, st)


def test_keep_with_a_bad_list_writes_no_shared_page(sgd):
    # entries in place around others out of order: whatever is made of such a list, the shared pages stay
    for at, value in ((0, 5), (30, 2), (10, 190), (63, 64), (150, 149)):
        cache, st = forked(sgd, 200, 3)
        rows = np.arange(199)
        rows[at] = value
        idx, cu = lists([[rows, rows], [np.arange(200)] * 2, [np.arange(300)] * 2])
        _, ws = sgd.pages_keep(cache, ints(idx), ints(cu))
        assert sgd.workspace_status(ws) & 0x48
        shared = st.ref > 1
        for name in ("k", "v"):
            got, want = getattr(cache, name).float().cpu().numpy(), getattr(st, name)
            assert np.array_equal(got[shared], want[shared])


def test_accept_of_shared_pages_that_are_not_written(sgd):
    """A step's row forked before its drafts were accepted: nodes that stay where they are write nothing."""
    n = M = 64
    for path, ok in (([0, 1, 2], True), ([0, 2, 3], False), ([], True), (list(range(M)), True)):
        cache, st = forked(sgd, 192, 9)
        p = np.full((3, M), -1, np.int32)
        p[0, :len(path)] = path
        p[2, :2] = (1, 3)
        n_path = np.array([len(path), 0, 2], np.int32)
        n_nodes = np.array([n, 0, 5], np.int32)
        new, ws = sgd.pages_accept(cache, ints(p), ints(n_path), ints(n_nodes))
        if ok:
            assert sgd.workspace_status(ws) == 0 and np.array_equal(new.cpu().numpy(), st.accept(p, n_path, n_nodes))
        else:
            assert sgd.workspace_status(ws) == 0x40 and new.tolist() == [192, 192, 297]
            for h in range(2):
                st._compact(2, h, 295, (1, 3))
        same_state(cache, st)


# ---------------------------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "int8"])
def test_append_writes_the_rows_own_pages_alone(sgd, dtype):
    """Where lens does not count the new tokens (a reserve was refused) or the row has ended, the last entries lie in
    pages that a fork shares, that are free, or that another row has taken: they stay as they are."""
    rng = np.random.default_rng(3)
    new = torch.from_numpy(rng.standard_normal((2, 70, 128), dtype=np.float32)).bfloat16().cuda()

    def go(cache, cu, held=True, n=70):
        c = sgd.PagedKv(cache.k, cache.v, cache.page_table, cache.lens, cache.held if held else None, cache.ref_count,
                        cache.k_scale, cache.v_scale)
        return sgd.workspace_status(sgd.pages_append(c, new[:, :n].contiguous(), new[:, :n].contiguous(), ints(cu)))

    def make():
        case = Case((200, 0, 64), seed=12, spare=4, max_pages=8, dtype=dtype)
        case.k, case.v = (t.nan_to_num(0.0) if dtype == "bf16" else t for t in (case.k, case.v))
        return case.gpu(sgd)

    # 200 tokens forked: the last 8 in a page of their own, 62 of the 70 in a shared one
    cache = make()
    sgd.pages_fork(cache, ints([0]), ints([1]))
    k = cache.k.clone()
    assert go(cache, [0, 70, 70, 70]) == 0x40
    changed = (cache.k != k).flatten(1).any(1).nonzero()[:, 0].tolist()
    assert changed == [int(cache.page_table[0, 3])] and (cache.k[changed[0], :, 8:] == k[changed[0], :, 8:]).all()
    # an ended row, its pages free
    cache = make()
    sgd.pages_release(cache, ints([0, 0, 64]))
    k, v = cache.k.clone(), cache.v.clone()
    assert go(cache, [0, 70, 70, 70]) == 0x4 and torch.equal(cache.k, k) and torch.equal(cache.v, v)
    assert go(cache, [0, 70, 70, 70], held=False) == 0x8 and torch.equal(cache.k, k) and torch.equal(cache.v, v)
    # taken by row 2
    _, ws = sgd.pages_reserve(cache.with_lens(ints([0, 0, 64])), ints([0, 0, 250]))
    assert sgd.workspace_status(ws) == 0
    assert go(cache, [0, 70, 70, 70]) == 0x4 and torch.equal(cache.k, k) and torch.equal(cache.v, v)
    # without the counts a caller answers for the pages
    cache = make()
    c = sgd.PagedKv(cache.k, cache.v, cache.page_table, cache.lens, k_scale=cache.k_scale, v_scale=cache.v_scale)
    assert sgd.workspace_status(sgd.pages_append(c, new, new, ints([0, 70, 70, 70]))) == 0


def test_append_of_nothing_checks_its_offsets(sgd):
    cache = Case((100, 70), seed=4).gpu(sgd)
    none = torch.zeros(2, 0, 128, dtype=torch.bfloat16, device="cuda")
    for cu, code in (([0, 0, 0], 0), ([0, 3, 6], 0x4), ([0, 1, 0], 0), ([1, 1, 1], 0x4)):
        assert sgd.workspace_status(sgd.pages_append(cache, none, none, ints(cu))) == code, cu


# ---------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "int8"])
@pytest.mark.parametrize("M", [3, 40])
def test_attn_asks_nothing_of_pages_that_no_query_sees(sgd, dtype, M):
    """Table entries between the first tokens and the window may hold anything, beside seen pages too."""
    lens, window, sinks = (700, 130, 901, 1500), 70, 5
    case = Case(lens, dtype=dtype, seed=9)
    q = case.query(M, 8).cuda()
    want = sgd.paged_attn(q, 8, case.gpu(sgd), window=window, sinks=sinks)
    assert sgd.workspace_status(want[2]) == 0
    gone, seen = 0, []
    for b, L in enumerate(lens):
        first = max(L - M + 1 - window, 0)  # the first entry of any window
        for j in range(-(-L // PAGE)):
            if j * PAGE >= sinks and (j + 1) * PAGE <= first:
                case.table[b, j] = (-1, case.n_pages, 2 ** 31 - 1)[gone % 3]
                gone += 1
            else:
                seen.append((b, j))
    assert gone > 25
    got = sgd.paged_attn(q, 8, case.gpu(sgd), window=window, sinks=sinks)
    assert sgd.workspace_status(got[2]) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # a row without nodes sees nothing at all
    n = ints([M, 0, M, M])
    bare = case.gpu(sgd)
    bare.page_table[1] = -1
    got = sgd.paged_attn(q, 8, bare, n_nodes=n, window=window, sinks=sinks)
    assert sgd.workspace_status(got[2]) == 0 and (got[0][1] == 0).all() and torch.isneginf(got[1][1]).all()
    for b, j in seen:  # every other one counts
        cache = case.gpu(sgd)
        cache.page_table[b, j] = -1
        assert sgd.workspace_status(sgd.paged_attn(q, 8, cache, window=window, sinks=sinks)[2]) == 0x8, (b, j)


# ---------------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------------
def test_a_step_whose_reserve_was_refused_changes_nothing(sgd):
    """The step's counts taken from what the reserve granted, on the device: where the pool has too few pages the calls
    that follow write, answer and accept nothing."""
    B, M, Hkv, G, D, V = 3, 6, 2, 4, 128, 50
    case = Case((64, 640, 128), Hkv=Hkv, D=D, seed=6, spare=0, max_pages=14)  # one free page, two needed
    case.k.nan_to_num_(0.0)
    case.v.nan_to_num_(0.0)
    cache, st = case.gpu(sgd), case.host()
    nodes, parent = ints([6, 0, 5]), ints([[-1, 0, 0, 1, 2, 2]] * B)
    grown, ws = sgd.pages_reserve(cache, nodes)
    assert sgd.workspace_status(ws) == 0x20
    n = grown - cache.lens
    cu = torch.nn.functional.pad(n.cumsum(0, dtype=torch.int32), (1, 0))
    step = cache.with_lens(grown)
    new = torch.ones(Hkv, 11, D, dtype=torch.bfloat16, device="cuda")
    assert sgd.workspace_status(sgd.pages_append(step, new, new, cu)) == 0x4  # cu ends at 0, not at 11
    out, lse, ws = sgd.paged_attn(case.query(M, G).cuda(), G, step, parent, n)
    assert sgd.workspace_status(ws) == 0 and (out == 0).all() and torch.isneginf(lse).all()
    u = torch.zeros(B, M, device="cuda")
    n_path, path, token, ws = sgd.verify_tree(torch.full((B, M, V), 1 / V, device="cuda"), ints([[0] * M] * B), parent, u, u[:, 0].contiguous(),
                                              n_nodes=n)
    assert sgd.workspace_status(ws) == 0 and n_path.tolist() == [0] * B and token.tolist() == [-1] * B
    lens, ws = sgd.pages_accept(step, path, n_path, n)
    assert sgd.workspace_status(ws) == 0 and lens.tolist() == case.lens.tolist()
    sgd.pages_release(step, lens)
    same_state(cache, st)


def test_int8_attention_is_closer_than_bf16_probabilities(sgd):
    """On an INT8 cache p enters the second product as float16 with 2^7 (off by at most 2^-11 of itself, or by 2^-32
    of the largest), where bfloat16 would allow 2^-8: sums that nearly cancel show the difference.
    Bounds beside the output's 2^-8 |out| and the logits' error as in the other attention tests: Q's bits below 2^-38
    of its row's maximum are lost; the running sum of L / 16 products of 16 tokens, and 16 of a merge, is rounded (or
    truncated) to 2^-23 each, twice for the two operands of a sum."""
    import math

    from oracle import paged as orc
    lens, G, M, D = (2, 3, 5, 9, 40, 300, 2053), 8, 2, 128
    case = Case(lens, D=D, dtype="int8", seed=77)
    case.ks = 0.002  # logits of a few tenths: their own error is far below the bound
    q = case.query(M, G)
    out, lse, ws = sgd.paged_attn(q.cuda(), G, case.gpu(sgd))
    assert sgd.workspace_status(ws) == 0
    ks, vs = (float(np.float32(x)) for x in (case.ks, case.vs))
    args = (q.float().numpy(), G, case.k.float().numpy(), case.v.float().numpy(), case.table, case.lens, None, None, 0, 0, ks, vs)
    ref, rlse, mass, zabs = orc.attn(*args)
    L = np.array(lens, float)[:, None, None, None]
    qmax = np.abs(q.float().numpy()).max(-1)[..., None]
    tz = 2.0 ** -15.9 * zabs[..., None] + 2.0 ** -18 + 2.0 ** -38 * qmax * 127 * ks * math.sqrt(D)
    tol = (2.0 ** -11 + 2 * tz + 2.0 ** -22 * (L / 16 + 16)) * mass + L * 2.0 ** -32 * 127 * vs + 2.0 ** -8 * np.abs(ref)
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    # the same bound finds probabilities that were rounded to bfloat16
    off = 0
    for b, n in enumerate(lens):
        for h in range(2):
            kk, vv = orc.rows(args[2], case.table[b], n, h) * ks, orc.rows(args[3], case.table[b], n, h) * vs
            for m in range(M):
                see = n - M + m + 1
                z = kk[:see] @ args[0][b, m, h * G:h * G + G].astype(np.float64).T / math.sqrt(D)
                e = np.exp(z - z.max(0))
                p = torch.from_numpy(e).bfloat16().double().numpy() / e.sum(0)
                here = slice(h * G, h * G + G)
                off += (np.abs(p.T @ vv[:see] - ref[b, m, here]) > tol[b, m, here]).sum()
    assert off > 20


@pytest.mark.parametrize("D,Hkv", [(64, 3), (128, 1)])
def test_append_codes_at_other_sizes(sgd, D, Hkv):
    import oracle
    rng = np.random.default_rng(D)
    new = [33, 0, 130, 1]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    case = Case((70, 3, 200, 64), Hkv=Hkv, D=D, dtype="int8", seed=D)
    cache, st = case.gpu(sgd), case.host()
    k, v = (torch.from_numpy(rng.standard_normal((Hkv, cu[-1], D), dtype=np.float32) * np.float32(1.5)).bfloat16() for _ in range(2))
    assert sgd.workspace_status(sgd.pages_append(cache, k.cuda(), v.cuda(), ints(cu))) == 0
    codes = [oracle.quantize(x.float().numpy(), np.float32(s)) for x, s in ((k, case.ks), (v, case.vs))]
    st.append(codes[0].reshape(k.shape), codes[1].reshape(v.shape), cu)
    same_state(cache, st)


def test_calls_from_two_host_threads(sgd):
    """Each thread with a stream, a cache and workspaces of its own, the same kernels at the same time."""
    import threading
    cases = [Case([int(x) for x in np.random.default_rng(s).integers(10, 3000, 6)], seed=s, spare=40, max_pages=60) for s in (3, 4)]
    qs = [c.query(5, 8).cuda() for c in cases]
    add = ints([5] * 6)

    def work(i, stream):
        cache = cases[i].gpu(sgd)
        torch.cuda.synchronize()
        done = []
        with torch.cuda.stream(stream):
            for _ in range(20):
                out, lse, ws = sgd.paged_attn(qs[i], 8, cache)
                new, ws2 = sgd.pages_reserve(cache, add)
                ws3 = sgd.pages_release(cache, cache.lens)
                done.append((out, lse, new, ws, ws2, ws3))
        stream.synchronize()
        return done

    want = [work(i, torch.cuda.Stream())[0] for i in (0, 1)]
    got, failed = [None, None], []

    def thread(i):
        try:
            got[i] = work(i, torch.cuda.Stream())
        except BaseException as e:  # noqa: BLE001  (reported by the test, not lost with the thread)
            failed.append(e)

    threads = [threading.Thread(target=thread, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for i in (0, 1):
        for out, lse, new, *ws in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1]) and torch.equal(new, want[i][2])
            assert all(sgd.workspace_status(w) == 0 for w in ws)
