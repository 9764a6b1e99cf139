"""The paged cache on the GPU against the fp64 oracle: attention of trees, chains and single tokens
(windows, first tokens, padded batches, garbage behind the masks), draft verification, the upkeep
of the pages, and a whole speculative step of them together.

Tolerances of the attention, element by element and from the arithmetic: the probabilities p enter the
second product as bfloat16, off by at most 2^-8 of themselves, so out is off by at most
2^-8 sum p |v|; the output's own rounding adds 2^-8 |out|.  A logit is a sum of D exact products in
float32: at most D + 2 roundings of 2^-24 (the running sum, the scale; twice that, since a tensor core
may truncate) of sum |q k| / sqrt(D), D <= 128, so 2^-15.9 of it with the factor 2; exp2, log2 and
the sums of positive terms add less than 2^-18 to lse.  A logit's error e scales p by 1 + e, twice
(numerator and sum).  Verification and page upkeep are exact.
"""
import numpy as np
import pytest
import torch

from oracle import paged as orc

pytestmark = pytest.mark.gpu

PAGE = 64


@pytest.fixture(scope="module")
def sgd():
    from conftest import build_library
    m = build_library()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Case:
    """A pool whose pages are handed out in random order; slots behind the last token hold NaN (bf16)."""

    def __init__(self, lens, Hkv=2, D=128, dtype="bf16", seed=0, spare=0, rows=0, max_pages=0, gain=1.0, hold=None):
        rng = np.random.default_rng(seed)
        self.rng, self.lens = rng, np.array(list(lens) + [0] * rows, np.int32)
        B = len(self.lens)
        need = [-(-int(L) // PAGE) for L in (hold or lens)] + [0] * rows
        self.n_pages = sum(need) + spare + 1
        order = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.zeros((B, max(max(need), max_pages, 1)), np.int32)
        self.ref, self.held = np.zeros(self.n_pages, np.int32), np.array(need, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            self.ref[order[at:at + n]] = 1
            at += n
        shape = (self.n_pages, Hkv, PAGE, D)
        self.ks = self.vs = None
        if dtype == "int8":
            self.k, self.v = (torch.from_numpy(rng.integers(-127, 128, shape, dtype=np.int8)) for _ in range(2))
            self.ks, self.vs = 0.0173, 0.0211
        else:
            self.k, self.v = (torch.from_numpy(rng.standard_normal(shape, dtype=np.float32) * np.float32(gain)).bfloat16()
                              for _ in range(2))
            seen = np.zeros((self.n_pages, PAGE), bool)
            for b, L in enumerate(self.lens):
                for j in range(-(-int(L) // PAGE)):
                    seen[self.table[b, j], :min(PAGE, L - j * PAGE)] = True
            hide = torch.from_numpy(~seen)[:, None, :, None]
            self.k.masked_fill_(hide, float("nan"))
            self.v.masked_fill_(hide, float("nan"))

    def gpu(self, sgd):
        sc = lambda x: None if x is None else torch.tensor([x], dtype=torch.float32, device="cuda")  # noqa: E731
        return sgd.PagedKv(self.k.cuda(), self.v.cuda(), ints(self.table), ints(self.lens), ints(self.held),
                           ints(self.ref), sc(self.ks), sc(self.vs))

    def host(self):
        return orc.Pages(self.k.float().numpy() if self.ks is None else self.k.numpy(),
                         self.v.float().numpy() if self.ks is None else self.v.numpy(), self.table, self.lens, self.held,
                         self.ref)

    def query(self, M, G, gain=1.0):
        shape = (len(self.lens), M, self.k.shape[1] * G, self.k.shape[3])
        return torch.from_numpy(self.rng.standard_normal(shape, dtype=np.float32) * np.float32(gain)).bfloat16()


def tree(rng, B, M, back=6, roots=False):
    lo = -1 if roots else 0
    return np.array([[-1] + [int(rng.integers(max(lo, m - back), m)) for m in range(1, M)] for _ in range(B)], np.int32)


def check_attn(sgd, case, q, G, parent=None, n_nodes=None, window=0, sinks=0, cache=None, **kw):
    cache = cache or case.gpu(sgd)
    out, lse, ws = sgd.paged_attn(q.cuda(), G, cache, None if parent is None else ints(parent),
                                  None if n_nodes is None else ints(n_nodes), window, sinks, **kw)
    one = lambda x: 1.0 if x is None else float(np.float32(x))  # noqa: E731
    ref, rlse, mass, zabs = orc.attn(q.float().numpy(), G, case.k.float().numpy(), case.v.float().numpy(), case.table,
                                     case.lens, parent, n_nodes, window, sinks, one(case.ks), one(case.vs))
    compare_attn(out, lse, ref, rlse, mass, zabs)
    assert sgd.workspace_status(ws) == 0
    return out, lse


def compare_attn(out, lse, ref, rlse, mass, zabs):
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isneginf(rlse)
    assert (np.isneginf(lse) == empty).all()
    assert (out[empty] == 0).all()
    tz = 2.0 ** -15.9 * zabs + 2.0 ** -18
    err = np.abs(np.where(empty, 0, lse) - np.where(empty, 0, rlse))
    assert (err <= tz).all(), f"lse off by {err.max():.2e}"
    tol = (2.0 ** -8 + 2 * tz[..., None]) * mass + 2.0 ** -8 * np.abs(ref) + 1e-30
    bad = ~(np.abs(out - ref) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outputs off, worst {np.nanmax(np.abs(out - ref) / tol):.2f} of the bound"


# ---------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "int8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 8, 16])
def test_attn_one_token(sgd, dtype, D, G):
    case = Case((1, 2, 63, 64, 65, 127, 128, 129, 1000, 2053), D=D, dtype=dtype, seed=G + D)
    check_attn(sgd, case, case.query(1, G), G)


@pytest.mark.parametrize("dtype", ["bf16", "int8"])
@pytest.mark.parametrize("D,G,M", [(128, 8, 5), (128, 8, 16), (64, 3, 7), (128, 5, 26), (64, 16, 64), (128, 8, 64),
                                   (128, 1, 64), (64, 7, 19), (128, 16, 17)])
def test_attn_tree(sgd, dtype, D, G, M):
    case = Case((M, M + 1, 64 + M, 300, 1111), D=D, dtype=dtype, seed=M)
    check_attn(sgd, case, case.query(M, G), G, parent=tree(case.rng, 5, M))


@pytest.mark.parametrize("M,G", [(4, 8), (33, 4), (64, 5)])
def test_attn_chain_and_forest(sgd, M, G):
    case = Case((M, 200, 640), seed=M + 1)
    q = case.query(M, G)
    chain, _ = check_attn(sgd, case, q, G)
    same, _ = check_attn(sgd, case, q, G, parent=np.tile(np.arange(-1, M - 1), (3, 1)))
    assert torch.equal(chain, same)
    check_attn(sgd, case, q, G, parent=tree(case.rng, 3, M, back=M, roots=True))
    check_attn(sgd, case, q, G, parent=np.full((3, M), -1))


@pytest.mark.parametrize("dtype", ["bf16", "int8"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 2), (64, 0), (64, 64), (127, 4), (128, 129), (1000, 7),
                                          (5000, 3), (300, 5000)])
@pytest.mark.parametrize("M", [1, 6])
def test_attn_window(sgd, dtype, window, sinks, M):
    case = Case((M, 64, 200, 401, 1500), D=64 if sinks == 7 else 128, dtype=dtype, seed=window)
    check_attn(sgd, case, case.query(M, 4), 4, window=window, sinks=sinks)
    check_attn(sgd, case, case.query(M, 4), 4, parent=tree(case.rng, 5, M), window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["bf16", "int8"])
@pytest.mark.parametrize("M", [3, 40])
def test_attn_windows_and_sinks_of_any_size(sgd, dtype, M):
    """More than any position, up to sizes past 32 bits: all tokens are in the window, or among the first ones."""
    case = Case((300, 70), seed=5, dtype=dtype)
    q = torch.randn(2, M, 8, 128, device="cuda").bfloat16()
    cache = case.gpu(sgd)
    want = sgd.paged_attn(q, 4, cache)
    big = [1000, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 40] + [x + d for n in range(20, 31) for x in (2 ** n, 3 * 2 ** (n - 1)) for d in (-1, 1)]
    for kw in [dict(window=x) for x in big] + [dict(window=1, sinks=x) for x in big] + [dict(window=x, sinks=x) for x in big]:
        got = sgd.paged_attn(q, 4, cache, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), kw


def test_attn_window_over_evicted_tokens(sgd):
    # entries that no query of the row sees may hold anything: NaN in K and V between the first
    # tokens and the window, up to the edge of either
    lens, window, sinks, M = (700, 130, 901), 70, 5, 3
    case = Case(lens, seed=9)
    for b, L in enumerate(lens):
        for t in range(sinks, L - M + 1 - window):
            p = case.table[b, t // PAGE]
            case.k[p, :, t % PAGE] = float("nan")
            case.v[p, :, t % PAGE] = float("inf")
    clean = Case(lens, seed=9)
    q = case.query(M, 8)
    out, lse, ws = sgd.paged_attn(q.cuda(), 8, case.gpu(sgd), window=window, sinks=sinks)
    ref = orc.attn(q.float().numpy(), 8, clean.k.float().numpy(), clean.v.float().numpy(), clean.table, clean.lens, None,
                   None, window, sinks)
    compare_attn(out, lse, *ref)


def test_attn_padded_batch(sgd):
    # rows without tokens, rows without nodes, fewer nodes than M, more nodes than tokens
    M = 9
    case = Case((0, 500, 77, 4, 64, 1), seed=3, max_pages=12)
    n = np.array([9, 0, 5, 9, 1, 2], np.int32)
    n[0] = 0
    check_attn(sgd, case, case.query(M, 8), 8, parent=tree(case.rng, 6, M), n_nodes=n)
    case2 = Case((0, 3, 0), seed=4)
    out, lse = check_attn(sgd, case2, case2.query(4, 2), 2)  # a chain longer than its row
    assert torch.isneginf(lse[0]).all() and torch.isneginf(lse[1, 0]).all() and torch.isfinite(lse[1, 1:]).all()


def test_attn_large_and_small_logits(sgd):
    case = Case((300, 129), seed=12, gain=9.0)
    check_attn(sgd, case, case.query(5, 8, gain=6.0), 8, parent=tree(case.rng, 2, 5))
    case = Case((300, 129), seed=13, gain=1e-20)
    check_attn(sgd, case, case.query(5, 8), 8)


@pytest.mark.parametrize("dtype,M", [("bf16", 4), ("bf16", 40), ("int8", 4)])
def test_attn_nan_query_stays_in_its_row(sgd, dtype, M):
    case = Case((3000, 129), Hkv=1, dtype=dtype, seed=14)
    q = case.query(M, 8)
    clean = sgd.paged_attn(q.cuda(), 8, case.gpu(sgd))
    q[0, 1, 3, 7] = float("nan")
    q[1, 0, 0, :] = float("inf")
    out, lse, _ = sgd.paged_attn(q.cuda(), 8, case.gpu(sgd))
    bad = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    bad[0, 1, 3] = bad[1, 0, 0] = True
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    # another row's reference may move at another tile (the warp's rows decide together): equal but for roundings
    assert torch.isfinite(out[~bad]).all()
    assert (out[~bad].float() - clean[0][~bad].float()).abs().max() <= 2.0 ** -7 * float(clean[0].float().abs().max())
    assert (lse[~bad] - clean[1][~bad]).abs().max() <= 1e-4


def test_attn_running_maximum_grows(sgd):
    # keys whose logits climb along the row, so that the running maximum moves in every tile
    L, D = 2000, 128
    case = Case((L,), Hkv=1, seed=21)
    for t in range(L):
        case.k[case.table[0, t // PAGE], 0, t % PAGE] = float(t) / 40
    q = torch.full((1, 1, 4, D), 0.25).bfloat16()
    q[:, :, 1] = -0.25
    q[:, :, 2] = 0
    check_attn(sgd, case, q, 4)


def test_attn_many_rows_and_long_row(sgd):
    rng = np.random.default_rng(5)
    case = Case([int(x) for x in rng.integers(1, 200, 333)], Hkv=1, seed=6)
    check_attn(sgd, case, case.query(2, 4), 4)
    case = Case((40000, 1, 9000), Hkv=1, seed=7)  # one row split over many CTAs
    check_attn(sgd, case, case.query(3, 4), 4, parent=tree(case.rng, 3, 3))
    check_attn(sgd, case, case.query(40, 8), 8, parent=tree(case.rng, 3, 40))


def dense_attn64(case, q, G, parent=None, window=0, sinks=0):
    """The oracle's formula in float64 torch on the GPU, for sizes that numpy loops are too slow for."""
    B, M, Hq, D = q.shape
    one = lambda x: 1.0 if x is None else float(np.float32(x))  # noqa: E731
    k, v, q = case.k.cuda(), case.v.cuda(), q.cuda().double()
    out, mass = torch.zeros(B, M, Hq, D, dtype=torch.float64), torch.zeros(B, M, Hq, D, dtype=torch.float64)
    lse, zabs = torch.zeros(B, M, Hq, dtype=torch.float64), torch.zeros(B, M, Hq, dtype=torch.float64)
    for b in range(B):
        L = int(case.lens[b])
        see = torch.from_numpy(orc.visible(L, M, M, None if parent is None else parent[b], window, sinks)).cuda()
        pages = torch.from_numpy(case.table[b, :-(-L // PAGE)]).long().cuda()
        for h in range(Hq // G):
            kk = k[pages, h].reshape(-1, D)[:L].double() * one(case.ks)
            vv = v[pages, h].reshape(-1, D)[:L].double() * one(case.vs)
            qq = q[b, :, h * G:h * G + G]
            z = (qq @ kk.T / D ** 0.5).masked_fill(~see[:, None], -float("inf"))
            lse[b, :, h * G:h * G + G] = torch.logsumexp(z, -1)
            p = torch.softmax(z, -1)
            out[b, :, h * G:h * G + G], mass[b, :, h * G:h * G + G] = p @ vv, p @ vv.abs()
            zabs[b, :, h * G:h * G + G] = (qq.abs() @ kk.abs().T / D ** 0.5).masked_fill(~see[:, None], 0).amax(-1)
    return [t.numpy() for t in (out, lse, mass, zabs)]


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("int8", 128), ("int8", 64)])
@pytest.mark.parametrize("M,G,window", [(16, 8, 0), (4, 8, 0), (3, 5, 900), (32, 8, 0), (24, 8, 1500)])
def test_attn_many_tiles(sgd, dtype, D, M, G, window):
    # a CTA walks many tiles and several segments with ragged ends, the memory pipeline full all along;
    # run again and again, since a missing wait would show only now and then
    rng = np.random.default_rng(D + M)
    case = Case([int(x) for x in rng.integers(700, 9000, 20)], Hkv=4, D=D, dtype=dtype, seed=D)
    q, par = case.query(M, G), tree(case.rng, 20, M)
    ref = dense_attn64(case, q, G, par, window, 5)
    cache, qc = case.gpu(sgd), q.cuda()
    first = sgd.paged_attn(qc, G, cache, ints(par), window=window, sinks=5)
    compare_attn(first[0], first[1], *ref)
    for _ in range(20):
        out, lse, ws = sgd.paged_attn(qc, G, cache, ints(par), window=window, sinks=5)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert sgd.workspace_status(ws) == 0


def test_attn_repeats_bit_for_bit(sgd):
    case = Case((3000, 800, 5000, 20), seed=31)
    cache, q = case.gpu(sgd), case.query(8, 8).cuda()
    first = sgd.paged_attn(q, 8, cache)
    for _ in range(5):
        again = sgd.paged_attn(q, 8, cache, workspace=first[2])
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_attn_bad_device_data_is_reported(sgd):
    case = Case((200, 90), seed=41, max_pages=4)
    q = case.query(3, 4).cuda()
    good = sgd.paged_attn(q, 4, case.gpu(sgd))

    def status(**kw):
        c = Case((200, 90), seed=41, max_pages=4)
        for name in ("table", "lens"):
            if name in kw:
                getattr(c, name)[:] = kw[name]
        out, lse, ws = sgd.paged_attn(q, 4, c.gpu(sgd), kw.get("parent"), kw.get("n_nodes"))
        return sgd.workspace_status(ws), out

    st, out = status(table=np.where(np.arange(4) == 1, 10 ** 6, case.table))
    assert st == 0x8
    st, out = status(table=np.array([[-1] * 4, case.table[1]]))
    assert st == 0x8 and torch.equal(out[1], good[0][1])
    st, out = status(lens=np.array([10 ** 6, 90]))
    assert st & 0x4 and torch.equal(out[1], good[0][1])
    st, out = status(lens=np.array([-5, 90]))
    assert st == 0x4 and torch.equal(out[1], good[0][1]) and (out[0] == 0).all()
    assert status(parent=ints([[-1, 0, 7], [-1, 0, 1]]))[0] == 0x8
    assert status(parent=ints([[-1, 1, 1], [-1, 0, 1]]))[0] == 0x8
    assert status(n_nodes=ints([4, 3]))[0] == 0x8
    assert status(n_nodes=ints([-1, 3]))[0] == 0x8
    assert status()[0] == 0


def test_attn_bad_scale_is_reported(sgd):
    case = Case((100,), dtype="int8", seed=1)
    case.vs = float("nan")
    out, _, ws = sgd.paged_attn(case.query(1, 4).cuda(), 4, case.gpu(sgd))
    assert sgd.workspace_status(ws) == 0x10 and (out == 0).all()


def test_attn_streams_and_graph(sgd):
    case = Case((900, 64, 333), seed=51)
    cache, q = case.gpu(sgd), case.query(6, 8).cuda()
    par = ints(tree(case.rng, 3, 6))
    want = sgd.paged_attn(q, 8, cache, par)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [sgd.paged_attn(q, 8, cache, par, stream=s) for s in (s1, s2, s1)]  # workspaces of their own
    torch.cuda.synchronize()
    assert all(torch.equal(g[0], want[0]) and torch.equal(g[1], want[1]) for g in got)
    # captured once, replayed after the lengths, the tree and the query changed in place
    out, lse, ws = (torch.empty_like(t) for t in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sgd.paged_attn(q, 8, cache, par, out=(out, lse), workspace=ws)
    case.lens[:] = (700, 60, 6)
    cache.lens.copy_(ints(case.lens))
    q2 = case.query(6, 8)
    q.copy_(q2)
    par2 = tree(case.rng, 3, 6)
    par.copy_(ints(par2))
    for _ in range(2):
        g.replay()
    ref = orc.attn(q2.float().numpy(), 8, case.k.float().numpy(), case.v.float().numpy(), case.table, case.lens, par2)
    compare_attn(out, lse, *ref)


# ---------------------------------------------------------------------------------------------
# verification
# ---------------------------------------------------------------------------------------------
def _distributions(rng, B, M, V, dtype, near=0.5):
    x = rng.standard_normal((B, M, V)).astype(np.float32) * 2
    y = x + near * rng.standard_normal((B, M, V)).astype(np.float32)
    p, q = (torch.softmax(torch.from_numpy(t), -1) for t in (x, y))
    return (p.bfloat16(), q.bfloat16()) if dtype == "bf16" else (p, q)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("B,M,V", [(3, 1, 7), (40, 6, 5), (60, 12, 33), (9, 64, 1000), (5, 20, 8192), (6, 9, 8193),
                                   (4, 7, 50021), (2, 5, 131072)])
def test_verify(sgd, dtype, drawn, B, M, V):
    rng = np.random.default_rng(V + M)
    p, q = _distributions(rng, B, M, V, dtype)
    parent = tree(rng, B, M)
    src = (q if drawn else p).float().numpy()
    tok = np.zeros((B, M), np.int32)
    for b in range(B):
        for m in range(1, M):
            if drawn:
                c = np.cumsum(src[b, parent[b, m]].astype(np.float64))
                tok[b, m] = min(V - 1, int(np.searchsorted(c, rng.random() * c[-1], side="right")))
            else:  # chosen: among the likeliest after the parent, each child another
                rank = int((parent[b, :m] == parent[b, m]).sum())
                tok[b, m] = np.argsort(-src[b, parent[b, m]], kind="stable")[min(rank, V - 1)]
    ua, us = rng.random((B, M), dtype=np.float32), rng.random(B, dtype=np.float32)
    n = None if M < 6 else rng.integers(0, M + 1, B).astype(np.int32)
    got = sgd.verify_tree(p.cuda(), ints(tok), ints(parent), torch.from_numpy(ua).cuda(), torch.from_numpy(us).cuda(),
                          q=q.cuda() if drawn else None, n_nodes=None if n is None else ints(n))
    assert sgd.workspace_status(got[3]) == 0
    ref = orc.verify(p.float().numpy(), q.float().numpy() if drawn else None, tok, parent, n, ua, us)
    for g, r in zip(got, ref[:3]):
        assert np.array_equal(g.cpu().numpy(), r)


def test_verify_edges(sgd):
    V = 9000
    p = torch.zeros(5, 2, V)
    p[0, :, 17] = 1.0          # certain
    p[1, :, V - 1] = 0.5       # the last token, a total of a half
    p[2] = 0.0                 # nothing to draw from
    p[3, :, 5:7] = 0.5
    p[4, :, 0] = 1e-30
    tok, par = ints([[0, 17], [0, 3], [0, 4], [0, 5], [0, 0]]), ints([[-1, 0]] * 5)
    ua = torch.tensor([[0, 0.999], [0, 0.0], [0, 0.5], [0, 0.5], [0, 0.9]], device="cuda")
    us = torch.tensor([0.99999994, 0.99999994, 0.3, 0.0, 0.0], device="cuda")
    n_path, path, nxt, ws = sgd.verify_tree(p.cuda(), tok, par, ua, us)
    assert n_path.tolist() == [2, 1, 1, 1, 1] and path.tolist() == [[0, 1], [0, -1], [0, -1], [0, -1], [0, -1]]
    assert nxt.tolist() == [17, V - 1, 0, 6, 0] and sgd.workspace_status(ws) == 0x80
    # the draft's distribution equal to the target's: a refusal that only rounding can cause leaves p
    n_path, _, nxt, ws = sgd.verify_tree(p[3:4].cuda(), tok[3:4], par[3:4], torch.tensor([[0, 1.0]], device="cuda"),
                                         us[3:4], q=p[3:4].cuda())
    assert n_path.tolist() == [1] and nxt.tolist() == [5] and sgd.workspace_status(ws) == 0


def test_verify_bad_device_data_is_reported(sgd):
    p = torch.full((2, 3, 50), 0.02).cuda()
    u, us = torch.zeros(2, 3).cuda(), torch.zeros(2).cuda()
    go = lambda tok, par, n=None: sgd.verify_tree(p, ints(tok), ints(par), u, us, n_nodes=None if n is None else ints(n))  # noqa: E731
    good = [[-1, 0, 1]] * 2
    assert sgd.workspace_status(go([[0, 1, 2]] * 2, good)[3]) == 0
    n_path, path, _, ws = go([[0, 50, 2], [0, 1, -1]], good)
    assert n_path.tolist() == [1, 2] and sgd.workspace_status(ws) == 0x8
    n_path, path, _, ws = go([[0, 1, 2]] * 2, [[-1, 1, 0], [-1, -2, 0]])
    assert path.tolist() == [[0, 2, -1], [0, 2, -1]] and sgd.workspace_status(ws) == 0x8
    n_path, path, _, ws = go([[0, 1, 2]] * 2, [[-1, -1, 0], [-1, 0, 5]])  # a second root is no error
    assert path.tolist() == [[0, 2, -1], [0, 1, -1]] and sgd.workspace_status(ws) == 0x8
    n_path, _, nxt, ws = go([[0, 1, 2]] * 2, good, [7, -3])
    assert n_path.tolist() == [3, 0] and nxt.tolist()[1] == -1 and sgd.workspace_status(ws) == 0x8


# ---------------------------------------------------------------------------------------------
# page upkeep
# ---------------------------------------------------------------------------------------------
def same_state(cache, st, what=("k", "v", "page_table", "lens", "held", "ref_count")):
    ref = dict(k=st.k, v=st.v, page_table=st.table, lens=st.lens, held=st.held, ref_count=st.ref)
    for name in what:
        got = getattr(cache, name)
        got = (got.float() if got.dtype == torch.bfloat16 else got).cpu().numpy()
        assert np.array_equal(got, ref[name], equal_nan=name in "kv"), name


@pytest.mark.parametrize("B,spare", [(1, 10), (7, 100), (1500, 3000)])
def test_reserve(sgd, B, spare):
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, 200, B)]
    case = Case(lens, Hkv=1, D=64, seed=B, spare=spare, max_pages=8)
    cache, st = case.gpu(sgd), case.host()
    for _ in range(3):
        add = rng.integers(0, 60, B).astype(np.int32)
        new, ws = sgd.pages_reserve(cache, ints(add))
        want, status = st.reserve(add)
        assert sgd.workspace_status(ws) == status and np.array_equal(new.cpu().numpy(), want)
        same_state(cache, st)
        st.lens = want
        cache = cache.with_lens(new)


def test_reserve_refuses_whole_calls(sgd):
    case = Case((100, 64, 10), seed=2, spare=3, max_pages=4, rows=1)
    for add, code in (([200, 0, 0, 0], 0x4), ([-1, 0, 0, 0], 0x4), ([100, 100, 60, 0], 0x20)):
        cache, st = case.gpu(sgd), case.host()
        new, ws = sgd.pages_reserve(cache, ints(add))
        assert st.reserve(np.array(add))[1] == code
        assert sgd.workspace_status(ws) == code and new.tolist() == case.lens.tolist()
        same_state(cache, st)
    case.ref[case.table[0, 1]] = 2  # the page in which row 0 would grow has another owner
    cache = case.gpu(sgd)
    new, ws = sgd.pages_reserve(cache, ints([1, 0, 0, 0]))
    assert sgd.workspace_status(ws) == 0x40 and new.tolist() == case.lens.tolist()
    new, ws = sgd.pages_reserve(cache, ints([0, 1, 0, 0]))  # the others may
    assert sgd.workspace_status(ws) == 0 and new.tolist() == [100, 65, 10, 0]
    # in place
    new, ws = sgd.pages_reserve(cache, ints([0, 0, 5, 0]), out=cache.lens)
    assert cache.lens.tolist() == [100, 64, 15, 0]


def test_reserve_refuses_shared_pages_behind_the_last_token(sgd):
    """A forked row that was cut back at a page's end would grow inside the pages that it still shares."""
    for cut, add in ((64, 1), (64, 65), (0, 1), (0, 200), (10, 1), (128, 70)):
        case = Case((192,), seed=cut, spare=6, rows=1, max_pages=6)
        cache, st = case.gpu(sgd), case.host()
        sgd.pages_fork(cache, ints([0]), ints([1]))
        assert st.fork(np.array([0]), np.array([1])) == 0
        cache.lens[0] = cut
        st.lens[0] = cut
        want, status = st.reserve(np.array([add, 0]))
        assert status == 0x40
        new, ws = sgd.pages_reserve(cache, ints([add, 0]))
        assert sgd.workspace_status(ws) == 0x40 and new.tolist() == want.tolist()
        same_state(cache, st)
        # given back first, the row grows in pages of its own (unless it was cut inside one)
        sgd.pages_release(cache, cache.lens)
        st.release(st.lens)
        want, status = st.reserve(np.array([add, 0]))
        assert status == (0x40 if cut % PAGE else 0)
        new, ws = sgd.pages_reserve(cache, ints([add, 0]))
        assert sgd.workspace_status(ws) == status and new.tolist() == want.tolist()
        same_state(cache, st)
    case = Case((64, 10), seed=3, spare=2, max_pages=4, hold=(128, 64))
    cache = case.gpu(sgd)
    cache.page_table[0, 1] = case.n_pages
    for add, status in ((0, 0), (1, 0x8)):
        new, ws = sgd.pages_reserve(cache, ints([add, 1]))
        assert sgd.workspace_status(ws) == status and new.tolist() == ([64, 10] if status else [64, 11])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hkv", [1, 3])
def test_append(sgd, D, Hkv):
    rng = np.random.default_rng(D)
    new = [0, 1, 63, 64, 65, 500, 0, 3]
    old = [10, 63, 1, 0, 64, 130, 5, 61]
    case = Case([a + b for a, b in zip(old, new)], Hkv=Hkv, D=D, seed=D + Hkv)
    cache, st = case.gpu(sgd), case.host()
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    k, v = (torch.from_numpy(rng.standard_normal((Hkv, cu[-1], D), dtype=np.float32)).bfloat16() for _ in range(2))
    ws = sgd.pages_append(cache, k.cuda(), v.cuda(), ints(cu))
    st.append(k.float().numpy(), v.float().numpy(), cu)
    assert sgd.workspace_status(ws) == 0
    same_state(cache, st)
    # no tokens at all
    ws = sgd.pages_append(cache, k[:, :0].cuda(), v[:, :0].cuda(), ints([0] * 9))
    assert sgd.workspace_status(ws) == 0
    same_state(cache, st)


def test_append_codes_are_the_quantised_ones(sgd):
    import oracle
    rng = np.random.default_rng(8)
    case = Case((70, 200), Hkv=2, D=128, dtype="int8", seed=8)
    cache, st = case.gpu(sgd), case.host()
    cu = np.array([0, 20, 150], np.int32)
    k, v = (torch.from_numpy(rng.standard_normal((2, 150, 128), dtype=np.float32) * np.float32(1.5)).bfloat16() for _ in range(2))
    ws = sgd.pages_append(cache, k.cuda(), v.cuda(), ints(cu))
    assert sgd.workspace_status(ws) == 0
    codes = [oracle.quantize(x.float().numpy(), np.float32(s)) for x, s in ((k, case.ks), (v, case.vs))]
    st.append(codes[0].reshape(k.shape), codes[1].reshape(v.shape), cu)
    same_state(cache, st)


def test_append_bad_device_data_is_reported(sgd):
    k = torch.zeros(2, 6, 128, dtype=torch.bfloat16, device="cuda")
    for change, code in ((dict(cu=[0, 3, 5]), 0x4), (dict(cu=[1, 3, 6]), 0x4), (dict(lens=[2, 100]), 0x4),
                         (dict(lens=[100, 10 ** 6]), 0x4), (dict(page=-1), 0x8), (dict(page=999), 0x8), ({}, 0)):
        case = Case((100, 70), seed=4)
        if "page" in change:
            case.table[0, 1] = change["page"]
        cache = case.gpu(sgd)
        cache.lens.copy_(ints(change.get("lens", [100, 70])))
        ws = sgd.pages_append(cache, k, k, ints(change.get("cu", [0, 3, 6])))
        assert sgd.workspace_status(ws) == code, change


@pytest.mark.parametrize("dtype", ["bf16", "int8"])
@pytest.mark.parametrize("D,Hkv", [(128, 2), (64, 3)])
def test_fork_and_release(sgd, dtype, D, Hkv):
    case = Case((64, 1, 200, 0, 128, 391), Hkv=Hkv, D=D, dtype=dtype, seed=D, spare=12, rows=9)
    cache, st = case.gpu(sgd), case.host()
    src, dst = np.array([2, 2, 5, 0, 3, 1, 5], np.int32), np.array([8, 6, 14, 7, 9, 13, 10], np.int32)
    for _ in range(2):  # forked, released, forked again: the same pages
        ws = sgd.pages_fork(cache, ints(src), ints(dst))
        assert sgd.workspace_status(ws) == 0 and st.fork(src, dst) == 0
        same_state(cache, st)
        keep = case.lens.copy()
        ws = sgd.pages_release(cache, ints(keep))
        st.release(keep)
        assert sgd.workspace_status(ws) == 0
        same_state(cache, st)
        assert np.array_equal(cache.ref_count.cpu().numpy(), case.ref)
    keep = np.array([0, 0, 65, 5, 127, 2 ** 31 - 1] + [0] * 9, np.int64)
    ws = sgd.pages_release(cache, ints(keep))
    st.release(keep)
    assert sgd.workspace_status(ws) == 0
    same_state(cache, st)


def test_fork_refuses_whole_calls(sgd):
    for src, dst, code in (([0], [1], 0x8), ([0, 0], [3, 3], 0x8), ([3], [4], 0), ([0], [5], 0x8), ([-1], [3], 0x8),
                           ([0, 0, 0], [3, 4, 2], 0x8), ([0, 3], [3, 4], 0x8), ([0, 0], [3, 4], 0x20), ([3], [3], 0x8),
                           ([0], [3], 0)):
        case = Case((100, 64, 30), seed=2, spare=0, rows=2)  # one free page: the pool's extra one
        cache, st = case.gpu(sgd), case.host()
        ws = sgd.pages_fork(cache, ints(src), ints(dst))
        assert sgd.workspace_status(ws) == code, (src, dst)
        if code == 0:
            st.fork(np.array(src), np.array(dst))
        same_state(cache, st)
    case.lens[0] = 129
    ws = sgd.pages_fork(case.gpu(sgd), ints([0]), ints([3]))
    assert sgd.workspace_status(ws) == 0x4


def test_release_bad_device_data_is_reported(sgd):
    case = Case((100, 64), seed=2)
    cache = case.gpu(sgd)
    cache.ref_count[int(case.table[0, 1])] = 0
    cache.page_table[1, 0] = 77
    ws = sgd.pages_release(cache, ints([-4, 0]))
    assert sgd.workspace_status(ws) == 0xc
    assert (cache.ref_count >= 0).all() and cache.held.tolist() == [0, 0]


@pytest.mark.parametrize("dtype", ["bf16", "int8"])
@pytest.mark.parametrize("M,D", [(1, 128), (7, 64), (64, 128), (64, 64)])
def test_accept(sgd, dtype, M, D):
    rng = np.random.default_rng(M)
    B = 6
    case = Case([M, 64 + M, 63 + M, 200, 300, 64], Hkv=3, D=D, dtype=dtype, seed=M)
    n = np.array([M, M, M, max(1, M // 2), M, 0], np.int32)
    n_path, path = np.zeros(B, np.int32), np.full((B, M), -1, np.int32)
    for b in range(B):
        if n[b]:
            chosen = sorted(rng.choice(n[b], size=int(rng.integers(1, n[b] + 1)), replace=False))
            n_path[b] = len(chosen)
            path[b, :len(chosen)] = chosen
    n_path[4] = 0  # nothing accepted at all
    cache, st = case.gpu(sgd), case.host()
    new, ws = sgd.pages_accept(cache, ints(path), ints(n_path), ints(n))
    assert np.array_equal(new.cpu().numpy(), st.accept(path, n_path, n)) and sgd.workspace_status(ws) == 0
    same_state(cache, st)


@pytest.mark.parametrize("dtype", ["bf16", "int8"])
@pytest.mark.parametrize("D", [64, 128])
def test_keep(sgd, dtype, D):
    rng = np.random.default_rng(D)
    lens, kept = [1, 64, 5000, 700, 0, 130], [1, 64, 1300, 699, 0, 1]
    Hkv = 2
    case = Case(lens, Hkv=Hkv, D=D, dtype=dtype, seed=D, max_pages=3)
    cu = np.concatenate([[0], np.cumsum(kept)]).astype(np.int32)
    idx = np.stack([np.concatenate([np.sort(rng.choice(L, K, replace=False)) for L, K in zip(lens, kept) if K])
                    for _ in range(Hkv)]).astype(np.int32)
    cache, st = case.gpu(sgd), case.host()
    new, ws = sgd.pages_keep(cache, ints(idx), ints(cu))
    assert np.array_equal(new.cpu().numpy(), st.keep(idx, cu)) and sgd.workspace_status(ws) == 0
    same_state(cache, st)


def test_compact_bad_device_data_is_reported(sgd):
    case = Case((100, 70, 30), seed=4)
    go = lambda idx, cu, c=None: sgd.pages_keep(c or case.gpu(sgd), ints([idx, idx]), ints(cu))  # noqa: E731
    cu = [0, 2, 4, 5]
    assert sgd.workspace_status(go([3, 9, 0, 69, 29], cu)[1]) == 0
    for idx in ([9, 3, 0, 69, 29], [3, 3, 0, 69, 29], [3, 100, 0, 69, 29], [-1, 4, 0, 69, 29], [0, 1, 2, 3, 30]):
        assert sgd.workspace_status(go(idx, cu)[1]) == 0x8, idx
    assert sgd.workspace_status(go([0] * 5, [0, 2, 1, 5])[1]) & 0x4
    assert sgd.workspace_status(go([0] * 5, [0, 2, 4, 9])[1]) & 0x4
    # a page with another owner is not written, the row stays as it is; the others go ahead
    cache = case.gpu(sgd)
    cache.ref_count[int(case.table[1, 0])] = 2
    st = case.host()
    st.ref[case.table[1, 0]] = 2
    new, ws = go([3, 9, 0, 69, 29], cu, cache)
    assert sgd.workspace_status(ws) == 0x40 and new.tolist() == [2, 70, 1]
    idx = np.array([[3, 9, 29]] * 2)
    for b, part in ((0, idx[:, :2]), (2, idx[:, 2:])):
        for h in range(2):
            st._compact(b, h, 0, part[h])
    same_state(cache, st)
    acc = lambda path, n_path, n: sgd.pages_accept(case.gpu(sgd), ints(path), ints(n_path), ints(n))  # noqa: E731
    ok = [[0, 2, -1]] * 3
    assert sgd.workspace_status(acc(ok, [2, 2, 2], [3, 3, 3])[1]) == 0
    assert sgd.workspace_status(acc([[0, 3, -1], *ok[1:]], [2, 2, 2], [3, 3, 3])[1]) == 0x8
    assert sgd.workspace_status(acc(ok, [4, 2, 2], [3, 3, 3])[1]) & 0x4
    assert sgd.workspace_status(acc(ok, [2, 2, 2], [4, 3, 3])[1]) & 0x4


# ---------------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "int8"])
def test_speculative_steps(sgd, dtype):
    """Steps of a serving loop: room for the nodes, their keys and values, attention, verification, the
    accepted ones kept, unused pages back, a fork, an end; every state against the oracle's."""
    import oracle
    rng = np.random.default_rng(77)
    Hkv, G, D, M, V = 2, 4, 128, 7, 300
    case = Case((100, 64, 250, 1), Hkv=Hkv, D=D, dtype=dtype, seed=78, spare=30, rows=2, max_pages=10)
    if dtype == "bf16":
        case.k.nan_to_num_(0.0)
        case.v.nan_to_num_(0.0)
    cache, st = case.gpu(sgd), case.host()
    B = 6
    for step in range(4):
        n = np.where(st.lens > 0, rng.integers(1, M + 1, B), 0).astype(np.int32)
        parent = tree(rng, B, M)
        new, ws = sgd.pages_reserve(cache, ints(n))
        want, status = st.reserve(n)
        assert status == 0 and sgd.workspace_status(ws) == 0 and np.array_equal(new.cpu().numpy(), want)
        cache, st.lens = cache.with_lens(new), want
        cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        k, v = (torch.from_numpy(rng.standard_normal((Hkv, cu[-1], D), dtype=np.float32)).bfloat16() for _ in range(2))
        sgd.pages_append(cache, k.cuda(), v.cuda(), ints(cu))
        if dtype == "int8":
            put = [oracle.quantize(x.float().numpy(), np.float32(s)).reshape(x.shape) for x, s in ((k, case.ks), (v, case.vs))]
        else:
            put = [x.float().numpy() for x in (k, v)]
        st.append(*put, cu)
        q = torch.from_numpy(rng.standard_normal((B, M, Hkv * G, D), dtype=np.float32)).bfloat16()
        out, lse, ws = sgd.paged_attn(q.cuda(), G, cache, ints(parent), ints(n), window=90, sinks=4)
        assert sgd.workspace_status(ws) == 0
        one = lambda x: 1.0 if x is None else float(np.float32(x))  # noqa: E731
        compare_attn(out, lse, *orc.attn(q.float().numpy(), G, st.k, st.v, st.table, st.lens, parent, n, 90, 4, one(case.ks),
                                         one(case.vs)))
        p, dr = _distributions(rng, B, M, V, "f32")
        tok = rng.integers(0, V, (B, M)).astype(np.int32)
        for b in range(B):
            for m in range(1, M):
                tok[b, m] = int(np.argmax(p[b, parent[b, m]].numpy() * rng.random(V)))
        ua, us = rng.random((B, M), dtype=np.float32) * 0.3, rng.random(B, dtype=np.float32)
        n_path, path, nxt, ws = sgd.verify_tree(p.cuda(), ints(tok), ints(parent), torch.from_numpy(ua).cuda(),
                                                torch.from_numpy(us).cuda(), q=dr.cuda(), n_nodes=ints(n))
        ref = orc.verify(p.numpy(), dr.numpy(), tok, parent, n, ua, us)
        assert all(np.array_equal(a.cpu().numpy(), r) for a, r in zip((n_path, path, nxt), ref))
        new, ws = sgd.pages_accept(cache, path, n_path, ints(n))
        want = st.accept(ref[1], ref[0], n)
        assert sgd.workspace_status(ws) == 0 and np.array_equal(new.cpu().numpy(), want)
        cache, st.lens = cache.with_lens(new), want
        ws = sgd.pages_release(cache, new)
        st.release(want)
        same_state(cache, st)
        if step == 1:
            ws = sgd.pages_fork(cache, ints([2, 0]), ints([4, 5]))
            assert sgd.workspace_status(ws) == 0 and st.fork(np.array([2, 0]), np.array([4, 5])) == 0
            same_state(cache, st)
        if step == 2:
            keep = st.lens.copy()
            keep[2] = 0
            sgd.pages_release(cache, ints(keep))
            cache.lens[2] = 0
            st.release(keep)
            st.lens[2] = 0
            same_state(cache, st)


def test_captured_step_replays(sgd):
    """A whole speculative step in one graph, replayed on changing inputs, against the same calls made one by one."""
    rng = np.random.default_rng(5)
    B, M, Hkv, G, D, V = 3, 6, 2, 8, 64, 9001
    case = Case((70, 640, 1), Hkv=Hkv, D=D, seed=6, spare=20, max_pages=14)
    n = ints([6, 4, 5])
    cu = ints([0, 6, 10, 15])
    shapes = dict(k=(Hkv, 15, D), v=(Hkv, 15, D), q=(B, M, Hkv * G, D))
    x = {a: torch.zeros(sh, dtype=torch.bfloat16, device="cuda") for a, sh in shapes.items()}
    x |= dict(p=torch.zeros(B, M, V, device="cuda"), dr=torch.zeros(B, M, V, device="cuda"), tok=ints(np.zeros((B, M))),
              par=ints(tree(rng, B, M)), ua=torch.zeros(B, M, device="cuda"), us=torch.zeros(B, device="cuda"))

    def step(cache):
        grown, w0 = sgd.pages_reserve(cache, n)
        c = cache.with_lens(grown)
        w1 = sgd.pages_append(c, x["k"], x["v"], cu)
        out, lse, w2 = sgd.paged_attn(x["q"], G, c, x["par"], n, window=300, sinks=3)
        n_path, path, token, w3 = sgd.verify_tree(x["p"], x["tok"], x["par"], x["ua"], x["us"], q=x["dr"], n_nodes=n)
        new, w4 = sgd.pages_accept(c, path, n_path, n)
        w5 = sgd.pages_release(c, new)
        cache.lens.copy_(new)
        return out, lse, n_path, path, token, [w0, w1, w2, w3, w4, w5]

    eager, replayed = case.gpu(sgd), case.gpu(sgd)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):  # the kernels are loaded before the capture
        step(case.gpu(sgd))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(replayed)
    for turn in range(4):
        for a in ("k", "v", "q"):
            x[a].copy_(torch.from_numpy(rng.standard_normal(shapes[a], dtype=np.float32)))
        p, dr = _distributions(rng, B, M, V, "f32")
        par = tree(rng, B, M)
        tok = np.array([[int(np.argmax(dr[b, max(par[b, m], 0)].numpy() * rng.random(V))) for m in range(M)] for b in range(B)])
        for a, t in (("p", p), ("dr", dr), ("tok", ints(tok)), ("par", ints(par)), ("ua", torch.from_numpy(rng.random((B, M)))),
                     ("us", torch.from_numpy(rng.random(B)))):
            x[a].copy_(t)
        want = step(eager)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got[:5], want[:5]):
            assert torch.equal(a, b)
        assert all(sgd.workspace_status(w) == 0 for w in got[5] + want[5])
        for name in ("k", "v", "page_table", "lens", "held", "ref_count"):
            a, b = getattr(eager, name), getattr(replayed, name)
            assert torch.equal(a.nan_to_num(7.0) if name in "kv" else a, b.nan_to_num(7.0) if name in "kv" else b), name


def test_calls_on_two_streams_at_once(sgd):
    # two batches in flight at the same time, each with its own workspace, several times over
    cases = [Case([int(x) for x in np.random.default_rng(s).integers(100, 5000, 12)], Hkv=4, seed=s) for s in (1, 2)]
    qs = [c.query(5, 8).cuda() for c in cases]
    caches = [c.gpu(sgd) for c in cases]
    want = [sgd.paged_attn(q, 8, c) for q, c in zip(qs, caches)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for i in (0, 1):
            got[i].append(sgd.paged_attn(qs[i], 8, caches[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for out, lse, ws in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1]) and sgd.workspace_status(ws) == 0


def test_selected_tokens_kept_in_pages(sgd):
    """oam_select's kept set, made permanent in the pages: the paged attention over what is left is the
    kept-set decode over the packed cache."""
    import workloads
    wl = workloads.Workload("paged", B=3, Hkv=2, G=8, D=128, kv_dtype="bf16", dist="normal", lengths=(700, 64, 1999))
    bt = workloads.generate(wl, 5)
    q, k, v, cu = (t.cuda() for t in (bt.q, bt.k, bt.v, bt.cu_seqlens))
    idx, cu_kept, _ = sgd.oam_select(q, k, v, cu, 8, 1.0, 1e-6, 1, 4, bt.lengths)
    want, want_lse, _ = sgd.decode_attn(q, 8, k, v, cu, idx=idx, cu_kept=cu_kept, kept_total_=idx.shape[1])
    case = Case((0, 0, 0), spare=60, max_pages=40)
    cache = case.gpu(sgd)
    lens, _ = sgd.pages_reserve(cache, (cu[1:] - cu[:-1]).contiguous())
    cache = cache.with_lens(lens)
    sgd.pages_append(cache, k, v, cu)
    new, ws = sgd.pages_keep(cache, idx, cu_kept)
    assert sgd.workspace_status(ws) == 0
    cache = cache.with_lens(new)
    sgd.pages_release(cache, new)
    assert int((cache.ref_count > 0).sum()) == int(((new + 63) // 64).sum())
    out, lse, ws = sgd.paged_attn(q[:, None].contiguous(), 8, cache)
    # both paths round p to bf16 (2^-8 of sum p |v|, itself at most max |v|) and this one its output
    vmax = float(v.float().abs().max())
    assert (out[:, 0].float() - want).abs().max() <= 3 * 2.0 ** -8 * vmax
    assert (lse[:, 0] - want_lse).abs().max() <= 2e-3


# ---------------------------------------------------------------------------------------------
# waits that run out
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,M", [("bf16", 1), ("bf16", 40), ("int8", 4), ("int8", 40)])
def test_attn_waits_are_bounded(sgd, dtype, M):
    # with the producer idle every wait on the pipeline runs out, nothing in flight: the call ends, says so, and the
    # same call made afterwards is right
    import time
    case = Case((300, 2100, 70), dtype=dtype, seed=M)
    q, par = case.query(M, 8), tree(case.rng, 3, M)
    cache = case.gpu(sgd)
    torch.cuda.synchronize()
    sgd.test_pipeline_timeout(4096, True)
    try:
        t = time.perf_counter()
        _, _, ws = sgd.paged_attn(q.cuda(), 8, cache, ints(par))
        assert sgd.workspace_status(ws) & 0x2
        assert time.perf_counter() - t < 20
    finally:
        sgd.test_pipeline_timeout(0, False)
    check_attn(sgd, case, q, 8, parent=par, cache=cache)
