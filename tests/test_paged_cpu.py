"""The paged cache and draft verification without a GPU: the host-side refusals of every entry point and
of the binding, the struct's layout, and pins of the fp64 oracle that the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import paged as orc


@pytest.fixture(scope="module")
def sgd():
    from conftest import build_library
    return build_library()


def _kv(sgd, **kw):
    base = dict(dtype=sgd.SGD_BF16, B=3, Hkv=2, D=128, n_pages=40, max_pages=8, k=0x10000, v=0x20000, k_scale=None,
                v_scale=None, page_table=0x30000, lens=0x31000, held=0x32000, ref_count=0x33000)
    base.update(kw)
    return sgd._PagedKvStruct(**base)


P = ctypes.c_void_p
ALL_OK = (-1, -2, -3, -4, -5, -8)  # the refusals of the host checks: a valid call fails later, for want of a device


def calls(sgd):
    """name -> call(kv, workspace, bytes, **changed pointer arguments)."""
    L, ref = sgd.lib, ctypes.byref

    def attn(kv, ws=0x90000, n=1 << 26, q=0x40000, G=4, M=5, parent=0x41000, n_nodes=0x42000, window=0, sinks=0,
             out=0x43000, lse=0x44000):
        return L.sgd_paged_attn(q, G, M, ref(kv), parent, n_nodes, window, sinks, out, lse, ws, n, None)

    def reserve(kv, ws=0x90000, n=1 << 20, add=0x40000, new=0x41000):
        return L.sgd_pages_reserve(ref(kv), add, new, ws, n, None)

    def append(kv, ws=0x90000, n=1 << 20, k=0x40000, v=0x41000, cu=0x42000, T=9):
        return L.sgd_pages_append(ref(kv), k, v, cu, T, ws, n, None)

    def fork(kv, ws=0x90000, n=1 << 20, src=0x40000, dst=0x41000, count=2):
        return L.sgd_pages_fork(ref(kv), src, dst, count, ws, n, None)

    def release(kv, ws=0x90000, n=1 << 20, keep=0x40000):
        return L.sgd_pages_release(ref(kv), keep, ws, n, None)

    def accept(kv, ws=0x90000, n=1 << 20, path=0x40000, n_path=0x41000, n_nodes=0x42000, M=5, new=0x43000):
        return L.sgd_pages_accept(ref(kv), path, n_path, n_nodes, M, new, ws, n, None)

    def keep(kv, ws=0x90000, n=1 << 20, idx=0x40000, cu=0x41000, total=7, new=0x42000):
        return L.sgd_pages_keep(ref(kv), idx, cu, total, new, ws, n, None)

    return dict(attn=attn, reserve=reserve, append=append, fork=fork, release=release, accept=accept, keep=keep)


NAMES = ("attn", "reserve", "append", "fork", "release", "accept", "keep")


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("kw,code", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(page_table=None), -1), (dict(lens=None), -1),
    (dict(B=0), -2), (dict(Hkv=0), -2), (dict(D=96), -2), (dict(n_pages=0), -2), (dict(max_pages=0), -2),
    (dict(n_pages=1 << 24, Hkv=2), -2), (dict(max_pages=1 << 24), -2), (dict(B=1 << 23, Hkv=2), -2),
    (dict(dtype=0), -3), (dict(dtype=7), -3), (dict(dtype=2), -1),
    (dict(k=0x10008), -4), (dict(v=0x20004), -4), (dict(lens=0x31002), -4),
    (dict(dtype=2, k_scale=0x50002, v_scale=0x50004), -4),
])
def test_every_call_refuses_a_bad_cache(sgd, name, kw, code):
    assert calls(sgd)[name](_kv(sgd, **kw)) == code


@pytest.mark.parametrize("name", NAMES)
def test_every_call_takes_a_good_cache_and_checks_its_workspace(sgd, name):
    call = calls(sgd)[name]
    assert call(_kv(sgd)) not in ALL_OK
    assert call(_kv(sgd, dtype=2, k_scale=0x50000, v_scale=0x50010)) not in ALL_OK
    assert call(_kv(sgd), ws=None) == -1
    assert call(_kv(sgd), ws=0x90004) == -4
    assert call(_kv(sgd), n=128) == -5


def test_argument_refusals(sgd):
    c, kv = calls(sgd), _kv(sgd)
    attn = c["attn"]
    assert attn(kv, q=None) == -1 and attn(kv, out=None) == -1 and attn(kv, lse=None) == -1
    assert attn(kv, G=0) == -2 and attn(kv, G=17) == -2 and attn(kv, M=0) == -2 and attn(kv, M=65) == -2
    assert attn(kv, window=-1) == -8 and attn(kv, sinks=-1) == -8
    assert attn(kv, q=0x40008) == -4 and attn(kv, out=0x43008) == -4 and attn(kv, parent=0x41002) == -4
    assert attn(kv, parent=None, n_nodes=None) not in ALL_OK
    assert c["reserve"](kv, add=None) == -1 and c["reserve"](kv, new=None) == -1
    assert c["append"](kv, cu=None) == -1 and c["append"](kv, k=None) == -1 and c["append"](kv, T=-1) == -2
    assert c["append"](kv, T=1 << 30) == -2 and c["append"](kv, k=0x40008) == -4
    assert c["fork"](kv, count=0) == -2 and c["fork"](kv, count=3) == -2 and c["fork"](kv, src=None) == -1
    assert c["release"](kv, keep=None) == -1
    assert c["accept"](kv, M=65) == -2 and c["accept"](kv, M=0) == -2 and c["accept"](kv, path=None) == -1
    assert c["accept"](kv, new=0x31000) == -8  # new_lens must not be lens
    assert c["keep"](kv, total=0) == -2 and c["keep"](kv, idx=None) == -1 and c["keep"](kv, new=0x31000) == -8
    for name in ("reserve", "fork", "release"):
        assert c[name](_kv(sgd, held=None)) == -1 and c[name](_kv(sgd, ref_count=None)) == -1
    for name in ("accept", "keep"):
        assert c[name](_kv(sgd, held=None)) not in ALL_OK and c[name](_kv(sgd, ref_count=None)) == -1
    for name in ("attn", "append"):
        assert c[name](_kv(sgd, held=None, ref_count=None)) not in ALL_OK


def test_verify_refusals(sgd):
    def v(p=0x1000, dt=0, q=0x2000, B=2, M=3, V=10, tok=0x3000, par=0x4000, nn=0x5000, ua=0x6000, us=0x7000, n=0x8000,
          path=0x9000, nxt=0xa000, ws=0xb000, nb=256):
        return sgd.lib.sgd_verify_tree(p, dt, q, B, M, V, tok, par, nn, ua, us, n, path, nxt, ws, nb, None)

    assert v() not in ALL_OK and v(q=None, nn=None) not in ALL_OK and v(dt=1) not in ALL_OK
    for name in ("p", "tok", "par", "ua", "us", "n", "path", "nxt", "ws"):
        assert v(**{name: None}) == -1
    assert v(B=0) == -2 and v(M=0) == -2 and v(M=65) == -2 and v(V=0) == -2 and v(V=1 << 31) == -2
    assert v(dt=2) == -3 and v(p=0x1008) == -4 and v(tok=0x3002) == -4 and v(nb=255) == -5


def test_workspace_size(sgd):
    size = lambda kv, G=1, M=1: sgd.lib.sgd_paged_workspace_size(ctypes.byref(kv), G, M)  # noqa: E731
    kv = _kv(sgd)
    assert size(kv) >= 256 + 4 * (40 + 3 * 3)
    assert size(kv, 17, 1) == 0 and size(kv, 1, 65) == 0 and size(kv, 0, 1) == 0 and size(_kv(sgd, D=32)) == 0
    assert size(kv, 16, 64) >= size(kv, 1, 1)


def test_binding_refuses_wrong_tensors(sgd):
    i32 = torch.int32
    k = torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(3, 2, dtype=i32), torch.zeros(3, dtype=i32)
    ok = sgd.PagedKv(k, k.clone(), table, lens)
    assert (ok.B, ok.Hkv, ok.D) == (3, 2, 64)
    for bad in (
        lambda: sgd.PagedKv(k[0], k[0], table, lens),
        lambda: sgd.PagedKv(k.float(), k.float(), table, lens),
        lambda: sgd.PagedKv(k, k[:3], table, lens),
        lambda: sgd.PagedKv(k.transpose(0, 1), k.transpose(0, 1), table, lens),
        lambda: sgd.PagedKv(k, k, table.long(), lens),
        lambda: sgd.PagedKv(k, k, table, lens[:2]),
        lambda: sgd.PagedKv(k, k, table, lens, held=lens[:2]),
        lambda: sgd.PagedKv(k, k, table, lens, ref_count=lens),
        lambda: sgd.PagedKv(k.to(torch.int8), k.to(torch.int8), table, lens),
        lambda: sgd.PagedKv(k, k, table, lens, k_scale=torch.ones(1), v_scale=torch.ones(1)),
        lambda: sgd.PagedKv(k.to(torch.int8), k.to(torch.int8), table, lens, k_scale=torch.ones(1)),
        lambda: sgd.paged_attn(torch.zeros(3, 1, 8, 64), 4, ok),
        lambda: sgd.paged_attn(torch.zeros(3, 1, 7, 64, dtype=torch.bfloat16), 4, ok),
        lambda: sgd.paged_attn(torch.zeros(3, 2, 8, 64, dtype=torch.bfloat16), 4, ok, parent=table[:, :1]),
        lambda: sgd.verify_tree(torch.zeros(3, 2, 9, dtype=torch.float64), table, table, table, lens),
        lambda: sgd.pages_append(ok, k[0], k[0], lens),
        lambda: sgd.pages_accept(ok, table, lens, lens.long()),
        lambda: sgd.pages_keep(ok, table, lens),
        lambda: sgd.pages_fork(ok, lens, lens[:1]),
    ):
        with pytest.raises(ValueError):
            bad()


# ---------------------------------------------------------------------------------------------
# pins of the oracle
# ---------------------------------------------------------------------------------------------
def test_oracle_attention_is_masked_sdpa():
    rng = np.random.default_rng(3)
    B, M, Hkv, G, D = 2, 5, 2, 3, 64
    lens, parent = np.array([70, 130]), [[-1, 0, 0, 2, 1], [-1, 0, 1, -1, 3]]
    table = np.array([[4, 1, 0], [2, 5, 3]])
    k, v = rng.standard_normal((2, 6, Hkv, 64, D))
    q = rng.standard_normal((B, M, Hkv * G, D))
    for window, sinks in ((0, 0), (9, 2), (1, 0), (200, 3)):
        out, lse, _, _ = orc.attn(q, G, k, v, table, lens, parent, None, window, sinks)
        for b in range(B):
            L = int(lens[b])
            kk = np.concatenate([k[p] for p in table[b]], 1)[:, :L]
            vv = np.concatenate([v[p] for p in table[b]], 1)[:, :L]
            # the mask written out from paths to the root, not from the oracle's walk
            paths = [[0], [0, 1], [0, 2], [0, 2, 3], [0, 1, 4]] if b == 0 else [[0], [0, 1], [0, 1, 2], [3], [3, 4]]
            see = torch.zeros(M, L, dtype=torch.bool)
            for m, path in enumerate(paths):
                seen = list(range(L - M)) + [L - M + a for a in path]
                where = list(range(L - M)) + list(range(L - M, L - M + len(path)))
                for t, pos in zip(seen, where):
                    if window == 0 or where[-1] - pos < window or pos < sinks:
                        see[m, t] = True
            qq = torch.from_numpy(q[b]).transpose(0, 1)
            rep = lambda x: torch.from_numpy(x).repeat_interleave(G, 0)  # noqa: E731
            ref = torch.nn.functional.scaled_dot_product_attention(qq, rep(kk), rep(vv), attn_mask=see)
            assert np.allclose(out[b], ref.transpose(0, 1).numpy(), atol=1e-12)
            z = (qq @ rep(kk).transpose(1, 2) / math.sqrt(D)).masked_fill(~see, -math.inf)
            assert np.allclose(lse[b], torch.logsumexp(z, -1).T.numpy(), atol=1e-12)


@pytest.mark.parametrize("children,n", [(1, 40), (2, 10)])
def test_oracle_verification_keeps_the_targets_distribution(children, n):
    # independently drawn children of the root over four tokens: whatever the draft's distribution,
    # the token after the root is distributed as the target says.  All random numbers on a grid: the
    # drafts exactly by their probabilities, the uniforms by the midpoints of n steps.
    p, q = np.array([0.4, 0.3, 0.2, 0.1]), np.array([0.1, 0.2, 0.3, 0.4])
    got = np.zeros(4)
    grid = (np.arange(n) + 0.5) / n
    for draft in np.ndindex(*(4,) * children):
        u = [a.reshape(-1) for a in np.meshgrid(*(grid,) * (children + 1), indexing="ij")]
        B, M = len(u[0]), children + 1
        wide = lambda x, shape: np.broadcast_to(np.array(x), shape)  # noqa: E731
        tok = wide([0, *draft], (B, M))
        n_path, path, nxt, status = orc.verify(wide(p, (B, M, 4)), wide(q, (B, M, 4)), tok, wide([-1] + [0] * children, (B, M)),
                                               None, np.stack([np.zeros(B), *u[:-1]], 1), u[-1])
        assert status == 0
        first = np.where(n_path > 1, np.take_along_axis(tok, np.maximum(path[:, 1:2], 0), 1)[:, 0], nxt)
        got += np.prod(q[list(draft)]) * np.bincount(first, minlength=4) / B
    # a midpoint grid is off by at most half a step for each of the uniforms
    assert np.abs(got - p).max() <= (children + 1) * 0.5 / n


def test_oracle_verification_hand_cases():
    p = np.array([[[0.5, 0.5, 0.0], [0.0, 0.25, 0.75], [1.0, 0.0, 0.0]]])
    par, tok = [[-1, 0, 1]], [[9, 1, 2]]
    verify = lambda *a: orc.verify(*a[:5], np.array(a[5]), np.array(a[6]))  # noqa: E731
    # chosen drafts: 0.4 < 0.5 accepts node 1, 0.74 < 0.75 node 2, then the next token is certain
    r = verify(p, None, tok, par, None, [[0, 0.4, 0.74]], [0.99])
    assert r[0].tolist() == [3] and r[1].tolist() == [[0, 1, 2]] and r[2].tolist() == [0] and r[3] == 0
    # node 1 refused: its token falls out, token 0 is left whatever the number
    r = verify(p, None, tok, par, None, [[0, 0.5, 0.0]], [0.7])
    assert r[0].tolist() == [1] and r[1].tolist() == [[0, -1, -1]] and r[2].tolist() == [0]
    # drawn draft: refused where u q >= p; the residual max(p - q, 0) = (0.3, 0, 0) leaves token 0
    q = np.array([[[0.2, 0.8, 0.0]] * 3])
    r = verify(p, q, tok, par, None, [[0, 0.625, 0.0]], [0.999])
    assert r[0].tolist() == [1] and r[2].tolist() == [0]
    # no nodes; nothing positive
    r = verify(np.zeros((2, 1, 3)), None, [[0], [0]], [[-1], [-1]], [0, 1], [[0], [0]], [0.5, 0.5])
    assert r[0].tolist() == [0, 1] and r[2].tolist() == [-1, 0] and r[3] == orc.BAD_PROBS


def test_oracle_pages_by_hand():
    k = np.arange(6 * 1 * 64 * 1, dtype=float).reshape(6, 1, 64, 1)
    table = np.array([[5, 2, 0], [0, 0, 0], [0, 0, 0]], np.int32)
    st = orc.Pages(k, -k, table, np.array([70, 0, 0]), np.array([2, 0, 0]), np.array([0, 0, 1, 0, 0, 1]))
    assert st.fork(np.array([0, 0]), np.array([1, 2])) == 0
    assert st.ref.tolist() == [1, 1, 1, 0, 0, 3] and st.table[1, :2].tolist() == [5, 0] and st.table[2, :2].tolist() == [5, 1]
    assert (st.k[0, 0, :6] == k[2, 0, :6]).all() and (st.k[0, 0, 6:] == k[0, 0, 6:]).all()
    new, status = st.reserve(np.array([58, 60, 0]))
    assert status == 0 and new.tolist() == [128, 130, 70] and st.table[1, 2] == 3 and st.held.tolist() == [2, 3, 2]
    assert st.reserve(np.array([1000, 0, 0]))[1] == orc.SIZE_MISMATCH
    st.release(np.array([70, 0, 64]))
    assert st.ref.tolist() == [0, 0, 1, 0, 0, 2] and st.held.tolist() == [2, 0, 1]
    st.lens = np.array([70, 0, 64])
    assert st.keep(np.array([[1, 65, 3]]), np.array([0, 2, 2, 3])).tolist() == [2, 0, 1]
    assert st.k[5, 0, :2, 0].tolist() == [k[5, 0, 3, 0], k[2, 0, 1, 0]]  # row 2 shares page 5: 3 -> 0, after row 0's move
