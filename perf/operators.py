"""Measured cases of the paged-cache operators: attention of a step's query tokens (a tree or a chain
of drafted tokens, or one token) over a paged cache with an optional sliding window and visible first
tokens, verification of drafted tokens, and the upkeep of the pages (append, fork, release, keep,
accept).

``run`` with ``own`` false computes each operator from its definition with elementary torch
operations; with ``own`` true it makes the library's calls.  A cache is a pool of 64-token pages
[n_pages, Hkv, 64, D] and a page table [B, max_pages]; sequence b's token t is slot t % 64 of page
table[b, t // 64].
"""
import math
import random

import torch

own = False

PAGE = 64
_T = {"bf16": torch.bfloat16, "int8": torch.int8, "f32": torch.float32}


# ------------------------------------------------------------------------------------------
# the cases
# ------------------------------------------------------------------------------------------
def listed():
    attn = dict(op="attn", Hkv=8, G=8, D=128, dtype="bf16", tree=True, ragged=False, window=0, sinks=0)
    return [
        # one user, a short conversation, seven drafted tokens beside the last one: launch latency counts
        dict(attn, name="tree_1x700_m8", B=1, M=8, lo=700, hi=700),
        # an ordinary speculative serving step: eight users, 16-node trees (some smaller), bf16 cache
        dict(attn, name="tree_8x32k_m16", B=8, M=16, lo=16384, hi=32768, ragged=True),
        # wide trees, 512 query rows to a KV head: the matrix products bound it, not the cache
        dict(attn, name="tree_4x32k_m64", B=4, M=64, lo=30001, hi=32768),
        # the long INT8 cache with three drafted tokens a user
        dict(attn, name="tree_int8_8x128k_m4", B=8, M=4, lo=65536, hi=131072, dtype="int8"),
        # single-token decoding with a sliding window and four first tokens, many users of mixed lengths
        dict(attn, name="window_64x1tok_4096", B=64, M=1, lo=512, hi=32768, tree=False, window=4096, sinks=4),
        # a drafted chain under a window, odd head group, small heads, INT8 cache
        dict(attn, name="window_int8_d64_m5", B=16, Hkv=4, G=3, D=64, M=5, lo=300, hi=20000, dtype="int8", tree=False,
             window=1000, sinks=7),
        # verification for one user, an odd vocabulary
        dict(op="verify", name="verify_1_m8", B=1, M=8, V=32001, draft=True, dtype="f32"),
        # verification of a batch of wide trees over a large vocabulary
        dict(op="verify", name="verify_64_m24", B=64, M=24, V=128000, draft=True, dtype="f32"),
        # prompts written into their pages behind a cached prefix
        dict(op="append", name="append_8x4k", B=8, Hkv=8, D=128, lo=1000, hi=3000, new_lo=1001, new_hi=8192),
        # beams of 64 requests: last step's seven branches of each released, seven new ones forked
        dict(op="fork", name="fork_64x7", n_src=64, forks=7, Hkv=8, D=128, lo=1000, hi=8000),
        # a step's accepted drafted tokens moved to the front of the tail: latency counts
        dict(op="accept", name="accept_8_m16", B=8, M=16, Hkv=8, D=128, lo=1500, hi=4000),
        # long prompts cut to an eighth of their tokens after token selection
        dict(op="keep", name="keep_8x32k", B=8, Hkv=8, D=128, lo=16384, hi=32768, num=1, den=8),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "verify", "append", "fork", "accept", "keep"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    if op == "attn":
        window = rng.choice([0, 0, _logint(rng, 16, 8192)])
        B = _logint(rng, 1, 64)
        # at most about 1.2 M cached tokens x heads x (D / 128), and 4e8 (row, token) pairs
        hi = max(16, min(65536, int(1.2e6 * 128 / (B * Hkv * D))))
        hi = _logint(rng, 16, hi)
        lo = max(1, _logint(rng, max(1, hi // 16), hi))
        G = rng.randint(1, 16)
        M = max(1, min(_logint(rng, 1, 64), int(4e8 / (B * Hkv * G * hi))))
        return dict(op="attn", B=B, Hkv=Hkv, G=G, D=D, M=M, lo=max(lo, M), hi=max(hi, M), dtype=rng.choice(["bf16", "int8"]),
                    tree=rng.random() < 0.6, ragged=rng.random() < 0.5, window=window,
                    sinks=rng.choice([0, 4, _logint(rng, 1, 200)]) if window else 0)
    if op == "verify":
        B, V = _logint(rng, 1, 64), _logint(rng, 50, 130000)
        M = max(1, min(_logint(rng, 1, 64), int(1.9e8 / (B * V))))
        return dict(op="verify", B=B, M=M, V=V, draft=rng.random() < 0.7, dtype=rng.choice(["f32", "bf16"]))
    if op == "append":
        lo, new = _logint(rng, 1, 3000), _logint(rng, 2, 8000)
        return dict(op="append", B=_logint(rng, 1, 8), Hkv=Hkv, D=D, lo=lo, hi=lo + _logint(rng, 1, 3000),
                    new_lo=_logint(rng, 1, new), new_hi=new)
    if op == "fork":
        lo = _logint(rng, 1, 4000)
        return dict(op="fork", n_src=_logint(rng, 1, 64), forks=rng.randint(1, 7), Hkv=Hkv, D=D, lo=lo,
                    hi=lo + _logint(rng, 1, 4000))
    if op == "accept":
        M = rng.randint(2, 64)
        return dict(op="accept", B=_logint(rng, 1, 64), M=M, Hkv=Hkv, D=D, lo=M + _logint(rng, 1, 500),
                    hi=M + 500 + _logint(rng, 1, 3000))
    hi = _logint(rng, 20, 30000)
    return dict(op="keep", B=_logint(rng, 1, 8), Hkv=Hkv, D=D, lo=_logint(rng, 1, hi), hi=hi, num=1, den=rng.randint(2, 16))


# ------------------------------------------------------------------------------------------
# sizes that follow from a case alone
# ------------------------------------------------------------------------------------------
def _spread(n, lo, hi):
    """n whole numbers spread over the logarithm of [lo, hi], both ends among them."""
    return [int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) for i in range(n)]


def _nodes(case):
    """Real nodes of each sequence: M, or fewer for every third one of a ragged batch."""
    M = case["M"]
    return [max(1, M - M // 3) if case.get("ragged") and b % 3 == 2 else M for b in range(case["B"])]


def _kept(L, case):
    return max(1, min(L, -(-L * case["num"] // case["den"])))


def work(case):
    op = case["op"]
    if op == "attn":
        es = 1 if case["dtype"] == "int8" else 2
        lens, n = _spread(case["B"], case["lo"], case["hi"]), _nodes(case)
        per = lens
        if case["window"]:
            per = [min(L, case["sinks"] + case["window"] - 1 + m) for L, m in zip(lens, n)]
        tokens = sum(per)
        rows = case["B"] * case["M"] * case["Hkv"] * case["G"]
        pairs = sum(t * m for t, m in zip(per, n)) * case["Hkv"] * case["G"]
        return {"bytes": 2 * tokens * case["Hkv"] * case["D"] * es + rows * (4 * case["D"] + 4), "flops": 4 * pairs * case["D"]}
    if op == "verify":
        # one row of each distribution to sample from, and the tested tokens' probabilities
        es = 4 if case["dtype"] == "f32" else 2
        return {"bytes": case["B"] * (case["V"] * es * (2 if case["draft"] else 1) + case["M"] * 20), "flops": case["B"] * case["V"] * 3}
    row = 2 * case["Hkv"] * case["D"] * 2  # K and V of one token
    if op == "append":
        return {"bytes": 2 * row * sum(_spread(case["B"], case["new_lo"], case["new_hi"])), "flops": 0}
    if op == "fork":
        lens = _spread(case["n_src"], case["lo"], case["hi"])
        return {"bytes": case["forks"] * sum(2 * row * (L % PAGE) + 12 * (L // PAGE) for L in lens), "flops": 0}
    if op == "accept":
        return {"bytes": case["B"] * (case["M"] * 4 + 2 * row * (case["M"] // 4)), "flops": 0}
    kept = sum(_kept(L, case) for L in _spread(case["B"], case["lo"], case["hi"]))
    return {"bytes": kept * (2 * row + 4 * case["Hkv"]), "flops": 0}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tree(rng, M):
    """A parent for each node (-1 for the root), parents before their children."""
    return [-1] + [rng.randint(max(0, m - 6), m - 1) for m in range(1, M)]


def _cache(case, lens, rng, gen, spare=0, rows=None, cols=0):
    """A pool with its pages handed out in random order to rows of `lens` tokens."""
    B = rows or len(lens)
    need = [-(-L // PAGE) for L in lens]
    n_pages = sum(lens) // PAGE + len(lens) + spare + 3  # as many whatever the order of the lengths
    order = list(range(n_pages))
    rng.shuffle(order)
    table = torch.zeros((B, max(need + [cols])), dtype=torch.int32)
    ref = torch.zeros(n_pages, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        pages = torch.tensor(order[at:at + n], dtype=torch.int32)
        table[b, :n] = pages
        ref[pages.long()] = 1
        at += n
    shape = (n_pages, case["Hkv"], PAGE, case["D"])
    st = {}
    for name in ("k", "v"):
        if case.get("dtype") == "int8":
            st[name] = torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda", generator=gen)
        else:
            st[name] = torch.randn(shape, dtype=torch.bfloat16, device="cuda", generator=gen)
    st["k_scale"] = st["v_scale"] = None
    if case.get("dtype") == "int8":
        st["k_scale"], st["v_scale"] = (torch.full((1,), s, device="cuda") for s in (0.02, 0.015))
    st["table"], st["ref"] = table.cuda(), ref.cuda()
    st["lens"] = _ints(list(lens) + [0] * (B - len(lens)))
    st["held"] = _ints(need + [0] * (B - len(lens)))
    return st


def prepare(case, seed):
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op == "verify":
        B, M, V = case["B"], case["M"], case["V"]
        dt = _T[case["dtype"]]
        parent = [_tree(rng, M) for _ in range(B)]
        st["parent"] = _ints(parent)
        logits = torch.randn((B, M, V), device="cuda", generator=gen).mul_(2.5)
        st["p"] = torch.softmax(logits, -1).to(dt)
        logits.add_(torch.randn((B, M, V), device="cuda", generator=gen), alpha=0.6)
        draft = torch.softmax(logits, -1).to(dt)
        del logits
        # every node's token is drawn from the draft's distribution after its parent
        src = (torch.arange(B, device="cuda")[:, None] * M + st["parent"].clamp(min=0)).reshape(-1)
        u = torch.rand(B * M, device="cuda", generator=gen)
        rows = draft.reshape(B * M, V)
        st["tokens"] = torch.cat([_sample_rows(rows[src[i:i + 64]], u[i:i + 64]) for i in range(0, B * M, 64)]
                                 ).reshape(B, M).to(torch.int32)
        st["q"] = draft if case["draft"] else None
        st["u_accept"] = torch.rand((B, M), device="cuda", generator=gen)
        st["u_sample"] = torch.rand(B, device="cuda", generator=gen)
        if own:  # the outputs and the workspace that a serving loop keeps from step to step
            import sparse_gqa_decode_b200 as sgd
            out = sgd.verify_tree(st["p"], st["tokens"], st["parent"], st["u_accept"], st["u_sample"], q=st["q"])
            st["out"], st["ws"] = tuple(torch.zeros_like(t) for t in out[:3]), out[3]
        return st
    if op == "fork":
        n_src, forks = case["n_src"], case["forks"]
        lens = _spread(n_src, case["lo"], case["hi"])
        rng.shuffle(lens)
        st |= _cache(case, lens, rng, gen, spare=n_src * forks, rows=n_src * (1 + forks))
        st["src"] = _ints([i % n_src for i in range(n_src * forks)])
        st["dst"] = _ints([n_src + i for i in range(n_src * forks)])
        st["stay"] = _ints(lens + [0] * (n_src * forks))  # what each row keeps before the new forks
    else:
        lens = _spread(case["B"], case["lo"], case["hi"])
        rng.shuffle(lens)
        if op == "append":
            new = _spread(case["B"], case["new_lo"], case["new_hi"])
            rng.shuffle(new)
            st |= _cache(case, [a + b for a, b in zip(lens, new)], rng, gen, cols=-(-(case["hi"] + case["new_hi"]) // PAGE))
            cu = [0]
            for x in new:
                cu.append(cu[-1] + x)
            st["cu"] = _ints(cu)
            for name in ("k_new", "v_new"):
                st[name] = torch.randn((case["Hkv"], cu[-1], case["D"]), dtype=torch.bfloat16, device="cuda", generator=gen)
        else:
            st |= _cache(case, lens, rng, gen)
        if op == "attn":
            B, M = case["B"], case["M"]
            st["q"] = torch.randn((B, M, case["Hkv"] * case["G"], case["D"]), dtype=torch.bfloat16, device="cuda", generator=gen)
            n = _nodes(case)
            st["n_nodes"] = _ints(n) if case["ragged"] else None
            st["parent"] = _ints([_tree(rng, M) for _ in range(B)]) if case["tree"] else None
        if op == "accept":
            M, B = case["M"], case["B"]
            path, n_path = torch.full((B, M), -1, dtype=torch.int32), []
            for b in range(B):  # a path from the root towards a random leaf
                nodes = sorted(rng.sample(range(1, M), min(M - 1, rng.randint(0, max(1, M // 3)))))
                path[b, :1 + len(nodes)] = torch.tensor([0] + nodes, dtype=torch.int32)
                n_path.append(1 + len(nodes))
            st["path"], st["n_path"], st["n_nodes"] = path.cuda(), _ints(n_path), _ints([M] * B)
        if op == "keep":
            kept = [_kept(L, case) for L in st["lens"].tolist()]
            rows = [torch.cat([torch.rand(L, device="cuda", generator=gen).topk(K).indices.sort().values
                               for L, K in zip(st["lens"].tolist(), kept)]) for _ in range(case["Hkv"])]
            st["idx"] = torch.stack(rows).to(torch.int32)
            cu = [0]
            for x in kept:
                cu.append(cu[-1] + x)
            st["cu_kept"] = _ints(cu)
    if own:  # the handle, the outputs and the workspace that a serving loop keeps from step to step
        import sparse_gqa_decode_b200 as sgd
        st["cache"] = sgd.PagedKv(st["k"], st["v"], st["table"], st["lens"], held=st["held"], ref_count=st["ref"],
                                  k_scale=st["k_scale"], v_scale=st["v_scale"])
        M = case["M"] if op == "attn" else 1
        st["ws"] = torch.empty(sgd.paged_workspace_size(st["cache"], case.get("G", 1), M), dtype=torch.uint8, device="cuda")
        st["new_lens"] = torch.zeros_like(st["lens"])
        if op == "attn":
            st["out"] = (torch.empty_like(st["q"]), torch.empty(st["q"].shape[:3], device="cuda"))
    return st


def _sample_rows(p, u):
    """The first token of each row whose running sum passes u of the total."""
    c = torch.cumsum(p.double(), -1)
    return (c <= u.double()[:, None] * c[:, -1:]).sum(-1).clamp(max=p.shape[-1] - 1)


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    if own:
        return _own(op, st)
    with torch.no_grad():
        return {"attn": _attn, "verify": _verify, "append": _append, "fork": _fork, "accept": _accept, "keep": _keep}[op](st)


def _own(op, st):
    import sparse_gqa_decode_b200 as sgd
    case = st["case"]
    if op == "attn":
        out, lse, _ = sgd.paged_attn(st["q"], case["G"], st["cache"], parent=st["parent"], n_nodes=st["n_nodes"],
                                     window=case["window"], sinks=case["sinks"], out=st["out"], workspace=st["ws"])
        return out, lse
    if op == "verify":
        return sgd.verify_tree(st["p"], st["tokens"], st["parent"], st["u_accept"], st["u_sample"], q=st["q"],
                               out=st["out"], workspace=st["ws"])[:3]
    if op == "append":
        sgd.pages_append(st["cache"], st["k_new"], st["v_new"], st["cu"], workspace=st["ws"])
        return st["k"], st["v"]
    if op == "fork":
        sgd.pages_release(st["cache"], st["stay"], workspace=st["ws"])
        sgd.pages_fork(st["cache"], st["src"], st["dst"], workspace=st["ws"])
        return st["k"], st["v"], st["table"], st["lens"], st["held"], st["ref"]
    if op == "accept":
        new, _ = sgd.pages_accept(st["cache"], st["path"], st["n_path"], st["n_nodes"], out=st["new_lens"], workspace=st["ws"])
        return st["k"], st["v"], new
    new, _ = sgd.pages_keep(st["cache"], st["idx"], st["cu_kept"], out=st["new_lens"], workspace=st["ws"])
    return st["k"], st["v"], new


def _ancestors(parent, B, M):
    """[B, M, M]: node j is node m or an ancestor of it (a chain where parent is None)."""
    if parent is None:
        return torch.ones((M, M), dtype=torch.bool, device="cuda").tril().expand(B, M, M)
    j = torch.arange(M, device="cuda")
    a = ((parent[:, :, None] == j) | (j[:, None] == j)).float()
    for _ in range(6):  # 2^6 steps up reach the root of any 64-node tree
        a = (torch.bmm(a, a) > 0).float()
    return a > 0


def _attn(st):
    case, q, table, lens = st["case"], st["q"], st["table"], st["lens"].long()
    B, M, Hkv, G, D = case["B"], case["M"], case["Hkv"], case["G"], case["D"]
    window, sinks = case["window"], case["sinks"]
    n = st["n_nodes"].long() if st["n_nodes"] is not None else torch.full_like(lens, M)
    base = lens - n
    anc = _ancestors(st["parent"], B, M)
    pos = base[:, None] + anc.sum(-1) - 1  # [B, M] each node's position
    if window:  # the only tokens that any node can see: the first ones, then the window's
        start = (base + 1 - window).clamp(min=sinks)
        t = torch.cat([torch.arange(sinks, device="cuda").expand(B, -1),
                       start[:, None] + torch.arange(window - 1 + M, device="cuda")], 1)
    else:
        t = torch.arange(table.shape[1] * PAGE, device="cuda").expand(B, -1)
    inside = t < lens[:, None]
    ts = torch.where(inside, t, 0)
    page = torch.gather(table.long(), 1, ts // PAGE)
    k = st["k"][page, :, ts % PAGE].float()  # [B, N, Hkv, D]
    v = st["v"][page, :, ts % PAGE].float()
    if st["k_scale"] is not None:
        k, v = k * st["k_scale"], v * st["v_scale"]
    j = t - base[:, None]
    node = (j >= 0) & (j < n[:, None])
    jn = j.clamp(0, M - 1)
    see = torch.where(node[:, None], torch.gather(anc, 2, jn[:, None].expand(-1, M, -1)), (j < 0)[:, None]) & inside[:, None]
    if window:
        at = torch.where(node, torch.gather(pos, 1, jn), t)
        see = see & ((pos[:, :, None] - at[:, None] < window) | (at < sinks)[:, None])
    see = see & (torch.arange(M, device="cuda") < n[:, None])[:, :, None]
    qf = q.float().reshape(B, M, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, M * G, D)
    s = torch.matmul(qf, k.permute(0, 2, 3, 1)).mul_(1 / math.sqrt(D)).reshape(B, Hkv, M, G, -1)
    s.masked_fill_(~see[:, None, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top > -math.inf, top, 0)).exp_()
    z = p.sum(-1, keepdim=True)
    lse = (z.log() + top)[..., 0]
    o = torch.matmul(p.reshape(B, Hkv, M * G, -1), v.permute(0, 2, 1, 3)).reshape(B, Hkv, M, G, D)
    o = torch.where(z > 0, o / z, 0)
    return (o.permute(0, 2, 1, 3, 4).reshape(B, M, Hkv * G, D).to(torch.bfloat16),
            lse.permute(0, 2, 1, 3).reshape(B, M, Hkv * G))


def _verify(st):
    p, q, tok, parent, ua = st["p"], st["q"], st["tokens"].long(), st["parent"].long(), st["u_accept"].double()
    B, M, V = p.shape
    rows = torch.arange(B, device="cuda")
    cur = torch.zeros(B, dtype=torch.long, device="cuda")
    n_path = torch.ones(B, dtype=torch.long, device="cuda")
    path = torch.full((B, M), -1, dtype=torch.long, device="cuda")
    path[:, 0] = 0
    w, total = p[:, 0].double(), torch.ones(B, dtype=torch.float64, device="cuda")
    ids = torch.arange(V, device="cuda")
    for m in range(1, M):  # a node is tested when the walk stands at its parent
        x = tok[:, m]
        test = parent[:, m] == cur
        px = w[rows, x]
        qx = q[rows, cur, x].double() if q is not None else torch.ones_like(px)
        yes = test & (ua[:, m] * qx * total < px)
        no = test & ~yes
        if q is not None:
            r = (w / total[:, None] - q[rows, cur].double()).clamp(min=0)
        else:
            r = torch.where(ids == x[:, None], 0, w)
        z = r.sum(-1)
        no = no & (z > 0)
        cur = torch.where(yes, m, cur)
        w = torch.where(yes[:, None], p[:, m].double(), torch.where(no[:, None], r, w))
        total = torch.where(yes, 1.0, torch.where(no, z, total))
        path.scatter_(1, n_path.clamp(max=M - 1)[:, None],
                      torch.where(yes, m, path.gather(1, n_path.clamp(max=M - 1)[:, None])[:, 0])[:, None])
        n_path = n_path + yes
    return n_path.int(), path.int(), _sample_rows(w, st["u_sample"]).int()


def _append(st):
    k, v, cu, lens = st["k"], st["v"], st["cu"].long(), st["lens"].long()
    i = torch.arange(st["k_new"].shape[1], device="cuda")
    b = torch.searchsorted(cu, i, right=True) - 1
    t = lens[b] - (cu[b + 1] - i)  # the new tokens are the last ones of their sequence
    page = st["table"].long()[b, t // PAGE]
    k[page, :, t % PAGE] = st["k_new"].transpose(0, 1)
    v[page, :, t % PAGE] = st["v_new"].transpose(0, 1)
    return k, v


def _fork(st):
    k, v, table, lens, held, ref = (st[n] for n in ("k", "v", "table", "lens", "held", "ref"))
    cols = torch.arange(table.shape[1], device="cuda")
    # the branches of the last pass go
    stay = (st["stay"] + PAGE - 1) // PAGE
    gone = (cols >= stay[:, None]) & (cols < held[:, None])
    ref.index_add_(0, torch.where(gone, table, 0).reshape(-1).long(), -gone.reshape(-1).int())
    held.copy_(torch.minimum(held, stay))
    # full pages are shared, a part-filled last page is copied to the lowest free one
    src, dst = st["src"].long(), st["dst"].long()
    L = lens[src].long()
    free = torch.sort((ref != 0).to(torch.uint8), stable=True).indices
    need = L % PAGE != 0
    new = free[need.long().cumsum(0) - need.long()]
    shared = cols < (L // PAGE)[:, None]
    rows = table[src].long()
    ref.index_add_(0, torch.where(shared, rows, 0).reshape(-1), shared.reshape(-1).int())
    old = rows.gather(1, (L // PAGE).clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    to = torch.where(need, new, rows[:, 0])
    old = torch.where(need, old, rows[:, 0])
    ref.index_add_(0, to, need.int())
    mine = (cols == (L // PAGE)[:, None]) & need[:, None]
    table[dst] = torch.where(shared, rows, torch.where(mine, new[:, None], table[dst].long())).int()
    fill = (torch.arange(PAGE, device="cuda") < (L % PAGE)[:, None])[:, None, :, None]
    k[to] = torch.where(fill, k[old], k[to])
    v[to] = torch.where(fill, v[old], v[to])
    held[dst] = ((L + PAGE - 1) // PAGE).int()
    lens[dst] = L.int()
    return k, v, table, lens, held, ref


def _move(st, h, b, src, dst):
    """Token src of sequence b, head h to token dst, all of them at once."""
    table = st["table"].long()
    for x in (st["k"], st["v"]):
        rows = x[table[b, src // PAGE], h, src % PAGE]
        x[table[b, dst // PAGE], h, dst % PAGE] = rows


def _accept(st):
    B, M = st["path"].shape
    base = (st["lens"] - st["n_nodes"]).long()
    i = torch.arange(M, device="cuda")
    stays = (i < st["n_path"][:, None])[:, None].expand(B, st["case"]["Hkv"], M)
    to = (base[:, None] + i)[:, None].expand_as(stays)
    frm = torch.where(stays, (base[:, None] + st["path"])[:, None].expand_as(stays), to)
    h = torch.arange(st["case"]["Hkv"], device="cuda")[None, :, None].expand_as(stays)
    b = torch.arange(B, device="cuda")[:, None, None].expand_as(stays)
    _move(st, h, b, frm, to)
    return st["k"], st["v"], (base + st["n_path"]).int()


def _keep(st):
    cu = st["cu_kept"].long()
    Hkv, n = st["idx"].shape
    i = torch.arange(n, device="cuda")
    b = torch.searchsorted(cu, i, right=True) - 1
    to = (i - cu[b]).expand(Hkv, n)
    h = torch.arange(Hkv, device="cuda")[:, None].expand(Hkv, n)
    _move(st, h, b.expand(Hkv, n), st["idx"].long(), to)
    return st["k"], st["v"], (cu[1:] - cu[:-1]).int()


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers alone
    st = prepare(case, seed)
    op = case["op"]
    lens = st["lens"].tolist()
    table = st["table"].tolist()
    if op == "attn":
        return _exact_attn(case, st, lens, table)
    k, v = st["k"], st["v"]
    slot = lambda b, t: (table[b][t // PAGE], t % PAGE)  # noqa: E731
    if op == "append":
        cu = st["cu"].tolist()
        for b in range(case["B"]):
            n, t = cu[b + 1] - cu[b], lens[b] - (cu[b + 1] - cu[b])
            done = 0
            while done < n:  # to the end of a page at a time
                page, s = slot(b, t + done)
                c = min(PAGE - s, n - done)
                k[page, :, s:s + c] = st["k_new"][:, cu[b] + done:cu[b] + done + c]
                v[page, :, s:s + c] = st["v_new"][:, cu[b] + done:cu[b] + done + c]
                done += c
        return k.double(), v.double()
    if op == "fork":
        free = [p for p, r in enumerate(st["ref"].tolist()) if r == 0]
        for a in st["src"].tolist():
            if lens[a] % PAGE:
                frm, to = table[a][lens[a] // PAGE], free.pop(0)
                k[to, :, :lens[a] % PAGE] = k[frm, :, :lens[a] % PAGE]
                v[to, :, :lens[a] % PAGE] = v[frm, :, :lens[a] % PAGE]
        return k.double(), v.double(), None, None, None, None
    if op == "accept":
        path, n_path = st["path"].tolist(), st["n_path"].tolist()
        for b in range(case["B"]):
            base = lens[b] - case["M"]
            for i in range(n_path[b]):  # a node never moves back, so one after the other is right
                (p0, s0), (p1, s1) = slot(b, base + path[b][i]), slot(b, base + i)
                k[p1, :, s1] = k[p0, :, s0].clone()
                v[p1, :, s1] = v[p0, :, s0].clone()
        return k.double(), v.double(), None
    cu = st["cu_kept"].tolist()
    for b in range(case["B"]):
        K = cu[b + 1] - cu[b]
        pages = st["table"][b, :-(-lens[b] // PAGE)].long()
        for x in (k, v):
            for h in range(case["Hkv"]):
                rows = x[pages, h].reshape(-1, case["D"])
                rows[:K] = rows[st["idx"][h, cu[b]:cu[b + 1]].long()].clone()
                x[pages, h] = rows.reshape(len(pages), PAGE, case["D"])
    return k.double(), v.double(), None


def _exact_attn(case, st, lens, table):
    B, M, Hkv, G, D = case["B"], case["M"], case["Hkv"], case["G"], case["D"]
    n = st["n_nodes"].tolist() if st["n_nodes"] is not None else [M] * B
    parent = st["parent"].tolist() if st["parent"] is not None else [list(range(-1, M - 1))] * B
    out = torch.zeros((B, M, Hkv * G, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, M, Hkv * G), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        pages = st["table"][b, :-(-lens[b] // PAGE)].long()
        k = st["k"][pages].permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :lens[b]].double()
        v = st["v"][pages].permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :lens[b]].double()
        if st["k_scale"] is not None:
            k, v = k * st["k_scale"].double(), v * st["v_scale"].double()
        base = lens[b] - n[b]
        depth = []
        for m in range(M):
            depth.append(0 if parent[b][m] < 0 else depth[parent[b][m]] + 1)
        see = torch.zeros((n[b], lens[b]), dtype=torch.bool)
        for m in range(n[b]):
            here = base + depth[m]
            first = 0 if not case["window"] else max(0, here - case["window"] + 1)
            see[m, first:base] = True
            see[m, :min(case["sinks"], base)] = True
            a = m
            while a >= 0:
                if not case["window"] or base + depth[a] >= first or base + depth[a] < case["sinks"]:
                    see[m, base + a] = True
                a = parent[b][a]
        see = see.cuda()
        for h in range(Hkv):
            qh = st["q"][b, :n[b], h * G:(h + 1) * G].double()  # [n, G, D]
            s = (qh.reshape(-1, D) @ k[h].T / math.sqrt(D)).reshape(n[b], G, -1)
            s = torch.where(see[:, None], s, -math.inf)
            z = torch.logsumexp(s, -1)
            lse[b, :n[b], h * G:(h + 1) * G] = z
            p = torch.where(see[:, None], torch.exp(s - torch.where(z.isinf(), 0.0, z)[..., None]), 0.0)
            out[b, :n[b], h * G:(h + 1) * G] = (p.reshape(n[b] * G, -1) @ v[h]).reshape(n[b], G, D)
    return out, lse
