"""Host side of the paged calls: sizes and arguments at the ends of their ranges, without a GPU."""
import ctypes

import pytest

from test_paged_cpu import ALL_OK, _kv, calls, sgd  # noqa: F401


@pytest.mark.parametrize("D,dtype", [(128, 1), (64, 2)])
def test_a_workspace_serves_every_smaller_step(sgd, D, dtype):
    """sgd_paged_workspace_size promises bytes for up to M query tokens and G heads."""
    assert (sgd.SGD_BF16, sgd.SGD_I8) == (1, 2)
    kv = _kv(sgd, B=4, D=D, dtype=dtype, k_scale=0x50000, v_scale=0x50010)
    size = {(G, M): sgd.lib.sgd_paged_workspace_size(ctypes.byref(kv), G, M) for G in range(1, 17) for M in range(65)}
    assert all(size.values())
    for G in range(1, 17):
        for M in range(1, 65):
            assert size[G, M - 1] <= size[G, M], (G, M)
            assert G == 1 or size[G - 1, M] <= size[G, M], (G, M)


def test_narrower_steps_run_on_the_widest_steps_workspace(sgd):
    kv, attn = _kv(sgd, B=4), calls(sgd)["attn"]
    for G, M in ((16, 40), (9, 64), (12, 60), (8, 64)):
        n = sgd.lib.sgd_paged_workspace_size(ctypes.byref(kv), G, M)
        for g in range(1, G + 1):
            for m in range(1, M + 1):
                assert attn(kv, n=n, G=g, M=m) not in ALL_OK, (G, M, g, m)


def test_append_refuses_counts_beyond_32_bits(sgd):
    # T_new * Hkv wraps to 0 and to negative numbers in 64 bits
    for Hkv, T in ((2, 1 << 62), (4, 1 << 62), (2, (1 << 63) - 1), (2, 1 << 30), (1, 1 << 31)):
        assert calls(sgd)["append"](_kv(sgd, Hkv=Hkv), T=T) == -2, (Hkv, T)
    assert calls(sgd)["append"](_kv(sgd), T=(1 << 30) - 1) not in ALL_OK


def test_binding_refuses_tensors_that_are_not_on_a_gpu(sgd):
    """With a stream given, addresses of host memory reached the kernels."""
    import torch
    i32, stream = torch.int32, type("Stream", (), {"cuda_stream": 0})()
    k = torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16)
    table, lens, ref = torch.zeros(3, 2, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(4, dtype=i32)
    cache = sgd.PagedKv(k, k.clone(), table, lens, lens, ref)
    u = torch.zeros(3, 2)
    cu, out, ws = torch.zeros(4, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(1 << 24, dtype=torch.uint8)
    q = torch.zeros(3, 2, 8, 64, dtype=torch.bfloat16)
    for call in (
        lambda: sgd.paged_attn(q, 4, cache, out=(q.clone(), torch.zeros(3, 2, 8)), workspace=ws, stream=stream),
        lambda: sgd.verify_tree(torch.zeros(3, 2, 8), table, table, u, u[:, 0].contiguous(), out=(out, table, lens), workspace=ws,
                                stream=stream),
        lambda: sgd.pages_reserve(cache, lens, out=out, workspace=ws, stream=stream),
        lambda: sgd.pages_append(cache, k[0], k[0], cu, workspace=ws, stream=stream),
        lambda: sgd.pages_fork(cache, lens[:1], lens[1:2], workspace=ws, stream=stream),
        lambda: sgd.pages_release(cache, lens, workspace=ws, stream=stream),
        lambda: sgd.pages_accept(cache, table, lens, lens, out=out, workspace=ws, stream=stream),
        lambda: sgd.pages_keep(cache, table[:2], cu, out=out, workspace=ws, stream=stream),
    ):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_keeps_the_sign_of_a_window(sgd, monkeypatch):
    """A number below -2^31 wraps on its way into 32 bits, to 0 (no window at all) or to a positive one."""
    import types

    import torch
    k = torch.zeros(1, 1, 64, 64, dtype=torch.bfloat16)
    table = torch.zeros(1, 1, dtype=torch.int32)
    cache = sgd.PagedKv(k, k, table, table[0])
    q = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    host = types.SimpleNamespace(raw=0, empty=lambda shape, dtype: torch.empty(shape, dtype=dtype),
                                 workspace=lambda n, ws: ws)
    monkeypatch.setattr(sgd, "_On", lambda device, stream: host)
    ws = torch.zeros(1 << 26, dtype=torch.uint8)
    for n in (-1, -2 ** 31, -2 ** 31 - 1, -2 ** 32, -2 ** 32 + 1, -2 ** 40):
        for kw in (dict(window=n), dict(window=5, sinks=n)):
            with pytest.raises(sgd.SgdError, match=r"sgd_paged_attn.*-8"):
                sgd.paged_attn(q, 1, cache, workspace=ws, **kw)


def kernels_that_wait():
    """(name, parameters, body) of each kernel that is launched early and waits for the stream's last one."""
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_gqa_decode_b200", "csrc")
    for name in sorted(os.listdir(csrc)):
        if name.endswith(".cu"):
            text = open(os.path.join(csrc, name)).read()
            for part in text.split("__global__ void")[1:]:
                m = re.match(r"(?:\s|__launch_bounds__\([^)]*\))*(\w+)\((.*?)\) \{\n(.*?)\n\}\n", part, re.S)
                if m and "grid_dependency_wait()" in m.group(3):
                    yield m.groups()


def test_early_kernels_promise_nothing_about_their_inputs(sgd):
    """What the stream's last kernel writes is not read-only while an early kernel runs: __restrict__ on a const
    pointer and __ldg say that it is, and such a load may move in front of the wait."""
    found = {name: (args, body) for name, args, body in kernels_that_wait()}
    assert set(found) == {"paged_attn_kernel", "paged_merge_kernel", "reserve_kernel", "fork_plan_kernel", "fork_copy_kernel"}
    for name, (args, body) in found.items():
        assert "__restrict__" not in args, name
        for word in ("__ldg(", "calibrated_scale(", ".nc"):
            assert word not in body, (name, word)
