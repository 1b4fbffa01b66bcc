"""Calls with ``stream=``: what they allocate belongs to that stream.

The stream is kept busy while the call is made, so its kernels run only after
the host has gone on: the current stream then takes as much memory as the call
had for its workspace and results, fills it, and the results must still be
those of a plain call.  (Memory of the current stream's would be handed out
again at once, while the kernels still use it.)"""
import numpy as np
import pytest
import torch

from equivariant_interatomic_potential_gb300 import workloads, zs
from train_refs import csr

pytestmark = pytest.mark.gpu

BUSY = 20_000_000   # cycles: some 10 ms


def grouped(dtype):
    # rows off 16-byte boundaries, gathered: operands laid out anew, partial weight gradients
    gen = torch.Generator(device="cuda").manual_seed(1)
    M, K, N, G = 3000, 131, 67, 5
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    row_ptr, perm = (torch.from_numpy(a).cuda() for a in csr(np.random.default_rng(1).integers(0, G, M), G))
    x, w, dy = rnd(M, K), rnd(G, N, K), rnd(M, N)
    return {"y": lambda **kw: zs.zs_grouped_matmul(x, w, row_ptr, perm, **kw),
            "dx": lambda **kw: zs.zs_grouped_matmul_dx(dy, w, row_ptr, perm, **kw),
            "dw": lambda **kw: zs.zs_grouped_matmul_dw(dy, x, row_ptr, perm, **kw),
            "both": lambda **kw: zs.zs_grouped_matmul_backward(dy, x, w, row_ptr, perm, **kw)}


def norm():
    gen = torch.Generator(device="cuda").manual_seed(2)
    M, C = 4000, 129
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    ops = (rnd(M, C), rnd(M, C), rnd(M, C), rnd(C), rnd(C), rnd(C))
    dy, du = rnd(M, C), rnd(M, C)
    stats = zs.zs_norm_gate_residual(*ops)[2]
    return {"norm": lambda **kw: zs.zs_norm_gate_residual(*ops, **kw),
            "norm backward": lambda **kw: zs.zs_norm_gate_residual_backward(dy, du, *ops, stats, **kw)}


def scatter():
    w = workloads.make_random(500, 20000, 32, seed=3)
    coup, rad, dst = (torch.from_numpy(a).cuda() for a in (w.coup, w.rad, w.dst))
    row_ptr, perm, _ = zs.zs_build_csr(dst, w.N)
    scale = torch.rand(w.N, device="cuda") + 0.5
    out, raw = zs.zs_forward_scaled(coup, rad, row_ptr, perm, scale, w.N)
    return {"csr": lambda **kw: zs.zs_build_csr(dst, w.N, **kw),
            "forward": lambda **kw: zs.zs_forward(coup, rad, row_ptr, perm, w.N, **kw),
            "forward_ld": lambda **kw: zs.zs_forward_ld(coup, rad, row_ptr, perm, w.N, **kw),
            "forward_scaled": lambda **kw: zs.zs_forward_scaled(coup, rad, row_ptr, perm, scale, w.N, **kw),
            "backward": lambda **kw: zs.zs_backward(out, coup, rad, dst, w.N, **kw),
            "backward_csr": lambda **kw: zs.zs_backward_csr(out, coup, rad, row_ptr, perm, w.N, **kw),
            "backward_scaled": lambda **kw: zs.zs_backward_scaled(out, coup, rad, dst, scale, w.N, raw, **kw)}


def each(result):
    return result if isinstance(result, tuple) else (result,)


@pytest.mark.parametrize("handle", [False, True], ids=["object", "handle"])
@pytest.mark.parametrize("calls", [lambda: grouped(torch.float32), lambda: grouped(torch.bfloat16), norm, scatter],
                         ids=["grouped_f32", "grouped_bf16", "norm", "scatter"])
def test_memory_stays_the_streams(calls, handle):
    s = torch.cuda.Stream()
    for name, call in calls().items():
        want = each(call())
        sizes = {t.numel() * t.element_size() for t in want}
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        call()
        sizes.add(torch.cuda.max_memory_allocated() - before)
        torch.cuda.empty_cache()
        with torch.cuda.stream(s):
            torch.cuda._sleep(BUSY)
        got = each(call(stream=s.cuda_stream if handle else s))
        taken = []
        for n in sorted(sizes) + [1 << 12, 1 << 16, 1 << 20, 1 << 22]:
            for _ in range(4):
                taken.append(torch.full((max(n, 1),), 0xA5, dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        assert all((a is None) == (b is None) and (a is None or torch.equal(a, b)) for a, b in zip(got, want)), name


def test_results_dropped_on_the_callers_stream():
    # a result that the caller's stream still reads when it is dropped is not handed to the next call on the stream
    y = grouped(torch.bfloat16)["y"]
    want = y()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = y(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(BUSY)
    copy = got.clone()          # waits behind the sleep
    del got
    with torch.cuda.stream(s):
        other = torch.full_like(want, 7.0)
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and bool((other == 7.0).all())


def test_default_stream_by_its_handle():
    y = grouped(torch.float32)["y"]
    want = y()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = y(stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
