"""What is built: libzs, which needs nvcc alone, and zs_torch, without which the binding works too."""
import os
import sysconfig

import pytest
import torch

from equivariant_interatomic_potential_gb300 import build, zs


def test_extension_is_of_one_torch_and_python(monkeypatch):
    name = os.path.basename(build.ext_path())
    assert torch.__version__ in name and name.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert os.path.basename(build.ext_path()) != name and "9.9.9" in build.ext_path()


@pytest.fixture
def no_extension(monkeypatch, tmp_path):
    """Another torch's file name, a compiler that fails, and a binding that has not loaded anything yet."""
    monkeypatch.setattr(build, "ext_path", lambda: str(tmp_path / "zs_torch.so"))
    monkeypatch.setenv("CXX", "false")
    fast = zs._Fast()
    monkeypatch.setattr(zs, "_fast", fast)
    return fast


def test_library_without_the_extension(no_extension):
    with pytest.warns(UserWarning, match="zs_torch was not built"):
        assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert build.up_to_date()
    with pytest.raises(RuntimeError, match="zs_torch failed"):
        build.build_ext()
    with pytest.warns(UserWarning, match="zs_torch cannot be used"):
        assert no_extension.matmul(1, 2, 3) is NotImplemented
    assert no_extension.norm_backward() is NotImplemented      # without another warning
    with pytest.raises(AttributeError):
        no_extension.anything_else


@pytest.mark.gpu
def test_results_without_the_extension(no_extension, monkeypatch):
    gen = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, w, dy = rnd(700, 65), rnd(3, 40, 65), rnd(700, 40)
    row_ptr = torch.tensor([0, 100, 100, 600], dtype=torch.int32, device="cuda")
    perm = torch.randperm(700, generator=gen, device="cuda").int()
    ops, cot = (rnd(300, 96), rnd(300, 96), rnd(300, 96), rnd(96), rnd(96), rnd(96)), (rnd(300, 96), rnd(300, 96))

    def everything():
        y = zs.zs_grouped_matmul(x, w, row_ptr, perm)
        n = zs.zs_norm_gate_residual(*ops, kind="layer")
        return (y, *zs.zs_grouped_matmul_backward(dy, x, w, row_ptr, perm), *n,
                *zs.zs_norm_gate_residual_backward(*cot, *ops, n[2], kind="layer"))

    with pytest.warns(UserWarning, match="zs_torch cannot be used"):
        without = everything()
    monkeypatch.undo()
    assert all(torch.equal(a, b) for a, b in zip(without, everything()))


@pytest.mark.gpu
def test_allocations_that_fail():
    # results of 4 TB, refused by the allocator: the same exception from the extension and from the binding
    n = 1 << 20
    x, w = torch.zeros(n, 1, device="cuda"), torch.zeros(1, n, 1, device="cuda")
    row_ptr = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    for call in (lambda **kw: zs.zs_grouped_matmul(x, w, row_ptr, **kw), lambda **kw: zs.zs_grouped_matmul_dw(x.view(1, n), x.view(1, n), row_ptr, **kw)):
        for kw in ({}, {"stream": torch.cuda.Stream()}):
            with pytest.raises(torch.OutOfMemoryError):
                call(**kw)


@pytest.mark.gpu
@pytest.mark.parametrize("short", [True, False], ids=["extension", "binding"])
@pytest.mark.parametrize("want", [True, 1, "yes", False, 0, None])
def test_any_truth_value_asks_for_statistics(want, short, monkeypatch):
    if not short:
        monkeypatch.setattr(zs, "_fast", type("None", (), {"norm": staticmethod(lambda *a: NotImplemented)}))
    t, v = torch.ones(4, 8, device="cuda"), torch.ones(8, device="cuda")
    assert (zs.zs_norm_gate_residual(t, t, None, v, v, v, want_stats=want)[2] is not None) == bool(want)
