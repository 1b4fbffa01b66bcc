"""Operands on several devices, and on one that is not the current one.

With fake tensors, which have a device and a shape and no memory, and a stand-in
for the library: a call either refuses its operands or makes its launch with
their device current.  Nothing reaches a GPU."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from equivariant_interatomic_potential_gb300 import zs

# where there is a GPU, a fake tensor's device has to exist
pytestmark = [pytest.mark.filterwarnings("ignore:Accessing the data pointer"),
              pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.device_count() < 2, reason="one GPU")]


class Machine:
    """Two devices, the first one current, and a library that notes which device its calls see."""

    def __init__(self, monkeypatch):
        self.current, self.seen = 0, []
        machine = self

        class Enter:
            def __init__(self, device):
                self.device = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)

            def __enter__(self):
                self.before, machine.current = machine.current, self.device.index

            def __exit__(self, *exc):
                machine.current = self.before

        class Library:
            def __getattr__(self, name):
                def call(*args):
                    if not name.endswith("bytes"):
                        machine.seen.append((name, machine.current))
                    return 0
                return call

        class Fast:
            def __getattr__(self, name):
                return lambda *args: NotImplemented

        monkeypatch.setattr(zs, "_raw_device", lambda: self.current)
        monkeypatch.setattr(zs, "_raw_stream", lambda device: 100 + device)
        monkeypatch.setattr(torch.cuda, "device", Enter)
        monkeypatch.setattr(zs, "load", lambda: Library())
        monkeypatch.setattr(zs, "_fast", Fast())


@pytest.fixture
def machine(monkeypatch):
    with FakeTensorMode():
        yield Machine(monkeypatch)


def on(device, *shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device=f"cuda:{device}")


def calls(devices):
    """Each call and its operands, the i-th one on devices[i % len(devices)]."""
    n = len(devices)
    M, K, N, G = 6, 8, 4, 2
    x, w, dy = (lambda d: on(d, M, K)), (lambda d: on(d, G, N, K)), (lambda d: on(d, M, N))
    rp, pm = (lambda d: on(d, G + 1, dtype=torch.int32)), (lambda d: on(d, M, dtype=torch.int32))
    row, vec, st = (lambda d: on(d, M, K)), (lambda d: on(d, K)), (lambda d: on(d, M, 4))
    for fn, make in ((zs.zs_grouped_matmul, (x, w, rp, pm)), (zs.zs_grouped_matmul_dx, (dy, w, rp, pm)),
                     (zs.zs_grouped_matmul_dw, (dy, x, rp, pm)),
                     (zs.zs_norm_gate_residual, (row, row, row, vec, vec, vec)),
                     (zs.zs_norm_gate_residual_backward, (row, row, row, row, row, vec, vec, vec, st))):
        yield fn, [f(devices[i % n]) for i, f in enumerate(make)]


def test_mixed_devices_refused(machine):
    for fn, operands in calls((0, 1)):
        with pytest.raises(ValueError, match="one device, got cuda:0 and cuda:1"):
            fn(*operands)
    for fn, operands in calls((0,)):
        for i, t in enumerate(operands):
            other = list(operands)
            other[i] = on(1, *t.shape, dtype=t.dtype)
            with pytest.raises(ValueError, match="one device"):
                fn(*other)
    assert not machine.seen
    x, w, rp = on(0, 6, 8), on(0, 2, 4, 8), on(0, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="one device"):
        zs.zs_grouped_matmul(x, w, rp, out=on(1, 6, 4))


@pytest.mark.parametrize("device", [0, 1])
def test_launched_on_the_operands_device(machine, device):
    for fn, operands in calls((device,)):
        machine.seen.clear()
        fn(*operands)
        assert [d for _, d in machine.seen] == [device] and machine.current == 0, machine.seen


def test_optimiser_step(machine):
    plan = zs.AdamWPlan(*([on(1, 5)] for _ in range(4)))
    zs.zs_adamw_step(plan, 1, lr=1e-3)
    assert machine.seen == [("zs_adamw_step", 1)] and machine.current == 0
    with pytest.raises(ValueError, match="on cuda:0"):
        zs.AdamWPlan([on(1, 5)], [on(0, 5)], [on(1, 5)], [on(1, 5)])
    with pytest.raises(ValueError, match="grad_scale"):
        zs.zs_adamw_step(plan, 1, lr=1e-3, grad_scale=on(0, 1))


def test_stream_of_another_device(machine):
    class Stream:
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError, match="operands and the stream"):
        zs._one_device((on(0, 3), None, 2.0), Stream.device)
    assert zs._one_device((on(1, 3), None), Stream.device) == 1
