"""Barriers of clusters, whose CTAs read each other's parts: warps come to them together, and what is read has been written."""
import glob
import os
import re

import numpy as np
import pytest
import torch

from equivariant_interatomic_potential_gb300 import build, zs


def test_barriers_bring_warps_together():
    # barrier.cluster is an instruction of a whole warp, whose threads may come from branches: there is one place that has it
    found = {}
    for path in glob.glob(os.path.join(build.CSRC, "*")):
        if path.endswith((".cu", ".cuh")):
            with open(path) as f:
                found[os.path.basename(path)] = len(re.findall(r"barrier\.cluster\.", f.read()))
    assert [p for p, n in found.items() if n] == ["zs_common.cuh"]
    with open(os.path.join(build.CSRC, "zs_common.cuh")) as f:
        assert len(re.findall(r"__syncwarp\(\);\n\s*asm volatile\(\"barrier\.cluster\.(?:arrive\.release|wait\.acquire)\.aligned", f.read())) == 2


@pytest.mark.gpu
def test_parts_of_an_order():
    # the cluster that orders few keys, and those that count tiles of many
    rng = np.random.default_rng(3)
    r = torch.Generator(device="cuda").manual_seed(4)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(1500):
        E, N = (int(rng.integers(1025, 16385)), int(rng.integers(1, 1024))) if i % 10 else (int(rng.integers(140000, 600000)), 7921)
        ids = torch.randint(-1, N + 1, (E,), generator=r, device="cuda", dtype=torch.int32)
        row_ptr, perm, bad = zs.zs_build_csr(ids, N)
        key = torch.where((ids >= 0) & (ids < N), ids, N).long()
        sorted_, order = torch.sort(key, stable=True)
        start = torch.searchsorted(sorted_, torch.arange(N + 1, device="cuda"))
        wrong += (perm != order).sum() + (row_ptr != start).sum() + (bad[0] != E - start[N])
    assert int(wrong) == 0
