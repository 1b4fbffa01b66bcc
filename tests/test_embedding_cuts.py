"""The embedding's gradient where rows of the table are cut between the threads and the CTAs that add them up."""
import numpy as np
import pytest
import torch

from equivariant_interatomic_potential_gb300 import zs
from train_refs import HALF_ULP, STEP, TORCH


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_small_gradients_of_odd_widths(dtype):
    """Many small gradients, whose rows go on from one CTA to the next while others end inside a piece.  Sums of at most 500
    terms in fp32: each addition and the product with the scale is off by 2^-24 of the sum of magnitudes at most: 2^-15,
    then the rounding to the type."""
    rng = np.random.default_rng(21)
    r = torch.Generator(device="cuda").manual_seed(22)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(3000):
        M, V, C = int(rng.integers(100, 501)), int(rng.integers(1, 120)), int(rng.integers(25, 70))
        ids = torch.randint(-1, V + 1, (M,), generator=r, device="cuda", dtype=torch.int32)
        if i % 2:
            ids = ids.clamp_max(V // 4)                      # few ids, which go over several CTAs
        wide = torch.randn(M, C + 3, generator=r, device="cuda").to(TORCH[dtype])
        dy = wide[:, i % 4:i % 4 + C] if i % 3 else wide[:, :C].contiguous()
        row_ptr, perm, _ = zs.zs_build_csr(ids, V)
        dw = zs.zs_embedding_backward(dy, row_ptr, perm, 0.5).double()
        held_ids = torch.where((ids >= 0) & (ids < V), ids, V).long()
        want, mag = (torch.zeros(V + 1, C, dtype=torch.float64, device="cuda").index_add_(0, held_ids, t)[:V] * 0.5
                     for t in (dy.double(), dy.double().abs()))
        wrong += (~((dw - want).abs() <= 2.0 ** -15 * mag + HALF_ULP[dtype] * 1.001 * want.abs() + STEP[dtype])).sum()
    assert int(wrong) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("C,counts", [(53, (190, 0, 33, 10, 7, 4, 6)), (29, (420, 180, 33, 9, 4, 7, 5, 5, 5, 6)), (43, (247, 13, 10, 4, 7, 5, 3))])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_that_go_on_beside_others_that_end(C, counts, dtype):
    # ones: a row of dw is the count of its id, in every column; shifted by a few ids, so that each row comes to each place
    for lead in range(60):
        n = np.array((lead + 1,) + counts + tuple(counts[-1 - i % 4] for i in range(30)))
        ids = torch.from_numpy(np.repeat(np.arange(len(n)), n).astype(np.int32)).cuda()
        row_ptr, perm, _ = zs.zs_build_csr(ids, len(n))
        dw = zs.zs_embedding_backward(torch.ones(len(ids), C, dtype=TORCH[dtype], device="cuda"), row_ptr, perm)
        want = torch.from_numpy(n).cuda().to(TORCH[dtype])[:, None].expand(-1, C)
        assert torch.equal(dw, want), (lead, torch.nonzero(dw != want)[:8].tolist())
