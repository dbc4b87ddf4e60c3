"""Selection of experts on the GPU at its edges, against the oracle."""
import numpy as np
import pytest
import torch

import bit_weight_only_quantize_amd as w4
import oracle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,k,groups,top,best", [(64, 6, 1, 1, 1), (8, 3, 1, 1, 1), (96, 8, 8, 3, 2), (256, 8, 8, 4, 1),
                                                 (600, 12, 4, 2, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_logits_count_as_masked(score, E, k, groups, top, best, dtype):
    """Choices as if the NaN logits were -infinity, with a bias too; weights NaN. Rows with one NaN up to all of them."""
    g = torch.Generator().manual_seed(E)
    l = torch.randn((40, E), generator=g).to(torch.bfloat16).float()
    nan = torch.rand((40, E), generator=g) < torch.linspace(0, 0.9, 40)[:, None]
    nan[:, 3] = True
    l[nan] = float("nan")
    l[7, 5] = float("-inf")
    l[8] = float("nan")
    x = l.to(torch.bfloat16) if dtype == "bf16" else l
    bias = 0.01 * torch.randn((E,), generator=g)
    for b in (None, bias):
        for renorm in (False, True):
            ids, w = w4.moe_select(x.cuda(), k, score, None if b is None else b.cuda(), groups, top, best, renorm)
            want, _ = oracle.moe_select(l.numpy(), k, score, None if b is None else b.numpy(), groups, top, best, renorm)
            assert np.array_equal(ids.cpu().numpy(), want), (b is None, renorm)
            assert bool(w.isnan().all())
