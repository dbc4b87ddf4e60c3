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


@pytest.mark.parametrize("E,k,groups,top,best", [(1024, 32, 1, 1, 1), (1024, 16, 8, 4, 2), (512, 8, 4, 2, 1), (256, 8, 1, 1, 1), (100, 8, 10, 4, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choice_values_next_to_each_other(score, E, k, groups, top, best):
    """A bias that leaves all choice values within some 10^-8 of each other, over logits of which most lie 8 binades below
    the largest, where the sum of a softmax in fp32 is off most: choices are those of 64 bits all the same."""
    rng = np.random.default_rng(E + k)
    base = -5.5 + 0.3 * rng.normal(size=E)
    base[rng.choice(E, 3, replace=False)] = [0, -0.2, -1]
    l = (base + rng.uniform(-20, 20, size=(64, 1))).astype(np.float32)       # a row's shift rounds every logit anew
    l64 = l.astype(np.float64)
    s = np.exp(base) / np.exp(base).sum() if score == "softmax" else 1 / (1 + np.exp(-l64[0]))
    if score == "sigmoid":
        l = (l64[:1] + rng.normal(size=(64, E)) * 2.0 ** -22).astype(np.float32)
    for width in (1e-7, 1e-8, 1e-9):
        bias = (0.01 - s + width * rng.normal(size=E)).astype(np.float32)
        ids, w = w4.moe_select(torch.from_numpy(l).cuda(), k, score, torch.from_numpy(bias).cuda(), groups, top, best)
        want, ww = oracle.moe_select(l, k, score, bias, groups, top, best)
        assert np.array_equal(ids.cpu().numpy(), want), width
        assert (np.abs(w.cpu().double().numpy() - ww) <= 2.0 ** -18 * ww).all()


@pytest.mark.parametrize("scale", [1, 20, 60])
@pytest.mark.parametrize("E,k,groups,top", [(128, 8, 1, 1), (256, 8, 8, 4), (1024, 32, 1, 1), (5, 2, 1, 1)])
def test_weights_as_close_as_their_formula(E, k, groups, top, scale):
    """Scores are computed in 64 bits but for the sum of a softmax, which fp32 holds to 18 units of 2^-23 of itself: within 2^-18 of
    themselves. Where the sum does not enter (sigmoid, or divided out again) only the last rounding to fp32 is left, 2^-24,
    and for what 64 bits add 2^-40."""
    l = scale * torch.randn((50, E), generator=torch.Generator().manual_seed(E))
    bias = 0.1 * torch.randn((E,), generator=torch.Generator().manual_seed(k))
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            for renorm in (False, True):
                ids, w = w4.moe_select(l.cuda(), k, score, None if b is None else b.cuda(), groups, top, 1, renorm)
                want, ww = oracle.moe_select(l.numpy(), k, score, None if b is None else b.numpy(), groups, top, 1, renorm)
                assert np.array_equal(ids.cpu().numpy(), want)
                off = 2.0 ** -18 if score == "softmax" and not renorm else 2.0 ** -24 + 2.0 ** -40
                assert (np.abs(w.cpu().double().numpy() - ww) <= off * ww + 2.0 ** -149).all(), (score, b is None, renorm)
