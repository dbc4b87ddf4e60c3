"""The microscaled calls at the largest sizes that they take: as many rows as a matrix has, tokens as a selection, pairs as
the experts' FFN. Inputs repeat themselves; so must results."""
import numpy as np
import pytest
import torch

import bit_weight_only_quantize_amd as w4
import oracle
from mx4_util import bf16, device, integers, product

pytestmark = pytest.mark.gpu


def test_one_row_times_the_most_rows():
    K, N, rows = 32, 1 << 26, 1024
    wc, ws, wv = integers((rows, K), 1)
    xc, xs, xv = integers((1, K), 2)
    want, _ = product(xv, wv)
    small = device(wc, ws)
    W = w4.QuantizedMatrix("mx4_g32", N, K, small.codes.repeat(N // rows, 1), small.scale.repeat(N // rows, 1), None)
    y = w4.mx4_gemm(W, bf16(xv).cuda(), dtype=torch.float32)
    assert torch.equal(y[0, :rows].cpu().double(), want[0])
    assert bool((y.view(-1, rows) == y[0, :rows]).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_most_tokens_of_a_selection(dtype):
    M, E, rows = 1 << 26, 3, 1 << 12
    l = torch.randn((rows, E), generator=torch.Generator().manual_seed(1)).to(dtype)
    ids, w = w4.moe_select(l.cuda().repeat(M // rows, 1), 2, "sigmoid", renormalize=True)
    wi, ww = oracle.moe_select(l.double().numpy(), 2, "sigmoid", renormalize=True)
    assert np.array_equal(ids[:rows].cpu().numpy(), wi)
    assert np.abs(w[:rows].cpu().double().numpy() - ww).max() < 2.0 ** -22
    assert bool((ids.view(-1, rows, 2) == ids[:rows]).all()) and bool((w.view(-1, rows, 2) == w[:rows]).all())


def test_the_most_pairs_of_the_experts():
    M, E, D, F, rows = 1 << 24, 2, 32, 32, 1 << 12
    q = [device(*integers((E,) + s, i, 121, 123)[:2]) for i, s in enumerate(((F, D), (F, D), (D, F)))]
    g = torch.Generator().manual_seed(3)
    x = torch.randn((rows, D), generator=g).to(torch.bfloat16).cuda()
    ids = torch.randint(0, E, (rows, 1), generator=g, dtype=torch.int32).cuda()
    p = torch.rand((rows, 1), generator=g).cuda()
    few = w4.mx4_moe(*q, x, ids, p)                      # the same kernels: over 1000 pairs an expert
    assert bool(few.isfinite().all()) and bool(few.any())
    n = M // rows
    y = w4.mx4_moe(*q, x.repeat(n, 1), ids.repeat(n, 1), p.repeat(n, 1))
    assert bool((y.view(n, rows, D) == few).all())
