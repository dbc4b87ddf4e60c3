"""Every kernel of the microscaled products and experts, over several rounds of its stages, blocks of columns and pieces of
K. tests/test_mx4_plan_cpu.py asserts that these sizes reach them."""
import numpy as np
import pytest
import torch

import bit_weight_only_quantize_amd as w4
import oracle
from mx4_plan_util import BLOCKS, WAYS
from mx4_util import device, matrix

pytestmark = pytest.mark.gpu
GRID = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def random_matrix(N, K, seed):
    """Codes of all kinds with scales 1/2, 1 and 2: the library's matrix and its values in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(126, 129, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    v = GRID.cuda()[torch.stack((c & 15, c >> 4), -1).int().flatten(-2)]
    v = v * torch.pow(2.0, s.double() - 127).repeat_interleave(32, -1)
    return w4.QuantizedMatrix("mx4_g32", N, K, c, s, None), v


@pytest.mark.parametrize("case", BLOCKS, ids=lambda c: "-".join(str(int(v)) for v in c))
def test_products_are_exact_in_every_block(case):
    """Products are multiples of 2^-4, and sums of magnitudes lie under 2^20, so that fp32 sums in any order are exact."""
    x4, M, N, K, ws = case
    W, wv = random_matrix(N, K, M)
    X, xv = random_matrix(M, K, N)
    assert float((xv.abs() @ wv.abs().t().contiguous()).max()) < 2 ** 20
    want = xv @ wv.t().contiguous()
    x = X if x4 else xv.to(torch.bfloat16)
    workspace = None if ws else torch.empty(0, dtype=torch.uint8, device="cuda")
    y = torch.full((M, N + 1), -5.0, device="cuda")
    w4.mx4_gemm(W, x, out=y[:, :N], workspace=workspace)
    assert torch.equal(y[:, :N].double(), want) and bool((y[:, N] == -5).all())
    h = w4.mx4_gemm(W, x, workspace=workspace)
    assert torch.equal(h, want.float().to(torch.bfloat16))


@pytest.mark.parametrize("skewed", [False, True])
@pytest.mark.parametrize("case", WAYS, ids=lambda c: "-".join(map(str, c)))
def test_experts_in_every_way(case, skewed):
    """Idle slots and tokens; skewed: nearly all pairs with one expert, some experts with one pair or none."""
    M, E, k, D, F = case
    s = [matrix((E,) + z, M + i, std=1 / z[1] ** 0.5) for i, z in enumerate(((F, D), (F, D), (D, F)))]
    g = torch.Generator().manual_seed(D)
    x = torch.randn((M, D), generator=g).to(torch.bfloat16)
    ids = torch.randint(0, E, (M, k), generator=g, dtype=torch.int32)
    if skewed:
        ids = torch.where(torch.rand((M, k), generator=g) < 0.99, 1, ids).to(torch.int32)
    ids[torch.rand((M, k), generator=g) < 0.05] = -1
    if M > 3:
        ids[3] = -1
    w = torch.randn((M, k), generator=g)
    y = torch.full((M, D + 8), -5.0, dtype=torch.bfloat16, device="cuda")
    q = [device(c, sc) for c, sc, _ in s]
    ws = w4.mx4_moe_workspace(*q, M, k)
    ws.fill_(0xFF)
    w4.mx4_moe(*q, x.cuda(), ids.cuda(), w.cuda(), "silu", out=y[:, :D], workspace=ws)
    got = y.cpu().double().numpy()
    want, bound = oracle.mx4_moe(*(v for _, _, v in s), x.double().numpy(), ids.numpy(), w.double().numpy(), "silu")
    assert (np.abs(got[:, :D] - want) <= bound).all() and (got[:, D:] == -5).all()
    if M > 3:
        assert not got[3, :D].any()


@pytest.mark.parametrize("x4", [False, True])
@pytest.mark.parametrize("M", [1, 6, 40, 300])
def test_weights_past_the_range_of_bf16(M, x4):
    """Codes 4 and 6 at scale byte 253, and 2 to 6 at 254, are 2^128 and more: infinite beside bf16 X, so that their column of Y is
    infinite or NaN and no other one is touched; exact beside 4 bits. Smaller codes there are like any others. K ends inside a step."""
    N, K = 70, 224
    W, wv = random_matrix(N, K, 1)
    X, xv = random_matrix(M, K, 2)
    W.scale[:8, 3], X.scale[:, 3] = 127, 40              # 2^-87
    wide = torch.tensor([4, 6, 2, 3, 4, 6, 1.5, 0.5], dtype=torch.float64)
    at = torch.tensor([253, 253, 254, 254, 254, 254, 254, 253], dtype=torch.uint8)
    W.scale[:8, 3] = at.cuda()
    W.codes[:8, 48:64] = 0
    W.codes[:8, 50] = torch.tensor([(GRID[:8] == v).nonzero().item() for v in wide], dtype=torch.uint8).cuda()
    wv[:8, 96:128] = 0
    wv[:8, 100] = (wide * torch.pow(2.0, at.double() - 127)).cuda()
    xv[:, 96:128] *= torch.pow(2.0, 40 - 127.0 - (random_matrix(M, K, 2)[0].scale[:, 3:4].double() - 127))
    want = xv @ wv.t().contiguous()
    y = w4.mx4_gemm(W, X if x4 else xv.to(torch.bfloat16), dtype=torch.float32).double()
    first = 0 if x4 else 6
    assert bool(((y[:, first:] - want[:, first:]).abs() <= K * 2.0 ** -23 * (xv.abs() @ wv[first:].abs().t().contiguous())).all())
    if not x4:
        assert not bool(y[:, :6].isfinite().any())
