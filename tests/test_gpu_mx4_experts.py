"""The experts' FFN on microscaled weights, where results show what happens inside."""
import numpy as np
import pytest
import torch

import bit_weight_only_quantize_amd as w4
import oracle
from mx4_util import bf16, device, integers, matrix

pytestmark = pytest.mark.gpu


def differences(E, D, F, seed):
    """Stacks whose results are sums of small differences of large h: rows 2i and 2i + 1 of gate and up are the same but
    for one code of up, in a group of small scale, and a row of down has the negative of each even code beside it."""
    rng = np.random.default_rng(seed)
    gate, up, down = (list(integers((E,) + s, seed + i, 123, 125)[:2]) for i, s in enumerate(((F, D), (F, D), (D, F))))
    up[1][:, :, -1] = 119
    for c, s in (gate, up):
        c[:, 1::2], s[:, 1::2] = c[:, 0::2], s[:, 0::2]
    up[0][:, 1::2, -1] ^= rng.choice(np.array([1, 2, 3, 0x30], np.uint8), size=(E, F // 2))
    low = down[0] & 15
    down[0] = (low | ((low ^ 8) << 4)).astype(np.uint8)
    return [(c, s, oracle.mx4_values(c, s)) for c, s in (gate, up, down)]


@pytest.mark.parametrize("M,E,k,D,F", [(1, 4, 2, 64, 96), (1, 9, 3, 2080, 160), (11, 16, 2, 64, 544), (26, 4, 2, 96, 288),
                                       (100, 3, 2, 64, 352), (400, 2, 2, 160, 96), (700, 4, 2, 64, 480)])
@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
def test_h_is_kept_to_16_bits(M, E, k, D, F, act):
    """x in whole numbers: sums of gate and up are exact in fp32 (multiples of 2^-9 under 2^13), so h is off by its
    activation, 2^-18 of itself and 2^-22 |g u|, and by its rounding to 16 bits, 2^-16; y by that times down, its sum of F
    products (and k terms) in fp32, and its rounding to bf16. A rounding of h to 8 bits lies far outside."""
    s = differences(E, D, F, M + D)
    rng = np.random.default_rng(F)
    xv = rng.integers(-3, 4, size=(M, D)).astype(np.float64)
    xv[:, -2:] = rng.integers(1, 4, size=(M, 2))                     # the changed codes count
    ids = rng.integers(0, E, size=(M, k)).astype(np.int32)
    w = rng.choice([0.5, 1.0, -1.0, 2.0], size=(M, k))
    y = w4.mx4_moe(*(device(c, sc) for c, sc, _ in s), bf16(xv).cuda(), torch.from_numpy(ids).cuda(),
                   torch.from_numpy(w).float().cuda(), act).cpu().double().numpy()
    want, rough, bound = np.zeros((3, M, D))
    for m in range(M):
        for e, p in zip(ids[m], w[m]):
            gate, up, down = (v[e] for _, _, v in s)
            assert (np.abs(gate) @ np.abs(xv[m])).max() < 2 ** 13 and (np.abs(up) @ np.abs(xv[m])).max() < 2 ** 13
            g, u = gate @ xv[m], up @ xv[m]
            h = oracle.gated(g, u, act)
            dh = 2.0 ** -18 * np.abs(h) + 2.0 ** -22 * np.abs(g * u) + 2.0 ** -16 * np.abs(h)
            a = np.abs(down)
            want[m] += p * (down @ h)
            rough[m] += p * (down @ bf16(h).double().numpy())
            bound[m] += abs(p) * (a @ dh + (F + k + 2) * 2.0 ** -23 * (a @ (np.abs(h) + dh)))
    bound += 2.0 ** -8 * (np.abs(want) + bound)
    assert (np.abs(y - want) <= bound).all()
    far = np.abs(rough - want) > bound                   # the test can tell
    assert far.mean() > 0.25, far.mean()


@pytest.mark.parametrize("M,E,k,D,F", [(20, 16, 2, 64, 4352), (20, 16, 2, 64, 4384), (20, 16, 2, 8960, 64), (20, 16, 2, 8992, 64),
                                       (50, 8, 2, 64, 2048), (50, 8, 2, 64, 2080), (50, 8, 2, 4352, 32), (30, 4, 2, 608, 288),
                                       (1, 4, 8, 64, 4096), (1, 4, 8, 64, 4128), (20, 16, 2, 64, 8960), (20, 16, 2, 64, 8992),
                                       (50, 8, 2, 64, 4352), (50, 8, 2, 64, 4384), (20, 16, 2, 96, 8480)])
def test_rows_at_the_ends_of_lds(M, E, k, D, F):
    """The longest rows of x, and of both pieces of h, that tiles of 8 and 16 rows and single tokens hold
    in LDS, and the next longer ones, which take another way."""
    s = [matrix((E,) + z, M + i, std=1 / z[1] ** 0.5) for i, z in enumerate(((F, D), (F, D), (D, F)))]
    g = torch.Generator().manual_seed(F)
    x = torch.randn((M, D), generator=g).to(torch.bfloat16)
    ids = torch.randint(0, E, (M, k), generator=g, dtype=torch.int32)
    w = torch.randn((M, k), generator=g)
    y = w4.mx4_moe(*(device(c, sc) for c, sc, _ in s), x.cuda(), ids.cuda(), w.cuda(), "silu").cpu().double().numpy()
    want, bound = oracle.mx4_moe(*(v for _, _, v in s), x.double().numpy(), ids.numpy(), w.double().numpy(), "silu")
    assert (np.abs(y - want) <= bound).all()


@pytest.mark.parametrize("M", [1, 20, 700])
def test_the_ends_of_large_stacks(M):
    """Stacks past 2^32 code bytes, zero but for the last expert's last rows; tolerances of what is rounded: gate and up, sums of
    96 products that are not zero (2^-23 each), the activation (slope under 1.13, 2^-18 of itself and 2^-22 |g u|), h to 16 bits, y
    to bf16."""
    E, F, D = 70, 2048, 65536
    q = [w4.empty_quantized("mx4_g32", *s, num_experts=E) for s in ((F, D), (F, D), (D, F))]
    for m in q:
        m.codes.zero_()
        m.scale.fill_(127)
    gc, gs, gv = integers((2, D), 1, 120, 121)
    for m in q[:2]:
        m.codes[E - 1, F - 2:] = torch.from_numpy(gc).cuda()
        m.scale[E - 1, F - 2:] = torch.from_numpy(gs).cuda()
    q[2].codes[E - 1, D - 1, F // 2 - 1] = 0x22          # 1 times the last two h
    x = torch.zeros((M, D), dtype=torch.bfloat16)
    x[:, :96] = torch.randn((M, 96), generator=torch.Generator().manual_seed(M)).to(torch.bfloat16)
    ids = torch.full((M, 2), E - 1, dtype=torch.int32)
    y = w4.mx4_moe(*q, x.cuda(), ids.cuda(), torch.full((M, 2), 0.5).cuda()).cpu().double()
    xv = x[:, :96].double().numpy()
    g = xv @ gv[:, :96].T
    off = 96 * 2.0 ** -23 * (np.abs(xv) @ np.abs(gv[:, :96].T))
    h = oracle.gated(g, g, "gelu_tanh")
    dh = 1.13 * off * (np.abs(g) + off) + np.abs(g) * off + 2.0 ** -18 * np.abs(h) + 2.0 ** -22 * g * g + 2.0 ** -16 * np.abs(h)
    want, bound = h.sum(1), (dh + 2.0 ** -21 * np.abs(h)).sum(1)
    assert (np.abs(y[:, D - 1].numpy() - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound)).all()
    assert not bool(y[:, :D - 1].any())
