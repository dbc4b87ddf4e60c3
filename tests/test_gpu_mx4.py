"""The microscaled 4-bit format on the GPU: quantization and read-back bit for bit, products exactly where fp32
sums are exact and within the sums' bound elsewhere, the selection of experts, and their FFN."""
import numpy as np
import pytest
import torch

import bit_weight_only_quantize_amd as w4
import oracle
from mx4_util import DT, bf16, device, integers, matrix, product, strided

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- rows
def special_rows(K, dtype):
    """Rows over the whole range of the type: ties, borders, zeros, the ends, infinities and NaN."""
    rng = np.random.default_rng(K)
    x = rng.normal(size=(40, K)) * np.exp2(rng.integers(-130, 120, size=(40, 1)).astype(np.float64))
    ties = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, 7.9])
    x[0, :10], x[1, :10], x[2, :10] = ties, -ties * 2.0 ** 100, ties * 2.0 ** -126
    x[0, 10:], x[1, 10:] = 0, 0
    x[3] = 0
    x[4] = -0.0
    x[5, 0], x[5, 1:] = 2.0 ** -149, 0
    x[6] = 3e38
    t = torch.from_numpy(x.astype(np.float32)).to(DT[dtype])
    t[7, K - 1], t[8, 3], t[9, 0] = float("inf"), float("nan"), float("-inf")
    lo = torch.finfo(DT[dtype]).min
    t[10], t[11, 1] = lo, -lo
    return t


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K,slack", [(32, 0), (96, 8), (2048, 0), (4128, 40)])
def test_quantize_and_read_bit_for_bit(K, slack, dtype):
    t = special_rows(K, dtype)
    x = strided(t, slack)
    q = w4.mx4_quantize(x)
    c, s = oracle.mx4_quantize(t.double().numpy())
    assert np.array_equal(q.scale.cpu().numpy(), s)
    assert np.array_equal(q.codes.cpu().numpy(), c)
    v = torch.from_numpy(oracle.mx4_values(c, s))
    for out in ("f32", "bf16"):
        back = torch.full((40, K + 16), -5.0, dtype=DT[out], device="cuda")
        w4.mx4_read(q, out=back[:, :K])
        got = back.cpu()
        assert torch.equal(got[:, K:], torch.full((40, 16), -5.0, dtype=DT[out]))       # nothing beside the rows
        want = v.to(DT[out])
        assert torch.equal(got[:, :K].isnan(), want.isnan())
        assert torch.equal(got[:, :K].nan_to_num(7), want.nan_to_num(7))


def test_read_every_code_at_every_scale():
    c = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    q = device(c, s)
    v = torch.from_numpy(oracle.mx4_values(c, s))
    for dt in (torch.float32, torch.bfloat16):
        got, want = w4.mx4_read(q, dt).cpu(), v.to(dt)
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(7), want.nan_to_num(7))


@pytest.mark.parametrize("rows", [1, 5, 257])
def test_quantize_pack_takes_the_scheme(rows):
    x = np.random.default_rng(rows).normal(size=(rows, 160)).astype(np.float32)
    q = w4.quantize_pack(torch.from_numpy(x).cuda(), "mx4_g32")
    c, s = oracle.mx4_quantize(x)
    assert np.array_equal(q.codes.cpu().numpy(), c) and np.array_equal(q.scale.cpu().numpy(), s)
    stack = w4.empty_quantized("mx4_g32", rows, 160, num_experts=3)
    for e in range(3):
        w4.quantize_pack(torch.from_numpy(x * 2 ** e).cuda(), "mx4_g32", out=stack, expert=e)
    assert np.array_equal(stack.codes.cpu().numpy(), np.stack([c] * 3))
    assert np.array_equal(stack.scale.cpu().numpy(), np.stack([s, s + 1, s + 2]))


# ---------------------------------------------------------------- products
SIZES = [(1, 1, 32), (1, 16, 64), (1, 37, 4096), (2, 130, 96), (5, 257, 416), (7, 64, 11008), (16, 100, 2048), (17, 96, 160),
         (31, 500, 1056), (33, 64, 2080), (64, 1000, 512), (65, 129, 1024), (100, 300, 4096), (128, 256, 64), (129, 128, 128), (255, 257, 96),
         (257, 385, 608), (333, 640, 2048), (600, 1100, 1312)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("x4", [False, True])
def test_product_is_exact_where_sums_are(M, N, K, x4):
    """Codes with scales of three binades are multiples of 2^-2, so products are multiples of 2^-4; fp32 holds every
    such number under 2^20, which the sums of magnitudes, and so all partial sums in any order, stay below."""
    wc, ws, wv = integers((N, K), 7 * M + N)
    xc, xs, xv = integers((M, K), K + M)
    want, size = product(xv, wv)
    assert float(size.max()) < 2 ** 20
    W = device(wc, ws)
    X = device(xc, xs) if x4 else strided(bf16(xv), 8 if M % 2 else 0)
    Y = torch.full((M, N + 3), -5.0, device="cuda")
    w4.mx4_gemm(W, X, out=Y[:, :N])
    got = Y.cpu()
    assert torch.equal(got[:, N:], torch.full((M, 3), -5.0))
    assert torch.equal(got[:, :N].double(), want)
    # without a workspace, and rounded once to bf16
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    assert torch.equal(w4.mx4_gemm(W, X, dtype=torch.float32, workspace=none).cpu().double(), want)
    assert torch.equal(w4.mx4_gemm(W, X).cpu(), want.float().to(torch.bfloat16))


@pytest.mark.parametrize("M,N,K", [(1, 300, 4096), (9, 200, 2048), (40, 256, 1024), (300, 384, 4096)])
@pytest.mark.parametrize("x4", [False, True])
def test_product_of_real_weights(M, N, K, x4):
    """Sums of K exact products in fp32: at most K additions, each off by 2^-23 of the sum of magnitudes."""
    wc, ws, wv = matrix((N, K), N)
    rng = np.random.default_rng(M)
    x = bf16(rng.normal(size=(M, K)) * np.exp(rng.normal(size=(M, 1))))
    xv = x.double().numpy()
    X = x.cuda()
    if x4:
        X = w4.mx4_quantize(X)
        xv = oracle.mx4_values(*oracle.mx4_quantize(xv))
    want, size = product(xv, wv)
    got = w4.mx4_gemm(device(wc, ws), X, dtype=torch.float32).cpu().double()
    bound = K * 2.0 ** -23 * size
    assert bool(((got - want).abs() <= bound).all())
    # and, as rounding errors have either sign, far inside on the whole
    assert float((got - want).norm() / want.norm()) < 2e-6
    half = w4.mx4_gemm(device(wc, ws), X).cpu().double()
    assert bool(((half - want).abs() <= bound + 2.0 ** -8 * (want.abs() + bound)).all())


@pytest.mark.parametrize("M", [1, 20, 300])
def test_product_of_one_sign(M):
    """All products positive: the sum is as large as the sum of magnitudes, and fp32 sums of K terms in
    pieces stay within K 2^-23 of it."""
    K, N = 4096, 160
    c = np.random.default_rng(M).integers(1, 8, size=(N, K))
    wc = (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)
    ws = np.full((N, K // 32), 127, np.uint8)
    x = bf16(np.abs(np.random.default_rng(1).normal(size=(M, K))) + 0.01)
    want, _ = product(x.double().numpy(), oracle.mx4_values(wc, ws))
    got = w4.mx4_gemm(device(wc, ws), x.cuda(), dtype=torch.float32).cpu().double()
    assert bool(((got - want).abs() <= K * 2.0 ** -23 * want).all())


@pytest.mark.parametrize("M", [1, 6, 40, 300])
@pytest.mark.parametrize("x4", [False, True])
def test_extreme_scales_and_non_finite_rows(M, x4):
    """Scales from 2^-100 to 2^103; a NaN scale of W makes its column NaN, one of X (or a NaN in X) its row, and nothing else."""
    N, K = 70, 128
    wc, ws, _ = integers((N, K), 1)
    xc, xs, _ = integers((M, K), 2)
    ws[0], xs[0] = 27, 225
    ws[1] = 230
    wv, xv = oracle.mx4_values(wc, ws), oracle.mx4_values(xc, xs)
    X = device(xc, xs) if x4 else bf16(xv).cuda()
    got = w4.mx4_gemm(device(wc, ws), X, dtype=torch.float32).cpu()
    with np.errstate(over="ignore"):
        want = torch.from_numpy((xv @ wv.T).astype(np.float32))
    if M > 1:                                            # row 0 times column 1 passes fp32: infinite or NaN there
        assert torch.equal(got[1:], want[1:])
    assert torch.equal(got[0, :1], want[0, :1]) and torch.equal(got[0, 2:], want[0, 2:])
    ws[3, 2] = 255
    wd = device(wc, ws)
    got = w4.mx4_gemm(wd, X, dtype=torch.float32).cpu()
    assert bool(got[:, 3].isnan().all()) and torch.equal(got[1:, 4:], want[1:, 4:])
    if M > 1:
        if x4:
            X.scale[M - 1, 1] = 255
        else:
            X[M - 1, 33] = float("nan")
        got = w4.mx4_gemm(wd, X, dtype=torch.float32).cpu()
        assert bool(got[M - 1].isnan().all()) and torch.equal(got[1:M - 1, 4:], want[1:M - 1, 4:])


def test_products_of_nothing():
    W = device(*integers((8, 64), 1)[:2])
    assert w4.mx4_gemm(W, torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")).shape == (0, 8)
    E = w4.empty_quantized("mx4_g32", 0, 64)
    assert w4.mx4_gemm(E, torch.ones((3, 64), dtype=torch.bfloat16, device="cuda")).shape == (3, 0)
    assert w4.mx4_gemm(W, E).shape == (0, 8)
    assert w4.mx4_quantize(torch.empty((0, 64), device="cuda")).N == 0
    assert w4.mx4_read(E).shape == (0, 64)


# ---------------------------------------------------------------- selection
def logits_of(M, E, kind, seed):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn((M, E), generator=g) * 2
    if kind == "ties":
        l = torch.randint(-3, 4, (M, E), generator=g).float()
    if kind == "bf16":
        l = l.to(torch.bfloat16)
    if kind == "masked":
        l[torch.rand((M, E), generator=g) < 0.7] = float("-inf")
        l[0] = float("-inf")
        l[1, 1:] = float("-inf")
    if kind == "lowest":                                 # a mask by the type's lowest value
        l[torch.rand((M, E), generator=g) < 0.5] = torch.finfo(torch.float32).min
    if kind == "close":                                  # scores within an ulp of fp32 of each other
        l = 3 + torch.randint(0, 40, (M, E), generator=g).float() * 2.0 ** -22
    if kind == "wide":
        l = l * 60
    return l


SELECT = [dict(E=128, k=8), dict(E=8, k=1), dict(E=1, k=1), dict(E=60, k=4, groups=4, top=2), dict(E=64, k=6, groups=8, top=3),
          dict(E=256, k=8, groups=8, top=4, best=2), dict(E=160, k=6, groups=8, top=3, best=1), dict(E=96, k=12, groups=2, top=1, best=2),
          dict(E=512, k=32, groups=64, top=32, best=2), dict(E=1024, k=32), dict(E=33, k=33 - 1), dict(E=24, k=3, groups=8, top=1), dict(E=72, k=9, groups=8, top=8)]


@pytest.mark.parametrize("kind", ["normal", "ties", "bf16", "masked", "lowest", "close", "wide"])
@pytest.mark.parametrize("s", SELECT, ids=lambda s: "-".join(f"{a}{b}" for a, b in s.items()))
def test_selection(s, kind):
    """Ids equal; weights (formula in fp32 or more) within 2^-18 of themselves: exp of a rounded difference |d| <= 200 is off by
    200 * 2^-24, the sum by 1024 * 2^-24, ties of neither sign."""
    E, k, G = s["E"], s["k"], s.get("groups", 1)
    how = dict(groups=G, top_groups=s.get("top", 1), group_best=s.get("best", 1))
    l = logits_of(37, E, kind, E + k)
    bias = torch.randn((E,), generator=torch.Generator().manual_seed(E)) * 0.3
    if kind == "close":
        bias = bias.sign() * 2.0 ** -24
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            for renorm in (False, True):
                x = strided(l, 5 if renorm else 0)
                ids, w = w4.moe_select(x, k, score, None if b is None else b.cuda(), renormalize=renorm, scale=2.5, **how)
                want, ww = oracle.moe_select(l.double().numpy(), k, score, None if b is None else b.double().numpy(),
                                             renormalize=renorm, scale=2.5, **how)
                assert np.array_equal(ids.cpu().numpy(), want), (score, b is None, renorm)
                got = w.cpu().double().numpy()
                assert (np.abs(got - ww) <= 2.0 ** -12 * np.abs(ww) * (kind == "wide") + 2.0 ** -18 * np.abs(ww) + 1e-37).all(), \
                    (score, b is None, renorm, np.abs(got - ww).max())


def test_selection_of_nan_and_infinity():
    l = torch.randn((6, 64), generator=torch.Generator().manual_seed(0))
    l[0, 5], l[1, 7], l[2] = float("nan"), float("inf"), float("nan")
    for score in ("softmax", "sigmoid"):
        for groups in (1, 8):
            ids, w = w4.moe_select(l.cuda(), 8, score, groups=groups, top_groups=max(1, groups // 4))
            ids, w = ids.cpu(), w.cpu()
            assert bool(w[0].isnan().all()) and bool(w[2].isnan().all()) and bool(w[3:].isfinite().all())
            assert ids[1, 0] == 7
            for r in range(6):                           # always distinct experts in range
                assert len(set(ids[r].tolist())) == 8 and 0 <= int(ids[r].min()) and int(ids[r].max()) < 64


def test_selection_agrees_with_the_softmax_router():
    """Without options it selects what moe_route selects, and its weights are the same to fp32's rounding."""
    W = torch.randn((128, 256), generator=torch.Generator().manual_seed(1)).cuda() * 0.05
    router = w4.quantize_pack(W, "aff8_g64")
    x = torch.randn((50, 256), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    ids, w, logits = w4.moe_route(router, x, 8)
    ids2, w2 = w4.moe_select(logits, 8)
    assert torch.equal(ids, ids2) and bool(((w - w2).abs() <= 2.0 ** -17 * w).all())


# ---------------------------------------------------------------- experts
def stacks(E, D, F, seed):
    s = [matrix((E, F, D), seed, std=0.5 / D ** 0.5), matrix((E, F, D), seed + 1, std=1 / D ** 0.5), matrix((E, D, F), seed + 2, std=1 / F ** 0.5)]
    return [device(c, sc) for c, sc, _ in s], [v for _, _, v in s]


EXPERTS = [(1, 4, 2, 64, 32), (1, 8, 8, 2048, 96), (2, 8, 3, 128, 64), (5, 16, 4, 96, 160), (17, 3, 2, 256, 96), (40, 4, 2, 320, 64),
           (64, 8, 8, 128, 128), (150, 2, 1, 160, 96), (300, 5, 3, 96, 32), (700, 4, 2, 64, 64)]


@pytest.mark.parametrize("M,E,k,D,F", EXPERTS)
@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
def test_experts(M, E, k, D, F, act):
    q, v = stacks(E, D, F, M + E)
    g = torch.Generator().manual_seed(M)
    x = torch.randn((M, D), generator=g).to(torch.bfloat16)
    ids = torch.randint(0, E, (M, k), generator=g, dtype=torch.int32)     # the same expert twice among them
    ids[torch.rand((M, k), generator=g) < 0.1] = -1
    if M > 3:
        ids[1] = -1                                                       # a token without any
        ids[2, 0] = E
        ids[3, 0] = 1 << 30
    w = torch.randn((M, k), generator=g)
    y = torch.full((M, D + 8), -5.0, dtype=torch.bfloat16, device="cuda")
    ws = w4.mx4_moe_workspace(*q, M, k)
    ws.fill_(0xFF)                                                        # NaN wherever nothing is written
    w4.mx4_moe(*q, strided(x, 8 if M % 2 else 0), ids.cuda(), w.cuda(), act, out=y[:, :D], workspace=ws)
    got = y.cpu().double()
    assert bool((got[:, D:] == -5).all())
    want, bound = oracle.mx4_moe(*v, x.double().numpy(), ids.numpy(), w.double().numpy(), act)
    err = np.abs(got[:, :D].numpy() - want)
    assert (err <= bound).all(), float((err / np.maximum(bound, 1e-300)).max())
    if M > 3:
        assert not got[1, :D].any()


def test_experts_read_only_the_chosen():
    """Stacks whose other experts hold NaN; a token's result does not depend on the others' rows."""
    E, D, F = 6, 128, 64
    q, v = stacks(E, D, F, 3)
    for m in q:
        m.scale[4] = 255
    x = torch.randn((50, D), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    x[7] = float("nan")
    ids = torch.randint(0, 4, (50, 2), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    w = torch.rand((50, 2), generator=torch.Generator().manual_seed(2))
    y = w4.mx4_moe(*q, x.cuda(), ids.cuda(), w.cuda()).cpu()
    assert bool(y[7].isnan().all()) and bool(y[:7].isfinite().all()) and bool(y[8:].isfinite().all())
    x[7] = 1.0
    ids[9, 0] = 4
    z = w4.mx4_moe(*q, x.cuda(), ids.cuda(), w.cuda()).cpu()
    assert bool(z[9].isnan().all()) and torch.equal(z[10:], y[10:]) and torch.equal(z[:7], y[:7])


def test_a_layer_as_it_is_used():
    """Router logits from a 4-bit product, the selection, the experts and a dense projection of their sum."""
    M, E, k, D, F = 33, 16, 4, 128, 96
    q, v = stacks(E, D, F, 11)
    rc, rs, rv = matrix((E, D), 5, std=0.2)
    oc, os_, ov = matrix((64, D), 6)
    x = torch.randn((M, D), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    bias = 0.05 * torch.randn((E,), generator=torch.Generator().manual_seed(4))
    logits = w4.mx4_gemm(device(rc, rs), x.cuda(), dtype=torch.float32)
    ids, w = w4.moe_select(logits, k, "sigmoid", bias.cuda(), groups=4, top_groups=2, group_best=2, renormalize=True, scale=1.5)
    y = w4.mx4_moe(*q, x.cuda(), ids, w, "silu")
    z = w4.mx4_gemm(device(oc, os_), w4.mx4_quantize(y), dtype=torch.float32)
    wi, ww = oracle.moe_select(logits.cpu().double().numpy(), k, "sigmoid", bias.double().numpy(), 4, 2, 2, True, 1.5)
    assert np.array_equal(ids.cpu().numpy(), wi)
    want, bound = oracle.mx4_moe(*v, x.double().numpy(), wi, w.cpu().double().numpy(), "silu")
    assert (np.abs(y.cpu().double().numpy() - want) <= bound).all()
    yq = oracle.mx4_values(*oracle.mx4_quantize(y.cpu().double().numpy()))
    wz, size = product(yq, ov)
    assert bool(((z.cpu().double() - wz).abs() <= D * 2.0 ** -23 * size).all())


# ---------------------------------------------------------------- streams, graphs, repeats
def all_calls(M=40):
    E, D, F, k = 8, 256, 96, 3
    q, _ = stacks(E, D, F, 21)
    W = device(*matrix((200, D), 8)[:2])
    g = torch.Generator().manual_seed(M)
    x = torch.randn((M, D), generator=g).to(torch.bfloat16).cuda()
    logits = torch.randn((M, E), generator=g).cuda()
    xq = w4.empty_quantized("mx4_g32", M, D)
    s = dict(x=x, logits=logits, xq=xq, ids=torch.zeros((M, k), dtype=torch.int32, device="cuda"),
             w=torch.zeros((M, k), device="cuda"), y=torch.empty((M, 200), device="cuda"), y4=torch.empty((M, 200), device="cuda"),
             back=torch.empty((M, D), device="cuda"), z=torch.empty((M, D), dtype=torch.bfloat16, device="cuda"),
             ws=w4.mx4_gemm_workspace(W, M), ws4=w4.mx4_gemm_workspace(W, M, True), mw=w4.mx4_moe_workspace(*q, M, k))

    def run():
        w4.mx4_quantize(s["x"], out=s["xq"])
        w4.mx4_read(s["xq"], out=s["back"])
        w4.mx4_gemm(W, s["x"], out=s["y"], workspace=s["ws"])
        w4.mx4_gemm(W, s["xq"], out=s["y4"], workspace=s["ws4"])
        w4.moe_select(s["logits"], k, groups=4, top_groups=2, ids=s["ids"], weights=s["w"])
        w4.mx4_moe(*q, s["x"], s["ids"], s["w"], out=s["z"], workspace=s["mw"])
        return [s[n].clone() for n in ("back", "y", "y4", "ids", "w", "z")] + [s["xq"].codes.clone()]
    return s, run


@pytest.mark.parametrize("M", [1, 40, 300])
def test_captured_and_on_another_stream(M):
    s, run = all_calls(M)
    eager = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(eager, other):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed in (1, 2, 3):                               # new inputs in the same buffers
        s["x"].copy_(torch.randn(s["x"].shape, generator=torch.Generator().manual_seed(seed)))
        s["logits"].copy_(torch.randn(s["logits"].shape, generator=torch.Generator().manual_seed(seed + 9)))
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in out]
        for a, b in zip(replayed, run()):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_the_same_bits_every_time(M):
    _, run = all_calls(M)
    first = run()
    for _ in range(5):
        for a, b in zip(first, run()):
            assert torch.equal(a, b)


def test_binding_refuses():
    W = device(*integers((8, 64), 1)[:2])
    x = torch.ones((3, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (x.float(), x.cpu(), x[:, ::2], x[:, :32], x[0]):
        with pytest.raises((ValueError, IndexError)):
            w4.mx4_gemm(W, bad)
    with pytest.raises(ValueError):
        w4.mx4_gemm(W, x, out=torch.empty((3, 9), device="cuda"))
    with pytest.raises(ValueError):
        w4.mx4_gemm(w4.QuantizedMatrix("mx4_g32", 9, 64, W.codes, W.scale, None), x)
    with pytest.raises(ValueError):
        w4.mx4_gemm(w4.empty_quantized("aff4_g64", 8, 64), x)
    with pytest.raises(ValueError):
        w4.mx4_quantize(x, out=w4.empty_quantized("mx4_g32", 4, 64))
    with pytest.raises(w4.W4Error):
        w4.mx4_quantize(torch.ones((3, 48), device="cuda"))
    l = torch.zeros((3, 16), device="cuda")
    for kw in (dict(score="tanh"), dict(bias=torch.zeros(15, device="cuda")), dict(ids=torch.zeros((3, 2), device="cuda")),
               dict(weights=torch.zeros((3, 4), device="cuda"))):
        with pytest.raises(ValueError):
            w4.moe_select(l, 2, **kw)
    with pytest.raises(w4.W4Error):
        w4.moe_select(l, 17)
    q, _ = stacks(4, 64, 32, 1)
    ids, w = torch.zeros((3, 2), dtype=torch.int32, device="cuda"), torch.zeros((3, 2), device="cuda")
    for a in ((x, ids.long(), w), (x, ids, w.double()), (x, ids[:2], w), (x.float(), ids, w), (x, ids, w[:, :1])):
        with pytest.raises(ValueError):
            w4.mx4_moe(*q, *a)
    with pytest.raises(ValueError):
        w4.mx4_moe(*q, x, ids, w, act="relu")
    with pytest.raises(w4.W4Error):
        w4.mx4_moe(*q, x, ids, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


# ---------------------------------------------------------------- far ends, calls side by side
@pytest.mark.parametrize("x4", [False, True])
@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_weights_past_4_gib(M, x4):
    """Only the last rows of a matrix of more than 2^32 code bytes are not zero."""
    K, N = 65536, (1 << 17) + 19
    W = w4.QuantizedMatrix("mx4_g32", N, K, torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda"),
                           torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda"), None)
    c, s, v = integers((3, K), 5)
    W.codes[N - 3:] = torch.from_numpy(c).cuda()
    W.scale[N - 3:] = torch.from_numpy(s).cuda()
    xc, xs, xv = integers((M, K), M, 127, 128)
    xc[:, 64:], xv[:, 128:] = 0, 0                       # few enough products that fp32 holds every partial sum
    y = w4.mx4_gemm(W, device(xc, xs) if x4 else bf16(xv).cuda(), dtype=torch.float32)
    want, _ = product(xv, v)
    assert torch.equal(y[:, N - 3:].cpu().double(), want)
    assert not bool(y[:, :N - 3].any())


@pytest.mark.parametrize("M", [1, 20, 700])
def test_stacks_past_4_gib(M):
    E, F, D = 70, 2048, 65536
    q = [w4.empty_quantized("mx4_g32", *s, num_experts=E) for s in ((F, D), (F, D), (D, F))]
    for m in q:
        m.codes.zero_()
        m.scale.fill_(127)
    gc, gs, gv = integers((2, D), 1, 120, 121)
    for m in q[:2]:                                      # the last expert's last two rows of h
        m.codes[E - 1, F - 2:] = torch.from_numpy(gc).cuda()
        m.scale[E - 1, F - 2:] = torch.from_numpy(gs).cuda()
    q[2].codes[E - 1, D - 1, F // 2 - 1] = 0x22          # 1 times the last two h
    x = torch.zeros((M, D), dtype=torch.bfloat16)
    x[:, :96] = torch.randn((M, 96), generator=torch.Generator().manual_seed(M)).to(torch.bfloat16)
    ids = torch.full((M, 2), E - 1, dtype=torch.int32)
    w = torch.full((M, 2), 0.5)
    y = w4.mx4_moe(*q, x.cuda(), ids.cuda(), w.cuda()).cpu().double()
    g = x[:, :96].double().numpy() @ gv[:, :96].T
    want = oracle.gated(g, g, "gelu_tanh").sum(1)
    size = np.abs(oracle.gated(g, g, "gelu_tanh")).sum(1)
    # h to bf16, parts to bf16, y to bf16, and the activation's 2^-18
    assert (np.abs(y[:, D - 1].numpy() - want) <= 2.0 ** -6 * size + 1e-6).all()
    assert not bool(y[:, :D - 1].any())


def test_calls_side_by_side_on_two_streams():
    """Each with workspaces of its own, over the same weights."""
    runs = [all_calls(M) for M in (40, 300)]
    want = [run() for _, run in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(runs[i][1]())
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            for a, b in zip(want[i], outs):
                assert torch.equal(a, b)


@pytest.mark.parametrize("M", [1, 3, 40])
def test_experts_without_a_usual_shape(M):
    """More columns than LDS holds rows of, more experts than pairs, a token whose experts are all the same, weights of 0
    and large ones, and an output row stride that is no multiple of 16 bytes."""
    E, D, F, k = 40, 20480, 32, 2
    q, v = stacks(E, D, F, 5)
    g = torch.Generator().manual_seed(M)
    x = torch.randn((M, D), generator=g).to(torch.bfloat16)
    ids = torch.randint(0, E, (M, k), generator=g, dtype=torch.int32)
    ids[0] = 7
    w = torch.randn((M, k), generator=g) * 100
    w[0, 1] = 0
    y = torch.full((M, D + 3), -5.0, dtype=torch.bfloat16, device="cuda")
    w4.mx4_moe(*q, x.cuda(), ids.cuda(), w.cuda(), "silu", out=y[:, :D])
    want, bound = oracle.mx4_moe(*v, x.double().numpy(), ids.numpy(), w.double().numpy(), "silu")
    got = y.cpu().double().numpy()
    assert (np.abs(got[:, :D] - want) <= bound).all() and (got[:, D:] == -5).all()


def test_pair_counts_at_the_borders_between_ways():
    """One expert gets all pairs, or none, around every number of rows at which another kernel takes over."""
    E, D, F = 2, 64, 32
    q, v = stacks(E, D, F, 9)
    for M in (15, 16, 17, 23, 24, 33, 34, 35, 63, 65, 127, 129, 641, 643):
        x = torch.randn((M, D), generator=torch.Generator().manual_seed(M)).to(torch.bfloat16)
        for e in (0, 1):
            ids = torch.full((M, 1), e, dtype=torch.int32)
            w = torch.ones((M, 1))
            y = w4.mx4_moe(*q, x.cuda(), ids.cuda(), w.cuda()).cpu().double().numpy()
            want, bound = oracle.mx4_moe(*v, x.double().numpy(), ids.numpy(), w.double().numpy(), "gelu_tanh")
            assert (np.abs(y - want) <= bound).all(), (M, e)


@pytest.mark.parametrize("M,K", [(1, 24576), (1, 32768), (2, 14336), (9, 3584), (16, 2016)])
def test_x_at_the_default_size_of_lds(M, K):
    """X takes 48 to 64 KiB of LDS, beside what the kernels hold for themselves."""
    wc, ws, wv = integers((50, K), K, 127, 128)
    xc, xs, xv = integers((M, K), M, 127, 128)
    want, size = product(xv, wv)
    assert float(size.max()) < 2 ** 22                   # multiples of 1/4
    y = w4.mx4_gemm(device(wc, ws), bf16(xv).cuda(), dtype=torch.float32)
    assert torch.equal(y.cpu().double(), want)


@pytest.mark.parametrize("k,F", [(8, 4096), (8, 3104), (32, 1024), (9, 4096)])
def test_experts_of_one_token_at_the_default_size_of_lds(k, F):
    E, D = 9, 64
    q, v = stacks(E, D, F, 31)
    g = torch.Generator().manual_seed(F)
    x = torch.randn((1, D), generator=g).to(torch.bfloat16)
    ids = torch.randint(0, E, (1, k), generator=g, dtype=torch.int32)
    w = torch.randn((1, k), generator=g)
    y = w4.mx4_moe(*q, x.cuda(), ids.cuda(), w.cuda()).cpu().double().numpy()
    want, bound = oracle.mx4_moe(*v, x.double().numpy(), ids.numpy(), w.double().numpy(), "gelu_tanh")
    assert (np.abs(y - want) <= bound).all()


@pytest.mark.parametrize("M,N,K", [(4096, 4096, 160), (2048, 11008, 96), (2048, 4096, 96), (4097, 257, 224), (513, 8000, 352),
                                   (1000, 1000, 4128)])
@pytest.mark.parametrize("x4", [False, True])
def test_product_in_every_block(M, N, K, x4):
    """Sizes at which the large blocks of the plan are taken, exact as above."""
    wc, ws, wv = integers((N, K), 1)
    xc, xs, xv = integers((M, K), 2)
    want, size = product(xv, wv)
    assert float(size.max()) < 2 ** 20
    y = w4.mx4_gemm(device(wc, ws), device(xc, xs) if x4 else bf16(xv).cuda(), dtype=torch.float32)
    assert torch.equal(y.cpu().double(), want)
