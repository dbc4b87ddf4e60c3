"""Cases for measuring the microscaled 4-bit format (E2M1 codes, one power-of-two scale
byte for 32 values along a row) and what a mixture of experts does with it.

  kind "quantize" rows are quantized and read back as the values they stand for
  kind "product"  Y [M][N] = X [M][K] times W [N][K] transposed, W in 4 bits, X bf16
                  (`x4` false) or quantized to the same 4 bits inside the call (`x4` true)
  kind "select"   router logits [M][E] to top_k experts and their weights: softmax or
                  sigmoid scores, a bias that only the choice sees, groups of experts,
                  weights renormalized and scaled
  kind "experts"  the gated FFN of each token's chosen experts, weighted and added up,
                  for gate, up [E][F][D] and down [E][D][F] in 4 bits

A group of 32 values with the largest magnitude a has the scale X = 2^(floor(log2 a) - 2),
stored as the byte of its exponent plus 127, and each value's code is the E2M1 number
(0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives) nearest to value / X, ties to the even
code, magnitudes over 6 to 6. Codes lie low nibble first in bytes [rows][K / 2].

Case keys: M rows or tokens, N, K, `src` / `dst` types of rows in and out, `slack` columns
between the rows of a strided input; E, top_k, `score`, `bias`, `groups` / `top_groups` /
`group_best` (how many of a group's largest choice values make its value), `renorm`,
`scale`, `masked` experts whose logits are -infinity; D, F, `act`, `idle` tokens of a
padded batch, which have no expert.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _case(name, kind, **kw):
    c = {"quantize": dict(M=1, K=64, src="bf16", dst="bf16", slack=0),
         "product": dict(M=1, N=64, K=64, x4=False, dst="bf16", slack=0),
         "select": dict(M=1, E=8, top_k=1, score="softmax", bias=False, groups=1, top_groups=1, group_best=1,
                        renorm=False, scale=1.0, src="f32", masked=0),
         "experts": dict(M=1, E=8, top_k=1, D=64, F=64, act="gelu_tanh", idle=0)}[kind]
    c.update(kw, kind=kind)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the activations of a decode step of 48 users, slices of a wider matrix
        _case("quantize_step", "quantize", M=48, K=2048, src="bf16", dst="f32", slack=64),
        # a weight matrix of the 7B shape, fp32 as the checkpoint's conversion holds it
        _case("quantize_weights", "quantize", M=11008, K=4096, src="f32", dst="bf16"),
        # one token of the 7B shape's gate projection
        _case("product_one", "product", M=1, N=11008, K=4096, dst="f32"),
        # a decode batch of the 13B shape, an odd number of users
        _case("product_few", "product", M=13, N=13824, K=5120, dst="f32"),
        # the last, ragged chunk of a prompt through the 7B shape's down projection
        _case("product_chunk", "product", M=333, N=4096, K=11008),
        # a prompt of 2048 tokens of the 7B shape, bf16 activations
        _case("product_prompt", "product", M=2048, N=11008, K=4096),
        # a longer prompt, activations quantized as well
        _case("product_prompt4", "product", M=4097, N=11008, K=4096, x4=True),
        # one token over 128 experts
        _case("select_one", "select", M=1, E=128, top_k=8, renorm=True),
        # a prompt over 256 experts in eight groups, sigmoid scores balanced by a bias
        _case("select_prompt", "select", M=8192, E=256, top_k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
              group_best=2, renorm=True, scale=2.5),
        # one token of the 26B mixture's shape
        _case("experts_one", "experts", M=1, E=128, top_k=8, D=2048, F=768),
        # a padded decode batch, three slots empty
        _case("experts_batch", "experts", M=61, E=128, top_k=8, D=2048, F=768, idle=3),
        # a prompt of 4096 tokens
        _case("experts_prompt", "experts", M=4096, E=128, top_k=8, D=2048, F=768, act="silu"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    limit = {}
    for c in listed():
        limit[c["kind"]] = max(limit.get(c["kind"], 0), _cost(c))
    while True:
        kind = rng.choice(["quantize", "product", "product", "select", "experts", "experts"])
        if kind == "quantize":
            c = _case(None, kind, M=_spread(rng, 1, 16384), K=32 * _spread(rng, 1, 512), src=rng.choice(["f32", "bf16"]),
                      dst=rng.choice(["f32", "bf16"]), slack=rng.choice([0, 0, 8, 96]))
        elif kind == "product":
            c = _case(None, kind, M=_spread(rng, 1, 8192), N=_spread(rng, 1, 16384), K=32 * _spread(rng, 1, 448),
                      x4=rng.random() < 0.4, dst=rng.choice(["f32", "bf16"]), slack=rng.choice([0, 0, 8, 96]))
        elif kind == "select":
            E = rng.choice([8, 16, 24, 60, 64, 96, 128, 160, 256, 384, 512])
            g = rng.choice([v for v in (1, 1, 2, 4, 8) if E % v == 0])
            c = _case(None, kind, M=_spread(rng, 1, 16384), E=E, top_k=rng.randint(1, min(E // g, 12)),
                      score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=g,
                      top_groups=rng.randint(1, g), group_best=rng.choice([1, 2]) if g > 1 and E > g else 1,
                      renorm=rng.random() < 0.6, scale=rng.choice([1.0, 1.0, 2.5]), src=rng.choice(["f32", "bf16"]),
                      masked=rng.choice([0, 0, 0, 1]))
        else:
            E = rng.choice([4, 8, 16, 60, 64, 128])
            c = _case(None, kind, M=_spread(rng, 1, 4096), E=E, top_k=rng.randint(1, min(E, 8)),
                      D=32 * _spread(rng, 4, 128), F=32 * _spread(rng, 2, 64), act=rng.choice(["gelu_tanh", "silu"]))
            if c["M"] > 3:
                c["idle"] = rng.choice([0, 0, 1, 3])
        if _cost(c) <= limit[kind]:
            return c


# ---------------------------------------------------------------- sizes of a case
def work(c):
    if c["kind"] == "quantize":                      # rows in, codes and scales out, rows as they read back
        n = c["M"] * c["K"]
        return {"bytes": n * (_SIZE[c["src"]] + _SIZE[c["dst"]]) + n * 17 // 32, "flops": 6 * n}
    if c["kind"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": N * K * 17 // 32 + 2 * M * K + M * N * _SIZE[c["dst"]], "flops": 2 * M * N * K}
    if c["kind"] == "select":
        return {"bytes": c["M"] * (c["E"] * _SIZE[c["src"]] + 8 * c["top_k"]) + 4 * c["E"] * c["bias"],
                "flops": 8 * c["M"] * c["E"]}
    pairs = (c["M"] - c["idle"]) * c["top_k"]
    hit = c["E"] * (1 - (1 - c["top_k"] / c["E"]) ** (c["M"] - c["idle"]))   # experts that some token chose
    return {"bytes": int(hit * 3 * c["D"] * c["F"] * 17 / 32) + 4 * c["M"] * c["D"] + 8 * c["M"] * c["top_k"],
            "flops": 6 * pairs * c["D"] * c["F"]}


def _cost(c):
    w = work(c)
    stored = c["E"] * 3 * c["D"] * c["F"] if c["kind"] == "experts" else 0
    return max(w["bytes"], stored) + w["flops"] / 200


# ---------------------------------------------------------------- the format in elementary operations
def _quantized(x):
    """fp32 [..., K] -> codes uint8 [..., K / 2], scale bytes uint8 [..., K / 32]."""
    x = x.unflatten(-1, (-1, 32))
    e = (x.abs().amax(-1).view(torch.int32) >> 23) - 2           # exponent of the largest, plus 127
    e = e.clamp(min=0)
    r = x * ((254 - e) << 23).view(torch.float32)[..., None]     # times 2^(127 - e): exact
    a = r.abs()
    q = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
         + 8 * (r < 0)).flatten(-2)
    return q[..., 0::2] | (q[..., 1::2] << 4), e.to(torch.uint8)


def _values(codes, scales):
    """The fp32 values that codes [..., K / 2] and scale bytes [..., K / 32] stand for."""
    grid = torch.tensor(_GRID + tuple(-v for v in _GRID), device=codes.device)
    v = grid[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    e = scales.int()
    s = torch.where(e == 0, 1 << 22, e << 23).view(torch.float32)
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


# ---------------------------------------------------------------- inputs
def _weights(shape, g):
    """Quantized N(0, 0.02) weights, made some matrices at a time."""
    dev = g.device
    codes = torch.empty(shape[:-1] + (shape[-1] // 2,), dtype=torch.uint8, device=dev)
    scales = torch.empty(shape[:-1] + (shape[-1] // 32,), dtype=torch.uint8, device=dev)
    rows = math.prod(shape[:-1])
    c2, s2 = codes.view(rows, -1), scales.view(rows, -1)
    step = max(1, (1 << 27) // shape[-1])
    for a in range(0, rows, step):
        m = min(step, rows - a)
        c2[a:a + m], s2[a:a + m] = _quantized(0.02 * torch.randn((m, shape[-1]), generator=g, device=dev))
    return codes, scales


def _strided(M, K, slack, dtype, g, spread=0.0):
    x = torch.randn((M, K + slack), generator=g, device=g.device)
    if spread:                                       # rows and channels of different magnitudes
        x *= torch.exp(spread * torch.randn((M, 1), generator=g, device=g.device))
        x *= torch.exp(spread * torch.randn((1, K + slack), generator=g, device=g.device))
    return x.to(dtype)[:, :K]


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 29)
    s = dict(case=c)
    if c["kind"] == "quantize":
        s["x"] = _strided(c["M"], c["K"], c["slack"], _TYPES[c["src"]], g, 0.7)
    elif c["kind"] == "product":
        s["w"] = _weights((c["N"], c["K"]), g)
        s["x"] = _strided(c["M"], c["K"], c["slack"], torch.bfloat16, g, 0.4)
    elif c["kind"] == "select":
        l = torch.randn((c["M"], c["E"]), generator=g, device=dev)
        l += 0.5 * torch.randn((c["E"],), generator=g, device=dev)
        if c["masked"]:
            l[:, torch.randperm(c["E"], generator=g, device=dev)[:c["masked"]]] = float("-inf")
        s["logits"] = l.to(_TYPES[c["src"]])
        s["bias"] = 0.1 * torch.randn((c["E"],), generator=g, device=dev) if c["bias"] else None
    else:
        E, D, F, M, k = c["E"], c["D"], c["F"], c["M"], c["top_k"]
        s["gate"], s["up"], s["down"] = _weights((E, F, D), g), _weights((E, F, D), g), _weights((E, D, F), g)
        s["x"] = torch.randn((M, D), generator=g, device=dev).to(torch.bfloat16)
        l = torch.randn((M, E), generator=g, device=dev) + 0.5 * torch.randn((E,), generator=g, device=dev)
        p, ids = torch.softmax(l, -1).topk(k, -1)
        ids = ids.to(torch.int32)
        if c["idle"]:
            ids[M - c["idle"]:] = -1
        s["ids"], s["weights"] = ids, p / p.sum(-1, keepdim=True)
    if own:
        import bit_weight_only_quantize_amd as w4

        def matrix(w, N, K, E=1):
            return w4.QuantizedMatrix("mx4_g32", N, K, w[0], w[1], None, E)
        if c["kind"] == "quantize":
            s["q"] = w4.empty_quantized("mx4_g32", c["M"], c["K"])
            s["out"] = torch.empty((c["M"], c["K"]), dtype=_TYPES[c["dst"]], device=dev)
        elif c["kind"] == "product":
            s["W"] = matrix(s["w"], c["N"], c["K"])
            s["q"] = w4.empty_quantized("mx4_g32", c["M"], c["K"]) if c["x4"] else None
            s["out"] = torch.empty((c["M"], c["N"]), dtype=_TYPES[c["dst"]], device=dev)
            s["workspace"] = w4.mx4_gemm_workspace(s["W"], c["M"], x4=c["x4"])
        elif c["kind"] == "select":
            s["out"] = (torch.empty((c["M"], c["top_k"]), dtype=torch.int32, device=dev),
                        torch.empty((c["M"], c["top_k"]), dtype=torch.float32, device=dev))
        else:
            s["mats"] = (matrix(s["gate"], F, D, E), matrix(s["up"], F, D, E), matrix(s["down"], D, F, E))
            s["out"] = torch.empty((M, D), dtype=torch.bfloat16, device=dev)
            s["workspace"] = w4.mx4_moe_workspace(*s["mats"], M, k)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        import bit_weight_only_quantize_amd as w4
        if c["kind"] == "quantize":
            return w4.mx4_read(w4.mx4_quantize(s["x"], out=s["q"]), out=s["out"])
        if c["kind"] == "product":
            x = w4.mx4_quantize(s["x"], out=s["q"]) if c["x4"] else s["x"]
            return w4.mx4_gemm(s["W"], x, out=s["out"], workspace=s["workspace"])
        if c["kind"] == "select":
            return w4.moe_select(s["logits"], c["top_k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                                 top_groups=c["top_groups"], group_best=c["group_best"], renormalize=c["renorm"],
                                 scale=c["scale"], ids=s["out"][0], weights=s["out"][1])
        return w4.mx4_moe(*s["mats"], s["x"], s["ids"], s["weights"], act=c["act"], out=s["out"],
                          workspace=s["workspace"])
    if c["kind"] == "quantize":
        return _values(*_quantized(s["x"].float())).to(_TYPES[c["dst"]])
    if c["kind"] == "product":
        x = _values(*_quantized(s["x"].float())) if c["x4"] else s["x"].float()
        return (x @ _values(*s["w"]).t()).to(_TYPES[c["dst"]])
    if c["kind"] == "select":
        return _select(s)
    return _experts(s)


def _select(s):
    """Choices in 64 bits: scores lie next to each other."""
    c = s["case"]
    l = s["logits"].double()
    if c["score"] == "softmax":
        p = torch.exp(l - l.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-l))
    value = p + s["bias"].double() if c["bias"] else p
    masked = l == float("-inf")
    order = (value if c["bias"] else l).masked_fill(masked, -1e300)
    if c["groups"] > 1:
        by = value.masked_fill(masked, float("-inf")).unflatten(-1, (c["groups"], -1))
        best = by.sort(-1, descending=True)[0][..., :c["group_best"]].sum(-1)
        keep = best.sort(dim=-1, descending=True, stable=True)[1][..., :c["top_groups"]]
        kept = torch.zeros_like(best, dtype=torch.bool).scatter_(-1, keep, True)
        order = order.unflatten(-1, (c["groups"], -1)).masked_fill(~kept[..., None], float("-inf")).flatten(-2)
    ids = order.sort(dim=-1, descending=True, stable=True)[1][..., :c["top_k"]]   # ties to the lower index
    w = p.gather(-1, ids)
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return ids.to(torch.int32), (w * c["scale"]).float()


def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _experts(s):
    c = s["case"]
    E, k = c["E"], c["top_k"]
    x, ids, w = s["x"].float(), s["ids"].long().flatten(), s["weights"]
    live = ids >= 0
    if len(ids) <= E:                                # each pair's own matrices
        e = ids.clamp(min=0)
        t = x.repeat_interleave(k, 0)[:, :, None]
        g = torch.bmm(_values(s["gate"][0][e], s["gate"][1][e]), t)
        u = torch.bmm(_values(s["up"][0][e], s["up"][1][e]), t)
        y = torch.bmm(_values(s["down"][0][e], s["down"][1][e]), _act(g, c["act"]) * u)[..., 0]
    else:                                            # every expert over its tokens, padded to the busiest one
        e = torch.where(live, ids, E)
        at = e.sort(stable=True)[1]
        count = torch.bincount(e, minlength=E + 1)
        place = torch.empty_like(ids)
        place[at] = torch.arange(len(ids), device=ids.device) - (count.cumsum(0) - count)[e[at]]
        place = torch.where(live, place, 0)
        rows = int(count[:E].max())
        t = torch.zeros((E, rows, c["D"]), device=x.device)
        t[ids[live], place[live]] = x.repeat_interleave(k, 0)[live]
        g = torch.bmm(t, _values(*s["gate"]).transpose(1, 2))
        u = torch.bmm(t, _values(*s["up"]).transpose(1, 2))
        y = torch.bmm(_act(g, c["act"]) * u, _values(*s["down"]).transpose(1, 2))
        y = y[ids.clamp(min=0), place]
    y = torch.where(live[:, None], y, torch.zeros_like(y)).view(c["M"], k, c["D"])
    return (y * w[..., None]).sum(1).to(torch.bfloat16)


# ---------------------------------------------------------------- the definition in 64 bits
def _two_to(e):
    """2^e in fp64, exactly: pow on the GPU may be an ulp off, which decides ties wrongly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _grid_of(codes, scales):
    """fp64 values of codes and scale bytes, from the bits of an E2M1 number."""
    n = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.int64, device=codes.device)
    n[..., 0::2] = codes.long() % 16
    n[..., 1::2] = codes.long() // 16
    e, m = (n // 2) % 4, (n % 2).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * _two_to(e - 1))
    v = torch.where(n >= 8, -v, v)
    return v * _two_to(scales.long() - 127).repeat_interleave(32, -1)


def _nearest(x):
    """The values that rows x [M][K] have after quantization, fp64."""
    x = x.double().reshape(x.shape[0], -1, 32)
    a = x.abs().max(-1, keepdim=True).values
    _, e = torch.frexp(a)                            # a = m 2^e with m in [0.5, 1)
    unit = _two_to(torch.where(a > 0, (e - 3).clamp(min=-127), -127))
    r = (x / unit).abs().clamp(max=6)
    step = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0))     # the spacing of E2M1 numbers there
    return (torch.round(r / step) * step * torch.sign(x) * unit).reshape(x.shape[0], -1)


def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] == "quantize":
        return _nearest(s["x"])
    if c["kind"] == "product":
        x = _nearest(s["x"]) if c["x4"] else s["x"].double()
        return torch.matmul(x, _grid_of(*s["w"]).t())
    if c["kind"] == "select":
        l, M, E = s["logits"].double(), c["M"], c["E"]
        p = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
        ids = _select(s)[0].long()                   # whole numbers are compared with the plain form's
        w = torch.gather(p, 1, ids)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        return None, c["scale"] * w
    E, D, k = c["E"], c["D"], c["top_k"]
    x = s["x"].double()
    y = torch.zeros((c["M"], D), dtype=torch.float64, device=x.device)
    for e in range(E):
        m, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        if len(m) == 0:
            continue
        gate, up, down = (_grid_of(q[0][e], q[1][e]) for q in (s["gate"], s["up"], s["down"]))
        g, u = x[m] @ gate.t(), x[m] @ up.t()
        g = torch.nn.functional.silu(g) if c["act"] == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
        y.index_add_(0, m, ((g * u) @ down.t()) * s["weights"][m, j].double()[:, None])
    return y
