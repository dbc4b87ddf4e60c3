"""Cases for measuring the batched INT4 KV cache: writing rows into it, reading them
back, and attention over it for single tokens and for prompts.

Every case is a batch of sequences. Sequence b holds L_b positions after the call and
has n_b rows in the call; its row i stands at position L_b - n_b + i. The cache is a
pool of pages, codes uint8 [page][kv head][position in page][D / 2] (element 2j in the
low nibble of byte j, stored plus 8) and fp32 scales [page][kv head][position in page];
`page` 0 means no page table: sequence b owns page b, which holds `longest` positions.

  kind "write"  K and V rows are quantized into the cache and read back
  kind "read"   K and V rows are read back from a filled cache
  kind "decode" attention of one row a sequence over its cached positions
  kind "prompt" attention of many rows a sequence, each seeing the positions up to its own

Case keys: B sequences (`idle` of them empty slots of a padded batch: no cached
position, output 0), `longest` the largest L, `rows` the largest n, `mix` seeds the
spread of the lengths (0: all alike), Hq / Hkv heads, D, page, window / sinks (0: none),
`src` and `dst` the types of the rows given and returned, `lse` whether the log-sum-exp
of each row is returned too, `fused` whether the rows are slices of one Q-K-V matrix.
"""
import math
import random

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}


def _case(name, kind, **kw):
    c = dict(kind=kind, B=1, idle=0, longest=1, rows=1, mix=0, Hq=8, Hkv=8, D=128, page=0, window=0, sinks=0,
             src="bf16", dst="bf16", lse=False, fused=False)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one generated token for each of 64 users; the projections' GEMVs return fp32
        _case("write_step", "write", B=64, longest=2048, rows=1, mix=1, Hq=32, Hkv=32, page=64, src="f32", dst="f32"),
        # prompts of seven users packed one after the other, K and V slices of the prefill GEMM's output
        _case("write_prompts", "write", B=7, longest=4096, rows=4096, mix=2, Hq=32, Hkv=8, page=16, fused=True),
        # three short prefixes taken out for a host copy, odd lengths
        _case("read_prefixes", "read", B=3, longest=333, rows=333, mix=3, Hq=4, Hkv=2, D=256, page=0, dst="f32"),
        # a long context read back in the activations' type
        _case("read_long", "read", B=1, longest=131071, rows=131071, Hq=32, Hkv=8, page=64),
        # the start of one user's answer, a small model: latency is all
        _case("decode_short", "decode", B=1, longest=129, Hq=8, Hkv=2, D=64, page=0, src="f32", dst="f32", lse=True),
        # one user at 8K context, 32 heads of 128 without sharing (the 7B shape), fp32 queries from the GEMV
        _case("decode_one", "decode", B=1, longest=8193, Hq=32, Hkv=32, page=0, src="f32", dst="bf16"),
        # a serving batch of ragged contexts in a padded graph: three empty slots
        _case("decode_batch", "decode", B=48, idle=3, longest=8192, mix=4, Hq=32, Hkv=8, page=64),
        # wide heads, a window of 1024 and four sinks over contexts up to 32K
        _case("decode_window", "decode", B=24, longest=32768, mix=5, Hq=16, Hkv=4, D=256, page=16, window=1024,
              sinks=4, src="f32", dst="f32"),
        # two users with 128K contexts, five query heads a kv head
        _case("decode_long", "decode", B=2, longest=131072, mix=6, Hq=40, Hkv=8, page=256, lse=True),
        # short follow-up questions in fp32, a small model
        _case("prompt_short", "prompt", B=3, longest=377, rows=77, mix=7, Hq=8, Hkv=2, D=64, page=16, src="f32",
              dst="f32", lse=True),
        # chunks of five users' prompts behind what they cached before, window and sinks
        _case("prompt_chunks", "prompt", B=5, longest=6001, rows=1500, mix=8, Hq=32, Hkv=8, page=32, window=2048,
              sinks=4, fused=True),
        # one whole prompt of 8192 tokens, the 7B shape
        _case("prompt_long", "prompt", B=1, longest=8192, rows=8192, Hq=32, Hkv=32, page=64, fused=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    limit = {}
    for c in listed():                               # a window saves the plain form nothing
        limit[c["kind"]] = max(limit.get(c["kind"], 0), _cost(dict(c, window=0)))
    while True:
        kind = rng.choice(["write", "read", "decode", "prompt"])
        Hkv = rng.choice([1, 2, 4, 5, 8, 16, 32])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 8, 16] if Hkv <= 8 else [1, 2, 3])
        src, dst = rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"])
        c = _case(None, kind, Hq=Hq, Hkv=Hkv, D=rng.choice([64, 128, 128, 128, 256]), mix=rng.randrange(1, 1 << 20),
                  page=rng.choice([0, 16, 32, 64, 128, 256]), src=src, dst=dst, fused=rng.random() < 0.5)
        if kind == "write":
            c.update(B=_spread(rng, 1, 64), rows=_spread(rng, 1, 4096), dst=src)
            c["longest"] = c["rows"] + _spread(rng, 1, 2048)
        elif kind == "read":
            c.update(B=_spread(rng, 1, 16), rows=_spread(rng, 1, 131071))
            c["longest"] = c["rows"]
        elif kind == "decode":
            c.update(B=_spread(rng, 1, 64), longest=_spread(rng, 1, 131072), lse=rng.random() < 0.4)
            if not c["lse"] and c["B"] > 3:
                c["idle"] = rng.choice([0, 0, 1, 3])
        else:
            c.update(B=_spread(rng, 1, 8), rows=_spread(rng, 2, 8192), lse=rng.random() < 0.4)
            c["longest"] = c["rows"] + rng.choice([0, _spread(rng, 1, 16384)])
        if kind in ("decode", "prompt") and rng.random() < 0.5:
            c["window"] = _spread(rng, 1, 4096)
            c["sinks"] = rng.choice([0, 1, 4, 4, 16, 67])
        if _cost(dict(c, window=0)) <= limit[kind]:
            return c


# ---------------------------------------------------------------- sizes of a case
def _sizes(c):
    """Per sequence (L, n)."""
    rng = random.Random(c["mix"])
    L, n = [], []
    for b in range(c["B"]):
        if b >= c["B"] - c["idle"]:
            L.append(0)
            n.append(1)
            continue
        rows, old = c["rows"], c["longest"] - c["rows"]
        if b and c["mix"]:
            rows = max(1, int(rows * rng.uniform(0.1, 1.0)))
            old = int(old * rng.uniform(0.0, 1.0))
        L.append(old + rows)
        n.append(rows)
    return L, n


def _visible(L, n, window, sinks):
    """(query, key) pairs that the mask leaves, and distinct keys that any row sees, of one sequence."""
    if L == 0:
        return 0, 0
    pairs = 0
    for i in range(n):
        p = L - n + i
        near = p + 1 if window == 0 else min(p + 1, window)
        pairs += near + (0 if window == 0 else min(sinks, p + 1 - near))
    first = L - n                                    # the first row's position
    lo = 0 if window == 0 else max(0, first - window + 1)
    return pairs, (L - lo) + min(sinks if window else 0, lo)


def work(c):
    L, n = _sizes(c)
    D, Hkv, Hq = c["D"], c["Hkv"], c["Hq"]
    vec = D // 2 + 4                                 # codes and scale of one cached head vector
    rows = sum(n)
    if c["kind"] == "write":                         # rows in, codes out, rows as they read back
        return {"bytes": 2 * rows * Hkv * (D * _SIZE[c["src"]] + vec + D * _SIZE[c["dst"]]),
                "flops": 2 * rows * Hkv * D * 4}
    if c["kind"] == "read":
        return {"bytes": 2 * rows * Hkv * (vec + D * _SIZE[c["dst"]]), "flops": 2 * rows * Hkv * D}
    pairs = keys = 0
    for a, b in zip(L, n):
        p, k = _visible(a, b, c["window"], c["sinks"])
        pairs += p
        keys += k
    return {"bytes": 2 * keys * Hkv * vec + rows * Hq * (D * (_SIZE[c["src"]] + _SIZE[c["dst"]]) + 4 * c["lse"]),
            "flops": 4 * D * Hq * pairs}


def _cost(c):
    L, _ = _sizes(c)
    w = work(c)
    full = 2 * sum(L) * c["Hkv"] * (c["D"] // 2 + 4)  # the cache that the case keeps, seen or not
    return max(w["bytes"], full) + w["flops"] / 200


# ---------------------------------------------------------------- inputs
def _quantized(x):
    """fp32 vectors [..., D] -> codes uint8 [..., D / 2], scales fp32 [...]."""
    s = x.abs().amax(-1)
    s = s / torch.full_like(s, 7.5)                  # a true division: a Python number would turn into a product
    r = x / torch.where(s > 0, s, torch.ones_like(s))[..., None]
    q = (torch.sign(r) * torch.floor(r.abs() + 0.5)).clamp(-8, 7).to(torch.int16) + 8
    return (q[..., 0::2] | (q[..., 1::2] << 4)).to(torch.uint8), s


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 17)
    L, n = _sizes(c)
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    rows, width = sum(n), max(1, c["longest"])
    if c["page"]:
        size = c["page"]
        need = [(v + size - 1) // size for v in L]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32).tolist()
        table = torch.full((B, max(1, max(need))), -1, dtype=torch.int32)
        at = 0
        for b in range(B):                           # entries behind a sequence's last page stay -1
            table[b, :need[b]] = torch.tensor(order[at:at + need[b]], dtype=torch.int32)
            at += need[b]
        table = table.to(dev)
    else:
        size, pages, table = width, B, None
    # what was cached before: head vectors of a spread of magnitudes, quantized
    filled = []
    for _ in range(2):
        codes = torch.empty((pages, Hkv, size, D // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((pages, Hkv, size), dtype=torch.float32, device=dev)
        step = max(1, (1 << 26) // (Hkv * size * D))
        for a in range(0, pages, step):
            m = min(step, pages - a)
            x = torch.randn((m, Hkv, size, D), generator=g, device=dev)
            x *= torch.exp(0.3 * torch.randn((m, Hkv, size, 1), generator=g, device=dev))
            codes[a:a + m], scales[a:a + m] = _quantized(x)
        filled += [codes, scales]
    if c["fused"]:
        qkv = torch.randn((rows, (Hq + 2 * Hkv) * D), generator=g, device=dev).to(_TYPES[c["src"]])
        q = qkv[:, :Hq * D].view(rows, Hq, D)
        k = qkv[:, Hq * D:(Hq + Hkv) * D].view(rows, Hkv, D)
        v = qkv[:, (Hq + Hkv) * D:].view(rows, Hkv, D)
    else:
        q = torch.randn((rows, Hq, D), generator=g, device=dev).to(_TYPES[c["src"]])
        k = v = None
        if c["kind"] == "write":
            k = torch.randn((rows, Hkv, D), generator=g, device=dev).to(_TYPES[c["src"]])
            v = torch.randn((rows, Hkv, D), generator=g, device=dev).to(_TYPES[c["src"]])
    first = [0]
    for m in n:
        first.append(first[-1] + m)
    s = dict(case=c, L=L, n=n, first=first, size=size, table=table, kc=filled[0], ks=filled[1], vc=filled[2],
             vs=filled[3], q=q, k=k, v=v, lens=torch.tensor(L, dtype=torch.int32, device=dev),
             n_dev=torch.tensor(n, device=dev), first_dev=torch.tensor(first[:-1], device=dev))
    if own:
        import bit_weight_only_quantize_amd as w4
        starts = None if max(n) == 1 else torch.tensor(first, dtype=torch.int32, device=dev)
        s["cache"] = w4.KVPages(*filled)
        s["batch"] = w4.KVBatch(s["lens"], table=table, starts=starts, rows=rows, max_rows=max(n), max_len=max(L))
        if c["kind"] in ("decode", "prompt"):
            s["out"] = torch.empty((rows, Hq, D), dtype=_TYPES[c["dst"]], device=dev)
            s["workspace"] = w4.kv_attention_workspace(s["cache"], s["batch"], Hq, c["window"], c["sinks"])
        else:
            s["back"] = [torch.empty((rows, Hkv, D), dtype=_TYPES[c["dst"]], device=dev) for _ in range(2)]
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        import bit_weight_only_quantize_amd as w4
        if c["kind"] == "write":
            w4.kv_write(s["k"], s["v"], s["cache"], s["batch"])
        if c["kind"] in ("write", "read"):
            return w4.kv_read(s["cache"], s["batch"], k=s["back"][0], v=s["back"][1])
        return w4.kv_attention(s["q"], s["cache"], s["batch"], window=c["window"], sinks=c["sinks"], out=s["out"],
                               want_lse=c["lse"], workspace=s["workspace"])
    if c["kind"] in ("write", "read"):
        page, off = _places(s)
        if c["kind"] == "write":
            for x, codes, scales in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
                codes[page, :, off], scales[page, :, off] = _quantized(x.float())
        return tuple(_values(codes[page, :, off], scales[page, :, off]).to(_TYPES[c["dst"]])
                     for codes, scales in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
    return _attend(s)


def _values(codes, scales):
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8
    return q * scales[..., None]


def _places(s):
    """Page and offset in it of every row."""
    rows = torch.arange(s["first"][-1], device=s["n_dev"].device)
    b = torch.repeat_interleave(torch.arange(len(s["n"]), device=rows.device), s["n_dev"], output_size=len(rows))
    pos = (s["lens"] - s["n_dev"] - s["first_dev"])[b] + rows
    if s["table"] is None:
        return b, pos
    return s["table"][b, pos // s["size"]].long(), pos % s["size"]


def _attend(s):
    c = s["case"]
    shape = (s["first"][-1], c["Hq"])
    out = torch.empty(shape + (c["D"],), dtype=_TYPES[c["dst"]], device=s["lens"].device)
    lse = torch.empty(shape, dtype=torch.float32, device=out.device)
    if max(s["n"]) == 1:                             # the whole batch at once, padded to the longest
        b = torch.arange(c["B"], device=out.device)
        _attend_block(s, b, max(s["L"]), s["lens"][:, None] - 1, slice(0, c["B"]), out, lse)
    else:                                            # sequence by sequence, some rows at a time
        for b, (L, n) in enumerate(zip(s["L"], s["n"])):
            step = max(1, (1 << 29) // (L * (c["Hq"] // c["Hkv"])))
            for i in range(0, n, step):
                m = min(step, n - i)
                p = torch.arange(L - n + i, L - n + i + m, device=out.device)[None, :]
                r = s["first"][b] + i
                _attend_block(s, torch.tensor([b]).to(out.device, non_blocking=True), L, p, slice(r, r + m), out, lse)
    return (out, lse) if c["lse"] else out


def _attend_block(s, b, T, p, rows, out, lse):
    """Rows `rows` of sequences b, at positions p [len(b)][N], over T positions; some kv heads at a time."""
    c = s["case"]
    Hkv, D = c["Hkv"], c["D"]
    B, N, G = p.shape[0], p.shape[1], c["Hq"] // c["Hkv"]
    t = torch.arange(T, device=p.device)
    see = t <= p[..., None]
    if c["window"]:
        see = see & ((t > p[..., None] - c["window"]) | (t < c["sinks"]))          # [B][N][T]
    if s["table"] is None:
        page, off = b[:, None].expand(B, T), t.expand(B, T)
    else:
        page, off = s["table"][b][:, t // s["size"]].clamp(min=0).long(), (t % s["size"]).expand(B, T)
    step = max(1, (1 << 29) // (B * T * max(G * N, D)))
    for h in range(0, Hkv, step):
        hs = slice(h, min(Hkv, h + step))
        m = hs.stop - hs.start
        heads = slice(hs.start * G, hs.stop * G)
        k = _values(s["kc"][:, hs][page, :, off], s["ks"][:, hs][page, :, off])    # [B][T][m][D]
        k = k.permute(0, 2, 3, 1).contiguous()
        q = s["q"][rows, heads].float().view(B, N, m, G, D).permute(0, 2, 1, 3, 4).reshape(B, m, N * G, D)
        z = torch.matmul(q, k).view(B, m, N, G, T) / math.sqrt(D)
        del k
        z = z.masked_fill(~see[:, None, :, None], float("-inf"))
        top = z.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
        z = torch.exp(z - top)
        total = z.sum(-1, keepdim=True)
        v = _values(s["vc"][:, hs][page, :, off], s["vs"][:, hs][page, :, off])
        v = v.permute(0, 2, 1, 3).contiguous()
        o = torch.matmul(z.view(B, m, N * G, T), v).view(B, m, N, G, D)
        del v, z
        o = torch.where(total > 0, o / total, torch.zeros_like(o))
        out[rows, heads] = o.permute(0, 2, 1, 3, 4).reshape(B * N, m * G, D).to(out.dtype)
        lse[rows, heads] = (top + torch.log(total)).permute(0, 2, 1, 3, 4).reshape(B * N, m * G)


# ---------------------------------------------------------------- the definition in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    dev = s["lens"].device
    G, D, W, S = c["Hq"] // c["Hkv"], c["D"], c["window"], c["sinks"]

    def cached(codes, scales, b, h, lo, hi):
        """Positions lo .. hi - 1 of kv head h of sequence b, fp64 [hi - lo][D]."""
        t = torch.arange(lo, hi, device=dev)
        where = (torch.full_like(t, b), t) if s["table"] is None else \
            (s["table"][b].long()[t // s["size"]], t % s["size"])
        byte = codes[:, h][where].to(torch.int64)
        x = torch.empty((hi - lo, D), dtype=torch.float64, device=dev)
        x[:, 0::2] = (byte % 16 - 8).double()
        x[:, 1::2] = (torch.div(byte, 16, rounding_mode="floor") - 8).double()
        return x * scales[:, h][where].double()[:, None]

    if c["kind"] in ("write", "read"):
        back = []
        for x, codes, scales in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
            if c["kind"] == "write":
                # the scale is held in fp32, and the codec rounds the fp32 quotient, halves away from zero
                x = x.double()
                scale = x.abs().max(-1, keepdim=True).values
                scale = (scale / torch.full_like(scale, 7.5)).float().double()
                y = (x / scale.clamp(min=1e-300)).float().double()
                y = torch.where(y < 0, torch.ceil(y - 0.5), torch.floor(y + 0.5))
                back.append(torch.minimum(torch.maximum(y, y.new_tensor(-8)), y.new_tensor(7)) * scale)
            else:
                parts = []
                for b, (L, n) in enumerate(zip(s["L"], s["n"])):
                    parts.append(torch.stack([cached(codes, scales, b, h, L - n, L) for h in range(c["Hkv"])], 1))
                back.append(torch.cat(parts))
        return tuple(back)

    out = torch.zeros((s["first"][-1], c["Hq"], D), dtype=torch.float64, device=dev)
    lse = torch.full((s["first"][-1], c["Hq"]), float("-inf"), dtype=torch.float64, device=dev)
    for b, (L, n) in enumerate(zip(s["L"], s["n"])):
        if L == 0:
            continue
        r0 = s["first"][b]
        pos = torch.arange(L - n, L, device=dev)[:, None]
        key = torch.arange(L, device=dev)[None, :]
        hidden = key > pos
        if W:
            hidden = hidden | ((pos - key >= W) & (key >= S))
        for h in range(c["Hkv"]):
            k = cached(s["kc"], s["ks"], b, h, 0, L)
            v = cached(s["vc"], s["vs"], b, h, 0, L)
            for j in range(h * G, (h + 1) * G):
                z = (s["q"][r0:r0 + n, j].double() @ k.t()) * D ** -0.5
                z.masked_fill_(hidden, float("-inf"))
                e = torch.logsumexp(z, 1)
                lse[r0:r0 + n, j] = e
                out[r0:r0 + n, j] = torch.exp(z.sub_(e[:, None])) @ v
    return (out, lse) if c["lse"] else out
