"""GPU tests of the batched INT4 KV cache at unusual values: values and scales that a row does not
see or gives no weight, infinities and NaN, magnitudes near the ends of the types."""
import numpy as np
import pytest
import torch

import bit_weight_only_quantize_amd as w4
import oracle
from kv_batch_util import DT, Batch, bounds, to_dev, values

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def check_rows(s, q, got, lse, q_dtype, out_dtype, scale=None, terms=None, rows=None):
    """Causal rows (default: all) against the oracle. The weights' 16-bit format: a weight times value scale is
    off by 2^-25 of the format's unit where the column's largest is 2^8 of it at least, so by 2^-33 of that
    for each key, times codes of up to 8: of the largest p_t * 8 * scale_t that the row itself sees."""
    sc = float(np.float32(s.D ** -0.5 if scale is None else scale))
    pick = list(range(s.rows)) if rows is None else list(rows)
    refs, tops = [], []
    for r in pick:
        b = int(np.searchsorted(s.first, r, side="right")) - 1
        t = np.arange(s.lens[b] - s.n[b] + r - s.first[b] + 1)
        k, v, vs = s.deq[0][b][:, t], s.deq[1][b][:, t], s.quant[1][b][1][:, t].astype(np.float64)
        refs.append(oracle.kv_attention(q[r][None], k, v, sc))
        g = np.arange(q.shape[1]) // (q.shape[1] // s.Hkv)
        z = sc * (k[g] @ q[r].astype(np.float64)[..., None])[..., 0]
        tops.append((np.exp(z - refs[-1][1][0][:, None]) * 8 * vs[g]).max(1))
    ref = [np.concatenate(x) for x in zip(*refs)]
    e, el = bounds(ref, s.D, max(s.lens), np.stack(tops)[..., None], q_dtype, out_dtype, terms)
    g, l = got[pick].float().cpu().numpy().astype(np.float64), lse[pick].cpu().numpy().astype(np.float64)
    assert np.isfinite(g).all() and np.isfinite(l).all()
    worst, lw = (np.abs(g - ref[0]) / e).max(), (np.abs(l - ref[1]) / el).max()
    print(f"[kv values] out {worst:.3f} lse {lw:.3f} of the bounds", flush=True)
    assert worst <= 1.0 and lw <= 1.0


def set_values(s, scales, b=0):
    """Sequence b's value scales times `scales` [L] (before the cache is made)."""
    c, old = s.quant[1][b]
    s.quant[1][b] = (c, (old * np.asarray(scales, dtype=np.float64)[None]).astype(np.float32))
    s.deq[1][b] = oracle.kv_dequant(*s.quant[1][b])


def set_scores(s, q, z, b=0):
    """Sequence b's keys such that a row with q = 1 in element 0 and 0 elsewhere scores about z[t] (scale 1)."""
    k = np.zeros((s.Hkv, s.lens[b], s.D), dtype=np.float32)
    k[:, :, 0] = np.asarray(z, dtype=np.float32)[None]
    s.quant[0][b] = oracle.kv_quantize(k)
    s.deq[0][b] = oracle.kv_dequant(*s.quant[0][b])
    q[...] = 0
    q[..., 0] = 1


SPLIT = dict(lens=[50, 40], rows=[12, 1], Hkv=2, G=5, page=16)         # few columns, whole
PARTS = dict(lens=[5003, 700], rows=[3, 2], Hkv=1, G=4, page=64)       # few columns, keys in parts
PROMPT = dict(lens=[628, 530, 700, 611], rows=[128, 101, 120, 77], Hkv=2, G=64, page=16)   # many columns
SHARED = dict(lens=[5000, 4700, 4900, 4850], rows=[1000, 900, 1000, 800], Hkv=4, G=8, page=32)   # four rows a wavefront
PROMPT_PARTS = dict(lens=[9001], rows=[130], Hkv=1, G=64, page=64)


def make(shape, D, name, q_dtype="f32"):
    s = Batch(shape["lens"], shape["rows"], shape["Hkv"], D, shape["page"], name)
    return s, values((s.rows, shape["Hkv"] * shape["G"], D), name + ".q", q_dtype, seed=2)


def attend(s, cache, q, q_dtype, out_dtype, **kw):
    b = s.batch(max_rows=max(s.n), max_len=max(s.lens))
    out = torch.full(q.shape, 9.0, dtype=DT[out_dtype], device="cuda")
    return w4.kv_attention(to_dev(q, q_dtype), cache, b, out=out, want_lse=True, **kw)


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---------------------------------------------------------------- values without weight
@pytest.mark.parametrize("factor", [2.0 ** 20, 2.0 ** 40, 2.0 ** 100, INF, NAN])
@pytest.mark.parametrize("D,types", [(64, ("f32", "f32")), (128, ("bf16", "bf16")), (256, ("f32", "bf16"))])
@pytest.mark.parametrize("shape", [SPLIT, PARTS, SHARED], ids=["split", "parts", "prompt"])
def test_later_rows_do_not_reach_earlier_ones(shape, D, types, factor):
    """A key and value of any scale at a later row's position: the rows before it keep their bits."""
    s, q = make(shape, D, f"later.{D}", types[0])
    want = attend(s, s.cache(), q, *types)
    cache, before = s.cache(), []
    for b in range(s.B):
        n, L = s.n[b], s.lens[b]
        i = n - 1 - (n - 1) // 2                              # the row whose key and value change
        p, o = s.place(b, L - n + i)
        for scales in (cache.k_scales, cache.v_scales):
            scales[int(p), :, int(o)] *= factor
        before += range(s.first[b], s.first[b] + i)
    got = attend(s, cache, q, *types)
    assert len(before) > 0
    for x, y in zip(got, want):
        assert torch.isfinite(x[before]).all() and same_bits(x[before], y[before])


@pytest.mark.parametrize("factor", [2.0 ** 20, 2.0 ** 100, INF, NAN])
@pytest.mark.parametrize("D,types", [(64, ("f32", "f32")), (128, ("bf16", "bf16"))])
@pytest.mark.parametrize("shape,window", [(SPLIT, 9), (SHARED, 700)], ids=["split", "prompt"])
def test_values_behind_the_window_do_not_reach_its_rows(shape, window, D, types, factor):
    """A key and value that the window of the first rows still holds: the rows past it keep their bits."""
    s, q = make(shape, D, f"behind.{D}", types[0])
    mask = dict(window=window, sinks=2)
    want = attend(s, s.cache(), q, *types, **mask)
    cache, past = s.cache(), []
    for b in range(s.B):
        n, first = s.n[b], s.lens[b] - s.n[b]
        p, o = s.place(b, first)                               # seen by the first `window` rows
        for scales in (cache.k_scales, cache.v_scales):
            scales[int(p), :, int(o)] *= factor
        past += range(s.first[b] + window, s.first[b] + n)
    got = attend(s, cache, q, *types, **mask)
    for x, y in zip(got, want):
        assert torch.isfinite(x[past]).all() and same_bits(x[past], y[past])


@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("ratio", [2.0 ** 16, 2.0 ** 24, 2.0 ** 40, 2.0 ** 60])
def test_large_values_without_weight(ratio, types):
    """Visible values `ratio` times the others under a weight of e^-70: the rest keeps its precision."""
    for at in (0, 37, 99):
        s, q = make(dict(lens=[100], rows=[1], Hkv=1, G=3, page=16), 64, f"light.{at}")
        z = np.random.default_rng(1).uniform(-1, 1, 100)
        z[at] = -70
        set_scores(s, q, z)
        set_values(s, np.where(np.arange(100) == at, ratio, 1.0))
        got, lse = attend(s, s.cache(), q, *types, scale=1.0)
        check_rows(s, q, got, lse, *types, scale=1.0, terms=1)


@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("lens,rows,G", [([300], [2], 3), ([5000], [1], 2), ([700] * 4, [160] * 4, 64)],
                         ids=["split", "parts", "prompt"])
@pytest.mark.parametrize("fall", [30, 100])
def test_values_that_shrink_while_their_weights_grow(fall, lens, rows, G, types):
    """Scores grow by 84 along the sequence (weights by 2^121) and values shrink by 2^fall: what counts at
    the end is far under the first values."""
    s, q = make(dict(lens=lens, rows=rows, Hkv=1, G=G, page=16), 64, f"shrink.{fall}.{lens}")
    L = lens[0]
    for b in range(s.B):
        set_scores(s, q, np.linspace(-84, 0, L), b)
        set_values(s, np.exp2(np.linspace(0, -fall, L)), b)
    got, lse = attend(s, s.cache(), q, *types, scale=1.0)
    pick = [int(s.first[b]) + i for b in range(s.B) for i in {0, s.n[b] // 2, s.n[b] - 1}]
    check_rows(s, q, got, lse, *types, scale=1.0, terms=1, rows=pick)


@pytest.mark.parametrize("power,ahead", [(-115, 0), (-60, 30), (0, 30), (110, 0), (110, 30)])
def test_values_that_begin_with_zeros(power, ahead):
    """The first 70 values are zeros, their scores `ahead` of the others; the rest, of any magnitude, enters
    all the same."""
    s, q = make(dict(lens=[200], rows=[2], Hkv=1, G=3, page=16), 64, f"zeros.{power}")
    set_scores(s, q, np.where(np.arange(200) < 70, ahead, 0.0))
    set_values(s, np.where(np.arange(200) < 70, 0.0, 2.0 ** power))
    got, lse = attend(s, s.cache(), q, "f32", "f32", scale=1.0)
    check_rows(s, q, got, lse, "f32", "f32", scale=1.0, terms=1)


# ---------------------------------------------------------------- magnitudes
@pytest.mark.parametrize("shape", [
    dict(lens=[4000], rows=[1], Hkv=1, G=2, page=16, max_len=1),       # whole
    dict(lens=[4000], rows=[1], Hkv=1, G=2, page=16, max_len=4000),    # in parts
    dict(lens=[3000] * 4, rows=[100] * 4, Hkv=2, G=64, page=16, max_len=3000),
    dict(lens=[9001], rows=[130], Hkv=1, G=64, page=64, max_len=9001),
], ids=["whole", "parts", "prompt", "prompt in parts"])
@pytest.mark.parametrize("power", [115, 125, -121])
def test_sums_of_large_and_small_values_of_one_sign(shape, power):
    """Thousands of values of one sign near the ends of fp32 under equal weights: the mean, though their
    sum would pass the type's end."""
    s, q = make(shape, 64, f"mean.{power}")
    for b in range(s.B):
        set_scores(s, q, np.zeros(s.lens[b]), b)
        v = (np.abs(s.x[1][b]).clip(0.5, 1) * 2.0 ** power).astype(np.float32)
        s.quant[1][b] = oracle.kv_quantize(v)
        s.deq[1][b] = oracle.kv_dequant(*s.quant[1][b])
    b = s.batch(max_rows=max(s.n), max_len=shape["max_len"])
    got, lse = w4.kv_attention(torch.from_numpy(q).cuda(), s.cache(), b, want_lse=True)
    check_rows(s, q, got, lse, "f32", "f32", terms=1, rows=[0, s.rows // 2, s.rows - 1])


# ---------------------------------------------------------------- NaN
@pytest.mark.parametrize("D,types", [(64, ("f32", "f32")), (128, ("bf16", "bf16")), (256, ("bf16", "f32"))])
@pytest.mark.parametrize("shape", [SPLIT, PARTS, PROMPT, PROMPT_PARTS], ids=["split", "parts", "prompt", "prompt in parts"])
def test_nan_shows_in_out_and_lse(shape, D, types):
    """A query with a NaN, an infinite one, a key or value of NaN scale: NaN in the rows that have or see
    it, in lse as well (-infinity means a row that sees nothing), and the bits of all others unchanged."""
    s, q = make(shape, D, f"nan.{D}", types[0])
    want, wl = attend(s, s.cache(), q, *types)
    bad = q.copy()
    last = s.rows - 1
    bad[0, 0, 3], bad[0, 1], bad[last, -1, D - 1] = NAN, NAN, INF
    hit = np.zeros(q.shape[:2], dtype=bool)
    hit[0, 0] = hit[0, 1] = hit[last, -1] = True
    got, lse = attend(s, s.cache(), bad, *types)
    h = torch.from_numpy(hit).cuda()
    assert torch.isnan(got[h]).all() and torch.isnan(lse[h]).all()
    assert same_bits(got[~h], want[~h]) and same_bits(lse[~h], wl[~h])
    # keys and values: the second last row of the first sequence and what follows see them
    n, L = s.n[0], s.lens[0]
    p, o = (int(x) for x in s.place(0, L - 2))
    sees = np.arange(s.rows)
    sees = torch.from_numpy((sees >= n - 2) & (sees < n)).cuda()
    for half in "kv":
        cache = s.cache()
        (cache.k_scales if half == "k" else cache.v_scales)[p, 0, o] = NAN
        got, lse = attend(s, cache, q, *types)
        G = shape["G"]
        assert torch.isnan(got[sees][:, :G]).all()
        assert torch.isnan(lse[sees][:, :G]).all() if half == "k" else same_bits(lse, wl)
        assert same_bits(got[~sees], want[~sees]) and same_bits(lse[~sees], wl[~sees])
        assert same_bits(got[sees][:, G:], want[sees][:, G:]) and same_bits(lse[sees][:, G:], wl[sees][:, G:])


def test_all_scores_nan():
    """Every key of NaN scale: NaN, not the result of a row that sees nothing."""
    for shape in (SPLIT, PARTS, PROMPT, PROMPT_PARTS):
        s, q = make(shape, 64, "allnan")
        cache = s.cache()
        cache.k_scales.fill_(NAN)
        got, lse = attend(s, cache, q, "f32", "f32")
        assert torch.isnan(got).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("shape", [SPLIT, PROMPT], ids=["split", "prompt"])
@pytest.mark.parametrize("qp,kp,scale", [(-140, 94, 1.0), (-30, 94, 2.0 ** -100), (-109, 94, 1.0), (-149, 0, 1.0),
                                         (-120, 90, 2.0 ** 30), (124, 14, 2.0 ** -140)])
def test_small_queries_against_large_keys(shape, qp, kp, scale):
    """Queries and scales far under 1 against keys near 2^100, a subnormal scale: scores far from both ends."""
    s, q = make(shape, 64, "tiny")
    q = (np.sign(q) * np.exp2(np.float64(qp)) * np.ceil(np.abs(q))).astype(np.float32)
    for b in range(s.B):
        s.quant[0][b] = oracle.kv_quantize((s.x[0][b] * np.float32(2.0 ** kp)).astype(np.float32))
        s.deq[0][b] = oracle.kv_dequant(*s.quant[0][b])
    got, lse = attend(s, s.cache(), q, "f32", "f32", scale=scale)
    check_rows(s, q, got, lse, "f32", "f32", scale=scale, rows=[0, 3, s.rows - 1])


def test_nan_of_any_payload_stays_nan_in_bf16():
    """A NaN whose mantissa is all ones must not carry into the sign: read back and attended, rows are NaN."""
    s, q = make(SPLIT, 64, "payload")
    cache = s.cache()
    for bits in (0x7FFFFFFF, 0x7F800001, -1, 0x7FC00000):
        for t in (cache.k_scales, cache.v_scales):
            t.view(torch.int32).fill_(bits)
        for x in w4.kv_read(cache, s.batch(), dtype=torch.bfloat16):
            assert torch.isnan(x).all()
        assert torch.isnan(attend(s, cache, q, "f32", "bf16")[0]).all()


def test_rounding_to_bf16():
    """Values on, next to and between two bf16 values, subnormals and the ends of the type: to nearest, ties to
    even, bit for bit as the conversion of the fp32 value."""
    rng = np.random.default_rng(11)
    bits = rng.integers(0, 0x7F80, 4096).astype(np.uint32) << 16
    bits += np.array([0, 1, 0x7FFF, 0x8000, 0x8001, 0xFFFF], dtype=np.uint32)[rng.integers(0, 6, 4096)]
    bits[:8] = [0, 1, 0x8000, 0x8001, 0x00800000, 0x7F7FFFFF, 0x7F7F8000, 0x7F7F7FFF]
    cache = w4.kv_pages(1, 1, 4096, 64)
    cache.k_codes.fill_(0x79)                                  # codes 1 and -1: the scale itself, both signs
    cache.k_scales.copy_(torch.from_numpy(bits.view(np.float32)).view(1, 1, 4096))
    b = w4.KVBatch(torch.tensor([4096], dtype=torch.int32, device="cuda"), rows=4096)
    k = torch.empty((4096, 1, 64), dtype=torch.bfloat16, device="cuda")
    w4.kv_read(cache, b, k=k)
    want = torch.from_numpy(bits.view(np.float32)).bfloat16()
    assert torch.equal(k[:, 0, 0].cpu().view(torch.int16), want.view(torch.int16))
    assert torch.equal(k[:, 0, 63].cpu().view(torch.int16), (-want).view(torch.int16))


# ---------------------------------------------------------------- writing what is not finite
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_write_of_infinities_and_nan_equals_the_single_sequence_codec(dtype):
    """Infinities and NaN among the values: the same codes and scales as w4_kv_quantize's, bit for bit."""
    x = values((40, 3, 128), "wnan", dtype)
    x[0, 0, 5], x[1, 1, 127], x[2, :, 0], x[3, 2] = INF, -INF, NAN, NAN
    x[4, 0, :2], x[5, 0, :3], x[6, 1] = [INF, -INF], [NAN, INF, -INF], INF
    x[7, 2] = 0
    x[7, 2, 9] = NAN
    xd = to_dev(x, dtype)
    codes, scales = w4.kv_cache(3, 40)
    w4.kv_quantize(xd.float(), codes, scales, 0)
    cache = w4.kv_pages(1, 3, 40)
    w4.kv_write(xd, xd, cache, w4.KVBatch(torch.tensor([40], dtype=torch.int32, device="cuda"), rows=40))
    for c, t in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
        assert torch.equal(t[0].view(torch.int32), scales.view(torch.int32))
        assert torch.equal(c[0], codes)


def test_infinite_values_of_later_rows_end_to_end():
    """An overflowed row written into the cache: the rows before it are those of a cache without it."""
    s, q = make(SPLIT, 128, "overflow", "bf16")
    k, v = (to_dev(s.new_rows(i), "bf16") for i in (0, 1))
    cache, b = s.cache(upto=[38, 39]), s.batch()
    w4.kv_write(k, v, cache, b)
    want = w4.kv_attention(to_dev(q, "bf16"), cache, b)
    v[6, 0, 17], k[6, 1, 3] = INF, INF
    w4.kv_write(k, v, cache, b)
    got = w4.kv_attention(to_dev(q, "bf16"), cache, b)
    assert same_bits(got[:6], want[:6]) and same_bits(got[12:], want[12:])
    assert not torch.isfinite(got[6:12]).all()


# ---------------------------------------------------------------- sizes
def test_parts_of_more_rows_than_one_grid_holds():
    """2^26 (row, query head) pairs whose keys are taken in parts: one wavefront each would pass the most
    threads of a launch. One sequence of one row; the other rows belong to none and stay as they are."""
    rows, Hq = 1 << 20, 64
    s = Batch([512], [1], 1, 64, 16, "grid")
    cache = s.cache()
    lens = torch.tensor([512], dtype=torch.int32, device="cuda")
    b = w4.KVBatch(lens, table=torch.from_numpy(s.table).cuda(), rows=rows, max_rows=1, max_len=512,
                   starts=torch.tensor([rows - 1, rows], dtype=torch.int32, device="cuda"))
    assert w4.kv_attention_workspace(cache, b, Hq).numel() > 0
    q = torch.empty((1, Hq, 64), dtype=torch.bfloat16, device="cuda").expand(rows, Hq, 64)
    x = values((1, Hq, 64), "grid.q", "bf16")
    q[-1:].copy_(to_dev(x, "bf16"))                            # one row of queries for all
    out = torch.full((rows, Hq, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, Hq), 3.0, dtype=torch.float32, device="cuda")
    w4.kv_attention(q, cache, b, out=out, lse=lse)
    check_rows(s, x, out[-1:], lse[-1:], "bf16", "bf16")
    assert (out[:-1] == 3.0).all() and (lse[:-1] == 3.0).all()
    del q, out, lse
    torch.cuda.empty_cache()                                   # the workspace alone took 73 GB


# ---------------------------------------------------------------- refusals of the binding
def test_lse_that_is_not_16_byte_aligned_is_refused():
    """A slice of a larger tensor is taken where it begins on 16 bytes, and refused before the launch elsewhere."""
    s, q = make(dict(lens=[20], rows=[2], Hkv=1, G=5, page=16), 64, "align")
    cache, b, qd = s.cache(), s.batch(), torch.from_numpy(q).cuda()
    want = w4.kv_attention(qd, cache, b, want_lse=True)[1]
    hold = torch.full((8, 5), 2.0, device="cuda")
    with pytest.raises(ValueError, match="aligned"):
        w4.kv_attention(qd, cache, b, lse=hold[1:3])
    assert (hold == 2.0).all()
    w4.kv_attention(qd, cache, b, lse=hold[4:6])
    assert same_bits(hold[4:6], want) and (hold[:4] == 2.0).all() and (hold[6:] == 2.0).all()


def test_windows_past_64_bits():
    """A window or sinks past any position, however large a Python number: all positions; negative ones are refused."""
    s, q = make(dict(lens=[70], rows=[3], Hkv=1, G=5, page=16), 64, "span")
    cache, b, qd = s.cache(), s.batch(), torch.from_numpy(q).cuda()
    want = w4.kv_attention(qd, cache, b)
    for big in (2 ** 63 - 1, 2 ** 63, 2 ** 64 + 5):
        assert same_bits(w4.kv_attention(qd, cache, b, window=big), want)
        assert same_bits(w4.kv_attention(qd, cache, b, window=3, sinks=big), want)
        assert w4.kv_attention_workspace(cache, b, 5, window=3, sinks=big).numel() == \
            w4.kv_attention_workspace(cache, b, 5).numel()
    for bad in (-1, -2 ** 64 + 5):
        with pytest.raises(ValueError, match="negative"):
            w4.kv_attention(qd, cache, b, window=bad)
        with pytest.raises(ValueError, match="negative"):
            w4.kv_attention(qd, cache, b, window=3, sinks=bad)


# ---------------------------------------------------------------- repeated calls
@pytest.mark.parametrize("types", [("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("shape", [PARTS, PROMPT], ids=["parts", "prompt"])
def test_repeated_calls_of_mixed_types_give_the_same_bits(shape, types):
    s, q = make(shape, 128, "again", types[0])
    cache = s.cache()
    first = attend(s, cache, q, *types)
    for _ in range(3):
        for x, y in zip(attend(s, cache, q, *types), first):
            assert same_bits(x, y)
