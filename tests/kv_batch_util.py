"""A batch of sequences for the tests of the batched INT4 KV cache: seeded vectors,
their codes by the oracle, a shuffled page table, and the oracle's attention."""
import numpy as np
import torch

import bit_weight_only_quantize_amd as w4
import oracle
import synth

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def values(shape, name, dtype="f32", seed=0):
    """Seeded vectors with a spread of magnitudes, as the values `dtype` holds (fp32 array)."""
    x = synth.normal_f32(shape, 1.0, seed, name)
    x = x * np.exp(0.4 * synth.normal_f32(shape[:-1] + (1,), 1.0, seed, name + ".mag")).astype(np.float32)
    if dtype == "bf16":
        x = (synth.bf16_bits_from_f32(x).astype(np.uint32) << 16).view(np.float32)
    return np.ascontiguousarray(x)


def to_dev(x, dtype):
    return torch.from_numpy(x).to(DT[dtype]).cuda()      # exact: x holds values of dtype


class Batch:
    """Sequences of the given lengths, the last rows[b] positions of each being rows of the call."""

    def __init__(self, lens, rows, Hkv, D, page, name, spare=2, vec_dtype="f32"):
        self.lens, self.n, self.Hkv, self.D, self.page = list(lens), list(rows), Hkv, D, page
        self.B = len(self.lens)
        self.first = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        self.rows = int(self.first[-1])
        # vectors [Hkv][L][D] of every sequence
        self.x = [[values((Hkv, L, D), f"{name}.{kv}.{b}", vec_dtype) for b, L in enumerate(self.lens)]
                  for kv in "kv"]
        self.quant = [[oracle.kv_quantize(a) if a.shape[1] else (np.zeros((Hkv, 0, D // 2), np.uint8),
                                                                np.zeros((Hkv, 0), np.float32)) for a in half]
                      for half in self.x]
        self.deq = [[oracle.kv_dequant(c, s) for c, s in half] for half in self.quant]
        if page:
            self.size = page
            need = [-(-L // page) for L in self.lens]
            self.pages = sum(need) + spare
            order = np.random.default_rng(len(name) + sum(self.lens)).permutation(self.pages)
            self.table = np.full((self.B, max(1, max(need))), -7, dtype=np.int32)
            at = 0
            for b, m in enumerate(need):
                self.table[b, :m] = order[at:at + m]
                at += m
        else:
            self.size, self.pages, self.table = max(1, max(self.lens)) + 3, self.B, None

    def place(self, b, t):
        return (b, t) if self.table is None else (self.table[b, t // self.size], t % self.size)

    def host_pool(self, upto=None):
        """Codes and scales with each sequence's first upto[b] positions (default: all) in place, and
        everything else stale: codes 0x5A and scales NaN."""
        pool = []
        for half in self.quant:
            codes = np.full((self.pages, self.Hkv, self.size, self.D // 2), 0x5A, dtype=np.uint8)
            scales = np.full((self.pages, self.Hkv, self.size), np.nan, dtype=np.float32)
            for b, (c, s) in enumerate(half):
                t = np.arange(self.lens[b] if upto is None else upto[b])
                if t.size:
                    p, o = self.place(b, t)
                    codes[p, :, o] = c[:, t].transpose(1, 0, 2)
                    scales[p, :, o] = s[:, t].transpose(1, 0)
            pool += [codes, scales]
        return pool

    def cache(self, upto=None):
        return w4.KVPages(*[torch.from_numpy(a).cuda() for a in self.host_pool(upto)])

    def batch(self, starts=True, rows=None, **kw):
        dev = lambda a: None if a is None else torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()
        return w4.KVBatch(dev(self.lens), table=dev(self.table), starts=dev(self.first) if starts else None,
                          rows=self.rows if rows is None else rows, **kw)

    def new_rows(self, kv):
        """Rows of the call [rows][Hkv][D], packed in sequence order; rows at no position are zeros."""
        out = np.zeros((self.rows, self.Hkv, self.D), dtype=np.float32)
        for b, (L, n) in enumerate(zip(self.lens, self.n)):
            m = min(L, n)
            out[self.first[b] + n - m:self.first[b] + n] = self.x[kv][b][:, L - m:L].transpose(1, 0, 2)
        return out

    def attend(self, q, scale, window=0, sinks=0):
        """The oracle's attention of packed rows q [rows][Hq][D]."""
        parts = [oracle.kv_attention(q[self.first[b]:self.first[b + 1]], self.deq[0][b], self.deq[1][b], scale,
                                     window, sinks) for b in range(self.B)]
        return [np.concatenate(p) for p in zip(*parts)]


def bounds(ref, D, L, vmax, q_dtype, out_dtype, terms=None):
    """Bounds of the errors of out and lse that the arithmetic allows; u = 2^-24, half a step of fp32.

    Scores. A bf16 query is exact in the 16-bit format of the products but for what falls under its
    least step, 2^-25 of the row's maximum < u max|q|; an fp32 one goes in two pieces of 11 bits, off
    by 2^-22 |q| = 4 u |q| at most. Products with the integer codes (stored plus 8, the offset's part a
    term of its own: Z and Zmax count both) are exact, their 2 D terms (two pieces) add up in fp32 to
    2 D u, the scalings to 4 u, the exponent's argument to 4 u (Z + |m|) with
    the running maximum m, |m| <= Z, and the exponential is good to 2^-22:
        dz = u (Zmax + (2 D + 16) Z) + 2^-22.
    (`terms`: elements of a query that are not 0, in place of D; adding a zero product is exact.)
    Weights. e^z is off by w = e^(2 dz) - 1 (a row's weight and its maximum's), and sums of L terms by
    L u, in numerator and denominator. The weight times the value's scale enters the second product
    in 16 bits: half a step is 2^-11 of it, 2^-22 in the two pieces that an fp32 query or output
    takes; below that the format's least step is 2^-33 of the largest value for each of L keys.
    A bf16 output adds its own half step, 2^-8 of the value."""
    out, lse, A, Z, Zmax = ref
    u = 2.0 ** -24
    dz = u * ((Zmax if terms is None else 0) + (2 * (D if terms is None else terms) + 16) * Z) + 2.0 ** -22
    w = np.expm1(2 * dz) + L * u
    piece = 2.0 ** -22 if "f32" in (q_dtype, out_dtype) else 2.0 ** -11
    e = (2 * w + piece + 4 * u)[..., None] * A + L * 2.0 ** -33 * vmax
    if out_dtype == "bf16":
        e = e * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(out)
    return e, dz + w + 4 * u * (1 + np.abs(np.where(np.isfinite(lse), lse, 0)))
