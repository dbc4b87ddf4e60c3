"""Host-side checks of the microscaled 4-bit calls, the selection of experts and their FFN: sizes,
and the documented refusals, before anything is launched (no GPU)."""
import ctypes

import pytest

import bit_weight_only_quantize_amd as w4

pytestmark = pytest.mark.cpu
L = w4.lib()


def mat(N=64, K=128, E=1, scheme=3, codes=16, scale=16):
    return w4._W4Matrix(scheme, E, N, K, codes, scale, None)


def rows(stride=128, dtype=1, data=16):
    return w4._W4Rows(data, dtype, stride, 0)


def test_packed_sizes():
    assert w4.packed_sizes("mx4_g32", 3, 96) == (144, 9, 0)
    with pytest.raises(w4.W4Error) as e:
        w4.packed_sizes("mx4_g32", 3, 48)
    assert e.value.code == -2


def test_quantize_and_read_refuse():
    q = L.w4_mx4_quantize
    assert q(rows(), 0, 128, None, None, None) == 0
    assert q(rows(), 4, 48, 16, 16, None) == -2
    assert q(rows(), -1, 64, 16, 16, None) == -2
    assert q(rows(), 4, 0, 16, 16, None) == -2
    assert q(rows(), 1 << 31, 64, 16, 16, None) == -2
    assert q(None, 4, 64, 16, 16, None) == -1
    assert q(rows(data=None), 4, 64, 16, 16, None) == -1
    assert q(rows(dtype=2), 4, 64, 16, 16, None) == -1
    assert q(rows(), 4, 64, None, 16, None) == -1
    assert q(rows(), 4, 64, 8, 16, None) == -3
    assert q(rows(data=8), 4, 64, 16, 16, None) == -3
    assert q(rows(stride=132), 4, 64, 16, 16, None) == -3          # 264 bytes
    assert q(rows(stride=32), 4, 64, 16, 16, None) == -2           # rows overlap
    assert L.w4_quantize_pack(3, 16, 4, 48, 16, 16, None, None) == -2
    assert L.w4_quantize_pack(3, None, 4, 64, 16, 16, None, None) == -1
    assert L.w4_quantize_pack(3, 16, 0, 64, 16, 16, None, None) == 0
    r = L.w4_mx4_read
    assert r(mat(N=0), rows(), None) == 0
    assert r(mat(scheme=1), rows(), None) == -1
    assert r(mat(E=2), rows(), None) == -2
    assert r(mat(), rows(stride=64), None) == -2
    assert r(mat(), rows(stride=129, dtype=0), None) == -3
    assert r(mat(scale=None), rows(), None) == -1


def test_products_refuse():
    g = L.w4_mx4_gemm
    ok = dict(W=mat(), X=rows(), M=3, Y=rows(stride=64), ws=None, wb=0)

    def call(f=g, **kw):
        a = dict(ok, **kw)
        if f is L.w4a4_mx4_gemm:
            return f(a["W"], a["X"], a["Y"], a["ws"], a["wb"], None)
        return f(a["W"], a["X"], a["M"], a["Y"], a["ws"], a["wb"], None)

    assert call(M=0) == 0 and call(W=mat(N=0)) == 0
    assert call(W=mat(scheme=0)) == -1
    assert call(W=mat(E=2)) == -2
    assert call(W=mat(K=48)) == -2
    assert call(W=mat(codes=24)) == -3
    assert call(M=-1) == -2 and call(M=1 << 31) == -2
    assert call(X=rows(dtype=0)) == -1                             # fp32 activations
    assert call(X=rows(stride=120)) == -2
    assert call(X=rows(stride=130)) == -3
    assert call(X=None) == -1 and call(Y=None) == -1
    assert call(Y=rows(stride=63)) == -2
    assert call(Y=rows(stride=64, dtype=3)) == -1
    assert call(Y=rows(stride=64, data=2)) == -3
    assert call(ws=None, wb=64) == -5
    a4 = L.w4a4_mx4_gemm
    assert call(a4, X=mat(N=0)) == 0
    assert call(a4, X=mat(N=3, K=64)) == -2
    assert call(a4, X=mat(N=3, scheme=2)) == -1
    assert call(a4, X=mat(N=3, E=2)) == -2
    assert call(a4, X=mat(N=3), Y=rows(stride=10)) == -2
    assert L.w4_mx4_gemm_workspace_bytes(mat(), 0, 0) == 0 and L.w4_mx4_gemm_workspace_bytes(None, 4, 0) == 0
    # the other products do not take the scheme
    d = ctypes.byref(mat())
    assert L.w4a16_gemv(d, 16, 1, 16, None) == -1
    assert L.w4a16_gemm(d, 16, 1, 16, None) == -1
    assert L.w4a16_moe_gemv(d, d, d, None, None, None, 16, 1, 16, 16, 1, 16, 1 << 20, 16, None) == -1
    assert L.w4_mx4_gemm_workspace_bytes(mat(scheme=0), 4, 0) == 0


def test_selection_refuses():
    def call(M=3, E=64, x=None, score=0, k=4, groups=1, top=1, best=1, scale=1.0, bias=None, ids=16, w=16):
        how = w4._W4Select(score, k, groups, top, best, 0, scale, bias)
        return L.w4_moe_select(rows(stride=64, dtype=0) if x is None else x, M, E, how, ids, w, None)

    assert call(M=0) == 0
    assert call(score=2) == -1 and call(scale=float("inf")) == -1 and call(scale=float("nan")) == -1
    assert call(E=0) == -2 and call(E=1025) == -2 and call(M=-1) == -2
    assert call(groups=7) == -2 and call(groups=0) == -2 and call(groups=8, top=9) == -2 and call(top=0) == -2
    assert call(E=128, groups=128) == -2
    assert call(groups=64, top=64, best=2) == -2                   # groups of one expert
    assert call(best=3) == -2 and call(best=0) == -2
    assert call(k=0) == -2 and call(k=33) == -2 and call(k=9, groups=8, top=1) == -2
    assert call(E=4, k=5) == -2
    assert call(x=rows(stride=63, dtype=0)) == -2
    assert call(x=rows(stride=64, dtype=2)) == -1
    assert call(ids=None) == -1 and call(w=None) == -1
    assert call(ids=8) == -3 and call(w=8) == -3 and call(bias=8) == -3
    assert L.w4_moe_select(rows(), 3, 64, None, 16, 16, None) == -1


def test_experts_refuse():
    E, D, F = 4, 128, 64
    need = L.w4_mx4_moe_workspace_bytes(3, 2, E, D, F)
    assert need >= 3 * 2 * (2 * F + 2 * D)

    def call(gate=mat(F, D, E), up=mat(F, D, E), down=mat(D, F, E), x=rows(stride=D), M=3, ids=16, w=16, k=2, act=0,
             y=rows(stride=D), ws=16, wb=need):
        return L.w4_mx4_moe(gate, up, down, x, M, ids, w, k, act, y, ws, wb, None)

    assert call(M=0) == 0
    assert call(gate=mat(F, D, E, scheme=1)) == -1
    assert call(up=mat(F, D, 3)) == -2 and call(up=mat(F + 32, D, E)) == -2 and call(down=mat(D, F + 32, E)) == -2
    assert call(gate=mat(F, D, 1025), up=mat(F, D, 1025), down=mat(D, F, 1025)) == -2
    assert call(act=2) == -1 and call(k=0) == -2 and call(k=33) == -2 and call(M=-1) == -2
    assert call(M=(1 << 23) + 1) == -2                             # M * top_k > 2^24
    assert call(x=rows(stride=D, dtype=0)) == -1 and call(y=rows(stride=D, dtype=0)) == -1
    assert call(x=rows(stride=D - 8)) == -2 and call(y=rows(stride=D - 8)) == -2
    assert call(ids=None) == -1 and call(w=4) == -3
    assert call(ws=None) == -5 and call(wb=need - 1) == -5 and call(ws=8) == -3
    assert L.w4_mx4_moe_workspace_bytes(0, 2, E, D, F) == 0
    assert L.w4_mx4_moe_workspace_bytes(1 << 24, 2, E, D, F) == 0


def test_workspaces_of_all_kinds_of_sizes():
    """Host-only: every plan has a size, whole blocks of fp32 sums for each piece of K, 0 for up to 16 rows."""
    pieces = set()
    for x4 in (0, 1):
        for N in (1, 129, 1000, 4096, 11008, 152064):
            for K in (32, 992, 4096, 11008, 65536):
                for M in (1, 16, 17, 64, 100, 128, 129, 200, 256, 300, 512, 1000, 4097):
                    n = L.w4_mx4_gemm_workspace_bytes(mat(N, K), M, x4)
                    assert n % (64 * 128 * 4) == 0 and (M > 16 or n == 0), (x4, N, K, M)
                    assert n <= 16 * 4 * (M + 255) * (N + 255)
                    pieces.add((x4, n > 0))
    assert len(pieces) == 4
