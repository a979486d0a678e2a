"""Host-side checks of the residual RMS norm's and the MXFP4 calls' arguments
(no GPU needed: every call here fails validation or has nothing to do)."""
import ctypes

import pytest

import sigmoid_top_routing_02_amd as moe

F = ctypes.c_void_p(0x10000)        # aligned, never dereferenced
MIS = ctypes.c_void_p(0x10004)
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    return moe.load_library()


def test_add_rmsnorm(L):
    f = L.moe_add_rmsnorm
    assert f(F, 0, F, 0, F, 1, -1, 128, 1e-6, F, F, F, F, F, None) == -2             # T < 0
    assert f(F, 0, F, 0, F, 1, 4, 0, 1e-6, F, F, None, None, F, None) == -2          # d < 1
    assert f(F, 0, F, 0, F, 1, 4, 16385, 1e-6, F, F, None, None, F, None) == -3      # d above the limit
    assert f(F, 0, F, 0, F, 1, 4, 100, 1e-6, F, F, F, F, F, None) == -2              # q with d % 128
    assert f(F, 0, F, 0, F, 1, 4, 128, 1e-6, F, F, F, None, F, None) == -1           # q without scale
    assert f(F, 0, F, 0, F, 1, 4, 128, 1e-6, F, F, None, F, F, None) == -1           # scale without q
    assert f(F, 0, None, 0, F, 1, 4, 128, 1e-6, F, F, F, F, F, None) == -1           # h_out without a residual
    for eps in (-1e-6, NAN):
        assert f(F, 0, F, 0, F, 1, 4, 128, eps, F, F, F, F, F, None) == -3
    for types in ((2, 0, 1), (0, -1, 1), (0, 0, 7)):
        assert f(F, types[0], F, types[1], F, types[2], 4, 128, 1e-6, F, F, F, F, F, None) == -3
    ptrs = [F] * 8                                                                   # x, residual, weight, outputs
    for i in range(8):
        p = list(ptrs)
        p[i] = MIS
        r = f(p[0], 0, p[1], 0, p[2], 1, 4, 128, 1e-6, p[3], p[4], p[5], p[6], p[7], None)
        assert r == -5, i
    assert f(None, 0, F, 0, F, 1, 4, 128, 1e-6, F, F, F, F, F, None) == -1
    assert f(F, 0, F, 0, None, 1, 4, 128, 1e-6, F, F, F, F, F, None) == -1
    assert f(None, 0, None, 0, None, 1, 0, 128, 1e-6, None, None, None, None, None, None) == 0


def test_add_rmsnorm_backward(L):
    size = L.moe_add_rmsnorm_backward_workspace_bytes
    assert size(0, 128) == 0 and size(4, 0) == 0 and size(4, 16385) == 0 and size(-1, 128) == 0
    assert 0 < size(1, 1) and size(2 ** 62, 16384) == size(512, 16384) == 512 * 16384 * 4
    f, need = L.moe_add_rmsnorm_backward, size(4, 128)
    assert f(F, 0, F, 0, F, 1, F, F, -1, 128, F, 0, F, F, need, None) == -2
    assert f(F, 0, F, 0, F, 1, F, F, 4, 0, F, 0, F, F, need, None) == -2
    assert f(F, 0, F, 0, F, 1, F, F, 4, 16385, F, 0, F, F, 1 << 40, None) == -3
    assert f(F, 0, F, 0, F, 1, F, F, 4, 128, F, 0, F, F, need - 1, None) == -4
    for t in ((2, 0, 0, 0), (0, 2, 0, 0), (0, 0, 2, 0), (0, 0, 0, 2)):
        assert f(F, t[0], F, t[1], F, t[2], F, F, 4, 128, F, t[3], F, F, need, None) == -3
    for i in (0, 1, 2, 3, 5, 6, 7):                                                  # dh (4) may be NULL
        for bad, want in ((None, -1), (MIS, -5)):
            p = [F] * 8
            p[i] = bad
            r = f(p[0], 0, p[1], 0, p[2], 1, p[3], p[4], 4, 128, p[5], 0, p[6], p[7], need, None)
            assert r == want, (i, want)
    assert f(F, 0, F, 0, F, 1, F, MIS, 4, 128, F, 0, F, F, need, None) == -5
    assert f(None, 0, None, 0, None, 1, None, None, 0, 128, None, 0, None, None, 0, None) == -1   # dw, also with T = 0


def test_quantisers(L):
    for f, unit in ((L.mxfp4_quant_1x32, 32), (L.mxfp4_dequant_1x32, 32), (L.fp8_dequant_1x128, 128)):
        def call(p, dt, rows, cols, f=f):
            if f is L.mxfp4_quant_1x32:
                return f(p[0], dt, rows, cols, p[1], p[2], None)
            return f(p[0], p[1], rows, cols, p[2], dt, None)
        assert call([F] * 3, 0, -1, unit) == -2
        assert call([F] * 3, 0, 4, 0) == -2
        assert call([F] * 3, 0, 4, unit + 16) == -2
        assert call([F] * 3, 2, 4, unit) == -3
        assert call([F] * 3, 0, 1 << 32, unit) == -3
        for i in range(3):
            for bad, want in ((None, -1), (MIS, -5)):
                p = [F] * 3
                p[i] = bad
                assert call(p, 0, 4, unit) == want
        assert call([None] * 3, 0, 0, unit) == 0


def test_grouped_gemm_mxfp4(L):
    def f(p=None, a_rows=8, index=F, G=2, M=8, N=256, K=64, epi=0, out=F, out_q=None, out_s=None):
        p = p or [F] * 5
        return L.grouped_gemm_mxfp4(p[0], p[1], a_rows, index, p[2], G, M, p[3], p[4], N, K, epi, out, out_q, out_s,
                                    None)
    assert f(G=0) == -3 and f(G=1025) == -3
    assert f(M=-1) == -3 and f(M=2 ** 31 - 65535) == -3
    assert f(K=0) == -2 and f(K=48) == -2 and f(N=0) == -2
    assert f(epi=4) == -3 and f(epi=-1) == -3
    for epi, outs in ((2, dict()), (3, dict(out=None, out_q=F, out_s=F))):
        assert f(epi=epi, N=384, **outs) == -2
    assert f(a_rows=1 << 31) == -3 and f(a_rows=-1) == -3
    assert f(a_rows=1 << 20, K=16384) == -3                                          # A past 32-bit offsets
    assert f(N=1 << 20, K=16384) == -3                                               # a group's B past them
    assert f(index=None, a_rows=7) == -2
    for i in range(5):
        for bad, want in ((None, -1), (MIS, -5)):
            p = [F] * 5
            p[i] = bad
            assert f(p) == want
    assert f(index=MIS) == -5
    assert f(out=None) == -1 and f(out=MIS) == -5 and f(out_q=F) == -3 and f(out_s=F) == -3
    assert f(epi=3, out=F, out_q=F, out_s=F) == -3
    assert f(epi=3, out=None, out_q=None, out_s=F) == -1 and f(epi=3, out=None, out_q=F, out_s=MIS) == -5
    assert f([None] * 5, a_rows=0, index=None, M=0, out=None) == 0
