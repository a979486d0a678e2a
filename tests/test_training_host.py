"""Host-side checks of the arguments of the layer norm, the balance loss and its
gradient, the router's backward from all logits and the calls on z in 8 bits (no GPU
needed: every call here fails validation or has nothing to do)."""
import ctypes

import pytest

import sigmoid_top_routing_02_amd as moe

F = ctypes.c_void_p(0x10000)        # aligned, never dereferenced
MIS = ctypes.c_void_p(0x10004)
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    return moe.load_library()


def _each_pointer(call, n, optional=()):
    """call(pointers): every NULL and every misaligned one is refused."""
    for i in range(n):
        for bad, want in ((None, -1), (MIS, -5)):
            if bad is None and i in optional:
                continue
            p = [F] * n
            p[i] = bad
            assert call(p) == want, (i, want)


def test_add_layernorm(L):
    def f(p=None, x=0, r=0, w=1, T=4, d=128, eps=1e-5, **kw):
        p = p or [F] * 10
        return L.moe_add_layernorm(p[0], x, p[1], r, p[2], p[3], w, T, d, eps, *p[4:], None)
    assert f(T=-1) == -2 and f(d=0) == -2 and f(d=16385) == -3 and f(d=100) == -2
    for eps in (-1e-6, NAN):
        assert f(eps=eps) == -3
    assert f(x=2) == -3 and f(r=-1) == -3 and f(w=7) == -3
    p = [F] * 10
    p[6] = None
    assert f(p) == -1                                            # scale without q
    p = [F] * 10
    p[7] = None
    assert f(p) == -1                                            # q without scale
    p = [F] * 10
    p[1] = None
    assert f(p) == -1                                            # h_out without a residual
    for i in range(10):
        p = [F] * 10
        p[i] = MIS
        assert f(p) == -5, i
    for i in (0, 2):
        p = [F] * 10
        p[i] = None
        assert f(p) == -1
    assert f([None] * 10, T=0) == 0


def test_add_layernorm_backward(L):
    size = L.moe_add_layernorm_backward_workspace_bytes
    assert size(0, 128) == 0 and size(4, 0) == 0 and size(4, 16385) == 0 and size(-1, 128) == 0
    assert 0 < size(1, 1) and size(2 ** 62, 16384) == 2 * 512 * 16384 * 4
    need = size(4, 128)

    def f(p=None, t=(0, 0, 1, 0), T=4, d=128, n=need):
        p = p or [F] * 10
        return L.moe_add_layernorm_backward(p[0], t[0], p[1], t[1], p[2], t[2], p[3], p[4], p[5], T, d, p[6], t[3], p[7],
                                            p[8], p[9], n, None)
    assert f(T=-1) == -2 and f(d=0) == -2 and f(d=16385, n=1 << 40) == -3 and f(n=need - 1) == -4
    for t in ((2, 0, 0, 0), (0, 2, 0, 0), (0, 0, 2, 0), (0, 0, 0, 2)):
        assert f(t=t) == -3
    _each_pointer(f, 10, optional=(5, 8))                         # dh, db
    assert f([None] * 10, T=0, n=0) == -1                         # dw, also with T = 0


def test_balance_loss(L):
    size = L.moe_balance_loss_workspace_bytes
    assert size(-1, 1) == 0 and size(2 ** 30 + 1, 1) == 0 and size(4, 0) == 0 and size(4, 2 ** 20 + 1) == 0
    assert size(2 ** 30, 2 ** 20) > size(4096, 2) > 16
    assert size(0, 1) == size(64, 2) == 16                        # small calls take none

    def f(p=None, n_seq=2, T=4096, E=16, K=4, n=1 << 30):
        p = p or [F] * 7
        return L.moe_balance_loss(p[0], p[1], p[2], n_seq, T, E, K, 1e-3, p[3], p[4], p[5], p[6], n, None)

    def b(p=None, n_seq=2, T=64, E=16, K=4):
        p = p or [F] * 6
        return L.moe_balance_loss_backward(p[0], p[1], p[2], n_seq, T, E, K, 1e-3, p[3], p[4], p[5], None)
    for g in (f, b):
        assert g(T=-1) == -2 and g(T=2 ** 30 + 1) == -3 and g(E=0) == -3 and g(E=257) == -3
        assert g(K=0) == -3 and g(K=17, E=64) == -3 and g(K=5, E=4) == -3
        assert g(n_seq=0) == -3 and g(n_seq=2 ** 20 + 1) == -3
    _each_pointer(f, 7, optional=(5,))                            # without seq_start: two sequences
    _each_pointer(b, 6, optional=(3, 4))                          # dloss, dlogits_in
    assert f(n=size(4096, 2) - 1) == -4
    assert b([None] * 6, n_seq=1, T=0) == 0


def test_router_logits_backward(L):
    size = L.moe_router_logits_backward_workspace_bytes
    assert size(-1, 128, 4) == 0 and size(2 ** 24 + 1, 128, 4) == 0 and size(4, 100, 4) == 0 and size(4, 0, 4) == 0
    assert size(4, 65664, 4) == 0 and size(4, 128, 0) == 0 and size(4, 128, 257) == 0
    assert size(0, 128, 4) == size(4, 128, 4) == 16 < size(5000, 128, 4)          # small calls take none

    def f(p=None, T=5000, d=128, E=16, n=1 << 40):
        p = p or [F] * 8
        return L.moe_router_logits_backward(p[0], p[1], p[2], T, d, E, p[3], p[4], p[5], p[6], p[7], n, None)
    assert f(T=-1) == -2 and f(T=2 ** 24 + 1) == -3 and f(d=0) == -2 and f(d=192) == -2 and f(d=65664) == -3
    assert f(E=0) == -3 and f(E=257) == -3
    _each_pointer(f, 8, optional=(3, 4))
    assert f(n=size(5000, 128, 16) - 1) == -4
    assert f([F, F, F, None, None, None, None, F]) == -1          # nothing asked for
    assert f([F, F, F, F, None, None, F, F]) == -1                # du_in without du


def test_swiglu_zq(L):
    def g(p=None, G=2, M=8, N=256, K=128, n=1 << 30):
        p = p or [F] * 10
        return L.grouped_gemm_fp8_swiglu_zq(p[0], p[1], p[2], p[3], G, M, p[4], p[5], N, K, p[6], p[7], p[8], p[9], F, n, None)
    assert g(G=0) == -3 and g(M=-1) == -3 and g(N=128) == -2 and g(K=100) == -2 and g(K=16512) == -3
    _each_pointer(g, 10, optional=(2,))
    assert g(n=L.moe_gemm_workspace_bytes(2, 8, 256, 128) - 1) == -4
    assert g([None] * 10, M=0) == 0

    def f(p=None, R=4, I=128):
        p = p or [F] * 5
        return L.moe_swiglu_backward_zq(p[0], p[1], p[2], R, I, p[3], p[4], None)
    assert f(R=-1) == -2 and f(I=0) == -2 and f(I=100) == -2 and f(R=2 ** 31) == -3 and f(I=65664) == -3
    _each_pointer(f, 5)
    assert f([None] * 5, R=0) == 0

    def w(p=None, G=2, n_kb=3, T=4, K=2, d=128, I=128):
        p = p or [F] * 18
        return L.moe_wgrad_operands_zq(*p[:10], G, n_kb, T, K, d, I, 8, *p[10:], None)
    assert w(G=0) == -3 and w(n_kb=-1) == -3 and w(K=17) == -3 and w(d=100) == -2 and w(I=0) == -2 and w(T=-1) == -2
    _each_pointer(w, 18)
    assert L.moe_last_error().startswith(b"moe_wgrad_operands_zq: ")
    assert w([None] * 18, n_kb=0) == 0
