"""Refusals of the mixture-of-experts entry points (no GPU: every call fails
before anything is launched)."""
import ctypes

import pytest

from quantized_matmul_03_b200 import binding

FAKE = ctypes.c_void_p(0x10000)        # aligned, never dereferenced
ODD = ctypes.c_void_p(0x10002)
OFF16 = ctypes.c_void_p(0x10008)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6


@pytest.fixture(scope="module")
def L():
    from quantized_matmul_03_b200 import build
    build.build()
    return binding.lib()


def route(L, **kw):
    a = dict(logits=FAKE, dtype=0, T=4, E=16, bias=None, score=0, G=1, tg=1, gt=1, k=2, renorm=1, scale=1.0,
             idx=FAKE, w=FAKE)
    a.update(kw)
    return L.qmm_moe_route(a["logits"], a["dtype"], a["T"], a["E"], a["bias"], a["score"], a["G"], a["tg"],
                           a["gt"], a["k"], a["renorm"], a["scale"], a["idx"], a["w"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 0), (dict(T=0, logits=None), 0),
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(E=1025), INVALID), (dict(dtype=3), INVALID),
    (dict(score=2), INVALID), (dict(G=3), INVALID), (dict(G=0), INVALID), (dict(E=64, G=64), INVALID),
    (dict(G=4, tg=5), INVALID), (dict(G=4, tg=0), INVALID), (dict(gt=3), INVALID), (dict(gt=0), INVALID),
    (dict(k=0), INVALID), (dict(k=17), INVALID), (dict(E=64, k=33), INVALID), (dict(G=4, tg=1, k=5), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(logits=None), INVALID), (dict(logits=ODD), INVALID), (dict(idx=None), INVALID), (dict(w=ODD), INVALID),
    (dict(bias=ODD), INVALID), (dict(T=2 ** 31), UNSUPPORTED),
])
def test_route_refusals(L, kw, status):
    assert route(L, **kw) == status


def experts(L, **kw):
    a = dict(x=FAKE, T=4, K=128, dtype=1, idx=FAKE, w=FAKE, k=2, wq=FAKE, s=FAKE, b=None, down=FAKE, E=4, I=128,
             N=128, gs=32, bits=4, mode=b"mxfp4", act=0, y=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return L.qmm_moe_experts(a["x"], a["T"], a["K"], a["dtype"], a["idx"], a["w"], a["k"], a["wq"], a["s"], a["b"],
                             a["wq"], a["s"], a["b"], a["down"], a["s"], a["b"], a["E"], a["I"], a["N"], a["gs"],
                             a["bits"], a["mode"], a["act"], a["y"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 0), (dict(N=0), 0), (dict(T=0, x=None, ws=None), 0),
    (dict(T=-1), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID), (dict(I=0), INVALID),
    (dict(E=0), INVALID), (dict(E=1025), INVALID), (dict(k=0), INVALID), (dict(k=33), INVALID),
    (dict(act=2), INVALID), (dict(mode=b"fp5"), INVALID), (dict(gs=64), INVALID), (dict(bits=8), INVALID),
    (dict(mode=b"mxfp8", bits=8), UNSUPPORTED), (dict(mode=b"affine", bits=8, b=FAKE), UNSUPPORTED),
    (dict(dtype=0), UNSUPPORTED), (dict(K=96), UNSUPPORTED), (dict(I=96), UNSUPPORTED),
    (dict(K=48), INVALID), (dict(mode=b"affine", gs=128, b=FAKE, K=192), INVALID),
    (dict(T=2 ** 29 + 1), UNSUPPORTED), (dict(I=2 ** 25), UNSUPPORTED), (dict(N=2 ** 29), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(wq=OFF16), INVALID), (dict(s=None), INVALID),
    (dict(down=None), INVALID), (dict(b=FAKE), INVALID), (dict(mode=b"affine"), INVALID),
    (dict(idx=None), INVALID), (dict(w=ODD), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=OFF16), WORKSPACE), (dict(wsb=16), WORKSPACE),
])
def test_experts_refusals(L, kw, status):
    assert experts(L, **kw) == status


def test_workspace_size(L):
    f = L.qmm_moe_experts_workspace_size
    assert f(0, 128, 2, 4, 128, 128, 1) == 0
    assert f(4, 128, 2, 4, 128, 128, 0) == 0            # f32 is refused
    one, many = f(1, 128, 2, 4, 128, 128, 1), f(64, 128, 2, 4, 128, 128, 1)
    assert 0 < one <= many
    need = f(4, 128, 2, 4, 128, 128, 1)
    assert experts(L, wsb=need - 1) == WORKSPACE


def test_forced_decode_path_is_refused(L):
    assert L.qmm_set_path(binding.PATHS["decode_tc"]) == 0
    try:
        assert experts(L) == UNSUPPORTED
    finally:
        L.qmm_set_path(0)
