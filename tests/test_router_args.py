"""Refusals of the norm and the router, before any launch (CPU)."""
import ctypes

import pytest
import torch

import __graft_entry__
import lora_moe_expert_info_gb300 as mlr
from lora_moe_expert_info_gb300 import norm, router

BF, F32 = torch.bfloat16, torch.float32
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: the calls return before any launch
ODD = ctypes.c_void_p(0x1001)
INVALID, UNSUPPORTED, CAPACITY = mlr.MLR_ERR_INVALID, mlr.MLR_ERR_UNSUPPORTED, mlr.MLR_ERR_CAPACITY
BIG = ctypes.c_size_t(1 << 40)


@pytest.fixture(scope="module", autouse=True)
def lib():
    __graft_entry__.build()
    norm._lib(), router._lib()
    return mlr.library()


def rms(lib, x=FAKE, res=None, w=FAKE, T=4, H=64, dtype=0, w_dtype=0, eps=1e-6, y=FAKE, r=None, codes=None, exps=None):
    return lib.moe_rms_norm(x, res, w, T, H, dtype, w_dtype, eps, y, r, codes, exps, None)


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=16385), UNSUPPORTED), (dict(dtype=2), INVALID), (dict(w_dtype=-1), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(y=None), INVALID), (dict(res=FAKE), INVALID), (dict(r=FAKE), INVALID), (dict(codes=FAKE), INVALID),
    (dict(exps=FAKE), INVALID), (dict(x=ODD), INVALID), (dict(w=ODD), INVALID), (dict(y=ODD), INVALID),
    (dict(res=ODD, r=FAKE), INVALID), (dict(T=0), 0), (dict(T=0, x=None, y=FAKE), 0),
])
def test_norm_refusals(lib, bad, code):
    assert rms(lib, **bad) == code


def test_norm_gradient_refusals(lib):
    def f(dy=FAKE, r=FAKE, w=FAKE, d_r=None, T=4, H=64, dtype=0, w_dtype=0, eps=1e-6, dx=FAKE, dw=FAKE, ws=FAKE, n=BIG):
        return lib.moe_rms_norm_backward(dy, r, w, d_r, T, H, dtype, w_dtype, eps, dx, dw, ws, n, None)
    need = lib.moe_rms_norm_backward_workspace_bytes(4, 64, 0)
    assert need >= 64 * 4 and lib.moe_rms_norm_backward_workspace_bytes(0, 64, 0) > 0
    for bad in ((-1, 64, 0), (4, 0, 0), (4, 16385, 0), (4, 64, 2)):
        assert lib.moe_rms_norm_backward_workspace_bytes(*bad) == 0
    for bad in (dict(dy=None), dict(r=None), dict(dx=None), dict(dw=None), dict(w=None), dict(H=0), dict(dtype=5), dict(eps=-1.0),
                dict(d_r=ODD), dict(dx=ODD), dict(ws=ctypes.c_void_p(0x1010))):
        assert f(**bad) == INVALID, bad
    assert f(H=40000) == UNSUPPORTED
    assert f(ws=None) == CAPACITY and f(n=ctypes.c_size_t(255)) == CAPACITY


def test_dequantize_refusals(lib):
    f = lib.moe_fp8_dequantize
    assert f(FAKE, FAKE, -1, 4, 0, FAKE, None) == INVALID and f(FAKE, FAKE, 4, 0, 0, FAKE, None) == INVALID
    assert f(FAKE, FAKE, 4, 4, 3, FAKE, None) == INVALID and f(None, FAKE, 4, 4, 0, FAKE, None) == INVALID
    assert f(FAKE, FAKE, 4, 4, 0, ODD, None) == INVALID and f(FAKE, None, 4, 4, 0, FAKE, None) == INVALID
    assert f(FAKE, FAKE, 0, 4, 0, None, None) == 0


def route(lib, logits=FAKE, bias=None, mask=None, T=4, E=16, K=2, G=1, B=1, dtype=1, scoring=0, ids=FAKE, w=FAKE):
    return lib.moe_route(logits, bias, mask, T, E, K, G, B, dtype, scoring, 1, 1.0, ids, w, None, None)


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(E=4097), UNSUPPORTED), (dict(K=0), INVALID), (dict(E=64, K=33), UNSUPPORTED),
    (dict(K=17), INVALID), (dict(G=3), INVALID), (dict(G=0), INVALID), (dict(G=4, B=5), INVALID), (dict(G=4, B=0), INVALID),
    (dict(G=8, B=1, K=3), INVALID), (dict(dtype=2), INVALID), (dict(scoring=2), INVALID), (dict(bias=FAKE), INVALID),
    (dict(bias=ODD, scoring=1), INVALID), (dict(logits=None), INVALID), (dict(logits=ODD), INVALID), (dict(ids=None), INVALID),
    (dict(w=None), INVALID), (dict(E=1024, G=512, B=2), UNSUPPORTED), (dict(T=1 << 30, K=2), UNSUPPORTED), (dict(T=0), 0),
])
def test_route_refusals(lib, bad, code):
    assert route(lib, **bad) == code


def test_balance_and_gradient_refusals(lib):
    ws = lib.moe_balance_loss_workspace_bytes
    assert ws(0, 16) > 0 and ws(4, 16) > 0 and ws(-1, 16) == 0 and ws(4, 0) == 0 and ws(4, 4097) == 0

    def f(logits=FAKE, ids=FAKE, T=4, E=16, K=2, dtype=1, scoring=0, loss=FAKE, counts=FAKE, w=FAKE, n=BIG):
        return lib.moe_balance_loss(logits, ids, None, T, E, K, dtype, scoring, loss, counts, w, n, None, None)
    for bad in (dict(logits=None), dict(ids=None), dict(loss=None), dict(counts=None), dict(K=0), dict(w=ctypes.c_void_p(0x1010))):
        assert f(**bad) == INVALID, bad
    big = dict(T=4096, E=256)  # past the single launch, which takes no workspace
    assert ws(2048, 256) == 1 and ws(2049, 256) > 4 * 513 and ws(4, 257) >= 4 * 515
    assert f(w=None, **big) == CAPACITY and f(n=ctypes.c_size_t(16), **big) == CAPACITY and f(E=5000) == UNSUPPORTED

    def g(logits=FAKE, ids=FAKE, dw=FAKE, counts=FAKE, dl=FAKE, T=4, E=16, K=2, dtype=1, scoring=0, out=FAKE):
        return lib.moe_route_backward(logits, ids, dw, counts, dl, None, T, E, K, dtype, scoring, 1, 1.0, out, None, None)
    for bad in (dict(dw=None, counts=None, dl=None), dict(counts=None), dict(dl=None), dict(out=None), dict(out=ODD), dict(ids=None),
                dict(dtype=9)):
        assert g(**bad) == INVALID, bad
    assert g(K=40) == UNSUPPORTED and g(T=0) == 0


def test_binding_checks():
    """On host tensors, which every call refuses last."""
    x, w = torch.zeros(4, 64, dtype=BF), torch.zeros(64, dtype=BF)
    l, ids = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32)
    g, counts, one = torch.zeros(4, 2), torch.zeros(17, dtype=torch.int32), torch.zeros(1)
    for bad in (lambda: norm.rms_norm(x.double(), w), lambda: norm.rms_norm(x, w.half()), lambda: norm.rms_norm(x, w, 1e-6, x.float()),
                lambda: norm.rms_norm("x", w), lambda: norm.fp8_dequantize(x, x), lambda: norm.rms_norm_backward(x.float(), x, w),
                lambda: norm.fp8_dequantize(ids, ids, torch.half), lambda: router.moe_route(ids, 2), lambda: router.moe_route(l, 2, "sigmoid", l[0].double()),
                lambda: router.moe_route(l, 2, token_mask=ids[:, 0]), lambda: router.moe_balance_loss(l, ids.long()),
                lambda: router.moe_route_backward(l, ids, g.double())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: norm.rms_norm(x, w[:32]), lambda: norm.rms_norm(x[:, ::2], w[:32]), lambda: norm.rms_norm(x[0], w),
                lambda: norm.rms_norm(x, w, residual_out=x), lambda: norm.rms_norm(x, w, 1e-6, x[:2]), lambda: norm.rms_norm(x[:, :0], w[:0]),
                lambda: norm.rms_norm_fp8(x, w, y=x, with_y=False), lambda: norm.rms_norm_backward(x[:2], x, w),
                lambda: norm.fp8_dequantize(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)),
                lambda: router.moe_route(l, 0), lambda: router.moe_route(l, 2, "max"), lambda: router.moe_route(l, 2, "softmax", l[0]),
                lambda: router.moe_route(l, 2, "sigmoid", l[0, :8]), lambda: router.moe_route(l[:, :0], 2), lambda: router.moe_route(l.T, 2),
                lambda: router.moe_route(l, 2, token_mask=torch.ones(3, dtype=torch.bool)), lambda: router.moe_balance_loss(l, ids[:3]),
                lambda: router.moe_route_backward(l, ids), lambda: router.moe_route_backward(l, ids, g, counts),
                lambda: router.moe_route_backward(l, ids, g, d_loss=one), lambda: router.moe_route_backward(l, ids, g, counts[:16], one),
                lambda: router.moe_route_backward(l, ids, g[:3])):
        with pytest.raises(ValueError):
            bad()


def test_layer_in_8_bits_refusals(lib):
    """The W8A8 layer with x in 8 bits: both of codes and exponents, of x's shape."""
    T, K, E, H, I, L, R = 8, 2, 3, 128, 64, 2, 16
    f = lib.fused_moe_lora_forward_fp8_w8a8_xq
    big = ctypes.c_size_t(1 << 30)
    tail = [T, K, E, H, I, L, R, FAKE, FAKE, big, None, None]
    assert f(FAKE, None, FAKE, *[FAKE] * 13, *tail) == INVALID
    assert f(FAKE, FAKE, None, *[FAKE] * 13, *tail) == INVALID
    assert f(FAKE, ctypes.c_void_p(0x1008), FAKE, *[FAKE] * 13, *tail) == INVALID
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    x = torch.zeros(T, H, dtype=BF)
    args = (x, torch.zeros(T, K, dtype=torch.int32), torch.zeros(T, K), torch.zeros(T, dtype=torch.int32),
            torch.zeros(L, dtype=torch.int32), torch.zeros(L), u8(E, 2 * I, H), u8(E, 1, 1), u8(E, H, I), u8(E, 1, 1),
            torch.zeros(L, E, 2, R, H, dtype=BF), torch.zeros(L, E, 2, I, R, dtype=BF), torch.zeros(L, E, R, I, dtype=BF),
            torch.zeros(L, E, H, R, dtype=BF))
    for kw in (dict(x_codes=u8(T, H)), dict(x_exps=u8(T, 1)), dict(x_codes=u8(T, H - 1), x_exps=u8(T, 1)),
               dict(x_codes=u8(T, H), x_exps=u8(T, 2))):
        with pytest.raises(ValueError):
            mlr.fused_moe_lora_forward_fp8_w8a8(*args, **kw)
    with pytest.raises(TypeError):
        mlr.fused_moe_lora_forward_fp8_w8a8(*args, x_codes=x, x_exps=u8(T, 1))


def calls():
    x, w = torch.zeros(4, 64, dtype=BF), torch.zeros(64)
    l, ids, g = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    return {
        "rms_norm": lambda: norm.rms_norm(x, w), "rms_norm empty": lambda: norm.rms_norm(x[:0], w),
        "rms_norm_fp8": lambda: norm.rms_norm_fp8(x, w), "fp8_dequantize": lambda: norm.fp8_dequantize(u8(4, 64), u8(4, 1)),
        "rms_norm_backward": lambda: norm.rms_norm_backward(x, x, w), "RmsNorm": lambda: norm.RmsNorm.apply(x, w, 1e-6, x),
        "moe_route": lambda: router.moe_route(l, 2), "moe_route empty": lambda: router.moe_route(l[:0], 2),
        "moe_balance_loss": lambda: router.moe_balance_loss(l, ids), "moe_route_backward": lambda: router.moe_route_backward(l, ids, g),
        "MoeRoute": lambda: router.MoeRoute.apply(l, 2),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_host_tensors_are_refused(name):
    with pytest.raises(ValueError, match="must be on a CUDA device"):
        calls()[name]()
