"""Refusals of the router and of the mixture-of-experts layer (CPU): the C-ABI rejects what it can see
before any device work, the binding checks every tensor before the library is called."""
import pytest
import torch

import fine_grained_block_amd as fgb
from fine_grained_block_amd import _lib

FAKE = 0x10000
ERR = dict(OK=0, NULL=-1, SHAPE=-2, STRIDE=-3, ALIGN=-4, ENUM=-5, WORKSPACE=-6, DEVICE=-7)


def _route(**kw):
    a = dict(logits=FAKE, dt=1, ld=64, T=10, E=64, k=8, scoring=0, bias=None, renorm=1, scale=1.0, ids=FAKE, w=FAKE)
    a.update(kw)
    return _lib.lib().fgb_moe_route(*a.values(), None)


def _moe(**kw):
    a = dict(x=FAKE, ldx=256, ids=FAKE, w=FAKE, k=2, w13=FAKE, s13=FAKE, w2=FAKE, s2=FAKE, fmt=0, E=8, act=4, res=FAKE,
             rdt=0, ldr=256, y=2 * FAKE, ydt=0, ldy=256, T=5, H=256, I=384, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return _lib.lib().fgb_moe_ffn(*a.values(), None)


def test_route_abi_refusals():
    assert _route(E=0, k=0) == ERR["SHAPE"] and _route(E=1025, ld=1025) == ERR["SHAPE"]
    assert _route(k=0) == ERR["SHAPE"] and _route(k=33) == ERR["SHAPE"] and _route(E=4, k=5) == ERR["SHAPE"]
    assert _route(T=-1) == ERR["SHAPE"] and _route(T=0, logits=None) == ERR["OK"]
    assert _route(dt=2) == ERR["ENUM"] and _route(scoring=2) == ERR["ENUM"]
    assert _route(logits=None) == ERR["NULL"] and _route(ids=None) == ERR["NULL"] and _route(w=None) == ERR["NULL"]
    assert _route(ld=63) == ERR["STRIDE"]
    assert _route(logits=FAKE + 2) == ERR["ALIGN"] and _route(dt=0, logits=FAKE + 1) == ERR["ALIGN"]
    assert _route(bias=FAKE + 2) == ERR["ALIGN"] and _route(ids=FAKE + 1) == ERR["ALIGN"]


def test_moe_abi_refusals():
    for bad in (dict(T=65), dict(T=-1), dict(k=0), dict(T=64, k=17), dict(E=0), dict(E=1025), dict(H=200, ldx=256),
                dict(I=100), dict(H=0), dict(I=0), dict(H=32896, ldx=32896, ldy=32896, ldr=32896), dict(I=32896)):
        assert _moe(**bad) == ERR["SHAPE"], bad
    assert _moe(T=0, x=None, ws=None) == ERR["OK"]
    for bad in (dict(fmt=2), dict(act=0), dict(act=1), dict(act=5), dict(rdt=3), dict(ydt=2)):
        assert _moe(**bad) == ERR["ENUM"], bad
    for name in ("x", "ids", "w", "w13", "s13", "w2", "s2", "y"):
        assert _moe(**{name: None}) == ERR["NULL"], name
    for name in ("ldx", "ldy", "ldr"):
        assert _moe(**{name: 128}) == ERR["STRIDE"], name
        assert _moe(**{name: 260}) == ERR["ALIGN"], name
    for name in ("x", "w13", "w2", "res", "y", "ws"):
        assert _moe(**{name: FAKE + 8}) == ERR["ALIGN"], name
    assert _moe(ids=FAKE + 2) == ERR["ALIGN"] and _moe(s2=FAKE + 2) == ERR["ALIGN"]
    assert _moe(y=FAKE, rdt=1) == ERR["STRIDE"] and _moe(y=FAKE, ldy=264) == ERR["STRIDE"]
    need = fgb.moe_ffn_workspace_bytes(5, 2, 8, 256, 384)
    assert need > 0 and _moe(wsb=need - 1) == ERR["WORKSPACE"] and _moe(ws=None) == ERR["WORKSPACE"]


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="fake pointers must not reach a real device")
def test_valid_arguments_stop_at_the_device():
    assert _route() == ERR["DEVICE"] and _route(dt=0, logits=FAKE + 2, ld=65) == ERR["DEVICE"]
    assert _moe() == ERR["DEVICE"] and _moe(res=None, rdt=9, ldr=0) == ERR["DEVICE"]
    assert _moe(fmt=1, s13=FAKE + 1, s2=FAKE + 3) == ERR["DEVICE"]
    assert _moe(H=32768, I=32768, ldx=32768, ldy=32768, ldr=32768, E=1, k=1) == ERR["DEVICE"] and _moe(y=FAKE) == ERR["DEVICE"]


def test_workspace_query():
    """Room for every pair's row of the gated product at least; 0 for shapes that are refused."""
    for T, k, E, H, I in [(1, 1, 1, 128, 128), (64, 16, 1024, 256, 128), (64, 8, 32, 7168, 2048), (17, 3, 5, 512, 640)]:
        assert fgb.moe_ffn_workspace_bytes(T, k, E, H, I) >= T * k * I
    assert fgb.moe_ffn_workspace_bytes(0, 2, 8, 256, 256) == 0 and fgb.moe_ffn_workspace_bytes(65, 2, 8, 256, 256) == 0
    assert fgb.moe_ffn_workspace_bytes(4, 2, 8, 200, 256) == 0


@pytest.fixture
def no_library(monkeypatch):
    def boom():
        raise AssertionError("the library was called")
    monkeypatch.setattr(fgb.ops, "lib", boom)


@pytest.mark.parametrize("kw,match", [
    (dict(logits=torch.zeros((4, 8), dtype=torch.float16)), "logits"), (dict(logits=torch.zeros(8)), "logits"),
    (dict(logits=torch.zeros((8, 4)).t()), "logits"), (dict(top_k=0), "top_k"), (dict(top_k=9), "top_k"),
    (dict(scoring="relu"), "scoring"), (dict(select_bias=torch.zeros(7)), "select_bias"),
    (dict(select_bias=torch.zeros(8, dtype=torch.bfloat16)), "select_bias"),
    (dict(out=(torch.zeros((4, 2), dtype=torch.int64), torch.zeros((4, 2)))), "ids"),
    (dict(out=(torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 3)))), "weights"), (dict(), "on the GPU"),
])
def test_route_binding_refusals(no_library, kw, match):
    args = dict(logits=torch.zeros((4, 8)), top_k=2)
    args.update(kw)
    with pytest.raises(ValueError, match=match):
        fgb.moe_route(**args)


def _args(T=3, E=4, k=2, H=256, I=128):
    return dict(x=torch.zeros((T, H), dtype=torch.bfloat16), ids=torch.zeros((T, k), dtype=torch.int32),
                weights=torch.zeros((T, k)), w13_q=torch.zeros((E, 2 * I, H), dtype=torch.uint8),
                s_w13=torch.zeros((E, 2 * I // 128, H // 128)), w2_q=torch.zeros((E, H, I), dtype=torch.uint8),
                s_w2=torch.zeros((E, H // 128, I // 128)))


@pytest.mark.parametrize("kw,match", [
    (dict(x=torch.zeros((3, 256))), "x must be"), (dict(x=torch.zeros((65, 256), dtype=torch.bfloat16)), "T <= 64"),
    (dict(ids=torch.zeros((3, 2), dtype=torch.int64)), "ids"), (dict(ids=torch.zeros((2, 2), dtype=torch.int32)), "ids"),
    (dict(ids=torch.zeros(6, dtype=torch.int32)), "ids"), (dict(weights=torch.zeros((3, 1))), "weights"),
    (dict(weights=torch.zeros((3, 2), dtype=torch.bfloat16)), "weights"),
    (dict(w13_q=torch.zeros((4, 128, 256), dtype=torch.uint8)), "w13_q"),
    (dict(w2_q=torch.zeros((4, 128, 256), dtype=torch.uint8)), "w13_q|w2_q"),
    (dict(w2_q=torch.zeros((256, 128), dtype=torch.uint8)), "w2_q"), (dict(s_w13=torch.zeros((4, 1, 2))), "s_w13"),
    (dict(s_w2=torch.zeros((4, 2, 1), dtype=torch.uint8)), "s_w2"), (dict(activation="none"), "activation"),
    (dict(activation="relu"), "activation"), (dict(residual=torch.zeros((3, 128))), "residual"),
    (dict(out=torch.zeros((3, 256), dtype=torch.float16)), "out"), (dict(), "on the GPU"),
])
def test_moe_binding_refusals(no_library, kw, match):
    args = _args()
    args.update(kw)
    with pytest.raises(ValueError, match=match):
        fgb.moe_ffn(**args)
