"""Refusals of the epilogue GEMM (CPU): the binding checks every tensor before the library is called,
the C-ABI rejects what it can see before any device work."""
import pytest
import torch

import fine_grained_block_amd as fgb
from fine_grained_block_amd import _lib

FAKE = 0x10000
ERR = dict(OK=0, NULL=-1, SHAPE=-2, STRIDE=-3, ALIGN=-4, ENUM=-5, WORKSPACE=-6, DEVICE=-7)


def _abi(**kw):
    a = dict(a_q=FAKE, lda=1024, s_a=FAKE, ld_sa=512, w_q=FAKE, s_w=FAKE, fmt=0, bias=FAKE, bdt=0, act=4, res=FAKE,
             rdt=0, ldr=512, y=2 * FAKE, ydt=0, ldy=512, M=512, N=512, K=1024, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return _lib.lib().fgb_w8a8_block_gemm_epilogue(*a.values(), None)


def test_abi_refusals():
    assert _abi(act=5) == ERR["ENUM"] and _abi(act=-1) == ERR["ENUM"]
    assert _abi(bdt=2) == ERR["ENUM"] and _abi(rdt=-1) == ERR["ENUM"] and _abi(ydt=2) == ERR["ENUM"]
    assert _abi(bias=FAKE + 8) == ERR["ALIGN"] and _abi(res=FAKE + 4) == ERR["ALIGN"]
    assert _abi(ldr=516) == ERR["ALIGN"]             # bf16 rows of 1032 bytes
    assert _abi(ldr=256) == ERR["STRIDE"]
    assert _abi(y=FAKE, ldr=520) == ERR["STRIDE"]    # in place with another pitch
    assert _abi(y=FAKE, rdt=1) == ERR["STRIDE"]      # in place with another type
    assert _abi(w_q=None) == ERR["NULL"] and _abi(K=1000) == ERR["SHAPE"]
    # the unused dtypes are ignored; M == 0 is a no-op before any pointer or device check
    assert _abi(bias=None, bdt=9, res=None, rdt=9, ldr=0, M=0) == ERR["OK"]
    need = fgb.gemm_workspace_bytes(40, 6144, 4096)
    big = dict(M=40, N=6144, K=4096, lda=4096, ldy=6144, ldr=6144)
    assert need > 0 and _abi(**big, ws=None, wsb=0) == ERR["WORKSPACE"]
    assert _abi(**big, wsb=need - 1) == ERR["WORKSPACE"] and _abi(**big, ws=FAKE + 8) == ERR["ALIGN"]


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="fake pointers must not reach a real device")
def test_abi_valid_arguments_stop_at_the_device():
    assert _abi() == ERR["DEVICE"]
    assert _abi(bias=None, bdt=9, res=None, rdt=9, ldr=0, act=0) == ERR["DEVICE"]
    assert _abi(res=2 * FAKE) == ERR["DEVICE"]  # y itself


@pytest.fixture
def no_library(monkeypatch):
    def boom():
        raise AssertionError("the library was called")
    monkeypatch.setattr(fgb.ops, "lib", boom)


def _ops(M=20, N=256, K=512):
    return (torch.zeros((M, K), dtype=torch.uint8), torch.zeros((K // 128, (M + 3) // 4 * 4)),
            torch.zeros((N, K), dtype=torch.uint8), torch.zeros((N // 128, K // 128)))


@pytest.mark.parametrize("kw,match", [
    (dict(activation="tanh"), "activation"), (dict(activation=None), "activation"),
    (dict(bias=torch.zeros(255)), "bias"), (dict(bias=torch.zeros(256, dtype=torch.float16)), "bias"),
    (dict(bias=torch.zeros((1, 256))), "bias"), (dict(bias=torch.zeros(512)[::2]), "bias"),
    (dict(residual=torch.zeros((19, 256))), "residual"), (dict(residual=torch.zeros((20, 128))), "residual"),
    (dict(residual=torch.zeros((20, 256), dtype=torch.float64)), "residual"),
    (dict(residual=torch.zeros((256, 20)).t()), "residual"), (dict(residual=3.0), "residual"),
    (dict(out=torch.zeros((20, 256), dtype=torch.float16)), "out"), (dict(out=torch.zeros((21, 256))), "out"),
    (dict(), "on the GPU"),
])
def test_binding_refusals(no_library, kw, match):
    with pytest.raises(ValueError, match=match):
        fgb.gemm_epilogue(*_ops(), **kw)
