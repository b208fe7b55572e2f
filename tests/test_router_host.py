"""CPU checks of the router's C ABI (include/moe_gate.h): sizes, options and
pointers that are refused before anything touches a device, and the binding's
own tensor checks."""
import ctypes
import math
import os

import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    import combine_dispatch_amd as m
    if not os.path.exists(m.LIB_PATH):
        from combine_dispatch_amd import build
        build.build()
    m.lib()
    return m


NULL = ctypes.c_void_p(0)
FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 1)


def gate(moe, shape, opts=None, logits=FAKE, bias=NULL, idx=FAKE, w=FAKE):
    return moe.lib().moe_gate(moe.MoeGateShape(*shape), opts, logits, bias, NULL, idx, w, NULL)


def test_defaults(moe):
    o = moe.moe_default_gate_options()
    assert (o.dtype, o.score, o.renormalise, o.scale) == (moe.MOE_DTYPE_F32, moe.MOE_SCORE_SOFTMAX, 1, 1.0)


@pytest.mark.parametrize("shape,want", [((-1, 8, 2), "INVALID_ARG"), ((1, 0, 1), "UNSUPPORTED"),
                                        ((1, 1025, 1), "UNSUPPORTED"), ((1, 8, 0), "UNSUPPORTED"),
                                        ((1, 8, 9), "UNSUPPORTED"), ((1, 1024, 65), "UNSUPPORTED"),
                                        ((1 << 28, 8, 2), "UNSUPPORTED"),
                                        ((1 << 27, 64, 16), "UNSUPPORTED"), ((0, 8, 2), "OK")])
def test_gate_shapes(moe, shape, want):
    st = moe.MOE_OK if want == "OK" else getattr(moe, "MOE_ERR_" + want)
    assert gate(moe, shape) == st
    assert moe.lib().moe_gate_backward(moe.MoeGateShape(*shape), None, FAKE, NULL, FAKE, FAKE, None, FAKE, NULL) == st
    if want != "OK":
        assert moe.moe_balance_workspace_bytes(*shape) == 0


@pytest.mark.parametrize("opts", [(2, 0, 1, 1.0), (0, 2, 1, 1.0), (0, 0, 2, 1.0), (0, 0, 1, math.inf), (0, 0, 1, math.nan)])
def test_gate_options_refused(moe, opts):
    o = moe.MoeGateOptions(*opts)
    assert gate(moe, (4, 8, 2), o) == moe.MOE_ERR_INVALID_ARG
    assert moe.lib().moe_gate_backward(moe.MoeGateShape(4, 8, 2), o, FAKE, NULL, FAKE, FAKE, None, FAKE,
                                       NULL) == moe.MOE_ERR_INVALID_ARG
    assert moe.lib().moe_balance_loss(moe.MoeGateShape(4, 8, 2), o, FAKE, NULL, FAKE, NULL, 1, 0.1, FAKE, FAKE, FAKE,
                                      FAKE, 1 << 30, NULL) == moe.MOE_ERR_INVALID_ARG


def test_gate_pointers(moe):
    s = (4, 8, 2)
    assert gate(moe, s, logits=NULL) == moe.MOE_ERR_INVALID_ARG
    assert gate(moe, s, idx=NULL) == moe.MOE_ERR_INVALID_ARG
    assert gate(moe, s, w=NULL) == moe.MOE_ERR_INVALID_ARG
    assert gate(moe, s, logits=ODD) == moe.MOE_ERR_INVALID_ARG
    assert gate(moe, s, idx=ctypes.c_void_p((1 << 20) + 4)) == moe.MOE_ERR_INVALID_ARG
    # a selection bias goes with sigmoid scores
    assert gate(moe, s, bias=FAKE) == moe.MOE_ERR_UNSUPPORTED


def test_backward_parts(moe):
    s, L = moe.MoeGateShape(4, 8, 2), moe.lib()
    bad = moe.MOE_ERR_INVALID_ARG
    assert L.moe_gate_backward(s, None, FAKE, NULL, NULL, FAKE, None, FAKE, NULL) == bad  # half a gate part
    assert L.moe_gate_backward(s, None, FAKE, NULL, NULL, NULL, None, FAKE, NULL) == bad  # no part at all
    assert L.moe_gate_backward(s, None, FAKE, NULL, FAKE, FAKE, None, NULL, NULL) == bad
    for b in (moe.MoeBalanceGrad(None, 4096, None, 1), moe.MoeBalanceGrad(4096, None, None, 1),
              moe.MoeBalanceGrad(4096, 4096, None, 2), moe.MoeBalanceGrad(4096, 4096, 4096, 0)):
        assert L.moe_gate_backward(s, None, FAKE, NULL, NULL, NULL, ctypes.byref(b), FAKE, NULL) == bad
    big = moe.MoeBalanceGrad(4096, 4096, 4096, 1 << 17)
    assert L.moe_gate_backward(s, None, FAKE, NULL, NULL, NULL, ctypes.byref(big), FAKE,
                               NULL) == moe.MOE_ERR_UNSUPPORTED


def test_balance_arguments(moe):
    s, L = moe.MoeGateShape(100, 8, 2), moe.lib()
    need = moe.moe_balance_workspace_bytes(100, 8, 2, 5)
    assert 0 < need < 1 << 16
    assert moe.moe_balance_workspace_bytes(100, 8, 2, 0) == 0
    assert moe.moe_balance_workspace_bytes(100, 8, 2, 65537) == 0

    def call(seq=FAKE, S=5, loss=FAKE, ws=FAKE, n=need, logits=FAKE):
        return L.moe_balance_loss(s, None, logits, NULL, FAKE, seq, S, 0.1, loss, FAKE, FAKE, ws, n, NULL)

    assert call(n=need - 1) == moe.MOE_ERR_WORKSPACE
    assert call(ws=NULL) == moe.MOE_ERR_WORKSPACE
    assert call(ws=ctypes.c_void_p((1 << 20) + 8)) == moe.MOE_ERR_WORKSPACE
    assert call(seq=NULL) == moe.MOE_ERR_INVALID_ARG  # several sequences need their offsets
    assert call(S=0) == moe.MOE_ERR_INVALID_ARG
    assert call(loss=NULL) == moe.MOE_ERR_INVALID_ARG
    assert call(logits=NULL) == moe.MOE_ERR_INVALID_ARG
    assert call(S=65537, n=1 << 40) == moe.MOE_ERR_UNSUPPORTED


def test_binding_refuses_host_tensors_and_bad_options(moe):
    l = torch.zeros(4, 8)
    with pytest.raises(moe.MoeError, match="GPU"):
        moe.moe_gate(l, torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2))
    with pytest.raises(moe.MoeError, match="GPU"):
        moe.moe_gate_backward(l, l, topk_idx=torch.zeros(4, 2, dtype=torch.int64), d_topk_w=torch.zeros(4, 2))
    with pytest.raises(moe.MoeError, match="together"):
        moe.moe_gate_backward(l, l, topk_idx=torch.zeros(4, 2, dtype=torch.int64))
    with pytest.raises(moe.MoeError, match="together"):
        moe.moe_gate_backward(l, l, slope=torch.zeros(1, 8))
    with pytest.raises(moe.MoeError, match="score"):
        moe.gate_options(score="relu")
