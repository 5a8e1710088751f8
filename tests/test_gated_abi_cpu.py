"""Gated attention and the query/key norm with rotation without a GPU: every
refusal (before any HIP call), workspace arithmetic and the binding's checks."""
import ctypes
import math

import pytest
import torch

import token_level_head_block_amd as mh

BASE = 1 << 36          # fake, aligned, never dereferenced
INV, UNS, MIS = mh.MHLA_ERR_INVALID_ARG, mh.MHLA_ERR_UNSUPPORTED, mh.MHLA_ERR_MISALIGNED


def P(i, off=0):
    return BASE * i + off


def seq(**kw):
    s = mh.make_seq(2, 100, 4, 2, 64, mh.MHLA_BF16, 0.125)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


@pytest.mark.parametrize("kw,code", [
    ({}, mh.MHLA_OK), ({"batch": 0}, mh.MHLA_OK), ({"tokens": 0}, mh.MHLA_OK), ({"heads": 0, "kv_heads": 0}, mh.MHLA_OK),
    ({"batch": -1}, INV), ({"tokens": -1}, INV), ({"heads": -2}, INV), ({"kv_heads": -1}, INV), ({"kv_heads": 0}, INV),
    ({"kv_heads": 3}, INV), ({"heads": 2, "kv_heads": 4}, INV), ({"scale": math.nan}, INV), ({"scale": math.inf}, INV),
    ({"head_dim": 48}, UNS), ({"head_dim": 256}, UNS), ({"dtype": 2}, UNS), ({"tokens": (1 << 30) + 1}, UNS),
    ({"heads": 65538}, UNS), ({"q_stride": 255}, INV), ({"q_stride": 257}, MIS), ({"q_stride": 256}, mh.MHLA_OK),
    ({"k_stride": 120}, INV), ({"v_stride": 132}, MIS), ({"v_stride": (1 << 23) + 8}, UNS), ({"k_stride": -128}, INV),
    ({"batch": 1 << 30, "heads": 2, "kv_heads": 2, "tokens": 1}, UNS),
    ({"batch": 4, "tokens": 1 << 30, "heads": 64, "kv_heads": 64}, UNS), ({"heads": 0}, INV),
    ({"batch": 1398101, "heads": 2, "kv_heads": 2, "tokens": 1}, mh.MHLA_OK),
    ({"batch": 1398102, "heads": 2, "kv_heads": 2, "tokens": 1}, UNS),
    ({"batch": 1398101, "heads": 1, "kv_heads": 1, "tokens": 2048}, mh.MHLA_OK),
    ({"batch": 1398102, "heads": 1, "kv_heads": 1, "tokens": 2048}, UNS),
    ({"batch": 1, "tokens": 1 << 30, "heads": 2, "kv_heads": 2}, mh.MHLA_OK),
    ({"batch": (1 << 31) - 1, "tokens": 1 << 30, "heads": 65536, "kv_heads": 65536, "head_dim": 128}, UNS),
])
def test_check_seq(kw, code):
    s = seq(**kw)
    assert mh.mhla_check_seq(s) == code
    if code != mh.MHLA_OK:
        assert mh.mhla_gated_workspace_bytes(s) == 0 and mh.mhla_gated_backward_workspace_bytes(s) == 0
        assert fwd(s=s) == code and bwd(s=s) == code


def test_null_seq():
    L = mh.lib()
    assert L.mhla_check_seq(None) == INV
    assert L.mhla_gated_workspace_bytes(None) == 0
    assert L.mhla_gated_forward(P(1), P(2), P(3), P(4), None, None, None, P(5), None, None, 0, None) == INV


def fwd(q=P(1), k=P(2), v=P(3), g=P(4), lens=P(5), state=P(6), s=None, out=P(7), so=P(8), ws=P(9), n=1 << 40):
    return mh.lib().mhla_gated_forward(q, k, v, g, lens, state, ctypes.byref(s if s is not None else seq()), out, so,
                                       ws, n, None)


def bwd(q=P(1), k=P(2), v=P(3), g=P(4), lens=P(5), state=P(6), do=P(7), ds1=P(8), s=None, dq=P(9), dk=P(10),
        dv=P(11), dg=P(12), ds0=P(13), ws=P(14), n=1 << 40):
    return mh.lib().mhla_gated_backward(q, k, v, g, lens, state, do, ds1, ctypes.byref(s if s is not None else seq()),
                                        dq, dk, dv, dg, ds0, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    ({"q": None}, INV), ({"k": None}, INV), ({"v": None}, INV), ({"g": None}, INV), ({"out": None}, INV),
    ({"q": P(1, 8)}, MIS), ({"state": P(6, 4)}, MIS), ({"so": P(8, 4)}, MIS), ({"g": P(4, 2)}, MIS),
    ({"lens": P(5, 1)}, MIS), ({"ws": P(9, 8)}, MIS), ({"n": 100}, INV), ({"ws": None, "n": 16}, INV),
    ({"out": P(1)}, INV), ({"out": P(2, 64)}, INV), ({"out": P(4)}, INV), ({"out": P(5)}, INV), ({"out": P(6)}, INV),
    ({"so": P(7)}, INV), ({"so": P(6, 16)}, INV), ({"ws": P(1)}, INV), ({"ws": P(8)}, INV), ({"ws": P(6)}, INV),
])
def test_forward_refusals(kw, code):
    assert fwd(**{"s": seq(tokens=4000), **kw}) == code


@pytest.mark.parametrize("kw,code", [
    ({"do": None}, INV), ({"dq": None}, INV), ({"dk": None}, INV), ({"dv": None}, INV), ({"dg": None}, INV),
    ({"do": P(7, 8)}, MIS), ({"ds1": P(8, 4)}, MIS), ({"ds0": P(13, 8)}, MIS), ({"dg": P(12, 2)}, MIS),
    ({"dq": P(7)}, INV), ({"dk": P(2)}, INV), ({"dv": P(10)}, INV), ({"dg": P(4)}, INV), ({"ds0": P(6)}, INV),
    ({"ds0": P(8, 16)}, INV), ({"ds0": P(8)}, INV), ({"ws": P(9)}, INV), ({"ws": P(7)}, INV), ({"n": 1000}, INV), ({"ws": P(14, 4)}, MIS),
])
def test_backward_refusals(kw, code):
    assert bwd(**kw) == code


def test_injected_allocation_failure(monkeypatch):
    monkeypatch.setenv("MHLA_FAIL_ALLOC", "1")
    assert fwd(s=seq(tokens=4000), ws=None, n=0) == mh.MHLA_ERR_ALLOC
    assert bwd(ws=None, n=0) == mh.MHLA_ERR_ALLOC
    assert rope_b(ws=None, n=0) == mh.MHLA_ERR_ALLOC


def test_empty_problems_need_nothing():
    for kw in ({"batch": 0}, {"heads": 0, "kv_heads": 0}):
        s = seq(**kw)
        assert mh.mhla_gated_workspace_bytes(s) == 0 and mh.mhla_gated_backward_workspace_bytes(s) == 0
        n = (None,) * 6
        assert mh.lib().mhla_gated_forward(*n, ctypes.byref(s), None, None, None, 0, None) == mh.MHLA_OK
        assert mh.lib().mhla_gated_backward(*n, None, None, ctypes.byref(s), *(None,) * 6, 0, None) == mh.MHLA_OK


def test_workspace_holds_segment_states():
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    many = mh.make_seq(64, 4096, 16, 16, 64, mh.MHLA_BF16)
    assert mh.mhla_gated_workspace_bytes(many) == 0              # enough heads: a sequence is one segment
    short = mh.make_seq(1, 256, 1, 1, 64, mh.MHLA_BF16)          # few chunks: one segment as well
    assert mh.mhla_gated_workspace_bytes(short) == 0
    assert mh.mhla_gated_backward_workspace_bytes(short) == up(64 * 64 * 4) + 2 * up(256 * 4)
    few = mh.make_seq(1, 64 * 9, 1, 1, 64, mh.MHLA_BF16)         # a segment a chunk
    assert mh.mhla_gated_workspace_bytes(few) == up(9 * 64 * 64 * 4) + up(9 * 4)
    n = up(10 * 64 * 64 * 4) + up(9 * 4) + up(9 * 64 * 64 * 4) + 2 * up(576 * 4)
    assert mh.mhla_gated_backward_workspace_bytes(few) == n


def step(q=P(1), k=P(2), v=P(3), g=P(4), slots=P(5), s=None, state=P(6), n=10, out=P(7)):
    return mh.lib().mhla_gated_step(q, k, v, g, slots, ctypes.byref(s if s is not None else seq(tokens=1)), state, n,
                                    out, None)


@pytest.mark.parametrize("kw,code", [
    ({"s": seq()}, INV), ({"n": -1}, INV), ({"slots": None, "n": 1}, INV), ({"q": None}, INV), ({"k": None}, INV),
    ({"v": None}, INV), ({"g": None}, INV), ({"state": None}, INV), ({"out": None}, INV), ({"state": P(6, 8)}, MIS),
    ({"out": P(7, 2)}, MIS), ({"g": P(4, 2)}, MIS), ({"slots": P(5, 2)}, MIS), ({"out": P(6)}, INV),
    ({"out": P(1)}, INV), ({"state": P(2)}, INV), ({"state": P(5)}, INV), ({"s": seq(tokens=1, batch=0)}, mh.MHLA_OK),
])
def test_step_refusals(kw, code):
    assert step(**kw) == code


def rope(q=P(1), k=P(2), wq=P(3), wk=P(4), pos=P(5), freq=P(6), r=None, s=None, qo=P(7), ko=P(8)):
    return mh.lib().mhla_qk_norm_rope(q, k, wq, wk, pos, freq, ctypes.byref(r if r is not None else mh.make_rope((32,))),
                                      ctypes.byref(s if s is not None else seq()), qo, ko, None)


def rope_b(q=P(1), k=P(2), wq=P(3), wk=P(4), pos=P(5), freq=P(6), dqo=P(7), dko=P(8), dq=P(9), dk=P(10), dwq=P(11),
           dwk=P(12), ws=P(13), n=1 << 30):
    return mh.lib().mhla_qk_norm_rope_backward(q, k, wq, wk, pos, freq, ctypes.byref(mh.make_rope((32,))), dqo, dko,
                                               ctypes.byref(seq()), dq, dk, dwq, dwk, ws, n, None)


def bad_rope(**kw):
    r = mh.make_rope((16, 16))
    for k, v in kw.items():
        setattr(r, k, v)
    return r


@pytest.mark.parametrize("kw,code", [
    ({"r": bad_rope(style=2)}, INV), ({"r": bad_rope(axes=0)}, INV), ({"r": bad_rope(axes=4)}, INV),
    ({"r": bad_rope(axes=1)}, INV), ({"r": bad_rope(eps=0.0)}, INV), ({"r": bad_rope(eps=math.nan)}, INV),
    ({"r": mh.make_rope((20, 16))}, INV), ({"r": mh.make_rope((5,))}, INV), ({"r": mh.make_rope((0,))}, INV),
    ({"r": mh.make_rope((-8, 16))}, INV), ({"r": mh.make_rope((40,))}, INV), ({"q": None}, INV), ({"k": None}, INV),
    ({"pos": None}, INV), ({"freq": None}, INV), ({"qo": None}, INV), ({"ko": None}, INV), ({"q": P(1, 8)}, MIS),
    ({"wq": P(3, 4)}, MIS), ({"pos": P(5, 2)}, MIS), ({"freq": P(6, 1)}, MIS), ({"qo": P(1, 16)}, INV),
    ({"qo": P(2)}, INV), ({"ko": P(7)}, INV), ({"qo": P(3)}, INV), ({"ko": P(5)}, INV),
    ({"s": seq(q_stride=512), "qo": P(1)}, INV), ({"s": seq(kv_heads=3), "q": None}, INV),
    ({"s": seq(batch=0)}, mh.MHLA_OK), ({"s": seq(tokens=0)}, mh.MHLA_OK),
])
def test_rope_refusals(kw, code):
    assert rope(**kw) == code


@pytest.mark.parametrize("kw,code", [
    ({"dqo": None}, INV), ({"dko": None}, INV), ({"dq": None}, INV), ({"dq": P(1)}, INV), ({"dk": P(7)}, INV),
    ({"dq": P(7, 64)}, INV), ({"dwq": P(11, 8)}, MIS), ({"dwq": P(3)}, INV), ({"dwk": P(11)}, INV), ({"n": 64}, INV),
    ({"ws": P(7)}, INV), ({"ws": P(13, 4)}, MIS), ({"ws": None, "n": 4}, INV),
])
def test_rope_backward_refusals(kw, code):
    assert rope_b(**kw) == code


def test_rope_workspace_bytes():
    assert mh.mhla_qk_norm_rope_backward_workspace_bytes(seq()) == 200 * 2 * 64 * 4
    assert mh.mhla_qk_norm_rope_backward_workspace_bytes(seq(tokens=100000)) == 1024 * 2 * 64 * 4
    assert mh.mhla_qk_norm_rope_backward_workspace_bytes(seq(batch=0)) == 0
    assert mh.mhla_qk_norm_rope_backward_workspace_bytes(seq(kv_heads=3)) > 0


# ---------------------------------------------------------------- the binding

def test_binding_refuses_wrong_tensors():
    q, k = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16)
    g = torch.zeros(1, 4, 1)
    with pytest.raises(ValueError, match="GPU"):
        mh.gated_forward(q, k, k, g)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        mh.gated_forward(q.half(), k.half(), k.half(), g)
    with pytest.raises(ValueError, match="v must be"):
        mh.gated_forward(q, k, k.float(), g)
    with pytest.raises(ValueError, match="v must be"):
        mh.gated_forward(q, k, k[:, :2], g)
    with pytest.raises(ValueError, match="evenly spaced"):
        mh.gated_forward(q.transpose(1, 2).contiguous().transpose(1, 2), k, k, g)
    with pytest.raises(ValueError, match="batch, tokens"):
        mh.gated_forward(q[0], k[0], k[0], g)


@pytest.mark.parametrize("shape,sub,step", [
    ((2, 5, 4, 32), (2, 3), 4 * 32), ((1, 5, 4, 32), (2, 3), 4 * 32), ((3, 1, 4, 32), (0, 2), 4 * 32),
])
def test_strides_of_slices(shape, sub, step):
    t = torch.zeros(shape)
    part = t[:, :, sub[0]:sub[1]]
    h = sub[1] - sub[0]
    assert mh._stride_of("t", part, (shape[0], shape[1], h, shape[3]), t.dtype, t.device) == step
    with pytest.raises(ValueError):                      # tokens of the batch's items not evenly spaced
        mh._stride_of("t", torch.zeros(2, 7, 2, 32)[:, :5], (2, 5, 2, 32), t.dtype, t.device)
    with pytest.raises(ValueError):                      # heads apart
        mh._stride_of("t", torch.zeros(2, 5, 4, 32)[:, :, ::2], (2, 5, 2, 32), t.dtype, t.device)
    with pytest.raises(ValueError):                      # every token the same one
        mh._stride_of("t", torch.zeros(1, 1, 2, 32).expand(1, 5, 2, 32), (1, 5, 2, 32), t.dtype, t.device)
