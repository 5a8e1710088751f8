"""Query/key norm with rotation (mhla_qk_norm_rope, _backward) against the
float64 oracle on the same inputs, and the layer's chain of it with gated
attention.

Tolerances, elementwise.  A rotated value is a sum of two products of values
that are off by at most 8 2^-24 of their size (square sum of d terms, whose
relative error halves under the root, root, two products, sine and cosine to
2 units) plus the angle's rounding, 2^-25 turns of 2 pi: 32 2^-24 of the pair's
length in all, and d 2^-24 / 2 from the mean.  Gradients take a second sum of d
terms and a cancelling difference: (64 + 2 d) 2^-24 of the summed magnitudes.
The final rounding is at most eps / 2 of the value.
"""
import numpy as np
import pytest
import torch

import token_level_head_block_amd as mh
from oracle import gated as og

from gpu_util import say
from test_gpu_gated import dev, host

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
REL = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def make(seed, dt, B, T, H, Hk, d, sections, far=0):
    r = np.random.default_rng(seed)
    rnd = lambda s: host(torch.from_numpy(r.normal(size=s).astype(np.float32)).to(dt))  # noqa: E731
    f32 = lambda x: x.astype(np.float32).astype(np.float64)  # noqa: E731
    axes, P = len(sections), sum(sections)
    pos = r.integers(-40, 400, size=(B, T, axes)) + far
    freq = f32(np.concatenate([1e4 ** (-np.arange(n) / max(n, 1)) for n in sections]))
    assert freq.size == P
    return {"q": rnd((B, T, H, d)), "k": rnd((B, T, Hk, d)), "dq": rnd((B, T, H, d)), "dk": rnd((B, T, Hk, d)),
            "wq": f32(1 + 0.2 * r.normal(size=d)), "wk": f32(1 + 0.2 * r.normal(size=d)), "pos": pos, "freq": freq}


def within(name, got, ref, tol):
    got = host(got)
    assert got.shape == ref.shape
    over = float(np.max(np.abs(got - ref) / (tol + 1e-30)))
    say(f"    {name}: error at most {over:.3f} of its tolerance")
    assert np.isfinite(got).all() and over <= 1.0, name


CASES = [
    # B, T, H, Hk, d, sections, interleaved, dtype, far
    (1, 1, 1, 1, 32, (8,), False, BF, 0), (2, 3, 2, 1, 32, (16,), True, F32, 0),
    (1, 9, 6, 6, 64, (16, 16), False, BF, 0), (2, 5, 3, 2, 64, (11, 11, 10), True, BF, 0),
    (1, 17, 4, 1, 128, (64,), False, F32, 1 << 20), (1, 4, 5, 5, 128, (22, 21, 21), False, BF, 0),
    (1, 6, 2, 7, 64, (24,), False, F32, 0), (3, 2, 33, 3, 128, (8,), True, BF, (1 << 31) - 500),
    (1, 5, 1, 1, 64, (32,), False, F32, -(1 << 31) + 50), (2, 1500, 2, 1, 32, (0, 16), False, BF, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}+{c[3]}x{c[4]}-{c[5]}-{c[6]}-{str(c[7])[6:]}")
@pytest.mark.parametrize("weights", [True, False], ids=["w", "ones"])
def test_forward_and_backward(case, weights):
    B, T, H, Hk, d, sections, inter, dt, far = case
    eps = 1e-5
    x = make(H + T, dt, B, T, H, Hk, d, sections, far)
    one = np.ones(d)
    wq, wk = (x["wq"], x["wk"]) if weights else (one, one)
    wdev = [dev(x["wq"]), dev(x["wk"])] if weights else [None, None]
    q, k, pos, freq = dev(x["q"], dt), dev(x["k"], dt), torch.from_numpy(x["pos"].astype(np.int32)).cuda(), dev(x["freq"])
    say(f"  [gpu] qk_norm_rope {case} weights={weights}")
    qo, ko = mh.qk_norm_rope(q, k, *wdev, pos, freq, sections, style=int(inter), eps=eps)
    dq, dk, dwq, dwk = mh.qk_norm_rope_backward(q, k, *wdev, pos, freq, sections, dev(x["dq"], dt), dev(x["dk"], dt),
                                                style=int(inter), eps=eps)
    torch.cuda.synchronize()
    for name, a, w, got, g, gd, gw in (("q", x["q"], wq, qo, x["dq"], dq, dwq), ("k", x["k"], wk, ko, x["dk"], dk, dwk)):
        ref = og.norm_rope(a, w, x["pos"], x["freq"], sections, inter, eps)
        n = a / np.sqrt(np.mean(a * a, -1, keepdims=True) + eps) * w
        # a pair's length bounds both of its members
        size = np.max(np.abs(n), -1, keepdims=True) * 1.5
        within(name, got, ref, REL[dt] * np.abs(ref) * 1.001 + (32 + d / 2) * 2.0 ** -24 * size)
        dx, dw = og.norm_rope_backward(a, w, x["pos"], x["freq"], sections, inter, eps, g)
        rs = 1 / np.sqrt(np.mean(a * a, -1, keepdims=True) + eps)
        u = np.abs(a) * rs
        dn = np.max(np.abs(g), -1, keepdims=True) * 1.5 * np.max(np.abs(w))
        mag = rs * (dn + u * np.mean(dn * u, -1, keepdims=True))
        within("d" + name, gd, dx, REL[dt] * np.abs(dx) * 1.001 + (64 + 2 * d) * 2.0 ** -24 * mag)
        if weights:
            # each row's term off by (32 + d / 2) 2^-24 of its size; a lane adds at most 48 rows here, a workgroup
            # 64 partial sums
            mw = np.sum(np.max(np.abs(g), -1, keepdims=True) * 1.5 * u, axis=(0, 1, 2))
            within("dw" + name, gw, dw, (32 + d / 2 + 48 + 64) * 2.0 ** -24 * mw)
        else:
            assert gw is None


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_slices_and_in_place_give_the_same_bits(dt):
    B, T, H, Hk, d, sections = 2, 130, 6, 2, 64, (16, 8)
    x = make(1, dt, B, T, H, Hk, d, sections)
    q, k, pos, freq = dev(x["q"], dt), dev(x["k"], dt), torch.from_numpy(x["pos"].astype(np.int32)).cuda(), dev(x["freq"])
    wq, wk = dev(x["wq"]), dev(x["wk"])
    a = mh.qk_norm_rope(q, k, wq, wk, pos, freq, sections)
    row = torch.cat([q.flatten(2), k.flatten(2), torch.full((B, T, Hk * d), float("nan"), dtype=dt, device="cuda")], -1)
    qs, ks = (t.unflatten(-1, (-1, d)) for t in row.split([H * d, Hk * d, Hk * d], dim=-1)[:2])
    b = mh.qk_norm_rope(qs, ks, wq, wk, pos, freq, sections)
    seq, rope = mh.make_seq(B, T, H, Hk, d, mh.MHLA_BF16 if dt == BF else mh.MHLA_F32), mh.make_rope(sections)
    qi, ki = q.clone(), k.clone()
    assert mh.mhla_qk_norm_rope(qi, ki, wq, wk, pos, freq, rope, seq, qi, ki) == mh.MHLA_OK
    dqo, dko = dev(x["dq"], dt), dev(x["dk"], dt)
    ga = mh.qk_norm_rope_backward(q, k, wq, wk, pos, freq, sections, dqo, dko)
    gb = mh.qk_norm_rope_backward(qs, ks, wq, wk, pos, freq, sections, dqo, dko)
    n = mh.mhla_qk_norm_rope_backward_workspace_bytes(seq)
    ws, dwq, dwk = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(wq), torch.empty_like(wk)
    assert mh.mhla_qk_norm_rope_backward(q, k, wq, wk, pos, freq, rope, dqo, dko, seq, dqo, dko, dwq, dwk, ws,
                                         n) == mh.MHLA_OK
    torch.cuda.synchronize()
    for u, v, w in zip(a, b, (qi, ki)):
        assert torch.equal(u, v) and torch.equal(u, w)
    for u, v, w in zip(ga, gb, (dqo, dko, dwq, dwk)):
        assert torch.equal(u, v) and torch.equal(u, w)


def test_many_tokens_reach_the_weights_gradient():
    """More tokens than one pass of the workgroups: dw against the same sum in 64 bits on the device."""
    B, T, H, Hk, d = 1, 40000, 3, 2, 64
    gen = torch.Generator(device="cuda").manual_seed(2)
    q, k, dqo, dko = (torch.randn(B, T, h, d, generator=gen, device="cuda").to(BF) for h in (H, Hk, H, Hk))
    pos = torch.arange(T, dtype=torch.int32, device="cuda").reshape(1, T, 1)
    freq = torch.zeros(32, device="cuda")                    # no turn: dn is the gradient itself
    w = torch.ones(d, device="cuda")
    dq, dk, dwq, dwk = mh.qk_norm_rope_backward(q, k, w, w, pos, freq, None, dqo, dko)
    qo, ko = mh.qk_norm_rope(q, k, w, w, pos, freq)
    for x, dy, dw, y in ((q, dqo, dwq, qo), (k, dko, dwk, ko)):
        x, dy = x.double(), dy.double()
        u = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        ref, mag = (dy * u).sum((0, 1, 2)), (dy * u).abs().sum((0, 1, 2))
        over = ((dw.double() - ref).abs() / (mag * (32 + d / 2 + 48 + 64) * 2.0 ** -24)).max().item()
        say(f"    dw: {over:.3f} of its tolerance")
        assert over <= 1.0
        assert ((y.double() - u).abs() <= 2.0 ** -8 * u.abs() * 1.001 + 1e-5).all()


def test_no_tokens():
    e, w = torch.empty(2, 0, 3, 32, device="cuda"), torch.ones(32, device="cuda")
    pos, freq = torch.empty(2, 0, 1, dtype=torch.int32, device="cuda"), torch.ones(8, device="cuda")
    q, k = mh.qk_norm_rope(e, e, w, w, pos, freq)
    dq, dk, dwq, dwk = mh.qk_norm_rope_backward(e, e, w, w, pos, freq, None, e, e)
    torch.cuda.synchronize()
    assert q.shape == e.shape and dq.shape == e.shape and not dwq.any() and not dwk.any()


def chain(row, w, x, sections, scale, lens):
    """Projection row [B, T, (H + 2 Hk) d] -> norm and rotation -> gated attention; and back from dout."""
    H, Hk, d = x["H"], x["Hk"], x["d"]
    q, k, v = (t.unflatten(-1, (-1, d)) for t in row.split([H * d, Hk * d, Hk * d], dim=-1))
    qr, kr = mh.qk_norm_rope(q, k, *w, x["pos"], x["freq"], sections)
    out, S = mh.gated_forward(qr, kr, v, x["g"], scale, None, lens, want_state=True)
    dqr, dkr, dv, dg, _ = mh.gated_backward(qr, kr, v, x["g"], x["do"], scale, None, None, lens)
    dq, dk, dwq, dwk = mh.qk_norm_rope_backward(q, k, *w, x["pos"], x["freq"], sections, dqr, dkr)
    return out, S, torch.cat([dq.flatten(2), dk.flatten(2), dv.flatten(2)], -1), dg, dwq, dwk


def test_chain_of_a_layer():
    """The run of a layer in fp32: rows of a projection, norm and rotation, attention, and all gradients,
    against the oracle's own chain; then the same in bf16, within its roundings in norm."""
    B, T, H, Hk, d, sections = 2, 150, 4, 2, 64, (16, 16)
    r = np.random.default_rng(3)
    row = r.normal(size=(B, T, (H + 2 * Hk) * d)).astype(np.float32).astype(np.float64)
    m = make(4, F32, B, T, H, Hk, d, sections)
    g = -0.05 * np.abs(r.normal(size=(B, T, Hk))).astype(np.float32).astype(np.float64)
    do = r.normal(size=(B, T, H, d)).astype(np.float32).astype(np.float64)
    lens, scale = [150, 77], d ** -0.5
    split = np.split(row, [H * d, (H + Hk) * d], axis=-1)
    q, k, v = (s.reshape(B, T, -1, d) for s in split)
    rope = lambda a, w: og.norm_rope(a, w, m["pos"], m["freq"], sections, False, 1e-6)  # noqa: E731
    qr, kr = rope(q, m["wq"]), rope(k, m["wk"])
    out, S = og.gated_forward(qr, kr, v, g, scale, None, lens)
    dqr, dkr, dv, dg, _ = og.gated_backward(qr, kr, v, g, do, scale, None, None, lens)
    dq, dwq = og.norm_rope_backward(q, m["wq"], m["pos"], m["freq"], sections, False, 1e-6, dqr)
    dk, dwk = og.norm_rope_backward(k, m["wk"], m["pos"], m["freq"], sections, False, 1e-6, dkr)
    drow = np.concatenate([a.reshape(B, T, -1) for a in (dq, dk, dv)], -1)
    x = {"H": H, "Hk": Hk, "d": d, "pos": torch.from_numpy(m["pos"].astype(np.int32)).cuda(), "freq": dev(m["freq"]),
         "g": dev(g)}
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for dt, tol in ((F32, 1e-5), (BF, 2e-2)):
        # fp32: the framework's bar; bf16: q, k, v, their rotated forms and dout are each rounded at 2^-9 in the
        # mean, five roundings on the way of a gradient
        x["do"] = dev(do, dt)
        got = chain(dev(row, dt), (dev(m["wq"]), dev(m["wk"])), x, sections, scale, ln)
        torch.cuda.synchronize()
        for n, a, b in zip(("out", "state", "drow", "dg", "dwq", "dwk"), got, (out, S, drow, dg, dwq, dwk)):
            err = float(np.linalg.norm(host(a) - b) / np.linalg.norm(b))
            say(f"    {dt} {n}: {err:.2e}")
            assert err <= tol


def test_tokens_past_one_launch():
    """More tokens than the workgroups of one launch take: the last ones are those of a short call."""
    d, T, tail = 32, (1 << 27) + 5000, 300
    pos = torch.zeros(1, T, 1, dtype=torch.int32, device="cuda")
    pos[0, T - tail:, 0] = torch.arange(tail, dtype=torch.int32, device="cuda")
    freq = 0.5 ** torch.arange(8, device="cuda", dtype=F32)
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k = torch.ones(1, T, 1, d, dtype=BF, device="cuda"), torch.empty(1, T, 0, d, dtype=BF, device="cuda")
    q[:, T - tail:] = torch.randn(1, tail, 1, d, generator=gen, device="cuda").to(BF)
    say(f"  [gpu] qk_norm_rope over {T} tokens")
    qo, _ = mh.qk_norm_rope(q, k, None, None, pos, freq)
    want, _ = mh.qk_norm_rope(q[:, T - tail:].contiguous(), k[:, T - tail:], None, None, pos[:, T - tail:].contiguous(), freq)
    torch.cuda.synchronize()
    assert torch.equal(qo[:, T - tail:], want)
    # ones of mean square 1, position 0: themselves, to 2^-20
    assert (qo[:, :T - tail] == 1).all()
