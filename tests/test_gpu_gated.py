"""Gated linear attention (mhla_gated_forward, _backward, _step) against the
float64 oracle on the same inputs.

Tolerances, elementwise.  Every output is a sum of products; `mag` is the same
sum over the products' absolute values (the oracle on |q|, |k|, |v|, ..).
A sum of n fp32 terms is off by at most n 2^-24 mag; here n counts the head
values and tokens of a chunk that one output adds, the chunks its state has
been carried over and 16 for exponentials, scales and the running gate sums.
The bf16 kernels take states and pair weights as two bf16 terms: 2^-16 mag
(twice 2^-17).  The final rounding is at most eps / 2 of the value.
"""
import numpy as np
import pytest
import torch

import token_level_head_block_amd as mh
from oracle import gated as og

from gpu_util import say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
CHUNK = 64


def dev(x, dt=F32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(dt).cuda()


def host(t):
    return t.double().cpu().numpy()


def inputs(seed, dt, B, T, H, Hk, d, state=True, gate=0.05, resets=0.0):
    """Values as the device sees them (rounded to dt), as float64 arrays."""
    r = np.random.default_rng(seed)
    rnd = lambda x: host(torch.from_numpy(x.astype(np.float32)).to(dt))  # noqa: E731
    x = {"q": rnd(r.normal(size=(B, T, H, d))), "k": rnd(r.normal(size=(B, T, Hk, d))),
         "v": rnd(r.normal(size=(B, T, Hk, d))), "do": rnd(r.normal(size=(B, T, H, d)))}
    g = -gate * np.abs(r.normal(size=(B, T, Hk)))
    g[r.random(size=g.shape) < resets] = -np.inf
    x["g"] = g.astype(np.float32).astype(np.float64)
    f = lambda: r.normal(size=(B, Hk, d, d)).astype(np.float32).astype(np.float64)  # noqa: E731
    x["s0"], x["ds1"] = (f(), f()) if state else (None, None)
    return x


def check(name, got, ref, mag, dt, d, T, terms=True):
    got = host(got)
    assert got.shape == ref.shape
    n = d + CHUNK + T / CHUNK + 16
    rel = {BF: 2.0 ** -8, F32: 2.0 ** -24}[dt]
    unit = n * 2.0 ** -24 + (2.0 ** -16 if terms else 0.0)
    tol = rel * np.abs(ref) * 1.001 + unit * mag + 1e-30
    over = float(np.max(np.abs(got - ref) / tol)) if ref.size else 0.0
    say(f"    {name}: error at most {over:.3f} of its tolerance")
    assert np.isfinite(got).all() and over <= 1.0, name


def mags(x, scale, lens=None):
    a = {k: None if v is None else np.abs(v) for k, v in x.items() if k != "g"}
    out, S = og.gated_forward(a["q"], a["k"], a["v"], x["g"], scale, a["s0"], lens)
    grads = og.gated_backward(a["q"], a["k"], a["v"], x["g"], a["do"], scale, a["s0"], a["ds1"], lens)
    return out, S, grads


def run_forward(x, dt, scale, lens=None, pad=0, **kw):
    q, k, v = (dev(x[n], dt) for n in "qkv")
    if pad:
        # slices of a wider row
        B, T, H, d = q.shape
        Hk = k.shape[2]
        row = torch.full((B, T, (H + 2 * Hk) * d + pad), float("nan"), dtype=dt, device="cuda")
        row[..., pad:] = torch.cat([q.flatten(2), k.flatten(2), v.flatten(2)], -1)
        q, k, v = (s.unflatten(-1, (-1, d)) for s in row[..., pad:].split([H * d, Hk * d, Hk * d], dim=-1))
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    s0 = None if x["s0"] is None else dev(x["s0"])
    say(f"  [gpu] gated_forward {tuple(q.shape)} Hk={k.shape[2]} {dt} lens={lens} pad={pad} state={s0 is not None}")
    out, S = mh.gated_forward(q, k, v, dev(x["g"]), scale, s0, ln, want_state=True)
    torch.cuda.synchronize()
    return (q, k, v, ln, s0), out, S


SHAPES = [
    # B, T, H, Hk, d, dtype
    (1, 1, 1, 1, 32, BF), (2, 1, 4, 2, 64, F32), (1, 63, 2, 2, 64, BF), (2, 64, 3, 1, 32, F32),
    (1, 65, 2, 1, 128, BF), (1, 130, 2, 2, 128, F32), (3, 200, 6, 2, 64, BF), (2, 321, 4, 4, 32, BF),
    (1, 577, 2, 2, 64, F32), (2, 260, 4, 1, 128, BF), (1, 700, 3, 3, 32, F32), (1, 1300, 1, 1, 64, BF),
    (32, 200, 8, 8, 32, BF), (1, 900, 6, 2, 128, F32), (2, 1100, 3, 1, 128, BF), (1, 128, 3, 3, 128, F32),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(i).replace("torch.", "") for i in s))
@pytest.mark.parametrize("state", [False, True], ids=["zero", "state"])
def test_forward_and_backward(shape, state):
    B, T, H, Hk, d, dt = shape
    x = inputs(sum(shape[:5]), dt, B, T, H, Hk, d, state)
    scale = d ** -0.5
    ref, Sr = og.gated_forward(x["q"], x["k"], x["v"], x["g"], scale, x["s0"])
    mo, mS, mg = mags(x, scale)
    (q, k, v, _, s0), out, S = run_forward(x, dt, scale)
    check("out", out, ref, mo, dt, d, T, dt == BF)
    check("state", S, Sr, mS, F32, d, T, False)
    say("  [gpu] gated_backward")
    grads = mh.gated_backward(q, k, v, dev(x["g"]), dev(x["do"], dt), scale, s0, dev(x["ds1"]) if state else None)
    torch.cuda.synchronize()
    refs = og.gated_backward(x["q"], x["k"], x["v"], x["g"], x["do"], scale, x["s0"], x["ds1"])
    for n, got, r, m in zip(("dq", "dk", "dv"), grads, refs, mg):
        check(n, got, r, m, dt, d, T, dt == BF)
    check_gate_gradient(grads[3], refs[3], x, scale, d, T)
    if state:
        check("dstate", grads[4], refs[4], mg[4], F32, d, T, False)
    else:
        assert grads[4] is None


def check_gate_gradient(dg, ref, x, scale, d, T, lens=None):
    """dg is a sum of q . dq - k . dk over a segment's tokens (at most 16 chunks) and one <S, dS>: each
    term off by (d + 64 + 16 + chunks) 2^-24 of its magnitude."""
    a = {k: None if v is None else np.abs(v) for k, v in x.items() if k != "g"}
    dq, dk, _, _, _ = og.gated_backward(a["q"], a["k"], a["v"], x["g"], a["do"], scale, a["s0"], a["ds1"], lens)
    Hk = x["k"].shape[2]
    B, _, H, _ = x["q"].shape
    r = np.sum(a["q"] * dq, -1).reshape(B, T, Hk, H // Hk).sum(-1) + np.sum(a["k"] * dk, -1)
    # the sums from t to the segment's end, and what crosses that end, whose magnitude is below that of
    # the crossing products at any token: bounded by the running maximum of r
    seg = 16 * CHUNK
    tail = np.zeros_like(r)
    for t0 in range(0, T, seg):
        tail[:, t0:t0 + seg] = np.cumsum(r[:, t0:t0 + seg][:, ::-1], 1)[:, ::-1]
    _, _, _, mag, _ = og.gated_backward(a["q"], a["k"], a["v"], x["g"], a["do"], scale, a["s0"], a["ds1"], lens)
    cross = np.max(mag, axis=1, keepdims=True)
    got = host(dg)
    tol = (d + CHUNK + T / CHUNK + 16) * 2.0 ** -24 * (tail + cross) + 2.0 ** -24 * np.abs(ref) + 1e-30
    over = float(np.max(np.abs(got - ref) / tol)) if ref.size else 0.0
    rel = float(np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30))
    say(f"    dg: error at most {over:.3f} of its tolerance, {rel:.2e} in all")
    assert np.isfinite(got).all() and over <= 1.0


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_lengths_and_what_lies_behind_them(dt):
    """Rows behind a sequence hold NaN and infinities: they reach nothing, and results there are zero."""
    B, T, H, Hk, d = 5, 300, 4, 2, 64
    lens = [300, 0, 1, 129, 5000]
    x = inputs(3, dt, B, T, H, Hk, d)
    scale = 0.1
    ref, Sr = og.gated_forward(x["q"], x["k"], x["v"], x["g"], scale, x["s0"], lens)
    refs = og.gated_backward(x["q"], x["k"], x["v"], x["g"], x["do"], scale, x["s0"], x["ds1"], lens)
    mo, mS, mg = mags(x, scale, lens)
    bad = {n: a if a is None or n in ("s0", "ds1") else a.copy() for n, a in x.items()}
    for n in ("q", "k", "v", "do", "g"):
        for b, ln in enumerate(lens):
            bad[n][b, min(ln, T):] = np.nan if b % 2 else np.inf
    (q, k, v, ln, s0), out, S = run_forward(bad, dt, scale, lens)
    check("out", out, ref, mo, dt, d, T, dt == BF)
    check("state", S, Sr, mS, F32, d, T, False)
    grads = mh.gated_backward(q, k, v, dev(bad["g"]), dev(bad["do"], dt), scale, s0, dev(x["ds1"]), ln)
    torch.cuda.synchronize()
    for n, got, r, m in zip(("dq", "dk", "dv"), grads, refs, mg):
        check(n, got, r, m, dt, d, T, dt == BF)
    check_gate_gradient(grads[3], refs[3], x, scale, d, T, lens)
    check("dstate", grads[4], refs[4], mg[4], F32, d, T, False)
    for t in (out, *grads[:4]):
        for b, n in enumerate(lens):
            assert not t[b, min(n, T):].any()


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("gate,resets", [(0.0, 0.0), (30.0, 0.0), (0.05, 0.1), (200.0, 0.3)])
def test_gates_from_one_to_zero(dt, gate, resets):
    """Gates of 1, gates far below fp32's range of products, and gates of 0."""
    B, T, H, Hk, d = 1, 200, 2, 1, 32
    x = inputs(4, dt, B, T, H, Hk, d, True, gate, resets)
    scale = 1.0
    with np.errstate(invalid="ignore"):
        ref, Sr = og.gated_forward(x["q"], x["k"], x["v"], x["g"], scale, x["s0"])
        refs = og.gated_backward(x["q"], x["k"], x["v"], x["g"], x["do"], scale, x["s0"], x["ds1"])
        mo, mS, mg = mags(x, scale)
    (q, k, v, _, s0), out, S = run_forward(x, dt, scale)
    # exponents of size |g| in powers of two are off by at most 2^-24 of their own size, and a weight
    # exp(-a) a 2^-24 is below 2^-24: the count of 16 in the tolerance holds them
    check("out", out, ref, mo, dt, d, T, dt == BF)
    check("state", S, Sr, mS, F32, d, T, False)
    grads = mh.gated_backward(q, k, v, dev(x["g"]), dev(x["do"], dt), scale, s0, dev(x["ds1"]))
    torch.cuda.synchronize()
    for n, got, r, m in zip(("dq", "dk", "dv"), grads, refs, mg):
        check(n, got, r, m, dt, d, T, dt == BF)
    check_gate_gradient(grads[3], refs[3], x, scale, d, T)
    assert not host(grads[3])[np.exp(x["g"].astype(np.float32)) == 0].any()


def test_packed_sequences_do_not_see_each_other():
    """A gate of 0 at each sequence's first token packs sequences: each gives what it gives alone."""
    H, Hk, d = 2, 2, 64
    parts = [1, 70, 64, 130, 3]
    x = inputs(5, BF, 1, sum(parts), H, Hk, d, False)
    t0 = 0
    for n in parts:
        x["g"][0, t0] = -np.inf
        t0 += n
    (q, k, v, _, _), out, S = run_forward(x, BF, 1.0)
    t0 = 0
    for n in parts:
        y = {m: a if a is None else a[:, t0:t0 + n] for m, a in x.items()}
        ref, Sr = og.gated_forward(y["q"], y["k"], y["v"], y["g"], 1.0)
        mo, mS, _ = mags(y, 1.0)
        check(f"out of {n}", out[:, t0:t0 + n], ref, mo, BF, d, sum(parts))
        t0 += n
    check("state", S, Sr, mS, F32, d, sum(parts), False)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_slices_of_a_projection_give_the_same_bits(dt, d):
    x = inputs(6, dt, 2, 150, 4, 2, d)
    (q, k, v, _, s0), a, Sa = run_forward(x, dt, 0.3)
    (qs, ks, vs, _, _), b, Sb = run_forward(x, dt, 0.3, pad=8)
    assert torch.equal(a, b) and torch.equal(Sa, Sb)
    g, do, ds1 = dev(x["g"]), dev(x["do"], dt), dev(x["ds1"])
    ga = mh.gated_backward(q, k, v, g, do, 0.3, s0, ds1)
    gb = mh.gated_backward(qs, ks, vs, g, do, 0.3, s0, ds1)
    torch.cuda.synchronize()
    for u, w in zip(ga, gb):
        assert torch.equal(u, w)


def test_repeats_give_the_same_bits_on_another_stream_and_workspace():
    x = inputs(7, BF, 1, 2000, 4, 2, 64)
    (q, k, v, _, s0), a, Sa = run_forward(x, BF, 0.3)
    seq = mh.make_seq(1, 2000, 4, 2, 64, mh.MHLA_BF16, 0.3)
    n = mh.mhla_gated_workspace_bytes(seq)
    assert n > 0                                             # few heads: the sequence is split
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, S = torch.empty_like(a), torch.empty_like(Sa)
    assert mh.mhla_gated_forward(q, k, v, dev(x["g"]), seq, out, None, s0, S, ws, n, s) == mh.MHLA_OK
    torch.cuda.synchronize()
    assert torch.equal(a, out) and torch.equal(Sa, S)
    # the workspace allocated by the call, and the state updated in place
    st = s0.clone()
    assert mh.mhla_gated_forward(q, k, v, dev(x["g"]), seq, out, None, st, st) == mh.MHLA_OK
    torch.cuda.synchronize()
    assert torch.equal(a, out) and torch.equal(Sa, st)


def test_packed_gradients_do_not_see_each_other():
    """Gates' gradients of packed sequences, one of them with values 10^6 times as large: each sequence's are
    those it gives alone, within its own sums' tolerance."""
    H, Hk, d = 2, 2, 64
    parts = [1, 70, 64, 130, 3, 90]
    x = inputs(14, F32, 1, sum(parts), H, Hk, d, False)
    t0 = 0
    for i, n in enumerate(parts):
        x["g"][0, t0] = -np.inf
        if i == 3:
            x["q"][:, t0:t0 + n] *= 2.0 ** 20
            x["v"][:, t0:t0 + n] *= 2.0 ** 20
        t0 += n
    q, k, v, g, do = (dev(x[n]) for n in ("q", "k", "v", "g", "do"))
    dg = mh.gated_backward(q, k, v, g, do, 1.0)[3]
    torch.cuda.synchronize()
    t0 = 0
    for n in parts:
        y = {m: a if a is None else a[:, t0:t0 + n] for m, a in x.items()}
        ref = og.gated_backward(y["q"], y["k"], y["v"], y["g"], y["do"], 1.0)[3]
        check_gate_gradient(dg[:, t0:t0 + n], ref, y, 1.0, d, n)
        t0 += n


def test_two_streams_at_once():
    """Two calls with workspaces of their own, running side by side many times, give what each gives alone."""
    xs = [inputs(30 + i, BF, 1, 3000, 2, 2, 64) for i in range(2)]
    alone = []
    for x in xs:
        (q, k, v, _, s0), a, Sa = run_forward(x, BF, 0.3)
        g, do, ds1 = dev(x["g"]), dev(x["do"], BF), dev(x["ds1"])
        alone.append(((q, k, v, g, do, s0, ds1), (a, Sa, *mh.gated_backward(q, k, v, g, do, 0.3, s0, ds1))))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            q, k, v, g, do, s0, ds1 = alone[i][0]
            with torch.cuda.stream(s):
                out, S = mh.gated_forward(q, k, v, g, 0.3, s0, want_state=True)
                got[i] = (out, S, *mh.gated_backward(q, k, v, g, do, 0.3, s0, ds1))
    torch.cuda.synchronize()
    for (_, want), have in zip(alone, got):
        for a, b in zip(want, have):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 values: the last tokens, behind a gate of 0, give what they give alone."""
    H, d, T, tail = 64, 64, 560000, 200
    assert T * H * d > 1 << 31
    gen = torch.Generator(device="cuda").manual_seed(0)
    small = [torch.randn(1, tail, H, d, generator=gen, device="cuda").to(BF) for _ in range(4)]
    gs = -0.1 * torch.rand(1, tail, H, generator=gen, device="cuda")
    gs[:, 0] = -float("inf")
    q, k, v, do = (torch.zeros(1, T, H, d, dtype=BF, device="cuda") for _ in range(4))
    g = torch.zeros(1, T, H, device="cuda")
    for a, b in zip((q, k, v, do, g), (*small, gs)):
        a[:, T - tail:] = b
    say(f"  [gpu] gated forward and backward over {q.numel()} values")
    # the short call starts at a chunk of its own, the long one inside a chunk: other sums of the same terms
    want = (mh.gated_forward(*small[:3], gs, 0.1), *mh.gated_backward(*small[:3], gs, small[3], 0.1)[:4])
    out = mh.gated_forward(q, k, v, g, 0.1)
    grads = mh.gated_backward(q, k, v, g, do, 0.1)[:4]
    torch.cuda.synchronize()
    for name, a, b in zip(("out", "dq", "dk", "dv", "dg"), (out, *grads), want):
        x, y = a[:, T - tail:].double(), b.double()
        err = ((x - y).abs().max() / y.abs().max()).item()
        say(f"    {name}: {err:.2e}")
        assert err <= (2.0 ** -8 if a.dtype == BF else 1e-5)
        assert not a[:, :T - tail].any()


def test_no_tokens_copies_the_state():
    s0 = torch.randn(2, 3, 32, 32, device="cuda")
    e = torch.empty(2, 0, 3, 32, device="cuda")
    out, S = mh.gated_forward(e, e, e, torch.empty(2, 0, 3, device="cuda"), 1.0, s0, want_state=True)
    dq, dk, dv, dg, ds = mh.gated_backward(e, e, e, torch.empty(2, 0, 3, device="cuda"), e, 1.0, s0, s0 * 2)
    torch.cuda.synchronize()
    assert out.shape == e.shape and torch.equal(S, s0) and torch.equal(ds, s0 * 2)


def test_long_sequence_carries_its_state():
    """Sums over 20000 tokens with gates close to 1: the state is an fp32 sum."""
    B, T, H, Hk, d = 1, 20001, 1, 1, 32
    x = inputs(8, BF, B, T, H, Hk, d, True, 1e-4)
    ref, Sr = og.gated_forward(x["q"], x["k"], x["v"], x["g"], 1.0, x["s0"])
    _, out, S = run_forward(x, BF, 1.0)
    err = np.linalg.norm(host(S) - Sr) / np.linalg.norm(Sr)
    say(f"    state: {err:.2e}")
    # 20001 products of random sign, each partial sum rounded at 2^-25 of a value that grows as the
    # square root: about sqrt(chunks) 2^-25 of the last one, times the products' own 2^-24
    assert err <= (T / CHUNK) ** 0.5 * 2.0 ** -24
    mo = og.gated_forward(*(np.abs(x[n]) for n in "qkv"), x["g"], 1.0, np.abs(x["s0"]))[0]
    check("out", out, ref, mo, BF, d, T)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hk,d", [(1, 6, 6, 64), (3, 4, 2, 128), (5, 3, 1, 32), (2, 8, 8, 128)])
def test_step(dt, B, H, Hk, d):
    x = inputs(9, dt, B, 1, H, Hk, d)
    q, k, v, g = x["q"][:, 0], x["k"][:, 0], x["v"][:, 0], x["g"][:, 0]
    ref, pr = og.gated_step(q, k, v, g, x["s0"], 0.2)
    mo, mp = og.gated_step(abs(q), abs(k), abs(v), g, abs(x["s0"]), 0.2)
    pool = dev(x["s0"])
    say(f"  [gpu] gated_step {B} {H} {Hk} {d} {dt}")
    out = mh.gated_step(dev(q, dt), dev(k, dt), dev(v, dt), dev(g), pool, 0.2)
    torch.cuda.synchronize()
    check("out", out, ref, mo, dt, d, 1, False)
    check("pool", pool, pr, mp, F32, d, 1, False)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_step_slots(dt):
    """Slots in any order, outside the pool, and the same one more than once (rows far apart too)."""
    d, H, Hk, n = 64, 4, 2, 9
    slots = [3, -1, 0, 3, 9, 8, 3, 1 << 30, 0] + list(range(n)) * 1 + [-(1 << 31)] + [3] * 2
    slots += [n + 5] * 300 + [8]                     # the last row lies in another pass of the search
    B = len(slots)
    r = np.random.default_rng(10)
    x = inputs(11, dt, B, 1, H, Hk, d, False)
    q, k, v, g = x["q"][:, 0], x["k"][:, 0], x["v"][:, 0], x["g"][:, 0]
    pool0 = r.normal(size=(n, Hk, d, d)).astype(np.float32).astype(np.float64)
    ref, pr = og.gated_step(q, k, v, g, pool0, 1.0, slots)
    mo, mp = og.gated_step(abs(q), abs(k), abs(v), g, abs(pool0), 1.0, slots)
    pool = dev(pool0)
    say(f"  [gpu] gated_step slots B={B}")
    out = mh.gated_step(dev(q, dt), dev(k, dt), dev(v, dt), dev(g), pool, 1.0,
                        torch.tensor(slots, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    check("out", out, ref, mo, dt, d, 64 * 6, False)
    check("pool", pool, pr, mp, F32, d, 64 * 6, False)
    for b, s in enumerate(slots):
        if not 0 <= s < n:
            assert not out[b].any()


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_prefill_then_steps_equal_the_whole(dt):
    """A prompt by the chunk form, then a token at a time from the state it leaves: the oracle's outputs of
    the whole sequence, with rows of the batch at different lengths."""
    B, T, H, Hk, d, new = 3, 130, 4, 2, 64, 5
    lens = [130, 7, 64]
    x = inputs(12, dt, B, T + new, H, Hk, d, False)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, k, v = (dev(x[n][:, :T], dt) for n in "qkv")
    out, pool = mh.gated_forward(q, k, v, dev(x["g"][:, :T]), 0.5, None, ln, want_state=True)
    outs = [mh.gated_step(dev(x["q"][:, T + i], dt), dev(x["k"][:, T + i], dt), dev(x["v"][:, T + i], dt),
                          dev(x["g"][:, T + i]), pool, 0.5) for i in range(new)]
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        y = {m: np.concatenate([x[m][b:b + 1, :n], x[m][b:b + 1, T:]], 1) for m in ("q", "k", "v", "g")}
        ref, S = og.gated_forward(y["q"], y["k"], y["v"], y["g"], 0.5)
        mo, mS = og.gated_forward(abs(y["q"]), abs(y["k"]), abs(y["v"]), y["g"], 0.5)
        got = torch.cat([out[b, :n]] + [o[b:b + 1] for o in outs])
        check(f"row {b}", got, ref[0], mo[0], dt, d, T, dt == BF)
        check(f"state {b}", pool[b], S[0], mS[0], F32, d, T, False)


def test_graph_replays():
    """Forward, backward and a step in one captured graph, replayed with other inputs and eager work of the
    same calls between: every replay equals the eager results bit for bit."""
    B, T, H, Hk, d = 1, 1500, 4, 2, 64
    xs = [inputs(20 + i, BF, B, T, H, Hk, d) for i in range(4)]
    seq, one = mh.make_seq(B, T, H, Hk, d, mh.MHLA_BF16, 0.4), mh.make_seq(B, 1, H, Hk, d, mh.MHLA_BF16, 0.4)
    nf, nb = mh.mhla_gated_workspace_bytes(seq), mh.mhla_gated_backward_workspace_bytes(seq)

    def buffers():
        e = lambda *s, dt=BF: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        return {"q": e(B, T, H, d), "k": e(B, T, Hk, d), "v": e(B, T, Hk, d), "g": e(B, T, Hk, dt=F32),
                "do": e(B, T, H, d), "s0": e(B, Hk, d, d, dt=F32), "ds1": e(B, Hk, d, d, dt=F32),
                "out": e(B, T, H, d), "S": e(B, Hk, d, d, dt=F32), "dq": e(B, T, H, d), "dk": e(B, T, Hk, d),
                "dv": e(B, T, Hk, d), "dg": e(B, T, Hk, dt=F32), "ds0": e(B, Hk, d, d, dt=F32), "o1": e(B, H, d),
                "wf": torch.empty(nf, dtype=torch.uint8, device="cuda"),
                "wb": torch.empty(nb, dtype=torch.uint8, device="cuda")}

    def fill(b, x):
        for n in ("q", "k", "v", "g", "do", "s0", "ds1"):
            b[n].copy_(dev(x[n], b[n].dtype))

    def work(b):
        assert mh.mhla_gated_forward(b["q"], b["k"], b["v"], b["g"], seq, b["out"], None, b["s0"], b["S"], b["wf"],
                                     nf) == mh.MHLA_OK
        assert mh.mhla_gated_backward(b["q"], b["k"], b["v"], b["g"], b["do"], seq, b["dq"], b["dk"], b["dv"],
                                      b["dg"], None, b["s0"], b["ds1"], b["ds0"], b["wb"], nb) == mh.MHLA_OK
        assert mh.mhla_gated_step(b["q"][:, 0], b["k"][:, 0], b["v"][:, 0], b["g"][:, 0], one, b["S"],
                                  b["o1"]) == mh.MHLA_OK

    a, e = buffers(), buffers()
    fill(a, xs[0])
    work(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(a)
    for x in xs[1:] + xs[:1]:
        fill(a, x)
        fill(e, x)
        work(e)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in ("out", "S", "dq", "dk", "dv", "dg", "ds0", "o1"):
            assert torch.equal(a[n], e[n]), n


def test_gradients_against_differences():
    """dL/dx along random directions against central differences of the fp32 forward."""
    B, T, H, Hk, d = 1, 150, 2, 1, 32
    x = inputs(13, F32, B, T, H, Hk, d, True, 0.1)
    q, k, v, g, s0, do, ds1 = (dev(x[n]) for n in ("q", "k", "v", "g", "s0", "do", "ds1"))
    grads = mh.gated_backward(q, k, v, g, do, 0.2, s0, ds1)

    def loss(args):
        out, S = mh.gated_forward(*args[:4], 0.2, args[4], want_state=True)
        return (out.double() * do.double()).sum() + (S.double() * ds1.double()).sum()
    args = [q, k, v, g, s0]
    gen = torch.Generator(device="cuda").manual_seed(0)
    for i, gr in enumerate(grads):
        u = torch.randn(args[i].shape, generator=gen, device="cuda")
        h = 1e-2 if i != 3 else 1e-3
        up, dn = (loss([a + s * h * u if j == i else a for j, a in enumerate(args)]) for s in (1, -1))
        num, ana = ((up - dn) / (2 * h)).item(), (gr.double() * u.double()).sum().item()
        # the loss is linear in each of q, k, v and the state but for their own roundings at 2^-24; its values
        # of size |L| are off by about 2^-22 |L| in all.  Along g it is smooth: an error of order h^2
        size = abs(loss(args).item()) + (gr.double() * u.double()).abs().sum().item()
        tol = 2.0 ** -20 * size / h + (h * h * 1e3 * size if i == 3 else 0.0)
        say(f"    input {i}: {num:.6g} against {ana:.6g} (tolerance {tol:.2g})")
        assert abs(num - ana) <= tol
