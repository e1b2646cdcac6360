"""Linear attention with one decay per head on the GPU against the fp64 token
recurrence (oracle/head_decay.py).

Tolerances.  A is the value of the same formula with every input replaced by its
magnitude, so every partial sum of the kernel is at most A.
  * a sum of n fp32 terms is off by at most n 2^-24 A; the kernels add at most
    256 channels, 64 tokens of a chunk, and one term per chunk and segment, and a
    decay factor exp(x g) is off by about (2 + |x g|) 2^-24: 512 roundings cover
    them all: 512 * 2^-24 = 2^-15.
  * bf16 inputs: the state and the decayed writes are bf16 hi + lo, each off by at
    most 2^-16 of itself: a state is off by at most 2^-16 A more per split it went
    through (two at most: 2^-15), so fp32 outputs get 2^-14 A;
  * an output in bf16 is rounded once, 2^-8 of itself, and its pairs are rounded
    to bf16 before they meet the third operand, 2^-8 A in all.
  * dg adds the parts of a pair's distance, each through two splits: 2^-13 A.
Inputs are converted to their dtype before both sides see them.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_26_amd as gdr
from oracle import head_decay as ref
from tests.gpu_util import DEV, host

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(seed, lens, H, Hk, Dk, Dv, dt, *, g=None, s0=True, packed=False):
    r = np.random.default_rng(seed)
    lead = (sum(lens),) if packed else (len(lens), lens[0])
    N = len(lens)

    def t(*shape, dtype=DT[dt]):
        return torch.from_numpy(r.normal(size=shape).astype(np.float32)).to(dtype).to(DEV)

    x = dict(q=t(*lead, H, Dk), k=t(*lead, Hk, Dk) / Dk ** 0.5, v=t(*lead, Hk, Dv))
    x["k"] = x["k"].to(DT[dt])
    gs = np.asarray(g if g is not None else -np.exp(r.uniform(-7, 0.5, size=H)), np.float32)
    x["g"] = torch.from_numpy(np.resize(gs, H).astype(np.float32)).to(DEV)
    x["s0"] = t(N, H, Dk, Dv, dtype=torch.float32) if s0 else None
    x["d_o"] = t(*lead, H, Dv)
    x["ds_final"] = t(N, H, Dk, Dv, dtype=torch.float32) if s0 else None
    x["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV) if packed else None
    return x


def sequences(x, lens, packed):
    at = 0
    for b, n in enumerate(lens):
        sl = slice(at, at + n) if packed else b
        at += n
        yield b, {k: host(x[k][sl]) for k in ("q", "k", "v", "d_o")}, {
            k: None if x[k] is None else host(x[k][b]) for k in ("s0", "ds_final")}


def mag(d):
    return {k: None if v is None else np.abs(v) for k, v in d.items()}


def close(name, got, want, A, rounded):
    """rounded: the output's dtype is bf16."""
    bf16_in = rounded is not None
    tol = 2.0 ** -15 * A if not bf16_in else 2.0 ** -14 * A if not rounded else 2.0 ** -8 * (np.abs(want) + A)
    err = np.abs(host(got).astype(np.float64) - want)
    assert np.all(np.isfinite(host(got))), name
    bad = err > tol + 1e-37
    assert not bad.any(), (name, int(bad.sum()), float((err / (tol + 1e-37)).max()), np.argwhere(bad)[:4].tolist())


def check_fwd(x, lens, dt, o, s, scale, packed=False):
    g, r = host(x["g"]), {"bf16": True, "f32": None}[dt]
    at = 0
    for b, tk, st in sequences(x, lens, packed):
        tk.pop("d_o")
        want, S = ref.forward(**tk, g=g, s0=st["s0"], scale=scale)
        A, SA = ref.forward(**mag(tk), g=g, s0=mag(st)["s0"], scale=abs(scale))
        got = o[at:at + lens[b]] if packed else o[b]
        at += lens[b]
        close(f"o[{b}]", got, want, A, r)
        if s is not None:
            close(f"s[{b}]", s[b], S[-1], SA[-1], None if r is None else False)


def check_bwd(x, lens, dt, out, scale, packed=False):
    g, r = host(x["g"]), {"bf16": True, "f32": None}[dt]
    at, dg, dgA = 0, 0.0, 0.0
    for b, tk, st in sequences(x, lens, packed):
        want = ref.backward(**tk, g=g, **st, scale=scale)
        A = ref.backward(**mag(tk), g=g, **mag(st), scale=abs(scale))
        for name in ("dq", "dk", "dv"):
            got = out[name][at:at + lens[b]] if packed else out[name][b]
            close(f"{name}[{b}]", got, want[name], A[name], r)
        if out["ds0"] is not None:
            close(f"ds0[{b}]", out["ds0"][b], want["ds0"], A["ds0"], None if r is None else False)
        at += lens[b]
        dg, dgA = dg + want["dg"], dgA + A["dg"]
    if out["dg"] is not None:
        err = np.abs(host(out["dg"]) - dg)
        assert np.all(err <= 2.0 ** -13 * dgA + 1e-37), ("dg", (err / (2.0 ** -13 * dgA + 1e-37)).max())


# B, T, H, Hk, Dk, Dv
SHAPES = [(1, 1, 1, 1, 8, 8), (2, 2, 2, 1, 16, 24), (1, 15, 3, 3, 64, 64), (2, 16, 4, 2, 64, 40), (1, 17, 2, 2, 72, 128),
          (1, 31, 1, 1, 128, 128), (1, 33, 2, 1, 128, 64), (2, 63, 2, 2, 40, 136), (1, 64, 4, 1, 128, 128),
          (1, 65, 2, 2, 256, 256), (3, 129, 6, 3, 64, 128), (1, 200, 2, 2, 136, 72), (1, 300, 2, 1, 96, 192)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(shape, dt):
    B, T, H, Hk, Dk, Dv = shape
    x = make(1, [T] * B, H, Hk, Dk, Dv, dt, s0=T % 2 == 1)
    o, s = gdr.head_decay_fwd(x["q"], x["k"], x["v"], x["g"], scale=0.25, s0=x["s0"])
    assert o.dtype == DT[dt] and s.dtype == torch.float32
    check_fwd(x, [T] * B, dt, o, s, 0.25)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_backward(shape, dt):
    B, T, H, Hk, Dk, Dv = shape
    x = make(2, [T] * B, H, Hk, Dk, Dv, dt, s0=T % 2 == 1)
    for need_dg in (False, True):
        out = gdr.head_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], scale=0.25, s0=x["s0"],
                                 ds_final=x["ds_final"], need_dg=need_dg, need_ds0=x["s0"] is not None)
        assert (out["dg"] is not None) == need_dg and out["dq"].dtype == DT[dt]
        check_bwd(x, [T] * B, dt, out, 0.25)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T, H", [(65, 2), (257, 2), (1100, 2), (5000, 1)])
def test_segments(T, H, dt):
    """A few heads of a long sequence are walked in segments (64 at most); the state is updated in place."""
    x = make(3, [T], H, 1, 64, 72, dt, g=[-0.003, -0.5])
    s = x["s0"].clone()
    o, s2 = gdr.head_decay_fwd(x["q"], x["k"], x["v"], x["g"], s0=s, s_final=s)
    assert s2 is s
    check_fwd(x, [T], dt, o, s, 1.0)
    out = gdr.head_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], s0=x["s0"], ds_final=x["ds_final"])
    check_bwd(x, [T], dt, out, 1.0)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_decays_at_the_ends(dt):
    """No decay, a decay that underflows within a chunk, and one that forgets at once."""
    x = make(4, [330], 4, 4, 64, 64, dt, g=[0.0, -3.0, -90.0, -np.inf])
    o, s = gdr.head_decay_fwd(x["q"], x["k"], x["v"], x["g"], s0=x["s0"])
    check_fwd(x, [330], dt, o, s, 1.0)
    out = gdr.head_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], s0=x["s0"], ds_final=x["ds_final"])
    check_bwd(x, [330], dt, out, 1.0)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[5], [0], [1, 0, 0, 70], [64, 128, 1], [300, 0, 700, 33, 0]],
                         ids=lambda s: "_".join(map(str, s)))
def test_packed(lens, dt):
    x = make(5, lens, 4, 2, 40, 128, dt, packed=True)
    o, s = gdr.head_decay_fwd_varlen(x["q"], x["k"], x["v"], x["g"], x["cu"], s0=x["s0"])
    check_fwd(x, lens, dt, o, s, 1.0, packed=True)
    out = gdr.head_decay_bwd_varlen(x["q"], x["k"], x["v"], x["g"], x["d_o"], x["cu"], s0=x["s0"],
                                    ds_final=x["ds_final"])
    check_bwd(x, lens, dt, out, 1.0, packed=True)


@pytest.mark.parametrize("Dv", [16, 72])
def test_packed_many_sequences(Dv):
    """More sequences than a workgroup has threads (256, or 512 for more than 64 columns)."""
    lens = [1 + i % 5 for i in range(600)]
    x = make(6, lens, 1, 1, 16, Dv, "f32", packed=True)
    o, s = gdr.head_decay_fwd_varlen(x["q"], x["k"], x["v"], x["g"], x["cu"], s0=x["s0"])
    check_fwd(x, lens, "f32", o, s, 1.0, packed=True)
    out = gdr.head_decay_bwd_varlen(x["q"], x["k"], x["v"], x["g"], x["d_o"], x["cu"], s0=x["s0"],
                                    ds_final=x["ds_final"])
    check_bwd(x, lens, "f32", out, 1.0, packed=True)


def test_packed_one_long_among_many():
    lens = [5] * 40 + [1500] + [3] * 40
    x = make(29, lens, 8, 4, 16, 24, "bf16", packed=True)
    o, s = gdr.head_decay_fwd_varlen(x["q"], x["k"], x["v"], x["g"], x["cu"], s0=x["s0"])
    check_fwd(x, lens, "bf16", o, s, 1.0, packed=True)
    out = gdr.head_decay_bwd_varlen(x["q"], x["k"], x["v"], x["g"], x["d_o"], x["cu"], s0=x["s0"],
                                    ds_final=x["ds_final"])
    check_bwd(x, lens, "bf16", out, 1.0, packed=True)


def test_packed_state_in_place():
    """Segments of a packed batch while s_final is s0."""
    lens = [700, 3, 450]
    x = make(21, lens, 2, 2, 64, 64, "bf16", packed=True)
    s = x["s0"].clone()
    o, s2 = gdr.head_decay_fwd_varlen(x["q"], x["k"], x["v"], x["g"], x["cu"], s0=s, s_final=s)
    assert s2 is s
    check_fwd(x, lens, "bf16", o, s, 1.0, packed=True)


def test_long_sequence_in_pieces():
    """A long sequence at once and in pieces that hand their state on; both are within the tolerance of the exact
    values, so within twice of each other, and the states' and outputs' A is bounded by the magnitudes' call."""
    T = 70001
    x = make(22, [T], 2, 1, 64, 128, "bf16", g=[-0.002, -0.2], s0=False)
    o, s = gdr.head_decay_fwd(x["q"], x["k"], x["v"], x["g"])
    A, SA = gdr.head_decay_fwd(x["q"].abs(), x["k"].abs(), x["v"].abs(), x["g"])
    st, parts = None, []
    for a, z in ((0, 20000), (20000, 20001), (20001, 61000), (61000, T)):
        p, st = gdr.head_decay_fwd(*(x[n][:, a:z] for n in "qkv"), x["g"], s0=st)
        parts.append(p)
    p = torch.cat(parts, 1)
    assert torch.all((o.double() - p.double()).abs() <= 2.0 ** -7 * (o.double().abs() + 1.01 * A.double()))
    assert torch.all((s.double() - st.double()).abs() <= 2.0 ** -13 * 1.01 * SA.double())


@pytest.mark.parametrize("cu, spans", [([3, 10, 20], [(3, 10), (10, 20)]), ([-5, 12, 4, 99], [(0, 12), (12, 12), (12, 40)]),
                                       ([40, 40], [(40, 40)]), ([7, 7, 7], [(7, 7), (7, 7)])])
def test_packed_offsets(cu, spans):
    """Tokens outside every sequence: rows of o stay, gradients are zero; offsets out of order are raised."""
    N = len(cu) - 1
    x = make(7, [40], 2, 1, 16, 16, "bf16", packed=True, s0=False)
    x["s0"] = torch.randn(N, 2, 16, 16, device=DEV)
    x["ds_final"] = torch.randn(N, 2, 16, 16, device=DEV)
    cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    o = torch.full((40, 2, 16), 7.0, dtype=torch.bfloat16, device=DEV)
    _, s = gdr.head_decay_fwd_varlen(x["q"], x["k"], x["v"], x["g"], cu, s0=x["s0"], o=o)
    out = gdr.head_decay_bwd_varlen(x["q"], x["k"], x["v"], x["g"], x["d_o"], cu, s0=x["s0"], ds_final=x["ds_final"])
    inside = np.zeros(40, bool)
    for n, (a, z) in enumerate(spans):
        inside[a:z] = True
        part = {k: x[k][a:z] for k in ("q", "k", "v", "d_o")}
        part.update({k: x[k][n:n + 1] for k in ("s0", "ds_final")}, g=x["g"])
        check_fwd(part, [z - a], "bf16", o[a:z], s[n:n + 1], 1.0, packed=True)
        one = {k: out[k][a:z] for k in ("dq", "dk", "dv")}
        check_bwd(part, [z - a], "bf16", dict(one, dg=None, ds0=out["ds0"][n:n + 1]), 1.0, packed=True)
    assert torch.all(o[torch.from_numpy(~inside).to(DEV)] == 7.0)
    for k in ("dq", "dk", "dv"):
        assert torch.all(out[k][torch.from_numpy(~inside).to(DEV)] == 0), k


def test_no_tokens():
    x = make(8, [0, 0], 2, 2, 16, 24, "bf16")
    o, s = gdr.head_decay_fwd(x["q"], x["k"], x["v"], x["g"], s0=x["s0"])
    assert o.shape == (2, 0, 2, 24) and torch.equal(s, x["s0"])
    _, s = gdr.head_decay_fwd(x["q"], x["k"], x["v"], x["g"])
    assert torch.all(s == 0)
    out = gdr.head_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], s0=x["s0"], ds_final=x["ds_final"])
    assert torch.equal(out["ds0"], x["ds_final"]) and torch.all(out["dg"] == 0)
    y = make(8, [0], 2, 2, 16, 24, "bf16", packed=True)
    e = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, s = gdr.head_decay_fwd_varlen(y["q"], y["k"], y["v"], y["g"], e)
    assert s.shape == (0, 2, 16, 24)


def fused(x):
    """q, k, v as views of one buffer, as a fused projection leaves them."""
    parts = [x[n].flatten(-2) for n in "qkv"]
    buf = torch.cat(parts, -1)
    out = dict(x)
    at = 0
    for n, p in zip("qkv", parts):
        out[n] = buf[..., at:at + p.shape[-1]].unflatten(-1, x[n].shape[-2:])
        at += p.shape[-1]
    return out


def test_views_and_broadcasts():
    x = make(9, [90, 90], 4, 2, 64, 128, "bf16")
    want = gdr.head_decay_fwd(x["q"], x["k"], x["v"], x["g"], s0=x["s0"])
    wb = gdr.head_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], s0=x["s0"], ds_final=x["ds_final"])
    y = fused(x)
    assert not y["k"].is_contiguous()
    y["d_o"] = x["d_o"].transpose(1, 2).contiguous().transpose(1, 2)
    got = gdr.head_decay_fwd(y["q"], y["k"], y["v"], y["g"], s0=y["s0"])
    gb = gdr.head_decay_bwd(y["q"], y["k"], y["v"], y["g"], y["d_o"], s0=y["s0"], ds_final=y["ds_final"])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for n in wb:
        assert torch.equal(gb[n], wb[n]), n
    # one key head and one sequence for all, by strides of zero
    k1 = x["k"][:1, :, :1].expand(2, 90, 2, 64)
    v1 = x["v"][:, :1].expand(2, 90, 2, 128)
    a = gdr.head_decay_fwd(x["q"], k1, v1, x["g"])
    b = gdr.head_decay_fwd(x["q"], k1.contiguous(), v1.contiguous(), x["g"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # the same key at every token
    k1 = x["k"][:, :1].expand(2, 90, 2, 64)
    a = gdr.head_decay_bwd(x["q"], k1, x["v"], x["g"], x["d_o"])
    b = gdr.head_decay_bwd(x["q"], k1.contiguous(), x["v"], x["g"], x["d_o"])
    for n in ("dq", "dk", "dv", "dg", "ds0"):
        assert torch.equal(a[n], b[n]), n
    a = gdr.head_decay_fwd(x["q"], k1, x["v"], x["g"])
    b = gdr.head_decay_fwd(x["q"], k1.contiguous(), x["v"], x["g"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_calls_at_once():
    """Calls on two streams without order between them, each with its own workspace."""
    xs = [make(23 + i, [900], 2, 1, 64, 64, "bf16") for i in range(2)]
    want = [gdr.head_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], s0=x["s0"]) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [[gdr.head_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], s0=x["s0"], stream=st)
            for x, st in zip(xs, streams)] for _ in range(3)]
    for st in streams:
        torch.cuda.current_stream().wait_stream(st)
    for run in got:
        for a, b in zip(run, want):
            for n in b:
                assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("Dk, Dv", [(64, 72), (72, 64), (16, 24), (128, 128), (200, 40), (40, 200), (136, 256)])
def test_a_workspace_used_again(Dk, Dv, dt):
    """The contents of a workspace do not matter: filled with NaN, and left by another call."""
    x = make(25, [700], 2, 1, Dk, Dv, dt)
    args = [x[n] for n in ("q", "k", "v", "g")]
    kw = dict(s0=x["s0"], ds_final=x["ds_final"])
    o, s = gdr.head_decay_fwd(*args, s0=x["s0"])
    check_fwd(x, [700], dt, o, s, 1.0)
    want = gdr.head_decay_bwd(*args, x["d_o"], **kw)
    check_bwd(x, [700], dt, want, 1.0)
    ws = torch.full((1 << 28,), 255, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        got = gdr.head_decay_fwd(*args, s0=x["s0"], workspace=ws)
        assert torch.equal(got[0], o) and torch.equal(got[1], s)
        ws.fill_(255)
        got = gdr.head_decay_bwd(*args, x["d_o"], workspace=ws, **kw)
        for n in want:
            assert torch.equal(got[n], want[n]), n
    lens = [300, 0, 400]
    y = make(26, lens, 2, 1, Dk, Dv, dt, packed=True)
    ws.fill_(255)
    out = gdr.head_decay_bwd_varlen(y["q"], y["k"], y["v"], y["g"], y["d_o"], y["cu"], s0=y["s0"],
                                    ds_final=y["ds_final"], workspace=ws)
    check_bwd(y, lens, dt, out, 1.0, packed=True)


def test_refusals():
    x = make(27, [40], 2, 1, 16, 16, "bf16")
    with pytest.raises(gdr.GdrError, match="ALIGN"):
        buf = torch.zeros(40 * 2 * 16 + 1, dtype=torch.bfloat16, device=DEV)
        gdr.head_decay_fwd(buf[1:].view(1, 40, 2, 16), x["k"], x["v"], x["g"])
    with pytest.raises(ValueError, match="contiguous"):
        gdr.head_decay_bwd(x["q"], x["k"], x["v"], x["g"], torch.ones(1, device=DEV).bfloat16().expand(1, 40, 2, 16))
    with pytest.raises(TypeError):
        gdr.head_decay_fwd(x["q"], x["k"].float(), x["v"], x["g"])
    with pytest.raises(TypeError):
        gdr.head_decay_fwd(x["q"].half(), x["k"].half(), x["v"].half(), x["g"])
    with pytest.raises(ValueError):
        gdr.head_decay_fwd(x["q"], x["k"][:, :39], x["v"], x["g"])
    with pytest.raises(gdr.GdrError, match="ALIAS"):
        gdr.head_decay_fwd(x["q"], x["k"], x["v"], x["g"], o=x["q"])
    with pytest.raises(gdr.GdrError, match="WORKSPACE"):
        y = make(28, [2000], 2, 1, 16, 16, "bf16")
        gdr.head_decay_fwd(y["q"], y["k"], y["v"], y["g"], workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    st = torch.zeros(1, 2, 16, 16, device=DEV)
    one = [x[n][:, 0] for n in "qkv"]
    with pytest.raises(ValueError, match="state_out"):
        gdr.head_decay_step(*one, x["g"], st, parents=torch.zeros(1, dtype=torch.int32, device=DEV))
    with pytest.raises(gdr.GdrError, match="SHAPE"):
        gdr.head_decay_step(*one, x["g"], st.repeat(2, 1, 1, 1))


def test_equal_calls_give_equal_bits():
    x = make(10, [700], 2, 1, 64, 64, "bf16")
    runs = [gdr.head_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], s0=x["s0"]) for _ in range(3)]
    for n in runs[0]:
        assert torch.equal(runs[0][n], runs[1][n]) and torch.equal(runs[0][n], runs[2][n]), n


def test_a_sequence_alone_and_in_a_batch():
    """Heads and sequences do not reach each other: a batch's parts have the bits of the calls on them alone
    (lengths within one segment, so that both are cut alike)."""
    x = make(11, [100, 100], 4, 4, 64, 64, "bf16")
    o, s = gdr.head_decay_fwd(x["q"], x["k"], x["v"], x["g"], s0=x["s0"])
    for b in range(2):
        o1, s1 = gdr.head_decay_fwd(*(x[n][b:b + 1] for n in "qkv"), x["g"], s0=x["s0"][b:b + 1])
        assert torch.equal(o[b:b + 1], o1) and torch.equal(s[b:b + 1], s1)
    bad = {n: x[n].clone() for n in "qkv"}
    for n in "qkv":
        bad[n][1] = float("nan")
    o2, s2 = gdr.head_decay_fwd(bad["q"], bad["k"], bad["v"], x["g"], s0=x["s0"])
    assert torch.equal(o2[0], o[0]) and torch.equal(s2[0], s[0])


# ---- the single token

# N, H, Hk, Dk, Dv
STEPS = [(1, 1, 1, 8, 8), (3, 4, 2, 64, 64), (2, 6, 1, 72, 40), (5, 2, 2, 128, 128), (2, 2, 2, 256, 256), (3, 2, 1, 24, 200)]


def step_case(seed, N, M, H, Hk, Dk, Dv, dt):
    x = make(seed, [N], H, Hk, Dk, Dv, dt, s0=False, packed=True)
    x["state"] = torch.randn(M, H, Dk, Dv, device=DEV, generator=torch.Generator(DEV).manual_seed(seed))
    return x


def check_step(x, dt, o, state_of, new_of, scale):
    """state_of(n): the state that row n continues from (None: padded row); new_of(n): its new state."""
    g, r = host(x["g"]), {"bf16": True, "f32": None}[dt]
    for n in range(x["q"].shape[0]):
        s = state_of(n)
        if s is None:
            assert torch.all(o[n] == 0)
            continue
        tk = {k: host(x[k][n:n + 1]) for k in "qkv"}
        want, S = ref.forward(**tk, g=g, s0=host(s), scale=scale)
        A, SA = ref.forward(**mag(tk), g=g, s0=np.abs(host(s)), scale=scale)
        # one fp32 sum over the channels; no operand below fp32
        err = np.abs(host(o[n]) - want[0])
        assert np.all(err <= 2.0 ** -15 * A[0] + (2.0 ** -8 * np.abs(want[0]) if r else 0)), n
        assert np.all(np.abs(host(new_of(n)) - S[-1]) <= 2.0 ** -21 * SA[-1]), n


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", STEPS, ids=lambda s: "x".join(map(str, s)))
def test_step(shape, dt):
    N, H, Hk, Dk, Dv = shape
    x = step_case(12, N, N, H, Hk, Dk, Dv, dt)
    old = x["state"].clone()
    out = torch.empty_like(old)
    o2 = gdr.head_decay_step(x["q"], x["k"], x["v"], x["g"], x["state"], scale=0.5, state_out=out)
    assert torch.equal(x["state"], old)
    y = fused(x)
    o = gdr.head_decay_step(y["q"], y["k"], y["v"], y["g"], x["state"], scale=0.5)
    check_step(x, dt, o, lambda n: old[n], lambda n: x["state"][n], 0.5)
    assert torch.equal(o, o2) and torch.equal(out, x["state"])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_step_slots(dt):
    """Padded rows, rows in any order, and a slot named twice: the first row has it."""
    x = step_case(13, 8, 6, 4, 2, 40, 64, dt)
    slots = [3, -1, 0, 6, 5, 3, 0, 4]
    has = [True, False, True, False, True, False, False, True]
    old = x["state"].clone()
    o = gdr.head_decay_step(x["q"], x["k"], x["v"], x["g"], x["state"],
                            slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    check_step(x, dt, o, lambda n: old[slots[n]] if has[n] else None, lambda n: x["state"][slots[n]], 1.0)
    for m in (1, 2):
        assert torch.equal(x["state"][m], old[m])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_step_parents(dt):
    """Beams that share a parent, and new rows that start from zero."""
    x = step_case(14, 5, 3, 2, 2, 64, 72, dt)
    parents = [2, 2, -1, 0, 3]
    out = torch.full((5, 2, 64, 72), float("nan"), device=DEV)
    o = gdr.head_decay_step(x["q"], x["k"], x["v"], x["g"], x["state"], state_out=out,
                            parents=torch.tensor(parents, dtype=torch.int32, device=DEV))
    zero = torch.zeros_like(x["state"][0])
    check_step(x, dt, o, lambda n: x["state"][parents[n]] if 0 <= parents[n] < 3 else zero, lambda n: out[n], 1.0)


def test_steps_continue_a_prefill():
    """A prompt's prefill and the tokens behind it one by one are the sequence as a whole."""
    x = make(15, [70, 70], 4, 2, 64, 64, "f32")
    whole, last = gdr.head_decay_fwd(x["q"], x["k"], x["v"], x["g"], s0=x["s0"])
    o, s = gdr.head_decay_fwd(*(x[n][:, :50] for n in "qkv"), x["g"], s0=x["s0"])
    rows = [o] + [gdr.head_decay_step(*(x[n][:, t] for n in "qkv"), x["g"], s)[:, None] for t in range(50, 70)]
    check_fwd(x, [70, 70], "f32", torch.cat(rows, 1), s, 1.0)
    check_fwd(x, [70, 70], "f32", whole, last, 1.0)


# ---- streams and graphs

def test_on_another_stream():
    x = make(16, [500], 4, 2, 64, 128, "bf16")
    want = gdr.head_decay_fwd(x["q"], x["k"], x["v"], x["g"], s0=x["s0"])
    wb = gdr.head_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], s0=x["s0"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gdr.head_decay_fwd(x["q"], x["k"], x["v"], x["g"], s0=x["s0"], stream=side)
    gb = gdr.head_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], s0=x["s0"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for n in wb:
        assert torch.equal(gb[n], wb[n]), n


def test_graph_replays_like_eager_calls():
    """Prefill, backward and decode steps captured once; the inputs change between the replays, and eager work
    runs between them."""
    static = make(17, [300, 300], 4, 2, 64, 64, "bf16")
    state = torch.empty(2, 4, 64, 64, device=DEV)

    def calls(x, st):
        o, s = gdr.head_decay_fwd(x["q"], x["k"], x["v"], x["g"], s0=x["s0"])
        out = gdr.head_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], s0=x["s0"], ds_final=x["ds_final"])
        st.copy_(s)
        steps = [gdr.head_decay_step(*(x[n][:, t] for n in "qkv"), x["g"], st) for t in range(3)]
        return [o, s, *out.values(), st, *steps]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(static, state)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls(static, state)
    for seed in (18, 19, 20):
        fresh = make(seed, [300, 300], 4, 2, 64, 64, "bf16")
        want = [t.clone() for t in calls(fresh, torch.empty_like(state))]
        for n, t in fresh.items():
            if t is not None:
                static[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(held, want)):
            assert torch.equal(a, b), (seed, i)
