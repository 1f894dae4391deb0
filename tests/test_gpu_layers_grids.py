"""The sequence-layer kernels that larger grids reach: heads in blocks and lists of several vectors, 128 columns of states to a
CTA, sequences in parts.  Each test asserts that its sizes reach them.

Bounds are those of test_gpu_layers.py; those of the weights' gradients are derived below.
"""
import ctypes

import pytest
import torch

import layer_oracle as lo
import newton_evaluation_nonlinear_b200 as pn
import test_gpu_layers as base
from test_gpu_layers import TYPES, half_step, rnd

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------------------------------------------
# rotary positions and norms
# ---------------------------------------------------------------------------------------------------------------------

def turned(x, pos, rot, layout, inverse=False, **how):
    """lo.rotate for many rows, on the GPU: angles below 2^17 times 2^-52 are off by less than 2^-35."""
    f, m = lo.frequencies(rot, **how)
    w = pos.double()[..., None, None] * torch.tensor([float(v) for v in f], dtype=torch.float64, device=pos.device)
    c, s = m * w.cos(), (-m if inverse else m) * w.sin()
    x = x.double()
    if layout == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def within(name, got, want, bound):
    off = (got.double() - want).abs() - bound - 2.0 ** -100
    assert bool((off <= 0).all()), (name, float(off.max()), float((got.double() - want).abs().max()))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H, K, dim, rot, layout, pad", [(17, 12, 128, 128, "half", 0), (12, 5, 128, 64, "interleaved", 0),
                                                         (9, 3, 72, 24, "half", 0), (17, 3, 10, 6, "half", 0),
                                                         (10, 9, 64, 64, "interleaved", 3)])
def test_heads_in_blocks(H, K, dim, rot, layout, pad, dtype):
    """So many vectors that groups take blocks of heads (two and more from 2 x 148 x 4 CTAs' worth of groups on, eight from four
    times that; head counts that blocks of 8 do not divide) and lists of several tokens, forward and backward.

    A weight's gradient is a sum of float32 terms, each 2^-21 off, added up one after the other by a group (rows x heads over
    at least 32 groups of a CTA's share of 296), then a CTA's groups (256 at most), then CTAs in eights (37, and 8): fewer
    than 2^9 additions for these sizes, each off by 2^-24 of the sum of the terms' magnitudes at most: 2^-15 of it."""
    T = 18500 * 16 // (H + K) + 1   # 296000 vectors
    assert T * (H + K) >= 8 * 148 * 4 * 32
    big = torch.zeros(2, T // 2, H + K, dim + pad, dtype=dtype, device="cuda")
    x = big[..., :dim]
    gen = torch.Generator(device="cuda").manual_seed(7)
    x.copy_(torch.randn(x.shape, device="cuda", generator=gen))
    tx = torch.randn(x.shape, device="cuda", generator=gen).to(dtype)
    q, k, tq, tk = x[:, :, :H], x[:, :, H:], tx[:, :, :H], tx[:, :, H:]
    pos = torch.arange(T // 2, device="cuda")[None] + torch.tensor([[0], [70000]], device="cuda")
    wq, wk = rnd(5, dim).cuda(), rnd(6, dim).cuda()
    r = pn.Rotary(rot, layout=layout)
    u = half_step(dtype)
    for inverse, call in ((False, r.apply), (True, r.apply_backward)):
        for name, y, got in zip("qk", (q, k), call(q, k, pos)):
            want = turned(y, pos, rot, layout, inverse)
            within(name, got, want, u * want.abs() + 2.0 ** -20 * want.abs().amax(-1, keepdim=True))
    for name, y, w, got in zip("qk", (q, k), (wq, wk), r.norm_apply(q, k, pos, wq, wk, 1e-5)):
        want = turned(lo.norm(y, w, 1e-5), pos, rot, layout)
        within(name, got, want, u * want.abs() + 2.0 ** -20 * want.abs().amax(-1, keepdim=True))
    got = r.norm_backward(tq, tk, q, k, pos, wq, wk, 1e-5)
    for a, b in zip(got, r.norm_backward(tq, tk, q, k, pos, wq, wk, 1e-5)):
        assert torch.equal(a, b)
    for name, y, t, w, dx, dw in (("q", q, tq, wq, got[0], got[2]), ("k", k, tk, wk, got[1], got[3])):
        t = turned(t, pos, rot, layout, True)
        want, want_w = lo.norm_gradient(t, y, w, 1e-5)
        rms = torch.sqrt((y.double() ** 2).mean(-1, keepdim=True) + 1e-5)
        size = ((t * w.double()).abs() / rms).amax(-1, keepdim=True)
        within("d" + name, dx, want, u * want.abs() + 2.0 ** -19 * size)
        within("dw" + name, dw, want_w, 2.0 ** -15 * (t * y.double() / rms).abs().reshape(-1, dim).sum(0))


# ---------------------------------------------------------------------------------------------------------------------
# linear attention
# ---------------------------------------------------------------------------------------------------------------------

def split(dk, dv, H, K, pass_, lens):
    """(columns, parts) of a pass over ragged bfloat16 sequences."""
    att = pn.LinearAttention(H, K, dk, dv, [0.0] * H, dtype=torch.bfloat16)
    c, p = ctypes.c_int(), ctypes.c_int()
    assert pn.lib.pn_linattn_split(att.h, pass_, len(lens), sum(lens), 1, max(lens), ctypes.byref(c), ctypes.byref(p)) == pn.PN_OK
    return c.value, p.value


@pytest.mark.parametrize("K", [6, 2])
@pytest.mark.parametrize("dk, dv", [(128, 128), (64, 128), (128, 72), (96, 160), (72, 96)])
def test_linear_many_ctas(dk, dv, K):
    """So many sequences and heads that CTAs take 128 columns, with decays on both sides of what one accumulator holds (from
    none at all to one that forgets at once), short sequences and rows of no sequence; gradients of shared heads go out in
    float32."""
    H, lens = 6, [0, 1, 63, 65, 130] * 3
    assert split(dk, dv, H, K, 0, lens) == (128, 1)
    assert split(dk, dv, H, K, 1, lens)[0] == (0 if dv > 128 else 64 if dk <= 64 else 128)
    base.run_linear(lens, H, K, dk, dv, torch.bfloat16, lead=3, tail=70)


@pytest.mark.parametrize("states", [True, False])
def test_linear_many_ctas_long(states):
    """The same over several chunks each, more than there are stages, equal lengths."""
    base.run_linear([333] * 13, 6, 2, 128, 128, torch.bfloat16, ragged=False, states=states)


@pytest.mark.parametrize("dk, dv, n", [(128, 128, 20), (64, 64, 3), (64, 128, 20), (128, 64, 20)])
def test_linear_outputs_that_tma_cannot_store(dk, dv, n):
    """Outputs at odd strides and offsets, of whole and short chunks: the bits of contiguous ones, and nothing beside them."""
    H, K, T = 4, 2, 150
    att = pn.LinearAttention(H, K, dk, dv, base.decays(H + 1)[1:], dtype=torch.bfloat16)
    q, k, v, do = (rnd(i, n, T, h, w, dtype=torch.bfloat16).cuda() for i, h, w in ((1, H, dk), (2, K, dk), (3, K, dv), (4, H, dv)))
    s0, ds = rnd(5, n, H, dk, dv).cuda(), rnd(6, n, H, dk, dv).cuda()
    want, S = att.forward(q, k, v, initial_state=s0)
    grads = att.backward(do, q, k, v, initial_state=s0, dstate=ds)
    full = pn.LinearAttention(H, H, dk, dv, base.decays(H + 1)[1:], dtype=torch.bfloat16)   # gradients without a sum over heads
    kf, vf = k.repeat_interleave(2, 2), v.repeat_interleave(2, 2)
    grads_full = full.backward(do, q, kf, vf, initial_state=s0, dstate=ds)

    def outside(x, step, off):
        """Memory for x with rows `step` elements further apart, `off` elements behind an aligned address."""
        b, t, h, d = x.shape
        mem = torch.full((b * t * h * (d + step) + off,), 7.0, dtype=x.dtype, device="cuda")
        return mem, mem[off:].view(b, t, h, d + step)[..., :d]

    for step, off in ((8, 0), (8, 4), (4, 0), (1, 1)):   # 16, 8, 8 and 2 byte alignment
        mem, out = outside(want, step, off)
        o, S2 = att.forward(q, k, v, initial_state=s0, out=out)
        assert torch.equal(o, want) and torch.equal(S2, S)
        assert int((mem != 7).sum()) <= o.numel() and bool((mem[off:].view(*o.shape[:3], -1)[..., dv:] == 7).all())
        for handle, args, right in ((att, (do, q, k, v), grads), (full, (do, q, kf, vf), grads_full)):
            mems, outs = zip(*[outside(x, step, off) for x in right[:3]])
            got = handle.backward(*args, initial_state=s0, dstate=ds, grads=outs)
            for x, y, mem in zip(got, right, (*mems, None)):
                assert torch.equal(x, y)
                if mem is not None:
                    assert bool((mem[off:].view(*x.shape[:3], -1)[..., x.shape[-1]:] == 7).all())


@pytest.mark.parametrize("g", [[-0.01, -0.8], [-1e-3, -3.0], [0.0, -0.05]])
@pytest.mark.parametrize("K", [1, 2])
@pytest.mark.parametrize("dk, dv", [(64, 64), (128, 128), (128, 64), (64, 96)])
def test_linear_ragged_parts(dk, dv, K, g, monkeypatch):
    """Ragged sequences in parts, some shorter than a part or empty; against time the first part begins with a short chunk.
    Decays on both sides of what one accumulator holds."""
    monkeypatch.setattr(base, "decays", lambda H: torch.tensor(g))
    lens = [1100, 0, 20, 513]
    for p in range(4):
        columns, parts = split(dk, dv, 2, K, p, lens)
        assert columns == 64 and parts > 1
    base.run_linear(lens, 2, K, dk, dv, torch.bfloat16, lead=2, tail=5)


@pytest.mark.parametrize("n, H, T, d", [(1, 4, 640, 128), (1, 4, 640, 64), (40, 4, 200, 128)])
def test_linear_bfloat16_rounds_what_it_says(n, H, T, d):
    """Outputs of the tcgen05 kernel are those of 64-bit chunks in which two things are rounded to bfloat16, once each: the
    weights between rows and the state before the chunk, both times the powers of the decay that one accumulator for both
    wants.  What is left are values that float32 and 64 bits round to neighbours: with products and sums up to 2^-17 off and
    steps of 2^-8 that is one value in 2^8 or fewer, each 2^-7.5 off: 2^-11.5 in the mean square, where a third rounding to
    bfloat16 would add 2^-9.2 (a half step of 2^-8, uniform, over a uniform mantissa)."""
    g = torch.tensor([0.0, -1e-3, -0.05, -0.8])[:H]
    q, k, v = (rnd(i, n, T, H, d, dtype=torch.bfloat16) for i in (1, 2, 3))
    att = pn.LinearAttention(H, H, d, d, g, dtype=torch.bfloat16)
    c = ctypes.c_int()
    assert pn.lib.pn_linattn_split(att.h, 0, n, T, 0, 0, ctypes.byref(c), ctypes.byref(ctypes.c_int())) == pn.PN_OK and c.value > 0
    o, _ = att.forward(q.cuda(), k.cuda(), v.cuda())
    C, i = 64, torch.arange(64).double()
    G = g.double()[:, None]
    pad = (-T) % C
    a, b, c = (torch.nn.functional.pad(x[:2].double(), (0, 0, 0, 0, 0, pad)).permute(0, 2, 1, 3) for x in (q, k, v))   # two will do
    once = lambda x: x.bfloat16().double()  # noqa: E731
    S, parts = torch.zeros(min(n, 2), H, d, d, dtype=torch.float64), []
    for r in range(0, T, C):
        x, y, z = (t[:, :, r:r + C] for t in (a, b, c))
        P = (x @ y.transpose(-1, -2)).tril() * torch.exp(G * (32 - (i + 1)))[:, None, :]
        o2 = x @ once(S * torch.exp(G * 32)[:, :, None]) + once(P) @ z
        parts.append(d ** -0.5 * torch.exp(G * (i + 1 - 32))[..., None] * o2)
        S = S * torch.exp(G * 64)[:, :, None] + (y * torch.exp(G * (63 - i))[..., None]).transpose(-1, -2) @ z
    want = torch.cat(parts, 2)[:, :, :T].permute(0, 2, 1, 3)
    got = o[:2].double().cpu()
    off = float((got - once(want)).norm() / want.norm())
    assert off < 2.0 ** -11, off
