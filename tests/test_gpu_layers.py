"""Rotary positions, norms of queries and keys, and linear attention on the GPU against plain 64-bit implementations.

Tolerances, from the arithmetic.  u is half a step of the output's type (finfo.eps / 2): one rounding at the end.
- Rotations and norms: for float32 sine and cosine carry at most 2^-22 (the angle's conversion to float, half a step of half
  a turn, times pi, and sincospif's own error) and each output adds about 8 roundings of float32; for the 16-bit types they
  carry 2^-21.4 and the angle 2^-22.4, together 2^-20.8, and an output takes two of them, sqrt 2 of its pair's size at most:
  2^-20.3, with four roundings of float32 below 2^-20.  So 2^-20 of the vector's largest value, plus u of the value.
- Norm gradients of a weight: sums over n rows of terms of one size, in float32: 2^-24 log2(n) + the terms' own 2^-21
  relative errors, of the sum of the terms' magnitudes: 2^-19 of it.
- Linear attention: A is the output's formula with every factor replaced by its magnitude.  Products, sums and powers of
  the decay in float32 are off by less than 2^-17 A for the lengths here (the powers by up to 20 steps, sums of at most
  2^9 terms).  Powers below float32's smallest normal number, 2^-126, are lost: 2^-100 for products with factors up to
  2^26.  Where a 16-bit type's matrix products take the weights between rows and the entering state rounded to that
  type (u each, on disjoint shares of A), u A is added.  States are float32 throughout: 2^-17 A.
"""
import pytest
import torch

import layer_oracle as lo
import newton_evaluation_nonlinear_b200 as pn

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def rnd(seed, *shape, dtype=torch.float32, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=gen)).to(dtype)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def check(name, got, want, bound):
    """|got - want| <= bound element by element (a tensor or a number), with no NaN."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape, name
    off = (got - want).abs() - bound - 2.0 ** -100   # what underflows, see above
    assert bool((off <= 0).all()), (name, float(off.max()), float((got - want).abs().max()))


def close_heads(name, got, want, dtype):
    """The bound of rotations and norms: u of the value and 2^-20 of the vector's largest."""
    check(name, got, want, half_step(dtype) * want.abs() + 2.0 ** -20 * want.abs().amax(-1, keepdim=True))


# ---------------------------------------------------------------------------------------------------------------------
# rotary positions and norms
# ---------------------------------------------------------------------------------------------------------------------

HEAD_CASES = [
    # B, T, Hq, Hk, dim, rot, layout, how
    (1, 1, 1, 1, 64, 64, "half", {}),
    (2, 3, 4, 2, 128, 128, "half", {}),
    (1, 5, 3, 1, 128, 64, "interleaved", dict(scaling="yarn", factor=16.0)),
    (3, 2, 2, 2, 80, 40, "half", dict(scaling="linear", factor=4.0)),
    (1, 7, 5, 5, 96, 32, "half", dict(scaling="ntk", factor=8.0)),
    (2, 2, 1, 3, 256, 256, "interleaved", {}),
    (1, 3, 2, 1, 256, 256, "half", {}),
    (1, 3, 2, 1, 2, 2, "half", {}),
    (1, 4, 2, 2, 10, 6, "interleaved", {}),
    (2, 3, 2, 2, 72, 24, "half", dict(scaling="yarn", factor=2.0)),
    (1, 2, 17, 1, 40, 12, "half", {}),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", HEAD_CASES)
def test_rotary(case, dtype):
    B, T, Hq, Hk, d, rot, layout, how = case
    q, k = rnd(1, B, T, Hq, d, dtype=dtype), rnd(2, B, T, Hk, d, dtype=dtype)
    pos = torch.arange(T)[None] + torch.tensor([0, 123456, -77][:B])[:, None]
    r = pn.Rotary(rot, layout=layout, **how)
    for inverse, call in ((False, r.apply), (True, r.apply_backward)):
        gq, gk = call(q.cuda(), k.cuda(), pos.cuda())
        close_heads("q", gq, lo.rotate(q, pos, rot, layout, inverse, **how), dtype)
        close_heads("k", gk, lo.rotate(k, pos, rot, layout, inverse, **how), dtype)


def test_rotary_far_positions():
    """Positions beyond what float32 or even a 64-bit float angle resolves.  A frequency is 2^-64 turns fixed point, rounded
    by half a step, 2 pi 2^-65 < 2^-62 radians, from an 80-bit power that is off by a few 2^-64 of at most one radian: the
    angle is off by at most |p| 2^-61, and so is each output, times its pair's size (sqrt 2 of the vector's largest)."""
    pos = torch.tensor([2 ** 24 + 1, 2 ** 31 + 7, 2 ** 40 + 12345, 2 ** 44 + 3, -(2 ** 40) - 9])
    q = rnd(3, 5, 2, 64)
    gq, gk = pn.Rotary(64).apply(q.cuda(), q[:, :1].cuda(), pos.cuda())
    want = lo.rotate(q, pos, 64)
    size = want.abs().amax(-1, keepdim=True)
    far = pos.double().abs()[:, None, None] * 2.0 ** -61 * 2 ** 0.5
    check("q", gq, want, 2.0 ** -24 * want.abs() + (2.0 ** -20 + far) * size)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", HEAD_CASES)
def test_norm_rotary(case, dtype):
    B, T, Hq, Hk, d, rot, layout, how = case
    q, k = rnd(1, B, T, Hq, d, dtype=dtype), rnd(2, B, T, Hk, d, dtype=dtype)
    q[0, 0, 0] = 0   # a vector of zeros: its norm is that of eps
    wt = torch.float32 if T % 2 else dtype
    wq, wk = rnd(5, d, dtype=wt), rnd(6, d, dtype=wt)
    pos = torch.arange(T)[None] + torch.tensor([0, 9999, -77][:B])[:, None]
    r = pn.Rotary(rot, layout=layout, **how)
    gq, gk = r.norm_apply(q.cuda(), k.cuda(), pos.cuda(), wq.cuda(), wk.cuda(), 1e-5)
    close_heads("q", gq, lo.rotate(lo.norm(q, wq, 1e-5), pos, rot, layout, **how), dtype)
    close_heads("k", gk, lo.rotate(lo.norm(k, wk, 1e-5), pos, rot, layout, **how), dtype)

    tq, tk = rnd(7, B, T, Hq, d, dtype=dtype), rnd(8, B, T, Hk, d, dtype=dtype)
    args = [x.cuda() for x in (tq, tk, q, k, pos, wq, wk)]
    got = r.norm_backward(*args, 1e-5)
    again = r.norm_backward(*args, 1e-5)
    for a, b in zip(got, again):
        assert torch.equal(a, b)
    for name, x, t, w, dx, dw in (("q", q, tq, wq, got[0], got[2]), ("k", k, tk, wk, got[1], got[3])):
        t = lo.rotate(t, pos, rot, layout, True, **how)
        want, want_w = lo.norm_gradient(t, x, w, 1e-5)
        # dx subtracts a mean from u = t w: its errors are those of r |u|
        rms = torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + 1e-5)
        size = ((t * w.double()).abs() / rms).amax(-1, keepdim=True)
        check("d" + name, dx, want, half_step(dtype) * want.abs() + 2.0 ** -19 * size)
        terms = (t * x.double() / rms).abs().reshape(-1, d).sum(0)
        check("dw" + name, dw, want_w, 2.0 ** -19 * terms + 1e-30)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_heads_strides(dtype):
    """Slices of one projection, transposed heads, rows at odd offsets; outputs strided too, and in place."""
    B, T, H, K, d = 2, 3, 4, 2, 64
    r = pn.Rotary(d)
    pos = torch.arange(B * T).reshape(B, T)
    w = rnd(4, d)
    qkv = rnd(1, B, T, H + 2 * K, d, dtype=dtype)
    want_q = lo.rotate(lo.norm(qkv[:, :, :H], w, 1e-6), pos, d)
    want_k = lo.rotate(lo.norm(qkv[:, :, H:H + K], w, 1e-6), pos, d)
    base = torch.zeros(B * T * (H + 2 * K) * (d + 3) + 1, dtype=dtype, device="cuda")
    odd = base[1:].view(B, T, H + 2 * K, d + 3)[..., :d]   # unaligned rows
    odd.copy_(qkv)
    moved = qkv.cuda().transpose(1, 2).contiguous().transpose(1, 2)   # heads outside tokens
    for x in (qkv.cuda(), odd, moved):
        q, k, rest = x[:, :, :H], x[:, :, H:H + K], x[:, :, H + K:].clone()
        gq, gk = r.norm_apply(q, k, pos.cuda(), w.cuda(), w.cuda())
        close_heads("q", gq, want_q, dtype)
        close_heads("k", gk, want_k, dtype)
        r.norm_apply(q, k, pos.cuda(), w.cuda(), w.cuda(), out=(q, k))   # in place
        close_heads("q in place", q, want_q, dtype)
        close_heads("k in place", k, want_k, dtype)
        assert torch.equal(x[:, :, H + K:], rest)
    assert float(base[0]) == 0


def test_norm_without_rotation():
    """The C entry takes no plan: the norm alone."""
    import ctypes
    q, k, w = rnd(1, 6, 2, 64).cuda(), rnd(2, 6, 1, 64).cuda(), rnd(3, 64).cuda()
    oq, ok = torch.empty_like(q), torch.empty_like(k)
    hs = [pn.pn_heads(t.data_ptr(), 0, t.stride(0), t.stride(1)) for t in (q, k, oq, ok)]
    st = pn.lib.pn_norm_rotary_apply(None, pn.PN_F32, 1, 6, 2, 1, 64, hs[0], hs[1], None, w.data_ptr(), w.data_ptr(), pn.PN_F32,
                                     ctypes.c_float(1e-6), hs[2], hs[3], torch.cuda.current_stream().cuda_stream)
    assert st == pn.PN_OK, pn.pn_last_error(None)
    close_heads("q", oq, lo.norm(q.cpu(), w.cpu(), 1e-6), torch.float32)
    close_heads("k", ok, lo.norm(k.cpu(), w.cpu(), 1e-6), torch.float32)


def test_heads_many_rows():
    """Enough rows that groups take several heads and several tokens; an empty batch gives zero weight gradients."""
    B, T, H, K, d = 2, 1500, 12, 3, 64
    q, k = rnd(1, B, T, H, d, dtype=torch.bfloat16).cuda(), rnd(2, B, T, K, d, dtype=torch.bfloat16).cuda()
    w = torch.ones(d, device="cuda")
    pos = torch.arange(B * T, device="cuda").reshape(B, T)
    r = pn.Rotary(d)
    gq, gk = r.norm_apply(q, k, pos, w, w)
    for at in ((0, 0), (0, T - 1), (1, 777), (1, T - 1)):   # each row alone gives the same bits
        sq, sk = r.norm_apply(q[at][None], k[at][None], pos[at][None], w, w)
        assert torch.equal(gq[at], sq[0]) and torch.equal(gk[at], sk[0])
    dq, dk, dwq, dwk = r.norm_backward(gq[:, :0], gk[:, :0], q[:, :0], k[:, :0], pos[:, :0].contiguous(), w, w)
    assert dq.shape == (B, 0, H, d) and float(dwq.abs().sum()) == 0 and float(dwk.abs().sum()) == 0


def test_heads_refusals():
    r = pn.Rotary(64)
    q, k = torch.zeros(2, 3, 4, 64, device="cuda"), torch.zeros(2, 3, 2, 64, device="cuda")
    pos = torch.zeros(2, 3, dtype=torch.int64, device="cuda")
    w = torch.ones(64, device="cuda")
    for args in [(q.double(), k.double(), pos), (q, k.half(), pos), (q, k[..., :32], pos), (q, k[:1], pos),
                 (q, k, pos.int()), (q, k, pos[:, :2]), (q, k, pos.cpu()), (q[..., ::2], k[..., ::2], pos),
                 (q[0, 0], k[0, 0], pos)]:
        with pytest.raises(ValueError):
            r.apply(*args)
    with pytest.raises(ValueError):
        r.apply(q, k, pos, out=(q[:, :, :1].expand_as(q), k))
    with pytest.raises(pn.PnError):
        pn.Rotary(128).apply(q, k, pos)
    for a, b in [(w[:32], w), (w, w.half()), (w.cpu(), w), (w.bfloat16(), w.bfloat16())]:
        with pytest.raises((ValueError, pn.PnError)):
            r.norm_apply(q, k, pos, a, b)


# ---------------------------------------------------------------------------------------------------------------------
# linear attention
# ---------------------------------------------------------------------------------------------------------------------

def decays(H):
    """From none at all to one that forgets at once."""
    g = torch.tensor([0.0, -1e-3, -0.05, -0.7, -3.0, -200.0])
    return g[torch.arange(H) % 6]


def mixed(dtype):
    """u of the operand roundings of the 16-bit types' matrix products."""
    return 0.0 if dtype == torch.float32 else half_step(dtype)


def run_linear(lens, H, K, dk, dv, dtype, seed=0, ragged=True, lead=0, tail=0, states=True):
    """Forward and backward of packed (or equal) sequences against the oracle; returns the GPU tensors."""
    n, total = len(lens), sum(lens)
    g = decays(H)
    scale = dk ** -0.5
    rows = lead + total + tail
    q, k, v = rnd(seed + 1, rows, H, dk, dtype=dtype), rnd(seed + 2, rows, K, dk, dtype=dtype), rnd(seed + 3, rows, K, dv, dtype=dtype)
    do = rnd(seed + 4, rows, H, dv, dtype=dtype)
    s0 = rnd(seed + 5, n, H, dk, dv) if states else None
    ds = rnd(seed + 6, n, H, dk, dv) if states else None
    if lead + tail:   # rows of no sequence hold anything
        for x in (q, k, v, do):
            x[:lead] = float("nan")
            x[lead + total:] = float("inf")
    att = pn.LinearAttention(H, K, dk, dv, g, dtype=dtype)
    cu = torch.tensor([lead + sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32)
    dev = [x.cuda() for x in (q, k, v)]
    shape = lambda x: x if ragged else x.view(n, lens[0], *x.shape[1:])  # noqa: E731
    how = dict(initial_state=None if s0 is None else s0.cuda())
    if ragged:
        how.update(cu_seqlens=cu.cuda(), max_len=max(lens))
    out = torch.full((rows, H, dv), 7.0, dtype=dtype, device="cuda")
    o, S = att.forward(*map(shape, dev), out=shape(out), **how)
    grads = tuple(torch.full_like(x, 7.0) for x in dev)
    dq, dk_, dv_, ds0 = att.backward(shape(do.cuda()), *map(shape, dev), dstate=None if ds is None else ds.cuda(),
                                     grads=tuple(map(shape, grads)), **how)
    got = [out, *grads]
    for x in got:   # rows of no sequence are left as they were
        assert bool((x[:lead] == 7).all()) and bool((x[lead + total:] == 7).all())
    c, u = 2.0 ** -17, half_step(dtype)
    m = mixed(dtype)
    for i, length in enumerate(lens):
        r = slice(lead + sum(lens[:i]), lead + sum(lens[:i]) + length)
        a = [x[r] for x in (q, k, v)]
        b = [x.double().abs() for x in a]
        e = None if s0 is None else s0[i]
        f = None if ds is None else ds[i]
        ea, fa = (None if x is None else x.abs() for x in (e, f))
        wo, wS = lo.linear(*a, g, scale, e)
        Ao, AS = lo.linear(*b, g, scale, ea)
        check(f"o[{i}]", out[r], wo, u * wo.abs() + (m + c) * Ao)
        check(f"S[{i}]", S[i], wS, c * AS)
        want = lo.linear_gradient(do[r], *a, g, scale, e, f)
        A = lo.linear_gradient(do[r].double().abs(), *b, g, scale, ea, fa)
        for name, x, w, y in zip(("dq", "dk", "dv"), grads, want, A):
            check(f"{name}[{i}]", x[r], w, u * w.abs() + (m + c) * y)
        check(f"ds0[{i}]", ds0[i], want[3], c * A[3])
    return att, dev, do, s0, cu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("length", [1, 2, 31, 63, 64, 65, 127, 128, 129, 200])
def test_linear_lengths(length, dtype):
    run_linear([length], 6, 6, 64, 64, dtype, ragged=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk, dv", [(8, 8), (32, 64), (64, 96), (80, 80), (96, 32), (128, 128), (128, 160), (64, 256),
                                    (256, 64), (136, 128), (200, 24)])
def test_linear_widths(dk, dv, dtype):
    run_linear([70, 130], 2, 1, dk, dv, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H, K", [(1, 1), (4, 2), (6, 1), (12, 4)])
def test_linear_shared_heads(H, K, dtype):
    run_linear([67, 67], H, K, 32, 64, dtype, ragged=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens, lead, tail", [([0], 0, 3), ([0, 5, 0, 130, 64, 1, 0], 3, 9), ([300, 1], 0, 0), ([1] * 9, 2, 200),
                                              ([128, 128], 0, 1)])
def test_linear_ragged(lens, lead, tail, dtype):
    run_linear(lens, 3, 3, 64, 64, dtype, lead=lead, tail=tail)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens", [[1100], [700, 20, 513]])
@pytest.mark.parametrize("dk, dv", [(64, 64), (128, 128), (136, 40)])
def test_linear_parts(lens, dk, dv, dtype):
    """Few heads and long sequences: the work is split along the sequence."""
    run_linear(lens, 2, 1, dk, dv, dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_linear_without_states(dtype):
    run_linear([90, 13], 4, 2, 64, 64, dtype, states=False)


def test_linear_large_values():
    """Inputs near the ends of the 16-bit ranges: nothing inside overflows where the outputs do not."""
    for dtype, big in ((torch.float16, 200.0), (torch.bfloat16, 1e15)):
        T, H, d = 150, 2, 64
        g = torch.tensor([0.0, -0.05])
        q, k = rnd(1, T, H, d, dtype=dtype), rnd(2, T, H, d, dtype=dtype)
        v = rnd(3, T, H, d, dtype=dtype)
        q, k = (q.double() / big).to(dtype), (k.double() * big).to(dtype)
        att = pn.LinearAttention(H, H, d, d, g, dtype=dtype)
        o, S = att.forward(q.cuda()[None], k.cuda()[None], v.cuda()[None])
        wo, wS = lo.linear(q, k, v, g, d ** -0.5)
        Ao, AS = lo.linear(q.double().abs(), k.double().abs(), v.double().abs(), g, d ** -0.5)
        # the smallest fp16 steps (2^-25 of rounding) of the outputs and of rounded operands, times the sum's other factor
        tiny = 2.0 ** -25 * (1 + float(v.abs().double().sum())) if dtype == torch.float16 else 0.0
        check("o", o[0], wo, half_step(dtype) * (wo.abs() + Ao) + 2.0 ** -17 * Ao + tiny)
        check("S", S[0], wS, 2.0 ** -17 * AS)


@pytest.mark.parametrize("dtype", TYPES)
def test_linear_strides(dtype):
    """Slices of one projection, heads outside tokens, rows at odd offsets: the same values as packed ones, bit for bit where
    the aligned kernels run and within two bounds of the value elsewhere."""
    B, T, H, K, d = 2, 140, 4, 2, 64
    g = decays(H)
    att = pn.LinearAttention(H, K, d, d, g, dtype=dtype)
    qkv = rnd(1, B, T, H + 2 * K, d, dtype=dtype)
    cut = lambda x: (x[:, :, :H], x[:, :, H:H + K], x[:, :, H + K:])  # noqa: E731
    base = torch.zeros(B * T * (H + 2 * K) * (d + 3) + 1, dtype=dtype, device="cuda")
    odd = base[1:].view(B, T, H + 2 * K, d + 3)[..., :d]
    odd.copy_(qkv)
    moved = qkv.cuda().transpose(1, 2).contiguous().transpose(1, 2)
    for x in (qkv.cuda(), odd, moved):
        q, k, v = cut(x)
        out = torch.zeros(B, H, T, d, dtype=dtype, device="cuda").transpose(1, 2)
        o, S = att.forward(q, k, v, out=out)
        for b in range(B):
            a = [y[b] for y in cut(qkv)]
            wo, wS = lo.linear(*a, g, d ** -0.5)
            Ao, AS = lo.linear(*[y.double().abs() for y in a], g, d ** -0.5)
            check("o", o[b], wo, half_step(dtype) * wo.abs() + (mixed(dtype) + 2.0 ** -17) * Ao)
            check("S", S[b], wS, 2.0 ** -17 * AS)


def test_linear_neighbours_do_not_leak():
    """NaN in one sequence or head stays there."""
    for dtype in TYPES:
        lens, H, d = [70, 90, 50], 2, 64
        cu = torch.tensor([0, 70, 160, 210], dtype=torch.int32).cuda()
        q, k, v = (rnd(i, 210, H, d, dtype=dtype) for i in (1, 2, 3))
        att = pn.LinearAttention(H, H, d, d, decays(H), dtype=dtype)
        clean, S = att.forward(q.cuda(), k.cuda(), v.cuda(), cu_seqlens=cu, max_len=90)
        gc = att.backward(q.cuda(), q.cuda(), k.cuda(), v.cuda(), cu_seqlens=cu, max_len=90)
        for x in (q, k, v):
            x[70:160, 1] = float("nan")
        o, S2 = att.forward(q.cuda(), k.cuda(), v.cuda(), cu_seqlens=cu, max_len=90)
        gn = att.backward(q.cuda(), q.cuda(), k.cuda(), v.cuda(), cu_seqlens=cu, max_len=90)
        keep = torch.ones(210, H, dtype=torch.bool)
        keep[70:160, 1] = False
        for a, b in zip((clean, *gc[:3]), (o, *gn[:3])):
            assert torch.equal(a.cpu()[keep], b.cpu()[keep])
        for i, h in ((0, 0), (0, 1), (1, 0), (2, 0), (2, 1)):
            assert torch.equal(S[i, h], S2[i, h]) and torch.equal(gc[3][i, h], gn[3][i, h])


def test_linear_state_in_place():
    """final_state may be initial_state, and d_initial_state d_final_state, split sequences included (C entries)."""
    for dtype, code in ((torch.float32, pn.PN_F32), (torch.bfloat16, pn.PN_BF16)):
        T, H, d = 1200, 2, 64
        q, k, v = (rnd(i, T, H, d, dtype=dtype).cuda() for i in (1, 2, 3))
        s0 = rnd(4, 1, H, d, d).cuda()
        att = pn.LinearAttention(H, H, d, d, decays(H), dtype=dtype)
        o, S = att.forward(q[None], k[None], v[None], initial_state=s0)
        grads = att.backward(q[None], q[None], k[None], v[None], initial_state=s0, dstate=s0)
        hs = lambda t: pn.pn_heads(t.data_ptr(), 0, t.stride(0), t.stride(1))  # noqa: E731
        st = torch.cuda.current_stream().cuda_stream
        n = pn.lib.pn_linattn_workspace(att.h, 1, 1, T, 0, 0)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        s1, o1 = s0.clone(), torch.empty_like(o[0])
        assert pn.lib.pn_linattn_forward(att.h, 1, T, None, 0, hs(q), hs(k), hs(v), s1.data_ptr(), hs(o1), s1.data_ptr(),
                                         ws.data_ptr(), n, st) == pn.PN_OK
        assert torch.equal(s1, S) and torch.equal(o1, o[0])
        d1 = s0.clone()
        outs = [torch.empty_like(x) for x in (q, k, v)]
        assert pn.lib.pn_linattn_backward(att.h, 1, T, None, 0, hs(q), hs(q), hs(k), hs(v), s0.data_ptr(), d1.data_ptr(),
                                          *map(hs, outs), d1.data_ptr(), ws.data_ptr(), n, st) == pn.PN_OK
        assert torch.equal(d1, grads[3])
        for a, b in zip(outs, grads):
            assert torch.equal(a, b[0])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows, H, K, dk, dv", [(1, 1, 1, 8, 8), (3, 4, 2, 64, 64), (2, 2, 2, 128, 160), (5, 6, 3, 80, 40),
                                                (1, 2, 1, 256, 256), (40, 8, 2, 64, 128)])
@pytest.mark.parametrize("rotate", [False, True])
def test_step(rows, H, K, dk, dv, dtype, rotate):
    g = decays(H)
    att = pn.LinearAttention(H, K, dk, dv, g, dtype=dtype)
    q, k, v = rnd(1, rows, H, dk, dtype=dtype), rnd(2, rows, K, dk, dtype=dtype), rnd(3, rows, K, dv, dtype=dtype)
    states = rnd(4, rows + 3, H, dk, dv)
    slots = torch.randperm(rows + 3, generator=torch.Generator().manual_seed(5))[:rows]
    wq, wk = 1 + rnd(6, dk, scale=0.2), 1 + rnd(7, dk, scale=0.2)
    pos = torch.arange(rows) * 1000 - 3
    how, eq, ek = {}, q.double(), k.double()
    if rotate:
        rot = dk // 2
        how = dict(rotary=pn.Rotary(rot, layout="interleaved" if dk == 80 else "half"), positions=pos.cuda(), wq=wq.cuda(),
                   wk=wk.cuda(), eps=1e-5)
        layout = "interleaved" if dk == 80 else "half"
        eq, ek = lo.rotate(lo.norm(q, wq, 1e-5), pos, rot, layout), lo.rotate(lo.norm(k, wk, 1e-5), pos, rot, layout)
    gs = states.cuda()
    o = att.step(q.cuda(), k.cuda(), v.cuda(), gs, slots=slots.cuda(), **how)
    touched = torch.zeros(rows + 3, dtype=torch.bool)
    for b in range(rows):
        s = int(slots[b])
        touched[s] = True
        a = (eq[b][None], ek[b][None], v[b][None])
        wo, wS = lo.linear(*a, g, dk ** -0.5, states[s])
        mag = [x.double().abs() for x in a]
        if rotate:   # an element turned to near zero carries its pair's error
            mag[0], mag[1] = (x + 0.25 * x.amax(-1, keepdim=True) for x in mag[:2])
        Ao, AS = lo.linear(*mag, g, dk ** -0.5, states[s].abs())
        check("o", o[b], wo[0], half_step(dtype) * wo[0].abs() + 2.0 ** -17 * Ao[0])
        check("S", gs[s], wS, 2.0 ** -17 * AS)
    assert torch.equal(gs.cpu()[~touched], states[~touched])


def test_step_padding_and_repeated_slots():
    """Rows outside the states and rows that repeat a slot are left as they are; the first row of a slot counts."""
    H, d = 2, 64
    att = pn.LinearAttention(H, H, d, d, decays(H))
    slots = torch.tensor([2, -1, 0, 2, 9, 0, 1], dtype=torch.int64)
    q, k, v = (rnd(i, 7, H, d).cuda() for i in (1, 2, 3))
    states = rnd(4, 3, H, d, d).cuda()
    one, out = states.clone(), torch.full((7, H, d), 5.0, device="cuda")
    att.step(q, k, v, one, slots=slots.cuda(), out=out)
    live = [0, 2, 6]
    two = states.clone()
    o = att.step(q[live], k[live], v[live], two, slots=slots[live].cuda())
    assert torch.equal(one, two) and torch.equal(out[live], o)
    assert bool((out[[1, 3, 4, 5]] == 5).all())
    before = states.clone()
    att.step(q[:3], k[:3], v[:3], states)   # without slots: row b is state b
    att.step(q[:3], k[:3], v[:3], before, slots=torch.arange(3, device="cuda"))
    assert torch.equal(states, before)
    assert att.step(q[:0], k[:0], v[:0], states).shape == (0, H, d)


@pytest.mark.parametrize("dtype", TYPES)
def test_linear_offsets_are_clamped(dtype):
    """Offsets outside the buffer are cut to it, a decreasing one makes an empty sequence: nothing else is read or written."""
    T, H, d = 200, 2, 64
    att = pn.LinearAttention(H, H, d, d, decays(H), dtype=dtype)
    q, k, v = (rnd(i, T, H, d, dtype=dtype).cuda() for i in (1, 2, 3))
    s0 = rnd(4, 3, H, d, d).cuda()

    def run(cu):
        out = torch.full((T, H, d), 7.0, dtype=dtype, device="cuda")
        o, S = att.forward(q, k, v, initial_state=s0, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), max_len=T, out=out)
        return o, S

    for bad, good in (([-5, 90, 90, 1000000], [0, 90, 90, T]), ([0, 120, 60, 60], [0, 120, 120, 120]),
                      ([150, 2 ** 31 - 1, 40, 40], [150, T, T, T])):
        for a, b in zip(run(bad), run(good)):
            assert torch.equal(a, b), bad
    pn.LinearAttention.check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_linear_many_sequences(dtype):
    """More sequences than are taken by length, most of them of one to three rows."""
    n, H, d = 600, 1, 16
    lens = [(7 * i) % 4 for i in range(n)]
    lens[311] = 140
    att = pn.LinearAttention(H, H, d, d, [-0.05], dtype=dtype)
    T = sum(lens)
    q, k, v = (rnd(i, T, H, d, dtype=dtype) for i in (1, 2, 3))
    s0 = rnd(4, n, H, d, d)
    cu = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32)
    o, S = att.forward(q.cuda(), k.cuda(), v.cuda(), initial_state=s0.cuda(), cu_seqlens=cu.cuda())   # no max_len
    g = torch.tensor([-0.05])
    for i in (0, 1, 2, 3, 310, 311, 312, n - 1):
        r = slice(int(cu[i]), int(cu[i + 1]))
        wo, wS = lo.linear(q[r], k[r], v[r], g, d ** -0.5, s0[i])
        Ao, AS = lo.linear(q[r].double().abs(), k[r].double().abs(), v[r].double().abs(), g, d ** -0.5, s0[i].abs())
        check(f"o[{i}]", o[r], wo, half_step(dtype) * wo.abs() + (mixed(dtype) + 2.0 ** -17) * Ao)
        check(f"S[{i}]", S[i], wS, 2.0 ** -17 * AS)


@pytest.mark.parametrize("dtype", TYPES)
def test_linear_long(dtype):
    """A sequence of many parts.  Its sums have 2^13 terms where nothing is forgotten: 2^-15 A in place of 2^-17 A (errors of
    float32 sums grow with the square root of the terms, 2^2 for 2^4 times as many; the powers' by the exponent's size, which
    the decay keeps within the same 20 steps)."""
    T, H, d = 9001, 2, 32
    g = torch.tensor([0.0, -0.002])
    att = pn.LinearAttention(H, 1, d, d, g, dtype=dtype)
    q, k, v = rnd(1, T, H, d, dtype=dtype), rnd(2, T, 1, d, dtype=dtype), rnd(3, T, 1, d, dtype=dtype)
    do = rnd(4, T, H, d, dtype=dtype)
    o, S = att.forward(q[None].cuda(), k[None].cuda(), v[None].cuda())
    grads = att.backward(do[None].cuda(), q[None].cuda(), k[None].cuda(), v[None].cuda())
    wo, wS = lo.linear(q, k, v, g, d ** -0.5)
    want = lo.linear_gradient(do, q, k, v, g, d ** -0.5)
    mag = [x.double().abs() for x in (q, k, v)]
    Ao, AS = lo.linear(*mag, g, d ** -0.5)
    A = lo.linear_gradient(do.double().abs(), *mag, g, d ** -0.5)
    u, c = half_step(dtype), 2.0 ** -15
    check("o", o[0], wo, u * wo.abs() + (mixed(dtype) + c) * Ao)
    check("S", S[0], wS, c * AS)
    for name, x, w, y in zip(("dq", "dk", "dv"), grads, want, A):
        check(name, x[0], w, u * w.abs() + (mixed(dtype) + c) * y)
    check("ds0", grads[3][0], want[3], c * A[3])


@pytest.mark.parametrize("dtype", TYPES)
def test_linear_strongest_decays(dtype):
    """Decays down to the least float32: nothing is kept, and no exponent becomes a NaN (bounds as in run_linear: every sum
    has one term)."""
    n, T, H, d = 2, 70, 4, 64
    g = torch.tensor([-3.4e38, -1e38, -1e6, -0.5])
    q, k, v, do = (rnd(i, n, T, H, d, dtype=dtype) for i in range(4))
    s0, ds = rnd(5, n, H, d, d), rnd(6, n, H, d, d)
    att = pn.LinearAttention(H, H, d, d, g, dtype=dtype)
    dev = [x.cuda() for x in (q, k, v)]
    o, S = att.forward(*dev, initial_state=s0.cuda())
    grads = att.backward(do.cuda(), *dev, initial_state=s0.cuda(), dstate=ds.cuda())
    states = s0.cuda()
    o1 = att.step(*[x[:, 0] for x in dev], states)
    u, m, c = half_step(dtype), mixed(dtype), 2.0 ** -17
    for i in range(n):
        a, mag = (q[i], k[i], v[i]), [x[i].double().abs() for x in (q, k, v)]
        wo, wS = lo.linear(*a, g, d ** -0.5, s0[i])
        Ao, AS = lo.linear(*mag, g, d ** -0.5, s0[i].abs())
        check("o", o[i], wo, u * wo.abs() + (m + c) * Ao)
        check("S", S[i], wS, c * AS)
        want = lo.linear_gradient(do[i], *a, g, d ** -0.5, s0[i], ds[i])
        A = lo.linear_gradient(do[i].double().abs(), *mag, g, d ** -0.5, s0[i].abs(), ds[i].abs())
        for name, x, w, y in zip(("dq", "dk", "dv"), grads, want, A):
            check(name, x[i], w, u * w.abs() + (m + c) * y)
        check("ds0", grads[3][i], want[3], c * A[3])
        check("step", o1[i], wo[0], u * wo[0].abs() + (m + c) * Ao[0])


@pytest.mark.parametrize("dk, dv", [(64, 96), (128, 64), (40, 24)])
def test_linear_mean_square(dk, dv):
    """How far float32 results are off in the mean square, relative to theirs.  The sums are of terms of either sign, so what
    is lost adds up by squares: over K terms, eights of them truncated at 2^-23 three times (3 2^-23 sqrt(8) sqrt(K / 8)
    against sqrt(K), at 0.6 of the full truncation) give 2^-22.2, K / 8 <= 16 float32 sums 2^-24 sqrt(16 / 2) / sqrt(3) <=
    2^-23.3, left-out products of two low halves 2^-24, the decay's powers at weights that count 2^-23: 2^-21.4 by squares,
    where an accumulator that is truncated 48 times for one sign's worth of its value is off by 2^-20 and more."""
    T, H = 1500, 4
    g = torch.tensor([0.0, -0.004, -0.05, -0.7])
    q, k, v, do = rnd(1, T, H, dk), rnd(2, T, 2, dk), rnd(3, T, 2, dv), rnd(4, T, H, dv)
    att = pn.LinearAttention(H, 2, dk, dv, g, dtype=torch.float32)
    dev = [x[None].cuda() for x in (q, k, v)]
    o, S = att.forward(*dev)
    got = (o[0], S[0], *[x[0] for x in att.backward(do[None].cuda(), *dev)[:3]])
    want = (*lo.linear(q, k, v, g, dk ** -0.5), *lo.linear_gradient(do, q, k, v, g, dk ** -0.5)[:3])
    for name, x, w in zip(("o", "S", "dq", "dk", "dv"), got, want):
        off = ((x.double().cpu() - w).norm() / w.norm()).item()
        assert off < 2.0 ** -21, f"{name}: {off:.3g}"


def test_offsets_beyond_32_bits():
    """Rows whose element offsets, and states whose slots, pass 2^31."""
    far = 1 << 30
    base = torch.empty(3 * far + 1024, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(base, (4, 2, 64), (far - 64, 64, 1))   # token 3 lies at element 3 2^30 - 192
    src = rnd(1, 4, 2, 64, dtype=torch.bfloat16)
    x.copy_(src)
    pos = torch.arange(4, device="cuda")
    near = src.cuda()
    r, att = pn.Rotary(64), pn.LinearAttention(2, 2, 64, 64, [-0.1, 0.0], dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda")
    for a, b in zip(r.norm_apply(x, x, pos, w, w), r.norm_apply(near, near, pos, w, w)):
        assert torch.equal(a, b)
    for a, b in zip(att.forward(x[None], x[None], x[None]), att.forward(near[None], near[None], near[None])):
        assert torch.equal(a, b)
    half = pn.LinearAttention(2, 2, 64, 64, [-0.1, 0.0], dtype=torch.float16)   # the other kernel
    xh, nh = x.view(torch.float16), near.view(torch.float16)
    for a, b in zip(half.forward(xh[None], xh[None], xh[None]), half.forward(nh[None], nh[None], nh[None])):
        assert torch.equal(a.view(torch.int16) if a.dtype == torch.float16 else a.view(torch.int32),
                           b.view(torch.int16) if b.dtype == torch.float16 else b.view(torch.int32))
    del base, x, xh
    one = pn.LinearAttention(1, 1, 256, 256, [-0.1])
    states = torch.zeros(33000, 1, 256, 256, device="cuda")   # 2^31 elements at slot 32768
    q = rnd(2, 1, 1, 256).cuda()
    o = one.step(q, q, q, states, slots=torch.tensor([32999], device="cuda"))
    small = torch.zeros(1, 1, 256, 256, device="cuda")
    assert torch.equal(o, one.step(q, q, q, small)) and torch.equal(states[32999], small[0])
    assert float(states[:32999].abs().amax()) == 0


def test_one_handle_on_two_streams():
    """Handles hold nothing that a call changes: two streams at once give what each gives alone."""
    T, H, d = 2000, 4, 64
    att = pn.LinearAttention(H, 2, d, d, decays(H), dtype=torch.bfloat16)
    r = pn.Rotary(d)
    w, pos = torch.ones(d, device="cuda"), torch.arange(T, device="cuda")
    ins = [(rnd(i, T, H, d, dtype=torch.bfloat16).cuda(), rnd(i + 9, T, 2, d, dtype=torch.bfloat16).cuda()) for i in range(2)]

    def layer(q, k):
        nq, nk = r.norm_apply(q, k, pos, w, w)
        o, S = att.forward(nq[None], nk[None], k[None])
        return (o, S, *att.backward(o, nq[None], nk[None], k[None], dstate=S))

    want = [layer(*x) for x in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = layer(*ins[i])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_linear_refusals():
    att = pn.LinearAttention(4, 2, 64, 32, [-0.1] * 4)
    q, k, v = torch.zeros(2, 5, 4, 64).cuda(), torch.zeros(2, 5, 2, 64).cuda(), torch.zeros(2, 5, 2, 32).cuda()
    cu = torch.tensor([0, 3, 5], dtype=torch.int32).cuda()
    s0 = torch.zeros(2, 4, 64, 32).cuda()
    bad = [dict(q=q.half(), k=k.half(), v=v.half()), dict(k=k[:, :4]), dict(v=v[..., :16]), dict(q=q[:, :, :2]), dict(k=k.half()),
           dict(initial_state=s0[:1]), dict(initial_state=s0.half()), dict(cu_seqlens=cu), dict(out=torch.zeros_like(v)),
           dict(q=q.cpu(), k=k.cpu(), v=v.cpu()), dict(out=torch.zeros(1, 1, 1, 32).cuda().expand(2, 5, 4, 32))]
    for kw in bad:
        with pytest.raises(ValueError):
            att.forward(**{**dict(q=q, k=k, v=v), **kw})
    for c in (cu.long(), cu.cpu(), cu[:0], cu[None]):
        with pytest.raises(ValueError):
            att.forward(q[0], k[0], v[0], cu_seqlens=c)
    with pytest.raises(ValueError):
        att.backward(torch.zeros(2, 5, 4, 64).cuda(), q, k, v)
    with pytest.raises(ValueError):
        att.backward(torch.zeros(2, 5, 4, 32).cuda(), q, k, v, grads=(k, k, v))
    states = torch.zeros(3, 4, 64, 32).cuda()
    for kw in [dict(states=states.half()), dict(states=states[..., :16]), dict(slots=torch.zeros(5, dtype=torch.int32).cuda()),
               dict(slots=torch.zeros(4, dtype=torch.int64).cuda()), dict(wq=torch.ones(64).cuda()),
               dict(rotary=pn.Rotary(64)), dict(out=torch.zeros(5, 4, 64).cuda())]:
        with pytest.raises(ValueError):
            att.step(q[0], k[0], v[0], **{**dict(states=states, slots=torch.zeros(5, dtype=torch.int64).cuda()), **kw})
    with pytest.raises(pn.PnError, match="n_slots"):
        att.step(q[0], k[0], v[0], states)
    with pytest.raises(pn.PnError, match="rot_dim"):
        att.step(q[0][:3], k[0][:3], v[0][:3], states, rotary=pn.Rotary(128), positions=torch.zeros(3, dtype=torch.int64).cuda())


def test_workspace_too_small_is_refused():
    att = pn.LinearAttention(2, 1, 64, 64, [-0.1] * 2)
    T = 5000
    q, k, o = (torch.zeros(T, h, 64, device="cuda") for h in (2, 1, 2))
    hs = lambda t: pn.pn_heads(t.data_ptr(), 0, t.stride(0), t.stride(1))  # noqa: E731
    n = pn.lib.pn_linattn_workspace(att.h, 0, 1, T, 0, 0)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    assert n > 0
    assert pn.lib.pn_linattn_forward(att.h, 1, T, None, 0, hs(q), hs(k), hs(k), None, hs(o), None, ws.data_ptr(), n - 1,
                                     None) == pn.PN_ERR_INVALID
    assert "workspace" in pn.pn_last_error(None)


# ---------------------------------------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES)
def test_layer_prompt_then_tokens(dtype):
    """As a model runs them: norm and rotation, a prompt, then tokens one by one from its state, against the oracle over the
    whole sequence."""
    T, more, H, K, d = 97, 4, 4, 2, 64
    g = decays(H)[[1, 2, 0, 3]]
    wq, wk = 1 + rnd(6, d, scale=0.2), 1 + rnd(7, d, scale=0.2)
    q, k, v = rnd(1, T + more, H, d, dtype=dtype), rnd(2, T + more, K, d, dtype=dtype), rnd(3, T + more, K, d, dtype=dtype)
    pos = torch.arange(T + more) + 500
    r = pn.Rotary(d, scaling="yarn", factor=4.0)
    att = pn.LinearAttention(H, K, d, d, g, dtype=dtype)
    nq, nk = r.norm_apply(q[:T].cuda(), k[:T].cuda(), pos[:T].cuda(), wq.cuda(), wk.cuda())
    o, state = att.forward(nq[None], nk[None], v[None, :T].cuda())
    rows = [o[0]]
    pool = torch.zeros(3, H, d, d, device="cuda")
    pool[1] = state[0]
    slot = torch.tensor([1], device="cuda")
    for t in range(T, T + more):
        rows.append(att.step(q[t:t + 1].cuda(), k[t:t + 1].cuda(), v[t:t + 1].cuda(), pool, slots=slot, rotary=r,
                             positions=pos[t:t + 1].cuda(), wq=wq.cuda(), wk=wk.cuda()))
    eq = lo.rotate(lo.norm(q, wq, 1e-6), pos, d, scaling="yarn", factor=4.0)
    ek = lo.rotate(lo.norm(k, wk, 1e-6), pos, d, scaling="yarn", factor=4.0)
    wo, wS = lo.linear(eq, ek, v, g, d ** -0.5)
    Ao, AS = lo.linear(eq.abs() + 0.25, ek.abs() + 0.25, v.double().abs(), g, d ** -0.5)
    u = half_step(dtype)   # the norm's output is rounded before the prompt reads it: u on q and on k
    check("o", torch.cat(rows), wo, u * wo.abs() + (2 * u + mixed(dtype) + 2.0 ** -16) * Ao)
    check("S", pool[1], wS, (u + 2.0 ** -16) * AS)
    assert float(pool[0].abs().sum()) == 0 and float(pool[2].abs().sum()) == 0


def test_layer_gradients_chain():
    """Gradients through norm, rotation and attention together, float32, against autograd in 64 bits of the oracle's formulas."""
    T, H, K, d = 70, 4, 2, 32
    g = decays(H)[[1, 2, 0, 3]]
    x = [rnd(1, T, H, d), rnd(2, T, K, d), rnd(3, T, K, d), 1 + rnd(6, d, scale=0.2), 1 + rnd(7, d, scale=0.2)]
    do, pos = rnd(4, T, H, d), torch.arange(T)
    r = pn.Rotary(d)
    att = pn.LinearAttention(H, K, d, d, g)
    q, k, v, wq, wk = [t.cuda() for t in x]
    nq, nk = r.norm_apply(q, k, pos.cuda(), wq, wk)
    dnq, dnk, dv, _ = att.backward(do.cuda(), nq, nk, v)
    dq, dk, dwq, dwk = r.norm_backward(dnq, dnk, q, k, pos.cuda(), wq, wk)

    leaves = [t.double().requires_grad_() for t in x]
    ang = pos.double()[:, None] * torch.tensor([float(f) for f in lo.frequencies(d)[0]], dtype=torch.float64)
    c, s = ang.cos()[:, None], ang.sin()[:, None]

    def prep(t, w):
        n = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w
        a, b = n[..., : d // 2], n[..., d // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    eq, ek, ev = prep(leaves[0], leaves[3]), prep(leaves[1], leaves[4]).repeat_interleave(2, 1), leaves[2].repeat_interleave(2, 1)
    i = torch.arange(T)
    D = torch.where(i[:, None] >= i[None], torch.exp(g.double()[:, None, None] * (i[:, None] - i[None]).clamp(min=0)), 0.0)
    a = torch.einsum("ihd,jhd->hij", eq, ek) * D * d ** -0.5
    (torch.einsum("hij,jhe->ihe", a, ev) * do.double()).sum().backward()
    for name, got, leaf in zip(("dq", "dk", "dv", "dwq", "dwk"), (dq, dk, dv, dwq, dwk), leaves):
        # sums of up to 70 * 70 products of order one in float32
        check(name, got, leaf.grad, 2.0 ** -15 * float(leaf.grad.abs().max()))


def test_layer_streams_and_graphs():
    """On another stream than torch's default, and captured into two graphs that replay in turn on new inputs."""
    T, H, d = 300, 2, 64
    dtype = torch.bfloat16
    att = pn.LinearAttention(H, H, d, d, decays(H), dtype=dtype)
    r = pn.Rotary(d)
    w = torch.ones(d, device="cuda")
    pos = torch.arange(T, device="cuda")

    def layer(x):
        q, k = r.norm_apply(x[0], x[1], pos, w, w)
        o, S = att.forward(q[None], k[None], x[2][None])
        dq, dk, dv, ds0 = att.backward(o, q[None], k[None], x[2][None], initial_state=S, dstate=S)
        gq, gk, dwq, dwk = r.norm_backward(dq[0], dk[0], x[0], x[1], pos, w, w)
        y = att.step(x[0][:1], x[1][:1], x[2][:1], S, rotary=r, positions=pos[:1], wq=w, wk=w)
        return o, S, dv, ds0, gq, gk, dwq, dwk, y

    ins = [rnd(20 + i, 3, T, H, d, dtype=dtype).cuda() for i in range(3)]
    want = [layer(x) for x in ins]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer(ins[0])
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want[0]):
        assert torch.equal(a, b)
    graphs = []
    for i in range(2):
        x = ins[i].clone()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = layer(x)
        graphs.append((gr, x, out))
    for turn in range(2):
        for i, (gr, x, out) in enumerate(graphs):
            x.copy_(ins[(i + turn + 1) % 3])
            gr.replay()
        torch.cuda.synchronize()
        for i, (gr, x, out) in enumerate(graphs):
            for a, b in zip(out, want[(i + turn + 1) % 3]):
                assert torch.equal(a, b)
