"""Calls of the sequence-layer operators at the edges of what their documentation allows: empty sequences, elements that do
not rotate, offsets out of order, outputs of unusual inputs, and the kernels that only larger grids reach.

Bounds are those of test_gpu_layers.py, which derives them; what is compared bit for bit here has no rounding in it.
"""
import pytest
import torch

import newton_evaluation_nonlinear_b200 as pn
from test_gpu_layers import TYPES, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n_copies, dk, dv", [(1, 64, 64), (1, 128, 96), (20, 128, 128)])
def test_empty_sequences_keep_their_states(n_copies, dk, dv, dtype):
    """The final state of an empty sequence is its initial one, and the gradient of its initial state that of its final one,
    to the last bit, whatever the decays and the size of the values."""
    lens = [0, 5, 0, 130, 64, 1, 0] * n_copies
    n, H, K, T = len(lens), 4, 2, sum(lens)
    att = pn.LinearAttention(H, K, dk, dv, [-1e-3, -0.05, -0.8, -3.0], dtype=dtype)
    q, do = rnd(1, T, H, dk, dtype=dtype).cuda(), rnd(2, T, H, dv, dtype=dtype).cuda()
    k, v = rnd(3, T, K, dk, dtype=dtype).cuda(), rnd(4, T, K, dv, dtype=dtype).cuda()
    s0, ds = rnd(5, n, H, dk, dv).cuda(), rnd(6, n, H, dk, dv).cuda()
    s0[:, :, 1] *= 1e-35   # small enough that a detour by way of other powers of two would lose bits
    ds[:, :, 2] *= 1e30
    cu = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
    o, S = att.forward(q, k, v, initial_state=s0, cu_seqlens=cu, max_len=130)
    ds0 = att.backward(do, q, k, v, initial_state=s0, dstate=ds, cu_seqlens=cu, max_len=130)[3]
    for i, length in enumerate(lens):
        if length == 0:
            assert torch.equal(S[i], s0[i]) and torch.equal(ds0[i], ds[i]), i
    o, S = att.forward(q[:0], k[:0], v[:0], initial_state=s0, cu_seqlens=torch.zeros_like(cu))   # nothing but empty ones
    assert torch.equal(S, s0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim, rot, layout", [(128, 64, "half"), (128, 64, "interleaved"), (72, 24, "half"), (40, 12, "half"),
                                              (40, 12, "interleaved"), (10, 6, "half"), (10, 6, "interleaved"), (256, 8, "half"),
                                              (256, 2, "interleaved")])
def test_elements_that_do_not_rotate_pass_through(dim, rot, layout, dtype):
    """Elements behind rot_dim come out as they went in, infinities, NaN and negative zeros too, and reach no other element."""
    B, T, H, K = 2, 5, 3, 1
    r = pn.Rotary(rot, layout=layout, scaling="yarn", factor=4.0)
    pos = (torch.arange(T)[None] + torch.tensor([[0], [99]])).cuda()
    clean = [rnd(i, B, T, h, dim, dtype=dtype).cuda() for i, h in ((1, H), (2, K))]
    odd = torch.tensor([float("inf"), float("-inf"), float("nan"), -0.0, 1.0], dtype=dtype, device="cuda")
    gen = torch.Generator().manual_seed(3)
    filled = []
    for x in clean:
        x = x.clone()
        x[..., rot:] = odd[torch.randint(0, 5, (*x.shape[:-1], dim - rot), generator=gen).cuda()]
        filled.append(x)
    bits = torch.int32 if dtype == torch.float32 else torch.int16
    for call in (r.apply, r.apply_backward):
        for x, got, want in zip(filled, call(*filled, pos), call(*clean, pos)):
            assert torch.equal(got[..., :rot], want[..., :rot])
            a, b = got[..., rot:], x[..., rot:]
            assert torch.equal(a.isnan(), b.isnan())
            assert torch.equal(a.contiguous().view(bits)[~a.isnan()], b.contiguous().view(bits)[~b.isnan()])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [1, 2])
def test_gradients_with_offsets_out_of_order(K, dtype):
    """Gradients take the rows that the forward pass takes whatever the offsets say, shared heads included: offsets outside the
    buffer are cut to it and a decreasing one makes an empty sequence."""
    T, H, d = 200, 2, 64
    att = pn.LinearAttention(H, K, d, d, [-0.05, -0.8], dtype=dtype)
    q, do = rnd(1, T, H, d, dtype=dtype).cuda(), rnd(2, T, H, d, dtype=dtype).cuda()
    k, v = rnd(3, T, K, d, dtype=dtype).cuda(), rnd(4, T, K, d, dtype=dtype).cuda()
    s0, ds = rnd(5, 3, H, d, d).cuda(), rnd(6, 3, H, d, d).cuda()

    def run(cu):
        grads = tuple(torch.full_like(x, 7.0) for x in (q, k, v))
        return att.backward(do, q, k, v, initial_state=s0, dstate=ds, max_len=T, grads=grads,
                            cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())

    for bad, good in (([-5, 90, 90, 1000000], [0, 90, 90, T]), ([0, 120, 60, 60], [0, 120, 120, 120]),
                      ([150, 2 ** 31 - 1, 40, 40], [150, T, T, T]), ([190, 100, 100, 160], [100, 100, 100, 160])):
        for name, a, b in zip(("dq", "dk", "dv", "ds0"), run(bad), run(good)):
            assert torch.equal(a, b), (bad, name)
    dq, dk, dv, _ = run([190, 100, 100, 160])   # rows of no sequence are left as they were
    for x in (dq, dk, dv):
        assert bool((x[:100] == 7).all()) and bool((x[160:] == 7).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_gradients_of_shared_heads_in_many_sequences(dtype):
    """Sequences of very different lengths beside each other: each row of dk and dv is that of its sequence alone, to the bit
    where both runs take the same parts."""
    H, K, d = 4, 1, 16
    lens = [(5 * i) % 7 for i in range(300)] + [400, 0, 131]
    T = sum(lens) + 9
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    att = pn.LinearAttention(H, K, d, d, [-0.01, -0.1, -0.9, -3.0], dtype=dtype)
    q, do = rnd(1, T, H, d, dtype=dtype).cuda(), rnd(2, T, H, d, dtype=dtype).cuda()
    k, v = rnd(3, T, K, d, dtype=dtype).cuda(), rnd(4, T, K, d, dtype=dtype).cuda()
    grads = tuple(torch.full_like(x, 7.0) for x in (q, k, v))
    att.backward(do, q, k, v, cu_seqlens=cu, max_len=400, grads=grads)
    for i in (0, 1, 3, 299, 300, 302):
        r = slice(int(cu[i]), int(cu[i + 1]))
        one = torch.tensor([r.start] + [r.stop] * len(lens), dtype=torch.int32, device="cuda")
        alone = att.backward(do, q, k, v, cu_seqlens=one, max_len=400)
        for x, y in zip(grads, alone):
            assert torch.equal(x[r], y[r]), i
    for x in grads:
        assert bool((x[T - 9:] == 7).all())


@pytest.mark.parametrize("n", [2, 33, 512, 513])
def test_order_of_sequences_does_not_matter(n):
    """Sequences are taken by length; packed in another order each gives the same bits."""
    H, d = 2, 64
    gen = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 150, (n,), generator=gen).tolist()
    lens[n // 2] = 700
    lens[n - 1] = lens[0]
    T = sum(lens)
    att = pn.LinearAttention(H, H, d, d, [-0.01, -0.9], dtype=torch.bfloat16)
    x = [rnd(i, T, H, d, dtype=torch.bfloat16) for i in (1, 2, 3)]
    s0 = rnd(4, n, H, d, d)
    parts = [list(y.split(lens)) for y in x]

    def run(order):
        cu = torch.tensor([0] + [lens[i] for i in order]).cumsum(0).int().cuda()
        packed = [torch.cat([p[i] for i in order]).cuda() for p in parts]
        o, S = att.forward(*packed, initial_state=s0[order].cuda(), cu_seqlens=cu, max_len=700)
        rows = dict(zip(order, o.split([lens[i] for i in order])))
        return [rows[i] for i in range(n)], S[torch.tensor(order).argsort().cuda()]

    o, S = run(list(range(n)))
    o2, S2 = run(torch.randperm(n, generator=gen).tolist())
    assert torch.equal(S, S2)
    assert all(torch.equal(a, b) for a, b in zip(o, o2))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_windows_that_overlap(dtype):
    """Heads that are windows of one row, each an element on from the one before (any strides are allowed): results are those of
    a copy, and come in tensors of their own with contiguous rows."""
    T, H, d = 70, 4, 64
    base = rnd(1, T, d + H - 1, dtype=dtype).cuda()
    x = base.as_strided((T, H, d), (d + H - 1, 1, 1))
    y = x.clone(memory_format=torch.contiguous_format)
    pos, w = torch.arange(T, device="cuda"), rnd(2, d).cuda()
    r, att = pn.Rotary(d), pn.LinearAttention(H, H, d, d, [0.0, -0.05, -0.8, -3.0], dtype=dtype)
    s0 = rnd(3, 1, H, d, d).cuda()
    one = dict(initial_state=s0, cu_seqlens=torch.tensor([0, T], dtype=torch.int32, device="cuda"))
    for a, b in zip(r.apply(x, x, pos), r.apply(y, y, pos)):
        assert torch.equal(a, b)
    for a, b in zip((*r.norm_apply(x, x, pos, w, w), *r.norm_backward(x, x, x, x, pos, w, w)[:2]),
                    (*r.norm_apply(y, y, pos, w, w), *r.norm_backward(y, y, y, y, pos, w, w)[:2])):
        # one rounding on each side, and float32 sums in two orders: test_gpu_layers.py has 2^-19 of a vector's size for one
        # (of y forward; of r |t w| in the gradient, at most sqrt(2) max|x| max|w| max r = 22 here)
        size = (b.double().abs().amax(-1, keepdim=True) + 22).cpu()
        off = (a.double() - b.double()).abs().cpu() - 2 * torch.finfo(dtype).eps / 2 * b.double().abs().cpu() - 2.0 ** -18 * size
        assert float(off.max()) <= 0
    for a, b in zip((*att.forward(x, x, x, **one), *att.backward(x, x, x, x, **one)),
                    (*att.forward(y, y, y, **one), *att.backward(y, y, y, y, **one))):
        assert torch.equal(a, b)
    states = [rnd(4, T, H, d, d).cuda() for _ in range(2)]
    assert torch.equal(att.step(x, x, x, states[0]), att.step(y, y, y, states[1]))
    assert torch.equal(*states)


def test_outputs_in_the_place_of_other_arrays_are_refused():
    """Where a pass would read what it has overwritten.  Rotations and norms may write over what they replace, no further."""
    T, H, d = 8, 2, 64
    r, att = pn.Rotary(d), pn.LinearAttention(H, H, d, d, [-0.1] * H)
    q, k, v, do = (rnd(i, T, H, d).cuda() for i in range(4))
    pos, w = torch.arange(T, device="cuda"), torch.ones(d, device="cuda")
    e = lambda: torch.empty_like(q)  # noqa: E731
    for out in [(k, q), (q, q), (e(), q), (k, e())]:
        with pytest.raises(pn.PnError, match="memory"):
            r.apply(q, k, pos, out=out)
        with pytest.raises(pn.PnError, match="memory"):
            r.norm_apply(q, k, pos, w, w, out=out)
        with pytest.raises(pn.PnError, match="memory"):
            r.norm_backward(q, k, do, v, pos, w, w, out=out)
    long = torch.zeros(2 * T, H, d, device="cuda")
    with pytest.raises(pn.PnError, match="memory"):   # in place, but with other strides
        r.apply(long[::2], k, pos, out=(long[:T], e()))
    for out in (q, k, v):
        with pytest.raises(pn.PnError, match="memory"):
            att.forward(q[None], k[None], v[None], out=out[None])
        with pytest.raises(pn.PnError, match="memory"):
            att.step(q, k, v, torch.zeros(T, H, d, d, device="cuda"), out=out)
    both = torch.zeros(T, H, d, d, device="cuda")
    with pytest.raises(pn.PnError, match="memory"):
        att.step(q, k, v, both, out=both.view(-1)[: T * H * d].view(T, H, d))
    for grads in [(q, e(), e()), (e(), k, e()), (e(), e(), do)] + [(k, e(), e())]:
        with pytest.raises(pn.PnError, match="memory"):
            att.backward(do[None], q[None], k[None], v[None], grads=tuple(x[None] for x in grads))
    one = e()
    with pytest.raises(pn.PnError, match="memory"):
        att.backward(do[None], q[None], k[None], v[None], grads=(one[None], e()[None], one[None]))
    windows = torch.zeros(T * H * d, device="cuda").as_strided((T, H, d), (d, 8, 1))
    with pytest.raises(ValueError, match="overlapping"):
        r.apply(q, k, pos, out=(windows, e()))
    with pytest.raises(ValueError, match="overlapping"):
        att.forward(q[None], k[None], v[None], out=windows[None])
    h = lambda t: pn.pn_heads(t.data_ptr(), 0, t.stride(0), t.stride(1))  # noqa: E731
    assert pn.lib.pn_rotary_apply(r.h, pn.PN_F32, 1, T, H, H, d, h(q), h(k), pos.data_ptr(), 0, h(windows), h(e()),
                                  None) == pn.PN_ERR_INVALID
    assert "overlapping" in pn.pn_last_error(None)


@pytest.mark.parametrize("dtype", TYPES)
def test_in_place_gradients(dtype):
    """apply_backward over the gradients it takes, norm_backward over those or over the inputs: the same bits."""
    T, H, K, d = 300, 4, 2, 64
    r = pn.Rotary(d)
    q, k, gq, gk = (rnd(i, T, n, d, dtype=dtype).cuda() for i, n in ((1, H), (2, K), (3, H), (4, K)))
    pos, w = torch.arange(T, device="cuda"), rnd(5, d).cuda()
    want = r.apply_backward(gq, gk, pos)
    a, b = gq.clone(), gk.clone()
    r.apply_backward(a, b, pos, out=(a, b))
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    want = r.norm_backward(gq, gk, q, k, pos, w, w)
    a, b = gq.clone(), gk.clone()
    for x, y in zip(r.norm_backward(a, b, q, k, pos, w, w, out=(a, b)), want):
        assert torch.equal(x, y)
    a, b = q.clone(), k.clone()
    for x, y in zip(r.norm_backward(gq, gk, a, b, pos, w, w, out=(a, b)), want):
        assert torch.equal(x, y)
    # the gradients side by side in one buffer, as one projection's gradient wants them
    both = torch.zeros(T, H + K, d, dtype=dtype, device="cuda")
    r.norm_backward(gq, gk, q, k, pos, w, w, out=(both[:, :H], both[:, H:]))
    assert torch.equal(both[:, :H], want[0]) and torch.equal(both[:, H:], want[1])


@pytest.mark.parametrize("chunk", [0, 1, 5])
@pytest.mark.parametrize("dk, dv, n, backward", [(64, 64, 1, False), (128, 128, 1, True), (128, 64, 40, True), (64, 128, 40, False),
                                                 (128, 128, 40, False)])
def test_waits_that_give_up_are_reported(dk, dv, n, backward, chunk):
    """Where a chunk is never loaded the waits for it run out after 100 us and the pass ends; every stream's check says so once,
    and later passes are right."""
    T, H = 2000, 2   # (n = 1: in parts of a few chunks)
    att = pn.LinearAttention(H, H, dk, dv, [-0.01, -0.9], dtype=torch.bfloat16)
    q, k, v, do = (rnd(i, n, T, H, w, dtype=torch.bfloat16).cuda() for i, w in enumerate((dk, dk, dv, dv)))
    s0 = rnd(9, n, H, dk, dv).cuda()

    def run():
        return att.backward(do, q, k, v, initial_state=s0, dstate=s0) if backward else att.forward(q, k, v, initial_state=s0)

    want = run()
    streams = [torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.current_stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            try:   # whatever other passes have left
                att.check()
            except pn.PnError:
                pass
            att.check()
    assert pn.lib.pn_linattn_debug_waits(att.h, 100000, chunk if n > 1 else min(chunk, 1)) == pn.PN_OK
    with torch.cuda.stream(streams[0]):
        run()
    streams[0].synchronize()
    assert pn.lib.pn_linattn_debug_waits(att.h, 2000000000, -1) == pn.PN_OK
    for s in reversed(streams):   # the other streams' checks first: they take nothing from this one's
        with torch.cuda.stream(s):
            with pytest.raises(pn.PnError) as e:
                att.check()
            assert e.value.status == pn.PN_ERR_TIMEOUT
            att.check()
    for a, b in zip(run(), want):
        assert torch.equal(a, b)
    for s in streams:
        with torch.cuda.stream(s):
            att.check()


FIRST_CAPTURED = """
import torch, newton_evaluation_nonlinear_b200 as pn
x = [torch.randn(300, 2, 64, device="cuda").to(t) for t in (torch.float32, torch.bfloat16, torch.float16)]
pos, w = torch.arange(300, device="cuda"), torch.ones(64, device="cuda")
r = pn.Rotary(64)
atts = [pn.LinearAttention(2, 2, 64, 64, [-0.1, 0.0], dtype=y.dtype) for y in x]
states = [torch.zeros(300, 2, 64, 64, device="cuda") for _ in x]
torch.cuda.synchronize()
def run():
    out = []
    for y, att, s in zip(x, atts, states):
        s.zero_()
        out += [*r.apply(y, y, pos), *r.norm_apply(y, y, pos, w, w), *r.norm_backward(y, y, y, y, pos, w, w),
                *att.forward(y[None], y[None], y[None]), *att.backward(y[None], y[None], y[None], y[None]), att.step(y, y, y, s)]
    return out
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = run()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, run()))
print("captured")
"""


def test_first_calls_in_a_capture():
    """A process whose first calls are captured (no kernel has been loaded before)."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FIRST_CAPTURED], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "captured" in run.stdout, run.stderr[-2000:]


def test_lists_beyond_31_bits():
    """More vectors than 2^30: rows and heads are found by 64-bit divisions."""
    T, H, K, d = (1 << 24) + 5, 63, 1, 8
    q, k = torch.zeros(T, H, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, K, d, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(T, device="cuda")
    r, w = pn.Rotary(d), torch.ones(d, device="cuda")
    rows = torch.tensor([0, 1, 77, 1 << 23, (1 << 24) - 1, 1 << 24, T - 1], device="cuda")
    q[rows], k[rows] = rnd(1, 7, H, d, dtype=torch.bfloat16).cuda(), rnd(2, 7, K, d, dtype=torch.bfloat16).cuda()
    gq, gk = r.norm_apply(q, k, pos, w, w)
    wq, wk = r.norm_apply(q[rows], k[rows], rows, w, w)
    assert torch.equal(gq[rows], wq) and torch.equal(gk[rows], wk)
    assert int((gq != 0).any(-1).any(-1).sum()) == 7 and int((gk != 0).any(-1).any(-1).sum()) == 7
    _, _, dwq, dwk = r.norm_backward(q, k, q, k, pos, w, w, out=(gq, gk))
    dq, dk, wwq, wwk = r.norm_backward(q[rows], k[rows], q[rows], k[rows], rows, w, w)
    assert torch.equal(gq[rows], dq) and torch.equal(gk[rows], dk)
    # sums in two orders of 7 x heads terms that are not zero, each 6 sqrt(8) at most: n additions are 2^-24 n of the terms' sum off
    for a, b, n in ((dwq, wwq, 7 * H), (dwk, wwk, 7 * K)):
        assert float((a - b).abs().max()) <= 2 * n * 2.0 ** -24 * n * 17


@pytest.mark.parametrize("lens, H, K", [([1], 1, 1), ([7], 8, 2), ([63], 1, 1), ([3, 0, 2, 10], 4, 2), ([1] * 15, 4, 4)])
@pytest.mark.parametrize("dk, dv", [(64, 64), (128, 128), (96, 96)])
def test_few_rows_are_rounded_once(lens, H, K, dk, dv, monkeypatch):
    """bfloat16 calls of a few rows, where the rounding of a weight would show in whole rows: only the outputs are rounded (the
    bound of float32, and half a step)."""
    import test_gpu_layers as base
    monkeypatch.setattr(base, "mixed", lambda dtype: 0.0)
    base.run_linear(lens, H, K, dk, dv, torch.bfloat16, lead=0, tail=0)
