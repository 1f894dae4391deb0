"""CPU checks of the sequence-layer wrappers: copies of plans and handles, and calls that are refused before any device is
asked."""
import copy
import pickle

import numpy as np
import pytest
import torch

import newton_evaluation_nonlinear_b200 as pn


@pytest.mark.parametrize("make", [copy.copy, copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x))])
def test_copies_are_handles_of_their_own(make):
    """A copy holds a handle of its own, made from the same arguments, and outlives its original (as in the copy of a model
    that holds one)."""
    r = pn.Rotary(64, 5e5, "interleaved", "yarn", 8.0, 2048, 16.0, 2.0, 1.25)
    s = make(r)
    assert s.h and s.h != r.h and s.rot_dim == 64 and s._args == r._args
    a = pn.LinearAttention(4, 2, 64, 96, torch.tensor([0.0, -0.1, -1.0, -9.0]), scale=0.25, dtype=torch.bfloat16)
    b = make(a)
    assert b.h and b.h != a.h
    assert (b.heads, b.kv_heads, b.dk, b.dv, b.scale, b.dtype) == (4, 2, 64, 96, 0.25, torch.bfloat16)
    assert np.array_equal(a._args[4], b._args[4])
    del r, a
    assert pn.lib.pn_linattn_workspace(b.h, 1, 2, 4096, 0, 0) > 0
    both = make([b, s, b])
    del both, s, b


def test_tensors_that_require_a_gradient_are_refused():
    """Results carry no graph: while torch records one, an argument that requires a gradient would lose it in silence.  (The
    refusal comes first; the same calls without recording go on to the next check, that of the device.)"""
    r, att = pn.Rotary(8), pn.LinearAttention(2, 2, 8, 8, [0.0, -0.1])
    x, w, pos = torch.zeros(1, 3, 2, 8), torch.ones(8), torch.zeros(1, 3, dtype=torch.int64)
    s = torch.zeros(3, 2, 8, 8)
    calls = [(r.apply, dict(q=x, k=x, positions=pos), "q k"), (r.apply_backward, dict(dq=x, dk=x, positions=pos), "dq dk"),
             (r.norm_apply, dict(q=x, k=x, positions=pos, wq=w, wk=w), "q k wq wk"),
             (r.norm_backward, dict(dq_out=x, dk_out=x, q=x, k=x, positions=pos, wq=w, wk=w), "dq_out dk_out q k wq wk"),
             (att.forward, dict(q=x, k=x, v=x, initial_state=s[:1], out=x), "q k v initial_state out"),
             (att.backward, dict(do=x, q=x, k=x, v=x, initial_state=s[:1], dstate=s[:1]), "do q k v initial_state dstate"),
             (att.step, dict(q=x[0], k=x[0], v=x[0], states=s, wq=w, wk=w), "q k v states wq wk")]
    for call, kw, names in calls:
        for name in names.split():
            leaf = kw[name].clone().requires_grad_()
            with pytest.raises(ValueError, match="requires a gradient"):
                call(**{**kw, name: leaf})
            with pytest.raises(ValueError, match="requires a gradient"):
                call(**{**kw, name: leaf * 1})
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
                call(**{**kw, name: leaf})
        with pytest.raises(ValueError, match="CUDA"):
            call(**kw)
    for call, kw, key in ((r.apply, calls[0][1], "out"), (r.norm_backward, calls[3][1], "out")):
        with pytest.raises(ValueError, match="requires a gradient"):
            call(**kw, **{key: (x, x.clone().requires_grad_())})
    with pytest.raises(ValueError, match="requires a gradient"):
        att.backward(x, x, x, x, grads=(x, x, x.clone().requires_grad_()))


def test_debug_waits_refusals():
    att = pn.LinearAttention(2, 2, 8, 8, [0.0, -0.1])
    for args, needle in [((None, 1000, -1), "handle"), ((att.h, 999, -1), "timeout"), ((att.h, 4000000001, -1), "timeout"), ((att.h, 1000, -2), "stall_chunk")]:
        assert pn.lib.pn_linattn_debug_waits(*args) == pn.PN_ERR_INVALID and needle in pn.pn_last_error(None)
    assert pn.lib.pn_linattn_debug_waits(att.h, 1000, 3) == pn.PN_OK


def test_sizes_beyond_32_bits_are_refused():
    """Not cut to their low bits."""
    far = 2 ** 32 + 8
    for make in (lambda: pn.Rotary(far), lambda: pn.LinearAttention(2, 2, far, 8, [0.0, 0.0], scale=1.0),
                 lambda: pn.LinearAttention(2, 2, 8, far, [0.0, 0.0])):
        with pytest.raises(ValueError, match="32 bits"):
            make()
    r, att = pn.Rotary(8), pn.LinearAttention(2, 2, 8, 8, [0.0, 0.0])
    small = torch.zeros(1, 1, 1, 8)
    for shape in ((far, 1, 1, 8), (1, far, 1, 8), (1, 1, far, 8)):
        x = small.expand(shape)
        pos = torch.zeros(1, 1, dtype=torch.int64).expand(shape[:2])
        with pytest.raises(ValueError, match="2\\^31"):
            r.apply(x, x, pos)
        with pytest.raises(ValueError, match="2\\^31"):
            att.forward(x, x, x)
    with pytest.raises(ValueError, match="2\\^31"):
        att.step(small[0].expand(far, 2, 8), small[0], small[0], torch.zeros(1, 2, 8, 8))


def test_attention_scales_beyond_float32_are_refused():
    """The factor is applied as a float32: one that would become zero or infinite is refused."""
    for m in (1e-50, 1e39, float("inf"), float("nan")):
        with pytest.raises((pn.PnError, ValueError), match="attention_scale"):
            pn.Rotary(64, attention_scale=m)
    pn.Rotary(64, attention_scale=1e-30)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32, torch.float64])
def test_decays_of_any_floating_type(dtype):
    g = torch.tensor([0.0, -0.5, -2.0], dtype=dtype)
    att = pn.LinearAttention(3, 1, 8, 8, g)
    assert np.array_equal(att._args[4], np.array([0.0, -0.5, -2.0], np.float32))


@pytest.mark.parametrize("dk", [0, -8])
def test_widths_below_one_are_refused_as_others_are(dk):
    """With the default scale too, which dk ** -0.5 would be."""
    with pytest.raises(pn.PnError, match=f"dk={dk}"):
        pn.LinearAttention(2, 2, dk, 8, [0.0, 0.0])


def test_split():
    """Which kernel, how many columns to a CTA, how many parts: the rules at their edges."""
    import ctypes

    def split(att, pass_, n, T, ragged=0, max_len=0):
        c, p = ctypes.c_int(-1), ctypes.c_int(-1)
        assert pn.lib.pn_linattn_split(att.h, pass_, n, T, ragged, max_len, ctypes.byref(c), ctypes.byref(p)) == pn.PN_OK
        return c.value, p.value

    att = pn.LinearAttention(2, 2, 128, 96, [0.0, 0.0], dtype=torch.bfloat16)
    assert split(att, 0, 37, 100) == (64, 1) and split(att, 0, 38, 100) == (128, 1)   # 37 x 2 heads x 2 CTAs fit 148 SMs
    assert split(att, 0, 1, 65536)[1] > 1 and split(att, 0, 1, 65536, 1, 100)[1] == 1
    wide = pn.LinearAttention(2, 2, 136, 96, [0.0, 0.0], dtype=torch.bfloat16)
    assert [split(wide, p, 1, 100)[0] for p in range(4)] == [0, 64, 64, 0]
    assert split(pn.LinearAttention(2, 2, 128, 96, [0.0, 0.0], dtype=torch.float16), 0, 1, 100)[0] == 0
    c = ctypes.c_int()
    for args, needle in [((None, 0, 1, 1, 0, 0, c, c), "NULL"), ((att.h, 4, 1, 1, 0, 0, c, c), "pass"),
                         ((att.h, 0, -1, 1, 0, 0, c, c), "shape"), ((att.h, 0, 1, 1, 0, -1, c, c), "max_len")]:
        assert pn.lib.pn_linattn_split(*args[:6], *map(ctypes.byref, args[6:])) == pn.PN_ERR_INVALID
        assert needle in pn.pn_last_error(None)
