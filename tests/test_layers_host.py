"""CPU checks of the sequence-layer operators: the oracle against differences, and every refusal that needs no GPU."""
import ctypes

import numpy as np
import pytest
import torch

import layer_oracle as lo
import newton_evaluation_nonlinear_b200 as pn


def test_oracle_gradients_against_differences():
    """The oracle's gradients are those of its forward pass: central differences in 64 bits, step 1e-6; the loss is
    at most cubic in each input, so the error is a few 1e-9 (1e-16 / 1e-6 of cancellation) of values of order one."""
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, dtype=torch.float64, generator=gen)  # noqa: E731
    q, k, v, s0 = rnd(5, 4, 3), rnd(5, 2, 3), rnd(5, 2, 6), rnd(4, 3, 6)
    g = torch.tensor([0.0, -0.1, -0.7, -3.0])
    do, ds = rnd(5, 4, 6), rnd(4, 3, 6)

    def loss():
        o, S = lo.linear(q, k, v, g, 0.4, s0)
        return float((o * do).sum() + (S * ds).sum())

    for x, dx in zip((q, k, v, s0), lo.linear_gradient(do, q, k, v, g, 0.4, s0, ds)):
        for at in range(0, x.numel(), 7):
            flat = x.view(-1)
            old = float(flat[at])
            flat[at] = old + 1e-6
            up = loss()
            flat[at] = old - 1e-6
            down = loss()
            flat[at] = old
            assert abs((up - down) / 2e-6 - float(dx.reshape(-1)[at])) < 1e-7

    x, w, t = rnd(3, 2, 6), rnd(6), rnd(3, 2, 6)
    dx, dw = lo.norm_gradient(t, x, w, 1e-3)
    for y, dy in ((x, dx), (w, dw)):
        for at in range(y.numel()):
            flat = y.view(-1)
            old = float(flat[at])
            flat[at] = old + 1e-6
            up = float((lo.norm(x, w, 1e-3) * t).sum())
            flat[at] = old - 1e-6
            down = float((lo.norm(x, w, 1e-3) * t).sum())
            flat[at] = old
            assert abs((up - down) / 2e-6 - float(dy.reshape(-1)[at])) < 1e-7


def test_oracle_rotation_is_orthogonal_and_relative():
    gen = torch.Generator().manual_seed(4)
    x, y = torch.randn(1, 2, 12, dtype=torch.float64, generator=gen), torch.randn(1, 2, 12, dtype=torch.float64, generator=gen)
    for layout in ("half", "interleaved"):
        def dot(p, s):
            a = lo.rotate(x, torch.tensor([p]), 8, layout)
            b = lo.rotate(y, torch.tensor([s]), 8, layout)
            return (a * b).sum(-1)
        torch.testing.assert_close(dot(7, 3), dot(1007, 1003), rtol=0, atol=1e-9)
        back = lo.rotate(lo.rotate(x, torch.tensor([77]), 8, layout), torch.tensor([77]), 8, layout, inverse=True)
        torch.testing.assert_close(back, x, rtol=0, atol=1e-12)


@pytest.mark.parametrize("kw, needle", [
    (dict(rot_dim=0), "rot_dim"), (dict(rot_dim=7), "rot_dim"), (dict(rot_dim=258), "rot_dim"),
    (dict(base=1.0), "base"), (dict(base=float("nan")), "base"),
    (dict(scaling="linear", factor=0.5), "factor"), (dict(scaling="ntk", factor=float("inf")), "factor"),
    (dict(scaling="ntk", factor=2.0, rot_dim=2), "rot_dim"),
    (dict(scaling="yarn", factor=2.0, original_length=0), "yarn"),
    (dict(scaling="yarn", factor=2.0, beta_fast=1.0, beta_slow=1.0), "yarn"),
])
def test_rotary_plan_refusals(kw, needle):
    with pytest.raises(pn.PnError, match=needle):
        pn.Rotary(**{"rot_dim": 64, **kw})


def test_rotary_wrapper_refusals():
    for kw in (dict(layout="other"), dict(scaling="other"), dict(attention_scale=0.0)):
        with pytest.raises(ValueError):
            pn.Rotary(64, **kw)
    r = pn.Rotary(64)
    q, k = torch.zeros(2, 3, 4, 64), torch.zeros(2, 3, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        r.apply(q, k, torch.zeros(2, 3, dtype=torch.int64))


@pytest.mark.parametrize("args, needle", [
    ((0, 1, 64, 64), "H=0"), ((257, 1, 64, 64), "H=257"), ((4, 3, 64, 64), "divide"), ((4, 0, 64, 64), "Hkv"),
    ((4, 4, 12, 64), "dk=12"), ((4, 4, 64, 264), "dv=264"), ((4, 4, 0, 64), "dk=0"),
])
def test_linear_attention_shape_refusals(args, needle):
    with pytest.raises(pn.PnError, match=needle):
        pn.LinearAttention(*args, np.zeros(args[0], np.float32), scale=1.0)


def test_linear_attention_decay_refusals():
    for bad in (0.1, float("nan"), float("-inf")):
        with pytest.raises(pn.PnError, match="log_decay"):
            pn.LinearAttention(2, 1, 8, 8, [0.0, bad])
    with pytest.raises(ValueError, match="log_decay"):
        pn.LinearAttention(2, 1, 8, 8, [0.0])
    with pytest.raises(ValueError, match="fixed"):
        pn.LinearAttention(2, 1, 8, 8, torch.zeros(2, requires_grad=True))
    with pytest.raises(pn.PnError, match="scale"):
        pn.LinearAttention(2, 1, 8, 8, [0.0, 0.0], scale=float("inf"))
    with pytest.raises(ValueError, match="dtype"):
        pn.LinearAttention(2, 1, 8, 8, [0.0, 0.0], dtype=torch.float64)


def _call(name, *args):
    return getattr(pn.lib, name)(*args), pn.pn_last_error(None)


def test_c_entry_refusals():
    """Bad arguments of the C entry points are refused before anything touches a device."""
    r = pn.Rotary(64)
    a = pn.LinearAttention(4, 2, 64, 32, np.full(4, -0.5, np.float32))
    x = np.zeros(4096, np.float32)   # a host array: refused as a device pointer
    h = pn.pn_heads(x.ctypes.data, 0, 256, 64)
    neg = pn.pn_heads(x.ctypes.data, 0, -256, 64)
    bad = pn.PN_ERR_INVALID
    f = ctypes.c_float
    assert _call("pn_rotary_create", None, None)[0] == bad
    assert _call("pn_rotary_apply", None, 0, 1, 1, 1, 1, 64, h, h, None, 0, h, h, None)[0] == bad
    for args, needle in [((9, 1, 1, 1, 1, 64), "dtype"), ((0, -1, 1, 1, 1, 64), "shape"), ((0, 1, 1, 0, 1, 64), "shape"),
                         ((0, 1, 1, 1, 1, 32), "rot_dim"), ((0, 1, 1, 1, 1, 258), "dim"), ((0, 1, 1, 1, 1, 65), "dim")]:
        st, text = _call("pn_rotary_apply", r.h, *args, h, h, x.ctypes.data, 0, h, h, None)
        assert st == bad and needle in text, (args, text)
    st, text = _call("pn_rotary_apply", r.h, 0, 1, 1, 1, 1, 64, h, neg, x.ctypes.data, 0, h, h, None)
    assert st == bad and "stride" in text
    st, text = _call("pn_rotary_apply", r.h, 0, 1, 1, 1, 1, 64, h, None, x.ctypes.data, 0, h, h, None)
    assert st == bad and "k is NULL" in text
    st, text = _call("pn_rotary_apply", r.h, 0, 1, 1, 1, 1, 64, h, h, x.ctypes.data, 2, h, h, None)
    assert st == bad and "inverse" in text
    st, text = _call("pn_rotary_apply", r.h, 0, 1, 1, 1, 1, 64, h, h, x.ctypes.data, 0, h, h, None)
    assert st == bad and ("CUDA" in text or "device" in text)
    assert _call("pn_rotary_apply", r.h, 0, 0, 5, 1, 1, 64, h, h, None, 0, h, h, None)[0] == pn.PN_OK   # no rows: no work
    p = x.ctypes.data
    for w, wd, eps, needle in [((None, p), 0, 1e-6, "NULL"), ((p, p), 1, 1e-6, "weights"), ((p, p), 0, -1.0, "eps"),
                               ((p, p), 0, float("nan"), "eps")]:
        st, text = _call("pn_norm_rotary_apply", r.h, 0, 1, 1, 1, 1, 64, h, h, p, *w, wd, f(eps), h, h, None)
        assert st == bad and needle in text, (needle, text)
    assert pn.lib.pn_norm_rotary_workspace(1, 1, 0, 1, 64) == 0
    st, text = _call("pn_norm_rotary_backward", r.h, 0, 1, 1, 1, 1, 64, None, h, h, h, p, p, p, 0, f(1e-6), h, h, p, p, p, 0,
                     None)
    assert st == bad

    assert _call("pn_linattn_forward", None, 1, 1, None, 0, h, h, h, None, h, None, None, 0, None)[0] == bad
    for n, T, needle in [(-1, 1, "shape"), (1, -1, "shape"), (1, 1 << 33, "rows"), (20000, 1, "65535")]:
        st, text = _call("pn_linattn_forward", a.h, n, T, None, 0, h, h, h, None, h, None, None, 0, None)
        assert st == bad and needle in text, (n, T, text)
    st, text = _call("pn_linattn_forward", a.h, 1, 1, None, -1, h, h, h, None, h, None, None, 0, None)
    assert st == bad and "max_len" in text
    assert _call("pn_linattn_forward", a.h, 0, 5, None, 0, h, h, h, None, h, None, None, 0, None)[0] == pn.PN_OK   # no rows
    st, text = _call("pn_linattn_forward", a.h, 1, 4, None, 0, h, None, h, None, h, None, None, 0, None)
    assert st == bad
    assert pn.lib.pn_linattn_workspace(None, 0, 1, 1, 0, 0) == 0
    for rows, n_slots, needle in [(-1, 1, "rows"), (70000, 70000, "rows"), (3, 2, "n_slots"), (1, -1, "n_slots")]:
        st, text = _call("pn_linattn_step", a.h, rows, h, h, h, h, p, n_slots, None, None, None, None, None, 0, f(0), None)
        assert st == bad and needle in text, (rows, text)
    st, text = _call("pn_linattn_step", a.h, 1, h, h, h, h, p, 1, None, None, None, p, None, 0, f(0), None)
    assert st == bad and "together" in text
    big = pn.Rotary(128)
    st, text = _call("pn_linattn_step", a.h, 1, h, h, h, h, p, 1, None, big.h, None, None, None, 0, f(0), None)
    assert st == bad and "rot_dim" in text
