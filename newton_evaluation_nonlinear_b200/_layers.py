"""torch-facing wrappers of the sequence-layer operators (include/pn.h): argument checks and marshalling only.

:class:`Rotary` rotates queries and keys by position, with or without the norm of each head vector before it;
:class:`LinearAttention` is the recurrence S_t = exp(g_h) S_{t-1} + k_t v_t^T, o_t = scale q_t S_t, over whole prompts
and for single tokens.  Gradients are explicit calls (``apply_backward``, ``norm_backward``, ``backward``); results
carry no autograd graph, so tensors that require a gradient are refused while torch records one: call from a
torch.autograd.Function, under torch.no_grad(), or with detached tensors.

Tensors are [tokens, heads, dim] or [batch, tokens, heads, dim], CUDA, of one of the types float32, bfloat16 and
float16, with contiguous rows and any other strides (slices of one projection's output go in as they are).  The work
is asynchronous on torch's current stream of the tensors' device; the calls can be captured into a CUDA graph.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

import numpy as np

from ._binding import (LIB_PATH, PN_BF16, PN_F16, PN_F32, PN_OK, PN_ROT_HALF, PN_ROT_INTERLEAVED, PN_ROT_LINEAR, PN_ROT_NTK,
                       PN_ROT_PLAIN, PN_ROT_YARN, PnError, SIGNATURES, lib, pn_heads, pn_last_error,
                       pn_rotary_desc)

_LAYOUTS = {"half": PN_ROT_HALF, "interleaved": PN_ROT_INTERLEAVED}
_SCALINGS = {"none": PN_ROT_PLAIN, "linear": PN_ROT_LINEAR, "ntk": PN_ROT_NTK, "yarn": PN_ROT_YARN}
_DTYPES = None
_HEADS_BYTES = ctypes.sizeof(pn_heads)


def _addresses() -> ctypes.CDLL:
    """The library again with every pointer as a plain address: the pn_heads of one call are rows of one array."""
    fast = ctypes.CDLL(LIB_PATH)
    for name in ("pn_rotary_apply", "pn_norm_rotary_apply", "pn_norm_rotary_backward", "pn_linattn_forward",
                 "pn_linattn_backward", "pn_linattn_step"):
        res, args = SIGNATURES[name]
        fn = getattr(fast, name)
        fn.restype, fn.argtypes = res, [ctypes.c_void_p if issubclass(a, ctypes._Pointer) else a for a in args]
    return fast


fast = _addresses()
_ROWS = {n: (struct.Struct(f"{4 * n}q"), ctypes.c_char * (_HEADS_BYTES * n), _HEADS_BYTES * n) for n in (4, 6, 7)}


def _dtypes():
    global _DTYPES
    if _DTYPES is None:
        import torch
        _DTYPES = {torch.float32: PN_F32, torch.bfloat16: PN_BF16, torch.float16: PN_F16}
    return _DTYPES


def _dtype(name, t):
    code = _dtypes().get(t.dtype)
    if code is None:
        raise ValueError(f"{name} is {t.dtype}: float32, bfloat16 or float16 is wanted")
    return code


def _ok(status: int) -> None:
    if status != PN_OK:
        raise PnError(status, pn_last_error(None))


_INT = 2 ** 31 - 1


def _int(name, n):
    """n as the C entries' 32-bit int (ctypes would keep the low bits of a larger one)."""
    n = int(n)
    if not -_INT <= n <= _INT:
        raise ValueError(f"{name}={n} does not fit 32 bits")
    return n


def _no_graph(*tensors):
    """Refuses tensors whose gradients torch would expect to be recorded."""
    for t in tensors:
        if t is not None and t.requires_grad:
            import torch
            if torch.is_grad_enabled():
                raise ValueError("a tensor requires a gradient, which this call does not record: call it under torch.no_grad() "
                                 "or from a torch.autograd.Function, or detach the tensor")


def _first(name, t):
    """The tensor that the others are held to: (dims, B, T, heads, dim, dtype, device number)."""
    nd = t.dim()
    if nd == 4:
        B, T, h, d = t.shape
    elif nd == 3:
        T, h, d = t.shape
        B = 1
    else:
        raise ValueError(f"{name} must be [tokens, heads, dim] or [batch, tokens, heads, dim]")
    if t.numel() > _INT and max(t.shape) > _INT:
        raise ValueError(f"{name} is {tuple(t.shape)}: sizes of up to 2^31 - 1 are taken")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return nd, B, T, h, d, t.dtype, t.get_device()


def _heads(name, t, like, heads, dim):
    """(address, batch, token and head stride) of a tensor with the first one's rows, type and device."""
    nd, B, T, _, _, dtype, device = like
    if t.dim() != nd:
        raise ValueError(f"{name} has {t.dim()} dimensions; {nd} are wanted")
    if nd == 4:
        b, n, h, e = t.shape
        x, y, z, w = t.stride()
    else:
        n, h, e = t.shape
        y, z, w = t.stride()
        b, x = 1, 0
    if n != T or e != dim or h != heads or b != B or t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{name} is {tuple(t.shape)} {t.dtype} on {t.device}; {(B, T, heads, dim)[4 - nd:]} {dtype} on "
                         f"cuda:{device} is wanted")
    if w != 1 and e > 1 and t.numel():
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), x, y, z


def _output(name, t, like, heads, dim):
    """The same of an output: tensors whose rows overlap (expanded ones, windows) are refused."""
    row = _heads(name, t, like, heads, dim)
    if min(row[1:]) < dim:
        for n, s in zip(t.shape[:-1], t.stride()):
            if n > 1 and s < dim:
                raise ValueError(f"{name} has overlapping elements")
    return row


def _fresh(t, nd):
    """(tensor, row as of :func:`_heads`) of one that empty_like has made.  (It orders dimensions by the strides of its model;
    windows that overlap by all but one element have two of one element, and then the rows need not be contiguous: another
    tensor takes its place.)"""
    if nd == 4:
        x, y, z, w = t.stride()
    else:
        x = 0
        y, z, w = t.stride()
    if w != 1:
        import torch
        return _fresh(torch.empty_like(t, memory_format=torch.contiguous_format), nd)
    return t, (t.data_ptr(), x, y, z)


def _rows(*heads):
    """Memory that holds the pn_heads of all of them, and the address of each."""
    layout, kind, n = _ROWS[len(heads)]
    memory = kind()
    at = ctypes.addressof(memory)
    layout.pack_into(memory, 0, *[v for row in heads for v in row])
    return memory, range(at, at + n, _HEADS_BYTES)


def _ints(name, t, shape, dtype, device):
    """Address of a contiguous tensor of integers; device: its number."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{device}")
    return t.data_ptr()


def _float32(name, t, shape, device):
    import torch
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.get_device() != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {tuple(shape)} on cuda:{device}")
    return t.data_ptr()


def _weights(wq, wk, dim, device):
    """Addresses and type of a norm's weights: float32, or the queries' type (which the library checks)."""
    dtype = wq.dtype
    for name, w in (("wq", wq), ("wk", wk)):
        if w.shape != (dim,) or not w.is_contiguous() or w.get_device() != device or w.dtype is not dtype:
            raise ValueError(f"{name} must be a contiguous [{dim}] tensor on cuda:{device}, both weights of one type")
    return wq.data_ptr(), wk.data_ptr(), _dtype("wq", wq)


def _stream(device):
    """torch's current stream of a device (by its number)."""
    import torch
    try:   # torch.cuda.current_stream without its Stream object
        return torch._C._cuda_getCurrentRawStream(device)
    except AttributeError:
        return torch.cuda.current_stream(device).cuda_stream


def _workspace(n, device):
    """(tensor that keeps it, pointer) of n bytes of torch's own memory, used on the current stream."""
    import torch
    if not n:
        return None, None
    w = torch.empty(n, dtype=torch.uint8, device=device)
    return w, w.data_ptr()


class Rotary:
    """The rotation of the first ``rot_dim`` elements of each head vector by its position.

    layout    "half" (pair i: elements i and i + rot_dim/2) or "interleaved" (2i and 2i + 1)
    scaling   "none"; "linear" (positions divided by ``factor``); "ntk" (the base stretched by ``factor``); "yarn"
              (per frequency, by a ramp linear in its turns over ``original_length``, as in the method's paper; models trained
              with a ramp linear in the pair's number have other frequencies)
    attention_scale   factor on the rotated elements; None: 1, or 0.1 ln(factor) + 1 for "yarn"

    The plan holds no device memory; one object serves every device and stream.  Copies, pickled ones too, are plans of
    their own.
    """

    def __init__(self, rot_dim: int, base: float = 10000.0, layout: str = "half", scaling: str = "none",
                 factor: float = 1.0, original_length: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 attention_scale: Optional[float] = None):
        if layout not in _LAYOUTS:
            raise ValueError(f"layout {layout!r}: one of {sorted(_LAYOUTS)}")
        if scaling not in _SCALINGS:
            raise ValueError(f"scaling {scaling!r}: one of {sorted(_SCALINGS)}")
        if attention_scale is not None and not attention_scale > 0:
            raise ValueError("attention_scale must be > 0")
        self.h = None
        self.rot_dim = _int("rot_dim", rot_dim)
        desc = pn_rotary_desc(self.rot_dim, _LAYOUTS[layout], _SCALINGS[scaling], float(base), float(factor),
                              int(original_length), float(beta_fast), float(beta_slow), float(attention_scale or 0.0))
        h = ctypes.c_void_p()
        _ok(lib.pn_rotary_create(ctypes.byref(h), ctypes.byref(desc)))
        self.h = h.value
        self._args = (rot_dim, base, layout, scaling, factor, original_length, beta_fast, beta_slow, attention_scale)

    def __reduce__(self):   # (a copy of the address alone would be destroyed twice)
        return type(self), self._args

    def __del__(self):
        try:
            if self.h:
                lib.pn_rotary_destroy(self.h)
                self.h = None
        except Exception:   # the interpreter is going down
            pass

    @staticmethod
    def _operands(q, k, positions):
        """(what k and the others are held to, key heads, rows of q and of k, address of positions)."""
        import torch
        like = nd, B, T, H, d, _, device = _first("q", q)
        K = k.shape[-2] if k.dim() == nd else 0
        if K > _INT:
            raise ValueError(f"k is {tuple(k.shape)}: sizes of up to 2^31 - 1 are taken")
        return (like, K, _heads("q", q, like, H, d), _heads("k", k, like, K, d),
                _ints("positions", positions, (B, T) if nd == 4 else (T,), torch.int64, device))

    @staticmethod
    def _out(q, k, like, K, out):
        nd, _, _, H, d, _, _ = like
        if out is None:
            import torch
            (oq, hq), (ok, hk) = _fresh(torch.empty_like(q), nd), _fresh(torch.empty_like(k), nd)
            return (oq, ok), hq, hk
        oq, ok = out
        return (oq, ok), _output("out[0]", oq, like, H, d), _output("out[1]", ok, like, K, d)

    def _rotate(self, q, k, positions, out, inverse):
        if q.requires_grad or k.requires_grad or out is not None:
            _no_graph(q, k, *(out or ()))
        like, K, hq, hk, pos = self._operands(q, k, positions)
        _, B, T, H, d, _, device = like
        out, oq, ok = self._out(q, k, like, K, out)
        keep, at = _rows(hq, hk, oq, ok)
        _ok(fast.pn_rotary_apply(self.h, _dtype("q", q), B, T, H, K, d, at[0], at[1], pos, inverse, at[2], at[3],
                                 _stream(device)))
        return out

    def apply(self, q, k, positions, out=None):
        """(q, k) rotated.  positions: int64, the shape of q without heads and dim.  ``out``: a pair of tensors, which may
        be (q, k) themselves and must overlap nothing else of the call."""
        return self._rotate(q, k, positions, out, 0)

    def apply_backward(self, dq, dk, positions, out=None):
        """Gradients of the inputs of :meth:`apply` from those of its outputs: the rotation by the opposite angles."""
        return self._rotate(dq, dk, positions, out, 1)

    def norm_apply(self, q, k, positions, wq, wk, eps: float = 1e-6, out=None):
        """x_j w_j / sqrt(mean(x^2) + eps) of each head vector, then the rotation, in one pass.  The weights are [dim],
        float32 or of the queries' type."""
        if q.requires_grad or k.requires_grad or wq.requires_grad or wk.requires_grad or out is not None:
            _no_graph(q, k, wq, wk, *(out or ()))
        like, K, hq, hk, pos = self._operands(q, k, positions)
        _, B, T, H, d, _, device = like
        w = _weights(wq, wk, d, device)
        out, oq, ok = self._out(q, k, like, K, out)
        keep, at = _rows(hq, hk, oq, ok)
        _ok(fast.pn_norm_rotary_apply(self.h, _dtype("q", q), B, T, H, K, d, at[0], at[1], pos, *w, eps, at[2], at[3],
                                      _stream(device)))
        return out

    def norm_backward(self, dq_out, dk_out, q, k, positions, wq, wk, eps: float = 1e-6, out=None):
        """(dq, dk, dwq, dwk) of :meth:`norm_apply`; dwq and dwk are float32 [dim].  ``out`` may be (dq_out, dk_out) and must
        overlap nothing else of the call."""
        import torch
        _no_graph(dq_out, dk_out, q, k, wq, wk, *(out or ()))
        like, K, hq, hk, pos = self._operands(q, k, positions)
        _, B, T, H, d, _, device = like
        gq, gk = _heads("dq_out", dq_out, like, H, d), _heads("dk_out", dk_out, like, K, d)
        w = _weights(wq, wk, d, device)
        out, oq, ok = self._out(q, k, like, K, out)
        dw = torch.empty((2, d), dtype=torch.float32, device=q.device)
        n = lib.pn_norm_rotary_workspace(B, T, H, K, d)
        keep_w, ws = _workspace(n, q.device)
        keep, at = _rows(gq, gk, hq, hk, oq, ok)
        at_w = dw.data_ptr()
        _ok(fast.pn_norm_rotary_backward(self.h, _dtype("q", q), B, T, H, K, d, *at[:4], pos, *w, eps, at[4], at[5], at_w,
                                         at_w + 4 * d, ws, n, _stream(device)))
        return out[0], out[1], dw[0], dw[1]


class LinearAttention:
    """Linear attention with a decay for each head: S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T, o_t = scale q_t S_t.

    heads, kv_heads   query heads, and key and value heads (query head h reads key head h // (heads / kv_heads))
    dk, dv            multiples of 8 up to 256
    log_decay         [heads], finite and <= 0, on the host or a device (read once, here; no gradient is formed for it)
    scale             None: dk ** -0.5
    dtype             of q, k, v and o: torch.float32, bfloat16 or float16; states are float32

    Sums and states are float32.  bfloat16 prompts and gradients of widths up to 128 and 64 rows times heads or more round the
    weights between rows and the state before each chunk of 64 rows to bfloat16 for the outputs: these are 0.0023 off in the
    mean square, where their own rounding makes 0.0017.  An infinite or NaN row makes outputs of its sequence and head
    undefined from up to 63 rows before it.

    Copies, pickled ones too, are handles of their own.
    """

    def __init__(self, heads: int, kv_heads: int, dk: int, dv: int, log_decay, scale: Optional[float] = None, dtype=None):
        import torch
        self.h = None
        self.heads, self.kv_heads = _int("heads", heads), _int("kv_heads", kv_heads)
        self.dk, self.dv = _int("dk", dk), _int("dv", dv)
        self.dtype = torch.float32 if dtype is None else dtype
        if self.dtype not in _dtypes():
            raise ValueError(f"dtype {dtype}: float32, bfloat16 or float16 is wanted")
        if isinstance(log_decay, torch.Tensor):
            if log_decay.requires_grad:
                raise ValueError("log_decay requires a gradient: the decays are fixed, detach it")
            log_decay = log_decay.to("cpu", torch.float32).numpy()   # (numpy has no bfloat16)
        g = np.ascontiguousarray(log_decay, dtype=np.float32)
        if g.shape != (self.heads,):
            raise ValueError(f"log_decay has shape {g.shape}; ({self.heads},) is wanted")
        self.scale = max(float(dk), 1.0) ** -0.5 if scale is None else float(scale)   # (a dk below 1 is refused below)
        h = ctypes.c_void_p()
        _ok(lib.pn_linattn_create(ctypes.byref(h), self.heads, self.kv_heads, self.dk, self.dv, _dtypes()[self.dtype],
                                  g.ctypes.data, self.scale))
        self.h = h.value
        self._args = (self.heads, self.kv_heads, self.dk, self.dv, g.copy(), self.scale, self.dtype)

    def __reduce__(self):   # (a copy of the address alone would be destroyed twice)
        return type(self), self._args

    def __del__(self):
        try:
            if self.h:
                lib.pn_linattn_destroy(self.h)
                self.h = None
        except Exception:   # the interpreter is going down
            pass

    def _operands(self, q, k, v):
        """What the others are held to, and the rows of q, k and v."""
        like = _first("q", q)
        if like[5] is not self.dtype:
            raise ValueError(f"q is {q.dtype}; {self.dtype} is wanted")
        return (like, _heads("q", q, like, self.heads, self.dk), _heads("k", k, like, self.kv_heads, self.dk),
                _heads("v", v, like, self.kv_heads, self.dv))

    def _sequences(self, like, cu_seqlens, max_len):
        """(n_seq, T, address of cu_seqlens, max_len) of the rows."""
        import torch
        nd, B, T, _, _, _, device = like
        if cu_seqlens is None:
            return B, T, None, 0
        if nd != 3:
            raise ValueError("packed sequences (cu_seqlens) are [tokens, heads, dim]")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be [sequences + 1]")
        return (_int("sequences", cu_seqlens.numel() - 1), T, _ints("cu_seqlens", cu_seqlens, cu_seqlens.shape, torch.int32, device),
                int(max_len or 0))

    def _empty(self, q, nd):
        import torch
        return _fresh(torch.empty_like(q) if self.dv == self.dk else q.new_empty(q.shape[:-1] + (self.dv,)), nd)

    def forward(self, q, k, v, initial_state=None, cu_seqlens=None, max_len: Optional[int] = None, out=None):
        """(o, final state) of whole sequences.

        q [batch, tokens, heads, dk], k and v with kv_heads; or, with ``cu_seqlens`` (int32 [sequences + 1], on the
        device), packed [rows, heads, dk], where rows before the first and behind the last sequence are neither read nor
        written.  ``max_len``: the longest sequence, a hint for the work's split.  States: float32
        [sequences, heads, dk, dv].  ``out``: a tensor for o, which overlaps no input."""
        import torch
        _no_graph(q, k, v, initial_state, out)
        like, hq, hk, hv = self._operands(q, k, v)
        n, T, cu, max_len = self._sequences(like, cu_seqlens, max_len)
        shape, device = (n, self.heads, self.dk, self.dv), like[-1]
        s0 = _float32("initial_state", initial_state, shape, device)
        state = q.new_empty(shape, dtype=torch.float32) if s0 is None else torch.empty_like(initial_state)
        if out is None:
            out, ho = self._empty(q, like[0])
        else:
            ho = _output("out", out, like, self.heads, self.dv)
        size = lib.pn_linattn_workspace(self.h, 0, n, T, cu is not None, max_len)
        keep_w, ws = _workspace(size, q.device)
        keep, at = _rows(hq, hk, hv, ho)
        _ok(fast.pn_linattn_forward(self.h, n, T, cu, max_len, *at[:3], s0, at[3], state.data_ptr(), ws, size, _stream(device)))
        return out, state

    def backward(self, do, q, k, v, initial_state=None, dstate=None, cu_seqlens=None, max_len: Optional[int] = None,
                 grads=None):
        """(dq, dk, dv, gradient of the initial state) of :meth:`forward` with the same inputs, from the gradients of o
        and (None: zero) of the final state.  ``grads``: a triple of tensors for dq, dk and dv, which overlap neither each
        other nor an input."""
        import torch
        _no_graph(do, q, k, v, initial_state, dstate, *(grads or ()))
        like, hq, hk, hv = self._operands(q, k, v)
        n, T, cu, max_len = self._sequences(like, cu_seqlens, max_len)
        shape, device = (n, self.heads, self.dk, self.dv), like[-1]
        hdo = _heads("do", do, like, self.heads, self.dv)
        s0 = _float32("initial_state", initial_state, shape, device)
        ds = _float32("dstate", dstate, shape, device)
        if grads is None:
            grads, outs = zip(*[_fresh(torch.empty_like(t), like[0]) for t in (q, k, v)])
        else:
            sizes = ((self.heads, self.dk), (self.kv_heads, self.dk), (self.kv_heads, self.dv))
            outs = [_output(f"grads[{i}]", g, like, *size) for i, (g, size) in enumerate(zip(grads, sizes))]
        ds0 = q.new_empty(shape, dtype=torch.float32)
        size = lib.pn_linattn_workspace(self.h, 1, n, T, cu is not None, max_len)
        keep_w, ws = _workspace(size, q.device)
        keep, at = _rows(hdo, hq, hk, hv, *outs)
        _ok(fast.pn_linattn_backward(self.h, n, T, cu, max_len, *at[:4], s0, ds, *at[4:], ds0.data_ptr(), ws, size,
                                     _stream(device)))
        return (*grads, ds0)

    @staticmethod
    def check(device=None):
        """Wait for the current stream and raise where a bounded device wait of a forward or backward pass on the device, in any
        stream, has given up since the last check of this stream (results are invalid).  The passes are asynchronous and
        cannot tell."""
        import torch
        with torch.cuda.device(device):
            _ok(lib.pn_linattn_check(torch.cuda.current_stream().cuda_stream))

    def step(self, q, k, v, states, slots=None, rotary: Optional[Rotary] = None, positions=None, wq=None, wk=None,
             eps: float = 1e-6, out=None):
        """o [rows, heads, dv] of one token of each of the rows; ``states`` [slots, heads, dk, dv] is updated in place.

        q [rows, heads, dk], k and v with kv_heads.  ``slots``: int64 [rows], the state of each row (None: row b has
        state b); a slot outside the states, or one that an earlier row names, makes its row padding, which is left as it
        is (in ``out`` too, which overlaps no other argument; without ``out`` such rows are undefined).  ``wq``, ``wk``: the
        norm of q and k, ``rotary`` with ``positions`` (int64 [rows]): their rotation, both in the same pass."""
        import torch
        _no_graph(q, k, v, states, wq, wk, out)
        if q.dim() != 3:
            raise ValueError("q must be [rows, heads, dk]")
        like, hq, hk, hv = self._operands(q, k, v)
        rows, device = like[2], like[-1]
        if out is None:
            out, ho = self._empty(q, 3)
        else:
            ho = _output("out", out, like, self.heads, self.dv)
        if states.dim() != 4:
            raise ValueError("states must be [slots, heads, dk, dv]")
        n = states.shape[0]
        st = _float32("states", states, (n, self.heads, self.dk, self.dv), device)
        sl = None if slots is None else _ints("slots", slots, (rows,), torch.int64, device)
        if (wq is None) != (wk is None):
            raise ValueError("wq and wk come together")
        w = (None, None, PN_F32) if wq is None else _weights(wq, wk, self.dk, device)
        if (rotary is None) != (positions is None):
            raise ValueError("rotary and positions come together")
        turn, pos = None, None
        if rotary is not None:
            turn, pos = rotary.h, _ints("positions", positions, (rows,), torch.int64, device)
        # rows lie at the batch stride
        keep, at = _rows(*[(p, y, 0, z) for p, _, y, z in (hq, hk, hv, ho)])
        _ok(fast.pn_linattn_step(self.h, rows, *at, st, n, sl, turn, pos, *w, eps, _stream(device)))
        return out
