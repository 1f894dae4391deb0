"""Cases of the sequence-layer operators: rotary positions, norms of queries and keys with the rotation, and linear
attention with a decay for each head, each in its plain form and through the library's entry points.

A case is a dict of plain values.  ``prepare`` makes its inputs on the GPU from a seed, ``run`` makes one pass (the
plain form, or with ``own`` the library's calls), ``exact`` gives the same outputs in 64 bits from the definitions, and
``work`` counts the bytes and operations a pass cannot do without.

Definitions, for query head h and its key head h' = h // (heads / kv_heads):

  rotation   pair i of a head vector, position p:  (a, b) -> m (a cos w - b sin w, b cos w + a sin w),  w = p f_i
  norm       y_j = x_j w_j / sqrt(mean(x^2) + eps), then the rotation
  attention  S_t = exp(g_h) S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t,   g_h <= 0
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
CHUNK = 64   # steps per chunk of the plain form of linear attention


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one token of one conversation: the rotation's smallest call
        dict(name="rope_token", op="rope", direction="forward", dtype="bf16", batch=1, tokens=1, heads=32, kv_heads=8,
             dim=128, rot=128, layout="half", scaling="none", factor=1.0, start=5000, packed=False),
        # a long prompt far into a stretched context, rotation of half of the head
        dict(name="rope_prompt", op="rope", direction="forward", dtype="bf16", batch=1, tokens=65536, heads=16,
             kv_heads=4, dim=128, rot=64, layout="interleaved", scaling="yarn", factor=16.0, start=1000000,
             packed=False),
        # training in single precision with odd sizes: the rotation's gradient
        dict(name="rope_gradient", op="rope", direction="backward", dtype="fp32", batch=3, tokens=2045, heads=12,
             kv_heads=12, dim=80, rot=40, layout="half", scaling="linear", factor=4.0, start=0, packed=False),
        # a decoding batch: one token for each of 64 conversations
        dict(name="norm_rope_tokens", op="norm", direction="forward", dtype="fp16", batch=64, tokens=1, heads=32,
             kv_heads=8, dim=64, rot=64, layout="half", scaling="ntk", factor=4.0, start=700, packed=True),
        # prompts, queries and keys lying in the output of one projection
        dict(name="norm_rope_prompt", op="norm", direction="forward", dtype="bf16", batch=4, tokens=4096, heads=32,
             kv_heads=8, dim=128, rot=128, layout="half", scaling="none", factor=1.0, start=0, packed=True),
        # the same in training: gradients of queries, keys and both weights
        dict(name="norm_rope_gradient", op="norm", direction="backward", dtype="bf16", batch=4, tokens=4096, heads=32,
             kv_heads=8, dim=128, rot=128, layout="half", scaling="none", factor=1.0, start=0, packed=True),
        # one token of one conversation through the recurrence
        dict(name="step_token", op="step", dtype="bf16", batch=1, heads=16, kv_heads=16, dk=128, dv=128, slots=4,
             rotate=False),
        # a decoding batch, its states at their slots of a pool, norm and rotation in the same pass
        dict(name="step_batch", op="step", dtype="bf16", batch=192, heads=32, kv_heads=8, dk=128, dv=128, slots=200,
             rotate=True),
        # a few short prompts in single precision, values wider than keys
        dict(name="prompt_short", op="linear", direction="forward", dtype="fp32", ragged=True, batch=7, tokens=1500,
             heads=8, kv_heads=4, dk=64, dv=96),
        # a serving batch of prompts of different lengths, packed
        dict(name="prompt_ragged", op="linear", direction="forward", dtype="bf16", ragged=True, batch=16, tokens=32768,
             heads=32, kv_heads=8, dk=128, dv=128),
        # one long document with few, narrow heads
        dict(name="prompt_long", op="linear", direction="forward", dtype="bf16", ragged=False, batch=1, tokens=65536,
             heads=16, kv_heads=16, dk=64, dv=64),
        # a training batch: all gradients
        dict(name="train_gradient", op="linear", direction="backward", dtype="bf16", ragged=False, batch=4,
             tokens=4096, heads=16, kv_heads=16, dk=128, dv=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    kv = rng.choice([1, 2, 3, 4, 8])
    heads = kv * rng.choice([1, 1, 2, 4])
    op = rng.choice(["rope", "norm", "step", "linear", "linear"])
    if op in ("rope", "norm"):
        dim = rng.choice([32, 64, 72, 80, 96, 128, 128, 256])
        rot = dim if rng.random() < 0.6 else 8 * rng.randint(1, dim // 8)
        batch = _log(rng, 1, 64)
        tokens = _log(rng, 1, max(1, min(65536, 100_000_000 // (batch * (heads + kv) * dim))))
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return dict(op=op, direction=rng.choice(["forward", "backward"]), dtype=dtype, batch=batch, tokens=tokens,
                    heads=heads, kv_heads=kv, dim=dim, rot=rot, layout=rng.choice(["half", "interleaved"]),
                    scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]),
                    start=_log(rng, 1, 4000000) - 1, packed=rng.random() < 0.5)
    dk = rng.choice([32, 64, 64, 80, 96, 128, 128])
    dv = dk if rng.random() < 0.6 else rng.choice([32, 64, 96, 128, 160, 256])
    if op == "step":
        batch = _log(rng, 1, 256)
        batch = max(1, min(batch, 90_000_000 // (heads * dk * dv)))
        return dict(op=op, dtype=dtype, batch=batch, heads=heads, kv_heads=kv, dk=dk, dv=dv,
                    slots=batch + rng.randint(0, 9), rotate=rng.random() < 0.5)
    most = 32768 * 32 * 256 // 4 if dtype != "fp32" else 32768 * 32 * 256 // 16
    ragged = rng.random() < 0.5
    batch = _log(rng, 1, 16)
    tokens = _log(rng, 1, max(1, min(65536, most // (heads * (dk + dv)))))
    if not ragged:
        tokens = max(1, tokens // batch)
    return dict(op=op, direction=rng.choice(["forward", "backward"]), dtype=dtype, ragged=ragged, batch=batch,
                tokens=tokens, heads=heads, kv_heads=kv, dk=dk, dv=dv)


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------

def _lengths(case, seed):
    """Lengths of a ragged batch: uneven, an empty sequence among several, and some rows behind the last one."""
    n, total = case["batch"], case["tokens"]
    rng = random.Random(seed * 7919 + 17)
    total -= min(total // 16, 5)   # rows of the buffer that belong to no sequence
    if n == 1:
        return [total]
    weights = [rng.uniform(0.1, 1.0) for _ in range(n)]
    weights[rng.randrange(n)] = 0.0
    lens = [int(total * w / sum(weights)) for w in weights]
    lens[max(range(n), key=lambda i: lens[i])] += total - sum(lens)
    return lens


def _log_decay(heads):
    """log(1 - 2^-x), x from 1 to 11 over the heads: memories from two steps to two thousand."""
    x = torch.linspace(1.0, 11.0, heads, dtype=torch.float64) if heads > 1 else torch.tensor([6.0], dtype=torch.float64)
    return torch.log1p(-torch.exp2(-x)).float()


def _rotary(rot, layout, scaling, factor):
    import newton_evaluation_nonlinear_b200 as pn
    return pn.Rotary(rot, base=10000.0, layout=layout, scaling=scaling, factor=factor, original_length=4096)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype = TYPES[case["dtype"]]

    def normal(*shape, dtype=dtype):
        return torch.randn(*shape, device="cuda", dtype=torch.float32, generator=gen).to(dtype)

    op, H, K = case["op"], case["heads"], case["kv_heads"]
    s = {"case": case}
    if op in ("rope", "norm"):
        B, T, d = case["batch"], case["tokens"], case["dim"]
        if case["packed"]:   # queries, keys and values side by side, as one projection leaves them
            qkv = normal(B, T, H + 2 * K, d)
            s["q"], s["k"] = qkv[:, :, :H], qkv[:, :, H:H + K]
        else:
            s["q"], s["k"] = normal(B, T, H, d), normal(B, T, K, d)
        s["positions"] = (torch.arange(T, device="cuda")[None] + case["start"]
                          + torch.randint(0, 50, (B, 1), device="cuda", generator=gen))
        if case["direction"] == "backward":
            s["dq"], s["dk"] = normal(B, T, H, d), normal(B, T, K, d)
        if op == "norm":
            s["wq"], s["wk"] = 1 + 0.1 * normal(d), 1 + 0.1 * normal(d)
        if own:
            s["rotary"] = _rotary(case["rot"], case["layout"], case["scaling"], case["factor"])
        return s
    dk, dv = case["dk"], case["dv"]
    s["log_decay"] = _log_decay(H)
    s["g"] = s["log_decay"].cuda()
    s["scale"] = dk ** -0.5
    if op == "step":
        B = case["batch"]
        s["q"], s["k"], s["v"] = normal(B, H, dk), normal(B, K, dk), normal(B, K, dv)
        s["states"] = 4.0 * normal(case["slots"], H, dk, dv, dtype=torch.float32)
        s["slots"] = torch.randperm(case["slots"], device="cuda", generator=gen)[:B]
        if case["rotate"]:
            s["positions"] = torch.randint(0, 30000, (B,), device="cuda", generator=gen)
            s["wq"], s["wk"] = 1 + 0.1 * normal(dk), 1 + 0.1 * normal(dk)
            s["rotary"] = _rotary(dk, "half", "none", 1.0) if own else None
    else:
        B, T = case["batch"], case["tokens"]
        lead = (T,) if case["ragged"] else (B, T)
        s["q"], s["k"], s["v"] = normal(*lead, H, dk), normal(*lead, K, dk), normal(*lead, K, dv)
        s["lens"] = _lengths(case, int(seed)) if case["ragged"] else [T] * B
        s["max_len"] = max(s["lens"])
        s["cu"] = torch.tensor([sum(s["lens"][:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
        s["s0"] = normal(B, H, dk, dv, dtype=torch.float32)
        if case["direction"] == "backward":
            s["do"] = normal(*lead, H, dv)
            s["ds"] = normal(B, H, dk, dv, dtype=torch.float32)
    if own:
        import newton_evaluation_nonlinear_b200 as pn
        s["attention"] = pn.LinearAttention(H, K, dk, dv, s["log_decay"], scale=s["scale"], dtype=dtype)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# the plain forms, in 32 bits
# ---------------------------------------------------------------------------------------------------------------------

def _frequencies(rot, scaling, factor, original=4096, fast=32.0, slow=1.0):
    """Angle per position of each pair, in 64 bits, and the factor on the rotated vector."""
    base = 10000.0
    if scaling == "ntk":
        base *= factor ** (rot / (rot - 2))
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        keep = ((original * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        return f * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _rotate(x, positions, case, sign=1.0):
    """x [..., heads, d] in 32 bits, its first `rot` values turned by the angles of its row's position (taken in 64)."""
    rot = case["rot"]
    f, m = _frequencies(rot, case["scaling"], case["factor"])
    w = positions.double()[..., None, None] * f
    cos, sin = (m * w.cos()).float(), (sign * m * w.sin()).float()
    if case["layout"] == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


EPS = 1e-6


def _norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _norm_gradient(dy, x, w):
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    dn = dy * w
    return r * (dn - n * (dn * n).mean(-1, keepdim=True)), (dy * n).flatten(0, -2).sum(0)


def _plain_heads(s):
    case = s["case"]
    q, k, p = s["q"].float(), s["k"].float(), s["positions"]
    dtype = s["q"].dtype
    if case["op"] == "rope":
        if case["direction"] == "forward":
            return {"q": _rotate(q, p, case).to(dtype), "k": _rotate(k, p, case).to(dtype)}
        return {"dq": _rotate(s["dq"].float(), p, case, -1.0).to(dtype),
                "dk": _rotate(s["dk"].float(), p, case, -1.0).to(dtype)}
    wq, wk = s["wq"].float(), s["wk"].float()
    if case["direction"] == "forward":
        return {"q": _rotate(_norm(q, wq), p, case).to(dtype), "k": _rotate(_norm(k, wk), p, case).to(dtype)}
    dq, dwq = _norm_gradient(_rotate(s["dq"].float(), p, case, -1.0), q, wq)
    dk, dwk = _norm_gradient(_rotate(s["dk"].float(), p, case, -1.0), k, wk)
    return {"dq": dq.to(dtype), "dk": dk.to(dtype), "dwq": dwq, "dwk": dwk}


def _plain_step(s):
    case, slots = s["case"], s["slots"]
    G = case["heads"] // case["kv_heads"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if case["rotate"]:
        how = dict(rot=case["dk"], layout="half", scaling="none", factor=1.0)
        q = _rotate(_norm(q, s["wq"].float()), s["positions"], how)
        k = _rotate(_norm(k, s["wk"].float()), s["positions"], how)
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    S = s["g"].exp()[:, None, None] * s["states"][slots] + k[..., None] * v[..., None, :]
    s["states"][slots] = S
    o = s["scale"] * (q[..., None] * S).sum(-2)
    return {"o": o.to(s["q"].dtype), "states": s["states"]}


def _chunks(s, names):
    """The rows of each sequence, padded with zeros to whole chunks, in 32 bits: [B, chunks, CHUNK, heads, d]."""
    case = s["case"]
    n = max(1, -(-s["max_len"] // CHUNK))
    t = torch.arange(n * CHUNK, device="cuda")
    lens = s["cu"].diff().long()
    valid = t[None] < lens[:, None]
    at = (s["cu"][:-1, None].long() + t[None]).clamp(max=max(0, sum(s["lens"]) - 1))
    G = case["heads"] // case["kv_heads"]
    got = []
    for name in names:
        x = s[name] if case["ragged"] else s[name].flatten(0, 1)
        x = torch.where(valid[..., None, None], x[at].float(), 0.0)
        if name in ("k", "v") and G > 1:
            x = x.repeat_interleave(G, 2)
        got.append(x.unflatten(1, (n, CHUNK)))
    return got, lens, valid, at


def _powers(g, n):
    """exp(g_h n) for the exponents n >= 0, zero where n < 0, the exponent taken in 64 bits: [H, ...]."""
    e = g.double().view(-1, *([1] * n.dim())) * n.double().clamp(min=0)
    return torch.where(n >= 0, e.exp(), 0.0).float()


def _scan(q, k, v, g, s0):
    """Outputs of the recurrence by chunks (forward in time), and what leaves each chunk for the next ones."""
    n = q.shape[1]
    i = torch.arange(CHUNK, device="cuda")
    c = torch.arange(n, device="cuda")
    inside = _powers(g, i[:, None] - i[None])                                       # [H, C, C]
    a = torch.einsum("bcihd,bcjhd->bchij", q, k) * inside[None, None]
    o = torch.einsum("bchij,bcjhe->bcihe", a, v)
    kw = k * _powers(g, CHUNK - 1 - i).t()[None, None, :, :, None]
    left = torch.einsum("bcjhd,bcjhe->bchde", kw, v)
    S = torch.einsum("hcx,bxhde->bchde", _powers(g, CHUNK * (c[:, None] - 1 - c[None])), left)
    S = S + _powers(g, CHUNK * c).t()[None, :, :, None, None] * s0[:, None]
    qw = q * _powers(g, 1 + i).t()[None, None, :, :, None]
    return o + torch.einsum("bcihd,bchde->bcihe", qw, S)


def _scan_back(q, k, v, g, s0, lens):
    """The same against time: row i takes rows j >= i of its sequence, and s0 from behind the last row."""
    n = q.shape[1]
    i = torch.arange(CHUNK, device="cuda")
    c = torch.arange(n, device="cuda")
    a = torch.einsum("bcihd,bcjhd->bchij", q, k) * _powers(g, i[None] - i[:, None])[None, None]
    o = torch.einsum("bchij,bcjhe->bcihe", a, v)
    left = torch.einsum("bcjhd,bcjhe->bchde", k * _powers(g, i).t()[None, None, :, :, None], v)
    S = torch.einsum("hcx,bxhde->bchde", _powers(g, CHUNK * (c[None] - 1 - c[:, None])), left)
    qw = q * _powers(g, CHUNK - i).t()[None, None, :, :, None]
    o = o + torch.einsum("bcihd,bchde->bcihe", qw, S)
    t = torch.arange(n * CHUNK, device="cuda")
    far = _powers(g, lens[:, None] - 1 - t[None]).permute(1, 2, 0).unflatten(1, (n, CHUNK))
    return o + torch.einsum("bcihd,bhde->bcihe", q * far[..., None], s0)


def _plain_linear(s):
    case, g, dtype = s["case"], s["g"], s["q"].dtype
    H, K = case["heads"], case["kv_heads"]
    back = case["direction"] == "backward"
    (q, k, v, *do), lens, valid, at = _chunks(s, ["q", "k", "v"] + ["do"] * back)

    def rows(x, heads):
        """[B, chunks, CHUNK, heads, d] back to the rows of the input; rows of no sequence are zero."""
        x = x.flatten(1, 2)
        if heads < H:
            x = x.unflatten(2, (heads, H // heads)).sum(3)
        if not case["ragged"]:
            return x[:, : case["tokens"]].to(dtype)
        out = torch.zeros(case["tokens"] + 1, heads, x.shape[-1], device="cuda")
        out[torch.where(valid, at, case["tokens"])] = x
        return out[:-1].to(dtype)

    end = lens[:, None] - 1 - torch.arange(q.shape[1] * CHUNK, device="cuda")[None]
    last = _powers(g, end).permute(1, 2, 0)                                         # [B, t, H]: decay to the last row
    whole = _powers(g, lens).t()[..., None, None]
    if not back:
        o = s["scale"] * _scan(q, k, v, g, s["s0"])
        kw = k.flatten(1, 2) * last[..., None]
        state = whole * s["s0"] + torch.einsum("bthd,bthe->bhde", kw, v.flatten(1, 2))
        return {"o": rows(o, H), "state": state}
    do = s["scale"] * do[0]
    dq = _scan(do, v, k, g, s["s0"].transpose(-1, -2))
    dk = _scan_back(v, do, q, g, s["ds"].transpose(-1, -2), lens)
    dv = _scan_back(k, q, do, g, s["ds"], lens)
    first = _powers(g, 1 + torch.arange(q.shape[1] * CHUNK, device="cuda")).t()[None, :, :, None]
    ds0 = whole * s["ds"] + torch.einsum("bthd,bthe->bhde", q.flatten(1, 2) * first, do.flatten(1, 2))
    return {"dq": rows(dq, H), "dk": rows(dk, K), "dv": rows(dv, K), "ds0": ds0}


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------

def run(s):
    case = s["case"]
    if not own:
        return {"rope": _plain_heads, "norm": _plain_heads, "step": _plain_step, "linear": _plain_linear}[case["op"]](s)
    if case["op"] == "rope":
        if case["direction"] == "forward":
            q, k = s["rotary"].apply(s["q"], s["k"], s["positions"])
            return {"q": q, "k": k}
        dq, dk = s["rotary"].apply_backward(s["dq"], s["dk"], s["positions"])
        return {"dq": dq, "dk": dk}
    if case["op"] == "norm":
        if case["direction"] == "forward":
            q, k = s["rotary"].norm_apply(s["q"], s["k"], s["positions"], s["wq"], s["wk"], EPS)
            return {"q": q, "k": k}
        dq, dk, dwq, dwk = s["rotary"].norm_backward(s["dq"], s["dk"], s["q"], s["k"], s["positions"], s["wq"],
                                                     s["wk"], EPS)
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    if case["op"] == "step":
        how = dict(rotary=s["rotary"], positions=s["positions"], wq=s["wq"], wk=s["wk"], eps=EPS) if case["rotate"] else {}
        return {"o": s["attention"].step(s["q"], s["k"], s["v"], s["states"], slots=s["slots"], **how),
                "states": s["states"]}
    how = dict(initial_state=s["s0"])
    if case["ragged"]:
        how.update(cu_seqlens=s["cu"], max_len=s["max_len"])
    if case["direction"] == "forward":
        out = torch.zeros(*s["q"].shape[:-1], case["dv"], device="cuda", dtype=s["q"].dtype) if case["ragged"] else None
        o, state = s["attention"].forward(s["q"], s["k"], s["v"], out=out, **how)
        return {"o": o, "state": state}
    grads = None
    if case["ragged"]:   # rows of no sequence are left as they are
        grads = (torch.zeros_like(s["q"]), torch.zeros_like(s["k"]), torch.zeros_like(s["v"]))
    dq, dk, dv, ds0 = s["attention"].backward(s["do"], s["q"], s["k"], s["v"], dstate=s["ds"], grads=grads, **how)
    return {"dq": dq, "dk": dk, "dv": dv, "ds0": ds0}


def work(case):
    size, H, K = SIZE[case["dtype"]], case["heads"], case["kv_heads"]
    if case["op"] in ("rope", "norm"):
        rows = case["batch"] * case["tokens"]
        values = rows * (H + K) * case["dim"]
        gradient = case["op"] == "norm" and case["direction"] == "backward"
        more = case["dim"] * size * 2 if case["op"] == "norm" else 0
        return {"bytes": (3 if gradient else 2) * values * size + 8 * rows + more + (8 * case["dim"] if gradient else 0),
                "flops": values * (12 if gradient else 7 if case["op"] == "norm" else 3)}
    dk, dv = case["dk"], case["dv"]
    if case["op"] == "step":
        row = (H * dk + K * dk + K * dv + H * dv) * size
        return {"bytes": case["batch"] * (8 * H * dk * dv + row + 8), "flops": case["batch"] * 5 * H * dk * dv}
    rows = case["tokens"] * (1 if case["ragged"] else case["batch"])
    if case["direction"] == "forward":
        row, per = H * dk + K * (dk + dv) + H * dv, 4
    else:
        row, per = 2 * H * dk + 2 * K * (dk + dv) + H * dv, 10
    states = case["batch"] * H * dk * dv * 4 * (2 if case["direction"] == "forward" else 3)
    return {"bytes": rows * row * size + states, "flops": rows * H * dk * dv * per}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------

def _turns(case, positions, back=False):
    """The rotation of each (row, pair) as a complex number."""
    rot, factor = case["rot"], case["factor"]
    spread = math.log(10000.0)
    if case["scaling"] == "ntk":
        spread += math.log(factor) * rot / (rot - 2)
    pace, size = [], 1.0
    for i in range(rot // 2):
        f = math.exp(-spread * 2 * i / rot)
        if case["scaling"] == "linear":
            f /= factor
        elif case["scaling"] == "yarn":
            turns = 4096 * f / (2 * math.pi)
            share = min(1.0, max(0.0, (turns - 1.0) / 31.0))
            f = share * f + (1.0 - share) * f / factor
        pace.append(f)
    if case["scaling"] == "yarn":
        size = 1.0 + 0.1 * math.log(factor)
    w = positions.to(torch.float64)[..., None, None] * torch.tensor(pace, dtype=torch.float64, device="cuda")
    return torch.polar(torch.full_like(w, size), -w if back else w)


def _turned(x, z, case):
    """x in 64 bits with its pairs, as complex numbers, multiplied by z."""
    rot, y = case["rot"], x.clone()
    if case["layout"] == "half":
        p = torch.complex(x[..., : rot // 2], x[..., rot // 2: rot]) * z
        y[..., : rot // 2], y[..., rot // 2: rot] = p.real, p.imag
    else:
        p = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * z
        y[..., 0:rot:2], y[..., 1:rot:2] = p.real, p.imag
    return y


def _unit(x):
    return x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()


def _exact_heads(s, case):
    out = {}
    back = case["direction"] == "backward"
    z = _turns(case, s["positions"], back)
    for name in ("q", "k"):
        x = s[name].double()
        if case["op"] == "rope":
            out["d" + name if back else name] = _turned(s["d" + name].double() if back else x, z, case)
            continue
        w = s["w" + name].double()
        if not back:
            out[name] = _turned(_unit(x) * w, z, case)
            continue
        t = _turned(s["d" + name].double(), z, case)
        n = _unit(x)
        rms = (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
        u = t * w
        out["d" + name] = (u - n * (u * n).sum(-1, keepdim=True) / x.shape[-1]) / rms
        out["dw" + name] = (t * n).sum((0, 1, 2))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rope", "norm"):
        return _exact_heads(s, case)
    H, G = case["heads"], case["heads"] // case["kv_heads"]
    decay = s["log_decay"].double().exp().cuda()[:, None, None]
    share = torch.arange(H, device="cuda") // G   # the key head of each head
    scale = float(s["scale"])
    if case["op"] == "step":
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        if case["rotate"]:
            how = dict(rot=case["dk"], layout="half", scaling="none", factor=1.0)
            z = _turns(how, s["positions"])
            q, k = _turned(_unit(q) * s["wq"].double(), z, how), _turned(_unit(k) * s["wk"].double(), z, how)
        states = s["states"].double()
        S = states[s["slots"]] * decay + k[:, share].unsqueeze(-1) * v[:, share].unsqueeze(-2)
        states[s["slots"]] = S
        return {"o": scale * torch.matmul(q.unsqueeze(-2), S).squeeze(-2), "states": states}
    lens = torch.tensor(s["lens"], device="cuda")
    start, longest = s["cu"][:-1].long(), s["max_len"]
    flat = {n: (s[n] if case["ragged"] else s[n].flatten(0, 1)).double() for n in ("q", "k", "v", "do") if n in s}
    rows = flat["q"].shape[0]
    for n in flat:   # one row of zeros behind all others
        flat[n] = torch.cat([flat[n], torch.zeros_like(flat[n][:1])]) if rows else flat[n].new_zeros(1, *flat[n].shape[1:])
    back = case["direction"] == "backward"
    wide = {"o": case["dv"]} if not back else {"dq": case["dk"], "dk": case["dk"], "dv": case["dv"]}
    out = {n: torch.zeros(rows + 1, H, d, dtype=torch.float64, device="cuda") for n, d in wide.items()}
    t = torch.arange(max(longest, 1), device="cuda")[:, None]
    at = torch.where(t < lens, start + t, rows)                       # [t, B]: the row of each step, or the row of zeros
    live = (t < lens).double()[..., None, None, None]
    S = s["s0"].double()
    for n in range(longest):
        r = at[n]
        k, v = flat["k"][r][:, share], flat["v"][r][:, share]
        S = torch.where(live[n] > 0, S * decay + k.unsqueeze(-1) * v.unsqueeze(-2), S)
        if back:
            out["dq"][r] = scale * torch.matmul(S, flat["do"][r].unsqueeze(-1)).squeeze(-1)
        else:
            out["o"][r] = scale * torch.matmul(flat["q"][r].unsqueeze(-2), S).squeeze(-2)
    if back:
        S = s["ds"].double()   # the gradient of the state, against time
        for n in reversed(range(longest)):
            r = at[n]
            here = S + scale * flat["q"][r].unsqueeze(-1) * flat["do"][r].unsqueeze(-2)
            out["dk"][r] = torch.matmul(here, flat["v"][r][:, share].unsqueeze(-1)).squeeze(-1)
            out["dv"][r] = torch.matmul(flat["k"][r][:, share].unsqueeze(-2), here).squeeze(-2)
            S = torch.where(live[n] > 0, here * decay, S)
    for n in out:
        x = out[n][:-1]
        if n in ("dk", "dv") and G > 1:
            x = x.unflatten(1, (H // G, G)).sum(2)
        out[n] = x if case["ragged"] else x.unflatten(0, (case["batch"], case["tokens"]))
    return {**out, ("ds0" if back else "state"): S}
