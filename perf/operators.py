"""Cases of the gated linear recurrence and of the layer norm, with their plain forms.

The gated recurrence has one real state per channel,

    w_t = c softplus(lam) sigmoid(r_t),  a_t = exp(-w_t),  beta_t = sqrt(1 - a_t^2),
    h_t = a_t h_{t-1} + beta_t sigmoid(i_t) x_t,  y_t = h_t

(at a reset, where a new document begins, a_t = 0 and beta_t = 1). The layer norm
normalises the rows of s = x + residual, the residual stream being kept in float32.

`run` computes a case in plain torch operations, or, where `own` is true, through the
library's entry points; `exact` gives the same outputs in 64 bits from the definitions,
step by step.
"""
import math

import torch

own = False

_C = 8.0
_EPS = 1e-5
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}

# No more elements than these in a drawn case (the largest listed ones have as many).
_MOST = {"scan": 262144 * 5120, "train": 8 * 4096 * 2048, "step": 256 * 5120, "norm": 32768 * 2048,
         "norm_train": 32768 * 2048}


def _recurrence(name, op, batch, seqlen, dim, dtype, reset=False, h0=False, last=False, sliced=False):
    return {"name": name, "op": op, "batch": batch, "seqlen": seqlen, "dim": dim, "dtype": dtype, "reset": reset,
            "h0": h0, "last": last, "sliced": sliced}


def _norm(name, op, rows, dim, dtype, residual, bias):
    return {"name": name, "op": op, "rows": rows, "dim": dim, "dtype": dtype, "residual": residual, "bias": bias}


def listed():
    return [
        # A short prompt continued from a kept state, in float32: latency counts.
        _recurrence("scan_tiny", "scan", 1, 256, 64, "f32", h0=True, last=True),
        # Documents packed into one long row of a narrow layer, the gates being slices of one projection.
        _recurrence("scan_packed", "scan", 1, 131071, 1030, "bf16", reset=True, last=True, sliced=True),
        # The long-context layer.
        _recurrence("scan_long", "scan", 1, 262144, 5120, "bf16", last=True),
        # A training pass of a small layer.
        _recurrence("train_small", "train", 4, 2048, 1536, "bf16"),
        # A training pass over a piece of longer documents, in float32, odd sizes.
        _recurrence("train_ragged", "train", 2, 1023, 517, "f32", reset=True, h0=True, last=True),
        # A training pass of a middle-sized layer.
        _recurrence("train_mid", "train", 8, 4096, 2048, "bf16"),
        # One token of one sequence, and of a batch of 256.
        _recurrence("step_one", "step", 1, 1, 2048, "bf16"),
        _recurrence("step_batch", "step", 256, 1, 5120, "bf16"),
        # The norm in front of the mixer while decoding a batch, behind the residual sum.
        _norm("norm_decode", "norm", 256, 5120, "bf16", True, True),
        # The same over a prompt.
        _norm("norm_prompt", "norm", 32768, 2048, "bf16", True, False),
        # Training passes: a middle-sized layer, and an odd-sized one in float32 without a residual.
        _norm("norm_train_mid", "norm_train", 32768, 2048, "bf16", True, True),
        _norm("norm_train_ragged", "norm_train", 1023, 517, "f32", False, True),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "train", "train", "step", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    most = _MOST[op] * 2 // _SIZE[dtype]
    if op in ("norm", "norm_train"):
        dim = _spread(rng, 16, 8192)
        return _norm("drawn", op, _spread(rng, 1, min(32768, most // dim)), dim, dtype, rng.random() < 0.5,
                     rng.random() < 0.5)
    dim = _spread(rng, 1, 5120)
    if op == "step":
        return _recurrence("drawn", op, _spread(rng, 1, min(256, most // dim)), 1, dim, dtype,
                           sliced=rng.random() < 0.5)
    batch = _spread(rng, 1, 8)
    seqlen = _spread(rng, 1, min(262144 if op == "scan" else 16384, most // (dim * batch)))
    flip = [rng.random() < 0.5 for _ in range(4)]
    return _recurrence("drawn", op, batch, seqlen, dim, dtype, *flip)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    gen = torch.Generator(device=dev).manual_seed(seed)
    tok = _TYPES[case["dtype"]]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=dev, dtype=dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    s = {"op": case["op"], "case": dict(case)}
    D = case["dim"]
    if case["op"] in ("norm", "norm_train"):
        R = case["rows"]
        s["x"] = normal(R, D, dtype=tok)
        s["weight"] = 1.0 + 0.1 * normal(D)
        s["bias"] = 0.1 * normal(D) if case["bias"] else None
        # the residual stream: larger than one layer's output, and off centre
        s["residual"] = 3.0 * normal(R, D) + 0.5 if case["residual"] else None
        if case["op"] == "norm_train":
            s["dy"] = normal(R, D, dtype=tok)
            s["dres"] = normal(R, D) if case["residual"] else None
            _leaves(s, "x", "weight", "bias", "residual")
        return s
    B, L = case["batch"], case["seqlen"]
    lead = (B,) if case["op"] == "step" else (B, L)
    s["x"] = normal(*lead, D, dtype=tok)
    if case["sliced"]:  # the two gates as halves of one projection
        both = normal(*lead, 2 * D, dtype=tok)
        s["r"], s["i"] = both[..., :D], both[..., D:]
    else:
        s["r"], s["i"] = normal(*lead, D, dtype=tok), normal(*lead, D, dtype=tok)
    # rates: exp(-c softplus(lam)) between 0.9 and 0.999, as such layers are initialised
    rate = -torch.log(0.9 + 0.099 * uniform(D)) / _C
    s["lam"] = torch.log(torch.expm1(rate))
    if case["op"] == "step":
        s["h"] = normal(B, D)
        s["h_out"] = torch.empty_like(s["h"])
        return s
    s["h0"] = normal(B, D) if case["h0"] else None
    # a document begins at one token in 512, on average
    s["reset"] = uniform(B, L) < 1.0 / 512 if case["reset"] else None
    if case["op"] == "train":
        s["dy"] = normal(B, L, D, dtype=tok)
        s["dlast"] = normal(B, D) if case["last"] else None
        _leaves(s, "x", "r", "i", "lam", "h0")
    return s


def _leaves(s, *names):
    for n in names:
        if s[n] is not None:
            s[n] = s[n].detach().requires_grad_(True)
    s["leaves"] = [n for n in names if s[n] is not None]


def run(state):
    f = {"scan": (_plain_scan, _own_scan), "train": (_plain_train, _own_train), "step": (_plain_step, _own_step),
         "norm": (_plain_norm, _own_norm), "norm_train": (_plain_norm_train, _own_norm_train)}[state["op"]]
    if own:
        return f[1](state)
    with torch.no_grad():
        return f[0](state)


# ------------------------------------------------- the library's entry points
def _own_scan(s):
    import selective_state_space_47_b200 as ssm
    kw = dict(reset=s["reset"], c=_C, return_last_state=s["case"]["last"])
    out = ssm.gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], s["h0"], **kw)
    return {"y": out[0], "h_last": out[1]} if s["case"]["last"] else {"y": out}


def _own_train(s):
    import selective_state_space_47_b200 as ssm
    out = ssm.gated_scan(s["x"], s["r"], s["i"], s["lam"], s["h0"], reset=s["reset"], c=_C,
                         return_last_state=s["case"]["last"])
    out = list(out) if s["case"]["last"] else [out]
    grads = torch.autograd.grad(out, [s[n] for n in s["leaves"]], [s["dy"], s["dlast"]][:len(out)])
    res = dict(zip(("y", "h_last"), (t.detach() for t in out)))
    res.update({"d" + n: g for n, g in zip(s["leaves"], grads)})
    return res


def _own_step(s):
    import selective_state_space_47_b200 as ssm
    y = ssm.gated_step(s["x"], s["r"], s["i"], s["lam"], s["h"], c=_C, h_out=s["h_out"])
    return {"y": y, "h": s["h_out"]}


def _own_norm(s):
    import selective_state_space_47_b200 as ssm
    out = ssm.layer_norm_fwd(s["x"], s["weight"], s["bias"], s["residual"], eps=_EPS)
    return {"y": out} if s["residual"] is None else {"y": out[0], "residual": out[1]}


def _own_norm_train(s):
    import selective_state_space_47_b200 as ssm
    out = ssm.layer_norm(s["x"], s["weight"], s["bias"], s["residual"], eps=_EPS)
    out = [out] if s["residual"] is None else list(out)
    grads = torch.autograd.grad(out, [s[n] for n in s["leaves"]], [s["dy"], s["dres"]][:len(out)])
    res = dict(zip(("y", "s"), (t.detach() for t in out)))
    res.update({"d" + n: g for n, g in zip(s["leaves"], grads)})
    return res


# ------------------------------------------------------------- plain forms
def _linear_scan(a, b, h0):
    """h_t = a_t h_{t-1} + b_t over dim 1 of [B, L, D]: pieces of 32 steps from a zero start, the pieces'
    ends chained by the same scan, and each piece's start carried into its steps."""
    B, L, D = a.shape
    if L <= 32:
        out = torch.empty_like(b)
        h = h0
        for t in range(L):
            h = a[:, t] * h + b[:, t]
            out[:, t] = h
        return out
    n = -(-L // 32)
    pad = n * 32 - L
    if pad:
        a = torch.cat([a, torch.ones_like(a[:, :1]).expand(B, pad, D)], 1)
        b = torch.cat([b, torch.zeros_like(b[:, :1]).expand(B, pad, D)], 1)
    a, b = a.view(B, n, 32, D), b.view(B, n, 32, D)
    hs, ps = torch.empty_like(b), torch.empty_like(a)
    hs[:, :, 0], ps[:, :, 0] = b[:, :, 0], a[:, :, 0]
    for t in range(1, 32):
        hs[:, :, t] = a[:, :, t] * hs[:, :, t - 1] + b[:, :, t]
        ps[:, :, t] = a[:, :, t] * ps[:, :, t - 1]
    ends = _linear_scan(ps[:, :, -1], hs[:, :, -1], h0)
    starts = torch.cat([h0[:, None], ends[:, :-1]], 1)
    ps *= starts[:, :, None]
    ps += hs
    return ps.view(B, n * 32, D)[:, :L]


def _plain_gates(s):
    x, r, i = (s[n].float() for n in ("x", "r", "i"))
    lam = s["lam"]
    p = _C * (torch.clamp(lam, min=0) + torch.log1p(torch.exp(-lam.abs())))
    sr, si = 1.0 / (1.0 + torch.exp(-r)), 1.0 / (1.0 + torch.exp(-i))
    w = p * sr
    a, beta = torch.exp(-w), torch.sqrt(-torch.expm1(-2.0 * w))
    if s.get("reset") is not None:
        m = s["reset"][..., None]
        a, beta = torch.where(m, 0.0, a), torch.where(m, 1.0, beta)
    return x, sr, si, w, a, beta


def _plain_start(s):
    h0 = s["h0"]
    return torch.zeros_like(s["x"][:, 0], dtype=torch.float32) if h0 is None else h0.float()


def _plain_scan(s):
    x, _, si, _, a, beta = _plain_gates(s)
    h = _linear_scan(a, beta * si * x, _plain_start(s))
    out = {"y": h.to(s["x"].dtype)}
    if s["case"]["last"]:
        out["h_last"] = h[:, -1].clone()
    return out


def _plain_train(s):
    x, sr, si, w, a, beta = _plain_gates(s)
    tok = s["x"].dtype
    u = si * x
    start = _plain_start(s)
    h = _linear_scan(a, beta * u, start)
    # v_t = dy_t + a_{t+1} v_{t+1}: the same scan from the other end
    dy = s["dy"].float()
    if s["dlast"] is not None:
        dy = torch.cat([dy[:, :-1], dy[:, -1:] + s["dlast"][:, None]], 1)
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    v = _linear_scan(after.flip(1), dy.flip(1), torch.zeros_like(start)).flip(1)
    before = torch.cat([start[:, None], h[:, :-1]], 1)
    dw = v * (a * a / beta * u - a * before)
    out = {"y": h.to(tok)}
    if s["case"]["last"]:
        out["h_last"] = h[:, -1].clone()
    vb = v * beta
    out["dx"] = (vb * si).to(tok)
    out["dr"] = (dw * w * (1.0 - sr)).to(tok)
    out["di"] = (vb * u * (1.0 - si)).to(tok)
    out["dlam"] = (dw * sr).sum((0, 1)) * _C / (1.0 + torch.exp(-s["lam"]))
    if s["h0"] is not None:
        out["dh0"] = a[:, 0] * v[:, 0]
    return out


def _plain_step(s):
    x, _, si, _, a, beta = _plain_gates(s)
    h = a * s["h"] + beta * si * x
    s["h_out"].copy_(h)
    return {"y": h.to(s["x"].dtype), "h": s["h_out"]}


def _plain_rows(s):
    t = s["x"].float()
    if s["residual"] is not None:
        t = t + s["residual"]
    centred = t - t.mean(1, keepdim=True)
    k = 1.0 / torch.sqrt((centred * centred).mean(1, keepdim=True) + _EPS)
    y = centred * k * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return t, centred * k, k, y.to(s["x"].dtype)


def _plain_norm(s):
    t, _, _, y = _plain_rows(s)
    return {"y": y} if s["residual"] is None else {"y": y, "residual": t}


def _plain_norm_train(s):
    t, xh, k, y = _plain_rows(s)
    dy = s["dy"].float()
    g = dy * s["weight"]
    ds = k * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    out = {"y": y}
    if s["residual"] is not None:
        out["s"] = t
        ds = ds + s["dres"]
    out["dx"] = ds.to(s["x"].dtype)
    out["dweight"] = (dy * xh).sum(0)
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0)
    if s["residual"] is not None:
        out["dresidual"] = ds
    return out


# ------------------------------------------------------------------- work
def work(case):
    size, D = _SIZE[case["dtype"]], case["dim"]
    if case["op"] in ("norm", "norm_train"):
        n = case["rows"] * D
        token, per, flops = 2 * size, 8 if case["residual"] else 0, 8
        params = 4 * D * (2 if case["bias"] else 1)
        if case["op"] == "norm_train":  # x, dy in and y, dx out; the residual stream and its gradient in and out
            token, per, params, flops = 4 * size, 2 * per, 2 * params, 24
        return {"bytes": n * (token + per) + params, "flops": n * flops}
    n = case["batch"] * case["seqlen"] * D
    state = 4 * case["batch"] * D
    if case["op"] == "step":
        return {"bytes": n * 4 * size + 2 * state + 4 * D, "flops": 20 * n}
    states = case["h0"] + case["last"]
    marks = case["batch"] * case["seqlen"] if case["reset"] else 0
    if case["op"] == "scan":
        return {"bytes": n * 4 * size + states * state + 4 * D + marks, "flops": 20 * n}
    return {"bytes": n * 8 * size + 2 * states * state + 8 * D + marks, "flops": 60 * n}


# --------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        d = {k: v.detach().double() if isinstance(v, torch.Tensor) and v.is_floating_point() and k not in ("x", "r", "i", "dy")
             else v for k, v in s.items()}
        if case["op"] in ("norm", "norm_train"):
            return _exact_norm(case, d)
        return _exact_recurrence(case, d)


def _exact_norm(case, d):
    t = d["x"].double()
    if case["residual"]:
        t = t + d["residual"]
    mean = t.sum(1, keepdim=True) / case["dim"]
    dev = ((t - mean) ** 2).sum(1, keepdim=True) / case["dim"] + _EPS
    xh = (t - mean) * dev ** -0.5
    out = {"y": xh * d["weight"] + (d["bias"] if case["bias"] else 0.0)}
    if case["residual"]:
        out["residual" if case["op"] == "norm" else "s"] = t
    if case["op"] == "norm":
        return out
    dy = d["dy"].double()
    g = dy * d["weight"]
    inner = (g * xh).sum(1, keepdim=True) / case["dim"]
    ds = (g - g.sum(1, keepdim=True) / case["dim"] - xh * inner) * dev ** -0.5
    if case["residual"]:
        ds = ds + d["dres"]
    out["dx"], out["dweight"] = ds, (dy * xh).sum(0)
    if case["bias"]:
        out["dbias"] = dy.sum(0)
    if case["residual"]:
        out["dresidual"] = ds
    return out


def _exact_recurrence(case, d):
    step = case["op"] == "step"
    x, r, i = ((d[n].unsqueeze(1) if step else d[n]) for n in ("x", "r", "i"))
    B, L, D = x.shape
    rate = _C * torch.logaddexp(d["lam"], torch.zeros_like(d["lam"]))
    h = d["h"] if step else d["h0"]
    h = torch.zeros(B, D, dtype=torch.float64, device=x.device) if h is None else h
    start = h
    # y, and for a training pass the factors of every step, in pieces of time
    y = torch.empty(B, L, D, dtype=torch.float64, device=x.device)
    decay = torch.empty_like(y) if case["op"] == "train" else None
    for t0 in range(0, L, 4096):
        part = slice(t0, min(L, t0 + 4096))
        a = torch.exp(-rate * torch.sigmoid(r[:, part].double()))
        b = torch.sigmoid(i[:, part].double()) * x[:, part].double()
        norm = (-torch.expm1(-2.0 * rate * torch.sigmoid(r[:, part].double()))).sqrt()
        if d.get("reset") is not None:
            m = d["reset"][:, part, None]
            a, norm = a.masked_fill(m, 0.0), norm.masked_fill(m, 1.0)
        b *= norm
        for t in range(a.shape[1]):
            h = torch.addcmul(b[:, t], a[:, t], h)
            y[:, t0 + t] = h
        if decay is not None:
            decay[:, part] = a
    if step:
        return {"y": y[:, 0], "h": h}
    out = {"y": y}
    if case["last"]:
        out["h_last"] = h
    if case["op"] == "scan":
        return out
    v = torch.zeros_like(h) if d["dlast"] is None else d["dlast"]
    dx, dr, di = (torch.empty_like(y) for _ in range(3))
    dlam = torch.zeros_like(rate)
    for t in range(L - 1, -1, -1):
        v = v + d["dy"][:, t].double()
        sr, si, xt = torch.sigmoid(r[:, t].double()), torch.sigmoid(i[:, t].double()), x[:, t].double()
        prev, a = (y[:, t - 1] if t else start), decay[:, t]
        fresh = d["reset"][:, t, None] if d["reset"] is not None else None
        norm = (-torch.expm1(-2.0 * rate * sr)).sqrt()
        dlog = a * prev * v - (a * a / norm) * (si * xt * v)  # with respect to log a = -rate sr
        if fresh is not None:
            dlog, norm = dlog.masked_fill(fresh, 0.0), norm.masked_fill(fresh, 1.0)
        dx[:, t] = v * norm * si
        di[:, t] = v * norm * xt * si * (1.0 - si)
        dr[:, t] = -dlog * rate * sr * (1.0 - sr)
        dlam -= (dlog * sr).sum(0)
        v = a * v
    out.update(dx=dx, dr=dr, di=di, dlam=dlam * _C * torch.sigmoid(d["lam"]))
    if case["h0"]:
        out["dh0"] = v
    return out
