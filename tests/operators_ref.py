"""Plain float64 forms of the gated linear recurrence and of the layer norm, step by step,
each with a bound on what float32 arithmetic may leave of it.

The bounds follow the arithmetic (u = 2^-24, half a float32 step), to first order and doubled for the rest:
a sigmoid from an exponential of 2^-22 and a reciprocal of 2^-23 is off by at most
(|v| + 7) u, 13 u for |v| <= 6; the rate by 4 u; 1 - exp(-w) by the sum and its own 4 u: 22 u
relative, so a decay a by 22 u (1 - a) + u; the input's factors by 40 u. They pass through the
recurrence with the state itself: E_t = a_t E_{t-1} + da_t |h_{t-1}| + 40 u |b_t| + 2 u M_t, where
M_t = a_t M_{t-1} + |b_t|. The roundings go by M_t and not by |h_t|: where time is cut into pieces, a
state is the sum P h + H of what was carried in and what the piece added, each rounded on its own
(half a step of up to |P h| and of up to the piece's sum of |b| carried on, together at most M_t),
and the two may cancel. A piece of n steps takes part in fewer than n such sums, so two
roundings a step cover them. A value stored in the tokens' type adds half a step of that type.
"""
import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def _gates(x, r, i, lam, reset, c):
    x, r, i, lam = (t.double() for t in (x, r, i, lam))
    p = c * torch.logaddexp(lam, torch.zeros_like(lam))
    sr, si = torch.sigmoid(r), torch.sigmoid(i)
    w = p * sr
    a, beta = torch.exp(-w), torch.sqrt(-torch.expm1(-2 * w))
    if reset is not None:
        a, beta = a.masked_fill(reset[..., None], 0.0), beta.masked_fill(reset[..., None], 1.0)
    return x, sr, si, w, a, beta


def gated_scan(x, r, i, lam, h0=None, reset=None, c=8.0):
    """y and, elementwise, the bound on float32's error in it (both float64, [B, L, D])."""
    xd, _, si, _, a, beta = _gates(x, r, i, lam, reset, c)
    b = beta * si * xd
    B, L, D = x.shape
    h = torch.zeros(B, D, dtype=torch.float64) if h0 is None else h0.double()
    err, mag = torch.zeros_like(h), h.abs()
    ys, es = torch.empty_like(b), torch.empty_like(b)
    for t in range(L):
        at = a[:, t]
        da = torch.where(at == 0, 0.0, 22 * U * (1 - at) + U)
        hn = at * h + b[:, t]
        if reset is not None:  # dropped, whatever it was
            fresh = reset[:, t, None]
            hn = torch.where(fresh, b[:, t], hn)
            h, err, mag = h.masked_fill(fresh, 0.0), err.masked_fill(fresh, 0.0), mag.masked_fill(fresh, 0.0)
        mag = at * mag + b[:, t].abs()
        err = at * err + da * h.abs() + 40 * U * b[:, t].abs() + 2 * U * mag
        h = hn
        ys[:, t], es[:, t] = h, err
    return ys, 2 * es


def gated_scan_bwd(x, r, i, lam, dy, h0=None, dh_last=None, reset=None, c=8.0):
    """The gradients by the formulas, and their bounds: two dicts."""
    xd, sr, si, w, a, beta = _gates(x, r, i, lam, reset, c)
    ys, es = gated_scan(x, r, i, lam, h0, reset, c)
    B, L, D = x.shape
    lam = lam.double()
    u = si * xd
    start = torch.zeros(B, D, dtype=torch.float64) if h0 is None else h0.double()
    v = torch.zeros_like(start) if dh_last is None else dh_last.double()
    ev, mv = torch.zeros_like(v), v.abs()
    g = {k: torch.empty_like(xd) for k in ("dx", "dr", "di")}
    e = {k: torch.empty_like(xd) for k in ("dx", "dr", "di")}
    dlam, elam, mlam = torch.zeros_like(lam), torch.zeros_like(lam), torch.zeros_like(lam)
    for t in range(L - 1, -1, -1):
        v = v + dy[:, t].double()
        mv = mv + dy[:, t].double().abs()
        ev = ev + 2 * U * mv
        at, bt, ut = a[:, t], beta[:, t], u[:, t]
        prev = ys[:, t - 1] if t else start
        eprev = es[:, t - 1] if t else torch.zeros_like(start)
        ratio = torch.where(bt > 0, at * ut / bt.clamp(min=1e-300), 0.0)
        dw, edw = at * v * (ratio - prev), at * (ev * (ratio - prev).abs() + v.abs() * (
            eprev + 50 * U * (ratio.abs() + prev.abs())))
        if reset is not None:
            fresh = reset[:, t, None]
            dw, edw = dw.masked_fill(fresh, 0.0), edw.masked_fill(fresh, 0.0)
        s, ws = 1 - si[:, t], w[:, t] * (1 - sr[:, t])
        g["dx"][:, t], e["dx"][:, t] = v * bt * si[:, t], bt * si[:, t] * (ev + 50 * U * v.abs())
        g["di"][:, t] = v * bt * ut * s
        e["di"][:, t] = (bt * ut).abs() * (ev * s + 50 * U * v.abs())
        g["dr"][:, t], e["dr"][:, t] = dw * ws, edw * ws + 40 * U * (dw * w[:, t]).abs()
        dlam = dlam + (dw * sr[:, t]).sum(0)
        elam = elam + (edw * sr[:, t]).sum(0)
        mlam = mlam + (dw * sr[:, t]).abs().sum(0)
        da = torch.where(at == 0, 0.0, 22 * U * (1 - at) + U)
        ev = at * ev + da * v.abs()
        v, mv = at * v, at * mv
        if reset is not None:
            v, ev, mv = v.masked_fill(fresh, 0.0), ev.masked_fill(fresh, 0.0), mv.masked_fill(fresh, 0.0)
    k = c * torch.sigmoid(lam)
    # dlam: a tile sums 64 steps one by one and across its warps, then tiles; 200 u covers any order
    g["dlam"], e["dlam"] = dlam * k, k * (elam + 200 * U * mlam)
    g["dh0"], e["dh0"] = v, ev + 2 * U * mv
    return g, {n: 2 * t for n, t in e.items()}


def check(got, ref, bound, dtype=torch.float32, what=""):
    """|got - ref| <= bound + half a step of the stored type, elementwise; the values are finite."""
    got, ref = got.detach().cpu(), ref
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got.float()).all(), f"{what}: not finite"
    tol = bound * (1 + HALF_STEP[dtype]) + HALF_STEP[dtype] * ref.abs() + 1e-36
    over = ((got.double() - ref).abs() / tol)
    worst = over.max().item() if over.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.2f} of the bound at {over.argmax().item()}"
    return worst


# Row sums: at most 64 values one after the other in a thread, then 5 + 32 partial sums: 100 u.
DEPTH = 100 * U


def layer_norm(x, weight, bias=None, residual=None, eps=1e-5):
    """dict y, s, mean, rstd and the bounds."""
    s = x.double() + (0.0 if residual is None else residual.double())
    n = s.shape[-1]
    mean = s.mean(-1, keepdim=True)
    cen = s - mean
    var = (cen * cen).mean(-1, keepdim=True)
    rstd = (var + eps) ** -0.5
    xh = cen * rstd
    y = xh * weight.double() + (0.0 if bias is None else bias.double())
    es = U * s.abs() if residual is not None else torch.zeros_like(s)
    em = DEPTH * s.abs().mean(-1, keepdim=True) + es.mean(-1, keepdim=True) + U * mean.abs()
    ec = es + em + U * cen.abs()
    # var: 2 E|cen ec| plus its own sum; rstd: half of that, relative to var + eps, plus 4 u
    ev = 2 * (cen.abs() * ec).mean(-1, keepdim=True) + (ec * ec).mean(-1, keepdim=True) + DEPTH * var
    er = rstd * (0.5 * ev / (var + eps) + 4 * U)
    ey = weight.double().abs() * (ec * rstd + cen.abs() * er) + 4 * U * (xh * weight.double()).abs() + U * y.abs()
    sq = lambda t: t.squeeze(-1)
    return (dict(y=y, s=s, mean=sq(mean), rstd=sq(rstd)),
            dict(y=2 * ey, s=2 * es, mean=2 * sq(em), rstd=2 * sq(er)))


def layer_norm_bwd(dy, s, weight, mean, rstd, dresidual_out=None):
    """dict dx (= dresidual), dweight, dbias for the given float32 mean and rstd, and the bounds. A row of the parts
    sums its rows one by one, then the parts are summed: at most rows + 12 additions."""
    dy, s, w = dy.double(), s.double(), weight.double()
    mean, rstd = mean.double().unsqueeze(-1), rstd.double().unsqueeze(-1)
    xh, g = (s - mean) * rstd, dy * w
    m0, m1 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    ds = rstd * (g - m0 - xh * m1)
    e0 = (DEPTH + U) * g.abs().mean(-1, keepdim=True)
    e1 = (DEPTH + 4 * U) * (g * xh).abs().mean(-1, keepdim=True)
    e = rstd * (4 * U * g.abs() + e0 + 4 * U * m0.abs() + xh.abs() * (e1 + 6 * U * m1.abs())) + 2 * U * ds.abs()
    if dresidual_out is not None:
        ds = ds + dresidual_out.double()
        e = e + U * ds.abs()
    rows = dy.reshape(-1, dy.shape[-1]).shape[0]
    flat = lambda t: t.reshape(rows, -1)
    out = dict(dx=ds, dweight=flat(dy * xh).sum(0), dbias=flat(dy).sum(0))
    n = (rows + 12) * U
    return out, dict(dx=2 * e, dweight=2 * (n + 3 * U) * flat(dy * xh).abs().sum(0), dbias=2 * n * flat(dy).abs().sum(0))
