"""GPU checks of the layer norm (forward, backward) against its float64 form, elementwise
within the bounds derived there, and of a recurrent residual layer made of both operators."""
import pytest
import torch

from tests import operators_ref as ref
from tests.conftest import cuda_available

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ssm():
    if not cuda_available():
        pytest.skip("needs a CUDA device")
    import selective_state_space_47_b200 as m
    return m


def make(rows, D, dtype, seed, residual, offset=0.5):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    return dict(x=(n(rows, D) + offset).to(dtype), weight=1 + 0.2 * n(D), bias=0.3 * n(D),
                residual=2 * n(rows, D) + offset if residual else None, dy=n(rows, D).to(dtype),
                dres=n(rows, D) if residual else None)


def cuda(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def check_all(ssm, d, dtype, bias=True, eps=1e-5):
    g = cuda(d)
    if not bias:
        d["bias"] = g["bias"] = None
    want, bound = ref.layer_norm(d["x"], d["weight"], d["bias"], d["residual"], eps)
    out = ssm.layer_norm_fwd(g["x"], g["weight"], g["bias"], g["residual"], eps=eps, return_stats=True)
    torch.cuda.synchronize()
    mean, rstd = out[-2:]
    ref.check(out[0], want["y"], bound["y"], dtype, "y")
    ref.check(mean, want["mean"], bound["mean"], what="mean")
    ref.check(rstd, want["rstd"], bound["rstd"], what="rstd")
    s = g["x"]
    if d["residual"] is not None:
        s = out[1]
        assert torch.equal(s.cpu(), d["x"].float() + d["residual"])
    gw, gb = ref.layer_norm_bwd(d["dy"], s.cpu(), d["weight"], mean.cpu(), rstd.cpu(), d["dres"])
    got = ssm.layer_norm_bwd(g["dy"], s, g["weight"], mean, rstd, g["dres"], residual=d["residual"] is not None, bias=bias)
    torch.cuda.synchronize()
    ref.check(got["dx"], gw["dx"], gb["dx"], dtype, "dx")
    ref.check(got["dweight"], gw["dweight"], gb["dweight"], what="dweight")
    if bias:
        ref.check(got["dbias"], gw["dbias"], gb["dbias"], what="dbias")
    else:
        assert got["dbias"] is None
    if d["residual"] is None:
        assert got["dresidual"] is None
    else:
        ref.check(got["dresidual"], gw["dx"], gb["dx"], what="dresidual")


DIMS = [1, 2, 7, 8, 31, 32, 33, 64, 100, 127, 128, 256, 264, 500, 512, 513, 1000, 1024, 1026, 1032, 2048, 2049, 4096, 4100, 5120,
        8192, 8200, 16383, 16384]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("residual", [False, True], ids=["alone", "residual"])
@pytest.mark.parametrize("dim", DIMS)
def test_dims(ssm, dim, residual, dtype):
    check_all(ssm, make(5, dim, dtype, dim, residual), dtype, bias=dim % 2 == 0)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 149, 600, 1185, 1400])
def test_rows(ssm, rows, dtype):
    check_all(ssm, make(rows, 40, dtype, rows, rows % 2 == 1), dtype)
    check_all(ssm, make(rows, 300, dtype, rows, rows % 2 == 0), dtype)


def test_rows_far_from_zero_and_flat_rows(ssm):
    """A row whose mean dwarfs its spread keeps its variance; a constant row gives bias, with finite gradients."""
    d = make(6, 640, F32, 7, False, offset=4096.0)
    d["x"][3] = 17.25
    d["x"][4] = 0.0
    check_all(ssm, d, F32)
    g = cuda(d)
    y = ssm.layer_norm_fwd(g["x"], g["weight"], g["bias"])
    assert torch.equal(y[3], g["bias"]) and torch.equal(y[4], g["bias"])


def test_a_bad_row_stays_in_its_row(ssm):
    d = make(9, 96, F32, 8, True)
    g = cuda(d)
    good = ssm.layer_norm_fwd(g["x"], g["weight"], g["bias"], g["residual"])[0]
    g["x"][4, 5] = float("nan")
    g["x"][6, 0] = float("inf")
    y = ssm.layer_norm_fwd(g["x"], g["weight"], g["bias"], g["residual"])[0]
    rest = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(y[rest], good[rest]) and torch.isnan(y[4]).all() and not torch.isfinite(y[6]).any()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_misaligned_arrays(ssm, dtype):
    """Arrays that start off 16 bytes take the element-wise form."""
    d = make(4, 64, dtype, 12, True)
    g = cuda(d)
    want, bound = ref.layer_norm(d["x"], d["weight"], d["bias"], d["residual"])
    for name in ("x", "weight", "bias", "residual"):
        h = dict(g)
        buf = torch.empty(h[name].numel() + 1, dtype=h[name].dtype, device="cuda")
        buf[1:] = h[name].reshape(-1)
        h[name] = buf[1:].view(h[name].shape)
        y, s = ssm.layer_norm_fwd(h["x"], h["weight"], h["bias"], h["residual"])
        ref.check(y, want["y"], bound["y"], dtype, name)


def test_empty_and_shapes(ssm):
    w = torch.ones(8, device="cuda")
    y, s = ssm.layer_norm_fwd(torch.zeros(0, 3, 8, device="cuda"), w, None, torch.zeros(0, 3, 8, device="cuda"))
    assert y.shape == s.shape == (0, 3, 8)
    z = torch.zeros(0, 8, device="cuda")
    g = ssm.layer_norm_bwd(z, z, w, z[:, 0], z[:, 0])
    assert torch.equal(g["dweight"], 0 * w) and torch.equal(g["dbias"], 0 * w)
    assert ssm.layer_norm_fwd(torch.zeros(8, device="cuda"), w).shape == (8,)
    with pytest.raises(RuntimeError):
        ssm.layer_norm_fwd(torch.zeros(2, 16385, device="cuda"), torch.zeros(16385, device="cuda"))


def test_residual_in_place_and_repeats(ssm):
    d = make(700, 520, BF16, 15, True)
    g = cuda(d)
    y, s, mean, rstd = ssm.layer_norm_fwd(g["x"], g["weight"], g["bias"], g["residual"], return_stats=True)
    r = g["residual"].clone()
    y2, s2 = ssm.layer_norm_fwd(g["x"], g["weight"], g["bias"], r, residual_out=r)
    assert s2 is r and torch.equal(s, r) and torch.equal(y, y2)
    first = ssm.layer_norm_bwd(g["dy"], s, g["weight"], mean, rstd, g["dres"], residual=True)
    for _ in range(5):
        again = ssm.layer_norm_bwd(g["dy"], s, g["weight"], mean, rstd, g["dres"], residual=True)
        for k in first:
            assert torch.equal(first[k], again[k]), k


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_autograd(ssm, dtype):
    d = make(30, 72, dtype, 16, True)
    g = cuda(d)
    leaf = {k: g[k].clone().requires_grad_(True) for k in ("x", "weight", "bias", "residual")}
    y, s = ssm.layer_norm(*leaf.values())
    torch.autograd.backward([y, s], [g["dy"], g["dres"]])
    _, _, mean, rstd = ssm.layer_norm_fwd(*(g[k] for k in leaf), return_stats=True)
    want, bound = ref.layer_norm_bwd(d["dy"], s.detach().cpu(), d["weight"], mean.cpu(), rstd.cpu(), d["dres"])
    for k, n in (("x", "dx"), ("weight", "dweight"), ("bias", "dbias"), ("residual", "dx")):
        ref.check(leaf[k].grad, want[n], bound[n], leaf[k].dtype, k)
    assert leaf["x"].grad.data_ptr() != leaf["residual"].grad.data_ptr()  # also where the two are equal
    # only the residual stream's gradient arrives: it passes through
    y, s = ssm.layer_norm(*leaf.values())
    gr, gw = torch.autograd.grad(s, (leaf["residual"], leaf["weight"]), g["dres"])
    assert torch.equal(gr, g["dres"]) and torch.equal(gw, torch.zeros_like(gw))


def test_no_gradient_asked(ssm):
    d = cuda(make(5, 64, BF16, 18, True))
    y, s = ssm.layer_norm(d["x"], d["weight"], d["bias"], d["residual"])
    assert not y.requires_grad
    for a, b in zip((y, s), ssm.layer_norm_fwd(d["x"], d["weight"], d["bias"], d["residual"])):
        assert torch.equal(a, b)
    x = torch.randn(1, 90, 64, device="cuda", requires_grad=True)
    lam = torch.zeros(64, device="cuda")
    with torch.no_grad():
        y, h = ssm.gated_scan(x, x, x, lam, return_last_state=True)
    assert not y.requires_grad and torch.equal(h, ssm.gated_scan_fwd(x, x, x, lam, return_last_state=True)[1])
    assert torch.equal(y, ssm.gated_scan(x, x, x, lam))


def test_a_second_derivative_is_refused(ssm):
    x = torch.randn(4, 32, device="cuda", requires_grad=True)
    w = torch.ones(32, device="cuda")
    for y in (ssm.layer_norm(x, w), ssm.gated_scan(x[None], x[None], x[None], w)):
        g, = torch.autograd.grad(y.square().sum(), x, create_graph=True)  # the first one is as without a graph
        y2 = ssm.layer_norm(x, w) if y.dim() == 2 else ssm.gated_scan(x[None], x[None], x[None], w)
        assert torch.equal(g, torch.autograd.grad(y2.square().sum(), x)[0])
        with pytest.raises(RuntimeError):
            torch.autograd.grad(g.sum(), x)


def test_graph(ssm):
    d = make(64, 256, BF16, 17, True)
    g = cuda(d)

    def both():
        y, s, m, k = ssm.layer_norm_fwd(g["x"], g["weight"], g["bias"], g["residual"], return_stats=True)
        return y, ssm.layer_norm_bwd(g["dy"], s, g["weight"], m, k, g["dres"], residual=True)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, grads = both()
    g["x"].mul_(1.5)
    graph.replay()
    torch.cuda.synchronize()
    y2, grads2 = both()
    assert torch.equal(y, y2)
    for k in grads:
        assert torch.equal(grads[k], grads2[k]), k


def test_a_recurrent_residual_layer(ssm):
    """Two layers of norm, projections, gated recurrence and residual sum, as they are used: in training against
    the same layers in float64, and token by token against the whole sequence."""
    B, L, D, c = 2, 150, 32, 8.0
    gen = torch.Generator().manual_seed(77)
    n = lambda *s: torch.randn(*s, generator=gen)
    params = []
    for _ in range(2):
        params.append(dict(weight=1 + 0.1 * n(D), bias=0.1 * n(D), proj=n(D, 3 * D) / D ** 0.5,
                           lam=torch.log(torch.expm1(-torch.log(0.9 + 0.09 * torch.rand(D, generator=gen)) / c))))
    x0, target = n(B, L, D), n(B, L, D)
    reset = torch.zeros(B, L, dtype=torch.bool)
    reset[0, 70] = True

    def plain(ps, x):
        out, s = x, torch.zeros_like(x)
        for p in ps:
            s = s + out
            m = s.mean(-1, keepdim=True)
            h = (s - m) / torch.sqrt(((s - m) ** 2).mean(-1, keepdim=True) + 1e-5) * p["weight"] + p["bias"]
            a = h @ p["proj"]
            xt, r, i = a.split(D, -1)
            w = c * torch.logaddexp(p["lam"], torch.zeros_like(p["lam"])) * torch.sigmoid(r)
            dec, inp = torch.exp(-w), torch.sqrt(-torch.expm1(-2 * w))
            st, ys = torch.zeros(B, D, dtype=x.dtype), []
            for t in range(L):
                f = reset[:, t, None]
                st = torch.where(f, 0.0, dec[:, t]) * st + torch.where(f, 1.0, inp[:, t]) * torch.sigmoid(i[:, t]) * xt[:, t]
                ys.append(st)
            out = torch.stack(ys, 1)
        return s + out

    def ours(ps, x, rs):
        out, s = x, torch.zeros_like(x)
        for p in ps:
            h, s = ssm.layer_norm(out, p["weight"], p["bias"], s)
            xt, r, i = (h @ p["proj"]).split(D, -1)
            out = ssm.gated_scan(xt, r, i, p["lam"], reset=rs, c=c)
        return s + out

    leaves = [{k: v.double().requires_grad_(True) for k, v in p.items()} for p in params]
    (plain(leaves, x0.double()) * target.double()).sum().backward()
    old = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        mine = [{k: v.cuda().requires_grad_(True) for k, v in p.items()} for p in params]
        y = ours(mine, x0.cuda(), reset.cuda())
        (y * target.cuda()).sum().backward()
        # float32 through two layers of depth-32 products and a recurrence with a memory of 100 steps:
        # about 100 roundings of 1.2e-7 in a row on sums of terms of either sign
        with torch.no_grad():
            want = plain(leaves, x0.double())
        assert (y.cpu().double() - want).abs().max() <= 2e-5 * want.abs().max()
        for a, b in zip(mine, leaves):
            for k in a:
                e = (a[k].grad.cpu().double() - b[k].grad).abs().max() / b[k].grad.abs().max()
                assert e <= 1e-4, (k, e.item())
        with torch.no_grad():
            hs = [torch.zeros(B, D, device="cuda") for _ in params]
            for t in range(70):
                out, s = x0[:, t].cuda(), torch.zeros(B, D, device="cuda")
                for p, h in zip(mine, hs):
                    z, s = ssm.layer_norm_fwd(out, p["weight"], p["bias"], s)
                    xt, r, i = (z @ p["proj"]).split(D, -1)
                    out = ssm.gated_step(xt, r, i, p["lam"], h, c=c)
                assert (s + out - y[:, t]).abs().max() <= 2e-5 * want.abs().max()
    finally:
        torch.backends.cuda.matmul.allow_tf32 = old


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 66, 4100, 4102])
@pytest.mark.parametrize("residual", [False, True], ids=["alone", "residual"])
def test_misaligned_arrays_backward(ssm, dtype, dim, residual):
    """Arrays that start off 16 bytes, one at a time."""
    d = make(9, dim, dtype, 13, residual)
    g = cuda(d)
    out = ssm.layer_norm_fwd(g["x"], g["weight"], g["bias"], g["residual"], return_stats=True)
    mean, rstd = out[-2:]
    t = dict(dy=g["dy"], s=out[1] if residual else g["x"], weight=g["weight"], dres=g["dres"])
    want, bound = ref.layer_norm_bwd(d["dy"], t["s"].cpu(), d["weight"], mean.cpu(), rstd.cpu(), d["dres"])
    for name in [k for k in t if t[k] is not None]:
        h = dict(t)
        buf = torch.empty(h[name].numel() + 1, dtype=h[name].dtype, device="cuda")
        buf[1:] = h[name].reshape(-1)
        h[name] = buf[1:].view(h[name].shape)
        got = ssm.layer_norm_bwd(h["dy"], h["s"], h["weight"], mean, rstd, h["dres"], residual=residual)
        for k in ("dx", "dweight", "dbias"):
            ref.check(got[k], want[k], bound[k], dtype if k == "dx" else F32, f"{k}, {name} off its place")


def test_streams_and_workspaces(ssm):
    """Both directions on a stream of the caller's, and the backward with a workspace of exactly the bytes it asks for."""
    import ctypes
    from selective_state_space_47_b200 import _native
    d = make(700, 264, BF16, 19, True)
    g = cuda(d)
    args = [g[k] for k in ("x", "weight", "bias", "residual")]
    want = ssm.layer_norm_fwd(*args, return_stats=True)
    grads = ssm.layer_norm_bwd(g["dy"], want[1], g["weight"], want[2], want[3], g["dres"], residual=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ssm.layer_norm_fwd(*args, return_stats=True, stream=s)
    gs = ssm.layer_norm_bwd(g["dy"], got[1], g["weight"], got[2], got[3], g["dres"], residual=True, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    a = _native.NormBwdArgs(700, 264, _native.SSM_BF16, 1)
    need = _native.lib().ssm_layer_norm_bwd_workspace_size(ctypes.byref(a))
    buf = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    gw = ssm.layer_norm_bwd(g["dy"], want[1], g["weight"], want[2], want[3], g["dres"], residual=True, workspace=buf[:need])
    for k in grads:
        assert torch.equal(grads[k], gs[k]) and torch.equal(grads[k], gw[k]), k
    assert (buf[need:] == 0xA5).all()
    for bad in (buf[:need - 1], torch.empty(need, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            ssm.layer_norm_bwd(g["dy"], want[1], g["weight"], want[2], want[3], workspace=bad, residual=True)


@pytest.mark.parametrize("dim,dtype", [(4099, BF16), (4098, BF16), (4099, F32)])
def test_as_many_blocks_as_the_row_allows(ssm, dim, dtype):
    """Where the backward's sums lie in shared memory, short rows leave room for several blocks on an SM, each with a row of
    partial sums in the workspace; the gradients are right for any number of them."""
    rows = 2400
    d = make(rows, dim, dtype, 20, False)
    g = cuda(d)
    _, mean, rstd = ssm.layer_norm_fwd(g["x"], g["weight"], return_stats=True)
    ws = torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device="cuda")  # NaNs, where nothing is written
    got = ssm.layer_norm_bwd(g["dy"], g["x"], g["weight"], mean, rstd, workspace=ws)
    parts = ws[:600 * dim * 4].view(torch.float32).view(600, dim)
    used = int((~torch.isnan(parts)).all(1).sum())
    assert used > torch.cuda.get_device_properties(0).multi_processor_count
    want, bound = ref.layer_norm_bwd(d["dy"], d["x"], d["weight"], mean.cpu(), rstd.cpu())
    for k in want:
        ref.check(got[k], want[k], bound[k], dtype if k == "dx" else F32, k)


def test_offsets_beyond_32_bits(ssm):
    """2.2e9 elements: the last rows, both directions."""
    rows, D = 1050001, 2112
    x = torch.empty(rows, D, device="cuda", dtype=BF16).normal_()
    w = 1 + 0.2 * torch.randn(D, device="cuda")
    y, mean, rstd = ssm.layer_norm_fwd(x, w, return_stats=True)
    tail = x[-5:].cpu()
    want, bound = ref.layer_norm(tail, w.cpu())
    ref.check(y[-5:], want["y"], bound["y"], BF16, "y")
    ref.check(mean[-5:], want["mean"], bound["mean"], what="mean")
    g = ssm.layer_norm_bwd(y, x, w, mean, rstd, bias=False)
    want, bound = ref.layer_norm_bwd(y[-5:].cpu(), tail, w.cpu(), mean[-5:].cpu(), rstd[-5:].cpu())
    ref.check(g["dx"][-5:], want["dx"], bound["dx"], BF16, "dx")
    assert torch.isfinite(g["dweight"]).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_one_tensor_in_two_places(ssm, dtype):
    """x as its own residual, and one tensor as token and both gates: gradients add up."""
    d = make(7, 72, dtype, 21, False)
    x, w = d["x"].cuda().requires_grad_(True), d["weight"].cuda().requires_grad_(True)
    y, s = ssm.layer_norm(x, w, w, x if dtype is F32 else x.float())
    gx, gw = torch.autograd.grad([y, s], [x, w], [d["dy"].cuda(), torch.ones_like(s)])
    _, _, mean, rstd = ssm.layer_norm_fwd(x.detach(), w.detach(), w.detach(), x.detach().float(), return_stats=True)
    want, bound = ref.layer_norm_bwd(d["dy"], s.detach().cpu(), d["weight"], mean.cpu(), rstd.cpu(), torch.ones(7, 72))
    # bfloat16: each part and the sum are rounded, half a step of values of up to twice |dx| each
    half = ref.HALF_STEP[dtype]
    ref.check(gx, 2 * want["dx"], 2 * bound["dx"] + 3 * half * want["dx"].abs(), dtype, "dx")
    ref.check(gw, want["dweight"] + want["dbias"], bound["dweight"] + bound["dbias"] + ref.U * (want["dweight"] + want["dbias"]).abs(), what="dweight")
    n = torch.randn(2, 70, 8, generator=torch.Generator().manual_seed(1)).to(dtype)
    t = n.cuda().requires_grad_(True)
    lam = torch.full((8,), -3.0)
    g, = torch.autograd.grad(ssm.gated_scan(t, t, t, lam.cuda()), t, n.cuda())
    want, bound = ref.gated_scan_bwd(n, n, n, lam, n)
    parts = [want[k] for k in ("dx", "dr", "di")]
    mag = sum(p.abs() for p in parts)
    ref.check(g, sum(parts), sum(bound[k] for k in ("dx", "dr", "di")) + 4 * half * mag, dtype, "d of all three")
