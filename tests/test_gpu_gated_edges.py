"""GPU checks of the gated linear recurrence where a value that the formulas never use is NaN,
and in the forms that other sizes than the plain tests' reach."""
import pytest
import torch

from tests import operators_ref as ref
from tests.conftest import cuda_available
from tests.test_gpu_gated import FWD, check_bwd, check_fwd, cuda, make

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
BWD = ("x", "r", "i", "lam", "dy", "h0", "dh_last")
NAN = float("nan")


@pytest.fixture(scope="module")
def ssm():
    if not cuda_available():
        pytest.skip("needs a CUDA device")
    import selective_state_space_47_b200 as m
    return m


# whole tiles by TMA, rows in pieces, odd rows, two passes over few columns, a few tokens by tiles and by threads
FORMS = [(2, 400, 64), (2, 400, 34), (2, 400, 33), (1, 5000, 72), (300, 9, 12), (300, 9, 7), (1500, 9, 12), (1500, 9, 7)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("slow", [True, False], ids=["rates_small", "rates_any"])
@pytest.mark.parametrize("size", FORMS, ids=lambda s: "x".join(map(str, s)))
def test_the_decay_gate_is_not_used_at_a_reset(ssm, size, slow, dtype):
    """At a reset a = 0 and beta = 1 whatever r is: a NaN there reaches no output and no gradient, and dr is 0."""
    d = make(*size, dtype, seed=11, h0=True, reset=0.05, slow=slow)
    d["reset"][:, size[1] // 2] = True
    want, bound = ref.gated_scan(*(d[k] for k in FWD), reset=d["reset"])
    gw, gb = ref.gated_scan_bwd(*(d[k] for k in BWD), reset=d["reset"])
    g = cuda(d)
    g["r"] = g["r"].masked_fill(g["reset"][..., None], NAN)
    y, h, states = ssm.gated_scan_fwd(*(g[k] for k in FWD), reset=g["reset"], return_last_state=True, return_states=True)
    ref.check(y, want, bound, dtype, "y")
    ref.check(h, want[:, -1], bound[:, -1], what="h_last")
    assert torch.isfinite(states).all()
    got = ssm.gated_scan_bwd(*(g[k] for k in BWD), states=states, reset=g["reset"])
    for k in gw:
        ref.check(got[k], gw[k], gb[k], dtype if k in ("dx", "dr", "di") else F32, k)
    assert not got["dr"][g["reset"]].any()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", FORMS, ids=lambda s: "x".join(map(str, s)))
def test_a_bad_input_gate_leaves_the_adjoint(ssm, size, dtype):
    """A NaN in i spoils the states from its step on, but the adjoint goes by r alone: dx and di are as
    without it at every other step, and so are dr before it and dh0."""
    B, L, D = size
    d = make(B, L, D, dtype, seed=12, h0=True)
    at = L // 2
    gw, gb = ref.gated_scan_bwd(*(d[k] for k in BWD))
    g = cuda(d)
    g["i"][0, at] = NAN
    y, states = ssm.gated_scan_fwd(*(g[k] for k in FWD), return_states=True)
    want, bound = ref.gated_scan(*(d[k] for k in FWD))
    ref.check(y[0, :at], want[0, :at], bound[0, :at], dtype, "y")
    assert torch.isnan(y[0, at:]).all()
    got = ssm.gated_scan_bwd(*(g[k] for k in BWD), states=states)
    cut = lambda t: torch.cat([t[0, :at], t[0, at + 1:]])
    for k in ("dx", "di"):
        ref.check(cut(got[k]), cut(gw[k]), cut(gb[k]), dtype, k)
        ref.check(got[k][1:], gw[k][1:], gb[k][1:], dtype, k)
    ref.check(got["dr"][0, :at], gw["dr"][0, :at], gb["dr"][0, :at], dtype, "dr")
    ref.check(got["dh0"], gw["dh0"], gb["dh0"], what="dh0")


def test_refusals_on_another_stream(ssm):
    """Outputs and states elsewhere than on the call's device are refused alike on any stream."""
    g = cuda(make(2, 70, 8, F32, seed=13, h0=True))
    args, w = [g[k] for k in FWD], torch.ones(8, device="cuda")
    here = torch.zeros(2, 70, 8)
    other = torch.cuda.Stream()
    for s in (None, other):
        for bad in (lambda: ssm.gated_scan_fwd(*args, out=here, stream=s),
                    lambda: ssm.gated_scan_fwd(*args, h_last=here[:, 0], stream=s),
                    lambda: ssm.gated_scan_bwd(*(g[k] for k in BWD), states=here[:, :2], stream=s),
                    lambda: ssm.gated_step(*(g[k][:, 0] for k in "xri"), g["lam"], g["h0"], out=here[:, 0], stream=s),
                    lambda: ssm.layer_norm_fwd(g["x"], w, out=here, stream=s),
                    lambda: ssm.layer_norm_fwd(g["x"], w, None, g["dy"], residual_out=here, stream=s)):
            with pytest.raises(ValueError):
                bad()


@pytest.mark.parametrize("kind", ["tensor", "ScanWorkspace"])
def test_a_workspace_is_held_on_another_stream(ssm, kind):
    """A caller's workspace dropped right after a call on another stream is not handed out again before that call has run."""
    g = cuda(make(2, 600, 96, F32, seed=14, h0=True))
    args, grads, w = [g[k] for k in FWD], [g[k] for k in BWD], torch.ones(96, device="cuda")
    _, states = ssm.gated_scan_fwd(*args, return_states=True)
    _, mean, rstd = ssm.layer_norm_fwd(g["x"], w, return_stats=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for call in (lambda ws: ssm.gated_scan_fwd(*args, workspace=ws, stream=s),
                 lambda ws: ssm.gated_scan_bwd(*grads, states=states, workspace=ws, stream=s),
                 lambda ws: ssm.layer_norm_bwd(g["x"], g["x"], w, mean, rstd, workspace=ws, stream=s)):
        buf = torch.empty(5 << 20, dtype=torch.uint8, device="cuda")
        at, ws = buf.data_ptr(), buf
        if kind == "ScanWorkspace":
            ws = ssm.ScanWorkspace()
            ws.buf = buf
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(200_000_000)  # about 0.1 s
        out = call(ws)
        del buf, ws
        again = torch.empty(5 << 20, dtype=torch.uint8, device="cuda")
        busy = not s.query()
        torch.cuda.synchronize()
        assert busy and again.data_ptr() != at
        del out, again


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 1, 3), (2, 64, 70), (2, 65, 70), (3, 190, 64), (1, 700, 200), (1, 1100, 33), (4, 300, 2048), (40, 130, 600),
                                  (1, 6000, 5120), (1, 50000, 72), (300, 3, 7), (2500, 16, 8), (300, 30, 64), (300, 64, 64), (40, 32, 5120),
                                  (40, 16, 5120)],
                         ids=lambda s: "x".join(map(str, s)))
def test_calls_keep_to_their_workspace(ssm, size, dtype):
    """With exactly the bytes asked for, and whatever they hold, results are as with scratch of the call's own, and what lies behind stays."""
    import ctypes
    from selective_state_space_47_b200 import _native
    B, L, D = size
    gen = torch.Generator(device="cuda").manual_seed(B + L + D)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    x, r, i, dy = (n(B, L, D).to(dtype) for _ in range(4))
    lam, h0, dl = n(D) - 3, n(B, D), n(B, D)
    a, b = _native.GatedArgs(), _native.GatedBwdArgs()
    for q in (a, b):
        q.batch, q.seqlen, q.dim, q.dtype, q.c = B, L, D, ssm._TOKEN_DTYPES[dtype], 8.0
    fore = _native.lib().ssm_gated_scan_workspace_size(ctypes.byref(a))
    back = _native.lib().ssm_gated_scan_bwd_workspace_size(ctypes.byref(b))
    def exactly(nbytes):
        buf = torch.full((nbytes + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        return buf, buf[:nbytes]
    y, h, st = ssm.gated_scan_fwd(x, r, i, lam, h0, return_last_state=True, return_states=True)
    buf, ws = exactly(fore)
    for p, q in zip((y, h, st), ssm.gated_scan_fwd(x, r, i, lam, h0, return_last_state=True, return_states=True, workspace=ws)):
        assert torch.equal(p, q)
    assert ssm.workspace_status(ws) == 0 and (buf[fore:] == 0xA5).all()
    want = ssm.gated_scan_bwd(x, r, i, lam, dy, h0, dl, states=st)
    buf, ws = exactly(back)
    got = ssm.gated_scan_bwd(x, r, i, lam, dy, h0, dl, states=st, workspace=ws)
    for k in want:
        assert torch.equal(want[k], got[k]), k
    assert ssm.workspace_status(ws) == 0 and (buf[back:] == 0xA5).all()


def test_a_dropped_handoff_is_reported(ssm):
    """A state that a segment does not hand on (a test hook of the library) makes its successor's bounded wait run out,
    forward and backward: the workspace's status says so, and so does the device's where the scratch is gone; the calls
    after it are right."""
    from selective_state_space_47_b200 import _native
    B, L, D = 1, 6000, 5120  # 80 columns of 47 tiles (94 in the backward): segments handed on in turn
    gen = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    x, r, i, dy = (n(B, L, D).to(BF16) for _ in range(4))
    lam = torch.full((D,), -4.0, device="cuda")
    drop, late = _native.SSM_TEST_DROP_HANDOFF, _native.SSM_ERR_TIMEOUT
    y, st = ssm.gated_scan_fwd(x, r, i, lam, return_states=True)
    want = ssm.gated_scan_bwd(x, r, i, lam, dy, states=st)
    assert ssm.gated_status() == 0
    ws = ssm.ScanWorkspace()
    for call, right in ((lambda **k: ssm.gated_scan_fwd(x, r, i, lam, **k), y),
                        (lambda **k: ssm.gated_scan_bwd(x, r, i, lam, dy, states=st, **k)["dx"], want["dx"])):
        call(_test_flags=drop)
        assert ssm.gated_status() == late and ssm.gated_status("cuda") == 0
        call(_test_flags=drop, workspace=ws)
        assert ssm.workspace_status(ws) == late and ssm.gated_status(stream=torch.cuda.current_stream()) == late
        assert torch.equal(call(workspace=ws), right) and torch.equal(call(), right)
        assert ssm.workspace_status(ws) == 0 and ssm.gated_status(0) == 0


@pytest.mark.parametrize("extras", [False, True], ids=["plain", "h0_reset"])
@pytest.mark.parametrize("B,L,D,dtype", [(4, 700, 517, F32), (8, 700, 330, F32), (8, 700, 330, BF16), (4, 700, 517, BF16), (5, 333, 320, BF16),
                                         (5, 333, 320, F32), (30, 200, 66, F32), (30, 200, 66, BF16)])
def test_every_loader_over_several_rounds(ssm, B, L, D, dtype, extras):
    """More than 24 columns of several tiles each, by TMA, in pieces of two elements and one by one."""
    d = make(B, L, D, dtype, seed=B * L + D, h0=extras, reset=0.01 if extras else 0.0, slow=not extras)
    g = cuda(d)
    _, (_, _, states) = check_fwd(ssm, d, g, dtype)
    check_bwd(ssm, d, g, dtype, states)


@pytest.mark.parametrize("B,L,D,dtype", [(1, 6000, 5120, BF16), (1, 5000, 2050, F32), (1, 9001, 1030, BF16), (1, 9001, 1031, BF16),
                                         (2, 3000, 5120, F32), (1, 30000, 72, F32)])
def test_dlam_over_segments_blocks_and_warps(ssm, B, L, D, dtype):
    """dlam of chosen channels, a sum over everything that a plan cuts time and sequences into, against the formula over all
    sequences."""
    gen = torch.Generator(device="cuda").manual_seed(D - L)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    g = {k: n(B, L, D).clamp(-6, 6).to(dtype) for k in ("x", "r", "i", "dy")}
    g["lam"] = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * torch.rand(D, device="cuda", generator=gen)) / 8.0))
    g["h0"], g["dh_last"] = n(B, D), n(B, D)
    reset = torch.rand(B, L, device="cuda", generator=gen) < 1e-3
    got = ssm.gated_scan_bwd(*(g[k] for k in BWD), reset=reset)
    sel = torch.tensor([0, 1, 63, 64, D // 2, D - 2, D - 1], device="cuda")
    d = {k: v.index_select(v.dim() - 1, sel).cpu() for k, v in g.items()}
    want, bound = ref.gated_scan_bwd(*(d[k] for k in BWD), reset=reset.cpu())
    for k in want:
        ref.check(got[k].index_select(got[k].dim() - 1, sel), want[k], bound[k], dtype if k in ("dx", "dr", "di") else F32, k)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,L,D", [(3, 150, 64), (2, 200, 33), (300, 9, 24), (40, 1, 64)], ids=lambda n: str(n))
def test_tokens_laid_out_step_by_step(ssm, B, L, D, dtype):
    """Tokens [L, B, D] in memory: the sequences lie closer together than the steps. In the step kernel too."""
    d = make(B, L, D, dtype, seed=B + L + D, h0=True, reset=0.02)
    g = cuda(d)
    for k in "xri":
        g[k] = g[k].transpose(0, 1).contiguous().transpose(0, 1)
    _, (y, _, states) = check_fwd(ssm, d, g, dtype)
    check_bwd(ssm, d, g, dtype, states)
    h = g["h0"].clone()
    d["reset"] = None
    want, bound = ref.gated_scan(*(d[k][:, :1] if k in "xri" else d[k] for k in FWD))
    out = ssm.gated_step(*(g[k][:, 0] for k in "xri"), g["lam"], h)
    ref.check(out, want[:, 0], bound[:, 0], dtype, "y")
    ref.check(h, want[:, 0], bound[:, 0], what="h")


@pytest.mark.parametrize("extras", [False, True], ids=["plain", "h0_reset"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,L,D", [(3, 1, 200), (3, 2, 200), (3, 3, 200), (3, 4, 200), (3, 5, 200), (3, 6, 200), (3000, 9, 7), (2500, 16, 6), (2500, 20, 4),
                                   (2500, 21, 4), (3000, 12, 5), (700, 16, 258), (700, 17, 257), (90, 32, 2050), (90, 33, 2048), (180, 24, 2049),
                                   (180, 25, 2048)], ids=lambda n: str(n))
def test_the_few_token_kernels_up_to_their_borders(ssm, B, L, D, dtype, extras):
    """Sizes at both sides of the rules that choose between a thread a channel and tiles, in every width of a thread's piece."""
    d = make(B, L, D, dtype, seed=B + L + D, h0=extras, reset=0.1 if extras else 0.0, slow=not extras)
    g = cuda(d)
    if extras:  # slices of one projection
        both = torch.cat([g["r"], g["i"]], 2)
        g["r"], g["i"] = both[:, :, :D], both[:, :, D:]
    _, (_, _, states) = check_fwd(ssm, d, g, dtype)
    got = check_bwd(ssm, d, g, dtype, states)
    again = ssm.gated_scan_bwd(*(g[k] for k in BWD), reset=g["reset"])
    for k in got:
        assert torch.equal(got[k], again[k]), k


def test_the_few_token_kernels_at_the_gates_ends(ssm):
    """By threads, as by tiles: tiny rates keep their weight, a closed gate holds the state exactly with finite gradients, and a
    reset keeps an infinity or NaN of what came before out of what follows."""
    B, L, D = 1500, 9, 12
    d = make(B, L, D, F32, seed=6, h0=True)
    d["lam"] = torch.linspace(-60, -8, D)
    g = cuda(d)
    _, (_, _, states) = check_fwd(ssm, d, g, F32)
    check_bwd(ssm, d, g, F32, states)
    d["r"][:] = float("-inf")
    g = cuda(d)
    y, h, states = ssm.gated_scan_fwd(*(g[k] for k in FWD), return_last_state=True, return_states=True)
    assert torch.equal(y, g["h0"][:, None].expand(-1, L, -1)) and torch.equal(h, g["h0"])
    got = ssm.gated_scan_bwd(g["x"], g["r"], g["i"], g["lam"], g["dy"], None, g["dh_last"], states=states)
    for k in ("dx", "dr", "di", "dlam"):
        assert torch.equal(got[k], torch.zeros_like(got[k])), k
    d = make(B, L, D, F32, seed=9, h0=True)
    d["reset"] = torch.zeros(B, L, dtype=torch.bool)
    d["reset"][:, 4] = True
    bad = {k: None if v is None else v.clone() for k, v in d.items()}
    bad["h0"][0] = float("inf")
    bad["x"][1, 2] = NAN
    bad["dy"][2, 6] = NAN
    g = cuda(bad)
    y, states = ssm.gated_scan_fwd(*(g[k] for k in FWD), reset=g["reset"], return_states=True)
    want, bound = ref.gated_scan(*(d[k] for k in FWD), reset=d["reset"])
    ref.check(y[:, 4:], want[:, 4:], bound[:, 4:], what="y after the reset")
    ref.check(y[2:], want[2:], bound[2:], what="y")
    got = ssm.gated_scan_bwd(g["x"], g["r"], g["i"], g["lam"], g["dy"], None, g["dh_last"], states=states, reset=g["reset"])
    want, bound = ref.gated_scan_bwd(*(d[k] for k in BWD), reset=d["reset"])
    for k in ("dx", "dr", "di"):
        ref.check(got[k][:2, 4:], want[k][:2, 4:], bound[k][:2, 4:], what=k)
        ref.check(got[k][2, :4], want[k][2, :4], bound[k][2, :4], what=k)
        ref.check(got[k][3:], want[k][3:], bound[k][3:], what=k)


def test_two_calls_at_once(ssm):
    """Calls that hand segments on in turn, on two streams that share the GPU, each forward and backward: the same bits as alone."""
    B, L, D = 1, 6000, 5120
    gen = torch.Generator(device="cuda").manual_seed(5)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    x, r, i, dy = (n(B, L, D).to(BF16) for _ in range(4))
    lam = torch.full((D,), -4.0, device="cuda")
    def both(a):
        y, st = ssm.gated_scan_fwd(a, r, i, lam, return_states=True)
        return (y, *ssm.gated_scan_bwd(a, r, i, lam, dy, states=st).values())
    want = [both(a) for a in (x, dy)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(6):
        for a, s in zip((x, dy), streams):
            with torch.cuda.stream(s):
                got.append(both(a))
    torch.cuda.synchronize()
    for k, res in enumerate(got):
        for p, q in zip(res, want[k % 2]):
            assert torch.equal(p, q)
    assert ssm.gated_status() == 0


def test_offsets_beyond_32_bits(ssm):
    """2.2e9 elements a tensor: the last steps of the last sequence, forward from their kept state and backward from the end,
    against the formulas; and the first steps of the first."""
    B, L, D = 2, 215041, 5120
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.empty(B, L, D, device="cuda", dtype=BF16).normal_(generator=gen).clamp_(-6, 6)
    lam = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * torch.rand(D, device="cuda", generator=gen)) / 8.0))
    y, h, states = ssm.gated_scan_fwd(x, x, x, lam, return_last_state=True, return_states=True)
    sel = torch.tensor([0, 1, 2559, D - 1], device="cuda")
    pick = lambda t: t.index_select(t.dim() - 1, sel).cpu()
    t0 = L // 64 * 64 - 64  # a whole chunk and the last, short one
    tail, l4 = pick(x[1:, t0:]), lam[sel].cpu()
    want, bound = ref.gated_scan(tail, tail, tail, l4, pick(states[1:, t0 // 64]))
    ref.check(pick(y[1:, t0:]), want, bound, BF16, "y")
    ref.check(pick(h[1:]), want[:, -1], bound[:, -1], what="h_last")
    head = pick(x[:1, :200])
    want, bound = ref.gated_scan(head, head, head, l4)
    ref.check(pick(y[:1, :200]), want, bound, BF16, "y")
    del y
    g = ssm.gated_scan_bwd(x, x, x, lam, x, states=states)
    want, bound = ref.gated_scan_bwd(tail, tail, tail, l4, tail, pick(states[1:, t0 // 64]))
    for k in ("dx", "dr", "di"):
        ref.check(pick(g[k][1:, t0:]), want[k], bound[k], BF16, k)
    assert all(torch.isfinite(g[k]).all() for k in ("dlam", "dh0"))
    del g, states
    # beyond 65535 sequences of a few tokens
    d = make(70000, 2, 12, F32, seed=70, h0=True, reset=0.2)
    c = cuda(d)
    _, (_, _, states) = check_fwd(ssm, d, c, F32)
    check_bwd(ssm, d, c, F32, states)


def test_a_training_step_captured(ssm):
    """Norm, recurrence and their backward by autograd in one graph, replayed on new values, against the same step eager. No eager
    graph of the captured leaves lives meanwhile (autograd would tie its stream into the capture)."""
    B, L, D = 2, 300, 64
    d = make(B, L, D, F32, seed=15, h0=True, reset=0.02)
    g = cuda(d)
    leaf = {k: g[k].clone().requires_grad_(True) for k in FWD}
    w, b, s0 = (torch.ones(D, device="cuda").requires_grad_(True), torch.zeros(D, device="cuda").requires_grad_(True), torch.randn(B, L, D, device="cuda"))
    inputs = [*leaf.values(), w, b]
    def step():
        z, s = ssm.layer_norm(leaf["x"], w, b, s0)
        y, h = ssm.gated_scan(z, leaf["r"], leaf["i"], leaf["lam"], leaf["h0"], reset=g["reset"], return_last_state=True)
        return [y.detach(), h.detach(), *torch.autograd.grad([y, h, s], inputs, [g["dy"], g["dh_last"], s0])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for scale in (1.0, 0.7, 1.3):
        with torch.no_grad():
            for k in ("x", "r"):
                leaf[k].copy_(g[k] * scale)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, step()):
            assert torch.equal(p, q)
