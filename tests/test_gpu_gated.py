"""GPU checks of the gated linear recurrence (scan, backward, step) against its float64
form, elementwise within the bounds derived there."""
import subprocess
import sys

import pytest
import torch

from tests import operators_ref as ref
from tests.conftest import ROOT, cuda_available

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssm():
    if not cuda_available():
        pytest.skip("needs a CUDA device")
    import selective_state_space_47_b200 as m
    return m


def make(B, L, D, dtype, seed, h0=False, reset=0.0, slow=True):
    """Inputs as such a layer sees them: gates around 0 (|v| <= 6), decays between 0.9 and 0.999 a step, or
    (slow false) rates from next to nothing to forgetting at once."""
    gen = torch.Generator().manual_seed(seed)
    tok = lambda: torch.randn(B, L, D, generator=gen).clamp(-6, 6).to(dtype)
    d = dict(x=tok(), r=tok(), i=tok())
    q = torch.rand(D, generator=gen)
    d["lam"] = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * q) / 8.0)) if slow else 16 * q - 12
    d["h0"] = torch.randn(B, D, generator=gen) if h0 else None
    d["reset"] = (torch.rand(B, L, generator=gen) < reset) if reset else None
    d["dy"] = tok()
    d["dh_last"] = torch.randn(B, D, generator=gen) if h0 else None
    return d


def cuda(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


FWD = ("x", "r", "i", "lam", "h0")


def check_fwd(ssm, d, g, dtype):
    y_ref, bound = ref.gated_scan(*(d[k] for k in FWD), reset=d["reset"])
    y, h, states = ssm.gated_scan_fwd(*(g[k] for k in FWD), reset=g["reset"], return_last_state=True, return_states=True)
    torch.cuda.synchronize()
    w = [ref.check(y, y_ref, bound, dtype, "y"), ref.check(h, y_ref[:, -1], bound[:, -1], what="h_last")]
    if y_ref.shape[1] > 64:
        w.append(ref.check(states[:, 1:], y_ref[:, 63:-1:64], bound[:, 63:-1:64], what="states"))
    first = torch.zeros_like(d["lam"]).expand(y_ref.shape[0], -1) if d["h0"] is None else d["h0"]
    assert torch.equal(states[:, 0].cpu(), first)
    return w, (y, h, states)


def check_bwd(ssm, d, g, dtype, states):
    want, bound = ref.gated_scan_bwd(*(d[k] for k in ("x", "r", "i", "lam", "dy", "h0", "dh_last")), reset=d["reset"])
    got = ssm.gated_scan_bwd(*(g[k] for k in ("x", "r", "i", "lam", "dy", "h0", "dh_last")), states=states, reset=g["reset"])
    torch.cuda.synchronize()
    for k in want:
        ref.check(got[k], want[k], bound[k], dtype if k in ("dx", "dr", "di") else torch.float32, k)
    return got


SIZES = [(1, 1, 1), (2, 1, 64), (3, 2, 31), (1, 63, 64), (2, 64, 33), (2, 65, 66), (1, 127, 130), (5, 128, 2),
         (2, 129, 7), (1, 300, 200), (2, 1025, 40), (1, 3000, 10), (2, 70, 8), (1, 200, 16), (300, 5, 24), (1, 65, 264)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("extras", [False, True], ids=["plain", "h0_reset"])
def test_scan_and_backward(ssm, size, dtype, extras):
    d = make(*size, dtype, seed=sum(size), h0=extras, reset=0.02 if extras else 0.0, slow=not extras)
    g = cuda(d)
    _, (_, _, states) = check_fwd(ssm, d, g, dtype)
    check_bwd(ssm, d, g, dtype, states)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("every", [1, 2, 64, 128], ids=lambda n: f"every{n}")
def test_resets_on_and_off_the_borders(ssm, dtype, every):
    """Resets at each step, each second one, and at the first or the last step of pieces of time."""
    for shift in (0, every - 1):
        d = make(2, 400, 34, dtype, seed=every + shift, h0=True)
        d["reset"] = torch.zeros(2, 400, dtype=torch.bool)
        d["reset"][:, shift::every] = True
        g = cuda(d)
        _, (_, _, states) = check_fwd(ssm, d, g, dtype)
        check_bwd(ssm, d, g, dtype, states)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_strided_and_misaligned_tokens(ssm, dtype):
    """Slices of one projection, also ones that start on an odd element or have an odd stride."""
    B, L, D = 2, 150, 48
    d = make(B, L, D, dtype, seed=5)
    for width, at in ((3 * D, (0, D, 2 * D)), (3 * D + 7, (1, D + 3, 2 * D + 6)), (3 * D + 2, (0, D, 2 * D + 1))):
        buf = torch.full((B, L, width), float("nan"), dtype=dtype, device="cuda")
        g = cuda(d)
        for k, o in zip("xri", at):
            buf[:, :, o:o + D] = g[k]
            g[k] = buf[:, :, o:o + D]
        _, (_, _, states) = check_fwd(ssm, d, g, dtype)
        check_bwd(ssm, d, g, dtype, states)
    # a sequence of which every second step is read, and one shared by the batch (stride 0)
    g = cuda(d)
    d2 = {k: (v[:, ::2] if k in ("x", "r", "i", "dy") else v) for k, v in d.items()}
    g2 = {k: (v[:, ::2] if k in ("x", "r", "i") else v) for k, v in g.items()}
    d2["r"] = d2["r"][:1].expand(B, -1, -1)
    g2["r"] = g2["r"][:1].expand(B, -1, -1)
    g2["dy"] = g["dy"][:, ::2].contiguous()
    _, (_, _, states) = check_fwd(ssm, d2, g2, dtype)
    check_bwd(ssm, d2, g2, dtype, states)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,L,D", [(256, 1, 64), (300, 4, 70), (64, 16, 260), (257, 31, 65), (256, 32, 12), (256, 33, 12), (2500, 3, 8),
                                   (52, 7, 321)])
def test_a_few_tokens_of_many_sequences(ssm, B, L, D, dtype):
    for extras in (False, True):
        d = make(B, L, D, dtype, seed=B + L, h0=extras, reset=0.1 if extras else 0.0, slow=not extras)
        g = cuda(d)
        if extras:  # slices of one projection
            both = torch.cat([g["r"], g["i"]], 2)
            g["r"], g["i"] = both[:, :, :D], both[:, :, D:]
        _, (_, _, states) = check_fwd(ssm, d, g, dtype)
        got = check_bwd(ssm, d, g, dtype, states)
        again = ssm.gated_scan_bwd(*(g[k] for k in ("x", "r", "i", "lam", "dy", "h0", "dh_last")), reset=g["reset"])
        for k in got:
            assert torch.equal(got[k], again[k]), k


def test_a_few_tokens_at_the_gates_ends(ssm):
    """As the long sequences: tiny rates keep their weight, a closed gate holds the state exactly with finite
    gradients, and a reset keeps an infinity of the state before it out of what follows."""
    B, L, D = 300, 9, 12
    d = make(B, L, D, torch.float32, seed=6, h0=True)
    d["lam"] = torch.linspace(-60, -8, D)
    g = cuda(d)
    _, (_, _, states) = check_fwd(ssm, d, g, torch.float32)
    check_bwd(ssm, d, g, torch.float32, states)
    d["r"][:] = float("-inf")
    g = cuda(d)
    y, h, states = ssm.gated_scan_fwd(*(g[k] for k in FWD), return_last_state=True, return_states=True)
    assert torch.equal(y, g["h0"][:, None].expand(-1, L, -1)) and torch.equal(h, g["h0"])
    got = ssm.gated_scan_bwd(g["x"], g["r"], g["i"], g["lam"], g["dy"], None, g["dh_last"], states=states)
    for k in ("dx", "dr", "di", "dlam"):
        assert torch.equal(got[k], torch.zeros_like(got[k])), k
    d = make(B, L, D, torch.float32, seed=9, h0=True)
    d["reset"] = torch.zeros(B, L, dtype=torch.bool)
    d["reset"][:, 4] = True
    bad = {k: None if v is None else v.clone() for k, v in d.items()}
    bad["h0"][0] = float("inf")
    bad["x"][1, 2] = float("nan")
    bad["dy"][2, 6] = float("nan")
    g = cuda(bad)
    y, states = ssm.gated_scan_fwd(*(g[k] for k in FWD), reset=g["reset"], return_states=True)
    want, bound = ref.gated_scan(*(d[k] for k in FWD), reset=d["reset"])
    ref.check(y[:, 4:], want[:, 4:], bound[:, 4:], what="y after the reset")
    ref.check(y[2:], want[2:], bound[2:], what="y")
    got = ssm.gated_scan_bwd(g["x"], g["r"], g["i"], g["lam"], g["dy"], None, g["dh_last"], states=states, reset=g["reset"])
    want, bound = ref.gated_scan_bwd(*(d[k] for k in ("x", "r", "i", "lam", "dy", "h0", "dh_last")), reset=d["reset"])
    for k in ("dx", "dr", "di"):
        ref.check(got[k][:2, 4:], want[k][:2, 4:], bound[k][:2, 4:], what=k)
        ref.check(got[k][2, :4], want[k][2, :4], bound[k][2, :4], what=k)
        ref.check(got[k][3:], want[k][3:], bound[k][3:], what=k)


def test_long_sequences(ssm):
    """Many tiles in a row: a few channels over 40000 steps, and several groups of channels."""
    for B, L, D, dtype in ((1, 40000, 3, torch.float32), (2, 9000, 130, torch.bfloat16)):
        d = make(B, L, D, dtype, seed=L, h0=True, reset=1e-4)
        g = cuda(d)
        _, (_, _, states) = check_fwd(ssm, d, g, dtype)
        check_bwd(ssm, d, g, dtype, states)


@pytest.mark.parametrize("B,L,D,dtype", [(1, 6000, 5120, torch.bfloat16), (3, 5000, 1536, torch.bfloat16),
                                         (4, 3000, 2048, torch.float32), (1, 9001, 1030, torch.bfloat16),
                                         (1, 50000, 72, torch.bfloat16), (2, 6001, 515, torch.bfloat16),
                                         (2, 6001, 515, torch.float32)])
def test_every_way_of_dealing_out_time(ssm, B, L, D, dtype):
    """More columns than the GPU takes at once (segments handed on in turn), fewer (clusters share a column) and
    very few (two passes): three channels against the reference, and five runs bit for bit."""
    gen = torch.Generator(device="cuda").manual_seed(D + L)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    g = {k: n(B, L, D).clamp(-6, 6).to(dtype) for k in ("x", "r", "i", "dy")}
    g["lam"] = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * torch.rand(D, device="cuda", generator=gen)) / 8.0))
    g["h0"], g["dh_last"] = n(B, D), n(B, D)
    g["reset"] = torch.rand(B, L, device="cuda", generator=gen) < 1e-3
    args, grads = [g[k] for k in FWD], [g[k] for k in ("x", "r", "i", "lam", "dy", "h0", "dh_last")]
    run = lambda: (ssm.gated_scan_fwd(*args, reset=g["reset"], return_last_state=True, return_states=True))
    y, h, states = run()
    got = ssm.gated_scan_bwd(*grads, states=states, reset=g["reset"])
    for _ in range(4):
        for a, b in zip((y, h, states), run()):
            assert torch.equal(a, b)
        again = ssm.gated_scan_bwd(*grads, states=states, reset=g["reset"])
        for k in got:
            assert torch.equal(got[k], again[k]), k
    sel = torch.tensor([0, D // 2, D - 1], device="cuda")
    cut = lambda t: t[B - 1:].index_select(t.dim() - 1, sel).cpu()
    d = {k: cut(v) for k, v in g.items() if k not in ("lam", "reset")}
    lam, reset = g["lam"][sel].cpu(), g["reset"][B - 1:].cpu()
    want, bound = ref.gated_scan(d["x"], d["r"], d["i"], lam, d["h0"], reset)
    ref.check(cut(y), want, bound, dtype, "y")
    ref.check(cut(h), want[:, -1], bound[:, -1], what="h_last")
    want, bound = ref.gated_scan_bwd(d["x"], d["r"], d["i"], lam, d["dy"], d["h0"], d["dh_last"], reset)
    for k in ("dx", "dr", "di", "dh0"):
        ref.check(cut(got[k]), want[k], bound[k], torch.float32 if k == "dh0" else dtype, k)


def test_workspaces(ssm):
    """A caller's workspace is used, reports its status, and is refused when too small or elsewhere."""
    d = make(2, 900, 192, torch.bfloat16, seed=51, h0=True)
    g = cuda(d)
    args, grads = [g[k] for k in FWD], [g[k] for k in ("x", "r", "i", "lam", "dy", "h0", "dh_last")]
    want, states = ssm.gated_scan_fwd(*args, return_states=True)
    ws = ssm.ScanWorkspace()
    for _ in range(3):
        assert torch.equal(ssm.gated_scan_fwd(*args, workspace=ws), want)
        assert ssm.workspace_status(ws) == 0
        ws.buf.fill_(255)  # what a call finds there does not matter
        got = ssm.gated_scan_bwd(*grads, states=states, workspace=ws)
        assert ssm.workspace_status(ws) == 0
        ws.buf.fill_(255)
    first = ssm.gated_scan_bwd(*grads, states=states)
    for k in got:
        assert torch.equal(got[k], first[k]), k
    for bad in (torch.empty(64, dtype=torch.uint8, device="cuda"), torch.empty(1 << 24, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            ssm.gated_scan_fwd(*args, workspace=bad)
        with pytest.raises(ValueError):
            ssm.gated_scan_bwd(*grads, states=states, workspace=bad)


def test_first_call_captured():
    """A process whose first call is made while a graph is captured."""
    if not cuda_available():
        pytest.skip("needs a CUDA device")
    code = """
import torch, selective_state_space_47_b200 as ssm
x = torch.randn(2, 500, 64, device="cuda"); lam = torch.zeros(64, device="cuda"); w = torch.ones(64, device="cuda")
def run():
    y, st = ssm.gated_scan_fwd(x, x, x, lam, return_states=True)
    n, m, k = ssm.layer_norm_fwd(y, w, return_stats=True)
    return [y, n, *ssm.gated_scan_bwd(x, x, x, lam, x, states=st).values(), *ssm.layer_norm_bwd(x, y, w, m, k).values()]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a = run()
g.replay()
b = run()
torch.cuda.synchronize()
assert all(p is q is None or torch.equal(p, q) for p, q in zip(a, b))
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT, timeout=120)


def test_a_reset_drops_what_came_before(ssm):
    """Infinities and NaN in one document, or in h0, stay out of the next, in both directions; the documents
    without them are as if alone."""
    d = make(2, 500, 34, torch.float32, seed=9, h0=True)
    d["reset"] = torch.zeros(2, 500, dtype=torch.bool)
    d["reset"][:, 200] = True
    d["reset"][:, 333] = True
    bad = {k: None if v is None else v.clone() for k, v in d.items()}
    bad["h0"][0] = float("inf")
    bad["x"][0, 17] = float("nan")
    bad["x"][1, 250] = float("inf")
    bad["dy"][0, 400] = float("nan")
    g = cuda(bad)
    y, states = ssm.gated_scan_fwd(*(g[k] for k in FWD), reset=g["reset"], return_states=True)
    want, bound = ref.gated_scan(*(d[k] for k in FWD), reset=d["reset"])
    ref.check(y[0, 200:], want[0, 200:], bound[0, 200:], what="y after the NaN's document")
    ref.check(y[1, :200], want[1, :200], bound[1, :200], what="y before")
    ref.check(y[1, 333:], want[1, 333:], bound[1, 333:], what="y after the infinity's document")
    assert not torch.isfinite(y[0, 17:200]).any() and not torch.isfinite(y[1, 250:333]).any()
    got = ssm.gated_scan_bwd(g["x"], g["r"], g["i"], g["lam"], g["dy"], None, g["dh_last"], states=states, reset=g["reset"])
    want, bound = ref.gated_scan_bwd(*(d[k] for k in ("x", "r", "i", "lam", "dy", "h0", "dh_last")), reset=d["reset"])
    for k in ("dx", "dr", "di"):
        ref.check(got[k][0, 200:333], want[k][0, 200:333], bound[k][0, 200:333], what=k)
        ref.check(got[k][1, :200], want[k][1, :200], bound[k][1, :200], what=k)
        ref.check(got[k][1, 333:], want[k][1, 333:], bound[k][1, 333:], what=k)


def test_gates_at_their_ends(ssm):
    """A closed decay gate (w = 0) holds the state exactly and has finite gradients; an open one forgets."""
    B, L, D = 2, 200, 6
    for r in (-200.0, float("-inf")):
        d = make(B, L, D, torch.float32, seed=3, h0=True)
        d["r"][:] = r
        g = cuda(d)
        y, h, states = ssm.gated_scan_fwd(*(g[k] for k in FWD), return_last_state=True, return_states=True)
        assert torch.equal(y, g["h0"][:, None].expand(-1, L, -1)) and torch.equal(h, g["h0"])
        got = ssm.gated_scan_bwd(g["x"], g["r"], g["i"], g["lam"], g["dy"], None, g["dh_last"], states=states)
        for k in ("dx", "dr", "di", "dlam"):
            assert torch.equal(got[k], torch.zeros_like(got[k])), k
        want = d["dy"].double().sum(1) + d["dh_last"].double()
        tol = (L + 2) * ref.U * (d["dy"].abs().double().sum(1) + d["dh_last"].abs())
        ref.check(got["dh0"], want, tol, what="dh0")
    d = make(B, L, D, torch.float32, seed=4, h0=True, slow=False)
    d["lam"][:] = 30.0  # a = exp(-240 sigmoid(r)): no memory at all
    d["r"][:] = 200.0
    d["i"][:] = float("inf")
    g = cuda(d)
    y = ssm.gated_scan_fwd(*(g[k] for k in FWD))
    assert torch.equal(y, g["x"])


def test_small_rates_keep_their_weight(ssm):
    """Rates so small that a rounds to 1: the input's weight sqrt(2 w) still counts, and so do gradients."""
    d = make(2, 300, 12, torch.float32, seed=6, h0=True)
    d["lam"] = torch.linspace(-60, -8, 12)
    g = cuda(d)
    _, (_, _, states) = check_fwd(ssm, d, g, torch.float32)
    check_bwd(ssm, d, g, torch.float32, states)


def test_empty_calls(ssm):
    z = lambda *s: torch.zeros(*s, device="cuda")
    lam, h0 = z(8), torch.randn(2, 8, device="cuda")
    y, h = ssm.gated_scan_fwd(z(2, 0, 8), z(2, 0, 8), z(2, 0, 8), lam, h0, return_last_state=True)
    assert y.shape == (2, 0, 8) and torch.equal(h, h0)
    _, h = ssm.gated_scan_fwd(z(2, 0, 8), z(2, 0, 8), z(2, 0, 8), lam, return_last_state=True)
    assert torch.equal(h, z(2, 8))
    g = ssm.gated_scan_bwd(z(2, 0, 8), z(2, 0, 8), z(2, 0, 8), lam, z(2, 0, 8), h0, h0)
    assert torch.equal(g["dh0"], h0) and torch.equal(g["dlam"], z(8))
    g = ssm.gated_scan_bwd(z(0, 5, 8), z(0, 5, 8), z(0, 5, 8), lam, z(0, 5, 8))
    assert torch.equal(g["dlam"], z(8)) and g["dx"].shape == (0, 5, 8)
    assert ssm.gated_scan_fwd(z(0, 5, 8), z(0, 5, 8), z(0, 5, 8), lam).shape == (0, 5, 8)
    assert ssm.gated_scan_fwd(z(2, 5, 0), z(2, 5, 0), z(2, 5, 0), z(0)).shape == (2, 5, 0)
    assert ssm.gated_step(z(0, 8), z(0, 8), z(0, 8), lam, z(0, 8)).shape == (0, 8)


def test_results_repeat_and_states_are_recomputed(ssm):
    """Bit for bit: the same call twice, the backward with and without the forward's states, and the
    outputs whatever else is asked for."""
    d = make(3, 2000, 70, torch.bfloat16, seed=21, h0=True, reset=0.003)
    g = cuda(d)
    args = [g[k] for k in FWD]
    y, h, states = ssm.gated_scan_fwd(*args, reset=g["reset"], return_last_state=True, return_states=True)
    b = [g[k] for k in ("x", "r", "i", "lam", "dy", "h0", "dh_last")]
    first = ssm.gated_scan_bwd(*b, states=states, reset=g["reset"])
    for _ in range(5):
        y2, h2 = ssm.gated_scan_fwd(*args, reset=g["reset"], return_last_state=True)
        assert torch.equal(y, y2) and torch.equal(h, h2)
        again = ssm.gated_scan_bwd(*b, reset=g["reset"])
        for k in first:
            assert torch.equal(first[k], again[k]), k


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 1), (3, 7), (2, 64), (33, 130)], ids=lambda s: "x".join(map(str, s)))
def test_step_chain(ssm, size, dtype):
    """Single tokens one after the other follow the scan; h in place, or into another array."""
    B, D, L = *size, 9
    d = make(B, L, D, dtype, seed=B + D, h0=True)
    g = cuda(d)
    want, bound = ref.gated_scan(*(d[k] for k in FWD))
    h = g["h0"].clone()
    for t in range(L):
        tok = [g[k][:, t] for k in ("x", "r", "i")]  # strided rows
        other = torch.empty_like(h)
        y2 = ssm.gated_step(*tok, g["lam"], h, h_out=other)
        y = ssm.gated_step(*tok, g["lam"], h)
        assert torch.equal(y, y2) and torch.equal(h, other)
        ref.check(y, want[:, t], bound[:, t], dtype, "y")
        ref.check(h, want[:, t], bound[:, t], what="h")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,D", [(700, 1024), (4099, 258), (70001, 4)])
def test_step_of_large_batches(ssm, B, D, dtype):
    """Many sequences to a thread, batches that are no multiple of them, arrays that start off a whole piece, and
    a large rate."""
    d = make(B, 1, D, dtype, seed=B, h0=True, slow=False)
    g = cuda(d)
    want, bound = ref.gated_scan(*(d[k] for k in FWD))
    buf = torch.empty(B * D + 1, device="cuda")
    for h in (g["h0"].clone(), buf[1:].view(B, D).copy_(g["h0"])):
        y = ssm.gated_step(*(g[k][:, 0] for k in ("x", "r", "i")), g["lam"], h)
        ref.check(y, want[:, 0], bound[:, 0], dtype, "y")
        ref.check(h, want[:, 0], bound[:, 0], what="h")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_autograd(ssm, dtype):
    d = make(2, 260, 36, dtype, seed=31, h0=True, reset=0.01)
    g = cuda(d)
    leaf = {k: g[k].clone().requires_grad_(True) for k in FWD}
    y, h = ssm.gated_scan(*leaf.values(), reset=g["reset"], return_last_state=True)
    torch.autograd.backward([y, h], [g["dy"], g["dh_last"]])
    want, bound = ref.gated_scan_bwd(*(d[k] for k in ("x", "r", "i", "lam", "dy", "h0", "dh_last")), reset=d["reset"])
    for k in FWD:
        ref.check(leaf[k].grad, want["d" + k], bound["d" + k], leaf[k].dtype, "d" + k)
    # one output only, no h0: no gradient where none is asked
    x = g["x"].clone().requires_grad_(True)
    out = ssm.gated_scan(x, g["r"], g["i"], g["lam"])
    assert isinstance(out, torch.Tensor)
    gx, = torch.autograd.grad(out, x, g["dy"])
    want, bound = ref.gated_scan_bwd(*(d[k] for k in ("x", "r", "i", "lam", "dy")))
    ref.check(gx, want["dx"], bound["dx"], dtype, "dx")


def test_streams_and_graphs(ssm):
    """A call on a stream given by the caller, forward and backward captured into a graph and replayed on
    new values, and two graphs replayed at the same time."""
    d = make(2, 700, 64, torch.float32, seed=41, h0=True)
    g = cuda(d)
    y_ref, bound = ref.gated_scan(*(d[k] for k in FWD))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = ssm.gated_scan_fwd(*(g[k] for k in FWD), stream=s)
    got = ssm.gated_scan_bwd(*(g[k] for k in ("x", "r", "i", "lam", "dy", "h0", "dh_last")), stream=s)
    torch.cuda.current_stream().wait_stream(s)
    ref.check(y, y_ref, bound, what="y on a stream")
    want, wb = ref.gated_scan_bwd(*(d[k] for k in ("x", "r", "i", "lam", "dy", "h0", "dh_last")))
    for k in want:
        ref.check(got[k], want[k], wb[k], what=k)

    def both(x):
        y, st = ssm.gated_scan_fwd(x, g["r"], g["i"], g["lam"], g["h0"], return_states=True)
        return y, ssm.gated_scan_bwd(x, g["r"], g["i"], g["lam"], g["dy"], None, g["dh_last"], states=st)

    with torch.cuda.stream(s):
        both(g["x"])
    torch.cuda.synchronize()
    xs = [torch.empty_like(g["x"]) for _ in range(2)]
    graphs, outs = [], []
    for k in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[k]):
            outs.append(both(xs[k]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(2):
        xs[k].copy_(g["x"] * (k + 1))
    torch.cuda.synchronize()
    for _ in range(10):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                graphs[k].replay()
    torch.cuda.synchronize()
    for k in range(2):
        y, grads = both(g["x"] * (k + 1))
        torch.cuda.synchronize()
        assert torch.equal(outs[k][0], y)
        for n in grads:
            assert torch.equal(outs[k][1][n], grads[n]), n
