"""CPU checks of the gated recurrence's and the layer norm's entry points: the argument
structs' layout, sizes, and the calls that are refused before any launch. No compute runs."""
import ctypes
import os
import subprocess

import pytest
import torch

import selective_state_space_47_b200 as ssm
from selective_state_space_47_b200 import _native
from selective_state_space_47_b200 import build as lib_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, OK = _native.SSM_ERR_INVALID, _native.SSM_ERR_UNSUPPORTED, _native.SSM_OK
FAKE = 1 << 20  # never dereferenced: every call below fails or ends first


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return _native.lib()


@pytest.mark.parametrize("cname,pyname", [("ssm_gated_args", "GatedArgs"), ("ssm_gated_bwd_args", "GatedBwdArgs"),
                                          ("ssm_norm_args", "NormArgs"), ("ssm_norm_bwd_args", "NormBwdArgs")])
def test_struct_layouts(tmp_path, cname, pyname):
    cls = getattr(_native, pyname)
    names = [f[0] for f in cls._fields_]
    src = tmp_path / "layout.c"
    body = "".join(f'printf("%zu\\n", offsetof({cname}, {n}));' for n in names)
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "ssm_scan.h"\n'
                   f'int main(void){{ {body} printf("%zu\\n%d\\n", sizeof({cname}), SSM_GATED_CHUNK); return 0; }}\n')
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)])
    got = [int(v) for v in subprocess.check_output([str(exe)]).decode().split()]
    assert got == [getattr(cls, n).offset for n in names] + [ctypes.sizeof(cls), _native.SSM_GATED_CHUNK]


def _fill(a, names, **kw):
    for k, n in enumerate(names):
        setattr(a, n, FAKE + (k << 16))
    a.workspace, a.workspace_bytes = FAKE + (40 << 16), 1 << 40
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(a, k)[:] = v
        else:
            setattr(a, k, v)
    return a


def _gated(bwd=False, **kw):
    a = _native.GatedBwdArgs() if bwd else _native.GatedArgs()
    a.batch, a.seqlen, a.dim, a.dtype, a.c = 2, 200, 32, _native.SSM_BF16, 8.0
    for n in ("x_stride", "r_stride", "i_stride"):
        getattr(a, n)[:] = (200 * 32, 32)
    names = ("x", "r", "i", "reset", "lam") + (
        ("states", "dy", "dh_last", "dx", "dr", "di", "dlam", "dh0") if bwd else ("h0", "y", "h_last", "states"))
    return _fill(a, names, **kw)


BIG = 1 << 60
COMMON = [
    (dict(batch=-1), INVALID), (dict(seqlen=-1), INVALID), (dict(dim=-1), INVALID), (dict(dtype=5), INVALID),
    (dict(flags=1), INVALID), (dict(c=0.0), INVALID), (dict(c=-1.0), INVALID), (dict(c=float("nan")), INVALID),
    (dict(c=float("inf")), INVALID), (dict(x=None), INVALID), (dict(r=None), INVALID), (dict(i=None), INVALID),
    (dict(lam=None), INVALID), (dict(x_stride=(-1, 32)), INVALID), (dict(i_stride=(0, -2)), INVALID),
    (dict(workspace=None), INVALID), (dict(workspace_bytes=16), INVALID),
    (dict(workspace=FAKE + 8), UNSUPPORTED), (dict(x=FAKE + 1), UNSUPPORTED), (dict(i=FAKE + 3), UNSUPPORTED),
    (dict(lam=FAKE + 2), UNSUPPORTED), (dict(batch=BIG, seqlen=BIG), UNSUPPORTED), (dict(dim=BIG), UNSUPPORTED),
    (dict(batch=1 << 20, seqlen=1 << 20, dim=1 << 15), UNSUPPORTED), (dict(r_stride=(BIG, BIG)), UNSUPPORTED),
    (dict(dtype=_native.SSM_F32, x=FAKE + 2), UNSUPPORTED),
]


@pytest.mark.parametrize("bad,code", COMMON + [
    (dict(y=None, h_last=None, states=None), INVALID), (dict(y=FAKE + 1), UNSUPPORTED),
    (dict(h0=FAKE + 2), UNSUPPORTED), (dict(h_last=FAKE + 1), UNSUPPORTED), (dict(states=FAKE + 2), UNSUPPORTED)])
def test_gated_scan_fwd_refuses(lib, bad, code):
    assert lib.ssm_gated_scan_fwd(ctypes.byref(_gated(**bad)), None) == code
    assert lib.ssm_gated_scan_fwd(None, None) == INVALID


@pytest.mark.parametrize("bad,code", COMMON + [
    (dict(dy=None), INVALID), (dict(states=None), INVALID), (dict(dx=None), INVALID), (dict(dr=None), INVALID),
    (dict(di=None), INVALID), (dict(dlam=None), INVALID), (dict(dy=FAKE + 1), UNSUPPORTED),
    (dict(dr=FAKE + 1), UNSUPPORTED), (dict(dh_last=FAKE + 2), UNSUPPORTED), (dict(dh0=FAKE + 1), UNSUPPORTED),
    (dict(dlam=FAKE + 2), UNSUPPORTED), (dict(states=FAKE + 2), UNSUPPORTED)])
def test_gated_scan_bwd_refuses(lib, bad, code):
    assert lib.ssm_gated_scan_bwd(ctypes.byref(_gated(True, **bad)), None) == code
    assert lib.ssm_gated_scan_bwd(None, None) == INVALID


def test_overlapping_arrays_are_refused(lib):
    """An output over an input: h_last where h0 lies, y over the tokens or the gap of a strided input, a state half over another."""
    at = lambda k: FAKE + (k << 16)  # of the k-th array
    for bad in (dict(h_last=at(5)), dict(y=at(0)), dict(y=at(2) + 64), dict(states=at(5) + 128), dict(h_last=at(4)),
                dict(states=at(3)), dict(batch=2, x_stride=(1 << 20, 32), y=at(0) + (1 << 20))):
        assert lib.ssm_gated_scan_fwd(ctypes.byref(_gated(**bad)), None) == INVALID, bad
    for bad in (dict(dh0=at(7)), dict(dx=at(6)), dict(di=at(1) + 32), dict(dlam=at(4)), dict(dh0=at(5) + 64)):
        assert lib.ssm_gated_scan_bwd(ctypes.byref(_gated(True, **bad)), None) == INVALID, bad
    step = lambda h, h_out: lib.ssm_gated_step(2, 32, 1, 8.0, at(0), 32, at(1), 32, at(2), 32, at(3), h, h_out, at(6), None)
    assert step(at(4), at(4) + 128) == INVALID and step(at(4) + 252, at(4)) == INVALID


def test_gated_sizes_and_empty_calls(lib):
    assert lib.ssm_gated_states_size(2, 200, 32) == 2 * 4 * 32 * 4
    assert lib.ssm_gated_states_size(2, 0, 32) == 0
    assert lib.ssm_gated_states_size(-1, 2, 32) == 0
    for bwd, size, call in ((False, lib.ssm_gated_scan_workspace_size, lib.ssm_gated_scan_fwd),
                            (True, lib.ssm_gated_scan_bwd_workspace_size, lib.ssm_gated_scan_bwd)):
        need = size(ctypes.byref(_gated(bwd)))
        assert 0 < need < 1 << 20
        assert call(ctypes.byref(_gated(bwd, workspace_bytes=need - 1)), None) == INVALID
        assert size(ctypes.byref(_gated(bwd, batch=-1))) == 0 and size(None) == 0
        assert call(ctypes.byref(_gated(bwd, dim=0)), None) == OK
    assert lib.ssm_gated_scan_fwd(ctypes.byref(_gated(batch=0)), None) == OK
    assert lib.ssm_gated_scan_fwd(ctypes.byref(_gated(seqlen=0, h_last=None)), None) == OK


@pytest.mark.parametrize("B,L,D,most", [(256, 4, 5120, 6 << 20), (2048, 4, 4096, 34 << 20), (70000, 1, 64, 1 << 20), (256, 40, 5120, 43 << 20),
                                        (2048, 200, 4096, 2 << 30), (1, 64, 64, 1 << 12), (4, 2048, 1536, 10 << 20)])
def test_gated_workspace_goes_by_the_length(lib, B, L, D, most):
    """The backward's scratch: a few-token call leaves at most 2048 rows of sums (4 bytes a channel), a call of n tiles of 64
    steps at most 32 bytes a channel and tile (a cluster's last round rounded up) and, beyond one tile, the segments'
    16 bytes; the forward's is a part of that. So neither outgrows the tokens."""
    kw = dict(batch=B, seqlen=L, dim=D, x_stride=(L * D, D), r_stride=(L * D, D), i_stride=(L * D, D))
    back = lib.ssm_gated_scan_bwd_workspace_size(ctypes.byref(_gated(True, **kw)))
    fore = lib.ssm_gated_scan_workspace_size(ctypes.byref(_gated(**kw)))
    assert 256 <= back <= most and 256 <= fore <= back
    tiles = -(-L // 64)
    assert back <= 1024 + B * D * (2 * tiles * 32 + 16 * tiles)
    assert fore <= 1024 + (B * D * 16 * tiles if tiles > 1 else 0)


@pytest.mark.parametrize("B,L,D,few", [(1, 2, 64, True), (1, 3, 64, False), (16, 4, 1024, True), (16, 8, 1024, False), (32, 7, 1024, True),
                                       (32, 16, 1024, False), (64, 12, 1024, True), (64, 16, 1024, False), (128, 16, 1024, True), (300, 9, 12, False), (300, 8, 12, True),
                                       (32, 12, 1001, True), (32, 16, 1001, False),
                                       (2500, 16, 8, True), (256, 17, 5120, False), (256, 16, 5120, True)])
def test_few_token_backward_is_chosen_where_it_is_faster(lib, B, L, D, few):
    """By tokens and columns, as measured beside the rule; the scratch shows which form a call takes (4 bytes a channel of at
    most 2048 rows, or 32 of each sequence's)."""
    kw = dict(batch=B, seqlen=L, dim=D, x_stride=(L * D, D), r_stride=(L * D, D), i_stride=(L * D, D))
    size = lib.ssm_gated_scan_bwd_workspace_size(ctypes.byref(_gated(True, **kw)))
    assert size == 256 + (min(B, 2048) * D * 4 if few else B * D * 32)


def test_gated_step_refuses(lib):
    def call(batch=2, dim=32, dtype=1, c=8.0, x=FAKE, xs=32, r=FAKE, rs=32, i=FAKE, i_s=32, lam=FAKE, h=FAKE,
             h_out=FAKE, y=FAKE + (1 << 16)):
        return lib.ssm_gated_step(batch, dim, dtype, c, x, xs, r, rs, i, i_s, lam, h, h_out, y, None)
    for bad in (dict(batch=-1), dict(dim=-1), dict(dtype=2), dict(c=0.0), dict(c=float("nan")), dict(xs=-1), dict(x=None),
                dict(r=None), dict(i=None), dict(lam=None), dict(h=None), dict(h_out=None), dict(y=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(x=FAKE + 1), dict(y=FAKE + 1), dict(h=FAKE + 2), dict(h_out=FAKE + 2), dict(lam=FAKE + 1),
                dict(batch=BIG, dim=BIG), dict(batch=1 << 30, dim=1 << 12), dict(batch=16, rs=BIG)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(batch=0) == OK and call(dim=0) == OK


def _norm(**kw):
    a = _native.NormArgs()
    a.rows, a.dim, a.dtype, a.eps = 3, 64, _native.SSM_BF16, 1e-5
    for k, n in enumerate(("x", "weight", "bias", "residual", "y", "residual_out", "mean", "rstd")):
        setattr(a, n, FAKE + (k << 16))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad,code", [
    (dict(rows=-1), INVALID), (dict(dim=-1), INVALID), (dict(dtype=9), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(x=None), INVALID),
    (dict(weight=None), INVALID), (dict(y=None), INVALID), (dict(residual=None), INVALID),
    (dict(residual_out=None), INVALID), (dict(dim=16385), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(x=FAKE + 1), UNSUPPORTED), (dict(y=FAKE + 1), UNSUPPORTED), (dict(weight=FAKE + 2), UNSUPPORTED),
    (dict(bias=FAKE + 1), UNSUPPORTED), (dict(residual=FAKE + 2), UNSUPPORTED), (dict(mean=FAKE + 2), UNSUPPORTED),
    (dict(rstd=FAKE + 3), UNSUPPORTED), (dict(rows=0), OK), (dict(dim=0), OK)])
def test_layer_norm_fwd_refuses(lib, bad, code):
    assert lib.ssm_layer_norm_fwd(ctypes.byref(_norm(**bad)), None) == code
    assert lib.ssm_layer_norm_fwd(None, None) == INVALID


def _norm_bwd(**kw):
    a = _native.NormBwdArgs()
    a.rows, a.dim, a.dtype, a.has_residual = 3, 64, _native.SSM_BF16, 1
    return _fill(a, ("s", "dy", "weight", "mean", "rstd", "dresidual_out", "dx", "dresidual", "dweight", "dbias"), **kw)


@pytest.mark.parametrize("bad,code", [
    (dict(rows=-1), INVALID), (dict(dim=-1), INVALID), (dict(dtype=9), INVALID), (dict(s=None), INVALID),
    (dict(dy=None), INVALID), (dict(weight=None), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID),
    (dict(dx=None), INVALID), (dict(dweight=None), INVALID), (dict(workspace=None), INVALID),
    (dict(workspace_bytes=16), INVALID), (dict(workspace=FAKE + 4), UNSUPPORTED), (dict(dim=16385), UNSUPPORTED),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(s=FAKE + 2), UNSUPPORTED), (dict(dy=FAKE + 1), UNSUPPORTED),
    (dict(dx=FAKE + 1), UNSUPPORTED), (dict(weight=FAKE + 1), UNSUPPORTED), (dict(dresidual=FAKE + 2), UNSUPPORTED),
    (dict(dresidual_out=FAKE + 2), UNSUPPORTED), (dict(dweight=FAKE + 2), UNSUPPORTED),
    (dict(dbias=FAKE + 2), UNSUPPORTED), (dict(rstd=FAKE + 1), UNSUPPORTED), (dict(dim=0), OK)])
def test_layer_norm_bwd_refuses(lib, bad, code):
    assert lib.ssm_layer_norm_bwd(ctypes.byref(_norm_bwd(**bad)), None) == code
    assert lib.ssm_layer_norm_bwd(None, None) == INVALID


def test_layer_norm_bwd_workspace(lib):
    need = lib.ssm_layer_norm_bwd_workspace_size(ctypes.byref(_norm_bwd()))
    assert 2 * 64 * 4 <= need < 1 << 20
    assert lib.ssm_layer_norm_bwd(ctypes.byref(_norm_bwd(workspace_bytes=need - 1)), None) == INVALID
    assert lib.ssm_layer_norm_bwd_workspace_size(ctypes.byref(_norm_bwd(rows=0))) == 0
    assert lib.ssm_layer_norm_bwd_workspace_size(None) == 0


def test_binding_refuses():
    """Host tensors, wrong shapes, dtypes and dimensions are refused before any CUDA call."""
    x, lam = torch.zeros(2, 5, 8), torch.zeros(8)
    bad = [
        lambda: ssm.gated_scan_fwd(x, x, x, lam), lambda: ssm.gated_scan(x, x, x, lam),
        lambda: ssm.gated_scan_fwd(x[0], x[0], x[0], lam), lambda: ssm.gated_scan_fwd(x, x[:, :4], x, lam),
        lambda: ssm.gated_scan_bwd(x, x, x, lam, x), lambda: ssm.gated_step(x[:, 0], x[:, 0], x[:, 0], lam, x[:, 0]),
        lambda: ssm.gated_step(x, x, x, lam, x[:, 0]), lambda: ssm.layer_norm_fwd(x, lam),
        lambda: ssm.layer_norm_fwd(torch.zeros(()), lam), lambda: ssm.layer_norm(x, lam),
        lambda: ssm.layer_norm_bwd(x, x, lam, x[..., 0], x[..., 0]),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    h = x.half()
    for f in (lambda: ssm.gated_scan_fwd(h, h, h, lam), lambda: ssm.gated_step(h[0], h[0], h[0], lam, x[0]),
              lambda: ssm.layer_norm_fwd(h, lam), lambda: ssm.layer_norm_bwd(h, h, lam, lam, lam)):
        with pytest.raises(TypeError):
            f()


def test_reference_gradients_against_differences():
    """The float64 backward formulas the GPU tests compare with, against central differences of the float64 forward."""
    from tests import operators_ref as ref
    gen = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    B, L, D = 2, 6, 3
    t = dict(x=n(B, L, D), r=n(B, L, D), i=n(B, L, D), lam=n(D) - 2, h0=n(B, D))
    reset = torch.zeros(B, L, dtype=torch.bool)
    reset[1, 3] = True
    dy, dl = n(B, L, D), n(B, D)

    def loss():
        y, _ = ref.gated_scan(**t, reset=reset)
        return (y * dy).sum() + (y[:, -1] * dl).sum()

    g, _ = ref.gated_scan_bwd(t["x"], t["r"], t["i"], t["lam"], dy, t["h0"], dl, reset=reset)
    _differences(loss, t, {k: g["d" + k] for k in t})
    q = dict(x=n(4, 7), weight=n(7), bias=n(7))
    dy = n(4, 7)
    o, _ = ref.layer_norm(q["x"], q["weight"], q["bias"])
    g, _ = ref.layer_norm_bwd(dy, q["x"], q["weight"], o["mean"], o["rstd"])
    _differences(lambda: (ref.layer_norm(q["x"], q["weight"], q["bias"])[0]["y"] * dy).sum(), q,
                 dict(x=g["dx"], weight=g["dweight"], bias=g["dbias"]))


def _differences(loss, tensors, grads, eps=1e-6):
    for k, v in tensors.items():
        flat, gf = v.view(-1), grads[k].reshape(-1)
        for j in range(flat.numel()):
            keep = flat[j].item()
            flat[j] = keep + eps
            up = loss()
            flat[j] = keep - eps
            down = loss()
            flat[j] = keep
            # truncation eps^2 and cancellation 1e-16 / eps, on values of order 10
            assert abs((up - down).item() / (2 * eps) - gf[j].item()) <= 1e-7 * max(1.0, abs(gf[j].item())), (k, j)


@pytest.mark.parametrize("off", [torch.no_grad, torch.inference_mode])
def test_nothing_is_kept_where_no_graph_is(monkeypatch, off):
    """With gradients switched off the wrappers ask the kernels for neither states nor statistics, though the parameters
    require gradients; with a graph they do."""
    asked = []

    def scan(x, *rest, return_last_state=False, return_states=False, **kw):
        asked.append(return_states)
        res = (x + 0.0,) + ((x[:, 0] + 0.0,) if return_last_state else ()) + ((x[:, :1],) if return_states else ())
        return res if len(res) > 1 else res[0]

    def norm(x, weight, bias=None, residual=None, *, eps=1e-5, return_stats=False):
        asked.append(return_stats)
        res = (x + 0.0,) + ((residual + x,) if residual is not None else ()) + ((x[..., 0], x[..., 0]) if return_stats else ())
        return res if len(res) > 1 else res[0]

    monkeypatch.setattr(ssm, "gated_scan_fwd", scan)
    monkeypatch.setattr(ssm, "layer_norm_fwd", norm)
    x, p = torch.randn(2, 3, 4), torch.nn.Parameter(torch.zeros(4))
    calls = (lambda: ssm.gated_scan(x, x, x, p), lambda: ssm.gated_scan(x, x, x, p, return_last_state=True)[0],
             lambda: ssm.layer_norm(x, p), lambda: ssm.layer_norm(x, p, p, x)[0])
    with off():
        for call in calls:
            assert not call().requires_grad
    assert asked == [False] * 4
    assert all(call().requires_grad for call in calls) and asked[4:] == [True] * 4


def test_test_hook_and_status_arguments(lib):
    """The hand-off hook is a flag of the scan's calls, others are refused; the status is a CUDA device's."""
    hook = _native.SSM_TEST_DROP_HANDOFF
    assert lib.ssm_gated_scan_fwd(ctypes.byref(_gated(flags=hook, batch=0)), None) == OK
    assert lib.ssm_gated_scan_bwd(ctypes.byref(_gated(True, flags=hook, dim=0)), None) == OK
    for bad in (hook | 1, _native.SSM_SEQ_PARALLEL, _native.SSM_TEST_SHORT_SEGMENTS):
        assert lib.ssm_gated_scan_fwd(ctypes.byref(_gated(flags=bad, batch=0)), None) == INVALID
        assert lib.ssm_gated_scan_bwd(ctypes.byref(_gated(True, flags=bad, dim=0)), None) == INVALID
    with pytest.raises(ValueError):
        ssm.gated_status("cpu")
