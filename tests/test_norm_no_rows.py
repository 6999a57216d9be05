"""The norms' gradient of no rows (a rank that received no tokens): zeros for what is summed
over rows, whatever the architecture does with a division by zero."""
import ctypes
import os
import signal
import subprocess
import sys

import pytest
import torch

from fp8_moe_routed_gb300 import binding as fb

P = ctypes.c_void_p

# The host side of the launch behind the entry point, which turns to the device first: on a
# machine without one (none is visible to this process) it has to come back with an error.
LAUNCH = """
import ctypes, sys
P, I64, I32, F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float

class Args(ctypes.Structure):
    _fields_ = ([(n, P) for n in ("dr", "dh", "r", "y", "w_post", "w_pre", "rstd_post", "rstd_pre",
                                  "gate")] +
                [("gate_kind", I32), ("sigmoid", I32), ("residual_scale", F32),
                 ("branch_scale", F32), ("T", I64), ("H", I32), ("f32", I32)] +
                [(n, P) for n in ("dx", "dy", "dw_post", "dw_pre", "dgate", "part")])

f = ctypes.CDLL(sys.argv[1])["_Z22fp8moe_launch_norm_bwdRK11NormBwdArgsiP11CUstream_st"]
f.argtypes, f.restype = [ctypes.POINTER(Args), I32, P], I32
for f32 in (0, 1):
    a = Args(w_post=16, w_pre=16, dw_post=16, dw_pre=16, residual_scale=1.0, branch_scale=1.0,
             H=64, f32=f32)
    print(f(ctypes.byref(a), 152, None))
"""


def test_the_host_side_survives_no_rows():
    fb.load()
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    p = subprocess.run([sys.executable, "-c", LAUNCH, fb.library_path()], env=env, text=True,
                       capture_output=True, timeout=120)
    assert p.returncode == 0, signal.Signals(-p.returncode).name if p.returncode < 0 else p.stderr
    assert all(int(v) > 0 for v in p.stdout.split()) and len(p.stdout.split()) == 2


@pytest.mark.gpu
@pytest.mark.parametrize("given", ["nothing", "zero", "inf", "nan"])
def test_sums_over_no_rows_are_zero(given):
    """dw_pre, dw_post and a gate's gradient per channel; the gate may be missing, and what it
    and the weights hold has no part in an empty sum."""
    H = 200
    out = {k: torch.full((H,), 7.0, device="cuda") for k in ("dw_post", "dw_pre", "dgate")}
    value = {"nothing": 1.0, "zero": 0.0}.get(given, float(given) if given in ("inf", "nan") else 0)
    gate, w = (torch.full((H,), value, device="cuda") for _ in range(2))
    for sigmoid in (0, 1):
        for t in out.values():
            t.fill_(7.0)
        rc = fb.load().fp8moe_norm_bwd(
            None, None, None, None, 0, H, 0, P(w.data_ptr()), P(w.data_ptr()), None, None,
            None if given == "nothing" else P(gate.data_ptr()), fb.GATES["channel"], sigmoid, 1.0, 1.0,
            None, None, P(out["dw_post"].data_ptr()), P(out["dw_pre"].data_ptr()),
            P(out["dgate"].data_ptr()), None, 0, fb._stream(torch.device("cuda", 0)))
        assert rc == fb.OK
        torch.cuda.synchronize()
        assert all((t == 0).all() for t in out.values())
    assert fb.read_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [None, "token", "channel", "full"])
@pytest.mark.parametrize("parts", ["both", "post", "pre"])
def test_no_rows_through_the_binding(kind, parts):
    post, pre = parts != "pre", parts != "post"
    if kind is not None and not post:
        pytest.skip("a gate belongs to a block output")
    H = 64
    e = torch.empty(0, H, dtype=torch.bfloat16, device="cuda")
    z, w = torch.empty(0, device="cuda"), torch.ones(H, device="cuda")
    gate = {None: None, "token": z, "channel": w, "full": e}[kind]
    dx, dy, dw_post, dw_pre, dgate = fb.norm_bwd(
        e, e if pre else None, e, e if post else None, w if post else None, w if pre else None,
        z if post else None, z if pre else None, gate=gate, gate_kind=kind)
    assert dx.shape == (0, H) and (dy.shape == (0, H) if post else dy is None)
    assert (dw_post == 0).all() if post else dw_post is None
    assert (dw_pre == 0).all() if pre else dw_pre is None
    if kind is not None:
        assert dgate.shape == gate.shape and (dgate == 0).all()
