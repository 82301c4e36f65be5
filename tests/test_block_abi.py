"""Host checks of the grouped gate, the RMS norm and the combine's gradient, on
the CPU: bad arguments come back as documented codes before any GPU work."""

import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

import moe_token_dispatch_amd as M
from tests.test_abi import _defines

B = ctypes.byref


def test_constants_and_structures_match_the_header():
    d = _defines()
    assert (d["DISPATCH_MAX_GATE_GROUPS"], d["DISPATCH_MAX_NORM_WIDTH"]) == (M.MAX_GATE_GROUPS, M.MAX_NORM_WIDTH)
    assert ctypes.sizeof(M.GateGroups) == 16 and ctypes.sizeof(M.RmsNormProblem) == 24
    assert (M.RmsNormProblem.width.offset, M.RmsNormProblem.weight_bytes.offset, M.RmsNormProblem.eps.offset) == (8, 16, 20)


def test_structures_from_c(tmp_path):
    """The structures as a C99 compiler lays them out, and a host check called from C."""
    gcc = shutil.which("gcc")
    if gcc is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("gcc or the ROCm headers are not installed")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    structs = {"dispatch_gate_groups_t": M.GateGroups, "dispatch_rms_norm_problem_t": M.RmsNormProblem}
    lines = [f'printf("%zu %zu\\n", sizeof({c}), offsetof({c}, {f}));' for c, t in structs.items() for f, _ in t._fields_]
    want = [f"{ctypes.sizeof(t)} {getattr(t, f).offset}" for t in structs.values() for f, _ in t._fields_]
    source = tmp_path / "probe.c"
    source.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"moe_dispatch.h\"\nint main(void) {\n" + "\n".join(lines)
                      + "\ndispatch_rms_norm_problem_t p = {0, 264, 2, 1e-6f};\nsize_t n = 0;\n"
                        'printf("%d\\n", dispatch_rms_norm_workspace_size(&p, &n));\nreturn 0;\n}\n')
    M.load_library()
    pkg, exe = os.path.join(root, "moe_token_dispatch_amd"), str(tmp_path / "probe")
    built = subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
                            "-I", os.path.join(root, "include"), str(source), "-o", exe, "-L", pkg, "-lmoe_dispatch",
                            f"-Wl,-rpath,{pkg}"], capture_output=True, text=True)
    assert built.returncode == 0, built.stderr
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120).stdout.split("\n")
    assert out[:len(want)] == want and int(out[len(want)]) == M.ERR_ALIGN


# ------------------------------------------------------------- grouped gate


def _gate(**kw):
    p = M.GateProblem(100, 64, 8, M.GATE_SIGMOID, 2, 8, M.GATE_NORMALIZE, 1.0, 0.1)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _grouped(p, groups, z=4096, bias=4096, out=True, ws=4096, n=1 << 30, **ptrs):
    o = M.GateOutPtrs(*[4096] * 6)
    for k, v in ptrs.items():
        setattr(o, k, v)
    return M.load_library().dispatch_gate_grouped(B(p) if p is not None else None, B(groups) if groups is not None else None,
                                                  z, bias, 4097, B(o) if out else None, ws, n, None)


@pytest.mark.parametrize("groups", [
    M.GateGroups(0, 1, 1, 0), M.GateGroups(-8, 1, 1, 0), M.GateGroups(65, 4, 1, 0), M.GateGroups(7, 4, 1, 0),
    M.GateGroups(8, 0, 1, 0), M.GateGroups(8, 9, 1, 0), M.GateGroups(8, -1, 1, 0), M.GateGroups(8, 4, 0, 0),
    M.GateGroups(8, 4, 3, 0), M.GateGroups(8, 4, 1, 1), M.GateGroups(16, 1, 1, 0)], ids=lambda g: f"{g.num_groups}-{g.topk_groups}-{g.score_experts}-{g.reserved}")
def test_bad_groups(groups):
    # (16 groups of 4 experts, one taken: fewer than the 8 entries.)
    assert _grouped(_gate(), groups) == M.ERR_ARG


def test_grouped_gate_arguments():
    good = M.make_gate_groups(8, 4, 2)
    assert _grouped(None, good) == M.ERR_NULL and _grouped(_gate(), None) == M.ERR_NULL
    assert _grouped(_gate(scoring=M.GATE_SOFTMAX), good, bias=None) == M.ERR_ARG  # pairs need sigmoid scores
    assert _grouped(_gate(scoring=M.GATE_SOFTMAX), M.make_gate_groups(8, 4)) == M.ERR_ARG  # and so does a bias
    assert _grouped(_gate(), good, z=None) == M.ERR_NULL and _grouped(_gate(), good, out=False) == M.ERR_NULL
    assert _grouped(_gate(), good, loss=None) == M.ERR_NULL
    assert _grouped(_gate(), good, z=4097) == M.ERR_ALIGN and _grouped(_gate(), good, bias=4098) == M.ERR_ALIGN
    assert _grouped(_gate(), good, ws=None) == M.ERR_WORKSPACE
    assert _grouped(_gate(), good, n=M.dispatch_gate_workspace_size(_gate()) - 1) == M.ERR_WORKSPACE
    for bad in (dict(num_experts=0), dict(num_experts=4096 + 8), dict(num_topk=0), dict(num_tokens=-1), dict(flags=2)):
        assert _grouped(_gate(**bad), good) == M.ERR_ARG, bad


# ----------------------------------------------------------------- RMS norm


def _norm(rows=100, width=256, weight_bytes=2, eps=1e-6):
    return M.RmsNormProblem(rows, width, weight_bytes, eps)


def _forward(p=None, prob=True, x=4096, r=4096, w=4096, n=4096, h=4096, y=4096, q=4096, sf=4096):
    p = _norm() if p is None else p
    return M.load_library().dispatch_rms_norm(B(p) if prob else None, x, r, w, n, h, y, q, sf, None)


def _backward(p=None, prob=True, h=4096, w=4096, dy=4096, dh=4096, n=4096, dx=4096, dw=4096, ws=4096, nbytes=1 << 40):
    p = _norm() if p is None else p
    return M.load_library().dispatch_rms_norm_backward(B(p) if prob else None, h, w, dy, dh, n, dx, dw, ws, nbytes, None)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(rows=1 << 31), dict(width=0), dict(width=65536 + 16),
                                 dict(weight_bytes=1), dict(weight_bytes=8), dict(eps=0.0), dict(eps=-1e-6),
                                 dict(eps=math.nan), dict(eps=math.inf), dict(eps=1e-39)], ids=str)
def test_bad_norm_problems(bad):
    p, n = _norm(**bad), ctypes.c_size_t(0)
    assert _forward(p) == M.ERR_ARG and _backward(p) == M.ERR_ARG
    assert M.load_library().dispatch_rms_norm_workspace_size(B(p), B(n)) == M.ERR_ARG


def test_norm_arguments():
    lib, n = M.load_library(), ctypes.c_size_t(0)
    assert _forward(_norm(width=264)) == M.ERR_ALIGN and _backward(_norm(width=264)) == M.ERR_ALIGN
    assert _forward(prob=False) == M.ERR_NULL and _backward(prob=False) == M.ERR_NULL
    for name in ("x", "r", "w", "h", "sf", "q"):
        assert _forward(**{name: None}) == M.ERR_NULL, name  # r, h and q, sf come in pairs
    assert _forward(y=None, q=None, sf=None) == M.ERR_NULL
    for name in ("x", "r", "w", "h", "y", "q"):
        assert _forward(**{name: 4104}) == M.ERR_ALIGN, name
    assert _forward(n=4098) == M.ERR_ALIGN and _forward(sf=4098) == M.ERR_ALIGN
    for name in ("h", "w", "dy", "dx"):
        assert _backward(**{name: None}) == M.ERR_NULL, name
    for name in ("h", "w", "dy", "dh", "dx", "dw"):
        assert _backward(**{name: 4104}) == M.ERR_ALIGN, name
    assert _backward(n=4098) == M.ERR_ALIGN
    need = M.dispatch_rms_norm_workspace_size(_norm())
    assert need > 0 and need % 256 == 0
    assert _backward(ws=None) == M.ERR_WORKSPACE and _backward(ws=4096 + 128) == M.ERR_WORKSPACE
    assert _backward(nbytes=need - 1) == M.ERR_WORKSPACE
    assert lib.dispatch_rms_norm_workspace_size(B(_norm()), None) == M.ERR_NULL
    assert lib.dispatch_rms_norm_workspace_size(None, B(n)) == M.ERR_NULL


def test_norm_of_no_rows_needs_no_rows():
    assert _forward(_norm(rows=0), x=None, r=None, h=None, y=None, q=None, sf=None, n=None) == M.OK
    assert _backward(_norm(rows=0), h=None, dy=None, dh=None, dx=None, dw=None, ws=None, nbytes=0, n=None) == M.OK


# ------------------------------------------------------- combine's gradient


def _combine(rows=100, k=8, tokens=50, width=256, reserved=0, prob=True, slot=4096, w=4096, y=4096, d=4096, dw=4096,
             dy=4096, dq=None, dsf=None):
    p = M.CombineProblem(tokens, k, reserved, width, rows)
    return M.load_library().dispatch_combine_backward(B(p) if prob else None, slot, w, y, d, dw, dy, dq, dsf, None)


def test_combine_gradient_arguments():
    assert _combine(prob=False) == M.ERR_NULL
    for bad in (dict(tokens=-1), dict(tokens=1 << 31), dict(k=0), dict(k=33), dict(rows=-1), dict(width=0),
                dict(width=1 << 30), dict(reserved=1)):
        assert _combine(**bad) == M.ERR_ARG, bad
    assert _combine(width=260) == M.ERR_ALIGN
    assert _combine(width=264, dy=None, dq=4096, dsf=4096) == M.ERR_ALIGN  # fp8 rows are whole 16-byte vectors
    assert _combine(dq=4096, dsf=4096) == M.ERR_ARG                        # one of the two forms
    for name in ("slot", "w", "d", "y"):
        assert _combine(**{name: None}) == M.ERR_NULL, name
    assert _combine(dw=None, dy=None) == M.ERR_NULL
    assert _combine(dy=None, dq=4096) == M.ERR_NULL and _combine(dy=None, dsf=4096) == M.ERR_NULL
    for name in ("y", "d", "dy"):
        assert _combine(**{name: 4104}) == M.ERR_ALIGN, name
    assert _combine(dy=None, dq=4104, dsf=4096) == M.ERR_ALIGN
    for name in ("slot", "w", "dw"):
        assert _combine(**{name: 4098}) == M.ERR_ALIGN, name
    assert _combine(dy=None, dq=4096, dsf=4098) == M.ERR_ALIGN
    assert _combine(tokens=0, slot=None, w=None, y=None, d=None, dw=None, dy=None) == M.OK


def test_combine_gradient_without_expert_rows():
    """Buffers of no rows may be NULL, as an empty tensor's pointer is; the weights' gradient is asked for otherwise."""
    assert _combine(rows=0, y=None, dw=None, dy=None) == M.OK
    for name in ("slot", "w", "d"):
        assert _combine(rows=0, y=None, dw=None, dy=None, **{name: None}) == M.ERR_NULL, name
    assert _combine(rows=0, y=None, dw=None, dy=None, dsf=4096) == M.ERR_NULL
    assert _combine(rows=1, y=None, dw=None, dy=None) == M.ERR_NULL


def test_binding_refuses_host_tensors():
    x, w = torch.zeros((4, 32), dtype=torch.bfloat16), torch.ones(32)
    with pytest.raises(ValueError, match="x must be a device tensor"):
        M.dispatch_rms_norm(x, w, 1e-6, y=torch.zeros_like(x))
    with pytest.raises(ValueError, match="h must be a device tensor"):
        M.dispatch_rms_norm_backward(x, w, x, 1e-6, torch.zeros_like(x))
    with pytest.raises(ValueError, match="expert_slot must be a device tensor"):
        M.dispatch_combine_backward(torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2)), x, x)
    p = M.make_gate_problem(4, 32, 2, M.GATE_SIGMOID, torch.float32)
    with pytest.raises(ValueError, match="logits must be a device tensor"):
        M.dispatch_gate_grouped(p, M.make_gate_groups(4, 2), torch.zeros((4, 32)), M.alloc_gate(p, "cpu"))


@pytest.mark.parametrize("gpus,current,of,expected", [(1, 0, 0, 0), (2, 0, 0, 0), (2, 0, 1, 1), (8, 5, 2, 2)])
def test_a_prepared_call_runs_on_its_tensors_device(monkeypatch, gpus, current, of, expected):
    """With several GPUs the tensors' device is the current one during the call, and the caller's again after it."""
    now, calls, codes = [current], [], [M.OK, M.ERR_HIP]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *_):
            now[0] = self.before

    class Library:
        dispatch_strerror = M.load_library().dispatch_strerror

        @staticmethod
        def dispatch_something(*args):
            calls.append((args, now[0]))
            return codes[len(calls) - 1]

    monkeypatch.setattr(M._binding, "load_library", Library)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: gpus)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    call = M._binding._Prepared("dispatch_something", (1, 2), torch.device("cuda", of), None)
    call()
    with pytest.raises(M.DispatchError, match="dispatch_something"):
        call()
    assert calls == [((1, 2), expected)] * 2 and now == [current]
