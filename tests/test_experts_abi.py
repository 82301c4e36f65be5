"""Host checks of the gate, quantisation and product calls, on the CPU: bad
arguments come back as documented codes before any GPU work."""

import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

import moe_token_dispatch_amd as M
from tests import layer_reference as R
from tests.test_abi import _defines

B = ctypes.byref


def test_constants_match_the_header():
    d = _defines()
    assert (d["DISPATCH_GATE_SOFTMAX"], d["DISPATCH_GATE_SIGMOID"], d["DISPATCH_GATE_NORMALIZE"],
            d["DISPATCH_SF_BLOCK"]) == (M.GATE_SOFTMAX, M.GATE_SIGMOID, M.GATE_NORMALIZE, M.SF_BLOCK)


def _gate(**kw):
    p = M.GateProblem(100, 64, 8, M.GATE_SIGMOID, 2, 8, M.GATE_NORMALIZE, 1.0, 0.1)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


BAD_GATES = [
    dict(num_tokens=-1), dict(num_tokens=1 << 31), dict(num_tokens=1 << 28), dict(num_experts=0),
    dict(num_experts=4097), dict(num_topk=0), dict(num_topk=33), dict(num_topk=9, num_experts=8), dict(scoring=2),
    dict(scoring=-1), dict(logits_bytes=8), dict(topk_idx_bytes=2), dict(flags=2), dict(route_scale=math.inf),
    dict(loss_coef=math.nan),
]


@pytest.mark.parametrize("bad", BAD_GATES, ids=str)
def test_bad_gate_problems(bad):
    lib, p, n = M.load_library(), _gate(**bad), ctypes.c_size_t(0)
    out = M.GateOutPtrs(*[4096] * 6)
    assert lib.dispatch_gate_workspace_size(B(p), B(n)) == M.ERR_ARG
    assert lib.dispatch_gate(B(p), 4096, None, None, B(out), 4096, 1 << 30, None) == M.ERR_ARG
    assert lib.dispatch_gate_backward(B(p), 4096, None, 4096, 4096, 4096, 4096, 4096, 4096, None) == M.ERR_ARG


def test_gate_arguments():
    lib, p = M.load_library(), _gate()
    ws = M.dispatch_gate_workspace_size(p)
    assert ws > 0 and ws % 256 == 0

    def call(p=p, z=4096, bias=4096, mask=4097, out=True, ws_ptr=4096, n=ws, **ptrs):
        o = M.GateOutPtrs(*[4096] * 6)
        for k, v in ptrs.items():
            setattr(o, k, v)
        return lib.dispatch_gate(B(p) if p is not None else None, z, bias, mask, B(o) if out else None, ws_ptr, n, None)

    assert call(p=None) == M.ERR_NULL
    assert call(z=None) == M.ERR_NULL
    assert call(out=False) == M.ERR_NULL
    for f in ("topk_idx", "topk_weights", "expert_count", "prob_sum", "live_tokens", "loss"):
        assert call(**{f: None}) == M.ERR_NULL, f
        assert call(**{f: 4098}) == M.ERR_ALIGN, f
    assert call(topk_idx=4100) == M.ERR_ALIGN
    assert call(z=4097) == M.ERR_ALIGN and call(bias=4098) == M.ERR_ALIGN
    assert call(p=_gate(scoring=M.GATE_SOFTMAX)) == M.ERR_ARG  # a bias needs sigmoid scores
    assert call(ws_ptr=None) == M.ERR_WORKSPACE
    assert call(ws_ptr=4096 + 128) == M.ERR_WORKSPACE
    assert call(n=ws - 1) == M.ERR_WORKSPACE
    assert lib.dispatch_gate_workspace_size(B(p), None) == M.ERR_NULL
    assert lib.dispatch_gate_workspace_size(None, None) == M.ERR_NULL


def test_gate_backward_arguments():
    lib, p = M.load_library(), _gate()

    def call(*, i=None, v=None, prob=p):
        args = [4096, 4096, 4096, 4096, 4096, 4096, 4096, 4096]  # z mask idx dw count live dloss dz
        if i is not None:
            args[i] = v
        return lib.dispatch_gate_backward(B(prob) if prob is not None else None, *args, None)

    assert call(prob=None) == M.ERR_NULL
    for i in (0, 2, 4, 5, 7):
        assert call(i=i, v=None) == M.ERR_NULL, i
    for i, v in ((0, 4097), (2, 4100), (3, 4098), (4, 4098), (5, 4098), (6, 4098), (7, 4097)):
        assert call(i=i, v=v) == M.ERR_ALIGN, i


@pytest.mark.parametrize("name,grad,sf_per_block", [
    ("dispatch_quantize", False, 1), ("dispatch_swiglu_quantize", False, 1),
    ("dispatch_swiglu_backward_quantize", True, 2)])
def test_quantize_arguments(name, grad, sf_per_block):
    lib = M.load_library()

    def call(rows=100, width=256, x=4096, d=4096, n=4096, q=4096, sf=4096, prob=True):
        p = M.QuantizeProblem(rows, width)
        ins = (x, d) if grad else (x,)
        return getattr(lib, name)(B(p) if prob else None, *ins, n, q, sf, None)

    assert call(prob=False) == M.ERR_NULL
    assert call(rows=-1) == M.ERR_ARG and call(rows=1 << 31) == M.ERR_ARG
    assert call(width=0) == M.ERR_ARG and call(width=(1 << 30) + 128) == M.ERR_ARG
    assert call(width=264) == M.ERR_ALIGN
    assert call(rows=(1 << 31) // (2 * sf_per_block) + 1, width=256) == M.ERR_ARG  # blocks pass 2^31
    for k in ("x", "q", "sf") + (("d",) if grad else ()):
        assert call(**{k: None}) == M.ERR_NULL, k
        assert call(**{k: 4098}) == M.ERR_ALIGN, k
    assert call(n=4098) == M.ERR_ALIGN
    if name != "dispatch_quantize":
        assert call(width=144) == M.ERR_ALIGN


def _experts(**kw):
    p = M.ExpertProblem(4, 0, 256, 512, 1000, 800)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


BAD_EXPERTS = [
    (dict(num_experts=0), M.ERR_ARG), (dict(num_experts=4097), M.ERR_ARG), (dict(reserved=1), M.ERR_ARG),
    (dict(in_features=0), M.ERR_ARG), (dict(in_features=(1 << 20) + 16), M.ERR_ARG),
    (dict(out_features=0), M.ERR_ARG), (dict(out_features=(1 << 20) + 256), M.ERR_ARG),
    (dict(expert_rows=-1), M.ERR_ARG), (dict(expert_rows=1 << 31), M.ERR_ARG), (dict(max_routed_rows=-1), M.ERR_ARG),
    (dict(expert_rows=(1 << 31) - 1, out_features=1 << 20), M.ERR_ARG),
    (dict(in_features=24), M.ERR_ALIGN), (dict(out_features=516), M.ERR_ALIGN),
]


@pytest.mark.parametrize("bad,code", BAD_EXPERTS, ids=str)
def test_bad_expert_problems(bad, code):
    lib, p = M.load_library(), _experts(**bad)
    assert lib.dispatch_expert_product(B(p), *[4096] * 7, None, 0, None) == code
    assert lib.dispatch_expert_product_swiglu(B(p), *[4096] * 8, None, 0, None) == code


def test_expert_arguments():
    lib, p = M.load_library(), _experts()
    assert lib.dispatch_expert_product(None, *[4096] * 7, None, 0, None) == M.ERR_NULL
    for swiglu, n in ((False, 7), (True, 8)):
        call = lib.dispatch_expert_product_swiglu if swiglu else lib.dispatch_expert_product
        for i in range(n):
            args = [4096] * n
            args[i] = None
            assert call(B(p), *args, None, 0, None) == M.ERR_NULL, i
            args[i] = 4104 if i in (2, 4, 6) else 4098
            assert call(B(p), *args, None, 0, None) == M.ERR_ALIGN, i
    # Halves of the SwiGLU product are whole blocks.
    assert lib.dispatch_expert_product_swiglu(B(_experts(out_features=384)), *[4096] * 8, None, 0, None) == M.ERR_ALIGN


def test_expert_workspace():
    lib, n = M.load_library(), ctypes.c_size_t(0)
    assert lib.dispatch_expert_workspace_size(None, B(n)) == M.ERR_NULL
    assert lib.dispatch_expert_workspace_size(B(_experts()), None) == M.ERR_NULL
    few, many = _experts(in_features=8192, expert_rows=16, max_routed_rows=8), _experts(expert_rows=4000, max_routed_rows=4000)
    need = M.dispatch_expert_workspace_size(few)
    assert need > 0 and M.dispatch_expert_workspace_size(many) == 0
    for swiglu, ptrs in ((False, 7), (True, 8)):
        call = lib.dispatch_expert_product_swiglu if swiglu else lib.dispatch_expert_product
        assert call(B(few), *[4096] * ptrs, 4096 + 128, need, None) == M.ERR_WORKSPACE
        assert call(B(few), *[4096] * ptrs, 4096, need - 1, None) == M.ERR_WORKSPACE


STRUCTS = {
    "dispatch_gate_problem_t": M.GateProblem, "dispatch_gate_out_t": M.GateOutPtrs,
    "dispatch_quantize_problem_t": M.QuantizeProblem, "dispatch_expert_problem_t": M.ExpertProblem,
}


def test_struct_layouts_from_c(tmp_path):
    """The structs of the header, compiled as C99, against the binding's."""
    gcc = shutil.which("gcc")
    if gcc is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("gcc or the ROCm headers are not installed")
    lines, want = [], []
    for c_name, py in STRUCTS.items():
        lines.append(f'printf("%zu\\n", sizeof({c_name}));')
        want.append(ctypes.sizeof(py))
        for field, _ in py._fields_:
            lines.append(f'printf("%zu\\n", offsetof({c_name}, {field}));')
            want.append(getattr(py, field).offset)
    src, exe = tmp_path / "probe.c", str(tmp_path / "probe")
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"moe_dispatch.h\"\nint main(void) {\n"
                   + "\n".join(lines) + "\nreturn 0;\n}\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    build = subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I",
                            "/opt/rocm/include", "-I", os.path.join(root, "include"), str(src), "-o", exe],
                           capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    got = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert [int(v) for v in got.stdout.split()] == want


@pytest.mark.parametrize("sigmoid", [False, True])
def test_references_of_the_gate_agree(sigmoid):
    g = torch.Generator().manual_seed(1)
    z = torch.randint(-3, 4, (40, 21), generator=g).float()
    z[0] = -math.inf
    z[1, 2:] = -math.inf
    z[2, 3] = math.nan
    mask = torch.rand((40,), generator=g) > 0.2
    bias = torch.randn((21,), generator=g) if sigmoid else None
    z2 = z.clone()
    z2[2, 3] = 0.0  # (NaN shows in sums: the choice alone is compared with it)
    for x, names in ((z, ("idx", "count")), (z2, ("idx", "weights", "prob_sum", "count", "live", "loss", "order"))):
        a = R.gate(x, 4, sigmoid, True, 1.5, 0.1, bias, mask)
        b = R.gate_table(x, 4, sigmoid, True, 1.5, 0.1, bias, mask)
        for name in names:
            assert torch.equal(torch.as_tensor(a[name]), torch.as_tensor(b[name])), name


@pytest.mark.parametrize("width", [8, 256, 264, 1 << 20])
def test_largest_expert_problems(width):
    """The output's tiles of 16 rows x 256 channels are counted in 32 bits; what they hold is taken."""
    lib, n = M.load_library(), ctypes.c_size_t(0)
    most = min((1 << 31) - 1, ((((1 << 31) - 1) // -(-width // 256)) - 4) * 16 + 15)
    assert lib.dispatch_expert_workspace_size(B(_experts(out_features=width, expert_rows=most)), B(n)) == M.OK
    if most < (1 << 31) - 1:
        p = _experts(out_features=width, expert_rows=most + 1)
        assert lib.dispatch_expert_workspace_size(B(p), B(n)) == M.ERR_ARG
        assert lib.dispatch_expert_product(B(p), *[4096] * 7, None, 0, None) == M.ERR_ARG
