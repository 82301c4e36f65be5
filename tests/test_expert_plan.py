"""How an experts' product is cut (dispatch_expert_plan.hpp), compiled with the
host compiler and asked on the CPU: the GPU tests that mean to run every tile
shape, shared or not, do, and what the library says of a workspace is that plan."""

import os
import random
import shutil
import subprocess

import pytest

import moe_token_dispatch_amd as M
from tests import test_gpu_expert_product as T

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOKENS = [16, 32, 64, 128, 192, 256]


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path_factory.mktemp("probe") / "expert_plan_probe")
    res = subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I",
                          os.path.join(ROOT, "moe_token_dispatch_amd", "csrc"),
                          os.path.join(ROOT, "tests", "expert_plan_probe.cpp"), "-o", exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr

    def ask(problems):
        """(rows, experts, N, K, workspace) to (tokens of a tile, workgroups that share one, bytes, operands widened)."""
        lines = "\n".join(" ".join(str(int(v)) for v in p) for p in problems)
        out = subprocess.run([exe], input=lines, capture_output=True, text=True, check=True).stdout
        return [tuple(int(v) for v in line.split()) for line in out.splitlines()]

    return ask


def _parameters(test):
    """{names: values} of a test's parametrize marks."""
    return {m.args[0]: m.args[1] for m in test.pytestmark if m.name == "parametrize"}


def test_rows_in_every_tile_does(plan):
    marks = _parameters(T.test_rows_in_every_tile)
    for counts, k, n in marks["counts,k,n"]:
        got = plan([(a, len(counts), n, k, False) for a in marks["announced"]])
        assert [g[0] for g in got] == TOKENS, (counts, k, n)


def test_shared_tiles_of_every_size_are(plan):
    marks = _parameters(T.test_shared_tiles_of_every_size)
    for counts in marks["counts"]:
        got = plan([(a, len(counts), 512, 5008, True) for a in marks["announced"]])
        assert [g[0] for g in got] == [16, 32, 64] and all(g[1] > 1 for g in got), counts


def test_few_rows_are_widened(plan):
    marks = _parameters(T.test_swiglu_of_few_rows_in_fp32)
    for counts, k in marks["counts,k"]:
        for workspace in (False, True):
            assert plan([(sum(counts), len(counts), 512, k, workspace)])[0][::3] == (16, 1), counts
    assert [g[3] for g in plan([(128, 8, 2048, 2048, True), (129, 8, 2048, 2048, True), (4000, 8, 2048, 2048, True)])] \
        == [1, 0, 0]


def test_workspace_is_the_plan(plan):
    r = random.Random(1)
    problems = [(r.randint(0, 1 << r.randint(0, 16)), r.randint(1, 300), 8 * r.randint(1, 1200), 16 * r.randint(1, 600), True)
                for _ in range(2000)]
    shared = 0
    for (rows, e, n, k, _), (tokens, parts, nbytes, _) in zip(problems, plan(problems)):
        p = M.make_expert_problem(e, k, n, 1 << 17, rows)
        assert M.dispatch_expert_workspace_size(p) == nbytes
        assert tokens in TOKENS and 1 <= parts <= 16 and (parts == 1) == (nbytes == 0)
        shared += parts > 1
        # No part without four blocks of K, no more workgroups than CUs, none shared past 64 tokens.
        assert parts == 1 or (parts * 4 <= -(-k // 128) and tokens <= 64)
    assert shared > 100
