"""CPU checks of the mixture-of-experts entry points: struct layouts, size
helpers, and the refusals that the host makes before any CUDA call."""
from __future__ import annotations

import os
import subprocess

import pytest
import torch

from tests import moe_ref as R
from tests.conftest import ROOT

HEADER = os.path.join(ROOT, "include", "mxfp4.h")


@pytest.fixture(scope="module")
def abi():
    from mxfp4_block_fake_b200 import build
    build.build()
    from mxfp4_block_fake_b200 import _abi
    _abi.lib()
    return _abi


@pytest.mark.parametrize("cname,pyname", [("mxfp4_moe_route_args", "RouteArgs"), ("mxfp4_moe_move_args", "MoveArgs"),
                                          ("mxfp4_linear_args", "LinearArgs")])
def test_struct_layout_matches_c(abi, tmp_path, cname, pyname):
    cls = getattr(abi, pyname)
    fields = [f for f, _ in cls._fields_]
    body = "\n".join(f'  printf("{f} %zu\\n", offsetof({cname}, {f}));' for f in fields)
    src = tmp_path / "layout.c"
    src.write_text(f'#include <stddef.h>\n#include <stdio.h>\n#include "mxfp4.h"\nint main(void) {{\n'
                   f'  printf("sizeof %zu\\n", sizeof({cname}));\n{body}\n  return 0;\n}}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.dirname(HEADER), "-o", str(exe), str(src)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    import ctypes
    assert int(got.pop("sizeof")) == ctypes.sizeof(cls)
    assert {f: int(v) for f, v in got.items()} == {f: getattr(cls, f).offset for f in fields}


P = 1 << 16  # a pointer that is never followed: every case below is refused on the host


def route(abi, **kw):
    a = abi.RouteArgs()
    a.logits, a.tokens, a.experts, a.ld, a.dtype, a.k = P, 4, 16, 16, abi.F32, 2
    a.scale, a.num_groups, a.topk_groups = 1.0, 1, 1
    a.weights = a.chosen = a.rows = a.slots = a.counts = P
    for f, v in kw.items():
        setattr(a, f, v)
    return a


@pytest.mark.parametrize("kw,expected", [
    (dict(dtype=2), 1), (dict(tokens=-1), 1), (dict(experts=0), 1), (dict(k=0), 1), (dict(k=17), 1), (dict(ld=15), 1),
    (dict(score=2), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(experts=1025, ld=1025), 2), (dict(experts=64, ld=64, k=33), 2), (dict(tokens=2 ** 30), 2),
    (dict(num_groups=0), 1), (dict(num_groups=3), 1), (dict(num_groups=4, topk_groups=5), 1), (dict(num_groups=4, topk_groups=0), 1),
    (dict(num_groups=8, topk_groups=1, k=3), 1), (dict(experts=64, ld=64, num_groups=64, topk_groups=64), 2),
    (dict(group_score=2), 1), (dict(logits=None), 1), (dict(weights=None), 1), (dict(chosen=None), 1), (dict(rows=None), 1),
    (dict(slots=None), 1), (dict(counts=None), 1), (dict(logits=P + 2), 1), (dict(counts=P + 4), 1), (dict(bias=P + 1), 1),
    (dict(tokens=65), 1), (dict(tokens=65, workspace=P, workspace_bytes=127), 1),
])
def test_route_refuses_on_the_host(abi, kw, expected):
    assert abi.mxfp4_moe_route(route(abi, **kw), None) == expected


@pytest.mark.parametrize("kw,expected", [
    (dict(ld_grad=15), 1), (dict(grad_weights=None), 1), (dict(grad_logits=None), 1), (dict(chosen=None), 1),
    (dict(logits=None), 1), (dict(k=0), 1), (dict(grad_logits=P + 2), 1), (dict(experts=2000, ld=2000, ld_grad=2000), 2),
])
def test_route_bwd_refuses_on_the_host(abi, kw, expected):
    a = route(abi, **{**dict(grad_weights=P, grad_logits=P, ld_grad=16), **kw})
    assert abi.mxfp4_moe_route_bwd(a, None) == expected


def move(abi, **kw):
    a = abi.MoveArgs()
    a.rows, a.tokens, a.cols, a.row_count, a.k, a.dtype = P, 4, 64, 8, 2, abi.BF16
    a.ld_tokens = a.ld_rows = a.ld_out = a.ld_grad_rows = 64
    a.scale_factor = 6.0
    for f, v in kw.items():
        setattr(a, f, v)
    return a


@pytest.mark.parametrize("kw,expected", [
    (dict(), 1), (dict(values=P, x=None), 1), (dict(values=P, ld_tokens=63), 1), (dict(values=P, ld_rows=63), 1),
    (dict(values=P, rows=None), 1), (dict(values=P, rows=P + 2), 1), (dict(values=P, k=0), 1), (dict(values=P, k=33), 2),
    (dict(values=P, dtype=5), 1), (dict(values=P, tokens=-1), 1), (dict(values=P, x=P + 1), 1),
    (dict(codes=P, scales=None), 1), (dict(codes=P, scales=P, elem_format=2), 1), (dict(codes=P, scales=P, scale_mode=2), 1),
    (dict(codes=P, scales=P, scale_factor=0.0), 1), (dict(codes=P, scales=P, elem_format=1), 2),
    (dict(values=P, row_count=2 ** 31), 2),
])
def test_dispatch_refuses_on_the_host(abi, kw, expected):
    assert abi.mxfp4_moe_dispatch(move(abi, **{**dict(x=P), **kw}), None) == expected


@pytest.mark.parametrize("kw,expected", [
    (dict(out=None), 1), (dict(y=None), 1), (dict(ld_out=10), 1), (dict(ld_rows=10), 1), (dict(residual=P, ld_tokens=3), 1),
    (dict(weights=P + 2), 1), (dict(out=P + 1), 1), (dict(k=40), 2),
])
def test_combine_refuses_on_the_host(abi, kw, expected):
    assert abi.mxfp4_moe_combine(move(abi, **{**dict(y=P, out=P), **kw}), None) == expected


@pytest.mark.parametrize("kw,expected", [
    (dict(grad_rows=None, grad_weights=None), 1), (dict(grad_out=None), 1), (dict(y=None), 1), (dict(ld_grad_rows=10), 1),
    (dict(ld_rows=10), 1), (dict(grad_weights=P + 1), 1),
])
def test_combine_bwd_refuses_on_the_host(abi, kw, expected):
    a = move(abi, **{**dict(y=P, grad_out=P, grad_rows=P, grad_weights=P), **kw})
    assert abi.mxfp4_moe_combine_bwd(a, None) == expected


def linear(abi, **kw):
    a = abi.LinearArgs()
    a.m, a.n, a.k = 8, 32, 128
    a.a = a.b = a.a_scales = a.b_scales = a.y = P
    a.lda = a.ldb = 64
    a.group_list, a.num_groups, a.group_list_type, a.d_dtype = P, 2, 1, abi.BF16
    a.ld_y, a.ld_res, a.ld_preact, a.ld_grad = 32, 32, 32, 32
    for f, v in kw.items():
        setattr(a, f, v)
    return a


@pytest.mark.parametrize("kw,expected", [
    (dict(elem_format=2), 1), (dict(activation=6), 1), (dict(activation=-1), 1), (dict(d_dtype=2), 1), (dict(m=-1), 1), (dict(n=-2), 1),
    (dict(k=0), 1), (dict(k=96), 1), (dict(k=32), 1), (dict(elem_format=1, k=48), 1), (dict(activation=5, n=31), 1),
    (dict(num_groups=0), 1), (dict(group_list_type=2), 1), (dict(group_list=P + 4), 1), (dict(num_groups=4097), 2),
    (dict(lda=48), 1), (dict(lda=72), 1), (dict(a=P + 8), 1), (dict(b=P + 8), 1), (dict(a_scales=P + 2), 1), (dict(b_scales=P + 8), 1),
    (dict(a=None), 1), (dict(b_scales=None), 1), (dict(y=None), 1), (dict(ld_y=31), 1), (dict(residual=P, ld_res=31), 1),
    (dict(preact=P, ld_preact=31), 1), (dict(y=P + 1), 1), (dict(bias=P + 2), 1), (dict(status=P + 2), 1), (dict(m=2 ** 31), 2),
    (dict(n=2 ** 31 - 2, ld_y=2 ** 31), 2),
])
def test_linear_refuses_on_the_host(abi, kw, expected):
    assert abi.mxfp4_grouped_linear(linear(abi, **kw), None) == expected


@pytest.mark.parametrize("kw,expected", [
    (dict(grad_out=None), 1), (dict(preact=None), 1), (dict(grad_preact=None), 1), (dict(ld_grad=31), 1), (dict(ld_preact=31), 1),
    (dict(ld_y=31), 1), (dict(grad_bias=P), 1), (dict(grad_bias=P, workspace=P, workspace_bytes=255), 1), (dict(grad_preact=P + 1), 1),
    (dict(activation=5, n=31), 1), (dict(num_groups=4097), 2),
])
def test_linear_bwd_refuses_on_the_host(abi, kw, expected):
    a = linear(abi, **{**dict(grad_out=P, preact=P, grad_preact=P), **kw})
    assert abi.mxfp4_grouped_linear_bwd(a, None) == expected


def test_empty_matrices_are_checked_like_others(abi):
    for empty in (dict(m=0), dict(n=0)):
        for kw in (dict(status=P + 2), dict(group_list=P + 4), dict(num_groups=0), dict(group_list_type=2)):
            assert abi.mxfp4_grouped_linear(linear(abi, **{**empty, **kw}), None) == 1
            a = linear(abi, **{**dict(grad_out=P, preact=P, grad_preact=P), **empty, **kw})
            assert abi.mxfp4_grouped_linear_bwd(a, None) == 1


def test_nothing_to_do_is_ok_without_a_device(abi):
    assert abi.mxfp4_moe_route_bwd(route(abi, tokens=0, ld_grad=16), None) == 0
    assert abi.mxfp4_moe_combine(move(abi, tokens=0, rows=None), None) == 0
    assert abi.mxfp4_moe_combine_bwd(move(abi, tokens=0, rows=None, grad_rows=P), None) == 0
    assert abi.mxfp4_moe_dispatch(move(abi, cols=0, values=P), None) == 0
    assert abi.mxfp4_grouped_linear(linear(abi, m=0), None) == 0


def test_outputs_without_an_element_need_no_address(abi):
    assert abi.mxfp4_moe_dispatch(move(abi, tokens=0, row_count=0, rows=None), None) == 0
    assert abi.mxfp4_moe_dispatch(move(abi, x=P, row_count=0), None) == 0
    assert abi.mxfp4_moe_dispatch(move(abi, x=P, cols=0), None) == 0
    assert abi.mxfp4_moe_dispatch(move(abi, x=P, row_count=0, ld_tokens=63), None) == 1
    assert abi.mxfp4_moe_combine_bwd(move(abi, tokens=0, rows=None), None) == 0
    assert abi.mxfp4_moe_combine_bwd(move(abi, grad_out=P, row_count=0), None) == 0
    assert abi.mxfp4_moe_combine_bwd(move(abi, tokens=0, rows=None, ld_out=63), None) == 1


def test_workspace_sizes(abi):
    L = abi.lib()
    assert L.mxfp4_moe_route_workspace(64, 256) == 0
    assert L.mxfp4_moe_route_workspace(65, 256) == 2 * 256 * 4
    assert L.mxfp4_moe_route_workspace(-1, 4) == -1
    assert L.mxfp4_grouped_linear_workspace(130, 10, 3) == (4 + 3) * 10 * 4
    assert L.mxfp4_grouped_linear_workspace(130, 10, 0) == -1
    ws = abi.mxfp4_grouped_linear_fwd_workspace
    big = dict(m=8192, n=4096, k=7168, num_groups=8)
    assert ws(linear(abi, **{**big, "m": 8})) == 0
    assert ws(linear(abi, **big)) == (32 + 8) * 56 * 1024
    assert ws(linear(abi, **{**big, "k": 1024})) == 0
    assert ws(linear(abi, **{**big, "group_list": None})) == (32 + 1) * 56 * 1024
    assert ws(linear(abi, **{**big, "activation": 9})) == -1
    assert L.mxfp4_moe_dispatch_workspace(4, 8, 7168, 32) == 0
    assert L.mxfp4_moe_dispatch_workspace(8192, 8, 7168, 65536) == (8192 * 56 + 65536) * 4
    assert L.mxfp4_moe_dispatch_workspace(-1, 8, 7168, 1) == -1


@pytest.mark.parametrize("kw", [dict(elem_format=2), dict(k=0), dict(k=-64), dict(k=7200), dict(elem_format=1, k=7184), dict(activation=5, n=4097),
                                dict(num_groups=0), dict(m=-1), dict(k=2 ** 62), dict(n=2 ** 31), dict(m=2 ** 31), dict(num_groups=4097)])
def test_forward_workspace_of_invalid_arguments(abi, kw):
    a = linear(abi, **{**dict(m=8192, n=4096, k=7168, num_groups=8), **kw})
    assert abi.mxfp4_grouped_linear_fwd_workspace(a) == -1


def test_cpu_tensors_are_refused():
    from mxfp4_block_fake_b200 import ops
    x = torch.zeros(4, 64)
    i = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: ops.mxfp4_moe_route(x, 2), lambda: ops.mxfp4_moe_route_bwd(x[:, :2], x, i),
                 lambda: ops.mxfp4_moe_dispatch(x, i), lambda: ops.mxfp4_moe_combine(x, i),
                 lambda: ops.mxfp4_moe_combine_bwd(x, x, i), lambda: ops.mxfp4_grouped_linear_bwd(x, x),
                 lambda: ops.mxfp4_grouped_linear(x, x, x, x, k=64)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_reference_by_hand():
    """The tests' own plain form on rows worked by hand."""
    x = torch.tensor([[0.0, 1.0, 1.0, -1.0], [-torch.inf, -torch.inf, 2.0, -torch.inf], [0.0, torch.nan, 0.0, 0.0]])
    w, e = R.route(x, 2, renormalize=False)
    assert e == [[1, 2], [2, -1], [0, 1]] and w[1] == [1.0, 0.0]
    p = 2.718281828459045 / (1 + 2 * 2.718281828459045 + 0.36787944117144233)
    assert w[0] == pytest.approx([p, p], rel=1e-15)
    rows, slots, counts = R.plan(e, 4)
    assert rows == [[1, 3], [4, -1], [0, 2]] and slots == [4, 0, 5, 1, 2, -1] and counts == [1, 2, 2, 0]
    # group limit: groups {0, 1} and {2, 3}; the best two added decide
    y = torch.tensor([[1.0, -9.0, 0.9, 0.8]])
    assert R.route(y, 1, score="sigmoid", num_groups=2, topk_groups=1)[1] == [[2]]
    assert R.route(y, 1, score="sigmoid", num_groups=2, topk_groups=1, group_score="max")[1] == [[0]]
    # the bias decides the choice, not the weight
    w, e = R.route(y, 1, score="sigmoid", bias=torch.tensor([0.0, 5.0, 0.0, float("nan")]), renormalize=False)
    assert e == [[1]] and w[0][0] == pytest.approx(1 / (1 + 2.718281828459045 ** 9), rel=1e-12)
