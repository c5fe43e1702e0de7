"""CPU tests of the operators around a block's products: the header against the
library and the binding, every refusal (checked before any HIP call), and
hand-built pins of the FP64 oracle that they are compared with."""
from __future__ import annotations

import ctypes
import pathlib
import re

import numpy as np
import pytest
import torch

from oracle import block as ref

w4 = pytest.importorskip("gemm_w4_gemv_amd")
from gemm_w4_gemv_amd import block, step  # noqa: E402

lib = w4.lib
HEADER = pathlib.Path(__file__).resolve().parents[1] / "include" / "w4_block.h"
OK, NULL, SHAPE, UNSUP, ALIGN, WS, ALIAS, ARG = 0, 1, 2, 3, 4, 5, 6, 7
P = 1 << 40  # addresses that are never read: 64 GiB apart
at = lambda i: P + (i << 36)  # noqa: E731


# --------------------------------------------------------------- the header
def test_header_binding_and_exports_agree():
    text = HEADER.read_text()
    names = set(re.findall(r"W4_API\s+[\w\s\*]+?\b(w4_\w+)\s*\(", text))
    assert names == set(block.SIGNATURES)
    assert all(hasattr(lib, n) and hasattr(w4, n) for n in names)
    for name, value in (("W4_NORM_MAX_DIM", block.NORM_MAX_DIM), ("W4_MOE_MAX_TOP", block.MOE_MAX_TOP),
                        ("W4_MOE_SORT_MAX_EXPERTS", block.MOE_SORT_MAX_EXPERTS)):
        assert re.search(rf"#define {name} {value}\b", text)


# ---------------------------------------------------------------- refusals
def norm_struct(**k):
    D = k.get("D", 512)
    return block._NormArgs(
        h=k.get("h", at(0)), y=k.get("y", at(1)), h_out=k.get("ho", at(2)), z=k.get("z", at(3)),
        y_weight=k.get("wy", at(4)), z_weight=k.get("wz", at(5)), gate=k.get("gate", at(6)),
        h_stride=k.get("hs", D), y_stride=k.get("ys", D), h_out_stride=k.get("hos", D), z_stride=k.get("zs", D),
        gate_stride=k.get("gs", 0), T=k.get("T", 5), D=D, h_f32=k.get("wide", 0), residual_scale=k.get("a", 1.0),
        branch_scale=k.get("b", 1.0), eps=k.get("eps", 1e-6), weight_add=k.get("add", 0.0))


def norm(**k):
    return lib.w4_block_norm(ctypes.byref(norm_struct(**k)), None)


NORM_BAD = [
    (dict(h=None), NULL), (dict(T=-1), SHAPE), (dict(T=(1 << 21) + 1), SHAPE), (dict(D=0), SHAPE), (dict(D=12), SHAPE),
    (dict(D=16392), SHAPE), (dict(D=-8), SHAPE), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(eps=float("inf")), ARG), (dict(add=float("inf")), ARG), (dict(a=float("nan")), ARG), (dict(b=float("inf")), ARG),
    (dict(hs=504), ARG), (dict(hs=516), ARG), (dict(ys=0), ARG), (dict(ys=(1 << 40) + 8), ARG), (dict(gs=8), ARG),
    (dict(gs=-512), ARG), (dict(h=at(0) + 8), ALIGN), (dict(y=at(1) + 2), ALIGN), (dict(wy=at(4) + 8), ALIGN),
    (dict(wz=at(5) + 4), ALIGN), (dict(gate=at(6) + 2), ALIGN), (dict(y=None), ARG), (dict(y=None, wy=None), ARG),
]


@pytest.mark.parametrize("kwargs,status", NORM_BAD + [
    (dict(y=None, wy=None, gate=None), ARG), (dict(ho=None, z=None), NULL), (dict(hos=8), ARG), (dict(zs=520 + 4), ARG),
    (dict(ho=at(2) + 8), ALIGN), (dict(z=at(3) + 2), ALIGN), (dict(ho=at(3)), ALIAS), (dict(ho=at(1)), ALIAS),
    (dict(z=at(0)), ALIAS), (dict(ho=at(0), hos=1024), ALIAS), (dict(ho=at(0) + 16), ALIAS), (dict(z=at(1) + 1024), ALIAS),
    (dict(z=at(1), zs=520), ALIAS), (dict(z=at(4)), ALIAS), (dict(ho=at(6)), ALIAS), (dict(z=at(6) - 16), ALIAS),
    (dict(gs=512, z=at(6) + 4 * 1024), ALIAS), (dict(wide=1, z=at(2) + 5 * 1024), ALIAS), (dict(y=at(0), ho=at(0)), ALIAS),
])
def test_block_norm_refusals(kwargs, status):
    assert norm(**kwargs) == status
    assert "w4_block_norm" in w4.w4_last_error()


def test_block_norm_empty_problem_launches_nothing():
    assert norm(T=0) == OK
    assert norm(T=0, h=None, y=None, ho=None, z=None) == OK
    assert norm(T=0, ho=at(0), z=at(1)) == OK  # outputs that are their inputs


def grad(**k):
    D = k.get("D", 512)
    g = block._NormGradArgs(
        dh_out=k.get("dho", at(8)), dz=k.get("dz", at(9)), dh=k.get("dh", at(10)), dy=k.get("dy", at(11)),
        dh_out_stride=k.get("dhos", D), dz_stride=k.get("dzs", D), dh_stride=k.get("dhs", D), dy_stride=k.get("dys", D),
        d_gate_stride=k.get("dgs", D), d_y_weight=k.get("sy", at(12)), d_z_weight=k.get("sz", at(13)), d_gate=k.get("dg", at(14)))
    return lib.w4_block_norm_grad(ctypes.byref(norm_struct(**k)), ctypes.byref(g), k.get("ws", at(15)),
                                  k.get("wsb", 1 << 30), None)


@pytest.mark.parametrize("kwargs,status", NORM_BAD + [
    (dict(dho=None, dz=None), NULL), (dict(dh=None, dy=None, sy=None, sz=None, dg=None), NULL), (dict(wy=None), ARG),
    (dict(wz=None), ARG), (dict(gate=None), ARG), (dict(y=None, wy=None, gate=None, sy=None, dg=None), ARG),
    (dict(dhos=8), ARG), (dict(dzs=516), ARG), (dict(dhs=0), ARG), (dict(dys=504), ARG), (dict(gs=512, dgs=8), ARG),
    (dict(dho=at(8) + 8), ALIGN), (dict(dh=at(10) + 2), ALIGN), (dict(sy=at(12) + 4), ALIGN), (dict(dg=at(14) + 8), ALIGN),
    (dict(ws=None), WS), (dict(wsb=16), WS), (dict(ws=at(15) + 8), ALIGN), (dict(dh=at(0)), ALIAS), (dict(dy=at(1)), ALIAS),
    (dict(dh=at(9)), ALIAS), (dict(dy=at(8)), ALIAS), (dict(dh=at(8), dhs=520), ALIAS), (dict(dy=at(9) + 16), ALIAS),
    (dict(sy=at(13)), ALIAS), (dict(sz=at(9)), ALIAS), (dict(dg=at(6)), ALIAS), (dict(ws=at(10)), ALIAS), (dict(ws=at(0)), ALIAS),
    (dict(gs=512, dg=at(6)), ALIAS),
])
def test_block_norm_grad_refusals(kwargs, status):
    assert grad(**kwargs) == status
    assert "w4_block_norm_grad" in w4.w4_last_error()
    a = norm_struct()
    assert lib.w4_block_norm_grad(ctypes.byref(a), None, None, 0, None) == NULL
    assert lib.w4_block_norm_grad(None, None, None, 0, None) == NULL


def test_block_norm_grad_workspace():
    size = w4.w4_block_norm_grad_workspace_bytes
    assert size(0, 512) == size(-1, 512) == size(5, 0) == size(5, 16392) == size((1 << 21) + 1, 8) == 0
    assert 0 < size(1, 512) <= size(5000, 512) == size(1 << 21, 512)  # a bounded number of runs of rows
    assert grad(T=0, sy=None, sz=None, dg=None, ws=None, wsb=0) == OK  # nothing to write


def sort(**k):
    top, D = k.get("top", 4), k.get("D", 512)
    a = block._SortArgs(
        experts=k.get("experts", at(0)), row_start=k.get("start", at(1)), row_of=k.get("row_of", at(2)),
        source=k.get("source", at(3)), x=k.get("x", at(4)), rows=k.get("rows", at(5)), x_stride=k.get("xs", D),
        rows_stride=k.get("rs", D), T=k.get("T", 3000), top=top, num_experts=k.get("E", 64), capacity=k.get("cap", 0),
        R=k.get("R", 12000), D=D)
    return lib.w4_moe_sort(ctypes.byref(a), k.get("ws", at(6)), k.get("wsb", 1 << 30), None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(experts=None), NULL), (dict(start=None), NULL), (dict(row_of=None), NULL), (dict(x=None), NULL), (dict(rows=None), NULL),
    (dict(T=-1), SHAPE), (dict(top=0), SHAPE), (dict(top=65), SHAPE), (dict(T=1 << 23, top=2), SHAPE), (dict(E=0), SHAPE),
    (dict(E=1025), SHAPE), (dict(R=-1), SHAPE), (dict(D=0), SHAPE), (dict(D=12), SHAPE), (dict(D=(1 << 20) + 8), SHAPE),
    (dict(cap=-1), ARG), (dict(xs=504), ARG), (dict(rs=516), ARG), (dict(experts=at(0) + 2), ALIGN), (dict(source=at(3) + 1), ALIGN),
    (dict(x=at(4) + 8), ALIGN), (dict(rows=at(5) + 2), ALIGN), (dict(ws=None), WS), (dict(wsb=16), WS), (dict(ws=at(6) + 8), ALIGN),
    (dict(row_of=at(0)), ALIAS), (dict(source=at(2) + 400), ALIAS), (dict(rows=at(4) + 1024), ALIAS), (dict(start=at(2)), ALIAS),
    (dict(ws=at(5)), ALIAS), (dict(ws=at(0)), ALIAS), (dict(start=at(3)), ALIAS),
])
def test_moe_sort_refusals(kwargs, status):
    assert sort(**kwargs) == status
    assert "w4_moe_sort" in w4.w4_last_error()


def test_moe_sort_workspace():
    size = w4.w4_moe_sort_workspace_bytes
    assert size(0, 4, 64) == size(10, 0, 64) == size(10, 4, 0) == size(10, 65, 4) == size(1 << 23, 2, 4) == 0
    assert size(1, 6, 64) == 0  # a decode step's choices need no table
    assert size(8191, 6, 64) == 48 * 64 * 4  # counts of 48 chunks
    for T, top, E in ((8191, 8, 256), (1 << 23, 1, 1024), (1 << 17, 64, 1)):
        assert 0 < size(T, top, E) <= 4 * ((1 << 22) + 1024)  # of at most 2^22 and their sums


def combine(**k):
    N = k.get("N", 512)
    a = block._CombineArgs(
        y=k.get("y", at(0)), row_of=k.get("row_of", at(1)), weights=k.get("w", at(2)), add=k.get("add", at(3)),
        out=k.get("out", at(4)), y_stride=k.get("ys", N), add_stride=k.get("as_", N), out_stride=k.get("os", N),
        T=k.get("T", 5), top=k.get("top", 2), R=k.get("R", 10), N=N)
    return lib.w4_moe_combine(ctypes.byref(a), None)


CHOICES_BAD = [(dict(T=-1), SHAPE), (dict(top=0), SHAPE), (dict(top=65), SHAPE), (dict(T=1 << 22, top=3), SHAPE), (dict(R=-1), SHAPE),
               (dict(N=0), SHAPE), (dict(N=20), SHAPE), (dict(N=(1 << 20) + 8), SHAPE), (dict(row_of=at(1) + 2), ALIGN),
               (dict(w=at(2) + 1), ALIGN), (dict(y=at(0) + 8), ALIGN), (dict(ys=504), ARG), (dict(y=None), NULL)]


@pytest.mark.parametrize("kwargs,status", CHOICES_BAD + [
    (dict(out=None), NULL), (dict(as_=8), ARG), (dict(os=513), ARG), (dict(add=at(3) + 2), ALIGN), (dict(out=at(4) + 8), ALIGN),
    (dict(out=at(0) + 9 * 1024), ALIAS), (dict(out=at(1)), ALIAS), (dict(out=at(2)), ALIAS), (dict(out=at(3) + 16), ALIAS),
    (dict(out=at(3), os=1024), ALIAS),
])
def test_moe_combine_refusals(kwargs, status):
    assert combine(**kwargs) == status
    assert "w4_moe_combine" in w4.w4_last_error()


def combine_grad(**k):
    N = k.get("N", 512)
    a = block._CombineGradArgs(
        dout=k.get("dout", at(4)), y=k.get("y", at(0)), row_of=k.get("row_of", at(1)), weights=k.get("w", at(2)),
        dy=k.get("dy", at(5)), dweights=k.get("dw", at(6)), dout_stride=k.get("ds", N), y_stride=k.get("ys", N),
        dy_stride=k.get("dys", N), T=k.get("T", 5), top=k.get("top", 2), R=k.get("R", 10), N=N)
    return lib.w4_moe_combine_grad(ctypes.byref(a), None)


@pytest.mark.parametrize("kwargs,status", CHOICES_BAD + [
    (dict(dout=None), NULL), (dict(dy=None, dw=None), NULL), (dict(ds=0), ARG), (dict(dys=516), ARG), (dict(dout=at(4) + 8), ALIGN),
    (dict(dy=at(5) + 2), ALIGN), (dict(dw=at(6) + 2), ALIGN), (dict(dy=at(4)), ALIAS), (dict(dy=at(0) + 16), ALIAS),
    (dict(dy=at(0), dys=1024), ALIAS), (dict(dw=at(0) + 64), ALIAS), (dict(dw=at(5)), ALIAS), (dict(dw=at(1)), ALIAS), (dict(dw=at(2)), ALIAS),
])
def test_moe_combine_grad_refusals(kwargs, status):
    assert combine_grad(**kwargs) == status
    assert "w4_moe_combine_grad" in w4.w4_last_error()


def test_empty_problems_launch_nothing():
    assert combine(T=0) == combine_grad(T=0) == OK
    assert combine(T=0, out=None, y=None, add=None, row_of=None, w=None) == OK
    assert combine(T=0, out=at(3)) == combine_grad(T=0, dy=at(0)) == OK


# ------------------------------------------------- a shared prefix (w4_step.h)
def shared(**k):
    hq, dim, block_size = 4, 128, k.get("block", 64)
    c = step._CacheStruct(at(20), at(21), at(22), at(23), 100, block_size, 2, dim)
    a = step._AttnArgs(q=k.get("q", at(0)), out=k.get("out", at(1)), q_stride=hq * dim, out_stride=hq * dim,
                       block_table=at(2), kv_lens=at(3), q_start=k.get("q_start", at(4)), T=k.get("T", 6), B=k.get("B", 3),
                       q_heads=hq, max_blocks=80, max_q=k.get("max_q", 2), max_kv=5000, scale=k.get("scale", 0.1))
    return lib.w4_kv4_attn_shared(ctypes.byref(a), k.get("prefix_table", at(6)), k.get("prefix", 4096), ctypes.byref(c),
                                  k.get("ws", at(5)), k.get("wsb", 1 << 30), None)


@pytest.mark.parametrize("kwargs,status", [
    (dict(prefix=-1), SHAPE), (dict(prefix_table=None), NULL), (dict(prefix_table=at(6) + 2), ALIGN), (dict(q=None), NULL),
    (dict(scale=0.0), ARG), (dict(ws=None), WS), (dict(wsb=64), WS), (dict(ws=at(5) + 8), ALIGN), (dict(out=at(6)), ALIAS),
    (dict(ws=at(6) + 240), ALIAS), (dict(block=24), UNSUP), (dict(T=-1), SHAPE), (dict(q_start=None), SHAPE),
])
def test_attn_shared_refusals(kwargs, status):
    assert shared(**kwargs) == status
    assert "w4_kv4_attn_shared" in w4.w4_last_error()


def test_attn_shared_empty_and_its_workspace():
    assert shared(T=0, B=0) == shared(max_q=0) == OK
    c = step._CacheStruct(at(20), at(21), at(22), at(23), 100, 64, 2, 128)
    fake = type("Cache", (), {"ref": ctypes.byref(c)})()
    size = lambda prefix, B=16: w4.w4_kv4_attn_shared_workspace_bytes(fake, B, B, 4, 1, 5000, prefix)  # noqa: E731
    assert size(0) == size(31) == w4.w4_kv4_attn_workspace_bytes(fake, 16, 16, 4, 1, 5000)  # no whole tile of tokens
    assert size(-1) == 0 and size(4096) > 0 and size(2 ** 40) == size(2 ** 31 - 1)
    assert size(4096) <= 16 * 4 * 128 * (128 + 2) * 4  # at most 128 parts a row


def test_binding_refuses_host_tensors_and_wrong_layouts():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        w4.w4_block_norm(x, z=x)  # host memory
    with pytest.raises(TypeError):
        w4.w4_block_norm(x.half(), z=x)
    with pytest.raises(ValueError):
        w4.w4_block_norm(x[0], z=x)
    with pytest.raises(ValueError):
        w4.w4_moe_sort(ids, 4, ids, ids)
    with pytest.raises(ValueError):
        w4.w4_moe_sort(ids[0], 4, ids, ids)
    with pytest.raises(ValueError):
        w4.w4_moe_combine(x, x)
    with pytest.raises(ValueError):
        w4.w4_moe_combine_grad(x)
    with pytest.raises(ValueError):
        w4.w4_moe_combine_grad(x, x)
    with pytest.raises(TypeError):
        w4.w4_kv4_attn_shared(x, None, x, x, x, None, 0)


# -------------------------------------------------------- pins of the oracle
def test_pin_block_norm_by_hand():
    y = np.array([[3.0, -4.0] * 4])  # mean square 12.5
    h = np.ones((1, 8))
    x, z = ref.block_norm(h, y, np.full(8, 0.5), np.full(8, 2.0), np.full(8, 10.0), 2.0, 0.5, 3.5, 1.0)
    assert np.allclose(x, 2 + 0.5 * 10 * np.array([[3.0, -4.0] * 4]) / 4 * 1.5)  # sqrt(12.5 + 3.5) = 4
    assert np.allclose(z, x / np.sqrt(np.mean(x * x) + 3.5) * 3)
    x, z = ref.block_norm(h, y)
    assert np.array_equal(x, h + y) and z is x
    assert ref.block_norm(h)[0] is h


@pytest.mark.parametrize("post,pre,gated", [(1, 1, 1), (0, 1, 1), (1, 0, 0), (1, 1, 0), (0, 0, 1)])
def test_pin_block_norm_grad_against_differences(post, pre, gated):
    g = np.random.default_rng(3)
    T, D = 3, 16
    v = dict(h=g.normal(0, 2, (T, D)), y=g.normal(0, 1, (T, D)), y_weight=g.normal(1, 0.2, D) if post else None,
             z_weight=g.normal(1, 0.2, D) if pre else None, gate=g.normal(0, 1, (T, D)) if gated else None)
    dho, dz = g.normal(0, 1, (T, D)), g.normal(0, 1, (T, D))
    rest = dict(a=0.75, b=0.5, eps=2.0 ** -10, add=0.25)
    got = ref.block_norm_grad(dh_out=dho, dz=dz, **v, **rest)

    def loss(**changed):
        x, z = ref.block_norm(**{**v, **changed}, **rest)
        return (x * dho).sum() + (z * dz).sum()

    for name, grad_name in (("h", "dh"), ("y", "dy"), ("y_weight", "d_y_weight"), ("z_weight", "d_z_weight"), ("gate", "d_gate")):
        if v[name] is None:
            continue
        way, step_ = g.normal(0, 1, v[name].shape), 1e-5
        diff = (loss(**{name: v[name] + step_ * way}) - loss(**{name: v[name] - step_ * way})) / (2 * step_)
        assert np.isclose((got[grad_name] * way).sum(), diff, rtol=1e-7, atol=1e-7), name
    alone = ref.block_norm_grad(v["h"], dz=dz, z_weight=v["z_weight"], eps=rest["eps"], add=rest["add"])
    way = g.normal(0, 1, (T, D))
    f = lambda s: (ref.block_norm(v["h"] + s * way, z_weight=v["z_weight"], eps=rest["eps"], add=rest["add"])[1] * dz).sum()  # noqa: E731
    assert np.isclose((alone["dh"] * way).sum(), (f(1e-5) - f(-1e-5)) / 2e-5, rtol=1e-7, atol=1e-7)


def test_pin_moe_sort_by_hand():
    start, row_of, source = ref.moe_sort([[2, 0], [0, 2], [5, 0], [2, -1]], 3)
    assert start == [0, 3, 3, 6] and row_of.tolist() == [[3, 0], [1, 4], [-1, 2], [5, -1]]
    assert source == [1, 2, 5, 0, 3, 6, -1, -1]
    start, row_of, source = ref.moe_sort([[2, 0], [0, 2], [5, 0], [2, -1]], 3, capacity=2)
    assert start == [0, 2, 2, 4] and row_of.tolist() == [[2, 0], [1, 3], [-1, -1], [-1, -1]]
    assert source == [1, 2, 0, 3, -1, -1, -1, -1]


def test_pin_combine_by_hand():
    y = np.array([[1.0, 2.0], [10.0, 20.0], [100.0, 200.0]])
    rows = np.array([[2, 0], [1, -1], [7, -1]])
    w = np.array([[0.5, 2.0], [3.0, 9.0], [1.0, 1.0]])
    out, size = ref.combine(y, rows, w, np.ones((3, 2)))
    assert out.tolist() == [[53.0, 105.0], [31.0, 61.0], [1.0, 1.0]] and np.all(size >= np.abs(out))
    dy, dw, _ = ref.combine_grad(np.array([[1.0, 1.0], [2.0, 0.0], [5.0, 5.0]]), y, rows, w)
    assert dy.tolist() == [[2.0, 2.0], [6.0, 0.0], [0.5, 0.5]]
    assert dw.tolist() == [[300.0, 3.0], [20.0, 0.0], [0.0, 0.0]]
