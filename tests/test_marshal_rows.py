"""The compiled check of a call's matrices against the one in Python: the same addresses and row strides where a
tensor is as it should be, the same error where it is not."""
from __future__ import annotations

import pytest
import torch

w4 = pytest.importorskip("gemm_w4_gemv_amd")
from gemm_w4_gemv_amd import block  # noqa: E402
from test_marshal import same  # noqa: E402

marshal = pytest.importorskip("gemm_w4_gemv_amd._marshal")
bf16, f32 = torch.bfloat16, torch.float32


def test_the_compiled_check_is_in_use():
    assert block._rows is marshal.rows


@pytest.mark.parametrize("args", [
    (0, 2, 8, torch.zeros(2, 8, dtype=bf16), "x", bf16), (0, 2, 8, [1], "x", bf16), (0, 2, 8, torch.zeros(16), "x", f32),
    (0, 2, 8, torch.zeros(2, 9), "x", f32), (0, 2, 8, torch.zeros(2, 8, device="meta"), "x", f32),
    (0, 2, 8, torch.zeros(2, 8).to_sparse(), "x", f32), (-1, 2, 8, torch.zeros(2, 16)[:, ::2], "x", f32), (0,),
])
def test_others_are_refused_alike(args):
    same(marshal.rows, block._rows_in_python, *args)


def test_none_and_host_tensors_pass_alike():
    x = torch.zeros(5, 24)
    assert same(marshal.rows, block._rows_in_python, -1, 5, 8, None, "n", bf16, x[:, 8:16], "x", f32) == \
        (None, 0, x.data_ptr() + 32, 24)


def test_a_gate_that_is_no_tensor():
    assert isinstance(same(block._given, block._given, 0, 2, 8, None, None, [1.0]), tuple)
    with pytest.raises((TypeError, ValueError)):
        block._given(0, 2, 8, None, None, [1.0] * 8)


@pytest.mark.gpu
def test_on_the_gpu():
    assert torch.cuda.is_available()
    x = torch.zeros(6, 32, dtype=bf16, device="cuda")
    good = [(6, 32, x), (6, 16, x[:, 8:24]), (3, 32, x[::2]), (1, 32, x[:1]), (0, 32, x[:0]), (6, 32, x[0].expand(6, 32)),
            (6, 1, x[:, 3:4]), (0, 16, x[:0, ::2]), (1, 32, torch.zeros(32, 1, dtype=bf16, device="cuda").t())]
    for n, wide, t in good:
        got = same(marshal.rows, block._rows_in_python, 0, n, wide, t, "x", bf16, None, "n", f32)
        assert got[0] == t.data_ptr() and got[2:] == (None, 0)
    for n, wide, t, kind, device in ((6, 16, x[:, ::2], bf16, 0), (5, 32, x, bf16, 0), (6, 32, x, f32, 0), (6, 32, x, bf16, 1),
                                     (6, 32, x.cpu(), bf16, 0), (32, 6, x.t(), bf16, 0)):
        got = same(marshal.rows, block._rows_in_python, device, n, wide, t, "x", kind)
        assert isinstance(got[0], type)
