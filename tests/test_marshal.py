"""The binding's compiled tensor checks against the ones in Python: the same addresses and strides
where a tensor is as it should be, the same error where it is not."""
from __future__ import annotations

import pytest
import torch

w4 = pytest.importorskip("gemm_w4_gemv_amd")
from gemm_w4_gemv_amd import step  # noqa: E402

marshal = pytest.importorskip("gemm_w4_gemv_amd._marshal")
slow_addresses, slow_optional, slow_heads = step._in_python
bf16, i32, f32 = torch.bfloat16, torch.int32, torch.float32


def outcome(f, *args):
    try:
        return f(*args)
    except Exception as e:  # noqa: BLE001 - the kind and the words are what is compared
        return type(e), str(e)


def same(fast, slow, *args):
    got, want = outcome(fast, *args), outcome(slow, *args)
    assert got == want, (got, want)
    return got


def test_the_compiled_checks_are_in_use():
    assert step._addresses is marshal.addresses and step._heads is marshal.heads


@pytest.mark.parametrize("args", [
    (0, torch.zeros(3, dtype=i32), "x", i32, 3), (0, None, "x", i32, 3), (0, [1, 2], "x", i32, None),
    (0, torch.zeros(3), "x", i32, 4), (-1, torch.zeros(3, dtype=i32), "x", i32, 3), (None, torch.zeros(1, dtype=i32), "x", i32, 1),
    (0, torch.zeros(0, dtype=i32), "x", i32, 0), (0, torch.zeros(2, 2, dtype=i32).to_sparse(), "x", i32, None),
    (0, torch.zeros(3, dtype=i32, device="meta"), "x", i32, 3), (0,),
])
def test_host_tensors_and_others_are_refused_alike(args):
    same(marshal.addresses, slow_addresses, *args)
    same(marshal.optional_addresses, slow_optional, *args)


@pytest.mark.parametrize("t", [torch.zeros(2, 3, 64, dtype=bf16), torch.zeros(2, 3, dtype=bf16), None, 5])
def test_heads_are_refused_alike(t):
    got = same(marshal.heads, slow_heads, t, "q", 0)
    assert isinstance(got[0], type) and issubclass(got[0], Exception)
    same(marshal.heads, slow_heads, t, "q", 0, 2, 3, 64)


@pytest.mark.gpu
def test_on_the_gpu():
    assert torch.cuda.is_available()
    x, y = torch.zeros(7, dtype=i32, device="cuda"), torch.zeros(4, 6, dtype=f32, device="cuda")
    good = (0, x, "x", i32, 7, y, "y", f32, None)
    assert same(marshal.addresses, slow_addresses, *good) == (x.data_ptr(), y.data_ptr())
    assert same(marshal.optional_addresses, slow_optional, 0, None, "n", i32, 3, x, "x", i32, 7) == (None, x.data_ptr())
    empty = torch.zeros(0, dtype=i32, device="cuda")
    same(marshal.addresses, slow_addresses, 0, empty, "e", i32, 0)
    for bad in ((0, x, "x", i32, 8), (0, x, "x", f32, 7), (1, x, "x", i32, 7), (0, x[::2], "x", i32, 4), (0, y.t(), "y", f32, None),
                (0, y, "y", f32, 24), (0, x.cpu(), "x", i32, 7), (0, x, "x", i32, 7, None, "n", i32, 1)):
        assert same(marshal.addresses, slow_addresses, *bad)[0] in (TypeError, ValueError)
    q = torch.zeros(5, 12, 64, dtype=bf16, device="cuda")
    for t in (q, q[:, 2:6], q[1:2, 3:], q[:0], q[::2], q[:, :1], q[0:1, 0:1, 0:8], torch.zeros(3, 1, 1, dtype=bf16, device="cuda")):
        assert same(marshal.heads, slow_heads, t, "q", 0)[0] == t.data_ptr()
        same(marshal.heads, slow_heads, t, "q", 0, None, None, 64)
        same(marshal.heads, slow_heads, t, "q", 0, 5, 12, 64)
    for t in (q[:, ::2], q.transpose(0, 1), q[:, :, ::2], q.float(), q[0], q.cpu()):
        assert isinstance(same(marshal.heads, slow_heads, t, "q", 0)[0], type)
    same(marshal.heads, slow_heads, q, "q", 1)
