"""CPU tests of the decode step's operators: calls at the edge of what the header allows, answered before any HIP call."""
from __future__ import annotations

import importlib.util
import pathlib
import sys
import types

import pytest
import torch

from test_step import NULL, OK, SHAPE, attn, qk, read, sample, w4

ROOT = pathlib.Path(__file__).resolve().parents[1]


# ------------------------------------------------------------ empty problems
# An array without elements may have no address: torch gives 0 for such a tensor.
@pytest.mark.parametrize("call,kwargs", [
    (attn, dict(T=0, q=None, out=None)), (attn, dict(B=0, lens=None, table=None)),
    (attn, dict(T=0, B=0, q=None, out=None, lens=None, table=None, q_start=None)),
    (qk, dict(T=0, q=None, k=None, v=None, qo=None, ko=None, pos=None, slots=None)),
    (qk, dict(T=0, cache=False, q=None, k=None, qo=None, ko=None, pos=None)), (qk, dict(T=0, hq=0, q=None, qo=None, k=None)),
    (read, dict(n=0, slots=None, ko=None, vo=None)), (read, dict(n=0, slots=None, vo=None)),
    (sample, dict(rows=0, logits=None, u=None, tokens=None, t=None, k=None, p=None, m=None, ws=None, wsb=0)),
])
def test_empty_problems_need_no_addresses(call, kwargs):
    assert call(**kwargs) == OK


@pytest.mark.parametrize("call,kwargs,status", [
    (attn, dict(T=0, lens=None), NULL), (attn, dict(T=0, table=None), NULL), (attn, dict(B=0, q=None, lens=None), NULL),
    (qk, dict(T=0, cs=None), NULL), (qk, dict(T=0, reach=0), SHAPE), (qk, dict(T=0, kc=None), NULL),
    (read, dict(n=0, kc=None), NULL), (sample, dict(rows=0, vocab=0), SHAPE), (sample, dict(rows=1, u=None), NULL),
])
def test_empty_problems_are_checked_for_the_rest(call, kwargs, status):
    assert call(**kwargs) == status


# ---------------------------------------------------------------- launch sizes
@pytest.mark.parametrize("call,kwargs", [
    (qk, dict(T=1 << 26)), (qk, dict(T=(1 << 26) - 3, cache=False)), (qk, dict(T=2 ** 31 - 1, hq=1, hkv=1, dim=64, rot=64)),
    (read, dict(n=1 << 27, hkv=2)), (read, dict(n=(1 << 28) - 15, hkv=1)), (read, dict(n=1 << 29, hkv=1, dim=64)),
    (read, dict(n=1 << 22, hkv=32, dim=256)),
])
def test_launches_past_2_32_work_items_are_refused(call, kwargs):
    """A launch counts its work-items in 32 bits: 64 for each token from 8192 tokens on, one for 8 values read back."""
    assert call(**kwargs) == SHAPE
    assert "too many rows" in w4.w4_last_error()


# -------------------------------------------------- the binding's compiled checks
def build_module():
    spec = importlib.util.spec_from_file_location("w4_build", ROOT / "gemm_w4_gemv_amd" / "build.py")
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_compiled_checks_are_optional(tmp_path, monkeypatch, capfd):
    """Without a compiler, torch's headers or its version the build goes on, says so and leaves no older copy behind."""
    build = build_module()
    to = tmp_path / build.MARSHAL.name
    for way in ("compiler", "source", "version"):
        stale = [tmp_path / "_marshal.so", to]
        for f in stale:
            f.write_bytes(b"of another build")
        with monkeypatch.context() as m:
            if way == "compiler":
                m.setenv("CXX", str(tmp_path / "no such compiler"))
            elif way == "source":
                m.setattr(build, "CSRC", tmp_path)
            else:
                m.setattr(build.importlib.util, "find_spec", lambda name: None)
            assert build.build_marshal(to) is False
        assert "not compiled" in capfd.readouterr().err
        assert not list(tmp_path.glob("_marshal*"))


def test_compiled_checks_are_taken_for_this_torch_alone():
    from gemm_w4_gemv_amd import step
    built_for = (f"{torch.version.__version__} {torch.version.git_version}", sys.hexversion >> 16)
    assert step._fits(types.SimpleNamespace(built_for=built_for))
    for other in ((built_for[0] + "0", built_for[1]), (built_for[0], built_for[1] + 1), None):
        assert not step._fits(types.SimpleNamespace(built_for=other))
    assert not step._fits(types.SimpleNamespace())  # one that does not say


def test_compiled_checks_are_in_use_where_they_can_be_built(tmp_path):
    from gemm_w4_gemv_amd import step
    build = build_module()
    if not build.build_marshal(tmp_path / build.MARSHAL.name):
        pytest.skip("the checks do not compile here")
    assert build.MARSHAL.exists(), "the library was built without them"
    assert step._marshal is not None and step._marshal.__file__ == str(build.MARSHAL)
    assert step._addresses is step._marshal.addresses and step._heads is step._marshal.heads
    assert step._optional_addresses is step._marshal.optional_addresses


# ------------------------------------------------------------- the decode step
def linears(*names, layer=0):
    return [{"name": n, "layer": layer} for n in names]


ATTENTION = types.SimpleNamespace(caches=[None, None])


@pytest.mark.parametrize("lins,attention,sampler,what", [
    (linears("q", "k", "o", "v"), True, False, "o"), (linears("o", "q", "k", "v"), True, False, "o"),
    (linears("q", "v", "o"), True, False, "k"), (linears("q", "k", "v", "o") + linears("v", "o", layer=1), True, False, "q"),
    (linears("q", "k", "v", "q", "o"), True, False, "q"), (linears("q", "k", "v", "o", "o"), True, False, "o"),
    (linears("q", "k", "v", "o", layer=2), True, False, "layer 2"), (linears("q", "k", "v", "o", layer=-1), True, False, "layer -1"),
    (linears("q", "k", "v", "o"), True, True, "logits"), (linears("logits", "logits"), False, True, "logits"),
    ([], False, True, "logits"),
])
def test_decode_step_refuses_linears_out_of_order(lins, attention, sampler, what):
    """Before anything runs: an o that would read what its attention has not written, a layer without its three,
    one that the attention does not have, a sampler without logits."""
    from gemm_w4_gemv_amd.decode import DecodeStep
    with pytest.raises(ValueError, match=what):
        DecodeStep(lins, stream=object(), attention=ATTENTION if attention else None, sampler=object() if sampler else None)


# ----------------------------------------------------- sizes past 32 bits
FAR = 2 ** 32  # ctypes would take its lowest 32 bits: 0


def meta(*shape, dtype=torch.int32):
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("what", ["block_size", "rows", "pages", "requests", "width"])
def test_plan_refuses_sizes_past_32_bits(what):
    more = {k: FAR + 16 if k == what else 16 for k in ("block_size", "rows", "pages", "requests", "width")}
    B = more["requests"]
    table, lens, rows = meta(B, more["width"]), meta(B), meta(more["rows"])
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_kv4_plan(lens, lens, table, meta(more["pages"]), meta(1), more["block_size"], meta(B + 1), lens, rows, rows, meta(2))


def test_attn_and_sample_refuse_sizes_past_32_bits():
    from gemm_w4_gemv_amd import step
    cache = object.__new__(step.Kv4Cache)
    cache.head_dim, cache.device_index, cache.block_size, cache.ref = 64, 0, 16, None
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_sample(meta(1, FAR + 100, dtype=torch.bfloat16), None, None)
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_sample(meta(FAR + 1, 100, dtype=torch.bfloat16), None, None)
    q = meta(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="32 bits"):
        w4.w4_kv4_attn(q, cache, meta(FAR + 3, 0), meta(FAR + 3), q)
    assert w4.w4_sample_workspace_bytes(1, FAR + 40000) == 0


@pytest.mark.parametrize("name", ["max_q", "max_kv", "window", "sinks"])
def test_attn_far_negative_sizes_are_negative(name):
    """-2^32 is refused like -1, not taken for 0; and what is past the other end counts as the largest."""
    import ctypes
    from gemm_w4_gemv_amd import step
    cache = types.SimpleNamespace(ref=ctypes.byref(step._CacheStruct(1, 1, 1, 1, 100000, 64, 1, 128)))
    size = lambda **k: step.w4_kv4_attn_workspace_bytes(cache, **{**dict(T=4, B=4, q_heads=1, max_q=1, max_kv=100000), **k})  # noqa: E731
    assert size() > 0
    assert size(**{name: -1}) == 0 and size(**{name: -FAR}) == 0 and size(**{name: 1 - FAR}) == 0
    assert size(**{name: FAR}) == size(**{name: 2 ** 31 - 1})


