"""GPU parity of the operators around a block's products against the FP64 oracle.

Tolerances, from the arithmetic (a rounding to BF16 is off by at most 2^-8
relative, one to FP32 by 2^-24).  K = 2^-20 stands for the handful (at most 16)
of FP32 roundings of one term, the inverse root's among them:
  * h': a fused sum of two terms, so K (|a h| + |b g u|), and its type's rounding;
  * z: h' off by that much moves the root mean square by at most the same part,
    relative, of its norm; then K of the result and its rounding;
  * gradients: the same for each of the steps they are made of (``grad_bounds``);
    sums over tokens are of terms off by so much, at most 16 of them in FP32
    before FP64 takes over (a run of 512th of the rows), else one more 2^-24 each;
  * combine: ``top`` + 1 fused additions, each off by 2^-24 of the magnitudes so
    far, then the rounding to BF16; dweights: a lane adds at most
    8 ceil(N / 512) products, lanes and waves 12 sums more, each off by 2^-24
    of the magnitudes; dy one product, rounded once;
  * tables and copied rows: equal, bit for bit.
BF16 results below its normal numbers are off by half of 2^-133.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import seeded_inputs as si
from oracle import block as ref
from test_gpu_step import ints

pytestmark = pytest.mark.gpu

w4 = pytest.importorskip("gemm_w4_gemv_amd")

DEV = "cuda"
bf16, f32 = torch.bfloat16, torch.float32
K = 2.0 ** -20
ROUND = {bf16: 2.0 ** -8, f32: 2.0 ** -24}
TINY = 2.0 ** -134


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(got, want, bound, what=""):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - want) <= bound + TINY)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.nanmax((np.abs(got - want) / (bound + TINY))[bad]):.3g} x the bound"


def tensor(seed, shape, size=1.0, dtype=bf16, mean=0.0):
    g = si.rng(91, seed, *shape)
    return torch.from_numpy((mean + size * g.normal(0, 1, shape)).astype(np.float32)).to(dtype).to(DEV)


def padded(t, pad):
    """The same rows, ``pad`` values further apart."""
    space = torch.full((t.shape[0], t.shape[1] + pad), 7.0, dtype=t.dtype, device=DEV)
    space[:, :t.shape[1]] = t
    return space[:, :t.shape[1]]


# -------------------------------------------------------------------- norms
def norm_case(seed, T, D, kind, gate, post, pre):
    return dict(h=tensor(seed, (T, D), 3.0, kind), y=tensor(seed + 1, (T, D)),
                y_weight=tensor(seed + 2, (D,), 0.2, mean=1.0) if post else None,
                z_weight=tensor(seed + 3, (D,), 0.2, mean=1.0) if pre else None,
                gate=None if gate is None else tensor(seed + 4, (D,) if gate == "channel" else (T, D), 0.5))


def norm_bounds(v, a, b, eps, add):
    """(h', z, error of h' in FP32, of z)."""
    h, y, wy, wz, gate = (f64(v[n]) for n in ("h", "y", "y_weight", "z_weight", "gate"))
    x, z = ref.block_norm(h, y, wy, wz, gate, a, b, eps, add)
    size = np.abs(x) if y is None else np.abs(np.float32(a) * h) + np.abs(x - np.float32(a) * h)
    ex = K * size if y is not None else 0 * size
    if wz is None:
        return x, z, ex, ex + ROUND[bf16] * np.abs(z)
    r = ref.rms(x, eps)
    rho = np.sqrt((ex ** 2).mean(-1, keepdims=True)) / r + K
    w = np.abs(wz + float(np.float32(add)))
    return x, z, ex, w / r * (ex + np.abs(x) * rho) + ROUND[bf16] * np.abs(z)


def run_norm(v, a=1.0, b=1.0, eps=1e-6, add=0.0, h_out=True, z=True, pad=0, **kw):
    T, D = v["h"].shape
    fresh = lambda kind: torch.full((T, D + pad), 7.0, dtype=kind, device=DEV)[:, :D]  # noqa: E731
    ho, zo = fresh(v["h"].dtype) if h_out else None, fresh(bf16) if z else None
    given = {n: padded(t, pad) if pad and t is not None and t.dim() == 2 else t for n, t in v.items()}
    w4.w4_block_norm(given.pop("h"), given.pop("y"), h_out=ho, z=zo, residual_scale=a, branch_scale=b, eps=eps,
                     weight_add=add, **given, **kw)
    torch.cuda.synchronize()
    return ho, zo


DIMS = [8, 128, 504, 512, 520, 1024, 1032, 2048, 2056, 3840, 4096, 4104, 8192, 8200, 16384]


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("T,kind,gate", [(1, bf16, None), (3, f32, "channel"), (37, bf16, "token")])
def test_block_norm(T, D, kind, gate):
    v = norm_case(1, T, D, kind, gate, True, True)
    a, b, add = (1.0, 1.0, 0.0) if T == 1 else (0.75, 0.22, 1.0)
    x, z, ex, ez = norm_bounds(v, a, b, 1e-6, add)
    ho, zo = run_norm(v, a, b, add=add, pad=8 if T == 3 else 0)
    close(ho, x, ex + ROUND[kind] * np.abs(x), "h_out")
    close(zo, z, ez, "z")


@pytest.mark.parametrize("T,D,kind,post,pre,h_out,z,gate", [
    (5, 384, bf16, False, True, True, True, None), (5, 384, f32, True, False, True, True, "channel"),
    (2000, 640, f32, False, False, True, True, "token"), (9, 2304, bf16, True, True, True, False, None),
    (9, 2304, bf16, True, True, False, True, "channel"), (700, 96, bf16, True, True, True, True, None),
])
def test_block_norm_parts(T, D, kind, post, pre, h_out, z, gate):
    """Without one of the norms, without one of the outputs; many rows."""
    v = norm_case(2, T, D, kind, gate, post, pre)
    x, zz, ex, ez = norm_bounds(v, 1.0, 0.5, 1e-5, 0.0)
    got_h, got_z = run_norm(v, 1.0, 0.5, 1e-5, h_out=h_out, z=z)
    if h_out:
        close(got_h, x, ex + ROUND[kind] * np.abs(x), "h_out")
    if z:
        close(got_z, zz, ez, "z")


@pytest.mark.parametrize("kind", [bf16, f32])
@pytest.mark.parametrize("D", [256, 5376])
def test_block_norm_of_the_stream_alone(D, kind):
    """No block's output yet: the first norm of a model."""
    v = dict(h=tensor(3, (6, D), 3.0, kind), y=None, y_weight=None, z_weight=tensor(4, (D,), 0.2, mean=1.0), gate=None)
    _, z, _, ez = norm_bounds(v, 1.0, 1.0, 1e-6, 0.0)
    close(run_norm(v, h_out=False)[1], z, ez, "z")


@pytest.mark.parametrize("kind", [bf16, f32])
@pytest.mark.parametrize("D", [320, 3840])
def test_block_norm_in_place(D, kind):
    v = norm_case(5, 17, D, kind, "channel", True, True)
    want_h, want_z = run_norm(v)
    h, y = padded(v["h"], 16), padded(v["y"], 24)
    w4.w4_block_norm(h, y, h_out=h, z=y, y_weight=v["y_weight"], z_weight=v["z_weight"], gate=v["gate"])
    torch.cuda.synchronize()
    assert torch.equal(h, want_h) and torch.equal(y, want_z)
    for t, wide in ((h, 16), (y, 24)):  # what lies between the rows stays
        assert torch.all(t.as_strided((17, wide), t.stride(), D) == 7.0)


@pytest.mark.parametrize("D", [512, 4096])
@pytest.mark.parametrize("size,eps", [(1e30, 1e-6), (3e37, 0.0), (1e-30, 0.0), (1e-38, 0.0), (1e-30, 1e-6), (2.0 ** -64, 2.0 ** -120)])
def test_block_norm_of_far_values(D, size, eps):
    """Squares that leave FP32: the norms are those of the values all the same."""
    v = norm_case(6, 4, D, bf16, None, True, True)
    v["y"], v["h"] = (v["y"].double() * size).to(bf16), (v["h"].double() * size / 8).to(bf16)
    x, z, ex, ez = norm_bounds(v, 1.0, 1.0, eps, 0.0)
    ho, zo = run_norm(v, eps=eps)
    close(ho, x, ex + ROUND[bf16] * np.abs(x), "h_out")
    close(zo, z, ez, "z")
    v["y"] = torch.zeros_like(v["y"])  # the second norm alone meets them
    x, z, ex, ez = norm_bounds(v, 1.0, 1.0, max(eps, 1e-30), 0.0)
    ho, zo = run_norm(v, eps=max(eps, 1e-30))
    close(ho, x, ex + ROUND[bf16] * np.abs(x), "h_out")
    close(zo, z, ez, "z")


def test_block_norm_rows_of_zeros_infinities_and_nan():
    """Each stays in its row; a row of zeros is 0 with eps and NaN without."""
    v = norm_case(7, 6, 1000, bf16, None, True, True)
    v["y"][1] = 0
    v["h"][1] = 0
    v["y"][2, 77] = float("inf")
    v["h"][3, 5] = float("nan")
    v["h"][4, 999] = float("-inf")
    clean = norm_case(7, 6, 1000, bf16, None, True, True)
    ho, zo = run_norm(v)
    want_h, want_z = run_norm(clean)
    for r in (0, 5):
        assert torch.equal(ho[r], want_h[r]) and torch.equal(zo[r], want_z[r])
    assert torch.all(ho[1] == 0) and torch.all(zo[1] == 0)
    # an infinity in y: its own channel is NaN (inf / inf), the others have nothing of y left
    assert torch.isnan(ho[2, 77]) and torch.equal(ho[2, :77], v["h"][2, :77]) and torch.all(torch.isnan(zo[2]))
    assert torch.isnan(ho[3, 5]) and not torch.isnan(ho[3, 6]) and torch.all(torch.isnan(zo[3]))
    assert ho[4, 999] == float("-inf") and torch.isnan(zo[4, 999]) and torch.all(zo[4, :999] == 0)
    _, zo = run_norm(v, eps=0.0)
    assert torch.all(torch.isnan(zo[1]))


# ---------------------------------------------------------- their gradients
def grad_bounds(v, dho, dz, a, b, eps, add, kind):
    """({gradient: value}, {gradient: bound}); sums over tokens for the weights and a shared gate."""
    h, y, wy, wz, gate = (f64(v[n]) for n in ("h", "y", "y_weight", "z_weight", "gate"))
    dho, dz = f64(dho), f64(dz)
    want = ref.block_norm_grad(h, y, dho, dz, wy, wz, gate, a, b, eps, add)
    x, _, ex, _ = norm_bounds(v, a, b, eps, add)
    a, b, add = (float(np.float32(s)) for s in (a, b, add))
    mean = lambda t: t.mean(-1, keepdims=True)  # noqa: E731
    T = len(h)
    in_f32 = K + max(0, -(-T // 512) - 16) * 2.0 ** -24
    bound = {}
    d = dho if dho is not None else np.zeros_like(x)
    ed = K * np.abs(d)
    dz = np.zeros_like(x) if dz is None else dz
    if wz is None:
        d, ed = d + dz, ed + K * np.abs(dz)
    else:
        r = ref.rms(x, eps)
        n, g = x / r, dz * (wz + add)
        rho = np.sqrt(mean(ex ** 2)) / r + K
        en = ex / r + np.abs(n) * rho
        m, em = mean(g * n), mean(np.abs(g) * en + K * np.abs(g * n))
        t = g - n * m
        ed = ed + (K * np.abs(g) + en * np.abs(m) + np.abs(n) * em + K * np.abs(n * m) + rho * np.abs(t)) / r
        d = d + t / r
        ed = ed + K * np.abs(d)
        bound["d_z_weight"] = (np.abs(dz) * en + in_f32 * np.abs(dz * n)).sum(0)
    if y is None:
        bound["dh"] = ed + ROUND[kind] * np.abs(want["dh"])
        return want, bound
    bound["dh"] = np.abs(a) * ed + ROUND[kind] * np.abs(want["dh"])
    n = y if wy is None else y / ref.rms(y, eps)
    w = np.ones(1) if wy is None else wy + add
    d, ed = b * d, np.abs(b) * ed + K * np.abs(b * d)
    if gate is not None:
        e = np.abs(n * w) * ed + K * np.abs(d * n * w)
        if gate.ndim == 1:
            want["d_gate"] = want["d_gate"].sum(0)
            bound["d_gate"] = (e + in_f32 * np.abs(d * n * w)).sum(0)
        else:
            bound["d_gate"] = e + ROUND[bf16] * np.abs(want["d_gate"])
        d, ed = d * gate, ed * np.abs(gate)
    if wy is None:
        bound["dy"] = ed + K * np.abs(d) + ROUND[bf16] * np.abs(want["dy"])
        return want, bound
    bound["d_y_weight"] = (np.abs(n) * ed + in_f32 * np.abs(d * n)).sum(0)
    g, eg = d * w, np.abs(w) * ed + K * np.abs(d * w)
    m, em = mean(g * n), mean(np.abs(n) * eg + K * np.abs(g * n))
    e = (eg + np.abs(n) * em + 2 * K * np.abs(n * m) + K * np.abs(g) + K * np.abs(g - n * m)) / ref.rms(y, eps)
    bound["dy"] = e + ROUND[bf16] * np.abs(want["dy"])
    return want, bound


def run_grad(v, dho, dz, a=1.0, b=1.0, eps=1e-6, add=0.0, leave=(), **kw):
    T, D = v["h"].shape
    out = {"dh": torch.full_like(v["h"], 7.0)}
    if v["y"] is not None:
        out["dy"] = torch.full((T, D), 7.0, dtype=bf16, device=DEV)
    for n, to in (("y_weight", "d_y_weight"), ("z_weight", "d_z_weight"), ("gate", "d_gate")):
        if v[n] is not None:
            out[to] = torch.full_like(v[n], 7.0) if v[n].dim() == 2 else torch.full((D,), 7.0, dtype=f32, device=DEV)
    for n in leave:
        out.pop(n, None)
    size = w4.w4_block_norm_grad_workspace_bytes(T, D)
    work = torch.full((size // 4,), float("nan"), dtype=f32, device=DEV)
    w4.w4_block_norm_grad(v["h"], v["y"], dh_out=dho, dz=dz, y_weight=v["y_weight"], z_weight=v["z_weight"],
                          gate=v["gate"], residual_scale=a, branch_scale=b, eps=eps, weight_add=add, workspace=work, **out,
                          **kw)
    torch.cuda.synchronize()
    return out


def check_grad(got, want, bound):
    for name, t in got.items():
        close(t, want[name], bound[name], name)


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("T,kind,gate", [(1, bf16, None), (5, f32, "channel"), (37, bf16, "token"), (3, bf16, "channel")])
def test_block_norm_grad(T, D, kind, gate):
    v = norm_case(11, T, D, kind, gate, True, True)
    dho, dz = tensor(12, (T, D), 0.3, kind), tensor(13, (T, D))
    rest = (1.0, 1.0, 1e-6, 0.0) if T == 1 else (0.75, 0.22, 1e-5, 1.0)
    check_grad(run_grad(v, dho, dz, *rest), *grad_bounds(v, dho, dz, *rest, kind))


@pytest.mark.parametrize("T,D,kind,post,pre,gate,dho,dz,leave", [
    (1100, 136, bf16, True, True, "channel", True, True, ()), (700, 2560, f32, True, True, "channel", True, True, ()),
    (9, 384, f32, False, True, "channel", True, True, ()), (9, 384, bf16, True, False, "token", True, True, ()),
    (9, 384, bf16, False, False, None, True, True, ()), (21, 1536, f32, True, True, None, False, True, ()),
    (21, 1536, bf16, True, True, "channel", True, False, ()), (6, 640, bf16, True, True, "channel", True, True, ("dh", "dy")),
    (6, 640, bf16, True, True, "channel", True, True, ("d_y_weight", "d_z_weight", "d_gate")),
    (600, 640, f32, True, True, "token", True, True, ("dh", "d_gate")), (5000, 64, bf16, True, True, "channel", True, True, ()),
])
def test_block_norm_grad_parts(T, D, kind, post, pre, gate, dho, dz, leave):
    """Without one of the norms, of the given gradients, of the asked ones; more rows than runs."""
    v = norm_case(14, T, D, kind, gate, post, pre)
    dho, dz = tensor(15, (T, D), 0.3, kind) if dho else None, tensor(16, (T, D)) if dz else None
    check_grad(run_grad(v, dho, dz, 0.9, 0.5, leave=leave), *grad_bounds(v, dho, dz, 0.9, 0.5, 1e-6, 0.0, kind))


@pytest.mark.parametrize("T,kind,gate", [(4095, f32, "token"), (4096, bf16, "token"), (4099, f32, "channel"), (4099, bf16, None)])
def test_block_norm_grad_of_many_rows(T, kind, gate):
    """On both sides of where two workgroups share a compute unit."""
    v = norm_case(24, T, 2064, kind, gate, True, True)
    dho, dz = tensor(25, (T, 2064), 0.3, kind), tensor(26, (T, 2064))
    check_grad(run_grad(v, dho, dz, 0.9, 0.5), *grad_bounds(v, dho, dz, 0.9, 0.5, 1e-6, 0.0, kind))


@pytest.mark.parametrize("kind", [bf16, f32])
@pytest.mark.parametrize("D", [512, 1024, 2048, 4096, 8192, 16384])
def test_block_norm_grad_of_far_gradients(D, kind):
    """Gradients whose products with y's norm, eight or more of one sign in a lane, pass FP32 where the result does not."""
    v = norm_case(27, 3, D, kind, None, True, True)
    dho = (0.7e38 * torch.sign(v["y"].float()) * torch.tensor([[1.0], [-1.0], [2.0 ** -120]], device=DEV)).to(kind)
    rest = (1.0, 1.0, 1e-6, 0.0)
    check_grad(run_grad(v, dho, None, *rest, leave=("d_y_weight", "d_z_weight")), *grad_bounds(v, dho, None, *rest, kind))


@pytest.mark.parametrize("kind", [bf16, f32])
def test_block_norm_grad_of_the_stream_alone_and_in_place(kind):
    v = dict(h=tensor(17, (20, 896), 3.0, kind), y=None, y_weight=None, z_weight=tensor(18, (896,), 0.2, mean=1.0), gate=None)
    dho, dz = tensor(19, (20, 896), 0.3, kind), tensor(20, (20, 896))
    check_grad(run_grad(v, dho, dz), *grad_bounds(v, dho, dz, 1.0, 1.0, 1e-6, 0.0, kind))
    v = norm_case(21, 20, 896, kind, "channel", True, True)
    want = run_grad(v, dho, dz)
    dh, dy = padded(dho, 8), padded(dz, 16)
    w4.w4_block_norm_grad(v["h"], v["y"], dh_out=dh, dz=dy, dh=dh, dy=dy, y_weight=v["y_weight"], z_weight=v["z_weight"],
                          gate=v["gate"])
    torch.cuda.synchronize()
    assert torch.equal(dh, want["dh"]) and torch.equal(dy, want["dy"])


def test_block_norm_grad_without_rows_sets_the_sums():
    v = norm_case(22, 0, 256, bf16, "channel", True, True)
    got = run_grad(v, torch.zeros_like(v["h"]), None)
    for n in ("d_y_weight", "d_z_weight", "d_gate"):
        assert torch.all(got[n] == 0)


def test_block_norm_grad_against_differences():
    """Of the operator itself, FP32 stream: the loss sum(h_out dh_out) + sum(z dz) along a direction of h."""
    T, D = 64, 256
    v = norm_case(23, T, D, f32, None, True, True)
    dho, dz = tensor(24, (T, D), 0.3, f32), tensor(25, (T, D))
    grad = f64(run_grad(v, dho, dz)["dh"])
    way, step = f64(tensor(26, (T, D), 1.0, f32)), 0.25

    def loss(s):
        x, z = run_norm({**v, "h": (v["h"].double() + s * torch.from_numpy(way).to(DEV)).float()})
        return (f64(x) * f64(dho)).sum() + (f64(z) * f64(dz)).sum()

    got = (loss(step) - loss(-step)) / (2 * step)
    # z's roundings to BF16, 2^-8 |z| each of random sign: 4 sigma of their sum against the gradient's direction
    x, z = ref.block_norm(f64(v["h"]), f64(v["y"]), f64(v["y_weight"]), f64(v["z_weight"]))
    noise = 4 * 2.0 ** -8 * np.sqrt(2 * ((z * f64(dz)) ** 2).sum()) / (2 * step)
    f = lambda s: sum((p * q).sum() for p, q in zip(ref.block_norm(  # noqa: E731
        f64(v["h"]) + s * way, f64(v["y"]), f64(v["y_weight"]), f64(v["z_weight"])), (f64(dho), f64(dz))))
    curved = abs((f(step) - f(-step)) / (2 * step) - (grad * way).sum())  # what the step itself is off by
    assert abs(got - (grad * way).sum()) <= noise + curved


# --------------------------------------------------------------------- sort
def run_sort(ids, E, capacity=0, D=None, R=None, source=True, pad=0):
    T, top = ids.shape
    full = lambda *s: torch.full(s, 77, dtype=torch.int32, device=DEV)  # noqa: E731
    start, row_of, src = full(E + 1), full(T, top), full(T * top) if source else None
    x = rows = None
    if D is not None:
        x = padded(tensor(31, (T, D)), pad) if pad else tensor(31, (T, D))
        rows = torch.full((T * top if R is None else R, D + pad), 7.0, dtype=bf16, device=DEV)[:, :D]
    size = w4.w4_moe_sort_workspace_bytes(T, top, E)
    work = torch.full((size // 4,), 12345, dtype=torch.int32, device=DEV) if size else None
    w4.w4_moe_sort(ints(ids), E, start, row_of, source=src, x=x, rows=rows, capacity=capacity, workspace=work)
    torch.cuda.synchronize()
    return start, row_of, src, x, rows


def check_sort(ids, E, capacity=0, D=None, R=None, **kw):
    start, row_of, src, x, rows = run_sort(ids, E, capacity, D, R, **kw)
    want = ref.moe_sort(ids, E, capacity)
    assert start.tolist() == want[0]
    assert np.array_equal(row_of.cpu().numpy(), want[1])
    if src is not None:
        assert src.tolist() == want[2]
    if D is not None:
        top = ids.shape[1]
        expect = torch.full_like(rows, 7.0)
        live = [(r, i // top) for r, i in enumerate(want[2]) if i >= 0 and r < len(expect)]
        if live:
            r, t = (torch.tensor(c, device=DEV) for c in zip(*live))
            expect[r] = x[t]
        assert torch.equal(rows, expect)


def routed(seed, T, top, E, bad=0.0):
    g = si.rng(92, seed, T, top, E)
    if top <= E:
        ids = np.argsort(g.uniform(size=(T, E)) + 0.3 * g.uniform(size=E), axis=1)[:, :top]
    else:
        ids = g.integers(0, E, (T, top))
    ids = np.where(g.uniform(size=(T, top)) < bad, g.choice([-1, E, 2 ** 31 - 1, -2 ** 31], (T, top)), ids)
    return ids.astype(np.int32)


@pytest.mark.parametrize("T,top,E,capacity,D,bad", [
    (1, 6, 64, 0, 256, 0.0), (1, 1, 1, 0, 8, 0.0), (64, 6, 64, 0, 4096, 0.0), (33, 8, 8, 0, 72, 0.1), (7, 64, 128, 0, 64, 0.0),
    (100, 2, 1024, 0, 128, 0.0), (500, 8, 256, 20, 64, 0.05), (4096, 1, 3, 0, 16, 0.0),          # counted by every workgroup
    (4097, 1, 3, 0, 16, 0.0), (2049, 2, 1, 0, 16, 0.0), (1500, 6, 64, 0, 264, 0.0), (3001, 5, 7, 900, 24, 0.2),
    (700, 64, 1024, 0, 8, 0.0), (9000, 3, 1024, 30, 8, 0.02), (20000, 8, 64, 0, None, 0.0),     # counted in chunks
])
def test_moe_sort(T, top, E, capacity, D, bad):
    check_sort(routed(32, T, top, E, bad), E, capacity, D)


@pytest.mark.parametrize("T", [40, 3000])
def test_moe_sort_extremes(T):
    """All to one expert, all to the last, to none, the same expert twice by a token; a capacity of 1; no sources."""
    for ids in (np.zeros((T, 4)), np.full((T, 4), 63), np.full((T, 4), -1), np.arange(4 * T).reshape(T, 4) % 64):
        for capacity in (0, 1, 70):
            check_sort(ids.astype(np.int32), 64, capacity, 32)
    check_sort(routed(33, T, 4, 64), 64, source=False)


@pytest.mark.parametrize("T,R", [(50, 100), (50, 0), (2000, 3000)])
def test_moe_sort_writes_no_row_past_the_last(T, R):
    check_sort(routed(34, T, 6, 16), 16, 0, 40, R, pad=16)


def test_moe_sort_without_tokens():
    start, row_of, src, *_ = run_sort(np.zeros((0, 6), dtype=np.int32), 10)
    assert start.tolist() == [0] * 11 and row_of.numel() == src.numel() == 0


# ------------------------------------------------------------------ combine
def rows_case(seed, T, top, R, N, bad=0.1):
    g = si.rng(93, seed, T, top, N)
    rows = g.permutation(R)[:T * top].reshape(T, top) if R >= T * top else g.integers(0, R, (T, top))
    rows = np.where(g.uniform(size=(T, top)) < bad, g.choice([-1, R, 2 ** 31 - 1, -2 ** 31], (T, top)), rows).astype(np.int32)
    w = g.uniform(0, 1, (T, top)).astype(np.float32)
    return rows, w


COMBINE = [(1, 6, 6, 4096), (1, 1, 1, 8), (3, 2, 9, 504), (64, 6, 384, 520), (17, 8, 200, 2048), (5, 9, 60, 2056), (2, 64, 128, 4104),
           (300, 4, 1200, 72), (4, 3, 12, 20000)]


@pytest.mark.parametrize("T,top,R,N", COMBINE)
@pytest.mark.parametrize("weighted,added", [(True, True), (False, False), (True, False)])
def test_moe_combine(T, top, R, N, weighted, added):
    rows, w = rows_case(41, T, top, R, N)
    y, add = tensor(42, (R, N)), tensor(43, (T, N)) if added else None
    out = torch.full((T, N + 8), 7.0, dtype=bf16, device=DEV)[:, :N]
    w4.w4_moe_combine(padded(y, 16), out, row_of=ints(rows), weights=torch.from_numpy(w).to(DEV) if weighted else None,
                      add=add)
    torch.cuda.synchronize()
    want, size = ref.combine(f64(y), rows, w if weighted else None, f64(add))
    close(out, want, (top + 1) * 2.0 ** -24 * size + ROUND[bf16] * np.abs(want))
    if added:  # onto add itself
        w4.w4_moe_combine(y, add, row_of=ints(rows), weights=torch.from_numpy(w).to(DEV), add=add)
        torch.cuda.synchronize()
        assert torch.equal(add, out)


def test_moe_combine_of_slots_and_unseen_rows():
    """Without row_of the rows follow the tokens; an infinity or NaN in a row that no choice has stays there."""
    y = tensor(44, (12, 264))
    w = torch.rand(3, 4, device=DEV)
    out, same = (torch.zeros(3, 264, dtype=bf16, device=DEV) for _ in range(2))
    w4.w4_moe_combine(y, out, weights=w)
    w4.w4_moe_combine(y, same, row_of=torch.arange(12, dtype=torch.int32, device=DEV).view(3, 4), weights=w)
    assert torch.equal(out, same)
    w4.w4_moe_combine(y, out)
    w4.w4_moe_combine(y, same, weights=torch.ones_like(w))
    assert torch.equal(out, same)
    bad = y.clone()
    bad[5], bad[6] = float("nan"), float("inf")
    rows = torch.tensor([[0, 1, -1, 2], [3, 4, 7, -1], [8, 9, 10, 11]], dtype=torch.int32, device=DEV)
    w4.w4_moe_combine(y, out, row_of=rows, weights=w)
    w4.w4_moe_combine(bad, same, row_of=rows, weights=w)
    assert torch.equal(out, same)
    none = torch.full((2, 3), -1, dtype=torch.int32, device=DEV)
    got = w4.w4_moe_combine(y[:0], out[:2], row_of=none)
    assert torch.all(got == 0)


@pytest.mark.parametrize("T,top,R,N", [c for c in COMBINE if c[2] >= c[0] * c[1]])
@pytest.mark.parametrize("weighted", [True, False])
def test_moe_combine_grad(T, top, R, N, weighted):
    rows, w = rows_case(45, T, top, R, N)
    y, dout = tensor(46, (R, N)), tensor(47, (T, N))
    dw = torch.full((T, top), 7.0, device=DEV)
    dy = torch.full((R, N + 16), 7.0, dtype=bf16, device=DEV)[:, :N]
    dev_w = torch.from_numpy(w).to(DEV) if weighted else None
    w4.w4_moe_combine_grad(padded(dout, 8), y, row_of=ints(rows), weights=dev_w, dy=dy, dweights=dw)
    torch.cuda.synchronize()
    want_y, want_w, size = ref.combine_grad(f64(dout), f64(y), rows, w if weighted else None)
    left = np.isnan(want_y)
    want_y[left] = 7.0
    close(dy, want_y, (2.0 ** -8 + 2.0 ** -23) * np.abs(want_y) * ~left, "dy")
    close(dw, want_w, (8 * -(-N // 512) + 12) * 2.0 ** -24 * size, "dweights")
    # one of the two alone, and over the rows themselves
    alone_w, alone_y, over = torch.full_like(dw, 7.0), torch.full((R, N), 7.0, dtype=bf16, device=DEV), y.clone()
    w4.w4_moe_combine_grad(dout, y, row_of=ints(rows), weights=dev_w, dweights=alone_w)
    w4.w4_moe_combine_grad(dout, row_of=ints(rows), weights=dev_w, dy=alone_y)
    both = torch.full_like(dw, 7.0)
    w4.w4_moe_combine_grad(dout, over, row_of=ints(rows), weights=dev_w, dy=over, dweights=both)
    torch.cuda.synchronize()
    assert torch.equal(alone_w, dw) and torch.equal(alone_y, dy) and torch.equal(both, dw)
    moved = torch.from_numpy(~left).to(DEV)
    assert torch.equal(over[moved], dy[moved]) and torch.equal(over[~moved], y[~moved])


def test_empty_calls():
    """No tokens, or rows of which none are asked for: nothing is written, nothing is wrong."""
    none, some = torch.zeros(0, 64, dtype=bf16, device=DEV), tensor(50, (6, 64))
    ids = torch.zeros(0, 3, dtype=torch.int32, device=DEV)
    assert w4.w4_moe_combine(none, none) is none
    w4.w4_moe_combine(some, none, row_of=ids)
    w4.w4_moe_combine_grad(none, none, dy=none)
    left = some.clone()
    w4.w4_moe_combine_grad(none, some, row_of=ids, dy=some, dweights=ids.float())
    w4.w4_block_norm(none, none, h_out=none, z=none)
    start, row_of, *_ = run_sort(np.zeros((0, 3), dtype=np.int32), 4)
    assert start.tolist() == [0] * 5
    torch.cuda.synchronize()
    assert torch.equal(some, left)
    with pytest.raises(ValueError):
        w4.w4_moe_combine(some, none)
    with pytest.raises(ValueError):
        w4.w4_moe_combine(some, some[:4])


def test_gradient_of_sorting_and_back_against_the_formula():
    """x -> rows -> (rows as they are) -> out: the gradients of the pair against those of the same sums in 64 bits."""
    T, top, E, N = 29, 4, 12, 136
    ids = routed(48, T, top, E, 0.1)
    start, row_of, _, x, rows = run_sort(ids, E, 9, N)
    w = torch.rand(T, top, device=DEV)
    dout = tensor(49, (T, N))
    drows, dw, dx = torch.zeros_like(rows), torch.zeros_like(w), torch.zeros_like(x)
    w4.w4_moe_combine_grad(dout, rows, row_of=row_of, weights=w, dy=drows, dweights=dw)
    w4.w4_moe_combine(drows, dx, row_of=row_of)
    torch.cuda.synchronize()
    kept = (row_of >= 0).cpu().numpy()
    xd, wd, dd = f64(x), f64(w), f64(dout)
    share = (wd * kept).sum(axis=1, keepdims=True)  # out = x * (the kept weights' sum)
    # drows is rounded (2^-8 of each term), then the sum
    close(dx, share * dd, 2 * 2.0 ** -8 * np.abs(share * dd) + 8 * 2.0 ** -24 * np.abs(share * dd))
    want = kept * (xd * dd).sum(axis=1, keepdims=True)
    close(dw, want, kept * (8 + 12) * 2.0 ** -24 * (np.abs(xd) * np.abs(dd)).sum(axis=1, keepdims=True))


# --------------------------------------------------- streams, graphs, repeats
def layer_calls(seed=51):
    """Closures over static buffers, one for each entry point, and what they write."""
    T, D, E, top = 70, 768, 16, 4
    v = norm_case(seed, T, D, bf16, "channel", True, True)
    dho, dz = tensor(seed + 1, (T, D), 0.3), tensor(seed + 2, (T, D))
    ids, w = ints(routed(seed, T, top, E)), torch.rand(T, top, device=DEV)
    many = ints(routed(seed, 1500, top, E))
    o = {n: torch.zeros(T, D, dtype=bf16, device=DEV) for n in ("h_out", "z", "dh", "dy", "out", "dx")}
    o.update({n: torch.zeros(T * top, D, dtype=bf16, device=DEV) for n in ("rows", "drows")})
    o.update({n: torch.zeros(D, device=DEV) for n in ("d_y_weight", "d_z_weight", "d_gate")})
    o.update(start=torch.zeros(E + 1, dtype=torch.int32, device=DEV), row_of=torch.zeros(T, top, dtype=torch.int32, device=DEV),
             start2=torch.zeros(E + 1, dtype=torch.int32, device=DEV), dweights=torch.zeros(T, top, device=DEV),
             row_of2=torch.zeros(1500, top, dtype=torch.int32, device=DEV))
    work = torch.zeros(w4.w4_block_norm_grad_workspace_bytes(T, D), dtype=torch.uint8, device=DEV)
    work2 = torch.zeros(w4.w4_moe_sort_workspace_bytes(1500, top, E), dtype=torch.uint8, device=DEV)
    ws = {n: v[n] for n in ("y_weight", "z_weight", "gate")}

    def run(stream):
        w4.w4_block_norm(v["h"], v["y"], h_out=o["h_out"], z=o["z"], stream=stream, **ws)
        w4.w4_moe_sort(ids, E, o["start"], o["row_of"], x=o["z"], rows=o["rows"], stream=stream)
        w4.w4_moe_sort(many, E, o["start2"], o["row_of2"], workspace=work2, stream=stream)
        w4.w4_moe_combine(o["rows"], o["out"], row_of=o["row_of"], weights=w, add=o["h_out"], stream=stream)
        w4.w4_moe_combine_grad(o["out"], o["rows"], row_of=o["row_of"], weights=w, dy=o["drows"], dweights=o["dweights"],
                               stream=stream)
        w4.w4_moe_combine(o["drows"], o["dx"], row_of=o["row_of"], stream=stream)
        w4.w4_block_norm_grad(v["h"], v["y"], dh_out=dho, dz=o["dx"], dh=o["dh"], dy=o["dy"], workspace=work, stream=stream,
                              d_y_weight=o["d_y_weight"], d_z_weight=o["d_z_weight"], d_gate=o["d_gate"], **ws)

    return v, ids, w, o, run


def test_block_graph_replays():
    """All of them in one graph, replayed four times with eager work between, inputs changed in place."""
    v, ids, w, o, run = layer_calls()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    w4.w4_graph_begin(stream)
    try:
        run(stream)
    finally:
        graph = w4.w4_graph_end(stream)
    for k in range(4):
        v["y"].copy_(tensor(60 + k, tuple(v["y"].shape)))
        ids.copy_(ints(routed(60 + k, 70, 4, 16, 0.1)))
        for t in o.values():
            t.fill_(3)
        torch.cuda.synchronize()
        graph.replay(stream)
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in o.items()}
        for t in o.values():
            t.fill_(3)
        torch.cuda.synchronize()
        run(stream)
        torch.cuda.synchronize()
        for n, t in o.items():
            assert torch.equal(got[n], t), n
    graph.destroy()


def test_block_calls_repeat_their_bits_on_another_stream():
    _, _, _, o, run = layer_calls(71)
    run(None)
    torch.cuda.synchronize()
    first = {n: t.clone() for n, t in o.items()}
    for t in o.values():
        t.fill_(5)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    run(other)
    other.synchronize()
    for n, t in o.items():
        if n == "drows" or n == "rows":  # rows behind the last are left: here every choice has one
            assert torch.equal(first[n], t)
        assert torch.equal(first[n], t), n


def test_the_most_tokens_of_one_call():
    """As many tokens as a call takes: a workgroup each must not pass what a launch counts."""
    T, N = 1 << 23, 2056
    dout = torch.empty(T, N, dtype=bf16, device=DEV)
    some = [0, (1 << 22) + 1, T - 1]
    values = tensor(60, (3, N))
    dout[some] = values
    y, row_of = tensor(61, (4, N)), torch.full((T, 1), -1, dtype=torch.int32, device=DEV)
    row_of[some, 0] = ints([2, 0, 3])
    dy, dw = torch.full_like(y, 7.0), torch.full((T, 1), 7.0, device=DEV)
    w4.w4_moe_combine_grad(dout, y, row_of=row_of, dy=dy, dweights=dw)
    torch.cuda.synchronize()
    assert torch.equal(dy[[2, 0, 3]], values) and torch.all(dy[1] == 7.0)
    want, size = (f64(values) * f64(y[[2, 0, 3]])).sum(1), np.abs(f64(values) * f64(y[[2, 0, 3]])).sum(1)
    close(dw[some, 0], want, (8 * -(-N // 256) + 12) * 2.0 ** -24 * size, "dweights")
    assert int((dw != 0).sum()) == 3
    del dout
    out = torch.full((T, 8), 7.0, dtype=bf16, device=DEV)
    w4.w4_moe_combine(y[:, :8], out, row_of=row_of)
    torch.cuda.synchronize()
    assert torch.equal(out[some], y[[2, 0, 3], :8]) and int((out != 0).any(1).sum()) == 3
    experts = torch.arange(T, dtype=torch.int32, device=DEV).remainder_(1000).view(T, 1)
    start, rows = torch.zeros(1025, dtype=torch.int32, device=DEV), torch.zeros(T, 1, dtype=torch.int32, device=DEV)
    work = torch.empty(w4.w4_moe_sort_workspace_bytes(T, 1, 1024), dtype=torch.uint8, device=DEV)
    w4.w4_moe_sort(experts, 1024, start, rows, workspace=work)
    torch.cuda.synchronize()
    sizes = [T // 1000 + (e < T % 1000) for e in range(1000)] + [0] * 24
    assert start.tolist() == [0, *np.cumsum(sizes).tolist()]
    at = torch.arange(T, device=DEV)
    assert torch.equal(rows[:, 0].long(), start[:1000].long()[at % 1000] + at // 1000)


def test_graphs_that_share_a_workspace():
    """Calls of several launches: three graphs over one workspace, replayed in turn with eager calls between."""
    v = norm_case(70, 4096, 2056, bf16, "channel", True, True)
    dz = tensor(71, (4096, 2056))
    grads = {n: torch.zeros(2056, device=DEV) for n in ("d_y_weight", "d_z_weight", "d_gate")}
    grads["dy"] = torch.zeros_like(v["y"])
    few, many = ints(routed(72, 3000, 6, 16, 0.1)), ints(routed(73, 3000, 8, 256, 0.1))
    x = tensor(74, (3000, 64))
    out = [(torch.zeros(E + 1, dtype=torch.int32, device=DEV), torch.zeros_like(ids), torch.zeros(ids.numel(), 64, dtype=bf16, device=DEV))
           for E, ids in ((16, few), (256, many))]
    sizes = [w4.w4_block_norm_grad_workspace_bytes(4096, 2056), w4.w4_moe_sort_workspace_bytes(3000, 6, 16),
             w4.w4_moe_sort_workspace_bytes(3000, 8, 256)]
    assert all(sizes)
    work = torch.full((max(sizes),), 0xAB, dtype=torch.uint8, device=DEV)
    calls = [lambda s: w4.w4_block_norm_grad(**v, dz=dz, workspace=work, stream=s, **grads)]
    for (start, row_of, rows), E, ids in ((out[0], 16, few), (out[1], 256, many)):
        calls.append(lambda s, start=start, row_of=row_of, rows=rows, E=E, ids=ids:
                     w4.w4_moe_sort(ids, E, start, row_of, x=x, rows=rows, capacity=500, workspace=work, stream=s))
    results = [list(grads.values()), list(out[0]), list(out[1])]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = []
    for call in calls:
        w4.w4_graph_begin(stream)
        try:
            call(stream)
        finally:
            graphs.append(w4.w4_graph_end(stream))
    for k in range(3):
        v["y"].copy_(tensor(75 + k, tuple(v["y"].shape)))
        few.copy_(ints(routed(75 + k, 3000, 6, 16, 0.1)))
        many.copy_(ints(routed(78 + k, 3000, 8, 256, 0.1)))
        got = []
        for graph, tensors in zip(graphs, results):
            for t in tensors:
                t.fill_(3)
            torch.cuda.synchronize()
            graph.replay(stream)
        torch.cuda.synchronize()
        got = [[t.clone() for t in tensors] for tensors in results]
        work.fill_(0xCD)
        for call, tensors in zip(calls, results):
            for t in tensors:
                t.fill_(3)
            torch.cuda.synchronize()
            call(stream)
        torch.cuda.synchronize()
        for first, tensors in zip(got, results):
            for a, b in zip(first, tensors):
                assert torch.equal(a, b)
        want = ref.moe_sort(many.cpu().numpy(), 256, 500)
        assert out[1][0].tolist() == list(want[0]) and np.array_equal(out[1][1].cpu().numpy(), want[1])
    for graph in graphs:
        graph.destroy()


# ------------------------------------------------- rows past the caches' keeping
# From 2^22 values of all choices on (block.hpp) rows go past the caches: kernels of their own.
@pytest.mark.parametrize("T,top,E,capacity,D,R,bad", [
    (1100, 6, 64, 0, 1024, None, 0.0), (1100, 6, 64, 90, 1024, 5000, 0.1), (600, 6, 16, 0, 1200, None, 0.05),  # by every workgroup
    (200, 64, 256, 0, 336, 12000, 0.0), (9000, 8, 512, 130, 64, None, 0.02),  # a table summed once
])
def test_moe_sort_of_many_values(T, top, E, capacity, D, R, bad):
    assert T * top * D >= 1 << 22
    check_sort(routed(81, T, top, E, bad), E, capacity, D, R, pad=8)


MANY_VALUES = [(1100, 8, 8900, 512), (950, 9, 8600, 504), (700, 6, 4200, 1024), (350, 6, 2200, 2048), (100, 12, 1300, 4104), (30, 64, 1920, 2304)]


@pytest.mark.parametrize("T,top,R,N", MANY_VALUES)
@pytest.mark.parametrize("weighted,added", [(True, True), (False, False)])
def test_moe_combine_of_many_values(T, top, R, N, weighted, added):
    assert T * top * N >= 1 << 22
    test_moe_combine(T, top, R, N, weighted, added)


@pytest.mark.parametrize("T,top,R,N", MANY_VALUES)
def test_moe_combine_grad_of_many_values(T, top, R, N):
    assert T * top * N >= 1 << 22
    test_moe_combine_grad(T, top, R, N, True)


@pytest.mark.parametrize("kind", [bf16, f32])
@pytest.mark.parametrize("D", [64, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 12288, 12296, 16384])
def test_block_norm_of_many_values(D, kind):
    """From 2^19 values on both outputs go past the caches; over their inputs too."""
    T = (1 << 19) // D + 3
    v = norm_case(82, T, D, kind, "token" if D % 16 else "channel", True, True)
    x, z, ex, ez = norm_bounds(v, 0.75, 0.22, 1e-6, 1.0)
    ho, zo = run_norm(v, 0.75, 0.22, add=1.0)
    close(ho, x, ex + ROUND[kind] * np.abs(x), "h_out")
    close(zo, z, ez, "z")
    w4.w4_block_norm(v["h"], v["y"], h_out=v["h"], z=v["y"], y_weight=v["y_weight"], z_weight=v["z_weight"], gate=v["gate"],
                     residual_scale=0.75, branch_scale=0.22, weight_add=1.0)
    torch.cuda.synchronize()
    assert torch.equal(v["h"], ho) and torch.equal(v["y"], zo)


@pytest.mark.parametrize("T,D,kind,teams", [(1 << 21, 8, bf16, 8), (150000, 136, f32, 8), (30000, 520, bf16, 4), (20000, 1032, f32, 2),
                                            (10000, 2056, f32, 1), (10000, 2056, bf16, 1)])
def test_block_norm_grad_sums_over_long_runs(T, D, kind, teams):
    """Sums over t of many rows.  A run is at most ceil(T / 256) of them, in turn over its teams: a lane's FP32 sum
    takes that part of them one after the other, each off by 2^-24 of the magnitudes so far, the teams' join three more
    roundings, which K has room for; FP64 joins the runs.  The terms are off as in ``grad_bounds``."""
    v = norm_case(83, T, D, kind, None, True, True)
    dho, dz = tensor(84, (T, D), 0.3, kind), tensor(85, (T, D))
    got = run_grad(v, dho, dz, 0.9, 0.5)
    want, bound = grad_bounds(v, dho, dz, 0.9, 0.5, 1e-6, 0.0, kind)
    h, y, wz = (f64(v[n]) for n in ("h", "y", "z_weight"))
    x, _ = ref.block_norm(h, y, f64(v["y_weight"]), wz, None, 0.9, 0.5, 1e-6, 0.0)
    r, n1 = ref.rms(x, 1e-6), y / ref.rms(y, 1e-6)
    n2, g = x / r, f64(dz) * wz
    dx = f64(dho) + (g - n2 * (g * n2).mean(-1, keepdims=True)) / r
    more = -(-(-(-T // 256)) // teams) * 2.0 ** -24
    bound["d_z_weight"] = bound["d_z_weight"] + more * np.abs(f64(dz) * n2).sum(0)
    bound["d_y_weight"] = bound["d_y_weight"] + more * np.abs(0.5 * dx * n1).sum(0)
    check_grad(got, want, bound)


# ------------------------------------------------------------ rows far apart
def far_rows(t):
    """The same rows 2^31 + 8 values apart: offsets past 32 bits from the third on, bytes from the second."""
    step = (1 << 31) + 8
    space = torch.empty((len(t) - 1) * step + t.shape[1], dtype=t.dtype, device=DEV)
    out = torch.as_strided(space, t.shape, (step, 1))
    out.copy_(t)
    return out


@pytest.mark.parametrize("kind", [bf16, f32])
def test_rows_far_apart(kind):
    """Each operator on rows whose offsets pass 32 bits: the bits of rows that lie together."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("less than 160 GiB of memory is free")
    T, D = 3, 520
    v = norm_case(86, T, D, kind, "token", True, True)
    want = run_norm(v)
    f = {n: far_rows(t) if t.dim() == 2 else t for n, t in v.items()}
    ho, z = far_rows(torch.full_like(v["h"], 7.0)), far_rows(torch.full_like(v["y"], 7.0))
    w4.w4_block_norm(f["h"], f["y"], h_out=ho, z=z, y_weight=v["y_weight"], z_weight=v["z_weight"], gate=f["gate"])
    assert torch.equal(ho, want[0]) and torch.equal(z, want[1])
    dho, dz = tensor(87, (T, D), 0.3, kind), tensor(88, (T, D))
    want = run_grad(v, dho, dz)
    ho.copy_(dho)
    z.copy_(dz)
    dgate = far_rows(torch.full_like(v["gate"], 7.0))
    w4.w4_block_norm_grad(f["h"], f["y"], dh_out=ho, dz=z, dh=ho, dy=z, y_weight=v["y_weight"], z_weight=v["z_weight"],
                          gate=f["gate"], d_gate=dgate)
    assert torch.equal(ho, want["dh"]) and torch.equal(z, want["dy"]) and torch.equal(dgate, want["d_gate"])
    del f, ho, dgate
    if kind is f32:
        return
    ids = ints([[1, 0], [1, 1], [0, 2]])
    start, row_of = torch.zeros(4, dtype=torch.int32, device=DEV), torch.zeros(T, 2, dtype=torch.int32, device=DEV)
    x = tensor(89, (T, D))
    z.copy_(x)
    rows = far_rows(torch.full((6, D), 7.0, dtype=bf16, device=DEV))
    w4.w4_moe_sort(ids, 3, start, row_of, x=z, rows=rows)
    assert row_of.tolist() == [[2, 0], [3, 4], [1, 5]]
    assert torch.equal(rows, x[[0, 2, 0, 1, 1, 2]])
    w, out = torch.rand(T, 2, device=DEV), torch.zeros(T, D, dtype=bf16, device=DEV)
    w4.w4_moe_combine(x[[0, 2, 0, 1, 1, 2]], out, row_of=row_of, weights=w, add=x)
    w4.w4_moe_combine(rows, z, row_of=row_of, weights=w, add=z)
    assert torch.equal(z, out)
    dy, dw = torch.zeros(6, D, dtype=bf16, device=DEV), torch.zeros_like(w)
    w4.w4_moe_combine_grad(out, x[[0, 2, 0, 1, 1, 2]], row_of=row_of, weights=w, dy=dy, dweights=dw)
    far_w = torch.zeros_like(w)
    w4.w4_moe_combine_grad(z, rows, row_of=row_of, weights=w, dy=rows, dweights=far_w)
    torch.cuda.synchronize()
    assert torch.equal(rows, dy) and torch.equal(far_w, dw)
