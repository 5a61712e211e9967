"""The norm of whole tokens with the residual's addition on the GPU against its
definition in float64.

Tolerances.  A norm's sum of up to 16384 squares is taken by lanes (at most 32 in
a row) and steps across them: 2^-18 of it, so y is off by 2^-18 of its value and
half a step u of the storage type; the sum by u and 2^-24.  8-bit values are off by
half a step: 2^-4 of the value in e4m3, or 2^-10 of the scale below its normal range,
half a scale in int8; and by what y and the scale are off, 2^-16 of the value.  dx is
2^-17 of the sum of absolute values of its terms, dweight 2^-17 of its own.
"""
import numpy as np
import pytest

import ends_ref
from gpu_util import say
from long_convolution_sequence_rfft_amd import hyena
from test_gpu_recurrence import IO, f64, torch_dtype

pytestmark = pytest.mark.gpu

CASES = [
    # B, N, d
    (1, 1, 1), (1, 1, 768), (2, 3, 64), (3, 37, 100), (1, 5, 33), (2, 50, 24), (1, 200, 770), (2, 9, 2048),
    (1, 3, 2056), (1, 4, 5003), (1, 2, 16384), (1, 2, 16383), (1, 3, 8200), (4, 700, 128), (1, 3000, 768),
]


def close(got, ref, size, dtype, what):
    err = np.abs(f64(got) - ref)
    bound = ends_ref.HALF_STEP[dtype] * np.abs(ref) + size + ends_ref.TINY[dtype]
    say(f"[gpu]   {what}: worst error / bound {float(np.max(err / bound)):.3f}")
    assert np.all(err <= bound), what


def make(case, dtype, seed, strided=False):
    import torch
    B, N, d = case
    gen = torch.Generator().manual_seed(seed)
    dt = torch_dtype(dtype)
    if strided:
        wide = torch.randn((N + 2, B, d + 3), generator=gen).to(dt).cuda()
        x = wide[1:N + 1, :, 1:d + 1].transpose(0, 1)
        res = torch.randn((B, N + 1, d + 1), generator=gen).to(dt).cuda()[:, :N, :d]
        dy = torch.randn((1, N, d), generator=gen).to(dt).cuda().expand(B, N, d)
        ds = torch.randn((B, N, 2 * d), generator=gen).to(dt).cuda()[..., d:]
    else:
        x, res, dy, ds = (torch.randn((B, N, d), generator=gen).to(dt).cuda() for _ in range(4))
    return x, res, dy, ds, (1 + 0.2 * torch.randn(d, generator=gen)).cuda()


def run(case, dtype, seed=1, strided=False, residual=True, weight=True, eps=1e-6):
    say(f"[gpu] residual_norm {case} {dtype} strided={strided} residual={residual} weight={weight}")
    x, res, dy, ds, w = make(case, dtype, seed, strided)
    if not residual:
        res = ds = None
    if not weight:
        w = None
    plan = hyena.ResidualNorm(*case, io_dtype=IO[dtype], eps=eps)
    y, total = plan.forward(x, res, w)
    wd = np.ones(case[2]) if w is None else f64(w)
    eps = float(np.float32(eps))
    ref, s = ends_ref.residual_norm(f64(x), None if res is None else f64(res), wd, eps)
    close(y, ref, 2.0 ** -18 * np.abs(ref), dtype, "y")
    if residual:
        close(total, s, 2.0 ** -24 * np.abs(s), dtype, "total")
    else:
        assert total is None
        total = x
    dx, dw = plan.backward(dy, total, w, ds=ds)
    rx, rw, ax, aw = ends_ref.residual_norm_grad(f64(dy), f64(total), wd, None if ds is None else f64(ds), eps)
    close(dx, rx, 2.0 ** -17 * ax, dtype, "dx")
    if weight:
        close(dw, rw, 2.0 ** -17 * aw, "f32", "dweight")
    else:
        assert dw is None


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", CASES)
def test_against_float64(case, dtype):
    run(case, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [CASES[3], CASES[4], CASES[6], CASES[8], CASES[13]])
def test_strided_views_and_broadcast_gradients(case, dtype):
    run(case, dtype, strided=True)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_without_residual_or_weight(dtype):
    run(CASES[3], dtype, residual=False)
    run(CASES[3], dtype, weight=False)
    run(CASES[9], dtype, residual=False, weight=False, eps=0.0)


EIGHT = [
    # B, N, d, group
    (1, 1, 768, None), (3, 7, 768, 128), (2, 5, 96, 32), (2, 33, 64, 64), (1, 4, 100, None), (1, 3, 77, None),
    (2, 3, 2176, 128), (1, 2, 16384, 32), (1, 2, 16384, None), (1, 40, 4096, 64), (1, 3, 160, 32), (5, 3, 5003, None),
]


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", EIGHT)
def test_eight_bits(case, dtype, kind):
    check_eight(case, dtype, kind)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("case", [EIGHT[1], EIGHT[2], EIGHT[5], EIGHT[6], EIGHT[10]])
def test_eight_bits_of_strided_views(case, kind):
    check_eight(case, "bf16", kind, strided=True)
    check_eight(case, "f32", kind, strided=True)


def check_eight(case, dtype, kind, strided=False):
    B, N, d, group = case
    say(f"[gpu] residual_norm in 8 bits {case} {dtype} {kind} strided={strided}")
    x, res, _, _, w = make((B, N, d), dtype, 2, strided)
    plan = hyena.ResidualNorm(B, N, d, io_dtype=IO[dtype], quantized=kind, group=group)
    y8, scales, total = plan.forward(x, res, w)
    ref, s = ends_ref.residual_norm(f64(x), f64(res), f64(w), float(np.float32(1e-6)))
    close(total, s, 2.0 ** -24 * np.abs(s), dtype, "total")
    g = group or d
    want = np.abs(ref.reshape(B, N, d // g, g)).max(-1) / ends_ref.LARGEST[kind]
    assert scales.shape == want.shape
    close(scales, want, 2.0 ** -17 * want, "f32", "scales")
    a = np.repeat(f64(scales), g, -1)
    got = y8.float().cpu().numpy().astype(np.float64) * a
    if kind == "e4m3":
        bound = (2.0 ** -4 + 2.0 ** -15) * np.abs(ref) + 2.0 ** -10 * a
    else:
        bound = 0.5 * a + 2.0 ** -16 * np.abs(ref)
    say(f"[gpu]   values: worst error / bound {float(np.max(np.abs(got - ref) / bound)):.3f}")
    assert np.all(np.abs(got - ref) <= bound)
    # the largest of a group is the type's largest
    assert np.all(np.abs(y8.float().cpu().numpy()).reshape(B, N, d // g, g).max(-1) == ends_ref.LARGEST[kind])


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_eight_bits_of_zeros_tiny_and_bad_rows(kind):
    import torch
    x = torch.randn((1, 6, 64), device="cuda")
    x[0, 1] = 0.0
    x[0, 2] = 1e-38
    x[0, 3, 40] = float("nan")
    w = torch.ones(64, device="cuda")
    plan = hyena.ResidualNorm(1, 6, 64, eps=1.0, quantized=kind, group=32)
    y8, scales, _ = plan.forward(x, None, w)
    values = y8.float()
    assert not values[0, 1:3].any() and not scales[0, 1:3].any()
    assert torch.isnan(scales[0, 3]).all()                     # the norm of the whole row is NaN
    good = [0, 4, 5]
    ref, _ = ends_ref.residual_norm(f64(x)[:, good], None, 1.0, 1.0)
    got = (values * scales.repeat_interleave(32, -1)).cpu().numpy()[:, good]
    assert np.abs(got - ref).max() <= 0.04 * np.abs(ref).max()


def test_the_sum_in_place():
    import torch
    x, res, dy, ds, w = make((2, 30, 96), "bf16", 4)
    plan = hyena.ResidualNorm(2, 30, 96, io_dtype=hyena.HYENA_BF16)
    y, total = plan.forward(x, res, w)
    for at in (0, 1):
        pair = [x.clone(), res.clone()]
        y2, t2 = plan.forward(*pair, w, total=pair[at])
        assert t2 is pair[at] and torch.equal(t2, total) and torch.equal(y2, y)
        assert torch.equal(pair[1 - at], (x, res)[1 - at])
    dx, dw = plan.backward(dy, total, w, ds=ds)
    kept = ds.clone()
    dx2, dw2 = plan.backward(dy, total, w, ds=kept, dx=kept)
    assert dx2 is kept and torch.equal(dx2, dx) and torch.equal(dw2, dw)
    with pytest.raises(hyena.HyenaError, match="overlaps"):
        plan.forward(x, res, w, y=x)
    with pytest.raises(hyena.HyenaError, match="overlaps"):
        plan.backward(dy, total, w, ds=ds, dx=dy)


def test_gradient_against_differences():
    import torch
    gen = torch.Generator().manual_seed(9)
    x, w, dy = torch.randn((1, 2, 20), generator=gen), torch.randn(20, generator=gen), torch.randn((1, 2, 20), generator=gen)
    plan = hyena.ResidualNorm(1, 2, 20)
    dx, dw = (f64(t) for t in plan.backward(dy.cuda(), x.cuda(), w.cuda()))
    f = lambda x, w: (f64(dy) * ends_ref.residual_norm(x, None, w, 1e-6)[0]).sum()  # noqa: E731
    h, xd, wd = 1e-5, f64(x), f64(w)
    for i in np.ndindex(1, 2, 20):
        e = np.zeros_like(xd)
        e[i] = h
        assert abs((f(xd + e, wd) - f(xd - e, wd)) / (2 * h) - dx[i]) < 1e-5
    for i in range(20):
        e = np.zeros(20)
        e[i] = h
        assert abs((f(xd, wd + e) - f(xd, wd - e)) / (2 * h) - dw[i]) < 1e-5


def test_another_stream_and_a_replayed_graph():
    import torch
    x, res, dy, ds, w = make((2, 500, 256), "bf16", 6)
    plan = hyena.ResidualNorm(2, 500, 256, io_dtype=hyena.HYENA_BF16)
    y, total = plan.forward(x, res, w)
    dx, dw = plan.backward(dy, total, w, ds=ds)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2, t2 = plan.forward(x, res, w)
        dx2, dw2 = plan.backward(dy, t2, w, ds=ds)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, t2 = plan.forward(x, res, w)
        dx2, dw2 = plan.backward(dy, t2, w, ds=ds)
    for _ in range(4):
        x.normal_()
        dy.normal_()
        graph.replay()
        torch.cuda.synchronize()
        y, total = plan.forward(x, res, w)
        dx, dw = plan.backward(dy, total, w, ds=ds)
        assert torch.equal(y, y2) and torch.equal(total, t2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)
