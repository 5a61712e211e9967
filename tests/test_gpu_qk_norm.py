"""Norms of queries and keys with the position rotation on the GPU against
their definition in float64.

Tolerances.  Every output is a few float32 operations on values of the size of
its pair's norm: 2^-20 of it (norm: a sum of up to 1024 squares by lanes and
shuffles, square root and reciprocal; sine and cosine: 2 units; the rotation:
3 roundings), plus half a step of the storage type.  Gradients of the weights
are sums of float32 terms of relative error 2^-20, in float32 within a
workgroup: 2^-17 of the sum of absolute values.
"""
import numpy as np
import pytest

import mixer_ref
from gpu_util import say
from long_convolution_sequence_rfft_amd import hyena
from test_gpu_recurrence import IO, f64, torch_dtype

pytestmark = pytest.mark.gpu

SMALL = 2.0 ** -20

CASES = [
    # B, N, q_heads, k_heads, D, rotary, norm, layout
    (1, 1, 1, 1, 64, 64, "rms", "half"), (2, 3, 12, 12, 64, 64, "rms", "half"),
    (2, 37, 6, 2, 64, 32, "l2", "interleaved"), (1, 100, 3, 1, 128, 128, "rms", "interleaved"),
    (1, 9, 2, 2, 80, 48, "rms", "half"), (2, 5, 3, 3, 20, 12, "l2", "half"), (1, 11, 2, 1, 7, 4, "rms", "interleaved"),
    (1, 6, 1, 2, 33, 32, "rms", "half"), (1, 4, 2, 2, 256, 64, "none", "half"), (1, 3, 1, 1, 1024, 1024, "rms", "half"),
    (1, 3, 1, 1, 1000, 10, "rms", "interleaved"), (1, 2, 1, 1, 1023, 1022, "l2", "half"), (1, 4, 2, 1, 1, 0, "rms", "half"),
    (3, 50, 2, 2, 24, 0, "rms", "half"), (1, 40, 5, 5, 16, 16, "none", "interleaved"),
    (1, 2500, 4, 1, 64, 64, "rms", "half"),
    (2, 7, 3, 2, 100, 100, "rms", "half"), (1, 5, 2, 2, 66, 64, "l2", "interleaved"), (1, 3, 1, 1, 1022, 1020, "rms", "half"),
    (1, 3, 2, 1, 514, 4, "rms", "interleaved"), (4, 2000, 4, 4, 128, 128, "rms", "half"),
]


def make(case, dtype, seed, sliced=False):
    import torch
    B, N, hq, hk, D, r, norm, layout = case
    gen = torch.Generator().manual_seed(seed)
    dt = torch_dtype(dtype)
    if sliced:
        full = torch.randn((B, N, hq + 2 * hk, D + 1), generator=gen).to(dt).cuda()
        q, k = full[:, :, :hq, 1:], full[:, :, hq:hq + hk, :D]
        dq = torch.randn((hq, B, N, D), generator=gen).to(dt).cuda().permute(1, 2, 0, 3)
        dk = torch.randn((B, 1, hk, D), generator=gen).to(dt).cuda().expand(B, N, hk, D)
    else:
        q, k, dq, dk = (torch.randn((B, N, h, D), generator=gen).to(dt).cuda() for h in (hq, hk, hq, hk))
    wq, wk = (1 + 0.2 * torch.randn(D, generator=gen).cuda() for _ in range(2))
    return q, k, dq, dk, wq, wk


def run(case, dtype, seed=1, sliced=False, positions=None, offset=0, weights=True, stretch=1.0, rscale=1.0):
    import torch
    say(f"[gpu] qk_norm {case} {dtype} sliced={sliced} positions={positions} offset={offset}")
    B, N, hq, hk, D, r, norm, layout = case
    q, k, dq, dk, wq, wk = make(case, dtype, seed, sliced)
    if not weights:
        wq = wk = None
    freqs = hyena.rotary_frequencies(r, stretch=stretch)
    pos = offset + np.arange(N)[None] + np.zeros((B, 1))
    at = None
    if positions is not None:
        pos = np.random.default_rng(seed).integers(*positions, (B, N)).astype(np.float64)
        at = torch.from_numpy(pos.astype(np.int32)).cuda()
    plan = hyena.QKNorm(B, N, hq, hk, D, io_dtype=IO[dtype], norm=norm, rotary_dim=r, layout=layout, freqs=freqs,
                        rotary_scale=rscale)
    args = (f64(freqs), norm, layout, r, 1e-6, rscale)
    u = mixer_ref.HALF_STEP[dtype]

    def close(got, ref, size, what, small=SMALL, step=u):
        err = np.abs(f64(got) - ref)
        bound = step * np.abs(ref) + small * size + 1e-30
        say(f"[gpu]   {what}: worst error / bound {float(np.max(err / bound)):.3f}")
        assert np.all(err <= bound), what

    def size(x, extra=0.0):  # a value's own size and its head's
        return np.abs(x).max(-1, keepdims=True) + extra

    qo, ko = plan.forward(q, k, wq, wk, positions=at, offset=offset)
    for got, x, w, what in ((qo, q, wq, "q"), (ko, k, wk, "k")):
        ref = mixer_ref.qk_norm(f64(x), None if w is None else f64(w), pos, *args)
        close(got, ref, size(ref), what)
    gq, gk, gwq, gwk = plan.backward(dq, dk, q, k, wq, wk, positions=at, offset=offset)
    for got, gw, dy, x, w, what in ((gq, gwq, dq, q, wq, "dq"), (gk, gwk, dk, k, wk, "dk")):
        dx, dw, aw = mixer_ref.qk_norm_grad(f64(dy), f64(x), None if w is None else f64(w), pos, *args)
        # the projection along x is subtracted: its terms are of the size of |dn w| / norm
        n = mixer_ref._norm(f64(x), norm, 1e-6)
        wmax = 1.0 if w is None else float(w.abs().max())
        m = D if norm == "rms" else 1
        along = (np.abs(f64(x)) * size(f64(dy))).sum(-1, keepdims=True) * np.abs(f64(x)) / (m * n * n) if norm != "none" else 0
        close(got, dx, 2 * wmax * abs(rscale) * (size(f64(dy)) + along) / n, what)
        if w is None or norm == "none":
            assert gw is None
        else:
            # a value's error is relative to its pair's size
            pair = (size(f64(dy)) * np.abs(f64(x)) / n).sum((0, 1, 2))
            close(gw, dw, aw + 2 * abs(rscale) * pair, what + "_weight", small=2.0 ** -17, step=2.0 ** -24)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", CASES)
def test_against_float64(case, dtype):
    run(case, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [CASES[2], CASES[4], CASES[6], CASES[12]])
def test_strided_views_and_broadcast_gradients(case, dtype):
    run(case, dtype, sliced=True)


@pytest.mark.parametrize("case", [CASES[1], CASES[2], CASES[6]])
def test_far_and_negative_positions(case):
    run(case, "f32", positions=(-1000, 1000))
    run(case, "f32", positions=(2 ** 31 - 5000, 2 ** 31 - 1))
    run(case, "f32", offset=(1 << 33) + 12345, stretch=32.0, rscale=1.3)


def test_without_weights():
    run(CASES[1], "f32", weights=False)
    run(CASES[2], "bf16", weights=False)


def test_zero_rows_have_finite_results():
    import torch
    plan = hyena.QKNorm(1, 2, 1, 1, 64)
    z = torch.zeros((1, 2, 1, 64), device="cuda")
    q, k = plan.forward(z, z)
    assert not q.any() and not k.any()
    d = torch.ones_like(z)
    w = torch.ones(64, device="cuda")
    dq, dk, dwq, dwk = plan.backward(d, d, z, z, w, w)
    assert torch.isfinite(dq).all() and not dwq.any() and not dwk.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_in_a_replayed_graph(dtype):
    import torch
    case = (2, 300, 4, 2, 64, 64, "rms", "half")
    q, k, dq, dk, wq, wk = make(case, dtype, 4)
    plan = hyena.QKNorm(2, 300, 4, 2, 64, io_dtype=IO[dtype])
    both = lambda: [*plan.forward(q, k, wq, wk), *plan.backward(dq, dk, q, k, wq, wk)]  # noqa: E731
    want = [t.clone() for t in both()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for _ in range(3):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(both(), want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_rotation_and_recurrence_as_a_mixer(dtype):
    """Training and decoding of a mixer: q, k, v from one projection, the norm with its rotation, the
    recurrence; gradients back through both against float64 differences of the whole, then one decoded
    token from the state with its own position against the longer sequence's last output."""
    import torch
    B, N, H, D = 2, 75, 3, 32
    gen = torch.Generator().manual_seed(8)
    dt = torch_dtype(dtype)
    qkv = torch.randn((B, N + 1, 3 * H, D), generator=gen).to(dt).cuda()
    g = -0.2 * torch.rand((B, N + 1, H), generator=gen).cuda()
    w = (1 + 0.2 * torch.randn(D, generator=gen)).cuda()
    do = torch.randn((B, N, H, D), generator=gen).to(dt).cuda()
    q, k, v = (qkv[:, :, i * H:(i + 1) * H] for i in range(3))
    norm = hyena.QKNorm(B, N, H, H, D, io_dtype=IO[dtype], norm="l2")
    rec = hyena.Recurrence(B, N, H, D, D, io_dtype=IO[dtype], training=True)
    qn, kn = norm.forward(q[:, :N], k[:, :N], w, w)
    o, state = rec.forward(qn, kn, v[:, :N], g[:, :N], scale=1.0, return_state=True)
    dqn, dkn, dv, dg, _ = rec.backward(do, qn, kn, v[:, :N], g[:, :N], scale=1.0)
    dq, dk, dwq, dwk = norm.backward(dqn, dkn, q[:, :N], k[:, :N], w, w)

    freqs = f64(norm.freqs)
    pos = np.arange(N + 1)[None] + np.zeros((B, 1))

    def whole(q, k, v, g, wq, wk, n):
        a = [mixer_ref.qk_norm(x[:, :n], y, pos[:, :n], freqs, "l2", "half", D, 1e-6, 1.0) for x, y in ((q, wq), (k, wk))]
        return mixer_ref.recurrence(*a, v[:, :n], g[:, :n], 1.0)

    at = [f64(x) for x in (q, k, v, g, w, w)]
    grads = [f64(x) for x in (dq, dk, dv, dg, dwq, dwk)]
    u = mixer_ref.HALF_STEP[dtype]
    rng = np.random.default_rng(1)
    for i, name in enumerate(("dq", "dk", "dv", "dg", "dwq", "dwk")):
        way = rng.standard_normal(at[i].shape)
        if i < 4:
            way[:, N:] = 0.0
        h = 1e-5
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * way, at[i] - h * way
        slope = sum(s * (whole(*x, N)[0] * f64(do)).sum() for s, x in ((1, up), (-1, down))) / (2 * h)
        mine = grads[i] * (way[:, :N] if i < 4 else way)
        # four roundings to the storage type on the way (q and k, their gradients, operands, the result);
        # their signs are independent over the tensor, 8 standard deviations
        size = np.sqrt((mine ** 2).sum())
        if i >= 4:  # sums over all tokens: the terms' size
            size = np.sqrt(sum((grads[j] * at[j][:, :N]) ** 2 for j in (0, 1)).sum()) + size
        assert abs(mine.sum() - slope) <= 8 * 4 * u * size + 1e-4 * abs(slope) + 1e-6, name

    ro, _, ao, _ = whole(*at, N + 1)
    one = hyena.QKNorm(B, 1, H, H, D, io_dtype=IO[dtype], norm="l2")
    last = torch.full((B, 1), N, dtype=torch.int32, device="cuda")
    q1, k1 = one.forward(q[:, N:], k[:, N:], w, w, positions=last)
    got = rec.step(q1[:, 0], k1[:, 0], v[:, N], g[:, N], state, scale=1.0)
    err = np.abs(f64(got) - ro[:, N])
    assert np.all(err <= 4 * u * ao[:, N] + 2.0 ** -15 * ao[:, N])
