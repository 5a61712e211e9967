"""The gated linear recurrence on the GPU against its definition in float64.

Tolerances.  An output is a sum of products; its bound is taken on the same
sum of absolute values A.  float32 accumulation of a tile's products (at most
128 channels, 64 tokens and a handful of carries) and the decays (a float32
exponent of at most 126 in size: relative error up to 126 ln 2 2^-24) stay
below 2^-15 A.  With 16-bit storage the scores between tokens, or the state,
are rounded once more as operands (half a step u of A) and the output is
rounded (u of its value): u |ref| + (u + 2^-15) A.  States are 2^-15 A at any
storage type.  A binary16 score below 2^-14 is subnormal: its rounding is off by
at most 2^-25 absolutely instead, times the other operand of the product, a
token's values, for the up to 64 tokens of a chunk.  dg is a sum over later tokens of q.dq - k.dk, each with the
error 2^-15 of its own absolute sum.
"""
import numpy as np
import pytest

import mixer_ref
from gpu_util import say
from long_convolution_sequence_rfft_amd import hyena

pytestmark = pytest.mark.gpu

IO = {"f32": hyena.HYENA_F32, "bf16": hyena.HYENA_BF16, "f16": hyena.HYENA_F16}
SMALL = 2.0 ** -15


def torch_dtype(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def f64(t):
    return t.detach().double().cpu().numpy()


class Case:
    """Inputs on the GPU (rounded to the storage type) and in float64."""

    def __init__(self, B, N, H, dk, dv, dtype, seed, carry=True, lengths=None, resets=(), decay=0.5, sliced=False):
        import torch
        say(f"[gpu] recurrence B={B} N={N} H={H} dk={dk} dv={dv} {dtype} carry={carry} lengths={lengths} "
            f"resets={resets} sliced={sliced}")
        gen = torch.Generator().manual_seed(seed)
        dt = torch_dtype(dtype)
        rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
        self.B, self.N, self.H, self.dk, self.dv, self.dtype = B, N, H, dk, dv, dtype
        self.scale = dk ** -0.5
        if sliced:  # q, k, v: odd slices of one projection, [B, H, N] order behind them
            full = rnd(B, H, N, 2 * dk + dv + 3).to(dt).cuda().transpose(1, 2)
            self.q, self.k, self.v = full[..., 1:1 + dk], full[..., 1 + dk:1 + 2 * dk], full[..., 2 + 2 * dk:2 + 2 * dk + dv]
            self.g = (-decay * torch.rand((B, H, N, 2), generator=gen)).cuda().transpose(1, 2)[..., 1]
            self.do = rnd(N, B, H, dv + 1).to(dt).cuda().transpose(0, 1)[..., :dv]
        else:
            self.q, self.k, self.v = (rnd(B, N, H, d).to(dt).cuda() for d in (dk, dk, dv))
            self.g = (-decay * torch.rand((B, N, H), generator=gen)).cuda()
            self.do = rnd(B, N, H, dv).to(dt).cuda()
        if resets:
            self.g = self.g.clone()
            for t, value in resets:
                if t < N:
                    self.g[:, t] = float(value)
        self.state = rnd(B, H, dk, dv).cuda() if carry else None
        self.d_final = rnd(B, H, dk, dv).cuda() if carry else None
        self.lengths = torch.tensor(lengths, dtype=torch.int32).cuda() if lengths is not None else None
        self.plan = hyena.Recurrence(B, N, H, dk, dv, io_dtype=IO[dtype], training=True)

    def inputs64(self):
        opt = lambda t: None if t is None else f64(t)  # noqa: E731
        n = None if self.lengths is None else self.lengths.cpu().numpy()
        return [f64(t) for t in (self.q, self.k, self.v, self.g)], opt(self.state), n, opt(self.d_final)

    def forward(self, **kw):
        return self.plan.forward(self.q, self.k, self.v, self.g, scale=self.scale, state=self.state,
                                 lengths=self.lengths, return_state=True, **kw)

    def backward(self):
        return self.plan.backward(self.do, self.q, self.k, self.v, self.g, scale=self.scale, state=self.state,
                                  lengths=self.lengths, d_final=self.d_final)


def close(got, ref, bound, what):
    err = np.abs(f64(got) - ref)
    worst = float(np.max(err / np.maximum(bound, 1e-30))) if err.size else 0.0
    say(f"[gpu]   {what}: worst error / bound {worst:.3f}")
    assert np.all(np.isfinite(f64(got))), what
    assert worst <= 1.0, what


def floor(c, values):
    """What subnormal binary16 scores may add, from the values [B, N, H, width] that they weight."""
    return 64 * 2.0 ** -25 * np.abs(values).max(1, keepdims=True) if c.dtype == "f16" else 0.0


def check_forward(c):
    (q, k, v, g), state, n, _ = c.inputs64()
    o, last = c.forward()
    ro, rs, ao, as_ = mixer_ref.recurrence(q, k, v, g, c.scale, state, n)
    u = mixer_ref.HALF_STEP[c.dtype]
    close(o, ro, u * np.abs(ro) + ((u if c.dtype != "f32" else 0) + SMALL) * ao + floor(c, v), "o")
    close(last, rs, SMALL * as_ + 1e-30, "state")


def check_backward(c):
    (q, k, v, g), state, n, df = c.inputs64()
    do = f64(c.do)
    dq, dk, dv, dg, ds = c.backward()
    ref = mixer_ref.recurrence_grad(do, q, k, v, g, c.scale, state, n, df)
    ab = [np.abs(x) if x is not None else None for x in (do, q, k, v)]
    absolute = mixer_ref.recurrence_grad(*ab, g, abs(c.scale), None if state is None else np.abs(state), n,
                                         None if df is None else np.abs(df))
    u = mixer_ref.HALF_STEP[c.dtype]
    for got, r, a, x, what in zip((dq, dk, dv), ref, absolute, (k, q, do), ("dq", "dk", "dv")):
        close(got, r, u * np.abs(r) + ((u if c.dtype != "f32" else 0) + SMALL) * a + floor(c, x), what)
    each = (ab[1] * absolute[0]).sum(-1) + (ab[2] * absolute[1]).sum(-1)
    over = np.flip(np.cumsum(np.flip(each, 1), 1), 1) + absolute[3]
    if df is not None:
        _, last, _, alast = mixer_ref.recurrence(q, k, v, g, c.scale, state, n)
        over = over + (alast * np.abs(df)).sum((-1, -2))[:, None]
    close(dg, ref[3], SMALL * over, "dg")
    if state is not None:
        close(ds, ref[4], SMALL * absolute[4] + 1e-30, "d_state")
    else:
        assert ds is None


SHAPES = [(1, 1, 1, 64, 64), (2, 2, 3, 64, 64), (1, 63, 2, 64, 64), (1, 64, 1, 64, 64), (2, 65, 2, 64, 64),
          (1, 129, 2, 64, 64), (1, 200, 1, 128, 128), (2, 130, 2, 64, 128), (1, 150, 2, 128, 64), (1, 97, 3, 40, 72),
          (1, 33, 2, 1, 1), (1, 140, 2, 7, 5), (1, 260, 1, 65, 33), (1, 31, 2, 16, 100), (3, 520, 2, 32, 16)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dtype):
    check_forward(Case(*shape, dtype, seed=sum(shape)))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, dtype):
    check_backward(Case(*shape, dtype, seed=sum(shape) + 1))


MASKS = [
    dict(lengths=(0, 1, 150)), dict(lengths=(64, 65, 200)), dict(lengths=(-3, 128, 1 << 30)),
    dict(resets=((0, -np.inf), (70, -np.inf), (71, -np.inf), (199, -np.inf))),
    dict(resets=((10, np.finfo(np.float32).min), (64, -88.0), (130, -87.0), (150, -1e4))),
    dict(lengths=(0, 0, 0)), dict(decay=40.0), dict(decay=0.0), dict(decay=1e-4, carry=False),
    dict(sliced=True), dict(sliced=True, lengths=(5, 199, 77), carry=False),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("mask", MASKS)
def test_masks_and_views(mask, dtype):
    c = Case(3, 200, 2, 20, 36, dtype, seed=5, **mask)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_padding_is_neither_read_nor_left(dtype):
    """NaN and infinities behind a row's length: outputs there are zero, the rest is what it was."""
    import torch
    c = Case(3, 150, 2, 64, 64, dtype, seed=9, lengths=(0, 70, 150))
    want = [*c.forward(), *c.backward()]
    for t in (c.q, c.k, c.v, c.g, c.do):
        t[0, :] = float("nan")
        t[1, 70:] = float("inf")
    got = [*c.forward(), *c.backward()]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for x in (got[0], got[2], got[3], got[4], got[5]):
        assert not x[0].any() and not x[1, 70:].any()
    assert torch.equal(got[1][0], c.state[0]) and torch.equal(got[6][0], c.d_final[0])


def test_shared_keys_through_a_zero_stride():
    """One key for all heads: the gradient is written per use, the caller sums."""
    import torch
    c = Case(2, 140, 4, 32, 48, "f32", seed=3)
    one = c.k[:, :, :1]
    c.k = one.expand(2, 140, 4, 32)
    check_forward(c)
    check_backward(c)
    dk = c.backward()[1].sum(2)
    c.k = c.k.contiguous()
    assert torch.equal(dk, c.backward()[1].sum(2))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_gradients_against_differences(dtype):
    """Central differences of the float64 definition along a random direction, at the stored inputs."""
    c = Case(2, 90, 2, 24, 20, dtype, seed=11, resets=((40, -np.inf),))
    (q, k, v, g), state, n, df = c.inputs64()
    do = f64(c.do)
    grads = [f64(x) for x in c.backward()]
    rng = np.random.default_rng(0)
    loss = lambda *x: (lambda o, s, *_: (o * do).sum() + (s * df).sum())(  # noqa: E731
        *mixer_ref.recurrence(*x[:4], c.scale, x[4], n))
    at = [q, k, v, g, state]
    for i, name in enumerate(("dq", "dk", "dv", "dg", "d_state")):
        way = rng.standard_normal(at[i].shape)
        if i == 3:
            way[np.isneginf(g)] = 0.0
        h = 1e-5
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * way, at[i] - h * way
        slope = (loss(*up) - loss(*down)) / (2 * h)
        # rounding: half a step of each gradient and of its operands, at random signs over the tensor
        scale = np.sqrt(((grads[i] * way) ** 2).sum())
        u = mixer_ref.HALF_STEP[dtype] if i < 3 else SMALL
        assert abs((grads[i] * way).sum() - slope) <= 8 * u * scale + 1e-4 * abs(slope) + 1e-6, name


def test_pieces_of_a_sequence_equal_the_whole_and_steps_go_on():
    """A prompt in two pieces, then tokens one at a time, against one call."""
    import torch
    B, N, H, dk, dv = 2, 300, 3, 64, 64
    c = Case(B, N, H, dk, dv, "f32", seed=21)
    o, last = c.forward()
    cut, end = 171, 290
    first = hyena.Recurrence(B, cut, H, dk, dv)
    second = hyena.Recurrence(B, end - cut, H, dk, dv)
    part = lambda t, a, b: t[:, a:b]  # noqa: E731
    o1, s1 = first.forward(*(part(t, 0, cut) for t in (c.q, c.k, c.v, c.g)), state=c.state, return_state=True)
    o2, s2 = second.forward(*(part(t, cut, end) for t in (c.q, c.k, c.v, c.g)), state=s1, return_state=True)
    table = torch.full((5, H, dk, dv), 7.0, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    table[slots.long()] = s2
    outs = [c.plan.step(c.q[:, t], c.k[:, t], c.v[:, t], c.g[:, t], table, slots=slots) for t in range(end, N)]
    got = torch.cat([o1, o2, torch.stack(outs, 1)], 1)
    (q, k, v, g), state, n, _ = c.inputs64()
    ro, rs, ao, as_ = mixer_ref.recurrence(q, k, v, g, c.scale, state, n)
    close(got, ro, 2 * SMALL * ao, "o in pieces")
    close(table[slots.long()], rs, 2 * SMALL * as_, "state in pieces")
    assert bool((table[[0, 2, 4]] == 7.0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 1, 64, 64), (3, 2, 128, 128), (2, 3, 40, 72), (2, 2, 7, 5), (1, 2, 1, 1),
                                   (2, 1, 128, 3), (1, 3, 5, 127)])
def test_step(shape, dtype):
    import torch
    B, H, dk, dv = shape
    say(f"[gpu] step {shape} {dtype}")
    gen = torch.Generator().manual_seed(B + H + dk + dv)
    dt = torch_dtype(dtype)
    q, k, v = (torch.randn((B, H, d), generator=gen).to(dt).cuda() for d in (dk, dk, dv))
    g = -torch.rand((B, H), generator=gen).cuda()
    g[0, 0] = -np.inf
    table = torch.randn((B + 2, H, dk, dv), generator=gen).cuda()
    before = table.clone()
    slots = torch.arange(B, 0, -1, dtype=torch.int32).cuda()
    plan = hyena.Recurrence(B, 1, H, dk, dv, io_dtype=IO[dtype])
    o = plan.step(q, k, v, g, table, scale=0.5, slots=slots)
    at = slots.long().cpu().numpy()
    ro, rs, ao, as_ = mixer_ref.recurrence(*(f64(t)[:, None] for t in (q, k, v, g)), 0.5, f64(before)[at])
    u = mixer_ref.HALF_STEP[dtype]
    close(o, ro[:, 0], u * np.abs(ro[:, 0]) + SMALL * ao[:, 0], "o")
    close(table[slots.long()], rs, SMALL * as_, "state")
    assert torch.equal(table[0], before[0]) and torch.equal(table[B + 1], before[B + 1])
    # rows outside the table take no part
    table.copy_(before)
    slots[0] = -1
    if B > 1:
        slots[1] = B + 2
    o2 = plan.step(q, k, v, g, table, scale=0.5, slots=slots)
    assert not o2[:2].any()
    if B > 2:
        assert torch.equal(o2[2:], o[2:])
    gone = [i for i in range(B + 2) if i not in slots.tolist()]
    assert torch.equal(table[gone], before[gone])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_in_a_replayed_graph_and_on_another_stream(dtype):
    import torch
    c = Case(2, 400, 2, 64, 64, dtype, seed=31)
    want = [t.clone() for t in (*c.forward(), *c.backward())]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [*c.forward(), *c.backward()]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [*c.forward(), *c.backward()]
    for _ in range(3):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        again = [*c.forward(), *c.backward()]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_long_row_far_offsets():
    """A row of 70000 tokens against the same row in float64 from its last 3000 tokens on (decays of at
    least 0.01 a token leave nothing of what came before)."""
    import torch
    B, N, H, d = 1, 70000, 2, 64
    gen = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn((B, N, H, d), generator=gen, device="cuda") for _ in range(3))
    g = -0.01 - 0.1 * torch.rand((B, N, H), generator=gen, device="cuda")
    plan = hyena.Recurrence(B, N, H, d, d)
    o, last = plan.forward(q, k, v, g, return_state=True)
    tail = 3000
    ro, rs, ao, as_ = mixer_ref.recurrence(*(f64(t[:, -tail:]) for t in (q, k, v, g)), d ** -0.5)
    close(o[:, -500:], ro[:, -500:], SMALL * ao[:, -500:], "o")
    close(last, rs, SMALL * as_, "state")
