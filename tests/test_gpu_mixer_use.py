"""The gated linear recurrence and the query/key norm as a program uses them
together and at their limits: graphs and streams side by side, tables of states
whose slots change between replays, very many rows or heads, offsets past 32
bits.  Tolerances: those of test_gpu_recurrence.py and test_gpu_qk_norm.py."""
import numpy as np
import pytest

import mixer_ref
from gpu_util import say
from long_convolution_sequence_rfft_amd import hyena
from test_gpu_recurrence import IO, SMALL, Case, check_backward, check_forward, close, f64, torch_dtype

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 2, 65536, 3, 2), (300, 70, 5, 16, 8), (4000, 1, 2, 8, 24)])
def test_many_rows_and_heads(shape, dtype):
    c = Case(*shape, dtype, seed=4)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 1500, 2, 64, 64), (12, 1100, 5, 16, 24), (7, 700, 9, 72, 40)])
def test_many_segments(shape, dtype):
    """Sequences cut into several segments, the backward's states (second shape) into finer ones than its
    gradients, with documents packed into the rows and rows that end inside a segment."""
    B, N = shape[:2]
    lengths = None if B == 1 else tuple((0, 1, N // 2, N - 1, N, N - 64, 65)[i % 7] for i in range(B))
    c = Case(*shape, dtype, seed=sum(shape), lengths=lengths, resets=((129, -np.inf), (N // 2 - 7, -np.inf)), decay=0.05)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_aligned_slices_of_one_projection(dtype):
    """16-byte vectors in rows that are not dense."""
    c = Case(2, 330, 3, 64, 64, dtype, seed=6)
    import torch
    qkv = torch.cat([c.q, c.k, c.v], 2)
    c.q, c.k, c.v = (qkv[:, :, 3 * i:3 * i + 3] for i in range(3))
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(2, 150, 2, 62, 62), (1, 130, 1, 126, 90), (1, 140, 2, 64, 75), (1, 140, 2, 75, 64),
                                   (2, 70, 3, 2, 6), (1, 90, 2, 30, 128)])
def test_rows_of_pairs_and_of_single_elements(shape, dtype):
    """Each tensor's rows are read by 16-byte vectors, by pairs or by elements, as its width and strides
    allow; here they differ from tensor to tensor."""
    c = Case(*shape, dtype, seed=sum(shape) + 2)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slices_that_start_at_an_even_or_odd_element(dtype):
    import torch
    c = Case(2, 140, 2, 24, 40, dtype, seed=14)
    for at in (2, 3):
        full = torch.zeros((2, 140, 2, 24 + 24 + 40 + 8), dtype=c.q.dtype, device="cuda")
        q, k, v = full[..., at:at + 24], full[..., at + 24:at + 48], full[..., 52:92]
        for view, x in ((q, c.q), (k, c.k), (v, c.v)):
            view.copy_(x)
        c.q, c.k, c.v = q, k, v
        check_forward(c)
        check_backward(c)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 1, 3, 64, 64), (2, 5, 3, 128, 96), (4, 64, 2, 40, 128), (3, 33, 5, 128, 128),
                                   (1, 64, 1, 7, 20)])
def test_calls_of_few_tokens_round_only_their_results(shape, dtype):
    """No score and no state is rounded to 16 bits on the way: half a step of the value, and 2^-15 of the
    sum of absolute values that float32 may lose."""
    import torch
    c = Case(*shape, dtype, seed=sum(shape) + 3)
    (q, k, v, g), state, n, df = c.inputs64()
    u, do = mixer_ref.HALF_STEP[dtype], f64(c.do)
    o, _ = c.forward()
    ro, _, ao, _ = mixer_ref.recurrence(q, k, v, g, c.scale, state, n)
    plain = c.plan.forward(c.q, c.k, c.v, c.g, scale=c.scale, state=c.state)[0]
    assert torch.equal(plain, o)
    close(o, ro, u * np.abs(ro) + SMALL * ao, "o")
    grads = c.backward()
    ref = mixer_ref.recurrence_grad(do, q, k, v, g, c.scale, state, n, df)
    size = mixer_ref.recurrence_grad(*(np.abs(x) for x in (do, q, k, v)), g, c.scale, np.abs(state), n, np.abs(df))
    for got, r, a, what in zip(grads[:3], ref, size, ("dq", "dk", "dv")):
        close(got, r, u * np.abs(r) + SMALL * a, what)


def test_large_values_and_scale():
    """States far from 1 (binary16: up to 2^26) and a negative scale."""
    for dtype in ("f32", "bf16", "f16"):
        c = Case(1, 150, 2, 32, 32, dtype, seed=12, decay=0.01)
        c.scale = -2.0 ** -12
        for t in (c.k, c.v):
            t.mul_(64.0)
        c.state.mul_(2.0 ** 20)
        c.d_final.mul_(2.0 ** -10)
        check_forward(c)
        check_backward(c)


def test_two_plans_on_two_streams_and_two_graphs_of_one_plan():
    import torch
    a, b = Case(2, 900, 2, 64, 64, "bf16", seed=41), Case(1, 700, 3, 64, 128, "f32", seed=42)
    run = lambda c: [*c.forward(), *c.backward()]  # noqa: E731
    want = [[t.clone() for t in run(c)] for c in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for s, c in zip(streams, (a, b)):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(run(c))
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for x, y in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(x, y))
    # two graphs that share a plan's workspace, one after the other, eager calls in between
    graphs, outs = [], []
    for direction in (lambda: [*a.forward()], lambda: [*a.backward()]):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(direction())
        graphs.append(g)
    for _ in range(3):
        for t in outs[0] + outs[1]:
            t.fill_(float("nan"))
        for g in graphs:
            g.replay()
        eager = run(a)
        torch.cuda.synchronize()
        for got in (outs[0] + outs[1], eager):
            assert all(torch.equal(p, q) for p, q in zip(got, want[0]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decoding_graph_with_changing_slots(dtype):
    """A decoding step (norm, rotation, recurrence) captured once; requests come and go between replays."""
    import torch
    B, H, D, n = 6, 2, 64, 9
    gen = torch.Generator().manual_seed(3)
    dt = torch_dtype(dtype)
    w = (1 + 0.1 * torch.randn(D, generator=gen)).cuda()
    table = torch.randn((n, H, D, D), generator=gen).cuda()
    qkv = torch.empty((B, 1, 3 * H, D), dtype=dt, device="cuda")
    g = torch.empty((B, H), device="cuda")
    slots = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    positions = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    norm = hyena.QKNorm(B, 1, H, H, D, io_dtype=IO[dtype])
    rec = hyena.Recurrence(B, 1, H, D, D, io_dtype=IO[dtype])

    def step(states):
        q, k = norm.forward(qkv[:, :, :H], qkv[:, :, H:2 * H], w, w, positions=positions)
        return rec.step(q[:, 0], k[:, 0], qkv[:, 0, 2 * H:], g, states, slots=slots)

    step(table.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(table)
    mine = table.clone()
    rng = np.random.default_rng(7)
    for i in range(5):
        qkv.copy_(torch.randn(qkv.shape, generator=gen).to(dt))
        g.copy_(-torch.rand(g.shape, generator=gen))
        at = rng.permutation(n)[:B]
        at[rng.integers(B)] = n + i  # one row without a request
        slots.copy_(torch.from_numpy(at.astype(np.int32)))
        positions.copy_(torch.from_numpy(rng.integers(0, 5000, (B, 1)).astype(np.int32)))
        say(f"[gpu] decoding graph, step {i}, slots {at.tolist()}")
        graph.replay()
        torch.cuda.synchronize()
        before = f64(mine)
        want = step(mine)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(table, mine)
        # against float64, from the stored q and k of the norm
        q, k = norm.forward(qkv[:, :, :H], qkv[:, :, H:2 * H], w, w, positions=positions)
        live = at < n
        ro, rs, ao, as_ = mixer_ref.recurrence(*(f64(x)[live] for x in (q, k, qkv[:, :, 2 * H:], g[:, None])), D ** -0.5,
                                               before[at[live]])
        u = mixer_ref.HALF_STEP[dtype]
        close(out[torch.from_numpy(live).cuda()], ro[:, 0], u * np.abs(ro[:, 0]) + SMALL * ao[:, 0], "o")
        close(mine[torch.from_numpy(at[live]).cuda()], rs, SMALL * as_, "state")
        assert not out[torch.from_numpy(~live).cuda()].any()


def test_recurrence_offsets_past_32_bits():
    """More than 2^31 elements per tensor.  Decays of at least 0.2 a token leave e^-60 of what came 300
    tokens before, so the last tokens of the last heads are compared with their own tail in float64."""
    import torch
    N, H, d, tail = 530000, 32, 128, 340
    say(f"[gpu] recurrence N={N} H={H} d={d}")
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k, v, do = (torch.randn((1, N, H, d), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    g = -0.2 - 0.2 * torch.rand((1, N, H), generator=gen, device="cuda")
    plan = hyena.Recurrence(1, N, H, d, d, io_dtype=hyena.HYENA_BF16, training=True)
    o, last = plan.forward(q, k, v, g, return_state=True)
    grads = plan.backward(do, q, k, v, g)
    cut = lambda t: t[:, -tail:, -2:]  # noqa: E731
    x = [f64(cut(t)) for t in (q, k, v, g)]
    ro, rs, ao, as_ = mixer_ref.recurrence(*x, d ** -0.5)
    ref = mixer_ref.recurrence_grad(f64(cut(do)), *x, d ** -0.5)
    size = mixer_ref.recurrence_grad(np.abs(f64(cut(do))), *(np.abs(t) for t in x[:3]), x[3], d ** -0.5)
    u, at = mixer_ref.HALF_STEP["bf16"], np.s_[:, 300:]
    close(cut(o)[at], ro[at], u * np.abs(ro[at]) + (u + SMALL) * ao[at], "o")
    close(last[:, -2:], rs, SMALL * as_, "state")
    for got, r, a, what in zip(grads[:3], ref, size, ("dq", "dk", "dv")):
        close(cut(got)[at], r[at], u * np.abs(r[at]) + (u + SMALL) * a[at], what)


def test_qk_norm_offsets_past_32_bits_and_more_tiles_than_workgroups():
    """A tile holds one token of 32 heads of 1024 channels, so the queries have more tiles than the
    kernel starts workgroups; their elements number more than 2^31."""
    import torch
    N, H, D = 65700, 32, 1024
    say(f"[gpu] qk_norm N={N} H={H} D={D}")
    gen = torch.Generator(device="cuda").manual_seed(6)
    q = torch.randn((1, N, H, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    k, dk = (torch.randn((1, N, 1, D), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
    plan = hyena.QKNorm(1, N, H, 1, D, io_dtype=hyena.HYENA_BF16, rotary_dim=64)
    qo, ko = plan.forward(q, k, w, w)
    dx = plan.backward(q, dk, q, k, w, w)  # q as its own gradient
    args = (f64(plan.freqs), "rms", "half", 64, 1e-6)
    u, small = mixer_ref.HALF_STEP["bf16"], 2.0 ** -20
    for rows in (slice(0, 3), slice(65534, 65540), slice(N - 3, N)):
        pos = np.arange(N)[None, rows].astype(np.float64)
        for got, x in ((qo, q), (ko, k)):
            ref = mixer_ref.qk_norm(f64(x[:, rows]), f64(w), pos, *args, 1.0)
            err = np.abs(f64(got[:, rows]) - ref)
            assert np.all(err <= u * np.abs(ref) + small * np.abs(ref).max(-1, keepdims=True))
        for got, x, dy in ((dx[0], q, q), (dx[1], k, dk)):
            ref, _, _ = mixer_ref.qk_norm_grad(f64(dy[:, rows]), f64(x[:, rows]), f64(w), pos, *args, 1.0)
            # the projection subtracted is at most |x| |dy w| / (D n^2) |x|, n near 1
            size = 4 * (np.abs(f64(dy[:, rows])).max(-1, keepdims=True) + np.abs(f64(x[:, rows])))
            assert np.all(np.abs(f64(got[:, rows]) - ref) <= u * np.abs(ref) + small * 2 * size)
    # the weights' gradient: float32 terms over all rows
    angle = torch.arange(N, device="cuda", dtype=torch.float64)[:, None] * plan.freqs
    cos, sin = torch.cos(angle)[None, :, None], torch.sin(angle)[None, :, None]
    x, dy = k.double(), dk.double()
    dn = dy.clone()
    dn[..., :32] = dy[..., :32] * cos + dy[..., 32:64] * sin
    dn[..., 32:64] = dy[..., 32:64] * cos - dy[..., :32] * sin
    term = dn * x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    dw, aw = term.sum((0, 1, 2)), term.abs().sum((0, 1, 2))
    # a term's error is relative to its pair's size: twice the sum covers it
    assert bool(((dx[3].double() - dw).abs() <= 2.0 ** -17 * 2 * aw).all())
