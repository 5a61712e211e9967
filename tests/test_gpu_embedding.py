"""Rows of a table by token and the table's gradient on the GPU against their
definition in float64.

Tolerances.  A row is one float32 product, rounded: half a step u of the storage
type and 2^-24 of the value.  A gradient is a sum of n float32 terms and at most
one more value: n 2^-24 of the sum of absolute values, and u of the result.
Values below the type's normal range are off by half its smallest step.
"""
import numpy as np
import pytest

import ends_ref
from gpu_util import say
from long_convolution_sequence_rfft_amd import hyena
from test_gpu_recurrence import IO, f64, torch_dtype

pytestmark = pytest.mark.gpu

CASES = [
    # B, N, V, d
    (1, 1, 1, 1), (1, 1, 7, 768), (2, 3, 50, 64), (3, 37, 211, 100), (1, 500, 3, 72), (4, 129, 1000, 33),
    (1, 1025, 257, 24), (2, 700, 5001, 10), (1, 5, 100000, 16), (1, 64, 300, 2056), (1, 9, 40, 5003), (2, 3000, 97, 8),
]


def text(rng, shape, V):
    """Tokens of a text: value v about as often as 1 / v."""
    return np.minimum((V ** rng.random(shape)).astype(np.int64), V) - 1


def close(got, ref, size, dtype, what):
    u = ends_ref.HALF_STEP[dtype]
    err = np.abs(f64(got) - ref)
    bound = u * np.abs(ref) + size + ends_ref.TINY[dtype]
    say(f"[gpu]   {what}: worst error / bound {float(np.max(err / bound)):.3f}")
    assert np.all(err <= bound), what


def run(case, dtype, seed=1, scale=1.5, tokens=None, strided=False, accumulate=False, bad=False):
    import torch
    B, N, V, d = case
    say(f"[gpu] embedding {case} {dtype} scale={scale} strided={strided} accumulate={accumulate}")
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    dt = torch_dtype(dtype)
    tok = text(rng, (B, N), V) if tokens is None else tokens
    if bad:
        tok = np.where(rng.random((B, N)) < 0.3, rng.choice([-1, -2 ** 31, V, 2 ** 31 - 1], (B, N)), tok)
    at = torch.from_numpy(tok.astype(np.int32)).cuda()
    table = torch.randn((V, d), generator=gen).to(dt).cuda()
    d_out = torch.randn((B, N, d), generator=gen).to(dt).cuda()
    if strided:
        # tokens without their last one, rows that are slices of wider ones
        wide = torch.zeros((B, N + 1), dtype=torch.int32, device="cuda")
        wide[:, :N] = at
        at = wide[:, :N]
        both = torch.zeros((B, N + 2, d + 3), dtype=dt, device="cuda")
        both[:, 1:N + 1, 2:d + 2] = d_out
        d_out = both[:, 1:N + 1, 2:d + 2]
    old = torch.randn((V, d), generator=gen).to(dt).cuda() if accumulate else None
    plan = hyena.Embedding(B, N, V, d, io_dtype=IO[dtype], scale=scale)
    f32scale = float(np.float32(scale))
    out = plan.forward(at, table)
    ref = ends_ref.embedding(tok, f64(table), f32scale)
    close(out, ref, 2.0 ** -24 * np.abs(ref), dtype, "out")
    g, a, n = ends_ref.embedding_grad(f64(d_out), tok, V, f32scale, None if old is None else f64(old))
    kept = None if old is None else old.clone()
    got = plan.backward(d_out, at, d_table=old)
    close(got, g, (n[:, None] + 3) * 2.0 ** -24 * a, dtype, "d_table")
    if accumulate:
        assert got is old
        assert torch.equal(got[torch.from_numpy(n == 0).cuda()], kept[torch.from_numpy(n == 0).cuda()])
    else:
        assert not got[torch.from_numpy(n == 0).cuda()].any()
        assert torch.equal(got, plan.backward(d_out, at))  # the same bits


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", CASES)
def test_against_float64(case, dtype):
    run(case, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [CASES[3], CASES[5], CASES[6], CASES[9]])
def test_strided_tokens_and_gradients(case, dtype):
    run(case, dtype, strided=True, bad=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", [CASES[2], CASES[3], CASES[5], CASES[11]])
def test_added_to_a_gradient(case, dtype):
    run(case, dtype, accumulate=True)
    run(case, dtype, accumulate=True, bad=True, scale=-0.3)


def test_tokens_that_take_no_part():
    run((3, 50, 60, 40), "bf16", bad=True)
    run((2, 40, 30, 8), "f32", tokens=np.full((2, 40), -1))
    run((2, 40, 30, 8), "f32", tokens=np.full((2, 40), 30), accumulate=True)
    # their gradients are not read
    import torch
    d_out = torch.full((1, 4, 8), float("nan"), device="cuda")
    d_out[0, 2] = 1.0
    at = torch.tensor([[-1, 9, 5, 1 << 30]], dtype=torch.int32, device="cuda")
    g = hyena.Embedding(1, 4, 9, 8).backward(d_out, at)
    want = torch.zeros((9, 8), device="cuda")
    want[5] = 1.0
    assert torch.equal(g, want)


def test_one_value_everywhere_and_runs_of_all_lengths():
    run((1, 4100, 500, 36), "f32", tokens=np.full((1, 4100), 123))
    # sorted lists whose values end at, before and after the ends of runs of 4
    rng = np.random.default_rng(3)
    tok = np.repeat(np.arange(300), rng.integers(0, 14, 300))
    rng.shuffle(tok)
    run((1, len(tok), 300, 16), "bf16", tokens=tok[None])
    # above 8192 runs of 4 tokens their length grows
    run((1, 40000, 37, 8), "f32", tokens=text(rng, (1, 40000), 37))


def test_a_broadcast_gradient():
    import torch
    d_out = torch.randn((1, 1, 24), device="cuda").expand(3, 50, 24)
    at = torch.arange(150, dtype=torch.int32, device="cuda").view(3, 50) % 7
    g = hyena.Embedding(3, 50, 7, 24).backward(d_out, at)
    n = np.bincount(np.arange(150) % 7)
    ref = f64(d_out)[0, 0][None] * n[:, None]
    close(g, ref, 25 * 2.0 ** -24 * np.abs(ref), "f32", "d_table")


def test_offsets_past_32_bits():
    # a table of 2^22 + 3 rows of 768 in bf16 is 6.4 GB
    import torch
    V, d = (1 << 22) + 3, 768
    table = torch.zeros((V, d), dtype=torch.bfloat16, device="cuda")
    tok = np.array([[0, V - 1, 1 << 21, V - 1, 12345]])
    at = torch.from_numpy(tok.astype(np.int32)).cuda()
    table[at.long().view(-1)] = torch.randn((5, d), device="cuda").bfloat16()
    plan = hyena.Embedding(1, 5, V, d, io_dtype=hyena.HYENA_BF16)
    assert torch.equal(plan.forward(at, table), table[at.long()])
    d_out = torch.ones((1, 5, d), dtype=torch.bfloat16, device="cuda")
    g = plan.backward(d_out, at)
    assert float(g[V - 1].float().min()) == 2.0 and float(g[V - 2].float().abs().max()) == 0.0
    assert float(g.sum(1, dtype=torch.float32).sum()) == 5.0 * d


def test_replayed_graphs_match_eager_calls():
    import torch
    V, d = 600, 64
    plan = hyena.Embedding(2, 300, V, d, io_dtype=hyena.HYENA_BF16, scale=2.0)
    at = torch.zeros((2, 300), dtype=torch.int32, device="cuda")
    table = torch.randn((V, d), device="cuda").bfloat16()
    d_out = torch.zeros((2, 300, d), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        plan.backward(d_out, at)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, g = plan.forward(at, table), plan.backward(d_out, at)
    rng = np.random.default_rng(5)
    for _ in range(4):
        at.copy_(torch.from_numpy(text(rng, (2, 300), V).astype(np.int32)))
        d_out.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, plan.forward(at, table)) and torch.equal(g, plan.backward(d_out, at))


@pytest.mark.parametrize("kind", ["text", "even", "same", "padded"])
def test_calls_of_many_tokens(kind):
    # from 131072 tokens on they are dealt out to the groups of values first
    rng = np.random.default_rng(8)
    for (B, N, V, d), strided in (((1, 131072, 1000, 8), False), ((3, 45000, 50000, 4), True), ((2, 70001, 300000, 4), False)):
        tok = text(rng, (B, N), V) if kind == "text" else rng.integers(0, V, (B, N))
        if kind == "same":
            tok[:] = V // 2
        if kind == "padded":
            tok[:, N // 3:] = -1
        run((B, N, V, d), "f32", tokens=tok, strided=strided, accumulate=kind == "even")


FEW = [
    # B, N, V, d: around the limit of tables of few values; teams of 8 to 64 lanes; several blocks of channels
    (1, 1, 32, 5), (2, 75, 31, 4), (1, 3000, 32, 1030), (3, 1111, 4, 100), (1, 70000, 16, 33), (1, 9000, 5, 256), (2, 500, 33, 40),
    (1, 40000, 2, 64),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", FEW)
def test_tables_of_few_values(case, dtype):
    rng = np.random.default_rng(6)
    run(case, dtype, tokens=rng.integers(0, case[2], case[:2]))
    run(case, dtype, strided=True, bad=True, scale=-0.7)
    run(case, dtype, accumulate=True, tokens=rng.integers(0, (case[2] + 1) // 2, case[:2]))


def test_rows_without_tokens_keep_their_bits():
    import torch
    for V in (9, 300):
        at = torch.tensor([[3, -1, 3, V]], dtype=torch.int32, device="cuda")
        d_out = torch.ones((1, 4, 8), device="cuda")
        old = torch.full((V, 8), -0.0, device="cuda")
        old[0, 0] = float("nan")
        bits = old.view(torch.int32).clone()
        plan = hyena.Embedding(1, 4, V, 8, scale=-2.0)
        plan.backward(d_out, at, d_table=old)
        rows = torch.arange(V, device="cuda") != 3
        assert torch.equal(old.view(torch.int32)[rows], bits[rows]) and bool((old[3] == -4).all())
        new = plan.backward(d_out, at)
        assert not new.view(torch.int32)[rows].any() and bool((new[3] == -4).all())


@pytest.mark.parametrize("case", [(1, 3000, 1200000, 4), (2, 70001, 1200000, 4), (1, 900, 1600000, 4)])
def test_tables_of_very_many_values(case):
    rng = np.random.default_rng(4)
    tok = rng.integers(0, case[2], case[:2])
    tok[0, ::3] = case[2] - 1
    tok[0, 1::7] = case[2] // 1024 * 1024 - 1
    run(case, "f32", tokens=tok)


@pytest.mark.parametrize("dtype,d", [("f32", 256), ("bf16", 600), ("bf16", 36), ("f16", 129)])
def test_values_that_fill_workgroups(dtype, d):
    # runs of 4 tokens by workgroups of 4 to 32 teams: values that begin and end at, before and
    # after their borders, and have one, some or many of them to themselves
    rng = np.random.default_rng(9)
    counts = np.concatenate([np.arange(1, 70), [127, 128, 129, 130, 255, 256, 257, 258, 400, 511, 513, 1025, 16, 16, 32, 32, 64, 64, 4, 4]])
    rng.shuffle(counts)
    tok = np.repeat(rng.permutation(120)[:len(counts)], counts)
    rng.shuffle(tok)
    run((1, len(tok), 120, d), dtype, tokens=tok[None])
    run((1, len(tok), 120, d), dtype, tokens=tok[None], accumulate=True, bad=True)
    run((1, 5000, 120, d), dtype, tokens=np.full((1, 5000), 119))
