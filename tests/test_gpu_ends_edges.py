"""Where the embedding, the norm of whole tokens and the loss over a vocabulary could lose
what their sums are made of: precision that depends on a call's size, and sizes at which
one kernel hands over to another.  Tolerances stand at each test."""
import numpy as np
import pytest

import ends_ref
from gpu_util import say
from long_convolution_sequence_rfft_amd import hyena
from test_gpu_embedding import run as embedding_run
from test_gpu_recurrence import IO, f64, torch_dtype
from test_gpu_token_loss import run as loss_run

pytestmark = pytest.mark.gpu


def rounded(a, dtype):
    """float64 values as the storage type holds them."""
    import torch
    return torch.from_numpy(np.asarray(a, dtype=np.float64)).to(torch_dtype(dtype)).double().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", [(5, 300, 40), (17, 131, 45), (150, 2000, 96), (1200, 3500, 64), (4200, 1100, 40), (4000, 15, 40), (3000, 259, 300)])
def test_loss_gradients_round_only_their_results(case, dtype):
    # All tokens are alike, and so are all rows of the table but the target's, which is zeros: G is
    # 1 + 0.95 u beside it, a value that the storage type rounds to 1.  Such a rounding would be in
    # every sum, 0.95 u of it beside the result's own u.  Behind that: what a probability is off by
    # (r, of two float32 logits, the exponential and lse), two terms of G (u^2; binary16's
    # subnormals 2^-39 of the largest |d_loss|), 2^-22 for the product with d_loss and the factor, and the
    # sum of K terms in float32.
    import torch
    T, V, d = case
    say(f"[gpu] token_loss, gradients of values beside the target {case} {dtype}")
    u = ends_ref.HALF_STEP[dtype]
    gen = torch.Generator().manual_seed(T)
    dt = torch_dtype(dtype)
    x = (torch.rand(d, generator=gen) + 0.5).to(dt)
    w = ((torch.rand(d, generator=gen) + 0.5) / d).to(dt)
    row = V * 3 // 7
    table = w.expand(V, d).clone()
    table[row] = 0.0
    xs, target = x.expand(1, T, d).contiguous().cuda(), torch.full((1, T), row, dtype=torch.int32, device="cuda")
    plan = hyena.TokenLoss(1, T, V, d, io_dtype=IO[dtype])
    _, lse = plan.forward(xs, table.cuda(), target)
    assert bool((lse == lse[0, 0]).all())
    xd, wd = f64(x), f64(w)
    p = np.exp(xd @ wd - float(lse[0, 0]))
    dl = float(np.float32((1 + 0.95 * u) / p))
    g = dl * p
    dx, d_table = plan.backward(torch.full((1, T), dl, device="cuda"), xs, table.cuda(), target, lse)
    size = np.abs(xd) @ np.abs(wd)
    r = 2 * (d + 8) * 2.0 ** -24 * size + 2.0 ** -20 + 2.0 ** -21 * size
    dg = (r + u * u + 2.0 ** -22) * g + (2.0 ** -39 * dl if dtype == "f16" else 0.0)
    for got, n, of, what in ((dx[0], V - 1, wd, "dx"), (d_table[torch.arange(V) != row], T, xd, "d_table")):
        ref = n * g * of
        bound = u * np.abs(ref) + n * (dg + (n + 16) * 2.0 ** -24 * g) * np.abs(of)
        once_more = rounded(n * float(rounded(g, dtype)) * of, dtype)
        assert np.any(np.abs(once_more - ref) > bound)  # the test tells the two apart
        err = np.abs(f64(got) - ref)
        say(f"[gpu]   {what}: worst error / bound {float(np.max(err / bound)):.3f}")
        assert np.all(err <= bound), what


@pytest.mark.parametrize("tokens", [7, 8, 9, 10])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_loss_of_few_tokens_at_the_limit_of_eight(dtype, tokens):
    # rows made of 16-byte pieces, and not; values that are no multiple of a wave's four
    loss_run((1, tokens, 777, 72), dtype, masked=0.0)
    loss_run((tokens, 1, 3001, 301), dtype, masked=0.3)


@pytest.mark.parametrize("case,strided", [((1, 140001, 1600001, 4), False), ((2, 70001, 5000003, 2), True)])
def test_many_tokens_of_a_table_beyond_the_dealt_groups(case, strided):
    # more values than 1024 groups of the sort hold: several groups share a list of dealt tokens.  Some
    # values have many tokens, more than a wave keeps; neighbours of the same list have some, too
    B, N, V, d = case
    rng = np.random.default_rng(7)
    tok = rng.integers(0, V, (B, N))
    tok[:, ::3] = 1024 * 5 + 3
    tok[:, 1::9] = 3
    tok[:, 2::9] = 1024 * (V // 1024 - 1) + 3
    hyena.hyena_timing_begin(64)
    try:
        embedding_run(case, "f32", tokens=tok, strided=strided)
    finally:
        kernels, _ = hyena.hyena_timing_end()
    assert any("hyena_embedding_deal" in k for k in kernels)


@pytest.mark.parametrize("rows,d", [((1 << 19) + 5, 256), (1 << 18, 1028)])
def test_norm_weight_gradient_of_very_many_rows(rows, d):
    # All rows are alike, +-1 and the same gradient, so that every term is exact. A team sums 16 of
    # them in float32, at worst 8.5 2^-24 off ((2 + ... + 16) / 16), which is the whole sum's error too; a
    # workgroup's part and the result are rounded: 2 2^-24.  The team's rows in one float32 sum would be
    # off by more, the rounding of each step being the same one over and over.
    import torch
    say(f"[gpu] norm, weight's gradient of {rows} rows of {d}")
    gen = torch.Generator().manual_seed(3)
    dy = (0.5 + 0.5 * torch.rand(d, generator=gen))
    x = torch.where(torch.rand(d, generator=gen) < 0.5, -1.0, 1.0)
    plan = hyena.ResidualNorm(1, rows, d, eps=0.0)
    _, dw = plan.backward(dy.cuda().expand(1, rows, d), x.cuda().expand(1, rows, d), torch.ones(d, device="cuda"))
    ref = rows * f64(dy) * f64(x)
    bound = 10.5 * 2.0 ** -24 * np.abs(ref)
    chain = np.cumsum(np.broadcast_to(dy.numpy(), (256, d)), axis=0, dtype=np.float32)[-1].astype(np.float64)
    assert np.any(np.abs(chain / 256 - f64(dy)) > 10.5 * 2.0 ** -24 * f64(dy))  # (256 rows of a team so)
    err = np.abs(f64(dw) - ref)
    say(f"[gpu]   worst error / bound {float(np.max(err / bound)):.3f}")
    assert np.all(err <= bound)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", [(1, 40000, 8), (1, 20000, 2048), (2, 9001, 96), (1, 30000, 33), (1, 2100, 5000), (1, 1500, 16380)])
def test_norm_gradients_of_teams_of_many_rows(case, dtype):
    # more rows for a team than it sums in float32, with some left at its end, by teams of every
    # width; against float64 on the GPU, at the tolerances of the other tests of the norm
    import torch
    B, N, d = case
    say(f"[gpu] norm gradients {case} {dtype}")
    gen = torch.Generator(device="cuda").manual_seed(1)
    dt = torch_dtype(dtype)
    s, dy = (torch.randn(case, generator=gen, device="cuda").to(dt) for _ in range(2))
    w = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda")
    dx, dw = hyena.ResidualNorm(*case, io_dtype=IO[dtype]).backward(dy, s, w)
    n = s.double() * torch.rsqrt(s.double().square().mean(-1, keepdim=True) + float(np.float32(1e-6)))
    ref = (dy.double() * n).sum((0, 1))
    size = (dy.double() * n).abs().sum((0, 1))
    assert bool(((dw.double() - ref).abs() <= 2.0 ** -24 * ref.abs() + 2.0 ** -20 * size).all())
    again = hyena.ResidualNorm(*case, io_dtype=IO[dtype]).backward(dy, s, w)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_gradients_of_a_packed_table_past_32_bits():
    # More than 4096 tokens: the table of 2^21 + 77 rows of 1024 in bf16 (4.3 GB) is packed, and G is made in
    # many pieces.  All rows but five are zeros, and so are their logits; those five, their neighbours
    # and others are compared.  Tolerances: those of the loss's other tests (r of a probability
    # from two logits' sums of absolute values), two terms of G, sums of as many terms as are not 0.
    import torch
    T, V, d, scale = 5000, (1 << 21) + 77, 1024, 0.2
    say(f"[gpu] token_loss gradients, packed table past 32 bits, {T} tokens")
    u = ends_ref.HALF_STEP["bf16"]
    gen = torch.Generator().manual_seed(3)
    at = torch.tensor([0, 5, V // 2, V - 2, V - 1])
    rows = torch.randn((5, d), generator=gen).bfloat16()
    table = torch.zeros((V, d), dtype=torch.bfloat16, device="cuda")
    table[at.cuda()] = rows.cuda()
    x = torch.randn((1, T, d), generator=gen).bfloat16()
    hit = torch.arange(T) % 5
    hit[::7] = -1
    target = torch.where(hit >= 0, at[hit], -1).to(torch.int32)[None].cuda()
    plan = hyena.TokenLoss(1, T, V, d, io_dtype=hyena.HYENA_BF16, scale=scale)
    _, lse = plan.forward(x.cuda(), table, target)
    dx, dt = plan.backward(torch.ones((1, T), device="cuda"), x.cuda(), table, target, lse)
    live = (hit >= 0).numpy()
    xs, ws, y = f64(x)[0][live], f64(rows), hit.numpy()[live]
    s = float(np.float32(scale))
    size = s * np.abs(xs) @ np.abs(ws).T
    p = np.exp(s * xs @ ws.T - f64(lse)[0][live][:, None])
    g = p.copy()
    g[np.arange(len(y)), y] -= 1
    r = 2 * (d + 8) * 2.0 ** -24 * size.max(-1) + 2.0 ** -20 + 2.0 ** -21 * size.max(-1)
    dg = r[:, None] * p + 2.0 ** -23 + u * u * np.abs(g)
    ref = s * g @ ws
    bound = u * np.abs(ref) + s * (dg + 21 * 2.0 ** -24 * np.abs(g)) @ np.abs(ws)
    assert np.all(np.abs(f64(dx)[0][live] - ref) <= bound) and not f64(dx)[0][~live].any()
    ref = s * g.T @ xs
    bound = u * np.abs(ref) + s * (dg + (len(y) + 16) * 2.0 ** -24 * np.abs(g)).T @ np.abs(xs)
    assert np.all(np.abs(f64(dt[at.cuda()]) - ref) <= bound)
    p = np.exp(-f64(lse)[0][live])  # of a row of zeros
    ref = s * p @ xs
    bound = u * np.abs(ref) + s * (p * (r + u * u + (len(y) + 16) * 2.0 ** -24)) @ np.abs(xs)
    for v in (1, 4, 6, V // 2 - 1, V // 2 + 1, V // 3, V - 3):
        assert np.all(np.abs(f64(dt[v]) - ref) <= bound + ends_ref.TINY["bf16"]), v
