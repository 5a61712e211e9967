"""The loss over a vocabulary and its gradients on the GPU against their
definition in float64.

Tolerances.  A logit is a float32 sum of d products: off by E = (d + 8) 2^-24 of
its sum of absolute values (float32 storage: the six products of three bfloat16
terms leave out 3 2^-24 of it, in the 8).  lse is off by the largest E of its token,
2^-16 for exponentials (2^-22) and their sum in float32 (at most 128 in a row), and 2^-22 of
its value; the loss by that and the target's E.

A probability is off by r = 2 E + 2^-20 + 2^-21 |logit| of its value (the factor log2 e and
the difference to lse are rounded).  G is off by r p + 2^-23 and, with 16-bit storage, by
half a step u of that type (binary16: also 2^-39 of the largest |d_loss|, its
subnormals at the scale G is kept at); float32 storage: 2^-23.  A gradient is the sum of
that over the table's (x's) absolute values, K 2^-24 of the sum of |G| times them for
the accumulation of K terms, and half a step of the storage type of itself.
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
    (1, 1, 1, 1), (1, 1, 1000, 64), (2, 3, 50, 32), (1, 128, 256, 128), (3, 43, 257, 40), (1, 130, 2000, 100),
    (2, 70, 513, 33), (1, 300, 700, 257), (1, 17, 5000, 768), (4, 100, 300, 96), (1, 5, 3, 1030),
]


def make(case, dtype, seed, masked=0.2, strided=False):
    import torch
    B, N, V, d = case
    gen = torch.Generator().manual_seed(seed)
    dt = torch_dtype(dtype)
    table = (torch.randn((V, d), generator=gen) * (2.0 / d ** 0.5)).to(dt).cuda()
    x = torch.randn((B, N, d), generator=gen).to(dt).cuda()
    target = torch.randint(0, V, (B, N), generator=gen, dtype=torch.int32)
    none = torch.rand((B, N), generator=gen) < masked
    target = torch.where(none, torch.tensor([-1, V, -2 ** 31], dtype=torch.int32)[torch.arange(B * N).view(B, N) % 3], target).cuda()
    d_loss = torch.randn((B, N), generator=gen).cuda()
    if strided:
        wide = torch.full((B, N + 1, d + 5), float("nan"), dtype=dt, device="cuda")
        wide[:, :N, 3:d + 3] = x
        x = wide[:, :N, 3:d + 3]
        more = torch.zeros((B, N + 2), dtype=torch.int32, device="cuda")
        more[:, 1:N + 1] = target
        target = more[:, 1:N + 1]
        d_loss = torch.tensor(0.37, device="cuda").expand(B, N)
    return x, table, target, d_loss


def compare(got, ref, bound, what):
    err = np.abs(f64(got) - ref)
    say(f"[gpu]   {what}: worst error / bound {float(np.max(err / bound)):.3f}")
    assert np.all(err <= bound), what


def check_grad(grads, case, dtype, x, table, target, d_loss, lse, scale):
    B, N, V, d = case
    u = ends_ref.HALF_STEP[dtype]
    xs, ws, t, dl = f64(x).reshape(-1, d), f64(table), target.cpu().numpy().reshape(-1), f64(d_loss).reshape(-1)
    live = (t >= 0) & (t < V)
    xs = np.where(live[:, None], xs, 0.0)
    rx, rt, g, p, size = ends_ref.token_loss_grad(dl, xs, ws, t, f64(lse).reshape(-1), scale)
    E = (d + 8) * 2.0 ** -24 * size
    r = 2 * E + 2.0 ** -20 + 2.0 ** -21 * size
    largest = np.abs(np.where(live, dl, 0.0)).max()
    dg = np.abs(np.where(live, dl, 0.0))[:, None] * (r[:, None] * p + 2.0 ** -23) + (2.0 ** -23 if dtype == "f32" else u) * np.abs(g)
    if dtype == "f16":
        dg = dg + 2.0 ** -39 * largest * live[:, None]
    scale = abs(scale)
    dx, dt = grads
    if dx is not None:
        more = scale * ((dg + (V + 16) * 2.0 ** -24 * np.abs(g)) @ np.abs(ws))
        compare(dx.reshape(-1, d), rx, u * np.abs(rx) + more + ends_ref.TINY[dtype], "dx")
        assert not f64(dx).reshape(-1, d)[~live].any()
    if dt is not None:
        more = scale * ((dg + (len(t) + 16) * 2.0 ** -24 * np.abs(g)).T @ np.abs(xs))
        compare(dt, rt, u * np.abs(rt) + more + ends_ref.TINY[dtype], "d_table")


def run(case, dtype, seed=1, masked=0.2, strided=False, scale=1.0, inputs=None):
    B, N, V, d = case
    say(f"[gpu] token_loss {case} {dtype} masked={masked} strided={strided} scale={scale}")
    x, table, target, d_loss = make(case, dtype, seed, masked, strided) if inputs is None else inputs
    plan = hyena.TokenLoss(B, N, V, d, io_dtype=IO[dtype], scale=scale)
    loss, lse = plan.forward(x, table, target)
    s = float(np.float32(scale))
    t = target.cpu().numpy().reshape(-1)
    live = (t >= 0) & (t < V)
    xs = np.where(live[:, None], f64(x).reshape(-1, d), 0.0)
    rl, rlse, size = ends_ref.token_loss(xs, f64(table), t, s)
    E = (d + 8) * 2.0 ** -24 * size
    assert not f64(loss).reshape(-1)[~live].any() and not f64(lse).reshape(-1)[~live].any()
    bound = E + 2.0 ** -16 + 2.0 ** -22 * (np.abs(rlse) + size)
    compare(lse.reshape(-1), rlse, bound, "lse")
    compare(loss.reshape(-1), rl, bound + E, "loss")
    check_grad(plan.backward(d_loss, x, table, target, lse), case, dtype, x, table, target, d_loss, lse, s)
    return plan, x, table, target, d_loss, loss, lse


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", CASES)
def test_against_float64(case, dtype):
    run(case, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", [CASES[2], CASES[4], CASES[6], CASES[9]])
def test_strided_views_and_one_gradient_for_all(case, dtype):
    run(case, dtype, strided=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scale(dtype):
    run(CASES[4], dtype, scale=0.125)
    run(CASES[4], dtype, scale=-3.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_no_token_takes_part(dtype):
    import torch
    plan, x, table, target, d_loss, loss, lse = run(CASES[4], dtype, masked=1.1)
    dx, dt = plan.backward(d_loss, x, table, target, lse)
    assert not dx.any() and not dt.any()
    # nothing of their rows or gradients is read
    x.fill_(float("nan"))
    d_loss = torch.full_like(d_loss, float("nan"))
    loss, lse = plan.forward(x, table, target)
    dx, dt = plan.backward(d_loss, x, table, target, lse)
    assert not loss.any() and not lse.any() and not dx.any() and not dt.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_masked_rows_may_hold_anything(dtype):
    import torch
    case = (2, 150, 300, 72)
    x, table, target, d_loss = make(case, dtype, 3, masked=0.5)
    live = (target >= 0) & (target < 300)
    clean = torch.where(live[..., None], x, 0)
    spoilt = torch.where(live[..., None], x, float("nan")).to(x.dtype)
    spoilt[~live.unsqueeze(-1).expand_as(x)] = float("inf")
    d_bad = torch.where(live, d_loss, float("nan"))
    plan = hyena.TokenLoss(2, 150, 300, 72, io_dtype=IO[dtype])
    a, b = plan.forward(clean, table, target), plan.forward(spoilt, table, target)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = plan.backward(torch.where(live, d_loss, 0), clean, table, target, a[1])
    gb = plan.backward(d_bad, spoilt, table, target, a[1])
    assert torch.equal(ga[0], gb[0]) and torch.equal(ga[1], gb[1])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gradients_of_very_different_sizes(dtype):
    # one token's gradient is 2^12 times the others'
    case = (1, 60, 400, 64)
    x, table, target, d_loss = make(case, dtype, 5)
    d_loss = d_loss * 1e-6
    d_loss[0, 7] = 4e-3
    run(case, dtype, inputs=(x, table, target, d_loss))
    run(case, dtype, inputs=(x, table, target, d_loss * 1e-20 if dtype == "bf16" else d_loss * 0))


def test_logits_of_any_size():
    # sure answers (probabilities 0 and 1) and logits of some hundreds
    for dtype in ("f32", "bf16"):
        x, table, target, d_loss = make((1, 40, 500, 48), dtype, 6, masked=0.0)
        run((1, 40, 500, 48), dtype, inputs=((x.float() * 60).to(x.dtype), table, target, d_loss))
        run((1, 40, 500, 48), dtype, inputs=(x * 0, table, target, d_loss))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_what_is_not_wanted(dtype):
    import torch
    plan, x, table, target, d_loss, loss, lse = run(CASES[9], dtype)
    dx, dt = plan.backward(d_loss, x, table, target, lse)
    a = plan.backward(d_loss, x, table, target, lse, want_table=False)
    b = plan.backward(d_loss, x, table, target, lse, want_dx=False)
    assert a[1] is None and b[0] is None and torch.equal(a[0], dx) and torch.equal(b[1], dt)
    assert plan.backward(d_loss, x, table, target, lse, want_dx=False, want_table=False) == (None, None)


def test_gradient_against_differences():
    import torch
    case = (1, 3, 11, 6)
    x, table, target, d_loss = make(case, "f32", 8, masked=0.0)
    plan = hyena.TokenLoss(*case)
    loss, lse = plan.forward(x, table, target)
    dx, dt = (f64(t) for t in plan.backward(d_loss, x, table, target, lse))
    t, dl = target.cpu().numpy().reshape(-1), f64(d_loss).reshape(-1)
    f = lambda x, w: (dl * ends_ref.token_loss(x, w, t, 1.0)[0]).sum()  # noqa: E731
    xd, wd, h = f64(x).reshape(3, 6), f64(table), 1e-5
    for i in np.ndindex(3, 6):
        e = np.zeros_like(xd)
        e[i] = h
        assert abs((f(xd + e, wd) - f(xd - e, wd)) / (2 * h) - dx[0][i]) < 1e-5
    for i in np.ndindex(11, 6):
        e = np.zeros_like(wd)
        e[i] = h
        assert abs((f(xd, wd + e) - f(xd, wd - e)) / (2 * h) - dt[i]) < 1e-5


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_several_pieces_of_the_vocabulary(dtype):
    # G of 16500 tokens fits 1 GiB for a part of these 40009 values (float32: a quarter): against
    # products in float64 on the GPU
    import torch
    say(f"[gpu] token_loss in pieces {dtype}")
    B, N, V, d = 3, 5500, 40009, 64
    x, table, target, d_loss = make((B, N, V, d), dtype, 4, masked=0.1)
    plan = hyena.TokenLoss(B, N, V, d, io_dtype=IO[dtype])
    assert plan.backward_bytes < (3 if dtype == "f32" else 1) * 2 * B * N * V
    loss, lse = plan.forward(x, table, target)
    dx, dt = plan.backward(d_loss, x, table, target, lse)
    live = ((target >= 0) & (target < V)).view(-1)
    xs, ws = x.view(-1, d).double(), table.double()
    l = xs @ ws.t().contiguous()
    ref = torch.where(live, torch.logsumexp(l, -1), 0)
    assert float((lse.view(-1) - ref).abs().max()) < 2e-4
    p = torch.exp(l - lse.view(-1, 1).double())
    p[torch.arange(B * N, device="cuda"), target.view(-1).long().clamp(0, V - 1)] -= 1
    p = torch.where(live[:, None], p * d_loss.view(-1, 1).double(), 0)
    u = ends_ref.HALF_STEP[dtype]
    # the norm of the errors: half a step of G and half a step of the result, each of every value
    for got, ref in ((dx.view(-1, d), p @ ws), (dt, p.t().contiguous() @ xs)):
        off = float(torch.linalg.vector_norm(got.double() - ref) / torch.linalg.vector_norm(ref))
        say(f"[gpu]   error norm {off:.3g}")
        assert off < (2 * u if dtype != "f32" else 1e-5)


def test_streams_and_replayed_graphs():
    import torch
    case = (2, 200, 1500, 96)
    x, table, target, d_loss = make(case, "bf16", 7)
    plan = hyena.TokenLoss(*case, io_dtype=hyena.HYENA_BF16)

    def both():
        loss, lse = plan.forward(x, table, target)
        return (loss, lse) + plan.backward(d_loss, x, table, target, lse)

    want = both()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in sides:  # two calls of one plan at once
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(both())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(want, g))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    for _ in range(4):
        x.normal_()
        target.random_(-3, 1500)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, both()))


@pytest.mark.parametrize("tokens", [2, 4, 5, 15, 16, 17, 31, 32, 33, 64, 65, 128, 129, 257])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_kernels_of_few_tokens_at_their_limits(dtype, tokens):
    # V that is no multiple of any tile; rows made of 16-byte pieces, and not
    run((1, tokens, 777, 72), dtype, masked=0.0)
    run((1, tokens, 131, 45), dtype, masked=0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_few_tokens_of_many(dtype):
    # the call is large, what takes part is not: tiles and rows behind the last token
    for count in (0, 1, 31, 33, 128):
        x, table, target, d_loss = make((2, 300, 321, 40), dtype, 9, masked=0.0)
        flat = target.view(-1)
        flat[count:] = -1
        run((2, 300, 321, 40), dtype, inputs=(x, table, target, d_loss))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_wide_rows(dtype):
    run((1, 70, 90, 2100), dtype)
    run((1, 3, 50, 16384), dtype, masked=0.0)
    run((1, 140, 40, 16380), dtype)


@pytest.mark.parametrize("tokens", [3, 40, 5000])
def test_tables_past_32_bits(tokens):
    # 2^21 + 77 rows of 1024 in bf16 are 4.3 GB: all rows but a few are zeros, and so are their logits
    import torch
    V, d = (1 << 21) + 77, 1024
    say(f"[gpu] token_loss with a table past 32 bits, {tokens} tokens")
    gen = torch.Generator().manual_seed(3)
    at = torch.tensor([0, 5, V // 2, V - 2, V - 1])
    table = torch.zeros((V, d), dtype=torch.bfloat16, device="cuda")
    rows = torch.randn((5, d), generator=gen).bfloat16()
    table[at.cuda()] = rows.cuda()
    x = torch.randn((1, tokens, d), generator=gen).bfloat16()
    target = at[torch.arange(tokens) % 5].to(torch.int32)[None].cuda()
    plan = hyena.TokenLoss(1, tokens, V, d, io_dtype=hyena.HYENA_BF16, scale=0.2)
    loss, lse = plan.forward(x.cuda(), table, target)
    l = 0.2 * x[0].double() @ rows.double().t()
    m = l.max(-1, keepdim=True).values.clamp(min=0)
    want = (torch.exp(l - m).sum(-1) + (V - 5) * torch.exp(-m[:, 0])).log() + m[:, 0]
    assert float((lse[0].cpu().double() - want).abs().max()) < 1e-4
    hit = l[torch.arange(tokens), torch.arange(tokens) % 5]
    assert float((loss[0].cpu().double() - (want - hit)).abs().max()) < 2e-4
    if tokens > 1000:  # (G of 2^21 values would take 85 pieces)
        return
    dx, dt = plan.backward(torch.ones((1, tokens), device="cuda"), x.cuda(), table, target, lse)
    g = torch.exp(l - want[:, None])
    g[torch.arange(tokens), torch.arange(tokens) % 5] -= 1
    u = ends_ref.HALF_STEP["bf16"]
    assert float((dx[0].cpu().double() - 0.2 * g @ rows.double()).abs().max()) < 3 * u * 0.2 * float((g.abs() @ rows.double().abs()).max())
    ref = 0.2 * g.t() @ x[0].double()
    assert float((dt[at.cuda()].cpu().double() - ref).abs().max()) < 3 * u * 0.2 * float((g.abs().t() @ x[0].double().abs()).max())
    p = torch.exp(-want)  # of a row of zeros
    other = 0.2 * (p[:, None] * x[0].double()).sum(0)
    for v in (1, V // 2 + 1, V - 3):
        assert float((dt[v].cpu().double() - other).abs().max()) < 3 * u * 0.2 * float((p[:, None] * x[0].double().abs()).sum(0).max())


def test_an_infinity_in_one_token_stays_there():
    import torch
    for dtype, shape in (("bf16", (1, 200, 300, 64)), ("bf16", (1, 3, 300, 64)), ("f32", (1, 40, 300, 64))):
        x, table, target, d_loss = make(shape, dtype, 2, masked=0.0)
        plan = hyena.TokenLoss(*shape, io_dtype=IO[dtype])
        loss, lse = plan.forward(x, table, target)
        x2 = x.clone()
        x2[0, 1, 5] = float("nan")
        loss2, lse2 = plan.forward(x2, table, target)
        keep = torch.arange(shape[1], device="cuda") != 1
        assert torch.isnan(loss2[0, 1]) and torch.equal(loss[0, keep], loss2[0, keep]) and torch.equal(lse[0, keep], lse2[0, keep])
        dx, _ = plan.backward(d_loss, x, table, target, lse, want_table=False)
        dx2, _ = plan.backward(d_loss, x2, table, target, lse2, want_table=False)
        assert torch.equal(dx[0, keep], dx2[0, keep])


def test_many_tokens_in_pieces_forward():
    # the sums of 600000 tokens' tiles do not fit one piece: some of the tokens against float64
    import torch
    T, V, d = 600000, 20011, 16
    say("[gpu] token_loss forward in pieces")
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((1, T, d), generator=gen, device="cuda").bfloat16()
    table = torch.randn((V, d), generator=gen, device="cuda").bfloat16()
    target = torch.randint(-1, V, (1, T), generator=gen, device="cuda", dtype=torch.int32)
    loss, lse = hyena.TokenLoss(1, T, V, d, io_dtype=hyena.HYENA_BF16).forward(x, table, target)
    for rows in (slice(0, 1500), slice(T // 2, T // 2 + 1500), slice(T - 1500, T)):
        l = x[0, rows].double() @ table.double().t().contiguous()
        t = target[0, rows].long()
        ref = torch.where(t >= 0, torch.logsumexp(l, -1), 0)
        hit = l.gather(1, t.clamp(min=0)[:, None])[:, 0]
        assert float((lse[0, rows] - ref).abs().max()) < 1e-4
        assert float((loss[0, rows] - torch.where(t >= 0, ref - hit, 0)).abs().max()) < 2e-4


MORE = [
    # whole tiles of logits, with rims on both axes; few values and many tokens: tokens dealt out and cut
    (1, 2100, 2305, 40), (1, 130, 33000, 33), (1, 33000, 65, 17), (3, 4000, 16, 256), (1, 9000, 200, 40), (1, 2396, 277, 25),
    (2, 600, 700, 513),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", MORE)
def test_shapes_of_tiles_against_float64(case, dtype):
    import torch
    plan, x, table, target, d_loss, loss, lse = run(case, dtype)
    again = plan.forward(x, table, target) + plan.backward(d_loss, x, table, target, lse)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
    more = plan.backward(d_loss, x, table, target, lse)
    assert torch.equal(again[2], more[0]) and torch.equal(again[3], more[1])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", [(1, 6000, 33000, 256), (1, 150, 300, 96), (1, 5000, 40, 64)])
def test_gradient_of_a_row_that_all_tokens_have_as_target(case, dtype):
    # G at the target is -(1 + 0.95 u) (1 - p) for every token, and x positive: that rounding's error, u of
    # the row in every channel, must not be in it.  Behind it is u for the row's own, u^2 for
    # the rest's, and what check_grad has for the sum.
    import torch
    B, N, V, d = case
    say(f"[gpu] token_loss, one target for all {case} {dtype}")
    u = ends_ref.HALF_STEP[dtype]
    x, table, target, _ = make(case, dtype, 11, masked=0.0)
    x, table = x.abs() + 0.5, table * 0.1
    row = V * 3 // 7
    target.fill_(row)
    target[0, N // 2] = -1
    dl = float(np.float32(1 + 0.95 * u))
    d_loss = torch.full((B, N), dl, device="cuda")
    plan = hyena.TokenLoss(B, N, V, d, io_dtype=IO[dtype])
    loss, lse = plan.forward(x, table, target)
    _, dt = plan.backward(d_loss, x, table, target, lse, want_dx=False)
    live = target.view(-1).cpu().numpy() == row
    xs, ws = f64(x)[0][live], f64(table)[row]
    size = np.abs(xs) @ np.abs(ws)
    p = np.exp(xs @ ws - f64(lse)[0][live])
    g = dl * (p - 1)
    r = 2 * (d + 8) * 2.0 ** -24 * size + 2.0 ** -20 + 2.0 ** -21 * size
    dg = dl * (r * p + 2.0 ** -23) + u * u * np.abs(g) + (2.0 ** -38 if dtype == "f16" else 0.0)
    ref = g @ xs
    bound = u * np.abs(ref) + (dg + (N + 16) * 2.0 ** -24 * np.abs(g)) @ np.abs(xs)
    assert np.all((1.95 * u - 2 * u * u) * np.abs(ref) > bound)  # (the error of one rounding more would show)
    compare(dt[row], ref, bound, "d_table of the target")


def test_as_many_tokens_as_there_may_be():
    # 2^22 tokens: offsets within a tile's blocks pass 2^31.  The last ones have targets, and a few
    # before them; against products in float64 on the GPU
    import torch
    T, V, d = 1 << 22, 300, 256
    say("[gpu] token_loss of 2^22 tokens")
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((1, T, d), generator=gen, device="cuda", dtype=torch.bfloat16)
    table = (torch.randn((V, d), generator=gen, device="cuda") * 0.1).bfloat16()
    target = torch.randint(0, V, (1, T), generator=gen, device="cuda", dtype=torch.int32)
    target[0, 1000] = -1
    target[0, 5000:5900] = V
    d_loss = torch.full((1, 1), 0.77, device="cuda").expand(1, T)
    plan = hyena.TokenLoss(1, T, V, d, io_dtype=hyena.HYENA_BF16)
    loss, lse = plan.forward(x, table, target)
    dx, dt = plan.backward(d_loss, x, table, target, lse)
    w = table.double()
    wt = w.t().contiguous()
    sums = torch.zeros((V, d), dtype=torch.float64, device="cuda")
    u = ends_ref.HALF_STEP["bf16"]
    for a in range(0, T, 1 << 17):
        rows = slice(a, a + (1 << 17))
        xs, t = x[0, rows].double(), target[0, rows].long()
        live = (t >= 0) & (t < V)
        l = xs @ wt
        ref = torch.where(live, torch.logsumexp(l, -1), 0)
        assert float((lse[0, rows] - ref).abs().max()) < 2e-4
        g = torch.exp(l - lse[0, rows, None].double())
        hit = t.clamp(0, V - 1)
        assert float((loss[0, rows] - torch.where(live, ref - l.gather(1, hit[:, None])[:, 0], 0)).abs().max()) < 4e-4
        g[torch.arange(len(t), device="cuda"), hit] -= 1
        g = torch.where(live[:, None], 0.77 * g, 0)
        sums += g.t().contiguous() @ xs
        want = g @ w
        # every element of G rounded, and the result; 0.77 * 2e-4 of every probability's error in lse
        off = (dx[0, rows].double() - want).abs() - u * want.abs() - (u + 2e-4) * (g.abs() @ w.abs())
        assert float(off.max()) <= 2.0 ** -20
    off = float(torch.linalg.vector_norm(dt.double() - sums) / torch.linalg.vector_norm(sums))
    say(f"[gpu]   error norm of d_table {off:.3g}")
    assert off < 2 * u  # the norm of the errors: half a step of G and half a step of the result
