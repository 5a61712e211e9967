"""The gated linear recurrence where sizes, decays, masks and magnitudes meet:
cuts into segments, the accuracy of the gradient of g, sequences packed side by
side, states far from 1, and results that do not depend on what else is in a
call.  References: float64, token by token (mixer_ref.py); SMALL and the half
steps of the storage types as in test_gpu_recurrence.py."""
import numpy as np
import pytest

import mixer_ref
from gpu_util import say
from long_convolution_sequence_rfft_amd import hyena
from test_gpu_recurrence import IO, SMALL, Case, check_backward, check_forward, close, f64, torch_dtype

pytestmark = pytest.mark.gpu

DTYPES = ["f32", "bf16", "f16"]


# ------------------------------------------------------------- cuts into segments

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(3, 300, 43, 16, 24), (2, 300, 96, 40, 8), (1, 700, 256, 8, 16), (129, 150, 1, 8, 8),
                                   (1, 300, 128, 8, 8), (1, 300, 257, 8, 8)])
def test_rows_that_only_dq_cuts(shape, dtype):
    """Without any state coming or going, 129 to 256 rows and heads of more than 128 tokens: one segment
    for dk and dv, several for dq, which need the states before them (and the sizes on both sides)."""
    check_backward(Case(*shape, dtype, seed=sum(shape), carry=False, decay=0.05))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(3, 300, 43, 16, 24), (2, 300, 96, 40, 8)])
def test_a_state_whose_gradient_is_not_asked_for(shape, dtype):
    """The C entry with a state and neither d_final nor d_state: the other gradients are the same bits."""
    import torch
    c = Case(*shape, dtype, seed=7, decay=0.05)
    c.d_final = None
    want = c.backward()
    check_backward(c)
    view = lambda t: hyena.View(t.data_ptr(), *t.stride()[:3])  # noqa: E731
    x = hyena.RecurrenceInputs(view(c.q), view(c.k), view(c.v), view(c.g), c.state.data_ptr(), None, c.scale)
    got = [torch.full_like(t, float("nan")) for t in want[:4]]
    grads = hyena.RecurrenceGrads(*(t.data_ptr() for t in got), None)
    st = hyena.hyena_recurrence_backward(c.plan.handle, x, view(c.do), None, grads, c.plan.workspace.data_ptr(),
                                         torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == hyena.HYENA_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------- the gradient of g
#
# dg_t is summed from q_s . dq_s - k_s . dk_s over the tokens s from t to the end of its sequence, a
# token's own pair left out of both.  With W_s = exp(g_s) <|S_{s-1}|, |dS_s|>, dg's own terms without
# their signs, the two products of token s are at most W_s and W_{s+1} in size, and what leaves the row
# with d_final is W of one token more.  Each is good to SMALL of its size, so dg_t to
#   SMALL (2 sum_{s >= t, same sequence} W_s + <|S_N|, |d_final|> in the last sequence).

def dg_bound(c):
    (q, k, v, g), state, n, df = c.inputs64()
    n = np.full(c.B, c.N) if n is None else np.clip(n, 0, c.N)
    ab = [np.abs(x) for x in (f64(c.do), q, k, v)]
    state = None if state is None else np.abs(state)
    W = mixer_ref.recurrence_grad(*ab, g, abs(c.scale), state, n, None if df is None else np.abs(df))[3]
    bound = np.zeros_like(W)
    if df is not None:
        leaves = (np.abs(mixer_ref.recurrence(*ab[1:], g, 1.0, state, n)[1]) * np.abs(df)).sum((-1, -2))
    for b in range(c.B):
        over = np.zeros(c.H) if df is None else leaves[b]
        for t in range(int(n[b]) - 1, -1, -1):
            over = over + 2 * W[b, t]
            bound[b, t] = over
            over = np.where(g[b, t] * np.log2(np.e) < -126, 0.0, over)
    return SMALL * bound


def check_dg(c):
    (q, k, v, g), state, n, df = c.inputs64()
    ref = mixer_ref.recurrence_grad(f64(c.do), q, k, v, g, c.scale, state, n, df)[3]
    close(c.backward()[3], ref, dg_bound(c), "dg")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("carry", [False, True])
@pytest.mark.parametrize("shape", [(2, 60, 2, 64, 64), (2, 200, 2, 64, 64), (1, 1500, 2, 16, 24), (1, 300, 200, 8, 8)])
def test_dg_of_fast_decays(shape, carry, dtype):
    for g in (-4.0, -12.0, -20.0):
        c = Case(*shape, dtype, seed=17, carry=carry)
        c.g.fill_(g)
        check_dg(c)


# second sequence's values, as many times the first one's (binary16: scores have to stay below 65504)
LARGER = {"f32": 1000.0, "bf16": 1000.0, "f16": 30.0}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(2, 60, 2, 32, 32), (1, 420, 3, 16, 24), (1, 420, 200, 8, 8), (1, 2600, 1, 64, 64)])
def test_dg_of_a_sequence_beside_a_larger_one(shape, dtype):
    """Sequences packed into a row: a sequence's gradient has the accuracy of its own terms, whatever
    follows it.  Starts at a chunk's first token, at its last, and two in one chunk."""
    B, N = shape[:2]
    starts = (20, 41) if N < 64 else (64, 127, 130, 256, N - 100)
    c = Case(*shape, dtype, seed=23, carry=False, resets=[(t, -np.inf) for t in starts])
    for i, t in enumerate(starts):
        if i % 2 == 0:
            end = starts[i + 1] if i + 1 < len(starts) else N
            c.v[:, t:end] *= LARGER[dtype]
            c.do[:, t:end] *= LARGER[dtype]
    check_dg(c)
    c = Case(*shape, dtype, seed=24, carry=True, lengths=(N - 1,) * B, resets=[(t, -88.0) for t in starts])
    check_dg(c)


# ------------------------------------------------------------- sequences side by side

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1, 470, 2, 64, 64), (1, 470, 400, 8, 8), (2, 1900, 1, 16, 100)])
def test_infinities_stay_near_their_sequence(shape, dtype):
    """Not finite: tokens in the middle of the second of three sequences, 64 tokens and more from both of
    its ends.  More than 63 tokens before its start and after its end everything is the same bits."""
    import torch
    N = shape[1]
    start, end = 130, N - 140
    c = Case(*shape, dtype, seed=31, resets=((start, -np.inf), (end, -100.0)))
    want = [*c.forward(), *c.backward()]
    for name, value in (("q", np.nan), ("k", np.inf), ("v", -np.inf), ("do", np.nan), ("g", np.nan)):
        t = getattr(c, name)
        kept = t.clone()
        t[:, 200] = float(value)
        say(f"[gpu]   {name} = {value}")
        got = [*c.forward(), *c.backward()]
        torch.cuda.synchronize()
        t.copy_(kept)
        for a, b, what in zip(got, want, ("o", "state", "dq", "dk", "dv", "dg", "d_state")):
            if "state" in what:
                assert torch.equal(a, b), (name, what)
                continue
            assert torch.equal(a[:, :start - 63], b[:, :start - 63]), (name, what)
            assert torch.equal(a[:, end + 63:], b[:, end + 63:]), (name, what)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(2, 50, 2, 64, 64), (1, 470, 2, 40, 72), (1, 300, 200, 8, 8)])
def test_a_state_in_front_of_a_start_is_not_seen(shape, dtype):
    """A row that begins with a new sequence: an initial state of NaN gives the bits of one of zeros."""
    import torch
    c = Case(*shape, dtype, seed=32)
    c.g[:, 0] = -np.inf
    c.state.zero_()
    want = [*c.forward(), *c.backward()]
    c.state.fill_(float("nan"))
    got = [*c.forward(), *c.backward()]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not got[-1].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dv", [64, 7])
def test_step_starts_a_sequence_over_whatever_the_slot_held(dv, dtype):
    """g = -infinity, and any below -87.34, leaves nothing of a state: the bits of a state of zeros."""
    import torch
    B, H, dk = 5, 2, 24
    gen = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn((B, H, d), generator=gen).to(torch_dtype(dtype)).cuda() for d in (dk, dk, dv))
    g = torch.tensor([-np.inf, -np.inf, -88.0, -103.0, -87.4], dtype=torch.float32)[:, None].expand(B, H).cuda()
    table = torch.zeros((B, H, dk, dv), device="cuda")
    plan = hyena.Recurrence(B, 1, H, dk, dv, io_dtype=IO[dtype])
    want = plan.step(q, k, v, g, table).clone()
    states = table.clone()
    for i, left in enumerate((float("nan"), float("inf"), 3e38, -3e38, 3e38)):
        table[i] = left
    got = plan.step(q, k, v, g, table)
    assert torch.isfinite(want.float()).all()
    assert torch.equal(got, want) and torch.equal(table, states)


# ------------------------------------------------------------- what else is in a call

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(2, 40, 3, 64, 64), (1, 64, 2, 40, 72), (1, 1, 5, 128, 128), (1, 17, 2, 7, 5)])
def test_a_short_row_has_the_same_bits_in_any_batch(shape, dtype):
    import torch
    B, N, H, dk, dv = shape
    c = Case(*shape, dtype, seed=3)
    many = -(-300 // (B * H))
    d = Case(B * many, N, H, dk, dv, dtype, seed=4)
    for name in ("q", "k", "v", "g", "do", "state", "d_final"):
        getattr(d, name)[-B:] = getattr(c, name)
    for a, b in zip([*c.forward(), *c.backward()], [*d.forward(), *d.backward()]):
        assert torch.equal(a, b[-B:])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(2, 100, 2, 64, 64), (1, 128, 3, 40, 128), (1, 300, 2, 128, 128), (1, 150, 800, 8, 8)])
def test_asking_for_the_final_state_leaves_the_outputs_as_they_are(shape, dtype):
    import torch
    c = Case(*shape, dtype, seed=5)
    o = c.plan.forward(c.q, c.k, c.v, c.g, scale=c.scale, state=c.state)[0]
    assert torch.equal(o, c.forward()[0])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [2, 400])
def test_states_are_held_in_32_bits(H, dtype):
    """Values that cancel: a first token's V, what decays leave of it less its rounding to the storage
    type, and less the rounding of that.  What bfloat16 leaves of V = 1..2 is about 2^-16; a token of another
    chunk reads it.  A state of 32 bits gets there with eleven roundings of at most 2^-24 of V (V times its
    decay, the state times its, two of each for the exponentials; the two subtracted values and their
    decays): below 2^-19.  Reading rounds the state and the result to the storage type."""
    import torch
    N, d = 192, 8
    say(f"[gpu] cancelling states H={H} {dtype}")
    dt, u = torch_dtype(dtype), mixer_ref.HALF_STEP[dtype]
    gen = torch.Generator().manual_seed(6)
    for reverse in (False, True):
        # e: the direction in which everything is; other keys and queries are 0
        g = torch.full((1, N, H), -0.013)
        V = (1 + torch.rand((1, H, d), generator=gen)).to(dt).double()
        at = (3, 70, 90, 180)          # a chunk of its own, two of the next, the reader in a third
        if reverse:
            at = tuple(N - 1 - t for t in at)
        write, read = torch.zeros((1, N, H, d), dtype=dt), torch.zeros((1, N, H, d), dtype=dt)
        write[:, at[0]] = V.to(dt)
        # decay from token i to a later one (reversed: earlier) is the sum of g between
        gd = g.double()
        left = V
        for i in (1, 2):
            left = left * torch.exp(gd[:, 0] * abs(at[i] - at[i - 1]))[..., None]
            write[:, at[i]] = -left.to(dt)
            left = left + write[:, at[i]].double()
        left = left * torch.exp(gd[:, 0] * abs(at[3] - at[2]))[..., None]
        one = torch.zeros((1, N, H, d), dtype=dt)
        for t in at[:3]:
            one[:, t, :, 0] = 1.0
        read[:, at[3], :, 0] = 1.0
        plan = hyena.Recurrence(1, N, H, d, d, io_dtype=IO[dtype], training=True)
        one, read, write, gg = (t.cuda() for t in (one, read, write, g))
        if not reverse:  # o of the reader
            got = plan.forward(read, one, write, gg, scale=1.0)[0][:, at[3]]
        else:            # dv of the reader, from do of the writers
            got = plan.backward(write, one, read, torch.zeros_like(write), gg, scale=1.0)[2][:, at[3]]
        ref = left.numpy()
        close(got, ref, 2 * u * np.abs(ref) + 2.0 ** -19 + (2.0 ** -25 if dtype == "f16" else 0.0), f"reverse={reverse}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(2, 65, 2, 64, 64), (1, 200, 3, 128, 128), (2, 330, 2, 40, 72), (1, 300, 2, 128, 64),
                                   (1, 900, 2, 64, 128), (1, 140, 300, 7, 5)])
@pytest.mark.parametrize("decay", [0.5, 0.01])
def test_rows_of_any_length_round_only_their_results(shape, decay, dtype):
    """No score and no state is rounded to 16 bits on the way: half a step of the value, and 2^-15 of the
    sum of absolute values (float32's 2^-15 less what its sums really lose leaves 2^-16 for scores and bfloat16
    states of two terms)."""
    c = Case(*shape, dtype, seed=sum(shape) + 4, decay=decay, resets=((70, -np.inf),))
    (q, k, v, g), state, n, df = c.inputs64()
    u, do = mixer_ref.HALF_STEP[dtype], f64(c.do)
    least = 2.0 ** -25 if dtype == "f16" else 0.0  # half a step of the smallest float16 results
    ro, _, ao, _ = mixer_ref.recurrence(q, k, v, g, c.scale, state, n)
    close(c.forward()[0], ro, u * np.abs(ro) + SMALL * ao + least, "o")
    ref = mixer_ref.recurrence_grad(do, q, k, v, g, c.scale, state, n, df)
    size = mixer_ref.recurrence_grad(*(np.abs(x) for x in (do, q, k, v)), g, c.scale, np.abs(state), n, np.abs(df))
    for got, r, a, what in zip(c.backward()[:3], ref, size, ("dq", "dk", "dv")):
        close(got, r, u * np.abs(r) + SMALL * a + least, what)


# ------------------------------------------------------------- magnitudes

@pytest.mark.parametrize("N", [50, 200])
@pytest.mark.parametrize("size", [2.0 ** -20, 2.0 ** -30, 2.0 ** 20])
@pytest.mark.parametrize("dtype", DTYPES)
def test_states_and_their_gradients_far_from_one(size, N, dtype):
    """Everything comes from the initial state (v = 0) and from d_final (do = 0), so that no score
    takes part; other operands around 64, so that 16-bit results are in their range.  One column of the
    state is 2^10 times the others."""
    import torch
    c = Case(2, N, 2, 24, 40, dtype, seed=9, decay=0.02)
    for t, by in ((c.state, size), (c.d_final, size), (c.v, 0.0), (c.do, 0.0)):
        t.mul_(by)
    c.state[..., 5] *= 1024.0
    c.d_final[..., 7] *= 1024.0
    for t in (c.q, c.k):
        t.mul_(64.0)
    if dtype == "f16" and size > 1:
        # o is q (64) times the largest column (2^30) summed over 24 channels, about 2^38: below 65504
        c.scale = 2.0 ** -30
    (q, k, v, g), state, n, df = c.inputs64()
    u = mixer_ref.HALF_STEP[dtype]
    least = 2.0 ** -25 if dtype == "f16" else 0.0  # half a step of the smallest float16 results
    o, last = c.forward()
    ro, rs, ao, as_ = mixer_ref.recurrence(q, k, v, g, c.scale, state, n)
    # bfloat16 reads the state rounded once
    held = u if dtype == "bf16" and N > 64 else 0.0
    close(o, ro, u * np.abs(ro) + (held + SMALL) * ao + least, "o")
    close(last, rs, SMALL * as_ + 1e-30, "state")
    if dtype == "f16" and size > 1:
        return  # gradients above float16's largest
    # dk is dS v: values for it alone
    c.v.copy_(64.0 * torch.randn(c.v.shape, generator=torch.Generator().manual_seed(10)))
    c.state.zero_()
    (q, k, v, g), state, n, df = c.inputs64()
    dq, dk, dv, dg, ds = c.backward()
    ref = mixer_ref.recurrence_grad(f64(c.do), q, k, v, g, c.scale, state, n, df)
    a = mixer_ref.recurrence_grad(np.abs(f64(c.do)), *(np.abs(x) for x in (q, k, v)), g, abs(c.scale), state, n, np.abs(df))
    assert not dq.any()
    close(dk, ref[1], u * np.abs(ref[1]) + SMALL * a[1] + least, "dk")
    close(dv, ref[2], u * np.abs(ref[2]) + (held + SMALL) * a[2] + least, "dv")
    close(ds, ref[4], SMALL * a[4] + 1e-30, "d_state")
    close(dg, ref[3], dg_bound(c), "dg")


@pytest.mark.parametrize("N", [30, 60])
@pytest.mark.parametrize("dtype", DTYPES)
def test_states_that_have_decayed_far(N, dtype):
    """One token, then nothing but decays of e^-1: down to e^-59 the state has the accuracy of its size, and
    so has the gradient of the initial state, which comes from the last token alone."""
    c = Case(2, N, 2, 24, 40, dtype, seed=12)
    c.g.fill_(-1.0)
    c.g[:, 5] = -np.inf
    c.v[:, 1:].zero_()
    c.v[:, 5].normal_()
    (q, k, v, g), state, n, df = c.inputs64()
    _, last = c.forward()
    _, rs, _, as_ = mixer_ref.recurrence(q, k, v, g, c.scale, state, n)
    close(last, rs, SMALL * as_, "state")
    c.g[:, 5] = -1.0
    c.do[:, :-1].zero_()
    c.d_final.zero_()
    (q, k, v, g), state, n, df = c.inputs64()
    ds = c.backward()[4]
    grad = lambda x, y: mixer_ref.recurrence_grad(x, y, k, v, g, c.scale, state, n, df)[4]  # noqa: E731
    close(ds, grad(f64(c.do), q), SMALL * grad(np.abs(f64(c.do)), np.abs(q)), "d_state")


# ------------------------------------------------------------- where outputs may lie

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("widths", [(5, 7), (16, 8)])
def test_float32_outputs_and_tables_at_any_element(widths, dtype):
    """States, their gradients and dg may start at any float32: a slice of a pool of states."""
    import torch
    dk, dv = widths
    c = Case(1, 150, 1, dk, dv, dtype, seed=10)
    o, last = c.forward()
    pool = torch.full((2 + dk * dv,), 7.0, device="cuda")
    mine = pool[1:1 + dk * dv].view(1, 1, dk, dv)
    o2, last2 = c.forward(final_state=mine)
    assert last2 is mine and torch.equal(o, o2) and torch.equal(last, mine)
    assert pool[0] == 7.0 and pool[-1] == 7.0
    # the backward pass through the C entry
    want = c.backward()
    view = lambda t: hyena.View(t.data_ptr(), *t.stride()[:3])  # noqa: E731
    x = hyena.RecurrenceInputs(view(c.q), view(c.k), view(c.v), view(c.g), c.state.data_ptr(), None, c.scale)
    got = [torch.empty_like(t) for t in want[:3]]
    floats = torch.full((1 + 150 + 1 + dk * dv + 1,), 7.0, device="cuda")
    dg, ds = floats[1:151], floats[152:152 + dk * dv]
    assert dg.data_ptr() % 16 and ds.data_ptr() % 4 == 0
    grads = hyena.RecurrenceGrads(*(t.data_ptr() for t in got), dg.data_ptr(), ds.data_ptr())
    st = hyena.hyena_recurrence_backward(c.plan.handle, x, view(c.do), c.d_final.data_ptr(), grads,
                                         c.plan.workspace.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == hyena.HYENA_OK
    assert torch.equal(dg, want[3].flatten()) and torch.equal(ds, want[4].flatten())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert floats[0] == 7.0 and floats[151] == 7.0 and floats[-1] == 7.0
    # one token on a table that is a slice of a pool
    one = hyena.Recurrence(1, 1, 1, dk, dv, io_dtype=IO[dtype])
    token = [t[:, 3] for t in (c.q, c.k, c.v, c.g)]
    table = torch.randn((3, 1, dk, dv), device="cuda")
    whole = torch.zeros(1 + 3 * dk * dv, device="cuda")
    part = whole[1:].view(3, 1, dk, dv)
    part.copy_(table)
    slots = torch.tensor([2], dtype=torch.int32, device="cuda")
    a, b = one.step(*token, table, slots=slots), one.step(*token, part, slots=slots)
    # (rows may be read in another order)
    close(b, f64(a), 2 * mixer_ref.HALF_STEP[dtype] * np.abs(f64(a)) + SMALL * np.abs(f64(table[2])).sum(1) * 20, "o")
    assert torch.equal(part, table) and whole[0] == 0.0
