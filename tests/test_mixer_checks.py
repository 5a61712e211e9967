"""Refusals of the gated linear recurrence and of the query/key norm, in the C
ABI and in the torch wrapper.  Every call here is refused before any GPU work,
so the addresses are never used and the tensors are host memory."""
import ctypes

import pytest
import torch

from long_convolution_sequence_rfft_amd import hyena

INVALID, UNSUPPORTED = hyena.HYENA_ERR_INVALID_ARGUMENT, hyena.HYENA_ERR_UNSUPPORTED


def ptr(i):
    """Aligned, distinct addresses 4 GiB apart."""
    return (1 << 40) + i * (1 << 32)


@pytest.mark.parametrize("args,code", [
    ((0, 8, 2, 4, 4), INVALID), ((1, 0, 2, 4, 4), INVALID), ((1, 8, 0, 4, 4), INVALID), ((1, 8, 2, 0, 4), INVALID),
    ((1, 8, 2, 4, -1), INVALID), ((1, 8, 2, 129, 4), UNSUPPORTED), ((1, 8, 2, 4, 129), UNSUPPORTED),
    ((1, 1 << 31, 2, 4, 4), UNSUPPORTED), ((1 << 13, 8, 1 << 12, 4, 4), UNSUPPORTED),
    ((1, 8, 65537, 4, 4), UNSUPPORTED), (((1 << 22) + 1, 8, 1, 4, 4), UNSUPPORTED),
    ((1 << 62, 8, 4, 4, 4), UNSUPPORTED), ((1, 8, 2, 4, 4, 3), UNSUPPORTED), ((1, 8, 2, 4, 4, -1), UNSUPPORTED),
])
def test_recurrence_plans(args, code):
    st, plan = hyena.hyena_recurrence_create(*args, check=False)
    assert st == code and plan is None
    assert "recurrence" in hyena.hyena_last_error()


def test_recurrence_largest_plans():
    for args in ((1 << 22, 1, 1, 128, 128), (1 << 6, 8, 1 << 16, 1, 1), (1, (1 << 31) - 65, 1, 1, 1)):
        _, plan = hyena.hyena_recurrence_create(*args)
        hyena.hyena_recurrence_destroy(plan)


def test_recurrence_null_plan_and_sizes():
    lib = hyena.load()
    assert lib.hyena_recurrence_create(None, 1, 8, 1, 4, 4, 0) == INVALID
    assert lib.hyena_recurrence_query(None, None, None) == INVALID
    assert hyena.hyena_recurrence_forward(None, None, ptr(0), None, None) == INVALID
    assert hyena.hyena_recurrence_backward(None, None, None, None, None, None) == INVALID
    assert hyena.hyena_recurrence_step(None, None, None, 1, ptr(0), ptr(1)) == INVALID
    assert hyena.hyena_recurrence_destroy(None) == hyena.HYENA_OK
    # one segment needs no forward workspace; several hold their states and decays
    _, p = hyena.hyena_recurrence_create(1, 64, 2, 16, 16)
    assert hyena.hyena_recurrence_query(p)[0] == 0
    hyena.hyena_recurrence_destroy(p)
    _, p = hyena.hyena_recurrence_create(1, 65536, 12, 64, 64)
    fwd, bwd = hyena.hyena_recurrence_query(p)
    assert 12 * 64 * 64 * 4 * 2 <= fwd <= bwd
    assert lib.hyena_recurrence_query(p, None, None) == hyena.HYENA_OK
    hyena.hyena_recurrence_destroy(p)


def inputs(**kw):
    """Valid inputs of a plan with B 2, N 300, heads 3, dk 8, dv 16, float32."""
    v = lambda i, d: hyena.View(ptr(i), 300 * 3 * d, 3 * d, d)  # noqa: E731
    x = hyena.RecurrenceInputs(v(0, 8), v(1, 8), v(2, 16), v(3, 1), None, None, 1.0)
    for name, value in kw.items():
        setattr(x, name, value)
    return x


@pytest.fixture
def plan():
    _, p = hyena.hyena_recurrence_create(2, 300, 3, 8, 16)
    yield p
    hyena.hyena_recurrence_destroy(p)


BAD_INPUTS = [
    dict(q=hyena.View(None, 7200, 24, 8)), dict(k=hyena.View(ptr(1) + 2, 7200, 24, 8)),
    dict(v=hyena.View(ptr(2), -1, 48, 16)), dict(g=hyena.View(ptr(3), 900, 3, -1)), dict(g=hyena.View(None, 0, 0, 0)),
    dict(state=ptr(4) + 1), dict(lengths=ptr(5) + 2),
]


def test_recurrence_token_strides(plan):
    far = hyena.View(ptr(0), 1 << 34, 1 << 23, 8)
    for name in ("q", "k", "v", "g"):
        x = inputs(**{name: far})
        assert hyena.hyena_recurrence_forward(plan, x, ptr(6), None, ptr(7)) == UNSUPPORTED
        assert name + " has a token stride" in hyena.hyena_last_error()
    out = hyena.RecurrenceGrads(ptr(8), ptr(9), ptr(10), ptr(11), None)
    assert hyena.hyena_recurrence_backward(plan, inputs(), far, None, out, ptr(7)) == UNSUPPORTED


@pytest.mark.parametrize("bad", BAD_INPUTS)
def test_recurrence_inputs(plan, bad):
    o, ws, d = ptr(10), ptr(11), hyena.View(ptr(12), 14400, 48, 16)
    grads = hyena.RecurrenceGrads(ptr(13), ptr(14), ptr(15), ptr(16), None)
    assert hyena.hyena_recurrence_forward(plan, inputs(**bad), o, None, ws) == INVALID
    assert hyena.hyena_recurrence_backward(plan, inputs(**bad), d, None, grads, ws) == INVALID
    if "state" not in bad and "lengths" not in bad:
        assert hyena.hyena_recurrence_step(plan, inputs(**bad), None, 2, ptr(13), o) == INVALID


def test_recurrence_forward_buffers(plan):
    x, o, last, ws = inputs(state=ptr(4)), ptr(10), ptr(11), ptr(12)
    call = lambda *a: hyena.hyena_recurrence_forward(plan, *a)  # noqa: E731
    assert call(None, o, last, ws) == INVALID
    assert call(x, None, last, ws) == INVALID
    assert call(x, o, last, None) == INVALID
    assert call(x, o, last, ws + 4) == INVALID
    assert call(x, o + 4, last, ws) == INVALID
    assert call(x, x.q.data + 16, last, ws) == INVALID          # o on q
    assert "overlaps" in hyena.hyena_last_error()
    assert call(x, o, o + 64, ws) == INVALID                    # the state on o
    assert call(x, o, x.state, ws) == INVALID                   # the final state on the initial one
    assert call(x, o, ws + 16, ws) == INVALID                   # on the workspace
    assert call(x, o, x.q.data - 16, ws) == INVALID             # reaching into q


def test_recurrence_backward_buffers(plan):
    x, ws, d = inputs(state=ptr(4)), ptr(12), hyena.View(ptr(13), 14400, 48, 16)
    outs = [ptr(20 + i) for i in range(5)]
    call = lambda x, d, df, o, ws: hyena.hyena_recurrence_backward(  # noqa: E731
        plan, x, d, df, None if o is None else hyena.RecurrenceGrads(*o), ws)
    assert call(None, d, None, outs, ws) == INVALID
    assert call(x, None, None, outs, ws) == INVALID
    assert call(x, hyena.View(None, 0, 0, 0), None, outs, ws) == INVALID
    assert call(x, d, ptr(14) + 1, outs, ws) == INVALID
    assert call(x, d, None, None, ws) == INVALID
    assert call(x, d, None, outs, None) == INVALID
    for i in range(4):
        assert call(x, d, None, outs[:i] + [None] + outs[i + 1:], ws) == INVALID
        assert call(x, d, None, outs[:i] + [outs[4] + 16] + outs[i + 1:], ws) == INVALID
        assert call(x, d, None, outs[:i] + [d.data] + outs[i + 1:], ws) == INVALID
    assert call(x, d, outs[4], outs, ws) == INVALID


def test_recurrence_step_buffers(plan):
    x, states, o = inputs(), ptr(10), ptr(11)
    call = lambda *a: hyena.hyena_recurrence_step(plan, *a)  # noqa: E731
    assert call(None, None, 2, states, o) == INVALID
    assert call(x, None, 1, states, o) == INVALID               # two rows, one state
    assert call(x, ptr(12), 0, states, o) == INVALID
    assert call(x, ptr(12), 1 << 31, states, o) == INVALID
    assert call(x, ptr(12) + 1, 2, states, o) == INVALID
    assert call(x, None, 2, None, o) == INVALID
    assert call(x, None, 2, states, None) == INVALID
    assert call(x, None, 2, states, states + 16) == INVALID
    assert call(x, None, 2, x.v.data, o) == INVALID


def qk(**kw):
    op = hyena.QkNorm(2, 10, 4, 2, 32, hyena.HYENA_F32, hyena.HYENA_NORM_RMS, hyena.HYENA_ROTARY_HALF, 16, 1e-6, 1.0,
                      ptr(0), ptr(1), ptr(2), ptr(3), 0, hyena.View(ptr(4), 1280, 128, 32), hyena.View(ptr(5), 640, 64, 32))
    for name, value in kw.items():
        setattr(op, name, value)
    return op


@pytest.mark.parametrize("bad,code", [
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(q_heads=0), INVALID), (dict(k_heads=-1), INVALID),
    (dict(D=0), INVALID), (dict(D=1025), UNSUPPORTED), (dict(q_heads=4097), UNSUPPORTED), (dict(k_heads=4097), UNSUPPORTED),
    (dict(B=1 << 20, N=1 << 20), UNSUPPORTED), (dict(B=1 << 62), UNSUPPORTED), (dict(io_dtype=3), UNSUPPORTED),
    (dict(norm=3), UNSUPPORTED), (dict(layout=2), UNSUPPORTED), (dict(rotary_dim=15), INVALID),
    (dict(rotary_dim=34), INVALID), (dict(rotary_dim=-2), INVALID), (dict(freqs=None), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
])
def test_qk_norm_descriptions(bad, code):
    d = hyena.View(ptr(10), 1280, 128, 32), hyena.View(ptr(11), 640, 64, 32)
    assert hyena.hyena_qk_norm_forward(qk(**bad), ptr(6), ptr(7)) == code
    assert hyena.hyena_qk_norm_scratch_bytes(qk(**bad))[0] == code
    assert hyena.hyena_qk_norm_backward(qk(**bad), *d, ptr(6), ptr(7), None, None, None) == code


def test_qk_norm_buffers():
    fwd = lambda op, q, k: hyena.hyena_qk_norm_forward(op, q, k)  # noqa: E731
    q, k = ptr(6), ptr(7)
    for bad in (dict(q=hyena.View(None, 0, 0, 0)), dict(k=hyena.View(ptr(5) + 1, 640, 64, 32)),
                dict(q=hyena.View(ptr(4), 1280, -128, 32)), dict(freqs=ptr(0) + 4), dict(q_weight=ptr(1) + 2),
                dict(k_weight=ptr(1) + 1), dict(positions=ptr(3) + 2)):
        assert fwd(qk(**bad), q, k) == INVALID
    assert fwd(None, q, k) == INVALID
    assert fwd(qk(), None, k) == INVALID
    assert fwd(qk(), q, None) == INVALID
    assert fwd(qk(), q + 8, k) == INVALID
    assert fwd(qk(), q, q + 16) == INVALID
    assert fwd(qk(), ptr(4), k) == INVALID          # in place
    assert fwd(qk(), q, ptr(3)) == INVALID          # on the positions
    assert hyena.load().hyena_qk_norm_scratch_bytes(ctypes.byref(qk()), None) == INVALID
    st, n = hyena.hyena_qk_norm_scratch_bytes(qk())
    assert st == hyena.HYENA_OK and n >= 2 * 32 * 4
    d = hyena.View(ptr(10), 1280, 128, 32), hyena.View(ptr(11), 640, 64, 32)
    back = lambda op, dq, dk, *a: hyena.hyena_qk_norm_backward(op, dq, dk, *a)  # noqa: E731
    assert back(qk(), None, d[1], q, k, None, None, None) == INVALID
    assert back(qk(), d[0], None, q, k, None, None, None) == INVALID
    assert back(qk(), *d, q, d[1].data, None, None, None) == INVALID
    assert back(qk(), *d, q, k, ptr(12), None, None) == INVALID             # no scratch
    assert back(qk(), *d, q, k, ptr(12), ptr(12), ptr(13)) == INVALID
    assert back(qk(), *d, q, k, ptr(12), ptr(14), ptr(12) - 256) == INVALID
    assert back(qk(), *d, q, k, ptr(12) + 2, None, ptr(13)) == INVALID
    assert back(qk(norm=hyena.HYENA_NORM_NONE), *d, q, k, ptr(12), None, ptr(13)) == INVALID


# ---------------------------------------------------------------- torch wrapper

def on_host(cls, **fields):
    """A plan bound to host memory: its checks run, no call of it is let through."""
    p = object.__new__(cls)
    p.torch, p.device, p.handle = torch, torch.device("cpu"), None
    for name, value in fields.items():
        setattr(p, name, value)
    return p


def host_recurrence(training=True):
    return on_host(hyena.Recurrence, B=2, N=20, heads=3, dk=8, dv=16, dtype=torch.float32, io_dtype=hyena.HYENA_F32,
                   training=training, workspace=None)


def rec_tensors():
    return dict(q=torch.zeros(2, 20, 3, 8), k=torch.zeros(2, 20, 3, 8), v=torch.zeros(2, 20, 3, 16), g=torch.zeros(2, 20, 3))


BAD_TENSORS = [
    dict(q=torch.zeros(2, 20, 3, 7)), dict(k=torch.zeros(2, 20, 3, 8, dtype=torch.bfloat16)), dict(v=torch.zeros(2, 19, 3, 16)),
    dict(v=torch.zeros(2, 20, 16, 3).transpose(2, 3)), dict(g=torch.zeros(2, 20, 3, dtype=torch.float64)), dict(q=None),
    dict(g=torch.zeros(2, 20, 3, 1)), dict(q=[1.0]), dict(state=torch.zeros(2, 3, 16, 8)),
    dict(state=torch.zeros(2, 3, 16, 8).transpose(2, 3)), dict(state=torch.zeros(2, 3, 8, 16, dtype=torch.bfloat16)),
    dict(lengths=torch.zeros(2, dtype=torch.int64)), dict(lengths=torch.zeros(3, dtype=torch.int32)),
    dict(lengths=torch.zeros(4, dtype=torch.int32)[::2]),
]


@pytest.mark.parametrize("bad", BAD_TENSORS)
def test_recurrence_rejects_bad_tensors(bad):
    p = host_recurrence()
    with pytest.raises(ValueError):
        p.forward(**{**rec_tensors(), **bad})
    with pytest.raises(ValueError):
        p.backward(torch.zeros(2, 20, 3, 16), **{**rec_tensors(), **bad})


def test_recurrence_rejects_bad_outputs_and_gradients():
    p = host_recurrence()
    x = rec_tensors()
    for kw in (dict(o=torch.zeros(2, 20, 3, 8)), dict(o=torch.zeros(2, 3, 20, 16).transpose(1, 2)),
               dict(final_state=torch.zeros(2, 3, 8, 15))):
        with pytest.raises(ValueError):
            p.forward(**x, **kw)
    with pytest.raises(ValueError):
        p.backward(torch.zeros(2, 20, 3, 8), **x)
    with pytest.raises(ValueError):
        p.backward(torch.zeros(2, 20, 3, 16), **x, d_final=torch.zeros(2, 3, 16, 8))
    with pytest.raises(ValueError, match="training"):
        host_recurrence(training=False).backward(torch.zeros(2, 20, 3, 16), **x)


def test_step_rejects_bad_tensors():
    p = host_recurrence()
    x = [torch.zeros(2, 3, 8), torch.zeros(2, 3, 8), torch.zeros(2, 3, 16), torch.zeros(2, 3)]
    good = torch.zeros(4, 3, 8, 16)
    for bad in (torch.zeros(4, 3, 16, 8), torch.zeros(4, 3, 8), None, good.to(torch.bfloat16), good.transpose(0, 1)):
        with pytest.raises(ValueError):
            p.step(*x, bad)
    for i, t in enumerate((torch.zeros(2, 3, 9), torch.zeros(2, 1, 3, 8), torch.zeros(3, 3, 16), torch.zeros(()))):
        with pytest.raises(ValueError):
            p.step(*x[:i], t, *x[i + 1:], good)
    with pytest.raises(ValueError):
        p.step(*x, good, slots=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        p.step(*x, good, o=torch.zeros(2, 3, 8))


def host_norm():
    return on_host(hyena.QKNorm, B=2, N=5, q_heads=4, k_heads=2, D=16, dtype=torch.float32, io_dtype=hyena.HYENA_F32,
                   norm="rms", layout="half", rotary_dim=8, eps=1e-6, rotary_scale=1.0, scratch_bytes=1024,
                   freqs=hyena.rotary_frequencies(8, device="cpu"))


@pytest.mark.parametrize("bad", [
    dict(q=torch.zeros(2, 5, 2, 16)), dict(k=torch.zeros(2, 5, 2, 16, dtype=torch.float16)), dict(q=None),
    dict(k=torch.zeros(2, 5, 16, 2).transpose(2, 3)), dict(q_weight=torch.zeros(15)),
    dict(k_weight=torch.zeros(16, dtype=torch.bfloat16)), dict(positions=torch.zeros(2, 5, dtype=torch.int64)),
    dict(positions=torch.zeros(5, dtype=torch.int32)),
])
def test_qk_norm_rejects_bad_tensors(bad):
    x = dict(q=torch.zeros(2, 5, 4, 16), k=torch.zeros(2, 5, 2, 16))
    p = host_norm()
    with pytest.raises(ValueError):
        p.forward(**{**x, **bad})
    with pytest.raises(ValueError):
        p.backward(x["q"], x["k"], **{**x, **bad})


def test_qk_norm_rejects_bad_outputs_and_gradients():
    p = host_norm()
    q, k = torch.zeros(2, 5, 4, 16), torch.zeros(2, 5, 2, 16)
    with pytest.raises(ValueError):
        p.forward(q, k, q_out=torch.zeros(2, 5, 4, 15))
    with pytest.raises(ValueError):
        p.backward(k, k, q, k)
    with pytest.raises(ValueError):
        p.backward(q, q, q, k)


def test_plans_refuse_other_devices_types_and_names():
    with pytest.raises(ValueError, match="GPU"):
        hyena.Recurrence(1, 8, 1, 4, 4, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        hyena.QKNorm(1, 8, 1, 1, 4, device="cpu")
    with pytest.raises(ValueError, match="dtype"):
        hyena.Recurrence(1, 8, 1, 4, 4, io_dtype=7)
    for kw in (dict(norm="layer"), dict(layout="quarter"), dict(rotary_dim=5), dict(rotary_dim=20)):
        p = on_host(hyena.QKNorm)
        p._place = lambda *a: None
        with pytest.raises(ValueError):
            p.__init__(1, 8, 1, 1, 16, **kw)


def test_rotary_frequencies():
    f = hyena.rotary_frequencies(8, base=16.0, stretch=2.0, device="cpu")
    assert f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([0.5, 0.25, 0.125, 0.0625], dtype=torch.float64), rtol=1e-15, atol=0.0)
    assert hyena.rotary_frequencies(0, device="cpu").numel() == 0
