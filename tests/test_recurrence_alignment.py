"""Alignment of the recurrence's outputs in the C ABI.  Every call here is
refused before any GPU work, so the addresses are never used."""
from long_convolution_sequence_rfft_amd import hyena
from test_mixer_checks import INVALID, inputs, plan, ptr  # noqa: F401


def test_forward_outputs(plan):  # noqa: F811
    x, o, last, ws = inputs(state=ptr(4)), ptr(10), ptr(11), ptr(12)
    for at in (2, 4, 8):
        assert hyena.hyena_recurrence_forward(plan, x, o + at, last, ws) == INVALID
        assert "o must be 16-byte aligned" in hyena.hyena_last_error()
    for at in (1, 2):
        assert hyena.hyena_recurrence_forward(plan, x, o, last + at, ws) == INVALID
        assert "final_state is not aligned to its element" in hyena.hyena_last_error()


def test_backward_outputs(plan):  # noqa: F811
    x, ws, d = inputs(state=ptr(4)), ptr(12), hyena.View(ptr(13), 14400, 48, 16)
    for i, name in enumerate(("dq", "dk", "dv", "dg", "d_state")):
        outs = [ptr(20 + j) for j in range(5)]
        outs[i] += 8 if i < 3 else 2
        assert hyena.hyena_recurrence_backward(plan, x, d, None, hyena.RecurrenceGrads(*outs), ws) == INVALID
        text = "must be 16-byte aligned" if i < 3 else "is not aligned to its element"
        assert f"{name} {text}" in hyena.hyena_last_error()


def test_step_outputs(plan):  # noqa: F811
    assert hyena.hyena_recurrence_step(plan, inputs(), None, 2, ptr(10) + 2, ptr(11)) == INVALID
    assert "states is not aligned to its element" in hyena.hyena_last_error()
    assert hyena.hyena_recurrence_step(plan, inputs(), None, 2, ptr(10), ptr(11) + 8) == INVALID
    assert "o must be 16-byte aligned" in hyena.hyena_last_error()
