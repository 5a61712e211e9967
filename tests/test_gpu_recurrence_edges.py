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
