"""Refusals of the embedding, the norm of whole tokens and the loss over a
vocabulary, in the C ABI and in the torch wrapper.  Every call here is refused
before any GPU work, so the addresses are never used and the tensors are host
memory."""
import ctypes

import pytest
import torch

from long_convolution_sequence_rfft_amd import hyena

INVALID, UNSUPPORTED = hyena.HYENA_ERR_INVALID_ARGUMENT, hyena.HYENA_ERR_UNSUPPORTED


def ptr(i):
    """Aligned, distinct addresses 4 GiB apart."""
    return (1 << 40) + i * (1 << 32)


def changed(op, kw):
    for name, value in kw.items():
        setattr(op, name, value)
    return op


def embedding(**kw):
    return changed(hyena.EmbeddingOp(2, 30, 100, 48, 1, 1.0, hyena.Rows(ptr(0), 30, 1)), kw)


def norm(**kw):
    return changed(hyena.ResidualNormOp(2, 30, 128, 1, 0, 0, 1e-6, ptr(1), hyena.Rows(ptr(0), 30 * 128, 128),
                                        hyena.Rows(ptr(2), 30 * 128, 128)), kw)


def loss(**kw):
    return changed(hyena.TokenLossOp(2, 30, 100, 48, 1, 1.0, hyena.Rows(ptr(0), 30 * 48, 48), ptr(1),
                                     hyena.Rows(ptr(2), 30, 1)), kw)


SIZES = [
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(d=0), INVALID), (dict(B=-1), INVALID), (dict(io_dtype=3), UNSUPPORTED),
    (dict(io_dtype=-1), UNSUPPORTED), (dict(d=1 << 20), UNSUPPORTED), (dict(B=1 << 20, N=1 << 20), UNSUPPORTED),
    (dict(B=1 << 62), UNSUPPORTED), (dict(N=1 << 33), UNSUPPORTED),
]


@pytest.mark.parametrize("bad,code", SIZES)
def test_sizes(bad, code):
    d = hyena.Rows(ptr(5), 30 * 48, 48)
    assert hyena.hyena_embedding_scratch_bytes(embedding(**bad))[0] == code
    assert "embedding" in hyena.hyena_last_error()
    assert hyena.hyena_embedding_forward(embedding(**bad), ptr(3), ptr(4)) == code
    assert hyena.hyena_embedding_backward(embedding(**bad), d, ptr(3), 0, ptr(4)) == code
    assert hyena.hyena_residual_norm_scratch_bytes(norm(**bad))[0] == code
    assert "residual norm" in hyena.hyena_last_error()
    assert hyena.hyena_residual_norm_forward(norm(**bad), ptr(3), ptr(4), None) == code
    assert hyena.hyena_residual_norm_backward(norm(**bad), d, None, ptr(3), None, None) == code
    assert hyena.hyena_token_loss_scratch_bytes(loss(**bad))[0] == code
    assert "token loss" in hyena.hyena_last_error()
    assert hyena.hyena_token_loss_forward(loss(**bad), ptr(3), ptr(4), ptr(6)) == code
    assert hyena.hyena_token_loss_backward(loss(**bad), d, ptr(3), ptr(4), ptr(6), ptr(7)) == code


def test_vocabularies_and_null_descriptions():
    for V, code in ((0, INVALID), (-5, INVALID), ((1 << 24) + 1, UNSUPPORTED)):
        assert hyena.hyena_embedding_scratch_bytes(embedding(V=V))[0] == code
        assert hyena.hyena_token_loss_scratch_bytes(loss(V=V))[0] == code
    assert hyena.hyena_embedding_scratch_bytes(embedding(V=1 << 24))[0] == 0
    assert hyena.hyena_token_loss_scratch_bytes(loss(V=1 << 22))[0] == 0
    lib = hyena.load()
    assert lib.hyena_embedding_scratch_bytes(None, None) == INVALID
    assert lib.hyena_residual_norm_scratch_bytes(None, None) == INVALID
    assert lib.hyena_token_loss_scratch_bytes(None, None, None) == INVALID
    assert lib.hyena_embedding_scratch_bytes(ctypes.byref(embedding()), None) == INVALID
    assert lib.hyena_residual_norm_scratch_bytes(ctypes.byref(norm()), None) == INVALID
    assert lib.hyena_token_loss_scratch_bytes(ctypes.byref(loss()), None, None) == hyena.HYENA_OK


def test_scratch_sizes():
    # largest calls of each limit still have a size that fits, and grow with the call
    n = [hyena.hyena_embedding_scratch_bytes(embedding(B=1, N=k, V=1 << 24, d=65536))[1] for k in (1, 1 << 20, 1 << 30)]
    assert 0 < n[0] < n[1] < n[2] < 1 << 44
    n = [hyena.hyena_token_loss_scratch_bytes(loss(B=1, N=k, V=1 << 22, d=16384, io_dtype=0))[1:] for k in (1, 1 << 12, 1 << 22)]
    assert n[0][0] < n[1][0] < n[2][0] < 1 << 50 and n[0][1] < n[1][1] < n[2][1] < 1 << 50
    # G is made in pieces: the logits would take this much in 16 bits
    assert hyena.hyena_token_loss_scratch_bytes(loss(B=2, N=8192, V=50257, d=768))[2] < 2 * 16384 * 50257
    assert hyena.hyena_token_loss_scratch_bytes(loss(B=8, N=8192, V=131072, d=768))[2] < 3 << 30


VIEWS = [hyena.Rows(None, 30 * 48, 48), hyena.Rows(ptr(0) + 1, 30 * 48, 48), hyena.Rows(ptr(0), -1, 48), hyena.Rows(ptr(0), 1, -48)]


@pytest.mark.parametrize("bad", VIEWS)
def test_views(bad):
    d = hyena.Rows(ptr(5), 30 * 48, 48)
    assert hyena.hyena_embedding_forward(embedding(tokens=bad), ptr(3), ptr(4)) == INVALID
    assert hyena.hyena_embedding_backward(embedding(tokens=bad), d, ptr(3), 0, ptr(4)) == INVALID
    assert hyena.hyena_embedding_backward(embedding(), bad, ptr(3), 0, ptr(4)) == INVALID
    assert hyena.hyena_residual_norm_forward(norm(x=bad), ptr(3), ptr(4), None) == INVALID
    if bad.data is not None:
        assert hyena.hyena_residual_norm_forward(norm(residual=bad), ptr(3), ptr(4), None) == INVALID
    assert hyena.hyena_residual_norm_backward(norm(x=bad), d, None, ptr(3), None, None) == INVALID
    assert hyena.hyena_residual_norm_backward(norm(), bad, None, ptr(3), None, None) == INVALID
    assert hyena.hyena_residual_norm_backward(norm(), d, bad, ptr(3), None, None) == INVALID
    for kw in (dict(x=bad), dict(targets=bad)):
        assert hyena.hyena_token_loss_forward(loss(**kw), ptr(3), ptr(4), ptr(6)) == INVALID
        assert hyena.hyena_token_loss_backward(loss(**kw), d, ptr(3), ptr(4), ptr(6), ptr(7)) == INVALID
    assert hyena.hyena_token_loss_backward(loss(), bad, ptr(3), ptr(4), ptr(6), ptr(7)) == INVALID
    far = hyena.Rows(ptr(0), 1 << 41, 48)
    assert hyena.hyena_embedding_forward(embedding(tokens=far), ptr(3), ptr(4)) == UNSUPPORTED


def test_embedding_buffers():
    f = lambda table, out: hyena.hyena_embedding_forward(embedding(), table, out)  # noqa: E731
    assert f(None, ptr(4)) == f(ptr(3), None) == f(ptr(3) + 1, ptr(4)) == f(ptr(3), ptr(4) + 1) == INVALID
    assert f(ptr(3), ptr(3) + 48) == f(ptr(3), ptr(0) - 16) == INVALID
    assert "overlaps" in hyena.hyena_last_error()
    d = hyena.Rows(ptr(5), 30 * 48, 48)
    b = lambda d, table, scratch: hyena.hyena_embedding_backward(embedding(), d, table, 1, scratch)  # noqa: E731
    assert b(None, ptr(3), ptr(4)) == b(d, None, ptr(4)) == b(d, ptr(3) + 1, ptr(4)) == INVALID
    assert b(d, ptr(3), None) == b(d, ptr(3), ptr(4) + 8) == INVALID
    assert b(d, ptr(5) + 96, ptr(4)) == b(d, ptr(3), ptr(5) + 16) == b(d, ptr(3), ptr(3) + 16) == b(d, ptr(0), ptr(4)) == INVALID


def test_norm_buffers():
    eight = dict(format=1)
    f = lambda op, s, y, a: hyena.hyena_residual_norm_forward(op, s, y, a)  # noqa: E731
    none = hyena.Rows(None, 0, 0)
    assert f(norm(), None, ptr(4), None) == f(norm(residual=none), ptr(3), ptr(4), None) == INVALID
    assert f(norm(), ptr(3), None, None) == f(norm(), ptr(3), ptr(4), ptr(6)) == f(norm(**eight), ptr(3), ptr(4), None) == INVALID
    assert f(norm(), ptr(3) + 1, ptr(4), None) == f(norm(), ptr(3), ptr(4) + 1, None) == INVALID
    assert f(norm(**eight), ptr(3), ptr(4), ptr(6) + 2) == f(norm(weight=ptr(1) + 2), ptr(3), ptr(4), None) == INVALID
    assert f(norm(format=3), ptr(3), ptr(4), ptr(6)) == UNSUPPORTED
    assert f(norm(group=32), ptr(3), ptr(4), None) == f(norm(format=1, group=48), ptr(3), ptr(4), ptr(6)) == INVALID
    assert f(norm(format=1, group=64, d=96), ptr(3), ptr(4), ptr(6)) == INVALID
    assert f(norm(eps=-1.0), ptr(3), ptr(4), None) == f(norm(eps=float("nan")), ptr(3), ptr(4), None) == INVALID
    # overlaps; the sum may lie on x or the residual, but only row on row
    assert f(norm(), ptr(3), ptr(0), None) == f(norm(), ptr(3), ptr(2), None) == f(norm(), ptr(3), ptr(3) + 16, None) == INVALID
    assert f(norm(), ptr(0) + 256, ptr(4), None) == f(norm(), ptr(1), ptr(4), None) == INVALID
    assert f(norm(x=hyena.Rows(ptr(0), 30 * 256, 256)), ptr(0), ptr(4), None) == INVALID
    assert f(norm(**eight), ptr(3), ptr(4), ptr(4) + 64) == f(norm(**eight), ptr(3), ptr(4), ptr(3) + 64) == INVALID
    d = hyena.Rows(ptr(5), 30 * 128, 128)
    b = lambda dy, ds, dx, dw, w: hyena.hyena_residual_norm_backward(norm(), dy, ds, dx, dw, w)  # noqa: E731
    assert b(None, None, ptr(3), None, None) == b(d, None, None, None, None) == b(d, None, ptr(3) + 1, None, None) == INVALID
    assert b(d, None, ptr(3), ptr(6), None) == b(d, None, ptr(3), ptr(6), ptr(7) + 4) == b(d, None, ptr(3), ptr(6) + 1, ptr(7)) == INVALID
    assert b(d, None, ptr(5), None, None) == b(d, None, ptr(0), None, None) == b(d, None, ptr(3), ptr(3), ptr(7)) == INVALID
    ds = hyena.Rows(ptr(8), 30 * 256, 256)
    assert b(d, ds, ptr(8), None, None) == b(d, ds, ptr(3), ptr(8), ptr(7)) == INVALID


def test_loss_buffers():
    f = lambda op, a, b, w: hyena.hyena_token_loss_forward(op, a, b, w)  # noqa: E731
    assert f(loss(table=None), ptr(3), ptr(4), ptr(6)) == f(loss(table=ptr(1) + 8), ptr(3), ptr(4), ptr(6)) == INVALID
    assert f(loss(), None, ptr(4), ptr(6)) == f(loss(), ptr(3), None, ptr(6)) == f(loss(), ptr(3) + 2, ptr(4), ptr(6)) == INVALID
    assert f(loss(), ptr(3), ptr(4), None) == f(loss(), ptr(3), ptr(4), ptr(6) + 8) == INVALID
    assert f(loss(), ptr(3), ptr(3) + 16, ptr(6)) == f(loss(), ptr(3), ptr(1), ptr(6)) == f(loss(), ptr(6) + 16, ptr(4), ptr(6)) == INVALID
    d = hyena.Rows(ptr(5), 30, 1)
    b = lambda d, lse, dx, dt, w: hyena.hyena_token_loss_backward(loss(), d, lse, dx, dt, w)  # noqa: E731
    assert b(None, ptr(3), ptr(4), ptr(6), ptr(7)) == b(d, None, ptr(4), ptr(6), ptr(7)) == INVALID
    assert b(d, ptr(3) + 2, ptr(4), ptr(6), ptr(7)) == b(d, ptr(3), None, None, ptr(7)) == INVALID
    assert b(d, ptr(3), ptr(4) + 8, ptr(6), ptr(7)) == b(d, ptr(3), ptr(4), ptr(6) + 8, ptr(7)) == INVALID
    assert b(d, ptr(3), ptr(4), ptr(6), None) == b(d, ptr(3), ptr(4), ptr(4) + 16, ptr(7)) == b(d, ptr(3), ptr(1), ptr(6), ptr(7)) == INVALID
    assert b(d, ptr(3), ptr(0), ptr(6), ptr(7)) == b(d, ptr(3), ptr(4), ptr(6), ptr(3) - 16) == INVALID


# ---------------------------------------------------------------- the torch wrapper

def bare(cls, **kw):
    """A plan without a GPU: what its checks use."""
    p = object.__new__(cls)
    p.torch, p.device, p.index, p._lib = torch, torch.device("cpu"), 0, hyena.load()
    p.io_dtype, p.dtype = hyena.HYENA_BF16, torch.bfloat16
    for name, value in kw.items():
        setattr(p, name, value)
    return p


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def refuses(f, match):
    with pytest.raises(ValueError, match=match):
        f()


def test_wrapper_constructors_refuse():
    for make in (lambda **k: hyena.Embedding(1, 4, 10, 8, **k), lambda **k: hyena.ResidualNorm(1, 4, 8, **k),
                 lambda **k: hyena.TokenLoss(1, 4, 10, 8, **k)):
        refuses(lambda: make(io_dtype=7), "unknown io dtype")
        refuses(lambda: make(device="cpu"), "must be a GPU")


def test_embedding_wrapper():
    p = bare(hyena.Embedding, B=2, N=5, V=9, d=8, scale=1.0, scratch_bytes=64)
    tok, table = zeros(2, 5, dtype=torch.int32), zeros(9, 8)
    refuses(lambda: p.forward(tok.long(), table), "tokens must be torch.int32")
    refuses(lambda: p.forward(tok[:, :4], table), "tokens must have shape")
    refuses(lambda: p.forward(tok, table.float()), "table must be torch.bfloat16")
    refuses(lambda: p.forward(tok, zeros(8, 9).t()), "table must be contiguous")
    refuses(lambda: p.forward(tok, None), "table must be a torch tensor")
    refuses(lambda: p.forward(tok, table, out=zeros(2, 5, 9)), "out must have shape")
    refuses(lambda: p.backward(zeros(2, 5, 8).float(), tok), "d_out must be torch.bfloat16")
    refuses(lambda: p.backward(zeros(2, 8, 5).transpose(1, 2), tok), "last axis of d_out")
    refuses(lambda: p.backward(zeros(2, 5, 8), tok, d_table=zeros(9, 8, dtype=torch.float32)), "d_table must be")


def test_norm_wrapper():
    kinds = dict(B=2, N=5, d=64, eps=1e-6, scratch_bytes=64, group=None, quantized=None, _y_dtype=torch.bfloat16)
    p = bare(hyena.ResidualNorm, **kinds)
    x, w = zeros(2, 5, 64), zeros(64, dtype=torch.float32)
    refuses(lambda: p.forward(x.float()), "x must be torch.bfloat16")
    refuses(lambda: p.forward(x, x[:, :4]), "residual must have shape")
    refuses(lambda: p.forward(x, x, w.bfloat16()), "weight must be torch.float32")
    refuses(lambda: p.forward(x, total=x), "only there with a residual")
    refuses(lambda: p.forward(x, scales=w), "only there with quantized")
    refuses(lambda: p.forward(x, y=x.float()), "y must be torch.bfloat16")
    refuses(lambda: p.forward(zeros(2, 64, 5).transpose(1, 2)), "last axis of x")
    refuses(lambda: p.backward(x, x, w, ds=x[:1]), "ds must have shape")
    refuses(lambda: p.backward(x, x, w, dx=x.float()), "dx must be torch.bfloat16")
    refuses(lambda: hyena.ResidualNorm(1, 1, 64, quantized="e5m2"), "quantized must be|must be a GPU|No HIP|NVIDIA|CUDA") \
        if torch.cuda.is_available() else None
    q = bare(hyena.ResidualNorm, **dict(kinds, quantized="int8", group=32, _y_dtype=torch.int8))
    assert q.scales_shape == (2, 5, 2)
    refuses(lambda: q.forward(x, y=x), "y must be torch.int8")
    refuses(lambda: q.forward(x, scales=zeros(2, 5, 1, dtype=torch.float32)), "scales must have shape")


def test_loss_wrapper():
    p = bare(hyena.TokenLoss, B=2, N=5, V=9, d=8, scale=1.0, forward_bytes=64, backward_bytes=64)
    x, table, t = zeros(2, 5, 8), zeros(9, 8), zeros(2, 5, dtype=torch.int32)
    f = zeros(2, 5, dtype=torch.float32)
    refuses(lambda: p.forward(x.float(), table, t), "x must be torch.bfloat16")
    refuses(lambda: p.forward(x, table[:8], t), "table must have shape")
    refuses(lambda: p.forward(x, None, t), "table must be a torch tensor")
    refuses(lambda: p.forward(x, table, t.long()), "targets must be torch.int32")
    refuses(lambda: p.forward(x, table, t, loss=f[:1]), "loss must have shape")
    refuses(lambda: p.backward(f.double(), x, table, t, f), "d_loss must be torch.float32")
    refuses(lambda: p.backward(f, x, table, t, None), "lse must be a torch tensor")
    refuses(lambda: p.backward(f, x, table, t, f.t().contiguous().t()), "lse must be contiguous")
