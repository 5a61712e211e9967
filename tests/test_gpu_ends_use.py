"""The operators at a model's ends and between its layers as a model uses them, with
a mixer between: tokens to rows, norm, queries and keys normed and rotated,
gated recurrence, residual, norm, loss; and back, the table shared by both ends.

The reference is the same model in torch's float64 on the CPU, its gradients by
autograd.  In float32 every operator is off by a few 2^-20 of its terms; a layer's
projections have 40 terms, the loss 90 and the recurrence 33 tokens: 2^-12 of the
largest value of each gradient stands for their sum over the layers.
"""
import numpy as np
import pytest

from gpu_util import say
from long_convolution_sequence_rfft_amd import hyena
from test_gpu_recurrence import f64

pytestmark = pytest.mark.gpu

B, N, V, H, DH, LAYERS = 2, 33, 90, 2, 20, 2
D = H * DH


def weights(gen):
    import torch
    w = dict(table=torch.randn((V, D), generator=gen), last=1 + 0.1 * torch.randn(D, generator=gen))
    for i in range(LAYERS):
        w[f"qkv{i}"] = torch.randn((D, 3 * D), generator=gen) / D ** 0.5
        w[f"out{i}"] = torch.randn((D, D), generator=gen) / D ** 0.5
        w[f"norm{i}"] = 1 + 0.1 * torch.randn(D, generator=gen)
        w[f"g{i}"] = -torch.rand((B, N, H), generator=gen)
    return w


def reference(w, tokens, targets, scale):
    import torch
    w = {k: v.double().requires_grad_() for k, v in w.items()}
    live = (tokens >= 0)[..., None]
    h = torch.where(live, w["table"][tokens.clamp(min=0).long()] * scale, 0.0)
    rms = lambda x, a: x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * a  # noqa: E731
    for i in range(LAYERS):
        qkv = (rms(h, w[f"norm{i}"]) @ w[f"qkv{i}"]).view(B, N, 3 * H, DH)
        q, k, v = qkv[:, :, :H], qkv[:, :, H:2 * H], qkv[:, :, 2 * H:]
        q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6) for x in (q, k))
        g = w[f"g{i}"].cumsum(1)
        decay = torch.exp(g[:, :, None] - g[:, None]).permute(0, 3, 1, 2).tril()
        scores = torch.einsum("bnhd,bmhd->bhnm", q, k) * decay * DH ** -0.5
        o = torch.einsum("bhnm,bmhd->bnhd", scores, v).reshape(B, N, D)
        h = h + o @ w[f"out{i}"]
    logits = rms(h, w["last"]) @ w["table"].t()
    loss = torch.nn.functional.cross_entropy(logits.view(-1, V), targets.long().view(-1), ignore_index=-1, reduction="none")
    loss.sum().backward()
    return loss.detach().view(B, N), {k: v.grad for k, v in w.items()}


def test_a_training_step_of_a_small_model():
    import torch
    say("[gpu] training step with embedding, residual norms, recurrence and loss")
    gen = torch.Generator().manual_seed(11)
    host = weights(gen)
    tokens = torch.randint(0, V, (B, N), generator=gen, dtype=torch.int32)
    targets = torch.roll(tokens, -1, 1)
    targets[:, -1] = -1
    tokens[1, 25:] = -1
    targets[1, 24:] = -1
    want, grads = reference(host, tokens, targets, 3.0)
    w = {k: v.cuda() for k, v in host.items()}
    tokens, targets = tokens.cuda(), targets.cuda()
    embed = hyena.Embedding(B, N, V, D, scale=3.0)
    norm = hyena.ResidualNorm(B, N, D)
    qk = hyena.QKNorm(B, N, H, H, DH, norm="l2", rotary_dim=0)
    rec = hyena.Recurrence(B, N, H, DH, DH, training=True)
    head = hyena.TokenLoss(B, N, V, D)
    # forward: the stream h is summed inside the norms
    stream, mixed, kept = embed.forward(tokens, w["table"]), None, []
    for i in range(LAYERS):
        y, total = norm.forward(stream, mixed, w[f"norm{i}"])
        stream = stream if total is None else total
        qkv = (y.view(-1, D) @ w[f"qkv{i}"]).view(B, N, 3 * H, DH)
        q, k, v = qkv[:, :, :H], qkv[:, :, H:2 * H], qkv[:, :, 2 * H:]
        qn, kn = qk.forward(q, k)
        o, _ = rec.forward(qn, kn, v, w[f"g{i}"])
        mixed = (o.view(-1, D) @ w[f"out{i}"]).view(B, N, D)
        kept.append((stream, y, q, k, v, qn, kn, o))
    y, stream = norm.forward(stream, mixed, w["last"])
    loss, lse = head.forward(y, w["table"], targets)
    assert np.abs(f64(loss) - f64(want)).max() < 1e-4
    # backward
    got = {}
    one = torch.ones((), device="cuda").expand(B, N)
    dy, got["table"] = head.backward(one, y, w["table"], targets, lse)
    dh, got["last"] = norm.backward(dy, stream, w["last"])
    for i in reversed(range(LAYERS)):
        s, y, q, k, v, qn, kn, o = kept[i]
        got[f"out{i}"] = o.view(-1, D).t() @ dh.view(-1, D)
        do = (dh.view(-1, D) @ w[f"out{i}"].t()).view(B, N, H, DH)
        dqn, dkn, dv, got[f"g{i}"], _ = rec.backward(do, qn, kn, v, w[f"g{i}"])
        dq, dk, _, _ = qk.backward(dqn, dkn, q, k)
        dqkv = torch.cat([dq, dk, dv], 2).view(-1, 3 * D)
        got[f"qkv{i}"] = y.view(-1, D).t() @ dqkv
        dy = (dqkv @ w[f"qkv{i}"].t()).view(B, N, D)
        dh, got[f"norm{i}"] = norm.backward(dy, s, w[f"norm{i}"], ds=dh)
    tied = embed.backward(dh, tokens, d_table=got["table"])
    assert tied is got["table"]
    for name, ref in grads.items():
        off = np.abs(f64(got[name]) - f64(ref)).max() / np.abs(f64(ref)).max()
        say(f"[gpu]   {name}: {off:.3g} of the largest value")
        assert off < 2.0 ** -12, name


def test_decoding_a_token_at_a_time():
    # one token per request through embedding, norm and recurrence equals the whole sequence's pass
    import torch
    say("[gpu] decoding with embedding, residual norm and recurrence")
    gen = torch.Generator().manual_seed(12)
    w = {k: v.cuda() for k, v in weights(gen).items()}
    tokens = torch.randint(0, V, (B, N), generator=gen, dtype=torch.int32).cuda()
    whole = hyena.ResidualNorm(B, N, D).forward(hyena.Embedding(B, N, V, D).forward(tokens, w["table"]), None, w["norm0"])[0]
    qkv = (whole.view(-1, D) @ w["qkv0"]).view(B, N, 3 * H, DH)
    o, _ = hyena.Recurrence(B, N, H, DH, DH).forward(*qkv.split(H, 2), w["g0"])
    embed, norm, rec = hyena.Embedding(B, 1, V, D), hyena.ResidualNorm(B, 1, D), hyena.Recurrence(B, 1, H, DH, DH)
    states = torch.zeros((B, H, DH, DH), device="cuda")
    for t in range(N):
        y, _ = norm.forward(embed.forward(tokens[:, t:t + 1], w["table"]), None, w["norm0"])
        assert torch.equal(y, whole[:, t:t + 1])
        q, k, v = (y.view(-1, D) @ w["qkv0"]).view(B, 3 * H, DH).split(H, 1)
        one = rec.step(q, k, v, w["g0"][:, t], states)
        assert float((one - o[:, t]).abs().max()) < 2.0 ** -12 * float(o.abs().max())
