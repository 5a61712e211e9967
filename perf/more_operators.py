"""Workloads of the operators at a model's ends and between its layers: inputs,
the plain form in elementary torch operations, the library's calls, and the
values in 64 bits.

A case's "op" names the operator:

  embed       rows of a table by token, times a factor
  embed_grad  the table's gradient: a new one, or added to one that is there
  norm        s = x + residual and its RMS norm, in the storage type or in 8 bits with scales
  norm_grad   its backward pass
  loss        softmax cross entropy of x table^T, per token
  loss_grad   its backward pass
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LARGEST = {"e4m3": 448.0, "int8": 127.0}


def listed():
    return [
        # the tokens of 32 requests that decode
        dict(name="embed_b32_bf16", op="embed", B=32, N=1, V=50257, d=768, scale=1.0, ragged=False, dtype="bf16"),
        # two 8K-token sequences enter a width-768 model that scales its embeddings by sqrt(width)
        dict(name="embed_8k_bf16", op="embed", B=2, N=8192, V=50257, d=768, scale=27.7128, ragged=False, dtype="bf16"),
        # training at 2K tokens in float32: padded rows, an odd vocabulary, a width that is no power of two
        dict(name="embed_grad_2k_f32", op="embed_grad", B=4, N=2048, V=31999, d=770, scale=1.0, ragged=True, adds=False,
             dtype="f32"),
        # training at 64K tokens a step with one table at both ends: the loss's gradient is there already
        dict(name="embed_grad_64k_tied_bf16", op="embed_grad", B=8, N=8192, V=50257, d=768, scale=27.7128, ragged=False,
             adds=True, dtype="bf16"),
        # one decoded token for each of 32 requests, the norm handed to an 8-bit projection
        dict(name="norm_b32_e4m3_bf16", op="norm", B=32, N=1, d=768, residual=True, eight="e4m3", group=0, dtype="bf16"),
        # between the layers of a width-768 model on two 8K-token sequences
        dict(name="norm_8k_bf16", op="norm", B=2, N=8192, d=768, residual=True, eight="", group=0, dtype="bf16"),
        # training at 2K tokens in binary16, the norm in front of the loss: no residual stream goes on
        dict(name="norm_grad_2k_f16", op="norm_grad", B=4, N=2048, d=1000, stream=False, dtype="f16"),
        # training at 8K tokens between layers: the stream's gradient comes in too
        dict(name="norm_grad_8k_bf16", op="norm_grad", B=2, N=8192, d=768, stream=True, dtype="bf16"),
        # scoring one more token of 8 candidates
        dict(name="loss_b8_bf16", op="loss", B=8, N=1, V=50257, d=768, masked=0.0, dtype="bf16"),
        # evaluating two 8K-token sequences
        dict(name="loss_8k_bf16", op="loss", B=2, N=8192, V=50257, d=768, masked=0.0, dtype="bf16"),
        # training on 2K tokens in float32
        dict(name="loss_grad_2k_f32", op="loss_grad", B=1, N=2048, V=31999, d=768, masked=0.0, dtype="f32"),
        # training on two 8K-token rows, a quarter of the tokens prompts without a target
        dict(name="loss_grad_8k_bf16", op="loss_grad", B=2, N=8192, V=50257, d=768, masked=0.25, dtype="bf16"),
    ]


def _log_uniform(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "loss", "loss_grad"])
    c = dict(op=op, B=_log_uniform(rng, 1, 8), N=_log_uniform(rng, 1, 16000),
             d=rng.choice([_log_uniform(rng, 24, 2500), 256, 768, 1024]))
    if op in ("embed", "embed_grad", "loss", "loss_grad"):
        c["V"] = rng.choice([_log_uniform(rng, 200, 100000), 50257])
    if op.startswith("embed"):
        c.update(scale=rng.choice([1.0, c["d"] ** 0.5]), ragged=rng.random() < 0.5)
    if op == "embed_grad":
        c.update(adds=rng.random() < 0.4)
    if op == "norm":
        c.update(residual=rng.random() < 0.8, eight=rng.choice(["", "", "e4m3", "int8"]), group=0)
    if op == "norm_grad":
        c.update(stream=rng.random() < 0.7)
    if op.startswith("loss"):
        c.update(masked=rng.choice([0.0, 0.0, round(rng.uniform(0.05, 0.9), 2)]))
    c["dtype"] = rng.choice(["f32", "bf16", "bf16", "f16"])
    if c.get("eight"):
        c["dtype"] = rng.choice(["bf16", "f16"])
        if rng.random() < 0.5:
            c["d"], c["group"] = rng.choice([256, 768, 1024, 1280]), rng.choice([32, 64, 128])
    key = "flops" if op.startswith("loss") else "bytes"
    # float32 products cost several times those in 16 bits
    heavy = 3 if op.startswith("loss") and c["dtype"] == "f32" else 1
    most = max(work(x)[key] for x in listed() if x["op"] == op)
    while heavy * work(c)[key] > most and (c["N"] > 1 or c.get("V", 0) > 200):
        if c["N"] > 1:
            c["N"] = max(1, c["N"] * 2 // 3)
        else:
            c["V"] = c["V"] * 2 // 3
    return c


def work(case):
    c, e = case, 4 if case["dtype"] == "f32" else 2
    n, d = c["B"] * c["N"], c["d"]
    if c["op"] == "embed":
        return dict(bytes=4 * n + (min(n, c["V"]) + n) * d * e, flops=n * d)
    if c["op"] == "embed_grad":  # rows that are added to are read and written: at most one for each token
        table = 2 * min(n, c["V"]) if c["adds"] else c["V"]
        return dict(bytes=4 * n + (n + table) * d * e, flops=n * d)
    if c["op"] == "norm":
        streams = (2 if c["residual"] else 0) + 1  # x, residual, their sum
        groups = n * (d // c["group"] if c["group"] else 1)
        out = n * d + 4 * groups if c["eight"] else n * d * e
        return dict(bytes=streams * n * d * e + out + 4 * d, flops=6 * n * d)
    if c["op"] == "norm_grad":
        return dict(bytes=(4 if c["stream"] else 3) * n * d * e + 8 * d, flops=12 * n * d)
    live = n - int(c["masked"] * n)
    if c["op"] == "loss":
        return dict(bytes=(live + c["V"]) * d * e + 12 * n, flops=2 * live * c["V"] * d)
    return dict(bytes=(live + n + 2 * c["V"]) * d * e + 12 * n, flops=6 * live * c["V"] * d)


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]
    B, N, d = c["B"], c["N"], c["d"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32)

    def tokens():
        """Token v about as often as 1 / v: text."""
        return (uniform(B, N) * math.log(c["V"])).exp().to(torch.int32).clamp(1, c["V"]) - 1

    s = dict(case=c)
    op = c["op"]
    if op.startswith("embed"):
        s["tokens"] = tokens()
        if c["ragged"]:  # rows are padded with tokens that are none
            n = torch.randint(0, N + 1, (B, 1), generator=gen, device="cuda")
            n[B // 2] = N
            s["tokens"] = torch.where(torch.arange(N, device="cuda") < n, s["tokens"], -1)
        if op == "embed":
            s["table"] = normal(c["V"], d).to(dt)
        else:
            s["d_out"] = normal(B, N, d).to(dt)
            s["d_table"] = normal(c["V"], d).to(dt) if c["adds"] else None
        if own:
            from long_convolution_sequence_rfft_amd import hyena
            s["plan"] = hyena.Embedding(B, N, c["V"], d, io_dtype=_io(hyena, c), scale=c["scale"])
        return s
    if op.startswith("norm"):
        s["weight"] = 1.0 + 0.1 * normal(d)
        x = normal(B, N, d) * (0.5 + uniform(B, N, 1))
        if op == "norm":
            s["x"], s["residual"] = x.to(dt), (2.0 * normal(B, N, d)).to(dt) if c["residual"] else None
        else:
            s["s"], s["dy"] = (2.0 * x).to(dt), normal(B, N, d).to(dt)
            s["ds"] = normal(B, N, d).to(dt) if c["stream"] else None
        if own:
            from long_convolution_sequence_rfft_amd import hyena
            s["plan"] = hyena.ResidualNorm(B, N, d, io_dtype=_io(hyena, c), eps=1e-6, quantized=c.get("eight") or None,
                                           group=c.get("group") or None)
        return s
    V = c["V"]
    s["table"] = (normal(V, d) * (2.0 / math.sqrt(d))).to(dt)  # logits of about 2
    target = tokens()
    # a model that has learnt something: x leans to the table's row of the target, more at some tokens than at others
    x = normal(B, N, d) + 2.0 * uniform(B, N, 1) * s["table"][target.long()].float()
    s["x"] = x.to(dt)
    masked = int(c["masked"] * B * N)
    if masked:
        none = torch.randperm(B * N, generator=gen, device="cuda")[:masked] if N < 4 else torch.arange(masked, device="cuda")
        target.view(-1)[none] = -1
    s["targets"] = target
    if op == "loss_grad":
        live = target >= 0
        s["d_loss"] = torch.where(live, 1.0 / live.sum().clamp(min=1), 0.0)
        lse = torch.zeros(B * N, device="cuda")
        table = s["table"].float()
        rows = s["x"].reshape(B * N, d).float()
        for i in range(0, B * N, 2048):
            lse[i:i + 2048] = torch.logsumexp(rows[i:i + 2048] @ table.t(), -1)
        s["lse"] = torch.where(live, lse.view(B, N), 0.0)
    if own:
        from long_convolution_sequence_rfft_amd import hyena
        s["plan"] = hyena.TokenLoss(B, N, V, d, io_dtype=_io(hyena, c))
    return s


def _io(hyena, c):
    return {"f32": hyena.HYENA_F32, "bf16": hyena.HYENA_BF16, "f16": hyena.HYENA_F16}[c["dtype"]]


# ---------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    c, p = s["case"], s["plan"]
    op = c["op"]
    if op == "embed":
        return dict(out=p.forward(s["tokens"], s["table"]))
    if op == "embed_grad":
        return dict(d_table=p.backward(s["d_out"], s["tokens"], d_table=s["d_table"]))
    if op == "norm":
        if c["eight"]:
            y8, scales, total = p.forward(s["x"], s["residual"], s["weight"])
            return dict(y=_values(y8, scales, c), scales=scales, total=total)
        y, total = p.forward(s["x"], s["residual"], s["weight"])
        return dict(y=y, total=total)
    if op == "norm_grad":
        dx, dw = p.backward(s["dy"], s["s"], s["weight"], ds=s["ds"])
        return dict(dx=dx, d_weight=dw)
    if op == "loss":
        loss, lse = p.forward(s["x"], s["table"], s["targets"])
        return dict(loss=loss, lse=lse)
    dx, dt = p.backward(s["d_loss"], s["x"], s["table"], s["targets"], s["lse"])
    return dict(dx=dx, d_table=dt)


def _values(y8, scales, c):
    """What the 8-bit values stand for, in the storage type."""
    wide = y8.float().unflatten(-1, (scales.shape[-1], -1)) * scales[..., None]
    return wide.flatten(-2).to(DTYPES[c["dtype"]])


def _run_plain(s):
    return {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "norm": _plain_norm, "norm_grad": _plain_norm_grad,
            "loss": _plain_loss, "loss_grad": _plain_loss_grad}[s["case"]["op"]](s)


def _plain_embed(s):
    t = s["tokens"].long()
    live = (t >= 0) & (t < s["case"]["V"])
    rows = s["table"][torch.where(live, t, 0)].float() * s["case"]["scale"]
    return dict(out=torch.where(live[..., None], rows, 0.0).to(s["table"].dtype))


def _plain_embed_grad(s):
    c = s["case"]
    t = s["tokens"].long().view(-1)
    live = (t >= 0) & (t < c["V"])
    rows = torch.where(live[:, None], s["d_out"].view(-1, c["d"]).float() * c["scale"], 0.0)
    if s["d_table"] is None:
        sums = torch.zeros((c["V"], c["d"]), device="cuda")
    else:
        sums = s["d_table"].float()
    sums = sums.index_add(0, torch.where(live, t, 0), rows).to(s["d_out"].dtype)
    if s["d_table"] is not None:
        return dict(d_table=s["d_table"].copy_(sums))
    return dict(d_table=sums)


def _plain_norm(s):
    c = s["case"]
    total = s["x"].float()
    if c["residual"]:
        total = total + s["residual"].float()
    y = total * torch.rsqrt(total.square().mean(-1, keepdim=True) + 1e-6) * s["weight"]
    kept = total.to(s["x"].dtype) if c["residual"] else None
    if not c["eight"]:
        return dict(y=y.to(s["x"].dtype), total=kept)
    y = y.unflatten(-1, (-1, c["group"] or c["d"]))
    scales = y.abs().amax(-1) / LARGEST[c["eight"]]
    q = torch.where(scales[..., None] > 0, y / scales[..., None], 0.0).clamp(-LARGEST[c["eight"]], LARGEST[c["eight"]])
    q = q.to(torch.float8_e4m3fn) if c["eight"] == "e4m3" else q.round().to(torch.int8)
    return dict(y=_values(q.flatten(-2), scales, c), scales=scales, total=kept)


def _plain_norm_grad(s):
    x, dy = s["s"].float(), s["dy"].float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    n = x * r
    dn = dy * s["weight"]
    dx = (dn - n * (dn * n).mean(-1, keepdim=True)) * r
    if s["ds"] is not None:
        dx = dx + s["ds"].float()
    return dict(dx=dx.to(s["s"].dtype), d_weight=(dy * n).sum((0, 1), dtype=torch.float64).float())


def _logits(s):
    c = s["case"]
    t = s["targets"].long().view(-1)
    live = (t >= 0) & (t < c["V"])
    x, table = s["x"].view(-1, c["d"]).float(), s["table"].float()
    return x, table, torch.matmul(x, table.t()), torch.where(live, t, 0), live


def _plain_loss(s):
    _, _, logits, at, live = _logits(s)
    m = logits.amax(-1, keepdim=True)
    lse = m[:, 0] + (logits - m).exp().sum(-1).log()
    loss = lse - logits.gather(1, at[:, None])[:, 0]
    shape = s["targets"].shape
    return dict(loss=torch.where(live, loss, 0.0).view(shape), lse=torch.where(live, lse, 0.0).view(shape))


def _plain_loss_grad(s):
    x, table, logits, at, live = _logits(s)
    g = (logits - s["lse"].view(-1, 1)).exp()
    g[torch.arange(at.numel(), device="cuda"), at] -= 1.0
    g = torch.where(live[:, None], g * s["d_loss"].view(-1, 1), 0.0)
    dx = torch.matmul(g, table).to(s["x"].dtype).view(s["x"].shape)
    return dict(dx=dx, d_table=torch.matmul(g.t(), x).to(s["table"].dtype))


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op, d = c["op"], c["d"]
    F = torch.nn.functional
    if op == "embed":
        t = s["tokens"]
        none = (t < 0) | (t >= c["V"])
        return dict(out=F.embedding(t.clamp(0, c["V"] - 1).long(), s["table"].double()).masked_fill(none[..., None], 0) * c["scale"])
    if op == "embed_grad":
        # a product with the tokens' marks, by a table with one more row for those that are none
        t = torch.where((s["tokens"] < 0) | (s["tokens"] >= c["V"]), c["V"], s["tokens"]).long()
        table = torch.zeros((c["V"] + 1, d), device="cuda", dtype=torch.float64, requires_grad=True)
        (F.embedding(t, table) * c["scale"]).backward(s["d_out"].double())
        g = table.grad[:c["V"]]
        return dict(d_table=g if s["d_table"] is None else g + s["d_table"].double())
    if op == "norm":
        total = s["x"].double() + (s["residual"].double() if c["residual"] else 0)
        size = torch.linalg.vector_norm(total, dim=-1, keepdim=True)
        y = total / torch.sqrt(size * size / d + 1e-6) * s["weight"].double()
        kept = total if c["residual"] else None
        if not c["eight"]:
            return dict(y=y, total=kept)
        g = c["group"] or d
        parts = y.reshape(*y.shape[:-1], d // g, g)
        scales = torch.linalg.vector_norm(parts, ord=math.inf, dim=-1) / LARGEST[c["eight"]]
        q = parts / scales[..., None].clamp(min=1e-300)
        if c["eight"] == "int8":
            q = torch.round(q)
        else:  # three bits behind the first, down to 2^-9
            step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
            q = torch.round(q / step) * step
        return dict(y=(q * scales[..., None]).reshape(y.shape), scales=scales, total=kept)
    if op == "norm_grad":
        x = s["s"].double().requires_grad_()
        w = s["weight"].double().requires_grad_()
        y = F.rms_norm(x, (d,), eps=1e-6) * w
        y.backward(s["dy"].double())
        return dict(dx=x.grad + (0 if s["ds"] is None else s["ds"].double()), d_weight=w.grad)
    grad = op == "loss_grad"
    t = torch.where((s["targets"] < 0) | (s["targets"] >= c["V"]), -100, s["targets"]).long().view(-1)
    x = s["x"].reshape(-1, d).double().requires_grad_(grad)
    table = s["table"].double().requires_grad_(grad)
    if not grad:
        logits = x @ table.t()
        loss = F.cross_entropy(logits, t, reduction="none", ignore_index=-100)
        lse = torch.logsumexp(logits, -1).masked_fill(t < 0, 0)
        return dict(loss=loss.view(s["targets"].shape), lse=lse.view(s["targets"].shape))
    # a piece of the rows at a time: their logits in 64 bits are large
    for i in range(0, t.numel(), 4096):
        F.cross_entropy(x[i:i + 4096] @ table.t(), t[i:i + 4096], reduction="none", ignore_index=-100).backward(
            s["d_loss"].view(-1)[i:i + 4096].double())
    return dict(dx=x.grad.view(s["x"].shape), d_table=table.grad)
