"""Workloads of the query/key norm with rotary positions and of the gated
linear recurrence: inputs, the plain form in elementary torch operations, the
library's calls, and the values in 64 bits.

A case's "op" names the operator:

  qk_norm        y = R(pos) (w * x / rms(x)) of queries and keys, per head
  qk_norm_grad   its backward pass
  recurrence     S_t = exp(g_t) S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t
  recurrence_grad  its backward pass
  step           one token of the recurrence on a table of states
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CHUNK = 64  # tokens that the plain form handles by one product


def listed():
    return [
        # one decoded token for each of 32 requests, at positions of their own
        dict(name="qk_norm_decode_b32_bf16", op="qk_norm", B=32, N=1, q_heads=12, k_heads=12, D=64, rotary=64,
             norm="rms", layout="half", dtype="bf16", far=131072, stretch=1.0),
        # the forward pass of a width-768 layer on two 8K-token sequences
        dict(name="qk_norm_8k_bf16", op="qk_norm", B=2, N=8192, q_heads=12, k_heads=12, D=64, rotary=64, norm="rms",
             layout="half", dtype="bf16", far=0, stretch=1.0),
        # training at 2K tokens in float32: L2 norms, half of each head rotated, neighbouring pairs
        dict(name="qk_norm_grad_2k_f32", op="qk_norm_grad", B=4, N=2048, q_heads=12, k_heads=12, D=64, rotary=32,
             norm="l2", layout="interleaved", dtype="f32", far=0, stretch=1.0),
        # training at 8K tokens, keys shared by three queries each, frequencies stretched for a longer context
        dict(name="qk_norm_grad_8k_bf16", op="qk_norm_grad", B=2, N=8192, q_heads=12, k_heads=4, D=64, rotary=64,
             norm="rms", layout="half", dtype="bf16", far=0, stretch=8.0),
        # a short prompt: the latency of one call
        dict(name="recurrence_17_f32", op="recurrence", B=1, N=17, H=4, dk=64, dv=64, dtype="f32", carry=True,
             ragged=False, packed=False),
        # the forward pass of a width-768 layer with wide heads on two 8K-token sequences
        dict(name="recurrence_8k_d128_bf16", op="recurrence", B=2, N=8192, H=6, dk=128, dv=128, dtype="bf16", carry=False,
             ragged=False, packed=False),
        # one 64K-token document at width 768, its final state kept for decoding
        dict(name="recurrence_64k_bf16", op="recurrence", B=1, N=65536, H=12, dk=64, dv=64, dtype="bf16", carry=True,
             ragged=False, packed=False),
        # training at 2K tokens in float32, documents packed into the rows
        dict(name="recurrence_grad_2k_f32", op="recurrence_grad", B=4, N=2048, H=12, dk=64, dv=64, dtype="f32", carry=False,
             ragged=False, packed=True),
        # training at 8K tokens, a piece of a longer sequence: states enter and leave
        dict(name="recurrence_grad_8k_bf16", op="recurrence_grad", B=2, N=8192, H=12, dk=64, dv=64, dtype="bf16", carry=True,
             ragged=False, packed=False),
        # a padded batch with odd sizes: 4100 tokens, heads of 40 and 72 channels
        dict(name="recurrence_grad_4100_f16", op="recurrence_grad", B=3, N=4100, H=5, dk=40, dv=72, dtype="f16", carry=True,
             ragged=True, packed=False),
        # one token of one request
        dict(name="step_b1_bf16", op="step", B=1, slots=4, H=12, dk=64, dv=64, dtype="bf16"),
        # one token of each of 256 requests, their states at scattered places of a table
        dict(name="step_b256_bf16", op="step", B=256, slots=320, H=12, dk=64, dv=64, dtype="bf16"),
    ]


def _log_uniform(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(["qk_norm", "qk_norm_grad", "recurrence", "recurrence_grad", "step"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    if op == "step":
        B = _log_uniform(rng, 1, 200)
        return dict(op=op, B=B, slots=B + rng.randint(0, 40), H=rng.randint(1, 16), dk=rng.randint(8, 128),
                    dv=rng.randint(8, 128), dtype=dtype)
    B, N = _log_uniform(rng, 1, 6), _log_uniform(rng, 1, 12000)
    if op.startswith("qk_norm"):
        k_heads = rng.randint(1, 12)
        D = rng.choice([rng.randint(8, 192), 64, 128])
        c = dict(op=op, B=B, N=N, q_heads=k_heads * rng.randint(1, 3), k_heads=k_heads, D=D,
                 rotary=rng.choice([D // 2 * 2, D // 4 * 2, 0]), norm=rng.choice(["rms", "rms", "l2", "none"]),
                 layout=rng.choice(["half", "interleaved"]), dtype=dtype, far=rng.choice([0, 1000, 1000000]),
                 stretch=rng.choice([1.0, 4.0]))
        least, most = 1, max(work(x)["bytes"] for x in listed() if x["op"].startswith("qk_norm"))
    else:
        c = dict(op=op, B=B, N=N, H=rng.randint(1, 12), dk=rng.choice([rng.randint(8, 128), 64, 128]),
                 dv=rng.choice([rng.randint(8, 128), 64, 128]), dtype=dtype, carry=rng.random() < 0.5,
                 ragged=rng.random() < 0.4, packed=rng.random() < 0.3)
        least, most = 1, max(work(x)["flops"] for x in listed() if x["op"] == op)
    key = "bytes" if op.startswith("qk_norm") else "flops"
    while work(c)[key] > most and c["N"] > least:
        c["N"] = c["N"] * 2 // 3
    return c


def work(case):
    c, e = case, 4 if case["dtype"] == "f32" else 2
    if c["op"].startswith("qk_norm"):
        n = c["B"] * c["N"] * (c["q_heads"] + c["k_heads"]) * c["D"]
        if c["op"] == "qk_norm":
            return dict(bytes=2 * n * e, flops=8 * n)
        return dict(bytes=3 * n * e, flops=16 * n)
    dk, dv = c["dk"], c["dv"]
    if c["op"] == "step":
        n = c["B"] * c["H"]
        return dict(bytes=n * (8 * dk * dv + (2 * dk + 2 * dv) * e + 4), flops=n * 5 * dk * dv)
    n = c["B"] * c["N"] * c["H"]
    state = c["B"] * c["H"] * dk * dv * 4
    if c["op"] == "recurrence":
        return dict(bytes=n * ((2 * dk + 2 * dv) * e + 4) + (2 * state if c["carry"] else 0), flops=n * 4 * dk * dv)
    return dict(bytes=n * ((4 * dk + 3 * dv) * e + 8) + (3 * state if c["carry"] else 0), flops=n * 10 * dk * dv)


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    s = dict(case=c)
    if c["op"].startswith("qk_norm"):
        B, N, D = c["B"], c["N"], c["D"]
        # queries and keys are slices of one projection's output, values behind them
        heads = c["q_heads"] + 2 * c["k_heads"]
        qkv = normal(B, N, heads, D).to(dt)
        s["q"] = qkv[:, :, :c["q_heads"]]
        s["k"] = qkv[:, :, c["q_heads"]:c["q_heads"] + c["k_heads"]]
        s["q_weight"] = 1.0 + 0.1 * normal(D) if c["norm"] != "none" else None
        s["k_weight"] = 1.0 + 0.1 * normal(D) if c["norm"] != "none" else None
        r = c["rotary"]
        s["freqs"] = (10000.0 ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / max(r, 1))) / c["stretch"]
        if c["far"]:
            s["positions"] = (torch.randint(0, c["far"], (B, 1), generator=gen, device="cuda")
                              + torch.arange(N, device="cuda")).to(torch.int32)
        else:
            s["positions"] = None
        if c["op"] == "qk_norm_grad":
            s["dq_out"] = normal(B, N, c["q_heads"], D).to(dt)
            s["dk_out"] = normal(B, N, c["k_heads"], D).to(dt)
        if own:
            from long_convolution_sequence_rfft_amd import hyena
            s["plan"] = hyena.QKNorm(B, N, c["q_heads"], c["k_heads"], D, io_dtype=_io(hyena, c), norm=c["norm"],
                                     rotary_dim=r, layout=c["layout"], eps=1e-6, freqs=s["freqs"])
        return s
    B, H, dk, dv = c["B"], c["H"], c["dk"], c["dv"]
    if c["op"] == "step":
        s["q"], s["k"], s["v"] = (normal(B, H, d).to(dt) for d in (dk, dk, dv))
        s["k"] = (s["k"].float() / math.sqrt(dk)).to(dt)
        s["g"] = _gates(normal(B, 1, H))[:, 0].contiguous()
        s["state"] = normal(c["slots"], H, dk, dv)
        s["slots"] = torch.randperm(c["slots"], generator=gen, device="cuda")[:B].to(torch.int32)
        if own:
            from long_convolution_sequence_rfft_amd import hyena
            s["plan"] = hyena.Recurrence(B, 1, H, dk, dv, io_dtype=_io(hyena, c))
        return s
    N = c["N"]
    # queries and keys leave the norm dense, values are a slice of the projection
    s["q"] = normal(B, N, H, dk).to(dt)
    s["k"] = (normal(B, N, H, dk) / math.sqrt(dk)).to(dt)
    s["v"] = normal(B, N, H, dk + dv).to(dt)[..., dk:]
    s["g"] = _gates(normal(B, N, H))
    if c["packed"]:  # a document starts where the gate is -inf
        starts = torch.rand((B, N, 1), generator=gen, device="cuda") < 1.0 / 300
        s["g"] = torch.where(starts, torch.full_like(s["g"], -math.inf), s["g"])
    s["lengths"] = None
    if c["ragged"]:
        n = torch.randint(0, N + 1, (B,), generator=gen, device="cuda")
        n[B // 2] = N
        if B >= 3:
            n[0] = 0
        s["lengths"] = n.to(torch.int32)
    s["state"] = normal(B, H, dk, dv) if c["carry"] else None
    grad = c["op"] == "recurrence_grad"
    if grad:
        s["do"] = normal(B, N, H, dv).to(dt)
        s["d_final"] = normal(B, H, dk, dv) if c["carry"] else None
    if own:
        from long_convolution_sequence_rfft_amd import hyena
        s["plan"] = hyena.Recurrence(B, N, H, dk, dv, io_dtype=_io(hyena, c), training=grad)
    return s


def _io(hyena, c):
    return {"f32": hyena.HYENA_F32, "bf16": hyena.HYENA_BF16, "f16": hyena.HYENA_F16}[c["dtype"]]


def _gates(x):
    """Log decays -softplus(x + b): heads from about 3 to about 3000 tokens of memory."""
    H = x.shape[-1]
    b = torch.linspace(-8.0, -1.0, H, device=x.device) if H > 1 else torch.full((1,), -4.0, device=x.device)
    return -torch.nn.functional.softplus(0.5 * x + b)


# ---------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    c = s["case"]
    p = s["plan"]
    if c["op"] == "qk_norm":
        q, k = p.forward(s["q"], s["k"], s["q_weight"], s["k_weight"], positions=s["positions"])
        return dict(q=q, k=k)
    if c["op"] == "qk_norm_grad":
        dq, dk, dqw, dkw = p.backward(s["dq_out"], s["dk_out"], s["q"], s["k"], s["q_weight"], s["k_weight"],
                                      positions=s["positions"])
        return dict(dq=dq, dk=dk, dq_weight=dqw, dk_weight=dkw)
    scale = 1.0 / math.sqrt(c["dk"])
    if c["op"] == "step":
        o = p.step(s["q"], s["k"], s["v"], s["g"], s["state"], scale=scale, slots=s["slots"])
        return dict(o=o, state=s["state"])
    if c["op"] == "recurrence":
        o, last = p.forward(s["q"], s["k"], s["v"], s["g"], scale=scale, state=s["state"], lengths=s["lengths"],
                            return_state=c["carry"])
        return dict(o=o, state=last)
    dq, dk, dv, dg, ds = p.backward(s["do"], s["q"], s["k"], s["v"], s["g"], scale=scale, state=s["state"],
                                    lengths=s["lengths"], d_final=s["d_final"])
    return dict(dq=dq, dk=dk, dv=dv, dg=dg, dstate=ds)


def _run_plain(s):
    op = s["case"]["op"]
    if op == "qk_norm":
        return dict(q=_plain_norm(s, s["q"], s["q_weight"]), k=_plain_norm(s, s["k"], s["k_weight"]))
    if op == "qk_norm_grad":
        dq, dqw = _plain_norm_grad(s, s["dq_out"], s["q"], s["q_weight"])
        dk, dkw = _plain_norm_grad(s, s["dk_out"], s["k"], s["k_weight"])
        return dict(dq=dq, dk=dk, dq_weight=dqw, dk_weight=dkw)
    return {"step": _plain_step, "recurrence": _plain_recurrence, "recurrence_grad": _plain_recurrence_grad}[op](s)


def _angles(s):
    c = s["case"]
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(c["N"], device="cuda")[None]
    a = (pos.double()[..., None] * s["freqs"])[:, :, None, :]
    return a.cos().float(), a.sin().float()


def _pairs(x, c):
    """The two members of each rotated pair, and the channels that stay."""
    r = c["rotary"]
    if c["layout"] == "half":
        return x[..., :r // 2], x[..., r // 2:r], x[..., r:]
    return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]


def _unpairs(a, b, rest, c):
    if c["layout"] == "half":
        return torch.cat([a, b, rest], -1)
    return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)


def _rstd(x, c):
    if c["norm"] == "none":
        return torch.ones_like(x[..., :1])
    n = x.square().sum(-1, keepdim=True)
    return torch.rsqrt((n / c["D"] if c["norm"] == "rms" else n) + 1e-6)


def _plain_norm(s, x, w):
    c = s["case"]
    cos, sin = _angles(s)
    y = x.float() * _rstd(x.float(), c)
    if w is not None:
        y = y * w
    a, b, rest = _pairs(y, c)
    return _unpairs(a * cos - b * sin, a * sin + b * cos, rest, c).to(x.dtype)


def _plain_norm_grad(s, dy, x, w):
    c = s["case"]
    cos, sin = _angles(s)
    a, b, rest = _pairs(dy.float(), c)
    dn = _unpairs(a * cos + b * sin, b * cos - a * sin, rest, c)
    if c["norm"] == "none":
        return dn.to(x.dtype), None
    r = _rstd(x.float(), c)
    xhat = x.float() * r
    dw = (dn * xhat).sum((0, 1, 2), dtype=torch.float64).float()
    t = dn * w
    mean = (t * xhat).sum(-1, keepdim=True) / (c["D"] if c["norm"] == "rms" else 1)
    return ((t - xhat * mean) * r).to(x.dtype), dw


def _plain_step(s):
    q, k, v = (s[n].float() for n in "qkv")
    at = s["slots"].long()
    S = s["state"][at] * s["g"].exp()[..., None, None] + k[..., :, None] * v[..., None, :]
    s["state"][at] = S
    o = (q[..., :, None] * S).sum(-2) / math.sqrt(s["case"]["dk"])
    return dict(o=o.to(s["q"].dtype), state=s["state"])


def _chunks(s, names):
    """Inputs as float32 [B, H, chunks, CHUNK, width], zero at padding; the log
    decays within a chunk, summed in 64 bits; the number of resets so far."""
    c = s["case"]
    B, N, H = c["B"], c["N"], c["H"]
    n = -(-N // CHUNK)
    keep = torch.ones((B, N), dtype=torch.bool, device="cuda")
    if s["lengths"] is not None:
        keep = torch.arange(N, device="cuda") < s["lengths"][:, None]

    def cut(x):
        x = torch.nn.functional.pad(x.transpose(1, 2), (0, 0, 0, n * CHUNK - N))
        return x.reshape(B, H, n, CHUNK, x.shape[-1])

    parts = [cut(torch.where(keep[..., None, None], s[name].float(), 0.0)) for name in names]
    g = cut(torch.where(keep[..., None], s["g"], 0.0)[..., None])[..., 0]
    resets = torch.isneginf(g)
    logs = torch.where(resets, 0.0, g).double().cumsum(-1)
    return parts, logs, resets.long().cumsum(-1), resets, keep


def _uncut(x, c, dtype):
    B, H, n, C, w = x.shape
    return x.reshape(B, H, n * C, w)[:, :, :c["N"]].transpose(1, 2).to(dtype).contiguous()


def _decays(logs, count):
    """exp of the log decays: between the tokens of a chunk (lower triangle),
    from a chunk's start to each token, from each token to the chunk's end, and
    between chunk boundaries: across[i, j] from the end of chunk j - 1 to the
    start of chunk i (row n: the end of the sequence)."""
    n, C = logs.shape[-2:]
    lower = torch.ones((C, C), dtype=torch.bool, device="cuda").tril()
    same = (count[..., :, None] == count[..., None, :]) & lower
    within = torch.where(same, (logs[..., :, None] - logs[..., None, :]).clamp(max=80.0).exp(), 0.0).float()
    head = torch.where(count == 0, logs.exp(), 0.0).float()
    last, total = logs[..., -1:], count[..., -1:]
    tail = torch.where(count == total, (last - logs).exp(), 0.0).float()
    pad = torch.nn.functional.pad
    ends, counts = pad(last[..., 0].cumsum(-1), (1, 0)), pad(total[..., 0].cumsum(-1), (1, 0))
    low = torch.ones((n + 1, n + 1), dtype=torch.bool, device="cuda").tril()
    same = (counts[..., :, None] == counts[..., None, :]) & low
    across = torch.where(same, (ends[..., :, None] - ends[..., None, :]).clamp(max=80.0).exp(), 0.0).float()
    return within, head[..., None], tail[..., None], across


def _states(k, v, tail, across, first):
    """The state before each chunk and, last, the final one."""
    B, H, n, C, dk = k.shape
    local = torch.matmul((k * tail).transpose(-1, -2).contiguous(), v).reshape(B, H, n, -1)
    start = torch.zeros_like(local[:, :, :1]) if first is None else first.reshape(B, H, 1, -1)
    return torch.matmul(across, torch.cat([start, local], 2)).reshape(B, H, n + 1, dk, v.shape[-1])


def _plain_recurrence(s):
    c = s["case"]
    (q, k, v), logs, count, _, _ = _chunks(s, ["q", "k", "v"])
    within, head, tail, across = _decays(logs, count)
    S = _states(k, v, tail, across, s["state"])
    scores = torch.matmul(q, k.transpose(-1, -2).contiguous()) * within
    o = torch.matmul(scores, v) + head * torch.matmul(q, S[:, :, :-1])
    o = _uncut(o / math.sqrt(c["dk"]), c, s["q"].dtype)
    return dict(o=o, state=S[:, :, -1].contiguous() if c["carry"] else None)


def _plain_recurrence_grad(s):
    c = s["case"]
    (q, k, v, do), logs, count, resets, keep = _chunks(s, ["q", "k", "v", "do"])
    B, H, n, C, dk = q.shape
    scale = 1.0 / math.sqrt(c["dk"])
    do = do * scale
    within, head, tail, across = _decays(logs, count)
    S = _states(k, v, tail, across, s["state"])
    # gradients of the states, back from the end: what each chunk's outputs add to the state before it
    local = torch.matmul((q * head).transpose(-1, -2).contiguous(), do).reshape(B, H, n, -1)
    end = torch.zeros_like(local[:, :, :1]) if s["d_final"] is None else s["d_final"].reshape(B, H, 1, -1)
    dS = torch.matmul(across.transpose(-1, -2).contiguous(), torch.cat([local, end], 2)).reshape(B, H, n + 1, dk, -1)
    before, after = S[:, :, :-1], dS[:, :, 1:]
    scores = torch.matmul(q, k.transpose(-1, -2).contiguous()) * within
    dscores = torch.matmul(do, v.transpose(-1, -2).contiguous()) * within
    dq = torch.matmul(dscores, k) + head * torch.matmul(do, before.transpose(-1, -2).contiguous())
    dk_ = torch.matmul(dscores.transpose(-1, -2).contiguous(), q) + tail * torch.matmul(v, after.transpose(-1, -2).contiguous())
    dv = torch.matmul(scores.transpose(-1, -2).contiguous(), do) + tail * torch.matmul(k, after)
    crossing = (q * dq).sum(-1).double() - (k * dk_).sum(-1).double()
    over = (S[:, :, 1:] * after).sum((-1, -2)).double()[..., None]
    dg = torch.where(resets, 0.0, crossing.flip(-1).cumsum(-1).flip(-1) + over)[..., None]
    dg = torch.where(keep[..., None], _uncut(dg, c, torch.float32)[..., 0], 0.0)
    dt = s["q"].dtype
    return dict(dq=_uncut(dq, c, dt), dk=_uncut(dk_, c, dt), dv=_uncut(dv, c, dt), dg=dg,
                dstate=dS[:, :, 0].contiguous() if c["carry"] else None)


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("qk_norm"):
        return _exact_norm(s, op == "qk_norm_grad")
    if op == "step":
        q, k, v, S = (s[n].double() for n in ("q", "k", "v", "state"))
        at = s["slots"].long()
        S[at] = torch.einsum("bh,bhkv->bhkv", s["g"].double().exp(), S[at]) + torch.einsum("bhk,bhv->bhkv", k, v)
        return dict(o=torch.einsum("bhk,bhkv->bhv", q, S[at]) / math.sqrt(case["dk"]), state=S)
    return _exact_recurrence(s, op == "recurrence_grad")


def _exact_norm(s, grad):
    """The rotation as a product of complex numbers, the norm's gradient by the
    Jacobian (I - x x^T / (|x|^2 + c eps)) w / norm."""
    c = s["case"]
    r, D = c["rotary"], c["D"]
    pos = torch.arange(c["N"], device="cuda")[None] if s["positions"] is None else s["positions"]
    turn = torch.polar(torch.ones((), device="cuda", dtype=torch.float64),
                       pos.double()[..., None] * s["freqs"])[:, :, None]
    # channel numbers of the pairs, one pair after the other
    pair = torch.arange(r, device="cuda")
    if c["layout"] == "half":
        pair = pair.reshape(2, r // 2).t().reshape(-1)

    def rotate(y, by):
        z = torch.view_as_complex(y[..., pair].reshape(*y.shape[:-1], r // 2, 2).contiguous()) * by
        y = y.clone()
        y[..., pair] = torch.view_as_real(z).flatten(-2)
        return y

    def norm(x):
        if c["norm"] == "none":
            return torch.ones_like(x[..., :1])
        m = D if c["norm"] == "rms" else 1
        return torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / m + 1e-6)

    def one(x, w, dy):
        x = x.double()
        w = torch.ones(D, device="cuda", dtype=torch.float64) if w is None else w.double()
        n = norm(x)
        if dy is None:
            return rotate(x / n * w, turn)
        dn = rotate(dy.double(), turn.conj())
        if c["norm"] == "none":
            return dn, None
        m = D if c["norm"] == "rms" else 1
        along = torch.linalg.vecdot(x, dn * w)[..., None]
        return dn * w / n - x * along / (m * n ** 3), torch.einsum("bnhd,bnhd->d", dn, x / n)

    if not grad:
        return dict(q=one(s["q"], s["q_weight"], None), k=one(s["k"], s["k_weight"], None))
    dq, dqw = one(s["q"], s["q_weight"], s["dq_out"])
    dk, dkw = one(s["k"], s["k_weight"], s["dk_out"])
    return dict(dq=dq, dk=dk, dq_weight=dqw, dk_weight=dkw)


def _exact_recurrence(s, grad):
    """Token by token."""
    c = s["case"]
    B, N, H, dk, dv = (c[n] for n in ("B", "N", "H", "dk", "dv"))
    scale = 1.0 / math.sqrt(dk)
    n = s["lengths"] if s["lengths"] is not None else torch.full((B,), N, device="cuda")
    live = (torch.arange(N, device="cuda")[None] < n[:, None])[..., None]

    def token_first(x):
        return torch.where(live[..., None], x.double(), 0.0).transpose(0, 1).contiguous()

    q, k, v = (token_first(s[x]) for x in "qkv")
    a = torch.where(live, s["g"].double(), 0.0).exp().transpose(0, 1)[..., None, None]
    S = torch.zeros((B, H, dk, dv), device="cuda", dtype=torch.float64) if s["state"] is None else s["state"].double()
    if not grad:
        o = torch.zeros((N, B, H, dv), device="cuda", dtype=torch.float64)
        for t in range(N):
            S = S * a[t] + k[t][..., None] * v[t][..., None, :]
            o[t] = (S * q[t][..., None]).sum(-2)
        return dict(o=(o * scale).transpose(0, 1).contiguous(), state=S if c["carry"] else None)
    do = token_first(s["do"])
    dq, dk_, dv_ = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for t in range(N):
        S = S * a[t] + k[t][..., None] * v[t][..., None, :]
        dq[t] = (S * do[t][..., None, :]).sum(-1) * scale
    dS = torch.zeros_like(S) if s["d_final"] is None else s["d_final"].double()
    # <S_t, dS_t> = <S_N, dS_N> + sum over later tokens of q.dq - k.dk
    dg = torch.zeros((N, B, H), device="cuda", dtype=torch.float64)
    over = (S * dS).sum((-1, -2))
    for t in range(N - 1, -1, -1):
        dS = dS + q[t][..., None] * (do[t] * scale)[..., None, :]
        dk_[t] = (dS * v[t][..., None, :]).sum(-1)
        dv_[t] = (dS * k[t][..., None]).sum(-2)
        over = over + (q[t] * dq[t]).sum(-1) - (k[t] * dk_[t]).sum(-1)
        dg[t] = over
        dS = dS * a[t]
    back = lambda x: x.transpose(0, 1).contiguous()  # noqa: E731
    dg = torch.where(live & ~torch.isneginf(s["g"]), back(dg), 0.0)
    live = live[..., None]
    return dict(dq=torch.where(live, back(dq), 0.0), dk=torch.where(live, back(dk_), 0.0),
                dv=torch.where(live, back(dv_), 0.0), dg=dg, dstate=dS if c["carry"] else None)
