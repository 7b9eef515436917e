"""Layer norm and the clipped policy loss, each forward and backward: what is timed.

Every case is one pass through one operator, as a training or serving program
makes it. With ``own`` false the operators run in their plain form (elementary
torch operations in binary32, binary64 where binary32 loses what matters); with
``own`` true through this package's entry points.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
CLIP_LOW, CLIP_HIGH, KL = 0.2, 0.28, 0.04


def norm(name, op, M, N, dtype, pdtype="f32", pad=0):
    """pad: elements between a row's end and the next row's start."""
    return {"name": name, "op": op, "M": M, "N": N, "dtype": dtype, "pdtype": pdtype, "pad": pad}


def loss(name, op, M, N, dtype, masked, ref, temperature, pad=0):
    """masked: the share of rows (padding, prompts) whose weight is 0. ref: with a KL term."""
    return {"name": name, "op": op, "M": M, "N": N, "dtype": dtype, "masked": masked, "ref": ref,
            "temperature": temperature, "pad": pad}


def listed():
    return [
        # one token of a decoding step: latency
        norm("norm forward 1x4096 bf16", "norm_forward", 1, 4096, "bf16"),
        # a training batch of 4 x 4096 tokens
        norm("norm forward 16384x4096 bf16", "norm_forward", 16384, 4096, "bf16"),
        # many narrow rows of a width that is no whole 16-byte vector
        norm("norm forward 100003x255 f32", "norm_forward", 100003, 255, "f32"),
        # a small network's step: latency and the weight's gradient
        norm("norm backward 1024x64 f32", "norm_backward", 1024, 64, "f32"),
        # an odd number of tokens, the columns a slice of a wider buffer, 16-bit parameters
        norm("norm backward 8191x1001 f16 pitch 1032", "norm_backward", 8191, 1001, "f16", "f16", pad=31),
        # the widest rows, a large training batch
        norm("norm backward 32768x8192 bf16", "norm_backward", 32768, 8192, "bf16"),
        # the few answer tokens of one short sequence, an odd vocabulary: the rows are split
        loss("loss forward 7x50001 f32", "loss_forward", 7, 50001, "f32", 0.0, True, 1.0),
        # a micro-batch with padding and a sampling temperature, no reference model
        loss("loss forward 4096x32000 bf16", "loss_forward", 4096, 32000, "bf16", 0.25, False, 0.7),
        # a large vocabulary and a long batch
        loss("loss forward 16384x131072 bf16", "loss_forward", 16384, 131072, "bf16", 0.0, True, 1.0),
        # the same short sequence's gradient
        loss("loss backward 7x50001 f32", "loss_backward", 7, 50001, "f32", 0.0, True, 1.0),
        # a micro-batch with padding; fp16 logits, an odd vocabulary
        loss("loss backward 4096x32003 f16", "loss_backward", 4096, 32003, "f16", 0.25, True, 0.7),
        # a large vocabulary
        loss("loss backward 8192x131072 bf16", "loss_backward", 8192, 131072, "bf16", 0.0, False, 1.0),
    ]


def _log_size(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm_forward", "norm_backward", "loss_forward", "loss_backward"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    pad = rng.choice([0, 0, 0, 8, 3, rng.randint(1, 64)])
    if op.startswith("norm"):
        N = _log_size(rng, 16, 8192)
        if rng.random() < 0.5:
            N = -(-N // 8) * 8
        M = _log_size(rng, 1, min(131072, (1 << 28) // (N + pad) * 2 // BYTES[dtype]))
        return {"op": op, "M": M, "N": N, "dtype": dtype, "pdtype": rng.choice(["f32", dtype]), "pad": pad}
    N = _log_size(rng, 500, 131072)
    if rng.random() < 0.5:
        N = -(-N // 8) * 8
    most = (1 << 31) if op == "loss_forward" else (1 << 30)
    M = _log_size(rng, 1, min(16384, most // (N + pad) * 2 // BYTES[dtype]))
    return {"op": op, "M": M, "N": N, "dtype": dtype, "masked": rng.choice([0.0, 0.1, 0.4]),
            "ref": rng.random() < 0.5, "temperature": rng.choice([1.0, 1.0, 0.6, 1.3]), "pad": pad}


def _rows(M, N, pad, dtype, gen, std, mean=0.0):
    """M rows of N values, N + pad elements apart."""
    a = torch.empty(M, N + pad, dtype=DTYPES[dtype], device="cuda")
    a.normal_(mean, std, generator=gen)
    return a[:, :N]


EPS = 1e-5


def _prepare_norm(case, gen):
    M, N, pad = case["M"], case["N"], case["pad"]
    x = _rows(M, N, pad, case["dtype"], gen, 1.3, 0.2)
    pd = DTYPES[case["pdtype"]]
    s = {"op": case["op"], "x": x,
         "gamma": (1 + 0.1 * torch.randn(N, device="cuda", generator=gen)).to(pd),
         "beta": (0.1 * torch.randn(N, device="cuda", generator=gen)).to(pd)}
    if case["op"] == "norm_backward":
        s["dy"] = _rows(M, N, pad, case["dtype"], gen, 1.0)
        mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        for i in range(0, M, 4096):  # what the forward pass of the step has left
            v = x[i:i + 4096].double()
            mean[i:i + 4096] = v.mean(-1)
            rstd[i:i + 4096] = (v.var(-1, unbiased=False) + EPS).rsqrt()
        s["mean"], s["rstd"] = mean, rstd
    return s


def _row_logs(z, tokens, T):
    """Each row's maximum, log of its sum, and its token's log probability, in binary64, a few rows at a time."""
    M, N = z.shape
    step = max(1, (1 << 26) // N)
    top, log, lp = (torch.empty(M, dtype=torch.float64, device=z.device) for _ in range(3))
    for i in range(0, M, step):
        v = z[i:i + step].double()
        a = v.amax(-1)
        v.sub_(a[:, None]).div_(T)
        hit = v.gather(1, tokens[i:i + step, None])[:, 0]
        b = v.exp_().sum(-1).log()
        top[i:i + step], log[i:i + step], lp[i:i + step] = a, b, hit - b
    return top, log, lp


def _prepare_loss(case, gen):
    M, N, T = case["M"], case["N"], case["temperature"]
    z = _rows(M, N, case["pad"], case["dtype"], gen, 2.5)
    tokens = torch.randint(0, N, (M,), device="cuda", generator=gen)
    # sampled tokens are likely ones: lift the token's logit
    z.scatter_add_(1, tokens[:, None], (6 * torch.rand(M, 1, device="cuda", generator=gen)).to(z.dtype))
    top, log, lp = _row_logs(z, tokens, T)
    # The policy has moved a little since the tokens were drawn. A ratio on a clip border up to rounding
    # has no gradient that both sides could agree on: such rows are moved off it.
    step = 0.12 * torch.randn(M, device="cuda", generator=gen)
    old = (lp - step).float()
    for border in (1 - CLIP_LOW, 1 + CLIP_HIGH):
        near = ((lp - old.double()).exp() - border).abs() < 1e-4
        old = torch.where(near, old - 1e-3, old)
    s = {"op": case["op"], "logits": z, "tokens": tokens, "old": old, "temperature": T,
         "advantage": torch.randn(M, device="cuda", generator=gen),
         "ref": (lp + 0.1 * torch.randn(M, device="cuda", generator=gen)).float() if case["ref"] else None}
    counted = torch.rand(M, device="cuda", generator=gen) >= case["masked"]
    s["weight"] = counted.float() / counted.sum().clamp(min=1)
    if case["masked"]:
        s["tokens"] = torch.where(counted, tokens, -100)  # what a padded batch holds there
    if case["op"] == "loss_backward":
        r = (lp - old.double()).exp()
        A = s["advantage"].double()
        d = -torch.where(r * A <= r.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * A, r * A, 0.0)
        if case["ref"]:
            d = d + KL * (1 - (s["ref"].double() - lp).exp())
        zero = torch.zeros((), dtype=torch.float64, device="cuda")
        s["coef"] = torch.where(counted, s["weight"] * d, zero).float()
        s["stats"] = torch.where(counted[:, None], torch.stack([top, log], 1), zero).float()
        # the loss is one of two that are averaged; fp16 gradients are scaled
        s["grad"] = torch.full((1,), 4096.0 if case["dtype"] == "f16" else 0.5, device="cuda")
    return s


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(int(seed))
    return (_prepare_norm if case["op"].startswith("norm") else _prepare_loss)(case, gen)


# ---- the plain forms ------------------------------------------------------------------------

def _norm_forward(s):
    x = s["x"].float()
    mean = x.sum(-1) / x.shape[1]
    c = x - mean[:, None]
    rstd = ((c * c).sum(-1) / x.shape[1] + EPS) ** -0.5
    y = c * rstd[:, None] * s["gamma"].float() + s["beta"].float()
    return y.to(s["x"].dtype), mean, rstd


def _norm_backward(s):
    x, dy, N = s["x"].float(), s["dy"].float(), s["x"].shape[1]
    h = (x - s["mean"][:, None]) * s["rstd"][:, None]
    dgamma, dbeta = (dy * h).sum(0), dy.sum(0)
    g = dy * s["gamma"].float()
    a, b = g.sum(-1, keepdim=True) / N, (g * h).sum(-1, keepdim=True) / N
    dx = (g - a - h * b) * s["rstd"][:, None]
    return dx.to(s["x"].dtype), dgamma.to(s["gamma"].dtype), dbeta.to(s["beta"].dtype)


def _loss_forward(s):
    counted = s["weight"] != 0
    z = s["logits"].float()
    top = z.amax(-1)
    e = (z - top[:, None]) / s["temperature"]
    hit = e.gather(1, s["tokens"].clamp(min=0)[:, None])[:, 0]
    log = e.exp().sum(-1).double().log()
    lp = hit.double() - log
    # ratios next to a clip border, and exp(d) - d - 1 for a small d, need binary64
    A, w = s["advantage"].double(), s["weight"].double()
    r = (lp - s["old"].double()).exp()
    c = r.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH)
    each = -torch.minimum(r * A, c * A)
    d = -torch.where(r * A <= c * A, r * A, 0.0)
    if s["ref"] is not None:
        q = s["ref"].double() - lp
        each = each + KL * (q.exp() - q - 1)
        d = d + KL * (1 - q.exp())
    total = torch.where(counted, w * each, 0.0).sum()
    stats = torch.stack([top.double(), log], 1)
    return (total.float(), torch.where(counted, lp, 0.0).float(),
            torch.where(counted[:, None], stats, 0.0).float(), torch.where(counted, w * d, 0.0).float())


def _loss_backward(s):
    z, T = s["logits"].float(), s["temperature"]
    p = ((z - s["stats"][:, :1]) / T - s["stats"][:, 1:]).exp()
    hit = torch.arange(z.shape[1], device=z.device) == s["tokens"][:, None]
    a = (s["grad"] * s["coef"] / T)[:, None]
    return torch.where(a == 0, 0.0, a * (hit.float() - p)).to(s["logits"].dtype)


PLAIN = {"norm_forward": _norm_forward, "norm_backward": _norm_backward, "loss_forward": _loss_forward,
         "loss_backward": _loss_backward}


def _own(s):
    import elementwise_reduction_b200 as dyt

    if s["op"] == "norm_forward":
        return dyt.layer_norm_forward(s["x"], s["gamma"], s["beta"], eps=EPS)
    if s["op"] == "norm_backward":
        return dyt.layer_norm_backward(s["x"], s["dy"], s["mean"], s["rstd"], s["gamma"], s["beta"])
    if s["op"] == "loss_forward":
        return dyt.policy_loss_forward(s["logits"], s["tokens"], s["old"], s["advantage"], ref_logp=s["ref"],
                                       weight=s["weight"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_coef=KL,
                                       temperature=s["temperature"])
    return dyt.policy_loss_backward(s["logits"], s["tokens"], s["stats"], s["coef"], grad=s["grad"],
                                    temperature=s["temperature"])


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


def work(case):
    M, N, e = case["M"], case["N"], BYTES[case["dtype"]]
    if case["op"] == "norm_forward":
        return {"bytes": 2 * M * N * e + 8 * M + 2 * N * BYTES[case["pdtype"]], "flops": 8 * M * N}
    if case["op"] == "norm_backward":
        return {"bytes": 3 * M * N * e + 8 * M + 3 * N * BYTES[case["pdtype"]], "flops": 15 * M * N}
    read = (1 - case["masked"]) * M * N * e  # rows of weight 0 need no logits
    row = 8 + 4 + 4 + 4 + (4 if case["ref"] else 0)
    if case["op"] == "loss_forward":
        return {"bytes": read + (row + 16) * M + 4, "flops": 4 * (1 - case["masked"]) * M * N}
    return {"bytes": read + M * N * e + 20 * M, "flops": 4 * (1 - case["masked"]) * M * N}


# ---- the definitions in binary64, a block of rows at a time --------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s)
    return _exact_loss(s)


def _exact_norm(s):
    M, N = s["x"].shape
    gamma, beta = s["gamma"].double(), s["beta"].double()
    step = max(1, (1 << 25) // N)
    blocks = [slice(i, min(M, i + step)) for i in range(0, M, step)]
    if s["op"] == "norm_forward":
        y = torch.empty(M, N, dtype=torch.float64, device="cuda")
        mean = torch.empty(M, dtype=torch.float64, device="cuda")
        rstd = torch.empty_like(mean)
        for b in blocks:
            x = s["x"][b].double()
            mean[b] = x.mean(-1)
            rstd[b] = 1 / torch.sqrt(x.var(-1, unbiased=False) + EPS)
            y[b] = torch.addcmul(beta, (x - mean[b, None]) * rstd[b, None], gamma)
        return y, mean, rstd
    dx = torch.empty(M, N, dtype=torch.float64, device="cuda")
    dgamma, dbeta = torch.zeros_like(gamma), torch.zeros_like(gamma)
    for b in blocks:
        r = s["rstd"][b, None].double()
        h = (s["x"][b].double() - s["mean"][b, None].double()) * r
        dy = s["dy"][b].double()
        dgamma += torch.einsum("ij,ij->j", dy, h)
        dbeta += dy.sum(0)
        g = dy * gamma
        dx[b] = r * (g - g.mean(-1, keepdim=True) - h * (g * h).mean(-1, keepdim=True))
    return dx, dgamma, dbeta


def _exact_loss(s):
    z, T = s["logits"], s["temperature"]
    M, N = z.shape
    tokens = s["tokens"].clamp(min=0)
    if s["op"] == "loss_backward":
        if M * N > 1 << 30:
            return None
        out = torch.empty(M, N, dtype=torch.float64, device="cuda")
        step = max(1, (1 << 25) // N)
        for i in range(0, M, step):
            b = slice(i, min(M, i + step))
            stats, a = s["stats"][b].double(), s["grad"].double() * s["coef"][b].double() / T
            v = -torch.exp((z[b].double() - stats[:, :1]) / T - stats[:, 1:])
            v[torch.arange(v.shape[0], device="cuda"), tokens[b]] += 1
            out[b] = torch.where(a[:, None] != 0, v * a[:, None], torch.zeros_like(v))
        return out
    top, log, lp = _row_logs(z, tokens, T)
    w, A = s["weight"].double(), s["advantage"].double()
    ratio = torch.exp(lp - s["old"].double())
    # the clipped side holds where it is the smaller: above for a positive advantage, below for a negative
    held = torch.where(A > 0, ratio > 1 + CLIP_HIGH, (ratio < 1 - CLIP_LOW) & (A < 0))
    border = torch.where(A > 0, torch.full_like(A, 1 + CLIP_HIGH), torch.full_like(A, 1 - CLIP_LOW))
    each = torch.where(held, -border * A, -ratio * A)
    d = torch.where(held, torch.zeros_like(A), -ratio * A)
    if s["ref"] is not None:
        q = s["ref"].double() - lp
        each = each + KL * (torch.expm1(q) - q)
        d = d - KL * torch.expm1(q)
    on = (w != 0).double()
    return (w * each).sum(), lp * on, torch.stack([top, log], 1) * on[:, None], d * w
