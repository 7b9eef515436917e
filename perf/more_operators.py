"""Root-mean-square norm with the residual's addition and log probabilities with
entropy and top alternatives, each forward and backward: what is timed.

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


def norm(name, op, M, N, dtype, residual, pdtype="f32", pad=0, group=0):
    """residual: forward, the block's input that is added first; backward, the gradient that its sum
    receives from later layers. pad: elements between a row's end and the next row's start. group:
    columns that share a scale of the 8-bit output (0: the whole row)."""
    return {"name": name, "op": op, "M": M, "N": N, "dtype": dtype, "residual": residual, "pdtype": pdtype,
            "pad": pad, "group": group}


def logps(name, op, M, N, dtype, top, masked, temperature=1.0, pad=0):
    """top: alternatives reported of each row (the backward has none). masked: the share of rows
    (padding, prompts) whose token is -100."""
    return {"name": name, "op": op, "M": M, "N": N, "dtype": dtype, "top": top, "masked": masked,
            "temperature": temperature, "pad": pad}


def listed():
    return [
        # one token of a decoding step: latency
        norm("rms forward 1x4096 bf16", "rms_forward", 1, 4096, "bf16", True),
        # a training batch of 4 x 4096 tokens
        norm("rms forward 16384x4096 bf16", "rms_forward", 16384, 4096, "bf16", True),
        # a decoding step of 64 requests, a scale for every 128 columns
        norm("rms quantize 64x8192 bf16", "rms_quantize", 64, 8192, "bf16", True, "bf16", group=128),
        # odd rows, the columns a slice of a wider buffer, no residual, a scale a row
        norm("rms quantize 8191x1001 f16", "rms_quantize", 8191, 1001, "f16", False, "f16", pad=31),
        # the prompts of a large serving batch
        norm("rms quantize 16384x8192 bf16", "rms_quantize", 16384, 8192, "bf16", True, "bf16"),
        # many narrow rows of a width that is no whole 16-byte vector, as in a norm over heads
        norm("rms backward 100003x255 f32", "rms_backward", 100003, 255, "f32", False),
        # the widest rows, a large training batch, inside a residual network
        norm("rms backward 32768x8192 bf16", "rms_backward", 32768, 8192, "bf16", True),
        # a few requests' next tokens, an odd vocabulary: the rows are split
        logps("logp forward 7x50001 f32", "logp_forward", 7, 50001, "f32", 20, 0.0),
        # the tokens of a micro-batch with prompts and padding, for a policy loss
        logps("logp forward 4096x32000 bf16", "logp_forward", 4096, 32000, "bf16", 0, 0.25, 0.7),
        # a large vocabulary, long sequences scored for distillation
        logps("logp forward 8192x131072 bf16", "logp_forward", 8192, 131072, "bf16", 8, 0.0),
        # a short answer's gradient
        logps("logp backward 7x50001 f32", "logp_backward", 7, 50001, "f32", 0, 0.0),
        # a micro-batch's gradient with an entropy bonus; fp16 logits, an odd vocabulary
        logps("logp backward 4096x32003 f16", "logp_backward", 4096, 32003, "f16", 0, 0.25, 0.7),
    ]


def _log_size(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rms_forward", "rms_quantize", "rms_backward", "logp_forward", "logp_backward"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    pad = rng.choice([0, 0, 0, 8, 3, rng.randint(1, 64)])
    if op.startswith("rms"):
        N = _log_size(rng, 16, 8192)
        if rng.random() < 0.5:
            N = -(-N // 8) * 8
        M = _log_size(rng, 1, min(131072, (1 << 28) // (N + pad) * 2 // BYTES[dtype]))
        return {"op": op, "M": M, "N": N, "dtype": dtype, "residual": rng.random() < 0.6,
                "pdtype": rng.choice(["f32", dtype]), "pad": pad,
                "group": rng.choice([0, 128]) if op == "rms_quantize" else 0}
    N = _log_size(rng, 500, 131072)
    if rng.random() < 0.5:
        N = -(-N // 8) * 8
    M = _log_size(rng, 1, min(16384, (1 << 30) // (N + pad) * 2 // BYTES[dtype]))
    return {"op": op, "M": M, "N": N, "dtype": dtype, "masked": rng.choice([0.0, 0.1, 0.4]),
            "top": rng.choice([0, 1, 5, 20, rng.randint(1, 32)]) if op == "logp_forward" else 0,
            "temperature": rng.choice([1.0, 1.0, 0.6, 1.3]), "pad": pad}


def _rows(M, N, pad, dtype, gen, std, mean=0.0):
    """M rows of N values, N + pad elements apart."""
    a = torch.empty(M, N + pad, dtype=DTYPES[dtype], device="cuda")
    a.normal_(mean, std, generator=gen)
    return a[:, :N]


EPS = 1e-6


def _prepare_norm(case, gen):
    M, N, pad = case["M"], case["N"], case["pad"]
    s = {"op": case["op"], "group": case["group"],
         "gamma": (1 + 0.1 * torch.randn(N, device="cuda", generator=gen)).to(DTYPES[case["pdtype"]]),
         "x": _rows(M, N, pad, case["dtype"], gen, 1.0),
         "residual": _rows(M, N, pad, case["dtype"], gen, 2.0, 0.1) if case["residual"] else None}
    if case["op"] == "rms_backward":
        s["dy"] = _rows(M, N, pad, case["dtype"], gen, 1.0)
        s["rstd"] = torch.empty(M, device="cuda")
        for i in range(0, M, 4096):  # what the forward pass of the step has left
            s["rstd"][i:i + 4096] = (s["x"][i:i + 4096].double().square().mean(-1) + EPS).rsqrt()
    return s


def _blocks(M, N, most=1 << 26):
    step = max(1, most // N)
    return [slice(i, min(M, i + step)) for i in range(0, M, step)]


def _prepare_logps(case, gen):
    M, N, T = case["M"], case["N"], case["temperature"]
    z = _rows(M, N, case["pad"], case["dtype"], gen, 2.5)
    tokens = torch.randint(0, N, (M,), device="cuda", generator=gen)
    # sampled tokens are likely ones: lift the token's logit
    z.scatter_add_(1, tokens[:, None], (6 * torch.rand(M, 1, device="cuda", generator=gen)).to(z.dtype))
    # eight sequences: a prompt before the answer and padding behind it, `masked` of the rows together
    length = -(-M // 8)
    out = int(length * case["masked"])
    at = torch.arange(M, device="cuda") % length
    prompt = (torch.rand(8, device="cuda", generator=gen) * (out + 1)).long()[torch.arange(M, device="cuda") // length]
    counted = (at >= prompt) & (at < prompt + length - out)
    s = {"op": case["op"], "logits": z, "tokens": torch.where(counted, tokens, -100), "top": case["top"],
         "temperature": T}
    if case["op"] == "logp_backward":
        stats, entropy = torch.zeros(M, 2, device="cuda"), torch.zeros(M, device="cuda")
        for b in _blocks(M, N):  # what the forward pass of the step has left
            v = z[b].double()
            m = v.amax(-1)
            v.sub_(m[:, None]).div_(T)
            log = v.exp().sum(-1).log()
            h = log - (v * (v - log[:, None]).exp()).sum(-1)
            on = counted[b]
            stats[b, 0], stats[b, 1], entropy[b] = m.float() * on, log.float() * on, h.float() * on
        s["stats"], s["entropy"] = stats, entropy
        scale = 64.0 if case["dtype"] == "f16" else 1.0  # fp16 gradients are scaled
        s["grad"] = scale * torch.randn(M, device="cuda", generator=gen)
        s["grad_entropy"] = scale * 0.1 * torch.rand(M, device="cuda", generator=gen)
    return s


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(int(seed))
    return (_prepare_norm if case["op"].startswith("rms") else _prepare_logps)(case, gen)


# ---- the plain forms ------------------------------------------------------------------------

QMAX, LEAST = 448.0, 2.0 ** -100  # the largest value of 8-bit floats with 3 bits behind the point; a scale's numerator


def _normed(s):
    """The sum with the residual, the rows' factors and the norm, in binary32."""
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    rstd = ((h * h).sum(-1) / h.shape[1] + EPS) ** -0.5
    return h, rstd, h * rstd[:, None] * s["gamma"].float()


def _rms_forward(s):
    h, rstd, y = _normed(s)
    dtype = s["x"].dtype
    return (y.to(dtype), h.to(dtype), rstd) if s["residual"] is not None else (y.to(dtype), rstd)


def _rms_quantize(s):
    h, _, y = _normed(s)
    M, N = y.shape
    group = s["group"] or N
    y = torch.cat([y, y.new_zeros(M, -N % group)], 1).view(M, -1, group) if N % group else y.view(M, -1, group)
    scale = torch.maximum(y.abs().amax(-1), y.new_tensor(LEAST)) / QMAX
    q = (y / scale[..., None]).view(M, -1)[:, :N].to(torch.float8_e4m3fn)
    scale = scale if s["group"] else scale[:, 0]
    return (q, scale, h.to(s["x"].dtype)) if s["residual"] is not None else (q, scale)


def _rms_backward(s):
    h, dy, r = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    n = h * r
    dgamma = (dy * n).sum(0)
    g = dy * s["gamma"].float()
    dx = (g - n * ((g * n).sum(-1, keepdim=True) / h.shape[1])) * r
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    return dx.to(s["x"].dtype), dgamma.to(s["gamma"].dtype)


def _logp_forward(s):
    z, K, counted = s["logits"].float(), s["top"], s["tokens"] != -100
    m = z.amax(-1)
    e = (z - m[:, None]) / s["temperature"]
    hit = e.gather(1, s["tokens"].clamp(min=0)[:, None])[:, 0]
    p = e.exp()
    total = p.sum(-1)
    log = total.double().log()
    entropy = log - ((p * e).sum(-1) / total).double()
    out = [torch.where(counted, v, 0.0).float() for v in (hit.double() - log, entropy)]
    stats = torch.where(counted[:, None], torch.stack([m.double(), log], 1), 0.0).float()
    if K == 0:
        return (*out, stats)
    del p
    # a whole number for each logit, in the logits' order, the lower column first among equal ones
    N = z.shape[1]
    v = (z + 0.0).view(torch.int32)
    key = torch.where(v < 0, v ^ 0x7FFFFFFF, v).long() * (1 << 32) + torch.arange(N - 1, -1, -1, device=z.device)
    ids = N - 1 - (key.topk(K, -1).values & 0xFFFFFFFF)
    best = torch.where(counted[:, None], e.gather(1, ids).double() - log[:, None], 0.0).float()
    return (*out, best, torch.where(counted[:, None], ids, -1), stats)


def _logp_backward(s):
    z, T, counted = s["logits"].float(), s["temperature"], (s["tokens"] != -100)[:, None]
    lp = (z - s["stats"][:, :1]) / T - s["stats"][:, 1:]
    p = lp.exp()
    hit = torch.arange(z.shape[1], device=z.device) == s["tokens"][:, None]
    a, b = s["grad"][:, None] / T, s["grad_entropy"][:, None] / T
    dz = a * (hit.float() - p) - b * (p * (lp + s["entropy"][:, None]))
    return torch.where(counted, dz, 0.0).to(s["logits"].dtype)


PLAIN = {"rms_forward": _rms_forward, "rms_quantize": _rms_quantize, "rms_backward": _rms_backward,
         "logp_forward": _logp_forward, "logp_backward": _logp_backward}


def _own(s):
    import elementwise_reduction_b200 as dyt

    if s["op"] == "rms_forward":
        y, h, rstd = dyt.rms_norm_forward(s["x"], s["gamma"], residual=s["residual"], eps=EPS)
        return (y, h, rstd) if s["residual"] is not None else (y, rstd)
    if s["op"] == "rms_quantize":
        q, scale, h = dyt.rms_norm_quantize(s["x"], s["gamma"], residual=s["residual"], eps=EPS, group=s["group"])
        return (q, scale, h) if s["residual"] is not None else (q, scale)
    if s["op"] == "rms_backward":
        return dyt.rms_norm_backward(s["x"], s["dy"], s["rstd"], s["gamma"], dresidual=s["residual"])
    if s["op"] == "logp_forward":
        logp, entropy, best, ids, stats = dyt.log_probs_forward(s["logits"], s["tokens"], top=s["top"],
                                                                temperature=s["temperature"])
        return (logp, entropy, best, ids, stats) if s["top"] else (logp, entropy, stats)
    return dyt.log_probs_backward(s["logits"], s["tokens"], s["stats"], s["entropy"], grad_logp=s["grad"],
                                  grad_entropy=s["grad_entropy"], temperature=s["temperature"])


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


def work(case):
    M, N, e = case["M"], case["N"], BYTES[case["dtype"]]
    if case["op"].startswith("rms"):
        res, gamma = case["residual"], N * BYTES[case["pdtype"]]
        if case["op"] == "rms_forward":
            return {"bytes": (4 if res else 2) * M * N * e + 4 * M + gamma, "flops": (5 if res else 4) * M * N}
        if case["op"] == "rms_quantize":
            scales = -(-N // case["group"]) if case["group"] else 1
            return {"bytes": M * N * ((3 if res else 1) * e + 1) + 4 * M * scales + gamma,
                    "flops": (7 if res else 6) * M * N}
        return {"bytes": (4 if res else 3) * M * N * e + 4 * M + 2 * gamma, "flops": (10 if res else 9) * M * N}
    length = -(-M // 8)
    read = (1 - int(length * case["masked"]) / length) * M * N  # rows that do not count need no logits
    if case["op"] == "logp_forward":
        return {"bytes": read * e + (8 + 16 + 12 * case["top"]) * M, "flops": 6 * read}
    return {"bytes": (read + M * N) * e + (8 + 20) * M, "flops": 7 * read}


# ---- the definitions in binary64, a block of rows at a time --------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rms_forward": _exact_norm, "rms_quantize": _exact_norm, "rms_backward": _exact_norm_backward,
            "logp_forward": _exact_logps, "logp_backward": _exact_logps_backward}[case["op"]](s)


def _exact_norm(s):
    M, N = s["x"].shape
    gamma, group = s["gamma"].double(), s["group"] or N
    ys, hs, rs, scales = [], [], [], []
    for b in _blocks(M, N, 1 << 25):
        h = s["x"][b].double()
        if s["residual"] is not None:
            h += s["residual"][b]
        r = 1 / torch.sqrt(torch.einsum("ij,ij->i", h, h) / N + EPS)
        y = torch.einsum("ij,i,j->ij", h, r, gamma)
        if s["op"] == "rms_quantize":
            parts = y.split(group, 1)
            scale = torch.stack([p.abs().amax(1).clamp(min=LEAST) / QMAX for p in parts], 1)
            y = torch.cat([p / scale[:, k:k + 1] for k, p in enumerate(parts)], 1)
            scales.append(scale if s["group"] else scale[:, 0])
        ys.append(y), hs.append(h if s["residual"] is not None else None), rs.append(r)
    last = torch.cat(scales if scales else rs)
    if s["residual"] is None:
        return torch.cat(ys), last
    # the forward gives (y, h, rstd), the 8-bit output (q, scale, h)
    return (torch.cat(ys), last, torch.cat(hs)) if scales else (torch.cat(ys), torch.cat(hs), last)


def _exact_norm_backward(s):
    M, N = s["x"].shape
    gamma = s["gamma"].double()
    dgamma, dx = torch.zeros_like(gamma), torch.empty(M, N, dtype=torch.float64, device="cuda")
    for b in _blocks(M, N, 1 << 25):
        h, r, dy = s["x"][b].double(), s["rstd"][b].double(), s["dy"][b].double()
        dgamma += torch.einsum("ij,ij,i->j", dy, h, r)
        g = dy * gamma
        dot = torch.einsum("ij,ij->i", g, h)
        # d(h_j rstd)/dh_k = rstd [j = k] - rstd^3 h_j h_k / N
        dx[b] = g * r[:, None] - h * (dot * r ** 3 / N)[:, None]
        if s["residual"] is not None:
            dx[b] += s["residual"][b]
    return dx, dgamma


def _exact_logps(s):
    z, T, K = s["logits"], s["temperature"], s["top"]
    M, N = z.shape
    on = s["tokens"] != -100
    tokens = torch.where(on, s["tokens"], 0)
    logp, entropy, top, log = (torch.empty(M, dtype=torch.float64, device="cuda") for _ in range(4))
    best = torch.empty(M, K, dtype=torch.float64, device="cuda")
    ids = torch.empty(M, K, dtype=torch.int64, device="cuda")
    for b in _blocks(M, N, 1 << 25):
        v = z[b].double()
        if K:
            order = z[b].sort(dim=-1, descending=True, stable=True).indices[:, :K]
        lp = torch.log_softmax(v / T, -1)
        logp[b] = lp[torch.arange(lp.shape[0], device="cuda"), tokens[b]]
        entropy[b] = -(lp.exp() * lp).sum(-1)
        top[b] = v.amax(-1)
        log[b] = top[b] / T + torch.log(torch.exp(v / T - top[b, None] / T).sum(-1)) - top[b] / T
        if K:
            best[b], ids[b] = lp.gather(1, order), order
    keep = on.double()
    out = (logp * keep, entropy * keep)
    stats = torch.stack([top, log], 1) * keep[:, None]
    if K == 0:
        return (*out, stats)
    return (*out, best * keep[:, None], torch.where(on[:, None], ids, -1), stats)


def _exact_logps_backward(s):
    z, T = s["logits"], s["temperature"]
    M, N = z.shape
    out = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    for b in _blocks(M, N, 1 << 25):
        lp = (z[b].double() - s["stats"][b, :1].double()) / T - s["stats"][b, 1:].double()
        a, e = s["grad"][b].double(), s["grad_entropy"][b].double()
        v = torch.exp(lp) * -(a[:, None] + e[:, None] * (lp + s["entropy"][b, None].double()))
        on = s["tokens"][b] != -100
        v[torch.arange(v.shape[0], device="cuda"), s["tokens"][b].clamp(min=0)] += a
        out[b] = torch.where(on[:, None], v / T, torch.zeros_like(v))
    return out
