"""The policy loss's kernels against its binary64 formulas: vocabularies from one
token, rows that are split and rows that share a CTA, masked rows, -inf and NaN
logits, strides, dtypes, gradients, and refusals."""
from __future__ import annotations

import pytest
import torch

from tests import row_helpers as R

pytestmark = pytest.mark.gpu

LO, HI, KL = 0.2, 0.28, 0.05
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")


def dyt():
    import elementwise_reduction_b200 as d
    return d


class Case:
    def __init__(self, M, N, dtype="f32", pitch=None, offset=0, T=1.0, ref=True, masked=0.0, seed=0, std=2.0,
                 token_dtype=torch.int64):
        g = torch.Generator("cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.z = R.Guarded(M, N, R.DT[dtype], pitch, offset)
        self.z.set(r(M, N) * std)
        self.tokens = torch.randint(0, N, (M,), device="cuda", generator=g).to(token_dtype)
        self.adv, self.T = r(M), T
        x = self.z.t.double() / T
        lp = (x - x.logsumexp(-1, keepdim=True)).gather(1, self.tokens.long()[:, None])[:, 0]
        # ratios on both sides of the clip range and inside it, none within 1e-3 of its ends
        step = torch.rand(M, device="cuda", generator=g) * 0.18 - 0.09
        step += torch.tensor([-0.6, 0.0, 0.0, 0.6], device="cuda")[torch.arange(M, device="cuda") % 4]
        self.old = (lp - step).float()
        self.ref = (lp + 0.3 * r(M)).float() if ref else None
        self.weight = None
        if masked:
            on = torch.rand(M, device="cuda", generator=g) >= masked
            on[0] = True
            self.weight = on.float() / on.sum()
            self.tokens = torch.where(on, self.tokens, torch.full_like(self.tokens, -100))

    def forward(self, **kw):
        return dyt().policy_loss_forward(self.z.t, self.tokens, self.old, self.adv, self.ref, self.weight, LO, HI,
                                         KL, self.T, **kw)

    def want_forward(self):
        return R.loss_forward(self.z.t, self.tokens, self.old, self.adv, self.ref, self.weight, LO, HI, KL, self.T)

    def check_forward(self):
        got = self.forward()
        info = dyt().dyt_last_launch_info()
        want, tol = self.want_forward()
        for g, w, t, name in zip(got, want, tol, ("loss", "logp", "stats", "coef")):
            assert g.dtype == torch.float32
            R.assert_close(g, w, t, name)
        return got, info

    def check_backward(self, got, grad=None, out_pitch=None, out_offset=0):
        M, N = self.z.t.shape
        dz = R.Guarded(M, N, self.z.t.dtype, out_pitch, out_offset, fill=5.0)
        gt = None if grad is None else torch.tensor([grad], device="cuda")
        dyt().policy_loss_backward(self.z.t, self.tokens, got[2], got[3], gt, self.T, dlogits=dz.t)
        info = dyt().dyt_last_launch_info()
        want, tol = R.loss_backward(self.z.t, self.tokens, got[2], got[3], 1.0 if grad is None else grad, self.T)
        R.assert_close(dz.t, want, tol + R.half_step(dz.t.dtype, want), "dlogits")
        dz.assert_surroundings_untouched("dlogits")
        return info


WIDTHS = [1, 2, 3, 7, 8, 9, 15, 31, 33, 64, 100, 255, 257, 1000, 1024, 2049, 4096, 5003, 16384, 50001]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", WIDTHS)
def test_widths(N, dtype):
    c = Case(7, N, dtype)
    got, info = c.check_forward()
    assert info["op"] == 7 and info["kernels"] == 2
    assert c.check_backward(got, grad=1000.0)["op"] == 8


@pytest.mark.parametrize("M", [1, 2, 5, 64, 65, 1183, 1184, 1185, 5000])
@pytest.mark.parametrize("N,dtype", [(515, "bf16"), (2051, "f32")])
def test_row_counts(M, N, dtype):
    c = Case(M, N, dtype, masked=0.3 if M > 2 else 0.0, T=0.7)
    got, _ = c.check_forward()
    c.check_backward(got, grad=100.0)


def test_paths():
    # many short rows are whole items, few or long ones are split; the backward gives a warp or a CTA to a row
    def both(M, N):
        c = Case(M, N, "bf16")
        got, fwd = c.check_forward()
        return fwd, c.check_backward(got)
    fwd, bwd = both(3000, 1000)
    assert fwd["col_chunks"] == 1 and bwd["path"] == 1
    fwd, bwd = both(1500, 8200)
    assert 1 < fwd["col_chunks"] <= 8 and bwd["path"] == 2 and bwd["col_chunks"] == 1
    fwd, bwd = both(2, 60000)
    assert fwd["col_chunks"] > 8 and bwd["col_chunks"] > 8


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,pitch,offset,out_pitch,out_offset", [
    (64, 72, 0, 64, 0), (64, 64, 1, 64, 1), (64, 65, 0, 67, 3), (1000, 1001, 2, 1000, 0), (4097, 4100, 1, 4099, 2),
    (9001, 9001, 3, 9001, 1), (9001, 9003, 0, 9005, 7), (20, 21, 1, 20, 0), (3, 3, 1, 3, 2)])
def test_strides_and_offsets(N, pitch, offset, out_pitch, out_offset, dtype):
    for M in (9, 1300):
        c = Case(M, N, dtype, pitch=pitch, offset=offset)
        got, _ = c.check_forward()
        c.check_backward(got, grad=30.0, out_pitch=out_pitch, out_offset=out_offset)


@pytest.mark.parametrize("T", [0.3, 1.0, 2.5])
@pytest.mark.parametrize("ref", [False, True])
def test_temperature_and_reference(T, ref):
    c = Case(21, 3001, "bf16", T=T, ref=ref)
    got, _ = c.check_forward()
    c.check_backward(got)


def test_int32_tokens_and_default_weight():
    a, b = Case(13, 700), Case(13, 700, token_dtype=torch.int32)
    ga, gb = a.forward(), b.forward()
    assert all(torch.equal(x, y) for x, y in zip(ga, gb))
    w = torch.full((13,), 1 / 13, device="cuda")
    a.weight = w
    want = a.want_forward()
    R.assert_close(ga[0], want[0][0], want[1][0] + 2 * R.U * want[0][0].abs(), "loss")
    assert torch.equal(dyt().policy_loss_backward(a.z.t, a.tokens, ga[2], ga[3]),
                       dyt().policy_loss_backward(b.z.t, b.tokens, gb[2], gb[3]))


@pytest.mark.parametrize("M,N", [(40, 600), (2000, 300), (40, 9000)])
def test_rows_without_weight_are_not_used(M, N):
    c = Case(M, N, "bf16", masked=0.5)
    clean = c.forward()
    dclean = dyt().policy_loss_backward(c.z.t, c.tokens, clean[2], clean[3])
    off = c.weight == 0
    assert off.any()
    c.z.t[off] = NAN
    for t in (c.old, c.adv, c.ref):
        t[off] = NAN
    got = c.forward()
    assert all(torch.equal(a, b) for a, b in zip(got, clean))
    assert not any(torch.isnan(t).any() for t in got)
    dz = dyt().policy_loss_backward(c.z.t, c.tokens, got[2], got[3])
    assert torch.equal(dz, dclean) and torch.equal(dz[off], torch.zeros_like(dz[off]))
    c.weight = torch.zeros_like(c.weight)
    assert all(torch.equal(t, torch.zeros_like(t)) for t in c.forward())


@pytest.mark.parametrize("M,N", [(8192, 2100), (8193, 2100), (8191, 517), (20000, 260), (3000, 9001)])
@pytest.mark.parametrize("masked", [0.5, 0.97])
def test_many_rows_of_which_few_count(M, N, masked):
    # up to 8192 rows the kernel lists those that count, beyond it looks their weights up
    c = Case(M, N, "bf16", masked=masked)
    got, _ = c.check_forward()
    c.check_backward(got, grad=1000.0)
    last = torch.zeros(M, device="cuda")
    last[-1] = 1.0
    c.weight, c.tokens = last, torch.where(last != 0, torch.full_like(c.tokens, N - 1), c.tokens)
    got, _ = c.check_forward()
    assert int((got[1] != 0).sum()) == 1


def test_runs_of_padding():
    # sequences of a padded batch: the first rows of each count
    M, N = 16 * 200, 1300
    c = Case(M, N, "bf16")
    lens = torch.tensor([200, 3, 150, 1, 0, 77, 200, 20, 0, 0, 9, 199, 64, 128, 32, 31], device="cuda")
    on = (torch.arange(200, device="cuda") < lens[:, None]).reshape(-1)
    c.weight = on.float() / on.sum()
    got, _ = c.check_forward()
    c.check_backward(got, grad=100.0)


def test_offsets_beyond_32_bits():
    # rows 2^30 + 1 elements apart: the last one starts past 2^31 elements, off 16-byte boundaries
    pitch, N = (1 << 30) + 1, 5000
    g = torch.Generator("cuda").manual_seed(2)
    z, dz = (torch.empty(2 * pitch + N + 8, dtype=torch.bfloat16, device="cuda").as_strided((3, N), (pitch, 1))
             for _ in range(2))
    z.copy_(torch.randn(3, N, device="cuda", generator=g))
    tokens = torch.tensor([0, 77, N - 1], device="cuda")
    lp = z.double().log_softmax(-1).gather(1, tokens[:, None])[:, 0].float()
    adv = torch.tensor([1.0, -2.0, 0.5], device="cuda")
    got = dyt().policy_loss_forward(z, tokens, lp - 0.03, adv)
    want, tol = R.loss_forward(z, tokens, lp - 0.03, adv)
    for a, b, t, name in zip(got, want, tol, ("loss", "logp", "stats", "coef")):
        R.assert_close(a, b, t, name)
    for out in (dz, torch.empty(3, N, dtype=torch.bfloat16, device="cuda")):
        dyt().policy_loss_backward(z, tokens, got[2], got[3], dlogits=out)
        want, tol = R.loss_backward(z, tokens, got[2], got[3])
        R.assert_close(out, want, tol + R.half_step(out.dtype, want), "dlogits")


def test_two_calls_at_once():
    c = Case(900, 6001, "bf16", masked=0.2)
    want = c.forward()
    dwant = dyt().policy_loss_backward(c.z.t, c.tokens, want[2], want[3])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [(c.forward(stream=s), dyt().policy_loss_backward(c.z.t, c.tokens, want[2], want[3], stream=s))
           for _ in range(8) for s in streams]
    torch.cuda.synchronize()
    for f, b in got:
        assert all(torch.equal(x, y) for x, y in zip(f, want)) and torch.equal(b, dwant)


@pytest.mark.parametrize("N,low", [(50, -INF), (5000, -INF), (5000, torch.finfo(torch.float32).min)])
def test_masked_vocabulary(N, low):
    # all but a few logits masked, by -inf or the type's lowest value, in whole vectors and single places
    c = Case(6, N)
    keep = torch.zeros(6, N, dtype=torch.bool, device="cuda")
    keep[:, ::7] = True
    keep[1] = False
    keep[1, N - 1] = True  # one logit left: probability 1
    keep[2, :N // 2] = False
    c.z.t.masked_fill_(~keep, low)
    c.tokens = torch.where(keep, torch.arange(N, device="cuda"), -1).amax(-1)
    c.old = torch.full((6,), -3.0, device="cuda")
    c.ref = None
    got, _ = c.check_forward()
    assert got[1][1] == 0.0
    dz = dyt().policy_loss_backward(c.z.t, c.tokens, got[2], got[3])
    want, tol = R.loss_backward(c.z.t, c.tokens, got[2], got[3])
    R.assert_close(dz, want, tol + R.half_step(dz.dtype, want), "dlogits")
    assert torch.equal(dz[~keep], torch.zeros_like(dz[~keep]))


@pytest.mark.parametrize("N", [40, 5000])
def test_logits_without_a_distribution_are_nan(N):
    c = Case(8, N)
    clean = c.forward()
    c.z.t[1] = -INF        # no token is left
    c.z.t[3, N // 2] = INF
    c.z.t[5, N - 1] = NAN
    c.tokens[6] = N        # outside the vocabulary
    c.tokens[7] = -1
    loss, logp, _, coef = c.forward()
    bad = torch.tensor([1, 3, 5, 6, 7], device="cuda")
    good = torch.tensor([0, 2, 4], device="cuda")
    assert torch.isnan(loss) and torch.isnan(logp[bad]).all() and torch.isnan(coef[bad]).all()
    assert torch.equal(logp[good], clean[1][good]) and torch.equal(coef[good], clean[3][good])
    # a token that is masked out has probability 0
    c = Case(2, N)
    c.z.t[0, int(c.tokens[0])] = -INF
    c.ref = None
    assert c.forward()[1][0] == -INF


def test_large_logits_keep_their_differences():
    # offsets far beyond the differences: the maximum is taken out before anything is rounded to it
    for offset in (1000.0, -30000.0):
        c = Case(5, 1200)
        c.z.t.copy_((c.z.t * 64).round() / 64 + offset)  # exact in binary32
        want = c.want_forward()
        c.old = want[0][1].float()
        got, _ = c.check_forward()
        c.check_backward(got)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [1.0, 0.25])
def test_rows_at_the_lowest_value_and_far_from_zero(dtype, T):
    # the backward takes the maximum out too before anything is rounded to its size:
    # rows all at the type's lowest value (equal probabilities), all but one there,
    # rows around the type's largest values, ordinary rows
    N, t = 1003, R.DT[dtype]
    c = Case(6, N, dtype, T=T, ref=False)
    big = torch.finfo(t)
    c.z.t[0] = big.min
    c.z.t[1] = big.min
    c.z.t[1, 5] = 1.0
    c.z.t[2] = big.max
    c.z.t[3] = big.max / 2 * (1 - torch.arange(N, device="cuda") % 4 * big.eps)  # neighbours there
    c.z.t[4] += 1000.0
    c.tokens[:5] = torch.tensor([N - 1, 6, 0, 4, 8], device="cuda")
    c.tokens[1] = 5
    lp = R.loss_forward(c.z.t, c.tokens, c.old, c.adv, T=T)[0][1]
    c.old = lp.float()
    got, _ = c.check_forward()
    for row in (0, 2):
        assert abs(float(got[1][row]) + float(torch.log(torch.tensor(float(N))))) < 1e-4
    c.check_backward(got)
    shifted = R.Guarded(6, N, t, offset=3)  # the input at another offset than the output
    shifted.set(c.z.t)
    c.z = shifted
    c.check_backward(got, out_pitch=N + 5, out_offset=1)


def test_clipped_rows_have_no_gradient():
    c = Case(8, 900, ref=False)
    got, _ = c.check_forward()
    r = (got[1] - c.old).exp()
    held = ((c.adv > 0) & (r > 1 + HI)) | ((c.adv < 0) & (r < 1 - LO))
    c8 = Case(64, 900, ref=False)
    got = c8.forward()
    r = (got[1] - c8.old).exp()
    held = ((c8.adv > 0) & (r > 1 + HI)) | ((c8.adv < 0) & (r < 1 - LO))
    assert held.any() and not held.all()
    assert torch.equal(got[3] == 0, held)
    dz = dyt().policy_loss_backward(c8.z.t, c8.tokens, got[2], got[3])
    assert torch.equal(dz.abs().amax(-1) == 0, held)


@pytest.mark.parametrize("M,N,dtype", [(9, 5003, "bf16"), (2000, 77, "f32"), (3, 70000, "f16")])
def test_in_place_and_deterministic(M, N, dtype):
    c = Case(M, N, dtype)
    z = c.z.t.clone()
    args = (c.tokens, c.old, c.adv, c.ref, c.weight, LO, HI, KL, 1.0)
    ws = dyt().policy_loss_workspace(z)
    first = None
    for fill in (0, 255):
        ws.fill_(fill)
        got = dyt().policy_loss_forward(z, *args, ws=ws)
        first = got if first is None else first
        assert all(torch.equal(a, b) for a, b in zip(got, first))
    dz = dyt().policy_loss_backward(z, c.tokens, got[2], got[3])
    assert dyt().policy_loss_backward(z, c.tokens, got[2], got[3], dlogits=z) is z and torch.equal(z, dz)


def test_module_gradient_and_differences():
    torch.manual_seed(1)
    M, N = 12, 90
    z = torch.randn(3, 4, N, device="cuda", requires_grad=True)
    tokens = torch.randint(0, N, (3, 4), device="cuda")
    lp = z.detach().log_softmax(-1).gather(-1, tokens[..., None])[..., 0]
    old, ref, adv = lp - 0.05, lp + 0.2, torch.randn(3, 4, device="cuda")
    weight = torch.rand(3, 4, device="cuda")
    loss = dyt().PolicyLoss(LO, HI, KL, temperature=0.8)
    old = old + torch.randn(3, 4, device="cuda").sign() * 0.02
    out = loss(z, tokens, old, adv, ref, weight)
    assert out.shape == ()
    (3 * out).backward()
    flat = z.detach().reshape(M, N)
    f = lambda t: None if t is None else t.reshape(M)  # noqa: E731
    got = dyt().policy_loss_forward(flat, f(tokens), f(old), f(adv), f(ref), f(weight), LO, HI, KL, 0.8)
    want, tol = R.loss_backward(flat, f(tokens), got[2], got[3], 3.0, 0.8)
    R.assert_close(z.grad.reshape(M, N), want, tol + R.half_step(torch.float32, want), "dlogits")
    # differences of the binary64 formula along a direction
    v = torch.randn(M, N, device="cuda").double()
    t = 1e-5
    g = lambda a: float(R.loss_forward(a, f(tokens), f(old), f(adv), f(ref), f(weight), LO, HI, KL, 0.8)[0][0])  # noqa: E731
    slope = 3 * (g(flat.double() + t * v) - g(flat.double() - t * v)) / (2 * t)
    mine = float((z.grad.reshape(M, N).double() * v).sum())
    assert abs(slope - mine) < 1e-4 * float((z.grad.reshape(M, N).double() * v).abs().sum())


def test_a_row_of_logits_and_an_empty_batch():
    z = torch.randn(300, device="cuda")
    one = lambda v, d=torch.float32: torch.tensor(v, device="cuda", dtype=d)  # noqa: E731
    loss, logp, stats, coef = dyt().policy_loss_forward(z, one(5, torch.int64), one(-4.0), one(1.0))
    assert logp.shape == () and stats.shape == (2,)
    lp = z.double().log_softmax(-1)[5]
    assert abs(float(logp) - float(lp)) < 64 * (R.U + R.EX2) + 2 * R.U * abs(float(lp)) + 3 * R.U * 12
    assert dyt().policy_loss_backward(z, one(5, torch.int64), stats, coef).shape == (300,)
    e = torch.empty(0, device="cuda")
    t = torch.empty(0, device="cuda", dtype=torch.int64)
    loss, logp, stats, coef = dyt().policy_loss_forward(torch.empty(0, 7, device="cuda"), t, e, e)
    assert float(loss) == 0.0 and logp.shape == (0,)
    assert dyt().policy_loss_backward(torch.empty(0, 7, device="cuda"), t, stats, coef).shape == (0, 7)


def test_norm_head_and_loss_together():
    # a network's end as it is trained: DyT, layer norm, the head's product, the loss; gradients of all
    # parameters against binary64 autograd of the same formulas
    torch.manual_seed(0)
    d = dyt()
    B, S, H, N = 2, 24, 128, 1003
    block = torch.nn.Sequential(d.DyT(H, 0.6, device="cuda"), d.LayerNorm(H, device="cuda"))
    with torch.no_grad():
        block[1].gamma.uniform_(0.5, 1.5)
    head = torch.randn(N, H, device="cuda").mul_(0.1).requires_grad_()
    x = torch.randn(B, S, H, device="cuda", requires_grad=True)
    tokens = torch.randint(0, N, (B, S), device="cuda")
    lens = torch.tensor([24, 9], device="cuda")
    weight = (torch.arange(S, device="cuda") < lens[:, None]).float() / lens.sum()
    adv = torch.randn(B, 1, device="cuda").expand(B, S)  # one value a sequence
    with torch.no_grad():
        lp = (block(x) @ head.t()).log_softmax(-1).gather(-1, tokens[..., None])[..., 0]
        old, ref = lp + 0.05, lp - 0.1
    loss = d.PolicyLoss(LO, HI, KL)(block(x) @ head.t(), tokens, old, adv, ref, weight)
    loss.backward()
    p64 = [t.detach().double().requires_grad_() for t in (x, head, block[0].alpha, block[0].gamma, block[0].beta,
                                                           block[1].gamma, block[1].beta)]
    x6, h6, al, g0, b0, g1, b1 = p64
    t6 = g0 * torch.tanh(al * x6) + b0
    n6 = (t6 - t6.mean(-1, keepdim=True)) / torch.sqrt(t6.var(-1, unbiased=False, keepdim=True) + 1e-5) * g1 + b1
    l6 = (n6 @ h6.t()).log_softmax(-1).gather(-1, tokens[..., None])[..., 0]
    r = (l6 - old.double()).exp()
    q = ref.double() - l6
    each = -torch.minimum(r * adv, r.clamp(1 - LO, 1 + HI) * adv) + KL * (q.exp() - q - 1)
    (each * weight.double()).sum().backward()
    # torch's float32 product of H terms is the largest rounding on the way: H u on logits of size ~1,
    # and as much again in its two backward products
    for got, want, name in zip((x, head, block[0].alpha, block[0].gamma, block[0].beta, block[1].gamma,
                                block[1].beta), p64, ("x", "head", "alpha", "gamma", "beta", "norm gamma",
                                                      "norm beta")):
        off = float((got.grad.double() - want.grad).norm() / want.grad.norm())
        assert off < 4 * H * R.U, (name, off)
    assert torch.equal(x.grad[1, 9:], torch.zeros_like(x.grad[1, 9:]))  # padding


def test_captured_and_replayed_on_another_stream():
    a, b = Case(30, 2003, "bf16"), Case(30, 2003, "bf16", seed=4)
    z, ws = a.z.t.clone(), dyt().policy_loss_workspace(a.z.t)
    call = lambda: dyt().policy_loss_forward(z, a.tokens, a.old, a.adv, a.ref, None, LO, HI, KL, ws=ws)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
        dz = dyt().policy_loss_backward(z, a.tokens, got[2], got[3])
    for c in (b, a):
        z.copy_(c.z.t)
        graph.replay()
        torch.cuda.synchronize()
        want = dyt().policy_loss_forward(z, a.tokens, a.old, a.adv, a.ref, None, LO, HI, KL, stream=s)
        s.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert torch.equal(dz, dyt().policy_loss_backward(z, a.tokens, want[2], want[3]))


def test_refusals():
    c = Case(4, 32)
    z, t, o, a = c.z.t.contiguous(), c.tokens, c.old, c.adv
    f, b = dyt().policy_loss_forward, dyt().policy_loss_backward
    _, _, stats, coef = f(z, t, o, a)
    for call in (lambda: f(z.t(), t, o, a), lambda: f(z, t[:3], o, a), lambda: f(z, t, o.cpu(), a),
                 lambda: f(z, t, o, a, weight=o[:2]), lambda: f(z.cpu(), t, o, a), lambda: f(z[:, :0], t, o, a),
                 lambda: f(z, t, o, a, ws=o), lambda: f(z, t, torch.zeros(8, device="cuda")[::2], a),
                 lambda: b(z, t, stats[:3], coef), lambda: b(z, t, stats, coef, dlogits=z[:2]),
                 lambda: b(z, t, stats, coef, grad=o)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: f(z.double(), t, o, a), lambda: f(z, t.float(), o, a), lambda: f(z, t, o.half(), a),
                 lambda: b(z, t, stats.double(), coef)):
        with pytest.raises(TypeError):
            call()
    for kw in ({"clip_low": -0.1}, {"clip_high": NAN}, {"kl_coef": INF}, {"temperature": 0.0},
               {"temperature": -1.0}, {"temperature": NAN}, {"ws": torch.empty(16, dtype=torch.uint8, device="cuda")}):
        with pytest.raises(dyt().DytError):
            f(z, t, o, a, **kw)
    with pytest.raises(dyt().DytError):
        b(z, t, stats, coef, temperature=0.0)
