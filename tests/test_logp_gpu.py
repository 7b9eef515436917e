"""The kernels for log probabilities, entropy and alternatives against their binary64
formulas: vocabularies from one token, rows that are split and rows that share a CTA,
rows that do not count, equal logits, -inf, NaN, strides, dtypes, gradients, refusals."""
from __future__ import annotations

import pytest
import torch

from tests import logp_helpers as L
from tests import row_helpers as R

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
LOWEST = torch.finfo(torch.float32).min


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")


def dyt():
    import elementwise_reduction_b200 as d
    return d


class Case:
    def __init__(self, M, N, dtype="f32", pitch=None, offset=0, T=1.0, top=None, masked=0.0, seed=0, std=2.0,
                 token_dtype=torch.int64, tokens=True):
        g = torch.Generator("cuda").manual_seed(seed)
        self.z = R.Guarded(M, N, R.DT[dtype], pitch, offset)
        self.z.set(torch.randn(M, N, device="cuda", generator=g) * std)
        self.top, self.T = min(N, 7) if top is None else min(N, top), T
        self.tokens = torch.randint(0, N, (M,), device="cuda", generator=g).to(token_dtype)
        if masked:
            off = torch.rand(M, device="cuda", generator=g) < masked
            self.tokens = torch.where(off, torch.full_like(self.tokens, -100), self.tokens)
        if not tokens:
            self.tokens = None
        self.da, self.db = (torch.randn(M, device="cuda", generator=g) for _ in range(2))

    def check_forward(self, **kw):
        got = dyt().log_probs_forward(self.z.t, self.tokens, self.top, self.T, **kw)
        info = dyt().dyt_last_launch_info()
        want, tol = L.forward(self.z.t, self.tokens, self.top, self.T)
        assert (got[0] is None) == (self.tokens is None)
        for g, w, t, name in zip(got, want, tol, ("logp", "entropy", "top_logp", "top_tokens", "stats")):
            if name == "top_tokens":
                assert (g is None) if self.top == 0 else torch.equal(g, w), name
            elif g is not None:
                assert g.dtype == torch.float32
                R.assert_close(g, w, t, name)
            else:
                assert name == "logp" or self.top == 0
        assert info["op"] == 12 and info["kernels"] == (1 if info["workspace_bytes"] == 0 else 2)
        return got, info

    def check_backward(self, got, scale=1.0, out_pitch=None, out_offset=0, da=True, db=True):
        M, N = self.z.t.shape
        dz = R.Guarded(M, N, self.z.t.dtype, out_pitch, out_offset, fill=5.0)
        da = self.da * scale if da and self.tokens is not None else None
        db = self.db * scale if db else None
        dyt().log_probs_backward(self.z.t, self.tokens, got[4], got[1], da, db, self.T, dlogits=dz.t)
        info = dyt().dyt_last_launch_info()
        want, tol = L.backward(self.z.t, self.tokens, got[4], got[1], da, db, self.T)
        R.assert_close(dz.t, want, tol + R.half_step(dz.t.dtype, want), "dlogits")
        dz.assert_surroundings_untouched("dlogits")
        assert info["op"] == 13 and info["kernels"] == 1
        return info


WIDTHS = [1, 2, 3, 7, 8, 9, 15, 31, 33, 64, 100, 255, 257, 1000, 1024, 2047, 2048, 2049, 2056, 4096, 5003, 16384,
          50001]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", WIDTHS)
def test_widths(N, dtype):
    for top in (0, 1, 5, 32):
        c = Case(7, N, dtype, top=top)
        got, _ = c.check_forward()
        if top in (0, 5):
            c.check_backward(got, scale=100.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [n for n in WIDTHS if n < 20000])
def test_widths_of_many_rows(N, dtype):
    c = Case(600, N, dtype, masked=0.2)
    got, info = c.check_forward()
    assert info["kernels"] == 2
    c.check_backward(got)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,top", [(1, 131072, 20), (74, 131072, 32), (75, 131072, 20), (8, 151936, 1),
                                     (1, 500001, 32), (64, 5000, 20), (592, 1000, 5), (593, 1000, 5), (1, 1, 1),
                                     (2, 1048571, 3)])
def test_few_rows(M, N, top, dtype):
    """One kernel where the rows' clusters are few, two beyond; rows among them that do not count."""
    for masked in (0.0, 0.5):
        c = Case(M, N, dtype, top=top, masked=masked)
        got, info = c.check_forward()
        batches = -(-N * c.z.t.element_size() // 4096)
        ctas = min(8, 1 << max(0, -(-batches // 8) - 1).bit_length())
        assert info["kernels"] == (1 if batches <= 256 and M * ctas <= 592 else 2)
        out = Case(M, N, dtype, top=0, masked=masked).check_forward()[0]
        assert all(torch.equal(got[i], out[i]) for i in (0, 1, 4))  # (with alternatives or without)
    none = Case(M, N, dtype, top=top, tokens=False)
    none.check_forward()


@pytest.mark.parametrize("M", [1, 2, 5, 64, 65, 1183, 1184, 1185, 5000])
@pytest.mark.parametrize("N,dtype", [(515, "bf16"), (2051, "f32")])
def test_row_counts(M, N, dtype):
    c = Case(M, N, dtype, masked=0.3 if M > 2 else 0.0, T=0.7)
    got, _ = c.check_forward()
    c.check_backward(got, scale=100.0)


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
        c.check_backward(got, 100.0, out_pitch, out_offset)


@pytest.mark.parametrize("T", [0.1, 0.6, 1.0, 3.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_temperatures_and_token_types(T, dtype):
    for kind in (torch.int64, torch.int32):
        c = Case(100, 3001, dtype, T=T, masked=0.2, token_dtype=kind, top=20)
        got, _ = c.check_forward()
        c.check_backward(got, 100.0)


@pytest.mark.parametrize("N", [5, 1000, 30001])
def test_single_gradients_and_no_tokens(N):
    for tokens in (True, False):
        c = Case(50, N, "f32", tokens=tokens)
        got, _ = c.check_forward()
        c.check_backward(got, da=False)
        if tokens:
            c.check_backward(got, db=False)
    # neither gradient: zeros, whatever the logits are
    c.z.t.fill_(NAN)
    dz = dyt().log_probs_backward(c.z.t, None, got[4])
    assert (dz == 0).all()


@pytest.mark.parametrize("M,N,masked", [(4000, 16001, 0.9), (4000, 16000, 0.5), (9000, 515, 0.5), (8192, 9000, 0.3),
                                        (3000, 300, 0.999), (500, 4000, 1.0)])
def test_rows_that_do_not_count(M, N, masked):
    c = Case(M, N, "bf16", masked=masked, top=3)
    off = c.tokens == -100
    c.z.t[off] = NAN  # not read
    got = dyt().log_probs_forward(c.z.t, c.tokens, 3)
    zero = c.z.t.clone()
    zero[off] = 0
    want, tol = L.forward(zero, c.tokens, 3)
    for g, w, t in zip(got, want, tol):
        assert torch.equal(g, w) if t is None else R.assert_close(g, w, t, "forward") is None
    dz = dyt().log_probs_backward(c.z.t, c.tokens, got[4], got[1], c.da, c.db)
    want, tol = L.backward(zero, c.tokens, got[4], got[1], c.da, c.db)
    R.assert_close(dz, want, tol + R.half_step(dz.dtype, want), "dlogits")
    assert (dz[off] == 0).all()


def test_another_ignored_token():
    c = Case(20, 100)
    c.tokens[3:7] = 0
    got = dyt().log_probs_forward(c.z.t, c.tokens, 2, ignore_index=0)
    off = c.tokens == 0
    want, tol = L.forward(c.z.t, c.tokens, 2, ignore=0)
    R.assert_close(got[0], want[0], tol[0], "logp")
    assert torch.equal(got[3], want[3]) and (got[3][off] == -1).all() and (got[4][off] == 0).all()
    dz = dyt().log_probs_backward(c.z.t, c.tokens, got[4], got[1], c.da, None, ignore_index=0)
    assert (dz[off] == 0).all() and (dz[~off] != 0).any()


@pytest.mark.parametrize("N", [10, 1000, 40001])
def test_tokens_outside_the_vocabulary(N):
    c = Case(12, N)
    c.tokens[2], c.tokens[5], c.tokens[7], c.tokens[9] = -1, N, 1 << 40, -100
    got, _ = c.check_forward()
    assert torch.isnan(got[0][[2, 5, 7]]).all() and got[0][9] == 0 and torch.isfinite(got[1]).all()
    c.da[7] = 0.0  # not wanted: the entropy's gradient stands
    c.check_backward(got)


# ---- equal logits, masks, infinities -------------------------------------------------------------

SHAPES = [(6, 20), (6, 33), (5, 2048), (5, 2049), (4, 12345), (3, 131072), (1500, 4000),
          (700, 20), (700, 33), (600, 2049), (600, 12345), (80, 131072)]  # (few rows take a kernel of their own)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", SHAPES)
def test_equal_logits_go_by_column(M, N, dtype):
    for top in (1, 5, 32):
        c = Case(M, N, dtype, top=top)
        c.z.t.fill_(0.5)
        c.z.t[1::2] = 0.0
        c.z.t[2] = c.z.t[2].clone().zero_()
        c.z.t[2, ::3] = -0.0  # equal to 0
        c.check_forward()
        g = torch.Generator("cuda").manual_seed(top)
        c.z.set(torch.randint(0, 3, (M, N), device="cuda", generator=g).float())  # three values
        c.check_forward()
        c.z.set(torch.randint(-40, 0, (M, N), device="cuda", generator=g).float())
        c.z.t[:, -1] = 0.0
        c.check_forward()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N", SHAPES)
def test_rising_and_falling_rows(M, N, dtype):
    # every logit passes the ones before it, or none does
    c = Case(M, N, dtype, top=20)
    ramp = torch.linspace(-20, 20, N, device="cuda")
    c.z.t.copy_(ramp)
    c.z.t[1::2] = -ramp
    got, _ = c.check_forward()
    c.check_backward(got)


@pytest.mark.parametrize("value", [-INF, "lowest"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N", SHAPES)
def test_masked_vocabularies(M, N, dtype, value):
    # all but a few logits masked: fewer left than alternatives, one left, the mask before and behind
    value = torch.finfo(R.DT[dtype]).min if value == "lowest" else value
    c = Case(M, N, dtype, top=9)
    keep = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    keep[0, [N - 1, N // 2, 3]] = True
    keep[1, N // 3] = True
    keep[2, : N // 2] = True
    if M > 3:
        keep[3:, N // 2:] = True
    c.z.t.masked_fill_(~keep, value)
    c.tokens = keep.to(torch.uint8).argmax(-1)
    got, _ = c.check_forward()
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all() and got[1][1] == 0 and got[0][1] == 0
    c.check_backward(got)
    c.tokens[1] = (N // 3 + 1) % N  # a token without probability
    got = dyt().log_probs_forward(c.z.t, c.tokens)
    assert got[0][1] == -INF if value == -INF else got[0][1] < -1e4


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", SHAPES)
def test_nan_and_infinity(M, N, dtype):
    c = Case(M, N, dtype, top=6)
    clean = dyt().log_probs_forward(c.z.t, c.tokens, 6)
    c.z.t[0, N // 2] = NAN
    c.z.t[1] = -INF
    c.z.t[2, [1, N - 2]] = INF
    got, want = dyt().log_probs_forward(c.z.t, c.tokens, 6), L.alternatives(c.z.t, 6)
    assert torch.equal(got[3], want)
    for t in (got[0], got[1], got[2]):
        assert torch.isnan(t[:3]).all()
    for a, b in zip(got, clean):
        assert torch.equal(a[3:], b[3:])
    c.z.t[0] = NAN
    c.z.t[0, [N - 3, 2, 4]] = 1.0
    c.z.t[2] = NAN
    got = dyt().log_probs_forward(c.z.t, c.tokens, 6)
    assert got[3][0].tolist() == [2, 4, N - 3, -1, -1, -1] and (got[3][2] == -1).all()
    assert torch.equal(got[3][1].cpu(), torch.arange(6))


def test_rows_far_from_zero():
    # the maximum leaves first: shifts that binary32 holds do not change a row
    for dtype, shift in (("f32", 4096.0), ("f32", -65536.0), ("bf16", 64.0)):
        c = Case(9, 3000, dtype, top=8)
        c.z.t.copy_((c.z.t.float() * 4).round() / 4)
        base = dyt().log_probs_forward(c.z.t, c.tokens, 8)
        if dtype == "bf16":
            c.z.t.copy_((c.z.t.float() * 2).round() / 2)
            base = dyt().log_probs_forward(c.z.t, c.tokens, 8)
        c.z.t.add_(shift)
        got, _ = c.check_forward()
        if dtype == "f32":
            for k in range(4):
                assert torch.equal(got[k], base[k])


def test_one_likely_token():
    c = Case(64, 50000, "f32", top=4)
    c.z.t[torch.arange(64), c.tokens] = 40.0
    got, _ = c.check_forward()
    c.check_backward(got)
    assert torch.equal(got[3][:, 0], c.tokens)


def test_offsets_beyond_32_bits():
    pitch, N = (1 << 30) + 8, 3001
    z = torch.empty(2 * pitch + N + 8, dtype=torch.bfloat16, device="cuda").as_strided((3, N), (pitch, 1))
    z.copy_(torch.randn(3, N, device="cuda", generator=torch.Generator("cuda").manual_seed(3)))
    tokens = torch.tensor([3000, 0, 1500], device="cuda")
    got = dyt().log_probs_forward(z, tokens, 10)
    want, tol = L.forward(z, tokens, 10)
    R.assert_close(got[0], want[0], tol[0], "logp")
    assert torch.equal(got[3], want[3])
    g = torch.randn(3, device="cuda")
    dz = dyt().log_probs_backward(z, tokens, got[4], got[1], g, g, dlogits=z)
    assert dz is z
    back, tol = L.backward(z.clone(), tokens, got[4], got[1], g, g)
    assert torch.isfinite(dz.float()).all()


def test_logits_beyond_32_bits_of_bytes():
    # 3 GiB of logits and alternatives in every row
    M, N = 12289, 131072
    z = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    z.normal_(0, 2.0, generator=torch.Generator("cuda").manual_seed(8))
    tokens = torch.randint(0, N, (M,), device="cuda")
    got = dyt().log_probs_forward(z, tokens, 4)
    at = torch.tensor([0, 1, 4095, 8191, 8192, M - 2, M - 1], device="cuda")
    want, tol = L.forward(z[at], tokens[at], 4)
    for g, w, t in zip(got, want, tol):
        assert torch.equal(g[at], w) if t is None else R.assert_close(g[at], w, t, "forward") is None
    g = torch.ones(M, device="cuda")
    part = z[at].clone()
    dyt().log_probs_backward(z, tokens, got[4], got[1], g, g, dlogits=z)
    want, tol = L.backward(part, tokens[at], got[4][at], got[1][at], g[at], g[at])
    R.assert_close(z[at], want, tol + R.half_step(z.dtype, want), "dlogits")


@pytest.mark.parametrize("N,dtype", [(64, "bf16"), (1001, "f16"), (5000, "f32"), (20003, "bf16")])
def test_in_place(N, dtype):
    for M in (5, 1400):
        c = Case(M, N, dtype)
        got = dyt().log_probs_forward(c.z.t, c.tokens)
        want = dyt().log_probs_backward(c.z.t, c.tokens, got[4], got[1], c.da, c.db)
        dyt().log_probs_backward(c.z.t, c.tokens, got[4], got[1], c.da, c.db, dlogits=c.z.t)
        assert torch.equal(c.z.t, want)


def test_the_same_bits_twice():
    c = Case(3000, 20001, "bf16", masked=0.3, top=20)
    once = dyt().log_probs_forward(c.z.t, c.tokens, 20)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(once, dyt().log_probs_forward(c.z.t, c.tokens, 20)))


def test_streams_and_graphs():
    c, e = Case(300, 20001, "bf16", masked=0.1, top=9), Case(40, 131072, "bf16", top=32, seed=5)
    def step(c):
        got = dyt().log_probs_forward(c.z.t, c.tokens, c.top)
        return (*got, dyt().log_probs_backward(c.z.t, c.tokens, got[4], got[1], c.da, c.db))
    wants = [[t.clone() for t in step(x)] for x in (c, e)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):  # two calls at once
        for s, x in zip(streams, (c, e)):
            with torch.cuda.stream(s):
                outs.append(step(x))
    torch.cuda.synchronize()
    for k, got in enumerate(outs):
        assert all(torch.equal(a, b) for a, b in zip(got, wants[k % 2]))
    got = dyt().log_probs_forward(c.z.t, c.tokens, c.top, stream=streams[0])
    streams[0].synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, wants[0]))
    ws = dyt().log_probs_workspace(c.z.t, c.top)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = dyt().log_probs_forward(c.z.t, c.tokens, c.top, ws=ws), step(c)
        graphs.append((graph, out))
    c.z.t.mul_(0.5)
    want = step(c)
    for graph, _ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for _, (a, b) in graphs:
        assert all(torch.equal(x, y) for x, y in zip(a, want)) and all(torch.equal(x, y) for x, y in zip(b, want))


# ---- module --------------------------------------------------------------------------------------

def test_module_gradients_agree_with_autograd():
    g = torch.Generator("cuda").manual_seed(9)
    z = torch.randn(3, 11, 70, device="cuda", generator=g, requires_grad=True)
    tokens = torch.randint(0, 70, (3, 11), device="cuda", generator=g)
    tokens[1, 4:] = -100
    ua, ub = (torch.randn(3, 11, device="cuda", generator=g) for _ in range(2))
    logp, entropy, best, ids = dyt().LogProbs(top=4, temperature=0.8)(z, tokens)
    assert logp.shape == entropy.shape == (3, 11) and best.shape == ids.shape == (3, 11, 4)
    assert not best.requires_grad and not ids.requires_grad
    ((logp * ua).sum() + (entropy * ub).sum()).backward()
    y = z.detach().double().requires_grad_()
    lp = (y / 0.8).log_softmax(-1)
    on = tokens != -100
    hit = lp.gather(-1, tokens.clamp(min=0)[..., None])[..., 0]
    ((hit * ua)[on].sum() - ((lp.exp() * lp).sum(-1) * ub)[on].sum()).backward()
    assert torch.allclose(z.grad.double(), y.grad, rtol=1e-5, atol=1e-6)
    # sums: gradients of one value for all rows; one output alone; nothing used
    for use in (lambda o: o[0].sum(), lambda o: o[1].mean(), lambda o: o[0].sum() + o[1].sum()):
        z.grad = None
        use(dyt().LogProbs()(z, tokens)).backward()
        assert torch.isfinite(z.grad).all() and (z.grad[1, 4:] == 0).all() and (z.grad[0] != 0).any()


def test_module_without_tokens():
    # a sampler's view, before a token is drawn: the entropy has a gradient
    z = torch.randn(5, 300, device="cuda", requires_grad=True)
    logp, entropy, best, ids = dyt().LogProbs(top=2)(z)
    assert logp is None and torch.equal(ids[:, 0], z.argmax(-1))
    entropy.sum().backward()
    lp = z.detach().double().requires_grad_()
    p = lp.log_softmax(-1)
    (-(p.exp() * p).sum()).backward()
    assert torch.allclose(z.grad.double(), lp.grad, rtol=1e-5, atol=1e-7)


def test_module_gradient_against_differences():
    g = torch.Generator("cuda").manual_seed(10)
    z, v = (torch.randn(8, 50, device="cuda", generator=g) for _ in range(2))
    tokens = torch.randint(0, 50, (8,), device="cuda", generator=g)
    def f(t):
        out = L.forward(t, tokens)[0]
        return float(out[0].sum() + 0.3 * out[1].sum())
    a = z.clone().requires_grad_()
    logp, entropy, _, _ = dyt().LogProbs()(a, tokens)
    (logp.sum() + 0.3 * entropy.sum()).backward()
    t = 1e-5
    slope = (f(z.double() + t * v.double()) - f(z.double() - t * v.double())) / (2 * t)
    assert abs(slope - float((a.grad.double() * v.double()).sum())) < 1e-4


def test_module_on_views():
    z = torch.randn(4, 9, 33, device="cuda")
    tokens = torch.randint(0, 33, (4, 9), device="cuda")
    cut = z[:, :-1]  # no single pitch: copied by the module, refused by the function
    a = dyt().LogProbs()(cut, tokens[:, 1:])
    b = dyt().log_probs_forward(cut.contiguous(), tokens[:, 1:].contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(ValueError):
        dyt().log_probs_forward(cut, tokens[:, 1:].contiguous())
    one = torch.randn(33, device="cuda")
    assert dyt().log_probs_forward(one, top=2)[3].shape == (2,)


def test_module_captured_with_its_backward():
    z = torch.randn(64, 3000, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    tokens = torch.randint(0, 3000, (64,), device="cuda")
    layer = dyt().LogProbs(top=5)
    def step():
        logp, entropy, best, ids = layer(z, tokens)
        return logp.detach(), best, ids, torch.autograd.grad(logp.sum() + 0.01 * entropy.sum(), z)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    with torch.no_grad():
        z.mul_(1.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, step()))


def test_norm_head_log_probabilities_and_loss_together():
    # a rollout's log probabilities by the served network, its policy step on the same rows: ratios of 1
    d = dyt()
    g = torch.Generator("cuda").manual_seed(12)
    M, W, N = 96, 256, 2000
    x, r = (torch.randn(M, W, device="cuda", generator=g, dtype=torch.bfloat16) for _ in range(2))
    head = (torch.randn(N, W, device="cuda", generator=g) / 8).bfloat16().requires_grad_()
    norm = d.RMSNorm(W, device="cuda")
    x.requires_grad_()
    tokens = torch.randint(0, N, (M,), device="cuda", generator=g)
    tokens[::5] = -100
    on = (tokens != -100).float()
    with torch.no_grad():
        y, h = norm(x, r)
        logits = y @ head.t()
        old, _, best, ids = d.LogProbs(top=3)(logits, tokens)
        q, scale, h8 = d.rms_norm_quantize(x.detach(), norm.gamma.detach(), r)
    assert torch.equal(h8, h) and torch.equal(ids[tokens != -100][:, 0], logits.float().argmax(-1)[tokens != -100])
    near = (q.float() * scale[:, None] - y.float()).abs()
    assert (near <= y.float().abs() / 16 + scale[:, None] * 2.0 ** -9 + y.float().abs() / 128).all()
    y, h = norm(x, r)
    logits = y @ head.t()
    adv = torch.randn(M, device="cuda", generator=g)
    loss = d.PolicyLoss()(logits, tokens, old, adv, weight=on / on.sum())
    logp, entropy, _, _ = d.LogProbs()(logits, tokens)
    (loss - 0.01 * (entropy * on).sum() / on.sum() + h.float().square().mean()).backward()
    for t in (x.grad, head.grad, norm.gamma.grad):
        assert torch.isfinite(t).all() and (t != 0).any()
    # the ratio is 1: the loss is the mean of -advantage, and so is its gradient that of -advantage logp
    assert abs(float(loss.detach()) + float((adv * on).sum() / on.sum())) < 1e-4
    assert torch.allclose(logp, old, rtol=0, atol=1e-6)


# ---- refusals ------------------------------------------------------------------------------------

def test_refusals():
    d = dyt()
    z = torch.randn(6, 20, device="cuda")
    t, v = torch.zeros(6, dtype=torch.int64, device="cuda"), torch.zeros(6, device="cuda")
    st = torch.zeros(6, 2, device="cuda")
    bad = [lambda: d.log_probs_forward(z, t[:5]), lambda: d.log_probs_forward(z, t.float()),
           lambda: d.log_probs_forward(z, t.cpu()), lambda: d.log_probs_forward(z.double(), t),
           lambda: d.log_probs_forward(z.t(), t), lambda: d.log_probs_forward(z, t, 33),
           lambda: d.log_probs_forward(z, t, 21), lambda: d.log_probs_forward(z, t, -1),
           lambda: d.log_probs_forward(z, t, temperature=0.0), lambda: d.log_probs_forward(z, t, temperature=NAN),
           lambda: d.log_probs_forward(z[:, :0], t), lambda: d.log_probs_forward(v[0], t),
           lambda: d.log_probs_forward(z.repeat(100, 1), t.repeat(100),
                                       ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
           lambda: d.log_probs_forward(z, t, ws=v), lambda: d.log_probs_workspace(z, 40),
           lambda: d.log_probs_backward(z, None, st, None, v), lambda: d.log_probs_backward(z, t, st, None, v, v),
           lambda: d.log_probs_backward(z, t, st[:5], v, v), lambda: d.log_probs_backward(z, t, st, v[:5], v),
           lambda: d.log_probs_backward(z, t, st, v, v[:5]), lambda: d.log_probs_backward(z, t, st, v, v, v.half()),
           lambda: d.log_probs_backward(z, t, st, v, v, dlogits=z[:5]),
           lambda: d.log_probs_backward(z, t, st, v, v, temperature=-1.0),
           lambda: d.log_probs_backward(z, t[:5], st, v, v)]
    for k, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, d.DytError)):
            call()
            pytest.fail(f"call {k} was not refused")
    # no rows
    got = d.log_probs_forward(z[:0], t[:0], 3)
    assert got[0].shape == (0,) and got[2].shape == got[3].shape == (0, 3) and got[4].shape == (0, 2)
    assert d.log_probs_backward(z[:0], t[:0], got[4], got[1], v[:0], v[:0]).shape == (0, 20)
