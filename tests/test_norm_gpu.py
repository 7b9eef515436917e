"""Layer norm's kernels against its binary64 formulas: lengths from one element,
ragged and strided rows, dtypes, empty shapes, extreme values, and refusals."""
from __future__ import annotations

import pytest
import torch

from tests import row_helpers as R

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")


def dyt():
    import elementwise_reduction_b200 as d
    return d


def inputs(M, N, xd="f32", pd="f32", seed=0, mean=0.3, std=1.2, pitch=None, offset=0):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, dy = R.Guarded(M, N, R.DT[xd], pitch, offset), R.Guarded(M, N, R.DT[xd], pitch, offset)
    x.set(r(M, N) * std + mean)
    dy.set(r(M, N))
    return x, dy, (1 + 0.2 * r(N)).to(R.DT[pd]), (0.2 * r(N)).to(R.DT[pd])


def check(M, N, xd="f32", pd="f32", out_pitch=None, out_offset=0, **kw):
    x, dy, gamma, beta = inputs(M, N, xd, pd, **kw)
    y = R.Guarded(M, N, R.DT[xd], out_pitch, out_offset, fill=7.0)
    _, mean, rstd = dyt().layer_norm_forward(x.t, gamma, beta, EPS, out=y.t)
    fwd = dyt().dyt_last_launch_info()
    want, tol = R.norm_forward(x.t, gamma, beta, EPS)
    R.assert_close(mean, want[1], tol[1], "mean")
    R.assert_close(rstd, want[2], tol[2], "rstd")
    R.assert_close(y.t, want[0], tol[0] + R.half_step(R.DT[xd], want[0]), "y")
    y.assert_surroundings_untouched("y")
    dx = R.Guarded(M, N, R.DT[xd], out_pitch, out_offset, fill=7.0)
    _, dgamma, dbeta = dyt().layer_norm_backward(x.t, dy.t, mean, rstd, gamma, beta, dx=dx.t)
    bwd = dyt().dyt_last_launch_info()
    want, tol = R.norm_backward(x.t, dy.t, mean, rstd, gamma)
    R.assert_close(dx.t, want[0], tol[0] + R.half_step(R.DT[xd], want[0]), "dx")
    assert dgamma.dtype == dbeta.dtype == R.DT[pd]
    R.assert_close(dgamma, want[1], tol[1] + R.half_step(R.DT[pd], want[1]), "dgamma")
    R.assert_close(dbeta, want[2], tol[2] + R.half_step(R.DT[pd], want[2]), "dbeta")
    dx.assert_surroundings_untouched("dx")
    return fwd, bwd


WIDTHS = [1, 2, 3, 4, 7, 8, 9, 16, 17, 31, 32, 33, 64, 65, 100, 127, 128, 255, 256, 257, 511, 512, 513, 520, 1000,
          1024, 2047, 2048, 4096, 4100, 4104, 8191, 8192]


@pytest.mark.parametrize("xd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", WIDTHS)
def test_widths(N, xd):
    fwd, bwd = check(37, N, xd)
    assert fwd["op"] == 5 and bwd["op"] == 6 and fwd["kernels"] == 1 and bwd["kernels"] == 2


@pytest.mark.parametrize("xd", ["f32", "bf16"])
@pytest.mark.parametrize("N", [8200, 12001, 16383, 16384, 16385, 32776, 40001])
def test_long_rows(N, xd):
    check(5, N, xd)


@pytest.mark.parametrize("M", [1, 2, 3, 7, 8, 9, 63, 1000, 4097, 65537])
@pytest.mark.parametrize("N,xd", [(32, "bf16"), (17, "f32"), (640, "f16")])
def test_row_counts(M, N, xd):
    check(M, N, xd)


@pytest.mark.parametrize("N", [16, 1024, 9000])
def test_rows_beyond_one_run(N):
    # several runs of 128 rows per lane
    check(160000 if N == 16 else 90000 if N == 1024 else 3000, N, "bf16" if N != 16 else "f32")


@pytest.mark.parametrize("N,lanes", [(1024, 64), (512, 32), (1021, 64), (96, 8)])
def test_some_rows_short_of_a_full_run(N, lanes):
    # 128 steps, a run of column sums, of which some rows of one CTA do not make the last one
    rows = 512 // lanes
    step = torch.cuda.get_device_properties(0).multi_processor_count * rows
    for extra in (5 * rows + 3, 1):
        check(127 * step + extra, N, "bf16")
        assert dyt().dyt_last_launch_info()["rows_per_step"] == rows


def test_offsets_beyond_32_bits():
    # rows 2^30 + 8 elements apart: the last one starts past 2^31 elements
    pitch, N = (1 << 30) + 8, 1000
    g = torch.Generator("cuda").manual_seed(5)
    x, dy, y = (torch.empty(2 * pitch + N + 8, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    xv, dv, yv = (t.as_strided((3, N), (pitch, 1)) for t in (x, dy, y))
    xv.copy_(torch.randn(3, N, device="cuda", generator=g))
    dv.copy_(torch.randn(3, N, device="cuda", generator=g))
    gamma = torch.rand(N, device="cuda", generator=g)
    _, mean, rstd = dyt().layer_norm_forward(xv, gamma, gamma, EPS, out=yv)
    want, tol = R.norm_forward(xv, gamma, gamma, EPS)
    R.assert_close(yv, want[0], tol[0] + R.half_step(yv.dtype, want[0]), "y")
    dx, dgamma, _ = dyt().layer_norm_backward(xv, dv, mean, rstd, gamma, gamma, dx=yv)
    want, tol = R.norm_backward(xv, dv, mean, rstd, gamma)
    R.assert_close(dx, want[0], tol[0] + R.half_step(dx.dtype, want[0]), "dx")
    R.assert_close(dgamma, want[1], tol[1] + R.half_step(dgamma.dtype, want[1]), "dgamma")


@pytest.mark.parametrize("xd,pd", [(a, b) for a in ("f32", "bf16", "f16") for b in ("f32", "bf16", "f16")])
def test_dtype_matrix(xd, pd):
    check(65, 136, xd, pd)
    check(9, 1032, xd, pd)


@pytest.mark.parametrize("xd", ["f32", "bf16"])
@pytest.mark.parametrize("N,pitch,offset,out_pitch,out_offset", [
    (64, 72, 0, 64, 0), (64, 64, 1, 64, 1), (64, 65, 0, 67, 3), (100, 104, 0, 100, 0), (1000, 1001, 2, 1000, 0),
    (4096, 4104, 0, 4112, 0), (4096, 4104, 8, 4096, 0), (4097, 4100, 1, 4099, 2), (9001, 9008, 0, 9001, 1)])
def test_strides_and_offsets(N, pitch, offset, out_pitch, out_offset, xd):
    check(19, N, xd, pitch=pitch, offset=offset, out_pitch=out_pitch, out_offset=out_offset)


@pytest.mark.parametrize("xd,pd", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("N", [1, 2, 3, 5, 7, 9, 17, 31, 33, 61, 100, 127, 251, 257, 511, 513, 517, 1001, 2047, 4093,
                               4099, 8185, 8191])
def test_aligned_rows_with_a_part_of_a_vector_at_the_end(N, xd, pd):
    # rows on 16-byte boundaries, NaN between them; few rows, several rows a lane, and a single one
    pitch = (N + 7) // 8 * 8
    for M in (1, 37, 1500):
        check(M, N, xd, pd, pitch=pitch + 8, out_pitch=pitch)


def test_parameters_of_two_dtypes_and_none():
    x, dy, gamma, beta = inputs(33, 200, "bf16")
    g16, b16 = gamma.to(torch.bfloat16), beta.to(torch.float16)
    for g, b in ((g16, b16), (gamma, None), (None, beta), (None, None)):
        y, mean, rstd = dyt().layer_norm_forward(x.t, g, b, EPS)
        want, tol = R.norm_forward(x.t, g, b, EPS)
        R.assert_close(y, want[0], tol[0] + R.half_step(y.dtype, want[0]), "y")
        dx, dgamma, dbeta = dyt().layer_norm_backward(x.t, dy.t, mean, rstd, g, b)
        want, tol = R.norm_backward(x.t, dy.t, mean, rstd, g)
        R.assert_close(dx, want[0], tol[0] + R.half_step(dx.dtype, want[0]), "dx")
        for got, p, i in ((dgamma, g, 1), (dbeta, b, 2)):
            assert (got is None) == (p is None)
            if p is not None:
                assert got.dtype == p.dtype
                R.assert_close(got, want[i], tol[i] + R.half_step(p.dtype, want[i]), ("", "dgamma", "dbeta")[i])


@pytest.mark.parametrize("mean,std", [(1000.0, 1.0), (0.0, 1e-4), (-3e4, 100.0), (0.0, 1e15)])
@pytest.mark.parametrize("N", [48, 1500, 8192])
def test_shifted_and_scaled_rows(mean, std, N):
    check(11, N, "f32", mean=mean, std=std)


def test_constant_rows_and_one_column():
    x = torch.full((5, 300), 2.5, device="cuda")
    y, mean, rstd = dyt().layer_norm_forward(x, None, None, EPS)
    assert torch.equal(y, torch.zeros_like(y)) and torch.equal(mean, torch.full_like(mean, 2.5))
    want, tol = R.norm_forward(x, None, None, EPS)
    R.assert_close(rstd, want[2], tol[2], "rstd")
    y, mean, rstd = dyt().layer_norm_forward(x, None, None, 0.0)  # 0 * inf, as the formula has it
    assert torch.isnan(y).all() and torch.isinf(rstd).all()


@pytest.mark.parametrize("N", [40, 1000, 2048, 9000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_row_stays_its_own(N, bad):
    x, dy, gamma, beta = inputs(6, N)
    clean, mean0, rstd0 = dyt().layer_norm_forward(x.t, gamma, beta, EPS)
    x.t[2, N // 2] = bad
    y, mean, rstd = dyt().layer_norm_forward(x.t, gamma, beta, EPS)
    assert torch.isnan(y[2]).all()
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(y[keep], clean[keep]) and torch.equal(mean[keep], mean0[keep])
    dx, dgamma, dbeta = dyt().layer_norm_backward(x.t, dy.t, mean, rstd, gamma, beta)
    assert torch.isnan(dx[2]).all() and torch.isfinite(dx[keep]).all()
    assert torch.isnan(dgamma).all() and torch.isfinite(dbeta).all()  # dbeta does not read x


@pytest.mark.parametrize("M,N,xd", [(300, 100, "f32"), (300, 128, "bf16"), (50, 4096, "bf16"), (4, 9000, "f32")])
def test_in_place(M, N, xd):
    x, dy, gamma, beta = inputs(M, N, xd)
    y, mean, rstd = dyt().layer_norm_forward(x.t, gamma, beta, EPS)
    dx, dgamma, dbeta = dyt().layer_norm_backward(x.t, dy.t, mean, rstd, gamma, beta)
    a = x.t.clone()
    assert dyt().layer_norm_forward(a, gamma, beta, EPS, out=a)[0] is a and torch.equal(a, y)
    for which in (0, 1):
        a, b = x.t.clone(), dy.t.clone()
        got = dyt().layer_norm_backward(a, b, mean, rstd, gamma, beta, dx=(a, b)[which])
        assert torch.equal(got[0], dx) and torch.equal(got[1], dgamma) and torch.equal(got[2], dbeta)


def test_empty_shapes():
    g = torch.ones(8, device="cuda", dtype=torch.bfloat16)
    x = torch.empty(0, 8, device="cuda")
    y, mean, rstd = dyt().layer_norm_forward(x, g, g)
    assert y.shape == (0, 8) and mean.numel() == rstd.numel() == 0
    dg = torch.full_like(g, 3.0)
    dx, dgamma, dbeta = dyt().layer_norm_backward(x, x, mean, rstd, g, g, dgamma=dg)
    assert torch.equal(dgamma, torch.zeros_like(g)) and torch.equal(dbeta, torch.zeros_like(g))
    y, _, _ = dyt().layer_norm_forward(torch.empty(3, 0, device="cuda"))
    assert y.shape == (3, 0)


def test_a_part_of_a_vector_over_several_runs():
    check(148 * 128 * 129 + 5, 61, "bf16", pitch=64, out_pitch=64)


def test_rows_without_elements_have_no_statistics():
    mean, rstd = torch.zeros(3, device="cuda"), torch.zeros(3, device="cuda")
    dyt().layer_norm_forward(torch.empty(3, 0, device="cuda"), mean=mean, rstd=rstd)
    assert torch.isnan(mean).all() and torch.isnan(rstd).all()


@pytest.mark.parametrize("M,N,xd", [(5000, 64, "f32"), (3000, 1001, "f16"), (1000, 4096, "bf16"), (40, 20000, "bf16")])
def test_deterministic_with_a_garbage_workspace(M, N, xd):
    x, dy, gamma, beta = inputs(M, N, xd)
    _, mean, rstd = dyt().layer_norm_forward(x.t, gamma, beta, EPS)
    ws = dyt().layer_norm_workspace(x.t)
    first = None
    for fill in (0, 255, 77):
        ws.fill_(fill)
        got = dyt().layer_norm_backward(x.t, dy.t, mean, rstd, gamma, beta, ws=ws)
        first = got if first is None else first
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_leading_dimensions_and_other_stream():
    x = torch.randn(3, 5, 96, device="cuda")[:, :, :90]
    gamma = torch.rand(90, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, mean, rstd = dyt().layer_norm_forward(x, gamma, None, EPS, stream=s)
    dx, dgamma, dbeta = dyt().layer_norm_backward(x, x, mean, rstd, gamma, stream=s)
    s.synchronize()
    assert y.shape == x.shape and mean.shape == (3, 5) and dbeta is None
    flat = x.reshape(15, 90)
    want, tol = R.norm_forward(flat, gamma, None, EPS)
    R.assert_close(y.reshape(15, 90), want[0], tol[0] + R.half_step(y.dtype, want[0]), "y")
    want, tol = R.norm_backward(flat, flat, mean, rstd, gamma)
    R.assert_close(dgamma, want[1], tol[1] + R.half_step(dgamma.dtype, want[1]), "dgamma")


def test_module_gradients_and_differences():
    torch.manual_seed(3)
    layer = dyt().LayerNorm(70, device="cuda")
    with torch.no_grad():
        layer.gamma.uniform_(0.5, 1.5)
        layer.beta.uniform_(-1, 1)
    x = torch.randn(4, 6, 70, device="cuda", requires_grad=True)
    up = torch.randn(4, 6, 70, device="cuda")
    (layer(x) * up).sum().backward()
    flat = x.detach().reshape(24, 70)
    _, mean, rstd = dyt().layer_norm_forward(flat, layer.gamma.detach(), layer.beta.detach(), layer.eps)
    want, tol = R.norm_backward(flat, up.reshape(24, 70), mean, rstd, layer.gamma.detach())
    R.assert_close(x.grad.reshape(24, 70), want[0], tol[0] + R.half_step(torch.float32, want[0]), "dx")
    R.assert_close(layer.gamma.grad, want[1], tol[1] + R.half_step(torch.float32, want[1]), "dgamma")
    R.assert_close(layer.beta.grad, want[2], tol[2] + R.half_step(torch.float32, want[2]), "dbeta")
    # central differences of the kernel's own forward along a direction v of x: with a step t the
    # difference is off by t^2 / 6 times the third derivative (below 60 here: |h'''| stays under 8 per
    # element along a unit-scale direction) and by the forward's rounding, 2^-20 * 41 values / t
    v = torch.randn(4, 6, 70, device="cuda")
    v = v / v.norm()
    t = 2.0 ** -5
    with torch.no_grad():
        f = lambda a: float((layer(a).double() * up.double()).sum())  # noqa: E731
        slope = (f(x + t * v) - f(x - t * v)) / (2 * t)
    assert abs(slope - float((x.grad * v).sum())) < t * t / 6 * 60 + 41 * 2.0 ** -20 / t


def test_module_without_parameters_or_bias():
    x = torch.randn(7, 33, device="cuda", requires_grad=True)
    dyt().LayerNorm(33, affine=False)(x).square().sum().backward()
    a = dyt().LayerNorm(33, bias=False, device="cuda")
    assert a.beta is None and len(list(a.parameters())) == 1
    a(x).sum().backward()
    assert a.gamma.grad is not None
    with pytest.raises(ValueError):
        a(torch.randn(3, 32, device="cuda"))


def test_expanded_upstream_gradient_and_transposed_input():
    layer = dyt().LayerNorm(24, device="cuda")
    x = torch.randn(24, 10, device="cuda", requires_grad=True)
    layer(x.t()).sum().backward()  # dy is an expanded one, x has no dense rows
    want, tol = R.norm_forward(x.detach().t(), None, None, layer.eps)
    R.assert_close(layer.gamma.grad, want[0].sum(0), tol[0].sum(0) + 136 * R.U * want[0].abs().sum(0), "dgamma")


def test_captured_and_replayed():
    x, dy, gamma, beta = inputs(200, 520, "bf16")
    xs, ds = x.t.clone(), dy.t.clone()
    ws = dyt().layer_norm_workspace(xs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            y, mean, rstd = dyt().layer_norm_forward(xs, gamma, beta, EPS)
            dyt().layer_norm_backward(xs, ds, mean, rstd, gamma, beta, ws=ws)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, mean, rstd = dyt().layer_norm_forward(xs, gamma, beta, EPS)
        out = dyt().layer_norm_backward(xs, ds, mean, rstd, gamma, beta, ws=ws)
    for seed in (5, 6):
        a, b, _, _ = inputs(200, 520, "bf16", seed=seed)
        xs.copy_(a.t)
        ds.copy_(b.t)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        y2, m2, r2 = dyt().layer_norm_forward(xs, gamma, beta, EPS)
        want = dyt().layer_norm_backward(xs, ds, m2, r2, gamma, beta)
        assert torch.equal(y, y2) and all(torch.equal(p, q) for p, q in zip(out, want))


def test_two_calls_at_once():
    # on two streams, each with its own workspace
    x, dy, gamma, beta = inputs(3000, 520, "bf16")
    _, mean, rstd = dyt().layer_norm_forward(x.t, gamma, beta, EPS)
    want = dyt().layer_norm_backward(x.t, dy.t, mean, rstd, gamma, beta)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[dyt().layer_norm_backward(x.t, dy.t, mean, rstd, gamma, beta, stream=s) for s in streams] for _ in range(8)]
    torch.cuda.synchronize()
    for pair in got:
        for one in pair:
            assert all(torch.equal(a, b) for a, b in zip(one, want))


def test_refusals():
    x = torch.randn(4, 16, device="cuda")
    g = torch.ones(16, device="cuda")
    m = torch.zeros(4, device="cuda")
    f, b = dyt().layer_norm_forward, dyt().layer_norm_backward
    for call in (lambda: f(x, g[:8]), lambda: f(x, g.cpu()), lambda: f(x.cpu()), lambda: f(x.t()),
                 lambda: f(x, out=x[:2]), lambda: f(x, out=x.half()), lambda: f(x, mean=m[:3]),
                 lambda: f(x, torch.ones(32, device="cuda")[::2]), lambda: f(torch.tensor(1.0, device="cuda")),
                 lambda: b(x, x[:3], m, m), lambda: b(x, x, m[:3], m), lambda: b(x, x, m, m, g, dgamma=g[:4]),
                 lambda: b(x, x, m, m, dgamma=g), lambda: b(x, x, m, m, g, ws=g)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: f(x.double()), lambda: f(x, g.double()), lambda: b(x, x, m.double(), m)):
        with pytest.raises(TypeError):
            call()
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(dyt().DytError):
            f(x, eps=eps)
    with pytest.raises(dyt().DytError):
        b(x, x, m, m, g, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
