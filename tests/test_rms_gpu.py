"""The root-mean-square norm's kernels against its binary64 formulas: lengths from one
element, ragged and strided rows, with and without a residual, 8-bit output with a scale
a row and a scale for 128 columns, dtypes, extreme values, refusals."""
from __future__ import annotations

import threading

import pytest
import torch

from tests import rms_helpers as S
from tests import row_helpers as R

pytestmark = pytest.mark.gpu

EPS = 1e-6
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")


def dyt():
    import elementwise_reduction_b200 as d
    return d


def inputs(M, N, xd="f32", pd="f32", res=True, seed=0, pitch=None, offset=0):
    """x, residual (or None), the gradient of y, gamma."""
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, res, dy = (R.Guarded(M, N, R.DT[xd], pitch, offset) if want else None for want in (True, res, True))
    x.set(r(M, N) + 0.2)
    if res is not None:
        res.set(2 * r(M, N))
    dy.set(r(M, N))
    return x, res, dy, (1 + 0.2 * r(N)).to(R.DT[pd])


def check_forward(x, res, gamma, out_pitch=None, out_offset=0):
    M, N, t = x.M, x.N, x.t.dtype
    y, h = (R.Guarded(M, N, t, out_pitch, out_offset, fill=7.0) for _ in range(2))
    rt = None if res is None else res.t
    got = dyt().rms_norm_forward(x.t, gamma, rt, EPS, out=y.t, residual_out=None if res is None else h.t)
    info = dyt().dyt_last_launch_info()
    want, tol = S.forward(x.t, rt, gamma, EPS)
    R.assert_close(got[2], want[2], tol[2], "rstd")
    R.assert_close(y.t, want[0], tol[0] + R.half_step(t, want[0]), "y")
    y.assert_surroundings_untouched("y")
    if res is None:
        assert got[1] is x.t
    else:
        R.assert_close(h.t, want[1], tol[1] + R.half_step(t, want[1]), "h")
        h.assert_surroundings_untouched("h")
    assert info["op"] == 9 and info["kernels"] == 1
    return got, info


def check_quantize(x, res, gamma, group, out_pitch=None, out_offset=0):
    M, N, t = x.M, x.N, x.t.dtype
    pitch = N if out_pitch is None else out_pitch
    buf = torch.full((96 + out_offset + M * pitch,), 0x55, dtype=torch.uint8, device="cuda")
    q = buf.view(torch.float8_e4m3fn).as_strided((M, N), (pitch, 1), 32 + out_offset)
    h = R.Guarded(M, N, t, out_pitch, out_offset, fill=7.0)
    rt = None if res is None else res.t
    _, scale, hh = dyt().rms_norm_quantize(x.t, gamma, rt, EPS, group, out=q,
                                           residual_out=None if res is None else h.t)
    info = dyt().dyt_last_launch_info()
    S.assert_quantized(q, scale, x.t, rt, gamma, EPS, group)
    assert scale.shape == ((M, -(-N // 128)) if group else (M,))
    inside = torch.zeros_like(buf, dtype=torch.bool)
    inside.as_strided((M, N), (pitch, 1), 32 + out_offset).fill_(True)
    assert (buf[~inside] == 0x55).all(), "q: written outside its rows"
    if res is not None:
        want = S.forward(x.t, rt, gamma, EPS)
        R.assert_close(hh, want[0][1], want[1][1] + R.half_step(t, want[0][1]), "h")
        h.assert_surroundings_untouched("h")
    assert info["op"] == 10 and info["kernels"] == 1
    return info


def check_backward(h, dy, rstd, gamma, dres, out_pitch=None, out_offset=0):
    M, N, t = h.M, h.N, h.t.dtype
    dx = R.Guarded(M, N, t, out_pitch, out_offset, fill=7.0)
    rt = None if dres is None else dres.t
    _, dgamma = dyt().rms_norm_backward(h.t, dy.t, rstd, gamma, rt, dx=dx.t)
    info = dyt().dyt_last_launch_info()
    want, tol = S.backward(h.t, dy.t, rstd, gamma, rt)
    R.assert_close(dx.t, S.overflowed(want[0], t), tol[0] + R.half_step(t, want[0]), "dx")
    dx.assert_surroundings_untouched("dx")
    if gamma is None:
        assert dgamma is None
    else:
        assert dgamma.dtype == gamma.dtype
        R.assert_close(dgamma, want[1], tol[1] + R.half_step(gamma.dtype, want[1]), "dgamma")
    assert info["op"] == 11
    return info


def check(M, N, xd="f32", pd="f32", out_pitch=None, out_offset=0, **kw):
    infos = []
    for res in (False, True):
        x, r, dy, gamma = inputs(M, N, xd, pd, res, **kw)
        got, fwd = check_forward(x, r, gamma, out_pitch, out_offset)
        for group in (0, 128):
            check_quantize(x, r, gamma, group, out_pitch, out_offset)
        # (the residual in the place of the stored sum's gradient)
        infos = [fwd, check_backward(x, dy, got[2], gamma, r, out_pitch, out_offset)]
    return infos


WIDTHS = [1, 2, 3, 4, 7, 8, 9, 16, 17, 24, 31, 32, 33, 64, 65, 100, 127, 128, 129, 160, 255, 256, 257, 511, 512, 513,
          520, 640, 1000, 1024, 1040, 2047, 2048, 4096, 4100, 4104, 8191, 8192]


@pytest.mark.parametrize("xd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", WIDTHS)
def test_widths(N, xd):
    _, bwd = check(37, N, xd)
    assert bwd["kernels"] == (1 if bwd["grid"] == 1 else 2)


@pytest.mark.parametrize("xd", ["f32", "bf16"])
@pytest.mark.parametrize("N", [8200, 12001, 16383, 16384, 16385, 16520, 32776, 40001])
def test_long_rows(N, xd):
    check(5, N, xd)


def test_long_rows_more_than_ctas():
    check(700, 17000, "bf16")
    check(700, 9001, "f32")


# columns, dtype, CTAs that share a row forward, and at least in the backward (0: no cluster)
SHARED = [(8192, "f32", 0, 0), (8200, "f32", 2, 2), (12288, "f32", 2, 2), (16384, "f32", 2, 2), (16388, "f32", 4, 4),
          (32768, "f32", 4, 4), (32772, "f32", 0, 0), (8200, "bf16", 0, 2), (12288, "bf16", 0, 2),
          (16384, "f16", 0, 2), (16392, "bf16", 2, 4), (20480, "bf16", 2, 4), (32768, "f16", 2, 4),
          (32776, "bf16", 4, 0), (65536, "bf16", 4, 0), (65544, "bf16", 0, 0),
          (8193, "f32", 2, 2), (12290, "bf16", 0, 2), (16385, "f16", 2, 4), (20481, "bf16", 2, 4), (30001, "f32", 4, 4),
          (32767, "bf16", 2, 4),
          (8193, "bf16", 0, 2), (9216, "bf16", 0, 2), (18432, "f16", 2, 4), (32769, "f32", 0, 0), (65535, "f16", 4, 0)]


@pytest.mark.parametrize("N,xd,fwd,bwd", SHARED)
def test_rows_that_a_cluster_shares(N, xd, fwd, bwd):
    for M in (1, 5, 41, 200):
        infos = check(M, N, xd)
        assert infos[0]["col_chunks"] == max(1, fwd)
        assert infos[1]["col_chunks"] in ((bwd, 8) if bwd == 4 else (bwd, 2 * bwd, 4 * bwd) if bwd else (1,))
        assert all(i["grid"] % i["col_chunks"] == 0 for i in infos)


@pytest.mark.parametrize("N,xd,pitch", [(12288, "bf16", 12304), (16384, "f32", 16384), (20480, "f16", 20480),
                                       (12289, "bf16", 12289), (20480, "f16", 20481), (9217, "bf16", 9217)])
def test_many_rows_that_a_cluster_shares(N, xd, pitch):
    """More rows than run at once, beside a second call and from a graph: the same bits."""
    M = 20000 if xd != "f32" else 10000
    x, r, dy, gamma = inputs(M, N, xd, pitch=pitch)
    want = dyt().rms_norm_forward(x.t, gamma, r.t, EPS)
    q = dyt().rms_norm_quantize(x.t, gamma, r.t, EPS, 128)
    grads = dyt().rms_norm_backward(x.t, dy.t, want[2], gamma, r.t)
    for i in (0, 1, 149, 7000, M - 1):  # (rows stand alone)
        one = [t.t[i:i + 1] for t in (x, r, dy)]
        a = dyt().rms_norm_forward(one[0], gamma, one[1], EPS)
        assert all(torch.equal(u, v[i:i + 1]) for u, v in zip(a, want))
        b = dyt().rms_norm_quantize(one[0], gamma, one[1], EPS, 128)
        assert torch.equal(b[0].view(torch.uint8), q[0][i:i + 1].view(torch.uint8)) and torch.equal(b[1], q[1][i:i + 1])
        c = dyt().rms_norm_backward(one[0], one[2], want[2][i:i + 1], gamma, one[1])
        assert torch.equal(c[0], grads[0][i:i + 1])
    part = slice(0, 300)
    exact, tol = S.backward(x.t[part], dy.t[part], want[2][part], gamma, r.t[part])
    R.assert_close(grads[0][part], exact[0], tol[0] + R.half_step(x.t.dtype, exact[0]), "dx")
    _, some = dyt().rms_norm_backward(x.t[part], dy.t[part], want[2][part], gamma, r.t[part])
    R.assert_close(some, exact[1], tol[1] + R.half_step(gamma.dtype, exact[1]), "dgamma")
    total = torch.zeros(N, dtype=torch.float64, device="cuda")
    room = torch.zeros(N, dtype=torch.float64, device="cuda")
    for i in range(0, M, 2000):
        e, t = S.backward(x.t[i:i + 2000], dy.t[i:i + 2000], want[2][i:i + 2000], gamma, r.t[i:i + 2000])
        total += e[1]
        room += t[1]
    R.assert_close(grads[1], total, room + R.half_step(gamma.dtype, total), "dgamma")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = dyt().rms_norm_forward(x.t, gamma, r.t, EPS)
        back = dyt().rms_norm_backward(x.t, dy.t, again[2], gamma, r.t)
    for o in (*again, *back):
        o.zero_()
    torch.cuda.synchronize()
    graph.replay()
    with torch.cuda.stream(side):
        other = dyt().rms_norm_forward(x.t, gamma, r.t, EPS)
        obwd = dyt().rms_norm_backward(x.t, dy.t, want[2], gamma, r.t)
    torch.cuda.synchronize()
    for got in ((*again, *back), (*other, *obwd)):
        assert all(torch.equal(u, v) for u, v in zip(got, (*want, *grads)))


@pytest.mark.parametrize("xd,pd", [("f32", "f32"), ("bf16", "f32"), ("f16", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("N,rows", [(16, 128), (64, 128), (96, 64), (100, 64), (250, 32), (512, 16), (500, 16),
                                    (1024, 8), (1001, 8), (4096, 2), (8191, 1)])
def test_few_rows_are_one_ctas(N, rows, xd, pd):
    """One, a whole step, a row more, two steps, a row beyond them: the last with partial sums."""
    for M in sorted({1, rows, rows + 1, 2 * rows, 2 * rows + 1}):
        x, r, dy, gamma = inputs(M, N, xd, pd)
        rstd = torch.rand(M, device="cuda") + 0.5
        info = check_backward(x, dy, rstd, gamma, r)
        if info["grid"] == 1:
            assert info["kernels"] == 1 and info["workspace_bytes"] == 0
        else:
            assert info["kernels"] == 2 and M > rows
        dx, none = dyt().rms_norm_backward(x.t, dy.t, rstd, gamma, r.t, frozen=True)
        assert none is None and dyt().dyt_last_launch_info()["kernels"] == 1
        assert torch.equal(dx, dyt().rms_norm_backward(x.t, dy.t, rstd, gamma, r.t)[0])


def test_first_calls_of_a_cluster_inside_a_capture():
    """What the launch asks about the device is asked while a stream is captured."""
    M, N = 300, 8968  # (no other test has CTAs of this size)
    x, r, dy, gamma = inputs(M, N, "bf16")
    x32, r32, _, _ = inputs(M, N, "f32")
    rstd = torch.rand(M, device="cuda") + 0.5
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx, dgamma = dyt().rms_norm_backward(x.t, dy.t, rstd, gamma, r.t)
        y, h, _ = dyt().rms_norm_forward(x32.t, gamma, r32.t, EPS)
    graph.replay()
    want, tol = S.backward(x.t, dy.t, rstd, gamma, r.t)
    R.assert_close(dx, want[0], tol[0] + R.half_step(dx.dtype, want[0]), "dx")
    R.assert_close(dgamma, want[1], tol[1] + R.half_step(gamma.dtype, want[1]), "dgamma")
    want, tol = S.forward(x32.t, r32.t, gamma, EPS)
    R.assert_close(y, want[0], tol[0] + R.half_step(y.dtype, want[0]), "y")
    R.assert_close(h, want[1], tol[1] + R.half_step(h.dtype, want[1]), "h")


def test_threads_that_call_at_once():
    """Two threads on streams of their own, clusters and rows for free CTAs: the bits of one after the other."""
    cases = [inputs(2000, N, xd, seed=i) for i, (N, xd) in enumerate([(4096, "bf16"), (9216, "bf16"), (1001, "f16")])]
    run = lambda x, r, dy, g: (*(f := dyt().rms_norm_forward(x.t, g, r.t, EPS)),  # noqa: E731
                               *dyt().rms_norm_backward(f[1], dy.t, f[2], g, r.t))
    want = [run(*c) for c in cases]
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[k] = [run(*cases[(k + i) % 3]) for i in range(30)]
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for k in range(2):
        for i, o in enumerate(got[k]):
            assert all(torch.equal(a, b) for a, b in zip(o, want[(k + i) % 3]))


@pytest.mark.parametrize("M", [1, 2, 3, 7, 8, 9, 63, 147, 149, 297, 1000, 4097, 65537])
@pytest.mark.parametrize("N,xd", [(32, "bf16"), (17, "f32"), (640, "f16"), (1288, "bf16")])
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
        for res in (False, True):
            x, r, dy, gamma = inputs(127 * step + extra, N, "bf16", res=res)
            rstd = dyt().rms_norm_forward(x.t, gamma)[2]
            assert check_backward(x, dy, rstd, gamma, r)["rows_per_step"] == rows


@pytest.mark.parametrize("xd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,pitch,offset,out_pitch,out_offset", [
    (64, 72, 0, 64, 0), (64, 64, 1, 64, 1), (64, 65, 0, 67, 3), (256, 264, 0, 264, 8), (256, 256, 0, 256, 4),
    (1000, 1001, 2, 1000, 0), (4096, 4100, 1, 4099, 2), (9000, 9008, 0, 9003, 1), (9001, 9003, 3, 9005, 7),
    (20, 21, 1, 20, 0), (3, 3, 1, 3, 2), (1, 5, 1, 2, 1)])
def test_strides_and_offsets(N, pitch, offset, out_pitch, out_offset, xd):
    for M in (9, 1300):
        check(M, N, xd, pitch=pitch, offset=offset, out_pitch=out_pitch, out_offset=out_offset)


@pytest.mark.parametrize("xd,pd", [(a, b) for a in ("f32", "bf16", "f16") for b in ("f32", "bf16", "f16")])
def test_dtype_matrix(xd, pd):
    check(65, 136, xd, pd)
    check(9, 1032, xd, pd)
    check(4, 20001, xd, pd)


@pytest.mark.parametrize("N", [100, 1024, 9001, 20000])
def test_without_gamma(N):
    for res in (False, True):
        x, r, dy, _ = inputs(13, N, "bf16", res=res)
        got, _ = check_forward(x, r, None)
        check_quantize(x, r, None, 128)
        assert check_backward(x, dy, got[2], None, r)["kernels"] == 1


def test_offsets_beyond_32_bits():
    # rows 2^30 + 8 elements apart: the last one starts past 2^31 elements
    pitch, N = (1 << 30) + 8, 1000
    g = torch.Generator("cuda").manual_seed(5)
    x, r, y = (torch.empty(2 * pitch + N + 8, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    xv, rv, yv = (t.as_strided((3, N), (pitch, 1)) for t in (x, r, y))
    xv.copy_(torch.randn(3, N, device="cuda", generator=g))
    rv.copy_(torch.randn(3, N, device="cuda", generator=g))
    gamma = torch.rand(N, device="cuda", generator=g)
    _, h, rstd = dyt().rms_norm_forward(xv, gamma, rv, EPS, out=yv)
    want, tol = S.forward(xv, rv, gamma, EPS)
    R.assert_close(yv, want[0], tol[0] + R.half_step(yv.dtype, want[0]), "y")
    R.assert_close(h, want[1], tol[1] + R.half_step(yv.dtype, want[1]), "h")
    dx, dgamma = dyt().rms_norm_backward(xv, rv, rstd, gamma, yv, dx=yv.clone())
    want, tol = S.backward(xv, rv, rstd, gamma, yv)
    R.assert_close(dx, want[0], tol[0] + R.half_step(dx.dtype, want[0]), "dx")
    R.assert_close(dgamma, want[1], tol[1], "dgamma")
    q = y.view(torch.float8_e4m3fn).as_strided((3, N), (pitch, 1))
    _, scale, _ = dyt().rms_norm_quantize(xv, gamma, rv, EPS, 128, out=q)
    S.assert_quantized(q, scale, xv, rv, gamma, EPS, 128)


@pytest.mark.parametrize("N", [24, 100, 1000, 1024, 4096, 9001, 20000])
@pytest.mark.parametrize("xd", ["f32", "bf16"])
def test_rows_of_zeros_nan_and_infinity_keep_to_themselves(N, xd):
    for res in (False, True):
        x, r, dy, gamma = inputs(40, N, xd, res=res)
        clean = dyt().rms_norm_forward(x.t, gamma, None if r is None else r.t, EPS)
        plain = [dyt().rms_norm_quantize(x.t, gamma, None if r is None else r.t, EPS, k)[:2] for k in (0, 128)]
        bad = {3: NAN, 17: INF, 18: -INF, 39: 0.0}
        for row, v in bad.items():
            x.t[row, N // 2] = v
        x.t[39] = 0.0
        if r is not None:
            r.t[39] = 0.0
        rt = None if r is None else r.t
        y, h, rstd = dyt().rms_norm_forward(x.t, gamma, rt, EPS)
        good = [i for i in range(40) if i not in bad]
        for a, b in zip((y, h, rstd), clean):
            assert torch.equal(a[good], b[good])
        assert torch.isnan(y[3]).all() and torch.isnan(rstd[3])
        assert rstd[17] == 0 and rstd[18] == 0 and torch.isnan(y[17, N // 2])
        assert (y[39] == 0).all() and abs(float(rstd[39]) - EPS ** -0.5) < 1e-3 * EPS ** -0.5
        for k, (q0, s0) in zip((0, 128), plain):
            q, s, _ = dyt().rms_norm_quantize(x.t, gamma, rt, EPS, k)
            assert torch.equal(q.view(torch.uint8)[good], q0.view(torch.uint8)[good]) and torch.equal(s[good], s0[good])
            assert torch.isnan(q.float()[3]).all() and torch.isnan(s[3]).all()
            at = 0 if k == 0 else N // 2 // 128
            s = s.reshape(40, -1)
            assert torch.isnan(s[17, at]) and torch.isnan(q.float()[17, N // 2]) and torch.isnan(s[18, at])
            assert (q.float()[39] == 0).all()
            assert torch.allclose(s[39], s.new_tensor(S.LEAST / S.QMAX), rtol=1e-6, atol=0)


@pytest.mark.parametrize("xd,value", [("f32", 1e18), ("f32", 1e-18), ("bf16", 1e18), ("f16", 60000.0), ("f16", 1e-7)])
def test_rows_of_large_and_small_values(xd, value):
    for N in (100, 1024, 9000):
        x, r, dy, gamma = inputs(9, N, xd)
        x.t.mul_(value / x.t.abs().max())
        r.t.mul_(value / 2 / r.t.abs().max())
        x.t.sub_(r.t / 2)
        got, _ = check_forward(x, r, gamma)
        check_quantize(x, r, gamma, 0)
        check_quantize(x, r, gamma, 128)


def test_rows_of_the_lowest_value():
    # their squares pass binary32: a factor of 0, and nothing but 0 comes out
    x = torch.full((4, 500), torch.finfo(torch.float32).min, device="cuda")
    y, _, rstd = dyt().rms_norm_forward(x)
    assert (rstd == 0).all() and (y == 0).all()
    q, scale, _ = dyt().rms_norm_quantize(x, group=128)
    assert (q.float() == 0).all() and torch.isfinite(scale).all()


@pytest.mark.parametrize("M,N", [(0, 64), (0, 0), (5, 0)])
def test_empty(M, N):
    x = torch.empty(M, N, device="cuda")
    gamma = torch.ones(N, device="cuda")
    y, h, rstd = dyt().rms_norm_forward(x, gamma, x)
    assert y.shape == h.shape == (M, N) and rstd.shape == (M,) and torch.isnan(rstd).all()
    q, scale, _ = dyt().rms_norm_quantize(x, gamma, group=128)
    assert q.shape == (M, N) and scale.shape == (M, -(-N // 128))
    q, scale, _ = dyt().rms_norm_quantize(x, gamma)
    assert torch.isfinite(scale).all()
    dx, dgamma = dyt().rms_norm_backward(x, x, rstd, gamma)
    assert dx.shape == (M, N) and torch.equal(dgamma, torch.zeros(N, device="cuda"))


@pytest.mark.parametrize("N", [96, 100, 1024, 4100, 9001, 20000])
@pytest.mark.parametrize("xd", ["f32", "bf16"])
def test_in_place(N, xd):
    for M in (3, 400):
        x, r, dy, gamma = inputs(M, N, xd)
        y, h, rstd = dyt().rms_norm_forward(x.t, gamma, r.t, EPS)
        for out, into in (("x", "residual"), ("residual", "x")):
            a, b = x.t.clone(), r.t.clone()
            t = {"x": a, "residual": b}
            dyt().rms_norm_forward(a, gamma, b, EPS, out=t[out], residual_out=t[into])
            assert torch.equal(t[out], y) and torch.equal(t[into], h)
        q, scale, _ = dyt().rms_norm_quantize(x.t, gamma, r.t, EPS, 128)
        b = r.t.clone()
        q2, scale2, h2 = dyt().rms_norm_quantize(x.t, gamma, b, EPS, 128, residual_out=b)
        assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(scale, scale2)
        assert h2 is b and torch.equal(b, h)
        want = dyt().rms_norm_backward(h, dy.t, rstd, gamma, r.t)
        for k in range(3):
            t = [h.clone(), dy.t.clone(), r.t.clone()]
            got = dyt().rms_norm_backward(t[0], t[1], rstd, gamma, t[2], dx=t[k])
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_the_same_bits_twice_and_on_shifted_rows():
    for N in (1000, 4096):
        x, r, dy, gamma = inputs(3000, N, "bf16")
        once = dyt().rms_norm_forward(x.t, gamma, r.t, EPS)
        back = dyt().rms_norm_backward(once[1], dy.t, once[2], gamma, r.t)
        for _ in range(3):
            again = dyt().rms_norm_forward(x.t, gamma, r.t, EPS)
            assert all(torch.equal(a, b) for a, b in zip(once, again))
            again = dyt().rms_norm_backward(once[1], dy.t, once[2], gamma, r.t)
            assert all(torch.equal(a, b) for a, b in zip(back, again))


def test_streams_and_graphs():
    x, r, dy, gamma = (t.t if isinstance(t, R.Guarded) else t for t in inputs(300, 1000, "bf16"))
    def step():
        y, h, rstd = dyt().rms_norm_forward(x, gamma, r, EPS)
        q, scale, _ = dyt().rms_norm_quantize(h, gamma, group=128)
        dx, dgamma = dyt().rms_norm_backward(h, dy, rstd, gamma, y)
        return y, h, rstd, q.view(torch.uint8), scale, dx, dgamma
    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, h, rstd = dyt().rms_norm_forward(x, gamma, r, EPS, stream=side)
    dx, dgamma = dyt().rms_norm_backward(h, dy, rstd, gamma, y, stream=side)
    side.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(dx, want[5]) and torch.equal(dgamma, want[6])
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        graphs.append((graph, outs))
    x.mul_(2)
    want = [t.clone() for t in step()]
    for graph, _ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for _, outs in graphs:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("N,xd,pitch", [(4096, "bf16", 4096), (4100, "bf16", 4101), (1504, "f16", 1600),
                                        (8192, "f32", 8192), (640, "f32", 640), (16384, "bf16", 16384)])
def test_many_rows_go_to_free_ctas(N, xd, pitch):
    # more rows than CTAs at a time, each done once: alone, beside another call, and from graphs
    d = dyt()
    M = 5003 if N > 640 else 9001
    cases = []
    for seed in (0, 1):
        x, r, dy, gamma = inputs(M, N, xd, seed=seed, pitch=pitch)
        y, h, rstd = (torch.full_like(t, NAN) for t in (x.t, x.t, dy.t[:, 0].float()))
        q = torch.full((M, N), NAN, device="cuda").to(torch.float8_e4m3fn)
        scale = torch.full((M, -(-N // 128)), NAN, device="cuda")
        cases.append((x, r, gamma, y, h, rstd, q, scale))
    def step(c):
        x, r, gamma, y, h, rstd, q, scale = c
        d.rms_norm_forward(x.t, gamma, r.t, EPS, out=y, residual_out=h, rstd=rstd)
        d.rms_norm_quantize(x.t, gamma, r.t, EPS, 128, out=q, scale=scale, residual_out=h)
    def outputs(c):
        return [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in c[3:]]
    for c in cases:
        step(c)
        assert d.dyt_last_launch_info()["grid"] == M
        want, tol = S.forward(c[0].t, c[1].t, c[2], EPS)
        R.assert_close(c[5], want[2], tol[2], "rstd")
        R.assert_close(c[3], want[0], tol[0] + R.half_step(c[3].dtype, want[0]), "y")
        R.assert_close(c[4], want[1], tol[1] + R.half_step(c[3].dtype, want[1]), "h")
        S.assert_quantized(c[6], c[7], c[0].t, c[1].t, c[2], EPS, 128)
    want = [[t.clone() for t in outputs(c)] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    graphs = []
    for s, c in zip(streams, cases):
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step(c)
            step(c)
        graphs.append(graph)
    for c in cases:
        for t in outputs(c):
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for s, c, graph in zip(streams, cases, graphs):
            with torch.cuda.stream(s):
                step(c)
                graph.replay()
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert all(torch.equal(a, b) for a, b in zip(outputs(c), w))


# ---- module ------------------------------------------------------------------------------------

def test_module_gradients_agree_with_the_formula():
    d = dyt()
    g = torch.Generator("cuda").manual_seed(3)
    layer = d.RMSNorm(72, device="cuda")
    with torch.no_grad():
        layer.gamma.copy_(1 + 0.3 * torch.randn(72, device="cuda", generator=g))
    x, r = (torch.randn(4, 5, 72, device="cuda", generator=g, requires_grad=True) for _ in range(2))
    uy, uh = (torch.randn(4, 5, 72, device="cuda", generator=g) for _ in range(2))
    y, h = layer(x, r)
    ((y * uy).sum() + (h * uh).sum()).backward()
    a, b, c = (t.detach().double().requires_grad_() for t in (x, r, layer.gamma))
    s = a + b
    n = s * torch.rsqrt(s.square().mean(-1, keepdim=True) + layer.eps)
    ((n * c * uy).sum() + (s * uh).sum()).backward()
    for got, want in ((x.grad, a.grad), (r.grad, b.grad), (layer.gamma.grad, c.grad)):
        assert torch.allclose(got.double(), want, rtol=1e-5, atol=1e-5)
    assert torch.equal(x.grad, r.grad) and x.grad.data_ptr() != r.grad.data_ptr()


def test_module_gradient_against_differences():
    layer = dyt().RMSNorm(33, device="cuda")
    g = torch.Generator("cuda").manual_seed(4)
    x, r, v, u = (torch.randn(6, 33, device="cuda", generator=g) for _ in range(4))
    def f(t):
        return float((S.forward(t, r.double(), layer.gamma.detach(), layer.eps)[0][0] * u.double()).sum())
    a = x.clone().requires_grad_()
    (layer(a, r)[0] * u).sum().backward()
    t = 1e-5
    slope = (f(x.double() + t * v.double()) - f(x.double() - t * v.double())) / (2 * t)
    assert abs(slope - float((a.grad.double() * v.double()).sum())) < 1e-4


def test_module_uses_of_its_outputs():
    d = dyt()
    layer = d.RMSNorm(40, device="cuda")
    x, r = (torch.randn(7, 40, device="cuda", requires_grad=True) for _ in range(2))
    _, h = layer(x, r)  # the stream alone
    h.sum().backward()
    assert torch.equal(x.grad, torch.ones_like(x)) and layer.gamma.grad is None
    x.grad = r.grad = None
    y, _ = layer(x, r.detach())  # the norm alone, one input frozen
    y.sum().backward()
    assert x.grad is not None and r.grad is None and layer.gamma.grad is not None
    layer.gamma.requires_grad_(False)
    layer.gamma.grad = None
    layer(x)[0].sum().backward()
    assert layer.gamma.grad is None
    # broadcast and transposed inputs are copied
    row = torch.randn(40, device="cuda", requires_grad=True)
    wide = torch.randn(40, 7, device="cuda").t()
    y, h = layer(row.expand(7, 40), wide)
    assert torch.equal(h, row + wide)
    y.sum().backward()
    assert row.grad.shape == (40,)
    with pytest.raises(ValueError):
        layer(x[:, :39])


def test_module_captured_with_its_backward():
    layer = dyt().RMSNorm(256, device="cuda", param_dtype=torch.bfloat16)
    x, r, u = (torch.randn(30, 256, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    x.requires_grad_()
    def step():
        y, h = layer(x, r)
        (dx, dg) = torch.autograd.grad((y * u).sum() + h.sum(), (x, layer.gamma))
        return y.detach(), dx, dg
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
        x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, step()))


# ---- refusals ----------------------------------------------------------------------------------

def test_refusals():
    d = dyt()
    x, many = torch.randn(6, 64, device="cuda"), torch.randn(600, 64, device="cuda")
    gamma, rstd = torch.ones(64, device="cuda"), torch.ones(6, device="cuda")
    bad = [lambda: d.rms_norm_forward(x, gamma[:63]), lambda: d.rms_norm_forward(x, gamma.double()),
           lambda: d.rms_norm_forward(x, gamma.cpu()), lambda: d.rms_norm_forward(x.double()),
           lambda: d.rms_norm_forward(x, gamma, x.bfloat16()), lambda: d.rms_norm_forward(x, gamma, x[:5]),
           lambda: d.rms_norm_forward(x, gamma, x.t()), lambda: d.rms_norm_forward(x.t()),
           lambda: d.rms_norm_forward(x, gamma, residual_out=x), lambda: d.rms_norm_forward(x, gamma, out=x[:5]),
           lambda: d.rms_norm_forward(x, eps=-1.0), lambda: d.rms_norm_forward(x, rstd=rstd[:5]),
           lambda: d.rms_norm_forward(x, gamma, x.cpu()),
           lambda: d.rms_norm_forward(x, gamma, x, out=x, residual_out=x), lambda: d.rms_norm_quantize(x, group=64),
           lambda: d.rms_norm_quantize(x, out=torch.empty(6, 64, dtype=torch.uint8, device="cuda")),
           lambda: d.rms_norm_quantize(x, scale=rstd[:5]), lambda: d.rms_norm_quantize(x, group=-128),
           lambda: d.rms_norm_quantize(x, eps=NAN), lambda: d.rms_norm_backward(x, x, rstd[:5], gamma),
           lambda: d.rms_norm_backward(x, x.half(), rstd, gamma), lambda: d.rms_norm_backward(x, x[:5], rstd, gamma),
           lambda: d.rms_norm_backward(x, x, rstd, gamma, x[:, :63]),
           lambda: d.rms_norm_backward(x, x, rstd, dgamma=gamma),
           lambda: d.rms_norm_backward(x, x, rstd, gamma, dgamma=gamma, frozen=True),
           lambda: d.rms_norm_backward(many, many, many[:, 0].contiguous(), gamma,
                                       ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
           lambda: d.rms_norm_backward(x, x, rstd.double(), gamma)]
    for k, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, d.DytError)):
            call()
            pytest.fail(f"call {k} was not refused")
