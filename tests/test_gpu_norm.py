"""GPU parity of mhc_layer_norm and mhc_layer_norm_backward against the fp64 oracle; bounds derived in
rows_util.py."""

import numpy as np
import pytest
import torch

import mhc_hyper_connection_02_b200 as mhc
from oracle import rows
from rows_util import DTYPES, check, f64, norm_bounds, norm_bwd_bounds, rounded

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 7168), (3, 7), (5, 127), (64, 512), (33, 1000), (9, 1001), (4, 8192),
          (3, 16392), (200, 64), (1000, 1032), (300, 2048), (2, 40000), (700, 96), (301, 7168),
          (400, 4096), (310, 16384), (1200, 520), (900, 264), (3, 5000), (333, 3001), (300, 32768)]


def _make(T, H, dtype, weights, seed, gap=0, offset=0.3):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H + gap), generator=g) * (0.5 + torch.rand((T, 1), generator=g))
    x = (x + offset * torch.randn((T, 1), generator=g)).to(DTYPES[dtype]).cuda()[:, :H]
    dy = torch.randn((T, H + gap), generator=g).to(DTYPES[dtype]).cuda()[:, :H]
    wt = DTYPES[weights]
    gamma = (1 + 0.2 * torch.randn(H, generator=g)).to(wt).cuda()
    beta = (0.2 * torch.randn(H, generator=g)).to(wt).cuda()
    return x, dy, gamma, beta


def _check_forward(x, gamma, beta, got, dtype, eps=1e-6):
    xd, gd, bd = f64(x), None if gamma is None else f64(gamma), None if beta is None else f64(beta)
    y, mean, rstd = rows.layer_norm(xd, gd, bd, eps)
    ey, em, er = norm_bounds(xd, gd, bd, y, mean, rstd, eps)
    check(got[1], mean, em, "mean")
    check(got[2], rstd, er, "rstd")
    check(got[0], y, rounded(y, ey, dtype), "y")


def _check_backward(dy, x, gamma, mean, rstd, got, dtype):
    a = [f64(v) if v is not None else None for v in (dy, x, gamma, mean, rstd)]
    dx, dg, db = rows.layer_norm_backward(*a)
    ex, eg, eb = norm_bwd_bounds(*a, dtype)
    check(got[0], dx, rounded(dx, ex, dtype), "d_x")
    check(got[1], dg, eg, "d_gamma")
    check(got[2], db, eb, "d_beta")


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dtype,weights", [("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32"),
                                           ("bf16", "bf16")])
def test_layer_norm(T, H, dtype, weights):
    x, dy, gamma, beta = _make(T, H, dtype, weights, T + H)
    got = mhc.layer_norm(x, gamma, beta)
    _check_forward(x, gamma, beta, got, dtype)
    back = mhc.layer_norm_backward(dy, x, gamma, got[1], got[2])
    _check_backward(dy, x, gamma, got[1], got[2], back, dtype)


@pytest.mark.parametrize("H", [512, 1001, 7168])
@pytest.mark.parametrize("gap", [1, 8, 512])
def test_rows_apart_and_unaligned(H, gap):
    x, dy, gamma, beta = _make(37, H, "bf16", "fp32", H + gap, gap=gap)
    got = mhc.layer_norm(x, gamma, beta)
    _check_forward(x, gamma, beta, got, "bf16")
    _check_backward(dy, x, gamma, got[1], got[2],
                    mhc.layer_norm_backward(dy, x, gamma, got[1], got[2]), "bf16")
    # every array one element off a 16-byte boundary
    off = [torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape) for t in
           (x, dy, gamma, beta, x)]
    for o, t in zip(off, (x, dy, gamma, beta)):
        o.copy_(t)
    got2 = mhc.layer_norm(off[0], off[2], off[3], y=off[4])
    _check_forward(x, gamma, beta, got2, "bf16")
    _check_backward(dy, x, gamma, got[1], got[2],
                    mhc.layer_norm_backward(off[1], off[0], off[2], got[1], got[2]), "bf16")


@pytest.mark.parametrize("H", [64, 1000, 1001, 7168, 20000])
def test_without_weights_and_in_place(H):
    x, dy, gamma, beta = _make(19, H, "bf16", "fp32", H)
    for g, b in ((None, None), (gamma, None), (None, beta)):
        got = mhc.layer_norm(x, g, b, eps=1e-3)
        _check_forward(x, g, b, got, "bf16", eps=1e-3)
        _check_backward(dy, x, g, got[1], got[2],
                        mhc.layer_norm_backward(dy, x, g, got[1], got[2]), "bf16")
    ref = mhc.layer_norm(x, gamma, beta)[0]
    z = x.clone()
    out = mhc.layer_norm(z, gamma, beta, y=z)[0]
    assert out.data_ptr() == z.data_ptr() and torch.equal(out, ref)


def test_a_stream_of_the_residual():
    """One stream of R [T,4,H] is a set of rows 4H apart."""
    g = torch.Generator().manual_seed(5)
    R = torch.randn((50, 4, 1024), generator=g).to(torch.bfloat16).cuda()
    x = R[:, 2]
    got = mhc.layer_norm(x)
    _check_forward(x, None, None, got, "bf16")


@pytest.mark.parametrize("H", [1000, 7168])
def test_mean_far_above_the_deviation(H):
    """A row whose mean is 1000 times its deviation (fp32): the bound carries mean|x| through."""
    g = torch.Generator().manual_seed(H)
    x = (1000 + torch.randn((8, H), generator=g)).cuda()
    _check_forward(x, None, None, mhc.layer_norm(x), "fp32")


@pytest.mark.parametrize("H", [512, 1001, 7168])
def test_constant_zero_and_non_finite_rows(H):
    x = torch.randn((5, H), device="cuda").to(torch.bfloat16)
    x[1] = 0
    x[2] = 3
    x[3, H // 2] = float("nan")
    x[4, 0] = float("inf")
    y, mean, rstd = mhc.layer_norm(x)
    assert torch.equal(y[1:3], torch.zeros_like(y[1:3]))
    assert mean[2].item() == 3 and abs(rstd[1].item() - 1e3) < 1e-3
    assert torch.isnan(y[3:]).all()
    _check_forward(x[:1], None, None, (y[:1], mean[:1], rstd[:1]), "bf16")


def test_no_tokens_and_untouched_neighbours():
    gamma = torch.ones(64, device="cuda")
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = mhc.layer_norm(e, gamma)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dg, db = mhc.layer_norm_backward(e, e, gamma, mean, rstd)
    assert dx.shape == (0, 64) and not dg.any() and not db.any() and dg.shape == (64,)
    for H in (64, 1001, 7168):
        x, dy, gamma, beta = _make(6, H, "bf16", "fp32", H)
        big = torch.full((8 * H + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = big[H: 7 * H].view(6, H)
        _, mean, rstd = mhc.layer_norm(x, gamma, beta, y=out)
        assert (big[:H] == 7).all() and (big[7 * H:] == 7).all()
        mhc.layer_norm_backward(dy, x, gamma, mean, rstd, d_x=out)
        assert (big[:H] == 7).all() and (big[7 * H:] == 7).all()


def test_same_bits_each_time_and_in_a_graph():
    x, dy, gamma, beta = _make(777, 2048, "bf16", "fp32", 9)
    y, mean, rstd = mhc.layer_norm(x, gamma, beta)
    ref = [y, *mhc.layer_norm_backward(dy, x, gamma, mean, rstd)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        a, m, r = mhc.layer_norm(x, gamma, beta)
        got = [a, *mhc.layer_norm_backward(dy, x, gamma, m, r)]
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(got, ref):
            assert torch.equal(g, w)
    with_stream = mhc.layer_norm_backward(dy, x, gamma, mean, rstd, stream=side)
    side.synchronize()
    for g, w in zip(with_stream, ref[1:]):
        assert torch.equal(g, w)


def test_gradient_against_differences():
    """fp32 rows: the directional derivative of sum(d_y y) by a central difference of the forward
    (step h: truncation h^2, rounding U / h of the sizes involved)."""
    x, dy, gamma, beta = _make(4, 257, "fp32", "fp32", 2)
    _, mean, rstd = mhc.layer_norm(x, gamma, beta)
    dx, dg, db = mhc.layer_norm_backward(dy, x, gamma, mean, rstd)
    v = torch.randn_like(x)
    h = 2.0 ** -7
    up, dn = mhc.layer_norm(x + h * v, gamma, beta)[0], mhc.layer_norm(x - h * v, gamma, beta)[0]
    diff = ((up.double() - dn.double()) * dy.double()).sum().item() / (2 * h)
    size = (dy.double().abs() * v.double().abs() * rstd.double()[:, None]).sum().item()
    assert abs(diff - (dx.double() * v.double()).sum().item()) < 1e-3 * size


def _rows_at(t, first, stride, fill):
    """t's rows `stride` elements apart from element `first` of a buffer of `fill`, and the buffer."""
    T, H = t.shape
    buf = torch.full((first + (T - 1) * stride + H + 5,), fill, dtype=t.dtype, device="cuda")
    rows_ = torch.as_strided(buf, (T, H), (stride, 1), first)
    rows_.copy_(t)
    return rows_, buf


@pytest.mark.parametrize("T", [1, 2, 9, 331])
@pytest.mark.parametrize("H", [1, 15, 16, 17, 33, 255, 1001, 5003])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_arrays_of_unlike_phases(T, H, dtype):
    """x, d_y and the outputs begin at addresses and lie at distances of their own; what lies beside
    the rows is a NaN that reaches nothing, and stays."""
    x, dy, gamma, beta = _make(T, H, dtype, "fp32", T * H)
    nan = float("nan")
    for i, (fx, gx, fd, gd, fo) in enumerate([(0, 0, 0, 0, 0), (1, 0, 1, 0, 1), (3, 5, 0, 0, 2),
                                             (2, H, 5, 3, 0), (0, 1, 7, 0, 3)]):
        xs, bx = _rows_at(x, fx, H + gx, nan)
        ds, bd = _rows_at(dy, fd, H + gd, nan)
        out, bo = _rows_at(x, fo, H, nan)
        keep = [b.clone() for b in (bx, bd)]
        got = mhc.layer_norm(xs, gamma, beta, y=out)
        edge = torch.cat((bo[:fo], bo[fo + T * H:]))
        assert torch.isnan(edge).all() and edge.numel() == fo + 5
        _check_forward(x, gamma, beta, got, dtype)
        back = mhc.layer_norm_backward(ds, xs, gamma, got[1], got[2], d_x=out)
        assert torch.isnan(torch.cat((bo[:fo], bo[fo + T * H:]))).all()
        _check_backward(dy, x, gamma, got[1], got[2], back, dtype)
        for b, k in zip((bx, bd), keep):
            assert torch.equal(b.nan_to_num(7.0), k.nan_to_num(7.0))
        if gx == 0:  # in place: the bits of an output of the same phase (the phase orders the sums)
            ref = mhc.layer_norm(xs, gamma, beta, y=_rows_at(x, fx, H, nan)[0])[0]
            assert torch.equal(mhc.layer_norm(xs, gamma, beta, y=xs)[0], ref)


@pytest.mark.parametrize("T,H,dtype", [(310, 9001, "bf16"), (300, 14001, "fp16"),
                                       (299, 16383, "bf16"), (305, 8190, "fp32"),
                                       (300, 11000, "fp32"), (298, 8191, "fp32"),
                                       (6000, 17, "bf16"), (5001, 100, "bf16")])
def test_widths_at_the_forms_limits(T, H, dtype):
    x, dy, gamma, beta = _make(T, H, dtype, "fp32", T + H, gap=1)
    got = mhc.layer_norm(x, gamma, beta)
    _check_forward(x, gamma, beta, got, dtype)
    back = mhc.layer_norm_backward(dy, x, gamma, got[1], got[2])
    _check_backward(dy, x, gamma, got[1], got[2], back, dtype)


@pytest.mark.parametrize("H", [1000, 1001])
def test_gradient_where_the_mean_is_far_above_the_deviation(H):
    """fp32: x - mean is formed first."""
    g = torch.Generator().manual_seed(H)
    x = (1000 + torch.randn((300, H), generator=g)).cuda()
    dy = torch.randn((300, H), generator=g).cuda()
    _, mean, rstd = mhc.layer_norm(x)
    _check_backward(dy, x, None, mean, rstd, mhc.layer_norm_backward(dy, x, None, mean, rstd),
                    "fp32")


@pytest.mark.slow
def test_training_batch():
    """The training batch's size; all tokens' sums, sampled rows."""
    T, H = 8192, 7168
    x, dy, gamma, beta = _make(T, H, "bf16", "fp32", 3)
    y, mean, rstd = mhc.layer_norm(x, gamma, beta)
    dx, dg, db = mhc.layer_norm_backward(dy, x, gamma, mean, rstd)
    pick = torch.arange(0, T, 511, device="cuda")
    _check_forward(x[pick], gamma, beta, (y[pick], mean[pick], rstd[pick]), "bf16")
    a = [f64(v) for v in (dy[pick], x[pick], gamma, mean[pick], rstd[pick])]
    rx, _, _ = rows.layer_norm_backward(*a)
    check(dx[pick], rx, rounded(rx, norm_bwd_bounds(*a, "bf16")[0], "bf16"), "d_x")
    tot = [0, 0, 0, 0]
    for i in range(0, T, 1024):  # the token sums, in chunks on the device in fp64
        s = slice(i, i + 1024)
        xh = (x[s].double() - mean[s].double()[:, None]) * rstd[s].double()[:, None]
        d = dy[s].double()
        for j, v in enumerate((d * xh, d, (d * xh).abs(), d.abs())):
            tot[j] = tot[j] + v.sum(0)
    n = -(-T // 64) + 100
    check(dg, f64(tot[0]), (n + 4) * 2.0 ** -24 * f64(tot[2]), "d_gamma")
    check(db, f64(tot[1]), n * 2.0 ** -24 * f64(tot[3]), "d_beta")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 2, 9, 321, 2001])
def test_the_first_and_the_last_row_of_an_array(dtype, T):
    """Rows of one value set give one result wherever they stand: the first and the last row, whose
    ends are fetched element by element, and those between them (of one phase, so of one grouping of
    the sums). Fresh values each time: what an earlier call left in shared memory shows."""
    for i, H in enumerate((1001, 77, 3501, 9003) * 6):
        x1, dy1, gamma, beta = _make(8, H, dtype, "fp32", i)
        at = torch.arange(T, device="cuda") % 8
        nan = float("nan")
        x, bx = _rows_at(x1[at], 3, H, nan)
        dy, bd = _rows_at(dy1[at], 1, H, nan)
        y, mean, rstd = mhc.layer_norm(x, gamma, beta)
        dx = mhc.layer_norm_backward(dy, x, gamma, mean, rstd)[0]
        for a in (y, dx):
            assert torch.equal(a, a[at]), (H, i)
        if i < 4:
            _check_forward(x1[at[-1:]], gamma, beta, (y[-1:], mean[-1:], rstd[-1:]), dtype)


def test_the_default_stream_by_its_handle():
    """Handle 0 is the device's default stream, whichever stream is current: the call comes after
    what stands in that stream."""
    x, dy, gamma, beta = _make(64, 1000, "bf16", "fp32", 3)
    ref = mhc.layer_norm(x, gamma, beta)
    late, out = torch.zeros_like(x), [torch.empty_like(v) for v in ref]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # clocks: some 50 ms
    late.copy_(x)
    with torch.cuda.stream(side):
        mhc.layer_norm(late, gamma, beta, y=out[0], mean=out[1], rstd=out[2], stream=0)
    torch.cuda.synchronize()
    for g, w in zip(out, ref):
        assert torch.equal(g, w)


@pytest.mark.parametrize("dtype,low,high", [("fp16", 2000.0, 2001.0), ("bf16", 1000.0, 1004.0)])
@pytest.mark.parametrize("H", [264, 1000, 1001, 7168, 9000, 9001])
def test_gradient_of_rows_of_two_neighbouring_values(dtype, low, high, H):
    """16-bit rows whose deviation is far below a step of their mean, with d_y along x - mean, so
    that d_x is a small difference: x - mean has to be formed first (the bound of fp32 rows)."""
    T = 300
    g = torch.Generator().manual_seed(H)
    x = torch.where(torch.rand((T, H), generator=g) < 0.01, high, low)
    x[:, 5] = high
    x = x.to(DTYPES[dtype]).cuda()
    _, mean, rstd = mhc.layer_norm(x)
    dy = ((x.float() - mean[:, None]) * rstd[:, None]).to(DTYPES[dtype])
    got = mhc.layer_norm_backward(dy, x, None, mean, rstd)
    a = [f64(dy), f64(x), None, f64(mean), f64(rstd)]
    dx, dg, db = rows.layer_norm_backward(*a)
    ex, eg, eb = norm_bwd_bounds(*a)
    check(got[0], dx, rounded(dx, ex, dtype), "d_x")
    check(got[1], dg, eg, "d_gamma")
    check(got[2], db, eb, "d_beta")


@pytest.mark.parametrize("T,H,dtype,gap", [
    # rows that are not whole windows: the last staged width and the next, backward and forward
    (300, 14057, "bf16", 1), (300, 14058, "fp16", 1), (299, 14065, "fp16", 1),
    (299, 14066, "bf16", 1), (301, 8189, "fp32", 1), (301, 8190, "fp32", 1),
    (300, 9377, "fp32", 1), (300, 9378, "fp32", 1),
    # whole windows: the last width whose gradients are held, staged and neither; many tokens beyond
    (300, 8192, "fp16", 0), (300, 8200, "bf16", 0), (300, 16392, "bf16", 8),
    (300, 8196, "fp32", 0), (300, 11468, "fp32", 0), (300, 11472, "fp32", 4),
    (1500, 12288, "fp32", 0), (900, 16384, "fp32", 0)])
def test_widths_on_either_side_of_the_forms_limits(T, H, dtype, gap):
    x, dy, gamma, beta = _make(T, H, dtype, "fp32", T + H, gap=gap)
    got = mhc.layer_norm(x, gamma, beta)
    _check_forward(x, gamma, beta, got, dtype)
    back = mhc.layer_norm_backward(dy, x, gamma, got[1], got[2])
    _check_backward(dy, x, gamma, got[1], got[2], back, dtype)


@pytest.mark.parametrize("H", [7168, 3501])
def test_rows_written_just_before_on_another_stream(H):
    """Inputs that kernels of the same side stream write just before the call and overwrite just
    after it, forward and backward, twice over in one graph too."""
    x, dy, gamma, beta = _make(700, H, "bf16", "fp32", H)
    y, mean, rstd = mhc.layer_norm(x, gamma, beta)
    ref = [y, mean, rstd, *mhc.layer_norm_backward(dy, x, gamma, mean, rstd)]
    a, d = torch.zeros_like(x), torch.zeros_like(dy)

    def both():
        a.copy_(x)
        f = mhc.layer_norm(a, gamma, beta)
        d.copy_(dy)
        b = mhc.layer_norm_backward(d, a, gamma, f[1], f[2])
        a.zero_()
        d.zero_()
        return [*f, *b]

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = both()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        first, second = both(), both()
    graph.replay()
    torch.cuda.synchronize()
    for g, f, s, w in zip(got, first, second, ref):
        assert torch.equal(g, w) and torch.equal(f, w) and torch.equal(s, w)
