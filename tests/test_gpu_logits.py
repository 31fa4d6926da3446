"""GPU parity of mhc_token_logprobs, mhc_distill_topk and their backward passes against the fp64
oracle; bounds derived in rows_util.py. Top indices have to be equal."""

import numpy as np
import pytest
import torch

import mhc_hyper_connection_02_b200 as mhc
from oracle import rows
from rows_util import DTYPES, E2, LN2, U, check, f64, grad_bounds, logprob_bounds, rounded, \
    row_sum_error
from rows_util import norm_bounds, norm_bwd_bounds

pytestmark = pytest.mark.gpu

# one token to many, odd vocabularies, rows shorter than a block and split over a cluster
SHAPES = [(1, 1), (1, 3), (3, 7), (1, 131072), (2, 100003), (4, 32768), (5, 50021), (17, 4099),
          (300, 1000), (160, 8200), (700, 33)]


def _logits(T, V, dtype, seed, pad=0, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn((T, V + pad), generator=g)).to(DTYPES[dtype]).cuda()[:, :V]


def _targets(T, V, seed):
    g = np.random.default_rng(seed)
    y = g.integers(0, V, T)
    y[::5] = -100 if T > 4 else y[::5]
    return torch.from_numpy(y).cuda()


def _check_forward(z, y, tau, top, got):
    zd = f64(z)
    yn = None if y is None else y.cpu().numpy()
    r = rows.token_logprobs(zd, yn, tau, top)
    e_lp, e_ent, e_s = logprob_bounds(r, zd, tau)
    lp, ent, ti, tl, stats = got
    check(stats[:, 0], r["m"], 0, "m")
    check(stats[:, 1], r["s"], e_s, "s")
    if y is not None:
        check(lp, r["logprob"], np.take_along_axis(e_lp, np.clip(yn, 0, z.shape[1] - 1)[:, None],
                                                   1)[:, 0], "logprob")
    if ent is not None:
        check(ent, r["entropy"], e_ent, "entropy")
    if top:
        np.testing.assert_array_equal(ti.cpu().numpy(), r["top_index"])
        check(tl, r["top_logprob"], np.take_along_axis(e_lp, np.maximum(r["top_index"], 0), 1),
              "top_logprob")
    return r


def _check_backward(z, y, tau, a, b, stats, ent, got, dtype):
    zd = f64(z)
    r = rows.token_logprobs(zd, None, tau)
    T = zd.shape[0]
    an = np.zeros(T) if a is None else f64(a)
    bn = np.zeros(T) if b is None else f64(b)
    ref = rows.token_logprobs_backward(zd, None if y is None else y.cpu().numpy(), tau,
                                       None if a is None else an, None if b is None else bn)
    e_s = row_sum_error(zd, r["m"], tau)[:, None] + U
    e_ent = logprob_bounds(r, zd, tau)[1]
    err = grad_bounds(r["lp"], r["entropy"], tau, an, bn, e_s)
    with np.errstate(invalid="ignore"):
        p = np.where(np.isfinite(r["lp"]), np.exp(r["lp"]), 0.0)
    err = err + p * np.abs(bn)[:, None] * (e_ent[:, None] + 2 * e_s) / tau  # of the entropy given
    if a is not None:
        # The target's own term d_logprob / temperature does not shrink with p: temperature and its
        # reciprocal in fp32, their product with d_logprob and the sum with the dense term are four
        # roundings of U each, relative to it (at p -> 0 the dense term's bound vanishes).
        yn = y.cpu().numpy()
        t = np.nonzero((yn >= 0) & (yn < zd.shape[1]))[0]
        err[t, yn[t]] += 4 * U * np.abs(an[t]) / tau
    check(got, ref, rounded(ref, err, dtype), "d_logits")


@pytest.mark.parametrize("T,V", SHAPES)
@pytest.mark.parametrize("dtype,tau", [("bf16", 1.0), ("fp16", 0.7), ("fp32", 2.0)])
def test_token_logprobs(T, V, dtype, tau):
    z, y = _logits(T, V, dtype, T + V), _targets(T, V, T)
    top = min(V, 20)
    got = mhc.token_logprobs(z, y, temperature=tau, top=top)
    _check_forward(z, y, tau, top, got)
    plain = mhc.token_logprobs(z, y, temperature=tau, entropy=False)
    assert torch.equal(plain[0], got[0]) and torch.equal(plain[4], got[4])
    assert plain[1] is None and plain[2] is None and plain[3] is None
    a, b = torch.randn(T, device="cuda"), torch.randn(T, device="cuda")
    d = mhc.token_logprobs_backward(z, y, got[4], a, d_entropy=b, entropy=got[1], temperature=tau)
    _check_backward(z, y, tau, a, b, got[4], got[1], d, dtype)
    d = mhc.token_logprobs_backward(z, y, got[4], a, temperature=tau)
    _check_backward(z, y, tau, a, None, got[4], None, d, dtype)
    d = mhc.token_logprobs_backward(z, None, got[4], None, d_entropy=b, entropy=got[1],
                                    temperature=tau)
    _check_backward(z, None, tau, None, b, got[4], got[1], d, dtype)


@pytest.mark.parametrize("top", [1, 2, 7, 31, 32])
@pytest.mark.parametrize("T,V", [(1, 32), (3, 40), (2, 9001), (400, 5000), (1, 70000)])
def test_top_alternatives(top, T, V):
    z = _logits(T, V, "bf16", top * T + V)
    _check_forward(z, None, 1.0, top, mhc.token_logprobs(z, None, top=top))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("apart", [8, 256 * 8, 1024 * 4, 1024 * 8, 3 * 1024 * 8])
def test_best_ones_at_one_distance(dtype, apart):
    """The best elements lie `apart` elements from one another: in one window, one round or several
    rounds of the same thread, equal ones among them."""
    V = 70001
    z = _logits(6, V, dtype, apart)
    at = torch.arange(0, V, apart, device="cuda")[:40]
    for t in range(6):
        z[t, at + t] = (20 + torch.arange(at.numel(), device="cuda") % (3 + 7 * t)).to(z.dtype)
    for top in (1, 9, 32):
        _check_forward(z, None, 1.0, top, mhc.token_logprobs(z, None, top=top))


def test_a_gradient_is_laid_out_as_padded_logits_are():
    for V, stride, want in ((1000, 1024, 1024), (1001, 1008, 1008), (1000, 1000, 1000),
                            (1000, 2000, 1000)):
        z = torch.randn((5, stride), device="cuda").to(torch.bfloat16)[:, :V]
        y, a = _targets(5, V, 1), torch.randn(5, device="cuda")
        st = mhc.token_logprobs(z, y, entropy=False)[4]
        d = mhc.token_logprobs_backward(z, y, st, a)
        assert d.shape == (5, V) and d.stride() == (want, 1)
        out = torch.empty((5, V), dtype=z.dtype, device="cuda")
        mhc.token_logprobs_backward(z, y, st, a, d_logits=out)
        assert torch.equal(out, d)
        idx, t = _teacher(5, V, 4, "fp32", 1, ragged=False, twice=False)
        loss, w, st = mhc.distill_topk(z, idx, t)
        assert mhc.distill_topk_backward(z, idx, w, st, a).stride() == (want, 1)


def _special_rows(V, dtype):
    """Rows that no-order-in-particular does not cover, for the top alternatives and the sums."""
    lowest = torch.finfo(DTYPES[dtype]).min
    z = torch.randn((19, V), generator=torch.Generator().manual_seed(V)) * 2
    z[1] = 0.0                                   # one value
    z[2] = torch.arange(V) / V                   # rising: 16-bit types give long runs of one value
    z[3] = -torch.arange(V) / V                  # falling
    z[4] = -float("inf")                         # nothing left
    z[5] = -float("inf")
    z[5, [V - 1, V // 2, V // 3]] = torch.tensor([1.0, 2.0, 3.0])  # fewer left than asked for
    z[6] = lowest
    z[7] = lowest
    z[7, V // 2] = 1.5
    z[8, V // 4:] = 0.0                          # a run of one value with others above and below
    z[9] = z[9] * 0 - 5.0
    z[9, V - 100:] = 7.0                         # the ties at the row's end
    z[10] = torch.where(torch.arange(V) % 2048 < 8, 10 + torch.rand(V), torch.tensor(0.0))
    z[11] = (torch.arange(V) % 97).float()       # many equal maxima
    z[12, 5] = float("nan")
    z[13, V - 1] = float("inf")
    z[14] = torch.where(torch.rand(V) < 0.5, 0.0, -0.0)  # signed zeros are one value
    z[15] = 1e4 * torch.randn(V)                 # far apart
    z[16] = -float("inf")
    z[16, 0] = float("nan")
    z[17] = torch.randn(V) * 1e-3 - 6e4
    z[18] = torch.where(torch.arange(V) % 3 == 0, -lowest / 2, -lowest / 2.5)
    return z.to(DTYPES[dtype]).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("V", [600, 8192, 40001])
@pytest.mark.parametrize("many", [False, True])
def test_masked_tied_and_ordered_rows(dtype, V, many):
    """Both forms: a cluster per row (few rows), and one CTA per row (the rows repeated)."""
    z = _special_rows(V, dtype)
    if dtype == "fp16":
        z[15] = (z[15].float() / 4).half()  # inside fp16's range: no infinities made
        z[15].clamp_(-6e4, 6e4)
    n = z.shape[0]
    y = torch.full((n,), V // 2, dtype=torch.int64, device="cuda")
    y[11] = V + 3   # no such token
    y[12] = -1
    reps = 20 if many else 1
    zz, yy = z.repeat(reps, 1), y.repeat(reps)
    got = mhc.token_logprobs(zz, yy, top=20)
    for k in {0, reps - 1}:
        s = slice(k * n, (k + 1) * n)
        _check_forward(z, y, 1.0, 20, [v[s] for v in got])
    a = torch.randn(n, device="cuda")
    b = torch.randn(n, device="cuda")
    a[0], b[0] = 0.0, 0.0
    a[1] = 0.0
    d = mhc.token_logprobs_backward(zz, yy, got[4], a.repeat(reps), d_entropy=b.repeat(reps),
                                    entropy=got[1])
    _check_backward(z, y, 1.0, a, b, got[4][:n], got[1][:n], d[(reps - 1) * n:], dtype)


def test_zero_upstream_gradients_clear_whatever_stood_there():
    z = _logits(6, 5003, "bf16", 1)
    z[2] = float("nan")
    st = mhc.token_logprobs(z, None, entropy=False)[4]
    y = torch.tensor([1, -1, -1, 2, 3, -100], device="cuda")
    a = torch.tensor([0.0, 1.0, 5.0, 0.0, 1.0, 1.0], device="cuda")
    d = mhc.token_logprobs_backward(z, y, st, a, d_logits=z)
    assert d.data_ptr() == z.data_ptr()
    zero = [0, 1, 2, 3, 5]
    assert torch.equal(d[zero], torch.zeros_like(d[zero])) and d[4].any()


@pytest.mark.parametrize("pad,V", [(27, 50021), (1, 999), (3, 8192), (64, 1024)])
def test_padded_rows_and_in_place(pad, V):
    for dtype in ("bf16", "fp32"):
        z, y = _logits(9, V, dtype, V, pad=pad), _targets(9, V, 3)
        got = mhc.token_logprobs(z, y, top=5)
        _check_forward(z, y, 1.0, 5, got)
        a, b = torch.randn(9, device="cuda"), torch.randn(9, device="cuda")
        kw = dict(d_entropy=b, entropy=got[1])
        ref = mhc.token_logprobs_backward(z, y, got[4], a, **kw)
        _check_backward(z, y, 1.0, a, b, got[4], got[1], ref, dtype)
        wide = torch.full((9, V + pad + 2), 7.0, dtype=z.dtype, device="cuda")
        out = mhc.token_logprobs_backward(z, y, got[4], a, d_logits=wide[:, 1:V + 1], **kw)
        assert torch.equal(out, ref) and (wide[:, 0] == 7).all() and (wide[:, V + 1:] == 7).all()
        whole = torch.zeros((9, V + pad), dtype=z.dtype, device="cuda")
        zz = whole[:, :V]
        zz.copy_(z)
        whole[:, V:] = 7
        assert torch.equal(mhc.token_logprobs_backward(zz, y, got[4], a, d_logits=zz, **kw), ref)
        assert (whole[:, V:] == 7).all()


@pytest.mark.parametrize("tau", [1e-3, 50.0, 1e30])
def test_temperatures_far_from_one(tau):
    z, y = _logits(5, 3001, "fp32", 4), _targets(5, 3001, 1)
    got = mhc.token_logprobs(z, y, temperature=tau, top=3)
    _check_forward(z, y, tau, 3, got)
    a = torch.randn(5, device="cuda")
    d = mhc.token_logprobs_backward(z, y, got[4], a, temperature=tau)
    _check_backward(z, y, tau, a, None, got[4], None, d, "fp32")


def _teacher(T, V, K, dtype, seed, ragged=True, twice=True):
    g = np.random.default_rng(seed)
    idx = np.stack([g.permutation(V)[:K] if K <= V else g.integers(0, V, K) for _ in range(T)])
    if ragged:
        for t in range(0, T, 2):
            idx[t, g.integers(1, K + 1):] = -1
    if twice and K > 3:
        idx[0] = idx[0, 0]              # one token K times
        idx[T - 1, 3] = idx[T - 1, 0]
        idx[T // 2, K - 1] = idx[T // 2, K // 2]
    t = torch.from_numpy(3 * g.standard_normal((T, K))).to(DTYPES[dtype]).cuda()
    return torch.from_numpy(idx).cuda(), t


def _check_distill(z, idx, t, tau, got, dtype):
    zd, td, i = f64(z), f64(t), idx.cpu().numpy()
    K = i.shape[1]
    loss, w = rows.distill_topk(zd, i, td, tau)
    r = rows.token_logprobs(zd, None, tau)
    e_lp, _, e_s = logprob_bounds(r, zd, tau)
    # weights: a softmax over at most 4 entries a thread and 16 joins
    used = np.where(i >= 0, td, -np.inf)
    top = used.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        td_d = np.where(w > 0, np.abs(used - top) / tau / LN2, 0)
    e_w = 2 * E2 + 30 * U + 2 * LN2 * U * (2 * td_d + 2 * td_d.max(1, keepdims=True))
    check(got[1], w, w * e_w + 1e-44, "weights")
    with np.errstate(invalid="ignore", divide="ignore"):
        lw = np.where(w > 0, np.log(w), 0.0)
        lpk = np.take_along_axis(r["lp"], np.clip(i, 0, zd.shape[1] - 1), 1)
        size = np.abs(lw) + np.where(w > 0, np.abs(lpk), 0)
        e_l = w * (e_w * (size + 1) + np.take_along_axis(e_lp, np.clip(i, 0, zd.shape[1] - 1), 1)
                   + 8 * U * (size + np.log(K) + 1))
        e_l = e_l.sum(1) + 24 * U * (w * size).sum(1)
    check(got[0], loss, e_l, "loss")
    check(got[2][:, 1], r["s"], e_s, "s")
    return w


def _check_distill_backward(z, idx, w, tau, g, got, dtype):
    zd, i = f64(z), idx.cpu().numpy()
    ref = rows.distill_topk_backward(zd, i, f64(w), f64(g), tau)
    r = rows.token_logprobs(zd, None, tau)
    gn = f64(g)
    err = grad_bounds(r["lp"], r["entropy"], tau, gn, 0 * gn,
                      row_sum_error(zd, r["m"], tau)[:, None] + U)
    q = np.zeros_like(zd)
    for t in range(i.shape[0]):
        used = (i[t] >= 0) & (i[t] < zd.shape[1])
        np.add.at(q[t], i[t][used], np.abs(f64(w)[t][used]))
    # a token's weights: at most K additions, then four roundings as at a target above
    err = err + (i.shape[1] + 4) * U * q * np.abs(gn)[:, None] / tau
    check(got, ref, rounded(ref, err, dtype), "d_logits")


@pytest.mark.parametrize("T,V,K", [(1, 1, 1), (1, 131072, 64), (3, 7, 5), (4, 50021, 17),
                                   (300, 1000, 33), (9, 32003, 300), (2, 3000, 1024), (5, 600, 1000),
                                   (1, 9001, 1)])
@pytest.mark.parametrize("dtype,teacher,tau", [("bf16", "bf16", 2.0), ("fp16", "fp32", 1.0),
                                               ("fp32", "fp16", 0.5)])
def test_distill(T, V, K, dtype, teacher, tau):
    z = _logits(T, V, dtype, T + V + K)
    idx, t = _teacher(T, V, K, teacher, K)
    got = mhc.distill_topk(z, idx, t, temperature=tau)
    _check_distill(z, idx, t, tau, got, dtype)
    g = torch.randn(T, device="cuda")
    d = mhc.distill_topk_backward(z, idx, got[1], got[2], g, temperature=tau)
    _check_distill_backward(z, idx, got[1], tau, g, d, dtype)
    zz = z.clone()
    same = mhc.distill_topk_backward(zz, idx, got[1], got[2], g, temperature=tau, d_logits=zz)
    assert torch.equal(same, d)


@pytest.mark.parametrize("V", [700, 40001])
def test_distill_rows_without_a_teacher_and_masked_ones(V):
    inf = float("inf")
    z = _logits(9, V, "bf16", V)
    idx, t = _teacher(9, V, 6, "fp32", 5, ragged=False, twice=False)
    idx[0] = -1                      # no entry
    t[1] = -inf                      # nothing kept
    t[2, :5] = -inf                  # one kept
    z[3] = -inf                      # no student distribution
    z[4, idx[4, 2]] = -inf           # the student rules out a teacher's token: infinite loss
    t[5] = torch.finfo(torch.float32).min
    z[6, 1] = float("nan")
    idx[7, 3] = V                    # no such token
    t[8, 0] = float("nan")
    got = mhc.distill_topk(z, idx, t)
    _check_distill(z, idx, t, 1.0, got, "bf16")
    assert got[0][0] == 0 and got[0][1] == 0 and got[0][4] == inf and torch.isnan(got[0][6:]).all()
    g = torch.ones(9, device="cuda")
    d = mhc.distill_topk_backward(z, idx, got[1], got[2], g)
    _check_distill_backward(z, idx, got[1], 1.0, g, d, "bf16")
    assert not d[0].any() and not d[1].any() and torch.isnan(d[6:]).all()


def test_no_tokens():
    e = torch.empty((0, 50), dtype=torch.bfloat16, device="cuda")
    y = torch.empty(0, dtype=torch.int64, device="cuda")
    lp, ent, ti, tl, st = mhc.token_logprobs(e, y, top=3)
    assert lp.shape == (0,) and ent.shape == (0,) and ti.shape == (0, 3) and st.shape == (0, 2)
    assert mhc.token_logprobs_backward(e, y, st, lp).shape == (0, 50)
    idx = torch.empty((0, 4), dtype=torch.int64, device="cuda")
    loss, w, st = mhc.distill_topk(e, idx, torch.empty((0, 4), device="cuda"))
    assert loss.shape == (0,) and mhc.distill_topk_backward(e, idx, w, st, loss).shape == (0, 50)


def test_binding_refusals():
    z = _logits(4, 64, "bf16", 1)
    y = _targets(4, 64, 1)
    st = torch.zeros((4, 2), device="cuda")
    with pytest.raises(ValueError, match="top"):
        mhc.token_logprobs(z, y, top=33)
    with pytest.raises(ValueError, match="int64"):
        mhc.token_logprobs(z, y.int())
    with pytest.raises(ValueError, match="rows must not"):
        mhc.token_logprobs(z[0:1].expand(4, 64))
    with pytest.raises(ValueError, match="contiguous"):
        mhc.token_logprobs(z.t())
    with pytest.raises(ValueError, match="d_logits"):
        mhc.token_logprobs_backward(z, y, st, st[:, 0].contiguous(), d_logits=z.float())
    for kw, status in ((dict(temperature=0.0), mhc.MHC_ERR_INVALID_ARG),):
        with pytest.raises(mhc.MhcError) as e:
            mhc.token_logprobs(z, y, **kw)
        assert e.value.status == status
    with pytest.raises(mhc.MhcError) as e:
        mhc.token_logprobs_backward(z, y, st)
    assert e.value.status == mhc.MHC_ERR_INVALID_ARG
    flat = torch.zeros(4 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(mhc.MhcError) as e:
        mhc.token_logprobs_backward(flat[:256].view(4, 64), y, st, st[:, 0].contiguous(),
                                    d_logits=flat[8:264].view(4, 64))
    assert e.value.status == mhc.MHC_ERR_ALIAS
    with pytest.raises(ValueError, match="K"):
        mhc.distill_topk(z, torch.zeros((4, 1025), dtype=torch.int64, device="cuda"),
                         torch.zeros((4, 1025), device="cuda"))


def test_same_bits_in_graphs_and_on_another_stream():
    T, V, K = 6, 50021, 40
    z, y = _logits(T, V, "bf16", 8), _targets(T, V, 2)
    idx, t = _teacher(T, V, K, "fp32", 1)
    a = torch.randn(T, device="cuda")

    def all_of(**kw):
        lp, ent, ti, tl, st = mhc.token_logprobs(z, y, top=9, **kw)
        d = mhc.token_logprobs_backward(z, y, st, a, d_entropy=a, entropy=ent, **kw)
        loss, w, st2 = mhc.distill_topk(z, idx, t, **kw)
        return [lp, ent, ti, tl, st, d, loss, w, st2,
                mhc.distill_topk_backward(z, idx, w, st2, a, **kw)]

    ref = all_of()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_of()
    for _ in range(2):
        for v in got:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for v, w in zip(got, ref):
            assert torch.equal(v, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = all_of(stream=side)
    got2 = all_of(stream=side.cuda_stream)
    side.synchronize()
    for v, v2, w in zip(got, got2, ref):
        assert torch.equal(v, w) and torch.equal(v2, w)


@pytest.mark.parametrize("dtype,V", [("bf16", 66001), ("fp32", 33001)])
def test_rows_left_over_after_full_rounds(dtype, V):
    """As many rows as two launches share, between kernels that write the logits just before and
    clear them just after."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    K = 12
    for T in (sms * 5 + 9, sms * 6 + 9):
        src, y = _logits(T, V, dtype, T), _targets(T, V, 2)
        idx, t = _teacher(T, V, K, "fp32", 1)
        z = torch.zeros_like(src)
        pick = torch.tensor([0, 1, T // 2, *range(T - 12, T)], device="cuda")
        zs, ys = src[pick], y[pick]
        for top in (0, 6):
            z.copy_(src)
            got = mhc.token_logprobs(z, y, top=top)
            z.zero_()
            _check_forward(zs, ys, 1.0, top, [v if v is None else v[pick] for v in got])
        z.copy_(src)
        got = mhc.distill_topk(z, idx, t)
        z.zero_()
        _check_distill(zs, idx[pick], t[pick], 1.0, [v[pick] for v in got], dtype)
        a = torch.randn(T, device="cuda")
        z.copy_(src)
        st = mhc.token_logprobs(z, y, entropy=False)[4]
        d = mhc.token_logprobs_backward(z, y, st, a, d_logits=z)
        _check_backward(zs, ys, 1.0, a[pick], None, st[pick], None, d[pick], dtype)


def test_offsets_past_32_bits():
    """Rows whose byte and element offsets pass 2^31 and 2^32 (the last rows are checked)."""
    T, V = 3, 5000
    stride = (1 << 31) + 3
    free = torch.cuda.mem_get_info()[0]
    if free < 2 * (2 * stride * 2 + (1 << 20)):
        pytest.skip("not enough device memory")
    store = torch.zeros(2 * stride + V, dtype=torch.bfloat16, device="cuda")
    z = torch.as_strided(store, (T, V), (stride, 1))
    z.copy_(_logits(T, V, "bf16", 3))
    y = _targets(T, V, 1)
    got = mhc.token_logprobs(z, y, top=4)
    _check_forward(z, y, 1.0, 4, got)
    a = torch.randn(T, device="cuda")
    dense = mhc.token_logprobs_backward(z, y, got[4], a)
    assert torch.equal(mhc.token_logprobs_backward(z, y, got[4], a, d_logits=z), dense)


def test_gradients_against_differences():
    """fp32 logits, directional central differences (rounding U / h of the loss's size)."""
    z, y = _logits(4, 301, "fp32", 2, scale=1.0), _targets(4, 301, 4)
    idx, t = _teacher(4, 301, 8, "fp32", 3)
    v, a, b = torch.randn_like(z), torch.randn(4, device="cuda"), torch.randn(4, device="cuda")
    h = 2.0 ** -7
    lp, ent, _, _, st = mhc.token_logprobs(z, y)
    d = mhc.token_logprobs_backward(z, y, st, a, d_entropy=b, entropy=ent)

    def f(x):
        r = mhc.token_logprobs(x, y)
        return (r[0].double() * a + r[1].double() * b).sum().item()

    assert abs((f(z + h * v) - f(z - h * v)) / (2 * h) - (d.double() * v).sum().item()) < 5e-3
    _, w, st = mhc.distill_topk(z, idx, t)
    d = mhc.distill_topk_backward(z, idx, w, st, a)
    k = lambda x: (mhc.distill_topk(x, idx, t)[0].double() * a).sum().item()
    assert abs((k(z + h * v) - k(z - h * v)) / (2 * h) - (d.double() * v).sum().item()) < 5e-3


def test_the_answer_end_of_a_stack():
    """head -> norm -> logits -> log probabilities and distillation, and back to the head's row: the
    operators together, as a training step uses them, against the oracle's chain. The product with
    the vocabulary is the user's (torch, fp32)."""
    T, H, V, K = 24, 512, 4001, 12
    g = torch.Generator().manual_seed(0)
    R = torch.randn((T, 4, H), generator=g).to(torch.bfloat16).cuda()
    gamma = (1 + 0.1 * torch.randn(H, generator=g)).cuda()
    beta = (0.1 * torch.randn(H, generator=g)).cuda()
    W = (torch.randn((H, V), generator=g) / H ** 0.5).cuda()
    y = _targets(T, V, 6)
    idx, t = _teacher(T, V, K, "fp32", 2)
    x = mhc.head_mean(R).float()
    n, mean, rstd = mhc.layer_norm(x, gamma, beta)
    z = n @ W
    lp, ent, _, _, st = mhc.token_logprobs(z, y)
    loss, w, st2 = mhc.distill_topk(z, idx, t, temperature=2.0)
    a = torch.full((T,), -1.0 / T, device="cuda")
    dz = mhc.token_logprobs_backward(z, y, st, a, d_entropy=0.01 * a, entropy=ent)
    dz += mhc.distill_topk_backward(z, idx, w, st2, -a, temperature=2.0)
    dx, dg, db = mhc.layer_norm_backward(dz @ W.t(), x, gamma, mean, rstd)

    xo, Wo = f64(x), f64(W)
    no, mo, ro = rows.layer_norm(xo, f64(gamma), f64(beta))
    zo = no @ Wo
    an = f64(a)
    dzo = rows.token_logprobs_backward(zo, y.cpu().numpy(), 1.0, an, 0.01 * an)
    wo = rows.distill_topk(zo, idx.cpu().numpy(), f64(t), 2.0)[1]
    dzo = dzo + rows.distill_topk_backward(zo, idx.cpu().numpy(), wo, -an, 2.0)
    dxo, dgo, dbo = rows.layer_norm_backward(dzo @ Wo.T, xo, f64(gamma), mo, ro)
    r = rows.token_logprobs(zo, y.cpu().numpy(), 1.0)
    # The product's fp32 sums over H terms (H U of the sizes' sum) move z by ez, and the log
    # probability by at most 2 ez; the gradients move by their sizes times that.
    ez = (H + 64) * U * (np.abs(no) @ np.abs(Wo)).max()
    check(lp, r["logprob"], 2 * ez + 1e-5, "logprob")
    check(ent, r["entropy"], 2 * ez * np.log(V) + 1e-5, "entropy")
    back = (np.abs(dzo) @ np.abs(Wo).T)
    lim = (8 * ez + (V + 64) * U) * back.max() * np.abs(ro).max() * 4
    check(dx, dxo, lim, "d_x")
    check(dg, dgo, T * lim * 8, "d_gamma")
    check(db, dbo, T * lim * 8, "d_beta")


@pytest.mark.parametrize("dtype,tau,size", [("bf16", 1e-3, 1e6), ("bf16", 1e-4, 1e4),
                                            ("bf16", 1.0, 1e12), ("bf16", 1e-2, 1e35),
                                            ("fp32", 1e-2, 1e35), ("fp16", 1e-3, 1e-3)])
def test_entropy_gradient_of_masked_logits_under_a_large_scale(dtype, tau, size):
    """A masked logit's gradient is zero, however large d_entropy / temperature is. The others lie
    within 40 temperatures of the best, so that no probability is below the smallest normal
    number."""
    T, V = 6, 5003
    g = torch.Generator().manual_seed(T)
    z = (tau * 40 * torch.rand((T, V), generator=g)).to(DTYPES[dtype])
    z[:, ::3] = -float("inf")
    z[1, ::2] = torch.finfo(DTYPES[dtype]).min
    z[2, 1:] = -float("inf")
    z[2, 0] = tau
    z[3] = -float("inf")
    z[4, 7] = -float("inf")
    z, y = z.cuda(), _targets(T, V, 1)
    y[4] = 7                                        # the target itself is ruled out
    _, ent, _, _, st = mhc.token_logprobs(z, y, temperature=tau)
    a, b = size * torch.randn(T, device="cuda"), size * torch.randn(T, device="cuda")
    for glp in (None, a):
        d = mhc.token_logprobs_backward(z, y, st, glp, d_entropy=b, entropy=ent, temperature=tau)
        _check_backward(z, y, tau, glp, b, st, ent, d, dtype)
        assert not d[3].any() and not d[0, 3::3][: V // 8].isnan().any()


@pytest.mark.parametrize("tau", [1.0, 1e-3, 1e-6])
@pytest.mark.parametrize("V,reps", [(9000, 30), (140001, 1)])
def test_maxima_on_either_side_of_the_forms_border(tau, V, reps):
    """The exponents' form changes where |max z| log2(e) / temperature passes 2^22. A thread's
    maximum passes it from round to round of its windows (4096 elements), from below, from above
    (negative logits) and not at all; the logits lie within 20 temperatures of one another."""
    border = 2.0 ** 22 * LN2 * tau
    steps = [(-9, -2, 4), (-3, 5, 6), (-12, -11, 1), (1, 3, 7), (-8, -6, -4), (6, -5, 9)]
    g = torch.Generator().manual_seed(V)
    at = torch.arange(V) // 4096 % 3
    z = torch.stack([s * border + tau * (torch.tensor(p, dtype=torch.float64)[at]
                                         + 2 * torch.rand(V, generator=g, dtype=torch.float64))
                     for s in (1, -1) for p in steps]).float().cuda()
    T = z.shape[0]
    y = _targets(T, V, 1)
    zz, yy = z.repeat(reps, 1), y.repeat(reps)
    got = [None if v is None else v[-T:] for v in
           mhc.token_logprobs(zz, yy, temperature=tau, top=4)]
    _check_forward(z, y, tau, 4, got)
    plain = mhc.token_logprobs(zz, yy, temperature=tau, entropy=False)
    _check_forward(z, y, tau, 0, [plain[0][-T:], None, None, None, plain[4][-T:]])
    a, b = torch.randn(T, device="cuda"), torch.randn(T, device="cuda")
    d = mhc.token_logprobs_backward(z, y, got[4], a, d_entropy=b, entropy=got[1], temperature=tau)
    _check_backward(z, y, tau, a, b, got[4], got[1], d, "fp32")
    idx, t = _teacher(T, V, 5, "fp32", 2)
    k = mhc.distill_topk(z, idx, tau * t, temperature=tau)
    _check_distill(z, idx, tau * t, tau, k, "fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("V", [77, 3001, 40003])
def test_gradients_written_into_rows_of_another_phase(dtype, V):
    """Logits and gradient begin at addresses and lie at distances of their own; what stands beside
    the gradient's rows stays."""
    T, K = 7, 6
    z, y = _logits(T, V, dtype, V), _targets(T, V, 2)
    idx, t = _teacher(T, V, K, "fp32", 1, ragged=False)
    a, b = torch.randn(T, device="cuda"), torch.randn(T, device="cuda")
    _, ent, _, _, st = mhc.token_logprobs(z, y)
    _, w, _ = mhc.distill_topk(z, idx, t)
    for first, gap, out_first, out_gap in ((0, 0, 1, 0), (1, 0, 0, 0), (3, 2, 2, 5), (0, 1, 7, 8),
                                           (5, V, 5, V)):
        src = torch.zeros(first + T * (V + gap), dtype=z.dtype, device="cuda")
        zz = torch.as_strided(src, (T, V), (V + gap, 1), first)
        zz.copy_(z)
        buf = torch.full((out_first + T * (V + out_gap) + 3,), 7.0, dtype=z.dtype, device="cuda")
        out = torch.as_strided(buf, (T, V), (V + out_gap, 1), out_first)
        inside = torch.zeros_like(buf, dtype=torch.bool)
        torch.as_strided(inside, (T, V), (V + out_gap, 1), out_first).fill_(True)
        mhc.token_logprobs_backward(zz, y, st, a, d_entropy=b, entropy=ent, d_logits=out)
        _check_backward(z, y, 1.0, a, b, st, ent, out, dtype)
        mhc.distill_topk_backward(zz, idx, w, st, a, d_logits=out)
        _check_distill_backward(z, idx, w, 1.0, a, out, dtype)
        assert (buf[~inside] == 7).all()


def test_the_answer_end_of_a_stack_with_its_weights_gradients():
    """The chain above with every error carried through element by element, so that the bounds of
    d_x, d_gamma and d_beta lie far below their values: a lost or a wrong part of them shows."""
    T, H, V, K = 24, 512, 4001, 12
    g = torch.Generator().manual_seed(1)
    R = torch.randn((T, 4, H), generator=g).to(torch.bfloat16).cuda()
    gamma = (1 + 0.1 * torch.randn(H, generator=g)).cuda()
    beta = (0.1 * torch.randn(H, generator=g)).cuda()
    W = (torch.randn((H, V), generator=g) / H ** 0.5).cuda()
    y = _targets(T, V, 6)
    idx, t = _teacher(T, V, K, "fp32", 2)
    x = mhc.head_mean(R).float()
    n, mean, rstd = mhc.layer_norm(x, gamma, beta)
    z = n @ W
    lp, ent, _, _, st = mhc.token_logprobs(z, y)
    loss, w, st2 = mhc.distill_topk(z, idx, t, temperature=2.0)
    a = torch.full((T,), -1.0 / T, device="cuda")
    dz = mhc.token_logprobs_backward(z, y, st, a, d_entropy=0.01 * a, entropy=ent)
    dz += mhc.distill_topk_backward(z, idx, w, st2, -a, temperature=2.0)
    got = mhc.layer_norm_backward(dz @ W.t(), x, gamma, mean, rstd)
    ref, tol = _answer_end(f64(x), f64(gamma), f64(beta), f64(W), y.cpu().numpy(),
                           idx.cpu().numpy(), f64(t), f64(a))
    for v, r, e, what in zip(got, ref, tol, ("d_x", "d_gamma", "d_beta")):
        assert np.max(e) < np.max(np.abs(r)) / 50, what
        check(v, r, e, what)


def _answer_end(x, gamma, beta, W, y, idx, t, a):
    """(d_x, d_gamma, d_beta) of the chain in fp64, and bounds of their errors in fp32. To first
    order: an error ez of each logit moves ln p and the entropy's term by at most twice its largest,
    and p by that times p."""
    H, V = W.shape
    n, mean, rstd = rows.layer_norm(x, gamma, beta)
    ey, em, er = norm_bounds(x, gamma, beta, n, mean, rstd, 1e-6)
    z = n @ W
    # the product: sums of H terms, and the error of what it takes (rounded once)
    ez = (H + 8) * U * (np.abs(n) @ np.abs(W)) + rounded(n, ey, "fp32") @ np.abs(W)
    shift = 2 * ez.max(1)
    r, r2 = rows.token_logprobs(z, y, 1.0), rows.token_logprobs(z, None, 2.0)
    h = 0.01 * a
    dz = rows.token_logprobs_backward(z, y, 1.0, a, h)
    w = rows.distill_topk(z, idx, t, 2.0)[1]
    dz2 = rows.distill_topk_backward(z, idx, w, -a, 2.0)
    p, p2 = np.exp(r["lp"]), np.exp(r2["lp"])
    size = np.abs(r["lp"]) + r["entropy"][:, None]
    ab = np.abs(a)[:, None]
    s = shift[:, None]
    e_ent = logprob_bounds(r, z, 1.0)[1][:, None]
    ed = (grad_bounds(r["lp"], r["entropy"], 1.0, a, h,
                      row_sum_error(z, r["m"], 1.0)[:, None] + U)
          + ab * p * s + np.abs(h)[:, None] * p * (s * (size + 2) + e_ent)
          + grad_bounds(r2["lp"], r2["entropy"], 2.0, a, 0 * a,
                        row_sum_error(z, r2["m"], 2.0)[:, None] + U) + ab / 2 * p2 * s / 2)
    # the target's and the entries' own terms: weights within 64 U, sums of at most K + 8 terms
    own = np.zeros_like(z)
    rows_ = np.arange(len(a))
    own[rows_[y >= 0], y[y >= 0]] = 8 * U
    for k in range(idx.shape[1]):
        used = idx[:, k] >= 0
        np.add.at(own, (rows_[used], idx[used, k]), (64 + 2 * idx.shape[1]) * U * w[used, k])
    ed = ed + ab * own + 2 * U * (np.abs(dz) + np.abs(dz2))
    dz = dz + dz2
    dn = dz @ W.T
    edn = ed @ np.abs(W).T + (V + 8) * U * (np.abs(dz) @ np.abs(W).T)
    ref = rows.layer_norm_backward(dn, x, gamma, mean, rstd)
    ex, eg, eb = norm_bwd_bounds(dn, x, gamma, mean, rstd)
    # what the backward pass is given: d_y within edn, mean within em, rstd within er
    rs, er = rstd[:, None], er[:, None]
    xh = np.abs(x - mean[:, None]) * rs
    exh = rs * em[:, None] + xh * er / rs
    q, eq = np.abs(dn * gamma), edn * np.abs(gamma)
    c1, c2 = q.mean(1, keepdims=True), (q * xh).mean(1, keepdims=True)
    ec2 = (eq * xh + q * exh).mean(1, keepdims=True)
    ex = ex + rs * (eq + eq.mean(1, keepdims=True) + exh * c2 + xh * ec2) + er * (q + c1 + xh * c2)
    eg = eg + (edn * xh + np.abs(dn) * exh).sum(0)
    eb = eb + edn.sum(0)
    # second-order terms, and fp32's rounding of d_x
    return ref, (1.01 * ex + 2 * U * np.abs(ref[0]), 1.01 * eg, 1.01 * eb)


def test_rows_left_over_after_full_rounds_in_a_graph():
    """The two launches of such a call captured between writers of their logits, twice over, and
    replayed with other logits."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T, V = sms * 6 + 9, 66001
    src, y = _logits(T, V, "bf16", 1), _targets(T, V, 2)
    other = torch.randn((T, V), device="cuda").to(torch.bfloat16)
    ref = [mhc.token_logprobs(v, y) for v in (src, other)]
    z = torch.zeros_like(src)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = []
        for _ in range(2):
            z.copy_(src)
            got.append(mhc.token_logprobs(z, y))
            z.zero_()
    for want in ref:
        graph.replay()
        torch.cuda.synchronize()
        for one in got:
            for k in (0, 1, 4):
                assert torch.equal(one[k], want[k])
        src.copy_(other)
