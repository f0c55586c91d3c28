"""Layer norm and RMS norm against the float64 oracle.

Bounds, u = half a step of the output type (relative), v = 2^-24 (fp32):
a row's mean and mean square are sums whose longest chain is at most 32 adds in
a thread and ten in the two shuffle trees, so they are off by at most 42 v times
the sum of magnitudes; xh follows with twice that through the mean and through
the square root of the variance, and a few roundings of its own.  K = 128 covers
them: |dy_out| <= u |y| + K v (|w| (|xh| + mean|xh| + |mu| r) + |b|).
The backward sums have the same chains; dw and db add their terms in at most
T / parts + parts / 16 + 20 steps.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import operators_oracle as oo  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
V = 2.0 ** -24
K = 128


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _case(T, d, dt, wt, seed=0, mean=0.5):
    g = torch.Generator().manual_seed(1000 * T + d + seed)
    x = (torch.randn(T, d, generator=g) * torch.exp(0.5 * torch.randn(T, 1, generator=g)) + mean).to(TYPES[dt])
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(TYPES[wt])
    b = (0.2 * torch.randn(d, generator=g)).to(TYPES[wt])
    dy = torch.randn(T, d, generator=g).to(TYPES[dt])
    return x, w, b, dy


def _n(t):
    return t.detach().double().cpu().numpy()


def _check(got, ref, lim, what):
    got = _n(got)
    assert got.shape == ref.shape
    err = np.abs(got - ref)
    assert (err <= lim).all(), f"{what}: {float((err / lim).max()):.3f} of the bound"


def _smallest(dt):
    # the spacing below which fp16 rounds absolutely
    return 2.0 ** -25 if dt == "fp16" else 1e-37


SHAPES = [(1, 1), (3, 2), (2, 31), (5, 32), (9, 100), (130, 256), (17, 257), (40, 512), (33, 513), (300, 1001),
          (8, 1024), (1000, 768), (7, 4096), (1, 8192), (70, 8192), (3, 8200), (5, 12001), (2, 16384), (3, 20000),
          (2, 32768),
          # rows that start anywhere: first and last chunks in part, and lengths around the limits
          (9, 6), (70, 36), (33, 602), (21, 4092), (4, 4782), (3, 12004), (2, 18002), (70, 249), (90, 255), (40, 505),
          (37, 511), (9, 8185), (5, 8191), (12, 16383), (9, 32761), (3, 32767)]


@pytest.mark.parametrize("dt,wt", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"),
                                   ("fp32", "fp32")])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward_and_backward(T, d, rms, dt, wt):
    from compressive_fine_tuning_b200 import sk
    x, w, b, dy = _case(T, d, dt, wt)
    eps = 1e-5
    xd, wd, bd, dyd = (t.cuda() for t in (x, w, b, dy))
    y, mean, rstd, ck = sk.layer_norm_fwd(xd, wd, bd, eps, rms)
    assert ck is None
    X, W, B, DY = _n(x), _n(w), _n(b), _n(dy)
    ref, mu, r = oo.norm_forward(X, W, B, eps, rms)
    xh = (X - mu[:, None]) * r[:, None]
    spread = np.abs(xh) + np.abs(xh).mean(1, keepdims=True) + (np.abs(X).mean(1) * r)[:, None]
    _check(y, ref, HALF[dt] * np.abs(ref) + K * V * (np.abs(W) * spread + np.abs(B)) + _smallest(dt), "y")
    _check(rstd, r, K * V * r * (1 + (np.abs(X).mean(1) * r) ** 2), "rstd")
    if rms:
        assert mean is None
    else:
        _check(mean, mu, K * V * (np.abs(X).mean(1) + 1e-30), "mean")
    # without bias and without statistics: the same rows
    y2, m2, r2, _ = sk.layer_norm_fwd(xd, wd, None, eps, rms, stats=False)
    assert m2 is None and r2 is None
    assert torch.equal(y2, sk.layer_norm(xd, wd, None, eps, rms))

    dx, dw, db = sk.layer_norm_bwd(dyd, xd, wd, mean, rstd, rms)
    rdx, rdw, rdb = oo.norm_backward(DY, X, W, eps, rms)
    u = np.abs(DY * W)
    m2 = (u * np.abs(xh)).mean(1, keepdims=True)
    lim = HALF[dt] * np.abs(rdx) + _smallest(dt)
    lim = lim + K * V * r[:, None] * (u + (0 if rms else 1) * u.mean(1, keepdims=True) + spread * (m2 + u))
    _check(dx, rdx, lim, "dx")
    steps = K + T
    _check(dw, rdw, HALF[wt] * np.abs(rdw) + steps * V * (np.abs(DY) * spread).sum(0) + _smallest(wt), "dw")
    _check(db, rdb, HALF[wt] * np.abs(rdb) + steps * V * np.abs(DY).sum(0) + _smallest(wt), "db")
    # deterministic; each output alone is the same
    dx2, dw2, db2 = sk.layer_norm_bwd(dyd, xd, wd, mean, rstd, rms)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)
    only, n1, n2 = sk.layer_norm_bwd(dyd, xd, wd, mean, rstd, rms, bias=False, need_dw=False)
    assert n1 is None and n2 is None
    _check(only, rdx, lim, "dx alone")
    n0, dw3, n2 = sk.layer_norm_bwd(dyd, xd, wd, mean, rstd, rms, bias=False, need_dx=False)
    assert n0 is None and n2 is None and torch.equal(dw3, dw)


@pytest.mark.parametrize("T,d", [(1, 32), (9, 96), (65, 512), (33, 544), (50, 5120), (4, 8192), (2, 16416)])
@pytest.mark.parametrize("rms", [False, True])
def test_checkpoint_of_the_output(T, d, rms):
    from compressive_fine_tuning_b200 import sk
    x, w, b, _ = _case(T, d, "bf16", "fp32")
    x[0, d // 2] = 300.0
    y, _, _, ck = sk.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda(), 1e-6, rms, ckpt=True)
    same = sk.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda(), 1e-6, rms)[0]
    assert torch.equal(y, same)
    want = sk.ckpt8(y)                                    # the checkpoint is that of y as rounded
    assert torch.equal(ck.q, want.q) and torch.equal(ck.scale, want.scale)


def test_many_rows_take_turns():
    """More rows than teams: every row goes through the loop that a team repeats."""
    from compressive_fine_tuning_b200 import sk
    for T, d, dt, wt, rms in ((20011, 64, "bf16", "bf16", False), (9001, 520, "bf16", "fp32", False),
                              (3001, 4104, "bf16", "bf16", False), (1185, 1536, "fp16", "fp32", True),
                              (1184, 2056, "fp32", "fp32", False), (2367, 5120, "bf16", "bf16", True),
                              (1301, 8192, "bf16", "fp32", False), (1200, 8192, "fp32", "fp32", True),
                              (1300, 2048, "bf16", "fp32", False), (1500, 1024, "fp16", "fp16", True),
                              (2500, 600, "bf16", "bf16", False), (1300, 1034, "bf16", "fp32", False),
                              (1200, 2052, "fp16", "fp16", True), (5003, 251, "bf16", "fp32", False),
                              (5003, 509, "fp16", "fp16", True), (2503, 1021, "bf16", "bf16", False),
                              (1500, 4095, "bf16", "fp32", False), (703, 8187, "fp32", "fp32", False),
                              (605, 9001, "bf16", "bf16", True), (310, 20003, "bf16", "fp32", False), (1250, 4096, "bf16", "bf16", False),
                              (1201, 9000, "bf16", "bf16", False), (1186, 17000, "fp16", "fp16", True)):
        x, w, b, dy = _case(T, d, dt, wt)
        xd, wd, bd, dyd = (t.cuda() for t in (x, w, b, dy))
        y, mean, rstd, ck = sk.layer_norm_fwd(xd, wd, bd, 1e-5, rms, ckpt=dt == "bf16" and d % 32 == 0)
        X, W, B, DY = _n(x), _n(w), _n(b), _n(dy)
        ref, mu, r = oo.norm_forward(X, W, B, 1e-5, rms)
        xh = np.abs(X - mu[:, None]) * r[:, None]
        spread = xh + xh.mean(1, keepdims=True) + (np.abs(X).mean(1) * r)[:, None]
        _check(y, ref, HALF[dt] * np.abs(ref) + K * V * (np.abs(W) * spread + np.abs(B)) + _smallest(dt), "y")
        _check(rstd, r, K * V * r * (1 + (np.abs(X).mean(1) * r) ** 2), "rstd")
        if ck is not None:
            alone = sk.layer_norm_fwd(xd, wd, bd, 1e-5, rms)[0]
            _check(alone, ref, HALF[dt] * np.abs(ref) + K * V * (np.abs(W) * spread + np.abs(B)) + _smallest(dt), "y alone")
            want = sk.ckpt8(y)
            assert torch.equal(ck.q, want.q) and torch.equal(ck.scale, want.scale)
        dx, dw, db = sk.layer_norm_bwd(dyd, xd, wd, mean, rstd, rms)
        rdx, rdw, rdb = oo.norm_backward(DY, X, W, 1e-5, rms)
        u = np.abs(DY * W)
        m2 = (u * xh).mean(1, keepdims=True)
        lim = HALF[dt] * np.abs(rdx) + _smallest(dt)
        lim = lim + K * V * r[:, None] * (u + (0 if rms else 1) * u.mean(1, keepdims=True) + spread * (m2 + u))
        _check(dx, rdx, lim, "dx")
        _check(sk.layer_norm_bwd(dyd, xd, wd, mean, rstd, rms, bias=False, need_dw=False)[0], rdx, lim, "dx alone")
        _check(dw, rdw, HALF[wt] * np.abs(rdw) + (K + T) * V * (np.abs(DY) * spread).sum(0) + _smallest(wt), "dw")
        _check(db, rdb, HALF[wt] * np.abs(rdb) + (K + T) * V * np.abs(DY).sum(0) + _smallest(wt), "db")
        again = sk.layer_norm_bwd(dyd, xd, wd, mean, rstd, rms)
        assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))


def test_large_mean_keeps_the_spread():
    """The variance is that of the centred values: a mean 1000 times the spread costs
    only the digits that fp32 inputs of that size have lost already."""
    from compressive_fine_tuning_b200 import sk
    x, w, b, _ = _case(20, 2048, "fp32", "fp32", mean=1000.0)
    y = sk.layer_norm(x.cuda(), w.cuda(), b.cuda(), 1e-5)
    ref, mu, r = oo.norm_forward(_n(x), _n(w), _n(b), 1e-5, False)
    assert (np.abs(_n(y) - ref) <= 42 * V * 1001 * r[:, None] * np.abs(_n(w)) + K * V * (np.abs(ref) + 4)).all()


def test_rows_with_nothing_or_not_finite():
    from compressive_fine_tuning_b200 import sk
    x = torch.ones(4, 96, dtype=torch.bfloat16)
    x[1] = 0
    x[2, 3] = float("nan")
    x[3, 4] = float("inf")
    w, b = torch.full((96,), 2.0), torch.full((96,), 0.5)
    y = sk.layer_norm(x.cuda(), w.cuda(), b.cuda(), 1e-5).float().cpu()
    assert (y[:2] == 0.5).all() and torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
    y = sk.layer_norm(x.cuda(), w.cuda(), None, 1e-5, True).float().cpu()
    assert (y[1] == 0).all() and torch.isnan(y[2]).all()


def test_empty_batch():
    from compressive_fine_tuning_b200 import sk
    x = torch.empty((0, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    y, mean, rstd, _ = sk.layer_norm_fwd(x, w, w)
    dx, dw, db = sk.layer_norm_bwd(x, x, w, mean, rstd)
    assert y.shape == (0, 64) and dx.shape == (0, 64) and not dw.any() and not db.any()


def test_views_that_start_anywhere():
    """Rows, weights and incoming gradients that are views into the middle of a
    buffer, at no 16-byte boundary: the same numbers as their copies."""
    from compressive_fine_tuning_b200 import sk
    x, w, b, dy = _case(9, 33, "bf16", "bf16")
    flat = torch.cat([w, b, w]).cuda()
    ws, bs = flat[33:66].requires_grad_(), flat[66:]
    assert ws.data_ptr() % 16 and bs.data_ptr() % 16
    xs = x.cuda()[1:].requires_grad_()
    assert xs.data_ptr() % 16
    # the gradient of a concatenation is handed on as views of one buffer
    both = torch.cat([torch.zeros(1, 33, dtype=torch.bfloat16, device="cuda"), sk.layer_norm(xs, ws, bs)])
    got = torch.autograd.grad(both, [xs, ws], dy.cuda())
    xc, wc = x[1:].cuda().requires_grad_(), b.cuda().requires_grad_()
    y = sk.layer_norm(xc, wc, w.cuda())
    want = torch.autograd.grad(y, [xc, wc], dy[1:].cuda())
    assert torch.equal(both[1:], y) and all(torch.equal(p, q) for p, q in zip(got, want))
    with torch.no_grad():
        assert torch.equal(sk.layer_norm(xs, ws, bs), y)
    with pytest.raises(sk.SketchError):
        sk.layer_norm_fwd(xs.detach(), w.cuda())                     # the plain call refuses


@pytest.mark.parametrize("rms", [False, True])
def test_autograd_and_differences(rms):
    """The module's gradients against central differences of the float64 formula
    and the oracle's; leading dimensions and strided inputs."""
    from compressive_fine_tuning_b200 import sk
    g = torch.Generator().manual_seed(3)
    big = torch.randn(6, 5, 80, generator=g).cuda()
    x = big.transpose(0, 1)[:, ::2].requires_grad_()             # [5, 3, 80], not contiguous
    m = sk.LayerNorm(80, eps=1e-4, rms=rms, bias=True, device="cuda")
    with torch.no_grad():
        m.weight.copy_(torch.rand(80, generator=g) + 0.5)
        m.bias.copy_(torch.randn(80, generator=g))
    c = torch.randn(5, 3, 80, generator=g).cuda()
    y = m(x)
    assert y.shape == x.shape
    gx, gw, gb = torch.autograd.grad((y * c).sum(), [x, m.weight, m.bias])
    X, W, C = _n(x).reshape(15, 80), _n(m.weight), _n(c).reshape(15, 80)
    rdx, rdw, rdb = oo.norm_backward(C, X, W, 1e-4, rms)
    for got, ref in ((gx.reshape(15, 80), rdx), (gw, rdw), (gb, rdb)):
        np.testing.assert_allclose(_n(got), ref, rtol=1e-5, atol=1e-5)
    h = 1e-4
    rng = np.random.default_rng(0)
    for _ in range(10):
        t, j = rng.integers(15), rng.integers(80)
        e = np.zeros_like(X)
        e[t, j] = h
        f = [(oo.norm_forward(X + s * e, W, _n(m.bias), 1e-4, rms)[0] * C).sum() for s in (1, -1)]
        # the difference's own error is of order h^2 = 1e-8 times third derivatives of order one
        assert abs((f[0] - f[1]) / (2 * h) - _n(gx).reshape(15, 80)[t, j]) <= 1e-4
