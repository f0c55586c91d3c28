"""Linear cross entropy against the float64 oracle.

Bounds.  A logit is d / 16 accumulations of sixteen exact products, each off by
less than 2^-23 of the magnitudes: delta = (d / 16 + 4) 2^-23 max_v sum |h w|.
A loss moves by at most 2 delta plus a few fp32 roundings of its terms.
P moves by its two roundings (fp16 2^-11, bf16 2^-8), by 2 delta and 2^-18 for the
exponentials, and by 2^-25 of the tile's largest where fp16 runs out; the products
add V / 16 (T / 16) accumulations of 2^-23, the outputs a bf16 rounding (2^-8).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import operators_oracle as oo  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _case(T, V, d, seed=0, ignored=0.2, scale=1.0, lean=8.0):
    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + V + d)
    w = (scale * torch.randn(V, d, generator=g) / d ** 0.5).to(torch.bfloat16)
    y = torch.randint(0, V, (T,), generator=g)
    h = (torch.randn(T, d, generator=g) + lean * torch.rand(T, 1, generator=g) * w[y].float()).to(torch.bfloat16)
    y[torch.rand(T, generator=g) < ignored] = -100
    return h, w, y


def _n(t):
    return t.detach().double().cpu().numpy()


def _bounds(H, W, P, c, dh, dw):
    d, V, T = H.shape[1], W.shape[0], H.shape[0]
    delta = (d / 16 + 4) * 2.0 ** -23 * (np.abs(H) @ np.abs(W).T).max(1)
    rel = (2.0 ** -8 + 2.0 ** -11 + 2 * delta + 2.0 ** -18)[:, None]
    moved = rel * np.abs(P) + 2.0 ** -24 * np.abs(c)[:, None]
    lim_h = moved @ np.abs(W) + (V / 16 + 4) * 2.0 ** -23 * (np.abs(P) @ np.abs(W)) + 2.0 ** -8 * np.abs(dh) + 1e-30
    lim_w = moved.T @ np.abs(H) + (T / 16 + 4) * 2.0 ** -23 * (np.abs(P).T @ np.abs(H)) + 2.0 ** -8 * np.abs(dw) + 1e-30
    return delta, lim_h, lim_w


def _check(got, ref, lim, what):
    err = np.abs(_n(got) - ref)
    assert np.isfinite(_n(got)).all(), what
    assert (err <= lim).all(), f"{what}: {float((err / lim).max()):.3f} of the bound"


SHAPES = [(1, 1, 8), (1, 2, 64), (2, 255, 72), (3, 256, 64), (5, 257, 128), (127, 300, 520), (128, 1000, 64),
          (129, 511, 200), (256, 513, 256), (257, 100, 1000), (300, 3001, 320), (64, 20001, 64), (700, 777, 96),
          (40, 5000, 136), (1030, 2500, 264), (600, 4001, 520), (270, 20011, 96)]


@pytest.mark.parametrize("reduction", ["none", "mean", "sum"])
@pytest.mark.parametrize("T,V,d", SHAPES)
def test_loss_and_gradients(T, V, d, reduction):
    from compressive_fine_tuning_b200 import sk
    h, w, y = _case(T, V, d)
    hd, wd, yd = h.cuda(), w.cuda(), y.cuda()
    dl = None
    if reduction == "none":
        dl = torch.linspace(-1.0, 2.0, T)
    elif T % 2:
        dl = torch.tensor([0.375])
    loss, dH, dW = sk.cross_entropy(hd, wd, yd, reduction=reduction, dloss=None if dl is None else dl.cuda(),
                                    need_dh=True, need_dw=True)
    H, W, Y = _n(h), _n(w), y.numpy()
    rl, rh, rw, P = oo.cross_entropy(H, W, Y, -100, reduction, None if dl is None else _n(dl))
    keep = Y != -100
    c = keep * (1.0 if dl is None else _n(dl)) / (max(1, keep.sum()) if reduction == "mean" else 1)
    delta, lim_h, lim_w = _bounds(H, W, P, c * np.ones(T), rh, rw)
    each = 2 * delta + 2.0 ** -20 * (2 + np.abs(H @ W.T).max(1))
    _check(loss, rl, each if reduction == "none" else (each * keep).sum() / (max(1, keep.sum()) if reduction == "mean" else 1)
           + 2.0 ** -23 * np.abs(rl) + 1e-12, "loss")
    _check(dH, rh, lim_h, "dH")
    _check(dW, rw, lim_w, "dW")
    assert not _n(dH)[~keep].any()
    # The loss alone may cut the vocabulary into narrower tiles: another order of fewer
    # than 64 additions of 2^-24 on either side (2^-17 of the sum, absolute in its
    # logarithm) and the roundings of the largest logit's size.
    l2, a, b = sk.cross_entropy(hd, wd, yd, reduction=reduction)
    assert a is None and b is None
    near = 2.0 ** -17 + 2.0 ** -22 * np.abs(H @ W.T).max()
    assert np.abs(_n(l2) - _n(loss)).max() <= near * (max(1, keep.sum()) if reduction == "sum" else 1)
    assert torch.equal(l2, sk.cross_entropy(hd, wd, yd, reduction=reduction)[0])
    # each gradient alone, the same inputs again: the same numbers
    dlc = None if dl is None else dl.cuda()
    assert torch.equal(sk.cross_entropy(hd, wd, yd.int(), reduction=reduction, dloss=dlc, need_loss=False, need_dh=True)[1], dH)
    assert torch.equal(sk.cross_entropy(hd, wd, yd, reduction=reduction, dloss=dlc, need_loss=False, need_dw=True)[2], dW)
    assert sk.device_check() == 0


@pytest.mark.parametrize("scale", [0.0, 30.0, 200.0])
def test_flat_and_large_logits(scale):
    """Equal logits (loss log V), and logits of tens to hundreds, where only the
    shift by the largest keeps the exponentials finite."""
    from compressive_fine_tuning_b200 import sk
    h, w, y = _case(40, 1500, 128, scale=scale, ignored=0.0, lean=0.0)
    loss, dH, _ = sk.cross_entropy(h.cuda(), w.cuda(), y.cuda(), reduction="none", need_dh=True)
    H, W = _n(h), _n(w)
    rl, rh, rw, P = oo.cross_entropy(H, W, y.numpy(), -100, "none")
    delta, lim_h, _ = _bounds(H, W, P, np.ones(40), rh, rw)
    _check(loss, rl, 2 * delta + 2.0 ** -20 * (2 + np.abs(H @ W.T).max(1)), "loss")
    _check(dH, rh, lim_h, "dH")


def test_surely_predicted_tokens_keep_their_gradient():
    """softmax ~ 1 at the target: the gradient is 1 - p, formed without cancellation,
    so it stays near the float64 one relative to its own size."""
    from compressive_fine_tuning_b200 import sk
    V, d, T = 512, 64, 8
    w = torch.zeros(V, d)
    w[:64] = torch.eye(64)
    h = torch.zeros(T, d)
    y = torch.arange(T) * 5
    h[torch.arange(T), y] = torch.linspace(9.0, 16.0, T)
    loss, dH, _ = sk.cross_entropy(h.bfloat16().cuda(), w.bfloat16().cuda(), y.cuda(), reduction="none", need_dh=True)
    rl, rh, _, _ = oo.cross_entropy(_n(h.bfloat16()), _n(w), y.numpy(), -100, "none")
    # The sum of exponentials is 1 and small terms: an addition next to 1 rounds by at
    # most 2^-24, and the longest chain has 32 terms of a 32-column piece, 8 pieces of
    # a tile, and 9 joins of two roundings: fewer than 64, so 2^-18 absolute.
    assert (np.abs(_n(loss) - rl) <= 2.0 ** -18 + 2.0 ** -18 * rl).all()
    got = _n(dH)[np.arange(T), y.numpy()]
    ref = rh[np.arange(T), y.numpy()]
    assert (np.abs(got - ref) <= 2 * 2.0 ** -8 * np.abs(ref) + 2.0 ** -18).all()


def test_targets_out_of_range_and_all_ignored():
    from compressive_fine_tuning_b200 import sk
    h, w, y = _case(50, 400, 64, ignored=0.0)
    y[3], y[9] = 400, -7
    hd, wd = h.cuda(), w.cuda()
    loss, dH, dW = sk.cross_entropy(hd, wd, y.cuda(), reduction="mean", need_dh=True, need_dw=True)
    assert sk.device_check() == sk.SK_CHECK_TARGET_RANGE
    y[3] = y[9] = -100
    want = sk.cross_entropy(hd, wd, y.cuda(), reduction="mean", need_dh=True, need_dw=True)
    assert all(torch.equal(a, b) for a, b in zip((loss, dH, dW), want))
    none = torch.full((50,), -100, dtype=torch.int64, device="cuda")
    for red in ("mean", "sum", "none"):
        loss, dH, dW = sk.cross_entropy(hd, wd, none, reduction=red, need_dh=True, need_dw=True)
        assert not loss.any() and not dH.any() and not dW.any()
    # any id may be the ignored one, a class among them
    y[:] = 17
    loss = sk.cross_entropy(hd, wd, y.cuda(), ignore_index=17, reduction="none")[0]
    assert not loss.any() and sk.device_check() == 0


def test_not_finite_rows_stay_apart():
    from compressive_fine_tuning_b200 import sk
    h, w, y = _case(20, 600, 64, ignored=0.0)
    clean = sk.cross_entropy(h.cuda(), w.cuda(), y.cuda(), reduction="none", need_dh=True)
    h[4, 7] = float("nan")
    h[11, 0] = float("inf")
    loss, dH, _ = sk.cross_entropy(h.cuda(), w.cuda(), y.cuda(), reduction="none", need_dh=True)
    bad = torch.tensor([4, 11])
    good = torch.tensor([t for t in range(20) if t not in (4, 11)])
    assert torch.isnan(loss[bad]).all() and torch.isnan(dH[bad]).all()
    assert torch.equal(loss[good], clean[0][good]) and torch.equal(dH[good], clean[1][good])


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_targets_from_the_second_id_on(dtype):
    """A sequence's targets are its ids shifted by one: a view one value further on."""
    from compressive_fine_tuning_b200 import sk
    h, w, y = _case(70, 500, 64)
    ids = torch.cat([y[:1], y]).to(dtype).cuda()
    weights = torch.rand(71, device="cuda")
    assert ids[1:].data_ptr() % 16 and weights[1:].data_ptr() % 16
    for red in ("none", "mean"):
        dl = weights[1:] if red == "none" else weights[3:4]
        got = sk.cross_entropy(h.cuda(), w.cuda(), ids[1:], reduction=red, dloss=dl, need_dh=True, need_dw=True)
        want = sk.cross_entropy(h.cuda(), w.cuda(), y.cuda(), reduction=red, dloss=dl.clone(), need_dh=True, need_dw=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T,V,d", [(20, 600, 64), (300, 1000, 128), (520, 264, 72)])
@pytest.mark.parametrize("reduction", ["none", "mean"])
def test_rows_of_tokens_that_take_no_part_hold_anything(T, V, d, reduction):
    """NaN and infinities in ignored tokens' rows (uninitialised padding) reach
    neither the loss nor dW nor the other tokens' dH: the same numbers as with
    zeros there."""
    from compressive_fine_tuning_b200 import sk
    h, w, y = _case(T, V, d, ignored=0.0)
    out = torch.tensor([0, 7, T // 2, T - 1])
    y[out] = -100
    h[out] = 0.0
    wd, yd = w.cuda(), y.cuda()
    want = sk.cross_entropy(h.cuda(), wd, yd, reduction=reduction, need_dh=True, need_dw=True)
    for k, bad in enumerate((float("nan"), float("inf"), -float("inf"))):
        dirty = h.clone()
        dirty[out[k], d - 1 - k] = bad
        dirty[out[3]] = bad
        got = sk.cross_entropy(dirty.cuda(), wd, yd, reduction=reduction, need_dh=True, need_dw=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(sk.cross_entropy(dirty.cuda(), wd, yd, reduction=reduction)[0],
                           sk.cross_entropy(h.cuda(), wd, yd, reduction=reduction)[0])
    # a class out of range is treated the same way
    y[out[0]] = V
    got = sk.cross_entropy(dirty.cuda(), wd, y.cuda(), reduction=reduction, need_dh=True, need_dw=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert sk.device_check() == sk.SK_CHECK_TARGET_RANGE


def test_empty_batch():
    from compressive_fine_tuning_b200 import sk
    h = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((10, 64), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((0,), dtype=torch.int64, device="cuda")
    for red in ("none", "mean", "sum"):
        loss, dH, dW = sk.cross_entropy(h, w, y, reduction=red, need_dh=True, need_dw=True)
        assert loss.numel() == (0 if red == "none" else 1) and not loss.any()
        assert dH.shape == (0, 64) and not dW.any()


def test_autograd():
    """Reduced losses hand out the gradients of the forward pass, scaled; a second
    backward pass over a retained graph gives the same numbers again."""
    from compressive_fine_tuning_b200 import sk
    h, w, y = _case(60, 900, 128)
    hd = h.cuda().reshape(3, 20, 128).requires_grad_()
    wd = w.cuda().requires_grad_()
    yd = y.cuda().reshape(3, 20)
    loss = sk.linear_cross_entropy(hd, wd, yd)
    alone = sk.linear_cross_entropy(hd.detach(), wd.detach(), yd)
    assert abs(float(alone) - float(loss.detach())) <= 2.0 ** -17 + 2.0 ** -22 * np.abs(_n(h) @ _n(w).T).max()
    one = torch.autograd.grad(loss, [hd, wd], retain_graph=True)
    kept = [t.clone() for t in one]
    two = torch.autograd.grad(loss * 4.0, [hd, wd], retain_graph=True)
    for a, b, k in zip(one, two, kept):
        assert torch.equal(a, k)                                      # handed out once, not touched again
        assert torch.equal(b.float(), 4.0 * a.float())                # a power of two scales every rounding
    _, rh, rw, P = oo.cross_entropy(_n(h), _n(w), y.numpy(), -100, "mean")
    keep = y.numpy() != -100
    _, lim_h, lim_w = _bounds(_n(h), _n(w), P, keep / keep.sum(), rh, rw)
    _check(one[0].reshape(60, 128), rh, lim_h, "dH")
    _check(one[1], rw, lim_w, "dW")
    # scaled by something that is not a power of two: one more bf16 rounding
    loss = sk.linear_cross_entropy(hd, wd, yd)
    three, = torch.autograd.grad(loss * 0.3, [hd])
    _check(three.reshape(60, 128), 0.3 * rh, 0.3 * (lim_h * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(rh)) + 1e-7 * np.abs(rh), "scaled")
    # per-token losses with their own weights
    g = torch.rand(3, 20, device="cuda")
    each = sk.linear_cross_entropy(hd, wd, yd, reduction="none")
    assert each.shape == (3, 20)
    gh, = torch.autograd.grad(each, [hd], g)
    _, rh, rw, P = oo.cross_entropy(_n(h), _n(w), y.numpy(), -100, "none", _n(g).reshape(-1))
    _, lim_h, _ = _bounds(_n(h), _n(w), P, keep * _n(g).reshape(-1), rh, rw)
    _check(gh.reshape(60, 128), rh, lim_h, "dH")


def test_difference_quotient():
    """dH along random directions against central differences of the float64 loss."""
    h, w, y = _case(12, 200, 64)
    H, W, Y = _n(h), _n(w), y.numpy()
    from compressive_fine_tuning_b200 import sk
    _, dH, dW = sk.cross_entropy(h.cuda(), w.cuda(), y.cuda(), need_dh=True, need_dw=True)
    rng = np.random.default_rng(1)
    for _ in range(5):
        e, f = rng.standard_normal(H.shape), rng.standard_normal(W.shape)
        s = 1e-4
        quot = (oo.cross_entropy(H + s * e, W, Y, -100, "mean")[0] - oo.cross_entropy(H - s * e, W, Y, -100, "mean")[0]) / (2 * s)
        lim = 2.0 ** -6 * (np.abs(_n(dH)) * np.abs(e)).sum() + 1e-6
        assert abs((_n(dH) * e).sum() - quot) <= lim
        quot = (oo.cross_entropy(H, W + s * f, Y, -100, "mean")[0] - oo.cross_entropy(H, W - s * f, Y, -100, "mean")[0]) / (2 * s)
        lim = 2.0 ** -6 * (np.abs(_n(dW)) * np.abs(f)).sum() + 1e-6
        assert abs((_n(dW) * f).sum() - quot) <= lim
