"""The operators' oracle pinned against something other than itself: closed
forms, library routines and finite differences (CPU only)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import operators_oracle as oo  # noqa: E402


def test_checkpoint_by_hand():
    x = np.zeros((1, 64))
    x[0, :4] = [127.0, 0.5, 1.5, -2.5]                  # 2^0: ties to even
    x[0, 32:34] = [127.5, 3.0]                          # does not fit 127 * 2^0: 2^1
    q, s = oo.ckpt8_quantize(x)
    assert s.tolist() == [[127, 128]]
    assert q[0, :4].tolist() == [127, 0, 2, -2] and q[0, 32:34].tolist() == [64, 2]
    assert oo.ckpt8_values(q, s)[0, 32:34].tolist() == [128.0, 4.0]


def test_checkpoint_range():
    x = np.zeros((4, 32))
    x[0, 0] = 255 * 2.0 ** 120                          # the largest bf16: clipped to 127 * 2^121
    x[1, 0] = 2.0 ** -133                               # below half the smallest step
    x[2, 0] = np.nan
    q, s = oo.ckpt8_quantize(x)
    assert (q[0, 0], s[0, 0]) == (127, 248) and (q[1, 0], s[1, 0]) == (0, 1) and s[2, 0] == 255 and s[3, 0] == 1
    v = oo.ckpt8_values(q, s)
    assert np.isnan(v[2]).all() and v[0, 0] == 127 * 2.0 ** 121


def test_checkpoint_is_the_nearest_multiple():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 96)) * np.exp(8 * rng.standard_normal((50, 1)))
    q, s = oo.ckpt8_quantize(x)
    step = np.repeat(2.0 ** (s.astype(float) - 127), 32, axis=1)
    assert (np.abs(oo.ckpt8_values(q, s) - x) <= step / 2).all()
    top = np.abs(x).reshape(50, 3, 32).max(-1)
    assert (127 * 2.0 ** (s.astype(float) - 127) >= top).all() and (127 * 2.0 ** (s.astype(float) - 128) < top).all()


@pytest.mark.parametrize("rms", [False, True])
def test_norm_against_the_library(rms):
    g = torch.Generator().manual_seed(0)
    x = torch.randn(7, 40, dtype=torch.float64, generator=g).requires_grad_()
    w = torch.randn(40, dtype=torch.float64, generator=g).requires_grad_()
    b = torch.randn(40, dtype=torch.float64, generator=g).requires_grad_()
    dy = torch.randn(7, 40, dtype=torch.float64, generator=g)
    if rms:
        y = torch.nn.functional.rms_norm(x, (40,), w, 1e-3) + b
    else:
        y = torch.nn.functional.layer_norm(x, (40,), w, b, 1e-3)
    y.backward(dy)
    X, W, B = (t.detach().numpy() for t in (x, w, b))
    np.testing.assert_allclose(oo.norm_forward(X, W, B, 1e-3, rms)[0], y.detach().numpy(), rtol=1e-12, atol=1e-12)
    for got, ref in zip(oo.norm_backward(dy.numpy(), X, W, 1e-3, rms), (x.grad, w.grad, b.grad)):
        np.testing.assert_allclose(got, ref.numpy(), rtol=1e-11, atol=1e-11)


@pytest.mark.parametrize("reduction", ["none", "mean", "sum"])
def test_cross_entropy_against_the_library(reduction):
    g = torch.Generator().manual_seed(1)
    h = torch.randn(9, 12, dtype=torch.float64, generator=g).requires_grad_()
    w = torch.randn(30, 12, dtype=torch.float64, generator=g).requires_grad_()
    y = torch.randint(0, 30, (9,), generator=g)
    y[2] = -100
    loss = torch.nn.functional.cross_entropy(h @ w.T, y, reduction=reduction)
    dl = torch.randn(9, dtype=torch.float64, generator=g) if reduction == "none" else torch.tensor(0.7, dtype=torch.float64)
    loss.backward(dl)
    got = oo.cross_entropy(h.detach().numpy(), w.detach().numpy(), y.numpy(), -100, reduction, dl.numpy())
    np.testing.assert_allclose(got[0], loss.detach().numpy(), rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(got[1], h.grad.numpy(), rtol=1e-10, atol=1e-13)
    np.testing.assert_allclose(got[2], w.grad.numpy(), rtol=1e-10, atol=1e-13)


def test_cross_entropy_leaves_out_what_it_must():
    h, w = np.ones((3, 2)), np.ones((4, 2))
    loss, dh, dw, _ = oo.cross_entropy(h, w, np.array([-1, 4, 2]), 2, "mean")
    assert loss == 0 and not dh.any() and not dw.any()
