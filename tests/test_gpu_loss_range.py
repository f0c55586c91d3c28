"""The loss's gradients of surely predicted tokens, class by class.

Each token is sure of its target, and the other classes lie 6 to 32 nats (2^-9 to
2^-46) below it, in the target's tile of classes and in others.  Every class has a
column of its own in W, so that dH shows each probability by itself, and every row
of dW belongs to one class.

Bounds, relative to each value itself.  A probability's exponential: 2^-11 for its
16-bit form, 2^-8 for P in bf16, and 2^-16 for the exponentials (ex2.approx of an
argument up to 46 that is off by half a step of 2^-18, __expf of one up to 32 by 40
steps of 2^-24, and the row's lse by half a step of 2^-18).  fp16 has full precision down to
2^-14 and half a step of 2^-25 below; the exponentials are kept times 2^15, so that
is 2^-40 of the tile's largest, absolute.  The products: one accumulation of 2^-23
per 16 terms, all of one sign.  The outputs: 2^-8.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import operators_oracle as oo  # noqa: E402

pytestmark = pytest.mark.gpu

P_REL = (1 + 2.0 ** -8) * (1 + 2.0 ** -11) * (1 + 2.0 ** -16)
P_ABS = 2.0 ** -40 * (1 + 2.0 ** -7)


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _n(t):
    return t.detach().double().cpu().numpy()


# 256 tokens take tiles of 256 tokens, the others the exchanged product
@pytest.mark.parametrize("T,V", [(3, 100), (20, 512), (256, 100), (256, 512), (300, 700)])
def test_small_probabilities_next_to_a_sure_target(T, V):
    from compressive_fine_tuning_b200 import sk
    d = 8 + (V + 7) // 8 * 8
    first, second = 5, V * 3 // 5
    v, t = np.arange(V), np.arange(T)
    W = np.zeros((V, d))
    W[v, 8 + v] = 1.0
    W[:, 0] = v * 7 % 41 / 64.0                       # logits are exact: H has one value per row
    W[:, 1] = (v * 7 + 13) % 41 / 64.0
    W[first, 0] = W[second, 1] = 1.0
    H = np.zeros((T, d))
    H[t, t % 2] = 16.0 + t % 17
    y = np.where(t % 2 == 0, first, second)
    h, w = (torch.from_numpy(a).to(torch.bfloat16) for a in (H, W))
    assert (_n(h) == H).all() and (_n(w) == W).all()
    _, dH, dW = sk.cross_entropy(h.cuda(), w.cuda(), torch.from_numpy(y).cuda(), reduction="sum", need_dh=True, need_dw=True)
    _, rh, rw, P = oo.cross_entropy(H, W, y, -100, "sum")
    assert P[t, y].min() > -0.25                      # every target has at least 75 %, most far more
    others = np.ones((T, V), dtype=bool)
    others[t, y] = False
    got, ref = _n(dH)[:, 8:8 + V][others], rh[:, 8:8 + V][others]
    rel = P_REL * (1 + 2.0 ** -8) * (1 + (V / 16 + 4) * 2.0 ** -23) - 1
    err = np.abs(got - ref) / (rel * ref + P_ABS)
    assert (err <= 1).all(), float(err.max())
    rows = np.setdiff1d(v, [first, second])
    rel = P_REL * (1 + 2.0 ** -8) * (1 + (T / 16 + 4) * 2.0 ** -23) - 1
    for k in (0, 1):
        err = np.abs(_n(dW)[rows, k] - rw[rows, k]) / (rel * rw[rows, k] + P_ABS * np.abs(H[:, k]).sum())
        assert (err <= 1).all(), (k, float(err.max()))
    assert sk.device_check() == 0


@pytest.mark.parametrize("T,V,ignored,reduction,factor", [
    (255, 20001, 0, "mean", None), (300, 20001, 45, "mean", None), (510, 9000, 0, "mean", 3.0), (256, 9000, 0, "sum", 0.3),
    (40, 9000, 5, "mean", -0.7), (255, 20001, 0, "none", 1 / 255), (40, 9000, 5, "none", -0.7)])
def test_a_factor_that_tokens_share_is_not_rounded(T, V, ignored, reduction, factor):
    """1 / 255 lies halfway between two bf16 values: rounded together with the target's
    entry of P it moved all of dW by 2^-8.  The factor of a reduced loss, and what
    per-token weights have in common, belong to the fp32 sums: here every token is far from sure, so that 1 - p is nearly one and
    P's rounding small.  Limits: that rounding (known), 2^-8 and what the other test allows for the
    rest of the probabilities, and the output's 2^-8."""
    from compressive_fine_tuning_b200 import sk
    d = 64
    g = torch.Generator().manual_seed(T + V)
    h = torch.randn(T, d, generator=g).to(torch.bfloat16)
    w = (0.3 * torch.randn(V, d, generator=g) / 8).to(torch.bfloat16)
    y = torch.randperm(V, generator=g)[:T]               # a row of dW has one token
    y[:ignored] = -100
    dl = None if factor is None else torch.full((T if reduction == "none" else 1,), factor)
    _, dH, dW = sk.cross_entropy(h.cuda(), w.cuda(), y.cuda(), reduction=reduction, dloss=None if dl is None else dl.cuda(),
                                 need_dh=True, need_dw=True)
    H, W, Y = _n(h), _n(w), y.numpy()
    _, rh, rw, P = oo.cross_entropy(H, W, Y, -100, reduction, None if dl is None else _n(dl))
    keep = Y >= 0
    scale = (1.0 if dl is None else float(dl[0])) / (keep.sum() if reduction == "mean" else 1)
    t = np.arange(T)[keep]
    entry = P[t, Y[keep]] / scale                         # p - 1
    rounded = _n(torch.from_numpy(entry).float().to(torch.bfloat16))
    assert entry.max() < -0.99 and np.abs(rounded - entry).max() < 2.0 ** -10
    delta = (d / 16 + 4) * 2.0 ** -23 * (np.abs(H) @ np.abs(W).T).max()
    off = np.abs(P)
    off[t, Y[keep]] = 0.0
    other = (P_REL * (1 + 2 * delta) - 1) * off + P_ABS * np.abs(scale)
    moved = other.copy()
    moved[t, Y[keep]] = (np.abs(rounded - entry) + 2.0 ** -20 + 2 * delta) * np.abs(scale)
    lim = moved.T @ np.abs(H) + (T / 16 + 4) * 2.0 ** -23 * (np.abs(P).T @ np.abs(H)) + 2.0 ** -8 * np.abs(rw) + 1e-30
    err = np.abs(_n(dW) - rw) / lim
    assert (err <= 1).all(), float(err.max())
    # dH gets the rounding of the target's entry back
    moved[t, Y[keep]] = (2.0 ** -20 + 2 * delta) * np.abs(scale)
    lim = moved @ np.abs(W) + (V / 16 + 4) * 2.0 ** -23 * (np.abs(P) @ np.abs(W)) + 2.0 ** -8 * np.abs(rh) + 1e-30
    err = np.abs(_n(dH) - rh) / lim
    assert (err <= 1).all(), float(err.max())
    assert not _n(dH)[~keep].any() and sk.device_check() == 0
