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
