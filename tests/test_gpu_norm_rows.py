"""dw and db of the norm's backward pass, row by row: no row left out, none twice.

With dy zero in all rows but one, dw and db are that row's terms alone: every
other term of a sum is an exact zero, so what is left is the rounding of
xh = (x - mean) * rstd (three roundings, and those of the row's statistics,
K 2^-24 of the row's magnitudes as in the test of whole batches), of one product,
and of the output.  db is dy's row itself.

For whole batches the sums' bound goes with the longest chain of additions that
the kernels have: the rows of one partial sum, then the partial sums of one thread
and the joining of 16 or fewer groups of threads.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import operators_oracle as oo  # noqa: E402
from tests.test_gpu_norm import HALF, K, V, _case, _check, _n, _smallest  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


# warps, blocks, the ring of pairs of rows (16-byte and longer rows of 1184 rows and
# more), odd lengths, and rows beyond 8192 columns, each with an odd last row
CASES = [(20011, 64, "bf16", "bf16", False), (4737, 512, "fp16", "fp32", False), (9001, 520, "bf16", "fp32", False),
         (1301, 4096, "bf16", "fp32", False), (1185, 8192, "bf16", "bf16", True), (2369, 2048, "fp32", "fp32", False),
         (1301, 1034, "bf16", "fp32", False), (2503, 1021, "bf16", "bf16", False), (703, 8187, "fp32", "fp32", True),
         (77, 4096, "bf16", "bf16", False), (605, 9001, "bf16", "bf16", True), (1187, 16384, "bf16", "fp32", False)]


@pytest.mark.parametrize("T,d,dt,wt,rms", CASES)
def test_a_single_row_reaches_dw_and_db(T, d, dt, wt, rms):
    from compressive_fine_tuning_b200 import sk
    x, w, b, dy = _case(T, d, dt, wt)
    xd, wd = x.cuda(), w.cuda()
    _, mean, rstd, _ = sk.layer_norm_fwd(xd, wd, b.cuda(), 1e-5, rms)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for row in sorted({0, 1, T // 2, min(T - 1, 2 * sms), T - 2, T - 1}):
        one = torch.zeros_like(xd)
        one[row] = dy[row].cuda()
        _, dw, db = sk.layer_norm_bwd(one, xd, wd, mean, rstd, rms)
        X, DY = _n(x[row:row + 1]), _n(dy[row:row + 1])
        _, mu, r = oo.norm_forward(X, _n(w), None, 1e-5, rms)
        xh = (X - mu[:, None]) * r[:, None]
        spread = np.abs(xh) + np.abs(xh).mean(1, keepdims=True) + (np.abs(X).mean(1) * r)[:, None]
        want = (DY * xh)[0]
        _check(dw, want, HALF[wt] * np.abs(want) + K * V * (np.abs(DY) * spread)[0] + _smallest(wt), f"dw, row {row}")
        _check(db, DY[0], HALF[wt] * np.abs(DY[0]) + _smallest(wt), f"db, row {row}")


@pytest.mark.parametrize("T,d,dt,wt,rms", CASES)
def test_sums_over_rows(T, d, dt, wt, rms):
    from compressive_fine_tuning_b200 import sk
    x, w, b, dy = _case(T, d, dt, wt, seed=7)
    xd, wd, dyd = x.cuda(), w.cuda(), dy.cuda()
    _, mean, rstd, _ = sk.layer_norm_fwd(xd, wd, b.cuda(), 1e-5, rms)
    _, dw, db = sk.layer_norm_bwd(dyd, xd, wd, mean, rstd, rms)
    X, DY = _n(x), _n(dy)
    _, rdw, rdb = oo.norm_backward(DY, X, _n(w), 1e-5, rms)
    _, mu, r = oo.norm_forward(X, _n(w), None, 1e-5, rms)
    xh = np.abs((X - mu[:, None]) * r[:, None])
    spread = xh + xh.mean(1, keepdims=True) + (np.abs(X).mean(1) * r)[:, None]
    parts = sk.lib.sk_layer_norm_bwd_workspace_bytes(T, d) // (8 * d)
    # rows of a partial sum (two more for pairs of rows), partial sums of a thread, joins
    chain = -(-T // parts) + 2 + -(-parts // 16) + 20
    _check(dw, rdw, HALF[wt] * np.abs(rdw) + (K + chain) * V * (np.abs(DY) * spread).sum(0) + _smallest(wt), "dw")
    _check(db, rdb, HALF[wt] * np.abs(rdb) + chain * V * np.abs(DY).sum(0) + _smallest(wt), "db")
    # these limits see a row that is missing
    lost = np.abs(DY[-1])
    seen = lost > HALF[wt] * np.abs(rdb) + chain * V * np.abs(DY).sum(0) + _smallest(wt)
    assert HALF[wt] > 2.0 ** -20 or seen.mean() > 0.9
