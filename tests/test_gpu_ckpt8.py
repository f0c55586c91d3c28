"""8-bit activation checkpoints and the LUT gradient that reads them.

The quantiser is exact arithmetic, so q, scale and the values read back must
match the oracle bit for bit.  The LUT gradient must match the float64 gradient
of the values the checkpoint stands for, and on the tensor cores be the same
numbers that the bf16 gradient gives for those values.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from compressive_fine_tuning_b200 import synth  # noqa: E402
from oracle import operators_oracle as oo  # noqa: E402
from tests import gpu_cases as gc  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda(monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    monkeypatch.delenv("SK_BWD_PATH", raising=False)


def _rows(T, d, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, d, generator=g) * torch.exp(6 * torch.randn(T, 1, generator=g))
    x = x * torch.exp(2 * torch.randn(T, d, generator=g))
    return x.to(torch.bfloat16)


def _special(T, d):
    x = _rows(T, d, 5)
    bits = x.view(torch.int16)
    x[0] = 0
    x[1, :32] = 2.0 ** -133                    # subnormal: rounds to zero at the smallest scale
    x[1, 32:64] = -(2.0 ** -120)
    x[2, :32] = 255 * 2.0 ** 120               # the largest bf16
    x[2, 32:64] = -127 * 2.0 ** 121
    x[3, :32] = 127.0                          # exactly 127 * 2^0
    x[3, 5] = 0.5                              # ties to even: 0
    x[3, 6] = 1.5                              # and 2
    x[3, 32:64] = 127.5                        # needs the next exponent
    x[4, 7] = float("nan")
    x[4, 40] = float("inf")
    x[4, 70] = -float("inf")
    assert bits.data_ptr() == x.data_ptr()
    return x


def _f64(t):
    return gc.bf16_to_f64(t)


@pytest.mark.parametrize("T,d", [(1, 32), (7, 96), (5, 11008), (1000, 4096), (3, 160), (64, 64)])
def test_checkpoint_bits(T, d):
    from compressive_fine_tuning_b200 import sk
    x = _special(T, d) if T >= 5 and d >= 96 else _rows(T, d, T + d)
    ck = sk.ckpt8(x.cuda())
    q, scale = oo.ckpt8_quantize(_f64(x))
    np.testing.assert_array_equal(ck.scale.cpu().numpy(), scale)
    np.testing.assert_array_equal(ck.q.cpu().numpy(), q)
    back = _f64(sk.ckpt8_dequant(ck))
    np.testing.assert_array_equal(back, oo.ckpt8_values(q, scale))    # NaNs in the same places
    fin = np.isfinite(back)
    top = np.where(fin, np.abs(_f64(x)), 0.0).reshape(T, -1, 32).max(-1, keepdims=True)
    # half a step of 2^e, and 127 * 2^(e-1) is below the block's largest value unless e is at its least
    lim = np.maximum(top / 127.0, 2.0 ** -127) * np.ones((1, 1, 32))
    err = np.where(fin, np.abs(back - np.where(fin, _f64(x), 0.0)), 0.0)
    assert (err <= lim.reshape(T, d)).all()


def _dlut_bound(c, values, task, ntask, T):
    """|error| of a bin: T / 16 accumulations of sixteen exact products each and at
    most 512 additions of the binning, each off by less than 2^-23 of the sum of
    magnitudes."""
    mag = oracle.backward_lut(np.abs(values), np.abs(c.dy), c.idx, c.gpr, c.k, task, ntask)
    return (T / 16 + 512) * 2.0 ** -23 * mag + 1e-30


CASES = [
    # n, d, bits, gpr, T, sets
    (8, 32, 4, 1, 1, 1), (64, 64, 2, 2, 63, 1), (64, 64, 2, 2, 64, 1), (256, 512, 3, 4, 33, 1),
    (264, 1376, 3, 1, 300, 1), (1000, 2048, 4, 8, 129, 1), (512, 288, 2, 3, 1000, 1),
    (128, 512, 4, 4, 200, 8), (320, 1024, 3, 2, 700, 3), (64, 96, 2, 1, 5, 3), (256, 256, 4, 1, 64, 8),
    (256, 512, 4, 16, 15, 1), (256, 512, 4, 16, 16, 1), (1024, 4096, 3, 2, 17, 5), (520, 1056, 2, 33, 100, 2),
    (1024, 4096, 4, 1, 3000, 1), (2568, 2080, 4, 5, 2500, 1),
    # groups of whole column tiles with enough (set, group, row block) units for the pairs
    (2304, 2048, 4, 4, 300, 4), (2264, 1536, 3, 2, 333, 8), (2304, 512, 2, 2, 700, 16),
]


@pytest.mark.parametrize("n,d,bits,gpr,T,sets", CASES)
def test_lut_gradient(n, d, bits, gpr, T, sets):
    from compressive_fine_tuning_b200 import sk
    c = synth.layer_case(900 + n + T, n=n, d=d, bits=bits, gpr=gpr, T=T, ntask=sets)
    packed, lut, X, dY, task = gc.dev_case(c)
    ck = sk.ckpt8(X)
    values = oo.ckpt8_values(*oo.ckpt8_quantize(c.x))
    got = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, sets)
    again = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, sets)
    assert torch.equal(got, again)
    ref = oracle.backward_lut(values, c.dy, c.idx, gpr, c.k, c.task, sets).reshape(got.shape)
    lim = _dlut_bound(c, values, c.task, sets, T).reshape(got.shape)
    err = np.abs(got.cpu().numpy().astype(np.float64) - ref)
    assert (err <= lim).all(), float((err / lim).max())
    # accumulate
    start = torch.full_like(got, 0.25)
    acc = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, sets, out=start.clone(), accumulate=True)
    assert torch.equal(acc, start + got)
    if sets == 1 and T >= 64:
        # the same products and accumulations as the bf16 gradient of the same values;
        # only the order of the 256-column binning (and its tiles' joining) differs
        same = sk.linear_bwd_lut(packed, bits, gpr, sk.ckpt8_dequant(ck), dY)
        assert (np.abs((got - same).cpu().numpy()) <= lim * (1024 * 2.0 ** -24) / ((T / 16 + 512) * 2.0 ** -23)).all()
    assert sk.device_check() == 0


@pytest.mark.parametrize("n,d,bits,gpr,T,sets", [(8, 32, 2, 1, 40, 1), (8, 32, 4, 1, 700, 3), (56, 1280, 4, 8, 4063, 3),
                                                 (32, 512, 4, 8, 962, 1), (40, 64, 3, 2, 16, 8), (600, 32, 2, 1, 90, 2),
                                                 (48, 3712, 4, 4, 17, 8), (24, 160, 3, 5, 5000, 1)])
def test_lut_gradient_of_few_rows_or_columns(n, d, bits, gpr, T, sets):
    """Layers smaller than one tile in either direction."""
    from compressive_fine_tuning_b200 import sk
    c = synth.layer_case(500 + n + T, n=n, d=d, bits=bits, gpr=gpr, T=T, ntask=sets)
    packed, lut, X, dY, task = gc.dev_case(c)
    ck = sk.ckpt8(X)
    values = oo.ckpt8_values(*oo.ckpt8_quantize(c.x))
    got = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, sets)
    ref = oracle.backward_lut(values, c.dy, c.idx, gpr, c.k, c.task, sets).reshape(got.shape)
    assert (np.abs(got.cpu().numpy().astype(np.float64) - ref) <= _dlut_bound(c, values, c.task, sets, T).reshape(got.shape)).all()
    assert torch.equal(got, sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, sets))
    start = torch.full_like(got, 0.25)
    acc = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, sets, out=start.clone(), accumulate=True)
    assert torch.equal(acc, start + got)
    assert sk.device_check() == 0


@pytest.mark.parametrize("T", [1, 9, 15])
def test_few_tokens_of_few_of_the_sets(T):
    """Sets that no token names are zero, or left alone when accumulating; ids out
    of range are flagged on this path too."""
    from compressive_fine_tuning_b200 import sk
    n, d, bits, gpr, sets = 72, 320, 3, 5, 8
    c = synth.layer_case(70 + T, n=n, d=d, bits=bits, gpr=gpr, T=T, ntask=sets)
    packed, lut, X, dY, _ = gc.dev_case(c)
    ck = sk.ckpt8(X)
    names = np.array([5, 2, 5] * 5, dtype=np.int32)[:T]
    task = torch.from_numpy(names).cuda()
    values = oo.ckpt8_values(*oo.ckpt8_quantize(c.x))
    ref = oracle.backward_lut(values, c.dy, c.idx, gpr, c.k, names, sets)
    got = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, sets)
    # T products and additions in fp32 and at most 64 additions of the binning
    mag = oracle.backward_lut(np.abs(values), np.abs(c.dy), c.idx, gpr, c.k, names, sets)
    lim = ((T + 64) * 2.0 ** -23 * mag + 1e-30).reshape(got.shape)
    assert (np.abs(got.cpu().numpy() - ref.reshape(got.shape)) <= lim).all()
    assert not got[[0, 1, 3, 4, 6, 7]].any()
    start = torch.full_like(got, 0.25)
    acc = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, sets, out=start.clone(), accumulate=True)
    assert torch.equal(acc, start + got) and sk.device_check() == 0
    task[0] = sets
    sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, sets)
    assert sk.device_check() == sk.SK_CHECK_TASK_RANGE


def test_lut_gradient_cuda_core_path(monkeypatch):
    from compressive_fine_tuning_b200 import sk
    n, d, bits, gpr, T, sets = 72, 320, 3, 5, 150, 2
    c = synth.layer_case(77, n=n, d=d, bits=bits, gpr=gpr, T=T, ntask=sets)
    packed, lut, X, dY, task = gc.dev_case(c)
    ck = sk.ckpt8(X)
    tc = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, sets)
    monkeypatch.setenv("SK_BWD_PATH", "simt")
    simt = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, sets)
    values = oo.ckpt8_values(*oo.ckpt8_quantize(c.x))
    ref = oracle.backward_lut(values, c.dy, c.idx, gpr, c.k, c.task, sets).reshape(tc.shape)
    lim = _dlut_bound(c, values, c.task, sets, 16 * T).reshape(tc.shape)
    for got in (tc, simt):
        assert (np.abs(got.cpu().numpy() - ref) <= lim).all()


@pytest.mark.parametrize("T", [40, 200])
def test_tasks_without_tokens_and_out_of_range(T):
    """Sets that no token names get zeros; a task id out of range is flagged and
    its token left out; without task ids every token belongs to set 0."""
    from compressive_fine_tuning_b200 import sk
    n, d, bits, gpr = 128, 256, 4, 2
    c = synth.layer_case(31, n=n, d=d, bits=bits, gpr=gpr, T=T)
    packed, lut, X, dY, _ = gc.dev_case(c)
    ck = sk.ckpt8(X)
    task = torch.full((T,), 2, dtype=torch.int32, device="cuda")
    whole = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY)
    got = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, 4)
    assert torch.equal(got[2], whole[0]) and not got[[0, 1, 3]].any()
    none = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, None, 4)
    assert torch.equal(none[0], whole[0]) and not none[1:].any()
    assert sk.device_check() == 0
    task[3] = 9
    task[7] = -1
    bad = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, 4)
    assert sk.device_check() == sk.SK_CHECK_TASK_RANGE
    dY2 = dY.clone()
    dY2[[3, 7]] = 0
    want = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY2, None, 1)
    torch.testing.assert_close(bad[2], want[0], rtol=0, atol=float(want.abs().max()) * T * 2.0 ** -23)


def test_empty_batch():
    from compressive_fine_tuning_b200 import sk
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    ck = sk.ckpt8(x)
    assert ck.q.shape == (0, 64) and ck.scale.shape == (0, 2) and sk.ckpt8_dequant(ck).shape == (0, 64)
    packed = torch.zeros((8, sk.packed_row_bytes(64, 4)), dtype=torch.uint8, device="cuda")
    out = sk.linear_bwd_lut_ckpt8(packed, 4, 1, ck, torch.empty((0, 8), dtype=torch.bfloat16, device="cuda"))
    assert not out.any()


def test_non_finite_block_reaches_only_its_columns():
    """A NaN or an infinity in X makes its 32-column block NaN: the bins its
    columns feed are NaN, every other bin is what it was."""
    from compressive_fine_tuning_b200 import sk
    n, d, bits, gpr, T = 128, 512, 4, 8, 96          # 64 columns per group
    c = synth.layer_case(8, n=n, d=d, bits=bits, gpr=gpr, T=T)
    packed, lut, X, dY, _ = gc.dev_case(c)
    clean = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, sk.ckpt8(X), dY)
    X[50, 130] = float("inf")                        # columns 128..159: group 2
    got = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, sk.ckpt8(X), dY)[0]
    others = [g for g in range(gpr) if g != 2]
    assert torch.equal(got[:, others], clean[0][:, others])
    hit = np.zeros((n, 16), dtype=bool)
    for i in range(n):
        hit[i, c.idx[i, 128:160]] = True
    np.testing.assert_array_equal(torch.isnan(got[:, 2]).cpu().numpy(), hit)


def test_layer_with_checkpoint():
    """SketchedLinear(ckpt8=True): same output and input gradient, the LUT
    gradient of the checkpoint's values, shared checkpoints, no X kept."""
    from compressive_fine_tuning_b200 import sk
    c = synth.layer_case(55, n=256, d=512, bits=4, gpr=2, T=200)
    packed, lut, X, dY, _ = gc.dev_case(c)
    plain = sk.SketchedLinear(packed, lut, 4, 512)
    kept = sk.SketchedLinear(packed, lut, 4, 512, ckpt8=True)
    xs = [X.clone().requires_grad_() for _ in range(3)]
    outs = [plain(xs[0]), kept(xs[1]), kept(xs[2], None, sk.ckpt8(X))]
    grads = []
    for m, x, y in zip((plain, kept, kept), xs, outs):
        m.lut.grad = None
        y.backward(dY)
        grads.append(m.lut.grad.clone())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert torch.equal(xs[0].grad, xs[1].grad) and torch.equal(xs[0].grad, xs[2].grad)
    want = sk.linear_bwd_lut_ckpt8(packed, 4, 2, sk.ckpt8(X), dY)
    assert torch.equal(grads[1], want) and torch.equal(grads[2], want)
    # the checkpoint moves the gradient by no more than its rounding: 2^(e-1) per value
    step = np.repeat(2.0 ** (sk.ckpt8(X).scale.cpu().numpy().astype(np.float64) - 128.0), 32, axis=1)
    lim = oracle.backward_lut(step, np.abs(c.dy), c.idx, 2, 16).reshape(grads[0].shape)
    lim = lim + _dlut_bound(c, np.abs(c.x) + step, None, 1, 200).reshape(grads[0].shape) * 2
    assert (np.abs((grads[1] - grads[0]).cpu().numpy()) <= lim).all()
    # frozen LUTs: nothing is quantised, X still gets its gradient
    kept.lut.requires_grad_(False)
    x = X.clone().requires_grad_()
    kept(x).backward(dY)
    assert torch.equal(x.grad, xs[0].grad)
