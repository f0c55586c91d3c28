"""The LUT gradient from a checkpoint with many LUT sets, on both paths: the
tensor cores, which take the sets in blocks, and the CUDA cores, which walk the
tokens of the sets that have some."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from compressive_fine_tuning_b200 import synth  # noqa: E402
from oracle import operators_oracle as oo  # noqa: E402
from tests import gpu_cases as gc  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("path", ["", "tc", "simt"])
@pytest.mark.parametrize("n,d,bits,gpr,T,sets", [
    (64, 96, 2, 1, 16, 64), (72, 320, 3, 5, 40, 64), (136, 1280, 4, 1, 33, 100), (264, 512, 4, 2, 31, 256),
    (256, 512, 3, 1, 65, 256), (80, 96, 4, 3, 300, 256), (40, 64, 3, 2, 17, 300), (40, 1056, 3, 1, 90, 300)])
def test_many_sets(monkeypatch, n, d, bits, gpr, T, sets, path):
    """T / 16 accumulations of sixteen products on the tensor cores, or T on the CUDA
    cores, and at most 512 additions of the binning, each off by less than 2^-23
    of the sum of magnitudes."""
    from compressive_fine_tuning_b200 import sk
    if path:
        monkeypatch.setenv("SK_BWD_PATH", path)
    else:
        monkeypatch.delenv("SK_BWD_PATH", raising=False)
    c = synth.layer_case(300 + n + T, n=n, d=d, bits=bits, gpr=gpr, T=T, ntask=sets)
    names = c.task.copy()
    names[T // 2:] = names[:T - T // 2]                   # sets with several tokens, far apart and next to each other
    names[1] = names[0]
    packed, lut, X, dY, _ = gc.dev_case(c)
    task = torch.from_numpy(names).cuda()
    ck = sk.ckpt8(X)
    values = oo.ckpt8_values(*oo.ckpt8_quantize(c.x))
    got = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, sets)
    ref = oracle.backward_lut(values, c.dy, c.idx, gpr, c.k, names, sets).reshape(got.shape)
    mag = oracle.backward_lut(np.abs(values), np.abs(c.dy), c.idx, gpr, c.k, names, sets).reshape(got.shape)
    err = np.abs(got.cpu().numpy().astype(np.float64) - ref)
    assert (err <= (T + 512) * 2.0 ** -23 * mag + 1e-30).all()
    unnamed = np.setdiff1d(np.arange(sets), names)
    assert not got[torch.from_numpy(unnamed).cuda()].any()
    start = torch.full_like(got, 0.25)
    acc = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, sets, out=start.clone(), accumulate=True)
    assert torch.equal(acc, start + got)
    assert torch.equal(got, sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, sets))
    assert sk.device_check() == 0
    # ids out of range: flagged, and their tokens in no set
    task[[2, T - 1]] = torch.tensor([sets, -1], dtype=torch.int32, device="cuda")
    some = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, sets)
    assert sk.device_check() == sk.SK_CHECK_TASK_RANGE
    kept = names.copy()
    kept[[2, T - 1]] = -1
    ref = oracle.backward_lut(values, c.dy * (kept >= 0)[:, None], c.idx, gpr, c.k, names, sets).reshape(got.shape)
    assert (np.abs(some.cpu().numpy() - ref) <= (T + 512) * 2.0 ** -23 * mag + 1e-30).all()


def test_blocks_of_sets(monkeypatch):
    """More LUT sets than the partial bins' room holds: the sets go through it in
    blocks.  A set's numbers are those of a call for its tokens alone."""
    from compressive_fine_tuning_b200 import sk
    monkeypatch.setenv("SK_BWD_PATH", "tc")
    n, d, bits, gpr, T, sets = 2048, 4608, 4, 16, 300, 256
    one = 18 * n * 2 * 16 * 4                             # column tiles, rows, group slots, bins, fp32
    block = (512 << 20) // one
    rest = T + sets * 63
    room = sk.workspace_bytes(sk.SK_OP_BWD_LUT_CKPT8, n, d, bits, gpr, T, sets)
    assert 1 < block < sets and block * one <= room <= (512 << 20) + rest * (2 * n + 2 * d + 4) + sets * 8 + 4096
    c = synth.layer_case(41, n=n, d=d, bits=bits, gpr=gpr, T=T)
    packed, lut, X, dY, _ = gc.dev_case(c)
    ck = sk.ckpt8(X)
    named = [0, 1, block - 1, block, block + 1, 2 * block - 1, 2 * block, sets - 1]
    g = torch.Generator().manual_seed(2)
    task = torch.tensor(named, dtype=torch.int32)[torch.randint(0, len(named), (T,), generator=g)].cuda()
    got = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, sets)
    for k in range(sets):
        if k not in named:
            assert not got[k].any(), k
            continue
        own = (task == k).nonzero()[:, 0]
        alone = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, sk.ckpt8(X[own].contiguous()), dY[own].contiguous())
        assert torch.equal(got[k], alone[0]), k
    acc = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, task, sets, out=torch.full_like(got, 0.25), accumulate=True)
    assert torch.equal(acc, 0.25 + got)
    assert sk.device_check() == 0


@pytest.mark.parametrize("T", [16, 40, 150])
def test_many_sets_without_task_ids(T):
    """All tokens are set 0's: the numbers, and the path, of a call for one set."""
    from compressive_fine_tuning_b200 import sk
    n, d, bits, gpr, sets = 520, 1056, 4, 1, 256
    c = synth.layer_case(60 + T, n=n, d=d, bits=bits, gpr=gpr, T=T)
    packed, lut, X, dY, _ = gc.dev_case(c)
    ck = sk.ckpt8(X)
    whole = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY)
    got = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, None, sets)
    assert torch.equal(got[0], whole[0]) and not got[1:].any()
    acc = sk.linear_bwd_lut_ckpt8(packed, bits, gpr, ck, dY, None, sets, out=torch.full_like(got, 0.25), accumulate=True)
    assert torch.equal(acc, 0.25 + got) and sk.device_check() == 0
