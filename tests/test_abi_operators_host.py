"""Host-side validation of the norm, checkpoint and cross-entropy calls: bad
arguments are rejected before anything touches a device (no GPU needed), by the
C ABI and by the Python binding."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from compressive_fine_tuning_b200 import sk

OK, INVALID, UNSUPPORTED, CUDA = 0, 1, 2, 3
BIG = 1 << 30                     # room between the fake device addresses below
A, B, C, D, E, F, G, H = (0x1000000000 + i * (BIG * 16) for i in range(8))


def _rejected(status):
    assert status == INVALID
    assert sk.lib.sk_last_error() != b""


# ---- norms ------------------------------------------------------------------

def fwd(x=A, xt=sk.SK_BF16, T=4, d=64, w=B, b=None, wt=sk.SK_BF16, eps=1e-5, rms=0, y=C, mean=D, rstd=E, q=None,
        scale=None):
    return sk.lib.sk_layer_norm_fwd(x, xt, T, d, w, b, wt, eps, rms, y, mean, rstd, q, scale, None)


def bwd(dy=A, x=B, xt=sk.SK_BF16, T=4, d=64, w=C, wt=sk.SK_BF16, mean=D, rstd=E, rms=0, dx=F, dw=G, db=H, ws=A + BIG * 8,
        nb=BIG):
    return sk.lib.sk_layer_norm_bwd(dy, x, xt, T, d, w, wt, mean, rstd, rms, dx, dw, db, ws, nb, None)


@pytest.mark.parametrize("kw", [
    dict(xt=3), dict(xt=-1), dict(wt=sk.SK_F16), dict(xt=sk.SK_F32), dict(d=0), dict(d=32769), dict(T=-1), dict(T=1 << 31),
    dict(rms=2)])
@pytest.mark.parametrize("call", [fwd, bwd])
def test_norm_shapes(call, kw):
    _rejected(call(**kw))


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(w=None), dict(y=None), dict(eps=-1e-5), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(x=A + 8), dict(y=C + 4), dict(w=B + 2), dict(y=A), dict(y=A + 16), dict(mean=C + 16), dict(q=F), dict(scale=F),
    dict(q=F, scale=G, d=48), dict(q=F, scale=G, xt=sk.SK_F16, wt=sk.SK_F16), dict(q=C + 32, scale=G), dict(b=B + 8),
    dict(q=F, scale=F + 16)])
def test_norm_forward_arguments(kw):
    _rejected(fwd(**kw))


@pytest.mark.parametrize("kw", [
    dict(dy=None), dict(x=None), dict(w=None), dict(rstd=None), dict(mean=None), dict(dx=A), dict(dx=B + 32), dict(dw=C),
    dict(db=G), dict(ws=None), dict(nb=0), dict(ws=F), dict(ws=A + BIG * 8 + 4), dict(dx=F + 8)])
def test_norm_backward_arguments(kw):
    _rejected(bwd(**kw))


def test_norm_empty_calls():
    assert fwd(T=0, x=None, w=None, y=None) == OK
    assert bwd(dx=None, dw=None, db=None, ws=None, nb=0) == OK
    assert bwd(T=0, dw=None, db=None) == OK
    assert sk.lib.sk_layer_norm_bwd_workspace_bytes(0, 64) == 0
    assert sk.lib.sk_layer_norm_bwd_workspace_bytes(8, 0) == 0
    for T, d in ((1, 1), (7, 4096), (100000, 8192), (5, 32768)):
        need = sk.lib.sk_layer_norm_bwd_workspace_bytes(T, d)
        assert need >= 8 * d and need % (8 * d) == 0


# ---- checkpoints ------------------------------------------------------------

def quant(X=A, T=4, d=64, q=B, scale=C):
    return sk.lib.sk_ckpt8_quantize(X, T, d, q, scale, None)


def dequant(X=A, T=4, d=64, q=B, scale=C):
    return sk.lib.sk_ckpt8_dequantize(q, scale, T, d, X, None)


@pytest.mark.parametrize("call", [quant, dequant])
@pytest.mark.parametrize("kw", [dict(d=0), dict(d=48), dict(T=-1), dict(X=None), dict(q=None), dict(scale=None),
                                dict(X=A + 2), dict(q=A + 128), dict(scale=B + 16), dict(scale=C + 1)])
def test_checkpoint_arguments(call, kw):
    _rejected(call(**kw))
    assert call(T=0, X=None, q=None, scale=None) == OK


def lut8(packed=A, bits=4, gpr=1, n=256, d=512, q=B, scale=C, dY=D, T=100, task=None, ntask=1, dlut=E, acc=0, ws=F, nb=BIG):
    return sk.lib.sk_linear_bwd_lut_ckpt8(packed, bits, gpr, n, d, q, scale, dY, T, task, ntask, dlut, acc, ws, nb, None)


@pytest.mark.parametrize("kw", [
    dict(bits=1), dict(bits=5), dict(n=12), dict(d=48), dict(gpr=3), dict(gpr=32), dict(T=-1), dict(ntask=0),
    dict(packed=None), dict(q=None), dict(scale=None), dict(dY=None), dict(dlut=None), dict(acc=2), dict(scale=C + 1),
    dict(q=B + 8), dict(dlut=B), dict(dlut=C), dict(dlut=D + 64), dict(ws=None), dict(nb=64), dict(ws=F + 4), dict(ws=B),
    dict(ws=E), dict(ws=A)])
def test_lut_gradient_arguments(kw):
    _rejected(lut8(**kw))


def test_lut_gradient_workspace():
    size = lambda **kw: sk.workspace_bytes(sk.SK_OP_BWD_LUT_CKPT8, *[{**dict(n=256, d=512, bits=4, gpr=1, T=100, ntask=1), **kw}[k]  # noqa: E731
                                           for k in ("n", "d", "bits", "gpr", "T", "ntask")])
    assert size() >= 100 * 512 * 2                  # X as bf16 and the partial bins
    assert size(T=1) == 0 and size(n=8, T=15) == 0  # the CUDA-core path needs none
    assert size(ntask=3) >= size()                  # task ids may be missing: enough for one set, too
    # routed dY, X in bf16 and three sets' bins, once there are tokens enough
    assert size(ntask=3, T=5000) >= 5000 * (256 + 512) * 2 + 3 * 256 * 16 * 4
    assert size(ntask=300) == 0                     # more sets than the routing takes
    assert lut8(T=1, ws=None, nb=0) in (CUDA, UNSUPPORTED, OK)
    assert sk.workspace_bytes(4, 256, 512, 4, 1, 100, 1) == 0
    assert lut8(T=0, acc=1) == OK


# ---- cross entropy ----------------------------------------------------------

def ce(h=A, w=B, y=C, bits=64, T=4, V=100, d=64, ignore=-100, red=sk.SK_CE_MEAN, dloss=None, loss=D, dH=E, dW=F, ws=G, nb=BIG):
    return sk.lib.sk_cross_entropy(h, w, y, bits, T, V, d, ignore, red, dloss, loss, dH, dW, ws, nb, None)


@pytest.mark.parametrize("kw", [
    dict(bits=16), dict(T=-1), dict(T=1 << 31), dict(V=0), dict(V=1 << 24), dict(d=0), dict(d=12), dict(d=1 << 20),
    dict(red=3), dict(red=-1), dict(h=None), dict(w=None), dict(y=None), dict(ws=None), dict(nb=16), dict(ws=G + 8),
    dict(h=A + 8), dict(dH=A), dict(dW=B + 32), dict(dH=E + 2), dict(dW=E), dict(loss=A + 4), dict(ws=E), dict(ws=C),
    dict(dloss=E + 4), dict(y=C + 4), dict(dloss=F + 2), dict(loss=F + 2)])
def test_cross_entropy_arguments(kw):
    _rejected(ce(**kw))


def test_cross_entropy_empty_calls():
    assert ce(loss=None, dH=None, dW=None, ws=None, nb=0) == OK
    assert ce(T=0, loss=None, dW=None) == OK
    size = sk.lib.sk_cross_entropy_workspace_bytes
    assert size(0, 100, 64, 1, 1) == 0 and size(4, 100, 60, 1, 1) == 0 and size(4, 1 << 24, 64, 0, 0) == 0
    # the exponentials of one chunk bound the workspace: it stops growing with the tokens
    small, large = size(8192, 32000, 4096, 1, 0), size(1 << 20, 32000, 4096, 1, 0)
    assert large - small < (64 << 20)
    assert size(1 << 20, 32000, 4096, 0, 0) < (80 << 20)   # 32768 tokens' tile statistics and all losses


def test_scale_arguments():
    s = sk.lib.sk_scale_bf16
    for args in ((A, 12, B, 8, C), (A, -8, B, 8, C), (None, 8, B, 8, C), (A, 8, None, 8, C), (A, 8, B, 8, None),
                 (A + 2, 8, B, 8, C), (A, 64, A + 16, 64, C), (A, 64, B, 64, A + 4)):
        _rejected(s(*args, None))
    assert s(None, 0, None, 0, None, None) == OK


# ---- without a device -------------------------------------------------------

def test_valid_calls_without_a_device_fail_loudly():
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    for st in (fwd(), bwd(), quant(), dequant(), lut8(), ce(), sk.lib.sk_scale_bf16(A, 8, B, 8, C, None)):
        assert st in (CUDA, UNSUPPORTED)


# ---- the binding's own checks (CPU tensors never reach the library) ---------

def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("call", [
    lambda: sk.layer_norm_fwd(_bf(4, 64), _bf(64)),
    lambda: sk.ckpt8(_bf(4, 64)),
    lambda: sk.ckpt8_dequant(sk.Ckpt8(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8))),
    lambda: sk.cross_entropy(_bf(4, 64), _bf(10, 64), torch.zeros(4, dtype=torch.int64)),
    lambda: sk.linear_cross_entropy(_bf(4, 64), _bf(10, 64), torch.zeros(4, dtype=torch.int64)),
])
def test_cpu_tensors_are_refused(call):
    with pytest.raises(ValueError, match="CUDA"):
        call()


@pytest.mark.parametrize("call", [
    lambda: sk.layer_norm_fwd(torch.zeros(4, 64, dtype=torch.float64), torch.zeros(64)),
    lambda: sk.layer_norm(torch.zeros(4, 64, dtype=torch.int32), torch.zeros(64)),
    lambda: sk.ckpt8(torch.zeros(4, 64)),
    lambda: sk.cross_entropy(torch.zeros(4, 64), _bf(10, 64), torch.zeros(4, dtype=torch.int64)),
])
def test_wrong_types_are_refused(call):
    with pytest.raises(TypeError):
        call()


def test_target_shape_is_checked():
    with pytest.raises(ValueError, match="class per token"):
        sk.linear_cross_entropy(_bf(2, 4, 64), _bf(10, 64), torch.zeros(8, dtype=torch.int64))
