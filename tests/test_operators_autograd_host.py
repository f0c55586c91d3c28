"""What the autograd front ends of the norm, the loss and the layer decide on the
host.  The library calls are replaced by stubs that return empty results, so that
nothing here needs a device."""
import contextlib

import pytest

torch = pytest.importorskip("torch")
import torch.autograd.forward_ad as fwad  # noqa: E402

from compressive_fine_tuning_b200 import sk  # noqa: E402


@pytest.fixture
def stubs(monkeypatch):
    def norm(x, weight, bias=None, eps=1e-5, rms=False, ckpt=False, stats=True):
        ck = sk.Ckpt8(torch.zeros(x.shape, dtype=torch.int8),
                      torch.zeros((x.shape[0], x.shape[1] // 32), dtype=torch.uint8)) if ckpt else None
        return torch.zeros(x.shape), torch.zeros(x.shape[0]), torch.ones(x.shape[0]), ck

    def loss(H, W, target, ignore_index=-100, reduction="mean", dloss=None, need_loss=True, need_dh=False, need_dw=False):
        return (torch.zeros(H.shape[0] if reduction == "none" else ()), torch.zeros(H.shape) if need_dh else None,
                torch.zeros(W.shape) if need_dw else None)

    monkeypatch.setattr(sk, "layer_norm_fwd", norm)
    monkeypatch.setattr(sk, "cross_entropy", loss)


# ---- forward-mode derivatives: none of the operators has one, so they refuse -------

@pytest.mark.parametrize("which", ["x", "weight", "bias"])
@pytest.mark.parametrize("mode", [contextlib.nullcontext, torch.no_grad])
@pytest.mark.parametrize("ckpt", [False, True])
def test_layer_norm_refuses_a_tangent(stubs, which, mode, ckpt):
    args = {"x": torch.randn(2, 3, 64), "weight": torch.ones(64), "bias": torch.zeros(64)}
    with mode(), fwad.dual_level():
        plain = sk.layer_norm(**args, ckpt=ckpt)            # no tangent anywhere: the level alone changes nothing
        assert (plain[0] if ckpt else plain).shape == (2, 3, 64)
        args[which] = fwad.make_dual(args[which], torch.ones_like(args[which]))
        with pytest.raises(NotImplementedError):
            sk.layer_norm(**args, ckpt=ckpt)


@pytest.mark.parametrize("which", ["H", "W"])
@pytest.mark.parametrize("mode", [contextlib.nullcontext, torch.no_grad])
@pytest.mark.parametrize("reduction", ["none", "mean"])
def test_linear_cross_entropy_refuses_a_tangent(stubs, which, mode, reduction):
    args = {"H": torch.randn(5, 64), "W": torch.randn(9, 64)}
    target = torch.arange(5)
    with mode(), fwad.dual_level():
        assert sk.linear_cross_entropy(**args, target=target, reduction=reduction).numel() == (5 if reduction == "none" else 1)
        args[which] = fwad.make_dual(args[which], torch.ones_like(args[which]))
        with pytest.raises(NotImplementedError):
            sk.linear_cross_entropy(**args, target=target, reduction=reduction)


def test_backward_passes_refuse_a_tangent_of_the_incoming_gradient(stubs):
    x = torch.randn(4, 64, requires_grad=True)
    h = torch.randn(5, 64, requires_grad=True)
    y = sk.layer_norm(x, torch.ones(64))
    loss = sk.linear_cross_entropy(h, torch.randn(9, 64), torch.arange(5))
    with fwad.dual_level():
        for out, leaf in ((y, x), (loss, h)):
            with pytest.raises(NotImplementedError):
                torch.autograd.grad(out, leaf, fwad.make_dual(torch.ones(out.shape), torch.ones(out.shape)))


# ---- the layer that keeps its input in 8 bits --------------------------------------

@pytest.fixture
def layer(monkeypatch):
    """A SketchedLinear on the CPU, and the calls that it makes."""
    calls = []

    def fwd(packed, lut, bits, X, task=None, **kw):
        calls.append("fwd")
        return torch.zeros((X.shape[0], lut.shape[1]), dtype=torch.bfloat16)

    def ckpt8(X):
        calls.append("ckpt8")
        return sk.Ckpt8(torch.zeros(X.shape, dtype=torch.int8),
                        torch.zeros((X.shape[0], X.shape[1] // 32), dtype=torch.uint8))

    monkeypatch.setattr(sk, "linear_fwd", fwd)
    monkeypatch.setattr(sk, "ckpt8", ckpt8)
    packed = torch.zeros((64, sk.packed_row_bytes(96, 4)), dtype=torch.uint8)
    return sk.SketchedLinear(packed, torch.zeros(1, 64, 3, 16), 4, 96, ckpt8=True), calls


def _x(T=5, d=96, grad=True):
    return torch.randn(T, d).to(torch.bfloat16).requires_grad_(grad)


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_no_checkpoint_is_made_where_no_gradient_follows(layer, mode):
    m, calls = layer
    with mode():
        m(_x())
    assert calls == ["fwd"]
    m.lut.requires_grad_(False)
    m(_x())
    assert calls == ["fwd"] * 2
    m.lut.requires_grad_(True)
    m(_x(grad=False))
    assert calls == ["fwd"] * 3 + ["ckpt8"]


def _ck(T=5, d=96, q=torch.int8, scale=torch.uint8, groups=None, device="cpu"):
    return sk.Ckpt8(torch.zeros((T, d), dtype=q, device=device),
                    torch.zeros((T, groups if groups is not None else d // 32), dtype=scale, device=device))


@pytest.mark.parametrize("mode", [contextlib.nullcontext, torch.no_grad])
@pytest.mark.parametrize("ck,error", [
    (_ck(T=4), ValueError), (_ck(d=64), ValueError), (_ck(groups=4), ValueError), (_ck(groups=0), ValueError),
    (_ck(q=torch.uint8), TypeError), (_ck(scale=torch.int8), TypeError), (_ck(q=torch.float32), TypeError),
    (sk.Ckpt8(_ck().q, _ck(T=6).scale), ValueError), (_ck(device="meta"), ValueError),
    (sk.Ckpt8(_ck().q, _ck(device="meta").scale), ValueError), (sk.Ckpt8(_ck().q, None), TypeError)])
def test_a_checkpoint_that_does_not_fit_is_refused_before_the_forward_pass(layer, mode, ck, error):
    m, calls = layer
    with mode(), pytest.raises(error):
        m(_x(), None, ck)
    assert not calls


def test_a_part_of_a_checkpoint_is_taken(layer, monkeypatch):
    """Rows of a longer batch's checkpoint: their scales start at any byte."""
    m, calls = layer
    whole = sk.Ckpt8(torch.arange(9 * 96).to(torch.int8).reshape(9, 96), torch.arange(27).to(torch.uint8).reshape(9, 3))
    part = sk.Ckpt8(whole.q[2:7], whole.scale[2:7])
    assert part.scale.data_ptr() % 16
    got = []

    def bwd(packed, bits, gpr, ck, dY, task=None, ntask=1, **kw):
        got.append(ck)
        return torch.zeros((ntask, 64, gpr, 16))

    monkeypatch.setattr(sk, "linear_bwd_lut_ckpt8", bwd)
    m(_x(grad=False), None, part).backward(torch.ones((5, 64), dtype=torch.bfloat16))
    assert calls == ["fwd"]
    assert torch.equal(got[0].q, part.q) and torch.equal(got[0].scale, part.scale)
    assert got[0].q.data_ptr() % 16 == 0 and got[0].scale.data_ptr() % 16 == 0


@pytest.mark.parametrize("own", [False, True])
def test_the_layer_keeps_its_input_in_8_bits_only(layer, own):
    m, _ = layer
    saved = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: saved.append(t) or t, lambda t: t):
        m(_x(), None, _ck() if own else None)
    kept = [t for t in saved if t.dim() == 2 and t.shape[0] == 5]
    assert sorted(str(t.dtype) for t in kept) == ["torch.int8", "torch.uint8"]
    assert sum(t.numel() * t.element_size() for t in kept) == 5 * 96 * 33 // 32
    m.lut.requires_grad_(False)                         # and none where only X's gradient is wanted
    saved.clear()
    with torch.autograd.graph.saved_tensors_hooks(lambda t: saved.append(t) or t, lambda t: t):
        m(_x(), None, _ck() if own else None)
    assert not [t for t in saved if t.dim() == 2 and t.shape[0] == 5]
