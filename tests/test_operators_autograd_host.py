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
