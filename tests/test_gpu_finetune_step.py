"""The operators as a fine-tuning step uses them together: norm with checkpoint,
sketched projections that share it, norm, linear cross entropy, LUT update;
captured into graphs, on side streams, and with batches cut into chunks.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import operators_oracle as oo  # noqa: E402
from tests.test_gpu_loss import _bounds, _check  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda(monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    monkeypatch.delenv("SK_BWD_PATH", raising=False)


D, FF, V, T = 256, 512, 1000, 300


def _layer(sk, n, d, seed, sets=1):
    g = torch.Generator().manual_seed(seed)
    idx = torch.randint(0, 16, (n, d), generator=g, dtype=torch.uint8).cuda()
    lut = (torch.randn(sets, n, 2, 16, generator=g) / d ** 0.5).cuda()
    return sk.SketchedLinear(sk.pack(idx, 4), lut.half().float(), 4, d, ckpt8=True), idx


class Step:
    """h -> norm -> (gate, up) -> silu(gate) * up -> down -> + h -> norm -> loss."""

    def __init__(self, sk, sets=1):
        self.sk = sk
        self.n1 = sk.LayerNorm(D, rms=True, dtype=torch.bfloat16, device="cuda")
        self.n2 = sk.LayerNorm(D, device="cuda")
        self.gate, self.gate_idx = _layer(sk, FF, D, 1, sets)
        self.up, self.up_idx = _layer(sk, FF, D, 2, sets)
        self.down, self.down_idx = _layer(sk, D, FF, 3, sets)
        g = torch.Generator().manual_seed(4)
        self.head = (torch.randn(V, D, generator=g) / 4).bfloat16().cuda().requires_grad_()
        self.params = [self.n1.weight, self.gate.lut, self.up.lut, self.down.lut, self.n2.weight, self.n2.bias, self.head]

    def loss(self, h, y, task=None):
        x, ck = self.n1(h, ckpt=True)
        a = torch.nn.functional.silu(self.gate(x, task, ck)) * self.up(x, task, ck)
        return self.sk.linear_cross_entropy(self.n2(h + self.down(a, task)), self.head, y)

    def plain(self, h, y, task=None):
        """The same in float64 from the same parameters, without the roundings in between."""
        ps = [p.detach().double().requires_grad_() for p in self.params]
        w1, lg, lu, ld, w2, b2, head = ps
        H = h.detach().double().requires_grad_()

        def norm(x, w, b, rms):
            c = x if rms else x - x.mean(-1, keepdim=True)
            z = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + 1e-5) * w
            return z if b is None else z + b

        def lin(x, lut, idx):
            n, d = idx.shape
            i = idx.long().view(1, n, 2, d // 2).expand(lut.shape[0], -1, -1, -1)
            theta = torch.gather(lut, 3, i).reshape(lut.shape[0], n, d)
            ys = torch.einsum("td,snd->stn", x, theta)
            return ys[0] if task is None else ys[task.long(), torch.arange(len(x), device=x.device)]

        x = norm(H, w1, None, True)
        a = torch.nn.functional.silu(lin(x, lg, self.gate_idx)) * lin(x, lu, self.up_idx)
        out = norm(H + lin(a, ld, self.down_idx), w2, b2, False)
        loss = torch.nn.functional.cross_entropy(out @ head.T, y)
        return loss, torch.autograd.grad(loss, [H] + ps)


def _inputs(seed=9):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(T, D, generator=g).bfloat16().cuda()
    y = torch.randint(0, V, (T,), generator=g)
    y[::7] = -100
    return h, y.cuda()


def _rel(a, b):
    a, b = a.double(), b.double()
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("sets", [1, 3])
def test_gradients_of_the_step(sets):
    """Against float64 without roundings.  bf16 activations round by 2^-9 in the mean
    square (2^-8 at most) at about eight places on a path, weights once (2^-9), the
    checkpoint by at most 1/127 of a block's largest value, about 0.6 % of a value in
    the mean square: together under 3 % of any gradient's norm."""
    from compressive_fine_tuning_b200 import sk
    s = Step(sk, sets)
    h, y = _inputs()
    task = torch.randint(0, sets, (T,), generator=torch.Generator().manual_seed(5), dtype=torch.int32).cuda() if sets > 1 else None
    hh = h.clone().requires_grad_()
    loss = s.loss(hh, y, task)
    got = torch.autograd.grad(loss, [hh] + s.params)
    ref_loss, ref = s.plain(h, y, task)
    assert abs(float(loss.detach()) - float(ref_loss.detach())) <= 0.01 * float(ref_loss.detach())
    for name, a, b in zip(["h", "n1", "gate", "up", "down", "n2.w", "n2.b", "head"], got, ref):
        assert a.shape == b.shape and _rel(a, b) <= 0.03, (name, _rel(a, b))
    assert sk.device_check() == 0


def test_optimizer_step_runs_and_uses_the_gradients():
    from compressive_fine_tuning_b200 import sk
    s = Step(sk)
    h, y = _inputs()
    s.loss(h, y).backward()
    before = s.gate.lut.detach().clone()
    m, v = torch.zeros_like(before), torch.zeros_like(before)
    grad = s.gate.lut.grad.clone()
    s.gate.adamw_step(m, v, 1, 1e-3)
    # the first AdamW step moves every value by lr against the sign of its gradient
    moved = s.gate.lut.detach() - before
    big = grad.abs() > 1e-6
    assert big.any() and torch.equal(torch.sign(moved)[big], -torch.sign(grad)[big])
    assert torch.equal(s.gate.lut16, s.gate.lut.detach().half())


def test_captured_step_replays_with_new_inputs():
    """Forward and backward in one CUDA graph, replayed on other inputs; two graphs side
    by side keep their own workspaces.  No eager autograd graph of the parameters is
    alive at the capture: PyTorch ties a parameter's accumulation node to the stream
    of the graph that holds it, and a capture on another stream then fails."""
    from compressive_fine_tuning_b200 import sk
    s = Step(sk)
    h, y = _inputs(1)
    wanted = [(torch.autograd.grad(s.loss(*i), s.params), s.loss(*i).detach()) for i in (_inputs(2), _inputs(3))]
    graphs = []
    for _ in range(2):
        hs, ys = h.clone(), y.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(2):
                torch.autograd.grad(s.loss(hs, ys), s.params)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            loss = s.loss(hs, ys)
            grads = torch.autograd.grad(loss, s.params)
        graphs.append((g, hs, ys, loss, grads))
    for (g, hs, ys, _, _), seed in zip(graphs, (2, 3)):
        a, b = _inputs(seed)
        hs.copy_(a)
        ys.copy_(b)
    for g, *_ in graphs:
        g.replay()
    graphs[0][0].replay()
    torch.cuda.synchronize()
    for (g, hs, ys, loss, grads), (want, want_loss) in zip(graphs, wanted):
        assert torch.equal(loss, want_loss)
        for a, b in zip(grads, want):
            assert torch.equal(a, b)
    # and eager steps still run
    again = torch.autograd.grad(s.loss(*_inputs(2)), s.params)
    assert all(torch.equal(a, b) for a, b in zip(again, wanted[0][0]))
    assert sk.device_check() == 0


def test_calls_on_side_streams():
    """Two streams run steps at the same time; each call's workspace is its stream's."""
    from compressive_fine_tuning_b200 import sk
    s = Step(sk)
    ins = [_inputs(k) for k in (11, 12)]
    want = [torch.autograd.grad(s.loss(*i), s.params) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [None, None]
    for rep in range(3):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k] = torch.autograd.grad(s.loss(*ins[k]), s.params)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def _ce64(h, w, y, reduction):
    """(loss, dH, dW) in float64 on the GPU, tokens in pieces."""
    H, W = h.double(), w.double()
    keep = y != -100
    n = max(1, int(keep.sum())) if reduction == "mean" else 1
    losses = torch.zeros(len(y), dtype=torch.float64, device=h.device)
    dH, dW = torch.zeros_like(H), torch.zeros_like(W)
    for a in range(0, len(y), 128):
        k = torch.nonzero(keep[a:a + 128])[:, 0] + a
        z = H[k] @ W.T
        r = torch.arange(len(k), device=h.device)
        losses[k] = torch.logsumexp(z, 1) - z[r, y[k]]
        p = torch.softmax(z, 1)
        p[r, y[k]] -= 1
        p /= n
        dH[k] = p @ W
        dW += p.T @ H[k]
    return losses.sum() / n, dH, dW


@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_cross_entropy_in_chunks_of_tokens(reduction):
    """A vocabulary so large that the buffer of exponentials holds 768 of 1700 tokens:
    three chunks, the mean over all of them, dW summed over them in fp32.  Rounding of
    P (2^-8 of each value at most, 2^-9 in the mean square) and of the outputs:
    0.5 % of the norm, 2^-7 of the largest entry at most."""
    from compressive_fine_tuning_b200 import sk
    g = torch.Generator().manual_seed(0)
    n, v, d = 1700, 300001, 64
    w = (torch.randn(v, d, generator=g) / 4).bfloat16().cuda()
    h = torch.randn(n, d, generator=g).bfloat16().cuda()
    y = torch.randint(0, v, (n,), generator=g)
    y[5::9] = -100
    y = y.cuda()
    loss, dH, dW = sk.cross_entropy(h, w, y, reduction=reduction, need_dh=True, need_dw=True)
    rl, rh, rw = _ce64(h, w, y, reduction)
    assert abs(float(loss) - float(rl)) <= 1e-5 * float(rl)
    for a, b in ((dH, rh), (dW, rw)):
        assert _rel(a, b) <= 0.005
        assert float((a.double() - b).abs().max()) <= 2.0 ** -7 * float(b.abs().max())
    again = sk.cross_entropy(h, w, y, reduction=reduction, need_dh=True, need_dw=True)
    assert all(torch.equal(p, q) for p, q in zip(again, (loss, dH, dW)))
    # each gradient alone (without dW no fp32 sums are kept): the same
    assert torch.equal(sk.cross_entropy(h, w, y, reduction=reduction, need_dh=True)[1], dH)
    assert torch.equal(sk.cross_entropy(h, w, y, reduction=reduction, need_dw=True, need_loss=False)[2], dW)


def test_loss_of_many_tokens_without_gradients():
    """More tokens than one launch takes when only the loss is wanted (32768)."""
    from compressive_fine_tuning_b200 import sk
    g = torch.Generator().manual_seed(0)
    n, v, d = 33000, 300, 64
    w = torch.randn(v, d, generator=g).bfloat16().cuda()
    h = torch.randn(n, d, generator=g).bfloat16().cuda()
    y = torch.randint(0, v, (n,), generator=g)
    y[::11] = -100
    z = h.double() @ w.double().T
    keep = (y != -100).cuda()
    ref = torch.logsumexp(z, 1) - z.gather(1, y.clamp(min=0).cuda()[:, None])[:, 0]
    ref = torch.where(keep, ref, 0.0)
    y = y.cuda()
    each = sk.linear_cross_entropy(h, w, y, reduction="none")
    assert float((each.double() - ref).abs().max()) <= 1e-5 * float(z.abs().max())
    for red, want in (("sum", ref.sum()), ("mean", ref.sum() / keep.sum())):
        assert abs(float(sk.linear_cross_entropy(h, w, y, reduction=red)) - float(want)) <= 1e-5 * float(want)


def test_inputs_are_not_written():
    """No call writes its inputs, and rows outside a view stay as they were."""
    from compressive_fine_tuning_b200 import sk
    big = torch.randn(40, 256, device="cuda").bfloat16()
    kept = big.clone()
    x = big[8:24]
    w = torch.rand(256, device="cuda")
    y, mean, rstd, ck = sk.layer_norm_fwd(x, w, w, ckpt=True)
    sk.layer_norm_bwd(y, x, w, mean, rstd)
    sk.ckpt8(x)
    head = big[24:40]
    sk.cross_entropy(x, head, torch.arange(16, device="cuda"), need_dh=True, need_dw=True)
    torch.cuda.synchronize()
    assert torch.equal(big, kept)


def test_same_tensor_twice_and_refusals_on_the_device():
    from compressive_fine_tuning_b200 import sk
    x = torch.randn(16, 64, device="cuda").bfloat16()
    # hidden states and head may be one tensor (tied), the norm's weight and bias too
    loss, dH, dW = sk.cross_entropy(x, x, torch.arange(16, device="cuda"), need_dh=True, need_dw=True)
    # every token is its own class with a logit of about 64 over the others: gradients of
    # 1e-20, which fp16 exponentials hold as zero (2^-24 of the row's largest, in _bounds)
    X = x.double().cpu().numpy()
    rl, rh, rw, P = oo.cross_entropy(X, X, np.arange(16), -100, "mean")
    _, lim_h, lim_w = _bounds(X, X, P, np.full(16, 1 / 16), rh, rw)
    assert abs(float(loss) - rl) <= 1e-5 * (1 + abs(rl))
    _check(dH, rh, lim_h, "dH")
    _check(dW, rw, lim_w, "dW")
    with pytest.raises(sk.SketchError):
        sk.layer_norm_fwd(torch.zeros(2, 40000, device="cuda"), torch.zeros(40000, device="cuda"))
    with pytest.raises(sk.SketchError):
        sk.cross_entropy(torch.zeros(2, 12, device="cuda").bfloat16(), torch.zeros(3, 12, device="cuda").bfloat16(),
                         torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        sk.layer_norm_fwd(x.t(), torch.zeros(16, device="cuda").bfloat16())
    with pytest.raises(ValueError):
        sk.ckpt8(x[:, :48].contiguous())
    with pytest.raises(ValueError):
        sk.linear_cross_entropy(x, x, torch.zeros(16, dtype=torch.int64, device="cuda"), reduction="max")


def test_offsets_beyond_32_bits():
    """Tensors of more than 2^31 values: the last rows come out as they do alone.
    Two roundings to bf16 lie between two ways of summing a row: 2^-7 of the value."""
    from compressive_fine_tuning_b200 import sk
    d, rows, last = 4096, 540000, 64
    near = lambda a, b, slack: bool(((a.double() - b.double()).abs() <= 2.0 ** -7 * b.double().abs() + slack).all())  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.zeros(rows, d, device="cuda", dtype=torch.bfloat16)
    assert x.numel() > 2 ** 31
    x[-last:] = torch.randn(last, d, device="cuda", generator=g).bfloat16()
    w = torch.rand(d, device="cuda", generator=g) + 0.5
    tail = x[-last:].clone()
    y, mean, rstd, ck = sk.layer_norm_fwd(x, w, w, ckpt=True)
    ys = sk.layer_norm_fwd(tail, w, w)[0]
    assert near(y[-last:], ys, 1e-5) and near(y[:2], w.expand(2, d), 0.0)
    alone = sk.ckpt8(y[-last:].clone())
    assert torch.equal(ck.q[-last:], alone.q) and torch.equal(ck.scale[-last:], alone.scale)
    whole = sk.ckpt8(y)
    assert torch.equal(whole.q[-last:], alone.q) and torch.equal(whole.scale, ck.scale)
    del y
    assert torch.equal(sk.ckpt8_dequant(ck)[-last:], sk.ckpt8_dequant(alone))
    dy = torch.zeros_like(x)
    dy[-last:] = torch.randn(last, d, device="cuda", generator=g).bfloat16()
    dx, dw, db = sk.layer_norm_bwd(dy, x, w, mean, rstd)
    # the other rows' dy is zero: the sums are the last rows'
    sx, sw, sb = sk.layer_norm_bwd(dy[-last:].clone(), tail, w, mean[-last:].clone(), rstd[-last:].clone())
    assert near(dx[-last:], sx, 1e-5) and not dx[:2].any()
    assert near(dw, sw, 1e-3) and near(db, sb, 1e-3)
    del dx, dy
    # a LUT gradient over that many tokens: those with a gradient are the last
    n = 64
    idx = torch.randint(0, 4, (n, d), device="cuda", generator=g, dtype=torch.uint8)
    packed = sk.pack(idx, 2)
    dY = torch.zeros(rows, n, device="cuda", dtype=torch.bfloat16)
    dY[-last:] = torch.randn(last, n, device="cuda", generator=g).bfloat16()
    got = sk.linear_bwd_lut_ckpt8(packed, 2, 2, ck, dY)
    want = sk.linear_bwd_lut_ckpt8(packed, 2, 2, alone, dY[-last:].clone())
    assert near(got, want, 1e-3 * float(want.abs().max()))
    del ck, whole, got
    # many tokens' losses, and a head of that many values with its gradient
    y = torch.randint(0, 40, (rows,), device="cuda", generator=g)
    small = (torch.randn(40, d, device="cuda", generator=g) / 8).bfloat16()
    each = sk.cross_entropy(x, small, y, reduction="none")[0]
    assert near(each[-last:], sk.cross_entropy(tail, small, y[-last:].clone(), reduction="none")[0], 1e-4)
    y = torch.arange(rows - last, rows, device="cuda")
    loss, dH, dW = sk.cross_entropy(tail, x, y, need_dh=True, need_dw=True, reduction="sum")
    # every row of the head but the last 64 is zero: their logits are 0
    z = tail.double() @ tail.double().T
    lse = torch.logsumexp(torch.cat([z, z.new_full((last, 1), np.log(rows - last))], 1), 1)
    assert abs(float(loss) - float((lse - z.diagonal()).sum())) <= 1e-5 * float(lse.sum())
    p = torch.softmax(torch.cat([z, z.new_full((last, 1), np.log(rows - last))], 1), 1)[:, :last] - torch.eye(last, device="cuda")
    # logits of up to 4500 in fp32: an error of 2^-23 of them in the exponent
    assert float((dW[-last:].double() - p.T @ tail.double()).abs().max()) <= 2.0 ** -6 and dW[:2].isfinite().all()
    assert float((dH.double() - p @ tail.double()).abs().max()) <= 2.0 ** -6
    assert sk.device_check() == 0
