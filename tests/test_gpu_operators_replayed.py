"""Operators in CUDA graphs that hold a part of a step."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def test_backward_captured_without_its_forward_pass_replays():
    """A backward pass in a graph of its own gives the same gradients at every
    replay, and those of the factor that its buffer holds then."""
    from compressive_fine_tuning_b200 import sk
    g = torch.Generator().manual_seed(3)
    h = torch.randn(70, 64, generator=g).bfloat16().cuda().requires_grad_()
    w = (torch.randn(300, 64, generator=g) / 8).bfloat16().cuda().requires_grad_()
    y = torch.randint(0, 300, (70,), generator=g).cuda()
    plain = torch.autograd.grad(sk.linear_cross_entropy(h, w, y), [h, w])
    factor = torch.tensor(0.5, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        loss = sk.linear_cross_entropy(h, w, y)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = torch.autograd.grad(loss, [h, w], factor, retain_graph=True)
    for f in (0.5, 0.5, 2.0, 0.25):                     # powers of two: exact in every rounding
        factor.fill_(f)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, plain):
            assert torch.equal(a.float(), f * b.float()), f
    with torch.cuda.stream(side):                       # and outside the graph
        for a, b in zip(torch.autograd.grad(loss, [h, w], torch.tensor(4.0, device="cuda")), plain):
            assert torch.equal(a.float(), 4.0 * b.float())
    assert sk.device_check() == 0


def test_forward_and_backward_in_graphs_of_their_own():
    """The two passes of a step captured one after the other and replayed in turn."""
    from compressive_fine_tuning_b200 import sk
    g = torch.Generator().manual_seed(4)
    draws = [torch.randn(70, 64, generator=g).bfloat16().cuda() for _ in range(3)]
    w = (torch.randn(300, 64, generator=g) / 8).bfloat16().cuda().requires_grad_()
    y = torch.randint(0, 300, (70,), generator=g).cuda()
    h = draws[0].clone().requires_grad_()
    factor = torch.tensor(0.5, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first, stream=side):
        loss = sk.linear_cross_entropy(h, w, y)
    with torch.cuda.graph(second, pool=first.pool(), stream=side):
        got = torch.autograd.grad(loss, [h, w], factor)
    for k, f in ((1, 0.5), (2, 2.0), (1, 0.25), (0, 1.0)):
        with torch.no_grad():
            h.copy_(draws[k])
        factor.fill_(f)
        first.replay()
        second.replay()
        torch.cuda.synchronize()
        hk = draws[k].clone().requires_grad_()
        want = sk.linear_cross_entropy(hk, w, y)
        assert torch.equal(loss, want)
        for a, b in zip(got, torch.autograd.grad(want, [hk, w])):
            assert torch.equal(a.float(), f * b.float()), f
    assert sk.device_check() == 0
