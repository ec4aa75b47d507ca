"""Captured backwards of the differentiable packed calls beside an eager graph
that lives on: which are refused, and which go through and replay."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def rand(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def replays(run, want):
    """Capture run() and check every replay against want."""
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def linear_case(gpu_lib, between):
    x, w = rand((64, 32), 1, torch.float32), rand((96, 32), 2)
    leaves = (x.requires_grad_(True), w.requires_grad_(True))
    gy = rand((64, 96), 3)

    def forward():
        return gpu_lib.mx4_linear(between(leaves[0]), leaves[1])

    def run():
        y = forward()
        return torch.autograd.grad(y, leaves, gy.to(y.dtype))

    return leaves, forward, run


def mix_case(gpu_lib, between):
    x, lg = rand((4, 4, 64), 4, torch.float32), rand((4, 4, 4), 5, torch.float32)
    leaves = (x.requires_grad_(True), lg.requires_grad_(True))
    gy = rand((4, 4, 64), 6)

    def forward():
        return gpu_lib.projected_mix(between(leaves[0]).bfloat16(), leaves[1])

    return leaves, forward, lambda: torch.autograd.grad(forward(), leaves[:1], gy)


BETWEEN = {"view": lambda t: t.view(t.shape), "cast": lambda t: t.bfloat16(),
           "chain": lambda t: (t * 2.0).reshape(-1).view(t.shape).bfloat16()}


@pytest.mark.parametrize("between", list(BETWEEN))
@pytest.mark.parametrize("case", [linear_case, mix_case])
def test_an_eager_graph_behind_other_nodes_is_refused(gpu_lib, case, between):
    """The leaf is not the operator's own input: a cast or a view stands
    between, as for weights kept in 32 bits."""
    leaves, forward, run = case(gpu_lib, BETWEEN[between])
    print(f"{case.__name__} {between}", flush=True)
    held = BETWEEN[between](leaves[0])  # an eager graph of x alone
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="eager graph"):
        with torch.cuda.graph(graph):
            run()
    torch.cuda.synchronize()
    del held
    replays(run, [t.clone() for t in run()])


@pytest.mark.parametrize("case", [linear_case, mix_case])
def test_an_eager_graph_begun_on_another_stream_joins_the_capture(gpu_lib, case):
    """The usual warm-up on a side stream, its result still held."""
    leaves, forward, run = case(gpu_lib, BETWEEN["cast"])
    want = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        held = forward()
    torch.cuda.current_stream().wait_stream(side)
    replays(run, want)
    assert held.requires_grad


def test_a_gradient_that_is_not_asked_for_is_no_reason(gpu_lib):
    """An eager graph of the weight lives, and the captured backward is for x
    alone."""
    gy, x, w = rand((64, 96), 3), rand((64, 32), 1), rand((96, 32), 2).requires_grad_(True)
    held = w * 1.0

    def run():
        xr = x.detach().requires_grad_(True)
        return torch.autograd.grad(gpu_lib.mx4_linear(xr, w), (xr,), gy)

    replays(run, [t.clone() for t in run()])
    assert held.requires_grad
