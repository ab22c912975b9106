"""DobbGroup's workspaces where captures in MXFP4 make them grow: on a stream of the caller's, with two streams
and two token counts, and between the replays of a captured graph.  What the group leaves has to be bit for bit
what a twin leaves whose workspaces had their size from the start (every kernel is deterministic).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
dobb = pytest.importorskip("block_diagonal_eigenbasis_amd")
from block_diagonal_eigenbasis_amd.optimizer import DobbGroup, Mx4Capture  # noqa: E402

DEV = "cuda"
BF16 = torch.bfloat16
DIMS = [(64, 768, 192), (48, 768, 192), (32, 1024, 64), (16, 512, 32)]      # two wide weights and two with narrow blocks
TOKENS = [4096, 16384, 16384, 1500]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def randn(*shape, seed=0, dtype=torch.float32):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).to(DEV)


def group(streams=1):
    Ws = [0.02 * randn(m, n, seed=i) for i, (m, n, _) in enumerate(DIMS)]
    return DobbGroup(Ws, [nb for _, _, nb in DIMS], momentum=0.9, weight_decay=0.1, streams=streams)


def captures(tokens, seed):
    return [Mx4Capture.quantize(randn(N, n, seed=seed + i, dtype=BF16)) for i, (N, (_, n, _)) in enumerate(zip(tokens, DIMS))]


def roomy(streams=1):
    """A group whose workspaces need not grow for any capture of this file."""
    g = group(streams)
    g.accumulate(captures([65536] * len(DIMS), 1), 0.0)
    for a in g.A:
        a.zero_()
    torch.cuda.synchronize()
    return g


def same(a, b):
    for name in ("W", "M", "A", "Q"):
        for i, (x, y) in enumerate(zip(getattr(a, name), getattr(b, name))):
            assert torch.equal(x, y), (name, i)


@pytest.mark.parametrize("streams", [1, 2])
@pytest.mark.parametrize("own_stream", [False, True])
def test_growing_workspaces(streams, own_stream):
    print(f"growing workspaces: {streams} streams, own stream {own_stream}", flush=True)
    a, b = group(streams), roomy(streams)
    xs = captures(TOKENS, 10)
    grads = [randn(m, n, seed=20 + i) for i, (m, n, _) in enumerate(DIMS)]
    torch.cuda.synchronize()
    sizes = [p.ws.numel() for p in a._parts]
    s = torch.cuda.Stream() if own_stream else None
    a.accumulate(xs, 0.0, stream=s)
    assert any(p.ws.numel() > k for p, k in zip(a._parts, sizes))
    sizes = [p.ws.numel() for p in a._parts]
    # what a freed workspace left behind is taken and written at once, on the stream that is current
    junk = [torch.full((k // 4,), 7.0, device=DEV) for k in sizes for _ in range(3)]
    longer = captures([65536, 4096, 65536, 40000], 30)
    torch.cuda.current_stream().synchronize()
    a.refresh_step(longer, 0.9, dobb.DOBB_REFRESH_EXACT, 0, grads, warm_start=False, stream=s)
    junk += [torch.full((k // 4,), 7.0, device=DEV) for k in sizes for _ in range(3)]
    torch.cuda.synchronize()
    b.accumulate(xs, 0.0)
    b.refresh_step(longer, 0.9, dobb.DOBB_REFRESH_EXACT, 0, grads, warm_start=False)
    torch.cuda.synchronize()
    same(a, b)
    assert all(bool((j == 7.0).all()) for j in junk)


@pytest.mark.parametrize("streams", [1, 2])
def test_a_longer_capture_between_replays(streams):
    """An eager call that needs larger workspaces than the graph was captured with: replays use the old ones."""
    print(f"longer capture between replays: {streams} streams", flush=True)
    a, b = group(streams), roomy(streams)
    xs = captures(TOKENS, 40)
    longer = captures([65536, 65536, 65536, 65536], 50)
    grads = [randn(m, n, seed=60 + i) for i, (m, n, _) in enumerate(DIMS)]
    for g in (a, b):
        g.refresh_step(xs, 0.0, dobb.DOBB_REFRESH_EXACT, 0, grads, warm_start=False)
    torch.cuda.synchronize()
    graph = a.capture_refresh_step(xs, 0.9, dobb.DOBB_REFRESH_ORTH_ITER, 1, grads)
    used = [p.ws.data_ptr() for p in a._parts]
    junk = []
    for it in range(4):
        graph.replay()
        b.refresh_step(xs, 0.9, dobb.DOBB_REFRESH_ORTH_ITER, 1, grads)
        torch.cuda.synchronize()
        same(a, b)
        for g in (a, b):
            g.accumulate(longer, 0.5)
        junk += [torch.full((1 << 20,), 7.0, device=DEV) for _ in range(16)]
        torch.cuda.synchronize()
        assert any(p.ws.data_ptr() != u for p, u in zip(a._parts, used))
        same(a, b)
    assert all(bool((j == 7.0).all()) for j in junk)


@pytest.mark.parametrize("streams", [1, 2])
def test_a_longer_capture_between_replays_of_the_callers_own_graph(streams):
    print(f"the caller's own graph: {streams} streams", flush=True)
    a, b = group(streams), roomy(streams)
    xs = captures(TOKENS, 70)
    longer = captures([65536, 65536, 65536, 65536], 80)
    grads = [randn(m, n, seed=90 + i) for i, (m, n, _) in enumerate(DIMS)]
    for g in (a, b):
        g.refresh_step(xs, 0.0, dobb.DOBB_REFRESH_EXACT, 0, grads, warm_start=False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.accumulate(xs, 0.9)
        a.step(grads)
    used = [p.ws.data_ptr() for p in a._parts]
    junk = []
    for it in range(4):
        graph.replay()
        b.accumulate(xs, 0.9)
        b.step(grads)
        torch.cuda.synchronize()
        same(a, b)
        for g in (a, b):
            g.accumulate(longer, 0.5)
        junk += [torch.full((1 << 20,), 7.0, device=DEV) for _ in range(16)]
        torch.cuda.synchronize()
        assert any(p.ws.data_ptr() != u for p, u in zip(a._parts, used))
        same(a, b)
    assert all(bool((j == 7.0).all()) for j in junk)
