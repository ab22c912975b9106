"""Which memory a DobbGroup's calls use as workspace, and on which stream, shown without a GPU: streams are
stand-ins, the state and the captures are CPU tensors, the grouped C calls are logged instead of made, and the
workspace sizes are the library's.

A workspace may be used on the stream in whose order it was allocated, or on one it is recorded on; it has its
size before the streams of a call fork, and stays the same until they have joined.
"""
import contextlib
import types
import weakref

import pytest
import torch

import block_diagonal_eigenbasis_amd as dobb
from block_diagonal_eigenbasis_amd import _abi, _ops
from block_diagonal_eigenbasis_amd.optimizer import DobbGroup, Mx4Capture

BF16 = torch.bfloat16


class Stream:
    made = 0

    def __init__(self, log, *_):
        Stream.made += 1
        self.cuda_stream, self.log, self.device = Stream.made, log, torch.device("cpu")

    def wait_stream(self, other):
        self.log.append(("wait", self.cuda_stream, other.cuda_stream))


class Graph:
    """Stands in for torch.cuda.CUDAGraph: an object that can be held and weakly referenced."""


@pytest.fixture
def world(monkeypatch):
    """log: ("alloc", address, stream), ("record", address, stream), ("wait", ..), ("call", name, address, stream)."""
    log = []
    w = types.SimpleNamespace(log=log, stream=lambda: Stream(log))
    current = [Stream(log)]

    @contextlib.contextmanager
    def on(s):
        current.append(s)
        try:
            yield
        finally:
            current.pop()

    def empty(*a, make=torch.empty, **kw):
        t = make(*a, **kw)
        if kw.get("dtype") == torch.uint8:
            log.append(("alloc", t.data_ptr(), current[-1].cuda_stream))
        return t

    class Lib:
        """The library: sizes are asked for, grouped calls are logged (the workspace is their third last argument)."""

        def __init__(self, real):
            self.real = real

        def __getattr__(self, name):
            if not name.endswith("_grouped"):
                return getattr(self.real, name)

            def call(*args):
                w.current_devices.append(w.devices[-1] if w.devices else None)
                log.append(("call", name, args[-3], args[-1]))
                return 0
            return call

    lib, ops = Lib(_abi.lib()), Lib(_ops._lib())
    monkeypatch.setattr(_abi, "lib", lambda: lib)
    monkeypatch.setattr(_ops, "_lib", lambda: ops)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "Stream", lambda *a, **k: Stream(log))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(torch.cuda, "stream", on)
    w.devices, w.current_devices = [], []

    @contextlib.contextmanager
    def device(d):
        w.devices.append(d)
        try:
            yield
        finally:
            w.devices.pop()
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "CUDAGraph", Graph)
    captures = []

    @contextlib.contextmanager
    def graph(g):
        captures.append(g)
        with on(Stream(log)):
            yield
        captures.pop()
    monkeypatch.setattr(torch.cuda, "graph", graph)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: bool(captures))
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: log.append(("record", t.data_ptr(), s.cuda_stream)), raising=False)
    return w


def group(dims, streams):
    return DobbGroup([torch.zeros(8, n) for n, _ in dims], [nb for _, nb in dims], streams=streams)


def held(n, N):
    T = dobb.mx4_tiles(N)
    return Mx4Capture(torch.zeros(T, 4, n, 16, dtype=torch.uint8), torch.zeros(T, n, 4, dtype=torch.uint8), (N,))


def check(log):
    """Every workspace on a stream it belongs to; none allocated between a fork and the last call of a run."""
    allowed, forked, calls = {}, False, 0
    for kind, *rest in log:
        if kind == "alloc":
            assert not forked, "a workspace grew after the streams forked"
            allowed[rest[0]] = {rest[1]}
        elif kind == "record":
            allowed.setdefault(rest[0], set()).add(rest[1])
        elif kind == "wait":
            forked = not forked                 # one side stream: it waits for the caller's, then the caller's for it
        else:
            calls += 1
            name, ws, stream = rest
            assert stream in allowed[ws], f"{name}: its workspace belongs to other streams"
    return calls


def in_one_workspace(log):
    """The workspaces of the calls, by stream: one each."""
    by = {}
    for kind, *rest in log:
        if kind == "call":
            by.setdefault(rest[2], set()).add(rest[1])
    return all(len(v) == 1 for v in by.values())


# two 768-wide weights and a 1024-wide one with narrow blocks, as a model holds them; the second token count of
# the wide part needs more scratch than the first, and more than the step reserved
DIMS = [(768, 192), (768, 192), (1024, 64)]


def captures(kind):
    if kind == "mx4":
        return [held(768, 4096), held(768, 16384), held(1024, 16384)]
    if kind == "dense":
        return [torch.zeros(N, n, dtype=BF16) for n, N in ((768, 4096), (768, 16384), (1024, 16384))]
    return [torch.zeros(4096, 768, dtype=BF16), held(768, 16384), held(1024, 16384)]


@pytest.mark.parametrize("kind", ["mx4", "dense", "mixed"])
@pytest.mark.parametrize("streams", [1, 2])
@pytest.mark.parametrize("own_stream", [False, True])
def test_workspaces_are_sized_before_the_streams_fork(world, kind, streams, own_stream):
    g = group(DIMS, streams)
    xs = captures(kind)
    s = world.stream() if own_stream else None
    for go in (lambda: g.accumulate(xs, 0.9, stream=s),
               lambda: g.refresh_step(xs, 0.9, dobb.DOBB_REFRESH_ORTH_ITER, 1, [torch.zeros(8, n) for n, _ in DIMS], stream=s)):
        start = len(world.log)
        go()
        first = [e for e in world.log[:start] if e[0] in ("alloc", "record")]
        assert check(first + world.log[start:]) >= 2
        assert in_one_workspace(world.log[start:])


@pytest.mark.parametrize("streams", [1, 2])
def test_a_call_that_refuses_a_capture_enqueues_nothing(world, streams):
    g = group(DIMS, streams)
    good = captures("mixed")
    for k, bad in [(1, held(760, 16384)), (2, held(1000, 128)), (0, torch.zeros(4096, 760, dtype=BF16)),
                   (2, torch.zeros(1024, 64, dtype=BF16).T)]:
        xs = list(good)
        xs[k] = bad
        start = len(world.log)
        with pytest.raises(ValueError, match=f"capture {k}"):
            g.refresh_step(xs, 0.9, dobb.DOBB_REFRESH_ORTH_ITER, 1, [torch.zeros(8, n) for n, _ in DIMS])
        assert not [e for e in world.log[start:] if e[0] == "call"]


@pytest.mark.parametrize("streams", [1, 2])
def test_a_captured_graph_keeps_its_workspaces(world, streams):
    g = group(DIMS, streams)
    xs = captures("mx4")
    grads = [torch.zeros(8, n) for n, _ in DIMS]
    with pytest.raises(RuntimeError, match="once before"):
        g.capture_refresh_step(xs, 0.9, dobb.DOBB_REFRESH_ORTH_ITER, 1, grads)
    g.refresh_step(xs, 0.9, dobb.DOBB_REFRESH_ORTH_ITER, 1, grads)
    graph = g.capture_refresh_step(xs, 0.9, dobb.DOBB_REFRESH_ORTH_ITER, 1, grads)
    used = [weakref.ref(p.ws) for p in g._parts]
    g.accumulate([held(n, 1 << 19) for n, _ in DIMS], 0.9)          # an eager call that needs more
    assert all(p.ws is not u() for p, u in zip(g._parts, used))
    g.set_streams(1)
    assert all(u() is not None for u in used), "a workspace of the graph was freed"
    bound = [weakref.ref(t) for x in xs for t in (x.codes, x.scales)] + [weakref.ref(t) for t in grads]
    xs.clear()
    grads.clear()
    assert all(b() is not None for b in bound), "a tensor that the graph reads was freed"
    del graph
    assert all(u() is None for u in used) and all(b() is None for b in bound)


@pytest.mark.parametrize("streams", [1, 2])
def test_calls_are_made_with_the_groups_device_current(world, streams):
    g = group(DIMS, streams)
    xs, grads = captures("mixed"), [torch.zeros(8, n) for n, _ in DIMS]
    g.accumulate(xs, 0.9)
    g.refresh(dobb.DOBB_REFRESH_EXACT, 0)
    g.step(grads)
    g.refresh_step(xs, 0.9, dobb.DOBB_REFRESH_ORTH_ITER, 1, grads)
    g.capture_refresh_step(xs, 0.9, dobb.DOBB_REFRESH_ORTH_ITER, 1, grads)
    assert len(world.current_devices) >= 10 and set(world.current_devices) == {g.device}


@pytest.mark.parametrize("streams", [1, 2])
def test_a_capture_of_the_callers_own_keeps_its_workspaces(world, streams):
    """Calls captured with torch.cuda.graph: the group cannot know how long that graph lives, and holds what it
    was captured with for its own life."""
    g = group(DIMS, streams)
    xs, grads = captures("mx4"), [torch.zeros(8, n) for n, _ in DIMS]
    g.accumulate(xs, 0.9)
    with torch.cuda.graph(Graph()):
        g.accumulate(xs, 0.9)
        g.step(grads)
    used = [weakref.ref(p.ws) for p in g._parts]
    g.accumulate([held(n, 1 << 19) for n, _ in DIMS], 0.9)
    assert all(p.ws is not u() for p, u in zip(g._parts, used))
    g.set_streams(1)
    assert all(u() is not None for u in used), "a workspace of the graph was freed"
    del g
    assert all(u() is None for u in used)
