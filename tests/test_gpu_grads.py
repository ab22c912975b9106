"""Gradient norms and clipping (include/dobb_ops.h) against the formulas in 64 bits.

Tolerances.  u = 2^-24 is half a step of fp32 relative to the value.
* norms, total: fp64 sums (error far below u) rounded once to fp32: u, 1.01 u allowed.
* coefficient: max_norm and total (or, where it is the larger term, the constant 1e-6) are off by u each,
  their sum and the quotient are rounded (u each), the product adds u: 5 u, and rounding to bf16 2^-8.
  So 6 u relative, and 2^-8 (1 + 6 u) more for bf16; entries below the normal range round to half of the
  smallest subnormal (2^-150, and 2^-134 for bf16).
"""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
dobb = pytest.importorskip("block_diagonal_eigenbasis_amd")
DEV = "cuda"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def views(numels, dtypes, seed, scale=1.0, gap=0):
    """Tensors laid one behind the other in a buffer per type, `gap` entries of 7 between them, each
    unaligned by what the ones before leave; and the buffers."""
    held = {dt: torch.full((sum(k + gap for k, d in zip(numels, dtypes) if d == dt) + gap,), 7.0, dtype=dt, device=DEV)
            for dt in set(dtypes)}
    at = {dt: gap for dt in held}
    g = gen(seed)
    out = []
    for k, dt in zip(numels, dtypes):
        v = held[dt][at[dt]:at[dt] + k]
        v.copy_(torch.randn(k, generator=g, device=DEV) * scale)
        out.append(v)
        at[dt] += k + gap
    return out, held


def ref_norms(ts):
    sq = [float(t.double().square().sum()) for t in ts]
    return [math.sqrt(s) for s in sq], math.sqrt(sum(sq))


def check_norms(norms, total, ts):
    want, all_ = ref_norms(ts)
    for got, w in zip(norms.tolist(), want):
        assert abs(got - w) <= 1.01 * U * w + 2.0 ** -149, (got, w)
    assert abs(float(total) - all_) <= 1.01 * U * all_ + 2.0 ** -149, (float(total), all_)


def check_clipped(outs, ts, max_norm):
    _, total = ref_norms(ts)
    c = min(1.0, max_norm / (total + 1e-6))
    for o, t in zip(outs, ts):
        want = t.double() * c
        tol = 6 * U * want.abs() + 2.0 ** -150
        if o.dtype == BF16:
            tol = tol + 2.0 ** -8 * (1 + 6 * U) * want.abs() + 2.0 ** -134
        off = (o.double() - want).abs()
        assert bool((off <= tol).all()), (o.dtype, t.numel(), float((off / want.abs().clamp(min=1e-300)).max()))


RAGGED = [random.Random(11).choice([1, 2, 3, 7, 8, 9, 31, 255, 1000, 4095, 4096, 4097, 8192, 8193, 16385]) for _ in range(401)]
LISTS = {
    "one entry": ([1], [F32]), "one bf16 entry": ([1], [BF16]), "one weight": ([768 * 768], [F32]),
    "vector ends": ([3, 4, 5, 7, 8, 9, 15, 16, 17], [F32, BF16, F32, BF16, BF16, BF16, F32, BF16, BF16]),
    "empty ones among": ([0, 5, 0, 0, 9000, 0], [F32, F32, BF16, F32, BF16, F32]),
    "chunk borders": ([4096, 4097, 8192, 8191, 8193, 16384 * 3 + 1], [F32, F32, BF16, BF16, BF16, F32]),
    "several tables": (RAGGED, [F32 if i % 3 else BF16 for i in range(len(RAGGED))]),
    "wide": ([6400 * 1600, 1600 * 1600 + 1], [BF16, F32]),
}


@pytest.mark.parametrize("name", LISTS)
def test_norms(name):
    print(f"norms: {name}", flush=True)
    numels, dts = LISTS[name]
    ts, _ = views(numels, dts, 1)
    norms = torch.empty(len(ts), device=DEV)
    total = dobb.dobb_grad_norm_grouped(ts, norms=norms)
    check_norms(norms, total, ts)
    # without the tensors' own norms, and once more: the same bits
    again = dobb.dobb_grad_norm_grouped(ts, total=torch.empty((), device=DEV))
    assert torch.equal(total, again)


@pytest.mark.parametrize("name", LISTS)
@pytest.mark.parametrize("out", ["in place", "same", "fp32", "bf16"])
@pytest.mark.parametrize("ratio", [0.37, 3.0])
def test_clip(name, out, ratio):
    print(f"clip: {name} {out} {ratio}", flush=True)
    numels, dts = LISTS[name]
    ts, held = views(numels, dts, 2, gap=5)
    before = [t.clone() for t in ts]
    max_norm = ratio * ref_norms(ts)[1]
    norms = torch.empty(len(ts), device=DEV)
    if out == "in place":
        outs, oheld = ts, held
        total = dobb.dobb_clip_grad_norm_grouped(ts, max_norm, norms=norms)
    else:
        odt = dts if out == "same" else [{"fp32": F32, "bf16": BF16}[out]] * len(dts)
        outs, oheld = views(numels, odt, 3, gap=5)
        total = dobb.dobb_clip_grad_norm_grouped(ts, max_norm, outs=outs, norms=norms)
        assert all(torch.equal(a, b) for a, b in zip(ts, before))
    check_norms(norms, total, before)
    check_clipped(outs, before, max_norm)
    if ratio > 1 and out in ("in place", "same"):
        assert all(torch.equal(a, b) for a, b in zip(outs, before))
    for dt, buf in oheld.items():       # the entries between the tensors are as they were
        mask = torch.ones(buf.numel(), dtype=torch.bool, device=DEV)
        base = buf.data_ptr()
        for o in outs:
            if o.dtype == dt and o.numel():
                a = (o.data_ptr() - base) // buf.element_size()
                mask[a:a + o.numel()] = False
        assert bool((buf[mask] == 7.0).all())


@pytest.mark.parametrize("scale", [1e30, 3e-25, 1e-39])
def test_norm_of_entries_whose_squares_leave_fp32(scale):
    ts, _ = views([5000, 333], [F32, BF16], 4, scale=scale)
    norms = torch.empty(2, device=DEV)
    total = dobb.dobb_clip_grad_norm_grouped(ts, 0.25 * ref_norms(ts)[1], outs=(outs := [torch.empty_like(t) for t in ts]), norms=norms)
    check_norms(norms, total, ts)
    check_clipped(outs, ts, 0.25 * ref_norms(ts)[1])


def test_max_norm_zero_and_infinity():
    ts, _ = views([300, 77], [F32, BF16], 5)
    before = [t.clone() for t in ts]
    dobb.dobb_clip_grad_norm_grouped(ts, math.inf)
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    dobb.dobb_clip_grad_norm_grouped(ts, 0.0)
    assert all(bool((t == 0).all()) for t in ts)
    # a zero gradient: the coefficient is 1, whatever max_norm
    total = dobb.dobb_clip_grad_norm_grouped(ts, 1.0)
    assert float(total) == 0.0 and all(bool((t == 0).all()) for t in ts)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_nan_and_infinity_propagate(dt):
    ts, _ = views([3000, 50], [dt, F32], 6)
    ts[0][1234] = math.nan
    norms = torch.empty(2, device=DEV)
    outs = [torch.empty_like(t) for t in ts]
    total = dobb.dobb_clip_grad_norm_grouped(ts, 1.0, outs=outs, norms=norms)
    assert math.isnan(float(total)) and math.isnan(float(norms[0])) and math.isfinite(float(norms[1]))
    assert all(bool(o.isnan().all()) for o in outs)
    ts[0][1234] = -math.inf
    total = dobb.dobb_clip_grad_norm_grouped(ts, 1.0, outs=outs, norms=norms)
    assert float(total) == math.inf and float(norms[0]) == math.inf
    bad = outs[0].isnan()
    assert bool(bad[1234]) and int(bad.sum()) == 1 and bool((outs[0][~bad] == 0).all()) and bool((outs[1] == 0).all())


def test_a_tensor_listed_twice_counts_twice_and_is_not_scaled_twice():
    ts, _ = views([4000], [F32], 7)
    total = dobb.dobb_grad_norm_grouped([ts[0], ts[0]])
    want = ref_norms(ts)[1] * math.sqrt(2)
    assert abs(float(total) - want) <= 1.01 * U * want
    with pytest.raises(dobb.DobbError):
        dobb.dobb_clip_grad_norm_grouped([ts[0], ts[0]], 0.1)
    outs = [torch.empty_like(ts[0]) for _ in range(2)]
    dobb.dobb_clip_grad_norm_grouped([ts[0], ts[0]], 0.1, outs=outs)      # read twice, written apart
    check_clipped(outs, [ts[0], ts[0]], 0.1)


def test_clip_by_a_total_from_elsewhere():
    """Totals of two processes' shards combined between the two calls."""
    a, _ = views([5000, 17], [F32, BF16], 8)
    b, _ = views([900], [BF16], 9)
    parts = torch.stack([dobb.dobb_grad_norm_grouped(a), dobb.dobb_grad_norm_grouped(b)])
    total = torch.linalg.vector_norm(parts)
    want = ref_norms(a + b)[1]
    ca, cb = [t.clone() for t in a], [t.clone() for t in b]
    dobb.dobb_clip_grads_grouped(ca, total, 0.5 * want)
    dobb.dobb_clip_grads_grouped(cb, total.reshape(1), 0.5 * want)
    # the combined total has up to 4 u more (two norms, squares, a sum, a root), 2^-20 is far above it
    c = 0.5 * want / (want + 1e-6)
    for o, t in zip(ca + cb, a + b):
        tol = (2.0 ** -20 + (2.0 ** -8 if o.dtype == BF16 else 0)) * (t.double() * c).abs()
        assert bool(((o.double() - t.double() * c).abs() <= tol).all())


def test_more_than_2_31_entries():
    n = (1 << 31) + 4097
    t = torch.zeros(n, dtype=BF16, device=DEV)
    at = torch.tensor([0, 5, (1 << 30) + 3, (1 << 31) - 1, 1 << 31, n - 1], device=DEV)
    t[at] = torch.tensor([3.0, -4.0, 1.5, 2.0, -8.0, 0.5], dtype=BF16, device=DEV)
    want = math.sqrt(float(t[at].double().square().sum()))
    total = dobb.dobb_clip_grad_norm_grouped([t], 0.5 * want)
    assert abs(float(total) - want) <= 1.01 * U * want
    c = 0.5 * want / (want + 1e-6)
    got, src = t[at].double(), torch.tensor([3.0, -4.0, 1.5, 2.0, -8.0, 0.5], dtype=torch.float64, device=DEV) * c
    assert bool(((got - src).abs() <= 2.0 ** -7 * src.abs()).all())
    assert int(torch.count_nonzero(t)) == 6


def test_on_a_stream_of_its_own():
    ts, _ = views([200000, 33], [F32, BF16], 10)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    norms = torch.empty(2, device=DEV)
    outs = [torch.empty_like(t) for t in ts]
    s.wait_stream(torch.cuda.current_stream())
    total = dobb.dobb_clip_grad_norm_grouped(ts, 1.0, outs=outs, norms=norms, stream=s)
    junk = [torch.full((1 << 16,), 3.0, device=DEV) for _ in range(8)]      # takes freed blocks, if any were
    torch.cuda.current_stream().wait_stream(s)
    check_norms(norms, total, ts)
    check_clipped(outs, ts, 1.0)
    del junk


def test_graph_replays():
    ts, held = views(RAGGED[:230], [F32 if i % 2 else BF16 for i in range(230)], 11)
    norms, total = torch.empty(230, device=DEV), torch.empty((), device=DEV)
    outs = [torch.empty_like(t) for t in ts]
    dobb.dobb_clip_grad_norm_grouped(ts, 1.0, outs=outs, norms=norms, total=total)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dobb.dobb_clip_grad_norm_grouped(ts, 1.0, outs=outs, norms=norms, total=total)
    for it in range(4):
        g = gen(20 + it)
        for buf in held.values():
            buf.copy_(torch.randn(buf.numel(), generator=g, device=DEV) * 10.0 ** (it - 2))
        eager = [torch.empty_like(t) for t in ts]
        en = torch.empty_like(norms)
        et = dobb.dobb_clip_grad_norm_grouped(ts, 1.0, outs=eager, norms=en)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check_norms(norms, total, ts)
        assert torch.equal(et, total) and torch.equal(en, norms)
        assert all(torch.equal(a, b) for a, b in zip(outs, eager))


def test_refusals():
    t = torch.zeros(8, 8, device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        dobb.dobb_grad_norm_grouped([t.T[:, :3]])
    with pytest.raises(TypeError, match="dtype"):
        dobb.dobb_grad_norm_grouped([t.half()])
    with pytest.raises(ValueError, match="shapes"):
        dobb.dobb_clip_grad_norm_grouped([t], 1.0, outs=[torch.zeros(8, 4, device=DEV)])
    with pytest.raises(ValueError, match="shapes"):
        dobb.dobb_clip_grad_norm_grouped([t, t.clone()], 1.0, outs=[t])
    with pytest.raises(ValueError, match="norms must have shape"):
        dobb.dobb_grad_norm_grouped([t], norms=torch.empty(2, device=DEV))
    with pytest.raises(ValueError, match="total"):
        dobb.dobb_grad_norm_grouped([t], total=torch.empty(2, device=DEV))
    with pytest.raises(ValueError, match="workspace too small"):
        dobb.dobb_grad_norm_grouped([t], ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(dobb.DobbError):
        dobb.dobb_clip_grad_norm_grouped([t], -1.0)
    with pytest.raises(dobb.DobbError):
        dobb.dobb_clip_grad_norm_grouped([t], math.nan)


def test_sums_over_a_gradient_are_refused():
    t = torch.zeros(64, device=DEV)
    with pytest.raises(dobb.DobbError):
        dobb.dobb_grad_norm_grouped([t], total=t[3])
    with pytest.raises(dobb.DobbError):
        dobb.dobb_clip_grad_norm_grouped([t], 1.0, norms=t[:1])
    with pytest.raises(dobb.DobbError):
        dobb.dobb_clip_grads_grouped([t], t[63:], 1.0)


def test_iterables_and_integer_bounds():
    ts, _ = views([50, 60], [F32, BF16], 30)
    want = dobb.dobb_grad_norm_grouped(ts)
    assert torch.equal(dobb.dobb_grad_norm_grouped(t for t in ts), want)
    assert torch.equal(dobb.dobb_clip_grad_norm_grouped(tuple(ts), 10 ** 6), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    total = dobb.dobb_grad_norm_grouped((t for t in ts), stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(total, want)
