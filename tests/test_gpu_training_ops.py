"""Clipping and MXFP4 captures where the optimizer calls them: DobbGroup and the torch.optim wrapper
against the entry points they drive, bit for bit (every kernel is deterministic), and a whole training
loop that uses all of them.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
dobb = pytest.importorskip("block_diagonal_eigenbasis_amd")
from block_diagonal_eigenbasis_amd.optimizer import (Dobb, DobbGroup, Mx4Capture, clip_grad_norm_,  # noqa: E402
                                                     default_update_scale, default_update_scale_g)

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
DIMS = [(96, 256, 64), (64, 512, 256), (128, 256, 128), (80, 400, 200), (48, 96, 48)]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def randn(*shape, seed=0, dtype=F32, scale=1.0):
    g = torch.Generator()
    g.manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(dtype).to(DEV)


def group(streams=1, wdt=F32, **kw):
    Ws = [randn(m, n, seed=i, dtype=wdt, scale=0.02) for i, (m, n, _) in enumerate(DIMS)]
    return DobbGroup(Ws, [nb for _, _, nb in DIMS], momentum=0.9, weight_decay=0.1, streams=streams, **kw)


# ---- Mx4Capture ------------------------------------------------------------------------------------
def test_capture_holds_micro_batches():
    xs = [randn(k, 40, seed=k, dtype=BF16) for k in (100, 128, 1, 300)]
    caps = [Mx4Capture.quantize(x) for x in xs]
    c = Mx4Capture.cat(caps)
    assert c.shape == (529, 40) and c.parts == (100, 128, 1, 300) and c.tiles == 6 and c.device == xs[0].device
    want = torch.cat([dobb.dobb_mx4_dequantize(k.codes, k.scales, x.shape[0]) for k, x in zip(caps, xs)])
    assert torch.equal(c.dequantize(), want)
    assert torch.equal(c.dequantize(BF16), want.to(BF16))
    assert Mx4Capture.cat(caps[:1]) is caps[0]
    # nested: a capture of captures
    d = Mx4Capture.cat([c, caps[0]])
    assert d.parts == (100, 128, 1, 300, 100) and torch.equal(d.dequantize()[:529], want)
    with pytest.raises(ValueError, match="one width"):
        Mx4Capture.cat([caps[0], Mx4Capture.quantize(randn(5, 41))])
    with pytest.raises(ValueError, match="one width"):
        Mx4Capture.cat([])
    with pytest.raises(ValueError, match="add up"):
        Mx4Capture(c.codes, c.scales, (529,))


# ---- DobbGroup --------------------------------------------------------------------------------------
@pytest.mark.parametrize("streams", [1, 2])
def test_group_takes_captures_of_both_kinds(streams):
    """Weights 0 and 3 captured in bf16, the others in MXFP4, one of them from two micro-batches."""
    g = group(streams)
    Ns = [300, 300, 300, 300, 200]
    xs = [randn(N, n, seed=10 + i, dtype=BF16) for i, (N, (_, n, _)) in enumerate(zip(Ns, DIMS))]
    given = [x if i in (0, 3) else Mx4Capture.quantize(x) for i, x in enumerate(xs)]
    given[4] = Mx4Capture.cat([Mx4Capture.quantize(xs[4][:150]), Mx4Capture.quantize(xs[4][150:])])
    g.accumulate(given, 0.0)
    g.accumulate(given, 0.9)
    for i, (_, n, nb) in enumerate(DIMS):
        A = torch.zeros(n // nb, nb, nb, device=DEV)
        for beta in (0.0, 0.9):
            if i in (0, 3):
                dobb.dobb_accumulate_moment(xs[i], A, nb, beta)
            else:
                dobb.dobb_accumulate_moment_mx4(given[i].codes, given[i].scales, A, nb, Ns[i], beta)
        # how many splits a launch takes goes by its blocks, so sums may differ in their last bits
        # between a grouped and a single call: two roundings of 2^-24 of the magnitudes, and the EMA's
        off = (g.A[i].double() - A.double()).abs()
        x = (given[i].dequantize() if i not in (0, 3) else xs[i]).double().abs()
        m = torch.stack([x[:, b:b + nb].T @ x[:, b:b + nb] for b in range(0, n, nb)]) / Ns[i]
        assert bool((off <= 16 * 2.0 ** -24 * m).all()), i
    with pytest.raises(ValueError, match="capture 1"):
        g.accumulate([xs[0], given[2], *given[2:]], 0.0)


def test_two_streams_match_one_stream():
    gs = [group(s) for s in (1, 2)]
    xs = [Mx4Capture.quantize(randn(500, n, seed=20 + i, dtype=BF16)) for i, (_, n, _) in enumerate(DIMS)]
    for it in range(3):
        for g in gs:
            grads = [randn(m, n, seed=30 + 7 * it + i) for i, (m, n, _) in enumerate(DIMS)]
            first = it == 0
            g.refresh_step(xs, 0.0 if first else 0.9, dobb.DOBB_REFRESH_EXACT if first else dobb.DOBB_REFRESH_ORTH_ITER,
                           0 if first else 1, grads, warm_start=not first, max_grad_norm=1.5)
    for name in ("W", "M", "A", "Q"):
        for a, b in zip(getattr(gs[0], name), getattr(gs[1], name)):
            assert torch.equal(a, b), name
    assert torch.equal(gs[0].grad_norm, gs[1].grad_norm)


@pytest.mark.parametrize("gdt", [F32, BF16])
def test_group_clips_before_the_step(gdt):
    a, b = group(wdt=gdt), group(wdt=gdt)
    grads = [randn(m, n, seed=50 + i, dtype=gdt) for i, (m, n, _) in enumerate(DIMS)]
    ours = [x.clone() for x in grads]
    a.step(ours, max_grad_norm=0.8)
    want = math.sqrt(sum(float(x.double().square().sum()) for x in grads))
    assert abs(float(a.grad_norm) - want) <= 1.01 * 2.0 ** -24 * want
    dobb.dobb_clip_grads_grouped(grads, a.grad_norm, 0.8)
    assert all(torch.equal(x, y) for x, y in zip(ours, grads))
    b.step(grads)
    assert all(torch.equal(x, y) for x, y in zip(a.W, b.W)) and all(torch.equal(x, y) for x, y in zip(a.M, b.M))


def test_graph_of_a_step_that_clips_and_takes_mx4_captures():
    """Replays on refilled gradients and captures, against the same calls made eagerly."""
    a, b = group(2), group(2)
    raw = [randn(500, n, seed=20 + i, dtype=BF16) for i, (_, n, _) in enumerate(DIMS)]
    xs = [Mx4Capture.quantize(x) for x in raw]
    grads = [randn(m, n, seed=60 + i) for i, (m, n, _) in enumerate(DIMS)]
    big = [Mx4Capture.quantize(randn(5000, n, seed=3, dtype=BF16)) for _, n, _ in DIMS]
    with pytest.raises(RuntimeError, match="once before"):
        group().capture_refresh_step(big, 0.9, dobb.DOBB_REFRESH_ORTH_ITER, 1, grads)
    for g in (a, b):
        g.refresh_step(xs, 0.0, dobb.DOBB_REFRESH_EXACT, 0, [x.clone() for x in grads], warm_start=False, max_grad_norm=1.0)
    torch.cuda.synchronize()
    graph = a.capture_refresh_step(xs, 0.9, dobb.DOBB_REFRESH_ORTH_ITER, 1, grads, max_grad_norm=1.0)
    for it in range(4):
        for i, (m, n, _) in enumerate(DIMS):
            grads[i].copy_(randn(m, n, seed=70 + 9 * it + i, scale=10.0 ** (it - 3)))
            dobb.dobb_mx4_quantize(randn(500, n, seed=90 + 9 * it + i, dtype=BF16), xs[i].codes, xs[i].scales)
        eager = [x.clone() for x in grads]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        b.refresh_step(xs, 0.9, dobb.DOBB_REFRESH_ORTH_ITER, 1, eager, max_grad_norm=1.0)
        torch.cuda.synchronize()
        assert torch.equal(a.grad_norm, b.grad_norm) and all(torch.equal(x, y) for x, y in zip(grads, eager))
        for name in ("W", "M", "A", "Q"):
            assert all(torch.equal(x, y) for x, y in zip(getattr(a, name), getattr(b, name))), (it, name)


# ---- clip_grad_norm_ ---------------------------------------------------------------------------------
def test_clip_grad_norm_over_a_model():
    m = torch.nn.Sequential(torch.nn.Linear(33, 65), torch.nn.Linear(65, 7, bias=False), torch.nn.LayerNorm(7)).to(DEV)
    frozen = torch.nn.Parameter(torch.zeros(4, device=DEV))
    params = [*m.parameters(), frozen]
    for i, p in enumerate(m.parameters()):
        p.grad = randn(*p.shape, seed=i, scale=3.0)
    tied = torch.nn.Parameter(torch.zeros_like(params[0]))
    tied.grad = params[0].grad                                   # one gradient of two parameters
    before = [p.grad.clone() for p in m.parameters()]
    want = math.sqrt(sum(float(g.double().square().sum()) for g in before))
    total = clip_grad_norm_([*params, tied], 2.0)
    assert abs(float(total) - want) <= 1.01 * 2.0 ** -24 * want
    c = 2.0 / (want + 1e-6)
    for p, g in zip(m.parameters(), before):
        assert bool(((p.grad.double() - c * g.double()).abs() <= 6 * 2.0 ** -24 * c * g.double().abs() + 2.0 ** -150).all())
    assert float(clip_grad_norm_(params[0], 1e30)) > 0           # one parameter
    assert float(clip_grad_norm_([frozen], 1.0)) == 0.0          # nothing to clip
    assert float(clip_grad_norm_(iter(()), 1.0)) == 0.0


def test_clip_grad_norm_of_gradients_that_share_memory():
    whole, part, same = (torch.nn.Parameter(torch.zeros(k, device=DEV)) for k in (12, 8, 12))
    whole.grad = torch.full((12,), 2.0, device=DEV)
    part.grad, same.grad = whole.grad[:8], whole.grad.view(12)
    with pytest.raises(dobb.DobbError):
        clip_grad_norm_([whole, part], 1.0)                      # part of the entries would be scaled twice
    assert bool((whole.grad == 2.0).all())
    assert abs(float(clip_grad_norm_([whole, same], 1e30)) - math.sqrt(48.0)) <= 1e-5
    none = torch.nn.Parameter(torch.zeros(0, device=DEV))
    none.grad = torch.zeros(0, device=DEV)
    assert clip_grad_norm_([none], 1.0).device.type == "cuda"


# ---- the optimizer ------------------------------------------------------------------------------------
@pytest.mark.parametrize("basis", ["activation", "output_gradient"])
@pytest.mark.parametrize("policy", ["first", "all"])
def test_optimizer_matches_the_entry_points(basis, policy):
    print(f"optimizer: {basis} {policy}", flush=True)
    dims = [(64, 256), (128, 128)]
    side = 1 if basis == "activation" else 0
    params = [torch.nn.Parameter(randn(m, n, seed=i, scale=0.02)) for i, (m, n) in enumerate(dims)]
    lr, wd, mu, T, beta, cap = 2.5e-3, 0.1, 0.9, 2, 0.9, 1.25
    opt = Dobb(params, lr=lr, weight_decay=wd, momentum=mu, blocks=2, refresh_period=T, beta=beta, capture=policy, basis=basis,
               capture_format="mx4", max_grad_norm=cap)
    nbs = [d[side] // 2 for d in dims]
    W = [p.detach().clone() for p in params]
    M = [torch.zeros_like(w) for w in W]
    A = [torch.zeros(2, nb, nb, device=DEV) for nb in nbs]
    Q = [torch.eye(nb, device=DEV).expand(2, nb, nb).contiguous() for nb in nbs]
    scale = default_update_scale if side else default_update_scale_g
    hps = [dobb.make_hparams(lr, wd, mu, scale(m, n)) for m, n in dims]
    step = dobb.dobb_step if side else dobb.dobb_step_g
    for t in range(5):
        batches = [[randn(k, d[side], seed=100 * t + 10 * j + i, dtype=BF16) for i, d in enumerate(dims)]
                   for j, k in enumerate((200, 333))]
        if opt.wants_capture():
            for b in batches:
                for p, x in zip(params, b):
                    opt.capture(p, x.view(1, *x.shape))
        grads = [randn(m, n, seed=1000 + 10 * t + i) for i, (m, n) in enumerate(dims)]
        for p, g in zip(params, grads):
            p.grad = g.clone()
        opt.step()
        total = dobb.dobb_clip_grad_norm_grouped(grads, cap)
        assert torch.equal(opt.grad_norm, total) and all(torch.equal(p.grad, g) for p, g in zip(params, grads))
        if t % T == 0:
            used = batches if policy == "all" else batches[:1]
            caps = [Mx4Capture.cat([Mx4Capture.quantize(b[i]) for b in used]) for i in range(2)]
            dobb.dobb_accumulate_moment_mx4_grouped([c.codes for c in caps], [c.scales for c in caps], A, nbs, caps[0].shape[0],
                                                    beta if t else 0.0)
            for i in range(2):
                if t:
                    dobb.dobb_refresh_basis(A[i], Q[i], dobb.DOBB_REFRESH_ORTH_ITER, iters=1, warm_start=True)
                else:
                    dobb.dobb_refresh_basis(A[i], Q[i], dobb.DOBB_REFRESH_EXACT, warm_start=False)
        for i in range(2):
            step(W[i], grads[i], M[i], Q[i], nbs[i], hps[i])
    for i in range(2):
        assert torch.equal(opt._group.A[i], A[i]) and torch.equal(opt._group.Q[i], Q[i])
        assert torch.equal(params[i].detach(), W[i])


def test_a_training_loop_with_everything_on():
    """Hooks, micro-batches, clipping over the whole model beside another optimizer: it runs, its gradients
    are the model's, and the weights stay finite."""
    torch.manual_seed(0)
    model = torch.nn.Sequential(torch.nn.Linear(64, 128), torch.nn.GELU(), torch.nn.Linear(128, 32)).to(DEV)
    lin = [m for m in model if isinstance(m, torch.nn.Linear)]
    opt = Dobb([m.weight for m in lin], blocks=4, refresh_period=2, capture="all", capture_format="mx4")
    rest = torch.optim.SGD([m.bias for m in lin], lr=1e-2)
    hooks = opt.attach_capture_hooks(lin)
    x, y = randn(3, 50, 64, seed=1), randn(3, 50, 32, seed=2)
    for _ in range(4):
        for j in range(3):
            (model(x[j]) - y[j]).square().mean().backward()
        grads = [p.grad.clone() for p in model.parameters()]
        total = clip_grad_norm_(model.parameters(), 0.05)
        want = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
        assert abs(float(total) - want) <= 1.01 * 2.0 ** -24 * want
        opt.step()
        rest.step()
        model.zero_grad()
    for h in hooks:
        h.remove()
    assert opt._group.refreshes == 2 and all(bool(p.isfinite().all()) for p in model.parameters())
    assert np.isfinite(float((model(x[0]) - y[0]).square().mean().detach()))
