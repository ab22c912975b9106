"""Clipping where the norm or its limit is infinite: a coefficient of 0 for a finite limit, of 1 for none, and a
NaN only from a NaN (include/dobb_ops.h).  All results are exact.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
dobb = pytest.importorskip("block_diagonal_eigenbasis_amd")
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def grads(dt, kind):
    a = torch.arange(1, 3001, device=DEV, dtype=F32).to(dt)
    b = torch.full((77,), -2.5, device=DEV)
    if kind == "large":                      # finite entries whose norm is above the largest fp32 value
        a[5], a[2000] = 3.0e38, -3.0e38
    else:
        a[1234] = {"inf": math.inf, "-inf": -math.inf, "nan": math.nan}[kind]
    return [a, b]


def same(xs, ys):
    return all(torch.equal(x, y) for x, y in zip(xs, ys))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("kind", ["inf", "-inf", "large"])
@pytest.mark.parametrize("where", ["in place", "apart", "given total"])
def test_an_infinite_norm(dt, kind, where):
    print(f"infinite norm: {dt} {kind} {where}", flush=True)
    for limit in (math.inf, 1.0, 0.0, 3.0e38):
        ts = grads(dt, kind)
        before = [t.clone() for t in ts]
        outs = ts if where != "apart" else [torch.empty_like(t) for t in ts]
        if where == "given total":
            total = dobb.dobb_grad_norm_grouped(ts)
            dobb.dobb_clip_grads_grouped(ts, total, limit)
        else:
            total = dobb.dobb_clip_grad_norm_grouped(ts, limit, outs=None if where == "in place" else outs)
        assert float(total) == math.inf
        if limit == math.inf:
            assert same(outs, before)
        else:                                # 0 times everything, which an infinity turns into a NaN
            want = [torch.where(t.isinf(), math.nan, 0.0) for t in before]
            for o, w in zip(outs, want):
                assert torch.equal(o.isnan(), w.isnan()) and bool((o[~w.isnan()] == 0).all())


@pytest.mark.parametrize("dt", [F32, BF16])
def test_a_nan_stays_one_without_a_limit(dt):
    for with_inf in (False, True):
        ts = grads(dt, "nan")
        if with_inf:
            ts[1][3] = math.inf
        total = dobb.dobb_clip_grad_norm_grouped(ts, math.inf)
        assert math.isnan(float(total)) and all(bool(t.isnan().all()) for t in ts)
