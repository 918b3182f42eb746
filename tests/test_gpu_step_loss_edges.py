"""Edges of the step losses on the GPU: rows without entries, log-probabilities
at their upper end, students that are far surer of a list than of the rest,
lists with repeated ids, empty batches.  Tolerances are derived in
_rows_ref.py, but for those stated here."""
import math

import pytest
import torch

import _rows_ref as F

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]
# A wave per row, a block per row, a row in parts (and a block again in the
# one call, whose rows a wave takes up to 256 or 512 entries).
LAYOUTS = [(1100, 250), (1100, 3001), (9, 3001), (9, 140001)]


@pytest.fixture(scope="module")
def S():
    import differentiable_series_alignment_amd as pkg
    from differentiable_series_alignment_amd import _lib
    _lib.lib()   # loud failure if the HIP library is missing
    return pkg


def both_ways(S, z, ids, values, w, temperature, tail):
    """(loss, gradient) through autograd and of the one call, on the CPU."""
    zd = z.to(DEV).requires_grad_(True)
    i, v, wd = ids.to(DEV), values.to(DEV), w.to(DEV)
    loss = S.distillation_loss(zd, i, v, temperature=temperature, tail=tail)
    grad, = torch.autograd.grad([loss], [zd], [wd])
    one = S.distillation_value_and_grad(zd, i, v, wd, temperature, tail)
    return [(loss.detach().cpu(), grad.cpu()), tuple(x.cpu() for x in one)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("R,V", LAYOUTS)
def test_rows_without_entries(S, R, V, tail, dtype):
    """Loss 0 and gradient 0 whatever the logits and the upstream gradient
    hold; the rows beside them keep theirs."""
    g = torch.Generator().manual_seed(R + V)
    z = torch.randn(R, V, generator=g).to(dtype)
    ids = torch.randint(0, V, (R, 3), generator=g)
    ids[:, 1:] = F.IGNORE
    values = torch.full((R, 3), math.log(0.5))
    w = torch.rand(R, generator=g) + 0.5
    ids[:6] = F.IGNORE
    z[1] = -math.inf
    z[2, V // 2] = math.nan
    z[3, 5] = math.inf
    z[4] = math.nan
    w[5] = math.nan
    some = [6, 7, 8]
    ref, gref, mag, mags = F.distill(z[some], ids[some], values[some], 1.0, tail, w[some])
    for loss, grad in both_ways(S, z, ids, values, w, 1.0, tail):
        assert bool((loss[:6] == 0).all()), loss[:6]
        assert bool((grad[:6] == 0).all()), [bool((x == 0).all()) for x in grad[:6]]
        F.assert_within(loss[some], ref, 4 * F.SUM + 2.0 ** -24 * ref.abs() + 1e-12 * mags)
        F.check_grad(grad[some], gref, mag, dtype)
    # a listed entry of no probability is an entry with the tail, none without
    ids[2, 0], values[2, 0] = 1, -math.inf
    for loss, grad in both_ways(S, z, ids, values, w, 1.0, tail):
        assert math.isnan(float(loss[2])) if tail else float(loss[2]) == 0.0
        assert bool(torch.isnan(grad[2]).all()) if tail else bool((grad[2] == 0).all())
