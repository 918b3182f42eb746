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


def tail_formula(z, ids, values, w):
    """(loss, gradient, magnitude of its terms, magnitude of the loss's terms) of
    the form with the tail at temperature 1, with log p_r as a log-sum-exp of its own
    so that no p_r is too small for it."""
    z, values, w = z.double(), values.double(), w.double()[:, None]
    R, V = z.shape
    logp = torch.log_softmax(z, -1)
    some = ids != F.IGNORE
    spot = torch.where(some, ids, torch.full_like(ids, V))
    q = torch.where(some, torch.exp(values), torch.zeros_like(values))
    qv = torch.zeros(R, V + 1, dtype=torch.float64).scatter_add_(1, spot, q)[:, :V]
    on = torch.zeros(R, V + 1, dtype=torch.bool).scatter_(1, spot, True)[:, :V]
    far = torch.logsumexp(logp.masked_fill(on, -math.inf), -1, keepdim=True)
    rest = (1.0 - q.sum(-1, keepdim=True)).clamp_min(0.0)
    at = logp.gather(1, ids.clamp_min(0))
    loss = torch.where(some, q * (values - at), torch.zeros_like(q)).sum(-1) + (rest * (rest.log() - far))[:, 0]
    mags = torch.where(some, q * (values.abs() + at.abs()), torch.zeros_like(q)).sum(-1) \
        + (rest * (rest.log().abs() + far.abs()))[:, 0]
    # (Not exp(logp - far): at 3.4e38 a difference in fp64 has no units left.)
    share = torch.softmax(z.masked_fill(on, -math.inf), -1)
    grad = torch.where(on, logp.exp() - qv, share * (far.exp() - rest)) * w
    mag = torch.where(on, logp.exp() + qv, share * (far.exp() + rest)) * w.abs()
    return loss, grad, mag, mags


def check_tail(S, z, ids, values, w, dtype, rows):
    ref, gref, mag, mags = tail_formula(z[rows], ids[rows], values[rows], w[rows])
    # Each logarithm's sum is off by SUM, and the rounding of the scale
    # log2(e) / T to fp32 moves every log p by up to 2^-24 of itself; so it
    # does p_r in the gradient, whose ONE holds that up to 400 nats (4 ONE of
    # a p_r below e^-400 are nothing).
    bound = 4 * F.SUM + 2.0 ** -24 * (ref.abs() + mags)
    for loss, grad in both_ways(S, z, ids, values, w, 1.0, True):
        F.assert_within(loss[rows], ref, bound, "loss")
        F.check_grad(grad[rows], gref, mag, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["160 80", "120 60", "300", "-1e4", "lowest", "far"])
@pytest.mark.parametrize("R,V", LAYOUTS)
def test_tail_far_below_the_list(S, R, V, kind, dtype):
    """The probability off the list may be below fp32's range, with a listed
    entry between the largest one and those off the list or none, finite masks
    off the list among them: loss and gradient are finite, and depend neither on
    the layout nor on where the listed entries stand.  Upstream gradients of a
    scaled loss among them."""
    g = torch.Generator().manual_seed(R + V)
    z = torch.rand(R, V, generator=g) / 2
    ids = torch.stack([torch.randperm(V, generator=g)[:4] for _ in range(R)])
    ids[:, 3] = F.IGNORE
    ids[1, 2] = F.IGNORE
    listed = {"160 80": [160.0, 80.0, 80.5], "120 60": [120.0, 60.0, 1.0], "300": [300.0, 299.0, 298.0],
              "-1e4": [3.0, 2.0, 1.0], "lowest": [3.0, 2.0, 1.0], "far": [3e9, 3e9, 0.0]}[kind]
    if kind == "far" and dtype == torch.float16:
        listed = [60000.0, 30000.0, 0.0]
    if kind == "-1e4":
        z -= 10000.0
    if kind == "lowest":
        z[:] = torch.finfo(dtype).min
    for j, v in enumerate(listed):
        rows = ids[:, j] != F.IGNORE
        z[rows, ids[rows, j]] = v
    z = z.to(dtype)
    values = torch.log(torch.tensor([[0.5, 0.2, 0.1, 1.0]] * R))
    w = torch.rand(R, generator=g) + 0.5
    if dtype != torch.float16:
        w[2], w[3] = 65536.0, -65536.0
    check_tail(S, z, ids, values, w, dtype, list(range(6)))


@pytest.mark.parametrize("R,V", LAYOUTS)
@pytest.mark.parametrize("vtype", TYPES)
def test_complete_lists_of_masked_students(S, R, V, vtype):
    """A list of all that a student allows, the others masked by a finite
    value: what the rounding of the list's values leaves of one does not meet
    the masks."""
    g = torch.Generator().manual_seed(3)
    z = torch.full((R, V), -1e4)
    ids = torch.stack([torch.randperm(V, generator=g)[:5] for _ in range(R)])
    allowed = torch.randn(R, 5, generator=g)
    z.scatter_(1, ids, allowed)
    values = torch.log_softmax(torch.randn(R, 5, generator=g).double(), -1).to(vtype)
    w = torch.ones(R)
    q, logp = values.double().exp(), torch.log_softmax(allowed.double(), -1)
    ref = (q * (values.double() - logp)).sum(-1)
    for loss, grad in both_ways(S, z, ids, values, w, 1.0, True):
        F.assert_within(loss, ref, 4 * F.SUM + 2.0 ** -23 * ref.abs())
        off = torch.ones(R, V, dtype=torch.bool).scatter_(1, ids, False)
        assert bool((grad[off] == 0).all())
        # p - q: two exponentials of either, and the gradient's rounding
        F.assert_within(grad.gather(1, ids), logp.exp() - q, 4 * F.ONE * (logp.exp() + q) + 2.0 ** -24)


@pytest.mark.parametrize("R,V", [(2000, 1), (1100, 250), (1100, 3001), (300, 3001), (9, 140001)])
@pytest.mark.parametrize("dtype", TYPES)
def test_log_probabilities_are_never_positive(S, R, V, dtype):
    """One entry with all of the probability (a vocabulary of one, one allowed
    entry, a sure row): its log-probability is at most 0, and so are the others."""
    g = torch.Generator().manual_seed(V)
    z = (torch.randn(R, V, generator=g) * 5).to(dtype)
    best = torch.randint(0, V, (R, 1), generator=g)
    top = torch.rand(R, 1, generator=g) * 40
    z[: R // 2] = -math.inf                              # one allowed entry
    z.scatter_(1, best, (top + 60.0).to(dtype))
    z[-1, 0] = math.nan
    k = min(V, 5)
    r = S.token_logprobs(z.to(DEV), best[:, 0].to(DEV), temperature=0.7, top_k=k)
    assert bool(torch.isnan(r.logprobs[-1])) and bool(torch.isnan(r.top_logprobs[-1]).all())
    assert bool((r.logprobs[:-1] <= 0).all()), float(r.logprobs[:-1].max())
    assert bool((r.top_logprobs[:-1] <= 0).all()), float(r.top_logprobs[:-1].max())
    some = torch.arange(0, R, max(1, R // 8))
    F.check_token_values(S.TokenLogProbs(*(x[some] for x in r)), z[some], best[some, 0], 0.7, k)


@pytest.mark.parametrize("make", [lambda: torch.empty(2, 0, 3, 8), lambda: torch.empty(0, 8, 4).transpose(1, 2),
                                  lambda: torch.empty(3, 0, 8)])
def test_batches_without_rows(S, make):
    z = make().to(DEV).requires_grad_(True)
    shape = z.shape[:-1]
    r = S.token_logprobs(z, torch.zeros(shape, dtype=torch.int64, device=DEV), top_k=2)
    assert r.logprobs.shape == shape and r.top_tokens.shape == (*shape, 2)
    ids = torch.zeros(*shape, 3, dtype=torch.int32, device=DEV)
    loss = S.distillation_loss(z, ids, torch.zeros(*shape, 3, device=DEV), tail=True)
    (r.logprobs.sum() + r.entropy.sum() + r.top_logprobs.sum() + loss.sum()).backward()
    assert loss.shape == shape and z.grad.shape == z.shape
    loss, grad = S.distillation_value_and_grad(z, ids, torch.zeros(*shape, 3, device=DEV))
    assert loss.shape == shape and grad.shape == z.shape


@pytest.mark.parametrize("R,V,K", [(2000, 4000, 256), (300, 20011, 250), (1100, 500, 64)])
def test_repeated_ids_give_the_same_bits(S, monkeypatch, R, V, K):
    """A list whose ids stand several times, their copies in different waves:
    which of them counts in p does not go by the order in which waves get there
    (the build with pseudo-random delays mixes it).  The student is near the
    teacher, so that the loss is as small as its sums' last bits."""
    from differentiable_series_alignment_amd import _lib
    g = torch.Generator().manual_seed(K)
    z = torch.randn(R, V, generator=g) * 8     # (a narrow range of exponentials sums exactly)
    ids = torch.stack([torch.randperm(V, generator=g)[:K // 2].repeat(2)[torch.randperm(K, generator=g)]
                       for _ in range(R)])
    values = (torch.log_softmax(z.double(), -1).gather(1, ids) - math.log(2.0)).float()
    w = torch.rand(R, generator=g) + 0.5
    args = [x.to(DEV) for x in (z, ids, values, w)]
    loss, grad = S.distillation_value_and_grad(*args, tail=True)
    some = list(range(0, R, R // 6))
    ref, gref, mag, mags = F.distill(z[some], ids[some], values[some], 1.0, True, w[some])
    F.assert_within(loss[some], ref, 4 * F.SUM + 2.0 ** -24 * ref.abs() + 1e-12 * mags)
    F.check_grad(grad[some].cpu(), gref, mag, torch.float32)
    plain = S.distillation_loss(*args[:3], tail=True)
    monkeypatch.setattr(_lib, "_lib", _lib.load(_lib.STRESS_LIB_PATH))
    for _ in range(8):
        loss1, grad1 = S.distillation_value_and_grad(*args, tail=True)
        assert torch.equal(loss, loss1), int((loss != loss1).sum())
        assert torch.equal(grad, grad1)
        assert torch.equal(plain, S.distillation_loss(*args[:3], tail=True))


@pytest.mark.parametrize("vtype", TYPES)
@pytest.mark.parametrize("R,V", [(2000, 100), (9, 100)])
def test_complete_lists_of_computed_log_probabilities(S, R, V, vtype):
    """A teacher's log-probabilities over the whole vocabulary, computed in
    fp32: their log-sum-exp near 30 is off by up to half a step there, 2^-20,
    and so is the list's sum.  That is no class of its own, also where the
    teacher is sure."""
    g = torch.Generator().manual_seed(R)
    t = torch.randn(R, V, generator=g) * 2 + 15
    t[:, 3] = 30.0 + torch.rand(R, generator=g)
    z = torch.randn(R, V, generator=g)
    ids = torch.arange(V).repeat(R, 1)
    own = S.token_logprobs(t.to(DEV), top_k=V)
    plain = t - torch.logsumexp(t, -1, keepdim=True)
    for i, v in ((own.top_tokens.cpu(), own.top_logprobs.cpu()), (ids, plain)):
        v = v.to(vtype)
        q = torch.exp(v.double())
        ref = (q * (v.double() - torch.log_softmax(z.double(), -1).gather(1, i))).sum(-1)
        for loss, grad in both_ways(S, z, i, v, torch.ones(R), 1.0, True):
            F.assert_within(loss, ref, 4 * F.SUM + 2.0 ** -23 * ref.abs())
            assert bool(torch.isfinite(grad).all())
