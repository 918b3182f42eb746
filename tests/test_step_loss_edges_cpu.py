"""Edges of the step losses that need no GPU: how tensors are walked, and
refusals."""
import pytest
import torch

import differentiable_series_alignment_amd as S
from differentiable_series_alignment_amd import token_losses as T


@pytest.mark.parametrize("make", [lambda: torch.empty(2, 0, 3, 8), lambda: torch.empty(0, 2, 3, 8),
                                  lambda: torch.empty(2, 3, 0, 8), lambda: torch.empty(0, 8, 4).transpose(1, 2),
                                  lambda: torch.empty(3, 0, 2, 4).transpose(0, 2), lambda: torch.empty(0, 5)])
def test_walks_of_empty_tensors(make):
    """No rows: the tensor itself, whatever its strides."""
    t = make()
    walked, outer, inner = T._walk(t, t.dim() - 1)
    assert walked is t and (outer, inner) == (0, 0)


def test_walks():
    """Two strides reach every row, or a copy is walked."""
    z = torch.arange(2 * 3 * 4 * 5.0).view(2, 3, 4, 5)
    for t in (z, z[:, :, 1:], z.transpose(1, 2), z[:1], z[..., ::2], z[:, :1].expand(2, 3, 4, 5), z[0, 0], z[0, 0, 0]):
        lead = t.dim() - 1
        w, outer, inner = T._walk(t, lead)
        n = t.shape[-2] if lead else 1
        flat = w.as_strided((w.untyped_storage().nbytes() // 4 - w.storage_offset(),), (1,))
        rows = [flat[(r // n) * outer + (r % n) * inner:][:t.shape[-1]] for r in range(t[..., 0].numel())]
        assert torch.equal(torch.stack(rows), t.reshape(-1, t.shape[-1]))


CALLS = [lambda z, i, v: S.token_logprobs(z, i[:, 0]), lambda z, i, v: S.token_logprobs(z, top_k=2),
         S.distillation_loss, S.distillation_value_and_grad, S.DistillationLoss()]


@pytest.mark.parametrize("call", CALLS)
def test_forward_mode_is_refused(call):
    """A tangent would be lost without a word."""
    import torch.autograd.forward_ad as fw
    z, i, v = torch.randn(2, 10), torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, 3)
    with fw.dual_level():
        dual = fw.make_dual(z, torch.ones_like(z))
        with pytest.raises(ValueError, match="forward-mode"):
            call(dual, i, v)
        with pytest.raises(ValueError, match="forward-mode"):
            call(dual.clone().requires_grad_(True), i, v)
        with pytest.raises(ValueError, match="GPU"):       # no tangent, no refusal of that kind
            call(z, i, v)
        with torch.no_grad(), pytest.raises(ValueError, match="forward-mode"):
            call(dual, i, v)
    with pytest.raises(ValueError, match="forward-mode"):
        torch.func.jvp(lambda x: call(x, i, v), (z,), (torch.ones_like(z),))


def test_forward_mode_of_what_goes_beside_is_refused():
    import torch.autograd.forward_ad as fw
    z, i, v = torch.randn(2, 10), torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, 3)
    with fw.dual_level():
        dual = fw.make_dual(v, torch.ones_like(v))
        for call in CALLS[2:]:
            with pytest.raises(ValueError, match="forward-mode"):
                call(z, i, dual)
        w = fw.make_dual(torch.ones(2), torch.ones(2))
        with pytest.raises(ValueError, match="forward-mode"):
            S.distillation_value_and_grad(z, i, v, w)


@pytest.mark.parametrize("bad", [1 << 63, -(1 << 63) - 1, (1 << 64) - 100, -100.5, float("nan"), float("inf"), None, "x"])
def test_ignore_index_is_an_int64(bad):
    """One that wraps to another id, or is rounded to one, would drop that id."""
    z, i, v = torch.randn(2, 10), torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, 3)
    for call in (lambda: S.token_logprobs(z, i[:, 0], ignore_index=bad),
                 lambda: S.distillation_loss(z, i, v, ignore_index=bad),
                 lambda: S.distillation_value_and_grad(z, i, v, ignore_index=bad),
                 lambda: S.DistillationLoss(ignore_index=bad)):
        with pytest.raises(ValueError, match="ignore_index"):
            call()


@pytest.mark.parametrize("good", [0, -100, -100.0, (1 << 63) - 1, -(1 << 63), True])
def test_ignore_index_of_other_kinds(good):
    z, i, v = torch.randn(2, 10), torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, 3)
    assert S.DistillationLoss(ignore_index=good).ignore_index == int(good)
    with pytest.raises(ValueError, match="GPU"):
        S.token_logprobs(z, i[:, 0], ignore_index=good)
    with pytest.raises(ValueError, match="GPU"):
        S.distillation_value_and_grad(z, i, v, ignore_index=good)
