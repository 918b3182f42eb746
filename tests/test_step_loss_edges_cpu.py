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
