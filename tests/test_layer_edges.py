"""What the binding of the operators around the prefill sees of a call, without a GPU."""
import torch
from torch.autograd import forward_ad

from chunked_kda_prefill_b200 import _views


def test_tangents_count_as_wanted_gradients():
    t, leaf = torch.ones(3), torch.ones(3, requires_grad=True)
    assert not _views.needs_grad(t, None) and _views.needs_grad(None, t, leaf)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(t, t)
        for grad in (torch.enable_grad, torch.no_grad):
            with grad():
                assert _views.needs_grad(None, dual) and _views.needs_grad(leaf, dual)
                assert not _views.has_tangent(t, leaf, None)
    with torch.no_grad():
        assert not _views.needs_grad(leaf, t)
