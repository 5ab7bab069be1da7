"""The operators around a layer record no gradient: while autograd records they
refuse inputs that require one, before anything else is looked at."""
import pytest
import torch

import moe_token_re_amd as moe


def leaf(*shape):
    return torch.zeros(shape, requires_grad=True)


CALLS = {
    "rms_norm x": lambda t, w: moe.rms_norm(t, w.detach()),
    "rms_norm weight": lambda t, w: moe.rms_norm(t.detach(), w),
    "rms_norm residual": lambda t, w: moe.rms_norm(t.detach(), w.detach(), residual=t),
    "rms_norm quantize": lambda t, w: moe.rms_norm(t, w.detach(), quantize="int8"),
    "rms_norm out": lambda t, w: moe.rms_norm(t, w.detach(), out=(torch.zeros_like(t), None, None)),
    "moe_router_top_k": lambda t, w: moe.moe_router_top_k(t, 2),
    "moe_token_permute tokens": lambda t, w: moe.moe_token_permute(t, index(), 4),
    "moe_token_permute weight": lambda t, w: moe.moe_token_permute(t.detach(), index(), 4, expert_weight=leaf(2, 1)),
    "moe_token_permute scales": lambda t, w: moe.moe_token_permute(t.detach(), index(), 4, per_token_scales=leaf(2)),
    "moe_token_unpermute rows": lambda t, w: moe.moe_token_unpermute(t, index()),
    "moe_token_unpermute weight": lambda t, w: moe.moe_token_unpermute(t.detach(), index(), expert_weight=leaf(2, 1)),
}


def index():
    return torch.zeros(2, 1, dtype=torch.int32)


@pytest.mark.parametrize("name", CALLS)
def test_a_gradient_is_not_lost(name):
    with pytest.raises(ValueError, match=f"{name.split()[0]} records no gradient"):
        CALLS[name](leaf(2, 64), leaf(64))
    # nothing is recorded here: the next check refuses these tensors, of which none is on a GPU
    for quiet in (torch.no_grad, torch.inference_mode):
        with quiet(), pytest.raises(ValueError, match="GPU"):
            CALLS[name](leaf(2, 64), leaf(64))


def test_gradients_are_functions_of_any_tensors():
    """What comes back from a *_backward call is a gradient, and is not led further."""
    x, w, i = leaf(2, 64), leaf(64), index()
    for call in (lambda: moe.rms_norm_backward(x, x, w), lambda: moe.moe_router_top_k_backward(x, x, x, i),
                 lambda: moe.moe_token_permute_backward(x, i), lambda: moe.moe_token_unpermute_backward(x, x, i)):
        with pytest.raises(ValueError, match="GPU"):
            call()
