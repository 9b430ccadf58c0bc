"""What the differentiable routing calls hand to the library (the calls replaced; no GPU needed)."""
import torch

from moe_variable_size_amd import api


def test_strided_operands_are_laid_out_densely(monkeypatch):
    """As the differentiable linear layer does: any strides of the logits, the bias and the ids."""
    seen = {}

    def route(logits, k, *, bias=None, **kw):
        seen.update(logits=logits, bias=bias)
        return torch.zeros(logits.shape[0], k, dtype=torch.int32), torch.zeros(logits.shape[0], k)

    def loss(logits, ids, *, score):
        seen.update(logits=logits, ids=ids)
        return torch.zeros(2), torch.zeros(logits.shape[1] + 1)

    monkeypatch.setattr(api, "moe_route_fwd", route)
    monkeypatch.setattr(api, "moe_router_loss_fwd", loss)
    l = torch.arange(12.0).view(4, 3).t()
    bias = torch.arange(8.0)[::2]
    ids = torch.arange(6, dtype=torch.int32).view(2, 3).t()
    api.route(l, 2, bias=bias)
    assert seen["logits"].is_contiguous() and torch.equal(seen["logits"], l)
    assert seen["bias"].is_contiguous() and torch.equal(seen["bias"], bias)
    api.route(l, 2, bias=None)
    assert seen["bias"] is None
    api.router_loss(l, ids)
    assert seen["ids"].is_contiguous() and torch.equal(seen["ids"], ids)
