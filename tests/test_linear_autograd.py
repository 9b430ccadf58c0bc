"""What the differentiable linear layer asks of its product (the product replaced; no GPU needed)."""
import pytest
import torch

from moe_variable_size_amd import api


@pytest.fixture
def calls(monkeypatch):
    seen = []

    def fwd(x, W, *, bias=None, act="none", residual=None, out_dtype=None, save_z=False):
        seen.append(save_z)
        z = x @ W.t()
        return (z, z) if save_z else z

    monkeypatch.setattr(api, "moe_linear_fwd", fwd)
    return seen


@pytest.mark.parametrize("act", ["none", "silu"])
def test_pre_activations_are_kept_only_for_a_backward(calls, act):
    x, W = torch.ones(2, 3), torch.ones(4, 3)
    Wp, bp = torch.nn.Parameter(W), torch.nn.Parameter(torch.zeros(4))
    r = torch.zeros(2, 4, requires_grad=True)
    needs = act != "none"
    for args, kw, want in (((x, W), {}, False), ((x, Wp), {}, needs), ((x, W, bp), {}, needs),
                           ((x, W), dict(residual=r), False)):
        api.linear(*args, act=act, **kw)
        assert calls.pop() is want
    with torch.no_grad():
        y = api.linear(x, Wp, bp, act=act)
    assert calls.pop() is False and not y.requires_grad
    with torch.inference_mode():
        api.linear(x, Wp, bp, act=act)
    assert calls.pop() is False
    assert api.linear(x, Wp, act=act).requires_grad and calls.pop() is needs
