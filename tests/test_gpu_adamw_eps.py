"""AdamW's eps over its whole range: a parameter that never had a gradient (m = v = 0) stays, also with an eps that is not 0 but
below fp32's normal numbers; elsewhere such an eps changes nothing."""
import pytest
import torch

from moe_variable_size_amd import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-37, 1.1754943508222875e-38, 1e-38, 3e-39, 1e-44, 1e-50, 1e-300])
def test_least_eps(eps, bits):
    kind = torch.float32 if bits == 32 else torch.uint8
    n = 600

    def step(e):
        p, g = torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
        g[::2] = 0.25
        g[1] = 1e-12  # v = 1e-24 (1 - beta2)
        m, v = (torch.zeros(n, dtype=kind, device="cuda").view(torch.float32 if bits == 32 else torch.float8_e4m3fn) for _ in range(2))
        scales = dict(m_scales=[torch.zeros(3, device="cuda")], v_scales=[torch.zeros(3, device="cuda")]) if bits == 8 else {}
        api.moe_adamw_step([p], [g], [m], [v], step=1, lr=1e-2, eps=e, weight_decay=0.0, **scales)
        return p

    p = step(eps)
    assert (p[3::2] == 1).all()
    assert torch.equal(p[::2], step(0.0)[::2]) and p[1] == step(0.0)[1]
