"""The SwiGLU epilogue of the e4m3 gate/up product against its formula in 64 bits, where e4m3 does not hide its error."""
import numpy as np
import pytest
import torch

from test_gpu_fp8_block import workspace

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _build():
    from serve_invariant_moe_gb300 import build
    build.build()


def scales(g, T):
    """h_scale of rows whose gate and up values are all g: |silu(g) g| / 448."""
    from serve_invariant_moe_gb300 import binding
    F = H = 128
    a = torch.zeros(T, H)
    a[:, 5] = g.sign()
    w13 = torch.zeros(1, 2 * F, H)
    w13[:, :, 5] = 1.0                                       # one product per output: g and u are exact
    w = workspace()
    r = binding.moe_grouped_swiglu_fp8(a.to(torch.float8_e4m3fn).to(DEV), g.abs().unsqueeze(1).contiguous().to(DEV), None,
                                       w13.to(torch.float8_e4m3fn).to(DEV), torch.ones(1, 2, 1, device=DEV), T, 1, w)
    binding.check_status(w)
    x = g.double().numpy()
    return r, np.abs(x / (1 + np.exp(-x)) * x) / 448


@pytest.mark.parametrize("T", [3, 40, 300])                  # 40 rows: column tiles, 300: row tiles
def test_h_is_fp32_at_any_gate(T):
    """exp's 2 units in the last place (4 u, u = 2^-24), the sum, a reciprocal within a unit (2 u), two products and the
    division by 448: 10 u relative, which the fp32 scale of h shows."""
    g = torch.linspace(-80, 80, T)
    g[g.abs() < 1e-3] = 1.0
    r, want = scales(g, T)
    got = r["h_scale"].double().cpu().numpy()[:, 0]
    err = (np.abs(got - want) / want).max() * 2 ** 24
    assert err <= 10, f"{err:.1f} u"
    assert (r["h"].float().abs() == 448).all()


@pytest.mark.parametrize("T", [3, 40, 300])
def test_h_of_gates_at_the_edge_of_fp32(T):
    """exp(-g) near and above the largest fp32 number: its reciprocal is a subnormal with at least 20 bits, then 0, where the
    formula is below 89 * 2^-128 of u; nothing is NaN."""
    g = torch.linspace(-88.7, -86.0, T)
    r, want = scales(g, T)
    got = r["h_scale"].double().cpu().numpy()[:, 0]
    assert (np.abs(got - want) <= (10 * 2.0 ** -24 + 2.0 ** -20) * want + 2.0 ** -149).all()
    r, want = scales(torch.linspace(-120.0, -88.73, T), T)
    got = r["h_scale"].double().cpu().numpy()[:, 0]
    assert (np.abs(got - want) <= 89 * 2.0 ** -128 * 120 / 448 + 2.0 ** -126).all()
    assert torch.isfinite(r["h"].float()).all()
