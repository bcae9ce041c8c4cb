"""The gradient through the gate where the slope is small or changes its sign, relative to the slope itself."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_slope(dtype):
    """The gradient through the gate, relative to itself: s and 1 - s are off by 2.5 * 2^-22 (expf by 1 ulp, the division by 2), so the
    slope s + gate s (1 - s) by 6 * 2^-22 of the magnitudes in it and with the products around it by 8; below the normal numbers
    e = exp(-|gate|) has steps of 2^-149, of which each of s and gate s is off by two."""
    import combine_topk_ids_histogram_gb300 as ep
    values = torch.cat([torch.linspace(-110, 110, 881), torch.linspace(-1.4, -1.2, 401), torch.tensor([0.0, -1e4, 1e4, -200.0, 200.0])])
    gate = values[:len(values) // 16 * 16].to(dtype).cuda()[None].expand(16, -1).contiguous()
    R, K = gate.shape
    up = torch.tensor([1.0, -3.0, 0.125, 100.0] * 4).to(dtype).cuda()[:, None].expand(R, K)
    d = torch.tensor([2.0, 1.0, -0.5, 0.25] * 4).to(dtype).cuda()
    g = torch.zeros(R, 16, dtype=dtype, device="cuda")
    g[:, 3] = d
    w = torch.zeros(1, 16, K, dtype=dtype, device="cuda")
    w[0, 3] = 1                                          # the sum has one term and is exact
    L = ref.layout_of(ep, [R])
    gx, _ = ep.expert_linear_bwd(g, None, w, L, gate_up=torch.cat([gate, up], 1).contiguous(), need=(True, False))
    v, u, d = gate.double(), up.double(), d.double()[:, None]
    s, rest = torch.sigmoid(v), torch.sigmoid(-v)
    want = torch.cat([d * u * (s + v * s * rest), d * v * s], 1)
    floor = 2 * 2.0 ** -149 * (1 + v.abs())
    err = torch.cat([(d * u).abs() * (8 * 2.0 ** -22 * (s + v.abs() * s * rest) + floor), d.abs() * (8 * 2.0 ** -22 * (v * s).abs() + floor)], 1)
    ref.assert_within(gx, want, ref.rounded(want, err, dtype), "gradient of gate and up")
