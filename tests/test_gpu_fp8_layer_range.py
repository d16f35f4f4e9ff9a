"""The layer of a few tokens where an activation between its products lies at the
end of fp32's range: next to infinity in bf16, and still finite."""
import numpy as np
import pytest
import torch

from expert_ffn_execution_router_amd import fp8

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("to", [3.38e38, 3.393e38, 3.4e38])
def test_activations_next_to_the_largest(to, sign):
    """silu(20) u = h with u chosen so that h is `to`, past bf16's largest value
    (3.3895e38) and below fp32's (3.4028e38).  h is off by at most 8 * 2^-23 of
    itself (exp, sum, quotient, two products), the down product of a single
    term, its scale, the weight of one and the result by half a step each:
    16 * 2^-23 in all."""
    print(f"layer range {to} {sign}", flush=True)
    H = I = 128
    x = torch.zeros(1, H, dtype=torch.bfloat16, device="cuda")
    x[0, 3] = 1.0
    gu = torch.zeros(1, 2 * I, H, device="cuda")
    gu[0, 5, 3], gu[0, I + 5, 3] = 16.0, 448.0 * sign
    dn = torch.zeros(1, H, I, device="cuda")
    dn[0, :, 5] = 1.0
    s_up = np.float32(to / 20 / 448)
    sgu = torch.tensor([[[1.25], [float(s_up)]]], device="cuda")
    sdn = torch.full((1, 1, 1), 2.0 ** -120, device="cuda")
    out = torch.empty(1, H, device="cuda")
    ids, w = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, device="cuda")
    fp8.layer(x, torch.zeros(1, H, device="cuda"), gu.to(F8), sgu, dn.to(F8), sdn, out, ids, w)
    h = sign * 20.0 / (1.0 + np.exp(-20.0)) * 448.0 * float(s_up)
    want = h * 2.0 ** -120
    assert abs(h) < 3.4028e38
    off = float((out.double() - want).abs().max())
    assert off <= 16 * 2.0 ** -23 * abs(want), (off, want)
