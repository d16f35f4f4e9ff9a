"""GPU tests of the norms' C calls where the torch layer passes less: no rows."""
import pytest
import torch

from expert_ffn_execution_router_amd import binding as B

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("n", [40, 512, 700, 2048, 4096, 4100])
@pytest.mark.parametrize("per_column", [0, 1])
def test_no_rows_give_sums_of_zero_and_touch_nothing(n, per_column):
    """Rows and gate of no rows have addresses, as a C caller's empty arrays may
    (here inside other tensors): the column sums are zeros and nothing of a row,
    nor the workspace that holds rows' sums, is touched."""
    print(f"no rows n={n} per_column={per_column}", flush=True)
    rows = torch.zeros(8, n, dtype=BF, device="cuda")
    w = torch.ones(n, dtype=BF, device="cuda")
    need = B.moe_norm_backward_workspace_bytes(0, n)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
    dw, dw2 = (torch.full((n,), 9.0, device="cuda") for _ in range(2))
    bf16 = B.MOE_T_BF16
    at = [r.data_ptr() for r in rows]
    B.check(B.lib().moe_norm_backward(bf16, bf16, at[0], n, at[1], n, 1.0, bf16, w.data_ptr(), bf16, at[2],
                                      n if per_column else 1, per_column, at[3], n, at[4], n, w.data_ptr(), at[5], n,
                                      at[6], n, dw.data_ptr(), bf16, None, 0, 0, dw2.data_ptr(), 0, n, 1e-6, 1e-6,
                                      ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert (dw == 0).all() and (dw2 == 0).all()
    assert (ws == 0xA5).all() and (rows == 0).all()
