"""The norm's gradients without grad_weight on the host (no GPU): the workspace is not looked at.

The call has no rows, so nothing is launched."""
import os

import pytest

import moe_expert_load_ultraep_amd as U

pytestmark = pytest.mark.skipif(not os.path.exists(U.LIB_PATH), reason="libultraep.so not built")

F = 1 << 20   # never dereferenced


@pytest.mark.parametrize("workspace,size", [(None, 0), (F + 4, 0), (F + 8, 100), (F, 0)])
def test_workspace_without_grad_weight(workspace, size):
    ctx = U.ultraep_create(8, 4, 1, 4)
    assert U.lib().ultraep_residual_norm_backward(ctx.handle, F, F, 0, F, 0, F, None, 0, 64, F, None, None, 0, workspace, size, None) == 0
    assert U.lib().ultraep_residual_norm_backward(ctx.handle, F, F, 0, F, 0, F, None, 3, 64, F, None, F, 0, F + 8, 1 << 30, None) == -2
