"""What the combine's mask drops is selected away in both directions: an
infinity or a NaN under it, in the experts' rows or in dy, reaches no output."""
import pytest
import torch

import moe_expert_layer_topk_gb300 as m
import ops_ref
from test_gpu_dropout import combine_inputs, rng

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,k", [(1, 64, 1), (33, 192, 3), (40, 2048, 8), (7, 4160, 2), (9, 320, 17)])
def test_dropped_rows_and_gradients_do_not_show(T, H, k):
    p, seed = 0.5, 23
    c = {n: v.cuda() for n, v in combine_inputs(T, H, k, seed=H).items()}
    keep = torch.from_numpy(ops_ref.keep(seed, 0, 0, T * H, p).reshape(T, H)).cuda()

    def run():
        y, dyp, dw = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty_like(c["y_perm"]), torch.empty(T, k, device="cuda")
        m.moe_combine_dropout(c["y_perm"], c["topk_w"], c["row_of_slot"], c["residual"], T, H, k, p, rng(seed), y)
        m.moe_combine_dropout_bwd(c["dy"], c["y_perm"], c["topk_w"], c["row_of_slot"], T, H, k, p, rng(seed), dyp, dw)
        return y, dyp, dw

    clean = run()
    junk = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda")[torch.arange(H, device="cuda") % 3].bfloat16()
    rows = c["row_of_slot"].long()
    c["y_perm"][rows] = torch.where(keep[:, None, :], c["y_perm"][rows], junk)
    c["dy"] = torch.where(keep, c["dy"], junk)
    for got, want, name in zip(run(), clean, ("y", "dy_perm", "d_w")):
        assert torch.equal(got, want), name
    # and under a mask that drops everything
    c["y_perm"][:], c["dy"][:] = float("nan"), float("inf")
    p = 1.0
    y, dyp, dw = run()
    assert torch.equal(y, c["residual"]) and not dyp.any() and not dw.any()
