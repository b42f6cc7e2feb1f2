"""Rows of the expert-contiguous row space that hold no token: what the layer's
backward pass says of them does not depend on what the buffers held before."""
import pytest
import torch

from mixture_experts_layer_59_b200 import binding as B
from mixture_experts_layer_59_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("round_mode,capacity", [(B.MOE_ROUND_NONE, -1), (B.MOE_ROUND_NEAREST, -1), (B.MOE_ROUND_CAPACITY, 70)])
def test_dS_of_rows_without_a_token_is_zero(dtype, round_mode, capacity):
    T, d, f, E, k = 500, 256, 128, 16, 3
    cfg = synth.MoEConfig("padding", T, d, f, E, k, std=0.05, routing="zipf")
    inp = synth.make_inputs(cfg, seed=3, device="cuda")
    x, wg, w1, w3, w2, dout = (inp[n].to(dtype) for n in ("x", "w_gate", "w1", "w3", "w2", "dout"))
    lo = torch.randn(T, E, generator=torch.Generator().manual_seed(1)).cuda()
    logits, idx, gate = B.moe_route(x, wg, k, logits_override=lo)
    plan = B.moe_permute(idx, gate, logits, E, round_mode, capacity=capacity)
    H, _ = B.moe_expert_ffn_fwd(x, w1, w3, w2, plan, k)
    cap, R = B.moe_row_capacity(T, E, k), int(plan["offsets"][-1])
    grads = []
    for fill in (float("nan"), 7.0):
        dS = torch.full((cap,), fill, device="cuda")
        g = B.moe_layer_bwd(dout, x, wg, w1, w3, w2, idx, gate, plan, H, out=dict(dS=dS), logits=logits)
        B.moe_check_status()
        grads.append(g)
    live = torch.zeros(cap, dtype=torch.bool, device="cuda")
    live[:R] = plan["row_token"][:R] >= 0
    assert 0 < int(live.sum()) < cap
    for g in grads:
        assert not g["dS"][~live].any()
        assert torch.isfinite(g["dS"]).all() and g["dS"][live].any()
    assert all(torch.equal(grads[0][n], grads[1][n]) for n in grads[0])


def test_dS_of_rows_without_a_token_is_zero_mxfp8():
    T, d, f, E, k = 500, 256, 128, 16, 3
    cfg = synth.MoEConfig("padding", T, d, f, E, k, std=0.05, routing="zipf")
    inp = synth.make_inputs(cfg, seed=3, device="cuda")
    from mixture_experts_layer_59_b200.layer import MoELayerStep
    step = MoELayerStep(T, d, f, E, k, precision="mxfp8")
    step.grads["dS"].fill_(float("nan"))
    lo = torch.randn(T, E, generator=torch.Generator().manual_seed(1)).cuda()
    step.forward(inp["x"], inp["w_gate"], inp["w1"], inp["w3"], inp["w2"], logits_override=lo)
    g = step.backward(inp["dout"])
    B.moe_check_status()
    R = int(step.plan["offsets"][-1])
    live = torch.zeros_like(g["dS"], dtype=torch.bool)
    live[:R] = step.plan["row_token"][:R] >= 0
    assert not g["dS"][~live].any() and torch.isfinite(g["dS"]).all()
