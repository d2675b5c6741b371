"""The few-token layer where intermediate values leave the ordinary range."""
import pytest
import torch

import mixture_experts_fp32_b200 as moe

pytestmark = pytest.mark.gpu

INF = float("inf")
BF16_MAX, FP32_MAX = torch.finfo(torch.bfloat16).max, torch.finfo(torch.float32).max


@pytest.fixture(scope="module", autouse=True)
def built():
    from mixture_experts_fp32_b200 import build
    build.build()
    moe.load()


def test_h_at_and_past_the_end_of_the_range():
    """h = silu(g) * u infinite, and finite next to the end of fp32's range, where bf16 has no value:
    h enters the down product as two bf16 parts, which have to stand for it.  One feature of h
    is not 0 and every weight of the down product is 2^-10 or -2^-10, so the result is known: off
    by the two parts' 2^-16 and half a step of bf16."""
    T, H, E, I = 5, 256, 4, 256
    x = torch.zeros(T, H)
    gate_up, down = torch.zeros(E, 2 * I, H), torch.empty(E, H, I)
    down[:] = torch.where(torch.randn(E, H, I, generator=torch.Generator().manual_seed(2)) > 0,
                          2.0 ** -10, -2.0 ** -10)
    gate_up[:, 5, 0] = 1.0                        # g = x[0]
    gate_up[:, I + 5, 1] = 1.0                    # u = x[1] + x[2]
    gate_up[:, I + 5, 2] = 1.0
    x[0, :2] = torch.tensor([1e30, 1e30])         # h infinite
    x[1, :2] = torch.tensor([1e30, -1e30])
    x[2, :3] = torch.tensor([2.0 ** 64, 1.9921875 * 2.0 ** 63, 0.005859375 * 2.0 ** 63])
    x[3, 0], x[3, 1:3] = x[2, 0], -x[2, 1:3]
    x[4, :2] = torch.tensor([1.5, 3.0])
    h = x[:, 0].double() / (1 + torch.exp(-x[:, 0].double())) * (x[:, 1] + x[:, 2]).double()
    assert BF16_MAX * (1 + 2.0 ** -9) < h[2] < FP32_MAX and h[3] == -h[2]
    h = torch.where(h.abs() > FP32_MAX, torch.sign(h) * INF, h)
    ref = down[0, :, 5].double() * h[:, None]     # one expert, its weight 1
    plan = moe.Plan(max_tokens=T, hidden=H, num_experts=E, top_k_max=1, inter=I)
    t = dict(router_w=torch.zeros(E, H), w_gate_up=gate_up.bfloat16(), w_down=down.bfloat16())
    t = {n: v.cuda() for n, v in t.items()}
    xb = x.bfloat16().cuda()
    assert torch.equal(xb.float().cpu(), torch.where(x.abs() == 1e30, x.bfloat16().float(), x))
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    plan.forward_few(plan.weights(t["router_w"], None, t["w_gate_up"], t["w_down"]), xb, None, 1, out)
    assert plan.device_status() == 0
    got = out.cpu().double()
    assert torch.equal(got[:2], ref[:2])
    assert ((got[2:] - ref[2:]).abs() <= (2.0 ** -8 + 2.0 ** -15) * ref[2:].abs()).all()
