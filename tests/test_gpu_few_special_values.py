"""The few-token layer where values leave the ordinary range, ties among experts of every lane, and the
quantiser's scale where it underflows."""
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


@pytest.mark.parametrize("E,equal,above", [(40, (39, 17, 18), ()), (40, (33, 1, 32, 0), ()),
                                           (256, (255, 17, 67, 200), ()),
                                           (256, (64, 63, 191, 31, 32), (250,)),
                                           (64, (63, 62, 61), (5, 40))])
def test_ties_among_high_experts(E, equal, above):
    """Experts with the same router row have the same logit in every token: they are taken in
    ascending order, after those above them and before the rest, wherever a lane holds them."""
    T, H = 6, 256
    g = torch.Generator().manual_seed(E + len(equal))
    x = (torch.rand(T, H, generator=g) + 0.5).bfloat16()
    router = -torch.rand(E, H, generator=g)       # the others' logits are negative
    router[list(equal)] = torch.rand(H, generator=g)
    for i, e in enumerate(above):
        router[e] = 2.0 + (len(above) - i)
    k = len(equal) + len(above)
    plan = moe.Plan(max_tokens=T, hidden=H, num_experts=E, top_k_max=k, inter=128)
    w = [t.cuda() for t in (router, torch.randn(E, 256, H, generator=g).bfloat16(),
                            torch.randn(E, H, 128, generator=g).bfloat16())]
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    wt = torch.full((T, k), -7.0, device="cuda")
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    plan.forward_few(plan.weights(w[0], None, w[1], w[2]), x.cuda(), None, k, out,
                     dbg=moe.make_debug(topk_ids=ids, topk_w=wt))
    assert plan.device_status() == 0
    assert ids.tolist() == [list(above) + sorted(equal)] * T
    tied = wt[:, len(above):]
    assert (tied == tied[:, :1]).all()
    assert above or (tied > 0).all()
    fewer = ids[:, :k - 1].clone()                # and the lowest of them where not all fit
    ids2 = torch.full((T, k - 1), -7, dtype=torch.int32, device="cuda")
    plan.forward_few(plan.weights(w[0], None, w[1], w[2]), x.cuda(), None, k - 1, out,
                     dbg=moe.make_debug(topk_ids=ids2))
    assert torch.equal(ids2, fewer)


def test_fp8_tokens_do_not_leak_into_one_another():
    """e4m3 weights: an infinite or NaN hidden state and an expert with NaN codes touch only the rows
    that read them; the others stay within the FP8 layer's 6e-2 x RMS (codes of h at a border may round
    the other way, since sums are cut elsewhere when the set of experts changes)."""
    import synth
    from moe_harness import plan_for, to_device, weights_of
    from synth.workloads import Workload
    w = Workload("leak8", T=12, H=384, E=16, k=2, I=256, S=1, Is=128, router_sigma=0.1, wtype="fp8",
                 w_sigma=0.05)
    d = to_device(synth.make_inputs(w))
    plan = plan_for(w)

    def run():
        out = torch.full((w.T, w.H), -1.0, dtype=torch.bfloat16, device="cuda")
        ids = torch.full((w.T, w.k), -7, dtype=torch.int32, device="cuda")
        plan.forward_few(weights_of(d), d["x"], None, w.k, out, dbg=moe.make_debug(topk_ids=ids))
        assert plan.device_status() == 0
        return out.double().cpu(), ids.cpu()

    clean, ids = run()
    hit = int(ids[0, 0])
    d["w_gate_up"][hit].view(torch.uint8)[3] = 0x7F
    d["x"][10, 5], d["x"][11, 200] = INF, float("nan")
    out, ids2 = run()
    assert torch.equal(ids[:10], ids2[:10])
    free = [t for t in range(10) if hit not in ids[t].tolist()]
    assert 0 not in free and len(free) >= 3
    scale = clean.square().mean().sqrt()
    assert ((out[free] - clean[free]).abs() <= 6e-2 * scale).all()
    for t in [0, 10, 11]:
        assert not torch.isfinite(out[t]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantiser_scale_that_underflows(dtype):
    """1e-44 / 448 is 0 in fp32: the scale is 1 and every code 0; the largest subnormal scale's values
    are divided by it as they are."""
    x = torch.zeros(4, 256)
    x[0] = 1e-44
    x[1, :128], x[1, 128:] = 1e-44, -1e-44
    x[2] = 1e-38                                  # scale subnormal
    x[3, 7] = 1e-44
    x = x.to(dtype).cuda()
    codes = torch.full((4, 256), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((4, 2), -1.0, device="cuda")
    moe.moe_quantize_groups(x, codes, scales)
    codes, scales, x = codes.cpu(), scales.cpu(), x.float().cpu()
    for r in (0, 1, 3):
        assert (scales[r] == 1.0).all() and (codes[r] & 0x7F == 0).all()
    want = x[2, 0] / torch.tensor(448.0)          # a tensor: not the number's reciprocal
    assert 0 < want < torch.finfo(torch.float32).tiny and (scales[2] == want).all()
    code = (x[2, 0] / want).clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert (codes[2] == code).all()
