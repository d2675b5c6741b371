"""One workspace for moe_forward and moe_forward_few: the few-token layer lives where the regions of
the other forwards lie, so that a plan costs what the larger of the two needs, and the entry
points that were there before take a workspace of the size they always took."""
import ctypes

import pytest
import torch

import mixture_experts_fp32_b200 as moe
from mixture_experts_fp32_b200 import build as moe_build

# (max_tokens, hidden, experts, top_k, inter, shared, shared inter, wtype): the bytes that
# moe_forward's own regions take
FORWARD_BYTES = [
    ((256, 7168, 48, 3, 5120, 1, 5120, moe.MOE_W_BF16), 67930368),
    ((16, 7168, 256, 8, 2048, 1, 2048, moe.MOE_W_BF16), 22601728),
    ((128, 7168, 256, 8, 2048, 1, 2048, moe.MOE_W_FP8_E4M3_B128), 42825728),
    ((8192, 7168, 256, 8, 2048, 1, 2048, moe.MOE_W_FP8_E4M3_B128), 1912687616),
    ((64, 256, 8, 2, 128, 1, 128, moe.MOE_W_FP8_E4M3_B128), 336128),
    ((1, 128, 1, 1, 128, 0, 0, moe.MOE_W_BF16), 32512),
]


@pytest.fixture(scope="module", autouse=True)
def lib():
    moe_build.build()
    return moe.load()


def config(c):
    T, H, E, k, I, S, Is, wtype = c
    return moe.moe_config(T, H, E, k, I, S, Is, 1, wtype)


@pytest.mark.parametrize("c,size", FORWARD_BYTES)
def test_forward_takes_a_workspace_of_its_own_regions(lib, c, size):
    plan, ws = moe.moe_plan_create(config(c))
    try:
        # no weights: an invalid argument once the workspace has been accepted, nothing launched
        def call(fn, n, T=1):
            return fn(plan, None, 0x6000, None, T, 1, 0x7000, 0x100000, n, None, None)

        assert call(lib.moe_forward, size) == moe.MOE_ERR_INVALID_ARG
        assert call(lib.moe_forward, size - 1) == moe.MOE_ERR_WORKSPACE
        assert call(lib.moe_forward, ws) == moe.MOE_ERR_INVALID_ARG
        assert call(lib.moe_forward_few, ws) == moe.MOE_ERR_INVALID_ARG
        assert call(lib.moe_forward_few, 256) == moe.MOE_ERR_WORKSPACE
        arr = (ctypes.c_void_p * 1)(0x7000)
        assert lib.moe_forward_scatter(plan, None, 0x6000, None, 1, 1, arr, 1, 1, 0, 0x100000,
                                       size - 1, None, None) == moe.MOE_ERR_WORKSPACE
        assert lib.moe_forward_scatter(plan, None, 0x6000, None, 1, 1, arr, 1, 1, 0, 0x100000,
                                       size, None, None) == moe.MOE_ERR_INVALID_ARG
    finally:
        moe.moe_plan_destroy(plan)


def test_plans_of_large_batches_pay_nothing_for_few_tokens(lib):
    for c, size in FORWARD_BYTES:
        plan, ws = moe.moe_plan_create(config(c))
        moe.moe_plan_destroy(plan)
        if c[0] >= 64 and c[1] >= 1024:
            assert ws == size
        else:                                     # partial tiles and h of at most 16 tokens
            T, H, E, k, I, S, Is, _ = c
            few = min(T, 16)
            most = (few * 160 * 4 * 256 * 4 + 16 * 16 * E * 4 +
                    16 * (min(E, few * k) + S) * max(I, Is) * 4 + 16 * H * 2)
            assert size <= ws <= max(size, most + (1 << 16))


@pytest.mark.gpu
@pytest.mark.parametrize("wtype", ["bf16", "fp8"])
@pytest.mark.parametrize("T", [3, 16])
def test_calls_in_turn_on_one_workspace(wtype, T):
    """Either call after the other on one workspace gives the bits it gives on a workspace of its own,
    whatever lay there, and nothing past the workspace's size is written."""
    import synth
    from moe_harness import plan_for, to_device, weights_of
    from synth.workloads import Workload
    w = Workload("sharing", T=T, H=640, E=24, k=4, I=256, S=1, Is=384, router_sigma=0.1, wtype=wtype,
                 w_sigma=0.05)
    d = to_device(synth.make_inputs(w))
    wts = weights_of(d)

    def call(fn, ws, n, plan):
        out = torch.full((T, w.H), float("nan"), dtype=torch.bfloat16, device="cuda")
        fn(plan.handle, wts, d["x"], None, T, w.k, out, ws, n)
        torch.cuda.synchronize()
        assert moe.moe_check_device_status(plan.handle, ws) == 0
        return out.view(torch.int16)

    plan = plan_for(w)
    pad = 1 << 16
    own = {fn: call(fn, torch.zeros(plan.ws_bytes, dtype=torch.uint8, device="cuda"), plan.ws_bytes,
                    plan) for fn in (moe.moe_forward, moe.moe_forward_few)}
    ws = torch.full((plan.ws_bytes + pad,), 0xA5, dtype=torch.uint8, device="cuda")
    for fn in (moe.moe_forward_few, moe.moe_forward, moe.moe_forward_few, moe.moe_forward_few,
               moe.moe_forward, moe.moe_forward):
        assert torch.equal(call(fn, ws, plan.ws_bytes, plan), own[fn])
    assert (ws[plan.ws_bytes:] == 0xA5).all()
