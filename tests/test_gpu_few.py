"""The few-token layer (moe_forward_few) against the CPU oracle, over head counts of one to
sixteen tokens, both weight types, shared experts of another width, padding rows, and the
ways a caller may use it: streams, captured graphs, shared workspaces.

Tolerances.  bf16 weights: the output's rounding is at most half a step, 2^-8 of the value;
h enters the down product as two bf16 parts, off by at most 2^-16 of each of the n = kI + Is
terms, so by at most 2^-16 sqrt(n) of the row's norm in a sum (Cauchy-Schwarz), and fp32 sums
of n terms by at most n 2^-24 sqrt(n); with n <= 4096 the two stay under 2^-9 of the root mean
square.  FP8: a code of h at the border of two values may fall to the other side (fp32 sums
against 64 bits), which moves single terms; the layer's tolerance of 6e-2 x RMS holds per value,
and 2^-8 + 2^-10 x RMS for the root mean square of the error, since such terms are rare (a sum
off by 2^-20 meets a border, 2^-4 apart at least, once in 2^15 values)."""
import numpy as np
import pytest
import torch

import mixture_experts_fp32_b200 as moe
import oracle
import synth
from synth.workloads import Workload

from moe_harness import LOGIT_TOL, WEIGHT_TOL, plan_for, rms, to_device, weights_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from mixture_experts_fp32_b200 import build
    build.build()
    moe.load()


def W(name, **kw):
    base = dict(T=16, H=256, E=8, k=2, I=128, router_sigma=0.1)
    base.update(kw)
    if base.get("wtype") == "fp8":
        base.setdefault("w_sigma", 0.05)
    return Workload(name, **base)


SHAPES = [
    dict(T=1), dict(T=16), dict(T=8, S=1, Is=128), dict(T=9, k=1, E=1, H=128),
    dict(T=3, H=640, E=40, k=8, I=384, S=1, Is=896, bias="zipf"),
    dict(T=16, H=384, E=256, k=8, I=256, bias="normal"),
    dict(T=13, H=1920, E=12, k=5, I=640, S=1, Is=128),
    dict(T=1, H=7168, E=48, k=3, I=256, S=1, Is=512, router_sigma=0.01),
    dict(T=12, H=512, E=8, k=3, I=256, S=1, Is=256, mask="dp_padded", dp_rows=(2, 0, 4, 1)),
    dict(T=16, H=256, E=16, k=4, I=128, mask="dp_padded", dp_rows=(0, 0, 0, 1)),
    dict(T=6, H=256, E=4, k=4, I=128, S=1, Is=384, mask="dp_padded", dp_rows=(0, 0)),
]
CASES = [W(f"{wtype}_{i}", wtype=wtype, **s) for wtype in ("bf16", "fp8")
         for i, s in enumerate(SHAPES)]


def run(plan, d, k, weights=None, valid=True):
    T, H = d["x"].shape
    E = d["workload"].E
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    dbg = {"logits": torch.full((T, E), float("nan"), device="cuda"),
           "topk_ids": torch.full((T, k), -7, dtype=torch.int32, device="cuda"),
           "topk_w": torch.full((T, k), float("nan"), device="cuda")}
    plan.forward_few(weights or weights_of(d), d["x"], d["valid"] if valid else None, k, out,
                     dbg=moe.make_debug(**dbg))
    torch.cuda.synchronize()
    assert plan.device_status() == 0
    return {"out": out.cpu(), **{n: t.cpu() for n, t in dbg.items()}}


def check(inp, res, k, renorm=True):
    w = inp["workload"]
    valid = inp["valid"].numpy().astype(bool)
    gl = res["logits"].numpy()
    ol = oracle.router_logits(inp["x"], inp["valid"], inp["router_w"], inp["router_b"])
    if valid.any():
        assert np.all(np.abs(gl - ol)[valid] <= LOGIT_TOL * (np.abs(ol[valid]) + rms(ol[valid])))
    assert np.all(gl[~valid] == 0)
    ids, wts = oracle.topk(gl, inp["valid"], k, renorm)
    assert np.array_equal(res["topk_ids"].numpy(), ids)
    assert np.all(np.abs(res["topk_w"].numpy() - wts) <= WEIGHT_TOL)
    out = res["out"]
    assert torch.equal(out[~valid].view(torch.int16), torch.zeros_like(out[~valid].view(torch.int16)))
    if not valid.any():
        return
    # routing weights as the kernel has them: their tolerance is checked above
    acc = oracle.moe_tokens(inp, ids, res["topk_w"].double().numpy())[valid]
    err = np.abs(out[valid].double().numpy() - acc)
    scale = rms(acc)
    if w.wtype == "bf16":
        assert np.all(err <= 2.0 ** -8 * np.abs(acc) + 2.0 ** -9 * scale), (err / scale).max()
    else:
        assert np.all(err <= 6e-2 * scale), (err / scale).max()
        assert rms(err) <= (2.0 ** -8 + 2.0 ** -10) * scale, rms(err) / scale


@pytest.mark.parametrize("w", CASES, ids=[c.name for c in CASES])
def test_matches_oracle(w):
    inp = synth.make_inputs(w, masked_fill="nan")
    plan = plan_for(w)
    d = to_device(inp)
    a = run(plan, d, w.k)
    check(inp, a, w.k)
    b = run(plan, d, w.k)                               # the same bits every time
    assert torch.equal(a["out"].view(torch.int16), b["out"].view(torch.int16))
    # routes as the plain forward does where its logits leave no near-tie to rounding
    full = torch.empty_like(d["x"])
    plan.forward(weights_of(d), d["x"], d["valid"], w.k, full)
    valid = inp["valid"].bool()
    diff = (full.cpu().double() - a["out"].double())[valid]
    if diff.numel():
        scale = a["out"][valid].double().square().mean().sqrt()
        assert diff.abs().max() <= (4e-2 if w.wtype == "bf16" else 12e-2) * scale


@pytest.mark.parametrize("wtype", ["bf16", "fp8"])
def test_every_token_count_and_fewer_experts_than_planned(wtype):
    w = W("counts", T=16, H=384, E=24, k=6, I=128, S=1, Is=256, wtype=wtype)
    inp = synth.make_inputs(w)
    plan = plan_for(w, max_tokens=40)                    # a plan for larger batches serves few too
    d = to_device(inp)
    for T in (1, 2, 7, 8, 9, 15, 16):
        for k in (1, 6):
            part = {**inp, "x": inp["x"][:T].contiguous(), "valid": inp["valid"][:T].contiguous()}
            pd = {**d, "x": d["x"][:T].contiguous(), "valid": d["valid"][:T].contiguous()}
            check(part, run(plan, pd, k, valid=T % 2 == 0), k)


def test_full_softmax_weights():
    w = W("full", T=5, H=256, E=32, k=4, I=128)
    inp = synth.make_inputs(w)
    plan = moe.Plan(max_tokens=5, hidden=256, num_experts=32, top_k_max=4, inter=128, renormalize=0)
    check(inp, run(plan, to_device(inp), 4), 4, renorm=False)


def test_ties_go_to_the_lower_expert():
    w = W("ties", T=4, H=256, E=40, k=3, I=128)
    inp = synth.make_inputs(w)
    inp["router_w"] = torch.zeros_like(inp["router_w"])
    inp["router_w"][17:19] = 0.0
    res = run(plan_for(w), to_device(inp), 3)
    assert res["topk_ids"].tolist() == [[0, 1, 2]] * 4


def test_tokens_do_not_leak_into_one_another():
    """An infinite hidden state and an expert with NaN weights touch only the rows that
    read them."""
    w = W("leak", T=10, H=256, E=16, k=2, I=128)
    inp = synth.make_inputs(w)
    plan = plan_for(w)
    d = to_device(inp)
    clean = run(plan, d, 2)
    hit = int(clean["topk_ids"][0, 0])
    d["w_gate_up"][hit] = float("nan")
    d["w_down"][hit] = float("inf")
    d["x"][9, 3] = float("inf")
    res = run(plan, d, 2)
    assert torch.equal(res["topk_ids"][:9], clean["topk_ids"][:9])
    free = [t for t in range(9) if hit not in clean["topk_ids"][t].tolist()]
    assert 0 not in free and len(free) >= 3
    a, b = res["out"][free].double(), clean["out"][free].double()
    # the same terms in sums cut at other places: fp32 rounding, then bf16
    assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -12).all()
    assert not torch.isfinite(res["out"][0].double()).all()


def test_shared_expert_alone_and_empty_batch():
    w = W("empty", T=4, S=1, Is=256, mask="dp_padded", dp_rows=(0, 0))
    inp = synth.make_inputs(w, masked_fill="nan")
    plan = plan_for(w)
    check(inp, run(plan, to_device(inp), w.k), w.k)
    none = torch.empty(0, w.H, dtype=torch.bfloat16, device="cuda")
    plan.forward_few(weights_of(to_device(inp)), none, None, w.k, none)      # no rows: nothing to do


@pytest.mark.parametrize("wtype", ["bf16", "fp8"])
def test_graph_replay_follows_its_inputs(wtype):
    w = W("graph", T=7, H=512, E=16, k=3, I=256, S=1, Is=128, wtype=wtype)
    inp = synth.make_inputs(w)
    d = to_device(inp)
    plan, wts = plan_for(w), weights_of(d)
    x = d["x"].clone()
    out, eager = torch.empty_like(x), torch.empty_like(x)
    plan.forward_few(wts, x, None, w.k, eager)           # first call outside capture
    graphs = []
    for _ in range(2):                                   # two graphs share the plan's workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            plan.forward_few(wts, x, None, w.k, out)
        graphs.append(g)
    for i, g in enumerate(graphs * 2):
        x.copy_(synth.normal_bf16(5 + i, synth.STREAM_X, (w.T, w.H), 1.0))
        out.zero_()
        g.replay()
        plan.forward_few(wts, x, None, w.k, eager)
        torch.cuda.synchronize()
        assert plan.device_status() == 0
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16))
    del graphs, g


def test_streams_and_neighbouring_calls():
    """Two plans on two streams, and forward and forward_few in turn on one workspace."""
    ws = [W("s0", T=9, H=512, E=16, k=3, I=256), W("s1", T=3, H=384, E=8, k=2, I=128, wtype="fp8")]
    jobs = []
    for w in ws:
        d = to_device(synth.make_inputs(w))
        plan, wts = plan_for(w), weights_of(d)
        ref = torch.empty_like(d["x"])
        plan.forward_few(wts, d["x"], None, w.k, ref)
        full = torch.empty_like(ref)
        plan.forward(wts, d["x"], None, w.k, full)
        jobs.append((w, d, plan, wts, ref, full, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for i in range(20):
        for w, d, plan, wts, ref, full, st in jobs:
            a, b = torch.empty_like(ref), torch.empty_like(ref)
            a.record_stream(st)
            b.record_stream(st)
            st.wait_stream(torch.cuda.current_stream())
            plan.forward_few(wts, d["x"], None, w.k, a, stream=st)
            plan.forward(wts, d["x"], None, w.k, b, stream=st)
            outs.append((a, b, ref, full))
    torch.cuda.synchronize()
    for a, b, ref, full in outs:
        assert torch.equal(a.view(torch.int16), ref.view(torch.int16))
        assert torch.equal(b.view(torch.int16), full.view(torch.int16))
    assert all(j[2].device_status() == 0 for j in jobs)


@pytest.mark.parametrize("wtype", ["bf16", "fp8"])
def test_expired_waits_report_and_leave_the_device_usable(wtype):
    w = W("limit", T=8, H=2048, E=16, k=4, I=512, S=1, Is=512, wtype=wtype)
    inp = synth.make_inputs(w)
    d = to_device(inp)
    plan = plan_for(w)
    plan.set_wait_limit(0)
    out = torch.empty_like(d["x"])
    plan.forward_few(weights_of(d), d["x"], None, w.k, out)
    assert plan.device_status() & moe.MOE_DEV_WAIT_TIMEOUT_FEW
    assert plan.device_status() == 0
    plan.set_wait_limit(2_000_000_000)
    check(inp, run(plan, d, w.k), w.k)
