"""Tiles that several CTAs finish together, and the ends of the ranges: sums of exactly zero, many
sharers, offsets past 32 bits, magnitudes at both ends of fp32.

Sums of zero are exact.  The 64-bit comparison of the product is that of its other tests: K terms
in fp32, each partial result off by at most a step, 2^-23, and half a step of the output type."""
import pytest
import torch

import mixture_experts_fp32_b200 as moe

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    from mixture_experts_fp32_b200 import build
    build.build()
    moe.load()


def groups(n):
    return -(-n // 128)


def spread(s, n):
    return s.repeat_interleave(128, -1)[..., :n]


# one row and 32, whole tiles in few CTAs, tiles of up to twenty CTAs, tiles cut along K
SHARED = [(1, 4096, 7168), (32, 1111, 7168), (16, 300, 16384), (20, 257, 1040), (40, 200, 8192),
          (100, 500, 7168), (256, 768, 6160), (70, 130, 4096)]


def operands(M, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    a = torch.randn(M, K, generator=g).to(E4M3).cuda()
    w = torch.randn(N, K, generator=g).to(E4M3).cuda()
    sa = (torch.rand(M, groups(K), generator=g) + 0.5).cuda()
    sw = (torch.rand(groups(N), groups(K), generator=g) + 0.5).cuda()
    return a, sa, w, sw


@pytest.mark.parametrize("M,N,K", SHARED)
def test_product_of_shared_tiles(M, N, K):
    a, sa, w, sw = operands(M, N, K, M + N + K)
    A = a.double() * spread(sa.double(), K)
    B = w.double() * spread(sw.double(), K).repeat_interleave(128, 0)[:N]
    ref, mag = A @ B.t(), A.abs() @ B.abs().t()
    for dtype in (torch.float32, torch.bfloat16):
        prod = moe.Product(max_rows=M, n=N, k=K, out_dtype=dtype)
        prod.workspace.fill_(0xA5)                # whatever lay there before
        out = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
        for _ in range(3):
            prod.forward(a, sa, w, sw, out)
        assert prod.device_status() == 0
        half = torch.finfo(dtype).eps / 2
        assert ((out.double() - ref).abs() <= K * 2.0 ** -23 * mag + half * ref.abs()).all()


@pytest.mark.parametrize("M,N,K", SHARED)
def test_product_of_zeros(M, N, K):
    a, sa, w, sw = operands(M, N, K, 1)
    prod = moe.Product(max_rows=M, n=N, k=K)
    prod.set_wait_limit(200_000_000)
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    for zero in (torch.zeros_like(a), torch.full_like(a.view(torch.uint8), 0x80).view(E4M3)):
        out.fill_(1.0)
        prod.forward(zero, sa, w, sw, out)
        assert prod.device_status() == 0
        assert (out == 0).all()
    # zeros in a part of K alone: some CTAs' sums vanish, others' do not
    a[:, K // 2:] = 0
    prod.forward(a, sa, w, sw, out)
    assert prod.device_status() == 0
    A = a.double() * spread(sa.double(), K)
    B = w.double() * spread(sw.double(), K).repeat_interleave(128, 0)[:N]
    ref, mag = A @ B.t(), A.abs() @ B.abs().t()
    assert ((out.double() - ref).abs() <= K * 2.0 ** -23 * mag + 2.0 ** -8 * ref.abs()).all()


@pytest.mark.parametrize("wtype", ["bf16", "fp8"])
@pytest.mark.parametrize("T,H,E,k,I,S,Is", [(1, 1024, 8, 2, 512, 1, 896), (16, 640, 12, 4, 256, 1, 640),
                                          (5, 2048, 4, 1, 128, 0, 0)])
def test_few_tokens_of_zeros(wtype, T, H, E, k, I, S, Is):
    g = torch.Generator(device="cuda").manual_seed(T)
    fp8 = wtype == "fp8"

    keep = []                                     # the weights' addresses are all that a plan holds

    def kept(t):
        keep.append(t)
        return t

    def weight(*shape):
        w = torch.randn(*shape, device="cuda", generator=g) * 0.1
        return kept(w.to(E4M3) if fp8 else w.to(torch.bfloat16))

    def scale(e, n, m):
        return kept(torch.ones(*((e,) if e else ()), groups(n), groups(m), device="cuda"))
    kw = dict(s_gate_up=scale(E, 2 * I, H), s_down=scale(E, H, I)) if fp8 else {}
    if S:
        kw.update(ws_gate_up=weight(2 * Is, H), ws_down=weight(H, Is))
        if fp8:
            kw.update(ss_gate_up=scale(0, 2 * Is, H), ss_down=scale(0, H, Is))
    plan = moe.Plan(max_tokens=T, hidden=H, num_experts=E, top_k_max=k, inter=I, num_shared=S,
                    shared_inter=Is, wtype=moe.MOE_W_FP8_E4M3_B128 if fp8 else moe.MOE_W_BF16)
    plan.set_wait_limit(200_000_000)
    w = plan.weights(kept(torch.randn(E, H, device="cuda", generator=g)), None, weight(E, 2 * I, H),
                     weight(E, H, I), **kw)
    valid = torch.ones(T, dtype=torch.uint8, device="cuda")
    out = torch.full((T, H), 1.0, dtype=torch.bfloat16, device="cuda")
    plan.forward_few(w, torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), valid, k, out)
    assert plan.device_status() == 0
    assert (out == 0).all()
    # values in half of the columns alone
    x = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    x[:, H // 2:] = 0
    other = torch.empty_like(out)
    plan.forward_few(w, x, valid, k, out)
    assert plan.device_status() == 0
    plan.forward(w, x, valid, k, other)
    assert plan.device_status() == 0
    # the two take their sums in other orders; FP8 rounds an expert's output to bf16 in one of them
    # (2^-8 of each, weights summing to 1) and may round codes at a border differently
    rms = other.double().norm() / other.numel() ** 0.5
    tol = 6e-2 if fp8 else 2.0 ** -7
    assert ((out.double() - other.double()).abs() <= tol * (rms + other.double().abs())).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_both_ends_of_the_range(dtype):
    g = torch.Generator().manual_seed(3)
    exps = torch.arange(-150, 121, 3, dtype=torch.float64)
    x = (torch.randn(len(exps), 256, generator=g).double() * torch.exp2(exps)[:, None]).to(dtype)
    x[:, 7] = 0.0
    codes = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty(len(exps), 2, device="cuda")
    moe.moe_quantize_groups(x.cuda(), codes, scales)
    v = x.float().view(len(exps), 2, 128)
    s = v.abs().amax(2) / 448.0
    s = torch.where(s == 0, torch.ones_like(s), s)
    want = (v / s[..., None]).clamp(-448, 448).view(x.shape).to(E4M3).view(torch.uint8)
    assert torch.equal(scales.cpu(), s)
    assert torch.equal(codes.cpu(), want)


def test_offsets_past_32_bits():
    rows, cols = 300_001, 7168                    # 2.15e9 codes, 4.3e9 bytes of values
    x = torch.randn(rows, cols, dtype=torch.bfloat16, device="cuda")
    codes = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, groups(cols), device="cuda")
    moe.moe_quantize_groups(x, codes, scales)
    last, last_s = torch.empty_like(codes[-2:]), torch.empty_like(scales[-2:])
    moe.moe_quantize_groups(x[-2:].clone(), last, last_s)
    assert torch.equal(codes[-2:], last) and torch.equal(scales[-2:], last_s)
    del x, codes, scales
    M, N, K, ldo = 40_000, 48, 256, 60_000        # rows of out 2.4e9 elements apart at the end
    a, sa, w, sw = operands(M, N, K, 5)
    out = torch.empty(M, ldo, dtype=torch.bfloat16, device="cuda")
    prod = moe.Product(max_rows=M, n=N, k=K)
    prod.forward(a, sa, w, sw, out[:, 1000:1000 + N])
    tail = torch.empty(300, N, dtype=torch.bfloat16, device="cuda")
    prod.forward(a[-300:].clone(), sa[-300:].clone(), w, sw, tail)
    assert prod.device_status() == 0
    assert torch.equal(out[-300:, 1000:1000 + N], tail)
