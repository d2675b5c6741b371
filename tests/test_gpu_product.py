"""The dense FP8 operators on the GPU: moe_quantize_groups and moe_block_scaled_product.

Quantiser: codes and scales equal, bit for bit, those of fp32 division and round-to-nearest-even
on the CPU; with silu(g) * u the fp32 expression is off by at most 2^-20 of its value (exp 2 ulp,
sum, quotient and product half an ulp each, and a scale's rounding), so a code's value is within
half a step (2^-4 of the value, 2^-10 of the scale below the normal range) of the 64-bit one.

Product: the products of codes are exact, and a sum of K terms in fp32, in any order, each
partial result off by at most a step (2^-23, which covers truncation as well as rounding), is off
by at most K 2^-23 sum |terms|; its errors are of random sign, so the 2-norm over all outputs is
held to sqrt(K) 2^-23 of the result's where no cancellation is built in (a random walk), plus half
a step of the output type."""
import math

import numpy as np
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


def quantize_cpu(v):
    """fp32 [R, C] on the CPU: codes (e4m3) and scales."""
    R, C = v.shape
    p = torch.nn.functional.pad(v, (0, groups(C) * 128 - C)).view(R, groups(C), 128)
    amax = p.abs().amax(2)
    s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    return (p / s[..., None]).view(R, -1)[:, :C].to(E4M3), s


def run_quantize(x, cols, valid=None, gated=False):
    rows = x.shape[0]
    codes = torch.full((rows, cols), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, groups(cols)), -1.0, device="cuda")
    moe.moe_quantize_groups(x, codes, scales, valid=valid, gated=gated)
    torch.cuda.synchronize()
    return codes.cpu(), scales.cpu()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 144), (17, 1200), (256, 7168),
                                       (1000, 272), (5000, 128)])
def test_quantize_codes_bit_exact(rows, cols, dtype):
    g = torch.Generator().manual_seed(rows * 7 + cols)
    x = torch.randn(rows, cols, generator=g)
    x *= torch.exp2(torch.randint(-30, 30, (rows, 1), generator=g).float())
    x[0, : min(cols, 128)] = 0.0                                   # an all-zero group: scale 1
    x = x.to(dtype)
    valid = (torch.rand(rows, generator=g) < 0.8).to(torch.uint8)
    for v in (None, valid):
        codes, scales = run_quantize(x.cuda(), cols, None if v is None else v.cuda())
        ref = x.float() if v is None else torch.where(v[:, None] != 0, x.float(), torch.zeros(()))
        q, s = quantize_cpu(ref)
        assert torch.equal(scales, s)
        assert torch.equal(codes, q.view(torch.uint8))


def test_quantize_special_values():
    x = torch.randn(6, 256)
    x[0, 5] = float("nan")                       # NaN stays where it is, the group's scale without it
    x[1, 7] = float("inf")                       # the group's finite values vanish beside it
    x[2, 130] = -float("inf")
    x[3, :] = float("nan")
    x[4, :128] = 1e-44                           # subnormal values: the scale is subnormal or zero
    x[5, :] = 3.4e38
    codes, scales = run_quantize(x.cuda(), 256)
    nan = (codes & 0x7F) == 0x7F
    assert nan[0].nonzero().flatten().tolist() == [5]
    q, s = quantize_cpu(torch.nan_to_num(x[:1], nan=0.0))
    keep = torch.arange(256) != 5
    assert torch.equal(scales[:1], s) and torch.equal(codes[0, keep], q.view(torch.uint8)[0, keep])
    assert nan[1].nonzero().flatten().tolist() == [7] and scales[1, 0] == float("inf")
    assert (codes[1, :128][torch.arange(128) != 7] & 0x7F == 0).all()
    assert nan[2].nonzero().flatten().tolist() == [130]
    assert nan[3].all() and (scales[3] == 1).all()
    assert (codes[5] & 0x7F == 0x7E).all()        # 448, the largest code


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 16), (5, 2064), (300, 640), (2, 5120)])
def test_quantize_gated(rows, cols, dtype):
    g = torch.Generator().manual_seed(cols)
    x = (torch.randn(rows, 2 * cols, generator=g) * 3).to(dtype)
    x[0, 0] = -100.0                              # silu(-100) = -4e-42 * ...: next to nothing
    valid = torch.ones(rows, dtype=torch.bool)
    valid[rows // 2] = rows == 1
    codes, scales = run_quantize(x.cuda(), cols, valid.cuda(), gated=True)
    xd = x.double()
    h = torch.where(valid[:, None], xd[:, :cols] / (1 + torch.exp(-xd[:, :cols])) * xd[:, cols:],
                    torch.zeros((), dtype=torch.float64))
    p = torch.nn.functional.pad(h, (0, groups(cols) * 128 - cols)).view(rows, -1, 128)
    amax = p.abs().amax(2)
    want = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    assert ((scales.double() - want).abs() <= 2.0 ** -20 * want).all()
    sc = spread(scales.double(), cols)
    got = codes.view(E4M3).double() * sc
    assert ((got - h).abs() <= (2.0 ** -4 + 2.0 ** -19) * h.abs() + 2.0 ** -10 * sc).all()
    assert (codes[~valid] == 0).all() and (scales[~valid] == 1).all()


def test_quantize_strided_rows_and_untouched_neighbours():
    big = torch.randn(9, 1000, dtype=torch.bfloat16, device="cuda")
    x = big[:, 40:40 + 304]                       # 80 bytes in: rows 16-byte aligned
    codes, scales = run_quantize(x, 304)
    q, s = quantize_cpu(x.float().cpu())
    assert torch.equal(codes, q.view(torch.uint8)) and torch.equal(scales, s)


# ------------------------------------------------------------------------ product

def operands(M, N, K, seed=0):
    g = torch.Generator().manual_seed(seed)
    a, sa = quantize_cpu(torch.randn(M, K, generator=g))
    w = torch.randn(N, K, generator=g).to(E4M3)
    sw = torch.exp2(torch.rand(groups(N), groups(K), generator=g) * 6 - 9)
    sa = sa * torch.exp2(torch.randint(-3, 4, sa.shape, generator=g).float())
    return a, sa, w, sw


def reference(a, sa, w, sw):
    """(result, sum of the terms' absolute values) in 64 bits, on the GPU's fp64 units."""
    N, K = w.shape
    A = a.cuda().double() * spread(sa.cuda().double(), K)
    B = w.cuda().double() * spread(sw.cuda().double(), K).repeat_interleave(128, 0)[:N]
    return (A @ B.t()).cpu(), (A.abs() @ B.abs().t()).cpu()


def check(got, ref, mag, K):
    half = torch.finfo(got.dtype).eps / 2
    err = (got.double() - ref).abs()
    assert torch.isfinite(got.float()).all()
    assert (err <= K * 2.0 ** -23 * mag + half * ref.abs()).all(), (err / mag).max()
    assert err.norm() <= (math.sqrt(K) * 2.0 ** -23 + half) * ref.norm(), err.norm() / ref.norm()


SHAPES = [(1, 1, 16), (1, 64, 128), (1, 4096, 512), (7, 100, 48), (8, 1111, 1200), (9, 129, 2048),
          (16, 7168, 256), (17, 65, 640), (33, 300, 144), (64, 512, 1024), (77, 1111, 1200),
          (128, 256, 128), (129, 257, 400), (200, 384, 7168), (256, 2000, 512), (300, 96, 2048),
          (513, 768, 272), (1000, 1040, 1152), (2048, 512, 384)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_matches_64_bits(M, N, K, dtype):
    a, sa, w, sw = operands(M, N, K, seed=M + N + K)
    ref, mag = reference(a, sa, w, sw)
    prod = moe.Product(max_rows=M, n=N, k=K, out_dtype=dtype)
    out = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
    args = a.cuda(), sa.cuda(), w.cuda(), sw.cuda()
    prod.forward(*args, out)
    assert prod.device_status() == 0
    check(out.cpu(), ref, mag, K)
    again = torch.empty_like(out)
    prod.forward(*args, again)
    assert torch.equal(out, again)                # the same bits every time


@pytest.mark.parametrize("M", [3, 40, 300])
def test_product_fewer_rows_than_planned_strided_output(M):
    N, K = 200, 256
    a, sa, w, sw = operands(M, N, K, seed=M)
    ref, mag = reference(a, sa, w, sw)
    for dtype in (torch.bfloat16, torch.float32):
        for off, width in ((0, N), (8, N + 16), (5, N + 7)):       # aligned and odd rows
            prod = moe.Product(max_rows=1000, n=N, k=K, out_dtype=dtype)
            big = torch.full((M + 2, width), 7.0, dtype=dtype, device="cuda")
            prod.forward(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), big[1:M + 1, off:off + N])
            assert prod.device_status() == 0
            big = big.cpu()
            check(big[1:M + 1, off:off + N].clone(), ref, mag, K)
            big[1:M + 1, off:off + N] = 7.0
            assert (big == 7.0).all()             # nothing beside the output was written


def test_product_padding_rows_and_special_codes():
    M, N, K = 150, 300, 384
    a, sa, w, sw = operands(M, N, K, seed=3)
    prod = moe.Product(max_rows=M, n=N, k=K, out_dtype=torch.float32)
    for rows in (M, 5):
        x = torch.randn(rows, K, device="cuda")
        valid = torch.ones(rows, dtype=torch.uint8, device="cuda")
        valid[2], valid[4] = 0, 0
        x[2] = float("nan")
        codes = torch.empty(rows, K, dtype=E4M3, device="cuda")
        scales = torch.empty(rows, groups(K), device="cuda")
        moe.moe_quantize_groups(x, codes, scales, valid=valid)
        codes.view(torch.uint8)[0, 7] = 0x7F                       # NaN in row 0 alone
        out = torch.empty(rows, N, device="cuda")
        prod.forward(codes, scales, w.cuda(), sw.cuda(), out)
        assert prod.device_status() == 0
        assert torch.isnan(out[0]).all() and torch.isfinite(out[1:]).all()
        assert (out[2] == 0).all() and (out[4] == 0).all()
        w2 = w.clone()
        w2.view(torch.uint8)[11, 380] = 0xFF                       # and in weight row 11 alone
        codes.view(torch.uint8)[0, 7] = 0
        prod.forward(codes, scales, w2.cuda(), sw.cuda(), out)
        assert torch.isnan(out[:, 11]).all()
        assert torch.isfinite(out[:, torch.arange(N, device="cuda") != 11]).all()


def test_product_graphs_and_streams():
    shapes = [(5, 640, 1024), (70, 500, 512), (400, 384, 640)]
    jobs = []
    for M, N, K in shapes:
        args = [t.cuda() for t in operands(M, N, K, seed=M)]
        prod = moe.Product(max_rows=M, n=N, k=K)
        ref = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        prod.forward(*args, ref)                  # first call outside capture
        out = torch.empty_like(ref)
        gs = []
        for _ in range(2):                        # two graphs share the workspace
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                prod.forward(*args, out)
            gs.append(g)
        jobs.append((prod, args, ref, out, gs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for prod, args, ref, out, gs, st in jobs:
        for g in gs + gs:
            out.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, ref)
        args[0].copy_(torch.zeros_like(args[0]))  # a replay follows its inputs
        gs[0].replay()
        torch.cuda.synchronize()
        assert (out == 0).all()
    fresh = []
    for i in range(10):
        for j, (prod, args, ref, out, gs, st) in enumerate(jobs):
            o = torch.empty_like(ref)
            o.record_stream(st)
            st.wait_stream(torch.cuda.current_stream())
            prod.forward(*args, o, stream=st)
            fresh.append(o)
    torch.cuda.synchronize()
    assert all((o == 0).all() for o in fresh)
    del jobs, gs, g


@pytest.mark.parametrize("M", [4, 500])
def test_product_expired_waits_report(M):
    N, K = 512, 2048
    a, sa, w, sw = operands(M, N, K, seed=1)
    prod = moe.Product(max_rows=M, n=N, k=K)
    prod.set_wait_limit(0)
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    args = a.cuda(), sa.cuda(), w.cuda(), sw.cuda()
    prod.forward(*args, out)
    assert prod.device_status() == moe.MOE_DEV_WAIT_TIMEOUT_PRODUCT
    prod.set_wait_limit(2_000_000_000)
    prod.forward(*args, out)
    assert prod.device_status() == 0
    ref, mag = reference(a, sa, w, sw)
    check(out.cpu(), ref, mag, K)


# ---------------------------------------------------------------------- together

@pytest.mark.parametrize("T", [1, 16, 200])
def test_dense_mlp_is_the_layer_with_one_expert(T):
    """quantise, product, gated quantise, product: the FP8 layer with one expert that every
    token selects with weight 1, in a captured graph beside the layer itself."""
    H, I = 512, 384
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    valid = torch.ones(T, dtype=torch.uint8, device="cuda")
    valid[T // 2] = T == 1
    gu, sgu = [t.cuda() for t in _weights(2 * I, H, g)]
    dn, sdn = [t.cuda() for t in _weights(H, I, g)]
    up = moe.Product(max_rows=T, n=2 * I, k=H, out_dtype=torch.float32)
    down = moe.Product(max_rows=T, n=H, k=I)
    new = lambda *s, dt: torch.empty(*s, dtype=dt, device="cuda")     # noqa: E731
    xq, xs = new(T, H, dt=E4M3), new(T, groups(H), dt=torch.float32)
    z = new(T, 2 * I, dt=torch.float32)
    hq, hs = new(T, I, dt=E4M3), new(T, groups(I), dt=torch.float32)
    out = new(T, H, dt=torch.bfloat16)

    def mlp():
        moe.moe_quantize_groups(x, xq, xs, valid=valid)
        up.forward(xq, xs, gu, sgu, z)
        moe.moe_quantize_groups(z, hq, hs, valid=valid, gated=True)
        down.forward(hq, hs, dn, sdn, out)

    plan = moe.Plan(max_tokens=T, hidden=H, num_experts=1, top_k_max=1, inter=I,
                    wtype=moe.MOE_W_FP8_E4M3_B128)
    w = plan.weights(torch.zeros(1, H, device="cuda"), None, gu[None], dn[None], sgu[None],
                     sdn[None])
    layer = torch.empty_like(out)
    call = plan.forward_few if T <= moe.MOE_FEW_TOKENS_MAX else plan.forward
    mlp()
    call(w, x, valid, 1, layer)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mlp()
        call(w, x, valid, 1, layer)
    x.copy_(torch.randn(T, H, generator=g).to(torch.bfloat16))
    graph.replay()
    torch.cuda.synchronize()
    assert up.device_status() == down.device_status() == plan.device_status() == 0
    # 64 bits, from the codes the quantiser gave for x (they are exact, tested above)
    zr, _ = reference(xq.cpu(), xs.cpu(), gu.cpu(), sgu.cpu())
    h = zr[:, :I] / (1 + torch.exp(-zr[:, :I])) * zr[:, I:]
    q, s = quantize_cpu(h.float())
    ref, _ = reference(q, s, dn.cpu(), sdn.cpu())
    ref[valid.cpu() == 0] = 0
    scale = ref.square().mean().sqrt()
    for got in (out, layer):
        err = got.cpu().double() - ref
        assert err.abs().max() <= 6e-2 * scale                        # the layer's tolerance
        assert err.square().mean().sqrt() <= (2.0 ** -8 + 2.0 ** -10) * scale
        assert (got[valid == 0] == 0).all()
    del graph


def _weights(rows, cols, g):
    w = torch.randn(rows, cols, generator=g) * 0.05
    p = w.view(rows // 128, 128, cols // 128, 128)
    s = p.abs().amax((1, 3)) / 448
    return (p / s[:, None, :, None]).view(rows, cols).to(E4M3), s
