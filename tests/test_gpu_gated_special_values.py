"""The gated quantiser where g or u is no ordinary number: infinities, NaN, and values on both
sides of |g| = 69, beyond which silu's quotient is taken by division.

v = silu(g) * u with silu(g) = g / (1 + e^-g) in fp32, then the rule of the values without a gate: a
NaN gives a NaN code and is left out of its group's maximum; an infinite value makes the scale
infinite, its own code NaN and the codes of the group's finite values 0."""
import pytest
import torch

import mixture_experts_fp32_b200 as moe

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
INF, NAN = float("inf"), float("nan")
COLS, AT = 256, 37                                # the special value's column


@pytest.fixture(scope="module", autouse=True)
def built():
    from mixture_experts_fp32_b200 import build
    build.build()
    moe.load()


def gated(g, u, dtype):
    """Codes and scales of silu(g) * u for rows of fp32 values."""
    x = torch.cat([g, u], 1).to(dtype).cuda()
    codes = torch.full(g.shape, 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((g.shape[0], -(-g.shape[1] // 128)), -1.0, device="cuda")
    moe.moe_quantize_groups(x, codes, scales, gated=True)
    return codes.cpu(), scales.cpu()


def ordinary(rows):
    gen = torch.Generator().manual_seed(11)
    g = torch.randn(rows, COLS, generator=gen) * 2
    u = torch.randn(rows, COLS, generator=gen)
    return g, u


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gv,uv", [(INF, 2.0), (INF, -0.25), (INF, INF), (INF, -INF), (3.0, INF),
                                   (-1.5, INF), (-1.5, -INF)])
def test_infinite_values_take_the_scale(gv, uv, dtype):
    g, u = ordinary(3)
    g[1, AT], u[1, AT] = gv, uv
    codes, scales = gated(g, u, dtype)
    assert scales[1, 0] == INF
    assert (codes[1, AT] & 0x7F) == 0x7F
    rest = torch.arange(128) != AT
    assert (codes[1, :128][rest] & 0x7F == 0).all()
    # the neighbouring rows and the row's other group are those of the ordinary values
    g[1, AT], u[1, AT] = 1.0, 1.0
    plain, plain_s = gated(g, u, dtype)
    assert torch.equal(scales[::2], plain_s[::2]) and torch.equal(codes[::2], plain[::2])
    assert scales[1, 1] == plain_s[1, 1] and torch.equal(codes[1, 128:], plain[1, 128:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gv,uv", [(NAN, 1.0), (1.0, NAN), (INF, 0.0), (0.0, INF), (-INF, 1.0),
                                   (INF, NAN)])
def test_nan_values_are_left_out_of_the_scale(gv, uv, dtype):
    g, u = ordinary(1)
    g[0, AT], u[0, AT] = gv, uv
    codes, scales = gated(g, u, dtype)
    g[0, AT], u[0, AT] = 0.0, 0.0                 # the same maximum
    plain, plain_s = gated(g, u, dtype)
    assert (codes[0, AT] & 0x7F) == 0x7F
    rest = torch.arange(COLS) != AT
    assert torch.equal(scales, plain_s) and torch.equal(codes[0, rest], plain[0, rest])


def test_large_gates():
    """|g| from 60 to 80 in every direction, then to the end of the range: v against 64 bits, off by at
    most 2^-20 of it (exp 2 ulp, sum, quotient and product half an ulp each) and half a step of the
    code (2^-4 of the value, 2^-10 of the scale below the normal range)."""
    g = torch.cat([torch.linspace(60, 80, 4096), torch.logspace(2, 38, 4096), torch.tensor([69.0] * 128)])
    g = torch.cat([g, -torch.linspace(60, 80, 4096)]).view(-1, 128)
    u = torch.randn(g.shape, generator=torch.Generator().manual_seed(5))
    u = torch.where(g > 1e30, u * 1e-3, u)
    codes, scales = gated(g, u, torch.float32)
    h = g.double() / (1 + torch.exp(-g.double())) * u.double()
    want = h.abs().amax(1, keepdim=True) / 448
    assert ((scales.double() - want).abs() <= 2.0 ** -20 * want).all()
    got = codes.view(E4M3).double() * scales.double()
    assert ((got - h).abs() <= (2.0 ** -4 + 2.0 ** -19) * h.abs() + 2.0 ** -10 * scales.double()).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_zeros_keep_their_sign(dtype):
    """silu(-0) = -0 and a product's sign is that of its factors: codes 0x80 and 0x00, beside values
    that make the scale ordinary and in a group of zeros."""
    signs = [(-0.0, 1.0), (-0.0, -1.0), (0.0, 1.0), (0.0, -1.0), (2.0, -0.0), (-2.0, -0.0),
             (2.0, 0.0), (-2.0, 0.0)]
    want = torch.tensor([0x80, 0, 0, 0x80, 0x80, 0, 0, 0x80], dtype=torch.uint8)
    g, u = ordinary(1)
    for at in (16, 136):
        g[0, at:at + 8] = torch.tensor([s[0] for s in signs])
        u[0, at:at + 8] = torch.tensor([s[1] for s in signs])
    g[0, 128:136], g[0, 144:] = 0.0, 0.0          # the second group: nothing but zeros
    codes, scales = gated(g, u, dtype)
    assert scales[0, 1] == 1.0 and scales[0, 0] != 1.0
    assert torch.equal(codes[0, 16:24], want) and torch.equal(codes[0, 136:144], want)
