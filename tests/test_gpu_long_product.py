"""A product that takes much longer than any of its waits: the limits are on single waits, so a correct
product reports nothing however long it runs.

K terms in fp32, each partial result off by at most a step, 2^-23, and half a step of bf16."""
import pytest
import torch

import mixture_experts_fp32_b200 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from mixture_experts_fp32_b200 import build
    build.build()
    moe.load()


def codes(rows, cols, seed):
    """e4m3 codes of every finite value, NaN's replaced by zeros."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(0, 256, (rows, cols), dtype=torch.uint8, device="cuda", generator=g)
    for part in c.split(4096):
        part[(part & 0x7F) == 0x7F] = 0
    return c


def test_no_limit_bounds_the_whole_product():
    n = 65536                                     # 5.6e14 operations, 17 GB
    a, w = codes(n, n, 1), codes(n, n, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    sa = torch.rand(n, n // 128, device="cuda", generator=g) + 0.5
    sw = torch.rand(n // 128, n // 128, device="cuda", generator=g) + 0.5
    out = torch.full((n, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    prod = moe.Product(max_rows=n, n=n, k=n)
    prod.set_wait_limit(50_000_000)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    prod.forward(a, sa, w, sw, out)
    end.record()
    assert prod.device_status() == 0
    assert begin.elapsed_time(end) > 120          # ms: past the limit set and those of 100 ms
    rows, cols = (torch.randperm(n, device="cuda", generator=g)[:96] for _ in range(2))
    A = a[rows].view(torch.float8_e4m3fn).double() * sa[rows].double().repeat_interleave(128, 1)
    B = w[cols].view(torch.float8_e4m3fn).double() * sw[cols // 128].double().repeat_interleave(128, 1)
    ref, mag = A @ B.t(), A.abs() @ B.abs().t()
    got = out[rows][:, cols].double()
    assert ((got - ref).abs() <= n * 2.0 ** -23 * mag + 2.0 ** -8 * ref.abs()).all()
    for part in out.split(8192):                  # every row was written
        assert torch.isfinite(part).all()
