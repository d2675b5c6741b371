"""Refusals of the few-token layer, the quantiser and the block-scaled product: on the host,
before anything is launched, without a GPU."""
import ctypes

import pytest
import torch

import mixture_experts_fp32_b200 as moe
from mixture_experts_fp32_b200 import build as moe_build

from test_binding_checks import FakeCuda

BAD, UNS, WSP, OK = (moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE,
                     moe.MOE_OK)
F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load()


class Fake(FakeCuda):
    """A CUDA tensor's attributes with a row stride."""

    def __init__(self, shape, dtype=BF16, ld=None, **kw):
        super().__init__(shape, dtype, **kw)
        self.ld = ld if ld is not None else (shape[1] if len(shape) > 1 else 1)

    def stride(self, d):
        return (self.ld, 1)[d]

    def get_device(self):
        return 0


@pytest.mark.parametrize("wtype", [moe.MOE_W_BF16, moe.MOE_W_FP8_E4M3_B128])
def test_few_rejects_before_launch(lib, wtype):
    plan, ws = moe.moe_plan_create(moe.moe_config(64, 256, 8, 2, 128, 1, 128, 1, wtype))
    try:
        s = [0x8000] * 4 if wtype else [None] * 4
        w = moe.moe_weights(0x1000, None, 0x2000, 0x3000, s[0], s[1], 0x4000, 0x5000, s[2], s[3])
        good = dict(w=w, x=0x6000, valid=None, T=4, k=2, out=0x7000, ws=0x100000, n=ws, dbg=None)

        def call(**kw):
            a = {**good, **kw}
            return lib.moe_forward_few(plan, ctypes.byref(a["w"]) if a["w"] else None, a["x"],
                                       a["valid"], a["T"], a["k"], a["out"], a["ws"], a["n"], None,
                                       None if a["dbg"] is None else ctypes.byref(a["dbg"]))

        assert lib.moe_forward_few(None, ctypes.byref(w), 0x6000, None, 4, 2, 0x7000, 0x100000, ws,
                                   None, None) == BAD
        assert call(T=0) == OK
        assert call(T=17) == UNS and call(T=64) == UNS          # the plan has room, the call not
        assert call(T=65) == BAD and call(T=-1) == BAD
        assert call(k=0) == BAD and call(k=3) == BAD
        assert call(w=None) == BAD and call(x=None) == BAD and call(out=None) == BAD
        assert call(x=0x6008) == BAD and call(out=0x7004) == BAD
        assert call(ws=None) == BAD and call(ws=0x100010) == BAD and call(n=ws - 1) == WSP
        no_shared = moe.moe_weights(0x1000, None, 0x2000, 0x3000, s[0], s[1])
        assert call(w=no_shared) == BAD
        if wtype:
            assert call(w=moe.moe_weights(0x1000, None, 0x2000, 0x3000, None, None, 0x4000,
                                          0x5000)) == BAD
        assert call(dbg=moe.moe_debug(perm=0x9000)) == UNS
        assert call(dbg=moe.moe_debug(offsets=0x9000)) == UNS
    finally:
        moe.moe_plan_destroy(plan)


def test_quantize_rejects_before_launch(lib):
    good = dict(x=0x1000, t=moe.MOE_T_BF16, rows=4, cols=256, ldx=256, gated=0, codes=0x8000,
                scales=0x9000)

    def call(**kw):
        a = {**good, **kw}
        return lib.moe_quantize_groups(a["x"], a["t"], a["rows"], a["cols"], a["ldx"], a["gated"],
                                       None, a["codes"], a["scales"], None)

    assert call(rows=0) == OK and call(rows=0, x=None, codes=None, scales=None) == OK
    assert call(rows=-1) == BAD and call(cols=0) == BAD
    assert call(cols=250) == UNS
    assert call(t=2) == BAD and call(gated=2) == BAD
    assert call(x=None) == BAD and call(codes=None) == BAD and call(scales=None) == BAD
    assert call(ldx=248) == BAD                                 # rows would overlap
    assert call(gated=1) == BAD                                 # a gated row is twice as wide
    assert call(ldx=260) == BAD                                 # rows not 16-byte aligned
    assert call(t=moe.MOE_T_FP32, ldx=258) == BAD
    assert call(x=0x1008) == BAD and call(codes=0x8008) == BAD and call(scales=0x9002) == BAD


def test_product_rejects_before_launch(lib):
    def create(**kw):
        c = {**dict(max_rows=64, n=100, k=256, t=0), **kw}
        h, n = ctypes.c_void_p(0x77), ctypes.c_size_t()
        st = lib.moe_product_create(
            ctypes.byref(moe.moe_product_config(c["max_rows"], c["n"], c["k"], c["t"])),
            ctypes.byref(h), ctypes.byref(n))
        if st != OK:
            assert h.value is None
        return st, h, n.value

    for kw, want in ((dict(max_rows=0), BAD), (dict(n=0), BAD), (dict(k=0), BAD), (dict(t=2), BAD),
                     (dict(t=-1), BAD), (dict(k=250), UNS), (dict(k=8), UNS),
                     (dict(k=(1 << 20) + 16), UNS), (dict(n=(1 << 24) + 1), UNS),
                     (dict(max_rows=(1 << 24) + 1), UNS)):
        assert create(**kw)[0] == want, kw
    assert lib.moe_product_create(None, None, None) == BAD
    assert lib.moe_product_set_wait_limit(None, 1) == BAD
    assert lib.moe_product_device_status(None, None, None, None) == BAD
    lib.moe_product_destroy(None)
    for t, width in ((moe.MOE_T_BF16, 2), (moe.MOE_T_FP32, 4)):
        st, h, ws = create(t=t)
        assert st == OK and ws > 0
        good = dict(a=0x1000, sa=0x2004, w=0x3000, sw=0x4000, rows=64, out=0x5000 + width, ldo=100,
                    wsp=0x100000, n=ws)

        def call(**kw):
            g = {**good, **kw}
            return lib.moe_block_scaled_product(h, g["a"], g["sa"], g["w"], g["sw"], g["rows"],
                                                g["out"], g["ldo"], g["wsp"], g["n"], None)

        assert call(rows=0) == OK
        assert call(rows=65) == BAD and call(rows=-1) == BAD
        for name in ("a", "sa", "w", "sw", "out", "wsp"):
            assert call(**{name: None}) == BAD, name
        assert call(a=0x1008) == BAD and call(w=0x3004) == BAD and call(sa=0x2002) == BAD
        assert call(out=0x5001) == BAD and call(ldo=99) == BAD
        assert call(wsp=0x100080) == BAD and call(n=ws - 1) == WSP
        assert lib.moe_block_scaled_product(None, 0x1000, 0x2000, 0x3000, 0x4000, 1, 0x5000, 100,
                                            0x100000, ws, None) == BAD
        lib.moe_product_destroy(h)


def test_binding_refuses_bad_tensors():
    x, codes, scales = Fake((4, 256)), Fake((4, 256), F8), Fake((4, 2), F32)
    q = moe.moe_quantize_groups
    with pytest.raises(ValueError, match="CUDA tensor"):
        q(torch.zeros(4, 256, dtype=BF16), codes, scales)
    with pytest.raises(ValueError, match="codes"):
        q(x, Fake((4, 256), BF16), scales)
    with pytest.raises(ValueError, match="contiguous"):
        q(x, Fake((4, 256), F8, contiguous=False), scales)
    with pytest.raises(ValueError, match="x: shape"):
        q(Fake((4, 256)), Fake((5, 256), F8), scales)
    with pytest.raises(ValueError, match="x: shape"):
        q(x, codes, scales, gated=True)
    with pytest.raises(ValueError, match="scales"):
        q(x, codes, Fake((4, 1), F32))
    with pytest.raises(ValueError, match="valid"):
        q(x, codes, scales, valid=Fake((3,), torch.uint8))
    with pytest.raises(ValueError, match="element type"):
        q(Fake((4, 256), torch.float16), codes, scales)
    with pytest.raises(ValueError, match="overlap"):
        q(Fake((4, 256), ld=0), codes, scales)                  # an expanded tensor
    with pytest.raises(ValueError, match="out_dtype"):
        moe.Product(max_rows=4, n=8, k=16, out_dtype=torch.float16)


def test_product_binding_shapes():
    class HostOnly(moe.Product):
        """The checks of ``forward`` without a workspace."""

        def __init__(self):
            self.handle = None
            self._set_shape(moe.moe_product_config(8, 300, 144, moe.MOE_T_BF16), BF16)

    p = HostOnly()
    good = dict(a=Fake((5, 144), F8), a_scales=Fake((5, 2), F32), w=Fake((300, 144), F8),
                w_scales=Fake((3, 2), F32), out=Fake((5, 300)))
    for name, bad in (("a", Fake((5, 128), F8)), ("a_scales", Fake((5, 1), F32)),
                      ("w", Fake((144, 300), F8)), ("w_scales", Fake((2, 2), F32)),
                      ("out", Fake((4, 300))), ("out", Fake((5, 300), F32)),
                      ("out", Fake((5, 300), ld=150))):
        with pytest.raises(ValueError, match=name):
            p.forward(**{**good, name: bad})
