"""Kernels that a device refuses take their own entry points out and no others: a fake device whose
preparation of some kernels fails, without a GPU."""
import ctypes
import os
import subprocess

import pytest

import mixture_experts_fp32_b200 as moe
from mixture_experts_fp32_b200 import build as moe_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FEW, LAYER = 1, 2                                # bits of the kernels that fail


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    moe_build.build()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(moe_build.nvcc())))
    path = tmp_path_factory.mktemp("fake") / "libmoe_fake.so"
    include = [os.path.join(ROOT, "include"), moe_build.CSRC, os.path.join(cuda, "include")]
    subprocess.check_call(
        ["g++", "-std=c++17", "-shared", "-fPIC",
         # its own symbols before those of a CUDA runtime in the process; the others unresolved
         "-Wl,-Bsymbolic,-z,lazy", "-Wl,--unresolved-symbols=ignore-all",
         *[a for d in include for a in ("-I", d)], "-x", "c++",
         os.path.join(moe_build.CSRC, "moe_api.cu"),
         os.path.join(ROOT, "tests", "c", "fake_device.cpp"), "-o", str(path)])
    return path


@pytest.fixture
def lib(library, tmp_path):
    """A fresh copy, which has prepared nothing yet."""
    copy = tmp_path / "libmoe_fake_fresh.so"
    copy.write_bytes(library.read_bytes())
    L = ctypes.CDLL(str(copy), mode=os.RTLD_LAZY | os.RTLD_LOCAL)
    for name in ("moe_forward", "moe_forward_few"):
        real = getattr(moe.load(), name)
        getattr(L, name).argtypes, getattr(L, name).restype = real.argtypes, real.restype
    return L


def calls(L):
    plan, ws = ctypes.c_void_p(), ctypes.c_size_t()
    cfg = moe.moe_config(16, 256, 8, 2, 128, 0, 0, 1, moe.MOE_W_BF16)
    assert L.moe_plan_create(ctypes.byref(cfg), ctypes.byref(plan), ctypes.byref(ws)) == moe.MOE_OK
    w = moe.moe_weights(0x1000, None, 0x2000, 0x3000)

    def call(fn):
        before = L.fake_launched()
        st = fn(plan, ctypes.byref(w), 0x6000, None, 4, 2, 0x7000, 0x100000, ws, None, None)
        return st, L.fake_launched() - before
    return (lambda: call(L.moe_forward)), (lambda: call(L.moe_forward_few))


def test_refused_few_token_kernels_leave_the_layer(lib):
    forward, few = calls(lib)
    lib.fake_fail(FEW)
    st, n = forward()
    assert st == moe.MOE_OK and n > 0
    assert few() == (moe.MOE_ERR_CUDA, 0)         # nothing launched
    assert forward()[0] == moe.MOE_OK
    lib.fake_fail(0)                              # and are asked for again
    assert few() == (moe.MOE_OK, 1)


def test_refused_layer_kernels_leave_few_tokens(lib):
    forward, few = calls(lib)
    lib.fake_fail(LAYER)
    assert forward() == (moe.MOE_ERR_CUDA, 0)
    assert few() == (moe.MOE_OK, 1)
    assert forward() == (moe.MOE_ERR_CUDA, 0)
    lib.fake_fail(0)
    assert forward()[0] == moe.MOE_OK


def test_prepared_once_and_for_what_is_called(lib):
    forward, few = calls(lib)
    for _ in range(3):
        assert forward()[0] == moe.MOE_OK
    assert (lib.fake_prepared(LAYER), lib.fake_prepared(FEW)) == (1, 0)
    for _ in range(3):
        assert few()[0] == moe.MOE_OK
    forward2, _ = calls(lib)                      # another plan of the same device
    assert forward2()[0] == moe.MOE_OK
    assert (lib.fake_prepared(LAYER), lib.fake_prepared(FEW)) == (1, 1)
