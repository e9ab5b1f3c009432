"""The layer norm's and the list step's launches on a runtime of two devices
that run nothing (tests/c_abi/fake_cudart.cpp): what a kernel is allowed and
how many of its blocks an SM keeps belong to a device, and a query that fails
is an error of the call that needed it, not a number for all later ones."""
import ctypes
import glob
import os
import subprocess

import pytest

import optimizer_step_resumable_gb300 as osr
from optimizer_step_resumable_gb300 import build as lib_build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def fake_path(lib, tmp_path_factory):
    """The library's own objects, linked with the fake runtime."""
    out = tmp_path_factory.mktemp("fake")
    objects = sorted(glob.glob(os.path.join(lib_build.BUILD_DIR, "*.o")))
    if len(objects) < len(lib_build.CUDA_SOURCES + lib_build.CXX_SOURCES):
        lib_build.build(force=True)
        objects = sorted(glob.glob(os.path.join(lib_build.BUILD_DIR, "*.o")))
    cuda = os.path.join(os.path.dirname(os.path.dirname(lib_build.nvcc())), "include")
    fake = str(out / "fake.o")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-I", cuda, "-c",
                    os.path.join(HERE, "c_abi", "fake_cudart.cpp"), "-o", fake], check=True)

    def symbols(flag, files):
        text = subprocess.run(["nm", flag, *files], capture_output=True, text=True, check=True).stdout
        return {line.split()[-1] for line in text.splitlines() if "cuda" in line}

    # every other call of the runtime does nothing and succeeds
    missing = symbols("--undefined-only", objects) - symbols("--defined-only", [fake])
    missing = sorted(s for s in missing if s.lstrip("_").startswith("cuda"))
    rest = out / "rest.c"
    rest.write_text("".join(f"long {s}(void) {{ return 0; }}\n" for s in missing))
    subprocess.run(["gcc", "-fno-builtin", "-fPIC", "-c", str(rest), "-o", str(out / "rest.o")],
                   check=True)
    path = str(out / "libfake.so")
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", path, *objects, fake,
                    str(out / "rest.o"), "-ldl", "-lpthread"], check=True)
    return path


@pytest.fixture
def fake(fake_path, tmp_path):
    """A library of its own for each test: what is kept per process starts anew."""
    own = str(tmp_path / "libfake.so")
    with open(fake_path, "rb") as f, open(own, "wb") as g:
        g.write(f.read())
    f = ctypes.CDLL(own)
    for name, (res, args) in osr.SIGNATURES.items():
        getattr(f, name).restype = res
        getattr(f, name).argtypes = args
    return f


# made-up addresses, apart from one another
X, Y, DY, DX, MEAN, RSTD, DW = (k << 40 for k in range(1, 8))


def forward(f, ln, cols, dtype, rows=1 << 20):
    return f.layernorm_forward(ln, X, cols, dtype, None, None, 0, Y, cols, MEAN, RSTD, rows, 1e-5,
                               None)


def backward(f, ln, cols, dtype, rows=1 << 20, dw=None):
    return f.layernorm_backward(ln, DY, cols, X, cols, dtype, None, 0, MEAN, RSTD, DX, cols, dw,
                                None, 0, rows, 0, None)


def context(f, cols):
    ln = ctypes.c_void_p()
    assert f.layernorm_create(cols, ctypes.byref(ln)) == osr.OK
    return ln


CASES = [(c, t) for c in (64, 600, 768, 1021, 4096, 8192, 12_000, 16_384)
         for t in (osr.DTYPE_F32, osr.DTYPE_BF16)]


@pytest.mark.parametrize("order", [(0, 1), (1, 0)])
@pytest.mark.parametrize("cols,dtype", CASES)
def test_layernorm_on_either_device(fake, cols, dtype, order):
    contexts = []
    for device in order:
        assert fake.cudaSetDevice(device) == 0
        contexts.append(context(fake, cols))
    assert fake.cudaSetDevice(0) == 0
    for _ in range(2):  # the first calls and the later ones
        for device, ln in zip(order, contexts):
            most = fake.fake_sms(device) * fake.fake_blocks(device) // 8 * 8
            for call in (forward, backward):
                assert call(fake, ln, cols, dtype) == osr.OK, (device, call.__name__)
                assert fake.fake_last_device() == device
                blocks = fake.fake_last_blocks()
                # as many as the device keeps, or as the partial sums have room for
                assert blocks == most or (call is backward and cols > 4096 and blocks == min(most, 304))
    for ln in contexts:
        assert fake.layernorm_destroy(ln) == osr.OK


@pytest.mark.parametrize("call", [forward, backward])
@pytest.mark.parametrize("attribute,occupancy", [(1, 0), (0, 1)])
def test_layernorm_reports_a_query_that_fails(fake, call, attribute, occupancy):
    cols = 4096
    ln = context(fake, cols)
    fake.fake_fail(attribute, occupancy)
    assert call(fake, ln, cols, osr.DTYPE_F32) == osr.ECUDA
    assert fake.fake_launches() == 0
    assert call(fake, ln, cols, osr.DTYPE_F32) == osr.OK
    assert fake.fake_last_blocks() == fake.fake_sms(0) * fake.fake_blocks(0) // 8 * 8


def make_list(f, numel, eight):
    h = ctypes.c_void_p()
    n = (ctypes.c_int64 * 1)(numel)
    assert f.adamw_list_create(1, n, (ctypes.c_uint8 * 1)(eight), ctypes.byref(h)) == osr.OK
    return h


def bind(f, h, g_dtype=osr.DTYPE_F32):
    row = ctypes.c_void_p * 1
    t = [row((k + 1) << 40) for k in range(6)]
    return f.adamw_list_bind(h, t[0], t[1], g_dtype, t[2], t[3], t[4], t[5], None, osr.DTYPE_BF16)


def step(f, h):
    return f.adamw_list_step(h, 1, 1e-3, 0.0, 1.0, 1.0, 0, 0, None)


@pytest.mark.parametrize("order", [(0, 1), (1, 0)])
@pytest.mark.parametrize("eight", [0, 1])
@pytest.mark.parametrize("g_dtype", [osr.DTYPE_F32, osr.DTYPE_BF16, osr.DTYPE_F16])
def test_list_step_on_either_device(fake, g_dtype, eight, order):
    lists = []
    for device in order:
        assert fake.cudaSetDevice(device) == 0
        lists.append(make_list(fake, 1 << 26, eight))
        assert bind(fake, lists[-1], g_dtype) == osr.OK
    assert fake.cudaSetDevice(0) == 0
    for device, h in zip(order, lists):
        assert step(fake, h) == osr.OK
        assert fake.fake_last_device() == device
        assert fake.fake_last_blocks() == fake.fake_sms(device) * fake.fake_blocks(device)
    for h in lists:
        assert fake.adamw_list_destroy(h) == osr.OK


@pytest.mark.parametrize("eight", [0, 1])
def test_list_reports_a_query_that_fails(fake, eight):
    h = make_list(fake, 1 << 26, eight)
    fake.fake_fail(0, 1)
    assert bind(fake, h) == osr.ECUDA
    assert step(fake, h) == osr.ESTATE and fake.fake_launches() == 0
    assert bind(fake, h) == osr.OK
    assert step(fake, h) == osr.OK
    assert fake.fake_last_blocks() == fake.fake_sms(0) * fake.fake_blocks(0)
