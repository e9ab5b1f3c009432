"""The linear layer's, the cross entropy's and the distillation's host code on a
runtime of two devices that run nothing (tests/c_abi/fake_cudart.cpp, with
fake_driver.cpp for tensor maps): workspaces, overlaps, devices, and what a
kernel that gave up leaves behind."""
import ctypes
import os
import random
import subprocess

import pytest

import optimizer_step_resumable_gb300 as osr
from optimizer_step_resumable_gb300 import build as lib_build

HERE = os.path.dirname(os.path.abspath(__file__))
F32, BF16, F16 = osr.DTYPE_F32, osr.DTYPE_BF16, osr.DTYPE_F16


@pytest.fixture(scope="module")
def fake_path(lib, tmp_path_factory):
    """The library's own objects, linked with the fake runtime and driver."""
    out = tmp_path_factory.mktemp("fake")
    names = lib_build.CUDA_SOURCES + lib_build.CXX_SOURCES
    objects = [os.path.join(lib_build.BUILD_DIR, s + ".o") for s in names]
    if not all(os.path.exists(o) for o in objects):
        lib_build.build(force=True)
    cuda = os.path.join(os.path.dirname(os.path.dirname(lib_build.nvcc())), "include")
    fakes = []
    for name in ("fake_cudart", "fake_driver"):
        fakes.append(str(out / (name + ".o")))
        subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-I", cuda, "-c",
                        os.path.join(HERE, "c_abi", name + ".cpp"), "-o", fakes[-1]], check=True)

    def symbols(flag, files):
        text = subprocess.run(["nm", flag, *files], capture_output=True, text=True, check=True).stdout
        return {line.split()[-1] for line in text.splitlines() if "cuda" in line}

    missing = symbols("--undefined-only", objects) - symbols("--defined-only", fakes)
    missing = sorted(s for s in missing if s.lstrip("_").startswith("cuda"))
    rest = out / "rest.c"
    rest.write_text("".join(f"long {s}(void) {{ return 0; }}\n" for s in missing))
    subprocess.run(["gcc", "-fno-builtin", "-fPIC", "-c", str(rest), "-o", str(out / "rest.o")],
                   check=True)
    path = str(out / "libfake.so")
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", path, *objects, *fakes,
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


def create(f, kind, *sizes):
    h = ctypes.c_void_p()
    assert getattr(f, kind + "_create")(*sizes, ctypes.byref(h)) == osr.OK
    return h


def place(k, at=0):
    """A made-up address, apart from the others."""
    return (k << 40) + 2 * at


WORK = place(20)


def workspace(f, kind, h, rows, flags):
    n = ctypes.c_int64(-1)
    assert getattr(f, kind + "_workspace")(h, rows, flags, ctypes.byref(n)) == osr.OK
    return n.value


def draw_size(r, most):
    n = int(2 ** r.uniform(0, most))
    return max(1, n // 8 * 8) if r.random() < 0.5 else n


def sizes(seed):
    """Sizes of a call, whether its matrices start anywhere, and their strides."""
    r = random.Random(seed)
    rows, a, b = draw_size(r, 21), draw_size(r, 14), draw_size(r, 17)
    any_address = r.random() < 0.5
    at = r.randrange(8) if any_address else 0

    def stride(n):
        return n + (r.randrange(9) if any_address else -n % 8)

    return r, rows, a, b, any_address, at, stride


# the bytes that the query names are enough for every call on these sizes, and
# every tensor map is one that the driver accepts
@pytest.mark.parametrize("seed", range(120))
def test_linear_workspaces_are_enough(fake, seed):
    r, rows, cin, cout, any_address, at, stride = sizes(seed)
    lin = create(fake, "linear", cin, cout)
    flag = osr.LINEAR_FOR_ANY_ADDRESS if any_address else 0
    for _ in range(4):
        dtype, act = r.choice((BF16, F16)), r.choice((0, 1, 2))
        in_out, grad_in_out = r.random() < 0.5, r.random() < 0.5
        w = (cin, cout) if in_out else (cout, cin)
        ws = stride(w[1])
        n = workspace(fake, "linear", lin, rows, flag)
        if rows * max(cin, cout) * 2 < 1 << 39:
            rc = fake.linear_forward(
                lin, place(1, at), stride(cin), place(2, at), ws, dtype, place(3), dtype, None, 0,
                act, place(4, at), stride(cout), place(5, at) if r.random() < 0.5 else None,
                stride(cout), rows, osr.LINEAR_IN_OUT if in_out else 0, WORK, n, None)
            assert rc == osr.OK, fake.adamw_last_error()
            grad = r.choice((F32, BF16, F16))
            flags = (osr.LINEAR_IN_OUT if in_out else 0) | r.choice((0, osr.LINEAR_ACCUMULATE)) | (
                osr.LINEAR_GRAD_IN_OUT if grad_in_out else 0)
            n = workspace(fake, "linear", lin, rows, flag | osr.LINEAR_FOR_BACKWARD)
            rc = fake.linear_backward(
                lin, place(6, at), stride(cout), place(1, at), stride(cin), place(2, at), ws, dtype,
                place(5, at), stride(cout), act, place(7, at) if r.random() < 0.8 else None,
                stride(cin), place(8) if r.random() < 0.8 else None,
                stride(cout if grad_in_out else cin), place(9) if r.random() < 0.8 else None, grad,
                rows, flags, WORK, n, None)
            assert rc == osr.OK, fake.adamw_last_error()
    assert fake.fake_maps_refused() == 0
    assert fake.linear_destroy(lin) == osr.OK


@pytest.mark.parametrize("seed", range(60))
def test_cross_entropy_workspaces_are_enough(fake, seed):
    r, rows, dim, vocab, any_address, at, stride = sizes(1000 + seed)
    ce = create(fake, "linear_cross_entropy", dim, vocab)
    flag = osr.LINEAR_FOR_ANY_ADDRESS if any_address else 0
    for _ in range(3):
        dtype, in_out, grad_in_out = r.choice((BF16, F16)), r.random() < 0.5, r.random() < 0.5
        ws = stride(vocab if in_out else dim)
        n = workspace(fake, "linear_cross_entropy", ce, rows, flag)
        rc = fake.linear_cross_entropy_forward(
            ce, place(1, at), stride(dim), place(2, at), ws, dtype, place(3), 0.0, place(4),
            place(5), rows, osr.LINEAR_IN_OUT if in_out else 0, WORK, n, None)
        assert rc == osr.OK, fake.adamw_last_error()
        n = workspace(fake, "linear_cross_entropy", ce, rows, flag | osr.LINEAR_FOR_BACKWARD)
        flags = (osr.LINEAR_IN_OUT if in_out else 0) | (osr.LINEAR_GRAD_IN_OUT if grad_in_out else 0)
        rc = fake.linear_cross_entropy_backward(
            ce, place(1, at), stride(dim), place(2, at), ws, dtype, place(3), place(5), None, 1.0,
            0.0, place(6, at) if r.random() < 0.8 else None, stride(dim),
            place(8) if r.random() < 0.8 else None, stride(vocab if grad_in_out else dim),
            r.choice((F32, BF16, F16)), rows, flags, WORK, n, None)
        assert rc == osr.OK, fake.adamw_last_error()
    assert fake.fake_maps_refused() == 0
    assert fake.linear_cross_entropy_destroy(ce) == osr.OK


def forward(f, lin, x=place(1), w=place(2), y=place(3), res=None, z=None, rows=100, xs=64, ys=48,
            rs=48, zs=48, act=0, dtype=BF16, work=WORK, n=1 << 30, flags=0):
    return f.linear_forward(lin, x, xs, w, 64, dtype, None, dtype, res, rs, act, y, ys, z, zs, rows,
                            flags, work, n, None)


def test_linear_refuses(fake):
    lin = create(fake, "linear", 64, 48)
    assert forward(fake, lin) == osr.OK and fake.fake_launches() > 0
    before = fake.fake_launches()
    for word, bad in (("d_x is NULL", dict(x=None)), ("d_weight is NULL", dict(w=None)),
                      ("aligned", dict(x=place(1) + 1)), ("rows", dict(rows=-1)),
                      ("rows", dict(rows=(1 << 30) + 1)), ("apart", dict(xs=63)),
                      ("apart", dict(ys=40)), ("activation", dict(act=5)), ("dtype", dict(dtype=F32)),
                      ("flags", dict(flags=osr.LINEAR_ACCUMULATE)), ("overlaps", dict(y=place(1) + 64)),
                      ("overlaps", dict(z=place(3) + 32)), ("overlaps", dict(res=place(3) + 2)),
                      ("overlaps", dict(res=place(3), rs=56)), ("overlaps", dict(y=place(2)))):
        assert forward(fake, lin, **bad) == osr.EINVAL, bad
        assert word in fake.adamw_last_error().decode(), (bad, fake.adamw_last_error())
    # an x that has to be copied needs a workspace
    assert forward(fake, lin, x=place(1, 1), work=None, n=0) == osr.EINVAL
    assert b"needs" in fake.adamw_last_error()
    assert forward(fake, lin, x=place(1, 1), work=WORK + 8) == osr.EINVAL
    assert forward(fake, lin, x=place(1, 1), n=100) == osr.EINVAL
    assert fake.fake_launches() == before
    assert forward(fake, lin, res=place(3)) == osr.OK  # in place
    # rows that lie between one another's (columns of one matrix) do not overlap
    assert forward(fake, lin, x=place(1), xs=112, y=place(1) + 128, ys=112) == osr.OK


def test_contexts_keep_to_their_device(fake):
    made = []
    for device in (1, 0):
        assert fake.cudaSetDevice(device) == 0
        made.append((device, create(fake, "linear", 64, 48), create(fake, "linear_cross_entropy", 64, 48),
                     create(fake, "distill", 1000, 8)))
    for device, lin, ce, ds in made:
        for call in (lambda: forward(fake, lin, rows=5000),
                     lambda: fake.linear_cross_entropy_forward(
                         ce, place(1), 64, place(2), 64, BF16, place(3), 0.0, place(4), place(5),
                         500, 0, WORK, 1 << 30, None),
                     lambda: fake.distill_forward(ds, place(1), 1000, F32, place(2), place(3), F32,
                                                  1.0, place(4), place(5), 10, None)):
            assert call() == osr.OK
            assert fake.fake_last_device() == device
            now = ctypes.c_int()
            assert fake.cudaGetDevice(ctypes.byref(now)) == 0 and now.value == 0
    # pairs of blocks on the device's SMs
    assert fake.cudaSetDevice(0) == 0
    big = create(fake, "linear", 512, 4096)
    assert fake.linear_forward(big, place(1), 512, place(2), 512, BF16, None, BF16, None, 0, 0,
                               place(3), 4096, None, 0, 1 << 16, 0, WORK, 1 << 30, None) == osr.OK
    assert fake.fake_last_blocks() == fake.fake_sms(0) // 2 * 2


def test_a_query_that_fails_is_the_calls_error(fake):
    lin = create(fake, "linear", 64, 48)
    fake.fake_fail(1, 0)
    assert forward(fake, lin) == osr.ECUDA and fake.fake_launches() == 0
    assert forward(fake, lin) == osr.OK


def test_a_kernel_that_gave_up_is_reported_once(fake):
    # the context's word in host memory, which such a kernel sets: device and SM
    # count come before its address
    for kind, call in (("linear", lambda h: forward(fake, h)),
                       ("linear_cross_entropy", lambda h: fake.linear_cross_entropy_forward(
                           h, place(1), 64, place(2), 64, BF16, place(3), 0.0, place(4), place(5),
                           10, 0, WORK, 1 << 30, None))):
        h = create(fake, kind, 64, 48)
        assert call(h) == osr.OK
        word = ctypes.cast(h.value + 8, ctypes.POINTER(ctypes.POINTER(ctypes.c_int32))).contents
        assert word[0] == 0
        word[0] = 1
        assert call(h) == osr.ESTATE and b"gave up" in fake.adamw_last_error()
        assert call(h) == osr.OK


def test_distillation_refuses(fake):
    ds = create(fake, "distill", 1000, 8)

    def back(l=place(1), ls=1000, dl=place(2), dls=1000, rows=10, dtype=F32, t=1.0, scale=1.0,
             vdtype=F32):
        return fake.distill_backward(ds, l, ls, dtype, place(3), place(4), vdtype, t, place(5), None,
                                     scale, dl, dls, rows, None)

    assert back() == osr.OK and back(dl=place(1)) == osr.OK
    for bad in (dict(l=None), dict(dl=None), dict(ls=999), dict(dls=10), dict(rows=-1),
                dict(rows=1 << 31), dict(dtype=3), dict(vdtype=-1), dict(t=0.0), dict(t=-2.0),
                dict(t=float("inf")), dict(t=1e-42), dict(scale=float("nan")), dict(scale=1e60),
                dict(dl=place(1) + 4), dict(dl=place(1), dls=1004), dict(l=place(1) + 2),
                dict(dl=place(3))):
        assert back(**bad) == osr.EINVAL, bad
    assert back(rows=0, l=None, dl=None) == osr.OK
