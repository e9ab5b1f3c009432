"""How the tiled products are divided and dealt out, read from the arguments of
their launches on a runtime that runs nothing (tests/c_abi/fake_products.cpp)."""
import ctypes
import os
import subprocess

import pytest

import optimizer_step_resumable_gb300 as osr
from optimizer_step_resumable_gb300 import build as lib_build

HERE = os.path.dirname(os.path.abspath(__file__))
F32, BF16, F16 = osr.DTYPE_F32, osr.DTYPE_BF16, osr.DTYPE_F16
WORK = 20 << 40


def place(k):
    """A made-up address, apart from the others."""
    return k << 40


@pytest.fixture(scope="module")
def fake(lib, tmp_path_factory):
    """The library's own objects, linked with the fake runtime, driver and launches."""
    out = tmp_path_factory.mktemp("fake")
    names = lib_build.CUDA_SOURCES + lib_build.CXX_SOURCES
    objects = [os.path.join(lib_build.BUILD_DIR, s + ".o") for s in names]
    if not all(os.path.exists(o) for o in objects):
        lib_build.build(force=True)
    cuda = os.path.join(os.path.dirname(os.path.dirname(lib_build.nvcc())), "include")
    fakes = []
    for name, more in (("fake_cudart", ["-DcudaLaunchKernelExC=fake_launch"]), ("fake_driver", []),
                       ("fake_products", [])):
        fakes.append(str(out / (name + ".o")))
        subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-I", cuda, *more, "-c",
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
    f = ctypes.CDLL(path)
    for name, (res, args) in osr.SIGNATURES.items():
        getattr(f, name).restype = res
        getattr(f, name).argtypes = args
    f.fake_product.restype = ctypes.POINTER(ctypes.c_int)
    return f


SHAPE = ("m", "n", "tiles_m", "tiles_n", "splits", "chains", "blocks")
DEAL = ("pairs", "longs", "ahead", "shorts", "after", "before")


def launches(f, call):
    """The products of a call: (first's shape, second's or None, the deal)."""
    f.fake_products_clear()
    assert call() == osr.OK, f.adamw_last_error()
    out = []
    for i in range(f.fake_products()):
        p = f.fake_product(i)
        one, two = (dict(zip(SHAPE, p[7 * k:7 * k + 7])) for k in (0, 1))
        out.append((one, two if two["blocks"] else None, dict(zip(DEAL, p[14:20]))))
    return out


def create(f, kind, *sizes):
    h = ctypes.c_void_p()
    assert getattr(f, kind + "_create")(*sizes, ctypes.byref(h)) == osr.OK
    return h


def ce_backward(f, dim, vocab, rows, dtype, grad, flags=0, dx=True, dw=True):
    ce = create(f, "linear_cross_entropy", dim, vocab)
    n = ctypes.c_int64()
    assert f.linear_cross_entropy_workspace(ce, rows, osr.LINEAR_FOR_BACKWARD,
                                            ctypes.byref(n)) == osr.OK
    got = launches(f, lambda: f.linear_cross_entropy_backward(
        ce, place(1), dim, place(2), dim, dtype, place(3), place(5), None, 1.0, 0.0,
        place(6) if dx else None, dim, place(8) if dw else None, dim, grad, rows, flags, WORK,
        n.value, None))
    f.linear_cross_entropy_destroy(ce)
    return got


def backward(f, cin, cout, rows, dtype, grad, flags=0, dx=True, dw=True):
    lin = create(f, "linear", cin, cout)
    n = ctypes.c_int64()
    assert f.linear_workspace(lin, rows, osr.LINEAR_FOR_BACKWARD, ctypes.byref(n)) == osr.OK
    got = launches(f, lambda: f.linear_backward(
        lin, place(1), cout, place(2), cin, place(3), cin, dtype, None, 0, 0,
        place(6) if dx else None, cin, place(8) if dw else None, cin, None, grad, rows, flags,
        WORK, n.value, None))
    f.linear_destroy(lin)
    return got


# Microseconds that an item takes, as the planner has it: its blocks of the inner
# dimension, its start and end, and each chain after the first.
def item_us(shape):
    each = -(-shape["blocks"] // shape["splits"])
    return 0.316 * each + 0.3 + 1.3 * (shape["chains"] - 1)


def items(shape):
    return shape["tiles_m"] * shape["tiles_n"] * shape["splits"]


def ends(deal, long_us, short_us):
    """When the last pair of blocks is done."""
    rounds = deal["longs"] // deal["pairs"]
    late = (rounds + 1) * long_us + deal["after"] * short_us if deal["ahead"] else 0.0
    return max(late, rounds * long_us + deal["before"] * short_us)


@pytest.mark.parametrize("dim,vocab,rows,grad", [
    (768, 32000, 8192, F32), (768, 32000, 8192, BF16), (2048, 50000, 16384, F32),
    (1024, 100000, 4096, F32), (640, 70001, 8192, F32)])
def test_two_products_are_dealt_out_by_the_time_they_take(fake, dim, vocab, rows, grad):
    # the pieces of a vocabulary write dx in float32 but for the last one
    for one, two, deal in ce_backward(fake, dim, vocab, rows, BF16, grad, osr.LINEAR_ACCUMULATE):
        if two is None:
            continue
        long_us, short_us = item_us(one), item_us(two)
        assert long_us >= short_us
        assert (deal["longs"], deal["shorts"]) == (items(one), items(two))
        assert deal["ahead"] == deal["longs"] % deal["pairs"]
        others, left = deal["pairs"] - deal["ahead"], deal["shorts"]
        best = min(ends(dict(deal, after=a, before=b), long_us, short_us)
                   for b in range(-(-left // others) + 1) for a in range(b + 1)
                   if a * deal["ahead"] + b * others >= left)
        assert ends(deal, long_us, short_us) <= best + 1e-6, (one, two, deal, best)


# each 16 products of equal signs lose up to 1.7 x 2^-24 of the sum: these many lose
# less than a quarter of the type's rounding, 2^-13 or 2^-10
CHAIN = {F16: 1 << 14, BF16: 1 << 17, F32: 1 << 10}


def products_in_a_row(shape):
    return -(-shape["blocks"] // (shape["splits"] * shape["chains"])) * 64


@pytest.mark.parametrize("rows", [1000, 16384, 16385, 100000, 131072, 131073, 1 << 20, (1 << 22) + 7])
@pytest.mark.parametrize("cin,cout", [(4096, 16128), (768, 768), (2048, 100), (100, 2048)])
def test_sums_for_16_bits_are_in_chains_where_the_cut_would_show(fake, rows, cin, cout):
    for dtype in (F16, BF16):
        for grad in (F16, BF16, F32):
            for dx in (False, True):
                shapes = [s for one, two, _ in backward(fake, cin, cout, rows, dtype, grad, dx=dx)
                          for s in (one, two) if s and s["blocks"] == -(-rows // 64)]
                assert shapes, "no product over the rows"
                for s in shapes:
                    assert products_in_a_row(s) <= CHAIN[grad], (s, dtype, grad)
                    if rows <= CHAIN[grad]:
                        assert s["chains"] == 1 or grad == F32


@pytest.mark.parametrize("features", [40000, 300000])
def test_long_sums_of_outputs_and_inputs_too(fake, features):
    for dtype in (F16, BF16):
        lin = create(fake, "linear", features, 64)
        n = ctypes.c_int64()
        assert fake.linear_workspace(lin, 500, 0, ctypes.byref(n)) == osr.OK
        (one, _, _), = launches(fake, lambda: fake.linear_forward(
            lin, place(1), features, place(2), features, dtype, None, dtype, None, 0, 0, place(4), 64,
            None, 0, 500, 0, WORK, n.value, None))
        assert products_in_a_row(one) <= CHAIN[dtype], one
        fake.linear_destroy(lin)
        for one, two, _ in backward(fake, 64, features, 500, dtype, dtype, dw=False):
            assert two is None and products_in_a_row(one) <= CHAIN[dtype], one


@pytest.mark.parametrize("rows,vocab", [(300, 1 << 20), (200000, 5000), (70000, 40000)])
def test_long_sums_of_the_cross_entropys_gradients(fake, rows, vocab):
    for dtype in (F16, BF16):
        for grad in (F16, BF16, F32):
            got = ce_backward(fake, 512, vocab, rows, dtype, grad)
            for one, two, _ in got:
                for s in (one, two):
                    if s is None or s["blocks"] == 512 // 64:
                        continue  # the logits
                    over_rows = s["blocks"] == -(-rows // 64)
                    assert products_in_a_row(s) <= CHAIN[grad if over_rows else dtype], s


def test_calls_in_turn_with_one_context_are_planned_as_alone(fake):
    # more different calls than a context keeps plans of, in every order
    cin, cout = 768, 1536
    work = ctypes.c_int64(1 << 40)

    def calls(lin, rows, dtype):
        yield lambda: fake.linear_forward(
            lin, place(1), cin, place(2), cin, dtype, None, dtype, None, 0, 0, place(4), cout, None,
            0, rows, 0, WORK, work, None)
        for grad, dx in ((F32, True), (dtype, True), (F32, False)):
            yield lambda grad=grad, dx=dx: fake.linear_backward(
                lin, place(1), cout, place(2), cin, place(3), cin, dtype, None, 0, 0,
                place(6) if dx else None, cin, place(8), cin, None, grad, rows, 0, WORK, work, None)

    def alone(rows, dtype):
        lin = create(fake, "linear", cin, cout)
        got = [launches(fake, c) for c in calls(lin, rows, dtype)]
        fake.linear_destroy(lin)
        return got

    sizes = [(rows, dtype) for rows in (40, 1000, 300000) for dtype in (F16, BF16)]
    want = {s: alone(*s) for s in sizes}
    assert len({str(w) for w in want.values()}) > 3
    lin = create(fake, "linear", cin, cout)
    for turn in range(2):
        for s in sizes if turn == 0 else reversed(sizes):
            assert [launches(fake, c) for c in calls(lin, *s)] == want[s]
    for i in range(4):
        for s in sizes:
            assert launches(fake, list(calls(lin, *s))[i]) == want[s][i]
    fake.linear_destroy(lin)


@pytest.mark.parametrize("kind", ["linear", "linear_cross_entropy"])
def test_a_call_without_rows_reports_a_kernel_that_gave_up(fake, kind):
    # how a caller who replays a graph asks: no launch, the state once
    h = create(fake, kind, 64, 48)

    def ask():
        if kind == "linear":
            return fake.linear_forward(h, None, 64, place(2), 64, BF16, None, BF16, None, 0, 0, None,
                                       48, None, 0, 0, 0, None, 0, None)
        return fake.linear_cross_entropy_forward(h, None, 64, place(2), 64, BF16, None, 0.0, None,
                                                 None, 0, 0, None, 0, None)

    before = fake.fake_launches()
    assert ask() == osr.OK
    # the context's word in host memory, behind device and SM count
    word = ctypes.cast(h.value + 8, ctypes.POINTER(ctypes.POINTER(ctypes.c_int32))).contents
    word[0] = 1
    assert ask() == osr.ESTATE and b"gave up" in fake.adamw_last_error()
    assert ask() == osr.OK and fake.fake_launches() == before
