"""Host-side checks of the 8-bit integer operators that need no GPU: argument
validation through the C ABI (no call here reaches a launch), workspace sizes
and the binding's tensor checks."""
import ctypes
import os
import subprocess

import pytest

from block_wise_mixed_b200 import _lib as B
from block_wise_mixed_b200 import build

P = ctypes.c_void_p
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


def mat(rows=4, cols=64, ld=None, codes=16, scales=16):
    return B.I8(rows, cols, (cols + 15) // 16 * 16 if ld is None else ld, codes, scales)


def ref(m):
    return None if m is None else ctypes.byref(m)


def status(st):
    return B.STATUS[st]


def test_header_declares_and_library_exports(lib):
    names = set(B.header_functions())
    want = {"mpq_i8_quantize", "mpq_i8_dequantize", "mpq_i8_linear", "mpq_i8_gated", "mpq_i8_linear_backward",
            "mpq_i8_gated_backward"}
    want |= {n + "_workspace_size" for n in want if "quantize" not in n}
    assert want <= names
    for n in want:
        assert hasattr(lib, n)


def test_struct_size():
    assert ctypes.sizeof(B.I8) == 32


# what every call refuses in an int8 matrix
BAD = [
    (dict(rows=-1), "MPQ_ERR_SHAPE"), (dict(cols=0), "MPQ_ERR_SHAPE"), (dict(cols=131072), "MPQ_ERR_SHAPE"),
    (dict(ld=48), "MPQ_ERR_ARG"), (dict(cols=60, ld=60), "MPQ_ERR_ARG"), (dict(codes=None), "MPQ_ERR_ARG"),
    (dict(codes=24), "MPQ_ERR_ARG"), (dict(scales=None), "MPQ_ERR_ARG"), (dict(scales=18), "MPQ_ERR_ARG"),
]


@pytest.mark.parametrize("kw,err", BAD)
def test_bad_matrices(lib, kw, err):
    bad, good = mat(**kw), mat()
    q = lib.mpq_i8_quantize
    assert status(q(P(16), 0, 1 << 20, ref(bad), None)) == err
    assert status(lib.mpq_i8_dequantize(ref(bad), P(16), 0, 1 << 20, None)) == err
    for x, w in ((bad, good), (good, bad)):
        assert status(lib.mpq_i8_linear(ref(x), ref(w), P(16), 0, 1 << 20, P(256), BIG, None)) == err
    for x, g, u in ((bad, good, good), (good, bad, good), (good, good, bad)):
        assert status(lib.mpq_i8_gated(ref(x), ref(g), ref(u), 0, P(16), 1, 1 << 20, P(256), BIG, None)) == err
        assert status(lib.mpq_i8_gated_backward(ref(x), ref(g), ref(u), 0, P(16), 1 << 20, P(16), P(16), 1 << 20,
                                                P(16), 1 << 20, P(256), BIG, None)) == err
    assert status(lib.mpq_i8_linear_backward(ref(bad), P(16), 4, 1 << 20, P(16), 1 << 20, P(256), BIG, None)) == err


def test_rows(lib):
    m = mat()
    q, d = lib.mpq_i8_quantize, lib.mpq_i8_dequantize
    assert status(q(P(16), 0, 64, None, None)) == "MPQ_ERR_ARG"
    assert status(q(None, 0, 64, ref(m), None)) == "MPQ_ERR_ARG"
    assert status(q(P(16), 2, 64, ref(m), None)) == "MPQ_ERR_ARG"     # no such type
    assert status(q(P(16), 0, 63, ref(m), None)) == "MPQ_ERR_ARG"     # rows overlap
    assert status(q(P(18), 0, 64, ref(m), None)) == "MPQ_ERR_ARG"     # fp32 at an odd half word
    assert status(q(P(17), 1, 64, ref(m), None)) == "MPQ_ERR_ARG"
    assert status(d(ref(m), None, 0, 64, None)) == "MPQ_ERR_ARG"
    assert status(d(ref(m), P(16), 3, 64, None)) == "MPQ_ERR_ARG"
    assert status(d(ref(m), P(16), 0, 63, None)) == "MPQ_ERR_ARG"
    empty = mat(rows=0, codes=None, scales=None)
    assert q(None, 0, 64, ref(empty), None) == 0
    assert d(ref(empty), None, 0, 64, None) == 0


def test_linear(lib):
    x, w = mat(rows=5), mat(rows=96)
    f = lib.mpq_i8_linear
    need = lib.mpq_i8_linear_workspace_size(5, 96, 64)

    def call(x=x, w=w, y=16, dt=0, ldy=96, ws=256, size=need):
        return status(f(ref(x), ref(w), P(y) if y else None, dt, ldy, P(ws) if ws else None, size, None))
    assert need >= 256
    assert call(x=None) == "MPQ_ERR_ARG" and call(w=None) == "MPQ_ERR_ARG"
    assert call(y=None) == "MPQ_ERR_ARG" and call(y=18) == "MPQ_ERR_ARG" and call(y=17, dt=1) == "MPQ_ERR_ARG"
    assert call(dt=2) == "MPQ_ERR_ARG" and call(dt=-1) == "MPQ_ERR_ARG"
    assert call(ldy=95) == "MPQ_ERR_ARG"
    assert call(ws=None) == "MPQ_ERR_WORKSPACE" and call(ws=128) == "MPQ_ERR_WORKSPACE"
    assert call(size=need - 1) == "MPQ_ERR_WORKSPACE"
    assert call(w=mat(rows=96, cols=65)) == "MPQ_ERR_SHAPE"
    assert call(w=mat(rows=0, codes=None, scales=None)) == "MPQ_ERR_SHAPE"
    assert call(x=mat(rows=0, codes=None, scales=None), y=None, ws=None) == "MPQ_OK"


def test_gated(lib):
    x, g, u = mat(rows=5), mat(rows=96), mat(rows=96)
    need = lib.mpq_i8_gated_workspace_size(5, 96, 64)

    def call(x=x, g=g, u=u, act=0, y=16, dt=1, ldy=96, ws=256, size=need):
        return status(lib.mpq_i8_gated(ref(x), ref(g), ref(u), act, P(y) if y else None, dt, ldy,
                                       P(ws) if ws else None, size, None))
    assert call(g=None) == "MPQ_ERR_ARG" and call(u=None) == "MPQ_ERR_ARG"
    assert call(act=2) == "MPQ_ERR_ARG" and call(act=-1) == "MPQ_ERR_ARG" and call(dt=2) == "MPQ_ERR_ARG"
    assert call(u=mat(rows=95)) == "MPQ_ERR_SHAPE" and call(u=mat(rows=96, cols=63)) == "MPQ_ERR_SHAPE"
    assert call(ldy=95) == "MPQ_ERR_ARG" and call(y=None) == "MPQ_ERR_ARG"
    assert call(ws=None) == "MPQ_ERR_WORKSPACE" and call(size=need - 1) == "MPQ_ERR_WORKSPACE"
    assert call(x=mat(rows=0, codes=None, scales=None), y=None, ws=None) == "MPQ_OK"


def test_backward(lib):
    w = mat(rows=96)
    need = lib.mpq_i8_linear_backward_workspace_size(5, 96, 64)

    def lin(w=w, dy=16, M=5, lddy=96, dx=16, lddx=64, ws=256, size=need):
        return status(lib.mpq_i8_linear_backward(ref(w), P(dy) if dy else None, M, lddy, P(dx) if dx else None, lddx,
                                                 P(ws) if ws else None, size, None))
    assert lin(w=None) == "MPQ_ERR_ARG" and lin(dy=None) == "MPQ_ERR_ARG" and lin(dx=None) == "MPQ_ERR_ARG"
    assert lin(dy=17) == "MPQ_ERR_ARG" and lin(dx=17) == "MPQ_ERR_ARG"
    assert lin(lddy=95) == "MPQ_ERR_ARG" and lin(lddx=63) == "MPQ_ERR_ARG"
    assert lin(M=-1) == "MPQ_ERR_SHAPE" and lin(M=0, dy=None, dx=None, ws=None) == "MPQ_OK"
    assert lin(w=mat(rows=0, codes=None, scales=None)) == "MPQ_ERR_SHAPE"
    assert lin(ws=None) == "MPQ_ERR_WORKSPACE" and lin(size=need - 1) == "MPQ_ERR_WORKSPACE"

    x, g, u = mat(rows=5), mat(rows=96), mat(rows=96)
    need = lib.mpq_i8_gated_backward_workspace_size(5, 96, 64)

    def gat(x=x, g=g, u=u, act=0, dh=16, lddh=96, dg=16, du=16, ldd=96, dx=16, lddx=64, ws=256, size=need):
        pp = [P(v) if v else None for v in (dh, dg, du, dx, ws)]
        return status(lib.mpq_i8_gated_backward(ref(x), ref(g), ref(u), act, pp[0], lddh, pp[1], pp[2], ldd, pp[3],
                                                lddx, pp[4], size, None))
    assert gat(act=2) == "MPQ_ERR_ARG" and gat(dh=None) == "MPQ_ERR_ARG" and gat(dx=None) == "MPQ_ERR_ARG"
    assert gat(dg=None) == "MPQ_ERR_ARG" and gat(du=None) == "MPQ_ERR_ARG"      # both or neither
    assert gat(lddh=95) == "MPQ_ERR_ARG" and gat(ldd=95) == "MPQ_ERR_ARG" and gat(lddx=63) == "MPQ_ERR_ARG"
    assert gat(dg=17) == "MPQ_ERR_ARG" and gat(du=17) == "MPQ_ERR_ARG"
    assert gat(u=mat(rows=95)) == "MPQ_ERR_SHAPE" and gat(x=mat(rows=5, cols=65)) == "MPQ_ERR_SHAPE"
    assert gat(ws=None) == "MPQ_ERR_WORKSPACE" and gat(size=need - 1) == "MPQ_ERR_WORKSPACE"
    assert gat(x=mat(rows=0, codes=None, scales=None), dh=None, dx=None, ws=None) == "MPQ_OK"


@pytest.mark.parametrize("name", ["linear", "gated", "linear_backward", "gated_backward"])
def test_workspace_sizes(lib, name):
    f = getattr(lib, "mpq_i8_%s_workspace_size" % name)
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 131072)):
        assert f(*bad) == 0
    for M in (0, 1, 17, 300, 5000):
        for N, K in ((1, 1), (1371, 2003), (28672, 8192)):
            assert f(M, N, K) >= 256 and f(M, N, K) % 256 == 0


def test_binding_refuses(lib):
    """Tensor checks of the binding; they raise before the library is called."""
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(B.MpqError) as ei:
        B.i8_quantize(x)                       # not on a CUDA device
    assert ei.value.name == "MPQ_ERR_ARG"
    with pytest.raises(B.MpqError):
        B.i8_quantize(x.half())                # neither bf16 nor fp32
    with pytest.raises(B.MpqError):
        B.i8_quantize(x[0])                    # one dimension
    with pytest.raises(B.MpqError):
        B.i8_matrix(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4))
    with pytest.raises(B.MpqError):
        B.i8_linear(x, x)                      # no int8 matrices


def test_row_words_end_at_the_last_column(tmp_path):
    """The host build of the row kernels' fetch of codes (tests/native/i8_words.cu)."""
    exe = tmp_path / "i8_words"
    src = os.path.join(os.path.dirname(__file__), "native", "i8_words.cu")
    nvcc = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_100a,code=sm_100a", "-o", str(exe), src],
                   check=True, capture_output=True, text=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout == "ok\n"


@pytest.mark.parametrize("name", ["linear", "gated", "linear_backward", "gated_backward"])
def test_workspace_of_the_largest_batch_serves_smaller_ones(lib, name):
    """Sizes never fall as the batch grows, through every change of plan."""
    f = getattr(lib, "mpq_i8_%s_workspace_size" % name)
    batches = list(range(0, 140)) + [191, 192, 255, 256, 257, 300, 511, 512, 513, 1000, 2048, 4096, 100000]
    for N, K in ((1, 1), (96, 64), (1371, 2003), (9728, 16384), (4096, 14336), (19100, 6000), (28672, 8192)):
        sizes = [f(M, N, K) for M in batches]
        assert sizes == sorted(sizes), (N, K)


def test_header_constants():
    text = open(B.HEADER).read()
    for name, value in (("MPQ_I8_MAX_COLS", B.I8_MAX_COLS), ("MPQ_I8_WS_ZERO", B.I8_WS_ZERO)):
        assert "#define %s %d\n" % (name, value) in text


def test_own_workspace_is_zeroed_where_it_has_to_be(lib, monkeypatch):
    """A call without a workspace clears the first bytes of its own, and no more."""
    import torch
    made = []
    empty = torch.empty

    def poisoned(*a, **k):
        made.append(empty(*a, **k).fill_(0xAB))
        return made[-1]
    monkeypatch.setattr(torch, "empty", poisoned)
    monkeypatch.setattr(B, "_call", lambda *a: None)
    B._call_ws("mpq_i8_gated_backward", (300, 1371, 2003), torch.device("cpu"), None, None)
    ws, = made
    assert ws.numel() == lib.mpq_i8_gated_backward_workspace_size(300, 1371, 2003)
    assert bool((ws[:B.I8_WS_ZERO] == 0).all()) and bool((ws[B.I8_WS_ZERO:] == 0xAB).all())


def test_plan_arguments(lib):
    work = (B.I8Work * 2)()
    assert ctypes.sizeof(B.I8Work) == 40
    assert status(lib.mpq_i8_plan(0, 1, 1, 1, None)) == "MPQ_ERR_ARG"
    for op in (-1, 4):
        assert status(lib.mpq_i8_plan(op, 1, 1, 1, work)) == "MPQ_ERR_ARG"
    for bad in ((0, 1, 1), (-1, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 131072)):
        assert status(lib.mpq_i8_plan(0, *bad, work)) == "MPQ_ERR_SHAPE"
    with pytest.raises(B.MpqError):
        B.i8_plan("dequantize", 1, 1, 1)
    for op, parts in (("linear", ["product"]), ("gated", ["product"]), ("linear_backward", ["gradient"]),
                      ("gated_backward", ["product", "gradient"])):
        for shape in ((1, 1, 1), (2 ** 31 - 1, 1, 1), (1, 2 ** 31 - 1, 16), (700, 5000, 3000)):
            assert list(B.i8_plan(op, *shape)) == parts


def test_shapes_of_every_plan(lib):
    """Each shape of i8_shapes.py is handed out the way it is listed for, and no
    shape in a wide sweep takes a way that has none listed."""
    import random

    import i8_shapes
    listed = set()
    for op, part, kernel, columns, how, M, N, K in i8_shapes.cases():
        assert i8_shapes.classes(B.i8_plan(op, M, N, K))[part] == (kernel, columns, how), (op, M, N, K)
        listed.add((op, part, kernel, columns, how))
    rng = random.Random(11)
    for _ in range(60000):
        op = rng.choice(("linear", "gated", "linear_backward", "gated_backward"))
        M, N, K = (int(round(2 ** rng.uniform(a, b))) for a, b in ((0, 12), (0, 15), (0, 15)))
        for part, way in i8_shapes.classes(B.i8_plan(op, M, N, K)).items():
            assert (op, part, *way) in listed, (op, M, N, K)


@pytest.mark.parametrize("name", ["linear", "gated", "linear_backward", "gated_backward"])
def test_workspace_holds_what_the_plan_takes(lib, name):
    """Partial sums of every batch fit behind the zeroed part of the size for larger ones."""
    f = getattr(lib, "mpq_i8_%s_workspace_size" % name)
    for N, K in ((96, 64), (1371, 2003), (9728, 16384), (4096, 14336), (19100, 6000), (28672, 8192), (128000, 4096)):
        for M in list(range(1, 140)) + [200, 255, 256, 257, 300, 511, 512, 1000, 2048, 4096]:
            need = max(w["slots"] for w in B.i8_plan(name, M, N, K).values())
            assert B.I8_WS_ZERO + need <= f(M, N, K), (M, N, K)
