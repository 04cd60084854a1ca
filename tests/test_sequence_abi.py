"""The sequence operators refuse bad arguments on the host, before anything reaches a GPU:
the C ABI's checks with pointers that are never read, and the binding's on CPU tensors
(no compute call; no GPU needed)."""
import ctypes

import pytest
import torch

import sparse_memory_linear_scoring_b200 as sdm
from sparse_memory_linear_scoring_b200 import build as sdm_build

OK, ERR_NULL, ERR_DIMS, ERR_ALIGN, ERR_WS, ERR_UNSUP = 0, 1, 2, 3, 4, 5
P, S, I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
GOOD = 1 << 20  # an aligned address that no check reads


class Strides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in "bht"]


class ConvDims(ctypes.Structure):
    _fields_ = [(n, I) for n in ("B", "H", "T", "d", "K", "silu", "in_dtype")]


class SsmDims(ctypes.Structure):
    _fields_ = [(n, I) for n in ("B", "H", "G", "T", "d_k", "d_v", "in_dtype")]


class BlockDims(ctypes.Structure):
    _fields_ = [(n, I) for n in ("B", "H", "G", "Tq", "Tk", "d", "block", "n_sel", "in_dtype")] + \
               [("scale", ctypes.c_float)]


class Views(ctypes.Structure):
    _fields_ = [(n, Strides) for n in "abcde"]


@pytest.fixture(scope="module")
def lib():
    sdm_build.build()
    l = sdm.load_library()
    sp, cd, sd, bd, vw = (ctypes.POINTER(t) for t in (Strides, ConvDims, SsmDims, BlockDims, Views))
    for name, args in (("conv_forward", [P] * 6 + [cd, sp, sp, P]),
                       ("conv_backward", [P] * 10 + [cd, sp, sp, sp, P, S, P]),
                       ("ssm_forward", [P] * 9 + [sd, vw, P, S, P]), ("ssm_step", [P] * 8 + [sd, vw, P]),
                       ("ssm_backward", [P] * 16 + [sd, vw, vw, P, S, P]),
                       ("block_pool", [P, P, I, bd, vw, P]), ("block_select", [P, P, I, P, P, bd, vw, P]),
                       ("block_forward", [P] * 7 + [bd, vw, P, S, P]),
                       ("block_backward", [P] * 11 + [bd, vw, vw, P, S, P])):
        fn = getattr(l, "sdm_" + name)
        fn.argtypes, fn.restype = args, ctypes.c_int
    for name, d in (("conv_backward", cd), ("ssm", sd), ("ssm_backward", sd), ("block", bd), ("block_backward", bd)):
        fn = getattr(l, "sdm_%s_workspace_bytes" % name)
        fn.argtypes, fn.restype = [d], S
    return l


def _views(**bad):
    v = Views(*[Strides(1 << 20, 1 << 16, 64) for _ in range(5)])
    for n, s in bad.items():
        setattr(v, n, Strides(*s))
    return v


# ---------------------------------------------------------------- convolution
CONV = dict(B=2, H=3, T=50, d=64, K=4, silu=1, in_dtype=1)


@pytest.mark.parametrize("field,value,code", [
    ("B", 0, ERR_DIMS), ("H", 0, ERR_DIMS), ("T", -1, ERR_DIMS), ("d", 0, ERR_DIMS), ("K", 0, ERR_DIMS),
    ("K", 1, ERR_UNSUP), ("K", 9, ERR_UNSUP), ("in_dtype", 2, ERR_DIMS), ("T", (1 << 30) + 1, ERR_DIMS),
    ("d", 1 << 25, ERR_DIMS)])
def test_conv_sizes(lib, field, value, code):
    d = ConvDims(**{**CONV, field: value})
    s = Strides(1 << 20, 1 << 16, 64)
    assert lib.sdm_conv_forward(GOOD, GOOD, None, None, None, GOOD, d, s, s, None) == code
    assert lib.sdm_conv_backward(*[GOOD] * 10, d, s, s, s, GOOD, 1 << 40, None) == code
    assert lib.sdm_conv_backward_workspace_bytes(d) == 0


def test_conv_pointers_and_workspace(lib):
    d, s = ConvDims(**CONV), Strides(1 << 20, 1 << 16, 64)
    for i, rc in ((0, ERR_NULL), (1, ERR_NULL), (5, ERR_NULL)):
        a = [GOOD, GOOD, None, None, None, GOOD]
        a[i] = None
        assert lib.sdm_conv_forward(*a, d, s, s, None) == rc
    for i in range(6):
        a = [GOOD] * 6
        a[i] = GOOD + 1
        assert lib.sdm_conv_forward(*a, d, s, s, None) == ERR_ALIGN
    assert lib.sdm_conv_forward(*[GOOD] * 6, d, Strides(-1, 0, 0), s, None) == ERR_DIMS
    assert lib.sdm_conv_forward(*[GOOD] * 6, None, s, s, None) == ERR_NULL
    n = lib.sdm_conv_backward_workspace_bytes(d)
    assert n > 0
    back = lambda ws, size: lib.sdm_conv_backward(*[GOOD] * 10, d, s, s, s, ws, size, None)  # noqa: E731
    assert back(None, n) == ERR_WS and back(GOOD, n - 1) == ERR_WS and back(GOOD + 8, n) == ERR_ALIGN
    # no step: the forward has nothing to do, the backward nothing to differentiate
    z = ConvDims(**{**CONV, "T": 0})
    assert lib.sdm_conv_forward(*[None] * 6, z, s, s, None) == OK
    assert lib.sdm_conv_backward(*[GOOD] * 10, z, s, s, s, GOOD, n, None) == ERR_DIMS


# ---------------------------------------------------------------- scan
SSM = dict(B=2, H=4, G=2, T=50, d_k=64, d_v=64, in_dtype=1)


@pytest.mark.parametrize("field,value,code", [
    ("B", 0, ERR_DIMS), ("G", 0, ERR_DIMS), ("G", 3, ERR_DIMS), ("T", -1, ERR_DIMS), ("d_k", 0, ERR_DIMS),
    ("d_k", 48, ERR_UNSUP), ("d_v", 256, ERR_UNSUP), ("d_v", 8, ERR_UNSUP), ("in_dtype", 3, ERR_DIMS)])
def test_ssm_sizes(lib, field, value, code):
    d = SsmDims(**{**SSM, field: value})
    v = _views()
    assert lib.sdm_ssm_forward(*[GOOD] * 9, d, v, GOOD, 1 << 40, None) == code
    assert lib.sdm_ssm_step(*[GOOD] * 8, d, v, None) == code
    assert lib.sdm_ssm_backward(*[GOOD] * 16, d, v, v, GOOD, 1 << 40, None) == code
    assert lib.sdm_ssm_workspace_bytes(d) == 0 and lib.sdm_ssm_backward_workspace_bytes(d) == 0


def test_ssm_pointers_and_workspace(lib):
    d, v = SsmDims(**SSM), _views()
    names = ("x", "dt", "A", "Bm", "Cm", "D", "S", "lengths", "y")
    for i, n in enumerate(names):
        a = [GOOD] * 9
        a[i] = None
        if n not in ("D", "lengths"):
            assert lib.sdm_ssm_forward(*a, d, v, GOOD, 1 << 40, None) == ERR_NULL, n
        a[i] = GOOD + 1
        assert lib.sdm_ssm_forward(*a, d, v, GOOD, 1 << 40, None) == ERR_ALIGN, n
    a = [GOOD] * 9
    a[6] = GOOD + 8  # the state is read in pieces of 16 bytes
    assert lib.sdm_ssm_forward(*a, d, v, GOOD, 1 << 40, None) == ERR_ALIGN
    assert lib.sdm_ssm_forward(*[GOOD] * 9, d, _views(b=(0, 0, -4)), GOOD, 1 << 40, None) == ERR_DIMS
    assert lib.sdm_ssm_forward(*[GOOD] * 9, d, None, GOOD, 1 << 40, None) == ERR_NULL
    n = lib.sdm_ssm_workspace_bytes(SsmDims(**{**SSM, "T": 50000}))
    big = SsmDims(**{**SSM, "T": 50000})
    assert n > 16 and lib.sdm_ssm_forward(*[GOOD] * 9, big, v, GOOD, n - 1, None) == ERR_WS
    assert lib.sdm_ssm_forward(*[GOOD] * 9, big, v, None, n, None) == ERR_WS
    assert lib.sdm_ssm_forward(*[None] * 9, SsmDims(**{**SSM, "T": 0}), v, None, 0, None) == OK
    n = lib.sdm_ssm_backward_workspace_bytes(d)
    assert lib.sdm_ssm_backward(*[GOOD] * 16, d, v, v, GOOD, n - 1, None) == ERR_WS
    assert lib.sdm_ssm_backward(*[GOOD] * 16, SsmDims(**{**SSM, "T": 0}), v, v, GOOD, n, None) == ERR_DIMS


# ---------------------------------------------------------------- block attention
BLOCK = dict(B=2, H=8, G=2, Tq=100, Tk=500, d=64, block=64, n_sel=4, in_dtype=1, scale=0.125)


@pytest.mark.parametrize("field,value,code", [
    ("B", 0, ERR_DIMS), ("G", 3, ERR_DIMS), ("Tq", 501, ERR_DIMS), ("Tq", -1, ERR_DIMS), ("d", 0, ERR_DIMS),
    ("d", 96, ERR_UNSUP), ("block", 48, ERR_UNSUP), ("block", 256, ERR_UNSUP), ("n_sel", 0, ERR_DIMS),
    ("n_sel", 65, ERR_UNSUP), ("scale", float("nan"), ERR_DIMS), ("scale", float("inf"), ERR_DIMS),
    ("Tk", (1 << 28) + 1, ERR_DIMS), ("in_dtype", -1, ERR_DIMS)])
def test_block_sizes(lib, field, value, code):
    d = BlockDims(**{**BLOCK, field: value})
    v = _views()
    assert lib.sdm_block_forward(*[GOOD] * 7, d, v, GOOD, 1 << 50, None) == code
    assert lib.sdm_block_backward(*[GOOD] * 11, d, v, v, GOOD, 1 << 50, None) == code
    assert lib.sdm_block_select(GOOD, GOOD, 10000000, GOOD, GOOD, d, v, None) == code
    assert lib.sdm_block_pool(GOOD, GOOD, 0, d, v, None) == code
    assert lib.sdm_block_workspace_bytes(d) == 0 and lib.sdm_block_backward_workspace_bytes(d) == 0


def test_block_blocks_past_the_limit(lib):
    d = BlockDims(**{**BLOCK, "Tk": 49153 * 32, "block": 32})
    assert lib.sdm_block_select(GOOD, GOOD, 49153, GOOD, GOOD, d, _views(), None) == ERR_UNSUP


def test_block_pointers_and_workspace(lib):
    d, v = BlockDims(**BLOCK), _views()
    for i, n in enumerate(("q", "k", "v", "idx", "lengths", "o", "lse")):
        a = [GOOD] * 7
        a[i] = None
        if n not in ("lengths", "lse"):
            assert lib.sdm_block_forward(*a, d, v, GOOD, 1 << 50, None) == ERR_NULL, n
        a[i] = GOOD + 1
        assert lib.sdm_block_forward(*a, d, v, GOOD, 1 << 50, None) == ERR_ALIGN, n
    n = lib.sdm_block_workspace_bytes(d)
    assert lib.sdm_block_forward(*[GOOD] * 7, d, v, GOOD, n - 1, None) == ERR_WS
    assert lib.sdm_block_forward(*[GOOD] * 7, d, v, GOOD + 8, n, None) == ERR_ALIGN
    assert lib.sdm_block_forward(*[GOOD] * 7, d, _views(c=(1, 1, -1)), GOOD, n, None) == ERR_DIMS
    zero = BlockDims(**{**BLOCK, "Tq": 0})
    assert lib.sdm_block_forward(*[None] * 7, zero, v, None, 0, None) == OK
    assert lib.sdm_block_select(None, None, 7, None, None, zero, v, None) == OK
    assert lib.sdm_block_backward(*[GOOD] * 11, zero, v, v, GOOD, 1 << 50, None) == ERR_DIMS
    n = lib.sdm_block_backward_workspace_bytes(d)
    assert lib.sdm_block_backward(*[GOOD] * 11, d, v, v, GOOD, n - 1, None) == ERR_WS
    # every block before the last key's own needs its mean
    assert lib.sdm_block_select(GOOD, GOOD, 6, None, GOOD, d, v, None) == ERR_DIMS
    assert lib.sdm_block_pool(GOOD, GOOD, 8, d, v, None) == ERR_DIMS      # 7 complete blocks
    assert lib.sdm_block_pool(GOOD, GOOD, -1, d, v, None) == ERR_DIMS
    assert lib.sdm_block_pool(None, None, 7, d, v, None) == OK            # none is left to do


# ---------------------------------------------------------------- binding
def t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("call,error,text", [
    (lambda: sdm.conv_forward(t(2, 3, 4), t(3, 4, 4)), ValueError, "must be"),
    (lambda: sdm.conv_forward(t(1, 2, 3, 4), t(2, 4)), ValueError, "must be"),
    (lambda: sdm.conv_forward(t(1, 2, 3, 4), t(3, 4, 4)), ValueError, "w has shape"),
    (lambda: sdm.conv_forward(t(1, 2, 3, 4, dtype=torch.float16), t(2, 4, 4)), TypeError, "dtype"),
    (lambda: sdm.conv_forward(t(1, 2, 3, 4), t(2, 4, 4, dtype=torch.bfloat16)), TypeError, "dtype"),
    (lambda: sdm.conv_forward(t(1, 2, 3, 4), t(2, 4, 4), state=t(1, 2, 4, 4)), ValueError, "state"),
    (lambda: sdm.conv_forward(t(1, 2, 3, 4), t(2, 4, 4), lengths=t(1)), TypeError, "lengths"),
    (lambda: sdm.conv_forward(t(1, 2, 3, 4), t(2, 4, 4)), ValueError, "CUDA"),
    (lambda: sdm.conv_backward(t(1, 2, 3, 4), t(2, 4, 4), t(1, 2, 4, 4)), ValueError, "dy has shape"),
    (lambda: sdm.conv_backward(t(1, 2, 3, 4), t(2, 4, 4), t(1, 2, 3, 4), dstate=t(1, 2, 3, 4).bfloat16()), TypeError, "dstate"),
    (lambda: sdm.ssm_forward(t(1, 2, 5, 16), t(1, 2, 4), t(2), t(1, 1, 5, 16), t(1, 1, 5, 16), t(1, 2, 16, 16)), ValueError, "dt"),
    (lambda: sdm.ssm_forward(t(1, 2, 5, 16), t(1, 2, 5), t(2), t(1, 1, 5, 16), t(1, 1, 5, 32), t(1, 2, 16, 16)), ValueError, "Cm"),
    (lambda: sdm.ssm_forward(t(1, 2, 5, 16), t(1, 2, 5), t(2), t(1, 1, 5, 16), t(1, 1, 5, 16), t(1, 2, 16, 16).double()), TypeError, "S has dtype"),
    (lambda: sdm.ssm_step(t(1, 2, 5, 16), t(1, 2, 5), t(2), t(1, 1, 5, 16), t(1, 1, 5, 16), t(1, 2, 16, 16), t(3)), ValueError, "D has shape"),
    (lambda: sdm.ssm_backward(t(1, 2, 5, 16), t(1, 2, 5), t(2), t(1, 1, 5, 16), t(1, 1, 5, 16), None, t(1, 2, 5, 16)), ValueError, "CUDA"),
    (lambda: sdm.block_pool(t(1, 2, 64, 32), first=1), ValueError, "first needs"),
    (lambda: sdm.block_pool(t(1, 2, 200, 32), t(1, 2, 2, 32)), ValueError, "kc must be"),
    (lambda: sdm.block_select(t(1, 4, 8, 32), t(1, 2, 3, 64), n_sel=2), ValueError, "kc has shape"),
    (lambda: sdm.block_forward(t(1, 4, 8, 32), t(1, 2, 8, 32), t(1, 2, 9, 32), t(1, 2, 8, 2).int()), ValueError, "v has shape"),
    (lambda: sdm.block_forward(t(1, 4, 8, 32), t(1, 2, 8, 32), t(1, 2, 8, 32), t(1, 2, 8, 2)), TypeError, "idx"),
    (lambda: sdm.block_forward(t(1, 4, 8, 32), t(1, 2, 8, 32), t(1, 2, 8, 32), t(1, 2, 7, 2).int()), ValueError, "idx"),
    (lambda: sdm.block_backward(t(1, 4, 8, 32), t(1, 2, 8, 32), t(1, 2, 8, 32), t(1, 2, 8, 2).int(), t(1, 4, 8, 32), t(1, 4, 7), t(1, 4, 8, 32)), ValueError, "lse"),
])
def test_binding_refuses(lib, call, error, text):
    with pytest.raises(error, match=text):
        call()
