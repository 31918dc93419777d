"""Refusals of the grouped products and the 8-bit row quantiser: synchronous
host validation through the C ABI and the binding (no GPU)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_moe_route_b200 import build
    build.build()
    from bit_quantized_moe_route_b200 import _lib
    return _lib.load_library()


FAKE, FAKE2 = 0x10000, 0x20000000


def _dims(**kw):
    from bit_quantized_moe_route_b200 import GmmDims
    d = dict(dtype=0, out_dtype=0, n_experts=4, rows=8, n_out=64, n_in=32, reserved=0)
    d.update(kw)
    return GmmDims(*[d[k] for k in ("dtype", "out_dtype", "n_experts", "rows", "n_out", "n_in", "reserved")])


def _mm(lib, d, ld_x=32, ld_y=64, off=FAKE, ws=FAKE, nbytes=1 << 30):
    return lib.moe_grouped_mm(None if d is None else ctypes.byref(d), FAKE, ld_x, FAKE, off, FAKE, ld_y, ws, nbytes,
                              None)


INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def test_dims(lib):
    assert _mm(lib, None) == INVALID
    for bad in (dict(n_experts=0), dict(n_experts=1025), dict(rows=-1), dict(rows=(1 << 30) + 1), dict(n_out=0),
                dict(n_in=0), dict(n_out=65537), dict(n_in=65537), dict(reserved=1)):
        assert _mm(lib, _dims(**bad), ld_x=1 << 20, ld_y=1 << 20) == INVALID, bad
        assert lib.moe_last_error_detail()
    for bad in (dict(dtype=2), dict(dtype=-1), dict(out_dtype=3), dict(out_dtype=1)):
        assert _mm(lib, _dims(**bad)) == UNSUPPORTED, bad
    assert _mm(lib, _dims(), ld_x=31) == INVALID and b"ld_x" in lib.moe_last_error_detail()
    assert _mm(lib, _dims(), ld_y=63) == INVALID and b"ld_y" in lib.moe_last_error_detail()
    assert _mm(lib, _dims(), off=None) == INVALID and b"expert_offsets" in lib.moe_last_error_detail()
    assert _mm(lib, _dims(rows=0)) == 0                      # nothing to do


def test_gradient_dims(lib):
    d = _dims()
    dx = lambda ld_dy, ld_dx: lib.moe_grouped_mm_dx(ctypes.byref(d), FAKE, ld_dy, FAKE, FAKE, FAKE, ld_dx, FAKE,
                                                    1 << 30, None)  # noqa: E731
    assert dx(63, 32) == INVALID and b"ld_dy" in lib.moe_last_error_detail()
    assert dx(64, 31) == INVALID and b"ld_dx" in lib.moe_last_error_detail()
    dw = lambda ld_dy, ld_x: lib.moe_grouped_mm_dw(ctypes.byref(d), FAKE, ld_dy, FAKE, ld_x, FAKE, FAKE, FAKE,
                                                   1 << 30, None)  # noqa: E731
    assert dw(63, 32) == INVALID and b"ld_dy" in lib.moe_last_error_detail()
    assert dw(64, 31) == INVALID and b"ld_x" in lib.moe_last_error_detail()


def test_workspace(lib):
    n = lib.moe_grouped_workspace_size()
    assert n == 40 << 20
    assert _mm(lib, _dims(), ws=None) == INVALID
    assert _mm(lib, _dims(), ws=FAKE + 16) == INVALID and b"aligned" in lib.moe_last_error_detail()
    assert _mm(lib, _dims(), nbytes=n - 1) == WORKSPACE


def test_fp8_dims(lib):
    def call(d, ld_x=32, ld_y=64, off=FAKE):
        return lib.moe_grouped_mm_fp8(ctypes.byref(d), FAKE, ld_x, FAKE, FAKE, FAKE, off, FAKE, ld_y, FAKE, 64, None)
    assert call(_dims()) == WORKSPACE
    for out in (0, 1, 2):
        assert call(_dims(dtype=9, out_dtype=out)) == WORKSPACE      # dtype is not read
    assert call(_dims(out_dtype=4)) == UNSUPPORTED
    assert call(_dims(), ld_x=31) == INVALID
    assert call(_dims(), off=None) == INVALID
    assert call(_dims(n_experts=1), off=None) == WORKSPACE


def test_quant_dims(lib):
    q = lambda dt, r, n, ld: lib.moe_quant_fp8(dt, r, n, FAKE, ld, FAKE, FAKE, None)  # noqa: E731
    assert q(2, 4, 64, 64) == UNSUPPORTED
    assert q(0, -1, 64, 64) == INVALID
    assert q(0, 4, 0, 64) == INVALID
    assert q(0, 4, 64, 63) == INVALID
    assert q(0, 4, 65537, 1 << 20) == INVALID
    assert q(0, 0, 64, 64) == 0


def test_binding_refuses(lib):
    import bit_quantized_moe_route_b200 as moe
    bf = torch.bfloat16
    x, w, y = torch.zeros(8, 32, dtype=bf), torch.zeros(4, 64, 32, dtype=bf), torch.zeros(8, 64, dtype=bf)
    off, ws = torch.zeros(5, dtype=torch.int32), torch.zeros(64, dtype=torch.uint8)

    def bad(match, call, *args):
        with pytest.raises(ValueError, match=match):
            call(*args)

    bad("CUDA", moe.grouped_mm, x, w, off, y, ws)
    bad("type", moe.grouped_mm, x.half(), w, off, y, ws)
    bad("operand type", moe.grouped_mm, x.float(), w.float(), off, y.float(), ws)
    bad("x must be", moe.grouped_mm, x[:, :31], w, off, y, ws)
    bad("y must be", moe.grouped_mm, x, w, off, y[:7], ws)
    bad("contiguous", moe.grouped_mm, torch.zeros(32, 8, dtype=bf).t(), w, off, y, ws)
    bad("overlap", moe.grouped_mm, torch.zeros(1, 32, dtype=bf).expand(8, 32), w, off, y, ws)
    bad("expert_offsets", moe.grouped_mm, x, w, off.long(), y, ws)
    bad("expert_offsets", moe.grouped_mm, x, w, off[:4], y, ws)
    bad("ws", moe.grouped_mm, x, w, off, y, ws.int())
    bad("output type", moe.grouped_mm, x, w, off, y.double(), ws)
    bad("dx must be", moe.grouped_mm_dx, y, w, off, x[:, :30], ws)
    bad("one type", moe.grouped_mm_dw, y, x.half(), off, w, ws)
    c, sx, sw = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(1, 8), torch.zeros(4, 1, 1)
    wc = torch.zeros(4, 64, 32, dtype=torch.uint8)
    bad("CUDA", moe.grouped_mm_fp8, c, sx, wc, sw, off, y, ws)
    bad("x_scales", moe.grouped_mm_fp8, c, sx.t(), wc, sw, off, y, ws)
    bad("w_scales", moe.grouped_mm_fp8, c, sx, wc, sw[:3], off, y, ws)
    bad("e4m3", moe.grouped_mm_fp8, x, sx, wc, sw, off, y, ws)
    bad("CUDA", moe.quant_fp8, x, c, sx)
    bad("codes", moe.quant_fp8, x, c[:7], sx)
    bad("scales", moe.quant_fp8, x, c, sx.t())
    bad("type", moe.quant_fp8, x.float(), c, sx)


@pytest.mark.parametrize("shape", [(), (64,), (2, 4, 32), (0,)])
def test_binding_refuses_what_is_no_matrix(lib, shape):
    import bit_quantized_moe_route_b200 as moe
    bf = torch.bfloat16
    x, w, off, ws = torch.zeros(shape, dtype=bf), torch.zeros(4, 64, 32, dtype=bf), torch.zeros(5, dtype=torch.int32), \
        torch.zeros(64, dtype=torch.uint8)
    y, codes = torch.zeros(8, 64, dtype=bf), torch.zeros(8, 32, dtype=torch.uint8)
    sx, sw, wc = torch.zeros(1, 8), torch.zeros(4, 1, 1), torch.zeros(4, 64, 32, dtype=torch.uint8)
    for call, args in ((moe.grouped_mm, (x, w, off, y, ws)), (moe.grouped_mm, (y[:, :32], w, off, x, ws)),
                       (moe.grouped_mm_dx, (x, w, off, y[:, :32], ws)), (moe.grouped_mm_dx, (y, w, off, x, ws)),
                       (moe.grouped_mm_dw, (x, y[:, :32], off, w, ws)), (moe.grouped_mm_dw, (y, x, off, w, ws)),
                       (moe.grouped_mm_dw, (y, y[:, :32], off, x, ws)), (moe.grouped_mm_fp8, (x.byte(), sx, wc, sw, off, y, ws)),
                       (moe.grouped_mm_fp8, (codes, sx, wc, sw, off, x, ws)), (moe.quant_fp8, (x, codes, sx)),
                       (moe.grouped_mm, (y[:, :32], x, off, y, ws))):
        if len(shape) == 3 and any(a is x for a in args[1:4]) and call is not moe.grouped_mm_fp8:
            continue                                              # a stack of matrices where one is taken
        with pytest.raises(ValueError, match="must be"):
            call(*args)
