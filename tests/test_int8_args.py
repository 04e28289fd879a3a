"""Arguments that the int8 quantiser and product refuse.  Every call here is
refused, or has nothing to do, before anything is launched (the pointers are
made up)."""

import ctypes
import os
import subprocess

import pytest

import entropy_decoding_amd as ed

L = ed.LIB
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def rows(**change):
    a = (ed.df11_int8_rows * 1)()
    r = a[0]
    r.src, r.codes, r.scales, r.src_stride, r.code_stride, r.rows, r.cols = 4096, 8192, 16384, 40, 48, 3, 40
    for k, v in change.items():
        setattr(r, k, v)
    return a


def tensor(**change):
    a = (ed.df11_int8_tensor * 1)()
    t = a[0]
    t.w, t.w_scale, t.x, t.x_scale, t.y = 4096, 8192, 16384, 32768, 65536
    t.w_stride, t.x_stride, t.y_stride, t.rows, t.cols = 48, 64, 20, 20, 40
    for k, v in change.items():
        setattr(t, k, v)
    return a


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("change", [
    {"src": 0}, {"src": 4097}, {"codes": 0}, {"codes": 8200}, {"scales": 0}, {"scales": 16386},
    {"src_stride": 39}, {"src_stride": 1 << 41}, {"code_stride": 40}, {"code_stride": 32},
    {"code_stride": (1 << 22) + 16}, {"cols": 131072}])
def test_quantiser_refuses(kind, change):
    assert L.df11_quantize_int8(kind, rows(**change), 1, None) == ed.DF11_E_INVALID


def test_quantiser_refuses_lists():
    assert L.df11_quantize_int8(3, rows(), 1, None) == ed.DF11_E_INVALID
    assert L.df11_quantize_int8(1, None, 1, None) == ed.DF11_E_INVALID
    many = (ed.df11_int8_rows * 17)(*[rows()[0]] * 17)
    assert L.df11_quantize_int8(1, many, 17, None) == ed.DF11_E_INVALID
    many = (ed.df11_int8_rows * 2)(*[rows(rows=0x7FFFFFFF, code_stride=48)[0]] * 2)
    assert L.df11_quantize_int8(1, many, 2, None) == ed.DF11_E_INVALID


@pytest.mark.parametrize("kind", [0, 1, 2])
def test_more_rows_than_a_grid_holds_are_refused(kind):
    """One workgroup of 256 threads a row: 2^24 rows would be 2^32 threads."""
    assert L.df11_quantize_int8(kind, rows(rows=1 << 24), 1, None) == ed.DF11_E_INVALID
    half = (ed.df11_int8_rows * 2)(*[rows(rows=1 << 23)[0]] * 2)
    assert L.df11_quantize_int8(kind, half, 2, None) == ed.DF11_E_INVALID


@pytest.mark.parametrize("kind", [0, 1, 2])
def test_more_tiles_than_a_grid_holds_are_refused(kind):
    """2^24 rows and 2^20 tokens are 2^28 tiles of 256 x 256, 512 threads each."""
    t = tensor(rows=1 << 24, y_stride=1 << 24)
    assert L.df11_gemm_int8(kind, t, 1, 1 << 20, None) == ed.DF11_E_INVALID
    many = (ed.df11_int8_tensor * 16)(*[t[0]] * 16)  # 2^24 workgroups of 16 rows
    nbytes = L.df11_linear_int8_scratch_bytes(many, 16, 1)
    assert linear(many, 16, kind, kind, 1, 4096, nbytes) == ed.DF11_E_INVALID


def test_quantiser_of_nothing():
    assert L.df11_quantize_int8(1, None, 0, None) == ed.DF11_OK
    assert L.df11_quantize_int8(1, rows(rows=0, src=0, codes=0, scales=0), 1, None) == ed.DF11_OK


@pytest.mark.parametrize("change", [
    {"w": 0}, {"w": 4104}, {"x": 0}, {"x": 16392}, {"w_scale": 0}, {"w_scale": 8194}, {"x_scale": 0},
    {"x_scale": 32769}, {"y": 0}, {"y": 65537}, {"w_stride": 40}, {"w_stride": 32}, {"x_stride": 40},
    {"x_stride": 32}, {"w_stride": (1 << 22) + 16}, {"x_stride": (1 << 22) + 16}, {"y_stride": 19},
    {"y_stride": 1 << 41}, {"cols": 131072}, {"rows": (1 << 24) + 1}])
@pytest.mark.parametrize("kind", [0, 1, 2])
def test_product_refuses(kind, change):
    assert L.df11_gemm_int8(kind, tensor(**change), 1, 5, None) == ed.DF11_E_INVALID


def test_product_refuses_lists():
    assert L.df11_gemm_int8(3, tensor(), 1, 5, None) == ed.DF11_E_INVALID
    assert L.df11_gemm_int8(0, tensor(y=65538), 1, 5, None) == ed.DF11_E_INVALID
    assert L.df11_gemm_int8(1, None, 1, 5, None) == ed.DF11_E_INVALID
    many = (ed.df11_int8_tensor * 17)(*[tensor()[0]] * 17)
    assert L.df11_gemm_int8(1, many, 17, 5, None) == ed.DF11_E_INVALID
    assert L.df11_gemm_int8(1, tensor(), 1, (1 << 20) + 1, None) == ed.DF11_E_INVALID


def test_product_of_nothing():
    assert L.df11_gemm_int8(1, None, 0, 5, None) == ed.DF11_OK
    assert L.df11_gemm_int8(1, tensor(w=0, x=0, y=0), 1, 0, None) == ed.DF11_OK
    assert L.df11_gemm_int8(1, tensor(rows=0, w=0, y=0), 1, 5, None) == ed.DF11_OK


def linear(t, n=1, x_kind=1, y_kind=1, tokens=5, scratch=4096, nbytes=1 << 20):
    return L.df11_linear_int8(x_kind, y_kind, t, n, tokens, scratch, nbytes, None)


@pytest.mark.parametrize("change", [
    {"w": 0}, {"w": 4104}, {"x": 0}, {"x": 16385}, {"w_scale": 0}, {"y": 0}, {"y": 65537},
    {"w_stride": 40}, {"x_stride": 39}, {"x_stride": 1 << 41}, {"y_stride": 19}, {"cols": 131072},
    {"rows": (1 << 24) + 1}])
def test_linear_refuses(change):
    assert linear(tensor(**change)) == ed.DF11_E_INVALID


def test_linear_refuses_scratch_and_types():
    need = L.df11_linear_int8_scratch_bytes(tensor(), 1, 5)
    assert need >= 5 * 48 + 5 * 4
    for change in ({"scratch": 0}, {"scratch": 4104}, {"nbytes": need - 1}, {"x_kind": 3},
                   {"y_kind": 3}, {"tokens": (1 << 20) + 1}):
        assert linear(tensor(), **change) == ed.DF11_E_INVALID
    assert linear(None) == ed.DF11_E_INVALID
    many = (ed.df11_int8_tensor * 17)(*[tensor()[0]] * 17)
    assert linear(many, 17) == ed.DF11_E_INVALID


@pytest.mark.parametrize("change", [
    {"w": 0}, {"x": 0}, {"x": 16385}, {"w_scale": 0}, {"y": 0}, {"y": 65537}, {"w_stride": 40},
    {"y_stride": 19}, {"cols": 131072}])
def test_linear_of_one_token_refuses(change):
    assert linear(tensor(**change), tokens=1) == ed.DF11_E_INVALID
    for bad in ({"x_kind": 3}, {"y_kind": 3}, {"scratch": 4104}):
        assert linear(tensor(), tokens=1, **bad) == ed.DF11_E_INVALID
    assert linear(tensor(x=16386), x_kind=0, tokens=1) == ed.DF11_E_INVALID


@pytest.mark.parametrize("cols,none", [(0, False), (1, True), (32768, True), (32769, False)])
def test_one_token_needs_no_scratch(cols, none):
    stride = max(16, (cols + 15) // 16 * 16)
    t = tensor(cols=cols, w_stride=stride, x_stride=stride)
    need = L.df11_linear_int8_scratch_bytes(t, 1, 1)
    assert (need == 0) == none
    assert L.df11_linear_int8_scratch_bytes(t, 1, 2) >= 2 * cols + 8
    if need:
        assert linear(t, tokens=1, scratch=0) == ed.DF11_E_INVALID
        assert linear(t, tokens=1, nbytes=need - 1) == ed.DF11_E_INVALID


def test_linear_of_nothing():
    assert linear(None, 0) == ed.DF11_OK
    assert linear(tensor(), tokens=0) == ed.DF11_OK


def test_structs_match_the_header(tmp_path):
    kinds = ("df11_int8_rows", "df11_int8_tensor")
    fields = {s: [f for f, _ in getattr(ed, s)._fields_] for s in kinds}
    body = "".join(f'printf("%zu ", offsetof({s}, {f}));' for s in kinds for f in fields[s])
    body += "".join(f'printf("%zu ", sizeof({s}));' for s in kinds)
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "df11.h"\nint main(void) {' + body +
                   'printf("%d %u %u", DF11_INT8_MAX_TENSORS, DF11_INT8_MAX_COLS, DF11_INT8_MAX_STRIDE);'
                   "return 0;}")
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "s")])
    got = [int(x) for x in subprocess.check_output([str(tmp_path / "s")], text=True).split()]
    assert got == ([getattr(getattr(ed, s), f).offset for s in kinds for f in fields[s]] +
                   [ctypes.sizeof(getattr(ed, s)) for s in kinds] +
                   [ed.DF11_INT8_MAX_TENSORS, ed.DF11_INT8_MAX_COLS, ed.DF11_INT8_MAX_STRIDE])
