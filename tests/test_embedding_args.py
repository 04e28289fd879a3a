"""Arguments that the embedding lookup and its gradient refuse.  Every call here
is refused, or has nothing to do, before anything is launched (the pointers are
made up)."""

import ctypes
import os
import subprocess

import pytest

import entropy_decoding_amd as ed

L = ed.LIB
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BIG = 1 << 40


def lookup(**change):
    a = dict(table=4096, tokens=8192, out=16384, table_stride=40, out_stride=48, rows=7, n=3, cols=40,
             table_type=1, out_type=0, token_bits=64, scale=1.0)
    a.update(change)
    return L.df11_embedding(ctypes.byref(ed.df11_embedding_lookup(**a)), None)


def gradient(scratch=1 << 20, nbytes=None, **change):
    a = dict(tokens=8192, dy=4096, dw=16384, dy_stride=40, dw_stride=48, rows=7, n=3, padding=-1, cols=40,
             dy_type=1, dw_type=0, token_bits=64, accumulate=0, scale=1.0)
    a.update(change)
    if nbytes is None:
        nbytes = L.df11_embedding_gradient_scratch_bytes(a["n"], a["rows"], a["cols"])
    return L.df11_embedding_gradient(ctypes.byref(ed.df11_embedding_grad(**a)), scratch, nbytes, None)


@pytest.mark.parametrize("change", [
    {"table": 0}, {"table": 4097}, {"tokens": 0}, {"tokens": 8196}, {"out": 0}, {"out": 16386},
    {"out_stride": 39}, {"out_stride": BIG}, {"table_stride": BIG}, {"table_type": 3}, {"out_type": 3},
    {"token_bits": 16}, {"token_bits": 0}, {"token_bits": 32, "tokens": 8194},
    {"rows": (1 << 24) + 1}, {"n": (1 << 24) + 1}, {"cols": (1 << 20) + 1, "out_stride": 1 << 21},
    {"n": 1 << 24, "cols": 8193, "out_stride": 8193}])  # 2^24 x 5 waves
def test_lookup_refuses(change):
    assert lookup(**change) == ed.DF11_E_INVALID


def test_lookup_of_nothing():
    assert L.df11_embedding(None, None) == ed.DF11_E_INVALID
    assert lookup(n=0, tokens=0, out=0) == ed.DF11_OK
    assert lookup(cols=0, table=0, out=0) == ed.DF11_OK


@pytest.mark.parametrize("change", [
    {"tokens": 0}, {"tokens": 8196}, {"dy": 0}, {"dy": 4097}, {"dw": 0}, {"dw": 16386}, {"dw_stride": 39},
    {"dw_stride": BIG}, {"dy_stride": BIG}, {"dy_type": 3}, {"dw_type": 3}, {"token_bits": 8},
    {"accumulate": 2}, {"rows": (1 << 24) + 1}, {"n": (1 << 24) + 1, "nbytes": 1 << 40},
    {"cols": (1 << 20) + 1, "dw_stride": 1 << 21, "nbytes": 1 << 40},
    {"n": 3000, "scratch": 0}, {"n": 3000, "scratch": (1 << 20) + 64}, {"n": 3000, "nbytes": 100}])
def test_gradient_refuses(change):
    assert gradient(**change) == ed.DF11_E_INVALID


def test_gradient_of_nothing():
    assert L.df11_embedding_gradient(None, 1 << 20, 1 << 20, None) == ed.DF11_E_INVALID
    assert gradient(rows=0, dw=0) == ed.DF11_OK
    assert gradient(cols=0, dw=0, dy=0) == ed.DF11_OK
    assert gradient(n=0, tokens=0, dy=0, accumulate=1) == ed.DF11_OK


def test_scratch_bytes():
    f = L.df11_embedding_gradient_scratch_bytes
    assert f((1 << 24) + 1, 8, 8) == f(3000, (1 << 24) + 1, 8) == f(3000, 8, (1 << 20) + 1) == 0
    assert f(2048, 16_383, 4096) == 0 < f(2049, 16_383, 4096)
    assert f(1, 16_384, 4096) > 0  # 2^26 elements
    assert gradient(n=0, tokens=0, dy=0, rows=1 << 24, accumulate=1, scratch=0, nbytes=0) == ed.DF11_OK
    assert f(3000, 8, 8) < f(100_000, 8, 8) < f(100_000, 1 << 20, 8) < f(100_000, 1 << 20, 80)
    assert f(8, 1 << 24, 1 << 20) > 0  # more workgroups than a grid holds: three launches


def test_struct_layouts(tmp_path):
    src = '''
#include <stdio.h>
#include <stddef.h>
#include "df11.h"
int main(void) {
  printf("%zu %zu %zu %zu\\n", sizeof(df11_embedding_lookup), offsetof(df11_embedding_lookup, n),
         offsetof(df11_embedding_lookup, token_bits), offsetof(df11_embedding_lookup, scale));
  printf("%zu %zu %zu %zu\\n", sizeof(df11_embedding_grad), offsetof(df11_embedding_grad, padding),
         offsetof(df11_embedding_grad, token_bits), offsetof(df11_embedding_grad, scale));
  printf("%u %u %u\\n", DF11_EMBEDDING_MAX_TOKENS, DF11_EMBEDDING_MAX_ROWS, DF11_EMBEDDING_MAX_COLS);
  return 0;
}
'''
    (tmp_path / "s.c").write_text(src)
    exe = str(tmp_path / "s")
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(tmp_path / "s.c"), "-o", exe])
    got = [list(map(int, line.split())) for line in subprocess.check_output([exe], text=True).splitlines()]
    a, g = ed.df11_embedding_lookup, ed.df11_embedding_grad
    assert got == [[ctypes.sizeof(a), a.n.offset, a.token_bits.offset, a.scale.offset],
                   [ctypes.sizeof(g), g.padding.offset, g.token_bits.offset, g.scale.offset],
                   [ed.DF11_EMBEDDING_MAX_TOKENS, ed.DF11_EMBEDDING_MAX_ROWS, ed.DF11_EMBEDDING_MAX_COLS]]


torch = pytest.importorskip("torch")


def test_binding_refuses():
    host = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device"):
        ed.Embedding(host)
    with pytest.raises(ValueError):
        ed.embedding_gradient(torch.zeros(4, dtype=torch.int64), host, 7)
