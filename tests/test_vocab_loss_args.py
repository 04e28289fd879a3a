"""Arguments that the cross entropy under an output head refuses.  Every call here
is refused, or has nothing to do, before anything is launched (the pointers are
made up)."""

import ctypes
import os
import subprocess

import pytest

import entropy_decoding_amd as ed

L = ed.LIB
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PIECE = dict(x=4096, targets=8192, w=16384, x_stride=64, w_stride=72, ignored=-100, n=3, cols=64, vocab=100, first=40,
             rows=60, target_bits=64, begin=1, end=1)
BAD_PIECES = [
    {"x": 0}, {"x": 4104}, {"targets": 0}, {"targets": 8196}, {"w": 0}, {"w": 16392}, {"x_stride": 60},
    {"x_stride": 56}, {"w_stride": 68}, {"w_stride": 56}, {"x_stride": (1 << 21) + 8},
    {"w_stride": (1 << 21) + 8}, {"cols": 60}, {"cols": (1 << 20) + 8, "x_stride": 1 << 21, "w_stride": 1 << 21},
    {"vocab": 0, "first": 0, "rows": 0}, {"vocab": 99}, {"first": 41}, {"first": 101, "rows": 0},
    {"vocab": (1 << 24) + 1}, {"target_bits": 16}, {"target_bits": 32, "targets": 8194},
    {"n": (1 << 20) + 1}, {"begin": 2}, {"end": 2}]


def loss(losses=32768, lse=65536, scratch=1 << 20, nbytes=None, sizes=None, **change):
    p = ed.df11_vocab_piece(**{**PIECE, **change})
    z = ed.df11_vocab_sizes(p.n, p.cols, p.rows, 0, 0)
    for k, v in (sizes or {}).items():
        setattr(z, k, v)
    if nbytes is None:
        nbytes = L.df11_vocab_loss_scratch_bytes(z)
    return L.df11_vocab_loss(p, losses, lse, z, scratch, nbytes, None)


def gradient(scratch=1 << 20, nbytes=None, sizes=None, grad=None, **change):
    p = ed.df11_vocab_piece(**{**PIECE, **change})
    g = dict(lse=65536, dx=1 << 17, dw=1 << 18, dx_stride=64, dw_stride=64, dx_type=1, dw_type=1)
    g.update(grad or {})
    z = ed.df11_vocab_sizes(p.n, p.cols, p.rows, 1, 0)
    for k, v in (sizes or {}).items():
        setattr(z, k, v)
    if nbytes is None:
        nbytes = L.df11_vocab_loss_gradient_scratch_bytes(z)
    return L.df11_vocab_loss_gradient(p, ed.df11_vocab_grad(**g), z, scratch, nbytes, None)


@pytest.mark.parametrize("change", BAD_PIECES + [
    {"losses": 0}, {"losses": 32770}, {"lse": 0}, {"lse": 65537}, {"scratch": 0}, {"scratch": (1 << 20) + 128},
    {"nbytes": 100}, {"sizes": {"n": 4}}, {"sizes": {"cols": 72}}, {"sizes": {"rows": 59}}])
def test_loss_refuses(change):
    assert loss(**change) == ed.DF11_E_INVALID


@pytest.mark.parametrize("change", BAD_PIECES + [
    {"scratch": 0}, {"scratch": (1 << 20) + 128}, {"nbytes": 100},
    {"sizes": {"n": 4}}, {"sizes": {"cols": 72}}, {"sizes": {"rows": 59}}, {"sizes": {"rows": (1 << 24) + 1}}] + [
    {"grad": g} for g in (
        {"lse": 0}, {"lse": 65538}, {"losses": 4098}, {"dx": 0}, {"dx": (1 << 17) + 1}, {"dx_stride": 63}, {"dx_stride": 1 << 40},
        {"dw": (1 << 18) + 1}, {"dw_stride": 63}, {"dw_stride": 1 << 40}, {"dx_type": 2}, {"dw_type": 2},
        {"dx_type": 0}, {"dw_type": 0},  # float32 without sizes for two terms
        {"accumulate": 2}, {"loss_grad": 4098, "loss_grads": 1}, {"loss_grad": 4096, "loss_grads": 2},
        {"lse_grad": 4098, "lse_grads": 1}, {"lse_grad": 4096, "lse_grads": 0})])
def test_gradient_refuses(change):
    assert gradient(**change) == ed.DF11_E_INVALID


def test_nothing_to_do():
    assert L.df11_vocab_loss(None, 4096, 4096, None, 1 << 20, 1 << 20, None) == ed.DF11_E_INVALID
    assert loss(n=0, x=0, targets=0) == ed.DF11_OK
    assert L.df11_vocab_loss_gradient(None, None, None, 1 << 20, 1 << 20, None) == ed.DF11_E_INVALID
    assert gradient(cols=0, x=0, w=0) == ed.DF11_OK


def test_more_than_a_grid_holds_is_refused():
    n, rows = 1 << 20, 1 << 24
    z = ed.df11_vocab_sizes(n, 8, rows, 0, 0)
    nbytes = L.df11_vocab_loss_scratch_bytes(z)
    assert nbytes > n * rows // 256 * 8
    assert loss(n=n, cols=8, x_stride=8, w_stride=8, vocab=rows, first=0, rows=rows,
                nbytes=nbytes) == ed.DF11_E_INVALID


def test_scratch_bytes():
    z = ed.df11_vocab_sizes
    f, g = L.df11_vocab_loss_scratch_bytes, L.df11_vocab_loss_gradient_scratch_bytes
    for bad in (z((1 << 20) + 1, 8, 8, 0, 0), z(8, 12, 8, 0, 0), z(8, (1 << 20) + 8, 8, 0, 0), z(8, 8, (1 << 24) + 1, 0, 0)):
        assert f(bad) == g(bad) == 0
    assert 0 < f(z(1, 64, 100, 0, 0)) <= f(z(100, 64, 100, 0, 0)) <= f(z(100, 64, 9000, 0, 0))
    assert 0 < g(z(100, 64, 9000, 0, 0)) < g(z(100, 64, 9000, 1, 0)) < g(z(100, 64, 9000, 1, 1))
    assert g(z(100, 64, 0, 1, 1)) < 2 ** 18  # no rows: room for one chunk of 256
    # g takes 2^29 elements at most, or 256 rows: not the logits' memory
    assert g(z(8192, 4096, 1 << 24, 1, 0)) < 2 ** 30 + 8192 * 4096 * 4 * 2 + 2 ** 20
    assert g(z(1 << 20, 8, 1 << 24, 0, 0)) < 2 ** 30 + 2 ** 20 * 200


def test_struct_layouts(tmp_path):
    src = '''
#include <stdio.h>
#include <stddef.h>
#include "df11.h"
int main(void) {
  printf("%zu %zu %zu %zu\\n", sizeof(df11_vocab_piece), offsetof(df11_vocab_piece, ignored),
         offsetof(df11_vocab_piece, first), offsetof(df11_vocab_piece, end));
  printf("%zu %zu\\n", sizeof(df11_vocab_sizes), offsetof(df11_vocab_sizes, two_terms));
  printf("%zu %zu %zu %zu\\n", sizeof(df11_vocab_grad), offsetof(df11_vocab_grad, dw_stride),
         offsetof(df11_vocab_grad, accumulate), offsetof(df11_vocab_grad, loss_grad_all));
  printf("%u %u %u %u\\n", DF11_VOCAB_MAX_TOKENS, DF11_VOCAB_MAX_ROWS, DF11_VOCAB_MAX_COLS, DF11_VOCAB_MAX_STRIDE);
  return 0;
}
'''
    (tmp_path / "s.c").write_text(src)
    exe = str(tmp_path / "s")
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(tmp_path / "s.c"), "-o", exe])
    got = [list(map(int, line.split())) for line in subprocess.check_output([exe], text=True).splitlines()]
    p, z, g = ed.df11_vocab_piece, ed.df11_vocab_sizes, ed.df11_vocab_grad
    assert got == [[ctypes.sizeof(p), p.ignored.offset, p.first.offset, p.end.offset],
                   [ctypes.sizeof(z), z.two_terms.offset],
                   [ctypes.sizeof(g), g.dw_stride.offset, g.accumulate.offset, g.loss_grad_all.offset],
                   [ed.DF11_VOCAB_MAX_TOKENS, ed.DF11_VOCAB_MAX_ROWS, ed.DF11_VOCAB_MAX_COLS,
                    ed.DF11_VOCAB_MAX_STRIDE]]


torch = pytest.importorskip("torch")


def test_binding_refuses():
    host = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        ed.VocabLoss([host])
    with pytest.raises(ValueError, match="pieces"):
        ed.VocabLoss([])
