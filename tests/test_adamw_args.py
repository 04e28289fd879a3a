"""Arguments that the optimiser step, the gradient norm and the reader of
8-bit states refuse.  Every call here is refused before anything is launched
(the pointers are made up)."""

import ctypes
import math
import os
import subprocess

import pytest

import entropy_decoding_amd as ed

L = ed.LIB
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def tensor(**change):
    a = (ed.df11_adamw_tensor * 1)()
    t = a[0]
    t.w, t.g, t.m, t.v, t.m_scale, t.v_scale = (4096 * (k + 1) for k in range(6))
    t.numel, t.lr_scale, t.weight_decay = 100, 1.0, 0.0
    for k, v in change.items():
        setattr(t, k, v)
    return a


def config(**change):
    c = ed.df11_adamw_config(1e-3, 0.9, 0.999, 1e-8, 1, 1, 1, 32, 0)
    for k, v in change.items():
        setattr(c, k, v)
    return c


def step(c, t, n=1):
    return L.df11_adamw_step(None if c is None else ctypes.byref(c), t, n, None)


@pytest.mark.parametrize("change", [
    {"w_type": 2}, {"w_type": 3}, {"g_type": 2}, {"state_bits": 16}, {"state_bits": 0},
    {"reserved": 1}, {"lr": math.nan}, {"lr": math.inf}, {"lr": -1e-3}, {"beta1": 1.0},
    {"beta1": -0.1}, {"beta2": 1.0}, {"beta2": math.nan}, {"eps": 0.0}, {"eps": -1.0},
    {"eps": math.inf}, {"eps": 1e-60}, {"step": 0}, {"d_lr": 2}, {"d_step": 4},
    {"d_grad_factor": 1}])
def test_step_refuses_numbers(change):
    assert step(config(**change), tensor()) == ed.DF11_E_INVALID


@pytest.mark.parametrize("bits,change", [
    (32, {"w": 0}), (32, {"g": 0}), (32, {"m": 0}), (32, {"v": 0}), (8, {"m_scale": 0}),
    (8, {"v_scale": 0}), (32, {"w": 4097}), (32, {"g": 4097}), (32, {"m": 4098}), (32, {"v": 4098}),
    (8, {"m_scale": 4098}), (32, {"master": 4098}), (32, {"counts": 4100}),
    (32, {"numel": 2 ** 40 + 1}), (32, {"lr_scale": -1.0}), (32, {"lr_scale": math.nan}),
    (32, {"weight_decay": math.inf}), (32, {"weight_decay": -0.1})])
def test_step_refuses_tensors(bits, change):
    assert step(config(state_bits=bits), tensor(**change)) == ed.DF11_E_INVALID


def test_step_refuses_masters_and_counts_of_float32_weights():
    for change in ({"master": 8192}, {"counts": 8192}):
        assert step(config(w_type=0), tensor(**change)) == ed.DF11_E_INVALID


def test_step_refuses_masters_for_some_tensors_only():
    t = (ed.df11_adamw_tensor * 2)(tensor(master=8192)[0], tensor()[0])
    assert step(config(), t, 2) == ed.DF11_E_INVALID


def test_step_refuses_null():
    assert step(None, tensor()) == ed.DF11_E_INVALID
    assert step(config(), None) == ed.DF11_E_INVALID


def test_step_of_nothing_launches_nothing():
    assert step(config(), None, 0) == ed.DF11_OK
    assert step(config(), tensor(numel=0, w=0, g=0, m=0, v=0)) == ed.DF11_OK


def counted(c, t, count=4096, n=1):
    return L.df11_adamw_step_counted(None if c is None else ctypes.byref(c), t, n, count, None)


def test_counted_step_refuses():
    """What the step refuses, and counters that are null, misaligned or beside
    the step's number on the device."""
    assert counted(config(), tensor(), None) == ed.DF11_E_INVALID
    assert counted(config(), tensor(), 4100) == ed.DF11_E_INVALID
    assert counted(config(d_step=8192), tensor(), 4096) == ed.DF11_E_INVALID
    assert counted(None, tensor()) == ed.DF11_E_INVALID
    assert counted(config(), None) == ed.DF11_E_INVALID
    assert counted(config(step=0), tensor()) == ed.DF11_E_INVALID
    assert counted(config(), tensor(w=4097)) == ed.DF11_E_INVALID
    assert counted(config(), None, n=0) == ed.DF11_OK


@pytest.mark.parametrize("kind,change", [
    (2, {}), (3, {}), (0, {"m": 0}), (0, {"v": 0}), (0, {"m_scale": 0}), (0, {"v_scale": 4097}),
    (0, {"numel": 2 ** 41})])
def test_values_refuse(kind, change):
    out = (ctypes.c_void_p * 1)(4096)
    assert L.df11_adamw_values(tensor(**change), 1, kind, out, out, None) == ed.DF11_E_INVALID


def test_values_refuse_outputs():
    for bad in (0, 4098):
        out = (ctypes.c_void_p * 1)(bad)
        assert L.df11_adamw_values(tensor(), 1, 0, out, None, None) == ed.DF11_E_INVALID
        assert L.df11_adamw_values(tensor(), 1, 0, None, out, None) == ed.DF11_E_INVALID


def norm(t, n=1, kind=1, most=1.0, out=4096, scratch=4096, nbytes=1 << 20):
    return L.df11_grad_norm(kind, t, n, most, out, scratch, nbytes, None)


def test_norm_refuses():
    ok = tensor()
    for change in ({"kind": 2}, {"most": 0.0}, {"most": -1.0}, {"most": math.nan}, {"out": 0},
                   {"out": 4098}, {"scratch": 0}, {"scratch": 4100}, {"nbytes": 7}):
        assert norm(ok, **change) == ed.DF11_E_INVALID
    assert norm(None) == ed.DF11_E_INVALID
    assert norm(tensor(g=0)) == ed.DF11_E_INVALID
    assert norm(tensor(g=4097)) == ed.DF11_E_INVALID
    assert norm(tensor(numel=2 ** 41)) == ed.DF11_E_INVALID


def test_norm_scratch_covers_every_chunk():
    for numel in (0, 1, 1024, 1025, 10 ** 9):
        assert L.df11_grad_norm_scratch_bytes(tensor(numel=numel), 1) >= 8 * max(1, numel // 65536)


def test_long_tensors_have_few_enough_chunks():
    """A workgroup of 256 threads a chunk, less than 2^32 threads a grid."""
    for numel in (2 ** 36, 2 ** 39 + 1, 2 ** 40):
        parts = L.df11_grad_norm_scratch_bytes(tensor(numel=numel), 1) // 8
        assert numel / 2 ** 30 <= parts <= 2 ** 23


def test_structs_match_the_header(tmp_path):
    names = [f for f, _ in ed.df11_adamw_tensor._fields_], [f for f, _ in ed.df11_adamw_config._fields_]
    body = "".join(f'printf("%zu ", offsetof({s}, {f}));' for s, fs in
                   (("df11_adamw_tensor", names[0]), ("df11_adamw_config", names[1])) for f in fs)
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "df11.h"\nint main(void) {' + body +
                   'printf("%zu %zu %d", sizeof(df11_adamw_tensor), sizeof(df11_adamw_config), DF11_ADAMW_BLOCK);'
                   "return 0;}")
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "s")])
    got = [int(x) for x in subprocess.check_output([str(tmp_path / "s")], text=True).split()]
    assert got == ([getattr(ed.df11_adamw_tensor, f).offset for f in names[0]] +
                   [getattr(ed.df11_adamw_config, f).offset for f in names[1]] +
                   [ctypes.sizeof(ed.df11_adamw_tensor), ctypes.sizeof(ed.df11_adamw_config),
                    ed.DF11_ADAMW_BLOCK])
