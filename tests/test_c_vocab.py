"""The embedding and the vocabulary loss used from plain C99, without the Python
binding: tests/c_abi/df11_vocab_check.c, as test_c_abi.py does for the codec."""

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "c_abi", "df11_vocab_check.c")
LIBDIR = os.path.join(ROOT, "entropy_decoding_amd")
ROCM = "/opt/rocm"


def _build(tmp_path, gpu: bool):
    exe = str(tmp_path / "df11_vocab_check")
    # c99: products and sums are not contracted
    cmd = ["gcc", "-std=c99", "-O1", "-Wall", "-Wextra", "-I", os.path.join(ROOT, "include"), SRC,
           "-o", exe, "-L", LIBDIR, "-ldf11", "-lm", f"-Wl,-rpath,{LIBDIR}"]
    if gpu:
        cmd += ["-DDF11_C_CHECK_GPU", "-D__HIP_PLATFORM_AMD__", "-I", f"{ROCM}/include",
                "-L", f"{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib"]
    else:
        cmd.insert(1, "-Werror")
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    return exe


def test_c_program_sizes_and_refusals(tmp_path):
    r = subprocess.run([_build(tmp_path, gpu=False)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    assert "sizes and refusals" in r.stdout


@pytest.mark.gpu
def test_c_program_runs_the_operators(tmp_path):
    exe = _build(tmp_path, gpu=True)
    print("[gpu] C program: df11_embedding, df11_embedding_gradient, df11_vocab_loss, df11_vocab_loss_gradient",
          flush=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.count("bit-exact") == 1 and "both gradients" in r.stdout
