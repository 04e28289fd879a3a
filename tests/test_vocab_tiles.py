"""What the compiler says of the vocabulary loss's tiles, in the built library: as
many workgroups fit a compute unit as their choice counts on, and no register
goes to memory."""

import math
import random
import re
import struct
import subprocess

import pytest

import entropy_decoding_amd as ed
import vocab_shapes
import vocab_tiles

READELF = "/opt/rocm/llvm/bin/llvm-readelf"
# (t, r): threads, workgroups of a compute unit
TILES = {(32, 64): (128, 2), (64, 64): (256, 2), (64, 128): (256, 2), (128, 128): (512, 1), (256, 128): (512, 1),
         (256, 256): (512, 1)}
KINDS = ["logits", "g", "dx", "dw", "dw past the caches"]


def kernels(tmp_path):
    """The metadata of the library's GPU kernels, by name."""
    with open(ed.LIB_PATH, "rb") as f:
        held = f.read()
    found, at = {}, -1
    while (at := held.find(b"\x7fELF", at + 1)) >= 0:
        if struct.unpack_from("<H", held, at + 18)[0] != 224:  # the GPU's
            continue
        (tmp_path / "gpu").write_bytes(held[at:])
        notes = subprocess.run([READELF, "--notes", str(tmp_path / "gpu")], capture_output=True, text=True).stdout
        for part in notes.split("- .agpr_count:")[1:]:
            values = dict(re.findall(r"^ +\.(\w+): +(\S+)$", "    .agpr_count: " + part, re.M))
            found[values["name"]] = values
    return found


def test_workgroups_of_a_compute_unit(tmp_path):
    seen = set()
    for name, v in kernels(tmp_path).items():
        m = re.search(r"5tilesI\w+?Li(\d)ELi(\d+)ELi(\d+)ELi", name)
        if not m:
            continue
        kind, shape = KINDS[int(m[1])], (int(m[2]), int(m[3]))
        threads, held = TILES[shape]
        seen.add((kind, shape))
        assert int(v["max_flat_workgroup_size"]) == threads
        assert held * int(v["group_segment_fixed_size"]) <= 160 * 1024, (kind, shape)
        # 512 registers a lane for a SIMD's waves, in groups of 8
        waves = held * threads // 64 / 4
        assert waves * -(-int(v["vgpr_count"]) // 8) * 8 <= 512, (kind, shape)
        assert int(v["vgpr_spill_count"]) == int(v["sgpr_spill_count"]) == 0, (kind, shape)
        assert int(v["private_segment_fixed_size"]) == 0, (kind, shape)
    assert seen == {(k, s) for k in KINDS for s in TILES}


def test_the_choice_of_tiles_is_the_librarys():
    """As far as the scratch tells it: a tile's rows, g's chunk and dx's parts."""
    rng = random.Random(1)

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    assert [tuple(map(int, t[:4])) for t in vocab_tiles.TILES] == [(*s, *v) for s, v in TILES.items()]
    for _ in range(4000):
        n, rows, cols = log(1, 1 << 20), log(1, 1 << 24), 8 * log(1, 1 << 17)
        z = ed.df11_vocab_sizes(n, cols, rows, rng.randint(0, 1), rng.randint(0, 1))
        assert ed.LIB.df11_vocab_loss_scratch_bytes(z) == vocab_tiles.loss_bytes(n, rows, cols)
        assert (ed.LIB.df11_vocab_loss_gradient_scratch_bytes(z) ==
                vocab_tiles.gradient_bytes(n, rows, cols, z.dx, z.two_terms))


def test_the_gpu_tests_reach_every_form():
    """All tiles of all products, and each of the logits at 16 stages and more.  Not among
    them: dw past the caches in tiles that only shapes of more than 2^28 elements
    of g or w take."""
    products = ["logits", "g", "dx", "dx in parts", *(f"dw {t}{a}" for t in ("bfloat16", "float32")
                                                      for a in ("", " added"))]
    want = {(p, k) for p in products for k in range(6)}
    want |= {("dw bfloat16 past", k) for k in (3, 4, 5)} | {("dw float32 added past", k) for k in (3, 4, 5)}
    want |= {("dw float32 past", k) for k in (1, 2, 4, 5)}
    seen, deep = set(), set()
    for n, rows, cols, dx, dw, add in vocab_shapes.SHAPES + vocab_shapes.PAST:
        found = vocab_tiles.forms(n, rows, cols, dw, add)
        seen |= found | vocab_tiles.forms(n, rows, cols, dw, add, on_half_lines=True)
        deep |= {k for p, k in found if p == "logits" and cols >= 1000}
    assert not want - seen and deep == set(range(6))
