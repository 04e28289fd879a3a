"""What the compiler says of the vocabulary loss's tiles, in the built library: as
many workgroups fit a compute unit as their choice counts on, and no register
goes to memory."""

import re
import struct
import subprocess

import pytest

import entropy_decoding_amd as ed

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
