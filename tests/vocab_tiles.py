"""Which of its tiles the vocabulary loss sends a shape to: the choice in
df11_vocab_loss.hip (tile_for, chunk_rows, dx_split) written again, with the table of
tiles read from there, so that tests can say which of them their shapes reach."""

import os
import re

import numpy as np

import entropy_decoding_amd as ed

F = np.float32
SOURCE = os.path.join(os.path.dirname(ed.__file__), "csrc", "df11_vocab_loss.hip")
with open(SOURCE) as f:
    _TABLE = re.search(r"kTiles\[\] = \{(\{.*?\})\};", f.read(), re.S)[1]
# (t, r, threads, workgroups of a compute unit, us of a stage with the chip full, alone)
TILES = [tuple(float(v.strip().rstrip("f")) for v in t.split(",")) for t in re.findall(r"\{(.*?)\}", _TABLE, re.S)]
DEPTH, UNITS, TWO_TERM_TOKENS, PAST = 64, 256, 64, 1 << 27


def terms_for(n, float32):
    return 3 if float32 else 2 if n <= TWO_TERM_TOKENS else 1


def up(n, to):
    return -(-n // to) * to


def tiles_of(tile, t, r):
    return up(t, int(tile[0])) // int(tile[0]) * (up(r, int(tile[1])) // int(tile[1]))


def time_of(tile, t, r, stages):
    n, at_once = tiles_of(tile, t, r), UNITS * int(tile[3])
    if n <= UNITS:
        return F(stages) * F(tile[5]) + F(3)
    return F(-(-n // at_once)) * (F(stages) * F(tile[4]) + F(3))


def tile_for(t, r, k):
    times = [time_of(tile, t, r, -(-k // DEPTH)) for tile in TILES]
    return times.index(min(times))


def chunk_rows(n, rows):
    most = max((1 << 29) // max(n, 1) // 256 * 256, 256)
    chunks = max(-(-rows // most), 1)
    return max(up(-(-rows // chunks), 256), 256)


def dx_split(n, cols, rows):
    stages, best, least = max(-(-rows // DEPTH), 1), (0, 1), None
    for i, tile in enumerate(TILES):
        parts = max(min(UNITS * int(tile[3]) // max(tiles_of(tile, n, cols), 1), stages // 8, 64), 1)
        time = time_of(tile, n, cols * parts, -(-stages // parts)) + F(parts * n * cols) * F(8 / 5e6)
        if least is None or time < least:
            least, best = time, (i, parts)
    return best


def forms(n, rows, cols, dw="bfloat16", add=False, on_half_lines=False):
    """The (product, tile) of a loss with gradients, a head in one piece; whether dw's
    rows lie on half lines.  The products
    of dw are told apart by type, by whether they are added, and stored past the caches;
    those of dx by whether they are in parts."""
    found = {("logits", tile_for(n, rows, cols))}
    chunk, size = chunk_rows(n, rows), 4 if dw == "float32" else 2
    past = rows * cols * size >= PAST and (not add if size == 2 else on_half_lines)
    name = f"dw {dw}{' added' if add else ''}{' past' if past else ''}"
    for c in range(0, rows, chunk):
        here = min(chunk, rows - c)
        found.add(("g", tile_for(n, here, cols)))
        found.add((name, tile_for(here, cols, n * terms_for(n, size == 4))))
    tile, parts = dx_split(n, cols, chunk)
    return found | {("dx in parts" if parts > 1 else "dx", tile)}


def loss_bytes(n, rows, cols):
    r = int(TILES[tile_for(n, rows, cols)][1])
    return up(8 * n, 256) + up(4 * n, 256) + up(8 * up(n, 16) * -(-rows // r), 256)


def gradient_bytes(n, rows, cols, dx, two_terms):
    chunk = chunk_rows(n, rows)
    parts = dx_split(n, cols, chunk)[1]
    total = 512 + 3 * up(4 * n, 256) + up(4 * n, 256) + up(8 * n, 256) + up(2 * n * up(cols, 64), 256)
    total += up(4 * parts * n * cols, 256) if dx else 0
    return total + up(2 * n * chunk * terms_for(n, two_terms), 256)
