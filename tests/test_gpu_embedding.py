"""GPU tests of the embedding lookup and of its gradient by sorted tokens.

Lookups are compared bit for bit: one float32 product and one rounding.  A
gradient's sum of k terms in float32, in any order, is off by at most
(k - 1) 2^-24 of the terms' magnitudes together (to first order), and the scale and an
addition round once each; the result's own rounding is at most half a step.
"""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import entropy_decoding_amd as ed  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
# half a step, at most, relative to the value: just above 1 the steps of types
# with 23, 7 and 10 bits behind the point are 2^-23, 2^-7 and 2^-10
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}


def say(msg):
    print(msg, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    torch.cuda.init()
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=gen(seed), device="cuda")


def some_tokens(n, rows, seed, kind=torch.int64):
    """Few common tokens and many rare ones."""
    u = torch.rand(n, generator=gen(seed), device="cuda")
    return ((u * u * u * rows).long().clamp(max=rows - 1) * 5 % rows).to(kind)


def plain_lookup(table, tokens, scale, kind):
    inside = (tokens >= 0) & (tokens < table.size(0))
    y = table[torch.where(inside, tokens, 0).long()].float() * torch.tensor(scale, dtype=F32, device="cuda")
    return torch.where(inside[:, None], y, float("nan")).to(kind)


def same(a, b):
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())


@pytest.mark.parametrize("kind", [F32, BF16, F16])
@pytest.mark.parametrize("out", [F32, BF16, F16])
@pytest.mark.parametrize("n,rows,cols", [(1, 1, 1), (1, 50, 4096), (5, 7, 8), (77, 33, 1001), (300, 999, 2056),
                                         (33, 5, 2049), (9, 40, 6151)])
def test_lookup(kind, out, n, rows, cols):
    say(f"[gpu] lookup {n} of {rows} x {cols}, {kind} to {out}")
    table = randn(rows, cols, seed=n).to(kind)
    tokens = some_tokens(n, rows, n + 1, torch.int64 if n % 2 else torch.int32)
    y = ed.Embedding(table, scale=1.7)(tokens, out)
    assert y.shape == (n, cols) and torch.equal(y, plain_lookup(table, tokens, 1.7, out))


def test_lookup_of_tokens_outside_the_table():
    say("[gpu] lookup of tokens outside the table")
    table = randn(10, 40)
    for kind in (torch.int32, torch.int64):
        tokens = torch.tensor([3, -1, 10, 9, 0, -2 ** 31, 2 ** 31 - 1], dtype=kind, device="cuda")
        assert same(ed.Embedding(table)(tokens), plain_lookup(table, tokens, 1.0, F32))
    far = torch.tensor([2 ** 32 + 3, -2 ** 63, 2 ** 63 - 1], device="cuda")
    assert ed.Embedding(table)(far).isnan().all()


def test_lookup_shapes_strides_and_outputs():
    """Tokens of any shape and strides; tables and outputs with rows apart, at
    any offset; what lies between an output's rows stays."""
    say("[gpu] lookup with strides")
    room = randn(30, 83, seed=3).to(BF16)
    table = room[:, 7:72]
    grid = some_tokens(60, 30, 4).view(5, 12)
    emb = ed.Embedding(table)
    for tokens in (grid, grid[:, 1:], grid.t(), grid[:, 0], grid[:0], grid[2, 3]):
        y = emb(tokens)
        assert y.shape == (*tokens.shape, 65)
        assert torch.equal(y.reshape(-1, 65), table[tokens.reshape(-1)])
    held = torch.full((60, 101), 7.0, dtype=BF16, device="cuda")
    version = held._version
    assert emb(grid, out=held[:, 3:68]).data_ptr() == held[:, 3:].data_ptr() and held._version > version
    assert torch.equal(held[:, 3:68], table[grid.reshape(-1)])
    assert (held[:, :3] == 7).all() and (held[:, 68:] == 7).all()


def test_lookup_beyond_32_bits():
    """A table and an output of more than 2^32 bytes and 2^31 elements."""
    say("[gpu] lookup beyond 32 bits")
    table = torch.zeros(150_000, 16_384, dtype=BF16, device="cuda")
    table[:, 0] = torch.arange(150_000, device="cuda") % 251
    table[:, -1] = torch.arange(150_000, device="cuda") % 241
    tokens = torch.randint(0, 150_000, (140_000,), generator=gen(1), device="cuda")
    tokens[-1], tokens[-2] = 149_999, 131_072
    y = ed.Embedding(table)(tokens)
    assert torch.equal(y[:, 0], table[:, 0][tokens]) and torch.equal(y[:, -1], table[:, -1][tokens])
    assert not y[:, 1:-1].any()


def test_a_table_that_requires_a_gradient_is_refused():
    table = torch.nn.Parameter(randn(10, 16))
    emb, tokens = ed.Embedding(table), torch.arange(3, device="cuda")
    with pytest.raises(RuntimeError, match="gradient"):
        emb(tokens)
    with torch.no_grad():
        assert torch.equal(emb(tokens), table[:3])


def check_gradient(got, tokens, dy, rows, scale=1.0, padding=None, before=None):
    """Against sums in float64; rows without a token bit for bit."""
    kept = (tokens >= 0) & (tokens < rows)
    if padding is not None:
        kept &= tokens != padding
    at, terms = tokens[kept].long(), dy.double()[kept] * scale
    zero = torch.zeros(rows, dy.size(1), dtype=torch.float64, device="cuda")
    want, size = zero.index_add(0, at, terms), zero.index_add(0, at, terms.abs())
    count = torch.bincount(at, minlength=rows)[:, None]
    base = zero if before is None else before.double()
    off = (count + 2) * 2.0 ** -24 * size + 2.0 ** -24 * base.abs()
    off += HALF[got.dtype] * ((want + base).abs() + off)
    if got.dtype == F16:
        off += 2.0 ** -25  # half a step of the smallest values
    off *= count > 0
    assert ((got.double() - want - base).abs() <= off).all()


@pytest.mark.parametrize("kind", [F32, BF16, F16])
@pytest.mark.parametrize("out", [F32, BF16, F16])
@pytest.mark.parametrize("n,rows,cols", [(1, 1, 1), (2, 3, 8), (16, 5, 40), (17, 5, 520), (300, 999, 513),
                                         (1000, 7, 24), (2048, 1, 8), (2048, 700, 1030), (2049, 700, 1030),
                                         (4100, 2500, 40)])
def test_gradient(kind, out, n, rows, cols):
    say(f"[gpu] gradient {n} of {rows} x {cols}, {kind} to {out}")
    tokens = some_tokens(n, rows, n, torch.int64 if n % 2 else torch.int32)
    dy = randn(n, cols, seed=rows).to(kind)
    got = ed.embedding_gradient(tokens, dy, rows, out, scale=0.37)
    assert got.dtype == out
    check_gradient(got, tokens, dy, rows, scale=float(torch.tensor(0.37, dtype=F32)))
    assert torch.equal(got, ed.embedding_gradient(tokens, dy, rows, out, scale=0.37))


@pytest.mark.parametrize("n", [1, 31, 32, 33, 48, 1024, 2047, 2048, 2049, 5000, 70_000])
@pytest.mark.parametrize("rows", [1, 5, 600_000])
def test_gradient_of_one_row(n, rows):
    """All tokens the same: a run over all chunks."""
    say(f"[gpu] gradient of {n} equal tokens, {rows} rows")
    dy = randn(n, 9, seed=n)
    tokens = torch.full((n,), rows - 1, device="cuda")
    check_gradient(ed.embedding_gradient(tokens, dy, rows), tokens, dy, rows)


@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("n", [1, 40, 3000])
def test_gradient_of_a_large_table(kind, n):
    """2^26 elements and more: rows that no token meets are cleared past the caches."""
    say(f"[gpu] gradient of a large table, {n} tokens, {kind}")
    rows, cols = 66_000, 1033
    tokens, dy = some_tokens(n, rows, n), randn(n, cols, seed=n)
    got = torch.full((rows, cols + 5), 7.0, dtype=kind, device="cuda")
    ed.embedding_gradient(tokens, dy, rows, out=got[:, 2:cols + 2])
    check_gradient(got[:, 2:cols + 2], tokens, dy, rows)
    assert (got[:, :2] == 7).all() and (got[:, cols + 2:] == 7).all()
    added = torch.zeros(rows, cols, device="cuda")
    ed.embedding_gradient(tokens, dy, rows, out=added, accumulate=True)
    check_gradient(added, tokens, dy, rows)


def test_gradient_of_runs_that_end_with_chunks():
    """Runs of 1 to 128 tokens, each length at many offsets of a chunk of 32."""
    say("[gpu] gradient of runs at chunk borders")
    for first in range(1, 33):
        lengths = [first] + [k for k in (16, 32, 1, 31, 33, 63, 64, 65, 128, 32, 32, 2) for _ in "abcde"]
        assert sum(lengths) > 2048
        tokens = torch.repeat_interleave(torch.arange(len(lengths), device="cuda"),
                                         torch.tensor(lengths, device="cuda"))
        tokens = tokens[torch.randperm(len(tokens), generator=gen(first), device="cuda")]
        dy = randn(len(tokens), 8, seed=first)
        check_gradient(ed.embedding_gradient(tokens, dy, len(lengths) + 3), tokens, dy, len(lengths) + 3)


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("n", [200, 2000, 3000])
def test_gradient_added(n, out):
    """Added to what is there; rows without a token are not touched, not even NaN."""
    say(f"[gpu] gradient added, {n} tokens, {out}")
    rows, cols, padding = 700, 136, 35
    tokens, dy = some_tokens(n, rows, 9), randn(n, cols, seed=2)
    tokens[::7] = padding
    tokens[3::50], tokens[4::50] = -100, rows
    dy[::7] = float("nan")  # what padding has is not looked at
    before = randn(rows, cols, seed=5).to(out)
    missed = torch.bincount(tokens[(tokens >= 0) & (tokens < rows) & (tokens != padding)], minlength=rows) == 0
    assert missed.any() and missed[padding]
    before[missed] = float("nan")
    dw = before.clone()
    version = dw._version
    got = ed.embedding_gradient(tokens, dy, rows, out=dw, accumulate=True, scale=3.0, padding_idx=padding)
    assert got is dw and dw._version > version and dw[missed].isnan().all()
    before[missed] = dw[missed] = 0
    check_gradient(dw, tokens, dy.nan_to_num(), rows, 3.0, padding, before)


def test_gradient_strides():
    """Rows apart and at any offset; one row of dy for all tokens; what lies between rows stays."""
    say("[gpu] gradient with strides")
    grid = some_tokens(96, 20, 8).view(8, 12)
    dy = randn(8, 12, 131, seed=1).to(BF16)
    flat = grid.reshape(-1)
    emb = ed.Embedding(randn(20, 131), scale=2.0, padding_idx=5)
    check_gradient(emb.gradient(grid, dy), flat, dy.view(96, 131), 20, 2.0, 5)
    room = torch.full((20, 151), 7.0, device="cuda")
    apart = randn(96, 150, seed=2)[:, 11:142]
    emb.gradient(flat, apart, out=room[:, 9:140])
    check_gradient(room[:, 9:140].contiguous(), flat, apart, 20, 2.0, 5)
    assert (room[:, :9] == 7).all() and (room[:, 140:] == 7).all()
    one = randn(1, 131).expand(96, 131)
    check_gradient(emb.gradient(flat, one), flat, one, 20, 2.0, 5)
    check_gradient(emb.gradient(grid[:, 3:7], dy[:, 3:7].contiguous()), grid[:, 3:7].reshape(-1),
                   dy[:, 3:7].reshape(32, 131), 20, 2.0, 5)


def test_gradient_of_no_tokens():
    say("[gpu] gradient of no tokens")
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    assert not ed.embedding_gradient(none, torch.zeros(0, 40, device="cuda"), 30).any()
    large = torch.ones(66_000, 1033, device="cuda")  # three launches otherwise
    assert not ed.embedding_gradient(none, torch.zeros(0, 1033, device="cuda"), 66_000, out=large).any()
    dw = torch.ones(30, 40, device="cuda")
    ed.embedding_gradient(none, torch.zeros(0, 40, device="cuda"), 30, out=dw, accumulate=True)
    assert (dw == 1).all()
    assert not ed.embedding_gradient(torch.tensor([-1, 30], device="cuda"), torch.ones(2, 40, device="cuda"), 30).any()


def test_gradient_of_nan_and_infinity():
    say("[gpu] gradient of NaN and infinities")
    tokens = torch.tensor([2, 0, 2, 4, 4, 0], device="cuda")
    dy = torch.ones(6, 8, device="cuda")
    dy[0, 1], dy[3, 2], dy[4, 2], dy[1, 3] = float("nan"), float("inf"), -float("inf"), float("inf")
    got = ed.embedding_gradient(tokens, dy, 5)
    want = torch.zeros(5, 8, device="cuda").index_add(0, tokens, dy)
    assert same(got, want)


def test_gradient_beyond_32_bits():
    say("[gpu] gradient beyond 32 bits")
    rows, cols, n = 140_000, 16_384, 150_000
    tokens = torch.randint(0, rows, (n,), generator=gen(1), device="cuda")
    tokens[:3] = rows - 1
    dy = torch.zeros(n, cols, dtype=BF16, device="cuda")
    dy[:, 0], dy[:, -1] = 1, torch.arange(n, device="cuda") % 4
    dw = ed.embedding_gradient(tokens, dy, rows)
    for c in (0, cols - 1):
        want = torch.zeros(rows, device="cuda").index_add(0, tokens, dy[:, c].float())
        assert torch.equal(dw[:, c].float(), want)
    assert not dw[:, 1:-1].any()


def test_against_differences():
    """The gradient is that of the lookup: changing one element of the table
    changes a sum of the outputs by that much (both are linear)."""
    say("[gpu] gradient against differences")
    table = randn(13, 24)
    tokens, dy = some_tokens(50, 13, 6), randn(50, 24, seed=7)
    emb = ed.Embedding(table, scale=1.5)
    dw = emb.gradient(tokens, dy)
    at = lambda: (emb(tokens).double() * dy).sum()  # noqa: E731
    for r, c in ((0, 0), (int(tokens[0]), 5), (12, 23)):
        base = at()
        held = table[r, c].clone()
        table[r, c] += 8.0
        slope = (at() - base) / 8.0
        table[r, c] = held
        # 50 products of float32 outputs, each half a step off, and dw's own roundings
        assert abs(float(slope - dw[r, c])) <= 50 * 2 * 16 * 5 * 2.0 ** -24


def test_captured_and_replayed_on_two_streams():
    """One graph per stream; new inputs between replays, eager calls beside them."""
    say("[gpu] lookup and gradient captured on two streams")
    table = randn(200, 72).to(BF16)
    emb = ed.Embedding(table)
    held = []
    for k in range(2):
        stream = torch.cuda.Stream()
        tokens, dy = some_tokens(500, 200, k), randn(500, 72, seed=k)
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            emb(tokens), emb.gradient(tokens, dy, dtype=F32)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            y, dw = emb(tokens), emb.gradient(tokens, dy, dtype=F32)
        held.append((stream, graph, tokens, dy, y, dw))
    for turn in range(4):
        for k, (stream, graph, tokens, dy, y, dw) in enumerate(held):
            tokens.copy_(some_tokens(500, 200, 10 * turn + k)), dy.copy_(randn(500, 72, seed=turn + 5 * k))
        torch.cuda.synchronize()
        for stream, graph, *_ in held:
            with torch.cuda.stream(stream):
                graph.replay()
        wanted = [(emb(h[2]), emb.gradient(h[2], h[3], dtype=F32)) for h in held]
        torch.cuda.synchronize()
        for h, (y, dw) in zip(held, wanted):
            assert torch.equal(h[4], y) and torch.equal(h[5], dw)


def test_named_stream():
    """A call on a named stream, its inputs freed and their memory reused at once."""
    say("[gpu] lookup and gradient on a named stream")
    emb, stream = ed.Embedding(randn(500, 1024)), torch.cuda.Stream()
    for turn in range(5):
        tokens, dy = some_tokens(3000, 500, turn), randn(3000, 1024, seed=turn)
        kept, want = tokens.clone(), dy.clone()
        stream.wait_stream(torch.cuda.current_stream())
        y = emb(tokens, stream=stream)
        dw = emb.gradient(tokens, dy, stream=stream)
        del tokens, dy
        torch.full((3000, 1024), 9.0, device="cuda"), torch.full((3000,), 9, device="cuda")
        torch.cuda.synchronize()
        assert torch.equal(y, emb.table[kept])
        check_gradient(dw, kept, want, 500)


@pytest.mark.parametrize("kind,n", [(F32, 65_500), (BF16, 130_000), (F16, 130_001)])
@pytest.mark.parametrize("out", [F32, BF16])
def test_gradient_added_from_much_that_is_read_once(kind, n, out):
    """2^28 bytes of dy and more pass the caches: runs of one token and runs over many
    chunks, added into rows that lie apart."""
    rows, cols = 4001, 1033
    say(f"[gpu] gradient added from {n} x {cols} of {kind}, to {out}")
    assert n * cols * (4 if kind == F32 else 2) >= 1 << 28
    tokens, dy = some_tokens(n, rows, 3), randn(n, cols, seed=4).to(kind)
    tokens[: n // 8], tokens[5::1000] = 17, rows + 3
    before = randn(rows, cols, seed=5).to(out)
    room = torch.full((rows, cols + 6), 7.0, dtype=out, device="cuda")
    dw = room[:, 3:cols + 3]
    dw.copy_(before)
    ed.embedding_gradient(tokens, dy, rows, out=dw, accumulate=True, scale=0.5, padding_idx=9)
    kept = (tokens < rows) & (tokens != 9)
    count = torch.bincount(tokens[kept], minlength=rows)
    assert count.max() > n // 8 - 100 and (count == 1).any() and (count == 0).any()
    assert torch.equal(dw[count == 0], before[count == 0])
    check_gradient(dw, tokens, dy, rows, 0.5, 9, before)
    assert (room[:, :3] == 7).all() and (room[:, cols + 3:] == 7).all()
