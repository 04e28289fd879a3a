"""Calls of the embedding and the vocabulary loss as programs make them, with the
stand-ins of test_lending.py for the library, the streams and the device: what
is passed on to the library is what the tensors hold."""

import ctypes

import pytest

import entropy_decoding_amd as ed

torch = pytest.importorskip("torch")

from test_lending import gpu  # noqa: E402,F401

BF16 = torch.bfloat16


def rows_at(address, stride, rows, cols, kind):
    """The rows that a call was given."""
    bits = {BF16: (ctypes.c_int16, torch.int16), torch.float32: (ctypes.c_float, torch.float32)}[kind]
    held = (bits[0] * (stride * (rows - 1) + cols)).from_address(address)
    return torch.frombuffer(held, dtype=bits[1]).view(kind).as_strided((rows, cols), (stride, 1)).clone()


@pytest.fixture
def seen(gpu, monkeypatch):  # noqa: F811
    """What the library's loss functions are given: (function, stream entered, rows of x)."""
    got = []

    def piece(name):
        def call(p, *_):
            got.append((name, gpu.inside, rows_at(p.x, p.x_stride, p.n, p.cols, BF16)))
            return ed.DF11_OK
        return call

    for name in ("df11_vocab_loss", "df11_vocab_loss_gradient"):
        monkeypatch.setattr(gpu.lib, name, piece(name), raising=False)
    return got


@pytest.mark.parametrize("stream", [None, 7])
def test_loss_of_a_batch_without_its_last_tokens(gpu, seen, stream):  # noqa: F811
    """Hidden states of several sequences, each without its last: no one stride
    reaches their rows."""
    head = ed.VocabLoss([torch.zeros(6, 16, dtype=BF16)])
    x = torch.randn(3, 5, 16).to(BF16)
    tokens = torch.zeros(3, 5, dtype=torch.int64)
    for part in (x[:, :-1], x[:, 1:], x.transpose(0, 1)[:4].transpose(0, 1)):
        seen.clear()
        gpu.lent.clear()
        losses, lse = head(part, tokens[:, 1:], stream=stream)
        assert losses.shape == lse.shape == (3, 4)
        dx, _ = head.gradient(part, tokens[:, 1:], lse, stream=stream)
        assert dx.shape == (12, 16)
        assert [s[0] for s in seen] == ["df11_vocab_loss", "df11_vocab_loss_gradient"]
        assert all(s[1] == (stream or gpu.current) and torch.equal(s[2], part.reshape(12, 16)) for s in seen)
        assert ((part.data_ptr(), 7) in gpu.lent) == (stream == 7)


@pytest.mark.parametrize("stream", [None, 7])
def test_loss_of_rows_that_the_library_does_not_reach(gpu, seen, stream):  # noqa: F811
    """The last token of each of several long sequences (rows further apart than
    DF11_VOCAB_MAX_STRIDE); rows that begin at any element, or any number of them apart."""
    head, targets = ed.VocabLoss([torch.zeros(6, 16, dtype=BF16)]), torch.zeros(2, dtype=torch.int64)
    long = torch.randn(2, (1 << 17) + 1, 16).to(BF16)
    odd = torch.randn(2, 27).to(BF16)
    for x in (long[:, -1], odd[:, 8:24], torch.randn(2, 32).to(BF16)[:, 3:19], torch.randn(1, 16).to(BF16).expand(2, 16)):
        seen.clear()
        gpu.lent.clear()
        _, lse = head(x, targets, stream=stream)
        head.gradient(x, targets, lse, stream=stream)
        assert len(seen) == 2 and all(s[1] == (stream or gpu.current) and torch.equal(s[2], x) for s in seen)
        assert ((x.data_ptr(), 7) in gpu.lent) == (stream == 7)
    assert all(p % 16 == 0 and s % 8 == 0 and s <= ed.DF11_VOCAB_MAX_STRIDE for p, s in given(head, long[:, -1], odd[:, 8:24]))


def given(head, *xs):
    """Where the rows lie that are passed on, and how far apart."""
    for x in xs:
        _, p = head._piece(x, torch.zeros(len(x), dtype=torch.int64), -100, None)
        yield p.x, p.x_stride


def test_hidden_states_that_are_refused(gpu, seen):  # noqa: F811
    head, tokens = ed.VocabLoss([torch.zeros(6, 16, dtype=BF16)]), torch.zeros(3, 4, dtype=torch.int64)
    x = torch.zeros(3, 16, 4, dtype=BF16)
    for bad in (x.transpose(1, 2), torch.zeros(3, 4, 32, dtype=BF16)[:, :, ::2], torch.zeros(3, 5, 16, dtype=BF16),
                torch.zeros(4, 3, 16, dtype=BF16), torch.zeros(3, 4, 24, dtype=BF16)):
        with pytest.raises(ValueError):
            head(bad, tokens)
        with pytest.raises(ValueError):
            head.gradient(bad, tokens, torch.zeros(3, 4))
    assert not seen


@pytest.mark.parametrize("stream", [None, 7])
def test_table_gradient_of_a_cut_batch(gpu, monkeypatch, stream):  # noqa: F811
    """The output's gradient of several sequences, each without its first; of one
    token that is a number of no dimension."""
    got = []

    def call(g, *_):
        got.append((gpu.inside, rows_at(g.dy, g.dy_stride, g.n, g.cols, torch.float32)))
        return ed.DF11_OK

    monkeypatch.setattr(gpu.lib, "df11_embedding_gradient", call, raising=False)
    dy, tokens = torch.randn(3, 5, 24), torch.zeros(3, 5, dtype=torch.int64)
    emb = ed.Embedding(torch.zeros(9, 24))
    for part, at in ((dy[:, 1:], tokens[:, 1:]), (dy.transpose(0, 1)[1:], tokens.t()[1:]), (dy[2, 3], tokens[2, 3]),
                     (dy[:, 1:, 3:11], tokens[:, 1:])):
        cols = part.size(-1)
        want = part.reshape(-1, cols)
        for f in (lambda: ed.embedding_gradient(at, part, 9, stream=stream),
                  lambda: emb.gradient(at, part, stream=stream)):
            got.clear()
            gpu.lent.clear()
            assert f().shape == (9, cols)
            assert len(got) == 1 and got[0][0] == (stream or gpu.current) and torch.equal(got[0][1], want)
            assert ((part.data_ptr(), 7) in gpu.lent) == (stream == 7)
    got.clear()
    for bad, at in ((dy.transpose(1, 2), torch.zeros(3, 24, dtype=torch.int64)), (dy[:, :, ::2], tokens),
                    (dy[:2], tokens), (dy[0, 0], tokens[0]), (dy[0, 0, 0], tokens[0, 0])):
        with pytest.raises(ValueError):
            ed.embedding_gradient(at, bad, 9)
    assert not got


def test_losses_under_a_head_that_requires_a_gradient_are_not_differentiated(gpu):  # noqa: F811
    """The call records no graph.  A loss summed with what has one must not leave the
    head without its gradient in silence."""
    pieces = [torch.zeros(6, 16, dtype=BF16), torch.nn.Parameter(torch.zeros(3, 16, dtype=BF16))]
    x, targets, other = torch.zeros(5, 16, dtype=BF16), torch.zeros(5, dtype=torch.int64), torch.ones(1).requires_grad_()
    head = ed.VocabLoss(pieces)
    losses, lse = head(x, targets)
    for out in (losses, lse):
        with pytest.raises(RuntimeError, match="gradient"):
            (out.sum() + other.sum()).backward()
    assert pieces[1].grad is None
    reached, todo = set(), [losses.grad_fn, lse.grad_fn]
    while todo:  # the outputs do not hold the node of the head's own leaf
        node = todo.pop()
        reached.add(getattr(node, "variable", None))
        todo += [f for f, _ in node.next_functions if f is not None]
    assert pieces[1] not in reached
    head.gradient(x, targets, lse, losses=losses)
    with torch.no_grad():
        assert not any(t.requires_grad for t in head(x, targets))
    pieces[1].requires_grad_(False)
    assert not any(t.requires_grad for t in head(x, targets))


def test_a_piece_of_more_tiles_than_a_grid_holds_is_refused():
    """2^12 x 2^11 tiles of 256 tokens x 256 rows, of 512 threads each: 2^32 threads (the
    pointers are made up)."""
    z = ed.df11_vocab_sizes(1 << 20, 8, 1 << 19, 0, 0)
    nbytes = ed.LIB.df11_vocab_loss_scratch_bytes(z)
    p = ed.df11_vocab_piece(x=4096, targets=8192, w=16384, x_stride=8, w_stride=8, ignored=-100, n=z.n, cols=8,
                            vocab=z.rows, first=0, rows=z.rows, target_bits=64, begin=1, end=1)
    assert ed.LIB.df11_vocab_loss(p, 32768, 65536, z, 1 << 20, nbytes, None) == ed.DF11_E_INVALID


def test_padding_outside_the_table_is_refused_at_once(gpu):  # noqa: F811
    table = torch.zeros(9, 16)
    for bad in (-1, 9, 1 << 70):
        with pytest.raises(ValueError, match="padding_idx"):
            ed.Embedding(table, padding_idx=bad)
    assert ed.Embedding(table, padding_idx=8).padding_idx == 8
