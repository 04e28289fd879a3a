"""GPU tests of calls of the embedding and the vocabulary loss as programs make
them: batches of several sequences, each without its first or last token."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import entropy_decoding_amd as ed  # noqa: E402
from test_gpu_vocab_loss import F32, Exact, check, inputs, randn, say  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    torch.cuda.init()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("side", [False, True])
def test_loss_of_a_batch_without_its_last_tokens(side):
    """The same bits as of the rows laid out one behind the other; on a named stream
    also where the batch is dropped at once."""
    say(f"[gpu] loss of a cut batch, on a stream of its own: {side}")
    x, w, targets = inputs(8 * 65, 700, 136, 3)
    x, targets = x.view(8, 65, 136), targets.view(8, 65)
    head, stream = ed.VocabLoss([w]), torch.cuda.Stream() if side else None
    flat, at = x[:, :-1].reshape(-1, 136), targets[:, 1:].reshape(-1)
    want, want_lse = head(flat, at)
    want_dx, (want_dw,) = head.gradient(flat, at, want_lse, 0.1, dw_dtype=F32)
    if side:
        stream.wait_stream(torch.cuda.current_stream())
    losses, lse = head(x[:, :-1], targets[:, 1:], stream=stream)
    dx, (dw,) = head.gradient(x[:, :-1], targets[:, 1:], lse, 0.1, dw_dtype=F32, stream=stream)
    del x, targets
    torch.full((8, 65, 136), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((8, 65), 9, device="cuda")
    torch.cuda.synchronize()
    assert losses.shape == (8, 64) and torch.equal(losses.view(-1), want) and torch.equal(lse.view(-1), want_lse)
    assert torch.equal(dx, want_dx) and torch.equal(dw, want_dw)


@pytest.mark.parametrize("side", [False, True])
def test_table_gradient_of_a_cut_batch(side):
    """The same bits as of the rows laid out one behind the other, and of one token's
    gradient, whose lookup gives a single row."""
    say(f"[gpu] table gradient of a cut batch, on a stream of its own: {side}")
    table, tokens = randn(300, 136, seed=1), torch.randint(0, 300, (8, 65), device="cuda")
    emb, dy, stream = ed.Embedding(table, scale=1.5), randn(8, 65, 136, seed=2), torch.cuda.Stream() if side else None
    want = emb.gradient(tokens[:, 1:].reshape(-1), dy[:, 1:].reshape(-1, 136))
    one = emb.gradient(tokens[2, 3].view(1), dy[2, 3].view(1, 136))
    if side:
        stream.wait_stream(torch.cuda.current_stream())
    got = emb.gradient(tokens[:, 1:], dy[:, 1:], stream=stream)
    got_one = emb.gradient(tokens[2, 3], dy[2, 3], stream=stream)
    del tokens, dy
    torch.full((8, 65, 136), 9.0, device="cuda"), torch.full((8, 65), 9, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got_one, one) and one.any()


def test_losses_under_a_head_that_requires_a_gradient():
    """The same bits; differentiated, also beside what has a gradient, they are an error."""
    say("[gpu] head that requires a gradient")
    x, w, targets = inputs(40, 300, 72, 5)
    want, want_lse = ed.VocabLoss([w])(x, targets)
    param, other = torch.nn.Parameter(w), torch.ones(1, device="cuda").requires_grad_()
    head = ed.VocabLoss([param])
    losses, lse = head(x, targets)
    assert torch.equal(losses, want) and torch.equal(lse, want_lse)
    with pytest.raises(RuntimeError, match="records no gradient for its head"):
        (losses.sum() + other.sum()).backward()
    dx, (dw,) = head.gradient(x, targets, lse, losses=losses)
    want_dx, (want_dw,) = ed.VocabLoss([w]).gradient(x, targets, want_lse, losses=want)
    assert torch.equal(dx, want_dx) and torch.equal(dw, want_dw)


def test_loss_of_many_tokens_under_many_rows():
    """2^22 tiles of 512 threads: half of what a grid holds.  Every block of the same
    1024 tokens has their bits."""
    say("[gpu] loss of 2^20 tokens under 262147 rows")
    x, w, targets = inputs(1024, 262_147, 8, 3)
    head, e = ed.VocabLoss([w]), Exact(x, w, targets)
    losses, lse = head(x, targets)
    check(lse, e.lse, e.off_lse, "lse")
    check(losses, e.loss, e.off_loss, "loss")
    del e
    many, many_lse = head(x.repeat(1024, 1), targets.repeat(1024))
    assert (many.view(1024, 1024) == losses).all() and (many_lse.view(1024, 1024) == lse).all()


@pytest.mark.parametrize("side", [False, True])
def test_loss_of_rows_that_the_library_does_not_reach(side):
    """The last token of each of several long sequences, rows that begin at any
    element, one row for all targets: the same bits as of rows one behind the other."""
    say(f"[gpu] loss of rows far apart or misaligned, on a stream of its own: {side}")
    long, w, _ = inputs(3 * 20_000, 300, 136, 2)
    targets, stream = torch.tensor([5, -100, 299], device="cuda"), torch.cuda.Stream() if side else None
    head = ed.VocabLoss([w])
    for x in (long.view(3, 20_000, 136)[:, -1], randn(3, 200, seed=1).to(long.dtype)[:, 3:139],
              randn(3, 139, seed=2).to(long.dtype)[:, :136], long[7:8].expand(3, 136)):
        want, want_lse = head(x.contiguous(), targets)
        want_dx, (want_dw,) = head.gradient(x.contiguous(), targets, want_lse)
        if side:
            stream.wait_stream(torch.cuda.current_stream())
        losses, lse = head(x, targets, stream=stream)
        dx, (dw,) = head.gradient(x, targets, lse, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(losses, want) and torch.equal(lse, want_lse)
        assert torch.equal(dx, want_dx) and torch.equal(dw, want_dw) and dw.any()
