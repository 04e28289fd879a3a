"""GPU tests of the embedding, the loss and their gradients as a program uses them
together: a head that stays compressed, and a training step of a table that is
embedding and head at once, through AdamW and the encoder back to a compressed
head."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import entropy_decoding_amd as ed  # noqa: E402
from test_gpu_vocab_loss import U, Exact, check, inputs, randn, say  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    torch.cuda.init()
    yield
    torch.cuda.synchronize()


def compressed(parts):
    tensors = [w.cpu().view(torch.int16).numpy().view(np.uint16).reshape(-1) for w in parts]
    cb = ed.df11_build_codebook(tensors)
    return ed.DeviceStream(ed.df11_encode(cb, tensors), cb, "cuda")


@pytest.mark.parametrize("n,sizes", [(1, [333]), (40, [128, 5, 200]), (300, [1000, 1001])])
@pytest.mark.parametrize("side", [False, True])
def test_compressed_head(n, sizes, side):
    """The same bits as of the head held in BF16, its pieces decompressed in turn."""
    say(f"[gpu] compressed head of {sizes} rows, {n} tokens, on a stream of its own: {side}")
    x, w, targets = inputs(n, sum(sizes), 72, n)
    parts = [t.contiguous() for t in w.split(sizes)]
    want, want_lse = ed.VocabLoss(parts)(x, targets)
    want_dx, want_dws = ed.VocabLoss(parts).gradient(x, targets, want_lse, 0.5, dw_dtype=F32)
    head = ed.VocabLoss.from_unit(compressed(parts), [(r, 72) for r in sizes])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream() if side else None
    if side:
        stream.wait_stream(torch.cuda.current_stream())
    losses, lse = head(x, targets, status=status, stream=stream)
    dx, dws = head.gradient(x, targets, lse, 0.5, dw_dtype=F32, status=status, stream=stream)
    torch.cuda.synchronize()
    assert int(status) == 0 and torch.equal(losses, want) and torch.equal(lse, want_lse)
    assert torch.equal(dx, want_dx) and all(torch.equal(a, b) for a, b in zip(dws, want_dws))


def test_unit_shapes_are_checked():
    unit = compressed([randn(10, 16).to(BF16), randn(6, 16).to(BF16)])
    ed.VocabLoss.from_unit(unit, [(10, 16), (6, 16)])
    for shapes in ([(16, 16)], [(6, 16), (10, 16)], [(10, 16), (12, 8)], []):
        with pytest.raises(ValueError):
            ed.VocabLoss.from_unit(unit, shapes)


def test_a_step_of_a_tied_table():
    """Lookup, loss, both gradients added up in float32 over two microbatches, AdamW
    with the norm clipped, encoded, and the compressed head's loss afterwards."""
    say("[gpu] training step of a table that is embedding and head")
    rows, cols, n = 700, 72, 150
    table = (randn(rows, cols, seed=1) / 4).to(BF16)
    tokens = torch.randint(0, rows, (2, n + 1), device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    tokens[:, -20:] = 3  # padding: looked up, without a gradient, not counted
    emb, head = ed.Embedding(table, padding_idx=3), ed.VocabLoss([table])
    grad = torch.zeros(rows, cols, device="cuda")
    want = torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
    off = torch.zeros_like(want)
    for part in tokens:
        seen, targets = part[:-1], part[1:]
        x = emb(seen)
        assert torch.equal(x, table[seen])
        losses, lse = head(x, targets, ignore_index=3)
        scale = 1.0 / int((targets != 3).sum())
        dx, _ = head.gradient(x, targets, lse, scale, ignore_index=3, dx_dtype=F32, dws=[grad], accumulate=True)
        emb.gradient(seen, dx, out=grad, accumulate=True)
        e = Exact(x, table, targets, ignored=3)
        check(losses, e.loss, e.off_loss, "loss")
        g, off_g = e.gradient(scale, 0.0, 2)
        (dx_want, dx_off), (dw_want, dw_off) = e.dx(g, off_g, F32), e.dw(g, off_g, F32)
        kept = seen != 3
        want += dw_want.index_add(0, seen[kept], dx_want[kept])
        off += dw_off.index_add(0, seen[kept], dx_off[kept])
        # a row's sum of up to n terms, and its additions to what is there
        size = dx_want.abs() + dx_off
        off += (n + 2) * U * torch.zeros_like(want).index_add(0, seen[kept], size[kept]) + 2 * U * want.abs()
    check(grad, want, off, "the table's gradient")
    opt = ed.AdamW([table], [grad], lr=1e-2, counts=True)
    before = table.clone()
    norm = opt.step(max_norm=1.0)
    exact = grad.double().norm()
    assert abs(norm[0].double() - exact) <= 4 * U * exact
    assert not torch.equal(table, before) and torch.equal(emb(tokens[0]), table[tokens[0]])
    unit, _ = opt.compress()
    x = emb(tokens[0, :-1])
    for a, b in zip(head(x, tokens[0, 1:]), ed.VocabLoss.from_unit(unit, [(rows, cols)])(x, tokens[0, 1:])):
        assert torch.equal(a, b)


def test_two_calls_of_one_head_at_once():
    """On two streams, each call with its own scratch."""
    say("[gpu] one head on two streams at once")
    x, w, targets = inputs(400, 20_000, 520, 3)
    other = inputs(400, 20_000, 520, 4)
    head = ed.VocabLoss([w])
    streams = [torch.cuda.Stream() for _ in range(2)]
    wants = []
    for a, t in ((x, targets), (other[0], other[2])):
        _, lse = head(a, t)
        wants.append((lse, head.gradient(a, t, lse, 0.1)))
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for stream, (a, t) in zip(streams, ((x, targets), (other[0], other[2]))):
            with torch.cuda.stream(stream):
                _, lse = head(a, t)
                got.append((lse, head.gradient(a, t, lse, 0.1)))
        torch.cuda.synchronize()
        for (lse, (dx, (dw,))), (lse2, (dx2, (dw2,))) in zip(got, wants):
            assert torch.equal(lse, lse2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_captured_on_a_stream_that_the_calls_name():
    say("[gpu] lookup, loss and gradients captured on a named stream")
    table = (randn(900, 136) / 10).to(BF16)
    emb, head = ed.Embedding(table), ed.VocabLoss([table])
    stream = torch.cuda.Stream()
    tokens = torch.randint(0, 900, (3001,), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    grad = torch.zeros(900, 136, device="cuda")

    def step(at):
        x = emb(tokens[:-1], stream=at)
        losses, lse = head(x, tokens[1:], stream=at)
        dx, _ = head.gradient(x, tokens[1:], lse, 0.01, losses=losses, dws=[grad], accumulate=True, stream=at)
        emb.gradient(tokens[:-1], dx, out=grad, accumulate=True, stream=at)
        return losses, dx

    stream.wait_stream(torch.cuda.current_stream())
    step(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        losses, dx = step(stream)
    for turn in range(3):
        tokens.copy_(torch.randint(0, 900, (3001,), device="cuda"))
        grad.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = losses.clone(), dx.clone(), grad.clone()
        grad.zero_()
        want = *step(None), grad
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_freed_while_another_stream_uses_them():
    """The head, the table and what the calls are given are dropped at once, with the
    stream still busy: new tensors must not lie there."""
    say("[gpu] table and head dropped while a busy stream uses them")
    from test_gpu_lifetimes import busy, refill

    table = (randn(3000, 264) / 10).to(BF16)
    tokens = torch.randint(0, 3000, (601,), device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    want = ed.VocabLoss([table])(ed.Embedding(table)(tokens[:-1]), tokens[1:])[0]
    used = [table.clone(), tokens.clone(), torch.zeros(600, 264, dtype=BF16, device="cuda")]
    emb, head = ed.Embedding(used[0]), ed.VocabLoss([used[0]])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    held = busy(side)
    emb(used[1][:-1], out=used[2], stream=side)
    losses, _ = head(used[2], used[1][1:], stream=side)
    at = {t.data_ptr() for t in used}
    sizes = [t.numel() * t.element_size() for t in used]
    del emb, head, used
    others, places = refill(sizes, torch.uint8)
    assert not at & places
    torch.cuda.synchronize()
    assert torch.equal(losses, want)
    del held, others
