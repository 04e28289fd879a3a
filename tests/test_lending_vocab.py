"""Which tensors the embedding and the vocabulary loss lend to a stream, with the
stand-ins of test_lending.py for the library, the streams and the device."""

import pytest

import entropy_decoding_amd as ed

torch = pytest.importorskip("torch")

from torch.multiprocessing.reductions import StorageWeakRef  # noqa: E402

from test_lending import gpu, unit  # noqa: E402,F401

BF16 = torch.bfloat16


def lent(gpu, tensors, stream):  # noqa: F811
    return {(t.data_ptr(), stream) for t in tensors} <= gpu.lent


def test_embedding(gpu):  # noqa: F811
    table, tokens, dy = torch.zeros(9, 16), torch.zeros(5, dtype=torch.int64), torch.zeros(5, 16)
    emb = ed.Embedding(table)
    y = emb(tokens)
    assert lent(gpu, [table], gpu.current) and not lent(gpu, [tokens], gpu.current)
    gpu.current = 5
    emb(tokens)
    assert lent(gpu, [table], 5)
    y = emb(tokens, stream=7)
    assert lent(gpu, [table, tokens, y], 7)
    given = torch.zeros(5, 16)
    emb(tokens, out=given, stream=8)
    assert lent(gpu, [given], 8)
    dw = torch.zeros(9, 16)
    ed.embedding_gradient(tokens, dy, 9)
    assert not lent(gpu, [dy], gpu.current)
    ed.embedding_gradient(tokens, dy, 9, out=dw, accumulate=True, stream=9)
    assert lent(gpu, [tokens, dy, dw], 9)
    assert gpu.lib.calls.count("df11_embedding") == 4 and gpu.lib.calls.count("df11_embedding_gradient") == 2


def test_loss(gpu):  # noqa: F811
    pieces = [torch.zeros(6, 16, dtype=BF16), torch.zeros(3, 16, dtype=BF16)]
    x, targets, lse = torch.zeros(5, 16, dtype=BF16), torch.zeros(5, dtype=torch.int32), torch.zeros(5)
    head = ed.VocabLoss(pieces)
    head(x, targets)
    assert lent(gpu, pieces, gpu.current) and not lent(gpu, [x], gpu.current)
    assert gpu.lib.calls.count("df11_vocab_loss") == 2
    gpu.current = 5
    head.gradient(x, targets, lse)
    assert lent(gpu, pieces, 5)
    out = head(x, targets, stream=7)
    assert lent(gpu, [*pieces, x, targets, *out], 7)
    a, c = torch.zeros(1), torch.zeros(5)
    dws = [torch.zeros(6, 16), torch.zeros(3, 16)]
    dx, got = head.gradient(x, targets, lse, a, c, dws=dws, accumulate=True, losses=out[0], stream=8)
    assert lent(gpu, [*pieces, x, targets, lse, out[0], a, c, dx, *dws], 8) and got is not None and all(p is q for p, q in zip(got, dws))


@pytest.mark.parametrize("stream", [None, 7])
def test_compressed_head(gpu, monkeypatch, stream):  # noqa: F811
    ds, status = unit([(4, 16), (3, 16)]), torch.zeros(1, dtype=torch.int32)
    ds.desc.n_tensors, ds.desc.tensor_offsets = 2, [0, 64, 112]
    decoded = []
    monkeypatch.setattr(ed, "df11_decompress_tensor",
                        lambda d, k, out, status, st: decoded.append((k, out.numel(), st)))
    head = ed.VocabLoss.from_unit(ds, [(4, 16), (3, 16)])
    head(torch.zeros(5, 16, dtype=BF16), torch.zeros(5, dtype=torch.int64), status=status, stream=stream)
    st = stream or gpu.current
    assert decoded == [(0, 64, st), (1, 48, st)]
    assert lent(gpu, [ds.stream, ds.sm, ds.gaps, ds.block_out_pos, ds.tables], st)
    assert lent(gpu, [status], 7) == (stream == 7)


def test_memory_that_calls_use_is_held(gpu):  # noqa: F811
    table, piece = torch.zeros(9, 16), torch.zeros(6, 16, dtype=BF16)
    emb, head = ed.Embedding(table), ed.VocabLoss([piece])
    memory = [StorageWeakRef(t.untyped_storage()) for t in (table, piece)]
    for t in (table, piece):
        t.data = torch.zeros_like(t)
    assert not any(m.expired() for m in memory)
    del emb, head
    assert all(m.expired() for m in memory)


def test_refusals(gpu):  # noqa: F811
    table, tokens = torch.zeros(9, 16), torch.zeros(5, dtype=torch.int64)
    emb = ed.Embedding(table)
    with pytest.raises(TypeError, match="int32 or int64"):
        emb(tokens.short())
    with pytest.raises(TypeError):
        ed.Embedding(table.double())
    with pytest.raises(ValueError):
        ed.Embedding(table.t())
    for out in (torch.zeros(4, 16), torch.zeros(5, 15), torch.zeros(1, 16).expand(5, 16), torch.zeros(16, 5).t()):
        with pytest.raises(ValueError):
            emb(tokens, out=out)
    with pytest.raises(ValueError):
        emb(tokens, torch.float16, out=torch.zeros(5, 16))
    grad = ed.embedding_gradient
    for kw in ({"dy": torch.zeros(4, 16)}, {"dy": torch.zeros(16, 5).t()}, {"dy": torch.zeros(5)},
               {"accumulate": True}, {"padding_idx": 9}, {"padding_idx": -1}, {"rows": -1},
               {"out": torch.zeros(8, 16)}, {"out": torch.zeros(9, 16), "dtype": torch.float16}):
        with pytest.raises(ValueError):
            grad(**{"tokens": tokens, "dy": torch.zeros(5, 16), "rows": 9, **kw})
    x, w, lse = torch.zeros(5, 16, dtype=BF16), torch.zeros(6, 16, dtype=BF16), torch.zeros(5)
    head = ed.VocabLoss([w])
    with pytest.raises(TypeError):
        head(x.float(), tokens)
    for bad in (x[:4], x[:, :8], torch.zeros(16, 5, dtype=BF16).t(), torch.zeros(2, 5, 16, dtype=BF16)):
        with pytest.raises(ValueError):
            head(bad, tokens)
    for pieces in ([w.float()], [w, torch.zeros(3, 8, dtype=BF16)], [w.t()]):
        with pytest.raises(ValueError):
            ed.VocabLoss(pieces)
    good = torch.zeros(6, 16)
    for kw in ({"lse": lse[:4]}, {"losses": lse[:4]}, {"lse": lse.double()}, {"loss_grad": torch.zeros(2)}, {"lse_grad": torch.zeros(4)},
               {"loss_grad": torch.zeros(1).double()}, {"accumulate": True}, {"dws": [good, good]}, {"dws": []},
               {"dws": [good[:5]]}, {"dws": [good], "dw_dtype": BF16}, {"dx": torch.zeros(4, 16)},
               {"dws": [good], "needs_dw": False}, {"dws": [good], "accumulate": True, "needs_dw": False}):
        with pytest.raises(ValueError):
            head.gradient(**{"x": x, "targets": tokens, "lse": lse, **kw})
    for kw in ({"dx_dtype": torch.float16}, {"dw_dtype": torch.float64}, {"dws": [good.half()]}):
        with pytest.raises(TypeError):
            head.gradient(**{"x": x, "targets": tokens, "lse": lse, **kw})
    assert not [c for c in gpu.lib.calls if not c.endswith("scratch_bytes")]
