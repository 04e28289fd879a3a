"""Which tensors the operators' binding lends to a stream, and what it makes on
one.  The library, the streams and the device are stand-ins here: the tensors
lie in host memory, and what would be recorded for a stream is written down."""

import contextlib
import types

import pytest

import entropy_decoding_amd as ed

torch = pytest.importorskip("torch")

from torch.multiprocessing.reductions import StorageWeakRef  # noqa: E402


class Fake:
    """Stands in for the library: every function succeeds, and is written down."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 1 << 10 if name.endswith("scratch_bytes") else ed.DF11_OK
        return call


@pytest.fixture
def gpu(monkeypatch):
    """lent: the (address, stream) pairs recorded; current: the current stream;
    inside: the stream whose guard is entered."""
    s = types.SimpleNamespace(lent=set(), current=1, inside=None, lib=Fake())

    @contextlib.contextmanager
    def guard(stream):
        s.inside = stream
        yield
        s.inside = None

    def on(device, stream):
        st = s.current if stream is None else stream
        return guard(st), st

    monkeypatch.setattr(ed, "LIB", s.lib)
    monkeypatch.setattr(ed, "_on", on)
    monkeypatch.setattr(ed, "_stream_of", lambda device, stream: stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: s.current)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: None)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, stream: s.lent.add((t.data_ptr(), stream)), raising=False)
    return s


def unit(shapes):
    """Something like a DeviceStream of a BF16 unit."""
    n = sum(r * c for r, c in shapes)
    return types.SimpleNamespace(
        stream=torch.zeros(64, dtype=torch.uint8), sm=torch.zeros(n, dtype=torch.uint8),
        gaps=torch.zeros(16, dtype=torch.uint8), block_out_pos=torch.zeros(16, dtype=torch.int32),
        tables=torch.zeros(64, dtype=torch.uint8), n_weights=n, desc=types.SimpleNamespace(format=0))


@pytest.mark.parametrize("stream", [None, 7])
def test_a_unit_is_lent_to_the_stream_that_decodes_it(gpu, monkeypatch, stream):
    ds, status = unit([(4, 32), (3, 16)]), torch.zeros(1, dtype=torch.int32)
    monkeypatch.setattr(ed, "df11_decompress_block", lambda *a: None)
    ed.Int8Linear.from_unit(ds, [(4, 32), (3, 16)], status, stream)
    want = {(t.data_ptr(), stream) for t in (ds.stream, ds.sm, ds.gaps, ds.block_out_pos, ds.tables, status)}
    assert want <= gpu.lent if stream is not None else not gpu.lent


def test_codes_are_lent_to_whatever_stream_multiplies_with_them(gpu):
    """Made on stream 7, used on the current one without naming it, and on another."""
    ws = [torch.zeros(4, 32), torch.zeros(3, 32)]
    layer = ed.Int8Linear.from_tensors(ws, stream=7)
    held = [t.data_ptr() for t in layer._memory]
    assert len(held) == 4
    x = torch.zeros(2, 32)
    layer([x, x], stream=7)
    for _ in range(2):
        layer([x, x])
    assert {(p, gpu.current) for p in held} <= gpu.lent
    assert (x.data_ptr(), gpu.current) not in gpu.lent  # the caller's, on the caller's stream
    gpu.current = 5
    layer([x, x])
    assert {(p, 5) for p in held} <= gpu.lent


def test_codes_given_to_a_layer_are_lent(gpu):
    (codes, scales), = ed.quantize_int8([torch.zeros(4, 32)])
    layer = ed.Int8Linear([codes], [scales], [(4, 32)])
    for stream in (7, None):  # they may have been made on another than the current one
        layer([torch.zeros(2, 32)], stream=stream)
        assert {(t.data_ptr(), stream or gpu.current) for t in layer._memory} <= gpu.lent


def optimiser(bits=8, sizes=(300, 5), **kw):
    ws = [torch.zeros(n) for n in sizes]
    return ed.AdamW(ws, [torch.zeros(n) for n in sizes], state_bits=bits, **kw)


@pytest.fixture
def host_tensors(monkeypatch):
    """AdamW takes tensors of the host."""
    monkeypatch.setattr(ed, "_same", lambda tensors, *a: list(tensors))


def test_values_are_made_on_the_stream_that_writes_them(gpu, host_tensors, monkeypatch):
    opt = optimiser()
    inside, empty = [], torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: (inside.append(gpu.inside), empty(*a, **kw))[1])
    for stream in (7, None):
        m, v = opt.state_values(stream=stream)
        assert [t.numel() for t in m] == [t.numel() for t in v] == [300, 5]
        assert inside == [7 if stream else gpu.current] * 4
        inside.clear()


def test_compressing_is_done_on_the_optimisers_device(gpu, host_tensors, monkeypatch):
    opt = optimiser()
    entered, at = [], []

    @contextlib.contextmanager
    def device(d):
        entered.append(d)
        yield
        entered.pop()

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(ed, "encode_on_device",
                        lambda tensors, stream=None: at.append((list(entered), tensors, stream)))
    for stream in (None, 7):
        opt.compress(stream)
        assert at.pop() == ([opt.device], opt.weights, stream) and not entered


@pytest.mark.parametrize("kind", [torch.float16, torch.float64])
def test_values_are_float32_whatever_torchs_default(gpu, host_tensors, kind):
    opt = optimiser()
    before = torch.get_default_dtype()
    torch.set_default_dtype(kind)
    try:
        values = opt.state_values()
    finally:
        torch.set_default_dtype(before)
    assert {t.dtype for part in values for t in part} == {torch.float32}


def test_an_optimisers_memory_is_lent_to_every_stream_that_steps(gpu, host_tensors):
    """Its states are made by the constructor: whoever drops it on another stream
    than that has no other hand on them."""
    opt = optimiser(counts=True)
    own = [t.data_ptr() for part in opt.state.values() for t in part]
    own += [opt.counts.data_ptr(), opt._skipped.data_ptr()]
    for current in (1, 5):
        gpu.current = current
        opt.step(max_norm=1.0)
        assert {(p, current) for p in own} <= gpu.lent
    opt = optimiser(device_step=True)
    gpu.current = 6
    opt.state_values()
    assert {(t.data_ptr(), 6) for part in opt.state.values() for t in part} <= gpu.lent
    opt.step(stream=9)
    given = [*opt.weights, *opt.grads, opt.d_step]
    assert {(t.data_ptr(), 9) for t in given} <= gpu.lent
    others = [torch.zeros(n) for n in (300, 5)]
    opt.set_grads(others)
    opt.step(stream=9)
    assert {(t.data_ptr(), 9) for t in others} <= gpu.lent


def test_views_of_one_storage_are_lent_with_it(gpu, host_tensors, monkeypatch):
    """Recording one tensor records the memory of all that share it."""
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, stream: gpu.lent.add((t.untyped_storage().data_ptr(), stream)))
    flat = torch.zeros(900)
    opt = ed.AdamW(list(flat.split([300, 599, 1])), [torch.zeros(n) for n in (300, 599, 1)])
    gpu.current = 5
    opt.step()
    want = [flat, *opt.state["m"], *opt.state["v"], opt._skipped]
    assert {(t.untyped_storage().data_ptr(), gpu.current) for t in want} <= gpu.lent


def test_memory_that_calls_use_is_held(gpu, host_tensors):
    """Not only the tensors, which may be given other memory (t.data = ..., as a
    module's to() does): calls go on with the addresses that were given."""
    opt = optimiser(masters=[torch.zeros(n) for n in (300, 5)])
    room, scales = torch.zeros(8 * 128, dtype=torch.int8), torch.zeros(4)
    codes = room[-room.data_ptr() % 128:][:4 * 128].view(4, 128)
    layer = ed.Int8Linear([codes], [scales], [(4, 128)])  # on cache lines: not copied
    given = [*opt.weights, *opt.masters, *opt.grads, *opt.state["m"], room, scales]
    del codes
    memory = [StorageWeakRef(t.untyped_storage()) for t in given]
    for t in given:
        t.data = torch.zeros_like(t)
    assert not any(m.expired() for m in memory)
    opt.set_grads([torch.zeros(n) for n in (300, 5)])
    assert sum(m.expired() for m in memory) == 2  # the gradients before
    del opt, layer
    assert all(m.expired() for m in memory)
