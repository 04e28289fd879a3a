"""GPU tests of tensors that are freed, or reused, while a call on another
stream is still to run.  A stream is kept busy for some ten milliseconds, the
call is queued behind, and the memory's owner lets go of it at once: new tensors
must not lie there, and the results have to be right."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import entropy_decoding_amd as ed  # noqa: E402


def say(msg):
    print(msg, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    torch.cuda.init()
    yield
    torch.cuda.synchronize()


def busy(stream, times=20):
    """Products on the stream; the caller holds the result."""
    a = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for _ in range(times):
            b = a @ a
    return a, b


def refill(sizes, kind, stream=None):
    """New tensors of the given sizes, filled, whose places are returned."""
    with torch.cuda.stream(stream or torch.cuda.current_stream()):
        held = [torch.full((n,), 85, dtype=kind, device="cuda") for n in sizes for _ in range(3)]
    return held, {t.data_ptr() for t in held}


def compressed(shapes, seed):
    g = torch.Generator().manual_seed(seed)
    ws = [(torch.randn(*s, generator=g) * 0.02).bfloat16() for s in shapes]
    tensors = [w.view(torch.int16).numpy().view(np.uint16).reshape(-1) for w in ws]
    cb = ed.df11_build_codebook(tensors)
    return ws, ed.DeviceStream(ed.df11_encode(cb, tensors), cb, "cuda")


def test_unit_freed_while_another_stream_decodes_it():
    shapes = [(512, 1024), (300, 512)]
    ws, ds = compressed(shapes, 1)
    xs = [torch.randn(20, c).bfloat16().cuda() for _, c in shapes]
    want = ed.Int8Linear.from_tensors([w.cuda() for w in ws])(xs, torch.float32)
    side = torch.cuda.Stream()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    held = busy(side)
    say("[gpu] Int8Linear.from_unit on a busy stream, the unit freed at once")
    layer = ed.Int8Linear.from_unit(ds, shapes, status, stream=side)
    arrays = [ds.stream, ds.sm, ds.gaps, ds.block_out_pos, ds.tables]
    sizes, at = [t.numel() * t.element_size() for t in arrays], {t.data_ptr() for t in arrays}
    del ds, arrays
    others, places = refill(sizes, torch.uint8)
    assert not at & places
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert all(torch.equal(a, b) for a, b in zip(layer(xs, torch.float32), want))
    del held, others


@pytest.mark.parametrize("tokens", [1, 40])
def test_layer_dropped_while_another_stream_uses_it(tokens):
    """Made on a side stream, whose memory its codes are; called on the current
    one without naming it."""
    shapes = [(512, 1024), (300, 512)]
    ws = [torch.randn(*s, device="cuda") for s in shapes]
    xs = [torch.randn(tokens, c, device="cuda").bfloat16() for _, c in shapes]
    want = ed.Int8Linear.from_tensors(ws)(xs, torch.float32)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    layer = ed.Int8Linear.from_tensors(ws, stream=side)
    torch.cuda.synchronize()
    tensors = layer._memory
    sizes = [t.untyped_storage().nbytes() for t in tensors]
    at = {t.data_ptr() for t in tensors}
    held = busy(torch.cuda.current_stream())
    say(f"[gpu] Int8Linear of {tokens} tokens on the busy current stream, the layer dropped at once")
    got = layer(xs, torch.float32)
    del layer, tensors
    others, places = refill(sizes, torch.uint8, side)
    assert not at & places
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del held, others


def test_values_on_a_stream_take_no_memory_in_use_elsewhere():
    """The current stream is busy with a buffer that is freed at once; the values
    written on another stream must not lie there."""
    n = 3 << 20
    w = torch.randn(n, device="cuda")
    opt = ed.AdamW([w], [torch.randn(n, device="cuda")], state_bits=8)
    opt.step()
    want = opt.state_values()
    side = torch.cuda.Stream()
    held = busy(torch.cuda.current_stream())
    buffers = [torch.empty(n, device="cuda") for _ in range(2)]
    for b in buffers:
        b.fill_(85.0)  # runs after the products
    at = {b.data_ptr() for b in buffers}
    say("[gpu] AdamW.state_values on a stream beside the busy current one")
    del b, buffers
    got = opt.state_values(stream=side)
    assert not at & {t.data_ptr() for part in got for t in part}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for p, q in zip(got, want) for a, b in zip(p, q))
    del held


def test_optimiser_dropped_while_another_stream_steps():
    """A step on a side stream that is current but not named."""
    n = 3 << 20
    w, g = torch.randn(n, device="cuda"), torch.randn(n, device="cuda")
    plain = ed.AdamW([w.clone()], [g])
    plain.step(max_norm=1.0)
    opt = ed.AdamW([w], [g])
    side = torch.cuda.Stream()
    held = busy(side)
    say("[gpu] AdamW step on a busy current stream, the optimiser dropped at once")
    with torch.cuda.stream(side):
        opt.step(max_norm=1.0)
    at = {t.data_ptr() for part in opt.state.values() for t in part}
    del opt
    others, places = refill([4 * n], torch.uint8)
    assert not at & places
    torch.cuda.synchronize()
    assert torch.equal(w, plain.weights[0])
    assert all((o == 85).all() for o in others)
    del held, others


def test_weights_given_other_memory():
    """As a module's to() does: a step after that must not write memory that is
    someone else's by then."""
    n = 1 << 20
    w, g = torch.nn.Parameter(torch.randn(n, device="cuda")), torch.randn(n, device="cuda")
    plain = ed.AdamW([w.detach().clone()], [g])
    opt = ed.AdamW([w], [g])
    old = w.data_ptr()
    w.data = torch.zeros(n, device="cuda")
    others, places = refill([4 * n], torch.uint8)
    assert old not in places
    say("[gpu] AdamW step after its weight was given other memory")
    opt.step(), plain.step()
    torch.cuda.synchronize()
    assert all((o == 85).all() for o in others) and not w.any()
    assert all(torch.equal(a, b) for a, b in zip(opt.state["m"], plain.state["m"]))
