"""GPU tests of what an AdamW object counts, refuses and tells torch, around
steps that are skipped, refused or never made."""

import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import entropy_decoding_amd as ed  # noqa: E402

BETAS = (0.9, 0.95)


def say(msg):
    print(msg, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    torch.cuda.init()
    yield
    torch.cuda.synchronize()


def make(sizes, bits=32, seed=0, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ws = [(torch.randn(n, device="cuda", generator=g) * 0.02).bfloat16() for n in sizes]
    gs = [torch.randn(n, device="cuda", generator=g) * 1e-3 for n in sizes]
    return ed.AdamW(ws, gs, masters=[w.float() for w in ws], state_bits=bits, lr=1e-2, betas=BETAS, **kw)


def parts(opt):
    return [opt.weights, opt.masters, *opt.state.values()]


def equal(a, b):
    torch.cuda.synchronize()
    return all(torch.equal(x, y) for p, q in zip(parts(a), parts(b)) for x, y in zip(p, q))


def skip(opt, how):
    if how == "factor":
        opt.step(grad_factor=torch.tensor([math.nan], device="cuda"))
        return
    grads = opt.grads
    opt.set_grads([torch.full_like(x, math.inf) for x in grads])
    opt.step(max_norm=0.01)
    opt.set_grads(grads)


def go(opt, how):
    if how == "factor":
        opt.step(grad_factor=torch.tensor([0.5], device="cuda"))
    else:
        opt.step(max_norm=0.01)


@pytest.mark.parametrize("sizes", [[300, 1025], [7] * 75, [500] * 36 + [0, 0]])
@pytest.mark.parametrize("how", ["factor", "norm"])
@pytest.mark.parametrize("device_step", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
def test_skipped_steps_are_not_counted(bits, device_step, how, sizes):
    """The updates after them are those of an optimiser that never met them."""
    a = make(sizes, bits, device_step=device_step)
    b = make(sizes, bits, device_step=True)
    say(f"[gpu] AdamW skipped steps bits={bits} device_step={device_step} {how} {len(sizes)} tensors")
    skip(a, how)
    assert equal(a, b)
    for made, skips in ((1, 2), (2, 0), (3, 1)):
        go(a, how), go(b, how)
        assert equal(a, b), made
        for _ in range(skips):
            skip(a, how)
        assert equal(a, b), made
    a.step(), b.step()  # and without a factor
    assert equal(a, b)
    assert a.steps == b.steps == 4 and int(b.d_step) == 4
    if device_step:
        assert int(a.d_step) == 4


@pytest.mark.parametrize("device_step", [False, True])
def test_skipped_steps_of_a_replayed_graph(device_step):
    """With the number on the device a replay that is skipped is not counted
    either; without it every replay is of the number that was captured."""
    a, b = (make([300, 70_000, 5], 8, device_step=device_step) for _ in range(2))
    say(f"[gpu] AdamW captured, some replays skipped, device_step={device_step}")
    for o in (a, b):
        go(o, "norm"), skip(o, "norm")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = a.step(max_norm=0.01)
    number = 2 if device_step else 3  # the host's does not know of the skipped one
    kept = [x.clone() for x in a.grads]
    for i, finite in enumerate([True, False, False, True, True, False, True]):
        for x, y in zip(a.grads, kept):
            x.copy_(y) if finite else x.fill_(math.nan)
        if finite:
            other = ed.AdamW(b.weights, b.grads, masters=b.masters, state_bits=8, state=b.state, lr=1e-2,
                             betas=BETAS, step=number - 1, device_step=device_step)
            want = other.step(max_norm=0.01)
            number += device_step
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert equal(a, b), i
        assert torch.equal(norm, want) if finite else not torch.isfinite(norm).any()
    if device_step:
        assert int(a.d_step) == number - 1 == a.steps


def test_steps_can_be_set():
    """As where a run goes on from saved states."""
    a, b = make([300], step=7), make([300])
    say("[gpu] AdamW.steps set")
    skip(b, "factor"), go(b, "factor")
    assert b.steps == 1
    for x, y in zip(parts(b), parts(a)):
        for p, q in zip(x, y):
            p.copy_(q)
    b.steps = 7
    go(a, "factor"), go(b, "factor")
    assert a.steps == b.steps == 8 and equal(a, b)


@pytest.mark.parametrize("device_step", [False, True])
def test_a_refused_step_is_not_counted(device_step):
    a, b = (make([300, 1025], device_step=device_step) for _ in range(2))
    say(f"[gpu] AdamW refused steps device_step={device_step}")
    for bad in (-1.0, math.nan):
        with pytest.raises(ed.Df11Error):
            a.step(lr=bad)
        with pytest.raises(ed.Df11Error):
            a.step(lr=bad, max_norm=1.0)
    with pytest.raises(ed.Df11Error):
        a.step(max_norm=-1.0)
    a.step(), b.step()
    assert equal(a, b) and a.steps == b.steps == 1
    if device_step:
        assert int(a.d_step) == 1


@pytest.mark.parametrize("kind", [torch.float64, torch.float16, torch.int8])
def test_refused_gradients_leave_the_old_ones(kind):
    sizes = [300, 1025]
    a, b = (make(sizes) for _ in range(2))
    say(f"[gpu] AdamW.set_grads of {kind}")
    with pytest.raises((TypeError, ed.Df11Error)):
        a.set_grads([torch.zeros(n, device="cuda").to(kind) for n in sizes])
    assert a.grads[0].dtype == torch.float32
    a.step(), b.step()
    assert equal(a, b)


def test_half_precision_is_refused_at_once():
    w = torch.zeros(10, dtype=torch.float16, device="cuda")
    say("[gpu] AdamW of float16")
    for pair in ((w, w.float()), (w.float(), w)):
        with pytest.raises(ed.Df11Error, match="float16"):
            ed.AdamW([pair[0]], [pair[1]])


def test_sizes_before_a_step_are_refused():
    say("[gpu] AdamW.compressed_sizes before a step")
    for opt in (make([300], counts=True, step=10), make([300], counts=True), make([300])):
        with pytest.raises(ValueError, match="counts"):
            opt.compressed_sizes()


def test_torch_sees_that_weights_change():
    """A graph that saved a weight must not go backward with the new one."""
    w = torch.randn(500, device="cuda", requires_grad=True)
    flat = torch.randn(900, device="cuda").bfloat16()
    views = list(flat.split([400, 500]))
    masters = [v.float() for v in views]
    one = ed.AdamW([w], [torch.ones(500, device="cuda")])
    two = ed.AdamW(views, [torch.ones_like(v) for v in views], masters=masters)
    say("[gpu] AdamW and torch's versions")
    loss = (w * w).sum()
    before = [t._version for t in (flat, *masters)]
    one.step(), two.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    assert all(t._version > v for t, v in zip((flat, *masters), before))
    with torch.inference_mode():  # such tensors have no version
        t = torch.randn(10, device="cuda")
        ed.AdamW([t], [torch.ones(10, device="cuda")]).step()


def test_numbers_of_steps_below_zero_are_refused():
    w, g = torch.zeros(10, device="cuda"), torch.zeros(10, device="cuda")
    say("[gpu] AdamW(step=-5)")
    for step in (-1, -5):
        with pytest.raises(ValueError, match="step"):
            ed.AdamW([w], [g], step=step)


def test_buffers_that_overlap_are_refused():
    """Whatever a step writes."""
    w = [torch.zeros(300, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    g = [torch.zeros(300, device="cuda") for _ in range(2)]
    flat = torch.zeros(900, device="cuda")
    zeros = lambda: [torch.zeros(300, device="cuda") for _ in range(2)]  # noqa: E731
    say("[gpu] AdamW of masters and states that overlap")
    for bad in ([flat[:300], flat[:300]], [flat[:300], flat[299:599]]):
        with pytest.raises(ValueError, match="overlap"):
            ed.AdamW(w, g, masters=bad)
        for name in "mv":
            with pytest.raises(ValueError, match="overlap"):
                ed.AdamW(w, g, state={"m": zeros(), "v": zeros(), name: bad})
    same = zeros()
    with pytest.raises(ValueError, match="overlap"):
        ed.AdamW(w, g, state={"m": same, "v": same})
    with pytest.raises(ValueError, match="overlap"):
        ed.AdamW(zeros(), g, state={"m": [flat[:300], flat[300:600]], "v": [flat[600:], flat[:300]]})
    f = zeros()
    with pytest.raises(ValueError, match="overlap"):
        ed.AdamW(f, g, state={"m": f, "v": zeros()})
    ed.AdamW(w, g, masters=[flat[:300], flat[300:600]]).step()  # side by side


@pytest.mark.parametrize("exponent", [-96, 0, 94])
def test_roots_of_every_mantissa(exponent):
    """The step's roots are correctly rounded: all 2^24 values of two binades, in
    the middle and at the ends of where they are formed without sqrtf.  Betas of
    1/2, late steps, no gradient and lr 1 make the new weight m / (2 sqrt(v / 2)) with
    one rounding for the root and one for the quotient (eps vanishes beside the
    root).  The quotient is just below 2, where its last place is the finest beside
    the root's: a root that is one off shows."""
    bits = np.arange(2 ** 24, dtype=np.uint32) + np.uint32((127 + exponent) << 23)
    v = bits.view(np.float32)
    r = np.sqrt(v)
    m = r * np.float32(1.999)
    n = v.size
    w = torch.zeros(n, device="cuda")
    state = {"m": [torch.from_numpy(m * np.float32(2)).cuda()], "v": [torch.from_numpy(v * np.float32(2)).cuda()]}
    opt = ed.AdamW([w], [torch.zeros(n, device="cuda")], state=state, lr=1.0, betas=(0.5, 0.5), eps=1e-30,
                   weight_decay=0.0, step=2999)
    say(f"[gpu] AdamW roots of [2^{exponent}, 2^{exponent + 2})")
    opt.step()
    torch.cuda.synchronize()
    assert np.array_equal(opt.state["v"][0].cpu().numpy(), v) and np.array_equal(opt.state["m"][0].cpu().numpy(), m)
    assert np.array_equal(w.cpu().numpy(), -(m / r))
    for other in (np.inf, -np.inf):  # one off either way would have been seen, but for 8 values
        assert (m / np.nextafter(r, np.float32(other)) == m / r).sum() <= 8
