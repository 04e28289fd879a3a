"""GPU tests of what an Int8Linear holds of the codes and scales it is given, and
of activations that require a gradient."""

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


@pytest.mark.parametrize("stride", [160, 128])
def test_codes_and_scales_live_alike(stride):
    """Codes on cache lines and their scales are used in place; others are laid
    out anew, and their scales with them."""
    a, b = (torch.randn(6, 20, device="cuda") for _ in range(2))
    (ca, sa), (cb, sb) = ed.quantize_int8([a, b])
    room = torch.zeros(6, stride, dtype=torch.int8, device="cuda")
    codes = room[:, :32]
    codes.copy_(ca)
    scales = sa.clone()
    x = torch.randn(3, 20, device="cuda")
    layer = ed.Int8Linear([codes], [scales], [(6, 20)])
    say(f"[gpu] Int8Linear whose codes of stride {stride} are requantised in place")
    first, = layer([x], torch.float32)
    other, = ed.Int8Linear([cb], [sb], [(6, 20)])([x], torch.float32)
    codes.copy_(cb), scales.copy_(sb)
    again, = layer([x], torch.float32)
    assert torch.equal(again, other if stride % 128 == 0 else first)
    assert not torch.equal(first, other)


def test_activations_that_require_a_gradient_are_refused():
    layer = ed.Int8Linear.from_tensors([torch.nn.Parameter(torch.randn(5, 20, device="cuda")) for _ in "ab"])
    x = torch.randn(3, 20, device="cuda")
    p = x.clone().requires_grad_()
    say("[gpu] Int8Linear of activations that require a gradient")
    want = layer([x, x])
    for xs in ([p, x], [x, p], [p * 1.0, x]):
        with pytest.raises(RuntimeError, match="gradient"):
            layer(xs)
        with torch.no_grad():
            assert all(torch.equal(y, z) for y, z in zip(layer(xs), want))
        assert all(torch.equal(y, z) for y, z in zip(layer([t.detach() for t in xs]), want))
