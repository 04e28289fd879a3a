"""GPU tests of the way from a compressed unit through AdamW and back, for
tensors as a unit or a module has them: at any offset, of any shape, parameters."""

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


def decoded(ds):
    out = torch.empty(ds.n_weights, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ed.df11_decompress_block(ds, out, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out.view(torch.int16)


@pytest.mark.parametrize("sizes", [[1], [5, 30_000, 1, 0, 4099], [70_001, 3], [8, 16, 65_536]])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_tensors_at_any_offset(sizes, shift):
    """A unit's tensors follow one another, so that after one of odd length none
    begins on 16 bytes."""
    g = torch.Generator(device="cuda").manual_seed(len(sizes))
    flat = (torch.randn(sum(sizes) + shift, device="cuda", generator=g) * 0.02).bfloat16()
    unit = flat[shift:]
    opt = ed.AdamW(list(unit.split(sizes)), [torch.ones(n, device="cuda") for n in sizes], counts=True, lr=1e-2)
    before = unit.clone()
    say(f"[gpu] AdamW step and compress, sizes {sizes} from element {shift}")
    opt.step()
    sz = opt.compressed_sizes()
    new, _ = opt.compress()
    assert int(new.desc.total_bits) == int(sz.total_bits) and new.n_weights == sum(sizes)
    assert torch.equal(decoded(new), unit.view(torch.int16)) and not torch.equal(unit, before)
    at = 0
    for k, n in enumerate(sizes):
        if at % 8 == 0:  # what a tensor is decoded alone from
            out = torch.empty(n, dtype=torch.bfloat16, device="cuda")
            ed.df11_decompress_tensor(new, k, out)
            assert torch.equal(out.view(torch.int16), unit[at:at + n].view(torch.int16)), k
        at += n


def test_parameters():
    ps = [torch.nn.Parameter((torch.randn(*s, device="cuda") * 0.02).bfloat16()) for s in ((64, 33), (7,), (128,))]
    opt = ed.AdamW(ps, [torch.ones_like(p) for p in ps], counts=True)
    say("[gpu] AdamW step and compress of parameters")
    opt.step()
    new, _ = opt.compress()
    want = torch.cat([p.detach().reshape(-1) for p in ps])
    assert torch.equal(decoded(new), want.view(torch.int16))
    assert np.isclose(int(opt.compressed_sizes().n_weights), want.numel())
