"""GPU tests of the AdamW step (df11_adamw_step), the gradient norm and the
reader of 8-bit states.

Two references.  The step's operations in float32, in the documented order,
each rounded (numpy): the kernel has to give the same bits.  And the formulas
in float64, with a bound that counts the roundings (u = 2^-24 is half a step of
float32): the factors b1, 1 - b1, ... are rounded once, so

  m: |dm| <= 5u (|b1 m| + |c1 f g|)            factor, product (twice with f), sum
  v: |dv| <= 7u v                              as m, with g twice; no cancellation
  d = sqrt(v) root + eps: |dd| <= 9u d         half of dv, the root, 3 factors, product, sum
  w: |dw| <= 2u |w keep| + size (|dm| / d + 12u |m| / d) + u |w'|

plus, for BF16 weights, half a step (2^-8 of the value).  8-bit states of value
S c^2 (m, or sqrt(v)) lie at most S (c + 1/4) from the value: |y - c| <= 1/2
with y = sqrt(value / S) gives |y^2 - c^2| <= (2c + 1/2) / 2; the arithmetic
before adds 20u of S 255^2 at most.
"""

import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import entropy_decoding_amd as ed  # noqa: E402

U = 2.0 ** -24
LR, BETAS, EPS = 1e-3, (0.9, 0.95), 1e-8
f32 = np.float32


def say(msg):
    print(msg, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    torch.cuda.init()
    yield
    torch.cuda.synchronize()


def to_bf16(a):
    """float32 to BF16 bits, to nearest, ties to even (no NaN)."""
    u = np.ascontiguousarray(a, dtype=f32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def from_bf16(b):
    return (b.astype(np.uint32) << 16).view(f32)


class Case:
    """Tensors at odd offsets of flat buffers with guards around them, on the
    host and on the device."""

    GUARD = 5

    def __init__(self, sizes, w="bf16", g="bf16", master=False, bits=32, seed=0, grads=None,
                 zero_state=False):
        rng = np.random.default_rng(seed)
        self.sizes, self.w_kind, self.g_kind, self.bits = sizes, w, g, bits
        self.dev, self.host = {}, {}
        blocks = [-(-s // 256) for s in sizes]
        each = [rng.standard_normal(s).astype(f32) * f32(0.02) for s in sizes]
        self._put("w", [to_bf16(x) if w == "bf16" else x for x in each])
        self._put("master", each)
        gs = grads or [(rng.standard_normal(s) * 1e-3 * np.exp(rng.standard_normal(s))).astype(f32)
                       for s in sizes]
        self._put("g", [to_bf16(x) if g == "bf16" else x for x in gs])
        if bits == 32:
            self._put("m", [(rng.standard_normal(s) * 3e-4).astype(f32) * (not zero_state) for s in sizes])
            self._put("v", [((1e-3 * rng.random(s)) ** 2).astype(f32) * (not zero_state) for s in sizes])
        else:
            on = 0 if zero_state else 1
            self._put("m", [rng.integers(-127, 128, s).astype(np.int8) * np.int8(on) for s in sizes])
            self._put("v", [rng.integers(0, 256, s).astype(np.uint8) * np.uint8(on) for s in sizes])
            self._put("m_scale", [(rng.random(b) * 1e-7 * on).astype(f32) for b in blocks])
            self._put("v_scale", [(rng.random(b) * 3e-8 * on).astype(f32) for b in blocks])
        self.has_master = master
        self.decay = [0.1 if k % 2 else 0.0 for k in range(len(sizes))]
        self.lr_scale = [1.0 if k % 3 else 0.5 for k in range(len(sizes))]

    def _put(self, name, arrays):
        g = self.GUARD
        flat, at = [], []
        n = g
        for a in arrays:
            at.append(n)
            n += a.size + g
        flat = np.full(n, 77, dtype=arrays[0].dtype)
        for a, o in zip(arrays, at):
            flat[o:o + a.size] = a
        kind = {np.dtype(np.uint16): torch.bfloat16}.get(flat.dtype)
        t = torch.from_numpy(flat.view(np.int16) if kind else flat.copy()).cuda()
        t = t.view(torch.bfloat16) if kind else t
        self.host[name] = [a.copy() for a in arrays]
        self.dev[name] = (t, flat, at, [t[o:o + a.size] for a, o in zip(arrays, at)])

    def views(self, name):
        return self.dev[name][3]

    def opt(self, **kw):
        names = ["m", "v"] + (["m_scale", "v_scale"] if self.bits == 8 else [])
        return ed.AdamW(self.views("w"), self.views("g"),
                        masters=self.views("master") if self.has_master else None,
                        state_bits=self.bits, state={k: self.views(k) for k in names}, lr=LR,
                        betas=BETAS, eps=EPS, weight_decay=self.decay, lr_scale=self.lr_scale,
                        **{"step": 4, **kw})

    def got(self, name):
        """The tensors after a step; fails if a guard was written."""
        t, flat, at, views = self.dev[name]
        now = (t.view(torch.int16) if t.dtype == torch.bfloat16 else t).cpu().numpy().view(flat.dtype)
        inside = np.zeros(flat.size, bool)
        for o, v in zip(at, views):
            inside[o:o + v.numel()] = True
        assert np.array_equal(now[~inside], flat[~inside]), f"{name}: written outside of a tensor"
        return [now[o:o + v.numel()].copy() for o, v in zip(at, views)]


def blockwise(s, x):
    return np.repeat(x, 256)[:s]


def step32(case, k, t, factor=None):
    """One tensor's step in float32, each operation rounded."""
    h = case.host
    s = case.sizes[k]
    b1, b2 = BETAS
    g = from_bf16(h["g"][k]) if case.g_kind == "bf16" else h["g"][k]
    x = (h["master"][k] if case.has_master else
         from_bf16(h["w"][k]) if case.w_kind == "bf16" else h["w"][k])
    if case.bits == 32:
        m, v = h["m"][k], h["v"][k]
    else:
        c = h["m"][k].astype(np.int32)
        m = blockwise(s, h["m_scale"][k]) * (c * np.abs(c)).astype(f32)
        c = h["v"][k].astype(np.int32)
        r = blockwise(s, h["v_scale"][k]) * (c * c).astype(f32)
        v = r * r
    with np.errstate(all="ignore"):
        if factor is not None:
            g = g * f32(factor)
        m = m * f32(b1) + g * f32(1 - b1)
        v = v * f32(b2) + (g * f32(1 - b2)) * g
        r = np.sqrt(v)
        u = m / (r * f32(1 / math.sqrt(1 - b2 ** t)) + f32(EPS))
        lr = LR * case.lr_scale[k]
        x = x * f32(1 - lr * case.decay[k]) - u * f32(lr / (1 - b1 ** t))
        out = {"master": x, "w": to_bf16(x) if case.w_kind == "bf16" else x}
        if case.bits == 32:
            return dict(out, m=m, v=v)

        def hold(x, most, tiny):
            top = np.array([np.abs(x[i:i + 256]).max() for i in range(0, s, 256)], dtype=f32)
            scale = np.where(top < f32(tiny), f32(0), top * (f32(1) / f32(most * most)))
            inv = np.where(scale > 0, f32(1) / scale, f32(0)).astype(f32)
            code = np.minimum(np.rint(np.sqrt(np.abs(x) * blockwise(s, inv))), f32(most))
            return scale.astype(f32), code

        ms, c = hold(m, 127, 2.0 ** -100)
        vs, d = hold(r, 255, 2.0 ** -149)
        d = np.where(r > 0, np.maximum(d, 1), 0)
        return dict(out, m=np.where(m < 0, -c, c).astype(np.int8), v=d.astype(np.uint8), m_scale=ms,
                    v_scale=vs)


def step64(case, k, t, factor=1.0):
    """The step in float64 from the same held values, and the bounds above."""
    h, s = case.host, case.sizes[k]
    b1, b2 = BETAS
    g = (from_bf16(h["g"][k]) if case.g_kind == "bf16" else h["g"][k]).astype(np.float64) * factor
    w = (h["master"][k] if case.has_master else
         from_bf16(h["w"][k]) if case.w_kind == "bf16" else h["w"][k]).astype(np.float64)
    if case.bits == 32:
        m0, v0 = h["m"][k].astype(np.float64), h["v"][k].astype(np.float64)
    else:
        c = h["m"][k].astype(np.float64)
        m0 = blockwise(s, h["m_scale"][k]).astype(np.float64) * c * np.abs(c)
        v0 = (blockwise(s, h["v_scale"][k]).astype(np.float64) * h["v"][k].astype(np.float64) ** 2) ** 2
    m = b1 * m0 + (1 - b1) * g
    v = b2 * v0 + (1 - b2) * g * g
    lr = LR * case.lr_scale[k]
    size, keep = lr / (1 - b1 ** t), 1 - lr * case.decay[k]
    d = np.sqrt(v) / math.sqrt(1 - b2 ** t) + EPS
    new = w * keep - size * m / d
    more = 0 if case.bits == 32 else 3  # roundings of the decoded states
    dm = (5 + more) * U * (np.abs(b1 * m0) + np.abs((1 - b1) * g))
    dw = (2 * U * np.abs(w * keep) + size * (dm / d + (12 + more) * U * np.abs(m) / d)
          + U * np.abs(new))
    return m, v, new, dm, (7 + more) * U * v, dw


KINDS = [("bf16", "bf16", False, 32), ("bf16", "f32", False, 32), ("bf16", "bf16", True, 32),
         ("bf16", "f32", True, 32), ("f32", "f32", False, 32), ("f32", "bf16", False, 32),
         ("bf16", "bf16", False, 8), ("bf16", "f32", False, 8), ("bf16", "bf16", True, 8),
         ("bf16", "f32", True, 8), ("f32", "f32", False, 8), ("f32", "bf16", False, 8)]
SIZES = [1, 3, 255, 0, 256, 257, 1000, 1023, 1024, 1025, 4099, 20001]


def same(case, want, names):
    for name in names:
        for k, (a, b) in enumerate(zip(case.got(name), [x[name] for x in want])):
            bad = a.view(np.uint8) != b.view(np.uint8)
            assert not bad.any(), (name, k, case.sizes[k], a[:4], b[:4])


def names_of(case):
    return (["w", "m", "v"] + (["m_scale", "v_scale"] if case.bits == 8 else []) +
            (["master"] if case.has_master else []))


@pytest.mark.parametrize("w,g,master,bits", KINDS)
def test_step_gives_the_bits_of_rounded_float32(w, g, master, bits):
    case = Case(SIZES, w, g, master, bits, seed=1)
    opt = case.opt()
    say(f"[gpu] df11_adamw_step w={w} g={g} master={master} bits={bits} sizes={SIZES}")
    opt.step()
    torch.cuda.synchronize()
    want = [step32(case, k, 5) for k in range(len(SIZES))]
    same(case, want, names_of(case))
    if not master:  # the masters are not this call's
        assert all(np.array_equal(a, b) for a, b in zip(case.got("master"), case.host["master"]))


@pytest.mark.parametrize("w,g,master,bits", KINDS)
def test_step_is_near_float64(w, g, master, bits):
    case = Case([777, 4097], w, g, master, bits, seed=2)
    say(f"[gpu] df11_adamw_step against float64 w={w} g={g} master={master} bits={bits}")
    case.opt().step()
    torch.cuda.synchronize()
    for k, s in enumerate(case.sizes):
        m, v, new, dm, dv, dw = step64(case, k, 5)
        got = case.got("w")[k]
        got = from_bf16(got) if w == "bf16" else got
        half = np.abs(new) * 2.0 ** -8 if w == "bf16" else 0.0
        assert (np.abs(got - new) <= (dw + half) * 1.001).all()
        if master:
            assert (np.abs(case.got("master")[k] - new) <= dw * 1.001).all()
        if bits == 32:
            assert (np.abs(case.got("m")[k] - m) <= dm * 1.001).all()
            assert (np.abs(case.got("v")[k] - v) <= dv * 1.001).all()
            continue
        for name, value in (("m", m), ("v", np.sqrt(v))):
            c = case.got(name)[k].astype(np.float64)
            sc = blockwise(s, case.got(name + "_scale")[k]).astype(np.float64)
            held = sc * c * np.abs(c)
            assert (np.abs(held - value) <= sc * (np.abs(c) + 0.25 + 20 * U * 255 ** 2) * 1.001).all()


def test_many_tensors_and_the_same_step_twice():
    """75 tensors are three launches; a second step goes on from the first."""
    rng = np.random.default_rng(3)
    case = Case([int(x) for x in rng.integers(0, 3000, 75)], bits=8, seed=3)
    opt = case.opt()
    say("[gpu] df11_adamw_step 75 tensors, two steps")
    for t in (5, 6):
        opt.step()
        torch.cuda.synchronize()
        want = [step32(case, k, t) for k in range(75)]
        same(case, want, names_of(case))
        for name in names_of(case):
            case.host[name] = [x[name] for x in want]


def test_large_tensor_chunks():
    """Several chunks of several iterations, and a ragged end."""
    case = Case([8_500_000 + 13, 2 ** 20], "bf16", "bf16", True, 8, seed=4)
    say("[gpu] df11_adamw_step 8.5 M elements")
    case.opt().step()
    torch.cuda.synchronize()
    same(case, [step32(case, k, 5) for k in range(2)], names_of(case))


@pytest.mark.parametrize("bits", [32, 8])
def test_more_than_2_32_elements(bits):
    """A tensor of 2^32 + 12345 elements beside a small one: the places around
    2^31, 2^32 and the end get what the same elements get in the small tensor."""
    n, blocks = 2 ** 32 + 12345, 16
    small = blocks * 256
    g = torch.Generator(device="cuda").manual_seed(5)
    w = torch.randn(small, device="cuda", generator=g).mul_(0.02).bfloat16()
    gr = torch.randn(small, device="cuda", generator=g).mul_(1e-3).bfloat16()
    big_w, big_g = (torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    places = [0, 2 ** 31 - 2048, 2 ** 32 - 2048, (n - small) // 256 * 256]
    for p in places:
        big_w[p:p + small], big_g[p:p + small] = w, gr
    opt = ed.AdamW([big_w, w], [big_g, gr], state_bits=bits, lr=1e-2, betas=BETAS)
    say(f"[gpu] df11_adamw_step of {n} elements, bits={bits}")
    norm = opt.step(max_norm=1e-2)
    torch.cuda.synchronize()
    want = math.sqrt((len(places) + 1) * float(gr.double().square().sum()))
    assert abs(float(norm[0]) - want) <= want * 1.01 * U
    for p in places:
        assert torch.equal(big_w[p:p + small], w), p
        for name in ("m", "v"):
            big, part = opt.state[name]
            assert torch.equal(big[p:p + small], part), (p, name)
    assert not big_w[small:2 ** 31 - 2048].any() and not big_w[2 ** 32 + small:places[-1]].any()
    assert not big_w[places[-1] + small:].any()


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_states_and_zero_gradients(bits):
    grads = [np.zeros(600, f32), np.concatenate([np.zeros(300, f32), np.full(300, 1e-4, f32)])]
    case = Case([600, 600], "bf16", "f32", True, bits, seed=5, grads=grads, zero_state=True)
    say(f"[gpu] df11_adamw_step from zeros bits={bits}")
    case.opt(step=0).step()
    torch.cuda.synchronize()
    same(case, [step32(case, k, 1) for k in range(2)], names_of(case))


def test_8bit_code_of_a_small_v_is_never_zero():
    g = np.full(256, 1e-7, f32)
    g[17] = 1.0
    case = Case([256], "bf16", "f32", True, 8, seed=6, grads=[g], zero_state=True)
    say("[gpu] df11_adamw_step 8-bit, v of very different sizes")
    case.opt(step=0).step()
    torch.cuda.synchronize()
    assert case.got("v")[0].min() == 1 and case.got("v")[0].max() == 255
    same(case, [step32(case, 0, 1)], names_of(case))


@pytest.mark.parametrize("value", [1e-30, 1e-42, 1e15])
def test_8bit_extreme_sizes(value):
    rng = np.random.default_rng(7)
    g = (rng.standard_normal(700) * value).astype(f32)
    case = Case([700], "f32", "f32", False, 8, seed=7, grads=[g], zero_state=True)
    say(f"[gpu] df11_adamw_step 8-bit, gradients about {value}")
    case.opt(step=0).step()
    torch.cuda.synchronize()
    same(case, [step32(case, 0, 1)], names_of(case))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf, 1e25])
@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_that_are_not_finite(value, bits):
    """They reach their own element; in 8 bits the states of its block."""
    rng = np.random.default_rng(8)
    g = (rng.standard_normal(1000) * 1e-3).astype(f32)
    g[300] = value
    case = Case([1000], "f32", "f32", False, bits, seed=8, grads=[g])
    say(f"[gpu] df11_adamw_step bits={bits} with a gradient of {value}")
    case.opt().step()
    torch.cuda.synchronize()
    want = step32(case, 0, 5)
    got = case.got("w")[0]
    rest = np.arange(1000) != 300
    assert np.array_equal(got[rest], want["w"][rest])
    assert np.array_equal(np.isnan(got), np.isnan(want["w"]))
    if bits == 32:
        for name in ("m", "v"):
            assert np.array_equal(case.got(name)[0][rest], want[name][rest])
            assert not np.isfinite(case.got(name)[0][300]) or value == 1e25
        return
    ms, vs = case.got("m_scale")[0], case.got("v_scale")[0]
    m_bad = not math.isclose(value, 1e25)  # a finite m beside a v that overflowed
    assert list(np.isnan(ms)) == [False, m_bad, False, False]
    assert list(np.isnan(vs)) == [False, True, False, False]
    assert not case.got("v")[0][256:512].any()
    out = np.r_[0:256, 512:1000]
    assert np.array_equal(case.got("m")[0][out], want["m"][out])
    assert np.array_equal(case.got("v")[0][out], want["v"][out])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("factor", [0.25, 0.0, math.nan, math.inf, -math.inf])
def test_gradient_factor(factor, bits):
    case = Case([300, 1025], "bf16", "bf16", True, bits, seed=9)
    opt = case.opt(counts=True)
    say(f"[gpu] df11_adamw_step factor={factor} bits={bits}")
    opt.step(grad_factor=torch.tensor([factor], dtype=torch.float32, device="cuda"))
    torch.cuda.synchronize()
    if math.isfinite(factor):
        same(case, [step32(case, k, 5, factor) for k in range(2)], names_of(case))
    else:  # nothing changes, and the histogram is of the weights that are there
        same(case, [{n: case.host[n][k] for n in names_of(case)} for k in range(2)], names_of(case))
    for k, w in enumerate(case.got("w")):
        want = np.bincount((w.astype(np.int64) >> 7) & 0xFF, minlength=256)
        assert np.array_equal(opt.counts[k].cpu().numpy(), want)


@pytest.mark.parametrize("master,bits", [(False, 32), (True, 8)])
def test_counts(master, bits):
    case = Case([1, 257, 0, 9000, 300_001], "bf16", "bf16", master, bits, seed=10)
    opt = case.opt(counts=True)
    opt.counts.fill_(123)  # the call clears them
    say(f"[gpu] df11_adamw_step counts master={master} bits={bits}")
    for _ in range(2):
        opt.step()
        torch.cuda.synchronize()
        for k, w in enumerate(case.got("w")):
            want = np.bincount((w.astype(np.int64) >> 7) & 0xFF, minlength=256)
            assert np.array_equal(opt.counts[k].cpu().numpy(), want), k
            if w.size:
                # df11_histogram_device wants 16-byte aligned weights
                d = torch.from_numpy(w.view(np.int16)).cuda()
                assert torch.equal(ed.df11_histogram_device(d), opt.counts[k])


def test_tensors_may_share_one_counts_array():
    case = Case([500, 700], "bf16", "bf16", seed=11)
    opt = case.opt(counts=True)
    opt.counts.fill_(9)
    opt._t[1].counts = opt._t[0].counts
    say("[gpu] df11_adamw_step shared counts")
    opt.step()
    torch.cuda.synchronize()
    w = np.concatenate(case.got("w")).astype(np.int64)
    assert np.array_equal(opt.counts[0].cpu().numpy(), np.bincount((w >> 7) & 0xFF, minlength=256))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_state_values(kind):
    case = Case([1, 255, 0, 257, 5000], bits=8, seed=12)
    opt = case.opt()
    dtype = torch.float32 if kind == "f32" else torch.bfloat16
    outs = [[torch.full((s,), 3.0, dtype=dtype, device="cuda") for s in case.sizes] for _ in "mv"]
    say(f"[gpu] df11_adamw_values {kind}")
    opt.state_values(*outs)
    torch.cuda.synchronize()
    for k, s in enumerate(case.sizes):
        c = case.host["m"][k].astype(np.int32)
        m = blockwise(s, case.host["m_scale"][k]) * (c * np.abs(c)).astype(f32)
        c = case.host["v"][k].astype(np.int32)
        r = blockwise(s, case.host["v_scale"][k]) * (c * c).astype(f32)
        for out, want in zip(outs, (m, r * r)):
            got = out[k].float().cpu().numpy()
            assert np.array_equal(got, want if kind == "f32" else from_bf16(to_bf16(want)))
    m_only, none = opt.state_values([t.float() for t in outs[0]], None)
    assert none is None
    got = opt.state_values()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[0], m_only))


@pytest.mark.parametrize("g", ["bf16", "f32"])
@pytest.mark.parametrize("sizes", [[1], [5, 0, 1025], [70_000, 3], [9_000_001], [11] * 80])
def test_grad_norm(sizes, g):
    case = Case(sizes, "bf16", g, seed=13)
    opt = case.opt()
    say(f"[gpu] df11_grad_norm {g} {sizes[:4]}")
    got = opt.grad_norm(1e-2).cpu().numpy()
    again = opt.grad_norm(1e-2).cpu().numpy()
    every = np.concatenate([from_bf16(x) if g == "bf16" else x for x in case.host["g"]]).astype(np.float64)
    norm = math.sqrt(math.fsum(every * every))
    # float64 inside; one rounding to float32, and n 2^-53 of summing at most
    assert abs(got[0] - norm) <= norm * 1.01 * U
    f = min(1.0, 1e-2 / (norm + 1e-6))
    assert abs(got[1] - f) <= f * 1.01 * U
    assert np.array_equal(got, again)


@pytest.mark.parametrize("g", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", [
    [65536], [65537], [65535, 0, 1], [32768, 32768, 1], [256] * 35 + [56576], [256] * 36 + [56320],
    [1] * 36, [1] * 37, [255, 257] * 18, [0] * 40 + [513], [33 * k for k in range(40)]])
def test_grad_norm_where_its_forms_meet(sizes, g):
    """Up to 65536 elements in up to 36 tensors one launch, two or more beyond.
    Every element counts: the norm of ones is the root of their number."""
    case = Case(sizes, "bf16", g, seed=18)
    say(f"[gpu] df11_grad_norm {g} {len(sizes)} tensors, {sum(sizes)} elements")
    got = case.opt().grad_norm(1e-2).cpu().numpy()
    every = np.concatenate([from_bf16(x) if g == "bf16" else x for x in case.host["g"]]).astype(np.float64)
    norm = math.sqrt(math.fsum(every * every))
    assert abs(got[0] - norm) <= norm * 1.01 * U
    ones = case.opt()
    for t in ones.grads:
        t.fill_(1.0)
    assert ones.grad_norm(1.0).cpu().numpy()[0] == f32(math.sqrt(sum(sizes)))
    last = [t for t in ones.grads if t.numel()][-1]
    last[-1] = math.inf
    assert math.isnan(ones.grad_norm(1.0).cpu().numpy()[1])


def test_grad_norm_of_nothing_and_of_large_values():
    case = Case([0, 0], "bf16", "f32", seed=14)
    say("[gpu] df11_grad_norm of nothing, of 1e30, of infinity")
    assert case.opt().grad_norm(0.5).tolist() == [0.0, 1.0]
    case = Case([1000], "bf16", "f32", seed=14, grads=[np.full(1000, 1e30, f32)])
    got = case.opt().grad_norm(1.0).cpu().numpy().astype(np.float64)
    norm = float(f32(1e30)) * math.sqrt(1000)
    assert abs(got[0] - norm) <= norm * 1.01 * U and abs(got[1] * norm - 1) <= 1.01 * U
    for value in (math.inf, math.nan):
        g = np.ones(1000, f32)
        g[999] = value
        case = Case([1000], "bf16", "f32", seed=14, grads=[g])
        before = case.views("w")[0].clone()
        norm = case.opt().step(max_norm=1.0).cpu().numpy()
        assert not math.isfinite(norm[0]) and math.isnan(norm[1])
        assert torch.equal(case.views("w")[0], before)  # the step changed nothing


@pytest.mark.parametrize("bits", [32, 8])
def test_clipped_step(bits):
    case = Case([4097, 600], "bf16", "bf16", True, bits, seed=15)
    say(f"[gpu] df11_adamw_step clipped, bits={bits}")
    norm = case.opt().step(max_norm=1e-3)
    torch.cuda.synchronize()
    factor = norm.cpu().numpy()[1]
    assert 0 < factor < 1
    same(case, [step32(case, k, 5, factor) for k in range(2)], names_of(case))


def test_numbers_on_the_device():
    """lr and the step's number read by the kernel give the bits of the host's."""
    a, b = (Case([300, 5000], "bf16", "bf16", True, 8, seed=16) for _ in range(2))
    one, two = a.opt(step=0), b.opt(step=0, device_step=True)
    lr = torch.zeros(1, device="cuda")
    say("[gpu] df11_adamw_step lr and step on the device")
    for t in range(1, 4):
        x = float(f32(1e-3 / t))
        one.step(lr=x)
        lr.fill_(x)
        two.step(lr=lr)
        torch.cuda.synchronize()
        for name in names_of(a):
            for p, q in zip(a.got(name), b.got(name)):
                assert np.array_equal(p, q), (t, name)
    assert int(two.d_step.item()) == 3


def test_replayed_from_a_graph():
    """A captured clipped step with the step's number on the device, replayed
    with eager work and synchronisation between, goes on as eager steps do."""
    eager, graphed = (Case([300, 70_000, 5], "bf16", "bf16", True, 8, seed=17) for _ in range(2))
    e, g = (c.opt(step=0, device_step=True, counts=True) for c in (eager, graphed))
    say("[gpu] df11_adamw_step captured in a graph")
    for o in (e, g):
        o.step(max_norm=0.01)  # warm-up, eager
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = g.step(max_norm=0.01)
    for i in range(4):
        want = e.step(max_norm=0.01)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, want)
        for name in names_of(eager):
            for p, q in zip(eager.got(name), graphed.got(name)):
                assert np.array_equal(p, q), (i, name)
        assert torch.equal(e.counts, g.counts)
        for c in (eager, graphed):  # other gradients for the next step
            for v in c.views("g"):
                v.mul_(0.5)


def test_two_streams():
    cases = [Case([30_000, 7], "bf16", "bf16", True, 8, seed=18 + k) for k in range(2)]
    opts = [c.opt() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    say("[gpu] df11_adamw_step on two streams at once")
    norms = [o.step(max_norm=1e-3, stream=s) for o, s in zip(opts, streams)]
    torch.cuda.synchronize()
    for c, norm in zip(cases, norms):
        same(c, [step32(c, k, 5, norm.cpu().numpy()[1]) for k in range(2)], names_of(c))


def test_binding_refuses():
    w = torch.zeros(10, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(10, device="cuda")
    with pytest.raises(ValueError):
        ed.AdamW([], [])
    with pytest.raises(ValueError):
        ed.AdamW([w], [g[:9]])
    with pytest.raises(ValueError):
        ed.AdamW([w[::2]], [g[:5]])
    with pytest.raises(ValueError):
        ed.AdamW([w.cpu()], [g])
    with pytest.raises(ValueError):
        ed.AdamW([w], [g], state_bits=4)
    with pytest.raises(TypeError):
        ed.AdamW([w], [g], masters=[w])
    with pytest.raises(TypeError):
        ed.AdamW([w], [g.to(torch.int32)])
    with pytest.raises(ed.Df11Error):
        ed.AdamW([w], [g.to(torch.float16)]).step()
    with pytest.raises(ValueError):
        ed.AdamW([w], [g], state={"m": [g]})
    with pytest.raises(ValueError):
        ed.AdamW([w], [g], weight_decay=[0.1, 0.2])
    with pytest.raises(ValueError):
        ed.AdamW([w], [g]).step(max_norm=1.0, grad_factor=g[:1])
    with pytest.raises(ValueError):
        ed.AdamW([w], [g]).step(grad_factor=g)
    with pytest.raises(ValueError):
        ed.AdamW([w], [g]).state_values()
    with pytest.raises(ed.Df11Error):
        ed.AdamW([g.clone()], [g], counts=True).step()
    with pytest.raises(ed.Df11Error):
        ed.AdamW([w], [g]).step(lr=-1.0)
    with pytest.raises(ed.Df11Error):
        ed.AdamW([w], [g]).grad_norm(0.0)


def test_update_then_compress():
    """A unit that is decoded, trained for two steps and encoded again: the
    sizes told from the step's histogram are the encoder's, and the unit
    decodes to the updated weights."""
    rng = np.random.default_rng(20)
    tensors = [to_bf16(rng.standard_normal(n).astype(f32) * 0.02) for n in (120_000, 4096, 30_008)]
    cb = ed.df11_build_codebook(tensors)
    ds = ed.DeviceStream(ed.df11_encode(cb, tensors), cb, "cuda")
    unit = torch.empty(ds.n_weights, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    say("[gpu] decode, two AdamW steps, encode, decode")
    ed.df11_decompress_block(ds, unit, status)
    weights = list(unit.split([t.size for t in tensors]))
    grads = [torch.randn(t.size, device="cuda").mul_(1e-3).bfloat16() for t in tensors]
    opt = ed.AdamW(weights, grads, masters=[w.float() for w in weights], state_bits=8, counts=True)
    before = unit.clone()
    for _ in range(2):
        opt.step(max_norm=1.0)
    sz = opt.compressed_sizes()
    new, _ = opt.compress()
    assert int(new.desc.total_bits) == int(sz.total_bits) and new.n_weights == int(sz.n_weights)
    out = torch.empty_like(unit)
    ed.df11_decompress_block(new, out, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(out.view(torch.int16), unit.view(torch.int16))
    assert not torch.equal(unit, before)


@pytest.mark.parametrize("sizes_first", [True, False])
def test_compressing_waits_for_a_step_on_another_stream(sizes_first):
    w = (torch.randn(200_000, device="cuda") * 0.02).bfloat16()
    g = torch.randn(200_000, device="cuda").bfloat16()
    opt = ed.AdamW([w], [g], counts=True, lr=0.5)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a = torch.randn(4096, 4096, device="cuda")
    say("[gpu] AdamW step behind products on another stream, then its sizes and unit")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(20):  # some ten milliseconds before the step
            b = a @ a
    opt.step(stream=side)
    if sizes_first:
        sz = opt.compressed_sizes()
        counts = np.bincount((w.view(torch.int16).cpu().numpy().view(np.uint16).astype(np.int64) >> 7)
                             & 0xFF, minlength=256)
        assert np.array_equal(opt.counts[0].cpu().numpy(), counts)
        assert int(sz.n_weights) == w.numel()
    new, _ = opt.compress()
    out, status = torch.empty_like(w), torch.zeros(1, dtype=torch.int32, device="cuda")
    ed.df11_decompress_block(new, out, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(out.view(torch.int16), w.view(torch.int16))
    del b


def test_weights_that_overlap_are_refused():
    flat = torch.zeros(300, device="cuda")
    g = [torch.zeros(n, device="cuda") for n in (100, 100, 0)]
    say("[gpu] AdamW of weights that overlap")
    for pair in ([flat[:100], flat[:100]], [flat[50:150], flat[:100]], [flat[:100], flat[99:199]]):
        with pytest.raises(ValueError, match="overlap"):
            ed.AdamW(pair, g[:2])
    ed.AdamW([flat[100:200], flat[:100], flat[50:50]], g).step()  # side by side, and an empty one


def test_gradients_freed_while_another_stream_uses_them():
    w = torch.randn(200_000, device="cuda")
    g = torch.randn(200_000, device="cuda")
    plain = ed.AdamW([w.clone()], [g.clone()])
    plain.step(max_norm=1.0)
    opt = ed.AdamW([w], [g])
    a = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    say("[gpu] AdamW step on a busy stream, its gradients freed at once")
    with torch.cuda.stream(side):
        for _ in range(20):
            b = a @ a
    opt.step(max_norm=1.0, stream=side)
    at = g.data_ptr()
    opt.set_grads([torch.zeros(200_000, device="cuda")])
    del g
    others = [torch.full((200_000,), 7.0, device="cuda") for _ in range(4)]
    assert all(o.data_ptr() != at for o in others)
    torch.cuda.synchronize()
    assert torch.equal(w, plain.weights[0])
    del b


def test_captured_with_its_stream_named():
    w, g = torch.randn(70_000, device="cuda"), torch.randn(70_000, device="cuda")
    side = torch.cuda.Stream()
    plain, opt = (ed.AdamW([w.clone()], [g.clone()], state_bits=8, device_step=True) for _ in range(2))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    say("[gpu] AdamW step captured, stream named")
    with torch.cuda.graph(graph, stream=side):
        opt.step(max_norm=1.0, stream=side)
    for _ in range(3):
        graph.replay()
        plain.step(max_norm=1.0)
        torch.cuda.synchronize()
        assert torch.equal(opt.weights[0], plain.weights[0])
        assert int(opt.d_step) == int(plain.d_step)
