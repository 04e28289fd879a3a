"""GPU tests of the int8 quantiser (df11_quantize_int8) and product
(df11_gemm_int8), and of the Int8Linear that calls both.

Codes are compared with round(127 x / a) in float64, which decides them: for
BF16, F16 and float32 inputs a quotient that is no tie is at least 2^-32 of
itself away from one, far more than float64's rounding, and ties are exact.
Sums are compared through the result: float(sum) * x_scale * w_scale, each
rounded in float32 and then to the type, has one right value of bits.  Against
float64 it is at most 3 half steps of float32 (2^-24 each) and one of the type
off (BF16 2^-8, F16 2^-11).
"""

import ctypes
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import entropy_decoding_amd as ed  # noqa: E402

U = 2.0 ** -24
KINDS = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def say(msg):
    print(msg, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    torch.cuda.init()
    yield
    torch.cuda.synchronize()


def reference_codes(x):
    """Codes and scales of the rows of a host tensor, by the definition."""
    x = x.double().numpy()
    with np.errstate(all="ignore"):
        top = np.abs(x).max(axis=1, initial=0.0)
        bad = ~np.isfinite(x).all(axis=1)
        ok = ~bad & (top > 0)
        codes = np.where(ok[:, None], np.rint(127.0 * x / np.where(ok, top, 1.0)[:, None]), 0.0)
        codes = np.where(np.isfinite(codes), codes, 0.0)
        scales = np.where(bad, np.float32(np.nan), top.astype(np.float32) / np.float32(127))
    return codes.astype(np.int8), scales.astype(np.float32)


def check_codes(x, label):
    """Quantises x (a host tensor) and compares every code, scale and pad."""
    r, c = x.shape
    say(f"[gpu] df11_quantize_int8 {label} {r}x{c} {x.dtype}")
    (codes, scales), = ed.quantize_int8([x.cuda()])
    torch.cuda.synchronize()
    want, sc = reference_codes(x)
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    assert codes.shape == (r, (c + 15) // 16 * 16)
    assert np.array_equal(codes[:, :c], want), np.argwhere(codes[:, :c] != want)[:5]
    assert not codes[:, c:].any()
    assert np.array_equal(scales, sc, equal_nan=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (2, 8), (5, 16), (4, 17), (3, 255), (2, 2048),
                                   (3, 2049), (1, 4096), (2, 9001), (300, 33), (1, 131071)])
def test_codes(kind, shape):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(*shape, generator=g) * torch.exp(torch.randn(shape[0], 1, generator=g) * 4)
    check_codes(x.to(KINDS[kind]), "normal")


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_codes_of_every_pattern(kind):
    """All 65536 patterns beside largest values with different mantissas, the
    ones that make ties among them; the rows of NaN and infinities too."""
    every = torch.from_numpy(np.arange(65536, dtype=np.uint16).view(np.int16)).view(KINDS[kind])
    f = every.float()
    finite = torch.where(torch.isfinite(f), f, torch.zeros(()))
    rows = []
    for top in (1.0, 1.5, 127 / 128, 1.0078125, 3.0, 0.75, 2.0 ** -20, 65504.0 if kind == "f16" else 3e38):
        top = torch.tensor(top).to(KINDS[kind]).float()
        row = torch.where(finite.abs() <= top, finite, torch.zeros(()))
        row[0] = top
        rows.append(row)
    check_codes(torch.stack(rows).to(KINDS[kind]), "every pattern")
    check_codes(every.view(1, -1).clone(), "with NaN")


@pytest.mark.parametrize("kind", KINDS)
def test_codes_next_to_ties(kind):
    """Values as near to a tie as the type has them, on both sides, and ties."""
    rng = np.random.default_rng(2)
    rows = []
    for _ in range(64):
        a = torch.tensor(float(rng.uniform(0.5, 2.0) * 2.0 ** int(rng.integers(-10, 10)))).to(KINDS[kind])
        h = torch.arange(0, 127, dtype=torch.float64) + 0.5
        x = (h * a.double() / 127).to(KINDS[kind])
        up, down = (torch.nextafter(x.float(), torch.tensor(s)).to(KINDS[kind]) if kind == "f32" else
                    (x.view(torch.int16) + d).view(KINDS[kind]) for s, d in ((math.inf, 1), (-math.inf, -1)))
        row = torch.cat([a.view(1), x, up, down, -x, a.view(1) / 2])
        rows.append(torch.where(row.float().abs() <= a.float(), row, a))
    check_codes(torch.stack(rows), "next to ties")


@pytest.mark.parametrize("kind", KINDS)
def test_codes_of_odd_rows(kind):
    tiny = {"bf16": 9.2e-41, "f16": 6e-8, "f32": 1.4e-45}[kind]
    large = torch.finfo(KINDS[kind]).max
    x = torch.zeros(9, 40)
    x[1, 3] = tiny
    x[2, 5], x[2, 6] = 3 * tiny, -tiny
    x[3, 0], x[3, 39] = large, -large / 2
    x[4, 7] = math.nan
    x[5, 39] = math.inf
    x[6, 0] = -math.inf
    x[7] = -1.0
    x[8, 2] = -0.0
    check_codes(x.to(KINDS[kind]), "odd rows")


def test_no_columns_and_no_rows():
    say("[gpu] df11_quantize_int8 of no columns")
    (codes, scales), (c2, s2) = ed.quantize_int8([torch.empty(3, 0, device="cuda"),
                                                  torch.empty(0, 5, device="cuda")])
    torch.cuda.synchronize()
    assert codes.shape == (3, 0) and scales.tolist() == [0.0] * 3
    assert c2.shape == (0, 16) and s2.numel() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_quantiser_strides_and_guards(kind):
    """Rows at odd offsets and strides; nothing outside of the rows is written."""
    base = torch.randn(7 * 61 + 9).to(KINDS[kind]).cuda()
    x = base[3:3 + 7 * 61].view(7, 61)[:, 5:50]
    codes = torch.full((9, 64), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((9,), 55.0, device="cuda")
    a = (ed.df11_int8_rows * 1)()
    a[0].src, a[0].codes, a[0].scales = x.data_ptr(), codes[1:].data_ptr(), scales[1:].data_ptr()
    a[0].src_stride, a[0].code_stride, a[0].rows, a[0].cols = x.stride(0), 64, 7, 45
    say(f"[gpu] df11_quantize_int8 strided {kind}")
    assert ed.LIB.df11_quantize_int8(ed.TYPES[str(KINDS[kind])[6:]], a, 1, None) == ed.DF11_OK
    torch.cuda.synchronize()
    want, sc = reference_codes(x.cpu())
    codes = codes.cpu().numpy()
    assert np.array_equal(codes[1:8, :45], want) and not codes[1:8, 45:48].any()
    assert (codes[1:8, 48:] == 99).all() and (codes[0] == 99).all() and (codes[8] == 99).all()
    assert np.array_equal(scales.cpu().numpy(), np.concatenate([[55], sc, [55]]).astype(np.float32))


def test_quantises_16_matrices_in_one_call():
    ms = [torch.randn(k + 1, 10 * k + 3).bfloat16() for k in range(16)]
    say("[gpu] df11_quantize_int8 16 matrices")
    for m, (codes, scales) in zip(ms, ed.quantize_int8([m.cuda() for m in ms])):
        want, sc = reference_codes(m)
        assert np.array_equal(codes.cpu().numpy()[:, :m.size(1)], want)
        assert np.array_equal(scales.cpu().numpy(), sc)


# ---------------------------------------------------------------- product


def rounded(a, kind):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(KINDS[kind])


def product(qx, qw, sx, sw, kind):
    """The result's bits: exact sums, then float32 and the type."""
    acc = qx.astype(np.float64) @ qw.astype(np.float64).T  # below 2^53: exact
    with np.errstate(all="ignore"):
        y = (acc.astype(np.float32) * sx[:, None].astype(np.float32)) * sw[None, :].astype(np.float32)
    return acc, rounded(y, kind)


class Product:
    """Matrices of random codes with garbage behind their columns, scales, and
    outputs inside larger buffers."""

    def __init__(self, shapes, tokens, kind, seed=0, extra=16, y_extra=3, code=lambda rng, s: rng.integers(-128, 128, s)):
        rng = np.random.default_rng(seed)
        self.kind, self.tokens, self.shapes = kind, tokens, shapes
        self.t = (ed.df11_int8_tensor * len(shapes))()
        self.parts = []
        for a, (r, c) in zip(self.t, shapes):
            stride = (c + 15) // 16 * 16 + extra
            w = rng.integers(-128, 128, (r, stride)).astype(np.int8)
            x = rng.integers(-128, 128, (tokens, stride)).astype(np.int8)
            w[:, :c], x[:, :c] = code(rng, (r, c)), code(rng, (tokens, c))
            sw = np.exp(rng.standard_normal(r)).astype(np.float32) * np.float32(1e-3)
            sx = np.exp(rng.standard_normal(tokens)).astype(np.float32) * np.float32(1e-2)
            y = torch.full((tokens, r + y_extra), 7.0, dtype=KINDS[kind], device="cuda")
            d = [torch.from_numpy(v).cuda() for v in (w, sw, x, sx)]
            a.w, a.w_scale, a.x, a.x_scale, a.y = [v.data_ptr() for v in d] + [y.data_ptr()]
            a.w_stride = a.x_stride = stride
            a.y_stride, a.rows, a.cols = r + y_extra, r, c
            self.parts.append((w[:, :c], x[:, :c], sw, sx, y, d))

    def run(self, stream=None):
        return ed.LIB.df11_gemm_int8(ed.TYPES[str(KINDS[self.kind])[6:]], self.t, len(self.t),
                                     self.tokens, stream)

    def check(self):
        for (r, c), (w, x, sw, sx, y, _) in zip(self.shapes, self.parts):
            acc, want = product(x, w, sx, sw, self.kind)
            got = y.cpu()
            assert torch.equal(got[:, :r], want), (r, c, np.argwhere((got[:, :r] != want).numpy())[:4])
            assert (got[:, r:] == 7.0).all(), "written behind the rows"
            exact = acc * sx[:, None].astype(np.float64) * sw[None, :].astype(np.float64)
            half = torch.finfo(KINDS[self.kind]).eps / 2 if self.kind != "f32" else 0.0
            low = torch.finfo(KINDS[self.kind]).smallest_normal * torch.finfo(KINDS[self.kind]).eps
            assert (np.abs(got[:, :r].double().numpy() - exact) <=
                    np.abs(exact) * (3 * U + half) * 1.001 + low).all()


SHAPES = [(1, 1), (15, 16), (16, 17), (17, 64), (33, 255), (64, 256), (1, 1024), (5, 1025), (130, 300)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens", [1, 2, 15, 16, 17, 32, 33, 64])
def test_product_of_few_tokens(tokens, kind):
    p = Product(SHAPES, tokens, kind, seed=tokens)
    say(f"[gpu] df11_gemm_int8 {tokens} tokens {kind} {SHAPES}")
    assert p.run() == ed.DF11_OK
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens", [65, 77, 127, 128, 129, 200, 256, 257, 300, 511, 515])
def test_product_of_many_tokens(tokens, kind):
    shapes = [(1, 1), (17, 64), (129, 127), (256, 128), (257, 129), (300, 1000), (511, 385), (64, 4111)]
    p = Product(shapes, tokens, kind, seed=tokens)
    say(f"[gpu] df11_gemm_int8 {tokens} tokens {kind} {shapes}")
    assert p.run() == ed.DF11_OK
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens,rows,cols", [
    (590, 8195, 1000), (601, 8130, 130), (997, 12003, 300), (1021, 12011, 257), (1000, 12003, 385),
    (2050, 12003, 300), (2047, 12289, 16), (2100, 11999, 641)])
def test_product_of_large_tiles(tokens, rows, cols, kind):
    """Enough work for tiles of 128 x 128, 256 x 128 and 256 x 256, with
    ragged ends in every direction and odd and even numbers of stages."""
    p = Product([(rows, cols), (70, cols + 33)], tokens, kind, seed=rows)
    say(f"[gpu] df11_gemm_int8 {tokens} tokens {rows}x{cols} {kind}")
    assert p.run() == ed.DF11_OK
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("tokens", [3, 100, 700])
@pytest.mark.parametrize("cols", [0, 16, 100, 128, 130, 256, 257, 384, 512, 640, 1040, 2048])
def test_product_columns(cols, tokens):
    p = Product([(270, cols)], tokens, "f32", seed=cols + tokens, extra=0)
    say(f"[gpu] df11_gemm_int8 {cols} columns, {tokens} tokens")
    assert p.run() == ed.DF11_OK
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("tokens", [1, 40, 300])
def test_sums_are_exact_at_the_limit(tokens):
    """131071 columns of -128 times -128: the largest sum that int32 holds."""
    def code(rng, s):
        v = np.full(s, -128)
        v[1::2] = rng.integers(-128, 128, s)[1::2]
        return v

    p = Product([(18, 131071)], tokens, "f32", seed=3, extra=0, code=code)
    say(f"[gpu] df11_gemm_int8 131071 columns, {tokens} tokens")
    assert p.run() == ed.DF11_OK
    torch.cuda.synchronize()
    p.check()


def far_product(rows, cols, tokens, kind, sample):
    """Large operands made on the device; rows and tokens of `sample` compared."""
    g = torch.Generator(device="cuda").manual_seed(7)
    w = torch.randint(-127, 128, (rows, cols), dtype=torch.int8, device="cuda", generator=g)
    x = torch.randint(-127, 128, (tokens, cols), dtype=torch.int8, device="cuda", generator=g)
    sw = torch.rand(rows, device="cuda", generator=g) + 0.5
    sx = torch.rand(tokens, device="cuda", generator=g) + 0.5
    y = torch.empty(tokens, rows, dtype=KINDS[kind], device="cuda")
    t = (ed.df11_int8_tensor * 1)()
    a = t[0]
    a.w, a.w_scale, a.x, a.x_scale, a.y = (v.data_ptr() for v in (w, sw, x, sx, y))
    a.w_stride = a.x_stride = cols
    a.y_stride, a.rows, a.cols = rows, rows, cols
    say(f"[gpu] df11_gemm_int8 {tokens} tokens {rows}x{cols} {kind}, beyond 32 bits")
    assert ed.LIB.df11_gemm_int8(ed.TYPES[str(KINDS[kind])[6:]], t, 1, tokens, None) == ed.DF11_OK
    torch.cuda.synchronize()
    r, s = (torch.tensor([i % n for i in sample], device="cuda") for n in (rows, tokens))
    _, want = product(x[s].cpu().numpy(), w[r].cpu().numpy(), sx[s].cpu().numpy(), sw[r].cpu().numpy(), kind)
    assert torch.equal(y[s][:, r].cpu(), want)


@pytest.mark.parametrize("rows,cols,tokens", [
    (140_000, 32_000, 1), (140_000, 32_000, 30), (140_000, 32_000, 50),  # weights of 4.5 GB
    (40_000, 16, 70_000),  # 2.8 G results
    (300, 32_000, 140_000)])  # activations of 4.5 GB
def test_offsets_beyond_32_bits(rows, cols, tokens):
    far_product(rows, cols, tokens, "bf16", [0, 1, 17, -1, -2, -300, 2 ** 17 + 3, 67_200, 134_300])


def test_quantiser_offsets_beyond_32_bits():
    x = torch.randn(1, 40_000, device="cuda").bfloat16().repeat(120_000, 1)  # 4.8 G elements
    x[-1] *= 2
    say("[gpu] df11_quantize_int8 of 4.8 G elements")
    (codes, scales), = ed.quantize_int8([x])
    want, sc = reference_codes(x[:1].cpu())
    for r in (0, 60_000, 107_380, 119_998, 119_999):
        assert np.array_equal(codes[r].cpu().numpy(), want[0]), r
        assert float(scales[r]) == float(sc[0]) * (2 if r == 119_999 else 1)


@pytest.mark.parametrize("tokens", [1, 9, 66, 600])
def test_random_sizes(tokens):
    rng = np.random.default_rng(30 + tokens)
    shapes = [(int(np.exp(rng.uniform(0, 6.5))), int(np.exp(rng.uniform(0, 8)))) for _ in range(16)]
    p = Product(shapes, tokens, ("bf16", "f16", "f32")[tokens % 3], seed=tokens)
    say(f"[gpu] df11_gemm_int8 {tokens} tokens {shapes}")
    assert p.run() == ed.DF11_OK
    torch.cuda.synchronize()
    p.check()


@pytest.mark.parametrize("tokens", [2, 150, 520])
def test_scales_that_are_not_finite(tokens):
    p = Product([(40, 64)], tokens, "f32", seed=5)
    w, x, sw, sx, y, d = p.parts[0]
    sw[3], sx[1] = np.nan, np.inf
    d[1].copy_(torch.from_numpy(sw)), d[3].copy_(torch.from_numpy(sx))
    say(f"[gpu] df11_gemm_int8 NaN and infinite scales, {tokens} tokens")
    assert p.run() == ed.DF11_OK
    torch.cuda.synchronize()
    _, want = product(x, w, sx, sw, "f32")
    assert np.array_equal(y.cpu().numpy()[:, :40], want.numpy(), equal_nan=True)


def linear_reference(x, w, kind):
    qx, sx = reference_codes(x)
    qw, sw = reference_codes(w)
    return product(qx, qw, sx, sw, kind)[1]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tokens", [1, 5, 70, 300])
def test_linear(tokens, kind):
    """Quantiser and product together, with a shared and a strided input, and
    the distance from the unquantised product: each factor is off by half a
    scale at most, so a sum is off by sum(|x| s_w + |w| s_x) / 2 + s_x s_w K / 4."""
    g = torch.Generator().manual_seed(tokens)
    shapes = [(96, 200), (33, 200), (50, 77)]
    ws = [(torch.randn(*s, generator=g) * 0.02).bfloat16() for s in shapes]
    a = torch.randn(tokens, 200, generator=g).to(KINDS[kind])
    b = torch.randn(tokens, 90, generator=g).to(KINDS[kind])[:, 4:81]
    layer = ed.Int8Linear.from_tensors([w.cuda() for w in ws])
    da, db = a.cuda(), torch.randn(tokens, 90).to(KINDS[kind]).cuda()
    db[:, 4:81] = b.cuda()
    say(f"[gpu] Int8Linear {tokens} tokens {kind}")
    ys = layer([da, da, db[:, 4:81]], KINDS[kind])
    out = [torch.full((tokens, r + 2), 5.0, dtype=KINDS[kind], device="cuda") for r, _ in shapes]
    layer([da, da.clone(), db[:, 4:81]], out=[o[:, 1:-1] for o in out])
    torch.cuda.synchronize()
    for x, w, y, o in zip((a, a, b), ws, ys, out):
        assert torch.equal(y.cpu(), linear_reference(x, w, kind))
        assert torch.equal(o[:, 1:-1], y) and (o[:, 0] == 5).all() and (o[:, -1] == 5).all()
        xd, wd = x.double(), w.double()
        sx, sw = xd.abs().amax(1) / 127, wd.abs().amax(1) / 127
        far = (xd.abs().sum(1)[:, None] * sw + wd.abs().sum(1) * sx[:, None]) / 2 + sx[:, None] * sw * x.size(1) / 4
        exact = xd @ wd.T
        # the rounding of a value that is itself off by `far`
        half = torch.finfo(KINDS[kind]).eps / 2
        assert ((y.cpu().double() - exact).abs() <= far * (1 + 1e-4) + (exact.abs() + far) * (half + 4 * U)).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cols", [1, 15, 16, 17, 127, 128, 129, 1000, 1024, 1025, 3975, 4095, 4096, 4097,
                                  4111, 5120, 9001, 32768, 32769])
def test_linear_of_one_token(cols, kind):
    """One token is quantised by the product's own workgroups (up to 32768
    columns): the same bits as by the quantiser, beside narrower matrices."""
    g = torch.Generator().manual_seed(cols)
    shapes = [(33, cols), (16, min(cols, 700)), (5, cols)]
    ws = [torch.randn(*s, generator=g).bfloat16() for s in shapes]
    a = (torch.randn(1, cols, generator=g) * 3).to(KINDS[kind])
    b = torch.randn(1, min(cols, 700), generator=g).to(KINDS[kind])
    layer = ed.Int8Linear.from_tensors([w.cuda() for w in ws])
    da, db = a.cuda(), b.cuda()
    say(f"[gpu] Int8Linear one token {kind} {cols} columns")
    for x, w, y in zip((a, b, a), ws, layer([da, db, da], KINDS[kind])):
        assert torch.equal(y.cpu(), linear_reference(x, w, kind)), w.shape


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("value", [0.0, math.nan, math.inf, -math.inf, "tiny"])
def test_linear_of_one_odd_token(value, kind):
    x = torch.zeros(1, 300)
    x[0, 299] = {"bf16": 9.2e-41, "f16": 6e-8, "f32": 1.4e-45}[kind] if value == "tiny" else value
    x = x.to(KINDS[kind])
    w = torch.randn(20, 300).bfloat16()
    say(f"[gpu] Int8Linear one token with {value} {kind}")
    y, = ed.Int8Linear.from_tensors([w.cuda()])([x.cuda()], torch.float32)
    assert np.array_equal(y.cpu().numpy(), linear_reference(x, w, "f32").numpy(), equal_nan=True)


def test_linear_of_a_compressed_unit():
    """Decode, quantise, multiply: the same as from the weights themselves."""
    rng = np.random.default_rng(6)
    shapes = [(64, 128), (48, 256), (130, 64)]
    ws = [(torch.randn(*s) * 0.02).bfloat16() for s in shapes]
    tensors = [w.view(torch.int16).numpy().view(np.uint16).reshape(-1) for w in ws]
    cb = ed.df11_build_codebook(tensors)
    ds = ed.DeviceStream(ed.df11_encode(cb, tensors), cb, "cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    xs = [torch.randn(20, c).bfloat16().cuda() for _, c in shapes]
    say("[gpu] Int8Linear of a compressed unit")
    ys = ed.Int8Linear.from_unit(ds, shapes, status)(xs, torch.float32)
    assert int(status.item()) == 0
    for x, w, y in zip(xs, ws, ys):
        assert torch.equal(y.cpu(), linear_reference(x.cpu(), w, "f32"))
    assert rng is not None


def test_update_requantise_multiply():
    """A block that is decoded, updated (8-bit states), requantised and used."""
    shapes = [(64, 128), (48, 256)]
    ws = [(torch.randn(*s) * 0.02).bfloat16() for s in shapes]
    tensors = [w.view(torch.int16).numpy().view(np.uint16).reshape(-1) for w in ws]
    cb = ed.df11_build_codebook(tensors)
    ds = ed.DeviceStream(ed.df11_encode(cb, tensors), cb, "cuda")
    unit = torch.empty(ds.n_weights, dtype=torch.bfloat16, device="cuda")
    ed.df11_decompress_block(ds, unit)
    parts = list(unit.split([r * c for r, c in shapes]))
    opt = ed.AdamW(parts, [torch.randn_like(p) * 1e-3 for p in parts], state_bits=8, lr=1e-2, counts=True)
    say("[gpu] decode, AdamW step, quantise, product; encode, decode, quantise, product")
    opt.step(max_norm=1.0)
    xs = [torch.randn(7, c).bfloat16().cuda() for _, c in shapes]
    mats = [p.view(s) for p, s in zip(parts, shapes)]
    ys = ed.Int8Linear.from_tensors(mats)(xs)
    again = ed.Int8Linear.from_unit(opt.compress()[0], shapes)(xs)
    torch.cuda.synchronize()
    for x, w, old, y, z in zip(xs, mats, ws, ys, again):
        assert not torch.equal(w.cpu(), old)
        assert torch.equal(y.cpu(), linear_reference(x.cpu(), w.cpu(), "bf16"))
        assert torch.equal(y, z)


@pytest.mark.parametrize("tokens,shapes", [
    (1, [(96, 200), (300, 528)]), (40, [(96, 200), (300, 528)]), (400, [(96, 200), (300, 528)]),
    (2050, [(12003, 300)])])
def test_replayed_from_a_graph(tokens, shapes):
    layer = ed.Int8Linear.from_tensors([torch.randn(*s, device="cuda") for s in shapes])
    xs = [torch.randn(tokens, c, device="cuda").bfloat16() for _, c in shapes]
    out = [torch.empty(tokens, r, dtype=torch.bfloat16, device="cuda") for r, _ in shapes]
    say(f"[gpu] Int8Linear captured in a graph, {tokens} tokens")
    layer(xs, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(xs, out=out)
    for i in range(4):
        for x in xs:
            x.copy_(torch.randn_like(x))
        want = [y.clone() for y in layer(xs)]
        for o in out:
            o.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_two_streams():
    shapes = [(300, 528), (64, 1000)]
    layer = ed.Int8Linear.from_tensors([torch.randn(*s, device="cuda") for s in shapes])
    streams = [torch.cuda.Stream() for _ in range(2)]
    inputs = [[torch.randn(t, c, device="cuda").bfloat16() for _, c in shapes] for t in (3, 200)]
    want = [[y.cpu() for y in layer(xs)] for xs in inputs]
    torch.cuda.synchronize()
    say("[gpu] Int8Linear on two streams at once")
    for _ in range(5):
        got = [layer(xs, stream=s) for xs, s in zip(inputs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p.cpu(), q) for p, q in zip(a, b))


@pytest.mark.parametrize("offset,stride", [(0, 128), (8, 32), (16, 48), (3, 37), (128, 37), (0, 144)])
def test_linear_takes_codes_anywhere(offset, stride):
    """Rows that do not start on cache lines are laid out anew."""
    w = torch.randn(6, 20).bfloat16()
    (codes, scales), = ed.quantize_int8([w.cuda()])
    room = torch.full((offset + 6 * stride,), 77, dtype=torch.int8, device="cuda")
    held = room[offset:].view(6, stride)[:, :32]
    held.copy_(codes)
    x = torch.randn(3, 20).bfloat16()
    say(f"[gpu] Int8Linear of codes at {offset}, stride {stride}")
    y, = ed.Int8Linear([held], [scales], [(6, 20)])([x.cuda()], torch.float32)
    assert torch.equal(y.cpu(), linear_reference(x, w, "f32"))
    one, = ed.Int8Linear([held[:1]], [scales[:1]], [(1, 20)])([x.cuda()], torch.float32)
    assert torch.equal(one, y[:, :1])


def test_linear_takes_one_row_of_codes_for_all():
    """Codes and scales of one row, broadcast over the matrix."""
    w = torch.randn(1, 200).bfloat16()
    (codes, scales), = ed.quantize_int8([w.cuda()])
    x = torch.randn(4, 200).bfloat16()
    say("[gpu] Int8Linear of broadcast codes")
    layer = ed.Int8Linear([codes.expand(9, -1)], [scales.expand(9).contiguous()], [(9, 200)])
    y, = layer([x.cuda()], torch.float32)
    assert torch.equal(y.cpu(), linear_reference(x, w.expand(9, -1), "f32"))
    again, = ed.Int8Linear.from_tensors(iter([w.cuda().expand(9, -1).contiguous()]))([x.cuda()], torch.float32)
    assert torch.equal(again, y)


def test_captured_with_its_stream_named():
    w = torch.randn(700, 272).bfloat16()
    layer = ed.Int8Linear.from_tensors([w.cuda(), w[:300].cuda()])
    side = torch.cuda.Stream()
    for tokens in (1, 90):
        x = torch.randn(tokens, 272).bfloat16()
        d = x.cuda()
        layer([d, d], torch.float32, stream=side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        say(f"[gpu] Int8Linear of {tokens} tokens captured, stream named")
        with torch.cuda.graph(graph, stream=side):
            ys = layer([d, d], torch.float32, stream=side)
        for k in range(3):
            d.copy_(x * (k + 1))
            graph.replay()
            eager = layer([d, d], torch.float32)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(ys, eager))
            assert torch.equal(ys[0].cpu(), linear_reference(x * (k + 1), w, "f32"))


def test_activations_freed_while_another_stream_uses_them():
    w = torch.randn(300, 512).bfloat16()
    layer = ed.Int8Linear.from_tensors([w.cuda()])
    x = torch.randn(64, 512).bfloat16()
    want = linear_reference(x, w, "f32")
    a = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    for tokens in (1, 64):
        d = x[:tokens].cuda()
        torch.cuda.synchronize()
        say(f"[gpu] Int8Linear of {tokens} tokens on a busy stream, its activations freed at once")
        with torch.cuda.stream(side):
            for _ in range(20):
                b = a @ a
        y, = layer([d], torch.float32, stream=side)
        at = d.data_ptr()
        del d
        others = [torch.zeros(tokens, 512, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        assert all(o.data_ptr() != at for o in others)
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), want[:tokens])
    del b


def test_no_tokens():
    layer = ed.Int8Linear.from_tensors([torch.randn(5, 20, device="cuda")])
    say("[gpu] Int8Linear of no tokens")
    assert layer([torch.randn(0, 20, device="cuda")])[0].shape == (0, 5)


def test_binding_refuses():
    w = torch.randn(6, 20, device="cuda")
    layer = ed.Int8Linear.from_tensors([w])
    x = torch.randn(3, 20, device="cuda")
    (codes, scales), = ed.quantize_int8([w])
    for bad in ([x.cpu()], [x[:, :19]], [x, x], [], [x.t()], [x[0]]):
        with pytest.raises(ValueError):
            layer(bad)
    for bad in ([x.double()], [x.to(torch.int8)]):
        with pytest.raises(TypeError):
            layer(bad)
    with pytest.raises(TypeError):
        layer([x], torch.float64)
    with pytest.raises(ValueError):
        layer([x], out=[torch.empty(3, 7, device="cuda")])
    with pytest.raises(ValueError):
        layer([x], torch.bfloat16, out=[torch.empty(3, 6, device="cuda")])
    with pytest.raises(ValueError):
        ed.Int8Linear([codes[:, :20]], [scales], [(6, 20)])
    with pytest.raises(ValueError):
        ed.Int8Linear([codes], [scales[:5]], [(6, 20)])
    with pytest.raises(ValueError):
        ed.Int8Linear([codes], [scales], [(7, 20)])
    with pytest.raises(ValueError):
        ed.Int8Linear([codes], [scales], [(6, 33)])
    with pytest.raises(ValueError):
        ed.Int8Linear([codes.float()], [scales], [(6, 20)])
    with pytest.raises(ValueError):
        ed.quantize_int8([w] * 17)
    assert ctypes.sizeof(ed.df11_int8_tensor) == 72
