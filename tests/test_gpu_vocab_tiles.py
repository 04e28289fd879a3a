"""GPU tests of every form of the vocabulary loss's tiles, at many stages and ragged
sizes, against float64.

Whole numbers: the operands are such that float32 holds every sum, in any order.
* Logits: x is whole, w whole times a power of two; a logit's sum is below 2^24 of
  their unit.  lse and losses are then off by what their exponentials, sums and
  logarithms are (test_gpu_vocab_loss.py), without a logit's share.
* Gradients, bit for bit: logits are 0 or -256 and the given lse 0, so that a
  token's exponentials are 1 or 0, and g is (a + c) times those, less a at the target: a
  dense matrix of whole numbers, or of numbers of 9 bits, which two terms hold, and
  one term rounds to 8.  Every sum is below 2^24 units (asserted), so dx and dw are the
  formula's, rounded once.
"""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import entropy_decoding_amd as ed  # noqa: E402
from test_gpu_vocab_loss import BF16, F32, U, Exact, check, gen, say  # noqa: E402
from vocab_shapes import PAST, SHAPES  # noqa: E402

TYPES = {"bfloat16": BF16, "float32": F32}


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    torch.cuda.init()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def whole(lo, hi, *shape, seed):
    return torch.randint(lo, hi + 1, shape, generator=gen(seed), device="cuda", dtype=torch.int32)


def some_targets(n, rows, seed):
    targets = torch.randint(0, rows, (n,), generator=gen(seed), device="cuda")
    if n > 4:
        targets[torch.rand(n, generator=gen(seed + 1), device="cuda") < 0.1] = -100
    return targets


class Whole(Exact):
    """Exact, where float32 holds every logit."""

    def __init__(self, x, w, targets):
        super().__init__(x, w, targets)
        roundings = (4 * math.log(len(w) + 1) + 700) * U
        self.off_lse = roundings + 4 * U * self.lse.abs()
        told = self.logits.gather(1, self.at[:, None])
        rest = self.logits.scatter(1, self.at[:, None], -math.inf)
        d = torch.logsumexp(rest, 1) - told[:, 0]
        off = roundings + 4 * U * (rest.amax(1) - told[:, 0]).abs()
        self.off_loss = torch.sigmoid(d) * off * (1 + off) + 8 * U * self.loss


def held(rows, cols, kind, left, right):
    """(a matrix of 7, the columns of it that a call is given)."""
    room = torch.full((rows, left + cols + right), 7.0, dtype=kind, device="cuda")
    return room, room[:, left:left + cols]


def outside_is_kept(room, left, cols):
    return bool((room[:, :left] == 7).all()) and bool((room[:, left + cols:] == 7).all())


@pytest.mark.parametrize("n,rows,cols,dx,dw,add", SHAPES)
def test_losses_and_gradients_of_whole_logits(n, rows, cols, dx, dw, add):
    say(f"[gpu] whole logits, {n} tokens, {rows} x {cols}, {dx}, {dw}, added {add}")
    x = whole(-2, 2, n, cols, seed=n).to(BF16)
    unit = 2.0 ** -round(math.log2(1.8 * cols ** 0.5))  # logits of a spread of about 2
    w = (whole(-4, 4, rows, cols, seed=rows).float() * unit).to(BF16)
    assert cols * 8 < 2 ** 24
    targets = some_targets(n, rows, cols)
    e = Whole(x, w, targets)
    head = ed.VocabLoss([w])
    losses, lse = head(x, targets)
    check(lse, e.lse, e.off_lse, "lse")
    check(losses, e.loss, e.off_loss, "loss")
    a = torch.randn(n, generator=gen(7), device="cuda")
    kinds = TYPES[dx], TYPES[dw]
    before = whole(-3, 3, rows, cols, seed=3).to(kinds[1]) if add else None
    got_dx, (got_dw,) = head.gradient(x, targets, lse, a, dx_dtype=kinds[0], dw_dtype=kinds[1], losses=losses,
                                      dws=[before.clone()] if add else None, accumulate=add)
    for got, kind, which in ((got_dx, kinds[0], "dx"), (got_dw, kinds[1], "dw")):
        g, off = e.gradient(a, 0.0, 2 if n <= 64 or kind == F32 else 1, True)
        check(got, *(e.dx(g, off, kind) if which == "dx" else e.dw(g, off, kind, before)), which)


@pytest.mark.parametrize("n,rows,cols,dx,dw,add", SHAPES + PAST)
def test_gradients_bit_for_bit(n, rows, cols, dx, dw, add):
    """Outputs that begin at any element; a float32 dw past the caches on half lines too."""
    check_bits(n, rows, cols, dx, dw, add, 1, 4)
    if dw == "float32" and rows * cols * 4 >= 1 << 27:
        check_bits(n, rows, cols, dx, dw, add, 16, 16 + -cols % 16)


def check_bits(n, rows, cols, dx, dw, add, left, right):
    say(f"[gpu] gradients bit for bit, {n} tokens, {rows} x {cols}, {dx}, {dw}, added {add}")
    dx, dw = TYPES[dx], TYPES[dw]
    # 8 columns say which logits are 0; of the others x has the even ones, w the odd
    group = whole(0, 7, n, seed=1)
    off = whole(0, 1, rows, 8, seed=2)  # a group's row: 1 where its logit is -256
    x, w = whole(-2, 2, n, cols, seed=n).to(BF16), whole(-1, 1, rows, cols, seed=rows).to(BF16)
    x[:, 9::2], w[:, 8::2] = 0, 0
    x[:, :8] = torch.nn.functional.one_hot(group.long(), 8)
    w[:, :8] = -256.0 * off
    targets = some_targets(n, rows, cols)
    fine = 2.0 ** -8 if rows < 60_000 else 0.0
    a = whole(1, 2, n, seed=5) * whole(0, 1, n, seed=6).mul(2).sub(1) * (1 + fine)
    a[(targets != -100).nonzero()[0]] = 1  # the digits of the first are taken out of g
    c = whole(0, 1, n, seed=8) * (1 + fine)
    before = whole(-100, 100, rows, cols, seed=9).to(dw) if add else None
    room_x, out_x = held(n, cols, dx, 3, 10)
    room_w, out_w = held(rows, cols, dw, left, right)
    if add:
        out_w.copy_(before)
    lse = torch.zeros(n, device="cuda")
    ed.VocabLoss([w]).gradient(x, targets, lse, a.float(), c.float(), dx=out_x, dws=[out_w], accumulate=add)
    assert outside_is_kept(room_x, 3, cols) and outside_is_kept(room_w, left, cols)

    counted = (targets != -100).double()
    a, c, x64 = a.double() * counted, c.double() * counted, x.double()
    unit = 2.0 ** -8 if fine else 1.0
    want, most = torch.zeros(n, cols, dtype=torch.float64, device="cuda"), 0.0
    step = max(1, 2 ** 27 // max(n, cols))
    for r in range(0, rows, step):
        w64, here = w[r:r + step].double(), torch.arange(r, min(r + step, rows), device="cuda")
        g = (a + c)[:, None] * (off[r:r + step, group.long()].t() == 0)
        g -= a[:, None] * (targets[:, None] == here)
        g_x, g_w = (g if n <= 64 or kind == F32 else g.to(BF16).double() for kind in (dx, dw))
        want += torch.matmul(g_x, w64)
        size = torch.matmul(g_x.abs(), (w64 / torch.where(torch.arange(cols, device="cuda") < 8, 256, 1)).abs())
        most += float(size.amax()) / unit
        of_x = torch.matmul(g_w.t(), x64)
        if add:
            of_x += before[r:r + step].double()
        assert n * 5 * 2 + 100 < 2 ** 24 * unit
        assert torch.equal(out_w[r:r + step], of_x.to(dw)), f"dw of rows from {r} on"
    assert 0 < most < 2 ** 24
    assert torch.equal(out_x, want.to(dx)), "dx"


@pytest.mark.parametrize("n,rows,cols", [(5, 300, 72), (64, 3000, 136), (65, 129, 264), (300, 2000, 520),
                                         (700, 24_500, 72), (1001, 5001, 1000)])
@pytest.mark.parametrize("dx,dw", [(F32, F32), (F32, BF16), (BF16, F32)])
def test_float32_gradients_hold_what_float32_does(n, rows, cols, dx, dw):
    """As above, g of 1 + 2^-9 + 2^-20, which BF16 holds in three terms, with so few
    entries in x and w that sums are below 16, so that float32 holds them too."""
    say(f"[gpu] gradients of {n} tokens, {rows} x {cols}, {dx}, {dw}, of 21 bits")
    group, off = whole(0, 7, n, seed=1), whole(0, 1, rows, 8, seed=2)

    def few(count, seed):
        keep = torch.rand(count, cols, generator=gen(seed), device="cuda") < 3 / count
        return (whole(-1, 1, count, cols, seed=seed + 1) * keep).to(BF16)

    x, w = few(n, 3), few(rows, 5)
    x[:, 9::2], w[:, 8::2] = 0, 0
    x[:, :8] = torch.nn.functional.one_hot(group.long(), 8)
    w[:, :8] = -256.0 * off
    targets = some_targets(n, rows, cols)
    a = torch.full((n,), 1 + 2.0 ** -9 + 2.0 ** -20, device="cuda")
    a[(targets != -100).nonzero()[0]] = 1
    got_dx, (got_dw,) = ed.VocabLoss([w]).gradient(x, targets, torch.zeros(n, device="cuda"), a, dx_dtype=dx,
                                                  dw_dtype=dw)
    here = torch.arange(rows, device="cuda")
    g = a.double()[:, None] * ((off[:, group.long()].t() == 0).double() - (targets[:, None] == here).double())
    g[targets == -100] = 0
    # the 8 columns that say which logits are 0 have long sums
    x64, w64 = x[:, 8:].double(), w[:, 8:].double()
    assert max((g.abs() @ w64.abs()).max(), (g.t().abs() @ x64.abs()).max()) < 16
    for got, want, kind in ((got_dx, g @ w64, dx), (got_dw, g.t() @ x64, dw)):
        if kind == F32:
            assert want.any() and torch.equal(got[:, 8:], want.float())


@pytest.mark.parametrize("n,rows,cols", [(20, 300, 72), (120, 3000, 136), (1500, 2000, 520)])
@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("given", ["number", "one", "each", "each but ignored"])
def test_one_gradient_of_all_losses_costs_no_digits(n, rows, cols, kind, given):
    """1 / 120, which BF16 holds to 1 in 290 only: g is whole but for it, and the
    gradients are those of whole numbers times it, rounded once more."""
    say(f"[gpu] gradients of {n} tokens, {rows} x {cols}, {kind}, of one 120th: {given}")
    group, off = whole(0, 7, n, seed=1), whole(0, 1, rows, 8, seed=2)
    x, w = whole(-2, 2, n, cols, seed=3).to(BF16), whole(-1, 1, rows, cols, seed=4).to(BF16)
    x[:, 9::2], w[:, 8::2] = 0, 0
    x[:, :8] = torch.nn.functional.one_hot(group.long(), 8)
    w[:, :8] = -256.0 * off
    targets = some_targets(n, rows, cols)
    targets[0], targets[1] = -100, 3
    a = torch.full((n,), 1 / 120, device="cuda")
    if given == "each but ignored":
        a[targets == -100] = float("nan")
    a = {"number": 1 / 120, "one": a[:1]}.get(given, a)
    dx, (dw,) = ed.VocabLoss([w]).gradient(x, targets, torch.zeros(n, device="cuda"), a, dx_dtype=kind, dw_dtype=kind)
    g = (off[:, group.long()].t() == 0).double()
    g -= (targets[:, None] == torch.arange(rows, device="cuda")).double()
    g[targets == -100] = 0
    one = torch.tensor(1 / 120, dtype=F32, device="cuda")
    for got, whole_ones in ((dx, g @ w.double()), (dw, g.t() @ x.double())):
        assert whole_ones.any() and whole_ones.abs().max() < 2 ** 24
        assert torch.equal(got, (whole_ones.float() * one).to(kind))
