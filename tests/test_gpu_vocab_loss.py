"""GPU tests of the cross entropy under an output head and of its gradients.

Bounds, with u = 2^-24 and K columns (everything to first order):
* a logit's K products are exact and its sums float32: off by at most
  K u sum |x w|, S being the largest of those sums for a token;
* an exponential exp(d) has an argument off by 2 |d| u and its own rounding of
  2 u, and the sum of all of them, in parts of at most 300 terms one behind
  another, rounds 600 times at most; the mean of |d| under the probabilities is
  at most log V, so lse is off by e = K u S + (4 log V + 700) u + 4 u |lse|, and
  the others' lse less the target's logit, d, by twice K u S and the same
  otherwise; the loss log(1 + exp d) by (1 - p) of that and its own roundings;
* a probability is off by the factor 2 e + 4 u (|l - lse| + 2), an entry of g by
  that times it, and by 2 u |g|, and by its rounding: 2^-8 of it, or with two
  terms (that of 2^-8 of what the first left) 2^-16;
* a gradient's sums are of M products, off by M u of their magnitudes together,
  then its own rounding, at most half a step.
"""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import entropy_decoding_amd as ed  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}  # half a step, at most, relative to the value


def say(msg):
    print(msg, flush=True)


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    torch.cuda.init()
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=gen(seed), device="cuda")


def inputs(n, rows, cols, seed=0, kind=torch.int64, ignored=0.2):
    """Hidden states that know their target more or less well; some targets ignored."""
    w = (randn(rows, cols, seed=seed) / max(1, cols) ** 0.5).to(BF16)
    targets = torch.randint(0, rows, (n,), generator=gen(seed + 1), device="cuda")
    x = (randn(n, cols, seed=seed + 2) + torch.rand(n, 1, generator=gen(seed + 3), device="cuda") * 12 *
         w[targets].float()).to(BF16)
    targets[torch.rand(n, generator=gen(seed + 4), device="cuda") < ignored] = -100
    return x, w, targets.to(kind)


class Exact:
    """The formulas in float64, and how far float32 may be from them."""

    def __init__(self, x, w, targets, ignored=-100):
        self.x, self.w = x.double(), w.double()
        rows, cols = w.shape
        self.logits = self.x @ self.w.t()
        self.lse = torch.logsumexp(self.logits, 1)
        self.counted = targets != ignored
        self.at = torch.where(self.counted, targets, 0).long()
        self.loss = torch.where(self.counted, self.lse - self.logits.gather(1, self.at[:, None])[:, 0], 0.0)
        size = (self.x.abs() @ self.w.abs().t()).amax(1)
        self.off_logit = cols * U * size
        self.off_lse = self.off_logit + (4 * math.log(rows + 1) + 700) * U + 4 * U * self.lse.abs()
        # the loss is log(1 + exp d), d what the others' lse is above the target's
        # logit; it changes with d by 1 - p
        told = self.logits.gather(1, self.at[:, None])
        rest = self.logits.scatter(1, self.at[:, None], -math.inf)
        d = torch.logsumexp(rest, 1) - told[:, 0]
        off_d = 2 * self.off_logit + (4 * math.log(rows + 1) + 700) * U + 4 * U * (rest.amax(1) - told[:, 0]).abs()
        off_d = torch.where(d == -math.inf, 0.0, off_d)
        self.loss = torch.where(self.counted, torch.logaddexp(d, torch.zeros_like(d)), 0.0)
        self.off_loss = torch.sigmoid(d) * off_d * (1 + off_d) + 8 * U * self.loss

    def gradient(self, loss_grad, lse_grad, terms, losses=False):
        """g and how far it may be off.  With the losses the target's entry is off by
        what they are, times a + c, and by 4 u of its two parts."""
        a = torch.where(self.counted, torch.as_tensor(loss_grad, dtype=torch.float64, device="cuda"), 0.0)
        c = torch.where(self.counted, torch.as_tensor(lse_grad, dtype=torch.float64, device="cuda"), 0.0)
        d = self.logits - self.lse[:, None]
        p = (a + c)[:, None] * d.exp()
        g = p.clone()
        g.scatter_add_(1, self.at[:, None], -a[:, None])
        off = p.abs() * (2 * self.off_lse[:, None] + 4 * U * (d.abs() + 2)) + 4 * U * (p.abs() + g.abs())
        if losses:
            told = torch.exp(-self.loss)
            g.scatter_(1, self.at[:, None], (a * torch.expm1(-self.loss) + c * told)[:, None])
            far = (a.abs() + c.abs()) * self.off_loss + 4 * U * (a.abs() * (1 - told) + c.abs() * told)
            off.scatter_(1, self.at[:, None], far[:, None])
        # exponentials below 2^-126 may be zero, and products with a small a + c
        off += (a + c).abs()[:, None] * 2.0 ** -126 + 2.0 ** -133
        return g, off + (g.abs() + off) * (2.0 ** -8 if terms == 1 else 2.0 ** -16)

    def dx(self, g, off, kind):
        want, size = g @ self.w, (g.abs() + off) @ self.w.abs()
        off = off @ self.w.abs() + (len(self.w) * 2 + 40) * U * size
        return want, off + HALF[kind] * (want.abs() + off)

    def dw(self, g, off, kind, before=None):
        want, size = g.t() @ self.x, (g.abs() + off).t() @ self.x.abs()
        off = off.t() @ self.x.abs() + (len(self.x) * 2 + 10) * U * size
        if before is not None:
            want = want + before.double()
            off = off + U * want.abs()
        return want, off + HALF[kind] * (want.abs() + off)


def check(got, want, off, what):
    far = (got.double() - want).abs() - off
    assert (far <= 0).all(), f"{what}: over the bound by {far.max().item():.3g}, {int((far > 0).sum())} values"


def check_all(n, rows, cols, seed=0, kind=torch.int64, dx=BF16, dw=BF16, add=False, pieces=None, factors=True,
              ignored=0.2):
    x, w, targets = inputs(n, rows, cols, seed, kind, ignored)
    parts = [w] if pieces is None else list(w.split(pieces))
    head = ed.VocabLoss(parts)
    losses, lse = head(x, targets)
    e = Exact(x, w, targets)
    check(lse, e.lse, e.off_lse, "lse")
    check(losses, e.loss, e.off_loss, "loss")
    assert (losses[targets == -100] == 0).all()
    a = randn(n, seed=seed + 7) if factors else 0.25
    c = 0.5 * randn(n, seed=seed + 8) if factors else None
    before = (randn(rows, cols, seed=seed + 9) * 0.1).to(dw) if add else None
    dws = list(before.clone().split(pieces or rows)) if add else None
    given = losses if seed % 2 else None
    got_dx, got_dw = head.gradient(x, targets, lse, a, c, dx_dtype=dx, dw_dtype=dw, dws=dws, accumulate=add,
                                   losses=given)
    assert got_dx.dtype == dx and all(t.dtype == dw for t in got_dw)
    for got, kind, which in ((got_dx, dx, "dx"), (torch.cat(got_dw), dw, "dw")):
        g, off = e.gradient(a, 0.0 if c is None else c, 2 if kind == F32 else 1, given is not None)
        want = e.dx(g, off, kind) if which == "dx" else e.dw(g, off, kind, before)
        check(got, *want, which)
    assert not got_dx[targets == -100].any()
    return head, x, targets, losses, lse, got_dx, got_dw


# small and large results, whole and ragged (test_gpu_vocab_tiles.py has every form
# of the tiles)
SIZES = [(1, 1, 8), (1, 2, 64), (1, 999, 256), (3, 17, 72), (16, 4000, 128), (31, 65, 8), (32, 64, 64),
         (33, 63, 136), (64, 700, 200), (65, 129, 64), (77, 1003, 1000), (128, 256, 256), (129, 255, 264),
         (300, 2000, 520), (257, 70_001, 40), (700, 24_500, 72), (40, 4300, 4104), (2100, 130, 8200)]


@pytest.mark.parametrize("n,rows,cols", SIZES)
def test_loss_and_gradient(n, rows, cols):
    say(f"[gpu] loss and gradient of {n} tokens, {rows} x {cols}")
    check_all(n, rows, cols, seed=n, kind=torch.int32 if n % 2 else torch.int64)


@pytest.mark.parametrize("dx,dw,add", [(F32, F32, False), (BF16, F32, True), (F32, BF16, False), (BF16, BF16, True)])
@pytest.mark.parametrize("n,rows,cols", [(1, 50, 64), (20, 333, 136), (100, 1003, 200), (300, 2000, 520),
                                         (40, 4300, 4104), (2100, 130, 8200)])
def test_types_and_accumulation(n, rows, cols, dx, dw, add):
    say(f"[gpu] gradient of {n} tokens, {rows} x {cols}, {dx}, {dw}, added {add}")
    check_all(n, rows, cols, seed=n, dx=dx, dw=dw, add=add)


@pytest.mark.parametrize("n,rows,cols,pieces", [(5, 300, 64, 128), (70, 1003, 136, 1), (200, 1003, 136, 500),
                                                (300, 5000, 72, 4999)])
def test_pieces(n, rows, cols, pieces):
    if pieces == 1:
        rows = 30
    say(f"[gpu] head of {rows} rows in pieces of {pieces}")
    check_all(n, rows, cols, seed=n, pieces=pieces, dx=F32)


@pytest.mark.parametrize("sizes", [[70_000, 40_000], [33_000, 1, 32_000], [5, 0, 300]])
@pytest.mark.parametrize("n", [1, 30])
def test_pieces_of_unlike_sizes(n, sizes):
    """Smaller pieces, for which another tile would be the faster one, fit where the
    largest does."""
    say(f"[gpu] pieces of {sizes} rows, {n} tokens")
    x, w, targets = inputs(n, sum(sizes), 8, n)
    head, e = ed.VocabLoss(list(w.split(sizes))), Exact(x, w, targets)
    losses, lse = head(x, targets)
    check(lse, e.lse, e.off_lse, "lse")
    check(losses, e.loss, e.off_loss, "loss")
    dx, dws = head.gradient(x, targets, lse, 0.5, dx_dtype=F32, losses=losses)
    g, off = e.gradient(0.5, 0.0, 2, True)
    check(dx, *e.dx(g, off, F32), "dx")
    check(torch.cat(dws), *e.dw(g, off, BF16), "dw")


def test_long_vocabulary_in_chunks():
    """g in several chunks of the vocabulary, with one and with two terms."""
    say("[gpu] g in several chunks")
    check_all(20_000, 60_000, 16, seed=1)
    check_all(20_000, 30_100, 16, seed=2, dx=F32, dw=F32, add=True)


def test_one_number_for_all():
    say("[gpu] one gradient for all losses")
    head, x, targets, _, lse, dx, (dw,) = check_all(50, 300, 64, seed=2, factors=False)
    one = torch.tensor([0.25], device="cuda")
    for a, c in ((one, None), (one.expand(50).contiguous(), torch.zeros(1, device="cuda"))):
        again, (dw_again,) = head.gradient(x, targets, lse, a, c)
        assert torch.equal(dx, again) and torch.equal(dw, dw_again)
    only, none = head.gradient(x, targets, lse, 0.25, needs_dw=False)
    assert none is None and torch.equal(only, dx)
    none, (only,) = head.gradient(x, targets, lse, 0.25, needs_dx=False)
    assert none is None and torch.equal(only, dw)


def test_against_differences():
    """Sums of float32 losses over a change that BF16 holds: the derivative along
    a line through x and along one through w."""
    say("[gpu] gradient against differences")
    n, rows, cols = 40, 200, 64
    x, w, targets = inputs(n, rows, cols, 5)
    a = randn(n, seed=6).abs()
    _, lse = ed.VocabLoss([w])(x, targets)
    dx, (dw,) = ed.VocabLoss([w]).gradient(x, targets, lse, a, dx_dtype=F32, dw_dtype=F32)

    def at(x, w):
        e = Exact(x, w, targets)
        losses, _ = ed.VocabLoss([w])(x, targets)
        return (losses.double() * a).sum(), (e.off_loss * a).sum()

    for which in "xw":
        base, grad = (x, dx) if which == "x" else (w, dw)
        step = torch.sign(randn(*base.shape, seed=8)) * 2.0 ** -6
        hi, lo = (base.float() + step).to(BF16), (base.float() - step).to(BF16)
        moved = hi.double() - lo.double()
        (up, off1), (down, off2) = (at(hi, w), at(lo, w)) if which == "x" else (at(x, hi), at(x, lo))
        # the central difference's error: a third derivative of a cross entropy along
        # a line is at most (the logits' spread)^3; steps from rounding are not even,
        # so the second derivative, at most spread^2, counts with their mean
        v = moved / 2
        spread = ((v @ w.double().t()) if which == "x" else (x.double() @ v.t())).abs().amax(1) * 2
        uneven = (hi.double() + lo.double() - 2 * base.double()) / 2
        drift = ((uneven @ w.double().t()) if which == "x" else (x.double() @ uneven.t())).abs().amax(1) * 2
        error = (a * (spread ** 3 / 3 + 2 * spread * drift + spread * spread * drift)).sum() + off1 + off2
        error += (grad.double().abs() * moved.abs()).sum() * 2.0 ** -14
        assert (up - down - (grad.double() * moved).sum()).abs() <= error
        assert error < 0.5 * (grad.double().abs() * moved.abs()).sum()


def test_targets_outside():
    """Outside the vocabulary: NaN, and no other token's loss or dx changes;
    ignore_index may be a row of the vocabulary, or any number."""
    say("[gpu] targets outside the vocabulary")
    x, w, targets = inputs(40, 130, 64, 3, ignored=0)
    head = ed.VocabLoss(list(w.split(50)))
    good = targets.clone()
    targets[[0, 7, 39]] = torch.tensor([-1, 130, 2 ** 31 + 5], device="cuda")
    losses, lse = head(x, targets)
    want, same_lse = head(x, good)
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[[0, 7, 39]] = True
    assert losses[bad].isnan().all() and torch.equal(losses[~bad], want[~bad])
    e = Exact(x, w, good)
    assert torch.equal(lse[~bad], same_lse[~bad])
    check(lse, e.lse, e.off_lse, "lse")
    dx, dws = head.gradient(x, targets, lse)
    dx_want, _ = head.gradient(x, good, lse)
    assert dx[bad].isnan().all() and torch.equal(dx[~bad], dx_want[~bad])
    assert all(t.isnan().all() for t in dws)
    losses, lse = head(x, good, ignore_index=int(good[5]))
    assert torch.equal(lse, same_lse)
    assert (losses[good == good[5]] == 0).all() and torch.equal(losses[good != good[5]], want[good != good[5]])
    far = torch.full((40,), -2 ** 62, device="cuda")
    assert not head(x, far, ignore_index=-2 ** 62)[0].any()


def test_all_ignored():
    say("[gpu] all tokens ignored")
    x, w, targets = inputs(70, 300, 136, 4, ignored=2)
    head = ed.VocabLoss([w])
    x[3] = float("nan")
    losses, lse = head(x, targets)
    assert not losses.any() and lse[3].isnan() and lse.isnan().sum() == 1
    dx, (dw,) = head.gradient(x, targets, lse)
    assert not dx.any() and not dw.any()
    held = torch.full((300, 136), 3.0, device="cuda")
    head.gradient(x, targets, lse, dws=[held], accumulate=True)
    assert (held == 3).all()


def test_nan_in_ignored_tokens_goes_nowhere():
    """A padded batch whose padding holds NaN and infinities: the counted tokens'
    results are those of a batch without it."""
    say("[gpu] NaN in ignored tokens")
    for n in (20, 150, 400, 1023, 1024, 1025, 3000):
        x, w, targets = inputs(n, 500, 72, n)
        head, on = ed.VocabLoss([w]), targets != -100
        x[~on] = float("nan")
        x[(~on).nonzero()[::2, 0]] = float("inf")
        losses, lse = head(x, targets)
        short, short_lse = head(x[on], targets[on])
        assert torch.equal(losses[on], short) and torch.equal(lse[on], short_lse) and not losses[~on].any()
        dx, (dw,) = head.gradient(x, targets, lse, 0.5, dw_dtype=F32)
        e = Exact(x[on], w, targets[on])
        check(dw, *e.dw(*e.gradient(0.5, 0.0, 2), F32), "dw")
        check(dx[on], *e.dx(*e.gradient(0.5, 0.0, 1), BF16), "dx")
        assert not dx[~on].any()


def test_infinite_and_extreme_logits():
    say("[gpu] infinite and extreme logits")
    n, rows, cols = 6, 400, 64
    w = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    x = torch.zeros(n, cols, dtype=BF16, device="cuda")
    w[:, 0], w[:, 1], w[:, 2] = torch.arange(rows, device="cuda") % 7, -1.0, 1.0
    w[200:, 3] = -float("inf")  # x[., 3] > 0: those rows count nothing
    w[:200, 3] = 1.0
    x[0, 0] = 3e4      # large differences
    x[1, 1] = 3e38     # all logits the lowest of the type, near enough
    x[2, 2] = 3e38
    x[3, 3] = 1.0      # half of them -infinity
    x[4, 2] = float("inf")
    targets = torch.tensor([5, 3, 3, 7, 3, 3], device="cuda")
    x[0, 3] = x[1, 3] = x[2, 3] = 1e-30  # keeps 0 * inf out: -inf there as well
    x[5, 3] = 2.0
    losses, lse = ed.VocabLoss([w])(x, targets)
    logits = x[:, :4].double() @ w[:, :4].double().t()
    want = torch.logsumexp(logits[[0, 1, 2, 3, 5]], 1)
    got = lse[[0, 1, 2, 3, 5]].double()
    assert ((got - want).abs() <= want.abs() * 8 * U + 800 * U).all()
    assert lse[4].isnan() and losses[4].isnan()
    all_low = torch.full((3, cols), -float("inf"), dtype=BF16, device="cuda")
    ones = torch.ones(1, cols, dtype=BF16, device="cuda")
    losses, lse = ed.VocabLoss([all_low])(ones, targets[:1] * 0)
    assert lse.item() == -float("inf") and losses.isnan().all()
    all_low[1:] = 1.0  # the target alone at -infinity, then the target at +infinity
    losses, lse = ed.VocabLoss([all_low])(ones, targets[:1] * 0)
    assert losses.item() == float("inf") and abs(lse.item() - 64 - math.log(2)) < 1e-4
    losses, lse = ed.VocabLoss([-all_low])(ones, targets[:1] * 0)
    assert losses.isnan().all() and lse.isnan().all()
    only = torch.ones(1, cols, dtype=BF16, device="cuda")
    losses, lse = ed.VocabLoss([only])(ones, targets[:1] * 0)
    assert losses.item() == 0 and lse.item() == 64


def test_certain_targets():
    """Losses down to 1e-24 keep their digits: differences of logarithms would not."""
    say("[gpu] nearly certain targets")
    rows, cols = 500, 64
    w = (randn(rows, cols) / 8).to(BF16)
    targets = torch.arange(60, device="cuda")
    x = (w[:60].float() * torch.linspace(1, 80, 60, device="cuda")[:, None]).to(BF16)
    losses, lse = ed.VocabLoss([w])(x, targets)
    e = Exact(x, w, targets)
    # of the inputs, in float64; the bound's largest part is 2 K u S, where S is up
    # to 80 |w|^2 = 80: 6e-4
    assert e.loss.min() < 1e-24 and (e.off_loss < 1e-3 * e.loss).all()
    check(losses, e.loss, e.off_loss, "loss")
    check(lse, e.lse, e.off_lse, "lse")
    for kind, terms in ((F32, 2), (BF16, 1)):
        dx, (dw,) = ed.VocabLoss([w]).gradient(x, targets, lse, losses=losses, dx_dtype=kind, dw_dtype=kind)
        g, off = e.gradient(1.0, 0.0, terms, True)
        # the entries of one token differ by the bound's relative error, 7e-4 at most,
        # and by their rounding, not by what lse has lost
        assert (off <= (2e-3 + 2.0 ** -8 * (terms == 1)) * g.abs() + 2.0 ** -125).all()
        check(dx, *e.dx(g, off, kind), "dx")
        check(dw, *e.dw(g, off, kind), "dw")


def test_shapes_and_strides():
    say("[gpu] loss with strides")
    room_w, room_x = randn(500, 200, seed=1).to(BF16), randn(60, 168, seed=2).to(BF16)
    w, x = room_w[:, 8:144], room_x[:, 16:152]
    targets = torch.randint(0, 500, (6, 21), generator=gen(3), device="cuda")
    head = ed.VocabLoss([w])
    part = targets[:, 1:11]
    losses, lse = head(x, part)
    flat, flat_lse = ed.VocabLoss([w.contiguous()])(x.contiguous(), part.reshape(-1))
    assert losses.shape == (6, 10) and torch.equal(losses.view(-1), flat) and torch.equal(lse.view(-1), flat_lse)
    cube = x.contiguous().view(6, 10, 136)
    assert torch.equal(head(cube, part)[0], losses)
    want, (want_w,) = head.gradient(cube, part, lse)
    held_x = torch.full((60, 151), 7.0, dtype=BF16, device="cuda")
    held_w = torch.full((500, 139), 7.0, dtype=BF16, device="cuda")
    got, (got_w,) = head.gradient(x, part, lse, dx=held_x[:, 3:139], dws=[held_w[:, 1:137]])
    assert torch.equal(got, want) and torch.equal(got_w, want_w)
    assert (held_x[:, :3] == 7).all() and (held_x[:, 139:] == 7).all()
    assert (held_w[:, :1] == 7).all() and (held_w[:, 137:] == 7).all()


def test_no_tokens():
    say("[gpu] loss of no tokens")
    w = randn(300, 64).to(BF16)
    head, none = ed.VocabLoss([w]), torch.zeros(0, dtype=torch.int64, device="cuda")
    x = torch.zeros(0, 64, dtype=BF16, device="cuda")
    losses, lse = head(x, none)
    assert losses.shape == lse.shape == (0,)
    dx, (dw,) = head.gradient(x, none, lse)
    assert dx.shape == (0, 64) and not dw.any()


def test_hidden_states_that_require_a_gradient_are_refused():
    x, w, targets = inputs(5, 30, 64)
    head = ed.VocabLoss([torch.nn.Parameter(w)])
    want = head(x, targets)[0]
    with pytest.raises(RuntimeError, match="gradient"):
        head(x.requires_grad_(), targets)
    with torch.no_grad():
        assert torch.equal(head(x, targets)[0], want)


def test_the_same_bits_each_time():
    say("[gpu] the same bits each time")
    x, w, targets = inputs(600, 9000, 136, 2)
    head = ed.VocabLoss([w])
    first = None
    for _ in range(4):
        losses, lse = head(x, targets)
        dx, (dw,) = head.gradient(x, targets, lse, 0.1, dw_dtype=F32)
        got = losses, lse, dx, dw
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_captured_and_replayed_on_two_streams():
    say("[gpu] loss and gradient captured on two streams")
    w = (randn(900, 136) / 10).to(BF16)
    head = ed.VocabLoss(list(w.split(400)))
    held = []
    for k in range(2):
        stream = torch.cuda.Stream()
        x, _, targets = inputs(120, 900, 136, k)
        scale = torch.full((1,), 0.5, device="cuda")
        stream.wait_stream(torch.cuda.current_stream())

        def step():
            losses, lse = head(x, targets)
            return losses, lse, head.gradient(x, targets, lse, scale, dw_dtype=F32, losses=losses)

        with torch.cuda.stream(stream):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = step()
        held.append((stream, graph, x, targets, scale, out))
    for turn in range(4):
        for k, (_, _, x, targets, scale, _) in enumerate(held):
            fresh = inputs(120, 900, 136, 20 * turn + k, ignored=0.3 * turn)
            x.copy_(fresh[0]), targets.copy_(fresh[2]), scale.fill_(turn + k + 0.5)
        torch.cuda.synchronize()
        for stream, graph, *_ in held:
            with torch.cuda.stream(stream):
                graph.replay()
        for _, _, x, targets, scale, (losses, lse, (dx, dws)) in held:
            want, want_lse = head(x, targets)
            want_dx, want_dws = head.gradient(x, targets, want_lse, scale, dw_dtype=F32, losses=want)
            torch.cuda.synchronize()
            assert torch.equal(losses, want) and torch.equal(lse, want_lse) and torch.equal(dx, want_dx)
            assert all(torch.equal(a, b) for a, b in zip(dws, want_dws))


def test_named_stream():
    say("[gpu] loss and gradient on a named stream")
    w = (randn(3000, 264) / 10).to(BF16)
    stream = torch.cuda.Stream()
    for turn in range(3):
        x, _, targets = inputs(500, 3000, 264, turn)
        kept = x.clone(), targets.clone()
        head = ed.VocabLoss([w.clone()])
        stream.wait_stream(torch.cuda.current_stream())
        losses, lse = head(x, targets, stream=stream)
        dx, (dw,) = head.gradient(x, targets, lse, 0.1, stream=stream)
        del x, targets, head
        torch.full((500, 264), 9.0, dtype=BF16, device="cuda"), torch.full((3000, 264), 9.0, dtype=BF16, device="cuda")
        torch.cuda.synchronize()
        head = ed.VocabLoss([w])
        assert torch.equal(losses, head(*kept)[0])
        want_dx, (want_dw,) = head.gradient(*kept, lse, 0.1)
        assert torch.equal(dx, want_dx) and torch.equal(dw, want_dw)
