"""The operators behind the selections on the GPU against their definitions in 64 bits
(behind_ref).  Tolerances follow from the roundings each kernel makes and are given where they are
used; places, tokens, offsets and 8-bit codes are equal."""
import math

import pytest

import behind_ref as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]
U = 2.0 ** -24  # half a step of fp32, relative


@pytest.fixture(scope="module")
def ds():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import top_selection_gb300 as m
    yield m
    assert m.ds_get_device_status() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ log probabilities ----
# A sum of V exponentials: each off by 2^-22 and by its argument's rounding (2^-23 y 2^-y ln 2 < 2^-23),
# added in fp32 by 256 threads and joined in at most 40 steps: (V / 256 + 40) 2^-24 in all, relative.
# x - m and the result are rounded once more each.

def sum_error(V):
    return 2.0 ** -22 + 2.0 ** -23 + (V / 256 + 40) * U


def check_logprobs(ds, x, tokens, top):
    V = x.shape[1]
    lp, lse, H, top_lp, top_tokens = ds.token_logprobs(x, tokens, top=top)
    want_lp, want_lse, want_H, want_top, want_tokens = ref.logprobs(x, tokens, top)
    assert torch.equal(top_tokens.long(), want_tokens)

    def near(got, want, limit):
        got = got.double()
        same = got == want  # infinities among them
        assert bool((same | ((got - want).abs() <= limit)).all())
    near(lp, want_lp, sum_error(V) + 4 * U * (want_lp.abs() + 1))
    near(lse, want_lse, sum_error(V) + 4 * U * (want_lse.abs() + 1))
    near(top_lp, want_top, sum_error(V) + 4 * U * (want_top.abs() + 1))
    # H = log s - w / s: both sums' errors, relative to sizes up to 1 + log V
    near(H, want_H, 4 * sum_error(V) * (1 + math.log(V)))


def rows_of(dtype, T, V, seed, pad=0, offset=0):
    """T rows of V logits, `pad` numbers between rows, the first `offset` numbers into the memory."""
    g = gen(seed)
    flat = torch.empty(T * (V + pad) + offset, dtype=dtype, device="cuda")
    flat.fill_(float("nan"))  # what lies between rows has no part
    x = flat[offset:].view(T, V + pad)[:, :V]
    x.copy_(2.0 * normal(g, T, V))
    tokens = torch.randint(V, (T,), device="cuda", generator=g).int()
    return x, tokens


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V,top,pad,offset", [
    (1, 1, 1, 0, 0),
    (1, 1, 0, 0, 1),
    (3, 2, 2, 1, 0),
    (5, 7, 3, 0, 3),
    (4, 32, 32, 0, 0),
    (4, 33, 32, 2, 5),
    (2, 129280, 20, 0, 0),
    (1, 129281, 32, 0, 1),
    (40, 32003, 5, 0, 0),
    (310, 8192, 1, 0, 0),
    (310, 8193, 20, 7, 1),
    (310, 20001, 32, 0, 0),
    (700, 300, 0, 0, 0),
    (9, 250007, 8, 0, 0),
])
def test_token_logprobs(ds, dtype, T, V, top, pad, offset):
    x, tokens = rows_of(dtype, T, V, T + V, pad, offset)
    tokens[0] = -1
    if T > 2:
        tokens[1], tokens[2] = V, 2 ** 31 - 1  # none of the columns
    check_logprobs(ds, x, tokens, top)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V", [(1, 20), (5, 1405), (400, 1405), (2, 129280)])
def test_nearly_certain_tokens(ds, dtype, T, V):
    """A token far above the others has a log probability -log(1 + t) near 0: its error is absolute, not
    relative to t.  The 1 is a sum's term like others, and each addition to a partial sum that holds it (in a
    thread, over lanes, warps and CTAs) rounds by up to a half step of a number in [1, 2), 2^-24: the V / 256 + 40
    additions of sum_error.  Its own exponential is off by 2^-22 and its argument moves it by 2^-23, the rest of
    sum_error; logarithm, difference and result round once more each."""
    x, _ = rows_of(dtype, T, V, V)
    tokens = torch.arange(T, device="cuda").int() % V
    gap = torch.linspace(4.0, 16.0, T, device="cuda") + math.log(V)
    x[torch.arange(T, device="cuda"), tokens.long()] = (x.amax(-1).float() + gap).to(dtype)
    lp = ds.token_logprobs(x, tokens, top=1)[0].double()
    want = ref.logprobs(x, tokens)[0]
    assert bool((want > -0.02).all()) and bool((want < 0).all())
    assert bool(((lp - want).abs() <= sum_error(V) + 4 * U * (want.abs() + 1)).all())


def masked_rows(dtype, V):
    """Rows whose masks leave little, and rows of equal or ordered numbers."""
    inf = math.inf
    g = gen(V)
    x = normal(g, 13, V).to(dtype)
    x[0] = -inf                                   # nothing
    x[1] = -inf
    x[1, V // 2] = 3.0                            # one token
    x[2] = -inf
    x[2, ::max(1, V // 5)] = x[3, ::max(1, V // 5)]  # a few
    x[4] = 1.25                                   # all alike
    x[5] = torch.where(torch.arange(V, device="cuda") % 2 == 0, 0.0, -0.0).to(dtype)  # zeros of both signs
    x[6] = x[6].sort().values                     # rising: the largest come last
    x[7] = x[7].sort(descending=True).values
    x[8] = torch.where(x[8] > 0.5, 2.0, x[8].float()).to(dtype)  # thousands share the largest
    x[9, : V // 2] = -inf
    x[10] = torch.finfo(dtype).min                # a mask of the type's lowest value throughout
    x[11] = torch.where(torch.arange(V, device="cuda") % 7 == 3, x[11].float(), torch.finfo(dtype).min).to(dtype)
    x[12] = (x[12].float() * 1000).to(dtype)      # far apart
    tokens = torch.randint(V, (13,), device="cuda", generator=g).int()
    tokens[1] = V // 2
    return x, tokens


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,top", [(5, 5), (40, 20), (513, 32), (9001, 20), (40000, 32), (40000, 1), (140000, 7)])
def test_token_logprobs_of_masked_rows(ds, dtype, V, top):
    x, tokens = masked_rows(dtype, V)
    check_logprobs(ds, x, tokens, top)
    many = x.repeat(30, 1)                        # as many rows as take a CTA each
    check_logprobs(ds, many, tokens.repeat(30), top)


def check_gradient(ds, x, tokens, g, h):
    T, V = x.shape
    lp, lse, H, _, _ = ds.token_logprobs(x, tokens)
    got = ds.token_logprobs_backward(g, x, tokens, lse, grad_entropy=h, entropy=H if h is not None else None)
    want = ref.logprobs_gradient(x, tokens, g, h)
    # p = exp(x - lse): lse is off by sum_error and rounded, the difference and the exponential's
    # argument too; then a few roundings, of terms |g|, |h| (|log p| + H)
    exact = ref.logprobs(x, tokens)[1][:, None]
    some = exact > -math.inf
    z = torch.where(some, exact, 0.0)
    lpd = torch.where(some, x.double() - z, -math.inf)
    p = torch.exp(lpd)
    size = g.double().abs()[:, None] + (0 if h is None else h.double().abs()[:, None] * (lpd.abs().clamp(max=1e6) + 1 + math.log(V)))
    rel = 2 * sum_error(V) + 4 * U * (z.abs() + lpd.abs().clamp(max=1e6)) + 8 * U
    limit = p * size * rel + half_step(x.dtype) * want.abs() * 1.01 + 2 * U * g.double().abs()[:, None] + 1e-37
    assert got.dtype == x.dtype and got.shape == x.shape
    assert bool(((got.double() - want).abs() <= limit).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("T,V,pad,offset", [(1, 1, 0, 0), (3, 50, 0, 0), (5, 33, 0, 0), (4, 129, 7, 1), (7, 9001, 0, 0),
                                            (6, 20000, 8, 0), (2, 129280, 0, 0), (300, 1000, 1, 0)])
def test_token_logprobs_backward(ds, dtype, entropy, T, V, pad, offset):
    x, tokens = rows_of(dtype, T, V, 3 * T + V, pad, offset)
    if T > 2:
        tokens[1], tokens[2] = -100, V
    g = gen(T)
    check_gradient(ds, x, tokens, normal(g, T), normal(g, T) if entropy else None)


@pytest.mark.parametrize("dtype", DTYPES)
def test_token_logprobs_backward_of_masked_rows(ds, dtype):
    x, tokens = masked_rows(dtype, 5003)
    g = gen(1)
    grad, h = normal(g, 13), normal(g, 13)
    lp, lse, H, _, _ = ds.token_logprobs(x, tokens)
    got = ds.token_logprobs_backward(grad, x, tokens, lse, grad_entropy=h, entropy=H)
    assert bool(torch.isfinite(got).all())
    assert not bool(got[0].any())
    keep = [1, 2, 3, 4, 5, 6, 7, 8, 9, 11, 12]
    # a given token that the mask excludes still has its own + g
    check_gradient(ds, x[keep], tokens[keep], grad[keep], h[keep])


def test_token_logprobs_gradient_against_differences(ds):
    """The kernel's gradient against differences of the kernel's own results: values of the order 5,
    off by 1e-6, over a step of 2 h = 0.04: 5e-5 each, and h^2 = 4e-4 for the slope."""
    g = gen(4)
    x, gl, gh = normal(g, 1, 12), normal(g, 1), normal(g, 1)
    t = torch.tensor([5], dtype=torch.int32, device="cuda")
    lp, lse, H, _, _ = ds.token_logprobs(x, t)
    got = ds.token_logprobs_backward(gl, x, t, lse, grad_entropy=gh, entropy=H)
    for v in range(12):
        total = 0.0
        for sign in (1, -1):
            y = x.clone()
            y[0, v] += sign * 0.02
            lp, _, H2, _, _ = ds.token_logprobs(y, t)
            total += sign * float(lp * gl + H2 * gh)
        assert abs(total / 0.04 - float(got[0, v])) < 6e-4 * (1 + float(gl.abs() + gh.abs()))


# ------------------------------------------------------------------ exchange -----

@pytest.mark.parametrize("T,k,E", [(0, 3, 4), (1, 1, 1), (1, 32, 512), (7, 3, 5), (33, 8, 256), (64, 32, 2), (1000, 8, 512),
                                   (4097, 1, 60), (9001, 7, 160), (40000, 8, 256)])
def test_expert_sort(ds, T, k, E):
    g = gen(T + E)
    for kind in range(4):
        e = torch.randint(E, (T, k), device="cuda", generator=g).int()
        if kind == 1:    # padded rows and what is no expert
            e[T // 2:] = -1
            e[::5] = torch.randint(-3, E + 3, e[::5].shape, device="cuda", generator=g).int()
        elif kind == 2:  # all choose one
            e.fill_(E - 1)
        elif kind == 3:
            e.fill_(-1)
        places, offsets = ds.expert_sort(e, E)
        want_places, want_offsets = ref.sort(e.cpu(), E)
        assert offsets.tolist() == want_offsets
        assert places.flatten().tolist() == want_places


def choices(T, k, E, seed, padded):
    g = gen(seed)
    e = torch.randint(E, (T, k), device="cuda", generator=g).int()
    if padded:
        e[T - T // 3:] = -1
        e[::4, 0] = -1
    return g, e


EXCHANGES = [(1, 1, 1, 1), (3, 2, 4, 64), (5, 3, 4, 65), (50, 8, 16, 200), (17, 32, 40, 136), (400, 4, 60, 1001),
             (6000, 2, 64, 48), (5500, 5, 8, 1030)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("T,k,E,D", EXCHANGES)
def test_exchange(ds, dtype, padded, T, k, E, D):
    g, e = choices(T, k, E, T + D, padded)
    places, offsets = ds.expert_sort(e, E)
    n = int(offsets[-1])
    for pad in (0, 1, 8):
        x, y, grad, rows = ((normal(g, r, D + pad).to(dtype))[:, :D] for r in (T, T * k, T, T * k))
        y[n:] = float("nan")  # rows behind the last choice have no part
        w = normal(g, T, k)
        assert torch.equal(ds.expert_gather(x, places, offsets), ref.gather(x, places, T * k))
        for weights in (w, None):
            got = ds.expert_combine(y, places, weights)
            want, size = ref.combine(y, places, weights)
            # k products and sums in fp32, one rounding
            assert got.dtype == dtype
            assert bool(((got.double() - want).abs() <= (k + 1) * U * size + half_step(dtype) * 1.01 * want.abs() + 1e-37).all())
        grad_y, grad_w = ds.expert_combine_backward(grad, y, places, offsets, w)
        p = places.long()
        for i in range(k):
            there = p[:, i] >= 0
            a, b = grad[there].double(), y[p[there, i]].double()
            want = w[there, i, None].double() * a
            got = grad_y[p[there, i]].double()
            # the product in fp32, then in the type
            assert bool(((got - want).abs() <= (half_step(dtype) + U) * 1.01 * want.abs() + 1e-37).all())
            want = (a * b).sum(-1)
            limit = (D / 32 + 16) * U * (a * b).abs().sum(-1) + 1e-37
            assert bool(((grad_w[there, i].double() - want).abs() <= limit).all())
            assert not bool(grad_w[~there, i].any())
        assert not bool(grad_y[n:].any())
        codes, scales = ds.expert_gather(x, places, offsets, quantise=True)
        want_codes, want_scales = ds.quantise_blocks(ref.gather(x, places, T * k))
        assert torch.equal(codes.view(torch.uint8), want_codes.view(torch.uint8)) and torch.equal(scales, want_scales)


def test_exchange_gradients_against_differences(ds):
    """sum_t r_t . combine(gather(x) * s, places, w), linear in x and w: differences over a step of 1 have
    only the values' own roundings, below 64 * 2^-24 * 100."""
    g, e = choices(6, 2, 3, 5, True)
    places, offsets = ds.expert_sort(e, 3)
    x, w, r, s = normal(g, 6, 8), normal(g, 6, 2), normal(g, 6, 8), normal(g, 12, 8)

    def f(x, w):
        return float((r.double() * ds.expert_combine(ds.expert_gather(x, places, offsets) * s, places, w).double()).sum())
    y = ds.expert_gather(x, places, offsets) * s
    grad_y, grad_w = ds.expert_combine_backward(r, y, places, offsets, w)
    grad_x = ds.expert_combine(grad_y * s, places)
    for t in range(6):
        for d in range(8):
            step = torch.zeros_like(x)
            step[t, d] = 1.0
            assert abs((f(x + step, w) - f(x - step, w)) / 2 - float(grad_x[t, d])) < 4e-4
        for i in range(2):
            step = torch.zeros_like(w)
            step[t, i] = 1.0
            assert abs((f(x, w + step) - f(x, w - step)) / 2 - float(grad_w[t, i])) < 4e-4


# ------------------------------------------------------------------ 8 bits -------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (1, 3, 16), (2, 5, 127), (3, 130, 300), (1, 257, 128), (2, 127, 264), (1, 60, 1000)])
def test_quantise_blocks(ds, dtype, E, N, K):
    g = gen(E * N + K)
    for pad in (0, 3, 8):
        big = (normal(g, E, N + 1, K + pad) * torch.exp(4 * normal(g, E, N + 1, 1))).to(dtype)
        x = big[:, :N, :K]
        x[0, 0] = 0.0
        for block in (1, 128):
            codes, scales = ds.quantise_blocks(x, block_rows=block)
            want, want_scales = ref.quantise(x, block)
            assert torch.equal(scales.double(), want_scales)
            assert torch.equal(codes.double(), want)
            c2, s2 = ds.quantise_blocks(x[0], block_rows=block)
            assert torch.equal(c2.double(), want[0]) and torch.equal(s2.double(), want_scales[0])


def test_quantise_blocks_at_the_ends(ds):
    """The borders between scales, ties of codes, the smallest and largest numbers."""
    x = torch.zeros(1, 12, 128, device="cuda")
    x[0, 0, 0], x[0, 0, 1] = 448.0, 2.0 ** -10                      # the border itself; half of the smallest code
    x[0, 1, 0] = torch.nextafter(torch.tensor(448.0), torch.tensor(500.0))  # one step above
    x[0, 2, 5] = 2.0 ** -149                                        # the smallest number
    x[0, 3, 127] = torch.finfo(torch.float32).max
    x[0, 3, 126] = -torch.finfo(torch.float32).max
    x[0, 4] = torch.linspace(-448, 448, 128, device="cuda")
    x[0, 5, :8] = torch.tensor([448, 17.0, 18, 19, 21, -17, -19, 2.0 ** -9 * 1.5], device="cuda")  # ties
    x[0, 6, 0] = 448 * 2.0 ** -126
    x[0, 7, 0] = 449 * 2.0 ** -126
    x[0, 8] = -0.0
    x[0, 9, :2] = torch.tensor([1e30, 1e-30], device="cuda")
    x[0, 10, 64] = 2.0 ** 127
    x[0, 11, 3] = -3.5
    for block in (1, 128):
        codes, scales = ds.quantise_blocks(x, block_rows=block)
        want, want_scales = ref.quantise(x, block)
        assert torch.equal(scales.double(), want_scales) and torch.equal(codes.double(), want)


# ------------------------------------------------------------------ product ------
# Products of codes are exact.  A block's 128 are summed by the tensor cores (4 instructions of 32,
# whose additions keep fp32's bits: less than a step, 2^-23, of the largest partial sum each, 2^-21
# in all), two roundings for the scales, and the blocks' sums added in fp32: (blocks + 10) 2^-23 of the
# sum of sizes.

def check_product(got, want, size, K, dtype):
    blocks = -(-K // 128)
    limit = (blocks + 10) * 2 * U * size + half_step(dtype) * 1.01 * want.abs() + 1e-37
    assert got.dtype == dtype and got.shape == want.shape
    assert bool(((got.double() - want).abs() <= limit).all())


def operands(g, T, E, N, K):
    x = normal(g, T, K).clamp(-4, 4).mul(100).to(torch.float8_e4m3fn)
    w = normal(g, E, N, K).clamp(-4, 4).mul(100).to(torch.float8_e4m3fn)
    blocks = -(-K // 128)
    return x, torch.exp(normal(g, T, blocks)), w, torch.exp(normal(g, E, -(-N // 128), blocks))


def spread(g, T, E, empty=0.3):
    """Offsets of T rows over E experts of unlike load, some without rows."""
    share = torch.rand(E, device="cuda", generator=g) ** 3
    share[torch.rand(E, device="cuda", generator=g) < empty] = 0.0
    share[E // 2] += 1e-3
    counts = torch.bincount(torch.multinomial(share, T, replacement=True, generator=g), minlength=E)
    return torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), counts.cumsum(0)]).int()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,E,N,K", [
    (1, 1, 1, 16), (1, 1, 128, 128), (1, 1, 1000, 4096), (2, 1, 129, 144), (31, 1, 260, 1040), (33, 1, 64, 2048),
    (127, 1, 256, 256), (128, 1, 257, 128), (129, 1, 640, 400), (300, 1, 200, 1536), (1000, 1, 1030, 528),
    (40, 8, 300, 1040), (700, 8, 130, 512), (5, 64, 72, 656), (900, 160, 136, 272), (3000, 3, 520, 640),
    (2000, 512, 24, 64), (20000, 4, 272, 144), (300, 2, 4096, 2064),
])
def test_expert_product(ds, dtype, T, E, N, K):
    g = gen(T + N + K)
    x, xs, w, ws = operands(g, T, E, N, K)
    offsets = spread(g, T, E)
    got = ds.expert_product(x, xs, w, ws, offsets, dtype=dtype)
    want, size = ref.product(x, xs, w, ws, offsets)
    check_product(got, want, size, K, dtype)
    if E == 1:
        assert torch.equal(ds.expert_product(x, xs, w, ws, dtype=dtype), got)
        assert torch.equal(ds.expert_product(x, xs, w[0], ws[0], dtype=dtype), got)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,E,N,K", [(60, 4, 200, 512), (900, 4, 300, 512), (6, 1, 130, 2048)])
def test_expert_product_rows_outside(ds, dtype, T, E, N, K):
    """Rows before the first offset and behind the last are zeros whatever they hold, and codes that are
    no numbers in one expert's rows or weights stay there."""
    g = gen(T)
    x, xs, w, ws = operands(g, T, E, N, K)
    a, b = T // 5, T - T // 4
    offsets = (a + spread(g, b - a, E, 0.0)).int()
    nan = torch.tensor(0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    x[:a], x[b:], xs[b:] = nan, nan, float("nan")
    want, size = ref.product(x, xs, w, ws, offsets)
    got = ds.expert_product(x, xs, w, ws, offsets, dtype=dtype)
    assert not bool(got[:a].any()) and not bool(got[b:].any())
    check_product(got, want, size, K, dtype)
    # a row of NaN codes, and an expert's weights of them
    bad = (a + b) // 2
    x[bad, 3] = nan
    w[E - 1, 5] = nan
    got = ds.expert_product(x, xs, w, ws, offsets, dtype=dtype)
    fine = torch.ones_like(got, dtype=torch.bool)
    fine[bad] = False
    fine[int(offsets[E - 1]):int(offsets[E]), 5] = False
    check_product(torch.where(fine, got, torch.zeros_like(got)), torch.where(fine, want, 0.0), size, K, dtype)
    assert bool(torch.isnan(got[bad]).all()) and bool(torch.isnan(got[int(offsets[E - 1]):int(offsets[E]), 5]).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,E,N,K", [(20000, 4, 261, 144), (20000, 4, 268, 144), (20000, 30, 1000, 64), (40001, 3, 520, 272),
                                     (25000, 9, 392, 400), (6000, 1, 1304, 528)])
def test_expert_product_of_many_rows(ds, dtype, T, E, N, K):
    """Tiles of 256 outputs, stored by bulk copies where rows allow it: experts' ends within 32 rows, outputs
    that end within a box, rows that start on 2, 4, 8 and 16 bytes, and rows of nobody around them."""
    g = gen(T + N + K)
    x, xs, w, ws = operands(g, T, E, N, K)
    a, b = 3, T - 77
    offsets = (a + spread(g, b - a, E)).int()
    want, size = ref.product(x, xs, w, ws, offsets)
    got = ds.expert_product(x, xs, w, ws, offsets, dtype=dtype)
    check_product(got, want, size, K, dtype)
    assert not bool(got[:a].any()) and not bool(got[b:].any())
    assert torch.equal(got, ds.expert_product(x, xs, w, ws, offsets, dtype=dtype))


def test_expert_product_strides(ds):
    g = gen(9)
    x, xs, w, ws = operands(g, 70, 3, 50, 160)
    offsets = spread(g, 70, 3, 0.0)
    want = ds.expert_product(x, xs, w, ws, offsets, dtype=torch.float32)
    wide = torch.zeros(70, 192, device="cuda").to(torch.float8_e4m3fn)
    wide[:, 16:176] = x
    big = torch.zeros(3, 60, 208, device="cuda").to(torch.float8_e4m3fn)
    big[:, 4:54, 32:192] = w
    got = ds.expert_product(wide[:, 16:176], xs, big[:, 4:54, 32:192], ws, offsets, dtype=torch.float32)
    assert torch.equal(got, want)
    with pytest.raises(ds.DSError):
        ds.expert_product(wide[:, 8:168], xs, w, ws, offsets)  # rows that do not start on 16 bytes


def test_expert_product_of_no_rows(ds):
    g = gen(10)
    x, xs, w, ws = operands(g, 20, 4, 130, 256)
    zeros = torch.zeros(5, dtype=torch.int32, device="cuda")
    assert ds.expert_product(x[:0], xs[:0], w, ws, zeros).shape == (0, 130)
    assert not bool(ds.expert_product(x, xs, w, ws, zeros).any())


def test_results_do_not_change(ds):
    """Calls again on the same inputs give the same bits (no order of atomics, no splits by time)."""
    g = gen(11)
    x, tokens = rows_of(torch.bfloat16, 3, 100003, 1)
    first = ds.token_logprobs(x, tokens, top=20)
    a, xs, w, ws = operands(g, 5, 2, 700, 4096)
    offsets = spread(g, 5, 2)
    p = ds.expert_product(a, xs, w, ws, offsets, dtype=torch.float32)
    for _ in range(20):
        assert all(torch.equal(u, v) for u, v in zip(first, ds.token_logprobs(x, tokens, top=20)))
        assert torch.equal(p, ds.expert_product(a, xs, w, ws, offsets, dtype=torch.float32))


# ------------------------------------------------------------------ together -----

class Layer:
    """A layer of experts with 8-bit weights: gate, sorting, two products, weighted sums."""

    def __init__(self, ds, D=256, F=384, E=16, k=4):
        g = gen(12)
        self.ds, self.E, self.k = ds, E, k
        self.gate = normal(g, D, E) * D ** -0.5
        self.up = ds.quantise_blocks(normal(g, E, 2 * F, D) * D ** -0.5, block_rows=128)
        self.down = ds.quantise_blocks(normal(g, E, D, F) * F ** -0.5, block_rows=128)

    def __call__(self, x):
        ds = self.ds
        weights, experts = ds.route(x.float() @ self.gate, self.k)
        places, offsets = ds.expert_sort(experts, self.E)
        rows = ds.expert_gather(x, places, offsets, quantise=True)
        both = ds.expert_product(*rows, *self.up, offsets)
        a, b = both.chunk(2, -1)
        hidden = torch.nn.functional.silu(a) * b
        codes = ds.quantise_blocks(hidden)
        y = ds.expert_product(*codes, *self.down, offsets)
        out = ds.expert_combine(y, places, weights)
        return out, (weights, experts, places, offsets, rows, both, hidden, codes, y)


@pytest.mark.parametrize("T", [1, 7, 130, 600])
def test_layer_of_experts(ds, T):
    """A run through the layer, each step against its definition in 64 bits from what the step
    before it gave, and each token's rows found again by the gate's choices: the steps' own limits
    hold, and 8 bits need no limit of their own."""
    layer = Layer(ds)
    x = normal(gen(T), T, 256).bfloat16()
    out, (weights, experts, places, offsets, rows, both, hidden, codes, y) = layer(x)
    assert int(offsets[-1]) == 4 * T and bool((places >= 0).all())
    e = experts.long()
    for i in range(4):  # choice i of each token lies among its expert's rows, and is the token
        at = places[:, i].long()
        assert bool(((at >= offsets[e[:, i]]) & (at < offsets[e[:, i] + 1])).all())
        want, scales = ref.quantise(x[None], 1)
        assert torch.equal(rows[0][at].double(), want[0]) and torch.equal(rows[1][at].double(), scales[0])
    check_product(both, *ref.product(*rows, *layer.up, offsets), 256, torch.bfloat16)
    want, scales = ref.quantise(hidden[None], 1)
    assert torch.equal(codes[0].double(), want[0]) and torch.equal(codes[1].double(), scales[0])
    check_product(y, *ref.product(*codes, *layer.down, offsets), 384, torch.bfloat16)
    want, size = ref.combine(y, places, weights)
    assert bool(((out.double() - want).abs() <= 5 * U * size + half_step(torch.bfloat16) * 1.01 * want.abs() + 1e-37).all())


def test_layer_captured_and_on_another_stream(ds):
    layer = Layer(ds)
    x = normal(gen(1), 64, 256).bfloat16()
    layer(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want, _ = layer(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    held = x.clone()
    with torch.cuda.graph(graph):
        out, _ = layer(held)
    other = normal(gen(2), 64, 256).bfloat16()
    for v in (x, other, x):
        held.copy_(v)
        graph.replay()
        assert torch.equal(out, layer(v)[0])
    assert torch.equal(out, want)


@pytest.mark.parametrize("T,V", [(1, 129280), (700, 1003)])
def test_log_probabilities_captured(ds, T, V):
    """Forward and backward in a graph, replayed on other logits: one row on a cluster, and many rows."""
    x, tokens = rows_of(torch.bfloat16, T, V, 5)
    grad = normal(gen(6), T)

    def step(x):
        lp, lse, H, top_lp, top = ds.token_logprobs(x, tokens, top=9)
        return lp, lse, H, top_lp, top, ds.token_logprobs_backward(grad, x, tokens, lse, grad_entropy=grad, entropy=H)
    step(x)
    held = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(held)
    other, _ = rows_of(torch.bfloat16, T, V, 7)
    for v in (x, other, x):
        held.copy_(v)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, step(v)))


def test_two_streams_at_once(ds):
    g = gen(13)
    streams = [torch.cuda.Stream() for _ in range(2)]
    data = []
    for i in range(2):
        x, tokens = rows_of(torch.float32, 50, 30001, i)
        a, xs, w, ws = operands(g, 400, 4, 500, 1024)
        data.append((x, tokens, a, xs, w, ws, spread(g, 400, 4)))
    want = [(ds.token_logprobs(d[0], d[1], top=5), ds.expert_product(*d[2:])) for d in data]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((ds.token_logprobs(data[i][0], data[i][1], top=5), ds.expert_product(*data[i][2:])))
    torch.cuda.synchronize()
    for i in range(2):
        for lp, p in got[i]:
            assert all(torch.equal(u, v) for u, v in zip(lp, want[i][0])) and torch.equal(p, want[i][1])


def test_a_stream_of_the_callers(ds):
    """`stream=`: the calls wait for what that stream does before, not for the current one."""
    side = torch.cuda.Stream()
    e = torch.zeros(100, 4, dtype=torch.int32, device="cuda")
    x = torch.zeros(100, 64, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        e.copy_(torch.arange(400, device="cuda").view(100, 4) % 7)
        x.fill_(3.0)
    h = side.cuda_stream
    places, offsets = ds.expert_sort(e, 7, stream=h)
    rows = ds.expert_gather(x, places, offsets, stream=h)
    back = ds.expert_combine(rows, places, stream=h)
    codes, scales = ds.quantise_blocks(x, stream=h)
    lp = ds.token_logprobs(x, e[:, 0].contiguous(), stream=None)  # the current stream: any order
    side.synchronize()
    assert offsets.tolist()[-1] == 400 and bool((back == 12.0).all()) and bool((codes.float() * scales == 3.0).all())
    assert lp[0].shape == (100,)


# ------------------------------------------------------------------ refusals -----

def test_refusals(ds):
    x = torch.zeros(4, 64, device="cuda")
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    p = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    o = torch.zeros(9, dtype=torch.int32, device="cuda")
    c = torch.zeros(8, 64, device="cuda").to(torch.float8_e4m3fn)
    s = torch.zeros(8, 1, device="cuda")
    w, ws = torch.zeros(8, 32, 64, device="cuda").to(torch.float8_e4m3fn), torch.zeros(8, 1, 1, device="cuda")
    for error, call in [
        (TypeError, lambda: ds.token_logprobs(x.half(), t)),
        (TypeError, lambda: ds.token_logprobs(x, t.long())),
        (ValueError, lambda: ds.token_logprobs(x, t[:3])),
        (ValueError, lambda: ds.token_logprobs(x.t(), t)),
        (ValueError, lambda: ds.token_logprobs(x[0], t)),
        (ValueError, lambda: ds.token_logprobs(x, t, top=65)),
        (ds.DSError, lambda: ds.token_logprobs(x, t, top=33)),
        (ds.DSError, lambda: ds.token_logprobs(x, t, top=-1)),
        (ds.DSError, lambda: ds.token_logprobs(x[:1].expand(4, 64), t)),     # rows that overlap
        (ValueError, lambda: ds.token_logprobs_backward(s[:4, 0], x, t, s[:4, 0], grad_entropy=s[:4, 0])),
        (ValueError, lambda: ds.token_logprobs_backward(s[:3, 0].clone(), x, t, s[:4, 0].clone())),
        (TypeError, lambda: ds.expert_sort(p.long(), 8)),
        (ValueError, lambda: ds.expert_sort(t, 8)),
        (ds.DSError, lambda: ds.expert_sort(p, 0)),
        (ds.DSError, lambda: ds.expert_sort(p, 513)),
        (ds.DSError, lambda: ds.expert_sort(torch.zeros(4, 33, dtype=torch.int32, device="cuda"), 8)),
        (ValueError, lambda: ds.expert_gather(x, p[:3], o)),
        (ValueError, lambda: ds.expert_gather(x, p, o[:1])),
        (TypeError, lambda: ds.expert_gather(x.half(), p, o)),
        (ValueError, lambda: ds.expert_combine(x, p, torch.zeros(4, 3, device="cuda"))),
        (TypeError, lambda: ds.expert_combine(x, p, torch.zeros(4, 2, device="cuda").bfloat16())),
        (ValueError, lambda: ds.expert_combine_backward(x, x, p, o, torch.zeros(4, 2, device="cuda"))),  # y of 4 rows
        (TypeError, lambda: ds.expert_combine_backward(x, torch.zeros(8, 64, device="cuda").bfloat16(), p, o, torch.zeros(4, 2, device="cuda"))),
        (ValueError, lambda: ds.quantise_blocks(x, block_rows=64)),
        (TypeError, lambda: ds.quantise_blocks(x.half())),
        (ValueError, lambda: ds.quantise_blocks(x.view(1, 1, 4, 64))),
        (TypeError, lambda: ds.expert_product(x, s[:4], w, ws, o)),
        (ValueError, lambda: ds.expert_product(c, s[:4], w, ws, o)),
        (ValueError, lambda: ds.expert_product(c, s, w, ws)),
        (ValueError, lambda: ds.expert_product(c, s, w, ws, o[:8])),
        (ValueError, lambda: ds.expert_product(c, s, w, ws[:, :, :0], o)),
        (ValueError, lambda: ds.expert_product(c[:, :48], s, w, ws, o)),
        (TypeError, lambda: ds.expert_product(c, s, w.view(torch.float8_e5m2), ws, o)),
    ]:
        with pytest.raises(error):
            call()
