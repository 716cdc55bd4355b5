"""The operators around the top-k on the GPU against their definitions in 64 bits
(operator_ref).  Tolerances follow from the roundings each kernel makes and are given where
they are used; whole numbers are equal wherever no comparison lies within fp32's rounding."""
import math

import numpy as np
import pytest

import operator_ref as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(scope="module")
def ds():
    import top_selection_gb300 as m
    return m


DTYPES = [torch.bfloat16, torch.float32]


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.detach().cpu().double().numpy() if t.is_floating_point() else t.cpu().numpy()


# ------------------------------------------------------------------ gate ---------
# fp32 steps: a score is off by the exponential's argument (2^-24 |x - max|, here below 20)
# and a few roundings; the sums of positive terms add less than 2^-24 * 10.  A choice value
# (score + bias, below 2) is off by less than 1e-6.
GATE_REL, GATE_MARGIN = 5e-6, 2e-6


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,k,scoring,bias,groups,topk_groups,score", [
    (256, 8, "sigmoid", True, 8, 4, "top2"),
    (256, 8, "softmax", False, 8, 3, "max"),
    (60, 4, "softmax", False, 1, 1, "max"),
    (8, 2, "softmax", False, 1, 1, "max"),
    (1, 1, "sigmoid", False, 1, 1, "max"),
    (2, 2, "softmax", True, 2, 2, "top2"),
    (33, 5, "sigmoid", True, 1, 1, "max"),
    (255, 32, "sigmoid", False, 1, 1, "max"),
    (512, 8, "softmax", True, 16, 2, "top2"),
    (511, 1, "softmax", False, 1, 1, "max"),
    (160, 6, "softmax", False, 8, 3, "top2"),
    (160, 6, "sigmoid", True, 8, 7, "max"),
    (96, 4, "sigmoid", True, 3, 2, "top2"),
    (480, 10, "sigmoid", True, 24, 11, "top2"),
    (32, 3, "sigmoid", True, 32, 5, "top2"),
])
def test_route(ds, dtype, E, k, scoring, bias, groups, topk_groups, score):
    rng = np.random.default_rng(E * 7 + k)
    for rows in (1, 9, 70):
        for renormalise, scale in ((True, 1.0), (False, 2.5)):
            x = dev((1.5 * rng.standard_normal((rows, E + 3))).astype(np.float32), dtype)[:, :E]
            b = (0.1 * rng.standard_normal(E)).astype(np.float32) if bias else None
            counts = torch.full((E,), 3, dtype=torch.int32, device="cuda")
            w, e = ds.route(x, k, scoring=scoring, bias=None if b is None else dev(b), groups=groups,
                            topk_groups=topk_groups, group_score=score, renormalise=renormalise, scale=scale,
                            counts=counts)
            xh = host(x)
            want, margin = ref.route(xh, k, scoring, b, groups, topk_groups, score)
            sure = (margin > GATE_MARGIN) | (margin == 0) if b is None else margin > GATE_MARGIN
            # bf16 logits tie often, and exactly; the lower index is then the answer
            eh = host(e)
            assert np.array_equal(eh[sure], want[sure])
            assert sure.mean() > 0.8 or rows < 9
            got = host(w)
            exact = ref.route_weights(xh, eh.astype(np.int64), scoring, renormalise, scale)
            assert np.allclose(got, exact, rtol=GATE_REL, atol=1e-37)
            assert np.array_equal(host(counts) - 3, np.bincount(eh.ravel(), minlength=E))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,k", [(256, 8), (60, 4), (33, 1), (8, 8), (512, 32)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_route_backward(ds, dtype, E, k, scoring, renormalise):
    """Against the chain rule in 64 bits.  An element is a difference of products g s of the
    order |g|max * max s * scale; fp32 keeps 1e-5 of that, bf16 rounds the result (2^-8)."""
    rng = np.random.default_rng(E + k)
    rows = 19
    x = dev((1.5 * rng.standard_normal((rows, E + 5))).astype(np.float32), dtype)[:, :E]
    g = rng.standard_normal((rows, k)).astype(np.float32)
    w, e = ds.route(x, k, scoring=scoring, renormalise=renormalise, scale=2.5)
    got = host(ds.route_backward(dev(g), x, e, scoring=scoring, renormalise=renormalise, scale=2.5))
    want = ref.route_gradient(g, host(x), host(e).astype(np.int64), scoring, renormalise, 2.5)
    size = 2.5 * np.abs(g).max(-1, keepdims=True)
    limit = 1e-5 * size + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0)
    assert np.all(np.abs(got - want) <= limit)


def test_route_gradient_against_differences(ds):
    """The kernel's gradient against differences of the kernel's own weights: fp32 weights of
    the order 1, off by 1e-6, over a step of 2 h = 0.02: 1e-4, and h^2 = 1e-4 for the slope."""
    rng = np.random.default_rng(8)
    x = rng.standard_normal((1, 16)).astype(np.float32)
    x[0, :4] += 4.0  # the choice stays the same under a step
    g = rng.standard_normal((1, 4)).astype(np.float32)
    for scoring in ("softmax", "sigmoid"):
        for renormalise in (False, True):
            w, e = ds.route(dev(x), 4, scoring=scoring, renormalise=renormalise)
            assert sorted(host(e)[0].tolist()) == [0, 1, 2, 3]
            got = host(ds.route_backward(dev(g), dev(x), e, scoring=scoring, renormalise=renormalise))[0]
            place = {int(v): j for j, v in enumerate(host(e)[0])}
            for c in range(16):
                total = 0.0
                for sign in (1, -1):
                    y = x.copy()
                    y[0, c] += np.float32(sign * 0.01)
                    w2, e2 = ds.route(dev(y), 4, scoring=scoring, renormalise=renormalise)
                    total += sign * sum(float(w2[0, j]) * g[0, place[int(e2[0, j])]] for j in range(4))
                assert abs(total / 0.02 - got[c]) < 4e-4 * (1 + np.abs(g).sum())


def test_route_ties_and_infinities(ds):
    inf = math.inf
    x = torch.tensor([[1.0, 3.0, 3.0, -2.0, 3.0, 1.0], [0.0, -0.0, 0.0, -0.0, 0.0, -0.0],
                      [-inf, 2.0, -inf, -inf, 1.0, -inf], [-inf] * 6], device="cuda")
    w, e = ds.route(x, 4)
    assert e.tolist() == [[1, 2, 4, 0], [0, 1, 2, 3], [1, 4, 0, 2], [0, 1, 2, 3]]
    z = math.e ** -1
    assert torch.allclose(w.cpu(), torch.tensor([[1 / (3 + z * z)] * 3 + [z * z / (3 + z * z)], [0.25] * 4,
                                                 [1 / (1 + z), z / (1 + z), 0, 0], [0] * 4]), rtol=GATE_REL, atol=0)
    # equal group scores: the lower group
    w, e = ds.route(x[1:2], 2, scoring="sigmoid", groups=3, topk_groups=1, group_score="top2")
    assert e.tolist() == [[0, 1]]
    back = ds.route_backward(torch.ones(4, 4, device="cuda"), x, ds.route(x, 4)[1])
    assert torch.isfinite(back).all() and back[3].abs().max() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_route_alignment(ds, dtype, shift):
    """Logits, bias, and the experts' and gradient's rows that start anywhere."""
    rng = np.random.default_rng(shift)
    rows, E, k = 5, 256, 8
    x = dev((1.5 * rng.standard_normal((rows, E))).astype(np.float32), dtype)
    b = dev((0.1 * rng.standard_normal(E)).astype(np.float32))
    kw = dict(scoring="sigmoid", groups=8, topk_groups=4, group_score="top2")
    w, e = ds.route(x, k, bias=b, **kw)
    wide = torch.zeros(E + 4, device="cuda")[shift:shift + E].copy_(b)
    w2, e2 = ds.route(x, k, bias=wide, **kw)
    assert torch.equal(w, w2) and torch.equal(e, e2)
    xs = torch.zeros(rows, E + 8, device="cuda", dtype=dtype)[:, shift:shift + E].copy_(x)
    w2, e2 = ds.route(xs, k, bias=wide, **kw)
    assert torch.equal(w, w2) and torch.equal(e, e2)
    g = dev(rng.standard_normal((rows, k)).astype(np.float32))
    assert torch.equal(ds.route_backward(g, xs, e, scoring="sigmoid"), ds.route_backward(g, x, e, scoring="sigmoid"))


def test_route_backward_ignores_outside_indices(ds):
    x = torch.randn(3, 20, device="cuda")
    e = torch.tensor([[2, -1, 5], [20, 3, 1 << 30], [-1, -1, -1]], dtype=torch.int32, device="cuda")
    got = ds.route_backward(torch.ones(3, 3, device="cuda"), x, e, renormalise=False)
    assert torch.isfinite(got).all()
    want = ref.route_gradient(np.array([[1.0, 1.0]]), host(x[:1]), np.array([[2, 5]]), "softmax", False, 1.0)
    assert np.allclose(host(got[:1]), want, atol=1e-6) and got[2].abs().max() == 0


def test_route_empty(ds):
    w, e = ds.route(torch.zeros(0, 64, device="cuda"), 4)
    assert w.shape == (0, 4) and e.shape == (0, 4)
    with pytest.raises(ds.DSError):
        ds.route(torch.zeros(2, 64, device="cuda"), 65)
    with pytest.raises(TypeError):
        ds.route(torch.zeros(2, 64, device="cuda", dtype=torch.float16), 4)
    with pytest.raises(ValueError):
        ds.route(torch.zeros(2, 64, device="cuda"), 4, scoring="linear")
    with pytest.raises(ValueError):
        ds.route(torch.zeros(2, 64, device="cuda"), 4, bias=torch.zeros(63, device="cuda"))


# ------------------------------------------------------------------ verification --
# A probability is off by its exponent's argument, 2^-23 * |x - max| / temperature (below 60
# in exponents that matter), and the sum: 1e-5.
VERIFY_REL = 1e-5


def verify_case(rng, B, S, V, dtype, probs, temp):
    x = 2.0 * rng.standard_normal((B, S + 1, V))
    at = rng.integers(V, size=(B, S + 1, 3))
    np.put_along_axis(x, at, 6.0 + 3.0 * rng.random((B, S + 1, 3)), -1)
    xt = dev(x.astype(np.float32), dtype)
    xh = host(xt)
    t = np.where(temp > 0, temp, 0.05)
    p = np.stack([ref.scores(xh[b, :S] / t[b], "softmax") for b in range(B)])
    if probs:
        other = ref.scores(2.0 * rng.standard_normal((B, S, V)), "softmax")
        q = (0.7 * p + 0.3 * other).astype(np.float32)
        drafts = (q / rng.exponential(size=q.shape)).argmax(-1)
    else:
        q = None
        drafts = np.where(rng.random((B, S)) < 0.6, p.argmax(-1), rng.integers(V, size=(B, S)))
    return xt, xh, q, drafts.astype(np.int32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,S,V", [(1, 1, 1), (3, 2, 7), (5, 4, 1000), (2, 3, 32003), (9, 5, 4097), (1, 0, 513),
                                   (2, 1, 129280), (40, 2, 2048)])
@pytest.mark.parametrize("probs", [True, False])
def test_verify(ds, dtype, B, S, V, probs):
    rng = np.random.default_rng(B * 100 + S * 10 + V)
    temp = rng.uniform(0.4, 1.5, B).astype(np.float32)
    temp[B // 2] = 0.0 if B > 1 else temp[B // 2]
    xt, xh, q, drafts = verify_case(rng, B, S, V, dtype, probs, temp)
    u = rng.random((B, S)).astype(np.float32)
    noise = rng.exponential(size=(B, V)).astype(np.float32).clip(1e-10)
    lens = rng.integers(S + 1, size=B).astype(np.int32) if B > 2 else None
    tok, acc, pr = ds.verify_drafts(xt, dev(drafts), dev(u), dev(noise), draft_probs=None if q is None else dev(q),
                                    draft_lens=None if lens is None else dev(lens), temperature=dev(temp))
    wt, wa, wp, margin = ref.verify(xh, drafts, u, noise, q, lens, temp)
    sure = margin > 1e-4
    assert sure.mean() >= 0.9 or B < 9
    assert np.array_equal(host(tok)[sure], wt[sure]) and np.array_equal(host(acc)[sure], wa[sure])
    assert np.allclose(host(pr)[sure], wp[sure], rtol=VERIFY_REL, atol=1e-30)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shift", [0, 1, 2, 3, 5, 7])
def test_verify_strides_and_alignment(ds, dtype, shift):
    """Rows that start anywhere: logits, probabilities and noise inside wider buffers."""
    rng = np.random.default_rng(shift)
    B, S, V = 4, 2, 1531
    temp = np.full(B, 0.8, dtype=np.float32)
    xt, xh, q, drafts = verify_case(rng, B, S, V, dtype, True, temp)
    u = rng.random((B, S)).astype(np.float32)
    noise = rng.exponential(size=(B, V)).astype(np.float32)
    wide = torch.full((B, S + 2, V + 13), math.inf, dtype=dtype, device="cuda")
    view = wide[:, 1:, shift:shift + V]
    view.copy_(xt)
    qw = torch.full((B, S, V + 9), math.inf, device="cuda")
    qv = qw[:, :, (shift + 1):(shift + 1) + V]
    qv.copy_(dev(q))
    nw = torch.full((B, V + 8), 1e-30, device="cuda")
    nv = nw[:, shift:shift + V]
    nv.copy_(dev(noise))
    tok, acc, pr = ds.verify_drafts(view, dev(drafts), dev(u), nv, draft_probs=qv, temperature=0.8)
    wt, wa, wp, margin = ref.verify(xh, drafts, u, noise, q, None, np.float32(0.8))
    assert margin.min() > 1e-4
    assert np.array_equal(host(tok), wt) and np.array_equal(host(acc), wa)
    assert np.allclose(host(pr), wp, rtol=VERIFY_REL)


def test_verify_edges(ds):
    inf = math.inf
    V = 6
    row = [0.0, 1.0, 1.0, -inf, 0.5, -inf]
    x = torch.tensor([[row, row], [[-inf] * V, row], [row, [-inf] * V], [row, row], [row, row], [row, row]],
                     device="cuda")
    u = torch.zeros(6, 1, device="cuda")
    noise = torch.ones(6, V, device="cuda")
    drafts = torch.tensor([[3], [1], [1], [-1], [V], [1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([1, 1, 1, 1, 1, -4], dtype=torch.int32, device="cuda")
    tok, acc, pr = ds.verify_drafts(x, drafts, u, noise, draft_lens=lens)
    p = ref.scores(np.array([row]), "softmax")[0]
    # an excluded token is refused at u = 0; a row of -inf alone has no distribution; tokens
    # outside the vocabulary are refused; a negative length is none; ties to the lowest index
    assert tok.tolist() == [[1, -1], [-1, -1], [1, -1], [1, -1], [1, -1], [1, -1]]
    assert acc.tolist() == [0, 0, 1, 0, 0, 0]
    assert np.allclose(host(pr), [[p[1], 0], [0, 0], [p[1], 0], [p[1], 0], [p[1], 0], [p[1], 0]], rtol=1e-6)
    # a draft distribution that covers the target's everywhere: the token comes from the target
    big = torch.full((6, 1, V), 2.0, device="cuda")
    tok, acc, pr = ds.verify_drafts(x[3:], drafts[:3], u[:3] + 0.99, noise[:3], draft_probs=big[:3])
    assert tok.tolist() == [[1, -1]] * 3 and acc.tolist() == [0, 0, 0]
    # temperature 0: the first maximum
    tok, acc, pr = ds.verify_drafts(x[3:], drafts[:3], u[:3] + 0.99, noise[:3], temperature=0.0)
    assert tok.tolist() == [[1, -1], [1, 1], [1, 1]] and acc.tolist() == [0, 1, 1]
    assert pr.tolist() == [[1, 0], [1, 1], [1, 1]]
    tok, acc, pr = ds.verify_drafts(x[:0], drafts[:0], u[:0], noise[:0])
    assert tok.shape == (0, 2) and acc.shape == (0,)
    with pytest.raises(ValueError):
        ds.verify_drafts(x, drafts[:, :0], u, noise)
    with pytest.raises(TypeError):
        ds.verify_drafts(x, drafts.long(), u, noise)
    with pytest.raises(ds.DSError):
        ds.verify_drafts(x, drafts, u, noise, temperature=-1.0)


def test_verify_emits_the_target_distribution(ds):
    """The first emitted token is distributed as the target's sample whatever the draft's
    distribution: shares of 60000 sequences within five standard deviations."""
    V, n = 5, 60000
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.tensor([0.3, 1.2, -0.5, 0.0, 0.9], device="cuda")
    q = torch.tensor([0.5, 0.1, 0.2, 0.15, 0.05], device="cuda")
    drafts = (q / torch.empty(n, V, device="cuda").exponential_(generator=g)).argmax(-1).int()[:, None]
    u = torch.rand(n, 1, device="cuda", generator=g)
    noise = torch.empty(n, V, device="cuda").exponential_(generator=g)
    tok, acc, _ = ds.verify_drafts(logits.expand(n, 2, V).contiguous(), drafts, u, noise,
                                   draft_probs=q.expand(n, 1, V).contiguous(), temperature=0.7)
    got = torch.bincount(tok[:, 0].long(), minlength=V).cpu().numpy() / n
    p = ref.scores(host(logits)[None] / 0.7, "softmax")[0]
    assert np.all(np.abs(got - p) <= 5 * np.sqrt(p * (1 - p) / n))


# ------------------------------------------------------------------ 4-bit cache ---

def new_cache(pages, heads, page, D, junk=True):
    """A cache full of junk (codes of 15, scales of NaN): what is not stored is not used."""
    cache = torch.full((pages, heads, page, 2, D // 2), 255 if junk else 0, dtype=torch.uint8, device="cuda")
    scales = torch.full((pages, heads, page, 4), math.nan if junk else 0.0, dtype=torch.bfloat16, device="cuda")
    return cache, scales


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,heads,D,page", [(1, 1, 64, 1), (5, 3, 128, 16), (67, 8, 128, 64), (130, 2, 64, 32), (33, 5, 64, 2)])
def test_cache_store_and_load(ds, dtype, T, heads, D, page):
    """The stored bits are the format's, exactly; reading back rounds once."""
    rng = np.random.default_rng(T)
    pages = -(-T // page) + 2
    cache, scales = new_cache(pages, heads, page, D)
    x = rng.standard_normal((2, T, heads, D)) * np.exp(rng.uniform(-9, 9, (2, T, heads, 1)))
    x[0, 0, 0] = 3.25           # a constant row
    x[1, 0, 0] = 0.0
    k, v = dev(x[0].astype(np.float32), dtype), dev(x[1].astype(np.float32), dtype)
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    slots[T // 2] = -1 if T > 1 else slots[T // 2]
    slots[T // 3] = pages * page if T > 3 else slots[T // 3]
    ds.cache_store(k, v, cache, scales, dev(slots))
    kb, vb = ds.cache_load(cache, scales, dev(slots), dtype=torch.float32)
    kh, vh = ds.cache_load(cache, scales, dev(slots))
    c, s = cache.cpu().numpy(), scales.cpu().float().numpy()
    used = np.zeros((pages, page), dtype=bool)
    for i, t in enumerate(slots):
        for n, (src, back, low) in enumerate(((k, kb, kh), (v, vb, vh))):
            if not 0 <= t < pages * page:
                assert back[i].abs().max() == 0 and low[i].abs().max() == 0
                continue
            used[t // page, t % page] = True
            codes, sc, m = ref.quantise(src[i].float().cpu().numpy())
            assert np.array_equal(c[t // page, :, t % page, n], ref.pack(codes))
            assert np.array_equal(s[t // page, :, t % page, 2 * n], sc)
            assert np.array_equal(s[t // page, :, t % page, 2 * n + 1], m)
            full = ref.value(codes, sc, m).astype(np.float32)
            assert np.array_equal(back[i].cpu().numpy(), full)
            assert np.array_equal(low[i].float().cpu().numpy(), ref.bf16(full))
    free = np.broadcast_to(~used[:, None], (pages, heads, page))
    assert np.all(c[free] == 255) and np.all(np.isnan(s[free]))


def test_cache_store_strides_and_refusals(ds):
    T, heads, D, page = 7, 2, 64, 16
    packed = torch.randn(T, 3, heads, D, device="cuda").bfloat16()  # q, k, v side by side
    k, v = packed[:, 1], packed[:, 2].transpose(0, 1).contiguous().transpose(0, 1)
    a, b = new_cache(2, heads, page, D), new_cache(2, heads, page, D)
    slots = torch.arange(3, 3 + T, dtype=torch.int32, device="cuda")
    ds.cache_store(k, v, *a, slots)
    ds.cache_store(k.contiguous(), v.contiguous(), *b, slots)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1].view(torch.int16), b[1].view(torch.int16))
    with pytest.raises(ds.DSError):
        ds.cache_store(torch.randn(T, heads, D + 1, device="cuda").bfloat16()[..., 1:], v, *a, slots)
    with pytest.raises(ValueError):
        ds.cache_store(k[:, :1], v, *a, slots)
    with pytest.raises(TypeError):
        ds.cache_store(k, v, *a, slots.long())
    with pytest.raises(TypeError):
        ds.cache_store(k, v, a[0], a[1].float(), slots)
    ds.cache_store(k[:0], v[:0], *a, slots[:0])


# ------------------------------------------------------------------ attention -----

class Paged:
    """Keys and values of a paged cache in 64 bits."""

    def __init__(self, cache, scales, table):
        self.c, self.s = cache.cpu().numpy(), scales.cpu().float().numpy().astype(np.float64)
        self.t = table.cpu().numpy()
        self.pages, self.heads, self.page = self.c.shape[:3]
        self.width = self.t.shape[1] * self.page

    def __call__(self, b, h, pos):
        pg = self.t[b, pos // self.page]
        there = (pg >= 0) & (pg < self.pages)
        at = np.where(there, pg, 0), h, pos % self.page
        codes, s = ref.unpack(self.c[at]).astype(np.float64), self.s[at]
        return codes[:, 0] * s[:, 0:1] + s[:, 1:2], codes[:, 1] * s[:, 2:3] + s[:, 3:4], there


def filled(ds, rng, B, heads, D, page, lens, extra=3, width=None):
    """A cache with the sequences' positions stored through cache_store, the rest junk."""
    width = width or max(1, -(-int(max(lens)) // page))
    pages = B * width + extra
    cache, scales = new_cache(pages, heads, page, D)
    table = rng.permutation(pages)[:B * width].reshape(B, width).astype(np.int32)
    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        pos = np.arange(n)
        slots = table[b][pos // page] * page + pos % page
        kv = rng.standard_normal((2, n, heads, D)).astype(np.float32)
        kv[0] += 0.5 * rng.standard_normal((1, heads, D))
        ds.cache_store(dev(kv[0]), dev(kv[1]), cache, scales, dev(slots.astype(np.int32)))
    return cache, scales, dev(table)


def check_attention(got, want, kv_max, dtype):
    """bf16: the result's rounding (2^-8 of it) and the weights' (16 bits, 2^-16 each); fp32:
    scores of up to ~40 keep 2^-23 * 40 * 2, the weights' error, times the values' size."""
    out, lse = host(got[0]), host(got[1])
    limit = 2.0 ** -8 * np.abs(want[0]) + 2.0 ** -13 * kv_max if dtype == torch.bfloat16 else 3e-5 * kv_max
    assert np.all(np.isfinite(out))
    assert np.all(np.abs(out - want[0]) <= limit)
    empty = np.isneginf(want[1])
    assert np.array_equal(np.isneginf(lse), empty)
    assert np.all(out[empty] == 0)
    assert np.all(np.abs(lse[~empty] - want[1][~empty]) <= 3e-5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,Q,hq,heads,D,page,lens", [
    (1, 1, 1, 1, 64, 16, [1]),
    (1, 1, 8, 8, 128, 64, [33]),
    (3, 1, 8, 2, 128, 16, [0, 1, 100]),
    (2, 1, 32, 4, 128, 64, [300, 129]),
    (4, 3, 8, 2, 64, 16, [2, 0, 3, 77]),          # fewer positions than tokens
    (2, 5, 16, 1, 128, 32, [500, 257]),           # 80 query rows on one key head
    (2, 2, 6, 2, 64, 1, [40, 5]),                 # pages of one position, 3 heads to a group
    (1, 1, 4, 1, 128, 128, [5000]),               # split over CTAs
    (1, 4, 16, 2, 64, 64, [3001]),
    (5, 1, 4, 4, 64, 8, [7, 8, 9, 31, 32]),
])
def test_attention(ds, dtype, B, Q, hq, heads, D, page, lens):
    rng = np.random.default_rng(sum(lens) + hq)
    cache, scales, table = filled(ds, rng, B, heads, D, page, lens)
    q = dev((1.5 * rng.standard_normal((B, Q, hq, D))).astype(np.float32), dtype)
    ln = dev(np.array(lens, dtype=np.int32))
    want = ref.attention(host(q), Paged(cache, scales, table), lens)
    check_attention(ds.cache_attention(q, cache, scales, table, ln), want, 5.0, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,Q,hq,heads,D,K,lens", [
    (2, 1, 8, 1, 128, 1, [50, 0]),
    (2, 1, 16, 2, 128, 40, [300, 20]),
    (1, 3, 4, 2, 64, 33, [90]),
    (3, 2, 32, 2, 64, 200, [1000, 1, 130]),
    (1, 1, 64, 1, 128, 2048, [4000]),             # 64 heads on one key head
])
def test_attention_selected(ds, dtype, B, Q, hq, heads, D, K, lens):
    rng = np.random.default_rng(K)
    cache, scales, table = filled(ds, rng, B, heads, D, 32, lens)
    q = dev((1.5 * rng.standard_normal((B, Q, hq, D))).astype(np.float32), dtype)
    idx = np.full((B, Q, K), -1, dtype=np.int32)
    for b in range(B):
        for i in range(Q):
            n = min(K, lens[b])
            idx[b, i, rng.permutation(K)[:n]] = rng.permutation(lens[b])[:n]  # -1 anywhere between
    if K > 10:
        idx[0, 0, 3] = idx[0, 0, 5]      # twice
        idx[0, 0, 7] = 1 << 30           # beyond the context
        idx[0, 0, 9] = -(1 << 30)
    want = ref.attention(host(q), Paged(cache, scales, table), lens, idx)
    got = ds.cache_attention(q, cache, scales, table, dev(np.array(lens, dtype=np.int32)), indices=dev(idx))
    check_attention(got, want, 5.0, dtype)


def test_attention_of_topk_selection(ds):
    """The indexer's path: scores, the top-k of them, attention over the selected positions."""
    rng = np.random.default_rng(2)
    B, n, heads, D, K = 3, 2000, 2, 128, 64
    cache, scales, table = filled(ds, rng, B, heads, D, 64, [n] * B)
    index_scores = torch.randn(B, 2048, device="cuda").bfloat16()
    _, idx = ds.topk(index_scores, K, 0, 0, N=n)
    q = dev(rng.standard_normal((B, 1, 8, D)).astype(np.float32), torch.bfloat16)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    got = ds.cache_attention(q, cache, scales, table, lens, indices=idx.view(B, 1, K))
    want = ref.attention(host(q), Paged(cache, scales, table), [n] * B, host(idx).reshape(B, 1, K))
    check_attention(got, want, 5.0, torch.bfloat16)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_strides_scale_and_large_scores(ds, dtype):
    rng = np.random.default_rng(3)
    B, Q, hq, heads, D, lens = 2, 2, 8, 2, 64, [200, 61]
    cache, scales, table = filled(ds, rng, B, heads, D, 16, lens)
    wide = torch.zeros(B, 20, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + table.shape[1]] = table
    view = wide[:, 2:2 + table.shape[1]]
    base = dev((3.0 * rng.standard_normal((hq, Q, B, D + 1))).astype(np.float32), dtype)
    q = base[..., 1:].permute(2, 1, 0, 3)          # any strides, rows at any alignment
    ln = dev(np.array(lens, dtype=np.int32))
    for scale in (0.05, -0.2, 0.0):
        want = ref.attention(host(q), Paged(cache, scales, view), lens, scale=scale)
        check_attention(ds.cache_attention(q, cache, scales, view, ln, scale=scale), want, 5.0, dtype)


def test_attention_pages_outside_the_cache(ds):
    """A table entry outside [0, pages) hides its positions and is not read."""
    rng = np.random.default_rng(9)
    cache, scales, table = filled(ds, rng, 1, 2, 64, 16, [160])
    table[0, 3], table[0, 6] = -1, cache.shape[0]
    q = dev(rng.standard_normal((1, 1, 4, 64)).astype(np.float32), torch.bfloat16)
    ln = torch.tensor([160], dtype=torch.int32, device="cuda")
    want = ref.attention(host(q), Paged(cache, scales, table), [160])
    check_attention(ds.cache_attention(q, cache, scales, table, ln), want, 5.0, torch.bfloat16)
    # lens beyond the table, and below zero
    ln = torch.tensor([1 << 30], dtype=torch.int32, device="cuda")
    check_attention(ds.cache_attention(q, cache, scales, table, ln), want, 5.0, torch.bfloat16)
    out, lse = ds.cache_attention(q, cache, scales, table, -ln)
    assert out.abs().max() == 0 and torch.isneginf(lse).all()
    with pytest.raises(ValueError):
        ds.cache_attention(q[..., :32], cache, scales, table, ln)
    with pytest.raises(TypeError):
        ds.cache_attention(q, cache, scales, table.long(), ln)
    with pytest.raises(ds.DSError):
        ds.cache_attention(q, cache, scales, table, ln, scale=math.inf)
    assert ds.cache_attention(q[:0], cache, scales, table[:0], ln[:0])[0].shape == (0, 1, 4, 64)
    out, lse = ds.cache_attention(q, cache, scales, table, ln,
                                  indices=torch.empty(1, 1, 0, dtype=torch.int32, device="cuda"))
    assert out.abs().max() == 0 and torch.isneginf(lse).all()


def test_attention_offsets_past_32_bits(ds):
    """A cache of 5 GiB: the pages in use lie behind 4 GiB."""
    rng = np.random.default_rng(10)
    heads, D, page = 8, 128, 128
    pages = (5 << 30) // (heads * page * D)
    cache = torch.empty(pages, heads, page, 2, D // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, heads, page, 4, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[pages - 1, pages - 5, pages - 2]], dtype=torch.int32, device="cuda")
    n = 300
    pos = torch.arange(n, device="cuda")
    slots = (table[0].long()[pos // page] * page + pos % page).int()
    kv = dev(rng.standard_normal((2, n, heads, D)).astype(np.float32))
    ds.cache_store(kv[0], kv[1], cache, scales, slots)
    q = dev(rng.standard_normal((1, 1, 16, D)).astype(np.float32), torch.bfloat16)
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    got = ds.cache_attention(q, cache, scales, table, ln)
    last = slice(pages - 5, pages)
    small = Paged(cache[last], scales[last], table - (pages - 5))
    check_attention(got, ref.attention(host(q), small, [n]), 5.0, torch.bfloat16)
    k, v = ds.cache_load(cache, scales, slots, dtype=torch.float32)
    codes, s, m = ref.quantise(kv[0].cpu().numpy())
    assert np.array_equal(k.cpu().numpy(), ref.value(codes, s, m).astype(np.float32))


def close_in_norm(got, want, dtype):
    """The error's norm against the result's: bf16's rounding is at most 2^-9 of each element and
    the weights' (11 bits) adds a random 2^-12 times a few; fp32: sums of n terms in fp32 by
    lanes, warps and splits, 2^-24 times the root of the additions and a few roundings each."""
    off = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert off <= (2.0 ** -8 if dtype == torch.bfloat16 else 3e-6), off


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("same", [False, True])
def test_attention_equal_weights_over_a_long_context(ds, dtype, same):
    """Equal weights average values out to 1/sqrt(n) of their size: errors of one sign would show.
    `same`: every value row has the same scale, so that the weights are rounded alike."""
    rng = np.random.default_rng(14)
    n, D = 60000, 64
    cache, scales, table = filled(ds, rng, 1, 1, D, 128, [n])
    if same:
        scales[..., 2] = 0.3359375
        scales[..., 3] = -2.53125
    q = torch.zeros(1, 1, 4, D, device="cuda", dtype=dtype)
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    want = ref.attention(host(q), Paged(cache, scales, table), [n])
    out, lse = ds.cache_attention(q, cache, scales, table, ln)
    close_in_norm(host(out), want[0], dtype)
    assert np.all(np.abs(host(lse) - math.log(n)) <= 1e-5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("order", ["up", "down", "spike"])
def test_attention_running_maximum(ds, dtype, order):
    """Scores that rise or fall all along the context, or stand out once: the running maximum
    moves in every step, in none, or once."""
    rng = np.random.default_rng(15)
    n, D = 3000, 64
    cache, scales, table = filled(ds, rng, 1, 1, D, 32, [n])
    k = rng.standard_normal((n, 1, D)).astype(np.float32) * 0.1
    k[:, 0, 0] += {"up": np.linspace(-40, 40, n), "down": np.linspace(40, -40, n),
                   "spike": np.where(np.arange(n) == 1234, 30.0, 0.0)}[order]
    v = rng.standard_normal((n, 1, D)).astype(np.float32)
    t = table[0].cpu().numpy()
    slots = dev((t[np.arange(n) // 32] * 32 + np.arange(n) % 32).astype(np.int32))
    ds.cache_store(dev(k), dev(v), cache, scales, slots)
    q = np.zeros((1, 1, 8, D), dtype=np.float32)
    q[..., 0] = np.linspace(-3, 3, 8)
    q = dev(q, dtype)
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    want = ref.attention(host(q), Paged(cache, scales, table), [n], scale=1.0)
    out, lse = ds.cache_attention(q, cache, scales, table, ln, scale=1.0)
    # scores reach 120: 2^-24 * 120 * log2(e) * 2 of a weight, and as much of lse
    limit = 2.0 ** -8 * np.abs(want[0]) + 2.0 ** -13 * 5 if dtype == torch.bfloat16 else 1e-4
    assert np.all(np.abs(host(out) - want[0]) <= limit)
    assert np.all(np.abs(host(lse) - want[1]) <= 1e-4)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("low,high", [(-30, 30), (30, -30), (-100, -90), (100, 110)])
def test_attention_values_of_every_size(ds, dtype, low, high):
    """Value rows whose sizes run from 2^low to 2^high along the context: the weights' common
    power of two follows the largest."""
    rng = np.random.default_rng(16)
    n, D = 700, 64
    cache, scales, table = filled(ds, rng, 1, 1, D, 32, [n])
    size = np.exp2(np.linspace(low, high, n)).astype(np.float32)[:, None, None]
    k = rng.standard_normal((n, 1, D)).astype(np.float32)
    v = rng.standard_normal((n, 1, D)).astype(np.float32) * size
    t = table[0].cpu().numpy()
    slots = dev((t[np.arange(n) // 32] * 32 + np.arange(n) % 32).astype(np.int32))
    ds.cache_store(dev(k), dev(v), cache, scales, slots)
    q = dev(rng.standard_normal((1, 1, 16, D)).astype(np.float32), dtype)
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    want = ref.attention(host(q), Paged(cache, scales, table), [n])
    out, _ = ds.cache_attention(q, cache, scales, table, ln)
    limit = 2.0 ** -8 * np.abs(want[0]) if dtype == torch.bfloat16 else 0
    top = (np.abs(want[0]).max(-1, keepdims=True))
    assert np.all(np.abs(host(out) - want[0]) <= limit + (2.0 ** -10 if dtype == torch.bfloat16 else 3e-5) * top)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [math.inf, math.nan, -math.inf])
def test_attention_bad_numbers_in_masked_places(ds, dtype, bad):
    """A later token's scales that are not finite do not reach the tokens that do not see it."""
    rng = np.random.default_rng(17)
    n, Q = 70, 3
    cache, scales, table = filled(ds, rng, 1, 2, 64, 16, [n])
    q = dev(rng.standard_normal((1, Q, 4, 64)).astype(np.float32), dtype)
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    want = ref.attention(host(q), Paged(cache, scales, table), [n])
    scales[table[0, (n - 1) // 16].item(), :, (n - 1) % 16] = bad
    out, lse = ds.cache_attention(q, cache, scales, table, ln)
    seen = slice(0, Q - 1)
    check_attention((out[:, seen], lse[:, seen]), (want[0][:, seen], want[1][:, seen]), 5.0, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_rows_that_see_something_late(ds, dtype):
    """Lists whose first hundreds of entries are not seen, differently for each token."""
    rng = np.random.default_rng(18)
    n, Q, K = 400, 2, 700
    cache, scales, table = filled(ds, rng, 1, 1, 128, 64, [n])
    q = dev(rng.standard_normal((1, Q, 16, 128)).astype(np.float32), dtype)
    idx = np.full((1, Q, K), -1, dtype=np.int32)
    idx[0, 0, 500:] = rng.integers(n, size=200)
    idx[0, 1, 131] = n - 1
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    want = ref.attention(host(q), Paged(cache, scales, table), [n], idx)
    check_attention(ds.cache_attention(q, cache, scales, table, ln, indices=dev(idx)), want, 5.0, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Q,group,D,K", [(1, 8, 128, 0), (2, 6, 64, 0), (1, 4, 64, 70), (1, 16, 128, 200)])
def test_attention_many_short(ds, dtype, Q, group, D, K):
    """Hundreds of contexts of a few pages: a key head's rows are one warp's work, or a few warps'."""
    rng = np.random.default_rng(19 + K)
    B, heads = 90, 8
    lens = rng.integers(0, 300, B)
    lens[:6] = [0, 1, 31, 32, 33, 299]
    cache, scales, table = filled(ds, rng, B, heads, D, 16, lens, width=20)
    q = dev((1.5 * rng.standard_normal((B, Q, heads * group, D))).astype(np.float32), dtype)
    idx = rng.integers(-1, 300, (B, Q, K), dtype=np.int32) if K else None
    want = ref.attention(host(q), Paged(cache, scales, table), lens, idx)
    got = ds.cache_attention(q, cache, scales, table, dev(lens.astype(np.int32)),
                             indices=None if idx is None else dev(idx))
    check_attention(got, want, 5.0, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,heads,group,Q,width", [
    ([9000], 1, 4, 1, 16384),                      # a table much wider than its context
    ([0, 1, 3000, 0, 7777, 129, 128, 8200], 2, 4, 1, 1024),
    ([1] * 40 + [6000, 0, 40], 1, 8, 2, 512),      # one context is nearly all of the work
    ([5000] * 5, 2, 16, 1, 1024),
    ([0, 0, 0], 2, 4, 1, 2560),
    ([16384, 16384, 1], 4, 2, 2, 1024),            # whole tables
])
def test_attention_splits_by_length(ds, dtype, lens, heads, group, Q, width):
    """Few contexts in wide tables, cut to splits by their lengths."""
    rng = np.random.default_rng(sum(lens) + group)
    cache, scales, table = filled(ds, rng, len(lens), heads, 64, 16, lens, width=width)
    q = dev((1.5 * rng.standard_normal((len(lens), Q, heads * group, 64))).astype(np.float32), dtype)
    want = ref.attention(host(q), Paged(cache, scales, table), lens)
    got = ds.cache_attention(q, cache, scales, table, dev(np.array(lens, dtype=np.int32)))
    check_attention(got, want, 5.0, dtype)


# ------------------------------------------------------------------ streams, graphs --

def test_other_stream_repeat_and_graph(ds):
    """The same bits on another stream, on a second call, and replayed from a graph."""
    rng = np.random.default_rng(11)
    cache, scales, table = filled(ds, rng, 2, 2, 128, 64, [3000, 700])
    q = dev(rng.standard_normal((2, 1, 16, 128)).astype(np.float32), torch.bfloat16)
    ln = torch.tensor([3000, 700], dtype=torch.int32, device="cuda")
    x = torch.randn(50, 256, device="cuda")
    logits = 3 * torch.randn(4, 3, 5000, device="cuda")
    drafts = logits[:, :2].argmax(-1).int()
    u, noise = torch.rand(4, 2, device="cuda"), torch.empty(4, 5000, device="cuda").exponential_()

    def all_():
        return (*ds.cache_attention(q, cache, scales, table, ln), *ds.route(x, 8),
                *ds.verify_drafts(logits, drafts, u, noise))
    first = all_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = all_()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            third = all_()
    for t in third:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_attention_workspace_under_capture(ds):
    """A capture that would have to grow the workspace is refused, and the stream goes on."""
    rng = np.random.default_rng(12)
    cache, scales, table = filled(ds, rng, 1, 1, 64, 64, [4000])
    q = dev(rng.standard_normal((1, 1, 8, 64)).astype(np.float32), torch.bfloat16)
    ln = torch.tensor([4000], dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(1, 1, 8, device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        st = ds.ds_cache_attention(q.data_ptr(), ds.DS_BF16, 1, 1, 8, 64, 512, 512, 64, cache.data_ptr(),
                                   scales.data_ptr(), cache.shape[0], 1, 64, table.data_ptr(), table.shape[1],
                                   table.shape[1], ln.data_ptr(), 0, 0, 0.125, out.data_ptr(), lse.data_ptr(),
                                   side.cuda_stream)
    assert st == 7          # DS_ERR_WORKSPACE
    want = ref.attention(host(q), Paged(cache, scales, table), [4000])
    check_attention(ds.cache_attention(q, cache, scales, table, ln), want, 5.0, torch.bfloat16)


def test_decode_step_example():
    """The example runs the operators together; the same seed gives the same tokens."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_step.py")
    spec = importlib.util.spec_from_file_location("decode_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    emitted, lens = example.main(steps=4, seed=1)
    assert (emitted >= 4).all() and (emitted <= 4 * (example.DRAFTS + 1)).all()
    assert torch.equal(lens.long(), example.CONTEXT + emitted)
    again, _ = example.main(steps=4, seed=1)
    assert torch.equal(emitted, again)
