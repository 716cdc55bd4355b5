"""The operators behind the selections at the ends of their ranges, on the GPU against their
definitions in 64 bits: logits of any size, numbers that are none, a kernel that gives
up, offsets in no order, and the products' gradient."""
import math

import pytest

import behind_ref as ref
import test_behind_gpu as base

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DTYPES, U = base.DTYPES, base.U
gen, normal, half_step, sum_error = base.gen, base.normal, base.half_step, base.sum_error


@pytest.fixture(scope="module")
def ds():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import top_selection_gb300 as m
    yield m
    assert m.ds_get_device_status() == 0


# ------------------------------------------------------------------ logits of any size ----

LARGE = [3e9, 1e10, 1e15, 1e30, 9e36, 3e38]


def large_rows(dtype, V):
    """Rows throughout at a large number, rows with one of them among ordinary numbers, rows masked with
    a finite number in part, and rows of numbers beside a large one."""
    g = gen(V)
    rows = []
    for c in LARGE:
        for c in (c, -c):
            rows.append(torch.full((V,), c, device="cuda"))
            one = normal(g, V)
            one[V // 3] = c
            rows.append(one)
    for c in (-1e9, -1e10, -1e20, -1e30):
        rows.append(torch.full((V,), c, device="cuda"))
        part = normal(g, V)
        part[: V // 2] = c                        # whole threads see nothing else
        rows.append(part)
        part = normal(g, V)
        part[torch.rand(V, device="cuda", generator=g) < 0.9] = c
        rows.append(part)
        part = torch.full((V,), c, device="cuda")
        part[V - 1] = -2.0 * abs(c)               # one below all the others
        rows.append(part)
    for c in (100.0, -3000.0, 1e5, -1e6, 1e7, 1e9):
        rows.append(c + 3.0 * normal(g, V))
    x = torch.stack(rows).to(dtype)
    return x, torch.randint(V, (x.shape[0],), device="cuda", generator=g).int()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,top", [(1, 1), (7, 5), (1000, 0), (1000, 20), (9001, 1), (40000, 32), (140000, 3)])
def test_token_logprobs_of_large_logits(ds, dtype, V, top):
    x, tokens = large_rows(dtype, V)
    for r in range(x.shape[0]):                   # one row: a cluster to it
        base.check_logprobs(ds, x[r:r + 1], tokens[r:r + 1], top)
    base.check_logprobs(ds, x.repeat(9, 1), tokens.repeat(9), top)  # as many rows as take a CTA each


def check_gradient(ds, x, tokens, g, h):
    """The gradient from the kernel's own lse.  log p = (x - lse) - rest, where rest is what lse lost when it was rounded:
    up to |lse| = 64 it is left out, which moves p by half a step of numbers in [32, 64], 2^-19 = 32 U; beyond
    that it is taken from a sum over the row again, off by sum_error and by 2 U |log|.  The two
    differences round by U of their results, of which the first is log p + rest, |rest| <= 43 (numbers' steps
    next to lse up to twice log V, beyond that log V itself); p's argument by U |log p|."""
    V = x.shape[1]
    _, lse, H, _, _ = ds.token_logprobs(x, tokens)
    got = ds.token_logprobs_backward(g, x, tokens, lse, grad_entropy=h, entropy=H if h is not None else None)
    # the formula, with the largest logit and log s apart: 64 bits lose log s beside 1e30 too
    y = x.double() - x.double().amax(-1, keepdim=True)
    lpd = y - torch.log(torch.exp(y).sum(-1, keepdim=True))
    p, lps = torch.exp(lpd), lpd.abs().clamp(max=1e6)
    plogp = torch.where(p > 0, p * lpd, 0.0)
    there = (tokens >= 0)[:, None]
    hot = (tokens[:, None] == torch.arange(V, device="cuda")).double()
    gd = torch.where(there, g.double()[:, None], 0.0)
    want = gd * (hot - p)
    size, more = gd.abs(), 0.0
    rel = 2 * sum_error(V) + U * (32 + 3 * 43 + 4 * lps) + 8 * U
    if h is not None:
        hd = h.double()[:, None]
        want = want - hd * (plogp - p * plogp.sum(-1, keepdim=True))
        size = size + hd.abs() * (lps + 1 + math.log(V))
        # the entropy's own error and log p's enter by h p
        more = hd.abs() * p * (4 * sum_error(V) * (1 + math.log(V)) + rel)
    limit = p * size * rel + more + half_step(x.dtype) * want.abs() * 1.01 + 2 * U * gd.abs() + 1e-37
    assert got.dtype == x.dtype and got.shape == x.shape
    assert bool(((got.double() - want).abs() <= limit).all())


def offset_rows(dtype, V, seed):
    g = gen(seed)
    rows = [torch.full((V,), c, device="cuda") for c in (-1e9, -1e30, -1e4, 77.0, 3e9, torch.finfo(dtype).min, torch.finfo(dtype).max)]
    rows += [c + 2.0 * normal(g, V) for c in (0.0, 50.0, -63.0, 66.0, 300.0, -1e4, 3e5, -1e7, 1e9)]
    part = torch.full((V,), -1e9, device="cuda")
    part[V // 2:] += 700.0 * normal(g, V - V // 2)  # steps of 64: the largest and few besides
    rows.append(part)
    part = torch.full((V,), -math.inf, device="cuda")
    part[::3] = -1e9                                # an exact mask within a finite one
    rows.append(part)
    x = torch.stack(rows).to(dtype)
    tokens = torch.randint(V, (x.shape[0],), device="cuda", generator=g).int()
    tokens[1] = tokens[9] = -1
    return g, x, tokens


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("V,pad,offset", [(1, 0, 0), (50, 0, 0), (5003, 0, 0), (5003, 4, 1), (20001, 8, 3), (129280, 0, 0)])
def test_token_logprobs_backward_of_large_logits(ds, dtype, entropy, V, pad, offset):
    """Every p keeps its digits whatever the logits' common offset: a row of -1e9 has 1 / V."""
    g, rows, tokens = offset_rows(dtype, V, V + pad)
    T = rows.shape[0]
    flat = torch.full((T * (V + pad) + offset,), math.nan, dtype=dtype, device="cuda")
    x = flat[offset:].view(T, V + pad)[:, :V]
    x.copy_(rows)
    check_gradient(ds, x, tokens, normal(g, T), normal(g, T) if entropy else None)


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_of_a_row_of_one_number(ds, dtype):
    """1 / V for every token but the given one, which has 1 / V - 1.  The sum is off by sum_error(4096) = 62 U, roundings of lse
    (8.3: 2^-21), differences, arguments and the exponential by less than 32 U: below 2^-17 in all."""
    V = 4096
    for c in (0.0, -1e4, -1e9, -1e30, 3e38, float(torch.finfo(dtype).min)):
        x = torch.full((3, V), c, device="cuda").to(dtype)
        t = torch.tensor([5, 4000, -1], dtype=torch.int32, device="cuda")
        _, lse, _, _, _ = ds.token_logprobs(x, t)
        got = ds.token_logprobs_backward(-torch.ones(3, device="cuda"), x, t, lse).double()
        want = torch.full((3, V), 1.0 / V, dtype=torch.float64, device="cuda")
        want[0, 5] -= 1.0
        want[1, 4000] -= 1.0
        want[2] = 0.0
        assert bool(((got - want).abs() <= (half_step(dtype) + 2.0 ** -17) * want.abs()).all())


# ------------------------------------------------------------------ numbers that are none ----

def order_of(x, top):
    """NaN first, then by value; equals by index.  (The CPU's stable sort puts NaN of either sign on top.)"""
    return x.double().cpu().sort(dim=-1, descending=True, stable=True).indices[:, :top].to(x.device)


def spoilt_rows(dtype, V):
    """Ordinary rows with a NaN or an infinity in their first, a middle and their last word, many of them, and nothing
    else; every other row is whole."""
    g, nan, inf = gen(V), math.nan, math.inf
    rows = []

    def add(change):
        rows.append(normal(g, V))
        rows.append(normal(g, V))
        change(rows[-1])
    for at in (0, V // 2, V - 1):
        for c in (nan, inf, -nan):
            add(lambda r: r.__setitem__(at, c))
    add(lambda r: r.fill_(nan))
    add(lambda r: r.fill_(inf))
    add(lambda r: (r.fill_(-inf), r.__setitem__(V // 3, nan)))
    add(lambda r: (r.__setitem__(slice(0, V // 2), -inf), r.__setitem__(V // 4, nan)))
    add(lambda r: (r.fill_(3e38), r.__setitem__(V // 3, nan)))
    add(lambda r: (r.__setitem__(slice(None, None, 3), nan), r.__setitem__(slice(1, None, 3), inf)))
    add(lambda r: (r.__setitem__(V - 1, nan), r.__setitem__(0, inf)))
    x = torch.stack(rows).to(dtype)
    tokens = torch.randint(V, (x.shape[0],), device="cuda", generator=g).int()
    tokens[3] = -1                                # a spoilt row without a token
    return x, tokens


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,top", [(1, 1), (9, 5), (300, 0), (1000, 20), (9001, 1), (40000, 32), (140000, 3)])
def test_numbers_that_are_none(ds, dtype, V, top):
    """A NaN or +inf among its logits makes a row's lse, log probabilities and entropy NaN, and its gradient; its top
    tokens are the NaN ones first, then +inf.  Rows beside it are as without it."""
    x, tokens = spoilt_rows(dtype, V)
    T = x.shape[0]
    bad = torch.arange(T, device="cuda") % 2 == 1
    order = order_of(x, top)
    clean = x.clone()
    clean[1::2] = x[::2]
    base.check_logprobs(ds, clean, tokens, top)
    for many in (1, 12):
        xs, ts, bads = x.repeat(many, 1), tokens.repeat(many), bad.repeat(many)
        lp, lse, H, top_lp, top_tokens = ds.token_logprobs(xs, ts, top=top)
        given = bads & (ts >= 0)
        assert bool(lse[bads].isnan().all()) and bool(H[bads].isnan().all()) and bool(lp[given].isnan().all())
        assert not bool(lp[ts < 0].any())
        assert bool(top_lp[bads].isnan().all())
        assert torch.equal(top_tokens.long(), order.repeat(many, 1))
        whole = ds.token_logprobs(clean.repeat(many, 1), ts, top=top)
        for a, b in zip((lp, lse, H, top_lp, top_tokens), whole):
            assert torch.equal(a[~bads], b[~bads])
        g = normal(gen(1), T * many)
        for h in (None, g):
            grad = ds.token_logprobs_backward(g, xs, ts, lse, grad_entropy=h, entropy=None if h is None else H)
            assert bool(grad[bads].isnan().all()) and not bool(grad[~bads].isnan().any())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,K", [(1, 8), (3, 300), (130, 264), (300, 1000)])
def test_8_bits_of_numbers_that_are_none(ds, dtype, N, K):
    """The codes of infinities and NaN are NaN.  An infinity counts as the largest number for its block's
    scale, a NaN not at all."""
    g = gen(N + K)
    x = normal(g, N, K).to(dtype)
    spoilt = x.clone()
    spoilt[0, K // 2] = math.inf
    spoilt[N - 1, K - 1] = -math.inf
    spoilt[N // 2, K // 3] = math.nan
    if N > 2:
        spoilt[1] = math.nan
    most = 3.3895313892515355e38                  # the largest bf16: 448 * 2^120 is above it, 448 * 2^119 below
    stand_in = torch.where(spoilt.isinf(), most, torch.where(spoilt.isnan(), 0.0, spoilt.float())).to(dtype)
    for block in (1, 128):
        for off in (0, 1):                        # rows on 16 bytes, and not
            held = torch.empty(N * K + off, dtype=dtype, device="cuda")[off:].view(N, K)
            held.copy_(spoilt)
            codes, scales = ds.quantise_blocks(held, block_rows=block)
            want, want_scales = ref.quantise(stand_in[None], block)
            assert torch.equal(scales.double(), want_scales[0])
            none = ~torch.isfinite(spoilt)
            assert bool(codes.float()[none].isnan().all())
            assert torch.equal(codes.double()[~none], want[0][~none])
    places, offsets = ds.expert_sort(torch.zeros(N, 1, dtype=torch.int32, device="cuda"), 1)
    codes, scales = ds.expert_gather(spoilt, places, offsets, quantise=True)
    want, want_scales = ds.quantise_blocks(spoilt)
    assert torch.equal(codes.view(torch.uint8), want.view(torch.uint8)) and torch.equal(scales, want_scales)


# ------------------------------------------------------------------ a product that gives up ----

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,E,N,K", [(1, 1, 1000, 4096), (300, 1, 400, 1536), (700, 8, 130, 512), (20000, 4, 272, 144),
                                     (6000, 1, 1304, 528)])
def test_product_that_gives_up(ds, dtype, T, E, N, K):
    """Blocks split over a cluster, narrow and wide tiles: each CTA gives up with copies, or copies and products, in
    flight.  The call records the timeout and returns; the next one is as ever."""
    g = gen(T + N)
    x, xs, w, ws = base.operands(g, T, E, N, K)
    offsets = base.spread(g, T, E)
    want = ds.expert_product(x, xs, w, ws, offsets, dtype=dtype)
    out = torch.empty_like(want)

    def probe(block):
        return ds.ds_expert_product_probe(block, x.data_ptr(), xs.data_ptr(), T, K, K, w.data_ptr(), ws.data_ptr(), E, N, K,
                                          N * K, offsets.data_ptr(), int(dtype == torch.float32), out.data_ptr(),
                                          torch.cuda.current_stream().cuda_stream)
    assert ds.ds_get_device_status() == 0
    for block in (0, 1):                           # every form here has two blocks to a tile at least
        assert probe(block) == 0
        again = ds.expert_product(x, xs, w, ws, offsets, dtype=dtype)  # right behind it on the stream
        assert ds.ds_get_device_status() == 5      # DS_ERR_TIMEOUT
        assert torch.equal(again, want)
    for block in (2, 3, 7):                        # some have no more
        assert probe(block) == 0
        assert ds.ds_get_device_status() in (0, 5)
    assert probe(2 ** 31 - 1) == 0                 # no tile has as many
    assert ds.ds_get_device_status() == 0 and torch.equal(out, want)


# ------------------------------------------------------------------ offsets ----

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,E,N,K", [(6, 4, 200, 2048), (900, 8, 130, 512), (20000, 5, 272, 144)])
def test_product_of_offsets_in_no_order(ds, dtype, T, E, N, K):
    """Offsets that descend, or lie outside of the rows: nothing outside of out is written, and rows of one expert alone
    have their products."""
    g = gen(T)
    x, xs, w, ws = base.operands(g, T, E, N, K)
    held = torch.full((T + 64, N), 7.0, device="cuda", dtype=dtype)
    out = held[32:32 + T]

    def product(offsets):
        o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        assert ds.ds_expert_product(x.data_ptr(), xs.data_ptr(), T, K, K, w.data_ptr(), ws.data_ptr(), E, N, K, N * K, o.data_ptr(),
                                    int(dtype == torch.float32), out.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        assert bool((held[:32] == 7.0).all()) and bool((held[32 + T:] == 7.0).all())
    product([T - T * e // E for e in range(E + 1)])
    product([0] + [(7919 * e) % (T + 1) for e in range(E)])
    product([-5] * E + [T + 100])                  # outside: the last expert has all rows
    want, size = ref.product(x, xs, w, ws, [0] * E + [T])
    base.check_product(out, want, size, K, dtype)
    product([2 ** 31 - 1] * (E + 1))               # all rows before the first expert
    assert not bool(out.any())


# ------------------------------------------------------------------ the products' gradient ----

@pytest.mark.parametrize("T,E,N,K", [(37, 3, 144, 272), (700, 4, 400, 512), (9, 1, 2048, 128)])
def test_gradient_of_the_products_rows(ds, T, E, N, K):
    """The gradient with respect to the rows: the outputs' gradient in 8 bits along N, times the transposed codes and
    scales, against 64 bits of the same codes, and against differences of the product itself."""
    g = gen(T + N)
    x, xs, w, ws = base.operands(g, T, E, N, K)
    ws = ws * 2.0 ** -10
    offsets = base.spread(g, T, E, 0.0)
    grad = normal(g, T, N)
    codes, scales = ds.quantise_blocks(grad)
    w_t, ws_t = w.transpose(1, 2).contiguous(), ws.transpose(1, 2).contiguous()
    got = ds.expert_product(codes, scales, w_t, ws_t, offsets, dtype=torch.float32)
    # grad_x[r, k] = sum_n grad[r, n] w[e, n, k]: the definition, of the codes' values
    tall, wide = torch.arange(N, device="cuda") // 128, torch.arange(K, device="cuda") // 128
    back = codes.double() * scales.double()[:, tall]
    want, size = torch.zeros(T, K, dtype=torch.float64, device="cuda"), torch.zeros(T, K, dtype=torch.float64, device="cuda")
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        m = w[e].double() * ws[e].double()[tall][:, wide]
        want[a:b], size[a:b] = back[a:b] @ m, back[a:b].abs() @ m.abs()
    base.check_product(got, want, size, N, torch.float32)
    # linear in the rows: a step of one code's value along k gives that column of the weights
    def f(x):
        return (back * ds.expert_product(x, xs, w, ws, offsets, dtype=torch.float32).double()).sum(-1)
    for k in (0, K // 2, K - 1):
        up, down = x.float(), x.float()
        up[:, k], down[:, k] = 8.0, -8.0
        slope = (f(up.to(x.dtype)) - f(down.to(x.dtype))) / (16.0 * xs.double()[:, k // 128])
        # each f is off by its product's error, (blocks + 11) 2^-23 of its sizes, summed over N
        for r in {0, T // 2, T - 1}:
            e = int((offsets[1:] <= r).sum())
            m = w[e].double() * ws[e].double()[tall][:, wide]
            sizes = (back[r].abs() * (m.abs() @ (x[r].double().abs().clamp(min=8.0) * xs[r].double()[wide]))).sum()
            off = 2 * (-(-K // 128) + 11) * 2 * U * sizes / (16.0 * xs[r, k // 128].double())
            assert abs(float(slope[r] - want[r, k])) <= float(off)
