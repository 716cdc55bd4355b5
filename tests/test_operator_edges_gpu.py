"""The operators around the top-k at the ends of their ranges, on the GPU against their definitions
in 64 bits: scales below zero, rows and values of very unlike size, lengths and scores at the edge
of their types."""
import math

import numpy as np
import pytest

import operator_ref as ref
import test_operators_gpu as base

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DTYPES = base.DTYPES
dev, host = base.dev, base.host


@pytest.fixture(scope="module")
def ds():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import top_selection_gb300 as m
    return m


def rows_to_cache(ds, k, v, page=16):
    """A cache of one sequence and key head that holds the fp32 rows k and v, the rest junk."""
    n, D = k.shape
    pages = -(-n // page)
    cache, scales = base.new_cache(pages + 1, 1, page, D)
    slots = torch.arange(n, dtype=torch.int32, device="cuda") + page
    ds.cache_store(dev(k[:, None]), dev(v[:, None]), cache, scales, slots)
    return cache, scales, torch.arange(1, pages + 1, dtype=torch.int32, device="cuda")[None]


# ------------------------------------------------------------------ attention -----

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,at,size,spread,below", [
    (1, slice(None), 0.1, 0.0, True),            # one position
    (1, slice(None), 1.005, 0.0, True),
    (50, slice(None), 1.003, 1e-5, False),       # every row's spread is below bf16's rounding
    (50, slice(None), 1.005, 1e-5, True),
    (700, slice(32, 64), 0.1, 0.0, True),        # one warp's tile of such rows beside ordinary ones
    (3000, slice(5, None, 7), -0.3, 1e-6, False),
    (3000, slice(5, None, 7), -0.301, 1e-6, True),
])
def test_attention_constant_values(ds, dtype, n, at, size, spread, below):
    """An fp32 row of nearly one value has m = bf16(its minimum), which may lie above its maximum
    (`below`): then s < 0 and the codes are 0, and the row stands for m.  Limits: the operator's
    (base.check_attention)."""
    rng = np.random.default_rng(n)
    k, v = rng.standard_normal((2, n, 64)).astype(np.float32)
    v[at] = size + spread * rng.standard_normal(v[at].shape)
    cache, scales, table = rows_to_cache(ds, k, v)
    codes, s, m = ref.quantise(v)
    stored = scales[1:].float().cpu().numpy().reshape(-1, 4)[:n]
    assert np.array_equal(stored[:, 2], s) and np.array_equal(stored[:, 3], m)
    assert (s[at] < 0).all() == below
    q = dev((1.5 * rng.standard_normal((1, 1, 4, 64))).astype(np.float32), dtype)
    want = ref.attention(host(q), base.Paged(cache, scales, table), [n])
    got = ds.cache_attention(q, cache, scales, table, torch.tensor([n], dtype=torch.int32, device="cuda"))
    base.check_attention(got, want, 5.0, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("which", [slice(None), slice(0, 1), slice(40, 45)])
def test_attention_scales_below_zero(ds, dtype, which):
    """Scales a caller wrote: negative ones, larger in size than the positive, with any codes."""
    rng = np.random.default_rng(21)
    n = 300
    k, v = rng.standard_normal((2, n, 64)).astype(np.float32)
    cache, scales, table = rows_to_cache(ds, k, v)
    flat = scales[1:].view(-1, 4)
    flat[which, 2] *= -1.5
    flat[which, 0] *= -1
    q = dev((1.5 * rng.standard_normal((1, 1, 8, 64))).astype(np.float32), dtype)
    want = ref.attention(host(q), base.Paged(cache, scales, table), [n])
    got = ds.cache_attention(q, cache, scales, table, torch.tensor([n], dtype=torch.int32, device="cuda"))
    # values of up to 2.5 + 1.5 * 15 * 0.35
    base.check_attention(got, want, 12.0, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,large", [(8, 2.0 ** 22), (16, 2.0 ** 25), (16, 1e8), (8, 1e10), (16, 1e30)])
def test_attention_query_rows_of_unlike_size(ds, dtype, heads, large):
    """A query row of any size leaves the rows beside it as they are."""
    rng = np.random.default_rng(22)
    n, D = 4096, 128
    k, v = rng.standard_normal((2, n, D)).astype(np.float32)
    cache, scales, table = rows_to_cache(ds, k, v, 64)
    x = (1.5 * rng.standard_normal((1, 1, heads, D))).astype(np.float32)
    x[0, 0, [1, heads - 2]] *= np.float32(large)
    q = dev(x, dtype)
    plain = [i for i in range(heads) if i not in (1, heads - 2)]
    want = ref.attention(host(q), base.Paged(cache, scales, table), [n])
    out, lse = ds.cache_attention(q, cache, scales, table, torch.tensor([n], dtype=torch.int32, device="cuda"))
    base.check_attention((out[:, :, plain], lse[:, :, plain]), (want[0][:, :, plain], want[1][:, :, plain]), 5.0, dtype)
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("large", [2.0 ** 14, 1e6, 1e15, 1e30])
@pytest.mark.parametrize("n,Q", [(70, 3), (33, 2), (1000, 5), (20, 2)])
def test_attention_large_numbers_in_masked_places(ds, dtype, large, n, Q):
    """A later token's scales of any size do not reach the tokens that do not see it (an unwritten
    slot behind a padded draft)."""
    rng = np.random.default_rng(n)
    k, v = rng.standard_normal((2, n, 64)).astype(np.float32)
    cache, scales, table = rows_to_cache(ds, k, v)
    q = dev((1.5 * rng.standard_normal((1, Q, 4, 64))).astype(np.float32), dtype)
    scales[1:].view(-1, 4)[n - 1, 2] = large
    scales[1:].view(-1, 4)[n - 1, 3] = -large
    want = ref.attention(host(q), base.Paged(cache, scales, table), [n])
    out, lse = ds.cache_attention(q, cache, scales, table, torch.tensor([n], dtype=torch.int32, device="cuda"))
    seen = slice(0, Q - 1)
    base.check_attention((out[:, seen], lse[:, seen]), (want[0][:, seen], want[1][:, seen]), 5.0, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_at_the_ends_of_the_range(ds, dtype):
    """Values of 2^90 and keys whose products with the query are ordinary but whose own size is not.
    Limits as for ordinary values (base.check_attention), relative to their size."""
    rng = np.random.default_rng(31)
    k, v = rng.standard_normal((2, 2500, 64)).astype(np.float32)
    big = np.float32(2.0 ** 90) / np.abs(v).max()
    cache, scales, table = rows_to_cache(ds, k * np.float32(2.0 ** 60), v * big)
    q = dev((rng.standard_normal((1, 1, 8, 64)) * 2.0 ** -60).astype(np.float32), dtype)
    want = ref.attention(host(q), base.Paged(cache, scales, table), [2500])
    out, lse = ds.cache_attention(q, cache, scales, table, torch.tensor([2500], dtype=torch.int32, device="cuda"))
    base.check_attention((out.double() / float(big), lse), (want[0] / float(big), want[1]), 5.0, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("order", ["up", "down", "mixed"])
@pytest.mark.parametrize("n,Q,heads,D", [(4, 5, 4, 64), (20, 6, 1, 64), (32, 5, 2, 128), (33, 5, 4, 64), (34, 8, 1, 64),
                                         (66, 5, 8, 128), (70, 3, 4, 64), (1000, 6, 4, 64), (5000, 5, 4, 128), (5121, 4, 16, 64)])
def test_attention_new_tokens_of_unlike_size(ds, dtype, order, n, Q, heads, D):
    """The step's own tokens have values of very unlike size, each seen by its token and the later
    ones: every row keeps its bits, relative to the largest value that it sees.  Limits: the operator's
    (base.check_attention), with that value."""
    rng = np.random.default_rng(n + Q)
    k, v = rng.standard_normal((2, n, D)).astype(np.float32)
    cache, scales, table = rows_to_cache(ds, k, v)
    sizes = 10.0 ** np.array([3, 9, 1, 20, 14, 25, 30, 28][:Q])
    sizes = {"up": np.sort(sizes), "down": np.sort(sizes)[::-1], "mixed": sizes}[order]
    for i in range(min(Q, n)):  # the new tokens, the last one last
        scales[1:].view(-1, 4)[n - 1 - i, 2:] *= float(sizes[Q - 1 - i])
    q = dev((1.5 * rng.standard_normal((1, Q, heads, D))).astype(np.float32), dtype)
    want = ref.attention(host(q), base.Paged(cache, scales, table), [n])
    out, lse = ds.cache_attention(q, cache, scales, table, torch.tensor([n], dtype=torch.int32, device="cuda"))
    sc = scales[1:].view(-1, 4)[:n].double().cpu().numpy()
    most = np.maximum(np.abs(sc[:, 3]), np.abs(15 * sc[:, 2] + sc[:, 3]))
    for i in range(Q):
        end = n - (Q - 1 - i)
        size = most[:end].max() / 5.0 if end > 0 else 1.0
        base.check_attention((out[:, i:i + 1].double() / size, lse[:, i:i + 1]),
                             (want[0][:, i:i + 1] / size, want[1][:, i:i + 1]), 5.0, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", ["many", "few", "wide"])
def test_attention_large_numbers_in_batches(ds, dtype, case):
    """The same in every sequence of a batch: hundreds of short contexts (one warp's work each), a few
    that are split by their lengths, and 40 rows on a key head."""
    rng = np.random.default_rng(34)
    B, Q, heads, group, D, width = {"many": (90, 2, 8, 4, 64, 20), "few": (4, 3, 2, 4, 64, 1024), "wide": (3, 5, 1, 8, 128, 64)}[case]
    lens = rng.integers(Q, 300, B) if case == "many" else np.array([3000, Q, 7777, 8161])[:B] if case == "few" else np.array([33, 900, 64])
    cache, scales, table = base.filled(ds, rng, B, heads, D, 16, lens, width=width)
    q = dev((1.5 * rng.standard_normal((B, Q, heads * group, D))).astype(np.float32), dtype)
    want = ref.attention(host(q), base.Paged(cache, scales, table), lens)
    for b in range(B):  # the last token's, seen by itself alone
        page = int(table[b, (lens[b] - 1) // 16])
        scales[page, :, (lens[b] - 1) % 16, 2:] = float(10.0 ** rng.uniform(3, 35))
    out, lse = ds.cache_attention(q, cache, scales, table, dev(lens.astype(np.int32)))
    seen = slice(0, Q - 1)
    base.check_attention((out[:, seen], lse[:, seen]), (want[0][:, seen], want[1][:, seen]), 5.0, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [40, 200])
def test_attention_scores_far_below_zero(ds, dtype, n):
    """Scores of -1e31 and below, and warps that have no position: the best one wins all the same.
    The scores' errors, 1e-6 of them, are far below their gaps, so the weights are 0 and 1."""
    rng = np.random.default_rng(33)
    k = (1.0 + rng.random((n, 64))).astype(np.float32)
    v = rng.standard_normal((n, 64)).astype(np.float32)
    cache, scales, table = rows_to_cache(ds, k, v)
    q = dev(np.full((1, 1, 4, 64), -1e31, dtype=np.float32) * np.array([1, 2, 3, 4], dtype=np.float32)[:, None], dtype)
    want = ref.attention(host(q), base.Paged(cache, scales, table), [n])
    out, lse = ds.cache_attention(q, cache, scales, table, torch.tensor([n], dtype=torch.int32, device="cuda"))
    assert np.all(np.abs(host(out) - want[0]) <= 2.0 ** -8 * np.abs(want[0]) + 2.0 ** -13 * 5)
    assert np.allclose(host(lse), want[1], rtol=1e-5)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_strides_of_one(ds, dtype):
    """The stride of an extent of 1 is never used, whatever it is."""
    k, v = np.random.default_rng(30).standard_normal((2, 200, 64)).astype(np.float32)
    cache, scales, table = rows_to_cache(ds, k, v)
    q = torch.randn(1, 1, 1, 64, device="cuda").to(dtype)
    ln = torch.tensor([200], dtype=torch.int32, device="cuda")
    want = ds.cache_attention(q, cache, scales, table, ln)
    got = ds.cache_attention(q.as_strided((1, 1, 1, 64), (3, 77, 5, 1)), cache, scales, table, ln)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("length", [-1, -(1 << 31), -(1 << 31) + 1])
@pytest.mark.parametrize("picked", [False, True])
def test_attention_lengths_below_zero(ds, length, picked):
    """A length below zero counts as zero, however far below."""
    k, v = np.random.default_rng(23).standard_normal((2, 40, 64)).astype(np.float32)
    cache, scales, table = rows_to_cache(ds, k, v)
    q = torch.randn(1, 4, 8, 64, device="cuda").bfloat16()
    idx = torch.arange(20, dtype=torch.int32, device="cuda").expand(1, 4, 20).contiguous() if picked else None
    out, lse = ds.cache_attention(q, cache, scales, table, torch.tensor([length], dtype=torch.int32, device="cuda"), indices=idx)
    assert out.abs().max() == 0 and torch.isneginf(lse).all()


# ------------------------------------------------------------------ 4-bit cache ---

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [2.0 ** 126, 2.0 ** -126])
def test_cache_at_the_ends_of_the_range(ds, dtype, size):
    """Rows of 2^126 come back finite, and those near fp32's smallest numbers by the format's rules;
    the bits are the format's."""
    rng = np.random.default_rng(32)
    x = rng.uniform(-1, 1, (40, 64)).astype(np.float32)
    x[:, 0], x[:, 1] = -1, 1
    x = dev(x * np.float32(size), dtype)
    cache, scales, table = rows_to_cache(ds, x.float().cpu().numpy(), -x.float().cpu().numpy())
    codes, s, m = ref.quantise(x.float().cpu().numpy())
    flat = scales[1:].float().cpu().numpy().reshape(-1, 4)[:40]
    assert np.array_equal(cache[1:, 0, :, 0].cpu().numpy().reshape(-1, 32)[:40], ref.pack(codes))
    assert np.array_equal(flat[:, 0], s) and np.array_equal(flat[:, 1], m)
    k, v = ds.cache_load(cache, scales, torch.arange(16, 56, dtype=torch.int32, device="cuda"), dtype=torch.float32)
    assert torch.isfinite(k).all() and torch.isfinite(v).all()
    assert np.array_equal(k[:, 0].cpu().numpy(), ref.value(codes, s, m).astype(np.float32))


# ------------------------------------------------------------------ gate ---------

@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_gradient_of_vanishing_scores(ds, scoring):
    """Logistic scores near fp32's smallest numbers: the weights are of the order 1, and so is their
    gradient.  Limits as for ordinary scores (1e-5 of scale * |g|); a score below 2^-126 keeps
    2^-149, 3e-7 of it."""
    x = np.array([[-88.0, -88.2, -200.0, -88.5, -300.0], [-85.0, -87.5, -88.5, -86.0, -88.0]], dtype=np.float32)
    w, e = ds.route(dev(x), 2, scoring=scoring, scale=2.5)
    g = np.array([[3.0, -3.0], [-5.0, 2.0]], dtype=np.float32)
    eh = host(e).astype(np.int64)
    assert np.allclose(host(w), ref.route_weights(x, eh, scoring, True, 2.5), rtol=base.GATE_REL)
    got = host(ds.route_backward(dev(g), dev(x), e, scoring=scoring, scale=2.5))
    want = ref.route_gradient(g, x, eh, scoring, True, 2.5)
    assert np.all(np.abs(got - want) <= 1e-5 * 2.5 * np.abs(g).max())


# ------------------------------------------------------------------ devices and streams --

def test_tensors_of_another_device(ds):
    """The tensors' device need not be the current one."""
    if torch.cuda.device_count() < 2:
        pytest.skip("needs two GPUs")
    x = torch.randn(9, 64, device="cuda:0")
    w, e = ds.route(x, 4)
    w1, e1 = ds.route(x.to("cuda:1"), 4)
    assert w1.device.index == 1 and torch.cuda.current_device() == 0
    assert torch.equal(w.cpu(), w1.cpu()) and torch.equal(e.cpu(), e1.cpu())


def busy(milliseconds=30):
    """Keeps the current stream at work for a while."""
    torch.cuda._sleep(int(milliseconds * 2e6))


def test_attention_of_an_empty_list_on_another_stream(ds):
    """No position is seen, whatever the current stream still has to do and the memory holds."""
    k, v = np.random.default_rng(24).standard_normal((2, 40, 64)).astype(np.float32)
    cache, scales, table = rows_to_cache(ds, k, v)
    q = torch.randn(1, 4, 8, 64, device="cuda").bfloat16()
    ln = torch.tensor([40], dtype=torch.int32, device="cuda")
    none = torch.empty(1, 4, 0, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        zeros = torch.zeros(1, 4, 1, dtype=torch.int32, device="cuda")  # a list of position 0, left behind
        del zeros
        busy()
        out, lse = ds.cache_attention(q, cache, scales, table, ln, indices=none, stream=side.cuda_stream)
        side.synchronize()
        torch.cuda.synchronize()
        assert out.abs().max() == 0 and torch.isneginf(lse).all()


def test_outputs_on_another_stream(ds):
    """Outputs of a call on another stream than the current one are not in memory that the current
    stream, behind in its work, still writes, and outlive their tensors on either."""
    rng = np.random.default_rng(25)
    k, v = rng.standard_normal((2, 300, 64)).astype(np.float32)
    cache, scales, table = rows_to_cache(ds, k, v)
    q = torch.randn(1, 2, 16, 64, device="cuda")
    ln = torch.tensor([300], dtype=torch.int32, device="cuda")
    x = torch.randn(70, 256, device="cuda")
    logits = 3 * torch.randn(4, 3, 5000, device="cuda")
    drafts = logits[:, :2].argmax(-1).int()
    u, noise = torch.rand(4, 2, device="cuda"), torch.empty(4, 5000, device="cuda").exponential_()
    experts = ds.route(x, 8)[1]
    g = torch.randn(70, 8, device="cuda")
    slots = torch.arange(16, 316, dtype=torch.int32, device="cuda")

    def all_(stream=None):
        return (*ds.cache_attention(q, cache, scales, table, ln, stream=stream), *ds.route(x, 8, stream=stream),
                ds.route_backward(g, x, experts, stream=stream), *ds.verify_drafts(logits, drafts, u, noise, stream=stream),
                *ds.cache_load(cache, scales, slots, stream=stream))
    want = all_()
    sizes = [t.numel() * t.element_size() for t in want]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        busy()
        for size in sizes:  # memory that is free for the host, and still to be written
            t = torch.empty(size, dtype=torch.uint8, device="cuda")
            t.fill_(77)
            del t
        got = all_(side.cuda_stream)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        # the current stream works on them, they are dropped, and the other stream calls again
        busy()
        sums = [t.double().abs().nan_to_num(posinf=1.0).sum() for t in got]
        del got
        again = all_(side.cuda_stream)
        for t in again:
            with torch.cuda.stream(side):
                t.zero_()
        torch.cuda.synchronize()
        assert [float(t) for t in sums] == [float(t.double().abs().nan_to_num(posinf=1.0).sum()) for t in want]
    torch.cuda.current_stream().synchronize()
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


def long_context(ds, seed, n=6000):
    rng = np.random.default_rng(seed)
    k, v = rng.standard_normal((2, n, 64)).astype(np.float32)
    cache, scales, table = rows_to_cache(ds, k, v, 64)
    q = dev(rng.standard_normal((1, 1, 8, 64)).astype(np.float32), torch.bfloat16)
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    return q, cache, scales, table, ln


def test_attention_captured_without_a_warm_up(ds):
    """A graph has a workspace of its own, whatever its stream has run before."""
    args = long_context(ds, 26)
    assert ds.ds_cache_attention_workspace_bytes(ds.DS_BF16, 1, 1, 8, 64, 1, 64, args[3].shape[1]) > 0
    want = ds.cache_attention(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        got = ds.cache_attention(*args)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_graphs_of_one_stream_at_the_same_time(ds):
    """Graphs captured on one stream and replayed side by side do not share a workspace."""
    capture, args = torch.cuda.Stream(), [long_context(ds, 27), long_context(ds, 28)]
    want, graphs, outs, sides = [], [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for a in args:
        want.append(ds.cache_attention(*a))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=capture):
            for _ in range(20):
                out = ds.cache_attention(*a)
        graphs.append(graph)
        outs.append(out)
    for _ in range(10):
        for graph, side in zip(graphs, sides):
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for got, expect in zip(outs, want):
            assert torch.equal(got[0], expect[0]) and torch.equal(got[1], expect[1])


def test_attention_with_a_workspace_of_the_caller(ds):
    q, cache, scales, table, ln = long_context(ds, 29)
    need = ds.ds_cache_attention_workspace_bytes(ds.DS_BF16, 1, 1, 8, 64, 1, 64, table.shape[1])
    want = ds.cache_attention(q, cache, scales, table, ln)
    buf = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")   # NaN wherever it is read before it is written
    out, lse = torch.empty_like(q), torch.empty(1, 1, 8, device="cuda")

    def call(ws, size):
        return ds.ds_cache_attention_ex(q.data_ptr(), ds.DS_BF16, 1, 1, 8, 64, 512, 512, 64, cache.data_ptr(),
                                        scales.data_ptr(), cache.shape[0], 1, 64, table.data_ptr(), table.shape[1],
                                        table.shape[1], ln.data_ptr(), 0, 0, 0.125, out.data_ptr(), lse.data_ptr(), ws,
                                        size, torch.cuda.current_stream().cuda_stream)
    assert call(buf.data_ptr(), need - 1) == 7      # DS_ERR_WORKSPACE
    assert call(buf.data_ptr() + 8, need) == 2      # DS_ERR_ALIGNMENT
    assert call(buf.data_ptr(), need) == 0
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert (buf[need:] == 255).all()
    assert call(0, 0) == 0                          # the library's
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    # a list that one cluster takes needs none
    assert ds.ds_cache_attention_workspace_bytes(ds.DS_BF16, 64, 1, 32, 128, 2, 64, 2048, picked=True, K=512) == 0
    with pytest.raises(ds.DSError):
        ds.ds_cache_attention_workspace_bytes(ds.DS_BF16, 1, 1, 8, 96, 1, 64, 4)
