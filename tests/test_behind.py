"""Host-side checks of the operators behind the selections that need no GPU: refusals come before
anything is launched, and the formulas the GPU tests compare against hold by themselves."""
import pytest

import behind_ref as ref

torch = pytest.importorskip("torch")

P = 1 << 20   # a 16-byte aligned address that is never read: the checks run first
INVALID, ALIGNMENT, UNSUPPORTED = 1, 2, 3


@pytest.fixture(scope="module")
def ds():
    from top_selection_gb300 import build
    build.build()
    import top_selection_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("change,want", [
    (dict(dtype=2), INVALID),
    (dict(rows=-1), INVALID),
    (dict(V=0), INVALID),
    (dict(row_stride=99), INVALID),
    (dict(top=-1), INVALID),
    (dict(V=10, top=11), INVALID),
    (dict(logits=0), INVALID),
    (dict(tokens=0), INVALID),
    (dict(out_logprobs=0), INVALID),
    (dict(out_lse=0), INVALID),
    (dict(out_entropy=0), INVALID),
    (dict(out_top_logprobs=0), INVALID),
    (dict(out_top_tokens=0), INVALID),
    (dict(logits=P + 2), ALIGNMENT),
    (dict(dtype=0, logits=P + 1), ALIGNMENT),
    (dict(tokens=P + 2), ALIGNMENT),
    (dict(out_top_tokens=P + 1), ALIGNMENT),
    (dict(top=33), UNSUPPORTED),
    (dict(V=(1 << 30) + 1, row_stride=1 << 31), UNSUPPORTED),
    (dict(rows=1 << 31), UNSUPPORTED),
    (dict(rows=0, logits=0), 0),
])
def test_token_logprobs_refuses(ds, change, want):
    a = dict(logits=P, dtype=1, rows=2, V=100, row_stride=100, tokens=P, top=5, out_logprobs=P, out_lse=P, out_entropy=P,
             out_top_logprobs=P, out_top_tokens=P)
    a.update(change)
    assert ds.ds_token_logprobs(**a) == want


@pytest.mark.parametrize("change,want", [
    (dict(dtype=-1), INVALID),
    (dict(row_stride=99), INVALID),
    (dict(grad_stride=99), INVALID),
    (dict(grad_logprobs=0), INVALID),
    (dict(lse=0), INVALID),
    (dict(entropy=0), INVALID),                       # a gradient of the entropy without the entropy
    (dict(grad_logits=0), INVALID),
    (dict(grad_logits=P + 2), ALIGNMENT),
    (dict(grad_entropy=P + 2), ALIGNMENT),
    (dict(V=(1 << 30) + 1, row_stride=1 << 31, grad_stride=1 << 31), UNSUPPORTED),
    (dict(rows=1 << 30, V=1 << 20, row_stride=1 << 20, grad_stride=1 << 20), UNSUPPORTED),
    (dict(rows=0, lse=0), 0),
])
def test_token_logprobs_backward_refuses(ds, change, want):
    a = dict(grad_logprobs=P, logits=P, dtype=1, rows=2, V=100, row_stride=100, tokens=P, lse=P, grad_entropy=P,
             entropy=P, grad_logits=P, grad_stride=100)
    a.update(change)
    assert ds.ds_token_logprobs_backward(**a) == want


@pytest.mark.parametrize("change,want", [
    (dict(tokens=-1), INVALID),
    (dict(k=0), INVALID),
    (dict(E=0), INVALID),
    (dict(experts=0), INVALID),
    (dict(places=0), INVALID),
    (dict(offsets=0), INVALID),
    (dict(offsets=0, tokens=0), INVALID),             # the offsets are written in any case
    (dict(experts=P + 2), ALIGNMENT),
    (dict(k=33), UNSUPPORTED),
    (dict(E=513), UNSUPPORTED),
    (dict(tokens=1 << 30), UNSUPPORTED),
])
def test_expert_sort_refuses(ds, change, want):
    a = dict(experts=P, tokens=4, k=2, E=8, places=P, offsets=P)
    a.update(change)
    assert ds.ds_expert_sort(**a) == want


EXCHANGE = [
    (dict(dtype=2), INVALID),
    (dict(tokens=-1), INVALID),
    (dict(D=0), INVALID),
    (dict(row_stride=63), INVALID),
    (dict(k=0), INVALID),
    (dict(places=0), INVALID),
    (dict(places=P + 2), ALIGNMENT),
    (dict(k=33), UNSUPPORTED),
    (dict(tokens=1 << 30), UNSUPPORTED),
    (dict(tokens=0), 0),
]


@pytest.mark.parametrize("change,want", EXCHANGE + [
    (dict(x=0), INVALID),
    (dict(out=0), INVALID),
    (dict(offsets=0), INVALID),
    (dict(E=0), INVALID),
    (dict(E=513), UNSUPPORTED),
    (dict(x=P + 1), ALIGNMENT),
    (dict(out=P + 1), ALIGNMENT),
])
def test_expert_gather_refuses(ds, change, want):
    a = dict(x=P, dtype=0, tokens=3, D=64, row_stride=64, places=P, k=2, offsets=P, E=8, out=P)
    a.update(change)
    assert ds.ds_expert_gather(**a) == want
    a["codes"] = a.pop("out")
    if a["codes"] == P:  # codes are bytes: any alignment
        assert ds.ds_expert_gather_quantised(**a, scales=P) == want
        assert ds.ds_expert_gather_quantised(**a, scales=P + 2) == (want or (ALIGNMENT if a["tokens"] else 0))


@pytest.mark.parametrize("change,want", EXCHANGE + [
    (dict(rows=-1), INVALID),
    (dict(y=0), INVALID),
    (dict(out=0), INVALID),
    (dict(weights=P + 2), ALIGNMENT),
    (dict(y=P + 1), ALIGNMENT),
])
def test_expert_combine_refuses(ds, change, want):
    a = dict(y=P, dtype=0, rows=6, D=64, row_stride=64, places=P, tokens=3, k=2, weights=P, out=P)
    a.update(change)
    assert ds.ds_expert_combine(**a) == want


@pytest.mark.parametrize("change,want", EXCHANGE + [
    (dict(grad=0), INVALID),
    (dict(y=0), INVALID),
    (dict(weights=0), INVALID),
    (dict(grad_y=0), INVALID),
    (dict(grad_weights=0), INVALID),
    (dict(offsets=0), INVALID),
    (dict(grad_stride=63), INVALID),
    (dict(E=513), UNSUPPORTED),
    (dict(grad_weights=P + 2), ALIGNMENT),
    (dict(grad=P + 1), ALIGNMENT),
])
def test_expert_combine_backward_refuses(ds, change, want):
    a = dict(grad=P, grad_stride=64, y=P, dtype=0, D=64, row_stride=64, places=P, tokens=3, k=2, offsets=P, E=8,
             weights=P, grad_y=P, grad_weights=P)
    a.update(change)
    assert ds.ds_expert_combine_backward(**a) == want


@pytest.mark.parametrize("change,want", [
    (dict(dtype=2), INVALID),
    (dict(matrices=-1), INVALID),
    (dict(rows=-1), INVALID),
    (dict(K=0), INVALID),
    (dict(row_stride=99), INVALID),
    (dict(matrix_stride=-1), INVALID),
    (dict(block_rows=64), INVALID),
    (dict(x=0), INVALID),
    (dict(codes=0), INVALID),
    (dict(scales=0), INVALID),
    (dict(x=P + 1), ALIGNMENT),
    (dict(scales=P + 2), ALIGNMENT),
    (dict(rows=1 << 40), UNSUPPORTED),
    (dict(matrices=1 << 40), UNSUPPORTED),
    (dict(row_stride=1 << 62), UNSUPPORTED),
    (dict(rows=0, x=0), 0),
    (dict(matrices=0, x=0), 0),
])
def test_quantise_blocks_refuses(ds, change, want):
    a = dict(x=P, dtype=0, matrices=2, rows=3, K=100, matrix_stride=300, row_stride=100, block_rows=1, codes=P, scales=P)
    a.update(change)
    assert ds.ds_quantise_blocks(**a) == want


@pytest.mark.parametrize("D", [(1 << 30) + 1, (1 << 31) - 1])
def test_exchange_refuses_long_rows(ds, D):
    """Columns are counted in 32 bits, a stretch of the row past the last one."""
    rows = dict(dtype=0, D=D, row_stride=D, places=P, tokens=1, k=1)
    assert ds.ds_expert_gather(x=P, out=P, offsets=P, E=1, **rows) == UNSUPPORTED
    assert ds.ds_expert_combine(y=P, out=P, rows=1, weights=P, **rows) == UNSUPPORTED
    assert ds.ds_expert_combine_backward(grad=P, grad_stride=D, y=P, offsets=P, E=1, weights=P, grad_y=P, grad_weights=P,
                                         **rows) == UNSUPPORTED


@pytest.mark.parametrize("K", [(1 << 26) + 1, (1 << 31) - 127, (1 << 31) - 1])
def test_8_bit_form_refuses_long_rows(ds, K):
    for block_rows in (1, 128):
        assert ds.ds_quantise_blocks(x=P, dtype=0, matrices=1, rows=1, K=K, matrix_stride=K, row_stride=K,
                                     block_rows=block_rows, codes=P, scales=P) == UNSUPPORTED
    assert ds.ds_expert_gather_quantised(x=P, dtype=0, tokens=1, D=K, row_stride=K, places=P, k=1, offsets=P, E=1, codes=P,
                                         scales=P) == UNSUPPORTED


@pytest.mark.parametrize("change,want", [
    (dict(dtype=2), INVALID),
    (dict(rows=-1), INVALID),
    (dict(K=0), INVALID),
    (dict(N=0), INVALID),
    (dict(E=0), INVALID),
    (dict(x_stride=240), INVALID),
    (dict(w_row_stride=240), INVALID),
    (dict(w_matrix_stride=-16), INVALID),
    (dict(w_matrix_stride=0), INVALID),               # one matrix for all experts
    (dict(offsets=0), INVALID),                       # several experts without offsets
    (dict(x=0), INVALID),
    (dict(x_scales=0), INVALID),
    (dict(w=0), INVALID),
    (dict(w_scales=0), INVALID),
    (dict(out=0), INVALID),
    (dict(x=P + 8), ALIGNMENT),
    (dict(w=P + 8), ALIGNMENT),
    (dict(x_stride=264), ALIGNMENT),
    (dict(w_row_stride=264), ALIGNMENT),
    (dict(w_matrix_stride=8), ALIGNMENT),
    (dict(x_scales=P + 2), ALIGNMENT),
    (dict(offsets=P + 2), ALIGNMENT),
    (dict(out=P + 1), ALIGNMENT),
    (dict(K=250), UNSUPPORTED),
    (dict(E=513), UNSUPPORTED),
    (dict(rows=(1 << 30) + 1), UNSUPPORTED),
    (dict(N=(1 << 24) + 1), UNSUPPORTED),
    (dict(rows=0, x=0), 0),
])
def test_expert_product_refuses(ds, change, want):
    a = dict(x=P, x_scales=P, rows=4, K=256, x_stride=256, w=P, w_scales=P, E=8, N=100, w_row_stride=256,
             w_matrix_stride=25600, offsets=P, dtype=0, out=P)
    a.update(change)
    assert ds.ds_expert_product(**a) == want


def test_python_entry_points_refuse_cpu_tensors(ds):
    x, i = torch.zeros(2, 64), torch.zeros(2, 4, dtype=torch.int32)
    codes = torch.zeros(2, 64, dtype=torch.float8_e4m3fn)
    for call in (lambda: ds.token_logprobs(x, i[:, 0]), lambda: ds.token_logprobs_backward(x[:, 0], x, i[:, 0], x[:, 0]),
                 lambda: ds.expert_sort(i, 8), lambda: ds.expert_gather(x, i, i[0]), lambda: ds.expert_combine(x, i),
                 lambda: ds.expert_combine_backward(x, x, i, i[0], x), lambda: ds.quantise_blocks(x),
                 lambda: ds.expert_product(codes, x[:, :1], codes, x[:1, :1])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError, match="dtype"):
        ds.expert_product(codes, x[:, :1], codes, x[:1, :1], dtype=torch.float16)


# ---------------------------------------------------- the formulas by themselves ----

def test_logprob_gradient_against_differences():
    """Central differences in 64 bits: the difference's own error is of the order h^2 = 1e-10, rounding's
    1e-16 / h = 1e-11, each times values of the order 1."""
    g = torch.Generator().manual_seed(1)
    x, gl, gh = (torch.randn(*s, dtype=torch.float64, generator=g) for s in ((4, 9), (4,), (4,)))
    t = torch.tensor([3, 0, -1, 9])  # the last two: none given
    got = ref.logprobs_gradient(x, t, gl, gh)
    h = 1e-5
    for v in range(9):
        total = 0.0
        for sign in (1, -1):
            y = x.clone()
            y[:, v] += sign * h
            lp, _, H, _, _ = ref.logprobs(y, t)
            total = total + sign * (lp * gl + H * gh)
        assert torch.allclose(got[:, v], total / (2 * h), rtol=0, atol=1e-8)


def test_logprob_gradient_against_autograd():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(3, 7, dtype=torch.float64, generator=g, requires_grad=True)
    t, gl, gh = torch.tensor([1, 6, 2]), torch.randn(3, generator=g).double(), torch.randn(3, generator=g).double()
    lp = torch.log_softmax(x, -1)
    ((lp[torch.arange(3), t] * gl).sum() - ((lp.exp() * lp).sum(-1) * gh).sum()).backward()
    assert torch.allclose(ref.logprobs_gradient(x.detach(), t, gl, gh), x.grad, rtol=0, atol=1e-13)


def test_sorted_places():
    e = torch.tensor([[2, 0], [0, -1], [5, 2], [2, 2]])
    places, offsets = ref.sort(e, 4)  # expert 5 is none
    assert places == [2, 0, 1, -1, -1, 3, 4, 5] and offsets == [0, 2, 2, 6, 6]


def test_rounding_to_8_bits():
    """Against torch's conversion, at every number that e4m3 holds, every midpoint and beside it."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    codes = codes[torch.isfinite(codes)].sort().values.unique()
    mid = (codes[1:] + codes[:-1]) / 2
    v = torch.cat([codes, mid, torch.nextafter(mid, mid + 1), torch.nextafter(mid, mid - 1)])
    assert torch.equal(ref.round_e4m3(v).float(), v.to(torch.float8_e4m3fn).float())


def test_scales_of_blocks():
    """The scale is enough for the block's largest number, and half of it is not; a number comes back
    within half a step of 3 bits, or of the smallest steps."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(1, 5, 300, generator=g) * torch.exp(8 * torch.randn(1, 5, 1, generator=g))
    codes, s = ref.quantise(x, 1)
    for r in range(5):
        for b in range(3):
            top, v = float(x[0, r, 128 * b:128 * b + 128].abs().max()), float(s[0, r, b])
            assert top <= 448 * v and top > 224 * v
    back = codes * s.repeat_interleave(128, 2)[:, :, :300]
    limit = torch.maximum(2.0 ** -4 * x.abs().double(), 2.0 ** -10 * s.repeat_interleave(128, 2)[:, :, :300])
    assert bool(((back - x).abs() <= limit).all())
