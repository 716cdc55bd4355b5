"""Host-side checks of the operators around the top-k that need no GPU: refusals come before
anything is launched, and the formulas the GPU tests compare against hold by themselves."""
import numpy as np
import pytest

import operator_ref as ref

P = 1 << 20   # a 16-byte aligned address that is never read: the checks run first


@pytest.fixture(scope="module")
def ds():
    from top_selection_gb300 import build
    build.build()
    import top_selection_gb300 as m
    m.load()
    return m


INVALID, ALIGNMENT, UNSUPPORTED = 1, 2, 3


@pytest.mark.parametrize("change,want", [
    (dict(dtype=2), INVALID),
    (dict(rows=-1), INVALID),
    (dict(E=0), INVALID),
    (dict(row_stride=63), INVALID),
    (dict(k=0), INVALID),
    (dict(k=65), INVALID),                                # more than there are experts
    (dict(groups=8, topk_groups=2, k=17), INVALID),       # more than the groups hold
    (dict(groups=7), INVALID),                            # 64 experts in 7 groups
    (dict(groups=8, topk_groups=9), INVALID),
    (dict(groups=8, topk_groups=0), INVALID),
    (dict(scoring=2), INVALID),
    (dict(group_score=-1), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(logits=0), INVALID),
    (dict(out_weights=0), INVALID),
    (dict(out_experts=0), INVALID),
    (dict(logits=P + 2), ALIGNMENT),
    (dict(bias=P + 2), ALIGNMENT),
    (dict(out_experts=P + 1), ALIGNMENT),
    (dict(E=513, row_stride=513), UNSUPPORTED),
    (dict(k=33), UNSUPPORTED),
    (dict(groups=64, topk_groups=8), UNSUPPORTED),
    (dict(rows=0, logits=0), 0),
])
def test_route_refuses(ds, change, want):
    a = dict(logits=P, dtype=1, rows=2, E=64, row_stride=64, k=4, scoring=0, bias=0, groups=1, topk_groups=1,
             group_score=0, renormalise=True, scale=1.0, out_weights=P, out_experts=P)
    a.update(change)
    assert ds.ds_route(**a) == want


@pytest.mark.parametrize("change,want", [
    (dict(dtype=7), INVALID),
    (dict(k=65), INVALID),
    (dict(k=0), INVALID),
    (dict(grad_stride=63), INVALID),
    (dict(scoring=3), INVALID),
    (dict(scale=float("nan")), INVALID),
    (dict(experts=0), INVALID),
    (dict(grad_logits=0), INVALID),
    (dict(grad_logits=P + 2), ALIGNMENT),
    (dict(k=40), UNSUPPORTED),
    (dict(E=1024, row_stride=1024, grad_stride=1024), UNSUPPORTED),
    (dict(rows=0), 0),
])
def test_route_backward_refuses(ds, change, want):
    a = dict(grad_weights=P, logits=P, dtype=1, rows=2, E=64, row_stride=64, k=4, experts=P, scoring=0,
             renormalise=True, scale=1.0, grad_logits=P, grad_stride=64)
    a.update(change)
    assert ds.ds_route_backward(**a) == want


@pytest.mark.parametrize("change,want", [
    (dict(dtype=2), INVALID),
    (dict(sequences=-1), INVALID),
    (dict(drafts_per_sequence=-1), INVALID),
    (dict(V=0), INVALID),
    (dict(row_stride=99), INVALID),
    (dict(noise_stride=99), INVALID),
    (dict(probs_row_stride=99), INVALID),
    (dict(temperature=-1.0), INVALID),
    (dict(temperature=float("inf")), INVALID),
    (dict(temperature=float("nan")), INVALID),
    (dict(logits=0), INVALID),
    (dict(drafts=0), INVALID),
    (dict(uniforms=0), INVALID),
    (dict(noise=0), INVALID),
    (dict(out_tokens=0), INVALID),
    (dict(out_accepted=0), INVALID),
    (dict(noise=P + 2), ALIGNMENT),
    (dict(logits=P + 2), ALIGNMENT),
    (dict(drafts_per_sequence=1025), UNSUPPORTED),
    (dict(V=(1 << 30) + 1, row_stride=1 << 31, noise_stride=1 << 31, probs_row_stride=1 << 31), UNSUPPORTED),
    (dict(sequences=0, logits=0), 0),
])
def test_verify_refuses(ds, change, want):
    a = dict(logits=P, dtype=1, sequences=2, drafts_per_sequence=3, V=100, seq_stride=400, row_stride=100, drafts=P,
             draft_lens=0, draft_probs=P, probs_seq_stride=300, probs_row_stride=100, uniforms=P, noise=P,
             noise_stride=100, temperatures=0, temperature=1.0, out_tokens=P, out_accepted=P)
    a.update(change)
    assert ds.ds_verify_drafts(**a) == want


@pytest.mark.parametrize("change,want", [
    (dict(dtype=2), INVALID),
    (dict(tokens=-1), INVALID),
    (dict(heads=0), INVALID),
    (dict(page=0), INVALID),
    (dict(pages=-1), INVALID),
    (dict(k=0), INVALID),
    (dict(slots=0), INVALID),
    (dict(cache=0), INVALID),
    (dict(v_head_stride=-8), INVALID),
    (dict(k_head_stride=100), ALIGNMENT),
    (dict(v=P + 8), ALIGNMENT),
    (dict(cache=P + 8), ALIGNMENT),
    (dict(scales=P + 4), ALIGNMENT),
    (dict(page=48), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED),
    (dict(tokens=0, k=0), 0),
])
def test_cache_store_refuses(ds, change, want):
    a = dict(k=P, v=P, dtype=0, tokens=3, heads=2, D=128, k_token_stride=256, k_head_stride=128, v_token_stride=256,
             v_head_stride=128, cache=P, scales=P, pages=4, page=16, slots=P)
    a.update(change)
    assert ds.ds_cache_store(**a) == want


@pytest.mark.parametrize("change,want", [
    (dict(dtype=9), INVALID),
    (dict(out_v=0), INVALID),
    (dict(out_k=P + 4), ALIGNMENT),
    (dict(D=32), UNSUPPORTED),
    (dict(tokens=0), 0),
])
def test_cache_load_refuses(ds, change, want):
    a = dict(cache=P, scales=P, pages=4, page=16, slots=P, tokens=3, heads=2, D=128, dtype=0, out_k=P, out_v=P)
    a.update(change)
    assert ds.ds_cache_load(**a) == want


@pytest.mark.parametrize("change,want", [
    (dict(dtype=2), INVALID),
    (dict(sequences=-1), INVALID),
    (dict(tokens=0), INVALID),
    (dict(q_heads=7), INVALID),                           # not a multiple of the key heads
    (dict(pages=0), INVALID),
    (dict(table_width=0), INVALID),
    (dict(table_stride=3), INVALID),
    (dict(K=-1), INVALID),
    (dict(K=8), INVALID),                                 # a list's length without a list
    (dict(q_head_stride=-1), INVALID),
    (dict(scale=float("nan")), INVALID),
    (dict(q=0), INVALID),
    (dict(lens=0), INVALID),
    (dict(out=0), INVALID),
    (dict(cache=P + 8), ALIGNMENT),
    (dict(scales=P + 4), ALIGNMENT),
    (dict(table=P + 2), ALIGNMENT),
    (dict(q=P + 1), ALIGNMENT),
    (dict(D=80), UNSUPPORTED),
    (dict(page=24), UNSUPPORTED),
    (dict(pages=1 << 28), UNSUPPORTED),                   # more entries than 32 bits count
    (dict(table_width=1 << 27, table_stride=1 << 27), UNSUPPORTED),
    (dict(sequences=0), 0),
])
def test_cache_attention_refuses(ds, change, want):
    a = dict(q=P, dtype=0, sequences=2, tokens=1, q_heads=8, D=128, q_seq_stride=1024, q_token_stride=1024,
             q_head_stride=128, cache=P, scales=P, pages=8, heads=2, page=16, table=P, table_width=4, table_stride=4,
             lens=P, indices=0, K=0, scale=0.1, out=P)
    a.update(change)
    assert ds.ds_cache_attention(**a) == want


def test_python_entry_points_refuse_cpu_tensors(ds):
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        ds.route(x, 4)
    with pytest.raises(ValueError, match="CUDA"):
        ds.verify_drafts(x.view(1, 2, 64), None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        ds.cache_load(torch.zeros(1, 1, 16, 2, 64, dtype=torch.uint8), None, torch.zeros(1))


# ---------------------------------------------------- the formulas by themselves ----

@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_gate_gradient_against_differences(scoring, renormalise):
    """The gradient's formula against central differences of the weights' formula, the choice
    held: with step h the difference's own error is of the order h^2 = 1e-10 and rounding's
    1e-16 / h = 1e-11, each times values of the order 1."""
    rng = np.random.default_rng(4)
    x, g = rng.standard_normal((5, 12)), rng.standard_normal((5, 3))
    chosen = np.stack([rng.permutation(12)[:3] for _ in range(5)])
    got = ref.route_gradient(g, x, chosen, scoring, renormalise, 2.5)
    h = 1e-5
    for e in range(12):
        up, down = x.copy(), x.copy()
        up[:, e] += h
        down[:, e] -= h
        w = [ref.route_weights(y, chosen, scoring, renormalise, 2.5) for y in (up, down)]
        diff = ((w[0] - w[1]) / (2 * h) * g).sum(-1)
        assert np.allclose(got[:, e], diff, rtol=0, atol=1e-8)


def test_race_draws_the_distribution():
    """argmax r / e with exponential e draws v with probability r_v / sum r: 20000 draws, five
    standard deviations of a share."""
    rng = np.random.default_rng(5)
    r = np.array([0.5, 0.0, 0.2, 0.05, 0.25]) * 3
    n = 20000
    got = np.bincount((r / rng.exponential(size=(n, 5))).argmax(-1), minlength=5) / n
    p = r / r.sum()
    assert np.all(np.abs(got - p) <= 5 * np.sqrt(p * (1 - p) / n))


def test_codes_round_trip():
    """A row's values come back within half a step, where the rounding of s and m to 8 bits
    lets the codes reach: s/2 + 15 s 2^-9 (s itself) + |m| 2^-8 (a minimum rounded up)."""
    rng = np.random.default_rng(6)
    x = rng.standard_normal((50, 64)).astype(np.float32) * np.exp(rng.uniform(-20, 20, (50, 1))).astype(np.float32)
    codes, s, m = ref.quantise(x)
    back = ref.value(codes, s, m)
    assert codes.min() >= 0 and codes.max() <= 15
    limit = s * (0.5 + 15 * 2.0 ** -9) + np.abs(m) * 2.0 ** -8
    assert np.all(np.abs(back - x) <= limit[:, None] * (1 + 1e-6))
    assert np.array_equal(ref.unpack(ref.pack(codes)), codes)
