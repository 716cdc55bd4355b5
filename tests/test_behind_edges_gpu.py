"""The operators behind the selections at the ends of their ranges, on the GPU against their
definitions in 64 bits: logits of any size."""
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
