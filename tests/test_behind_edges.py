"""Host-side checks of the operators behind the selections at the ends of their ranges, without a GPU."""
import pytest

P = 1 << 20   # a 16-byte aligned address that is never read: the checks run first
INVALID, ALIGNMENT = 1, 2


@pytest.fixture(scope="module")
def ds():
    from top_selection_gb300 import build
    build.build()
    import top_selection_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("change,want", [
    (dict(block=-1), INVALID),
    (dict(x=0), INVALID),
    (dict(out=P + 1), ALIGNMENT),
    (dict(rows=0, x=0), 0),
])
def test_expert_product_probe_refuses(ds, change, want):
    a = dict(block=0, x=P, x_scales=P, rows=4, K=256, x_stride=256, w=P, w_scales=P, E=8, N=100, w_row_stride=256,
             w_matrix_stride=25600, offsets=P, dtype=0, out=P)
    a.update(change)
    assert ds.ds_expert_product_probe(**a) == want
