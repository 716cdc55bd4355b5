"""Checks of the operators around the top-k that need no GPU: sizes whose products pass 32 or 64 bits
are refused before anything is launched, and a call is made on its tensors' device."""
import warnings

import pytest

P = 1 << 20   # a 16-byte aligned address that is never read: the checks run first
UNSUPPORTED = 3


@pytest.fixture(scope="module")
def ds():
    from top_selection_gb300 import build
    build.build()
    import top_selection_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("change", [
    dict(indices=P, K=(1 << 30) + 1),                                   # places of a list
    dict(indices=P, K=(1 << 31) - 1),
    dict(pages=1 << 30, page=1 << 30, heads=16, q_heads=16, table_width=1, table_stride=1),   # 2^64 entries
    dict(pages=(1 << 31) - 1, page=1 << 30, heads=(1 << 31) - 1, q_heads=(1 << 31) - 1, table_width=1, table_stride=1),
    dict(sequences=1 << 40, tokens=1 << 30, heads=8, indices=P, K=1),                          # 2^73 lists
    dict(sequences=1 << 62, heads=4),                                                          # 2^64 units
    dict(sequences=1 << 32),
])
def test_cache_attention_refuses_sizes(ds, change):
    a = dict(q=P, dtype=0, sequences=2, tokens=1, q_heads=8, D=128, q_seq_stride=1024, q_token_stride=1024,
             q_head_stride=128, cache=P, scales=P, pages=8, heads=2, page=16, table=P, table_width=4, table_stride=4,
             lens=P, indices=0, K=0, scale=0.1, out=P)
    a.update(change)
    assert ds.ds_cache_attention(**a) == UNSUPPORTED


@pytest.mark.parametrize("change", [dict(pages=1 << 40, page=1 << 30), dict(pages=1 << 62, page=2)])
def test_cache_store_refuses_sizes(ds, change):
    a = dict(k=P, v=P, dtype=0, tokens=3, heads=2, D=128, k_token_stride=256, k_head_stride=128, v_token_stride=256,
             v_head_stride=128, cache=P, scales=P, pages=4, page=16, slots=P)
    a.update(change)
    assert ds.ds_cache_store(**a) == UNSUPPORTED


def test_route_refuses_sizes(ds):
    rows = (1 << 63) - 1
    assert ds.ds_route(logits=P, dtype=1, rows=rows, E=64, row_stride=64, k=4, scoring=0, bias=0, groups=1, topk_groups=1,
                       group_score=0, renormalise=True, scale=1.0, out_weights=P, out_experts=P) == UNSUPPORTED
    assert ds.ds_route_backward(grad_weights=P, logits=P, dtype=1, rows=rows, E=64, row_stride=64, k=4, experts=P,
                                scoring=0, renormalise=True, scale=1.0, grad_logits=P, grad_stride=64) == UNSUPPORTED


def test_a_call_is_made_on_its_tensors_device(ds):
    """Tensors of a device that does not exist, and no tokens: the call has to fail in making that
    device current, where on the current device it would return with nothing to do."""
    torch = pytest.importorskip("torch")
    fake = pytest.importorskip("torch._subclasses.fake_tensor")
    at = f"cuda:{torch.cuda.device_count() + 1}"
    with fake.FakeTensorMode():
        kv = torch.empty(0, 2, 64, device=at, dtype=torch.bfloat16)
        cache = torch.empty(2, 2, 16, 2, 32, device=at, dtype=torch.uint8)
        scales = torch.empty(2, 2, 16, 4, device=at, dtype=torch.bfloat16)
        slots = torch.empty(0, device=at, dtype=torch.int32)
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")     # of reading a fake tensor's address
        with pytest.raises(RuntimeError):
            ds.cache_store(kv, kv, cache, scales, slots, stream=0)


def test_binding_of_another_torch(ds, monkeypatch):
    """A binding built against another torch is built anew, and not loaded."""
    pytest.importorskip("torch")
    from top_selection_gb300 import build
    assert build.up_to_date() and build.binding_matches()
    monkeypatch.setattr(build, "_torch_version", lambda: "0.1+other", raising=False)
    assert not build.up_to_date()
    monkeypatch.setattr(ds, "_binding", None)
    with pytest.raises(RuntimeError, match="another torch"):
        ds.route(None, 1)


def test_captures_of_the_topk_outlive_the_other_operators(tmp_path, monkeypatch):
    """An edit of another operator's source, which includes none of the top-k's kernels, leaves the
    digest of its captures as it is; an edit of a shared header does not."""
    import os
    import bench
    csrc = os.path.join(os.path.dirname(os.path.abspath(bench.__file__)), "top_selection_gb300", "csrc")
    kernels = ("ds_split.cuh", "ds_select.cuh")
    for name in bench.OTHER_OPERATORS:
        text = open(os.path.join(csrc, name)).read()
        assert not any(f'#include "{k}"' in text for k in kernels)
    tree = tmp_path / "top_selection_gb300" / "csrc"
    tree.mkdir(parents=True)
    for name in ("ds_topk.cu", "ds_common.cuh", *bench.OTHER_OPERATORS):
        (tree / name).write_text(name)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    digest = bench._source_digest()
    for name in bench.OTHER_OPERATORS:
        (tree / name).write_text("edited")
    assert bench._source_digest() == digest
    (tree / "ds_common.cuh").write_text("edited")
    assert bench._source_digest() != digest
