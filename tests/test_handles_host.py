"""The handles of the binding and the C structs made of them, without a GPU: what a struct says follows the handle."""
import pytest
import torch

from test_abi import K  # noqa: F401


@pytest.fixture
def host(K, monkeypatch):  # noqa: F811
    """The package, with host tensors let through the device check."""
    monkeypatch.setattr(K, "_dev_ptr", lambda t, *a, **kw: None if t is None else t.data_ptr())
    return K


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


@pytest.mark.parametrize("kind", ["block_tables", "block_tables_headwise"])
def test_the_width_follows_the_table(host, kind):
    p = host.Paging(i32(2), **{kind: i32(4, 5)})
    assert p.struct().max_blocks == 5 == p.max_blocks
    for width in (3, 9):
        t = i32(4, width)
        setattr(p, kind, t)
        assert p.struct().max_blocks == width == p.max_blocks
        assert getattr(p.struct(), kind) == t.data_ptr()
    late = host.Paging(i32(2))
    assert late.max_blocks == 0
    setattr(late, kind, i32(2, 7))
    assert late.struct().max_blocks == 7
    for t in (i32(14), i32(2, 7, 1)):    # a row stride only a two-dimensional table has
        setattr(late, kind, t)
        with pytest.raises(ValueError):
            late.struct()
