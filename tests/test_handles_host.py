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


def test_the_pools_are_checked_for_the_row_the_mode_has_now(host):
    c = host.PagedCache(host.KVQ_INT4_TOKEN_HEAD, 3, 2, 16, 64, device="cpu")
    c.struct()
    for name, value in (("mode", host.KVQ_BF16_CACHE), ("head_dim", 128), ("num_blocks", 4)):
        old = getattr(c, name)
        setattr(c, name, value)
        with pytest.raises(ValueError):
            c.struct()
        setattr(c, name, old)
        assert c.struct().num_blocks == 3
    c.mode = host.KVQ_INT2_TOKEN_HEAD
    assert c.struct().mode == host.KVQ_INT2_TOKEN_HEAD and c.row_bytes == 20


def test_signs_and_channel_maxima_are_as_long_as_the_head_now_is(host):
    c = host.PagedCache(host.KVQ_INT4_TOKEN_HEAD, 3, 2, 16, 64, rht_signs=torch.ones(64, dtype=torch.int8), device="cpu")
    c.struct()
    row = host.kvq_row_bytes(host.KVQ_INT4_TOKEN_HEAD, 128)
    c.k_pages = c.v_pages = torch.zeros((3, 2, 16, row), dtype=torch.uint8)
    c.head_dim = 128
    with pytest.raises(ValueError, match="rht_signs"):
        c.struct()
    c.rht_signs = torch.ones(128, dtype=torch.int8)
    assert c.struct().head_dim == 128
    c = host.PagedCache(host.KVQ_INT8_CHANNEL, 3, 2, 16, 64, device="cpu")
    c.struct()
    c.ch_amax = torch.zeros((2, 1, 64))
    with pytest.raises(ValueError, match="ch_amax"):
        c.struct()


def test_a_paging_state_resized_in_place_is_seen(host):
    """The number of sequences and the table's width come from the tensors as they are at the call."""
    lens, table = torch.zeros(4, dtype=torch.int32), i32(4, 6)
    p = host.Paging(lens, block_tables=table)
    assert (p.struct().batch, p.struct().max_blocks) == (4, 6)
    first = p.struct()
    assert p.struct() is first
    at = lens.data_ptr()
    lens.resize_(2)
    assert lens.data_ptr() == at and p.struct().batch == 2
    buf = torch.zeros(9, dtype=torch.int32)
    p.seq_lens = buf[:3]
    assert p.struct().batch == 3
    p.seq_lens.data = buf[:4]           # the same address, another length
    assert p.struct().batch == 4
    table.resize_(4, 3)
    assert p.struct().max_blocks == 3
    p.seq_lens.data = buf[:9]
    with pytest.raises(ValueError):     # more sequences than the table has rows
        p.struct()
