"""The binding's description of a pool of pages follows its tensor (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def fg():
    import __graft_entry__ as g
    g.build()
    from bit_compressed_throughput_gb300 import fg as mod
    return mod


def says(pool):
    s = pool.struct()
    assert (s.pages, s.page, s.h, s.H) == (pool.pages, pool.page, pool.h, pool.H)
    return s.blocks, s.pages, s.page, s.h, s.H


def test_replaced_blocks_are_the_ones_described(fg):
    pool = fg.KVPagesQ4(4, 16, 128, 2, device="cpu")
    first = pool.blocks
    assert says(pool) == (first.data_ptr(), 4, 16, 128, 2)
    pool.blocks = grown = torch.zeros((9, 2, 1152), dtype=torch.uint8)
    assert pool.blocks is grown and says(pool) == (grown.data_ptr(), 9, 16, 128, 2)
    assert pool.parts()[0].shape == (9, 2, 16, 32)
    pool.blocks = other = torch.zeros((3, 5, 64 * 72), dtype=torch.uint8)
    assert says(pool) == (other.data_ptr(), 3, 64, 320, 5)
    for bad in (grown.to(torch.int8), grown[:, :1], grown[0], torch.zeros((2, 2, 100)).byte(),
                torch.zeros((2, 2, 72 * 24)).byte()):
        with pytest.raises(ValueError):
            pool.blocks = bad
        assert pool.blocks is other and says(pool) == (other.data_ptr(), 3, 64, 320, 5)


def test_blocks_resized_in_place(fg):
    pool = fg.KVPagesQ4.of(torch.zeros((4, 2, 1152), dtype=torch.uint8), 64)
    pool.blocks.resize_((2, 2, 1152))
    assert says(pool) == (pool.blocks.data_ptr(), 2, 16, 128, 2)
    pool.blocks.set_(torch.zeros((1 << 22,), dtype=torch.uint8))
    with pytest.raises(ValueError):
        pool.struct()


@pytest.mark.parametrize("name", ["d", "H", "h", "page", "pages"])
def test_sizes_are_not_set_by_hand(fg, name):
    pool = fg.KVPagesQ4(4, 16, 128, 2, device="cpu")
    with pytest.raises(AttributeError):
        setattr(pool, name, 8)
    pool.label = "a caller's own"
    assert says(pool) == (pool.blocks.data_ptr(), 4, 16, 128, 2)
