"""What the binding hands to the library of a pool (no GPU needed)."""
import pytest
import torch


def _fields(kvq, pools):
    got = kvq._pool_structs(pools, -1)               # -1: tensors of the host
    return [(p.bits, p.num_heads, p.head_dim, p.page_size, p.num_pages, p.codes, p.scales) for p in got]


def _want(p):
    return (p.bits, p.num_heads, p.head_dim, p.page_size, p.num_pages, p.codes.data_ptr(), p.scales.data_ptr())


@pytest.mark.parametrize("bits", [8, 6, 4])
def test_pages_are_those_of_the_pool(kvq, bits):
    """However the codes are held: as bytes, as words, with a page's dimensions apart or in one."""
    p = kvq.Pool.empty(bits, 2, 64, 16, 7, "cpu")
    forms = [p.codes, p.codes.view(torch.int8), p.codes.view(torch.int32), p.codes.reshape(7, -1)]
    pools = [kvq.Pool(bits, 2, 64, 16, c, p.scales) for c in forms]
    assert _fields(kvq, pools) == [_want(x) for x in pools] and all(x.num_pages == 7 for x in pools)


def test_pools_of_other_classes(kvq):
    """Whatever has a pool's attributes: slots, properties."""
    base = kvq.Pool.empty(4, 2, 128, 16, 5, "cpu")

    class Slots:
        __slots__ = ("bits", "num_heads", "head_dim", "page_size", "codes", "scales", "num_pages")

    a = Slots()
    for name in Slots.__slots__:
        setattr(a, name, getattr(base, name))

    class Props:
        bits, num_heads, head_dim, page_size = 4, 2, 128, 16
        codes = property(lambda self: base.codes)
        scales = property(lambda self: base.scales)
        num_pages = property(lambda self: 5)

    assert _fields(kvq, [a, Props(), base]) == [_want(base)] * 3
    ref = kvq._PoolRef([a, Props()], -1)
    assert ref.at and len(ref.hold) == 10


def test_changed_pools(kvq):
    p = kvq.Pool.empty(4, 2, 64, 16, 5, "cpu")
    _fields(kvq, [p])
    q = kvq.Pool.empty(8, 1, 32, 32, 9, "cpu")
    for name in ("bits", "num_heads", "head_dim", "page_size", "codes", "scales"):
        setattr(p, name, getattr(q, name))
    assert _fields(kvq, [p]) == [_want(q)]


def test_negative_fields_are_left_to_the_library(kvq):
    p = kvq.Pool.empty(4, 2, 64, 16, 5, "cpu")
    p.page_size = -16
    assert kvq._pool_structs([p], -1)[0].page_size == -16
