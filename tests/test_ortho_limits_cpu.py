"""Sizes that zero_orthogonalize refuses before any launch."""
import pytest

Z = pytest.importorskip("zero_sharded_optimizer_device_gb300")


@pytest.mark.parametrize("m,n", [(1, 2 ** 28 + 1), (2 ** 28 + 1, 1), (2 ** 29, 1), (3, 2 ** 30)])
def test_sides_whose_products_would_outlast_their_waits(m, n):
    """A pair of CTAs walks a Gram product of one tile alone, some 400 cycles every 64 columns; whoever waits for it gives up after 4e9: 2^29 would come near that."""
    with pytest.raises(Z.ZeroError) as e:
        Z.zero_orthogonalize_workspace(m, n, 1)
    assert e.value.name == "ZERO_ERANGE"


def test_the_longest_sides():
    for m, n in ((1, 2 ** 28), (2 ** 28, 1), (2 ** 28 - 5, 40)):
        assert Z.zero_orthogonalize_workspace(m, n, 1) > 0
