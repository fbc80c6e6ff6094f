"""Limits of the operators between a layer's linears that follow from their number
ranges and workspaces.  No GPU: the pointers are never dereferenced."""
import pytest

from tests.test_layer_host import L, linear  # noqa: F401  (L: a fixture)


@pytest.mark.parametrize("scale,status", [(2.0 ** 65, -1), (-2.0 ** 65, -1), (1e30, -1)])
def test_scale(L, scale, status):  # noqa: F811
    """Outputs' factors are the scale times 2^40."""
    assert linear(L, scale=scale) == status
