"""Workspace queries of the 8-bit product and the experts: 0 for every size that the entry point refuses."""
import ctypes

import pytest

import int4_group_quantized_w4a16_amd as kaio
from tests.test_abi_host import PROB, UNSUP
from tests.test_products_host import experts, linear, moe


@pytest.mark.parametrize("m,n,k", [(1 << 24, 64, 256), (1 << 24, 64, 131056), (40, 1 << 26, 256), (1 << 20, 1 << 25, 256),
                                   (2 ** 32 - 1, 64, 256), (40, 2 ** 32 - 1, 256), (40, 64, 131072), (40, 64, 200)])
def test_linear_of_refused_sizes_needs_nothing(m, n, k):
    st, msg = linear(m=m, n=n, k=k, xs=0, size=1 << 62)
    assert st == PROB, msg
    for int8_x in (0, 1):
        assert kaio.lib().kaio_linear_w8a8_workspace_size(m, n, k, int8_x) == 0


def test_linear_of_the_largest_sizes_has_its_rows():
    size = kaio.lib().kaio_linear_w8a8_workspace_size
    for m, n, k in (((1 << 24) - 1, 16, 256), (1 << 17, (1 << 16) - 16, 131056), (40, (1 << 26) - 1, 256)):
        assert size(m, n, k, 0) >= m * k + 4 * m and size(m, n, k, 1) == 0


def test_experts_of_refused_sizes_need_nothing():
    for kw in (dict(group_size=64), dict(experts=513), dict(hidden=200), dict(inner=0), dict(hidden=1 << 24)):
        assert moe(**kw, size=1 << 40)[0] in (UNSUP, PROB)
        assert kaio.lib().kaio_moe_w4a16_workspace_size(ctypes.byref(experts(**kw)), 3, 2) == 0
