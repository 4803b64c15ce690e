"""Sizes at the ends of what the linear-attention calls take, on the host."""
import ctypes

import pytest

P = ctypes.c_void_p(1 << 20)  # an aligned placeholder, never dereferenced


@pytest.fixture(scope="module")
def g():
    from gated_delta_rule_159_b200 import build
    build.build()
    from gated_delta_rule_159_b200 import gdn2
    return gdn2


def _sizes(g, dims, packed):
    return [getattr(g.lib, f"gdn2_linattn_{n}_workspace_size")(ctypes.byref(dims), packed)
            for n in ("fwd", "bwd", "bwd_ckpt8")]


@pytest.mark.parametrize("d,dtype", [(1, 0), (128, 0), (24, 1)])
def test_token_numbers_stay_in_32_bits(g, d, dtype):
    """A loop steps up to 2^14 tokens past a sequence's end before it looks."""
    most = 2 ** 31 - 2 ** 15
    for n, length, packed in ((1, most, 0), (7, most, 1), (2 ** 16 - 1, 2 ** 15, 0)):
        dims = g.LinattnDims(n, length, 1, 1, d, d, dtype, dtype, 0, 0)
        assert all(_sizes(g, dims, packed))
    for n, length, packed in ((1, most + 1, 0), (1, 2 ** 31 - 1, 0), (7, most + 1, 1), (7, 2 ** 31 - 1, 1),
                              (2 ** 26 - 1, 32, 0)):
        dims = g.LinattnDims(n, length, 1, 1, d, d, dtype, dtype, 0, 0)
        assert not any(_sizes(g, dims, packed)), (n, length, packed)
        cu = P if packed else None
        assert g.lib.gdn2_linattn_fwd(P, P, P, P, None, cu, P, None, ctypes.byref(dims), P, 1 << 50,
                                      None) == g.ERR_UNSUPPORTED
