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


def test_short_sequences_need_no_state_each(g):
    """A packed batch has room for the states of cut sequences' pieces: no more than the balanced share calls for,
    however many sequences there are."""
    H, d = 16, 128
    state = 4 * d * d * H

    def fwd(n, tokens):
        return g.lib.gdn2_linattn_fwd_workspace_size(ctypes.byref(g.LinattnDims(n, tokens, H, H, d, d, 0, 0, 0, 0)), 1)

    few, many = fwd(32, 65536), fwd(1024, 65536)
    assert many - few < 1024 * 64               # offsets and order, no states
    assert many < 160 * 4 * d * d + (1 << 20)   # at most a piece for each of the SMs
    assert fwd(32, 65536) > state               # sequences long enough to be cut may be among them
    # the gradients': marks and dots grow with the batch, the pieces' states (three runs) do not
    bwd = [g.lib.gdn2_linattn_bwd_workspace_size(
        ctypes.byref(g.LinattnDims(n, 65536, H, H, d, d, 0, 0, g.LINATTN_HEAD_DECAY, 0)), 1) for n in (1, 1024)]
    assert bwd[1] < bwd[0] + 1024 * 64 and bwd[1] < 3 * 160 * 4 * d * d + (1 << 20)


def test_gradients_of_a_packed_batch_take_one_launch_by_its_size(g):
    """Seen from the workspace: two runs' marks of the state where the three share a launch, one run's else."""
    H, d = 16, 128
    mark = 4 * d * d * H

    def bwd(n, tokens, packed):
        return g.lib.gdn2_linattn_bwd_workspace_size(
            ctypes.byref(g.LinattnDims(n, tokens if packed else tokens // n, H, H, d, d, 0, 0, 0, 0)), packed)

    groups = 32768 // 256 + 8
    both = 2 * groups * mark
    assert bwd(8, 32768, 0) < both and bwd(8, 32768, 1) < both        # as many units as SMs, long: one after the other
    assert bwd(11, 9001, 1) > 2 * (9001 // 256 + 11) * mark           # short ones, ragged: one launch
    assert bwd(1, 4096, 0) > 2 * (4096 // 256) * mark                 # SMs idle: one launch


def test_every_output_apart_from_every_input(g):
    """S_T, the offsets and the indices as well: an address used twice is refused, but for S_T at S0's."""
    at = [ctypes.c_void_p((i + 1) << 20) for i in range(20)]
    dims = g.LinattnDims(2, 100, 2, 2, 128, 128, 0, 0, 0, 0)
    ws = ctypes.c_void_p(1 << 40)

    def fwd(**kw):
        a = dict(zip(("q", "k", "v", "log_a", "S0", "cu", "o", "S_T"), at), **kw)
        rc = g.lib.gdn2_linattn_fwd(a["q"], a["k"], a["v"], a["log_a"], a["S0"], a["cu"], a["o"], a["S_T"],
                                    ctypes.byref(dims), ws, 1 << 50, None)
        return rc, g.lib.gdn2_last_error().decode()

    for kw in (dict(S_T=at[0]), dict(S_T=at[1]), dict(S_T=at[2]), dict(S_T=at[3]), dict(S_T=at[5]), dict(o=at[4]),
               dict(o=at[5]), dict(o=at[7])):
        rc, msg = fwd(**kw)
        assert rc == g.ERR_INVALID_ARG and "address" in msg, kw
    one = g.LinattnDims(2, 1, 2, 2, 128, 128, 0, 0, 0, 0)
    for S, o in ((at[4], at[6]), (at[5], at[4])):  # the indices at at[4]
        rc = g.lib.gdn2_linattn_step(at[0], at[1], at[2], at[3], S, 2, at[4], o, ctypes.byref(one), None)
        assert rc == g.ERR_INVALID_ARG and "address" in g.lib.gdn2_last_error().decode()
    grads = [at[7 + i] for i in range(5)]
    for i in range(5):
        out = [at[6] if i == j else x for j, x in enumerate(grads)]  # the offsets at at[6]
        rc = g.lib.gdn2_linattn_bwd(at[0], at[1], at[2], at[3], None, at[6], at[4], None, *out, ctypes.byref(dims), ws,
                                    1 << 50, None)
        assert rc == g.ERR_INVALID_ARG and "address" in g.lib.gdn2_last_error().decode()
        rc = g.lib.gdn2_linattn_bwd_ckpt8(*[at[12 + j] for j in range(6)], at[3], None, at[6], at[4], None, *out,
                                          ctypes.byref(dims), ws, 1 << 50, None)
        assert rc == g.ERR_INVALID_ARG and "address" in g.lib.gdn2_last_error().decode()
