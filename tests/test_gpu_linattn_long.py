"""Linear attention on the GPU where many chunks, pieces and blocks meet: long uncut sequences, ragged
batches of more units than SMs, decays on both sides of the kernels' limits, and the bounded waits."""
import pytest
import torch

import linattn_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU test"
    from gated_delta_rule_159_b200 import gdn2
    return gdn2


def _check_units(g, p, cu, H, Hqk, tc, units):
    """Forward and gradients of a few (sequence, head) units against float64; the statuses are clean."""
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    o, S = g.linattn_fwd(p["q"], p["k"], p["v"], p["log_a"], p["S0"], p["cu"], workspace=ws)
    assert g.check_status(ws) == g.OK
    got = g.linattn_bwd(p["q"], p["k"], p["v"], p["log_a"], p["dO"], p["S0"], p["dS_T"], p["cu"])
    assert g.check_status(got["workspace"]) == g.OK
    share = H // Hqk
    for n, h in units:
        s = slice(cu[n], cu[n + 1])
        # the heads of h's group alone: a problem of one sequence
        heads = slice(h // share * share, h // share * share + share)
        one = {"cu": None, "q": p["q"][s, h // share:h // share + 1], "k": p["k"][s, h // share:h // share + 1],
               "v": p["v"][s, heads], "dO": p["dO"][s, heads],
               "log_a": p["log_a"][heads] if p["log_a"].dim() == 1 else p["log_a"][s, heads],
               "S0": None if p["S0"] is None else p["S0"][n:n + 1, heads],
               "dS_T": None if p["dS_T"] is None else p["dS_T"][n:n + 1, heads]}
        length = cu[n + 1] - cu[n]
        want = ref.forward(one, [0, length], share, 1, tc)
        ref.check("o", o[s, heads], *want["o"])
        ref.check("S_T", S[n:n + 1, heads], *want["S_T"])
        grads = ref.gradients(one, [0, length], share, 1, tc)
        for name in ("dq", "dk", "dv", "dlog_a", "dS0"):
            if got[name] is None:
                continue
            mine = {"dq": lambda: got["dq"][s, h // share:h // share + 1], "dk": lambda: got["dk"][s, h // share:h // share + 1],
                    "dv": lambda: got["dv"][s, heads], "dlog_a": lambda: got["dlog_a"][s, heads],
                    "dS0": lambda: got["dS0"][n:n + 1, heads]}[name]()
            ref.check(name, mine, *grads[name])


@pytest.mark.parametrize("decay", ["token", "reset", "none"])
def test_many_chunks_in_every_block(g, decay):
    """148 and more blocks of 16 chunks each, uncut: every barrier goes round many times."""
    lens = (2048,) * 8
    p, cu = ref.problem(lens, 20, 20, 128, 128, BF, decay, True, seed=31)
    _check_units(g, p, cu, 20, 20, True, [(0, 0), (7, 19)])


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 128, 128), (F32, 40, 72)])
def test_ragged_batch_of_more_units_than_blocks_run_at_once(g, dtype, dk, dv):
    """The blocks start in the order of the pieces' lengths; lengths of 0 and 1 among them."""
    lens = (5, 700, 0, 129, 1, 640, 128, 33, 257, 64, 2, 511, 300, 31, 127, 90, 12, 0, 260, 77)
    p, cu = ref.problem(lens, 32, 16, dk, dv, dtype, "token", True, seed=32)
    _check_units(g, p, cu, 32, 16, dtype == BF, [(1, 0), (4, 31), (6, 7), (11, 16)])


@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("lens", [(1700, 900, 40, 0, 1), (129, 300, 0, 7)])
def test_gradients_side_by_side(g, lens, decay):
    """Few units: the three gradients share a launch, with sequences cut and uncut, of shared q and k."""
    p, cu = ref.problem(lens, 4, 2, 128, 128, BF, decay, True, seed=39)
    _check_units(g, p, cu, 4, 2, True, [(0, 0), (1, 2), (3, 0), (len(lens) - 1, 2)])


@pytest.mark.parametrize("la", [-0.05, -0.17, -0.18, -0.36, -103.0, -104.5])
def test_decays_on_both_sides_of_the_limits(g, la):
    """A chunk of 128 tokens decays by 2^-32 at log_a = -0.1733: below it the state's accumulator is
    scaled back every chunk, above it now and then; e^-104 is 0."""
    p, cu = ref.problem((700, 260), 2, 1, 128, 128, BF, "head", True, seed=33)
    p["log_a"] = torch.tensor([la, la / 2], device="cuda")
    _check_units(g, p, cu, 2, 1, True, [(0, 0), (1, 0)])


def test_sharp_changes_of_the_decay(g):
    """Resets right at, before and behind the edges of chunks and of 32-token blocks."""
    p, cu = ref.problem((650,), 1, 1, 128, 128, BF, "token", True, seed=34)
    for t in (0, 31, 32, 127, 128, 129, 255, 383, 384, 511, 640, 649):
        p["log_a"][t] = -float("inf")
    p["log_a"][200:210] = -30.0
    _check_units(g, p, cu, 1, 1, True, [(0, 0)])


def test_wait_times_out_then_recovers(g):
    """The first block's wait for a load that never comes gives up; the next call is clean."""
    p, cu = ref.problem((300, 40), 2, 2, 128, 128, BF, "token", True, seed=35)
    args = [p[x] for x in ("q", "k", "v", "log_a")]
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    g.debug_timeout_once(g.DEBUG_LINATTN, 1_000_000)
    g.linattn_fwd(*args, p["S0"], p["cu"], workspace=ws)
    assert g.check_status(ws) == g.ERR_TIMEOUT
    o, S = g.linattn_fwd(*args, p["S0"], p["cu"], workspace=ws)
    assert g.check_status(ws) == g.OK
    want = ref.forward(p, cu, 2, 2, True)
    ref.check("o", o, *want["o"])
    ref.check("S_T", S, *want["S_T"])


@pytest.mark.parametrize("heads", [2, 80])
def test_wait_of_the_gradients_times_out_then_recovers(g, heads):
    """The same with the three runs in one launch (2 heads), and one after the other (80)."""
    p, cu = ref.problem((300, 40), heads, heads, 128, 128, BF, "token", True, seed=40)
    args = [p[x] for x in ("q", "k", "v", "log_a", "dO", "S0", "dS_T", "cu")]
    want = g.linattn_bwd(*args)
    assert g.check_status(want["workspace"]) == g.OK
    g.debug_timeout_once(g.DEBUG_LINATTN, 1_000_000)
    ws = g.linattn_bwd(*args)["workspace"]
    assert g.check_status(ws) == g.ERR_TIMEOUT
    got = g.linattn_bwd(*args, workspace=ws)
    assert g.check_status(ws) == g.OK
    for name in ("dq", "dk", "dv", "dlog_a", "dS0"):
        assert torch.equal(got[name], want[name])


def test_two_graphs_and_their_workspaces(g):
    """Two captured graphs with one workspace replay in turn; calls of other sizes run between them."""
    p, cu = ref.problem((900, 200), 4, 2, 128, 128, BF, "token", True, seed=36)
    r, _ = ref.problem((130,), 4, 2, 128, 128, BF, "token", True, seed=37)
    ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    first = [p[x] for x in ("q", "k", "v", "log_a")], [r[x] for x in ("q", "k", "v", "log_a")]
    want = [g.linattn_fwd(*a, x["S0"], x["cu"], workspace=ws) for a, x in zip(first, (p, r))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for a, x in zip(first, (p, r)):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                outs.append(g.linattn_fwd(*a, x["S0"], x["cu"], workspace=ws))
            graphs.append(graph)
    torch.cuda.synchronize()
    for i in (0, 1, 1, 0, 1):
        for t in outs[i]:
            t.zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        for a, b in zip(outs[i], want[i]):
            assert torch.equal(a, b)
        g.linattn_bwd(*first[1], r["dO"], r["S0"], r["dS_T"], r["cu"], workspace=ws)


def test_a_training_step_from_checkpoints(g):
    """Save q, k and v in 8 bits, run the prompt, take the gradients from the checkpoints: they are those
    at the restored values, bit for bit, and near those at the originals."""
    p, cu = ref.problem((400, 77), 4, 2, 128, 128, BF, "token", True, seed=38)
    saved = [g.ckpt8_save(p[x]) for x in "qkv"]
    g.linattn_fwd(p["q"], p["k"], p["v"], p["log_a"], p["S0"], p["cu"])
    got = g.linattn_bwd_ckpt8(*saved, p["log_a"], p["dO"], p["S0"], p["dS_T"], p["cu"])
    back = [g.ckpt8_restore(*s) for s in saved]
    want = g.linattn_bwd(*back, p["log_a"], p["dO"], p["S0"], p["dS_T"], p["cu"])
    plain = g.linattn_bwd(p["q"], p["k"], p["v"], p["log_a"], p["dO"], p["S0"], p["dS_T"], p["cu"])
    for x in ("dq", "dk", "dv", "dlog_a", "dS0"):
        assert torch.equal(got[x], want[x]), x
        if x == "dlog_a":  # differences of sums: no bound of its own on the relative error
            continue
        # A code is off by up to half a step, 1 / sqrt(12) of a step in the root mean square; the step is at
        # most the block's largest value / 63.5, and the largest of 32 normal values is about 2.4 times
        # their root mean square: 1.1% a saved factor, of which every gradient has two at most: 1.6%.
        off = (got[x].double() - plain[x].double()).norm() / plain[x].double().norm()
        assert off < 2 * 0.016, (x, float(off))


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 24)])
def test_the_first_token_decays_nothing_without_a_state(g, dtype, d):
    p, cu = ref.problem((1, 200, 1, 0, 2), 2, 1, d, d, dtype, "token", False, seed=39)
    dS_T = torch.randn(5, 2, d, d, device="cuda")
    got = g.linattn_bwd(p["q"], p["k"], p["v"], p["log_a"], p["dO"], None, dS_T, p["cu"])
    first = [c for c, e in zip(cu, cu[1:]) if e > c]
    assert (got["dlog_a"][first] == 0).all() and (got["dlog_a"][cu[1] + 1:cu[2]] != 0).any()
