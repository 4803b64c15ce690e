"""Linear attention on the GPU where a loose bound would hide a fault: states that nothing is written to,
errors in the norm, gradients of log_a, calls from two threads."""
import ctypes
import subprocess

import pytest
import torch

import linattn_ref as ref
from test_gpu_linattn_long import _check_units

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU test"
    from gated_delta_rule_159_b200 import gdn2
    return gdn2


CALLER = r"""
#include <pthread.h>
#include <stddef.h>
#include <stdint.h>
typedef int (*fwd_t)(const void *, const void *, const void *, const void *, const float *, const int32_t *, void *,
                     float *, const void *, void *, size_t, void *);
struct call { fwd_t fn; const void *q, *k, *v, *la, *S0; void *o, *S, *ws, *stream; const void *dims; int64_t n, bad; };
static void *work(void *arg) {
  struct call *c = arg;
  for (int64_t i = 0; i < c->n; ++i)
    c->bad += c->fn(c->q, c->k, c->v, c->la, c->S0, NULL, c->o, c->S, c->dims, c->ws, 256, c->stream) != 0;
  return NULL;
}
void run(struct call *c, int threads) {
  pthread_t t[16];
  for (int i = 0; i < threads; ++i) pthread_create(&t[i], NULL, work, &c[i]);
  for (int i = 0; i < threads; ++i) pthread_join(t[i], NULL);
}
"""


class Call(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("fn", "q", "k", "v", "log_a", "S0", "o", "S", "ws", "stream", "dims")] + [
        ("n", ctypes.c_int64), ("bad", ctypes.c_int64)]


def test_threads_with_heads_of_two_sizes(g, tmp_path):
    """The fp32 run's shared memory differs by head size; no thread's launches may see another's."""
    src, so = tmp_path / "caller.c", tmp_path / "caller.so"
    src.write_text(CALLER)
    subprocess.check_call(["gcc", "-O2", "-shared", "-fPIC", "-pthread", str(src), "-o", str(so)])
    calls, kept = (Call * 4)(), []
    for i, d in enumerate((40, 128, 40, 128)):
        p = ref.problem((3,), 1, 1, d, d, F32, "token", True, seed=50 + d)[0]
        want = g.linattn_fwd(p["q"], p["k"], p["v"], p["log_a"], p["S0"])
        dims = g.LinattnDims(1, 3, 1, 1, d, d, g.F32, g.F32, 0, 0)
        o, S, ws = torch.empty_like(p["v"]), torch.empty_like(p["S0"]), torch.empty(256, dtype=torch.uint8, device="cuda")
        stream = torch.cuda.Stream()
        calls[i] = Call(ctypes.cast(g.lib.gdn2_linattn_fwd, ctypes.c_void_p).value,
                        *(p[x].data_ptr() for x in ("q", "k", "v", "log_a", "S0")), o.data_ptr(), S.data_ptr(), ws.data_ptr(),
                        stream.cuda_stream, ctypes.addressof(dims), 20000, 0)
        kept.append((p, want, o, S, ws, stream, dims))
    torch.cuda.synchronize()
    ctypes.CDLL(str(so)).run(calls, 4)
    torch.cuda.synchronize()
    for call, (_, want, o, S, *_) in zip(calls, kept):
        assert call.bad == 0
        assert torch.equal(o, want[0]) and torch.equal(S, want[1])


# lengths and heads: 160 units of 16 chunks each, uncut; one sequence cut into many pieces; chunks of one token
STILL = [((2048,) * 8, 20), ((20000,), 1), ((1,) * 3, 4), ((300, 0, 129), 2)]


@pytest.mark.parametrize("lens,H", STILL, ids=["uncut", "cut", "one", "ragged"])
@pytest.mark.parametrize("zero", ["k", "v"])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 32)])
def test_a_state_that_nothing_is_written_to(g, dtype, d, zero, lens, H):
    """Without a decay it stays bit for bit, however many tokens pass; so does its gradient."""
    p, _ = ref.problem(lens, H, H, d, d, dtype, "none", True, seed=60)
    q, k, v, la, dO = (p[x] for x in ("q", "k", "v", "log_a", "dO"))
    o, S = g.linattn_fwd(q, torch.zeros_like(k) if zero == "k" else k, torch.zeros_like(v) if zero == "v" else v, la,
                         p["S0"], p["cu"])
    assert torch.equal(S, p["S0"])
    # dLoss/dS gains q_t dO_t^T with every token
    got = g.linattn_bwd(torch.zeros_like(q) if zero == "k" else q, k, v, la, torch.zeros_like(dO) if zero == "v" else dO,
                        p["S0"], p["dS_T"], p["cu"])
    assert torch.equal(got["dS0"], p["dS_T"])


@pytest.mark.parametrize("lens,H", STILL, ids=["uncut", "cut", "one", "ragged"])
@pytest.mark.parametrize("la", [-1e-9, -1e-4, -0.003, -0.3])
def test_a_state_that_only_decays(g, la, lens, H):
    """log_a is summed in steps of 2^-32 in log2 (half a step a token, and two fp32 roundings of the product); a
    chunk's factor rounds the state once and is off by less than that itself; a piece's takes three roundings
    and an exponential of 2 ulp (at most 40 pieces of 512 tokens)."""
    p, cu = ref.problem(lens, H, H, 128, 128, BF, "none", True, seed=61)
    decay = torch.full((H,), la, device="cuda")
    _, S = g.linattn_fwd(p["q"], torch.zeros_like(p["k"]), p["v"], decay, p["S0"], p["cu"])
    got = g.linattn_bwd(torch.zeros_like(p["q"]), p["k"], p["v"], decay, p["dO"], p["S0"], p["dS_T"], p["cu"])
    for n, length in enumerate(lens):
        total = length * decay.double()[:, None, None]
        roundings = 2 * (length // 128 + 1) + (8 * 40 if len(lens) == 1 else 0) + 2 * float(total.abs().max())
        bound = length * 2.0 ** -33 + roundings * ref.FP32
        for x, start in ((S, p["S0"]), (got["dS0"], p["dS_T"])):
            want = torch.exp(total) * start[n].double()
            off = (x[n].double() - want).abs() - bound * want.abs()
            assert (off <= 2.0 ** -120).all(), (n, float((off / want.abs()).max()), bound)  # below: fp32's last bits


def _norms(got, want):
    """|got - want| / |want| over everything, both float64."""
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape and torch.isfinite(got).all()
    return float((got - want).norm() / want.norm())


def test_states_near_the_end_of_the_range(g):
    """Values of 2^110 written under decays on both sides of 2^-32 a chunk: nothing in between is larger."""
    p, cu = ref.problem((1000, 40), 3, 3, 128, 128, BF, "none", False, seed=62)
    decay = torch.tensor([-0.01, -0.05, -0.3], device="cuda")
    p["log_a"] = decay
    k, v = p["k"] * 2.0 ** 56, p["v"] * 2.0 ** 54
    o, S = g.linattn_fwd(p["q"], k, v, decay, None, p["cu"])
    want = ref.forward(dict(p, k=k, v=v), cu, 3, 3, True)
    assert torch.isfinite(o).all() and _norms(S, want["S_T"][0]) < 1.2e-6


# lengths, H, H_qk, decay: few tokens and many, one launch and three, pieces
DENSE = [((500, 129, 1), 2, 1, "token"), ((2048,), 160, 160, "none"), ((2048,), 160, 80, "token"), ((6000,), 1, 1, "none"),
         ((300, 40), 2, 2, "reset"), ((385, 64), 2, 2, "strong"), ((700,), 2, 1, "head")]


def _problem(lens, H, Hqk, decay, dtype, d, seed):
    p, cu = ref.problem(lens, H, Hqk, d, d, dtype, decay, True, seed=seed)
    keep = min(H, 2 * (H // Hqk))  # heads that are checked: the first groups'
    one = dict(p)
    for x in ("q", "k"):
        one[x] = p[x][:, :keep * Hqk // H].contiguous()
    for x in ("v", "dO"):
        one[x] = p[x][:, :keep].contiguous()
    one["log_a"] = p["log_a"][:keep] if p["log_a"].dim() == 1 else p["log_a"][:, :keep].contiguous()
    for x in ("S0", "dS_T"):
        one[x] = p[x][:, :keep].contiguous()
    return p, cu, one, keep


@pytest.mark.parametrize("case", DENSE, ids=lambda c: f"{'-'.join(map(str, c[0]))}_h{c[1]}.{c[2]}_{c[3]}")
def test_states_in_the_norm(g, case):
    """S_T and dS0 of the tensor-core runs.  A weighted row of y keeps 26 bits.  A chunk's sum takes 32 products, each
    cut off in the last bit at most: on average less than half a step (2^-24 / 1.4 of the value), of partial sums that
    come to two thirds of the whole: 0.95e-6, and the state itself is rounded once a chunk (2^-24 / sqrt(3) each, at
    random).  1.2e-6; rows kept to 17 bits (2^-17 / sqrt(3) / 1.4) would be off by 3e-6."""
    lens, H, Hqk, decay = case
    p, cu, one, keep = _problem(lens, H, Hqk, decay, BF, 128, 70)
    _, S = g.linattn_fwd(p["q"], p["k"], p["v"], p["log_a"], p["S0"], p["cu"])
    got = g.linattn_bwd(p["q"], p["k"], p["v"], p["log_a"], p["dO"], p["S0"], p["dS_T"], p["cu"])
    heads = keep * Hqk // H
    want = ref.forward(one, cu, keep, heads, True)["S_T"][0]
    assert _norms(S[:, :keep], want) < 1.2e-6
    want = torch.zeros_like(want)
    for n, h, _, u in ref.units(one, cu, keep, heads):
        want[n, h] = ref.run(u["k"], u["q"], u["dO"], u["la"], u["dS_T"], back=True)["fin"]
    assert _norms(got["dS0"][:, :keep], want) < 1.2e-6


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 24)])
def test_cut_sequences_among_many_short_ones(g, dtype, d):
    """More sequences than the plan counts at once; the two long ones are cut, and only they."""
    lens = (2,) * 700 + (3000,) + (1, 0, 3) * 300 + (2500,) + (5,)
    p, cu = ref.problem(lens, 1, 1, d, d, dtype, "token", True, seed=80)
    _check_units(g, p, cu, 1, 1, dtype == BF, [(0, 0), (700, 0), (701, 0), (1601, 0), (1602, 0)])


@pytest.mark.parametrize("dtype,d,H", [(BF, 128, 2), (BF, 128, 160), (F32, 24, 2)])
def test_no_gradient_through_a_reset(g, dtype, d, H):
    """a_t <S_{t-1}, dLoss/dS_t> is 0 where a_t is."""
    p, cu = ref.problem((700, 90), H, H, d, d, dtype, "reset", True, seed=72)
    got = g.linattn_bwd(p["q"], p["k"], p["v"], p["log_a"], p["dO"], p["S0"], p["dS_T"], p["cu"])
    reset = p["log_a"].float() < -104.0
    assert reset.any() and (got["dlog_a"][reset] == 0).all()
    assert (got["dlog_a"][~reset] != 0).any()


@pytest.mark.parametrize("dtype,d,lens,H", [(BF, 128, (300, 200), 2), (BF, 128, (5000,), 1), (F32, 24, (300, 200), 2),
                                            (BF, 128, (200, 300), 160)])
def test_a_nan_decay_shows(g, dtype, d, lens, H):
    """As in the single-token call: the state behind it is NaN, and so is every gradient that passed it."""
    p, cu = ref.problem(lens, H, H, d, d, dtype, "token", True, seed=73)
    at = 150
    p["log_a"][at, 0] = float("nan")
    o, S = g.linattn_fwd(p["q"], p["k"], p["v"], p["log_a"], p["S0"], p["cu"])
    clean = torch.ones(len(lens), H, dtype=torch.bool, device="cuda")
    clean[0, 0] = False
    assert torch.isnan(S[0, 0]).all() and torch.isfinite(S[clean]).all()
    assert torch.isnan(o[at:cu[1], 0]).all() and torch.isfinite(o[:, 1:]).all() and torch.isfinite(o[cu[1]:]).all()
    assert torch.isfinite(o[:at, 0]).all()
    got = g.linattn_bwd(p["q"], p["k"], p["v"], p["log_a"], p["dO"], p["S0"], p["dS_T"], p["cu"])
    assert torch.isnan(got["dS0"][0, 0]).all() and torch.isfinite(got["dS0"][clean]).all()
    assert torch.isnan(got["dq"][at:cu[1], 0]).all() and torch.isnan(got["dv"][:at, 0]).all()
    assert torch.isfinite(got["dq"][:at, 0]).all() and torch.isfinite(got["dv"][at:, 0]).all()
    assert torch.isnan(got["dlog_a"][at, 0]) and torch.isfinite(got["dlog_a"][:, 1:]).all()
    step = p["log_a"][at:at + 1].contiguous()
    S1 = p["S0"][:1].clone()
    o1 = g.linattn_step(*(p[x][at:at + 1].contiguous() for x in "qkv"), step, S1)
    assert torch.isnan(S1[0, 0]).all() and torch.isnan(o1[0, 0]).all() and torch.isfinite(S1[0, 1:]).all()


# a decay per token only: a fixed one has no gradient
DLOG = [((1, 0, 127, 300, 128, 129), 4, 2, "token"), ((385, 64), 2, 2, "strong"), ((400, 31), 2, 2, "reset"),
        ((512,), 1, 1, "none"), ((1700, 90), 1, 1, "token"), ((2048,), 160, 160, "token"), ((2048,), 160, 80, "none"),
        ((900,), 80, 80, "reset")]


@pytest.mark.parametrize("dtype,d,limit", [
    # bf16: the weights, the state's copy and the result are rounded to 2^-8, 0.17% of the value in the root mean
    # square each; dlog_a is a sum of differences of two such dots, over 256 tokens at most
    (BF, 128, 1e-2),
    # fp32: some 2000 roundings of 2^-24, even if they all went one way
    (F32, 40, 1.2e-4)])
@pytest.mark.parametrize("case", DLOG, ids=lambda c: f"{'-'.join(map(str, c[0]))}_h{c[1]}.{c[2]}_{c[3]}")
def test_gradients_in_the_norm(g, case, dtype, d, limit):
    """Every gradient, log_a's above all: a bound from absolute values is larger than it is."""
    lens, H, Hqk, decay = case
    p, cu, one, keep = _problem(lens, H, Hqk, decay, dtype, d, 71)
    got = g.linattn_bwd(p["q"], p["k"], p["v"], p["log_a"], p["dO"], p["S0"], p["dS_T"], p["cu"])
    assert g.check_status(got["workspace"]) == g.OK
    heads = keep * Hqk // H
    want = ref.gradients(one, cu, keep, heads, dtype == BF)
    for name in ("dlog_a", "dq", "dk", "dv"):
        n = heads if name in ("dq", "dk") else keep
        assert _norms(got[name][:, :n], want[name][0]) < limit, name


def test_steps_do_not_drift(g):
    """A fixed decay over 1000 single tokens with nothing written.  The step's factor is off by 2^-28 at most (0.4e-5
    over all of them); a single float's error adds up, and these decays are some whose float is off by more than
    2^-25.5 (2.1e-5).  The states' own roundings are at random and leave the mean of 16384 of them alone."""
    la = -torch.exp2(torch.linspace(-14, -6, 4000, dtype=torch.float64)).float()
    a = torch.exp(la.double())
    worst = la[((a.float().double() - a).abs() / a) > 2.0 ** -25.5][:4]
    assert worst.numel() == 4
    H = 4
    S = torch.randn(1, H, 128, 128, device="cuda").abs() + 0.5
    want = torch.exp(1000 * worst.double()).cuda()[None, :, None, None] * S.double()
    q, v = torch.zeros(1, H, 128, device="cuda"), torch.randn(1, H, 128, device="cuda")
    for _ in range(1000):
        g.linattn_step(q, q, v, worst.cuda(), S)
    drift = ((S.double() - want) / want).mean((0, 2, 3)).abs()
    assert (drift < 1000 * 2.0 ** -28 + 4 * 2.0 ** -24 * (1000 / 16384) ** 0.5).all(), drift


def test_the_stream_is_the_current_one(g, monkeypatch):
    """With torch's quick query and without it."""
    dev = torch.device("cuda", torch.cuda.current_device())
    side = torch.cuda.Stream()
    for quick in (True, False):
        if not quick:
            monkeypatch.setattr(g, "_raw_stream", None)
        assert g._stream(dev) == torch.cuda.current_stream().cuda_stream
        with torch.cuda.stream(side):
            assert g._stream(dev) == side.cuda_stream
            assert g._stream(torch.device("cuda")) == side.cuda_stream


@pytest.mark.parametrize("dtype,d,tile", [(BF, 128, 128), (F32, 24, 32)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_how_far_a_nan_reaches(g, dtype, d, tile, bad):
    """One bad value: tokens in front of its tile (behind it, for what is summed backward) keep every bit, and so do
    the other head and the other sequence."""
    p, cu = ref.problem((400, 300), 2, 2, d, d, dtype, "token", False, seed=81)
    names = ("q", "k", "v", "log_a", "dO")
    clean_o, clean_S = g.linattn_fwd(*(p[x] for x in names[:4]), None, p["cu"])
    clean = g.linattn_bwd(*(p[x] for x in names), None, None, p["cu"])
    at = 300
    first, behind = at // tile * tile, (at // tile + 1) * tile
    p["v"][at, 0, d // 2] = bad
    o, S = g.linattn_fwd(*(p[x] for x in names[:4]), None, p["cu"])
    far = torch.ones(700, 2, dtype=torch.bool, device="cuda")
    far[first:400, 0] = False
    assert torch.equal(o[far], clean_o[far]) and not torch.isfinite(o[at, 0]).all()
    assert torch.equal(S[:, 1], clean_S[:, 1]) and torch.equal(S[1], clean_S[1])
    got = g.linattn_bwd(*(p[x] for x in names), None, None, p["cu"])
    assert torch.equal(got["dv"], clean["dv"])      # v is not in it
    assert torch.equal(got["dq"][far], clean["dq"][far])
    near = torch.zeros(700, 2, dtype=torch.bool, device="cuda")
    near[first:behind, 0] = True                    # dk is k's tile of v alone
    assert torch.equal(got["dk"][~near], clean["dk"][~near])
