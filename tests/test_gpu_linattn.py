"""Linear attention with a decay per head on the GPU against float64 (bounds: linattn_ref)."""
import pytest
import torch

import linattn_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
RAGGED = (1, 0, 127, 300, 128, 129)
# lengths, H, H_qk, d_k, d_v, type, decay, start
FWD = [
    ((1,), 2, 2, 128, 128, BF, "token", True),
    ((200,), 4, 4, 128, 128, BF, "token", False),
    (RAGGED, 4, 2, 128, 128, BF, "token", True),
    (RAGGED, 2, 1, 128, 128, BF, "head", True),
    ((385, 64), 2, 2, 128, 128, BF, "strong", True),
    ((400, 31), 2, 2, 128, 128, BF, "reset", True),
    ((512,), 1, 1, 128, 128, BF, "none", True),
    ((1700, 90), 1, 1, 128, 128, BF, "token", True),   # cut into pieces
    ((1, 0, 33, 200), 4, 2, 48, 80, F32, "token", True),
    ((600,), 2, 2, 16, 16, F32, "token", False),        # cut into pieces
    ((150, 2), 2, 2, 128, 128, F32, "reset", True),
    ((97,), 3, 1, 7, 13, F32, "head", True),
    ((140, 5), 2, 2, 64, 33, BF, "token", True),
    ((64,), 2, 1, 128, 1, BF, "strong", False),
    ((64,), 2, 1, 1, 128, F32, "none", True),
]


def _tc(dk, dv, dtype):
    return dk == 128 and dv == 128 and dtype == BF


def _ids(c):
    return f"{'-'.join(map(str, c[0]))}_h{c[1]}.{c[2]}_{c[3]}x{c[4]}_{str(c[5])[6:]}_{c[6]}"


@pytest.fixture(scope="module")
def g():
    assert torch.cuda.is_available(), "GPU test"
    from gated_delta_rule_159_b200 import gdn2
    return gdn2


@pytest.mark.parametrize("case", FWD, ids=_ids)
def test_forward(g, case):
    lens, H, Hqk, dk, dv, dtype, decay, start = case
    p, cu = ref.problem(lens, H, Hqk, dk, dv, dtype, decay, start, seed=1)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    o, S = g.linattn_fwd(p["q"], p["k"], p["v"], p["log_a"], p["S0"], p["cu"], workspace=ws)
    assert g.check_status(ws) == g.OK
    want = ref.forward(p, cu, H, Hqk, _tc(dk, dv, dtype))
    ref.check("o", o, *want["o"])
    ref.check("S_T", S, *want["S_T"])


@pytest.mark.parametrize("case", FWD, ids=_ids)
def test_backward(g, case):
    lens, H, Hqk, dk, dv, dtype, decay, start = case
    p, cu = ref.problem(lens, H, Hqk, dk, dv, dtype, decay, start, seed=2)
    got = g.linattn_bwd(p["q"], p["k"], p["v"], p["log_a"], p["dO"], p["S0"], p["dS_T"], p["cu"])
    assert g.check_status(got["workspace"]) == g.OK
    want = ref.gradients(p, cu, H, Hqk, _tc(dk, dv, dtype))
    for name, (value, bound) in want.items():
        if name == "dlog_a" and decay == "head":
            assert got["dlog_a"] is None
            continue
        ref.check(name, got[name], value, bound)


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 128, 128), (F32, 24, 40)])
def test_equal_lengths_match_packed(g, dtype, dk, dv):
    p, cu = ref.problem((150, 150, 150), 2, 2, dk, dv, dtype, "token", True, seed=3)
    four = lambda t: t.view(3, 150, *t.shape[1:])  # noqa: E731
    o, S = g.linattn_fwd(p["q"], p["k"], p["v"], p["log_a"], p["S0"], p["cu"])
    o4, S4 = g.linattn_fwd(four(p["q"]), four(p["k"]), four(p["v"]), four(p["log_a"]), p["S0"])
    assert torch.equal(o4.view_as(o), o) and torch.equal(S4, S)
    a = g.linattn_bwd(p["q"], p["k"], p["v"], p["log_a"], p["dO"], p["S0"], p["dS_T"], p["cu"])
    b = g.linattn_bwd(four(p["q"]), four(p["k"]), four(p["v"]), four(p["log_a"]), four(p["dO"]), p["S0"], p["dS_T"])
    for x in ("dq", "dk", "dv", "dlog_a", "dS0"):
        assert torch.equal(a[x].view_as(b[x]), b[x]), x


@pytest.mark.parametrize("dtype,dk,dv,Hqk", [(BF, 128, 128, 1), (BF, 128, 128, 2), (F32, 24, 40, 1)])
def test_rows_behind_the_last_sequence(g, dtype, dk, dv, Hqk):
    """NaN rows behind the last sequence reach nothing, and outputs there stay as they were."""
    p, cu = ref.problem((130, 61), 2, Hqk, dk, dv, dtype, "token", True, seed=4, tail=70)
    T = cu[-1]
    o = torch.full_like(p["v"], 7.0)
    o, S = g.linattn_fwd(p["q"], p["k"], p["v"], p["log_a"], p["S0"], p["cu"], o=o)
    cut = {k: (v[:T].contiguous() if k in ("q", "k", "v", "dO", "log_a") else v) for k, v in p.items()}
    o2, S2 = g.linattn_fwd(cut["q"], cut["k"], cut["v"], cut["log_a"], p["S0"], p["cu"])
    assert torch.equal(o[:T], o2) and (o[T:] == 7.0).all() and torch.equal(S, S2)
    a = g.linattn_bwd(p["q"], p["k"], p["v"], p["log_a"], p["dO"], p["S0"], p["dS_T"], p["cu"])
    b = g.linattn_bwd(cut["q"], cut["k"], cut["v"], cut["log_a"], cut["dO"], p["S0"], p["dS_T"], p["cu"])
    for x in ("dq", "dk", "dv", "dlog_a"):
        assert torch.equal(a[x][:T], b[x]), x
    assert torch.equal(a["dS0"], b["dS0"])


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 32)])
def test_sequences_do_not_mix(g, dtype, d):
    """A NaN in one sequence stays in it, in the forward and in every gradient."""
    p, cu = ref.problem((100, 140, 90), 2, 2, d, d, dtype, "token", False, seed=5)
    clean = g.linattn_bwd(p["q"], p["k"], p["v"], p["log_a"], p["dO"], None, None, p["cu"])
    o, S = g.linattn_fwd(p["q"], p["k"], p["v"], p["log_a"], None, p["cu"])
    for x in ("q", "k", "v", "dO"):
        p[x][cu[1]:cu[2]] = float("nan")
    bad = g.linattn_bwd(p["q"], p["k"], p["v"], p["log_a"], p["dO"], None, None, p["cu"])
    o2, S2 = g.linattn_fwd(p["q"], p["k"], p["v"], p["log_a"], None, p["cu"])
    for s in (slice(0, cu[1]), slice(cu[2], cu[3])):
        assert torch.equal(o[s], o2[s])
        for x in ("dq", "dk", "dv", "dlog_a"):
            assert torch.equal(clean[x][s], bad[x][s]), x
    assert torch.equal(S[::2], S2[::2]) and torch.equal(clean["dS0"][::2], bad["dS0"][::2])


STEP = [(1, 1, 1, 128, 128, BF, "token"), (5, 4, 2, 128, 128, BF, "head"), (3, 4, 4, 64, 96, F32, "head"),
        (2, 3, 1, 7, 13, F32, "token"), (7, 2, 2, 100, 1, BF, "token"), (2, 2, 2, 1, 128, F32, "token")]


@pytest.mark.parametrize("case", STEP, ids=lambda c: "_".join(map(str, c)))
@pytest.mark.parametrize("pool", [False, True])
def test_step(g, case, pool):
    N, H, Hqk, dk, dv, dtype, decay = case
    p, _ = ref.problem((N,), H, Hqk, dk, dv, dtype, decay, False, seed=6)
    gen = torch.Generator(device="cuda").manual_seed(7)
    P = N + 3 if pool else N
    S = torch.randn(P, H, dk, dv, generator=gen, device="cuda")
    idx = torch.randperm(P, generator=gen, device="cuda")[:N].to(torch.int32) if pool else None
    if pool and N > 1:
        idx[0] = P if N % 2 else -1  # a padding row
    before = S.double()
    o = g.linattn_step(p["q"], p["k"], p["v"], p["log_a"], S, idx)
    rows = torch.arange(N, device="cuda") if idx is None else idx.long()
    live = (rows >= 0) & (rows < P)
    share = H // Hqk
    q, k = (p[x].double().repeat_interleave(share, 1) for x in "qk")
    la = p["log_a"].double()
    a = torch.exp(la).expand(N, H)[..., None, None]
    at = rows.clamp(0, P - 1)
    kv = k[..., None] * p["v"].double()[..., None, :]
    new = a * before[at] + kv
    size = a * before[at].abs() + kv.abs()
    want = torch.where(live[:, None, None], (q[..., None] * new).sum(-2), 0.0)
    # 2 roundings and a 2-ulp exponential in the state, dk sums in o
    bound = torch.where(live[:, None, None], (dk + 16) * ref.FP32 * (q.abs()[..., None] * size).sum(-2), 0.0)
    ref.check("o", o, want.cpu(), bound.cpu())
    touched = at[live]
    ref.check("S", S[touched], new[live].cpu(), (8 * ref.FP32 * size[live]).cpu())
    rest = torch.ones(P, dtype=torch.bool, device="cuda")
    rest[touched] = False
    assert torch.equal(S[rest].double(), before[rest])


def test_step_in_bf16_output_and_reset(g):
    p, _ = ref.problem((4,), 2, 2, 128, 128, BF, "token", False, seed=8)
    S = torch.randn(4, 2, 128, 128, device="cuda")
    S2 = S.clone()
    o = g.linattn_step(p["q"], p["k"], p["v"], p["log_a"], S)
    ob = g.linattn_step(p["q"], p["k"], p["v"], p["log_a"], S2, out_dtype=BF)
    assert torch.equal(ob, o.to(BF)) and torch.equal(S, S2)
    p["log_a"].fill_(-float("inf"))
    g.linattn_step(p["q"], p["k"], p["v"], p["log_a"], S)
    assert torch.equal(S, p["k"].float()[..., None] * p["v"].float()[..., None, :])


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 40)])
def test_prompt_then_tokens(g, dtype, d):
    """A prompt and single-token steps behind it agree with one longer prompt."""
    p, cu = ref.problem((170,), 4, 2, d, d, dtype, "token", True, seed=9)
    want = ref.forward(p, cu, 4, 2, _tc(d, d, dtype))
    part = {x: p[x][:160].contiguous() for x in ("q", "k", "v", "log_a")}
    _, S = g.linattn_fwd(part["q"], part["k"], part["v"], part["log_a"], p["S0"])
    for t in range(160, 170):
        o = g.linattn_step(*(p[x][t:t + 1].contiguous() for x in ("q", "k", "v", "log_a")), S)
        ref.check("o", o[0], want["o"][0][t], want["o"][1][t] + 1e-5)
    ref.check("S_T", S, want["S_T"][0], 2 * want["S_T"][1])


@pytest.mark.parametrize("dtype,d", [(F32, 12)])
def test_gradients_against_differences(g, dtype, d):
    """Central differences of the forward call itself, along random directions."""
    p, cu = ref.problem((37, 20), 2, 1, d, d, dtype, "token", True, seed=10)
    gen = torch.Generator(device="cuda").manual_seed(11)
    grads = g.linattn_bwd(p["q"], p["k"], p["v"], p["log_a"], p["dO"], p["S0"], p["dS_T"], p["cu"])

    def loss(x):
        o, S = g.linattn_fwd(x["q"], x["k"], x["v"], x["log_a"], x["S0"], p["cu"])
        return float((o.double() * p["dO"].double()).sum() + (S.double() * p["dS_T"].double()).sum())

    h = 2.0 ** -8
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("log_a", "dlog_a"), ("S0", "dS0")):
        v = torch.randn(p[name].shape, generator=gen, device="cuda")
        up, down = (loss(dict(p, **{name: p[name] + s * h * v})) for s in (1, -1))
        want = float((grads[grad].double() * v.double()).sum())
        # the loss is linear in q, k, v and S0 (differences exact); the third derivative in log_a adds
        # h^2/6 of the loss's terms; fp32 sums of ~3000 terms of size ~1 round by 1e-5, over 2 h
        assert abs((up - down) / (2 * h) - want) <= 2e-2 + 1e-3 * abs(want), name


@pytest.mark.parametrize("lens", [(300,), (2100,)])
def test_graph_replay_and_streams(g, lens):
    """Captured calls replay on new data; two streams with their own workspaces run side by side."""
    p, cu = ref.problem(lens, 1, 1, 128, 128, BF, "token", True, seed=12)
    args = [p[x] for x in ("q", "k", "v", "log_a")]
    o = torch.empty_like(p["v"])
    S = torch.empty_like(p["S0"])
    g.linattn_fwd(*args, p["S0"], p["cu"], o=o, S_T=S)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            g.linattn_fwd(*args, p["S0"], p["cu"], o=o, S_T=S)
            grads = g.linattn_bwd(*args, p["dO"], p["S0"], p["dS_T"], p["cu"])
    torch.cuda.synchronize()
    p["v"].copy_(torch.randn_like(p["v"]))
    graph.replay()
    torch.cuda.synchronize()
    got = [o.clone(), S.clone()] + [grads[x].clone() for x in ("dq", "dk", "dv", "dlog_a", "dS0")]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            outs.append((g.linattn_fwd(*args, p["S0"], p["cu"]),
                         g.linattn_bwd(*args, p["dO"], p["S0"], p["dS_T"], p["cu"])))
    torch.cuda.synchronize()
    for (oo, SS), gr in outs:
        for a, b in zip(got, [oo, SS] + [gr[x] for x in ("dq", "dk", "dv", "dlog_a", "dS0")]):
            assert torch.equal(a, b)


def test_state_may_be_updated_in_place(g):
    p, cu = ref.problem((1300, 7), 1, 1, 128, 128, BF, "token", True, seed=13)
    args = [p[x] for x in ("q", "k", "v", "log_a")]
    o, S = g.linattn_fwd(*args, p["S0"], p["cu"])
    mine = p["S0"].clone()
    o2, S2 = g.linattn_fwd(*args, mine, p["cu"], S_T=mine)
    assert torch.equal(o, o2) and torch.equal(S, mine) and S2 is mine
    o3, none = g.linattn_fwd(*args, p["S0"], p["cu"], output_final_state=False)
    assert none is None and torch.equal(o, o3)


def test_empty_batch(g):
    S0 = torch.randn(2, 3, 128, 128, device="cuda")
    e = lambda *s: torch.empty(*s, dtype=BF, device="cuda")  # noqa: E731
    q, v, la = e(2, 0, 3, 128), e(2, 0, 3, 128), e(2, 0, 3)
    o, S = g.linattn_fwd(q, q, v, la, S0)
    assert o.numel() == 0 and torch.equal(S, S0)
    got = g.linattn_bwd(q, q, v, la, v, S0, S0)
    assert torch.equal(got["dS0"], S0)
