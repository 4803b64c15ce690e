"""Refusals of the linear-attention and checkpoint calls, on the host, before any CUDA call; and the
float64 reference of the GPU tests against the recurrence."""
import ctypes

import pytest
import torch

import linattn_ref as ref

P = ctypes.c_void_p(1 << 20)   # aligned placeholders, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 4)
WS = ctypes.c_void_p(1 << 21)


@pytest.fixture(scope="module")
def g():
    from gated_delta_rule_159_b200 import build
    build.build()
    from gated_delta_rule_159_b200 import gdn2
    return gdn2


def _dims(g, **kw):
    base = dict(n_seqs=2, seq_len=100, n_heads=4, n_qk_heads=2, d_k=128, d_v=128, dtype_in=g.BF16, dtype_out=g.BF16,
                flags=0, reserved=0)
    base.update(kw)
    return g.LinattnDims(*(base[n] for n, _ in g.LinattnDims._fields_))


BAD_DIMS = [(dict(n_seqs=0), -1), (dict(seq_len=-1), -1), (dict(n_heads=3), -1), (dict(n_qk_heads=0), -1),
            (dict(d_k=0), -1), (dict(d_v=129), -2), (dict(d_k=256), -2), (dict(dtype_in=3), -1), (dict(flags=2), -1),
            (dict(reserved=1), -1), (dict(n_seqs=1 << 20, seq_len=1 << 12), -2), (dict(n_seqs=1 << 28, seq_len=1), -2)]


def _fwd(g, dims, cu=None, ws=WS, nbytes=1 << 40, **p):
    a = dict(q=P, k=P, v=P, log_a=P, S0=None, o=P, S_T=None)
    a.update(p)
    return g.lib.gdn2_linattn_fwd(a["q"], a["k"], a["v"], a["log_a"], a["S0"], cu, a["o"], a["S_T"], ctypes.byref(dims),
                                  ws, nbytes, None), g.lib.gdn2_last_error().decode()


def _bwd(g, dims, cu=None, ws=WS, nbytes=1 << 40, ckpt8=False, **p):
    names = ("q", "k", "v") if not ckpt8 else ("q", "qs", "k", "ks", "v", "vs")
    a = {n: P for n in names + ("log_a", "dO", "dq", "dk", "dv", "dlog_a")}
    a.update(S0=None, dS_T=None, dS0=None)
    a.update(p)
    fn = g.lib.gdn2_linattn_bwd_ckpt8 if ckpt8 else g.lib.gdn2_linattn_bwd
    return fn(*(a[n] for n in names), a["log_a"], a["S0"], cu, a["dO"], a["dS_T"], a["dq"], a["dk"], a["dv"], a["dlog_a"],
              a["dS0"], ctypes.byref(dims), ws, nbytes, None), g.lib.gdn2_last_error().decode()


def _step(g, dims, n_slots=4, **p):
    a = dict(q=P, k=P, v=P, log_a=P, S=P, idx=None, o=P)
    a.update(p)
    return g.lib.gdn2_linattn_step(a["q"], a["k"], a["v"], a["log_a"], a["S"], n_slots, a["idx"], a["o"],
                                   ctypes.byref(dims), None), g.lib.gdn2_last_error().decode()


@pytest.mark.parametrize("bad,code", BAD_DIMS)
def test_bad_dims(g, bad, code):
    d = _dims(g, **bad)
    for rc, msg in (_fwd(g, d), _bwd(g, d), _bwd(g, d, ckpt8=True), _step(g, d)):
        assert rc == code and msg
    for size in (g.lib.gdn2_linattn_fwd_workspace_size, g.lib.gdn2_linattn_bwd_workspace_size,
                 g.lib.gdn2_linattn_bwd_ckpt8_workspace_size):
        assert size(ctypes.byref(d), 0) == 0
    assert _fwd(g, _dims(g, dtype_out=g.F32))[0] == g.ERR_UNSUPPORTED


@pytest.mark.parametrize("name", ["q", "k", "v", "log_a", "o"])
def test_forward_pointers(g, name):
    assert _fwd(g, _dims(g), **{name: None})[0] == g.ERR_INVALID_ARG
    assert _fwd(g, _dims(g), **{name: ctypes.c_void_p((1 << 20) + 1)})[0] == g.ERR_INVALID_ARG


def test_forward_states_and_workspace(g):
    d = _dims(g)
    assert _fwd(g, d, S0=ODD)[0] == g.ERR_INVALID_ARG and _fwd(g, d, S_T=ODD)[0] == g.ERR_INVALID_ARG
    assert _fwd(g, d, cu=ctypes.c_void_p((1 << 20) + 2))[0] == g.ERR_INVALID_ARG
    assert _fwd(g, d, ws=None)[0] == g.ERR_WORKSPACE
    assert _fwd(g, d, ws=ctypes.c_void_p((1 << 21) + 64))[0] == g.ERR_WORKSPACE
    assert _fwd(g, d, nbytes=255)[0] == g.ERR_WORKSPACE


@pytest.mark.parametrize("ckpt8", [False, True])
def test_backward_pointers(g, ckpt8):
    d = _dims(g)
    names = (("q", "k", "v") if not ckpt8 else ("q", "qs", "k", "ks", "v", "vs")) + (
        "log_a", "dO", "dq", "dk", "dv", "dlog_a")
    for name in names:
        assert _bwd(g, d, ckpt8=ckpt8, **{name: None})[0] == g.ERR_INVALID_ARG, name
    for name in ("S0", "dS_T", "dS0", "dO", "dq"):
        assert _bwd(g, d, ckpt8=ckpt8, **{name: ODD})[0] == g.ERR_INVALID_ARG, name
    rc, msg = _bwd(g, _dims(g, flags=g.LINATTN_HEAD_DECAY), ckpt8=ckpt8)
    assert rc == g.ERR_INVALID_ARG and "dlog_a" in msg
    assert _bwd(g, d, ckpt8=ckpt8, ws=None)[0] == g.ERR_WORKSPACE
    assert _bwd(g, d, ckpt8=ckpt8, nbytes=256)[0] == g.ERR_WORKSPACE


def test_step_refusals(g):
    d = _dims(g, seq_len=1)
    for name in ("q", "k", "v", "log_a", "S", "o"):
        assert _step(g, d, **{name: None})[0] == g.ERR_INVALID_ARG, name
    assert _step(g, d, S=ODD)[0] == g.ERR_INVALID_ARG
    assert _step(g, d, idx=P, n_slots=0)[0] == g.ERR_INVALID_ARG
    assert _step(g, _dims(g, seq_len=2))[0] == g.ERR_INVALID_ARG


def test_ckpt8_refusals(g):
    def call(x=P, codes=P, scales=P, rows=4, cols=64, dtype=0):
        return (g.lib.gdn2_ckpt8_save(x, codes, scales, rows, cols, dtype, None),
                g.lib.gdn2_ckpt8_restore(codes, scales, x, rows, cols, dtype, None))
    for bad in (dict(x=None), dict(codes=None), dict(scales=None), dict(x=ODD), dict(codes=ODD), dict(rows=-1),
                dict(cols=0), dict(dtype=2)):
        assert call(**bad) == (g.ERR_INVALID_ARG,) * 2, bad
    assert call(rows=1 << 40) == (g.ERR_UNSUPPORTED,) * 2
    assert call(x=None, codes=None, scales=None, rows=0) == (g.OK,) * 2


def test_outputs_apart_from_inputs(g):
    """An output at an input's address, or at another output's, is refused."""
    at = [ctypes.c_void_p((i + 1) << 20) for i in range(16)]
    ins = dict(zip(("q", "k", "v", "log_a", "dO", "S0", "dS_T"), at))
    outs = dict(zip(("dq", "dk", "dv", "dlog_a", "dS0"), at[8:]))
    ws = ctypes.c_void_p(1 << 30)
    d = _dims(g)
    for name in ("q", "k", "v", "log_a"):
        rc, msg = _fwd(g, d, ws=ws, q=at[0], k=at[1], v=at[2], log_a=at[3], o=ins[name])
        assert rc == g.ERR_INVALID_ARG and "address" in msg
        rc, msg = _step(g, _dims(g, seq_len=1), q=at[0], k=at[1], v=at[2], log_a=at[3], S=at[9], o=ins[name])
        assert rc == g.ERR_INVALID_ARG and "address" in msg
    for out in outs:
        for other in [n for n in {**ins, **outs} if n != out]:
            rc, msg = _bwd(g, d, ws=ws, **{**ins, **outs, out: {**ins, **outs}[other]})
            assert rc == g.ERR_INVALID_ARG and "address" in msg, (out, other)
    rc, msg = _bwd(g, d, ws=ws, ckpt8=True, qs=at[13], ks=at[14], vs=at[15], **{**ins, **outs, "dq": at[13]})
    assert rc == g.ERR_INVALID_ARG and "address" in msg
    for fn in (lambda a, b: g.lib.gdn2_ckpt8_save(at[0], a, b, 4, 64, g.BF16, None),
               lambda a, b: g.lib.gdn2_ckpt8_restore(a, b, at[0], 4, 64, g.BF16, None)):
        assert fn(at[0], at[1]) == g.ERR_INVALID_ARG and "address" in g.lib.gdn2_last_error().decode()
        assert fn(at[1], at[0]) == g.ERR_INVALID_ARG


def test_workspace_sizes(g):
    size = lambda d, packed=0: g.lib.gdn2_linattn_fwd_workspace_size(ctypes.byref(d), packed)  # noqa: E731
    assert size(_dims(g)) == 256                       # nothing to cut
    assert size(_dims(g, n_seqs=1, seq_len=65536)) > 256 + 4 * 65536 * 8  # pieces and their states
    assert size(_dims(g, n_seqs=3, seq_len=65536), 1) > size(_dims(g, n_seqs=3, seq_len=90), 1) == 256


def test_python_refusals(g):
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    q, v, la = t(10, 2, 128), t(10, 4, 128), t(10, 4)
    with pytest.raises(ValueError, match="CUDA"):
        g._ptr(q)
    with pytest.raises(ValueError):
        g.linattn_fwd(q, t(11, 2, 128), v, la)
    with pytest.raises(ValueError):
        g.linattn_fwd(q, q, t(9, 4, 128), la)
    with pytest.raises(ValueError):
        g.linattn_fwd(q, q, v, t(10, 3))
    with pytest.raises(TypeError):
        g.linattn_fwd(q, q, v, t(4))                   # a decay per head is fp32
    with pytest.raises(TypeError):
        g.linattn_fwd(q, q, v.float(), la)
    with pytest.raises(TypeError):
        g.linattn_fwd(q, q, v, la, None, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        g.linattn_fwd(q, q, v, la, t(1, 4, 64, 128, dtype=torch.float32))
    with pytest.raises(TypeError):
        g.linattn_fwd(q, q, v, la, t(1, 4, 128, 128))
    with pytest.raises(ValueError):
        g.linattn_bwd(q, q, v, la, t(10, 4, 64))
    with pytest.raises(ValueError):
        g.linattn_step(q, q, v, la, t(9, 4, 128, 128, dtype=torch.float32))
    with pytest.raises(TypeError):
        g.linattn_step(q, q, v, la, t(9, 4, 128, 128, dtype=torch.float32), torch.zeros(10, dtype=torch.int64))
    with pytest.raises(TypeError):
        g.ckpt8_save(t(4, 32, dtype=torch.float16))
    with pytest.raises(ValueError):
        g.ckpt8_restore(t(4, 33, dtype=torch.int8), t(4, 1, dtype=torch.uint8))


@pytest.mark.parametrize("back", [False, True])
def test_reference_is_the_recurrence(back):
    gen = torch.Generator().manual_seed(0)
    T, dy, dz = 300, 5, 7
    x, y, z = (torch.randn(T, d, generator=gen, dtype=torch.float64) for d in (dy, dy, dz))
    la = -torch.rand(T, generator=gen, dtype=torch.float64)
    la[17], la[200] = -torch.inf, 0.0
    S = start = torch.randn(dy, dz, generator=gen, dtype=torch.float64)
    r = ref.run(x, y, z, la, start, back)
    for t in reversed(range(T)) if back else range(T):
        if not back:
            S = torch.exp(la[t]) * S
        S = S + y[t][:, None] * z[t]
        torch.testing.assert_close(r["out"][t], x[t] @ S, rtol=1e-10, atol=1e-10)
        if back:
            S = torch.exp(la[t]) * S
    torch.testing.assert_close(r["fin"], S, rtol=1e-10, atol=1e-10)


@pytest.mark.parametrize("lens", [(5, 0, 9), (140,)])
def test_reference_gradients_are_autograd(lens):
    p, cu = ref.problem(lens, 2, 1, 4, 3, torch.float32, "token", True, seed=1, device="cpu")
    want = ref.gradients(p, cu, 2, 1, False)
    x = {n: p[n].double().requires_grad_() for n in ("q", "k", "v", "log_a", "S0")}
    loss = 0.0
    for n in range(len(lens)):
        S = x["S0"][n]
        for t in range(cu[n], cu[n + 1]):
            S = torch.exp(x["log_a"][t])[:, None, None] * S + x["k"][t][:, :, None] * x["v"][t][:, None, :]
            loss = loss + ((x["q"][t][:, :, None] * S).sum(1) * p["dO"][t].double()).sum()
        loss = loss + (S * p["dS_T"][n].double()).sum()
    loss.backward()
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("log_a", "dlog_a"), ("S0", "dS0")):
        torch.testing.assert_close(want[grad][0], x[name].grad, rtol=1e-9, atol=1e-9)
