"""8-bit checkpoints on the GPU against the definition in float64, and their use in gradients."""
import math

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


def define(x):
    """Codes and scale bytes block by block with Python numbers (exact: powers of two, halves)."""
    rows = x.reshape(-1, x.shape[-1]).cpu().double().tolist()
    codes, scales = [], []
    for row in rows:
        c, s = [], []
        for b in range(0, len(row), 32):
            block = row[b:b + 32]
            if not all(math.isfinite(v) for v in block):
                c += [0] * len(block)
                s.append(255)
                continue
            top = max(abs(v) for v in block)
            e = -127
            while top > 127 * 2.0 ** e:
                e += 1
            lim = 63 if e >= 122 else 127
            c += [max(-lim, min(lim, round(v / 2.0 ** e))) for v in block]  # round() takes ties to even
            s.append(e + 127)
        codes.append(c)
        scales.append(s)
    return torch.tensor(codes, dtype=torch.int8), torch.tensor(scales, dtype=torch.uint8)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(1, 1), (3, 31), (2, 32), (5, 33), (4, 40), (7, 128), (2, 3, 100), (9, 256), (1, 8)])
def test_codes_and_values(g, dtype, shape):
    gen = torch.Generator().manual_seed(sum(shape))
    x = torch.randn(shape, generator=gen) * torch.exp(4 * torch.randn(shape[:-1], generator=gen))[..., None]
    x = x.to(dtype)
    flat = x.view(-1)
    ends = torch.tensor([0.0, -0.0, 127.0, 127.5, 126.5, 2.0 ** -126, 2.0 ** -130, 0.5, 1.5, 2.5])
    flat[:min(10, flat.numel())] = ends[:min(10, flat.numel())].to(dtype)
    codes, scales = g.ckpt8_save(x.cuda())
    want_c, want_s = define(x)
    assert codes.shape == x.shape and torch.equal(codes.cpu().view_as(want_c), want_c)
    assert torch.equal(scales.cpu().view_as(want_s), want_s)
    step = torch.ldexp(torch.ones(want_s.shape).double(), want_s.int() - 127).repeat_interleave(32, -1)[:, :shape[-1]]
    value = (want_c.double() * step).view(shape)
    assert (value - x.double()).abs().max() <= (x.double().abs().max() / 127)
    for out in (BF, F32):  # a code times a power of two is exact in both
        assert torch.equal(g.ckpt8_restore(codes, scales, out).cpu().double(), value)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [64, 50])
def test_ends_of_the_range(g, dtype, cols):
    big = torch.finfo(dtype).max
    x = torch.zeros(5, cols, dtype=dtype)
    x[0, 0], x[0, 33] = float("inf"), 1.0
    x[1, 5], x[1, 40] = float("nan"), -2.0
    x[2, 3], x[2, 4], x[2, 45] = big, -big, big / 3
    x[3, 1], x[3, 40] = 2.0 ** -133, -(2.0 ** -127)  # subnormals
    codes, scales = g.ckpt8_save(x.cuda())
    want_c, want_s = define(x)
    assert torch.equal(codes.cpu(), want_c) and torch.equal(scales.cpu(), want_s)
    y = g.ckpt8_restore(codes, scales, dtype).cpu()
    assert torch.isnan(y[0, :32]).all() and torch.isnan(y[1, :32]).all()
    assert y[0, 33] == 1.0 and y[1, 40] == -2.0 and torch.isfinite(y[2:]).all()
    assert (y[2, 3] / big - 1).abs() <= 1 / 63 and (y[4] == 0).all()


def test_large_and_empty(g):
    x = torch.randn(4097, 2048, device="cuda").to(BF)
    y = g.ckpt8_restore(*g.ckpt8_save(x))
    step = x.float().view(4097, 64, 32).abs().amax(-1, keepdim=True) / 127
    assert ((y.float() - x.float()).view(4097, 64, 32).abs() <= step).all()
    again = g.ckpt8_restore(*g.ckpt8_save(y))
    assert torch.equal(again, y)  # restored values keep their codes
    codes, scales = g.ckpt8_save(x[:0])
    assert codes.shape == (0, 2048) and g.ckpt8_restore(codes, scales).shape == (0, 2048)


@pytest.mark.parametrize("lens,H,Hqk,dk,dv,dtype,decay", [
    ((1, 0, 129, 200), 2, 1, 128, 128, BF, "token"), ((300,), 2, 2, 128, 128, BF, "head"),
    ((1500,), 1, 1, 128, 128, BF, "token"), ((70, 41), 4, 2, 48, 80, F32, "token"), ((90,), 2, 2, 33, 100, BF, "token")])
def test_gradients_from_checkpoints(g, lens, H, Hqk, dk, dv, dtype, decay):
    p, cu = ref.problem(lens, H, Hqk, dk, dv, dtype, decay, True, seed=20)
    kept = {x: g.ckpt8_save(p[x]) for x in "qkv"}
    got = g.linattn_bwd_ckpt8(kept["q"], kept["k"], kept["v"], p["log_a"], p["dO"], p["S0"], p["dS_T"], p["cu"])
    assert g.check_status(got["workspace"]) == g.OK
    for x in "qkv":
        p[x] = g.ckpt8_restore(*kept[x], torch.float32)
    want = ref.gradients(p, cu, H, Hqk, dk == dv == 128 and dtype == BF)
    for name, (value, bound) in want.items():
        if got[name] is not None:
            ref.check(name, got[name], value, bound)


def test_training_step_from_checkpoints(g):
    """Forward, checkpoints, gradients; the delta rule's own backward reads restored tensors too."""
    p, cu = ref.problem((260,), 2, 2, 128, 128, BF, "token", True, seed=21)
    args = [p[x] for x in ("q", "k", "v", "log_a")]
    g.linattn_fwd(*args, p["S0"], p["cu"])
    kept = [g.ckpt8_save(t) for t in args[:3]]
    back = [g.ckpt8_restore(*t) for t in kept]
    a = g.linattn_bwd_ckpt8(*kept, p["log_a"], p["dO"], p["S0"], p["dS_T"], p["cu"])
    b = g.linattn_bwd(*back, p["log_a"], p["dO"], p["S0"], p["dS_T"], p["cu"])
    for x in ("dq", "dk", "dv", "dlog_a", "dS0"):
        assert torch.equal(a[x], b[x]), x
    gates = torch.sigmoid(torch.randn(260, 2, device="cuda")).to(BF)
    q, k, v = (t.clone() for t in back)
    d = g.chunk_bwd(q, k, v, p["log_a"], gates, None, p["dO"], p["S0"], scalar_decay=True, scalar_gates=True,
                    tied_gates=True)
    assert g.check_status(d["workspace"]) == g.OK and all(torch.isfinite(d[x]).all() for x in ("dq", "dk", "dv"))
