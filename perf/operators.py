"""Cases that time the linear-attention and 8-bit-checkpoint operators.

Each case is one pass through an operator as a user's program calls it.  With ``own`` false
``run`` computes it with elementary torch operations in 32 bits; with ``own`` true it calls the
library's entry points.  ``exact`` gives the same outputs from the definition, token by token in
64 bits.

The operators:

* linear attention with a decay for each head, per token t and head h (state S of d_k x d_v):
  ``S_t = a_t S_{t-1} + k_t v_t^T``, ``o_t = S_t^T q_t``, with ``a_t = exp(log_a_t)``; q and k may
  have fewer heads than v.  The prompt form, the single-token step and the gradients;
* checkpoints in 8 bits: blocks of 32 values share a power-of-two scale 2^e, the smallest with
  ``max|x| <= 127 * 2^e``, and every value is kept as the integer nearest to x / 2^e;
* the gradients of linear attention read from such checkpoints of q, k and v.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
CHUNK = 64  # tokens of a chunk of the plain form


def listed():
    full = dict(hqk=16, h=16, dk=128, dv=128, dtype="bf16")
    return [
        # one short prompt of a chat turn: latency
        dict(name="fwd prompt 200", op="fwd", n=1, tokens=200, ragged=False, decay="token", start=False, **full),
        # the framework's prefill batch
        dict(name="fwd batch 8x4096", op="fwd", n=8, tokens=32768, ragged=False, decay="token", start=True, **full),
        # one long document, fixed decays per head (retention)
        dict(name="fwd long 65000", op="fwd", n=1, tokens=65000, ragged=False, decay="head", start=False, **full),
        # a packed batch of ragged prompts, q and k shared by two heads each
        dict(name="fwd packed shared", op="fwd", n=19, tokens=30011, ragged=True, decay="token", start=True,
             hqk=8, h=16, dk=128, dv=128, dtype="bf16"),
        # a few users' next token in fp32, narrower heads than usual
        dict(name="step 4 fp32", op="step", n=4, slots=0, h=16, hqk=16, dk=64, dv=96, dtype="fp32", decay="head"),
        # the framework's decode batch, states in a pool
        dict(name="step 256 pool", op="step", n=256, slots=300, decay="token", **full),
        # a training step's gradients on the framework's batch
        dict(name="bwd batch 8x4096", op="bwd", n=8, tokens=32768, ragged=False, decay="token", start=True, **full),
        # gradients of a small fp32 model, odd head sizes, packed
        dict(name="bwd fp32 small heads", op="bwd", n=3, tokens=1201, ragged=True, decay="token", start=True,
             hqk=2, h=4, dk=48, dv=80, dtype="fp32"),
        # a layer's saved activations of one training batch, saved and restored
        dict(name="ckpt8 32768x2048", op="ckpt8", rows=32768, cols=2048, dtype="bf16"),
        # a small fp32 tensor whose rows end inside a block
        dict(name="ckpt8 fp32 777x1000", op="ckpt8", rows=777, cols=1000, dtype="fp32"),
        # the training step's gradients again, from 8-bit q, k and v
        dict(name="bwd_ckpt8 8x4096", op="bwd_ckpt8", n=8, tokens=32768, ragged=False, decay="token", start=True, **full),
        # packed fine-tuning samples with fixed decays and shared q and k
        dict(name="bwd_ckpt8 packed", op="bwd_ckpt8", n=11, tokens=9001, ragged=True, decay="head", start=False,
             hqk=8, h=16, dk=128, dv=128, dtype="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "step", "bwd", "bwd", "ckpt8", "bwd_ckpt8"])
    if op == "ckpt8":
        cols = _log_uniform(rng, 8, 8192)
        return dict(op=op, rows=_log_uniform(rng, 1, max(1, 67108864 // cols)), cols=cols,
                    dtype=rng.choice(["bf16", "fp32"]))
    hqk = rng.choice([1, 2, 3, 4, 8, 16])
    h = hqk * rng.choice([1, 1, 2, 4])
    wide = rng.random() < 0.7
    if wide:
        heads = dict(hqk=hqk, h=h, dk=128, dv=128, dtype="bf16")
    else:
        heads = dict(hqk=hqk, h=h, dk=rng.randint(8, 128), dv=rng.randint(8, 128), dtype=rng.choice(["bf16", "fp32"]))
    decay = rng.choice(["token", "head"])
    if op == "step":
        n = _log_uniform(rng, 1, max(1, 4096 // h))
        return dict(op=op, n=n, slots=rng.choice([0, n, n + rng.randint(1, 50)]), decay=decay, **heads)
    tokens = _log_uniform(rng, 1, min(65536, (524288 if wide else 65536) // h))
    n = min(tokens, _log_uniform(rng, 1, 32))
    ragged = rng.random() < 0.5
    if not ragged:
        tokens = tokens // n * n
    return dict(op=op, n=n, tokens=tokens, ragged=ragged, decay=decay, start=rng.random() < 0.5, **heads)


def work(case):
    if case["op"] == "ckpt8":
        size = case["rows"] * case["cols"]
        es = 2 if case["dtype"] == "bf16" else 4
        blocks = case["rows"] * (-(-case["cols"] // 32))
        return {"bytes": size * (2 * es + 2) + 2 * blocks, "flops": 0}
    h, hqk, dk, dv, n = (case[x] for x in ("h", "hqk", "dk", "dv", "n"))
    es = 2 if case["dtype"] == "bf16" else 4
    state = 4 * n * h * dk * dv
    if case["op"] == "step":
        decay = 4 * h if case["decay"] == "head" else es * n * h
        return {"bytes": es * n * (2 * hqk * dk + h * dv) + 4 * n * h * dv + decay + 2 * state,
                "flops": 4 * n * h * dk * dv}
    t = case["tokens"]
    decay = 4 * h if case["decay"] == "head" else es * t * h
    qkv = es * t * (2 * hqk * dk + h * dv)
    start = state if case["start"] else 0
    if case["op"] == "fwd":
        return {"bytes": qkv + es * t * h * dv + decay + start + state, "flops": 4 * t * h * dk * dv}
    saved = qkv if case["op"] == "bwd" else t * (2 * hqk * (dk + -(-dk // 32)) + h * (dv + -(-dv // 32)))
    grads = qkv + (decay if case["decay"] == "token" else 0)
    return {"bytes": saved + es * t * h * dv + decay + grads + start + 2 * state, "flops": 10 * t * h * dk * dv}


# ---------------------------------------------------------------- inputs


def _cu(case, seed):
    """Token offsets of the packed sequences: random lengths, one of them 0 and one of them 1 where there are enough."""
    n, t = case["n"], case["tokens"]
    r = np.random.RandomState(seed % (1 << 31))
    cut = np.sort(r.randint(0, t + 1, n - 1)) if n > 1 else np.zeros(0, np.int64)
    lens = np.diff(np.concatenate([[0], cut, [t]]))
    if n >= 4:
        i, j, big = *r.choice(n, 2, replace=False), int(np.argmax(lens))
        for at, to in ((i, 0), (j, min(1, t))):
            if at != big and lens[big] + lens[at] >= to:
                lens[big] += lens[at] - to
                lens[at] = to
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def _unit(g, shape, dtype):
    x = torch.randn(shape, generator=g, device="cuda")
    return (x / x.norm(dim=-1, keepdim=True)).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "ckpt8":
        # activations: normal, with a scale for each channel and a few outliers
        x = torch.randn(case["rows"], case["cols"], generator=g, device="cuda")
        x = x * torch.exp(torch.randn(case["cols"], generator=g, device="cuda"))
        x = x * torch.where(torch.rand(x.shape, generator=g, device="cuda") < 1e-3, 20.0, 1.0)
        return dict(op="ckpt8", x=x.to(dtype))
    h, hqk, dk, dv, n = (case[x] for x in ("h", "hqk", "dk", "dv", "n"))
    step = case["op"] == "step"
    t = n if step else case["tokens"]
    lead = (t,) if step or case["ragged"] else (n, t // n)
    s = dict(op=case["op"], q=_unit(g, (*lead, hqk, dk), dtype), k=_unit(g, (*lead, hqk, dk), dtype),
             v=torch.randn(*lead, h, dv, generator=g, device="cuda").to(dtype))
    if case["decay"] == "head":  # slopes of a geometric series over the heads
        s["log_a"] = -torch.exp2(-8.0 * (torch.arange(h, device="cuda", dtype=torch.float32) + 1) / h)
    else:
        s["log_a"] = (-torch.nn.functional.softplus(torch.randn(*lead, h, generator=g, device="cuda")) * 0.05).to(dtype)
    if step:
        pool = case["slots"] or n
        s["S"] = torch.randn(pool, h, dk, dv, generator=g, device="cuda") * 0.1
        s["idx"] = (torch.randperm(pool, generator=g, device="cuda")[:n].to(torch.int32) if case["slots"] else None)
        return s
    s["S0"] = torch.randn(n, h, dk, dv, generator=g, device="cuda") * 0.1 if case["start"] else None
    s["cu"] = torch.from_numpy(_cu(case, seed)).cuda() if case["ragged"] else None
    if case["op"] != "fwd":
        s["dO"] = torch.randn(*lead, h, dv, generator=g, device="cuda").to(dtype)
        s["dS_T"] = torch.randn(n, h, dk, dv, generator=g, device="cuda") * 0.1
        if case["op"] == "bwd_ckpt8":
            for x in "qkv":
                s[x] = _save8(s[x])
    return s


# ---------------------------------------------------------------- plain forms


def _power(e):
    """2^e in fp32 from its bits, e in [-127, 127]; 2^-127 is a subnormal."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _save8(x):
    """(int8 codes like x, uint8 scales [..., blocks]): byte e + 127 for the scale 2^e."""
    cols = x.shape[-1]
    pad = -cols % 32
    f = torch.nn.functional.pad(x.float(), (0, pad)).unflatten(-1, (-1, 32))
    m, e = torch.frexp(f.abs().amax(-1))  # max = m 2^e with m in [1/2, 1); 127 = (127/128) 2^7
    e = torch.where(m > 127 / 128, e - 6, e - 7)
    e = torch.where(m == 0, -127, e.clamp(min=-127))
    codes = torch.round(f * _power(-e)[..., None]).to(torch.int8)
    return codes.flatten(-2)[..., :cols].contiguous(), (e + 127).to(torch.uint8)


def _restore8(codes, scales, dtype):
    e = scales.to(torch.int32) - 127
    step = _power(e).repeat_interleave(32, dim=-1)
    return (codes.float() * step[..., :codes.shape[-1]]).to(dtype)


def _pad_index(cu, n):
    """[n, L] places of the packed tokens in a padded layout (L whole chunks) and their mask."""
    lens = cu[1:].long() - cu[:-1].long()
    length = -(-int(lens.max()) // CHUNK) * CHUNK
    at = torch.arange(max(length, CHUNK), device=cu.device)
    mask = at[None] < lens[:, None]
    return torch.where(mask, cu[:-1].long()[:, None] + at[None], 0), mask


def _padded(s):
    """The inputs as fp32 [n, L, ...] with zeros behind each sequence, and how to put results back."""
    q, k, v = s["q"], s["k"], s["v"]
    h = v.shape[-2]
    la = s["log_a"]
    la = la.expand(*v.shape[:-2], h) if la.dim() == 1 else la
    if s["cu"] is not None:
        index, mask = _pad_index(s["cu"], s["cu"].numel() - 1)

        def spread(x):
            y = x.float()[index]
            return torch.where(mask.reshape(*mask.shape, *([1] * (y.dim() - 2))), y, 0.0)

        def back(y):
            return y[mask]
    else:
        pad = -v.shape[1] % CHUNK

        def spread(x):
            return torch.nn.functional.pad(x.float(), (0, 0) * (x.dim() - 2) + (0, pad))

        def back(y):
            return y[:, :v.shape[1]]

    share = h // q.shape[-2]
    return spread, back, spread(q).repeat_interleave(share, 2), spread(k).repeat_interleave(share, 2), spread(v), spread(la)


def _chunked(x, y, z, la, start):
    """o_t = sum_{j <= t} exp(L_t - L_j) (x_t . y_j) z_j + exp(L_t) start^T x_t over the chunks of [n, L, h, d], and the last state."""
    n, length, h, _ = x.shape
    x, y, z = (t.unflatten(1, (-1, CHUNK)).permute(0, 3, 1, 2, 4) for t in (x, y, z))  # [n, h, c, C, d]
    cum = la.unflatten(1, (-1, CHUNK)).permute(0, 3, 1, 2).cumsum(-1)  # [n, h, c, C]
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=x.device).tril()
    decay = torch.where(low, cum[..., :, None] - cum[..., None, :], -torch.inf).exp()
    out = ((x @ y.transpose(-1, -2)) * decay) @ z
    total = cum[..., -1]
    added = (y * (total[..., None] - cum).exp()[..., None]).transpose(-1, -2) @ z  # [n, h, c, dk, dv]
    first = torch.zeros_like(added[:, :, 0]) if start is None else start
    parts = torch.cat([first[:, :, None], added], 2)
    run_ = torch.nn.functional.pad(total.double().cumsum(-1), (1, 0))  # log decay from the start to each chunk's start
    between = torch.ones(run_.shape[-1], run_.shape[-1], dtype=torch.bool, device=x.device).tril()
    weight = torch.where(between, run_[..., :, None] - run_[..., None, :], -torch.inf).exp().float()
    states = (weight @ parts.flatten(-2)).unflatten(-1, parts.shape[-2:])
    out = out + (x * cum.exp()[..., None]) @ states[:, :, :-1]
    return out.permute(0, 2, 3, 1, 4).reshape(n, length, h, -1), states[:, :, -1]


def _chunked_back(x, y, z, la, start):
    """The same sum over j >= t with exp(L_j - L_t), from the last token back; the state before the first token."""
    later = torch.cat([la[:, 1:], torch.zeros_like(la[:, :1])], 1)
    out, first = _chunked(x.flip(1), y.flip(1), z.flip(1), later.flip(1), start)
    return out.flip(1), first * la[:, 0].exp()[..., None, None]


def _plain_fwd(s):
    _, back, q, k, v, la = _padded(s)
    o, last = _chunked(q, k, v, la, s["S0"])
    return back(o).to(s["v"].dtype), last


def _plain_bwd(s):
    dtype = s["dO"].dtype
    if isinstance(s["q"], tuple):
        s = dict(s, **{x: _restore8(*s[x], dtype) for x in "qkv"})
    spread, back, q, k, v, la = _padded(s)
    do = spread(s["dO"])
    flip = lambda t: None if t is None else t.transpose(-1, -2)  # noqa: E731
    dq, last = _chunked(do, v, k, la, flip(s["S0"]))
    dv, first = _chunked_back(k, q, do, la, s["dS_T"])
    dk, _ = _chunked_back(v, do, q, la, flip(s["dS_T"]))
    share = v.shape[2] // s["q"].shape[-2]
    sum_heads = lambda t: t.unflatten(2, (-1, share)).sum(3)  # noqa: E731
    got = dict(dq=back(sum_heads(dq)).to(dtype), dk=back(sum_heads(dk)).to(dtype), dv=back(dv).to(dtype), dS0=first)
    if s["log_a"].dim() > 1:
        # every pair (i, j) with j < t <= i holds a_t once: sums over i >= t of q.dq less those of k.dk
        flow = (q.double() * dq.double()).sum(-1) - (k.double() * dk.double()).sum(-1)
        end = (last.transpose(-1, -2).double() * s["dS_T"].double()).sum((-1, -2))
        got["dlog_a"] = back((flow.flip(1).cumsum(1).flip(1) + end[:, None])).to(dtype)
    return got


def _plain_step(s):
    at = slice(None) if s["idx"] is None else s["idx"].long()
    share = s["v"].shape[1] // s["q"].shape[1]
    q, k = (s[x].float().repeat_interleave(share, 1) for x in "qk")
    a = s["log_a"].float().exp().expand(q.shape[:2])
    new = a[..., None, None] * s["S"][at] + k[..., None] * s["v"].float()[..., None, :]
    s["S"][at] = new
    return (q[..., None] * new).sum(-2), s["S"]


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "ckpt8":
        codes, scales = _save8(s["x"])
        return _restore8(codes, scales, s["x"].dtype), scales
    return {"fwd": _plain_fwd, "step": _plain_step, "bwd": _plain_bwd, "bwd_ckpt8": _plain_bwd}[s["op"]](s)


def _run_own(s):
    from gated_delta_rule_159_b200 import gdn2
    if s["op"] == "ckpt8":
        codes, scales = gdn2.ckpt8_save(s["x"])
        return gdn2.ckpt8_restore(codes, scales, s["x"].dtype), scales
    if s["op"] == "step":
        return gdn2.linattn_step(s["q"], s["k"], s["v"], s["log_a"], s["S"], s["idx"]), s["S"]
    if s["op"] == "fwd":
        return gdn2.linattn_fwd(s["q"], s["k"], s["v"], s["log_a"], s["S0"], s["cu"])
    call = gdn2.linattn_bwd if s["op"] == "bwd" else gdn2.linattn_bwd_ckpt8
    g = call(s["q"], s["k"], s["v"], s["log_a"], s["dO"], s["S0"], s["dS_T"], s["cu"])
    names = ("dq", "dk", "dv", "dS0") + (("dlog_a",) if s["log_a"].dim() > 1 else ())
    return {x: g[x] for x in names}


# ---------------------------------------------------------------- the definition, token by token in 64 bits


def _exact8(x):
    """The restored values and the scale bytes, block by block from logarithms."""
    x = x.double()
    cols = x.shape[-1]
    blocks = torch.cat([x, x.new_zeros(*x.shape[:-1], -cols % 32)], -1).reshape(*x.shape[:-1], -1, 32)
    top = blocks.abs().max(-1).values
    e = torch.ceil(torch.log2(top / 127).clamp(min=-127.0)).long()
    powers = torch.tensor([2.0 ** i for i in range(-128, 129)], dtype=torch.float64, device=x.device)
    e = torch.where(top > 127 * powers[e + 128], e + 1, e)
    e = torch.where((top <= 127 * powers[e + 127]) & (e > -127), e - 1, e)
    step = powers[e + 128][..., None]
    near = torch.floor(blocks / step)
    rest = blocks / step - near
    near = near + ((rest > 0.5) | ((rest == 0.5) & (near % 2 == 1)))
    return (near * step).reshape(*x.shape[:-1], -1)[..., :cols], (e + 127).to(torch.uint8)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "ckpt8":
        return _exact8(s["x"])
    if s["op"] == "bwd_ckpt8":
        powers = torch.tensor([2.0 ** (i - 127) for i in range(255)], dtype=torch.float64, device="cuda")
        s = dict(s, **{x: s[x][0].double() * powers[s[x][1].long()].repeat_interleave(32, -1)[..., :s[x][0].shape[-1]]
                       for x in "qkv"})
    share = case["h"] // case["hqk"]
    dt = torch.float64
    if s["op"] == "step":
        q, k = (s[x].to(dt).repeat_interleave(share, 1) for x in "qk")
        S = s["S"].to(dt)
        rows = torch.arange(case["n"], device="cuda") if s["idx"] is None else s["idx"].long()
        new = torch.exp(s["log_a"].to(dt)).expand(q.shape[:2])[..., None, None] * S[rows]
        new = new + torch.einsum("nhk,nhv->nhkv", k, s["v"].to(dt))
        S[rows] = new
        return torch.einsum("nhk,nhkv->nhv", q, new), S
    n, h, dk, dv = (case[x] for x in ("n", "h", "dk", "dv"))
    packed = s["cu"] is not None
    cu = s["cu"].tolist() if packed else [i * (case["tokens"] // n) for i in range(n + 1)]
    flat = lambda x: x.reshape(-1, *x.shape[-2:]).to(dt)  # noqa: E731
    q, k = (flat(s[x]).repeat_interleave(share, 1) for x in "qk")
    v = flat(s["v"])
    la = s["log_a"].to(dt)
    a = torch.exp(la.expand(v.shape[0], h) if la.dim() == 1 else la.reshape(-1, h))
    lens = [cu[i + 1] - cu[i] for i in range(n)]
    order = sorted(range(n), key=lambda i: -lens[i])  # longest first: the live sequences are the first ones
    first = torch.tensor([cu[i] for i in order], device="cuda")
    live = [sum(x > t for x in lens) for t in range(max(lens))]
    S = torch.zeros(n, h, dk, dv, dtype=dt, device="cuda") if s["S0"] is None else s["S0"].to(dt)[order]
    fwd = s["op"] == "fwd"
    do = None if fwd else flat(s["dO"])
    one = torch.zeros(v.shape[0], h, dv if fwd else dk, dtype=dt, device="cuda")
    for t, m in enumerate(live):
        at = first[:m] + t
        S[:m] = a[at][..., None, None] * S[:m] + k[at][..., None] * v[at][..., None, :]
        one[at] = torch.matmul(q[at][..., None, :], S[:m])[..., 0, :] if fwd else torch.matmul(S[:m], do[at][..., None])[..., 0]
    inverse = torch.tensor(order, device="cuda").argsort()
    shape = lambda x, like: x.reshape(*like.shape[:-1], x.shape[-1])  # noqa: E731
    if fwd:
        return shape(one, s["v"]), S[inverse]
    R = s["dS_T"].to(dt)[order]
    flow = (S * R).sum((-1, -2))
    dks, dvs, dla = torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(a)
    for t, m in reversed(list(enumerate(live))):
        at = first[:m] + t
        R[:m] += q[at][..., None] * do[at][..., None, :]
        dks[at] = torch.matmul(R[:m], v[at][..., None])[..., 0]
        dvs[at] = torch.matmul(k[at][..., None, :], R[:m])[..., 0, :]
        flow[:m] += (q[at] * one[at]).sum(-1) - (k[at] * dks[at]).sum(-1)
        dla[at] = flow[:m]
        R[:m] *= a[at][..., None, None]
    shared = lambda x: shape(x.reshape(x.shape[0], -1, share, dk).sum(2), s["q"])  # noqa: E731
    got = dict(dq=shared(one), dk=shared(dks), dv=shape(dvs, s["v"]), dS0=R[inverse])
    if la.dim() > 1:
        got["dlog_a"] = dla.reshape(s["log_a"].shape)
    return got
