"""Linear attention with a decay per head in float64 on the CPU, with rounding bounds.

``run`` is the definition of one head of one sequence,
out_t = sum_{j <= t} e^{L_t - L_j} (x_t . y_j) z_j + e^{L_t} start^T x_t, from its T x T weights;
``back`` sums over j >= t with e^{L_j - L_t} instead.  Beside every value it gives sums of absolute
values that bound the rounding of the two kernels.

Unit roundings: bf16 2^-8, fp32 2^-24 (half a step, relative).

The fp32 kernel updates a state T times (a product and a fused multiply-add each, and an
exponential of 2 ulp a token) and sums dy products: every term of out passes at most
3 T + dy + 16 roundings, so |error| <= (4 T + dy + 16) 2^-24 * big with
big = sum |weights| |x| . |y| |z|.

The tensor-core kernel rounds the chunk's weights e^{..} (x . y) to bf16, the state to bf16 for the
product with x, and out to bf16: |error| <= 2^-8 (|out| + within + through) + (fp32 part), with
within = sum over the chunk's j of |weight z_j| and through = e^{..} |x| . |state at the chunk's
start|.  The state itself takes bf16 triples of e^{..} y (24 bits): the fp32 part holds for it, with
accumulations that may truncate (2^-23).
"""
import torch

BF16, FP32 = 2.0 ** -8, 2.0 ** -24
CHUNK = 128


def _weights(la, back):
    """[T, T] e^{L_t - L_j} (j <= t), or e^{L_j - L_t} (j >= t); resets are exact zeros."""
    T = la.numel()
    w = torch.zeros(T, T, dtype=torch.float64)
    for t in range(T):  # products of decays, so that a reset does not meet inf - inf
        w[t, t] = 1.0
        if t:
            w[t, :t] = w[t - 1, :t] * torch.exp(la[t])
    return w.T.contiguous() if back else w


def run(x, y, z, la, start, back=False):
    """x, y [T, dy], z [T, dz], la [T], start [dy, dz] (float64).  Returns a dict with out, fin and the
    bounds' sums: big, within, through (like out), fin_big (like fin)."""
    T, dy = x.shape
    w = _weights(la, back)
    p = w * (x @ y.T)
    out = p @ z
    big = (w * (x.abs() @ y.abs().T)) @ z.abs()
    a = torch.exp(la)
    total = torch.exp(la.sum()) if T else torch.ones((), dtype=torch.float64)
    if T:
        # weight of the start: forward e^{L_t}, backward e^{L_end - L_t} = the last token's weight on t
        first = w[:, 0] * a[0] if not back else w[:, T - 1]
        out = out + first[:, None] * (x @ start)
        big = big + first[:, None] * (x.abs() @ start.abs())
        last = w[T - 1] if not back else w[0] * a[0]
        fin = total * start + (y * last[:, None]).T @ z
        fin_big = total * start.abs() + (y.abs() * last[:, None]).T @ z.abs()
    else:
        fin, fin_big = start.clone(), start.abs()
    within = torch.zeros_like(out)
    through = torch.zeros_like(out)
    S = start
    chunks = [(c, min(c + CHUNK, T)) for c in range(0, T, CHUNK)]
    for c0, c1 in reversed(chunks) if back else chunks:
        s = slice(c0, c1)
        within[s] = p[s, s].abs() @ z[s].abs()
        if not back:
            through[s] = (w[s, c0] * a[c0])[:, None] * (x[s].abs() @ S.abs())
            S = torch.exp(la[s].sum()) * S + (y[s] * w[c1 - 1, s][:, None]).T @ z[s]
        else:
            through[s] = w[s, c1 - 1][:, None] * (x[s].abs() @ S.abs())
            S = torch.exp(la[s].sum()) * S + (y[s] * (w[c0, s] * a[c0])[:, None]).T @ z[s]
    return dict(out=out, fin=fin, big=big, within=within, through=through, fin_big=fin_big)


def fp32_out(r, T, dy):
    return (4 * T + dy + 16) * FP32 * r["big"]


def fp32_fin(r, T):
    return (4 * T + 16) * FP32 * r["fin_big"]


def tc_out(r, T, dy):
    return BF16 * (r["out"].abs() + 1.01 * (r["within"] + r["through"])) + 2 * (T + dy + 64) * FP32 * r["big"]


def tc_fin(r, T):
    return 2 * (T + 64) * FP32 * r["fin_big"]


def problem(lens, H, Hqk, dk, dv, dtype, decay, start, seed, tail=0, device="cuda"):
    """Inputs of a packed batch (``tail`` rows behind the last sequence hold NaN)."""
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)

    def rnd(*shape, scale=1.0):
        v = (torch.randn(*shape, generator=g) * scale).to(dtype)
        return torch.cat([v, torch.full((tail, *shape[1:]), float("nan"), dtype=dtype)]) if tail else v

    p = dict(q=rnd(T, Hqk, dk, scale=dk ** -0.5), k=rnd(T, Hqk, dk, scale=dk ** -0.5), v=rnd(T, H, dv), dO=rnd(T, H, dv))
    if decay == "head":
        p["log_a"] = -torch.exp2(-8.0 * (torch.arange(H) + 1) / H)
    else:
        la = -torch.nn.functional.softplus(torch.randn(T, H, generator=g)) * (3.0 if decay == "strong" else 0.05)
        if decay == "none":
            la = torch.zeros(T, H)
        if decay == "reset":  # single resets, a stretch of them, and steps far below fp32's range
            la = torch.where(torch.rand(T, H, generator=g) < 0.02, -torch.inf, la)
            la[T // 3:T // 3 + 40] = -1000.0
        p["log_a"] = torch.cat([la.to(dtype), torch.full((tail, H), float("nan"), dtype=dtype)]) if tail else la.to(dtype)
    N = len(lens)
    p["S0"] = torch.randn(N, H, dk, dv, generator=g) * 0.3 if start else None
    p["dS_T"] = torch.randn(N, H, dk, dv, generator=g) * 0.3 if start else None
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    p["cu"] = torch.tensor(cu, dtype=torch.int32)
    return {k: None if v is None else v.to(device) for k, v in p.items()}, cu


def units(p, cu, H, Hqk):
    """(n, h, token slice, {name: float64 CPU tensor of the unit}) of every sequence and head."""
    share = H // Hqk
    dk, dv = p["q"].shape[-1], p["v"].shape[-1]
    c = {k: None if v is None else v.detach().cpu().double() for k, v in p.items() if k != "cu"}
    for n in range(len(cu) - 1):
        s = slice(cu[n], cu[n + 1])
        for h in range(H):
            u = dict(q=c["q"][s, h // share], k=c["k"][s, h // share], v=c["v"][s, h], dO=c["dO"][s, h],
                     la=(c["log_a"][h].expand(cu[n + 1] - cu[n]) if c["log_a"].dim() == 1 else c["log_a"][s, h]))
            zero = torch.zeros(dk, dv, dtype=torch.float64)
            u["S0"] = zero if c["S0"] is None else c["S0"][n, h]
            u["dS_T"] = zero if c["dS_T"] is None else c["dS_T"][n, h]
            yield n, h, s, u


def forward(p, cu, H, Hqk, tc):
    """o, S_T and their bounds (float64, CPU)."""
    T = cu[-1]
    dk, dv = p["q"].shape[-1], p["v"].shape[-1]
    o, ob = torch.zeros(T, H, dv, dtype=torch.float64), torch.zeros(T, H, dv, dtype=torch.float64)
    S, Sb = torch.zeros(len(cu) - 1, H, dk, dv, dtype=torch.float64), torch.zeros(len(cu) - 1, H, dk, dv, dtype=torch.float64)
    for n, h, s, u in units(p, cu, H, Hqk):
        length = cu[n + 1] - cu[n]
        r = run(u["q"], u["k"], u["v"], u["la"], u["S0"])
        o[s, h], S[n, h] = r["out"], r["fin"]
        ob[s, h] = tc_out(r, length, dk) if tc else fp32_out(r, length, dk)
        Sb[n, h] = tc_fin(r, length) if tc else fp32_fin(r, length)
    if not tc and p["q"].dtype == torch.bfloat16:
        ob = ob + BF16 * o.abs()
    return dict(o=(o, ob), S_T=(S, Sb))


def gradients(p, cu, H, Hqk, tc):
    """{name: (value, bound)} of dq, dk, dv, dlog_a, dS0 from the formulas of the three runs."""
    T, N = cu[-1], len(cu) - 1
    dk, dv = p["q"].shape[-1], p["v"].shape[-1]
    z = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    g = {x: (z(*s), z(*s)) for x, s in dict(dq=(T, Hqk, dk), dk=(T, Hqk, dk), dv=(T, H, dv), dlog_a=(T, H),
                                            dS0=(N, H, dk, dv)).items()}
    share = H // Hqk
    out_bound = tc_out if tc else fp32_out
    for n, h, s, u in units(p, cu, H, Hqk):
        length = cu[n + 1] - cu[n]
        rq = run(u["dO"], u["v"], u["k"], u["la"], u["S0"].T)
        rv = run(u["k"], u["q"], u["dO"], u["la"], u["dS_T"], back=True)
        rk = run(u["v"], u["dO"], u["q"], u["la"], u["dS_T"].T, back=True)
        for x, r, dim, head in (("dq", rq, dv, h // share), ("dk", rk, dv, h // share), ("dv", rv, dk, h)):
            g[x][0][s, head] += r["out"]
            g[x][1][s, head] += out_bound(r, length, dim)
        g["dS0"][0][n, h] = rv["fin"]
        g["dS0"][1][n, h] = tc_fin(rv, length) if tc else fp32_fin(rv, length)
        # dlog_a_t = sum of the pairs (i, j), j < t <= i, of e^{L_i - L_j} (q_i.k_j)(dO_i.v_j), with the
        # start and dS_T as a token before the first and one behind the last
        w = _weights(u["la"], False)
        pair = w * (u["q"] @ u["k"].T) * (u["dO"] @ u["v"].T)
        if length:
            e = torch.exp(u["la"])
            left = (w[:, 0] * e[0]) * torch.einsum("tk,kv,tv->t", u["q"], u["S0"], u["dO"])
            right = w[length - 1] * torch.einsum("tk,kv,tv->t", u["k"], u["dS_T"], u["v"])
            both = torch.exp(u["la"].sum()) * (u["S0"] * u["dS_T"]).sum()
            val, size = z(length), z(length)
            flow = (u["q"] * rq["out"]).sum(-1).abs() + (u["k"] * rk["out"]).sum(-1).abs()
            for t in range(length):
                val[t] = pair[t:, :t].sum() + left[t:].sum() + right[:t].sum() + both
            if tc:
                # every term of the chunk's sums carries a bf16 weight or state (2^-8 each), and so
                # does the product of the chunk's two states
                dots = (u["q"].abs() * (rq["within"] + rq["through"])).sum(-1) + (
                    u["k"].abs() * (rk["within"] + rk["through"])).sum(-1)
                for c0 in range(0, length, CHUNK):
                    sl = slice(c0, min(c0 + CHUNK, length))
                    size[sl] = dots[sl].sum()
                # the state product at the chunk's start, bounded by the flow through it
                bound = BF16 * (val.abs() + 1.01 * size) + BF16 * _through_chunks(u, w, left, right, both, length)
            else:
                bound = (4 * length + dk + dv + 32) * FP32 * (
                    (u["q"].abs() * rq["big"]).sum(-1).sum() + (u["k"].abs() * rk["big"]).sum(-1).sum()
                    + torch.exp(u["la"].sum()) * (u["S0"].abs() * u["dS_T"].abs()).sum()
                    + (rq["fin_big"].T * u["dS_T"].abs()).sum()) + z(length)
            g["dlog_a"][0][s, h], g["dlog_a"][1][s, h] = val, bound
            del flow
    if p["dO"].dtype == torch.bfloat16 and (not tc or share > 1):
        for x in ("dq", "dk", "dv", "dlog_a"):
            g[x] = (g[x][0], g[x][1] + BF16 * g[x][0].abs())
    return g


def _through_chunks(u, w, left, right, both, length):
    """For every chunk sum |S at its start| |dLoss/dS at its end| times the chunk's decay."""
    size = torch.zeros(length, dtype=torch.float64)
    S = u["S0"]
    starts = []
    for c0 in range(0, length, CHUNK):
        s = slice(c0, min(c0 + CHUNK, length))
        starts.append(S)
        S = torch.exp(u["la"][s].sum()) * S + (u["k"][s] * w[s.stop - 1, s][:, None]).T @ u["v"][s]
    R = u["dS_T"]
    for c0, S in reversed(list(zip(range(0, length, CHUNK), starts))):
        s = slice(c0, min(c0 + CHUNK, length))
        size[s] = torch.exp(u["la"][s].sum()) * (S.abs() * R.abs()).sum()
        back = w[s, c0] * torch.exp(u["la"][c0])
        R = torch.exp(u["la"][s].sum()) * R + (u["q"][s] * back[:, None]).T @ u["dO"][s]
    return size


def check(name, got, want, bound):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{name}: not finite"
    excess = (got - want).abs() - bound
    worst = float(excess.max()) if excess.numel() else 0.0
    assert worst <= 1e-30, f"{name}: {worst:.3g} above the bound (at {int(excess.argmax())}, |ref| max {float(want.abs().max()):.3g})"
