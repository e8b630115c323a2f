"""The causal mixer core in 64 bits, token by token on the CPU: what the
prompt scan and the token step are tested against."""
import math

import numpy as np
import torch


def draw(tokens, n, heads, headdim, d_state, dtype, seed, *, pool, a_range=(0.02, 16.0), bias=True):
    """Seeded inputs and a pool: xbc ~ N(0, 1) with B and C scaled by
    1/sqrt(N), dt = softplus(N(-2, 1/2)), A log-uniform in -[a_range]."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    H, P, N = heads, headdim, d_state
    ch = H * P + 2 * N
    xbc = r(tokens, ch)
    xbc[:, H * P:] /= math.sqrt(N)
    tail = r(pool, 4, ch)
    tail[..., H * P:] /= math.sqrt(N)
    lo, hi = a_range
    return {"xbc": xbc.to(dtype), "dt": torch.nn.functional.softplus(r(tokens, H) * math.sqrt(0.5) - 2).to(dtype),
            "A": -torch.exp(torch.rand(H, generator=g) * math.log(hi / lo) + math.log(lo)), "D": r(H),
            "conv_w": r(ch, 4) * 0.5, "conv_b": r(ch) * 0.1 if bias else None,
            "state": r(pool, H, P, N) * 0.2, "tail": tail.to(dtype),
            "slots": torch.randperm(pool, generator=g)[:n].to(torch.int32)}


def prompts(d, lens, resume, heads, headdim, d_state, cu=None):
    """(y, state pool, tail pool) in 64 bits; rows outside every prompt are 0."""
    H, P, N = heads, headdim, d_state
    f = lambda t: t.double().numpy()  # noqa: E731
    xbc, dt, A, D, w = (f(d[k]) for k in ("xbc", "dt", "A", "D", "conv_w"))
    bias = 0.0 if d["conv_b"] is None else f(d["conv_b"])
    state, tail = f(d["state"]).copy(), f(d["tail"]).copy()
    y = np.zeros((xbc.shape[0], H * P))
    if cu is None:
        cu = [0]
        for v in lens:
            cu.append(cu[-1] + v)
    for s, n in enumerate(lens):
        k = int(d["slots"][s])
        h = state[k].copy() if resume[s] else np.zeros((H, P, N))
        t0 = tail[k].copy() if resume[s] else np.zeros_like(tail[k])
        rows = np.concatenate([t0, xbc[cu[s]:cu[s] + n]])
        for t in range(n):
            pre = (rows[t + 1:t + 5] * w.T).sum(0) + bias
            u = pre / (1.0 + np.exp(-pre))
            x, B, C = u[:H * P].reshape(H, P), u[H * P:H * P + N], u[H * P + N:]
            step = dt[cu[s] + t]
            h *= np.exp(step * A)[:, None, None]
            h += (step[:, None] * x)[:, :, None] * B
            y[cu[s] + t] = (h @ C + D[:, None] * x).reshape(-1)
        state[k], tail[k] = h, rows[n:n + 4]
    return y, state, tail


def run(lib, d, lens, resume, heads, headdim, d_state, *, rows=None, cu=None, y=None, ws=None, stream=None,
        device="cuda"):
    """bimamba_prompt_scan on copies: (y, state pool, tail pool)."""
    c = {k: None if v is None else v.to(device) for k, v in d.items()}
    if cu is None:
        cu = [0]
        for v in lens:
            cu.append(cu[-1] + v)
    if y is None:
        y = torch.full((d["xbc"].shape[0], heads * headdim), float("nan"), dtype=d["xbc"].dtype, device=device)
    shape = dict(heads=heads, headdim=headdim, d_state=d_state)
    if ws is None:
        ws = lib.new_prompt_workspace(c["xbc"], batch=len(lens), **shape)
    lib.bimamba_prompt_scan(c["xbc"], c["dt"], c["A"], c["D"], c["conv_w"], c["conv_b"],
                            torch.tensor(cu, dtype=torch.int32, device=device), c["state"], c["tail"], c["slots"],
                            None if resume is None else torch.tensor(resume, dtype=torch.int32, device=device), y,
                            ws, stream=stream, **shape)
    return y, c["state"], c["tail"]


def far(got, want):
    """2-norm of the difference over the 2-norm of the value."""
    got = got.detach().cpu().double().numpy() if torch.is_tensor(got) else np.asarray(got)
    n = np.linalg.norm(want)
    off = np.linalg.norm(got - want)
    return off / n if n else off
