"""Workloads of the causal serving operators and of the block's layer norm.

Four operators around the bidirectional mixer core:

  prompt     causal conv + SiLU + selective scan over packed ragged prompts,
             whose states and conv tails live in a pool (in place)
  step       the same for one new token of each of a batch of streams
  norm       (residual add and) layer norm in front of the mixer's projection
  norm_grad  its backward pass with the weight and bias gradients

Each case is a dict of plain values; `prepare` draws its inputs, `run` makes
one pass: the plain torch form, or, where `own` is set, the library's calls.
"""
import math

import torch

own = False

Q = 64   # chunk of the plain prompt form


# --------------------------------------------------------------------------- cases
def _prompt(name, lens, dtype="bf16", heads=64, headdim=64, d_state=128, pool=None, resume="none",
            memory="mixed", bias=True):
    n = len(lens.split(","))
    return {"name": name, "op": "prompt", "dtype": dtype, "heads": heads, "headdim": headdim,
            "d_state": d_state, "lens": lens, "pool": n + 3 if pool is None else pool,
            "resume": resume, "memory": memory, "bias": bias}


def _step(name, rows, dtype="bf16", heads=64, headdim=64, d_state=128, pool=None, bias=True):
    return {"name": name, "op": "step", "dtype": dtype, "heads": heads, "headdim": headdim,
            "d_state": d_state, "rows": rows, "pool": rows + 3 if pool is None else pool,
            "memory": "mixed", "bias": bias}


def _norm(name, op, rows, cols, dtype="bf16", residual=True, bias=True):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype,
            "residual": residual, "bias": bias}


def listed():
    return [
        # a short follow-up turn of one cached stream: latency
        _prompt("prompt_turn_37", "37", resume="all"),
        # a serving batch of prompts of every length, some of them continuing a cached entry
        _prompt("prompt_ragged_8k", "1311,1,640,129,0,2777,63,1024,517,1536,128", resume="some"),
        # the 1.3B layer's batch: 8 sequences of 4096 tokens
        _prompt("prompt_8x4096", ",".join(["4096"] * 8)),
        # one long document: few walks, so the sequence itself has to be split
        _prompt("prompt_long_32k", "32768", memory="long"),
        # fp32 activations (the parity path), ragged
        _prompt("prompt_f32_ragged", "1024,517,1,300", dtype="f32", resume="some"),
        # one stream generating: latency
        _step("step_1", 1),
        # 32 streams (the decode workload's batch)
        _step("step_32", 32),
        # every stream of a 256-entry pool, fp32 activations
        _step("step_256_f32", 256, dtype="f32", pool=256),
        # the rows of a decode batch, at the model's width
        _norm("norm_32x2048", "norm", 32, 2048),
        # the 1.3B layer's tokens
        _norm("norm_32768x2048", "norm", 32768, 2048),
        _norm("norm_grad_32768x2048", "norm_grad", 32768, 2048),
        # fp32 training of a ragged batch at a width that is no power of two
        _norm("norm_grad_f32_1001x4104", "norm_grad", 1001, 4104, dtype="f32", residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _split(rng, tokens, n):
    """`tokens` over `n` prompts: uneven, empty ones and single tokens among them."""
    w = [rng.choice([0.0, rng.random() ** 3, rng.random(), 1.0]) for _ in range(n)]
    if not any(w):
        w[0] = 1.0
    lens = [int(tokens * x / sum(w)) for x in w]
    lens[max(range(n), key=lambda i: w[i])] += tokens - sum(lens)
    return lens


def draw(rng):
    op = rng.choice(["prompt", "prompt", "step", "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("norm", "norm_grad"):
        cols = 8 * _log(rng, 8, 1024)
        rows = _log(rng, 1, 32768)
        rows = max(1, min(rows, 32768 * 2048 // cols // (1 if dtype == "bf16" else 2)))
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype,
                "residual": rng.random() < 0.5, "bias": rng.random() < 0.7}
    heads, P, N = rng.choice([(2 * rng.randint(1, 32), 64, 128), (64, 64, 128),
                              (rng.randint(1, 16), rng.choice([32, 64, 128]), rng.choice([16, 32, 64, 256]))])
    d = {"op": op, "dtype": dtype, "heads": heads, "headdim": P, "d_state": N,
         "memory": rng.choice(["short", "mixed", "long"]), "bias": rng.random() < 0.7}
    if op == "step":
        rows = _log(rng, 1, 256)
        return {**d, "rows": rows, "pool": rows + rng.randint(0, 16)}
    tc = dtype == "bf16" and P == 64 and N == 128 and heads % 2 == 0
    tokens = _log(rng, 1, 32768 if tc else 2048)
    n = _log(rng, 1, 24)
    lens = _split(rng, tokens, n)
    return {**d, "lens": ",".join(str(v) for v in lens), "pool": n + rng.randint(0, 6),
            "resume": rng.choice(["none", "some", "all"])}


# --------------------------------------------------------------------------- inputs
_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _mixer(case, tokens, g):
    """Raw xBC, dt (positive), A, D and the conv of a mixer: the distributions
    of the repository's synthetic inputs.  memory: how fast the states decay."""
    H, P, N = case["heads"], case["headdim"], case["d_state"]
    ch = H * P + 2 * N
    dev, td = "cuda", _DTYPE[case["dtype"]]
    lo, hi = {"short": (1.0, 16.0), "mixed": (0.02, 16.0), "long": (1e-3, 1e-2)}[case["memory"]]
    xbc = torch.randn((tokens, ch), generator=g, device=dev)
    xbc[:, H * P:] /= math.sqrt(N)
    dt = torch.nn.functional.softplus(torch.randn((tokens, H), generator=g, device=dev) * math.sqrt(0.5) - 2.0)
    A = -torch.exp(torch.rand((H,), generator=g, device=dev) * math.log(hi / lo) + math.log(lo))
    D = torch.randn((H,), generator=g, device=dev)
    conv_w = torch.randn((ch, 4), generator=g, device=dev) * 0.5
    conv_b = torch.randn((ch,), generator=g, device=dev) * 0.1 if case["bias"] else None
    pool = case["pool"]
    state = torch.randn((pool, H, P, N), generator=g, device=dev) * 0.2
    tail = torch.randn((pool, 4, ch), generator=g, device=dev)
    tail[..., H * P:] /= math.sqrt(N)
    return {"xbc": xbc.to(td), "dt": dt.to(td), "A": A, "D": D, "conv_w": conv_w, "conv_b": conv_b,
            "state_pool": state, "tail_pool": tail.to(td)}


def _lens(case):
    return [int(v) for v in case["lens"].split(",")]


def _resumed(case, n):
    return [{"none": 0, "all": 1, "some": (i + 1) % 2}[case["resume"]] for i in range(n)]


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        rows, cols, td = case["rows"], case["cols"], _DTYPE[case["dtype"]]
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        scale = torch.exp(0.3 * rnd(rows, 1))
        x = (rnd(rows, cols) * scale + 0.2 * rnd(rows, 1)).to(td)
        s = {"x": x, "gamma": 1.0 + 0.2 * rnd(cols), "beta": 0.1 * rnd(cols) if case["bias"] else None,
             "residual": rnd(rows, cols).to(td) if case["residual"] else None, "eps": 1e-5}
        if op == "norm_grad":
            h = x.double()
            mean = h.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = torch.rsqrt((h - mean[:, None]).square().mean(1) + s["eps"]).float()
            s["dy"] = rnd(rows, cols).to(td)
        return s
    if op == "step":
        s = _mixer(case, case["rows"], g)
        s["slots"] = torch.randperm(case["pool"], generator=g, device="cuda")[:case["rows"]].to(torch.int32)
        return s
    lens = _lens(case)
    s = _mixer(case, sum(lens), g)
    n = len(lens)
    s["lens"] = lens
    s["cu_seqlens"] = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
    s["slots"] = torch.randperm(case["pool"], generator=g, device="cuda")[:n].to(torch.int32)
    s["resume"] = torch.tensor(_resumed(case, n), dtype=torch.int32, device="cuda")
    return s


def prepare(case, seed):
    """Inputs, the output buffers and the workspace that a serving or training
    program keeps."""
    s = _inputs(case, seed)
    s["case"] = case
    op = case["op"]
    if op in ("norm", "norm_grad"):
        x = s["x"]
        f32 = dict(dtype=torch.float32, device="cuda")
        if op == "norm":
            s["out"] = {"y": torch.empty_like(x), "mean": torch.empty(case["rows"], **f32),
                        "rstd": torch.empty(case["rows"], **f32)}
            if case["residual"]:
                s["out"]["sum"] = torch.empty_like(x)
        else:
            s["out"] = {"dx": torch.empty_like(x), "dgamma": torch.empty(case["cols"], **f32)}
            if case["bias"]:
                s["out"]["dbeta"] = torch.empty(case["cols"], **f32)
    else:
        s["y"] = torch.zeros((s["xbc"].shape[0], case["heads"] * case["headdim"]), dtype=s["xbc"].dtype,
                             device="cuda")
    if own and op != "norm":
        from bidirectional_mamba_ssm_b200 import _lib as bm
        if op == "norm_grad":
            s["ws"] = bm.new_layer_norm_workspace(s["x"])
        elif op == "prompt":
            s["ws"] = bm.new_prompt_workspace(s["xbc"], batch=len(s["lens"]), heads=case["heads"],
                                              headdim=case["headdim"], d_state=case["d_state"])
        else:
            s["ws"] = bm.new_step_workspace(case["rows"], heads=case["heads"], headdim=case["headdim"],
                                            d_state=case["d_state"], dtype=s["xbc"].dtype)
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    return {"prompt": _run_prompt, "step": _run_step, "norm": _run_norm, "norm_grad": _run_norm_grad}[case["op"]](s)


def _shape(case):
    return {"heads": case["heads"], "headdim": case["headdim"], "d_state": case["d_state"]}


def _run_prompt(s):
    if own:
        from bidirectional_mamba_ssm_b200 import _lib as bm
        bm.bimamba_prompt_scan(s["xbc"], s["dt"], s["A"], s["D"], s["conv_w"], s["conv_b"], s["cu_seqlens"],
                               s["state_pool"], s["tail_pool"], s["slots"], s["resume"], s["y"], s["ws"],
                               **_shape(s["case"]))
    else:
        _plain_prompt(s)
    return {"y": s["y"], "state": s["state_pool"], "tail": s["tail_pool"]}


def _run_step(s):
    if own:
        from bidirectional_mamba_ssm_b200 import _lib as bm
        bm.bimamba_token_step(s["xbc"], s["dt"], s["A"], s["D"], s["conv_w"], s["conv_b"], s["state_pool"],
                              s["tail_pool"], s["slots"], s["y"], s["ws"], **_shape(s["case"]))
    else:
        _plain_step(s)
    return {"y": s["y"], "state": s["state_pool"], "tail": s["tail_pool"]}


def _run_norm(s):
    o = s["out"]
    if own:
        from bidirectional_mamba_ssm_b200 import _lib as bm
        bm.bimamba_layer_norm(s["x"], s["gamma"], s["beta"], o["y"], o["mean"], o["rstd"],
                              residual=s["residual"], sum_out=o.get("sum"), eps=s["eps"])
        return o
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    mean = h.mean(1)
    d = h - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + s["eps"])
    y = d * rstd[:, None] * s["gamma"]
    if s["beta"] is not None:
        y = y + s["beta"]
    r = {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    if s["residual"] is not None:
        r["sum"] = h.to(s["x"].dtype)
    return r


def _run_norm_grad(s):
    o = s["out"]
    if own:
        from bidirectional_mamba_ssm_b200 import _lib as bm
        bm.bimamba_layer_norm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], o["dx"], o["dgamma"],
                                       o.get("dbeta"), s["ws"], dsum=s["residual"])
        return o
    dy = s["dy"].float()
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    a = dy * s["gamma"]
    dx = (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    r = {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xh).sum(0)}
    if s["beta"] is not None:
        r["dbeta"] = dy.sum(0)
    return r


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _plain_step(s):
    case = s["case"]
    H, P, N = case["heads"], case["headdim"], case["d_state"]
    slots = s["slots"].long()
    tail = torch.cat([s["tail_pool"][slots][:, 1:], s["xbc"][:, None]], 1)
    act = (tail.float() * s["conv_w"].t()).sum(1)
    if s["conv_b"] is not None:
        act = act + s["conv_b"]
    act = _silu(act)
    x = act[:, :H * P].view(-1, H, P)
    B, C = act[:, None, None, H * P:H * P + N], act[:, None, None, H * P + N:]
    dt = s["dt"].float()
    h = s["state_pool"][slots] * torch.exp(dt * s["A"])[:, :, None, None] + (dt[:, :, None] * x)[..., None] * B
    y = (h * C).sum(-1) + s["D"][:, None] * x
    s["y"].copy_(y.view(-1, H * P))
    s["state_pool"][slots] = h
    s["tail_pool"][slots] = tail


def _plain_prompt(s):
    """The chunked form: within chunks of Q tokens by masked products, across a
    prompt's chunks by one product with the decays between them.  Sums of
    dt * A in 64 bits (their differences are what counts)."""
    case, lens = s["case"], s["lens"]
    H, P, N = case["heads"], case["headdim"], case["d_state"]
    dev, n, total = s["xbc"].device, len(lens), sum(lens)
    slots = s["slots"].long()
    resume = s["resume"].bool()
    ln = torch.tensor(lens, device=dev)
    start = torch.cumsum(ln, 0) - ln
    tail0 = torch.where(resume[:, None, None], s["tail_pool"][slots], torch.zeros_like(s["tail_pool"][:1]))
    init = torch.where(resume[:, None, None, None], s["state_pool"][slots], torch.zeros_like(s["state_pool"][:1]))
    # raw rows: the packed tokens, then each prompt's 4 tokens before it
    rows = torch.cat([s["xbc"], tail0.reshape(4 * n, -1)])
    seq = torch.repeat_interleave(torch.arange(n, device=dev), ln, output_size=total)
    pos = torch.arange(total, device=dev) - start[seq]

    def source(p, q):   # the row of position p (may be -4..-1) of prompt q
        return torch.where(p >= 0, start[q] + p, total + 4 * q + 4 + p)

    if total:
        act = sum(rows[source(pos - 3 + j, seq)].float() * s["conv_w"][:, j] for j in range(4))
        if s["conv_b"] is not None:
            act = act + s["conv_b"]
        act = torch.cat([_silu(act), act.new_zeros(1, act.shape[1])])
        dtp = torch.cat([s["dt"].float(), s["dt"].new_zeros(1, H).float()])
        # chunks: a prompt's tokens from its own start, Q at a time, filled up with the zero row
        nch = (ln + Q - 1) // Q
        first = torch.cumsum(nch, 0) - nch
        nc = sum((v + Q - 1) // Q for v in lens)
        cseq = torch.repeat_interleave(torch.arange(n, device=dev), nch, output_size=nc)
        p = (torch.arange(nc, device=dev) - first[cseq])[:, None] * Q + torch.arange(Q, device=dev)
        idx = torch.where(p < ln[cseq][:, None], start[cseq][:, None] + p, total)
        a, dt = act[idx], dtp[idx]
        x = a[..., :H * P].view(nc, Q, H, P).transpose(1, 2)
        B, C = a[..., H * P:H * P + N], a[..., H * P + N:]
        c = torch.cumsum(dt.double() * s["A"].double(), 1).transpose(1, 2)           # nc, H, Q
        dth = dt.transpose(1, 2)
        below = torch.ones(Q, Q, dtype=torch.bool, device=dev).tril()
        decay = torch.exp((c[..., :, None] - c[..., None, :]).masked_fill(~below, -math.inf)).float()
        M = (C @ B.transpose(1, 2))[:, None] * decay * dth[:, :, None]
        y = M @ x
        w = torch.exp(c[..., -1:] - c).float() * dth                                  # nc, H, Q
        local = (x * w[..., None]).transpose(2, 3) @ B[:, None]                       # nc, H, P, N
        # across chunks: state entering chunk i = sum over j < i of the same prompt
        tot = torch.cumsum(c[..., -1], 0)                                             # nc, H
        before = tot - c[..., -1]
        same = (cseq[:, None] == cseq) & torch.ones(nc, nc, dtype=torch.bool, device=dev).tril(-1)
        E = torch.exp((before.t()[:, :, None] - tot.t()[:, None, :]).masked_fill(~same, -math.inf)).float()
        flat = local.transpose(0, 1).reshape(H, nc, P * N)
        base = before[first[cseq].clamp(max=nc - 1)]
        enter = (E @ flat).view(H, nc, P, N).transpose(0, 1)
        enter = enter + torch.exp(before - base).float()[..., None, None] * init[cseq]
        y = y + torch.exp(c).float()[..., None] * (C[:, None] @ enter.transpose(2, 3))
        y = y + s["D"][:, None, None] * x
        s["y"][:total] = y.transpose(1, 2).reshape(nc * Q, H * P)[(p < ln[cseq][:, None]).reshape(-1)].to(s["y"].dtype)
        final = torch.exp(c[..., -1]).float()[..., None, None] * enter + local
        last = (first + nch - 1).clamp(min=0)
        init = torch.where((ln > 0)[:, None, None, None], final[last], init)
    back = ln[:, None] - 4 + torch.arange(4, device=dev)
    s["tail_pool"][slots] = rows[source(back, torch.arange(n, device=dev)[:, None])]
    s["state_pool"][slots] = init


# --------------------------------------------------------------------------- counts
def work(case):
    esz = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("norm", "norm_grad"):
        n, r = case["rows"] * case["cols"], 1 if case["residual"] else 0
        params = 4 * case["cols"] * (2 if case["bias"] else 1)
        if op == "norm":
            return {"bytes": esz * n * (2 + 2 * r) + 8 * case["rows"] + params, "flops": 8 * n}
        return {"bytes": esz * n * (3 + r) + 8 * case["rows"] + 4 * case["cols"] + params, "flops": 14 * n}
    H, P, N = case["heads"], case["headdim"], case["d_state"]
    ch, st = H * P + 2 * N, 4 * H * P * N
    params = 4 * (2 * H + ch * (5 if case["bias"] else 4))
    if op == "step":
        r = case["rows"]
        return {"bytes": r * (2 * st + esz * (ch + H + H * P + 7 * ch)) + params, "flops": r * (5 * H * P * N + 8 * ch)}
    lens = _lens(case)
    t, n, k = sum(lens), len(lens), sum(_resumed(case, len(lens)))
    return {"bytes": esz * t * (ch + H + H * P) + (n + k) * st + esz * ch * (4 * n + 3 * k) + params,
            "flops": t * (2 * Q * N + H * (Q * P + 4 * P * N))}


# --------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The definitions in 64 bits: token by token for the scans, row by row
    (two passes) for the norm."""
    s = _inputs(case, seed)
    f = lambda t: None if t is None else t.double()  # noqa: E731
    op = case["op"]
    if op == "norm":
        h = f(s["x"]) if s["residual"] is None else f(s["x"]) + f(s["residual"])
        var, mean = torch.var_mean(h, dim=1, correction=0)
        inv = (var + s["eps"]) ** -0.5
        y = torch.einsum("rc,r,c->rc", h - mean[:, None], inv, f(s["gamma"]))
        out = {"y": y if s["beta"] is None else y + f(s["beta"]), "mean": mean, "rstd": inv}
        if s["residual"] is not None:
            out["sum"] = h
        return out
    if op == "norm_grad":
        m, inv, dy, cols = f(s["mean"])[:, None], f(s["rstd"])[:, None], f(s["dy"]), case["cols"]
        z = (f(s["x"]) - m) * inv
        u = dy * f(s["gamma"])
        dx = inv / cols * (cols * u - u.sum(1, keepdim=True) - z * torch.einsum("rc,rc->r", u, z)[:, None])
        out = {"dx": dx if s["residual"] is None else dx + f(s["residual"]), "dgamma": torch.einsum("rc,rc->c", dy, z)}
        if case["bias"]:
            out["dbeta"] = dy.sum(0)
        return out
    H, P, N = case["heads"], case["headdim"], case["d_state"]
    slots = s["slots"].long().tolist()
    if op == "step":
        lens, keep = [1] * case["rows"], [1] * case["rows"]
    else:
        lens, keep = s["lens"], _resumed(case, len(s["lens"]))
    steps = max(lens) if lens else 0
    if steps * max(1, len(lens)) * H * P * N > 3e11:
        return None
    n, ch = len(lens), H * P + 2 * N
    pool, tails = f(s["state_pool"]).clone(), f(s["tail_pool"]).clone()
    xbc, dt, A, D, w = f(s["xbc"]), f(s["dt"]), f(s["A"]), f(s["D"]), f(s["conv_w"])
    bias = 0.0 if s["conv_b"] is None else f(s["conv_b"])
    kept = torch.tensor(keep, device="cuda", dtype=torch.float64)
    h = pool[slots] * kept[:, None, None, None]
    window = tails[slots] * kept[:, None, None]                       # the last 4 raw tokens of each prompt
    starts = torch.tensor([sum(lens[:i]) for i in range(n)], device="cuda")
    count = torch.tensor(lens, device="cuda")
    y = torch.zeros((xbc.shape[0] + 1, H * P), dtype=torch.float64, device="cuda")
    if xbc.shape[0] == 0:
        steps = 0
    for t in range(steps):
        live = (count > t)
        row = torch.where(live, starts + t, 0)
        moved = torch.cat([window[:, 1:], xbc[row][:, None]], 1)
        window = torch.where(live[:, None, None], moved, window)
        pre = torch.einsum("bkc,ck->bc", window, w) + bias
        u = pre * torch.sigmoid(pre)
        x = u[:, :H * P].reshape(n, H, P)
        d = dt[row] * live[:, None]
        h = h * torch.exp(d * A)[:, :, None, None]
        h += torch.einsum("bhp,bn->bhpn", x * d[:, :, None], u[:, H * P:H * P + N])
        out = torch.einsum("bhpn,bn->bhp", h, u[:, H * P + N:ch]) + x * D[:, None]
        y[torch.where(live, starts + t, xbc.shape[0])] = out.reshape(n, H * P)
    pool[slots], tails[slots] = h, window
    return {"y": y[:-1], "state": pool, "tail": tails}
