"""Workloads of the operators around a TTT layer: layer norm, the gated linear recurrence and
the linear layer with its epilogue, each with its backward pass and its small serving form.

A block of a model that uses the library reads its hidden states through a norm, projects them
with linear layers, mixes them over time (the TTT layer, or a gated recurrence) and projects
the result back onto the residual stream. The widths are the repository's: 1024 and 2048 (16
heads of 64 and 128, the 410M and 1.45B shapes), 2560 and 9728 (the In-Place shape), 512 to
32768 tokens.

With `own` false the operators run in plain form (elementary torch operations in float32,
rounded once at the end); with `own` true they are the library's calls.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
# the In-Place shape: 32768 tokens of width 2560, hidden width 9728
MAX_ELEMS = 32768 * 2560
MAX_MNK = 32768 * 9728 * 2560


def listed():
    return [
        # one decode step of 8 sequences: residual add and norm of one row each (latency)
        dict(name="norm_fwd_decode", op="norm_fwd", B=1, H=1, T=8, d=2560, dtype="bf16",
             residual=True, token_major=False),
        # output norm of the 1.45B shape's TTT layer: per-head weights, heads to token-major rows
        dict(name="norm_fwd_heads", op="norm_fwd", B=4, H=16, T=4096, d=128, dtype="bf16",
             residual=False, token_major=True),
        # pre-norm of a long sequence at the In-Place width, with the residual stream's gradient
        dict(name="norm_bwd_long", op="norm_bwd", B=1, H=1, T=32768, d=2560, dtype="bf16",
             residual=True, token_major=False),
        # ragged float32 rows: odd width, odd count, two weight groups
        dict(name="norm_bwd_odd_f32", op="norm_bwd", B=3, H=2, T=683, d=1021, dtype="f32",
             residual=False, token_major=False),
        # one token of 64 running sequences in a cache of 96, some batch rows padding (latency)
        dict(name="recur_step_64", op="recur_step", B=64, D=2560, S=96, dtype="bf16",
             gate="sigmoid"),
        # packed documents of a 32768-token sequence, few channels, a long scan
        dict(name="recur_fwd_long", op="recur_fwd", B=1, T=32768, D=2560, dtype="bf16",
             gate="sigmoid", docs=True),
        # training batch of the 410M shape's tokens at the 1.45B width
        dict(name="recur_bwd_train", op="recur_bwd", B=8, T=2048, D=2048, dtype="bf16",
             gate="sigmoid", docs=False),
        # decay given as values (as the TTT layer's gamma), odd sizes, float32
        dict(name="recur_bwd_odd_f32", op="recur_bwd", B=3, T=1537, D=1021, dtype="f32",
             gate="decay", docs=True),
        # decode step of 8 sequences through the up projection (a weight read)
        dict(name="linear_fwd_decode", op="linear_fwd", M=8, N=9728, K=2560, act="silu",
             bias=True, mul=True, residual=False),
        # the gated-MLP activation Z = SiLU(H Wg^T) * U that the In-Place layer takes
        dict(name="linear_fwd_gated_mlp", op="linear_fwd", M=32768, N=9728, K=2560, act="silu",
             bias=False, mul=True, residual=False),
        # output projection onto the residual stream, ragged sizes
        dict(name="linear_fwd_ragged", op="linear_fwd", M=1537, N=1000, K=520, act="id",
             bias=True, mul=False, residual=True),
        # training step of a projection with bias and SiLU at the 1.45B shape
        dict(name="linear_bwd_train", op="linear_bwd", M=16384, N=2048, K=2048, act="silu",
             bias=True, mul=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "recur_fwd", "recur_bwd", "recur_step",
                     "linear_fwd", "linear_bwd"])
    if op.startswith("norm"):
        B, H, d = rng.randint(1, 8), rng.choice([1, 1, 1, 2, 3, 8, 16]), _log_int(rng, 16, 8192)
        T = _log_int(rng, 1, 16384)
        T = max(1, min(T, MAX_ELEMS // (B * H * d)))
        return dict(op=op, B=B, H=H, T=T, d=d, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    residual=rng.random() < 0.5, token_major=rng.random() < 0.5)
    if op == "recur_step":
        B = _log_int(rng, 1, 256)
        return dict(op=op, B=B, D=_log_int(rng, 16, 8192), S=B + rng.randint(0, 64),
                    dtype=rng.choice(["bf16", "bf16", "f32"]),
                    gate=rng.choice(["sigmoid", "decay"]))
    if op.startswith("recur"):
        B, T, D = rng.randint(1, 8), _log_int(rng, 1, 32768), _log_int(rng, 16, 4096)
        T = max(1, min(T, MAX_ELEMS // (2 * B * D)))
        return dict(op=op, B=B, T=T, D=D, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    gate=rng.choice(["sigmoid", "decay"]), docs=rng.random() < 0.5)
    M, N, K = _log_int(rng, 1, 16384), 8 * _log_int(rng, 2, 1216), 8 * _log_int(rng, 2, 512)
    M = max(1, min(M, MAX_MNK // (4 * N * K)))
    case = dict(op=op, M=M, N=N, K=K, act=rng.choice(["id", "silu"]), bias=rng.random() < 0.5,
                mul=rng.random() < 0.5)
    if op == "linear_fwd":
        case["residual"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------------------------ inputs
def _dt(case):
    return BF16 if case["dtype"] == "bf16" else F32


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = dict(device="cuda")

    def randn(*shape, dtype=F32, std=1.0, mean=0.0):
        x = torch.empty(shape, **dev).normal_(mean, std, generator=g)
        return x if dtype == F32 else x.to(dtype)

    def empty(*shape, dtype=F32):
        return torch.empty(shape, dtype=dtype, **dev)

    s = dict(case=case, out={})
    o = s["out"]
    op = case["op"]
    if op.startswith("norm"):
        B, H, T, d, dt = case["B"], case["H"], case["T"], case["d"], _dt(case)
        yshape = (B, T, H, d) if case["token_major"] else (B, H, T, d)
        # hidden states: unit spread about a row mean of the same size
        x = randn(B, H, T, d) + randn(B, H, T, 1)
        s["X"] = x.to(dt)
        s["weight"], s["bias"] = randn(H, d, std=0.2, mean=1.0), randn(H, d, std=0.2)
        if op == "norm_fwd":
            s["residual"] = randn(B, H, T, d, dtype=dt) if case["residual"] else None
            o["Y"] = empty(*yshape, dtype=dt)
            o["S"] = empty(B, H, T, d, dtype=dt) if case["residual"] else None
            o["mean"], o["rstd"] = empty(B, H, T), empty(B, H, T)
        else:
            xs = s["X"].float()
            s["mean"] = xs.mean(-1)
            s["rstd"] = torch.rsqrt(xs.var(-1, unbiased=False) + 1e-5)
            s["dY"] = randn(*yshape, dtype=dt)
            s["dS"] = randn(B, H, T, d, dtype=dt) if case["residual"] else None
            o["dX"] = empty(B, H, T, d, dtype=dt)
            o["dweight"], o["dbias"] = empty(H, d), empty(H, d)
        return s
    if op.startswith("recur"):
        B, D, dt = case["B"], case["D"], _dt(case)
        T = case.get("T", 1)
        shape = (B, T, D) if op != "recur_step" else (B, D)
        s["X"] = randn(*shape, dtype=dt)
        if case["gate"] == "sigmoid":  # gate logits: decays around 0.88, memories of 2 to 50 tokens
            s["G"] = randn(*shape, std=1.0, mean=2.0, dtype=dt)
        else:                          # decay values, as the TTT layer's gamma: sigmoid(N(3, 0.5))
            s["G"] = torch.sigmoid(randn(*shape, std=0.5, mean=3.0))
        if op == "recur_step":
            s["state"] = randn(case["S"], D, std=0.5)
            slots = torch.randperm(case["S"], generator=g, **dev)[:B].to(torch.int32)
            if B >= 8:  # the batch is padded to its bucket: the last rows name no sequence
                slots[B - B // 8:] = -1
            s["slots"] = slots
            o["Y"] = torch.zeros(shape, dtype=dt, **dev)
            return s
        s["reset"] = None
        if case["docs"]:  # documents of about 600 tokens, packed
            s["reset"] = (torch.rand((B, T), generator=g, **dev) < 1 / 600).to(torch.uint8)
        s["h0"] = randn(B, D, std=0.5)
        if op == "recur_fwd":
            o["Hs"], o["h_final"] = empty(B, T, D, dtype=dt), empty(B, D)
            return s
        s["dH"], s["dh_final"] = randn(B, T, D, dtype=dt), randn(B, D)
        s["Hs"] = _recur_plain(s)[0].to(dt)
        o["dX"], o["dh0"] = empty(B, T, D, dtype=dt), empty(B, D)
        o["dG"] = empty(B, T, D, dtype=s["G"].dtype)
        return s
    M, N, K = case["M"], case["N"], case["K"]
    s["X"] = randn(M, K, dtype=BF16)
    s["W"] = randn(N, K, std=K ** -0.5, dtype=BF16)
    s["bias"] = randn(N, std=0.5) if case["bias"] else None
    s["mul"] = randn(M, N, dtype=BF16) if case["mul"] else None
    if op == "linear_fwd":
        s["residual"] = randn(M, N, dtype=BF16) if case["residual"] else None
        o["Y"] = empty(M, N, dtype=BF16)
        return s
    s["P"] = randn(M, N, dtype=BF16) if case["act"] != "id" or case["mul"] else None
    s["dY"] = randn(M, N, dtype=BF16)
    o["dX"], o["dW"] = empty(M, K, dtype=BF16), empty(N, K, dtype=BF16)
    o["dbias"] = empty(N) if case["bias"] else None
    o["dmul"] = empty(M, N, dtype=BF16) if case["mul"] else None
    return s


# ------------------------------------------------------------------------------- plain forms
def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 1 with h_{-1} = 0, by doubling: after the step with
    offset k each entry holds the map of the last 2k tokens."""
    k, T = 1, a.shape[1]
    while k < T:
        u = torch.cat([u[:, :k], u[:, k:] + a[:, k:] * u[:, :-k]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return u


def _gates(s):
    """The decay of every token (0 where a document starts), the gate itself and the input."""
    x, g = s["X"].float(), s["G"].float()
    if s["case"]["gate"] == "sigmoid":
        a, u = _sigmoid(g), x * _sigmoid(-g)
    else:
        a, u = g, x
    r = s.get("reset")
    keep = a if r is None else torch.where(r[..., None] != 0, torch.zeros_like(a), a)
    return keep, a, u


def _recur_plain(s):
    keep, _, u = _gates(s)
    u = torch.cat([u[:, :1] + keep[:, :1] * s["h0"][:, None], u[:, 1:]], 1)
    h = _scan(keep, u)
    return h, h[:, -1]


def _act(p, act):
    return p * _sigmoid(p) if act == "silu" else p


def _dact(p, act):
    if act != "silu":
        return torch.ones_like(p)
    sg = _sigmoid(p)
    return sg * (1 + p * (1 - sg))


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm_fwd":
        h = s["X"].float() if s["residual"] is None else s["X"].float() + s["residual"].float()
        mean = h.mean(-1)
        xc = h - mean[..., None]
        rstd = 1 / torch.sqrt((xc * xc).mean(-1) + 1e-5)
        y = xc * rstd[..., None] * s["weight"][:, None] + s["bias"][:, None]
        y = y.transpose(1, 2).contiguous() if c["token_major"] else y
        return dict(Y=y.to(_dt(c)), S=None if s["residual"] is None else h.to(_dt(c)),
                    mean=mean, rstd=rstd)
    if op == "norm_bwd":
        dy = s["dY"].float()
        dy = dy.transpose(1, 2) if c["token_major"] else dy
        xh = (s["X"].float() - s["mean"][..., None]) * s["rstd"][..., None]
        g = dy * s["weight"][:, None]
        dx = s["rstd"][..., None] * (g - g.mean(-1, keepdim=True)
                                     - xh * (g * xh).mean(-1, keepdim=True))
        dx = dx if s["dS"] is None else dx + s["dS"].float()
        return dict(dX=dx.to(_dt(c)), dweight=(dy * xh).sum((0, 2)), dbias=dy.sum((0, 2)))
    if op == "recur_fwd":
        h, last = _recur_plain(s)
        return dict(Hs=h.to(_dt(c)), h_final=last.contiguous())
    if op == "recur_bwd":
        keep, a, _ = _gates(s)
        dh = s["dH"].float()
        dh = torch.cat([dh[:, :-1], dh[:, -1:] + s["dh_final"][:, None]], 1)
        # the adjoint runs backwards: D_t = dH_t + a_{t+1} D_{t+1}
        nxt = torch.cat([keep[:, 1:], torch.zeros_like(keep[:, :1])], 1)
        D = _scan(nxt.flip(1), dh.flip(1)).flip(1)
        prev = torch.cat([s["h0"][:, None], s["Hs"].float()[:, :-1]], 1)
        if s["reset"] is not None:
            prev = torch.where(s["reset"][..., None] != 0, torch.zeros_like(prev), prev)
        dh0 = keep[:, 0] * D[:, 0]
        if c["gate"] == "sigmoid":
            na = _sigmoid(-s["G"].float())
            return dict(dX=(D * na).to(_dt(c)),
                        dG=(D * (prev - s["X"].float()) * a * na).to(_dt(c)), dh0=dh0)
        return dict(dX=D.to(_dt(c)), dG=D * prev, dh0=dh0)
    if op == "recur_step":
        slots, st, y = s["slots"].long(), s["state"], s["out"]["Y"]
        live = torch.nonzero(slots >= 0)[:, 0]
        keep, _, u = _gates(s)
        h = keep[live] * st[slots[live]] + u[live]
        st[slots[live]] = h
        y[live] = h.to(y.dtype)
        return dict(Y=y, state=st)
    x, w = s["X"].float(), s["W"].float()
    if op == "linear_fwd":
        p = x @ w.t()
        p = p if s["bias"] is None else p + s["bias"]
        y = _act(p, c["act"])
        y = y if s["mul"] is None else y * s["mul"].float()
        y = y if s["residual"] is None else y + s["residual"].float()
        return dict(Y=y.to(BF16))
    dy = s["dY"].float()
    dp, dmul = dy, None
    if s["P"] is not None:
        p = s["P"].float()
        dmul = None if s["mul"] is None else (dy * _act(p, c["act"])).to(BF16)
        dp = dy * _dact(p, c["act"])
        dp = dp if s["mul"] is None else dp * s["mul"].float()
    return dict(dX=(dp @ w).to(BF16), dW=(dp.t() @ x).to(BF16),
                dbias=dp.sum(0) if c["bias"] else None, dmul=dmul)


# ------------------------------------------------------------------------- the library's calls
def _plan(s):
    """The config and the workspace a program makes once for its shapes and keeps."""
    if "plan" not in s:
        import weight_sequence_layers_b200 as ttt
        c, cfg, n = s["case"], None, 0
        op = c["op"]
        if op.startswith("norm"):
            cfg = ttt.make_norm_config(c["B"], c["H"], c["T"], c["d"], c["dtype"],
                                       c["token_major"], 1e-5)
            n = ttt.ttt_norm_bwd_workspace_bytes(cfg) if op == "norm_bwd" else 0
        elif op.startswith("recur"):
            cfg = ttt.make_recur_config(c["B"], c.get("T", 1), c["D"], c["dtype"], c["gate"])
        else:
            n = ttt.ttt_linear_workspace_bytes(c["M"], c["N"], c["K"], op == "linear_bwd")
        ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
        s["plan"] = (ttt, cfg, ws, n)
    return s["plan"]


def _run_own(s):
    ttt, cfg, ws, n = _plan(s)
    c, o = s["case"], s["out"]
    op = c["op"]
    if op == "norm_fwd":
        ttt.ttt_norm_fwd(cfg, s["X"], s["residual"], s["weight"], s["bias"], o["Y"], o["S"],
                         o["mean"], o["rstd"])
    elif op == "norm_bwd":
        ttt.ttt_norm_bwd(cfg, s["X"], s["weight"], s["mean"], s["rstd"], s["dY"], s["dS"],
                         o["dX"], o["dweight"], o["dbias"], ws, n)
    elif op == "recur_fwd":
        ttt.ttt_recur_fwd(cfg, s["X"], s["G"], s["reset"], s["h0"], o["Hs"], o["h_final"])
    elif op == "recur_bwd":
        ttt.ttt_recur_bwd(cfg, s["X"], s["G"], s["reset"], s["h0"], s["Hs"], s["dH"],
                          s["dh_final"], o["dX"], o["dG"], o["dh0"])
    elif op == "recur_step":
        ttt.ttt_recur_step(cfg, s["X"], s["G"], s["slots"], s["state"], o["Y"])
        return dict(Y=o["Y"], state=s["state"])
    elif op == "linear_fwd":
        ttt.ttt_linear_fwd(c["M"], c["N"], c["K"], c["act"], s["X"], s["W"], s["bias"], s["mul"],
                           s["residual"], o["Y"], None, ws, n)
    else:
        ttt.ttt_linear_bwd(c["M"], c["N"], c["K"], c["act"], s["X"], s["W"], s["P"], s["mul"],
                           s["dY"], o["dX"], o["dW"], o["dbias"], o["dmul"], ws, n)
    return dict(o)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op.startswith("norm"):
        rows, es = case["B"] * case["H"] * case["T"], 2 if case["dtype"] == "bf16" else 4
        n, wd = rows * case["d"], case["H"] * case["d"]
        if op == "norm_fwd":  # x, y (and the residual and the sum), weight and bias, mean and rstd
            return dict(bytes=n * es * (4 if case["residual"] else 2) + 8 * wd + 8 * rows,
                        flops=8 * n)
        # x, dy, dx (and the stream's gradient), weight, mean and rstd, the two weight gradients
        return dict(bytes=n * es * (4 if case["residual"] else 3) + 12 * wd + 8 * rows,
                    flops=14 * n)
    if op.startswith("recur"):
        es = 2 if case["dtype"] == "bf16" else 4
        gs = es if case["gate"] == "sigmoid" else 4
        n, bd = case["B"] * case.get("T", 1) * case["D"], case["B"] * case["D"]
        r = case["B"] * case.get("T", 1) if case.get("docs") else 0
        if op == "recur_step":  # x, gate, y, the live sequences' states in and out, slots
            live = case["B"] - (case["B"] // 8 if case["B"] >= 8 else 0)
            return dict(bytes=live * case["D"] * (2 * es + gs + 8) + 4 * case["B"], flops=6 * n)
        if op == "recur_fwd":  # x, gate, h; h0 and h_final
            return dict(bytes=n * (2 * es + gs) + 8 * bd + r, flops=6 * n)
        # gate twice (in, gradient), h, dh, dx, and x with the sigmoid; h0, dh_final, dh0
        return dict(bytes=n * (3 * es + 2 * gs + (es if case["gate"] == "sigmoid" else 0))
                    + 12 * bd + r, flops=12 * n)
    M, N, K = case["M"], case["N"], case["K"]
    if op == "linear_fwd":
        return dict(bytes=2 * (M * K + N * K + M * N * (1 + case["mul"] + case["residual"]))
                    + 4 * N * case["bias"], flops=2 * M * N * K)
    p = case["act"] != "id" or case["mul"]
    return dict(bytes=2 * (2 * M * K + 2 * N * K + M * N * (1 + p + 2 * case["mul"]))
                + 4 * N * case["bias"], flops=4 * M * N * K)


# ------------------------------------------------------------------------------------- exact
def _sig64(x):
    return torch.where(x >= 0, 1 / (1 + torch.exp(-x.abs())),
                       torch.exp(-x.abs()) / (1 + torch.exp(-x.abs())))


def exact(case, seed):
    """The operators from their definitions in 64 bits, token by token where they recur."""
    s = prepare(case, seed)
    op, f = case["op"], torch.float64
    d = {k: v.to(f) for k, v in s.items()
         if isinstance(v, torch.Tensor) and v.dtype in (BF16, F32)}
    if op.startswith("norm"):
        h = d["X"] + d["residual"] if "residual" in d else d["X"]
        w, b = d["weight"].unsqueeze(1), d["bias"].unsqueeze(1)
        n = case["d"]
        if op == "norm_fwd":
            mean = h.sum(-1) / n
            var = ((h - mean.unsqueeze(-1)) ** 2).sum(-1) / n
            rstd = (var + 1e-5) ** -0.5
            y = (h - mean.unsqueeze(-1)) * rstd.unsqueeze(-1) * w + b
            if case["token_major"]:
                y = y.permute(0, 2, 1, 3).contiguous()
            return dict(Y=y, S=h if "residual" in d else None, mean=mean, rstd=rstd)
        dy = d["dY"].permute(0, 2, 1, 3) if case["token_major"] else d["dY"]
        r = d["rstd"].unsqueeze(-1)
        xh = (h - d["mean"].unsqueeze(-1)) * r
        # y = w xh + b with xh = (x - mean) r: the adjoint of xh, then of x through mean and r
        dxh = dy * w
        dx = r * dxh - r / n * dxh.sum(-1, keepdim=True) - r / n * xh * (dxh * xh).sum(-1, keepdim=True)
        if "dS" in d:
            dx = dx + d["dS"]
        return dict(dX=dx, dweight=torch.einsum("bhtd,bhtd->hd", dy, xh),
                    dbias=torch.einsum("bhtd->hd", dy))
    if op.startswith("recur"):
        if case["gate"] == "sigmoid":
            a, na = _sig64(d["G"]), _sig64(-d["G"])
        else:
            a, na = d["G"], torch.ones_like(d["G"])
        if op == "recur_step":
            live = s["slots"] >= 0
            at = s["slots"][live].long()
            new = a[live] * d["state"][at] + na[live] * d["X"][live]
            state, y = d["state"].clone(), torch.zeros_like(d["X"])
            state[at], y[live] = new, new
            return dict(Y=y, state=state)
        B, T, D = d["X"].shape
        keep = torch.ones((B, T, 1), dtype=f, device="cuda")
        if s["reset"] is not None:
            keep = (s["reset"] == 0).to(f).unsqueeze(-1)
        ak = a * keep
        if op == "recur_fwd":
            u = na * d["X"]
            h, hs = d["h0"], torch.empty_like(u)
            for t in range(T):
                h = torch.addcmul(u[:, t], ak[:, t], h)
                hs[:, t] = h
            return dict(Hs=hs, h_final=h)
        carry = d["dh_final"]
        Ds = torch.empty_like(a)
        for t in range(T - 1, -1, -1):
            adj = d["dH"][:, t] + carry
            Ds[:, t] = adj
            carry = ak[:, t] * adj
        prev = torch.empty_like(a)
        prev[:, 0], prev[:, 1:] = d["h0"], d["Hs"][:, :-1]
        prev = prev * keep
        if case["gate"] == "sigmoid":
            # h = a prev + (1 - a) x, a = sigmoid(g): dh/dg = (prev - x) a (1 - a)
            return dict(dX=Ds * na, dG=Ds * (prev - d["X"]) * a * na, dh0=carry)
        return dict(dX=Ds, dG=Ds * prev, dh0=carry)
    silu = case["act"] == "silu"
    if op == "linear_fwd":
        p = d["X"] @ d["W"].T
        if "bias" in d:
            p += d["bias"]
        if silu:
            p *= _sig64(p)
        if "mul" in d:
            p *= d["mul"]
        if "residual" in d:
            p += d["residual"]
        return dict(Y=p)
    dp, dmul = d["dY"], None
    if "P" in d:
        p = d["P"]
        sg = _sig64(p) if silu else torch.ones_like(p)
        if "mul" in d:
            dmul = dp * p * sg
            dp = dp * d["mul"]
        if silu:
            dp = dp * (sg + p * sg * (1 - sg))
    return dict(dX=dp @ d["W"], dW=dp.T @ d["X"], dbias=dp.sum(0) if case["bias"] else None,
                dmul=dmul)
