"""The gated linear recurrence on the GPU against its definition in 64 bits, token by token."""
import pytest
import torch

import weight_sequence_layers_b200 as ttt
from _block import DT, F64, U32, Out, assert_within, randn, rng, sync_ok

pytestmark = pytest.mark.gpu

# Roundings charged to one token, relative to |a h_{t-1}| + |u_t|: the gate's exponential (2
# ulp + 1 per unit of the logit's size, |logit| < 12 here: 32 U32), its sum, quotient and
# product (8 U32), the recurrence's own (2 U32), and one token's part of the roundings of the
# partial products that join segments (a token's map enters at most 64 products or joins).
K = 110


def case(B, T, D, dtype, gate, reset=None, h0=True, seed=0):
    g, dt = rng(seed), DT[dtype]
    c = dict(B=B, T=T, D=D, dt=dt, sig=gate == "sigmoid",
             cfg=ttt.make_recur_config(B, T, D, dtype, gate), X=randn(g, B, T, D, dtype=dt))
    if gate == "sigmoid":
        c["G"] = randn(g, B, T, D, mean=2.0, dtype=dt)
    else:
        c["G"] = torch.sigmoid(randn(g, B, T, D, mean=3.0, std=0.5))
        c["G"][torch.rand((B, T, D), generator=g, device="cuda") < 0.01] = 0.0
        c["G"][torch.rand((B, T, D), generator=g, device="cuda") < 0.01] = 1.0
    if reset is None:
        c["reset"] = None
    else:
        c["reset"] = (torch.rand((B, T), generator=g, device="cuda") < reset).to(torch.uint8) * 3
    c["h0"] = randn(g, B, D) if h0 else None
    c["dH"], c["dh_final"] = randn(g, B, T, D, dtype=dt), randn(g, B, D) if h0 else None
    return c


def gates(c):
    G = c["G"].to(F64)
    a = torch.sigmoid(G) if c["sig"] else G
    na = torch.sigmoid(-G) if c["sig"] else torch.ones_like(G)
    keep = torch.ones((c["B"], c["T"], 1), dtype=F64, device="cuda")
    if c["reset"] is not None:
        keep = (c["reset"] == 0).to(F64)[..., None]
    return a, na, a * keep, keep


def zeros_bd(c):
    return torch.zeros((c["B"], c["D"]), dtype=F64, device="cuda")


def forward(c, final=True):
    H = Out(c["B"], c["T"], c["D"], dtype=c["dt"])
    hf = Out(c["B"], c["D"]) if final else None
    ttt.ttt_recur_fwd(c["cfg"], c["X"], c["G"], c["reset"], c["h0"], H.t, hf and hf.t)
    sync_ok()
    return H.check(), hf and hf.check()


def reference(c):
    a, na, ak, _ = gates(c)
    u = na * c["X"].to(F64)
    h = c["h0"].to(F64) if c["h0"] is not None else zeros_bd(c)
    err, hs, es = zeros_bd(c), [], []
    for t in range(c["T"]):
        err = ak[:, t] * err + K * U32 * ((ak[:, t] * h).abs() + u[:, t].abs())
        h = ak[:, t] * h + u[:, t]
        hs.append(h)
        es.append(err)
    return torch.stack(hs, 1), torch.stack(es, 1)


def check_forward(c):
    H, hf = forward(c)
    h, e = reference(c)
    assert_within("H", H, h, e)
    assert_within("h_final", hf, h[:, -1], e[:, -1])
    again, _ = forward(c, final=False)
    assert torch.equal(again, H)  # a fixed order of sums
    return H


def check_backward(c, H):
    dX, dG = Out(c["B"], c["T"], c["D"], dtype=c["dt"]), Out(c["B"], c["T"], c["D"],
                                                             dtype=c["G"].dtype)
    dh0 = Out(c["B"], c["D"])
    ttt.ttt_recur_bwd(c["cfg"], c["X"] if c["sig"] else None, c["G"], c["reset"], c["h0"], H,
                      c["dH"], c["dh_final"], dX.t, dG.t, dh0.t)
    sync_ok()
    a, na, ak, keep = gates(c)
    dH, X = c["dH"].to(F64), c["X"].to(F64)
    carry = c["dh_final"].to(F64) if c["dh_final"] is not None else zeros_bd(c)
    err, Ds, es = zeros_bd(c), [None] * c["T"], [None] * c["T"]
    for t in range(c["T"] - 1, -1, -1):
        Ds[t] = dH[:, t] + carry
        es[t] = err + 2 * U32 * (dH[:, t].abs() + carry.abs())
        err = ak[:, t] * (es[t] + K * U32 * (dH[:, t].abs() + carry.abs()))
        carry = ak[:, t] * Ds[t]
    D, e = torch.stack(Ds, 1), torch.stack(es, 1)
    h0 = c["h0"].to(F64) if c["h0"] is not None else zeros_bd(c)
    prev = torch.cat([h0[:, None], H.to(F64)[:, :-1]], 1) * keep
    if c["sig"]:
        assert_within("dX", dX.check(), na * D, na * e + 50 * U32 * (na * D).abs())
        s = (prev - X) * a * na
        assert_within("dG", dG.check(), D * s, e * s.abs() + 100 * U32 * (D * s).abs())
    else:
        assert_within("dX", dX.check(), D, e)
        assert_within("dG", dG.check(), D * prev, e * prev.abs() + 2 * U32 * (D * prev).abs())
    assert_within("dh0", dh0.check(), carry, err)
    dX2, dG2 = torch.empty_like(dX.t), torch.empty_like(dG.t)
    ttt.ttt_recur_bwd(c["cfg"], c["X"], c["G"], c["reset"], c["h0"], H, c["dH"], c["dh_final"],
                      dX2, dG2)
    sync_ok()
    assert torch.equal(dX2, dX.t) and torch.equal(dG2, dG.t)


def check(c):
    check_backward(c, check_forward(c).clone())


KINDS = [("bf16", "sigmoid"), ("bf16", "decay"), ("f32", "sigmoid"), ("f32", "decay")]


@pytest.mark.parametrize("dtype,gate", KINDS)
@pytest.mark.parametrize("T", [1, 2, 3, 4, 7, 8, 9, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257,
                               511, 512, 513, 1000, 1025, 2049])
def test_lengths(T, dtype, gate):
    check(case(2, T, 70, dtype, gate, seed=T))


@pytest.mark.parametrize("dtype,gate", KINDS)
@pytest.mark.parametrize("D", [1, 2, 3, 4, 6, 8, 15, 31, 32, 34, 63, 64, 65, 66, 127, 128, 129, 130,
                               200, 256, 264, 1021])
def test_widths(D, dtype, gate):
    check(case(3, 150, D, dtype, gate, seed=D, reset=0.05))


@pytest.mark.parametrize("dtype,gate", KINDS)
@pytest.mark.parametrize("B,T,D", [(1, 700, 2560), (8, 300, 1024), (40, 70, 512), (3, 1537, 1021),
                                   (1, 6000, 64), (5, 900, 2050), (1, 9000, 8), (150, 5, 300)])
def test_shapes(B, T, D, dtype, gate):
    check(case(B, T, D, dtype, gate, seed=B, reset=0.01))


@pytest.mark.parametrize("dtype,gate", KINDS)
@pytest.mark.parametrize("reset", [0.0, 0.02, 0.5, 1.0])
@pytest.mark.parametrize("T", [1, 65, 1100])
def test_resets(T, reset, dtype, gate):
    check(case(2, T, 130, dtype, gate, seed=7, reset=reset))
    check(case(2, T, 130, dtype, gate, seed=7, reset=reset, h0=False))


@pytest.mark.parametrize("dtype,gate", KINDS)
@pytest.mark.parametrize("D", [64, 65])
def test_nothing_crosses_a_reset(D, dtype, gate):
    # infinities and NaN before a document's start do not reach it, nor, backwards, the document
    # before; a reset on the first token drops h0 and gives dh0 = 0
    B, T = 2, 900
    cut = [0, 1, 64, 65, 200, 511, 512, 899]
    for at in cut:
        c = case(B, T, D, dtype, gate, seed=at)
        c["reset"] = torch.zeros((B, T), dtype=torch.uint8, device="cuda")
        c["reset"][0, at] = 255
        clean = case(B, T, D, dtype, gate, seed=at)
        clean["reset"] = c["reset"]
        c["h0"][0] = float("inf")
        if at:
            c["X"][0, at - 1, ::2] = float("nan")
            c["X"][0, at // 2, 1::2] = float("inf")
        H, hf = forward(c)
        Hc, hfc = forward(clean)
        assert torch.equal(H[0, at:], Hc[0, at:]) and torch.equal(H[1], Hc[1])
        assert torch.equal(hf, hfc)
        for k in ("dh_final",):
            c[k] = clean[k].clone()
        c["dH"] = clean["dH"].clone()
        c["dH"][0, at] = float("nan")
        dX, dG, dh0 = torch.empty_like(c["X"]), torch.empty_like(c["G"]), torch.empty_like(c["h0"])
        ttt.ttt_recur_bwd(c["cfg"], clean["X"], c["G"], c["reset"], clean["h0"], Hc, c["dH"],
                          c["dh_final"], dX, dG, dh0)
        dXc, dGc, dh0c = torch.empty_like(dX), torch.empty_like(dG), torch.empty_like(dh0)
        ttt.ttt_recur_bwd(c["cfg"], clean["X"], c["G"], c["reset"], clean["h0"], Hc, clean["dH"],
                          c["dh_final"], dXc, dGc, dh0c)
        sync_ok()
        for got, want in ((dX, dXc), (dG, dGc)):
            assert torch.equal(got[0, :at], want[0, :at]) and torch.equal(got[1], want[1])
            assert torch.equal(got[0, at + 1:], want[0, at + 1:])
        assert torch.equal(dh0, dh0c)
        if at == 0:
            assert not dh0[0].any()


@pytest.mark.parametrize("dtype,gate", KINDS)
def test_two_calls_with_the_state_carried_equal_one_call(dtype, gate):
    c = case(2, 700, 96, dtype, gate, seed=21, reset=0.01)
    H, hf = [o.clone() for o in forward(c)]
    cut = 333
    parts, h = [], c["h0"].clone()
    for lo, hi in ((0, cut), (cut, 700)):
        p = dict(c, T=hi - lo, cfg=ttt.make_recur_config(2, hi - lo, 96, dtype, gate))
        for k in ("X", "G", "reset"):
            p[k] = c[k][:, lo:hi].contiguous()
        Hp = torch.empty_like(p["X"])
        ttt.ttt_recur_fwd(p["cfg"], p["X"], p["G"], p["reset"], h, Hp, h)  # the state in place
        parts.append(Hp)
    sync_ok()
    h64, e = reference(c)
    assert_within("H", torch.cat(parts, 1), h64, e)
    assert_within("h_final", h, h64[:, -1], e[:, -1])


@pytest.mark.parametrize("gate", ["sigmoid", "decay"])
def test_saturated_gates(gate):
    # gates that are 0 or 1 to the last bit, tiny and huge logits
    c = case(1, 300, 64, "f32", gate, seed=4)
    if gate == "sigmoid":
        vals = torch.tensor([-200.0, -88.0, -20.0, 0.0, 20.0, 88.0, 200.0, 1e30], device="cuda")
    else:
        vals = torch.tensor([0.0, 1e-38, 1e-20, 0.5, 1.0, 1.0, 1.0, 1.0], device="cuda")
    c["G"] = vals[torch.randint(0, 8, (1, 300, 64), generator=rng(3), device="cuda")]
    H, hf = forward(c)
    a, na, ak, _ = gates(c)
    h = c["h0"].to(F64)
    u = na * c["X"].to(F64)
    err = zeros_bd(c)
    for t in range(300):
        # |logit| up to 200: the exponential's relative error grows to 236 ulp, where it is 1e-38
        # and below; 300 U32 covers every logit
        err = ak[:, t] * err + 400 * U32 * ((ak[:, t] * h).abs() + u[:, t].abs())
        h = ak[:, t] * h + u[:, t]
        assert_within("H", H[:, t], h, err + 1e-37)


def test_gradient_against_differences():
    # J = <dH, H> + <dh_final, h_final> along random directions, in 64 bits around the inputs;
    # step 1e-5 leaves 1e-9 of J's scale, the float32 gradients 1e-5 of it (K U32 per token over
    # a memory of up to 50 tokens would be 4e-4 at worst; rounding errors of mixed sign average
    # to under a tenth of that over 11,000 entries)
    for gate in ("sigmoid", "decay"):
        c = case(2, 90, 61, "f32", gate, seed=31, reset=0.05)
        H, _ = forward(c)
        dX, dG, dh0 = torch.empty_like(c["X"]), torch.empty_like(c["G"]), torch.empty_like(c["h0"])
        ttt.ttt_recur_bwd(c["cfg"], c["X"], c["G"], c["reset"], c["h0"], H, c["dH"],
                          c["dh_final"], dX, dG, dh0)
        sync_ok()

        def J(X, G, h0):
            p = dict(c, X=X, G=G, h0=h0)
            a, na, ak, _ = gates(p)
            h, total = h0, 0.0
            for t in range(c["T"]):
                h = ak[:, t] * h + na[:, t] * X[:, t]
                total = total + (c["dH"][:, t].to(F64) * h).sum()
            return float(total + (c["dh_final"].to(F64) * h).sum())

        g, s = rng(32), 1e-5
        at = [c["X"].to(F64), c["G"].to(F64), c["h0"].to(F64)]
        for k, grad in enumerate((dX, dG, dh0)):
            v = randn(g, *grad.shape).to(F64)
            up, dn = list(at), list(at)
            up[k], dn[k] = at[k] + s * v, at[k] - s * v
            num, ana = (J(*up) - J(*dn)) / (2 * s), float((grad.to(F64) * v).sum())
            scale = float((grad.to(F64) * v).abs().sum())
            assert abs(num - ana) <= 4e-5 * scale, (gate, k, num, ana, scale)


@pytest.mark.parametrize("gate", ["sigmoid", "decay"])
def test_more_than_2_31_elements(gate):
    # the last tokens sit past 32-bit element offsets; each token is checked against its own
    # predecessor as the kernel wrote it
    D, T = 4096, (1 << 19) + 70
    cfg = ttt.make_recur_config(1, T, D, "bf16", gate)
    X = torch.empty((T, D), device="cuda", dtype=torch.bfloat16).normal_(generator=rng(1))
    if gate == "sigmoid":
        G = torch.empty((T, D), device="cuda", dtype=torch.bfloat16).normal_(2, 1, generator=rng(2))
    else:
        G = torch.full((T, D), 0.9, device="cuda")
    H = torch.empty_like(X)
    hf = torch.empty(D, device="cuda")
    ttt.ttt_recur_fwd(cfg, X, G, None, None, H, hf)
    sync_ok()
    tail = slice(T - 200, T)
    a = torch.sigmoid(G[tail].to(F64)) if gate == "sigmoid" else G[tail].to(F64)
    u = (torch.sigmoid(-G[tail].to(F64)) if gate == "sigmoid" else 1.0) * X[tail].to(F64)
    prev = H[T - 201:T - 1].to(F64)
    # h_{t-1} is known to half a bf16 step
    assert_within("H", H[tail], a * prev + u, 2.0 ** -8 * (a * prev).abs() + 2 * K * U32 * 8)
    dX, dG = torch.empty_like(X), torch.empty_like(G)
    ttt.ttt_recur_bwd(cfg, X, G, None, None, H, X, None, dX, dG)
    sync_ok()
    c = zeros = torch.zeros(D, dtype=F64, device="cuda")
    for t in range(T - 1, T - 100, -1):
        Dt = X[t].to(F64) + c
        at = a[t - T]
        if gate == "sigmoid":
            na = torch.sigmoid(-G[t].to(F64))
            assert_within("dX", dX[t], Dt * na, 1e-4 * torch.ones_like(zeros))
        else:
            assert_within("dX", dX[t], Dt, 1e-4 * torch.ones_like(zeros))
            assert_within("dG", dG[t], Dt * H[t - 1].to(F64), 1e-3 * torch.ones_like(zeros))
        c = at * Dt


# ------------------------------------------------------------------------------------- step
def step_case(B, D, S, dtype, gate, seed=0):
    c = case(B, 1, D, dtype, gate, seed=seed)
    g = rng(seed + 1)
    c["X"], c["G"] = c["X"][:, 0].contiguous(), c["G"][:, 0].contiguous()
    c["state"] = randn(g, S, D)
    c["slots"] = torch.randperm(S, generator=g, device="cuda")[:B].to(torch.int32)
    return c


def step_reference(c, slots):
    """Rows in order, in 64 bits; returns Y (NaN where a row is skipped), the states and bounds."""
    G, X = c["G"].to(F64), c["X"].to(F64)
    a = torch.sigmoid(G) if c["sig"] else G
    na = torch.sigmoid(-G) if c["sig"] else torch.ones_like(G)
    st, err = c["state"].to(F64).clone(), torch.zeros_like(c["state"], dtype=F64)
    Y, E = torch.full_like(X, float("nan")), torch.zeros_like(X)
    for b, sl in enumerate(slots):
        if 0 <= sl < st.shape[0]:
            err[sl] = a[b] * err[sl] + K * U32 * ((a[b] * st[sl]).abs() + (na[b] * X[b]).abs())
            st[sl] = a[b] * st[sl] + na[b] * X[b]
            Y[b], E[b] = st[sl], err[sl]
    return Y, E, st, err


def run_step(c, slots):
    S, D = c["state"].shape
    st, Y = Out(S, D), Out(c["B"], D, dtype=c["dt"])
    st.t.copy_(c["state"])
    ttt.ttt_recur_step(c["cfg"], c["X"], c["G"], slots, st.t, Y.t)
    torch.cuda.synchronize()
    return st.check(), Y.check()


def check_step(c, slots, use=True):
    st, Y = run_step(c, slots if use else None)
    lst = slots.tolist() if use else list(range(c["B"]))
    Yr, E, sr, err = step_reference(c, lst)
    live = ~torch.isnan(Yr[:, 0])
    assert bool(torch.isnan(Y[~live].float()).all())  # a skipped row is left as it was
    assert_within("Y", Y[live], Yr[live], E[live])
    assert_within("state", st, sr, err)
    touched = sorted({s for s in lst if 0 <= s < st.shape[0]})
    rest = [s for s in range(st.shape[0]) if s not in set(touched)]
    assert torch.equal(st[rest], c["state"][rest])


@pytest.mark.parametrize("dtype,gate", KINDS)
@pytest.mark.parametrize("B,D,S", [(1, 1, 1), (1, 64, 3), (3, 65, 7), (8, 2560, 8), (64, 1024, 96),
                                   (257, 130, 300), (700, 33, 1000)])
def test_step(B, D, S, dtype, gate):
    c = step_case(B, D, S, dtype, gate, seed=B)
    check_step(c, c["slots"])
    check_step(c, c["slots"], use=False)
    s = c["slots"].clone()
    s[::3] = -1
    s[1::7] = -2 ** 31
    check_step(c, s)
    sync_ok()


@pytest.mark.parametrize("dtype,gate", KINDS)
@pytest.mark.parametrize("D", [65, 1024])
def test_step_rows_of_one_slot_are_applied_in_order(D, dtype, gate):
    c = step_case(40, D, 50, dtype, gate, seed=3)
    s = c["slots"].clone()
    s[3] = s[1] = s[30]
    s[5:9] = s[20]
    s[39] = s[0]
    s[10] = -1
    check_step(c, s)
    check_step(c, torch.full_like(s, 7))
    sync_ok()


def test_step_slot_out_of_range_is_recorded_and_skipped():
    c = step_case(6, 64, 9, "bf16", "sigmoid", seed=9)
    s = c["slots"].clone()
    s[2], s[4] = 9, 2 ** 31 - 1
    check_step(c, s)
    assert ttt.ttt_get_device_error() == ttt.ERR_RANGE
    assert ttt.ttt_get_device_error() == ttt.OK


@pytest.mark.parametrize("dtype,gate", KINDS)
def test_steps_equal_the_forward(dtype, gate):
    B, T, D = 5, 40, 192
    c = case(B, T, D, dtype, gate, seed=14)
    cfg = ttt.make_recur_config(B, 1, D, dtype, gate)
    st, Y = c["h0"].clone(), torch.empty((T, B, D), dtype=c["dt"], device="cuda")
    for t in range(T):
        ttt.ttt_recur_step(cfg, c["X"][:, t].contiguous(), c["G"][:, t].contiguous(), None, st, Y[t])
    sync_ok()
    h, e = reference(c)
    assert_within("Y", Y.transpose(0, 1), h, e)
    assert_within("state", st, h[:, -1], e[:, -1])


@pytest.mark.parametrize("dtype,gate", KINDS)
@pytest.mark.parametrize("B,T,D", [(1, 4001, 1), (1, 2999, 63), (5, 777, 129), (2, 2300, 70), (1, 1100, 2562),
                                   (9, 130, 2049)])
def test_long_sequences_of_odd_widths(B, T, D, dtype, gate):
    # clusters along the sequence, rows that start inside a 4- or 16-byte word, a last round that
    # some CTAs have no token of
    check(case(B, T, D, dtype, gate, seed=T, reset=0.003))


# Decays above one, over stretches whose product leaves float32's range (up to 1e300) while every
# state stays in it: zero states over a padded prefix, tiny states, growth after decay. All terms
# are positive, so that a token's roundings stay relative to the state and K covers them as above.
GROWTH = ["zero prefix", "tiny state", "decay then growth", "growth then decay", "huge decays"]


def growth_case(kind, B, T, D, dtype, seed=0):
    c = case(B, T, D, dtype, "decay", seed=seed)
    c["X"], c["dH"] = c["X"].abs(), c["dH"].abs()
    c["h0"] = c["dh_final"] = None
    G = 0.5 + 0.4 * torch.rand((B, T, D), generator=rng(seed + 1), device="cuda")
    third = max(T // 3, 1)
    if kind in ("zero prefix", "huge decays"):
        # features differ, and some never grow
        big = torch.tensor([2.0, 1.1, 0.9, 1e20 if kind == "huge decays" else 8.0], device="cuda")
        lo, hi = third, T - third
        G[:, :lo] = big[torch.arange(D, device="cuda") % 4]
        G[:, hi:] = big[torch.arange(D, device="cuda") % 4]
        c["X"][:, :lo], c["X"][:, hi:] = 0, 0
        c["dH"][:, :lo], c["dH"][:, hi:] = 0, 0
        G[:, lo], G[:, hi] = 0.0, 0.0  # no adjoint enters the first third, no state the last
    else:
        n = min(T, 180)
        up = torch.where(torch.arange(D, device="cuda") % 3 == 0, 2.0, 1.5)
        c["X"][:, :n] = 0
        c["dH"] *= 1e-30
        if kind == "tiny state":       # 1e-30 grows by up to 2^150
            G[:, :min(n, 150)] = up
            c["h0"] = torch.full((B, D), 1e-30, device="cuda")
        elif kind == "decay then growth":
            G[:, :n // 2], G[:, n // 2:n] = 1 / up, up
            c["h0"] = torch.full((B, D), 3.0, device="cuda")
        else:
            G[:, :n // 2], G[:, n // 2:n] = up, 1 / up
            c["h0"] = torch.full((B, D), 3.0, device="cuda")
    c["G"] = G
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", GROWTH)
@pytest.mark.parametrize("B,T,D", [(2, 100, 64), (1, 700, 65), (2, 1500, 70), (1, 2600, 33),
                                   (40, 200, 130), (1, 900, 1021)])
def test_decays_above_one(B, T, D, kind, dtype):
    c = growth_case(kind, B, T, D, dtype, seed=T)
    h, _ = reference(c)
    assert float(h.abs().max()) < 1e38  # the states stay in range: the kernel's have to
    check(c)
    # a document's start inside a stretch of growth
    c["reset"] = torch.zeros((B, T), dtype=torch.uint8, device="cuda")
    c["reset"][:, T // 5] = 1
    c["reset"][:, T - T // 5] = 1
    check(c)


def test_growth_of_one_sequence_leaves_the_others_alone():
    # sequences (and features) are independent: one that grows changes no bit of the rest
    c = case(3, 1300, 96, "f32", "decay", seed=2)
    H, hf = [o.clone() for o in forward(c)]
    c["G"][1], c["X"][1], c["h0"][1] = 2.0, 0.0, 0.0
    H2, hf2 = forward(c)
    for b in (0, 2):
        assert torch.equal(H2[b], H[b]) and torch.equal(hf2[b], hf[b])
    assert not H2[1].any() and not hf2[1].any()


def test_float32_gates_keep_float32():
    # A token's roundings with float32 logits do not grow with the logit: the exponential 5 U32 (two
    # float32 steps of the hardware's and a multiply-add), the sum 1, the reciprocal 2 (one step), the
    # gate's product 1 and the recurrence 1: 10 U32 for either gate; 24 U32 for the two of them with
    # the difference and the products of dG (the exponential enters a (1 - a) with a factor below 1).
    # X = 1 from a zero state gives 1 - a, X = 0 from a state of 1 gives a.
    D = 4096
    G = torch.linspace(-86, 86, D, device="cuda")
    G = torch.cat([G, torch.tensor([-0.0, 0.0, 1e-3, -1e-3, 30.25, -30.25, 5.5, -5.5], device="cuda")])
    D = G.numel()
    cfg = ttt.make_recur_config(1, 1, D, "f32", "sigmoid")
    g = G.to(F64)
    a, na = torch.sigmoid(g), torch.sigmoid(-g)
    one, zero = torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")
    # (the bounds are relative; assert_within adds half a step and the smallest normal)
    for x, h0, ref in ((one, zero, na), (zero, one, a), (one * 3, one * 5, 3 * na + 5 * a)):
        H, st, Y = Out(1, 1, D), h0.clone().view(1, D), Out(1, D)
        ttt.ttt_recur_fwd(cfg, x, G, None, h0, H.t)
        ttt.ttt_recur_step(cfg, x, G, None, st, Y.t)
        sync_ok()
        assert_within("H", H.check().view(-1), ref, 10 * U32 * ref)
        assert_within("Y", Y.check().view(-1), ref, 10 * U32 * ref)
        dX, dG, dh0 = Out(1, 1, D), Out(1, 1, D), Out(1, D)
        ttt.ttt_recur_bwd(cfg, x, G, None, h0, H.t, one, None, dX.t, dG.t, dh0.t)
        sync_ok()
        assert_within("dX", dX.check().view(-1), na, 10 * U32 * na)
        assert_within("dh0", dh0.check().view(-1), a, 10 * U32 * a)
        s = (h0 - x).to(F64) * a * na
        assert_within("dG", dG.check().view(-1), s, 24 * U32 * s.abs())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_logits(dtype):
    # gates that are exactly open or shut; a NaN logit reaches its own feature only
    inf = float("inf")
    G = torch.tensor([inf, -inf, 1e30, -1e30, 126.0, 127.0, -87.0, float("nan"), 0.0, 200.0],
                     device="cuda").to(DT[dtype])
    D = G.numel()
    X, h0 = torch.full((D,), 2.0, device="cuda").to(DT[dtype]), torch.full((D,), 5.0, device="cuda")
    want = [5, 2, 5, 2, 5, 5, 2, float("nan"), 3.5, 5]
    cfg = ttt.make_recur_config(1, 1, D, dtype, "sigmoid")
    H, Y, st = torch.empty_like(X), torch.empty_like(X), h0.clone().view(1, D)
    ttt.ttt_recur_fwd(cfg, X, G, None, h0, H)
    ttt.ttt_recur_step(cfg, X, G, None, st, Y)
    dX, dG, dh0 = torch.empty_like(X), torch.empty_like(X), torch.empty_like(h0)
    ttt.ttt_recur_bwd(cfg, X, G, None, h0, H, torch.ones_like(X), None, dX, dG, dh0)
    sync_ok()
    for got in (H, Y, st.view(-1)):
        for g, w in zip(got.tolist(), want):
            assert g == w or (g != g and w != w), (got.tolist(), want)
    ok = [i for i in range(D) if i != 7]
    assert torch.isfinite(dX[ok].float()).all() and torch.isfinite(dG[ok].float()).all()
    assert dh0.tolist()[0] == 1.0 and abs(dh0.tolist()[1]) < 1e-37 and dX.tolist()[1] == 1.0
