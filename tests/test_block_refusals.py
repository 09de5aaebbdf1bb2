"""The operators around the layer reject bad arguments on the host before anything is launched
(these run without a GPU), and the binding's structs agree with the header."""
import ctypes
import re

import pytest
import torch

import weight_sequence_layers_b200 as ttt

A = 4096  # a 16-byte aligned address that is never dereferenced on these paths
NAN, INF = float("nan"), float("inf")


def by(c):
    return ctypes.byref(c)


def norm_cfg(**kw):
    base = dict(B=2, H=3, T=5, d=64, dtype="f32", token_major=False, eps=1e-5)
    base.update(kw)
    return ttt.make_norm_config(**base)


def recur_cfg(**kw):
    base = dict(B=2, T=5, D=64, dtype="bf16", gate="sigmoid")
    base.update(kw)
    return ttt.make_recur_config(**base)


@pytest.mark.parametrize("name", ["ttt_norm_config", "ttt_recur_config"])
def test_config_structs_match_the_header(name):
    text = re.sub(r"/\*.*?\*/", " ", open(ttt.HEADER).read(), flags=re.S)
    body = re.findall(r"typedef struct \{([^{}]*)\} " + name + ";", text)[0]
    fields = []
    for decl in body.split(";"):
        words = decl.replace(",", " ").split()
        fields += [(w, words[0]) for w in words[1:]]
    ctype = {"int": ctypes.c_int, "float": ctypes.c_float}
    assert [(n, ctype[t]) for n, t in fields] == list(getattr(ttt, name)._fields_)
    enums = dict(re.findall(r"\b(TTT_GATE_[A-Z]+)\s*=\s*(\d+)", text))
    assert {k: int(enums["TTT_GATE_" + k.upper()]) for k in ttt.GATE} == ttt.GATE


BAD_NORM = [dict(B=0), dict(H=0), dict(T=0), dict(d=0), dict(eps=0.0), dict(eps=-1.0),
            dict(eps=NAN), dict(eps=INF), dict(B=1 << 16, H=1 << 8, T=1 << 7),
            dict(B=1 << 16, H=1 << 16), dict(B=1 << 15, H=1, T=1 << 15, d=16384)]


def norm_fwd(c, *p):
    return ttt.lib.ttt_norm_fwd(by(c), *p, None)


def norm_bwd(c, *p, ws=None, n=0):
    return ttt.lib.ttt_norm_bwd(by(c), *p, ws, n, None)


@pytest.mark.parametrize("bad", BAD_NORM)
def test_norm_config_errors(bad):
    c = norm_cfg(**bad)
    assert norm_fwd(c, A, None, A, A, A, None, A, A) == ttt.ERR_INVALID_ARG
    assert norm_bwd(c, A, A, A, A, A, None, A, A, A, ws=A, n=1 << 40) == ttt.ERR_INVALID_ARG
    with pytest.raises(ttt.TTTError):
        ttt.ttt_norm_bwd_workspace_bytes(c)


def test_norm_argument_errors():
    c = norm_cfg()
    for field, v in (("dtype", 2), ("token_major", 2)):
        bad = norm_cfg()
        setattr(bad, field, v)
        assert norm_fwd(bad, A, None, A, A, A, None, A, A) == ttt.ERR_INVALID_ARG
    assert ttt.lib.ttt_norm_fwd(None, A, None, A, A, A, None, A, A, None) == ttt.ERR_INVALID_ARG
    assert norm_fwd(norm_cfg(d=16385), A, None, A, A, A, None, A, A) == ttt.ERR_UNSUPPORTED
    assert norm_fwd(c, None, None, A, A, A, None, A, A) == ttt.ERR_INVALID_ARG
    assert norm_fwd(c, A, None, A, A, None, None, A, A) == ttt.ERR_INVALID_ARG
    assert norm_fwd(c, A, None, A, A, A, A, A, A) == ttt.ERR_INVALID_ARG  # S without residual
    for i in range(8):
        p = [A] * 8
        p[i] = A + 8
        assert norm_fwd(c, *p) == ttt.ERR_ALIGNMENT, i
    good = [A, A, A, A, A, None, A, A, A]  # S weight mean rstd dY dS dX dweight dbias
    for i in (0, 2, 3, 4, 6):
        p = list(good)
        p[i] = None
        assert norm_bwd(c, *p, ws=A, n=1 << 40) == ttt.ERR_INVALID_ARG, i
    for i in range(9):
        p = [A] * 9
        p[i] = A + 4
        assert norm_bwd(c, *p, ws=A, n=1 << 40) == ttt.ERR_ALIGNMENT, i
    need = ttt.ttt_norm_bwd_workspace_bytes(c)
    if need:
        assert norm_bwd(c, *good, ws=None, n=0) == ttt.ERR_WORKSPACE
        assert norm_bwd(c, *good, ws=A, n=need - 1) == ttt.ERR_WORKSPACE


BAD_RECUR = [dict(B=0), dict(T=0), dict(D=0), dict(B=1 << 16, T=1 << 15),
             dict(B=1 << 10, T=1 << 20, D=1 << 11)]


@pytest.mark.parametrize("bad", BAD_RECUR)
def test_recur_config_errors(bad):
    c = recur_cfg(**bad)
    assert ttt.lib.ttt_recur_fwd(by(c), A, A, A, A, A, A, None) == ttt.ERR_INVALID_ARG
    assert ttt.lib.ttt_recur_bwd(by(c), *[A] * 10, None) == ttt.ERR_INVALID_ARG
    assert ttt.lib.ttt_recur_step(by(c), A, A, A, 4, A, A, None) == ttt.ERR_INVALID_ARG


def test_recur_argument_errors():
    c = recur_cfg()
    fwd = lambda c, *p: ttt.lib.ttt_recur_fwd(by(c), *p, None)
    bwd = lambda c, *p: ttt.lib.ttt_recur_bwd(by(c), *p, None)
    for field, v in (("dtype", 2), ("gate", 2), ("gate", -1)):
        bad = recur_cfg()
        setattr(bad, field, v)
        assert fwd(bad, A, A, A, A, A, A) == ttt.ERR_INVALID_ARG
    assert ttt.lib.ttt_recur_fwd(None, A, A, A, A, A, A, None) == ttt.ERR_INVALID_ARG
    for i in (0, 1, 4):
        p = [A] * 6
        p[i] = None
        assert fwd(c, *p) == ttt.ERR_INVALID_ARG, i
    for i in range(6):
        p = [A] * 6
        p[i] = A + 1
        assert fwd(c, *p) == ttt.ERR_ALIGNMENT, i
    # X G reset h0 H dH dh_final dX dG dh0
    for i in (0, 1, 4, 5, 7, 8):
        p = [A] * 10
        p[i] = None
        assert bwd(c, *p) == ttt.ERR_INVALID_ARG, i
    for i in range(10):
        p = [A] * 10
        p[i] = A + 2
        assert bwd(c, *p) == ttt.ERR_ALIGNMENT, i


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", ["decay", "sigmoid"])
def test_recur_widths_whose_blocks_leave_32_bits(dtype, gate):
    # the last block of features ends past D: no index of it may pass 2^31 - 1
    for D in (2 ** 31 - 1, 2 ** 31 - 512):
        c = recur_cfg(B=1, T=1, D=D, dtype=dtype, gate=gate)
        assert ttt.lib.ttt_recur_fwd(by(c), A, A, A, A, A, A, None) == ttt.ERR_INVALID_ARG
        assert ttt.lib.ttt_recur_bwd(by(c), *[A] * 10, None) == ttt.ERR_INVALID_ARG
        assert ttt.lib.ttt_recur_step(by(c), A, A, A, 4, A, A, None) == ttt.ERR_INVALID_ARG


def test_recur_step_refuses_more_rows_than_it_can_match():
    # every row is compared with all others where slots are given
    c = recur_cfg(B=(1 << 20) + 1, T=1, D=1)
    assert ttt.lib.ttt_recur_step(by(c), A, A, A, 9, A, A, None) == ttt.ERR_UNSUPPORTED


def test_recur_step_argument_errors():
    c = recur_cfg(T=1, B=4)
    step = lambda c, X, G, sl, n, st, Y: ttt.lib.ttt_recur_step(by(c), X, G, sl, n, st, Y, None)
    assert step(recur_cfg(T=2), A, A, A, 9, A, A) == ttt.ERR_INVALID_ARG
    assert step(c, A, A, A, 0, A, A) == ttt.ERR_INVALID_ARG
    assert step(c, A, A, None, 3, A, A) == ttt.ERR_INVALID_ARG  # fewer states than rows
    for i in (0, 1, 4, 5):
        p = [A, A, A, 9, A, A]
        p[i] = None
        assert step(c, *p) == ttt.ERR_INVALID_ARG, i
    for i in (0, 1, 2, 4, 5):
        p = [A, A, A, 9, A, A]
        p[i] = A + 4
        assert step(c, *p) == ttt.ERR_ALIGNMENT, i


def test_linear_size_errors():
    q = ttt.lib.ttt_linear_workspace_bytes
    none = ctypes.c_size_t(-1).value
    fwd = lambda M, N, K, act=0: ttt.lib.ttt_linear_fwd(M, N, K, act, *[A] * 7, A, 1 << 50, None)
    bwd = lambda M, N, K, act=0: ttt.lib.ttt_linear_bwd(M, N, K, act, *[A] * 9, A, 1 << 50, None)
    for call in (fwd, bwd):
        for s in ((0, 64, 64), (4, 0, 64), (4, 64, 0), (-1, 64, 64),
                  (1 << 30, 1 << 20, 64), (1 << 30, 64, 1 << 20), (4, 1 << 30, 1 << 20)):
            assert call(*s) == ttt.ERR_INVALID_ARG, s
        assert call(4, 64, 64, 2) == ttt.ERR_INVALID_ARG
        for s in ((4, 60, 64), (4, 64, 60), (4, 1, 8), (4, 8, 1)):
            assert call(*s) == ttt.ERR_UNSUPPORTED, s
    for s in ((0, 64, 64), (4, 60, 64), (4, 64, 60)):
        assert q(*s, 0) == none and q(*s, 1) == none
    assert q(4, 64, 64, 2) == none
    with pytest.raises(ttt.TTTError):
        ttt.ttt_linear_workspace_bytes(4, 64, 60, 0)


def test_linear_argument_errors():
    M, N, K = 4, 64, 64
    nf, nb = (ttt.ttt_linear_workspace_bytes(M, N, K, b) for b in (0, 1))
    fwd = lambda *p, ws=A, n=1 << 40: ttt.lib.ttt_linear_fwd(M, N, K, 1, *p, ws, n, None)
    for i in (0, 1, 5):  # X W bias mul residual Y P
        p = [A] * 7
        p[i] = None
        assert fwd(*p) == ttt.ERR_INVALID_ARG, i
    for i in range(7):
        p = [A] * 7
        p[i] = A + 2
        assert fwd(*p) == ttt.ERR_ALIGNMENT, i
    assert fwd(*[A] * 7, ws=A + 8) == ttt.ERR_ALIGNMENT
    if nf:
        assert fwd(*[A] * 7, ws=None, n=0) == ttt.ERR_WORKSPACE
    bwd = lambda act, *p, ws=A, n=1 << 40: ttt.lib.ttt_linear_bwd(M, N, K, act, *p, ws, n, None)
    # X W P mul dY dX dW dbias dmul
    base = [A] * 9
    for act, gone in ((1, [4]), (1, [5, 6, 7, 8]), (0, [0]), (0, [1]), (1, [2]), (0, [2]),
                      (0, [3]), (1, [2, 3, 8])):
        p = [None if i in gone else v for i, v in enumerate(base)]
        assert bwd(act, *p) == ttt.ERR_INVALID_ARG, (act, gone)
    for i in range(9):
        p = [A] * 9
        p[i] = A + 2
        assert bwd(1, *p) == ttt.ERR_ALIGNMENT, i
    if nb:
        assert bwd(1, *base, ws=None, n=0) == ttt.ERR_WORKSPACE
        assert bwd(1, *base, ws=A, n=nb - 1) == ttt.ERR_WORKSPACE


def test_binding_refuses_tensors_that_do_not_fit():
    c = norm_cfg(B=1, H=1, T=2, d=8)
    x = torch.zeros(16)
    with pytest.raises(ValueError, match="CUDA"):
        ttt.ttt_norm_fwd(c, x, None, None, None, x)
    with pytest.raises(ValueError, match="expected 16"):
        ttt.ttt_norm_fwd(c, x[:8], None, None, None, x)
    with pytest.raises(ValueError, match="bfloat16"):
        ttt.ttt_norm_fwd(c, x.bfloat16(), None, None, None, x)
    with pytest.raises(ValueError, match="contiguous"):
        ttt.ttt_norm_fwd(c, torch.zeros(32)[::2], None, None, None, x)
    r = recur_cfg(B=1, T=2, D=8, gate="decay")
    b = torch.zeros(16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="G is"):  # a decay is float32
        ttt.ttt_recur_fwd(r, 4096, b, None, None, 4096)
    with pytest.raises(ValueError, match="reset is"):
        ttt.ttt_recur_bwd(r, None, 4096, torch.zeros(2, dtype=torch.bool), None, 4096, 4096, None,
                          4096, 4096)
    s = recur_cfg(B=2, T=1, D=8)
    with pytest.raises(ValueError, match="slots is"):
        ttt.ttt_recur_step(s, 4096, 4096, torch.zeros(2, dtype=torch.int64), torch.zeros(3, 8),
                           4096)
    with pytest.raises(ValueError, match="W is"):
        ttt.ttt_linear_fwd(2, 8, 8, "id", 4096, b, None, None, None, 4096)
    with pytest.raises(ValueError, match="dbias is"):
        ttt.ttt_linear_bwd(2, 8, 8, "id", 4096, 4096, None, None, 4096, dbias=torch.zeros(16))
    with pytest.raises(ValueError, match="workspace"):
        ttt.ttt_linear_bwd(2, 8, 8, "id", 4096, 4096, None, None, 4096, dX=4096,
                           workspace=torch.zeros(4), workspace_bytes=32)


def test_native_checks_agree_with_the_binding_s_own():
    # what the native checks do not take, the binding's own checks name; they never take what those
    # refuse (host tensors here: no address may come back for one)
    from weight_sequence_layers_b200 import _bind
    t = torch.zeros(6)
    assert _bind.ptrs((None, 4096), (1, 1), "ff", 0) == (None, 4096)
    for bad in ((t,), (t.view(2, 3).t(),), ("x",), (3.0,), (t.to(torch.bfloat16),), (t.to("meta"),)):
        assert _bind.ptrs(bad, (6,), "f", 0) is None
        assert _bind.ptrs(bad, (6,), "f", -1) is None
    assert _bind.ptrs((t,), (6, 6), "f", 0) is None and _bind.ptrs((t,), (6,), "ff", 0) is None
    assert _bind.ptrs([t], (6,), "f", 0) is None and _bind.ptrs((t,), (6,), "f") is None
