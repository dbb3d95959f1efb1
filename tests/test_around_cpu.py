"""The operators around the block, as far as no GPU is needed: the oracle's
gradients against differences, and every refusal of the C ABI and the binding.
Fake pointer values are never dereferenced: validation fails first."""
import ctypes

import numpy as np
import pytest
import torch

import learned_token_group_b200 as moga
from oracle import around

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P = 1 << 20
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return moga.get_lib()


def int3(*v):
    return (ctypes.c_int * 3)(*v)


# ----------------------------------------------------------------------------- the oracle
def _slope(f, x, dx, h=1e-6):
    return (f(x + h * dx) - f(x - h * dx)) / (2 * h)


@pytest.mark.parametrize("halves", [False, True])
def test_norm_oracle_gradients_are_the_differences(halves):
    rng = np.random.default_rng(1)
    x, w, dy = rng.normal(size=(5, 2, 64)), rng.normal(size=64), rng.normal(size=(5, 2, 64))
    ang = around.angles(around.grid_positions(5, (2, 2, 3), 4), (12, 10, 8), 64)
    g = around.norm_rope_backward(dy, x, w, 1e-3, ang, halves)
    f = lambda x, w: (around.norm_rope(x, w, 1e-3, ang, halves)[0] * dy).sum()  # noqa: E731
    for _ in range(3):
        e = rng.normal(size=x.shape)
        assert abs(_slope(lambda t: f(t, w), x, e) - (g["dx"] * e).sum()) < 1e-6
        e = rng.normal(size=w.shape)
        assert abs(_slope(lambda t: f(x, t), w, e) - (g["dw"] * e).sum()) < 1e-6


def test_norm_oracle_turns_and_keeps_lengths():
    rng = np.random.default_rng(2)
    x = rng.normal(size=(6, 1, 64))
    pos = np.array([[3, 0, 0]] * 3 + [[0, 0, 0]] * 3)
    for halves in (False, True):
        y, _ = around.norm_rope(x, None, 0.0, around.angles(pos, (4, 0, 0), 64), halves)
        z = x / np.sqrt((x ** 2).mean(-1, keepdims=True))
        assert np.allclose((y ** 2).sum(-1), 64.0)
        assert np.allclose(y[3:], z[3:])                      # position 0 does not turn
        a, b = (0, 32) if halves else (0, 1)
        assert np.allclose(y[:3, 0, a] + 1j * y[:3, 0, b], (z[:3, 0, a] + 1j * z[:3, 0, b]) * np.exp(3j))
        rest = np.setdiff1d(np.arange(64), [0, 1, 2, 3, 32, 33, 34, 35] if halves else range(8))
        assert np.allclose(y[..., rest], z[..., rest])        # pairs past the axes do not turn


def test_cross_oracle_gradients_are_the_differences():
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(7, 4, 8)), rng.normal(size=(9, 2, 8)), rng.normal(size=(9, 2, 8))
    dout = rng.normal(size=q.shape)
    seg = [(0, 3, 0, 4), (3, 4, 4, 4), (4, 7, 5, 9)]
    r = around.cross(q, k, v, seg, dout)
    f = lambda q, k, v: np.nansum(around.cross(q, k, v, seg)["out"] * dout)  # noqa: E731
    for _ in range(3):
        e = rng.normal(size=q.shape)
        assert abs(_slope(lambda t: f(t, k, v), q, e) - np.nansum(r["dq"] * e)) < 1e-6
        e = rng.normal(size=k.shape)
        assert abs(_slope(lambda t: f(q, t, v), k, e) - np.nansum(r["dk"] * e)) < 1e-6
        assert abs(_slope(lambda t: f(q, k, t), v, e) - np.nansum(r["dv"] * e)) < 1e-6
    assert (r["out"][3] == 0).all() and np.isneginf(r["lse"][:, 3]).all()
    assert np.isnan(r["dk"][4]).all() and not np.isnan(r["dk"][5]).any()


def test_cross_oracle_against_the_library_softmax():
    rng = np.random.default_rng(4)
    q, k, v = (torch.from_numpy(rng.normal(size=(n, 3, 16))) for n in (5, 11, 11))
    t = torch.nn.functional.scaled_dot_product_attention(*(x.transpose(0, 1) for x in (q, k, v))).transpose(0, 1)
    assert np.abs(around.cross(q, k, v, [(0, 5, 0, 11)])["out"] - t.numpy()).max() < 1e-12


# ----------------------------------------------------------------------------- refusals of the C ABI
def _norm(lib, q=P, qs=(256, 128), k=P, ks=(256, 128), dt=1, N=100, H=2, Hk=2, d=128, w=None, eps=1e-6, table=P, rows=64,
          axes=(22, 21, 21), grid=(4, 5, 6), token0=0, pos=None, halves=0, out=P, ws=P, wsb=BIG):
    return lib.moga_qk_norm_rope(q, *qs, k, *ks, dt, N, H, Hk, d, w, w, eps, table, rows,
                                 None if axes is None else int3(*axes), None if grid is None else int3(*grid), token0,
                                 pos, halves, out, out, ws, wsb, None)


NORM_REFUSALS = [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(out=None), INVALID), (dict(q=P + 2), INVALID),
    (dict(out=P + 8), INVALID), (dict(w=P + 2), INVALID), (dict(dt=2), INVALID), (dict(N=-1), INVALID),
    (dict(N=1 << 31), INVALID), (dict(H=0, Hk=0), INVALID), (dict(H=-1), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(H=70000), UNSUPPORTED), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(halves=2), INVALID), (dict(qs=(260, 128)), UNSUPPORTED),
    (dict(qs=(256, 4)), UNSUPPORTED), (dict(qs=(-256, 128)), INVALID), (dict(ks=(256, -8)), INVALID),
    (dict(dt=0, qs=(258, 128)), UNSUPPORTED), (dict(axes=None), INVALID), (dict(axes=(-1, 2, 2)), INVALID),
    (dict(axes=(22, 22, 21)), INVALID), (dict(rows=0), INVALID), (dict(table=P + 4), INVALID),
    (dict(table=None), INVALID), (dict(grid=None), INVALID), (dict(pos=P), INVALID), (dict(grid=(4, 0, 6)), INVALID),
    (dict(grid=(65, 5, 6)), INVALID), (dict(rows=5), INVALID), (dict(token0=-1), INVALID), (dict(token0=120), INVALID),
    (dict(grid=(1, 1 << 16, 1 << 16), axes=(1, 0, 0)), UNSUPPORTED), (dict(grid=None, pos=P + 2), INVALID),
    (dict(grid=None, pos=P, ws=None), INVALID), (dict(ws=P + 8), INVALID), (dict(wsb=128), WORKSPACE),
]


@pytest.mark.parametrize("bad,status", NORM_REFUSALS, ids=[str(b) for b, _ in NORM_REFUSALS])
def test_norm_refusals(lib, bad, status):
    assert _norm(lib, **bad) == status


def test_norm_backward_refusals(lib):
    need = lib.moga_qk_norm_rope_backward_workspace_size(128)
    assert need > lib.moga_qk_norm_rope_backward_workspace_size(64) > lib.moga_qk_norm_rope_workspace_size()
    assert lib.moga_qk_norm_rope_backward_workspace_size(-1) == 0

    def f(dy=P, q=P, dx=P, dw=P, d=128, ws=P, wsb=need):
        return lib.moga_qk_norm_rope_backward(dy, dy, q, 256, 128, P, 256, 128, 1, 10, 2, 2, d, None, None, 1e-6, None, 0,
                                              None, None, 0, None, 0, dx, dx, dw, dw, ws, wsb, None)
    assert f(dy=None) == f(q=None) == f(dx=None) == f(dx=P + 4) == f(dw=P + 1) == f(ws=None) == INVALID
    assert f(d=32) == UNSUPPORTED
    assert f(wsb=need - 1) == WORKSPACE


def test_rope_table_refusals(lib):
    f = lib.moga_rope_table
    assert f(0, 128, int3(1, 1, 1), 1e4, P, None) == INVALID
    assert f(8, 128, None, 1e4, P, None) == INVALID
    assert f(8, 128, int3(1, -1, 1), 1e4, P, None) == INVALID
    assert f(8, 128, int3(30, 30, 5), 1e4, P, None) == INVALID
    assert f(8, 96, int3(1, 1, 1), 1e4, P, None) == UNSUPPORTED
    for theta in (0.0, -1.0, float("nan"), float("inf")):
        assert f(8, 128, int3(1, 1, 1), theta, P, None) == INVALID
    assert f(8, 128, int3(1, 1, 1), 1e4, None, None) == f(8, 128, int3(1, 1, 1), 1e4, P + 4, None) == INVALID


CROSS = dict(q=P, qs=(512, 128), k=P, ks=(256, 128), v=P, vs=(256, 128), N=100, L=50, H=4, Hk=2, d=128, qo=None, ko=None,
             kl=None, S=1, out=P, lse=None, fill=0, ws=P, wsb=BIG)
CROSS_REFUSALS = [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q=P + 8), INVALID),
    (dict(H=0), INVALID), (dict(Hk=0), INVALID), (dict(H=5), INVALID), (dict(N=-1), INVALID), (dict(L=-1), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(N=1 << 30), UNSUPPORTED), (dict(L=1 << 30), UNSUPPORTED),
    (dict(N=1 << 29, H=4), UNSUPPORTED), (dict(S=0), INVALID), (dict(S=1025, qo=P, ko=P), INVALID),
    (dict(S=2), INVALID), (dict(S=2, qo=P), INVALID), (dict(S=2, ko=P), INVALID), (dict(qo=P + 1), INVALID),
    (dict(kl=P + 2), INVALID), (dict(qs=(516, 128)), UNSUPPORTED), (dict(qs=(512, 4)), UNSUPPORTED),
    (dict(qs=(0, 128)), INVALID), (dict(qs=(512, 0)), INVALID), (dict(ks=(256, -128)), INVALID),
    (dict(qs=(64, 128)), UNSUPPORTED), (dict(qs=(512, 64)), UNSUPPORTED),
    (dict(qs=(128, 12672)), UNSUPPORTED),              # heads overlap: 99 token strides, 100 tokens
    (dict(qs=(256, 12672 + 136)), UNSUPPORTED),        # the head stride is no whole number of token strides
    (dict(fill=2), INVALID), (dict(fill=-1), INVALID),
    (dict(qs=(448, 128)), UNSUPPORTED),                # a token's heads reach into the next token
]
CROSS_REFUSALS_FWD = CROSS_REFUSALS + [
    (dict(out=None), INVALID), (dict(out=P + 8), INVALID), (dict(lse=P + 2), INVALID), (dict(ws=None), INVALID),
    (dict(ws=P + 8), INVALID), (dict(wsb=64), WORKSPACE),
]


def _cross(lib, **kw):
    a = dict(CROSS, **kw)
    return lib.moga_cross_attn(a["q"], *a["qs"], a["k"], *a["ks"], a["v"], *a["vs"], a["N"], a["L"], a["H"], a["Hk"],
                               a["d"], a["qo"], a["ko"], a["kl"], a["S"], a["out"], a["lse"], a["fill"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad,status", CROSS_REFUSALS_FWD, ids=[str(b) for b, _ in CROSS_REFUSALS_FWD])
def test_cross_refusals(lib, bad, status):
    assert _cross(lib, **bad) == status


def _cross_back(lib, dout=P, dq=P, dk=P, dv=P, **kw):
    a = dict(CROSS, lse=P, **kw)
    return lib.moga_cross_attn_backward(dout, a["q"], *a["qs"], a["k"], *a["ks"], a["v"], *a["vs"], a["N"], a["L"],
                                        a["H"], a["Hk"], a["d"], a["qo"], a["ko"], a["kl"], a["S"], a["out"], a["lse"],
                                        dq, dk, dv, a["fill"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bad,status", CROSS_REFUSALS, ids=[str(b) for b, _ in CROSS_REFUSALS])
def test_cross_backward_refusals(lib, bad, status):
    assert _cross_back(lib, **bad) == status


def test_cross_backward_refuses_missing_outputs_and_small_workspaces(lib):
    for n in ("dout", "dq", "dk", "dv", "out"):
        assert _cross_back(lib, **{n: None}) == INVALID
        assert _cross_back(lib, **{n: P + 16}) == INVALID          # 32-byte sectors
    need = lib.moga_cross_attn_backward_workspace_size(100, 50, 4, 2, 128, 1)
    assert _cross_back(lib, wsb=need - 1) == WORKSPACE
    assert lib.moga_cross_attn_workspace_size(-1, 50, 4, 2, 128, 1) == 0
    assert lib.moga_cross_attn_backward_workspace_size(100, 50, 4, 2, 128, 0) == 0


# ----------------------------------------------------------------------------- refusals of the binding
def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    for f in (lambda: moga.qk_norm_rope(x, None), lambda: moga.qk_norm_rope(None, x), lambda: moga.cross_attn(x, x, x),
              lambda: moga.qk_norm_rope_backward(x, None, x, None),
              lambda: moga.cross_attn_backward(x, x, x, x, x, torch.zeros(2, 4))):
        with pytest.raises(ValueError, match="CUDA"):
            f()
    with pytest.raises(ValueError, match="one of q and k"):
        moga.qk_norm_rope(None, None)
    with pytest.raises(ValueError, match="positions"):
        moga.rope_table(0, 64, (1, 1, 1), device="cuda:0")


def test_fill_refusals(lib):
    """fill of the _ex calls is 0 or 1."""
    def f(fill):
        return lib.moga_qk_norm_rope_ex(P, 256, 128, P, 256, 128, 1, 10, 2, 2, 128, None, None, 1e-6, None, 0, None, None,
                                        0, None, 0, P, P, fill, None, 0, None)

    def b(fill):
        return lib.moga_qk_norm_rope_backward_ex(P, P, P, 256, 128, P, 256, 128, 1, 10, 2, 2, 128, None, None, 1e-6, None, 0,
                                                 None, None, 0, None, 0, P, P, P, P, fill, P, BIG, None)
    for fill in (-1, 2):
        assert f(fill) == b(fill) == INVALID


def test_rope_table_refuses_a_host_device():
    for dev in ("cpu", "meta"):
        with pytest.raises(ValueError, match="CUDA"):
            moga.rope_table(8, 64, (1, 1, 1), device=dev)
