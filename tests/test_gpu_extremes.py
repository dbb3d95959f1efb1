"""The block's attention where scores are far from ordinary ones: keys that a
channel masks with -inf or a hugely negative number, keys that are all the same
huge one, and rows whose scores are all -inf (taken as 0, with a log-sum-exp of
-inf).

exp of a masked score is 0 in 64 bits too (each is below -8e10), so results are
those of the keys left.  Where P is exactly 1 or 0, out is a mean of V rows:
sums and a division in fp32 (2^-12 of the magnitudes) and one rounding to bf16
(2^-8)."""
import numpy as np
import pytest
import torch

import learned_token_group_b200 as moga
import oracle
from parity import compare_out, np_cpu

pytestmark = pytest.mark.gpu

INF = float("inf")
LOWEST = torch.finfo(torch.bfloat16).min
MASKS = [-INF, LOWEST, -3e30, -1e30, -1e12]
HUGE = [LOWEST / 4, -1e30, -1e12, -3e9, 3e9, 1e12, 1e30, -LOWEST / 4]


def f64(t):
    return np_cpu(t).astype(np.float64)


def inputs(N, H, d, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q, k, v = (torch.randn(N, H, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    q[..., 0], k[..., 0] = 1, 0
    return q, k, v


def groups(q, k, v, sizes):
    off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")
    perm = torch.arange(len(q), dtype=torch.int32, device="cuda")
    ws = moga.workspace(moga.get_lib().moga_group_attn_workspace_size(*q.shape, len(sizes)), "cuda")
    out = moga.group_attn(q, k, v, perm, off, None, len(sizes), ws=ws)
    moga.sync_status(ws)
    return out


def attention(q, k, v):
    """Rows of q [n, H, d] over keys k, v [m, H, d], 64 bits."""
    s = np.einsum("ihd,jhd->hij", f64(q), f64(k)) / np.sqrt(q.shape[-1])
    p = np.exp(s - s.max(-1, keepdims=True))
    return np.einsum("hij,jhd->ihd", p / p.sum(-1, keepdims=True), f64(v))


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sizes,hidden", [([200], 128), ([300, 700], 140), ([129], 128), ([2000], 1300)])
def test_groups_with_hidden_first_tiles(sizes, hidden, d, mask):
    """Every score of a row's first key tiles is -inf or hugely negative, those behind are ordinary."""
    q, k, v = inputs(sum(sizes), 2, d)
    start = 0
    want = np.empty(q.shape)
    for n in sizes:
        k[start:start + hidden, :, 0] = mask
        want[start:start + n] = attention(q[start:start + n], k[start + hidden:start + n], v[start + hidden:start + n])
        start += n
    compare_out(groups(q, k, v, sizes), want)


@pytest.mark.parametrize("value", HUGE)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 77, 130, 1000])
def test_groups_of_keys_that_are_all_huge(N, d, value):
    """The mean of V; and with one key that is larger than the rest, its V."""
    q, k, v = inputs(N, 2, d, seed=N)
    q[..., 1:], k[..., 1:], k[..., 0] = 0, 0, value
    for top in (slice(0, N), slice(N // 2, N // 2 + 1)):
        if top.stop - top.start == 1:
            k[top, :, 0] = 0.75 * value if value < 0 else 1.25 * value
        want, size = f64(v)[top].mean(0), np.abs(f64(v)[top]).mean(0)
        off = np.abs(f64(groups(q, k, v, [N])) - want)
        assert (off <= 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * size).all()


@pytest.mark.parametrize("N", [1, 77, 130, 1000])
def test_groups_whose_scores_are_all_minus_infinity(N):
    q, k, v = inputs(N, 2, 64)
    k[..., 0] = -INF
    assert (groups(q, k, v, [N]) == 0).all()


WINDOWS = [((2, 10, 12), (2, 5, 6)), ((2, 8, 16), (2, 8, 8)), ((3, 16, 16), (3, 8, 8)), ((1, 30, 52), (1, 30, 52))]


@pytest.mark.parametrize("grid,window", WINDOWS)
@pytest.mark.parametrize("d", [64, 128])
def test_windows_far_from_ordinary(grid, window, d):
    """60-, 128- and 192-token windows, and one of a whole frame (through the grouped kernel)."""
    N = int(np.prod(grid))
    q, k, v = inputs(N, 1, d)
    idx = [np.asarray(i) for i in oracle.stga_windows(*grid, window)]
    for mask in MASKS:
        kk = k.clone()
        for i in idx:                                 # all but the last few keys of every window
            kk[torch.as_tensor(i[:-5], device="cuda"), :, 0] = mask
        want = np.empty(q.shape)
        for i in idx:
            want[i] = attention(q[i], k[i[-5:]], v[i[-5:]])
        compare_out(moga.stga_window_attn(q, kk, v, grid, window), want)
    q[..., 1:], k[..., 1:] = 0, 0
    for value in HUGE:
        k[..., 0] = value
        out = f64(moga.stga_window_attn(q, k, v, grid, window))
        for i in idx:
            want, size = f64(v)[i].mean(0), np.abs(f64(v)[i]).mean(0)
            assert (np.abs(out[i] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * size).all()
    k[..., 0] = -INF
    assert (moga.stga_window_attn(q, k, v, grid, window) == 0).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [LOWEST / 4, -1e12, 3e9])
def test_training_rows_with_a_huge_log_sum_exp_add_nothing(value, d):
    """Half of the rows meet a huge score in every key: |lse| is past 2^20, P cannot be formed from it, and they
    take P = 0.  The other rows' gradients are theirs alone (channel 0, which the huge numbers multiply, aside)."""
    grid, window, N, M = (3, 10, 12), (3, 8, 8), 360, 2
    q, k, v = inputs(N, 1, d)
    q[::2, :, 0], k[..., 0] = 0, value
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x, W = (torch.randn(n, 64, generator=g, device="cuda").to(torch.bfloat16) for n in (N, M))
    dout = torch.randn(N, 1, d, generator=g, device="cuda").to(torch.bfloat16)
    args = (x, W, None, q, k, v, M, grid, window)
    sv = moga.layer_train(*args)
    got = moga.layer_backward(dout, sv, *args)
    moga.sync_status(got["ws"])
    assert (got["dq"][1::2] == 0).all()
    quiet = dout.clone()
    quiet[1::2] = 0                                   # what those rows add is then 0 in the formulas too
    other = moga.layer_backward(quiet, sv, *args)
    for n in ("dq", "dk", "dv"):
        a, b = (f64(t[n])[..., 1:] for t in (got, other))
        assert np.isfinite(a).all() and np.array_equal(a, b), n
    assert np.isfinite(f64(got["dv"])).all() and np.abs(f64(got["dv"])).max() > 0
