"""Cross attention and its gradients on the GPU against the oracle (float64).

Tolerances, elementwise, for inputs given in bf16:
* a score is a sum of d_h exact products in fp32: off by at most
  delta = d_h 2^-23 max_ij sum_c |q_ic k_jc| / sqrt(d_h), and so, relatively,
  is exp(score); exp2 and its argument's rounding add under 2^-14.
* out: rounded once (2^-8 |out|); P enters the product as bf16 (2^-8); so
  2^-8 |out| + (2^-8 + 2^-12 + 2 delta) sum_j p_ij |v_j|.
* lse: delta, the sum's roundings (under 2^-16) and its own (2^-22 |lse|).
* dv: as out, with dO for v.
* dq, dk: rounded once; dS enters as bf16 (2^-8) and sums of some thousand
  terms in fp32 (2^-11); D comes from out rounded to bf16 (2^-8 of sum_c
  |dO_c O_c|); P = exp(S - lse) carries 2 delta + 2^-14; dP and D carry
  eta = d_h 2^-23 max sum_c |dO_c v_c| each.
* fp32 holds no normal number below 2^-126: a P under that may be 0.  Such an
  error reaches a sum at most 2^-126 x 2^11 rows x 2^12 (|dP| |Q| at most, here)
  < 2^-100 (TINY), which every tolerance includes.
"""
import numpy as np
import pytest
import torch

import learned_token_group_b200 as moga
import oracle
from oracle import around
from parity import np_cpu

pytestmark = pytest.mark.gpu

B = 2.0 ** -8
TINY = 2.0 ** -100
TIMEOUT, DEVICE_CHECK = 5, 6


def rnd(g, *s):
    return torch.randn(s, generator=g, device="cuda")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def layout_of(x, how):
    """x [n, h, d] with the same values in other memory."""
    n, h, d = x.shape
    if how == "packed":                               # beside another tensor of the same rows
        return torch.cat([x, torch.full_like(x, float("nan"))], 1)[:, :h]
    if how == "head_major":
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    if how == "head_rows":                            # head-major with rows to spare
        y = torch.full((h, n + 5, d), float("nan"), dtype=x.dtype, device=x.device)
        y[:, :n] = x.transpose(0, 1)
        return y[:, :n].transpose(0, 1)
    if how == "wide":                                 # a token stride that is no multiple of the head's
        y = torch.full((n, h * d + 24), float("nan"), dtype=x.dtype, device=x.device)
        y[:, :h * d] = x.reshape(n, h * d)
        return y.as_strided((n, h, d), (h * d + 24, d, 1))
    return x


class Case:
    def __init__(self, q_lens, k_lens, H, Hk, d, seed=0, layout="dense", padded=False, edge=0, peak=1.0, poison=True):
        """Segments of q_lens queries and k_lens keys; padded: each segment's
        keys in a place of the longest's size; edge: rows before the first and
        behind the last segment.  Whatever belongs to no segment is NaN."""
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        S = len(q_lens)
        qo = edge + np.concatenate([[0], np.cumsum(q_lens)])
        width = [max(k_lens)] * S if padded else k_lens
        ko = edge + np.concatenate([[0], np.cumsum(width)])
        N, L = int(qo[-1]) + edge, int(ko[-1]) + edge
        self.N, self.L, self.H, self.Hk, self.d = N, L, H, Hk, d
        q, k, v, dout = (rnd(g, n, h, d) for n, h in ((N, H), (L, Hk), (L, Hk), (N, H)))
        q = 1.3 * peak * q
        if peak > 1 and L:                            # some keys that queries match
            k[:min(N, L)] = peak * q[:min(N, L), ::H // Hk] / (1.3 * peak)
        self.seg = [(int(qo[s]), int(qo[s + 1]), int(ko[s]), int(ko[s]) + int(k_lens[s])) for s in range(S)]
        if poison:
            for t, (a, b) in ((q, (0, 1)), (k, (2, 3)), (v, (2, 3)), (dout, (0, 1))):
                dead = torch.ones(len(t), dtype=torch.bool, device="cuda")
                for s in self.seg:
                    dead[s[a]:s[b]] = False
                t[dead] = float("nan")
        self.q, self.k, self.v, self.dout = (t.to(torch.bfloat16) for t in (q, k, v, dout))
        whole = S == 1 and not edge
        self.seg_args = dict(q_offsets=None if whole else ints(qo), kv_offsets=None if whole else ints(ko),
                             kv_lens=ints(k_lens) if padded else None)
        self.in_place = [layout_of(t, layout) for t in (self.q, self.k, self.v)]

    def reference(self, dout=None):
        r = around.cross(self.q, self.k, self.v, self.seg, dout)
        sc = 1 / np.sqrt(self.d)
        f = lambda t: np.abs(around.f64(t))  # noqa: E731
        self.delta = self.eta = 0.0
        for q0, q1, k0, k1 in self.seg:
            if q1 > q0 and k1 > k0:
                for h in range(self.H):
                    kh = h // (self.H // self.Hk)
                    self.delta = max(self.delta, self.d * 2.0 ** -23 * sc * (f(self.q[q0:q1, h]) @ f(self.k[k0:k1, kh]).T).max())
                    if dout is not None:
                        self.eta = max(self.eta, self.d * 2.0 ** -23 * (f(dout[q0:q1, h]) @ f(self.v[k0:k1, kh]).T).max())
        return r


def near(got, want, tol, what=""):
    a = np_cpu(got).astype(np.float64)
    inside = ~np.isnan(want)
    a, want, tol = a[inside], want[inside], tol[inside]
    assert np.isfinite(a).all(), f"{what}: not finite"
    over = np.abs(a - want) - tol - TINY
    assert a.size == 0 or over.max() <= 0, f"{what}: off by {np.abs(a - want).max():.3e}, {over.max():.3e} over"


def check_forward(c, **kw):
    r = c.reference()
    out, lse = moga.cross_attn(*c.in_place, **c.seg_args, return_lse=True, **kw)
    near(out, r["out"], B * np.abs(r["out"]) + (B + 2.0 ** -12 + 2 * c.delta) * r["out_size"], what="out")
    got = np_cpu(lse)
    keys = np.isfinite(r["lse"])
    assert np.isneginf(got[np.isneginf(r["lse"])]).all()
    assert (np.abs(got[keys] - r["lse"][keys]) <= c.delta + 2.0 ** -16 + 2.0 ** -22 * np.abs(r["lse"][keys])).all()
    outside = np.isnan(r["out"][:, 0, 0]) if c.N else np.zeros(0, bool)
    assert (np_cpu(out)[outside] == 0).all() and np.isneginf(got[:, outside]).all()
    assert torch.equal(out, moga.cross_attn(*c.in_place, **c.seg_args))       # the same without lse, and again
    return out, lse


def check_backward(c, out, lse, **kw):
    r = c.reference(c.dout)
    g = moga.cross_attn_backward(c.dout, *c.in_place, out, lse, **c.seg_args, **kw)
    moga.sync_status(g["ws"])
    for n in ("dq", "dk"):
        near(g[n], r[n], B * np.abs(r[n]) + (B + 2.0 ** -11) * r[n + "_size"] + B * r[n + "_d"] +
             (2 * c.delta + 2.0 ** -14) * r[n + "_p"] + 2 * c.eta * r[n + "_1"], what=n)
    near(g["dv"], r["dv"], B * np.abs(r["dv"]) + (B + 2.0 ** -11 + 2 * c.delta) * r["dv_size"], what="dv")
    for n in ("dq", "dk", "dv"):
        assert (np_cpu(g[n])[np.isnan(r["dv" if n == "dv" else n])] == 0).all()
    return g


def check(*a, **kw):
    c = Case(*a, **kw)
    out, lse = check_forward(c)
    check_backward(c, out, lse)
    return c


ONE = [(1, 1, 1, 1, 128), (1, 77, 12, 12, 128), (1, 16, 2, 2, 64), (5, 128, 2, 1, 128), (128, 129, 1, 1, 64),
       (129, 127, 2, 2, 128), (257, 300, 3, 1, 128), (300, 512, 2, 2, 64), (130, 1, 2, 2, 128), (3, 2000, 2, 2, 128),
       (700, 1030, 4, 2, 64), (256, 256, 1, 1, 128), (77, 5003, 3, 3, 128), (1500, 77, 8, 1, 64), (2, 15, 1, 1, 128),
       (385, 640, 1, 1, 128), (64, 3000, 16, 4, 64)]


@pytest.mark.parametrize("N,L,H,Hk,d", ONE)
def test_one_segment(N, L, H, Hk, d):
    check([N], [L], H, Hk, d, seed=N + L)


@pytest.mark.parametrize("H,Hk", [(64, 1), (128, 2), (128, 1), (5, 1), (12, 4), (32, 1)])
def test_shared_key_heads(H, Hk):
    """Tiles of all query heads of a key head (up to 64, a power of two), or of one at a time."""
    check([9], [70], H, Hk, 64)
    check([37, 0, 130], [200, 5, 19], H, Hk, 64)


def test_a_thousand_segments():
    rng = np.random.default_rng(3)
    check(list(rng.integers(0, 5, 1024)), list(rng.integers(0, 40, 1024)), 4, 2, 64)
    check(list(rng.integers(0, 5, 100)), list(rng.integers(0, 300, 100)), 2, 2, 128)


def test_lengths_without_offsets():
    """One segment whose keys end early: the same bits as without the rows behind, whatever they hold."""
    c = Case([70], [90], 2, 2, 128)
    c.k[50:], c.v[50:] = float("nan"), float("inf")
    n = ints([50])
    out, lse = moga.cross_attn(c.q, c.k, c.v, kv_lens=n, return_lse=True)
    want, lse2 = moga.cross_attn(c.q, c.k[:50], c.v[:50], return_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, lse2)
    g = moga.cross_attn_backward(c.dout, c.q, c.k, c.v, out, lse, kv_lens=n)
    h = moga.cross_attn_backward(c.dout, c.q, c.k[:50], c.v[:50], out, lse)
    assert torch.equal(g["dq"], h["dq"])
    for x in ("dk", "dv"):
        assert torch.equal(g[x][:50], h[x]) and (g[x][50:] == 0).all()
    out, lse = moga.cross_attn(c.q, c.k, c.v, kv_lens=ints([0]), return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()
    g = moga.cross_attn_backward(c.dout, c.q, c.k, c.v, out, lse, kv_lens=ints([0]))
    assert all((g[x] == 0).all() for x in ("dq", "dk", "dv"))


def test_infinities_stay_in_their_rows():
    """An infinite query makes its own row NaN, an infinite value its own channel infinite; the rest keeps its bits."""
    c = Case([140], [200], 2, 2, 64)
    want = moga.cross_attn(c.q, c.k, c.v)
    q, v = c.q.clone(), c.v.clone()
    q[5, 0, 3] = float("inf")
    v[7, 1, 9] = float("inf")
    got = moga.cross_attn(q, c.k, v)
    assert torch.isnan(got[5, 0]).all() and torch.isinf(got[:, 1, 9]).all()
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[5, 0] = keep[:, 1, 9] = False
    assert torch.equal(got[keep], want[keep])


SEGS = {
    "one_and_two_tiles": ([100, 300, 1, 129, 128, 200, 5], [300, 129, 500, 100, 640, 128, 257]),
    "ragged": ([130, 0, 1, 300, 7, 256], [5, 64, 0, 257, 128, 33]),
    "singles": ([1] * 9, [1, 2, 0, 128, 129, 300, 17, 0, 64]),
    "empty": ([3, 0, 5], [0, 0, 0]),
    "many": (list(range(40)), [(7 * i) % 150 for i in range(40)]),
    "long_short": ([1000, 1], [3, 1500]),
}


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("edge", [0, 3])
@pytest.mark.parametrize("d,H,Hk", [(128, 2, 2), (64, 4, 1)])
@pytest.mark.parametrize("name", sorted(SEGS))
def test_segments(name, d, H, Hk, edge, padded):
    check(*SEGS[name], H, Hk, d, seed=edge, edge=edge, padded=padded)


@pytest.mark.parametrize("heads", [12, 16])
def test_many_units_of_every_kind_on_each_sm(heads):
    """More units than SMs, with one query tile and with two, of no to six key tiles, following one another."""
    rng = np.random.default_rng(heads)
    check(list(rng.integers(0, 420, 60)), list(rng.integers(0, 700, 60)), heads, heads // 4, 64)
    check(list(rng.integers(0, 300, 40)), list(rng.integers(0, 300, 40)), heads, heads, 128)


def test_many_queries_without_keys():
    """More units without keys than a CTA's ring holds, behind, before and between others."""
    check([300, 9000, 200, 9000, 130, 9000], [200, 0, 300, 0, 129, 0], 12, 12, 64)
    check([9000, 300], [0, 200], 12, 12, 64)


@pytest.mark.parametrize("layout", ["packed", "head_major", "head_rows", "wide"])
@pytest.mark.parametrize("d", [64, 128])
def test_layouts(layout, d):
    check([140, 200], [70, 150], 4, 2, d, layout=layout)
    check([150], [200], 1, 1, d, layout=layout)
    check([1], [200], 3, 3, d, layout=layout)


@pytest.mark.parametrize("peak", [2.0, 6.0])
def test_matched_keys(peak):
    """A query's own key takes nearly all of its row, and running maxima grow from tile to tile."""
    check([300], [700], 2, 2, 128, peak=peak)
    check([2], [3000], 2, 2, 64, peak=peak)


@pytest.mark.parametrize("N", [60, 200])
def test_growing_scores(N):
    """Keys sorted by their score: every tile's maximum is above the last one's by more than 2^8."""
    c = Case([N], [900], 1, 1, 128)
    u = torch.zeros(128, device="cuda")
    u[0] = 1
    c.q = (c.q.float() * 0.1 + 8 * u).to(torch.bfloat16)
    c.k = (c.k.float() * 0.1 + torch.linspace(-40, 40, 900, device="cuda")[:, None, None] * u).to(torch.bfloat16)
    c.in_place = [c.q, c.k, c.v]
    check_backward(c, *check_forward(c))


def test_no_rows():
    q, k = (torch.zeros(n, 2, 128, dtype=torch.bfloat16, device="cuda") for n in (0, 5))
    out, lse = moga.cross_attn(q, k, k, return_lse=True)
    assert out.shape == (0, 2, 128) and lse.shape == (2, 0)
    g = moga.cross_attn_backward(q, q, k, k, out, lse)
    assert (g["dk"] == 0).all() and (g["dv"] == 0).all() and g["dq"].shape == (0, 2, 128)
    out, lse = moga.cross_attn(k, q, q, return_lse=True)              # queries, no keys
    assert (out == 0).all() and torch.isneginf(lse).all()
    g = moga.cross_attn_backward(k, k, q, q, out, lse)
    assert (g["dq"] == 0).all() and g["dk"].shape == (0, 2, 128)


def test_rows_of_no_segment_are_left_as_they_were():
    c = Case([100, 30], [40, 0], 2, 2, 128, edge=4)
    out = torch.full((c.N, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    assert moga.cross_attn(*c.in_place, **c.seg_args, out=out) is out
    assert (out[:4] == 7).all() and (out[134:] == 7).all() and (out[104:134] == 0).all()


BAD = [dict(q_offsets=[0, 60, 50]), dict(q_offsets=[-1, 50, 100]), dict(q_offsets=[0, 50, 101]),
       dict(kv_offsets=[0, 60, 50]), dict(kv_offsets=[-2, 50, 80]), dict(kv_offsets=[0, 50, 81]),
       dict(kv_lens=[41, 3]), dict(kv_lens=[3, -1]), dict(kv_offsets=[0, 2 ** 31 - 1, 80]),
       dict(kv_lens=[2 ** 31 - 1, 3])]


@pytest.mark.parametrize("bad", BAD, ids=[str(b) for b in BAD])
def test_bad_segments_are_reported_and_nothing_is_written(bad):
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    q, k, v = (rnd(g, n, 2, 64).to(torch.bfloat16) for n in (100, 80, 80))
    seg = dict(q_offsets=[0, 50, 100], kv_offsets=[0, 40, 80], kv_lens=[40, 40])
    good = {n: ints(x) for n, x in seg.items()}
    broken = {n: ints(x) for n, x in dict(seg, **bad).items()}
    ws = moga.workspace(moga.cross_attn_workspace_size(q, k, 2, backward=True), "cuda")
    out = torch.full((100, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    moga.cross_attn(q, k, v, **broken, out=out, ws=ws)
    with pytest.raises(moga.MogaError) as e:
        moga.sync_status(ws)
    assert e.value.status == DEVICE_CHECK and (out == 7).all()
    out, lse = moga.cross_attn(q, k, v, **good, return_lse=True, ws=ws)
    moga.sync_status(ws)
    gr = moga.cross_attn_backward(q, q, k, v, out, lse, **broken, ws=ws)
    with pytest.raises(moga.MogaError):
        moga.sync_status(ws)
    assert all((gr[n] == 0).all() for n in ("dk", "dv"))
    moga.cross_attn_backward(q, q, k, v, out, lse, **good, ws=ws)
    moga.sync_status(ws)


def test_the_same_bits_again_with_a_used_workspace():
    """Calls of other sizes in between leave nothing behind; sums are taken in a fixed order."""
    cs = [Case([700], [300], 4, 2, 128), Case([3], [4000], 2, 2, 64), Case(*SEGS["ragged"], 4, 4, 128)]
    ws = moga.workspace(max(moga.cross_attn_workspace_size(c.q, c.k, len(c.seg), True) for c in cs), "cuda")
    runs = []
    for _ in range(2):
        for c in cs:
            out, lse = moga.cross_attn(*c.in_place, **c.seg_args, return_lse=True, ws=ws)
            g = moga.cross_attn_backward(c.dout, *c.in_place, out, lse, **c.seg_args, ws=ws)
            runs.append((out, lse, g["dq"], g["dk"], g["dv"]))
    moga.sync_status(ws)
    for a, b in zip(runs[:3], runs[3:]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_other_streams_and_replayed_graphs():
    cs = [Case([500], [300], 2, 2, 128, seed=1), Case([4], [3000], 2, 2, 128, seed=2)]
    ws = moga.workspace(max(moga.cross_attn_workspace_size(c.q, c.k, 1, True) for c in cs), "cuda")

    def step(c, ws=None):
        out, lse = moga.cross_attn(*c.in_place, return_lse=True, ws=ws)
        g = moga.cross_attn_backward(c.dout, *c.in_place, out, lse, ws=ws)
        return out, lse, g["dq"], g["dk"], g["dv"]
    want = [step(c) for c in cs]
    torch.cuda.synchronize()
    got = []
    for c in cs:                                      # at once, each with its own workspace
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got.append(step(c))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    graphs = []
    for c in cs:                                      # two graphs of one workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, step(c, ws)))
    old = [c.v.clone() for c in cs]
    for f in (2.0, 1.0):
        for c, v in zip(cs, old):
            c.v.copy_(v * f)
        for g, _ in graphs * 2:
            g.replay()
        torch.cuda.synchronize()
        now = [step(c) for c in cs]
        for (_, a), b in zip(graphs, now):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    moga.sync_status(ws)


@pytest.mark.parametrize("N,L", [(500, 300), (5, 3000)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(N, L):
    """The library's test hook withholds each CTA's first K tile: the bounded waits run out, nothing hangs."""
    lib = moga.get_lib()
    c = Case([N], [L], 2, 2, 128)
    ws = moga.workspace(moga.cross_attn_workspace_size(c.q, c.k), "cuda")
    old = lib.moga_set_wait_limit_ns(50_000_000)
    try:
        assert lib.moga_debug_inject(1) == 0
        moga.cross_attn(*c.in_place, ws=ws)
        with pytest.raises(moga.MogaError) as e:
            moga.sync_status(ws)
        assert e.value.status == TIMEOUT
    finally:
        lib.moga_debug_inject(0)
        lib.moga_set_wait_limit_ns(old)
    moga.sync_status(ws)
    check_forward(c, ws=ws)
    moga.sync_status(ws)


@pytest.mark.parametrize("layout", ["dense", "views", "broadcast"])
def test_autograd(layout):
    """The function's gradients against 64-bit autograd of the formula."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    q = rnd(g, 120, 4, 72).to(torch.bfloat16).requires_grad_()
    kv = rnd(g, 90, 2, 2, 72).to(torch.bfloat16).requires_grad_()
    co = rnd(g, 120, 4, 64).to(torch.bfloat16)
    if layout == "views":                             # heads off a 16-byte boundary, keys and values side by side
        view = lambda q, kv: (q[..., 3:67], kv[:, 0, :, :64], kv[:, 1, :, :64])  # noqa: E731
    elif layout == "broadcast":                       # one key head for all, one value row for all
        view = lambda q, kv: (q[..., :64], kv[:, 0, :1, :64].expand(90, 4, 64), kv[:1, 1, :1, :64].expand(90, 4, 64))  # noqa: E731
    else:
        view = lambda q, kv: (q[..., :64].contiguous(), kv[:, 0, :, :64].contiguous(), kv[:, 1, :, :64].contiguous())  # noqa: E731
    qo, ko = [0, 50, 120], [0, 60, 90]
    out = moga.CrossAttnFunction.apply(*view(q, kv), ints(qo), ints(ko))
    (out * co).float().sum().backward()
    q64, kv64 = (t.detach().double().requires_grad_() for t in (q, kv))
    a, b, c = view(q64, kv64)
    loss = 0
    for (q0, q1), (k0, k1) in zip(zip(qo, qo[1:]), zip(ko, ko[1:])):
        for h in range(4):
            kh = h * b.shape[1] // 4
            p = torch.softmax(a[q0:q1, h] @ b[k0:k1, kh].t() / 8, -1)
            loss = loss + ((p @ c[k0:k1, kh]) * co[q0:q1, h].double()).sum()
    loss.backward()
    # each gradient is rounded once and made of products with P or dS rounded once (their errors spread over the
    # sum); a broadcast adds its terms in bf16: 2^-8 of the largest each, at most 4 of them.  One value row for all
    # keys makes dq 0: dP is the same for all keys of a row, and what is left of dP - D is dP times the distance of
    # sum_j P_ij from 1.  S is the forward's, bit for bit, so that distance is made of the roundings of exp2, of its
    # argument (below 2^4: 2^-20), of the sum and of lse: under 2^-17.  |dP| < 2^6 (64 channels), |k| < 2^3, and the
    # scale is 2^-3: dq is off by under 2^-11 from that.
    for x, y in ((q.grad, q64.grad), (kv.grad, kv64.grad)):
        off, most = (x.double() - y).abs().max().item(), y.abs().max().item()
        assert off <= 4 * B * most + 2.0 ** -11


def test_refusals():
    q, k = (torch.zeros(n, h, 64, dtype=torch.bfloat16, device="cuda") for n, h in ((10, 4), (8, 2)))

    def no(match, *a, **kw):
        with pytest.raises((ValueError, moga.MogaError), match=match):
            moga.cross_attn(*a, **kw)
    no("bfloat16", q.float(), k, k)
    no("k and v must be", q, k, k[:5])
    no("k and v must be", q[:, :3], k, k)
    no("tokens, heads", q[0], k, k)
    no("dense", q[..., ::2], k, k)
    no("UNSUPPORTED", q[..., :32], k[..., :32], k[..., :32])
    no("several segments", q, k, k, q_offsets=ints([0, 5, 10]))
    no("_offsets must be", q, k, k, q_offsets=ints([0, 5, 10]), kv_offsets=ints([0, 8]))
    no("int32", q, k, k, q_offsets=ints([0]), kv_offsets=ints([0]))
    no("q_offsets", q, k, k, q_offsets=ints([0, 5, 10]).long(), kv_offsets=ints([0, 3, 8]))
    no("kv_lens", q, k, k, kv_lens=ints([1, 2]))
    no("out", q, k, k, out=torch.zeros(10, 4, 64, device="cuda"))
    no("must be on", q, k, k, kv_lens=torch.zeros(1, dtype=torch.int32))
    no("WORKSPACE", q, k, k, ws=moga.workspace(256, "cuda")[:128])
    no("INVALID_ARG", q, k[:, :1].expand(8, 2, 64), k)  # a head stride of zero: autograd's function copies it
    out, lse = moga.cross_attn(q, k, k, return_lse=True)
    for kw in (dict(dout=q.float()), dict(out=out[:5]), dict(lse=lse.t()), dict(lse=lse.double())):
        with pytest.raises(ValueError):
            moga.cross_attn_backward(**dict(dict(dout=q, q=q, k=k, v=k, out=out, lse=lse), **kw))


def test_block_with_its_text_attention():
    """As used: norm and rotation, the visual block, then attention to each shot's prompt; against the oracle."""
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    grid, N, H, d, M = (3, 10, 12), 360, 2, 128, 3
    qkv = rnd(g, N, 3 * H, d).to(torch.bfloat16)
    w = [1 + 0.2 * rnd(g, d) for _ in range(4)]
    x, W_r = rnd(g, N, 64).to(torch.bfloat16), (rnd(g, M, 64) / 8).to(torch.bfloat16)
    axes = (24, 20, 20)
    table = moga.rope_table(12, d, axes)
    q, k = moga.qk_norm_rope(qkv[:, :H], qkv[:, H:2 * H], w[0], w[1], table, axes, grid)
    v = qkv[:, 2 * H:].contiguous()
    res = moga.moga_layer(x, W_r, None, q, k, v, M, grid, (3, 8, 8))
    text = rnd(g, 50, 2, H, d).to(torch.bfloat16)
    q2, _ = moga.qk_norm_rope(res["out"], None, w[2], None)
    _, k2 = moga.qk_norm_rope(None, text[:, 0], None, w[3])
    qo, ko = [0, 120, 360], [0, 27, 50]
    ws = moga.workspace(moga.cross_attn_workspace_size(q2, k2, 2), "cuda")
    out = moga.cross_attn(q2, k2, text[:, 1], ints(qo), ints(ko), ws=ws)
    moga.sync_status(res["ws"])
    moga.sync_status(ws)
    # the oracle, step by step from the GPU's own inputs of each step (their roundings are tested above)
    ang = around.angles(around.grid_positions(N, grid), axes, d)
    for got, xi, wi in ((q, qkv[:, :H], w[0]), (k, qkv[:, H:2 * H], w[1])):
        want, size = around.norm_rope(xi, wi, 1e-6, ang, False)
        assert (np.abs(np_cpu(got) - want) <= B * np.abs(want) * 1.001 + 2.0 ** -19 * size).all()
    f = lambda t: np_cpu(t).astype(np.float64)  # noqa: E731
    ref = oracle.moga_layer(f(x), f(W_r), None, f(q), f(k), f(v), M, grid=grid, window=(3, 8, 8))
    assert np.abs(f(res["out"]) - ref["out"]).max() <= 2e-2
    want = around.cross(q2, k2, text[:, 1], [(0, 120, 0, 27), (120, 360, 27, 50)])
    assert (np.abs(f(out) - want["out"]) <= B * np.abs(want["out"]) + (B + 2.0 ** -11) * want["out_size"]).all()


def test_training_step_through_block_and_text_attention():
    """The three autograd functions in a row; each one's gradients are those of its own backward call."""
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    grid, N, H, d, M = (2, 10, 12), 240, 2, 64, 3
    qkv = rnd(g, N, 3 * H, d).to(torch.bfloat16).requires_grad_()
    text = rnd(g, 40, 2, H, d).to(torch.bfloat16).requires_grad_()
    w = [(1 + 0.2 * rnd(g, d)).requires_grad_() for _ in range(4)]
    x, W_r = (t.to(torch.bfloat16).requires_grad_() for t in (rnd(g, N, 64), rnd(g, M, 64) / 8))
    axes, table = (12, 10, 10), moga.rope_table(12, d, (12, 10, 10))
    qo, ko = ints([0, 120, 240]), ints([0, 25, 40])
    norm, block, cross = moga.QkNormRopeFunction.apply, moga.MogaFunction.apply, moga.CrossAttnFunction.apply
    q, k = norm(qkv[:, :H], qkv[:, H:2 * H], w[0], w[1], table, axes, grid)
    y = block(x, W_r, None, q, k, qkv[:, 2 * H:], M, grid, (2, 8, 8))
    q2, _ = norm(y, None, w[2])
    _, k2 = norm(None, text[:, 0], None, w[3])
    out = cross(q2, k2, text[:, 1], qo, ko)
    dout = rnd(g, N, H, d).to(torch.bfloat16)
    mid = torch.autograd.grad(out, [q2, k2, y, q, k], dout, retain_graph=True)
    out.backward(dout)
    with torch.no_grad():
        o, lse = moga.cross_attn(q2, k2, text[:, 1], qo, ko, return_lse=True)
        gc = moga.cross_attn_backward(dout, q2, k2, text[:, 1], o, lse, qo, ko)
        assert torch.equal(gc["dq"], mid[0]) and torch.equal(gc["dk"], mid[1])
        assert torch.equal(text.grad[:, 1], gc["dv"])
        g2 = moga.qk_norm_rope_backward(mid[0], None, y, None, w[2])
        assert torch.equal(g2["dq"], mid[2]) and torch.equal(g2["dw_q"], w[2].grad)
        g1 = moga.qk_norm_rope_backward(mid[3], mid[4], qkv[:, :H], qkv[:, H:2 * H], w[0], w[1], table, axes, grid)
        assert torch.equal(g1["dq"], qkv.grad[:, :H]) and torch.equal(g1["dk"], qkv.grad[:, H:2 * H])
        assert torch.equal(g1["dw_q"], w[0].grad)
    for t in (x, W_r, qkv, text, *w):
        assert torch.isfinite(t.grad).all() and t.grad.abs().max() > 0


def test_offsets_past_32_bits():
    """Keys that start past 2^31 elements of one buffer (4 GB, mostly untouched)."""
    L, d = 300, 128
    sn = (1 << 31) // 256 + 128
    buf = torch.empty((L - 1) * sn + 2 * d, dtype=torch.bfloat16, device="cuda")
    k = buf.as_strided((L, 2, d), (sn, d, 1))
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    c = Case([40], [L], 2, 2, d)
    k.copy_(c.k)
    c.in_place[1] = k
    check_backward(c, *check_forward(c))


# ----------------------------------------------------------------------------- scores far from ordinary ones
LOWEST = torch.finfo(torch.bfloat16).min
HIDDEN = [float("-inf"), LOWEST, -3e30, -1e30, -1e12]


class Masked(Case):
    """A case behind `hidden` keys that a channel masks: q holds 1 there, those
    keys `mask` and the others 0.  exp of their scores is 0 in 64 bits too
    (each is below -8e10), so that results are those of the keys behind."""

    def __init__(self, N, L, H, Hk, d, hidden, mask):
        super().__init__([N], [L], H, Hk, d, seed=hidden)
        self.q[..., 0], self.k[..., 0] = 1, 0
        g = torch.Generator(device="cuda")
        g.manual_seed(1)
        k, v = (rnd(g, hidden, Hk, d).to(torch.bfloat16) for _ in range(2))
        k[..., 0] = mask
        self.in_place = [self.q, torch.cat([k, self.k]), torch.cat([v, self.v])]


# one query tile and two, a whole hidden tile before the first key that counts, and part of one; in one range
# of keys (few keys, or enough heads) and in shares, with whole shares hidden
MASKED = [(60, 72, 2, 2, 128), (60, 40, 2, 1, 256 - 40), (200, 72, 2, 2, 128), (200, 300, 80, 80, 140),
          (60, 300, 80, 80, 256), (5, 2000, 2, 2, 1300), (200, 2000, 4, 2, 700)]


@pytest.mark.parametrize("mask", HIDDEN)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,L,H,Hk,hidden", MASKED)
def test_hidden_first_tiles(N, L, H, Hk, hidden, d, mask):
    """Every score of a row's first key tiles is -inf or hugely negative, those behind are ordinary."""
    c = Masked(N, L, H, Hk, d, hidden, mask)
    r = c.reference()
    out, lse = moga.cross_attn(*c.in_place, return_lse=True)
    near(out, r["out"], B * np.abs(r["out"]) + (B + 2.0 ** -12 + 2 * c.delta) * r["out_size"], what="out")
    near(lse, r["lse"], c.delta + 2.0 ** -16 + 2.0 ** -22 * np.abs(r["lse"]), what="lse")


HUGE = [LOWEST / 4, -1e30, -1e12, -3e9, 3e9, 1e12, 1e30, -LOWEST / 4]


@pytest.mark.parametrize("value", HUGE)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,L", [(3, 1), (60, 77), (200, 130), (5, 3000), (200, 3000)])
def test_keys_that_are_all_huge(N, L, d, value):
    """All keys the same huge one: the mean of V.  All but one: that one's V, where it is larger.

    P is exactly 1 or exactly 0 in both (the scores differ by over 2^20), so
    out is rounded once, behind sums and a division in fp32 (2^-12)."""
    c = Case([N], [L], 2, 2, d, seed=L)
    one = torch.zeros(d, dtype=torch.bfloat16, device="cuda")
    one[0] = 1
    c.q[:], c.k[:] = one, value * one
    v = around.f64(c.v)
    for _ in range(2):
        out, lse = moga.cross_attn(c.q, c.k, c.v, return_lse=True)
        s = around.f64(c.k)[:, :, 0] / np.sqrt(d)                     # [L, H]
        top = s == s.max(0)
        for h in range(2):
            w = v[top[:, h], h]
            want, size = w.mean(0)[None].repeat(N, 0), np.abs(w).mean(0)[None]
            near(out[:, h], want, B * np.abs(want) + 2.0 ** -12 * size, what="out")
            want = np.full(N, s[:, h].max() + np.log(top[:, h].sum()))
            near(lse[h], want, 2.0 ** -21 * np.abs(want), what="lse")
        c.k[L // 2, :, 0] = 0.75 * value if value < 0 else 1.25 * value


@pytest.mark.parametrize("N,L", [(3, 1), (60, 77), (200, 130), (5, 3000)])
def test_rows_whose_scores_are_all_minus_infinity(N, L):
    """As rows without keys: 0, and -inf.  Other rows of the tile are as ever."""
    c = Case([N], [L], 2, 2, 64, seed=L)
    c.q[..., 0], c.k[..., 0] = 0.25, float("-inf")
    out, lse = moga.cross_attn(c.q, c.k, c.v, return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()
    c.k[:, 1, 0] = 0                                                  # the second head's keys count again
    out, lse = moga.cross_attn(c.q, c.k, c.v, return_lse=True)
    assert (out[:, 0] == 0).all() and torch.isneginf(lse[0]).all()
    alone = moga.cross_attn(c.q[:, 1:].contiguous(), c.k[:, 1:].contiguous(), c.v[:, 1:].contiguous())
    assert torch.isfinite(lse[1]).all() and (L > 1000 or torch.equal(out[:, 1:], alone))


@pytest.mark.parametrize("mask", HIDDEN[1:])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,L,H,Hk,hidden", MASKED)
def test_gradients_behind_hidden_keys(N, L, H, Hk, hidden, d, mask):
    """Hidden keys get gradients of 0 and change no others (those of -inf make dS K's channel 0 * inf, as the formula has it)."""
    c = Masked(N, L, H, Hk, d, hidden, mask)
    r = c.reference(c.dout)
    out, lse = moga.cross_attn(*c.in_place, return_lse=True)
    g = moga.cross_attn_backward(c.dout, *c.in_place, out, lse)
    moga.sync_status(g["ws"])
    assert (g["dk"][:hidden] == 0).all() and (g["dv"][:hidden] == 0).all()
    g = dict(dq=g["dq"], dk=g["dk"][hidden:], dv=g["dv"][hidden:])
    for n in ("dq", "dk"):
        near(g[n], r[n], B * np.abs(r[n]) + (B + 2.0 ** -11) * r[n + "_size"] + B * r[n + "_d"] +
             (2 * c.delta + 2.0 ** -14) * r[n + "_p"] + 2 * c.eta * r[n + "_1"], what=n)
    near(g["dv"], r["dv"], B * np.abs(r["dv"]) + (B + 2.0 ** -11 + 2 * c.delta) * r["dv_size"], what="dv")


FAR = 2.0 ** 20


@pytest.mark.parametrize("value", [LOWEST / 4, -1e12, 3e9, 1.5 * FAR * 16, -1.5 * FAR * 16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,L,H,Hk", [(60, 77, 2, 2), (200, 130, 2, 1), (5, 3000, 2, 2), (200, 700, 80, 80)])
def test_rows_with_a_huge_log_sum_exp_add_nothing(N, L, H, Hk, d, value):
    """Half of the rows meet a huge score in every key: lse is past 2^20, and P cannot be formed from it.

    Their dq is 0, and dk, dv are those of the other rows.  channel 0 of dq and
    dk, which the huge numbers multiply, is left out."""
    c = Case([N], [L], H, Hk, d, seed=L)
    c.q[..., 0], c.k[..., 0] = 0, value
    c.q[1::2, :, 0] = 1
    out, lse = moga.cross_attn(c.q, c.k, c.v, return_lse=True)
    assert (lse[:, 1::2].abs() > FAR).all()
    g = moga.cross_attn_backward(c.dout, c.q, c.k, c.v, out, lse)
    moga.sync_status(g["ws"])
    # In channel 0 the terms of a sum dS K are up to sum_j |dS_ij| |value|; sum_j |dS_ij| <= 2 max |dP| passes 8 here,
    # and 8 |value| fp32's largest number at LOWEST / 4: that sum may be infinite.
    assert (g["dq"][1::2] == 0).all() and all(torch.isfinite(g[n][..., 1:]).all() for n in ("dq", "dk", "dv"))
    q, k, dout = c.q[::2].contiguous(), c.k.clone(), c.dout[::2].contiguous()
    k[..., 0] = 0                                                     # q's channel 0 is 0 in these rows
    c.q, c.k, c.seg = q, k, [(0, len(q), 0, L)]
    r = c.reference(dout)
    g["dq"] = g["dq"][::2]
    for n in ("dq", "dk"):
        tol = B * np.abs(r[n]) + (B + 2.0 ** -11) * r[n + "_size"] + B * r[n + "_d"] + \
            (2 * c.delta + 2.0 ** -14) * r[n + "_p"] + 2 * c.eta * r[n + "_1"]
        near(g[n][..., 1:], r[n][..., 1:], tol[..., 1:], what=n)
    near(g["dv"], r["dv"], B * np.abs(r["dv"]) + (B + 2.0 ** -11 + 2 * c.delta) * r["dv_size"], what="dv")


def test_gradients_of_rows_whose_scores_are_all_minus_infinity():
    """As of rows without keys: none.  (k holds no -inf here: q does, and k a positive channel.)"""
    for N, L in ((60, 77), (200, 130), (5, 3000)):
        c = Case([N], [L], 2, 2, 64, seed=L)
        c.k[..., 0] = 0.5
        q = c.q.clone()
        q[1::2, :, 0] = float("-inf")
        out, lse = moga.cross_attn(q, c.k, c.v, return_lse=True)
        assert torch.isneginf(lse[:, 1::2]).all() and (out[1::2] == 0).all()
        g = moga.cross_attn_backward(c.dout, q, c.k, c.v, out, lse)
        assert (g["dq"][1::2] == 0).all() and torch.isfinite(g["dq"]).all() and torch.isfinite(g["dv"]).all()
        even = [t[::2].contiguous() for t in (c.q, c.dout)]
        r = around.cross(even[0], c.k, c.v, [(0, len(even[0]), 0, L)], even[1])
        near(g["dv"], r["dv"], B * np.abs(r["dv"]) + (B + 2.0 ** -10) * r["dv_size"], what="dv")


@pytest.mark.parametrize("bad", BAD + [dict(q_offsets=[0, 101], one=True), dict(kv_lens=[81], one=True),
                                       dict(kv_offsets=[5, 3], one=True)], ids=str)
def test_refused_segments_leave_nan_in_outputs_made_by_the_call(bad):
    """What the memory held before never comes out as a result: out, lse and dq are NaN, dk and dv 0."""
    bad = dict(bad)
    seg = {} if bad.pop("one", False) else dict(q_offsets=[0, 50, 100], kv_offsets=[0, 40, 80], kv_lens=[40, 40])
    c = Case([100], [80], 2, 2, 64)
    good = {n: ints(x) for n, x in seg.items()}
    broken = {n: ints(x) for n, x in dict(seg, **bad).items()}
    for n in (1, 3):                                  # one range of keys for a CTA, and shares (3 x 2,000 keys)
        q, k, v, dout = c.q, c.k, c.v, c.dout
        if n == 3:
            if seg or "kv_lens" not in bad:
                break
            c = Case([3], [2000], 2, 2, 64)
            q, k, v, dout, broken = c.q, c.k, c.v, c.dout, dict(kv_lens=ints([2001]))
        out0, lse0 = moga.cross_attn(q, k, v, **(good if n == 1 else {}), return_lse=True)
        for t in [torch.full((200 * 2 * 64,), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(8)] + \
                 [torch.full_like(lse0, 5.0) for _ in range(8)]:
            del t
        out, lse = moga.cross_attn(q, k, v, **broken, return_lse=True)
        assert torch.isnan(out).all() and torch.isnan(lse).all()
        assert torch.isnan(moga.cross_attn(q, k, v, **broken)).all()
        g = moga.cross_attn_backward(dout, q, k, v, out0, lse0, **broken)
        assert torch.isnan(g["dq"]).all() and (g["dk"] == 0).all() and (g["dv"] == 0).all()
        with pytest.raises(moga.MogaError):
            moga.sync_status(g["ws"])


def test_autograd_reports_to_a_given_workspace():
    """Both passes of the function use the caller's ws: it reports what each refused, and is refused if too small."""
    c = Case([50, 50], [40, 40], 2, 2, 64)
    q, k, v = (t.clone().requires_grad_() for t in (c.q, c.k, c.v))
    ws = moga.workspace(moga.cross_attn_workspace_size(q, k, 2, backward=True), "cuda")
    qo, ko, kl = ints([0, 50, 100]), ints([0, 40, 80]), ints([40, 40])
    out = moga.CrossAttnFunction.apply(q, k, v, qo, ko, kl, ws)
    out.backward(c.dout)
    moga.sync_status(ws)
    good = [t.grad.clone() for t in (q, k, v)]
    plain = moga.CrossAttnFunction.apply(q, k, v, qo, ko, kl)
    assert torch.equal(plain, out)
    kl[1] = 41
    bad = moga.CrossAttnFunction.apply(q, k, v, qo, ko, kl, ws)
    with pytest.raises(moga.MogaError) as e:
        moga.sync_status(ws)
    assert e.value.status == DEVICE_CHECK and torch.isnan(bad).all()
    q.grad = k.grad = v.grad = None
    bad.backward(c.dout)
    with pytest.raises(moga.MogaError):
        moga.sync_status(ws)
    assert torch.isnan(q.grad).all() and (k.grad == 0).all() and (v.grad == 0).all()
    kl[1] = 40
    q.grad = k.grad = v.grad = None
    moga.CrossAttnFunction.apply(q, k, v, qo, ko, kl, ws).backward(c.dout)
    moga.sync_status(ws)
    assert all(torch.equal(t.grad, x) for t, x in zip((q, k, v), good))
    with pytest.raises(ValueError, match="ws"):
        moga.CrossAttnFunction.apply(q, k, v, qo, ko, kl, ws[:256])


def test_one_workspace_for_a_training_step():
    """Norm and cross attention of a step, one after the other, with one ws of the largest size."""
    c = Case([100], [80], 2, 2, 64)
    w = torch.ones(64, device="cuda", requires_grad=True)
    need = max(moga.cross_attn_workspace_size(c.q, c.k, backward=True), moga.qk_norm_rope_workspace_size(64, backward=True))

    def step(ws):
        q = c.q.clone().requires_grad_()
        k = c.k.clone().requires_grad_()
        w.grad = None
        rest = (None, None, None, None, 0, 1e-6, False, ws)
        a, _ = moga.QkNormRopeFunction.apply(q, None, w, None, *rest)
        _, b = moga.QkNormRopeFunction.apply(None, k, None, w, *rest)
        moga.CrossAttnFunction.apply(a, b, c.v, None, None, None, ws).backward(c.dout)
        return q.grad, k.grad, w.grad.clone()
    ws = moga.workspace(need, "cuda")
    want = step(None)
    for _ in range(2):
        assert all(torch.equal(x, y) for x, y in zip(step(ws), want))
    moga.sync_status(ws)


def test_a_unit_longer_than_the_wait_limit():
    """Softmax warps without a tile of their own wait as long as a unit takes: that is no wait that ran out.

    200 units of one query tile and 1,200,000 keys each (some 9,400 tiles, several
    milliseconds) against a limit of 2 ms a step."""
    lib = moga.get_lib()
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    L = 1_200_000
    q, k = rnd(g, 1, 200, 64).to(torch.bfloat16), rnd(g, L, 1, 64).to(torch.bfloat16)
    ws = moga.workspace(moga.cross_attn_workspace_size(q, k), "cuda")
    want = moga.cross_attn(q, k, k, ws=ws)
    moga.sync_status(ws)
    old = lib.moga_set_wait_limit_ns(2_000_000)
    try:
        got = moga.cross_attn(q, k, k, ws=ws)
        moga.sync_status(ws)
    finally:
        lib.moga_set_wait_limit_ns(old)
    assert torch.equal(got, want)


@pytest.mark.parametrize("N,L,H,Hk", [(500, 300, 2, 2), (5, 3000, 2, 2), (200, 38400, 2, 1)])
def test_a_wait_that_runs_out_in_the_backward_is_reported_and_the_next_call_is_right(N, L, H, Hk):
    """The test hook withholds each CTA's first K tile (dQ) or Q tile (dK, dV): the bounded waits run out, nothing hangs."""
    lib = moga.get_lib()
    c = Case([N], [L], H, Hk, 64)
    seg = dict(q_offsets=ints([0, N]))                # dk and dv then start as zeros
    out, lse = moga.cross_attn(*c.in_place, return_lse=True)
    ws = moga.workspace(moga.cross_attn_workspace_size(c.q, c.k, backward=True), "cuda")
    old = lib.moga_set_wait_limit_ns(50_000_000)
    try:
        assert lib.moga_debug_inject(1) == 0
        g = moga.cross_attn_backward(c.dout, *c.in_place, out, lse, **seg, ws=ws)
        with pytest.raises(moga.MogaError) as e:
            moga.sync_status(ws)
        assert e.value.status == TIMEOUT
        if L > 38000:                                 # one share of the queries: nothing adds up what was not written
            assert (g["dk"] == 0).all() and (g["dv"] == 0).all()
    finally:
        lib.moga_debug_inject(0)
        lib.moga_set_wait_limit_ns(old)
    moga.sync_status(ws)
    check_backward(c, out, lse, ws=ws)
    moga.sync_status(ws)


def test_autograd_with_a_workspace_refuses_as_the_call_does():
    q, k = (torch.zeros(n, 2, 64, dtype=torch.bfloat16, device="cuda") for n in (10, 8))
    ws = moga.workspace(1 << 20, "cuda")
    for bad in ((q[0], k, k), (q, k[0], k), (q, k[:, :0], k[:, :0]), (q, k, k, ints([0]), ints([0]))):
        args = list(bad) + [None] * (6 - len(bad))
        with pytest.raises((ValueError, moga.MogaError)):
            moga.CrossAttnFunction.apply(*args)
        with pytest.raises((ValueError, moga.MogaError)):
            moga.CrossAttnFunction.apply(*args, ws)
