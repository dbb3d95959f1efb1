"""The norm of query and key heads with their rotation, and its gradients, on
the GPU against the oracle (float64).

Tolerances, elementwise.  An output is rounded to bf16 once: half a step,
2^-8 |y|.  What comes before is fp32: the mean of squares (8 fused steps, 4
additions of the row sum, eps: 13 roundings, halved by the root), rsqrtf (2
ulp), two products, two products and a sum of the rotation, cos and sin
rounded to fp32: under 32 roundings of 2^-24 relative to |z_a| + |z_b| of the
pair, 2^-19.  The gradients add a second row sum and five more steps: under 64
roundings, 2^-18, of the sum of the terms' magnitudes.  dw's terms carry 2^-19
and its sum at most 4 + 64 + 3 + 8 additions here: under 128 roundings, 2^-17.
"""
import numpy as np
import pytest
import torch

import learned_token_group_b200 as moga
from oracle import around
from parity import np_cpu

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
FWD, BWD, SUM = 2.0 ** -19, 2.0 ** -18, 2.0 ** -17
EPS = 1e-6
DEVICE_CHECK = 6


def _axes(d):
    n = d // 2
    return (n - 2 * (n // 3) - 1, n // 3, n // 3)      # one pair does not turn


def make(N, H, Hk, d, dtype, layout, pos, seed=0, scale=1.0, P=64, weights=True):
    """The arguments of a call, and the oracle's angles."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if layout == "packed":
        x = (scale * rnd(N, H + 2 * Hk, d)).to(dtype)
        q, k = x[:, :H], x[:, H:H + Hk]
    elif layout == "head_major":
        q, k = ((scale * rnd(h, N, d)).to(dtype).transpose(0, 1) for h in (H, Hk))
    else:
        q, k = ((scale * rnd(N, h, d)).to(dtype) for h in (H, Hk))
    a = dict(q=q if H else None, k=k if Hk else None, w_q=1 + 0.3 * rnd(d) if weights else None,
             w_k=1 + 0.3 * rnd(d) if weights else None)
    ang = None
    if pos != "none":
        a["axes"] = _axes(d)
        a["table"] = moga.rope_table(P, d, a["axes"])
        if pos == "list":
            a["positions"] = torch.randint(0, P, (N, 3), generator=g, device="cuda", dtype=torch.int32)
            ang = around.angles(np_cpu(a["positions"]), a["axes"], d)
        else:
            a["grid"], a["token0"] = (5, 7, 9), 311                  # wraps around after 4 tokens
            ang = around.angles(around.grid_positions(N, a["grid"], 311), a["axes"], d)
    return a, ang


def near(got, want, size, rel, half):
    a = np_cpu(got).astype(np.float64)
    assert np.isfinite(a).all()
    over = np.abs(a - want) - half * np.abs(want) * (1 + rel) - rel * size
    assert (over <= 0).all(), f"off by {np.abs(a - want).max():.3e}, {over.max():.3e} over"


def check_forward(a, ang, halves=False, eps=EPS, **kw):
    out = moga.qk_norm_rope(**a, halves=halves, eps=eps, **kw)
    for y, x, w in zip(out, (a["q"], a["k"]), (a["w_q"], a["w_k"])):
        if x is None:
            assert y is None
            continue
        assert y.dtype == torch.bfloat16 and y.shape == x.shape and y.is_contiguous()
        near(y, *around.norm_rope(x, w, eps, ang, halves), FWD, HALF[torch.bfloat16])
    return out


def check_backward(a, ang, halves=False, eps=EPS, seed=1, ws=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dy = [None if a[n] is None else torch.randn(a[n].shape, generator=g, device="cuda").to(torch.bfloat16) for n in "qk"]
    got = moga.qk_norm_rope_backward(*dy, **a, halves=halves, eps=eps, ws=ws)
    moga.sync_status(got["ws"])
    for n, d in zip("qk", dy):
        x, w = a[n], a["w_" + n]
        if x is None:
            assert got["d" + n] is None and got["dw_" + n] is None
            continue
        r = around.norm_rope_backward(d, x, w, eps, ang, halves)
        assert got["d" + n].dtype == x.dtype
        near(got["d" + n], r["dx"], r["dx_size"], BWD, HALF[x.dtype])
        if w is None:
            assert got["dw_" + n] is None
        else:
            near(got["dw_" + n], r["dw"], r["dw_size"], SUM, HALF[torch.float32])
    return dy, got


SHAPES = [(1, 1, 1, 64), (1, 12, 12, 128), (3, 5, 0, 128), (2, 0, 3, 64), (130, 8, 2, 64), (67, 3, 1, 128),
          (1561, 12, 12, 128), (333, 40, 40, 128), (257, 17, 1, 64), (5000, 1, 1, 128)]


@pytest.mark.parametrize("N,H,Hk,d", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pos,halves", [("none", False), ("grid", False), ("grid", True), ("list", False), ("list", True)])
def test_forward_and_backward(N, H, Hk, d, dtype, pos, halves):
    layout = ("dense", "packed", "head_major")[(N + H) % 3]
    a, ang = make(N, H, Hk, d, dtype, layout, pos, seed=N)
    check_forward(a, ang, halves)
    check_backward(a, ang, halves)


@pytest.mark.parametrize("layout", ["dense", "packed", "head_major"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layouts(layout, dtype):
    a, ang = make(203, 6, 2, 128, dtype, layout, "grid", seed=5)
    check_forward(a, ang)
    check_backward(a, ang)


def test_one_stride_for_all_tokens_or_heads():
    """A token or a head broadcast by a stride of zero is read like any other."""
    a, ang = make(50, 4, 4, 64, torch.bfloat16, "dense", "grid")
    a["q"], a["k"] = a["q"][:1].expand(50, 4, 64), a["k"][:, :1].expand(50, 4, 64)
    check_forward(a, ang)
    check_backward(a, ang)


@pytest.mark.parametrize("scale", [1e-4, 300.0, 1e15])
def test_small_and_large_values(scale):
    a, ang = make(70, 3, 3, 128, torch.bfloat16, "dense", "grid", scale=scale)
    check_forward(a, ang)
    check_backward(a, ang)


def test_zero_rows_and_no_weights():
    a, ang = make(20, 2, 2, 64, torch.bfloat16, "dense", "grid", weights=False)
    a["q"][3] = 0
    a["k"][:, 1] = 0
    out = check_forward(a, ang)
    assert (out[0][3] == 0).all()
    check_backward(a, ang)


def test_a_row_without_length_stays_in_its_row():
    """eps = 0 and a zero row: 0 * inf is NaN there (as the formula has it) and nowhere else, dw apart."""
    a, ang = make(20, 3, 1, 64, torch.bfloat16, "dense", "none")
    a["q"][7, 1] = 0
    q, _ = moga.qk_norm_rope(**a, eps=0.0)
    bad = torch.isnan(q)
    assert bad[7, 1].all() and bad.sum() == 64
    # heads that do not exist (3 heads in lanes for 4) leave dw finite
    a, ang = make(20, 3, 1, 64, torch.bfloat16, "dense", "none")
    check_backward(a, ang, eps=0.0)


def test_infinities_and_nan_stay_in_their_rows():
    a, _ = make(40, 2, 2, 128, torch.bfloat16, "dense", "grid")
    want = moga.qk_norm_rope(**a)[0]
    a["q"][5, 0, 3], a["q"][6, 1, 9] = float("inf"), float("nan")
    got = moga.qk_norm_rope(**a)[0]
    assert torch.isnan(got[6, 1]).all() and torch.isnan(got[5, 0]).any()
    keep = torch.ones(40, 2, dtype=torch.bool)
    keep[5, 0] = keep[6, 1] = False
    assert torch.equal(got[keep], want[keep])


def test_far_positions():
    """2^20 positions: the table's angles are formed in 64 bits."""
    d, P = 64, 1 << 20
    a, _ = make(100, 2, 2, d, torch.float32, "dense", "none")
    a["axes"] = (32, 0, 0)
    a["table"] = moga.rope_table(P, d, a["axes"])
    p = torch.zeros(100, 3, dtype=torch.int32, device="cuda")
    p[:, 0] = torch.arange(P - 100, P)
    p[:, 1:] = -5                                     # axes that do not turn are not looked at
    a["positions"] = p
    ang = around.angles(np_cpu(p), a["axes"], d)
    t = np_cpu(a["table"])[P - 100:]
    assert np.abs(t - np.stack([np.cos(ang), np.sin(ang)], -1)).max() <= 2.0 ** -24 + 1e-9
    check_forward(a, ang)
    check_backward(a, ang)


def test_table_is_one_and_zero_where_nothing_turns():
    t = moga.rope_table(9, 64, (4, 0, 2))
    assert (t[:, 6:, 0] == 1).all() and (t[:, 6:, 1] == 0).all() and (t[0, :, 0] == 1).all()
    want = around.angles(np.stack([np.arange(9)] * 3, 1), (4, 0, 2), 64)
    assert np.abs(np_cpu(t) - np.stack([np.cos(want), np.sin(want)], -1)).max() <= 2.0 ** -24


def test_shards_of_tokens_and_samples_of_a_batch():
    """token0 places a shard of a sequence; a batch of grids wraps around."""
    a, ang = make(630, 2, 2, 128, torch.bfloat16, "dense", "grid")
    a["token0"] = 0
    whole = moga.qk_norm_rope(**a)                    # two samples of 315 places
    for s in (slice(100, 217), slice(0, 630), slice(400, 401)):
        part = dict(a, q=a["q"][s], k=a["k"][s], token0=s.start % 315)
        for x, y in zip(moga.qk_norm_rope(**part), whole):
            assert torch.equal(x, y[s])
    b = dict(a, q=a["q"][315:], k=a["k"][315:])
    assert torch.equal(moga.qk_norm_rope(**b)[0], whole[0][315:])


def test_positions_outside_the_table_are_skipped_and_reported():
    a, ang = make(60, 3, 2, 64, torch.bfloat16, "dense", "list")
    ws = moga.workspace(256, "cuda")
    bad = [4, 5, 59]
    a["positions"][4, 0], a["positions"][5, 1], a["positions"][59, 2] = -1, 64, 2 ** 31 - 1
    out = [torch.full((60, h, 64), 7.0, dtype=torch.bfloat16, device="cuda") for h in (3, 2)]
    moga.qk_norm_rope(**a, out=out, ws=ws)
    with pytest.raises(moga.MogaError) as e:
        moga.sync_status(ws)
    assert e.value.status == DEVICE_CHECK
    keep = np.setdiff1d(np.arange(60), bad)
    for y, x, w in zip(out, (a["q"], a["k"]), (a["w_q"], a["w_k"])):
        assert (y[bad] == 7).all()
        want, size = around.norm_rope(x, w, EPS, ang, False)
        near(y[keep], want[keep], size[keep], FWD, HALF[torch.bfloat16])
    moga.sync_status(ws)                              # cleared
    dy = [torch.randn_like(y) for y in out]
    g = moga.qk_norm_rope_backward(*dy, **a)
    with pytest.raises(moga.MogaError):
        moga.sync_status(g["ws"])
    r = around.norm_rope_backward(np_cpu(dy[0])[keep], np_cpu(a["q"])[keep], a["w_q"], EPS, ang[keep], False)
    near(g["dw_q"], r["dw"], r["dw_size"], SUM, HALF[torch.float32])


def test_no_tokens():
    a, ang = make(0, 3, 2, 64, torch.bfloat16, "dense", "grid")
    q, k = moga.qk_norm_rope(**a)
    assert q.shape == (0, 3, 64) and k.shape == (0, 2, 64)
    g = moga.qk_norm_rope_backward(q, k, **a)
    assert (g["dw_q"] == 0).all() and (g["dw_k"] == 0).all() and g["dq"].shape == (0, 3, 64)


def test_in_place():
    a, ang = make(300, 4, 2, 128, torch.bfloat16, "dense", "grid")
    want = moga.qk_norm_rope(**a)
    for halves in (False, True):
        b = dict(a, q=a["q"].clone(), k=a["k"].clone())
        want = moga.qk_norm_rope(**a, halves=halves)
        got = moga.qk_norm_rope(**b, halves=halves, out=(b["q"], b["k"]))
        assert got[0] is b["q"] and all(torch.equal(x, y) for x, y in zip(got, want))


def test_the_same_bits_again_and_a_used_workspace():
    a, ang = make(3000, 12, 4, 128, torch.bfloat16, "packed", "grid")
    dy, first = check_backward(a, ang)
    small, ang2 = make(3, 1, 1, 128, torch.bfloat16, "dense", "none")
    check_backward(small, ang2, ws=first["ws"])
    again = moga.qk_norm_rope_backward(*dy, **a, ws=first["ws"])
    assert again["ws"] is first["ws"]
    for n in ("dq", "dk", "dw_q", "dw_k"):
        assert torch.equal(first[n], again[n])


def test_other_streams_and_a_replayed_graph():
    a, ang = make(700, 6, 6, 128, torch.bfloat16, "dense", "grid")
    want, _ = moga.qk_norm_rope(**a), torch.cuda.synchronize()
    dy, g = check_backward(a, ang)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append((moga.qk_norm_rope(**a), moga.qk_norm_rope_backward(*dy, **a)))
    torch.cuda.synchronize()
    for out, h in got:
        assert all(torch.equal(x, y) for x, y in zip(out, want))
        assert all(torch.equal(h[n], g[n]) for n in ("dq", "dk", "dw_q", "dw_k"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moga.qk_norm_rope(**a)
        h = moga.qk_norm_rope_backward(*dy, **a)
    old = a["q"].clone()
    for x in (-old, old):
        a["q"].copy_(x)
        graph.replay()
        now = moga.qk_norm_rope(**a)
        assert all(torch.equal(x, y) for x, y in zip(out, now))
    assert all(torch.equal(h[n], g[n]) for n in ("dq", "dk", "dw_q", "dw_k"))


@pytest.mark.parametrize("layout", ["dense", "packed", "odd", "broadcast"])
def test_autograd(layout):
    """The function's gradients against 64-bit autograd of the formula, views and broadcast inputs included."""
    a, ang = make(90, 4, 2, 64, torch.bfloat16, "dense", "grid")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    base = torch.randn(90, 8, 72, generator=g, device="cuda").to(torch.bfloat16).requires_grad_()
    if layout == "packed":
        view = lambda b: (b[:, :4, :64], b[:, 4:6, :64])  # noqa: E731
    elif layout == "odd":                             # heads that start off a 16-byte boundary
        view = lambda b: (b[:, :4, 3:67], b[:, 4:6, 1:65])  # noqa: E731
    elif layout == "broadcast":
        view = lambda b: (b[:, :1, :64].expand(90, 4, 64), b[:1, 4:6, :64].expand(90, 2, 64))  # noqa: E731
    else:
        view = lambda b: (b[:, :4, :64].contiguous(), b[:, 4:6, :64].contiguous())  # noqa: E731
    ws = [a["w_q"].requires_grad_(), a["w_k"].requires_grad_()]
    q, k = moga.QkNormRopeFunction.apply(*view(base), *ws, a["table"], a["axes"], a["grid"], None, a["token0"], EPS, True)
    co = [torch.randn(t.shape, generator=g, device="cuda").to(torch.bfloat16) for t in (q, k)]
    ((q * co[0]).float().sum() + (k * co[1]).float().sum()).backward()
    b64 = base.detach().double().requires_grad_()
    w64 = [w.detach().double().requires_grad_() for w in ws]
    phase = torch.from_numpy(ang).cuda()[:, None]
    loss = 0
    for x, w, c in zip(view(b64), w64, co):
        z = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w
        u, v = z[..., :32], z[..., 32:]
        y = torch.cat([u * phase.cos() - v * phase.sin(), u * phase.sin() + v * phase.cos()], -1)
        loss = loss + (y * c.double()).sum()
    loss.backward()
    # dy is rounded once by the product's backward (exact: a factor of one), dx once, and a broadcast's sum of n
    # bf16 values in bf16 once more; 2^-8 each, with the fp32 part below 2^-9 of the largest
    n = 90 if layout == "broadcast" else 1
    for x, y in ((base.grad, b64.grad), (ws[0].grad, w64[0].grad), (ws[1].grad, w64[1].grad)):
        assert (x.double() - y).abs().max() <= (2.5 if n > 1 else 1.5) * 2.0 ** -8 * y.abs().max()


def test_one_output_without_a_gradient():
    a, ang = make(30, 2, 2, 64, torch.bfloat16, "dense", "grid")
    a["q"].requires_grad_()
    q, k = moga.QkNormRopeFunction.apply(a["q"], a["k"], a["w_q"], a["w_k"], a["table"], a["axes"], a["grid"], None, 0)
    q.float().sum().backward()                        # a gradient of stride zero, and none for k
    assert torch.isfinite(a["q"].grad).all()


def test_refusals():
    a, _ = make(10, 2, 2, 64, torch.bfloat16, "dense", "grid")

    def no(match, **kw):
        with pytest.raises((ValueError, moga.MogaError), match=match):
            moga.qk_norm_rope(**dict(a, **kw))
    no("same tokens", k=a["k"][:5])
    no("same tokens", k=torch.zeros(10, 2, 128, dtype=torch.bfloat16, device="cuda"))
    no("must be torch.bfloat16", k=a["k"].float())
    no("must be torch.bfloat16 or torch.float32", q=a["q"].half())
    no("tokens, heads", q=a["q"][0])
    no("dense", q=torch.zeros(10, 2, 128, dtype=torch.bfloat16, device="cuda")[..., ::2])
    no("w_q", w_q=a["w_q"].double())
    no("w_k", w_k=a["w_k"][:32])
    no("grid or positions", grid=None)
    no("need a table", table=None)
    no("axes", axes=None)
    no("table", table=a["table"][:, :16])
    no("INVALID_ARG", axes=(30, 30, 30))
    no("INVALID_ARG", token0=315)
    no("INVALID_ARG", grid=(65, 1, 1))
    no("positions", grid=None, positions=torch.zeros(10, 2, dtype=torch.int32, device="cuda"))
    no("positions", grid=None, positions=torch.zeros(10, 3, dtype=torch.int32))
    no("q_out", out=(torch.zeros(10, 2, 64, device="cuda"), None))
    no("UNSUPPORTED", q=torch.zeros(10, 2, 32, dtype=torch.bfloat16, device="cuda"), k=None, w_q=None, w_k=None, table=None, grid=None,
       axes=None, token0=0)
    no("INVALID_ARG", q=torch.zeros(10 * 2 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(10, 2, 64))
    with pytest.raises(ValueError, match="dq_out"):
        moga.qk_norm_rope_backward(None, a["k"], **a)
    with pytest.raises(ValueError, match="dk_out"):
        moga.qk_norm_rope_backward(a["q"], a["k"].float(), **a)


def test_numbers_past_32_bits_are_refused():
    # 2^32 + 1 and 2^64 would come down as 1 and 0.
    a, _ = make(10, 2, 2, 64, torch.bfloat16, "dense", "grid")
    big = (1 << 32) + 1
    for kw in (dict(grid=(big, *a["grid"][1:])), dict(axes=(big, 0, 0)), dict(token0=1 << 64), dict(token0=-1)):
        with pytest.raises(ValueError, match="grid"):
            moga.qk_norm_rope(**dict(a, **kw))
    with pytest.raises(ValueError, match="32 bits"):
        moga.rope_table(8, 64, (big, 0, 0))


def test_offsets_past_32_bits():
    """Tokens 2^31 elements apart in one buffer (4 GB of bf16, mostly untouched)."""
    N, H, d = 4100, 4, 128
    sn = (1 << 31) // 4096 + 128                      # the last tokens start past 2^31 elements
    buf = torch.empty((N - 1) * sn + H * d, dtype=torch.bfloat16, device="cuda")
    q = buf.as_strided((N, H, d), (sn, d, 1))
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    q.copy_(torch.randn(N, H, d, generator=g, device="cuda"))
    got, _ = moga.qk_norm_rope(q, None)
    want, size = around.norm_rope(q, None, EPS, None, False)
    near(got, want, size, FWD, HALF[torch.bfloat16])


def _used_memory(nbytes):
    """Leaves the caching allocator blocks that hold ordinary numbers."""
    for t in [torch.full((nbytes // 2,), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]:
        del t


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,Hk,d,halves", [(3, 2, 64, False), (1, 0, 128, True), (40, 40, 128, True), (17, 1, 64, False)])
def test_skipped_tokens_are_nan_in_outputs_made_by_the_call(H, Hk, d, halves, dtype):
    """What the memory held before never comes out as a result, from the calls or from autograd."""
    a, ang = make(60, H, Hk, d, dtype, "dense", "list")
    bad = [4, 5, 59]
    a["positions"][4, 0], a["positions"][5, 1], a["positions"][59, 2] = -1, 64, 2 ** 31 - 1
    keep = np.setdiff1d(np.arange(60), bad)
    _used_memory(60 * H * d * 4)
    dy = [None if a[n] is None else torch.ones(a[n].shape, dtype=torch.bfloat16, device="cuda") for n in "qk"]
    out = moga.qk_norm_rope(**a, halves=halves)
    g = moga.qk_norm_rope_backward(*dy, **a, halves=halves)
    for n, y, t in zip("qk", out, dy):
        if y is None:
            continue
        want, size = around.norm_rope(a[n], a["w_" + n], EPS, ang, halves)
        assert torch.isnan(y[bad]).all()
        near(y[keep], want[keep], size[keep], FWD, HALF[torch.bfloat16])
        r = around.norm_rope_backward(np_cpu(t)[keep], np_cpu(a[n])[keep], a["w_" + n], EPS, ang[keep], halves)
        assert torch.isnan(g["d" + n][bad]).all()
        near(g["d" + n][keep], r["dx"], r["dx_size"], BWD, HALF[dtype])
        near(g["dw_" + n], r["dw"], r["dw_size"], SUM, HALF[torch.float32])


def test_autograd_reports_to_a_given_workspace():
    """Both passes of the function use the caller's ws: it reports what each skipped, and is refused if too small."""
    a, _ = make(60, 3, 2, 64, torch.bfloat16, "dense", "list")
    a["q"].requires_grad_()
    ws = moga.workspace(moga.qk_norm_rope_workspace_size(64, backward=True), "cuda")
    args = [a[n] for n in ("q", "k", "w_q", "w_k", "table", "axes")] + [None, a["positions"], 0, EPS, False]
    q, k = moga.QkNormRopeFunction.apply(*args, ws)
    (q.float().sum() + k.float().sum()).backward()
    moga.sync_status(ws)
    good = a["q"].grad.clone()
    a["positions"][7, 0] = 64
    q, k = moga.QkNormRopeFunction.apply(*args, ws)
    with pytest.raises(moga.MogaError) as e:
        moga.sync_status(ws)
    assert e.value.status == DEVICE_CHECK and torch.isnan(q[7]).all() and torch.isnan(k[7]).all()
    a["q"].grad = None
    torch.autograd.backward([q, k], [torch.ones_like(q), torch.ones_like(k)])
    with pytest.raises(moga.MogaError):
        moga.sync_status(ws)
    keep = [n for n in range(60) if n != 7]
    assert torch.isnan(a["q"].grad[7]).all() and torch.equal(a["q"].grad[keep], good[keep])
    moga.sync_status(ws)
    with pytest.raises(ValueError, match="ws"):
        moga.QkNormRopeFunction.apply(*args, moga.workspace(256, "cuda"))


@pytest.mark.parametrize("first", [1, 3, 8])
def test_autograd_takes_gradients_that_start_anywhere(first):
    """An output's gradient may be a slice of a flat buffer, off a 16-byte boundary."""
    a, _ = make(30, 2, 1, 64, torch.bfloat16, "dense", "grid")
    a["q"].requires_grad_()
    a["k"].requires_grad_()
    args = [a[n] for n in ("q", "k", "w_q", "w_k", "table", "axes", "grid")] + [None, a["token0"]]
    flat = torch.randn(30 * 3 * 64 + 16, device="cuda").to(torch.bfloat16)
    dq = flat[first:first + 30 * 2 * 64].view(30, 2, 64)
    dk = flat[first + 30 * 2 * 64:][:30 * 64].view(30, 1, 64)
    got = torch.autograd.grad(moga.QkNormRopeFunction.apply(*args), [a["q"], a["k"]], [dq, dk])
    want = torch.autograd.grad(moga.QkNormRopeFunction.apply(*args), [a["q"], a["k"]], [dq.clone(), dk.clone()])
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_too_large_for_their_sum_give_zero(dtype):
    """A sum of squares past fp32's range: 1 / sqrt(inf) = 0.  The other rows are as ever."""
    a, ang = make(20, 2, 2, 64, dtype, "dense", "grid")
    a["q"][7, 1] *= 1e25
    out = moga.qk_norm_rope(**a)
    dy = [torch.ones(t.shape, dtype=torch.bfloat16, device="cuda") for t in out]
    g = moga.qk_norm_rope_backward(*dy, **a)
    assert (out[0][7, 1] == 0).all() and (g["dq"][7, 1] == 0).all() and torch.isfinite(g["dw_q"]).all()
    a["q"][7, 1] = 1
    near(out[1], *around.norm_rope(a["k"], a["w_k"], EPS, ang, False), FWD, HALF[torch.bfloat16])
    want, size = around.norm_rope(a["q"], a["w_q"], EPS, ang, False)
    keep = [n for n in range(20) if n != 7]
    near(out[0][keep], want[keep], size[keep], FWD, HALF[torch.bfloat16])
