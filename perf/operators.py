"""Cases and plain forms of the operators beside the visual block.

Two operators, each with its backward pass:

* the norm of every query and key head with the rotation by the token's place
  (``qk_norm_rope``), which makes the q and k that the attention calls take;
* cross attention of the video tokens to an encoder's states of another
  length (``cross_attn``), one segment of keys for each shot or sample.

Sizes are the latent grids of the repository's workloads (1,560 tokens a
frame, 32,760 and 187,200 tokens, 12 heads of 128 channels), and generic ones.
"""
import math
import random

import torch

own = False

DEV = "cuda"
THETA = 10000.0
EPS = 1e-6
ROWS, COLS = 30, 52  # latent frame


def listed():
    f = dict(op="norm", dtype="bf16", packed=True, halves=False, pos="grid")
    b = dict(f, op="norm_back")
    c = dict(op="cross", kind="one", S=1)
    t = dict(c, op="cross_train")
    return [
        # one latent frame, as a streaming generator makes it: latency counts
        dict(f, name="norm_frame", N=1560, H=12, Hk=12, d=128),
        # the 30 s video: queries and keys read in place from a packed projection
        dict(f, name="norm_187k", N=187200, H=12, Hk=12, d=128),
        # fp32 activations, shared key heads, listed positions far along the axis, an odd number of tokens
        dict(f, name="norm_f32_odd", N=20011, H=8, Hk=2, d=64, dtype="f32", packed=False, halves=True, pos="list"),
        # the norm without rotation, with its gradients: the text states of a few prompts
        dict(b, name="norm_back_text", N=2310, H=12, Hk=12, d=128, pos="none"),
        # a training step's gradients over the 30 s video
        dict(b, name="norm_back_187k", N=187200, H=12, Hk=12, d=128),
        # one query, one short prompt: the smallest call
        dict(c, name="cross_one", N=1, L=77, H=12, Hk=12, d=128),
        # a batch of single queries over padded prompts of different lengths, shared key heads
        dict(c, name="cross_batch", N=64, L=64 * 512, S=64, kind="padded", H=16, Hk=4, d=64),
        # a few pooling queries that read a whole video: many keys, few rows
        dict(c, name="cross_pool", N=77, L=187200, H=12, Hk=12, d=128),
        # seven shots of different lengths, each with its own prompt, one of them empty
        dict(c, name="cross_shots", N=32760, L=1907, S=7, kind="ragged", H=12, Hk=12, d=128),
        # the 30 s video against one long prompt
        dict(c, name="cross_187k", N=187200, L=512, H=12, Hk=12, d=128),
        # a training step (output, then gradients) over seven shots
        dict(t, name="cross_train_shots", N=32760, L=1907, S=7, kind="ragged", H=12, Hk=12, d=128),
        # a training step over the 30 s video
        dict(t, name="cross_train_187k", N=187200, L=512, H=12, Hk=12, d=128),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    d = rng.choice([64, 128])
    H = rng.choice([1, 2, 4, 6, 8, 12, 16])
    Hk = rng.choice([h for h in range(1, H + 1) if H % h == 0])
    if rng.random() < 0.45:
        N = _log(rng, 1, 187200 * 12 * 128 // (H * d) if H * d > 1536 else 187200)
        return dict(op=rng.choice(["norm", "norm_back"]), N=N, H=H, Hk=Hk, d=d, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    packed=rng.random() < 0.5, halves=rng.random() < 0.5, pos=rng.choice(["grid", "list", "none"]))
    op = rng.choice(["cross", "cross_train"])
    kind = rng.choice(["one", "ragged", "padded"])
    S = 1 if kind == "one" else _log(rng, 2, 24)
    most = 187200 * 512 * 12 * 128
    while True:  # the plain form pads every segment to the longest: bound that work too
        N, L = _log(rng, 1, 187200), _log(rng, 16 * S, 187200)
        if kind == "padded":
            L = L // S * S
        c = dict(op=op, kind=kind, S=S, N=N, L=L, H=H, Hk=Hk, d=d)
        q, k = _split(c)
        nq, nk = max(n for _, n in q), max(n for _, n in k)
        # with a single key the gradients of q and k are 0, and what is computed for them is rounding alone
        alone = op == "cross_train" and any(a and b == 1 for (_, a), (_, b) in zip(q, k))
        if not alone and S * nq * nk * H * d <= most and S * (nq + nk) * H * d <= most // 256:
            return c


def _parts(total, S, rng):
    """total in S parts of random lengths, some of them possibly zero."""
    cut = sorted(rng.randrange(total + 1) for _ in range(S - 1))
    edge = [0] + cut + [total]
    return [(a, b - a) for a, b in zip(edge, edge[1:])]


def _split(c):
    """(start, length) of each segment's queries and keys."""
    S, N, L = c["S"], c["N"], c["L"]
    if S == 1:
        return [(0, N)], [(0, L)]
    rng = random.Random(1000003 * N + 1009 * L + S)
    if c["kind"] == "padded":
        w = L // S
        q = [(s * N // S, (s + 1) * N // S - s * N // S) for s in range(S)]
        return q, [(s * w, rng.randrange(w + 1)) for s in range(S)]
    q, k = _parts(N, S, rng), _parts(L, S, rng)
    j = rng.randrange(S)  # one segment without keys: its keys go to the next
    k = [list(p) for p in k]
    i = (j + 1) % S
    if i > j:
        k[i] = [k[j][0], k[j][1] + k[i][1]]
        k[j] = [k[j][0], 0]
    return q, [tuple(p) for p in k]


def _axes(c):
    n = c["d"] // 2
    if c["pos"] == "none":
        return (0, 0, 0)
    return (n - 2 * (n // 3), n // 3, n // 3)


def _rows(c):
    """Rows of the position table."""
    return 4096 if c["pos"] == "list" else max(-(-c["N"] // (ROWS * COLS)), ROWS, COLS)


def _freqs(c):
    """Axis of each pair and its frequency (64 bits)."""
    axis, freq = [], []
    for a, n in enumerate(_axes(c)):
        axis += [a] * n
        freq += [THETA ** (-i / n) for i in range(n)]
    return axis, freq


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    N, H, Hk, d = c["N"], c["H"], c["Hk"], c["d"]
    if c["op"].startswith("norm"):
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        if c["packed"]:  # one projection's output: queries, keys and values of a token side by side
            x = torch.empty(N, H + 2 * Hk, d, dtype=dt, device=DEV)
            x.normal_(generator=g)
            q, k = x[:, :H], x[:, H:H + Hk]
        else:
            q, k = _randn(g, N, H, d).to(dt), _randn(g, N, Hk, d).to(dt)
        s = dict(c=c, q=q, k=k, w_q=1 + 0.2 * _randn(g, d), w_k=1 + 0.2 * _randn(g, d), axes=_axes(c))
        s["table"] = s["pos"] = s["grid"] = s["ws"] = None
        if c["pos"] != "none":
            _, freq = _freqs(c)
            ang = torch.arange(_rows(c), dtype=torch.float64, device=DEV)[:, None] * torch.tensor(freq, dtype=torch.float64, device=DEV)
            s["table"] = torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()
        if c["pos"] == "list":
            s["pos"] = torch.randint(0, _rows(c), (N, 3), generator=g, device=DEV, dtype=torch.int32)
        elif c["pos"] == "grid":
            s["grid"] = (-(-N // (ROWS * COLS)), ROWS, COLS)
        if c["op"] == "norm_back":
            s["dq"] = torch.empty(N, H, d, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
            s["dk"] = torch.empty(N, Hk, d, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
        return s
    L, S = c["L"], c["S"]
    q = (1.3 * _randn(g, N, H, d)).to(torch.bfloat16)
    kv = torch.empty(L, 2, Hk, d, dtype=torch.bfloat16, device=DEV).normal_(generator=g)  # one projection of the states
    s = dict(c=c, q=q, k=kv[:, 0], v=kv[:, 1], q_off=None, kv_off=None, kv_len=None, ws=None)
    qs, ks = _split(c)
    s["q_max"], s["k_max"] = max(n for _, n in qs), max(n for _, n in ks)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    if S > 1:
        s["q_off"] = ints([a for a, _ in qs] + [N])
        s["kv_off"] = ints([a for a, _ in ks] + [L])
        if c["kind"] == "padded":
            s["kv_len"] = ints([n for _, n in ks])
    if c["op"] == "cross_train":
        s["dout"] = torch.empty(N, H, d, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    return s


# ----------------------------------------------------------------------------- plain forms
def _pairs(x, halves):
    return x.unflatten(-1, (2, -1)).unbind(-2) if halves else x.unflatten(-1, (-1, 2)).unbind(-1)


def _join(a, b, halves):
    return torch.stack([a, b], -2 if halves else -1).flatten(-2)


def _angles(s):
    """cos and sin of each token's pairs, [N, 1, d/2]; None without rotation."""
    c = s["c"]
    if c["pos"] == "none":
        return None
    if s["pos"] is not None:
        pos = s["pos"].long()
    else:
        n = torch.arange(c["N"], device=DEV)
        pos = torch.stack([n // (ROWS * COLS), n // COLS % ROWS, n % COLS], -1)
    axis = torch.tensor(_freqs(c)[0], device=DEV)
    t = s["table"][pos[:, axis], torch.arange(c["d"] // 2, device=DEV)]
    return t[:, None, :, 0], t[:, None, :, 1]


def _plain_norm(s):
    rot, halves = _angles(s), s["c"]["halves"]

    def one(x, w):
        x = x.float()
        z = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        if rot is not None:
            a, b = _pairs(z, halves)
            z = _join(a * rot[0] - b * rot[1], a * rot[1] + b * rot[0], halves)
        return z.to(torch.bfloat16)

    return {"q": one(s["q"], s["w_q"]), "k": one(s["k"], s["w_k"])}


def _plain_norm_back(s):
    rot, halves = _angles(s), s["c"]["halves"]

    def one(x, w, dy):
        dt = x.dtype
        x, dy = x.float(), dy.float()
        if rot is not None:
            a, b = _pairs(dy, halves)
            dy = _join(a * rot[0] + b * rot[1], b * rot[0] - a * rot[1], halves)
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        n = x * r
        g = dy * w
        dx = r * (g - n * (g * n).mean(-1, keepdim=True))
        return dx.to(dt), (dy * n).sum((0, 1), dtype=torch.float64).float()

    dq, dw_q = one(s["q"], s["w_q"], s["dq"])
    dk, dw_k = one(s["k"], s["w_k"], s["dk"])
    return {"dq": dq, "dk": dk, "dw_q": dw_q, "dw_k": dw_k}


def _plain_cross(s, train):
    """Every segment padded to the longest by indexing, then batched products."""
    c = s["c"]
    N, L, H, Hk, d = c["N"], c["L"], c["H"], c["Hk"], c["d"]
    zero = lambda v: torch.tensor([0, v], dtype=torch.int32, device=DEV)  # noqa: E731
    q_off = (s["q_off"] if s["q_off"] is not None else zero(N)).long()
    kv_off = (s["kv_off"] if s["kv_off"] is not None else zero(L)).long()
    k_len = s["kv_len"].long() if s["kv_len"] is not None else kv_off[1:] - kv_off[:-1]
    at = torch.arange(s["q_max"], device=DEV)
    qm = at < (q_off[1:] - q_off[:-1])[:, None]
    qi = (q_off[:-1, None] + at).clamp(max=N - 1)
    at = torch.arange(s["k_max"], device=DEV)
    km = at < k_len[:, None]
    ki = (kv_off[:-1, None] + at).clamp(max=L - 1)
    head = torch.arange(H, device=DEV) // (H // Hk)
    Q = s["q"][qi].float().transpose(1, 2)                  # [S, H, q, d]
    K = s["k"][ki].float().transpose(1, 2)[:, head]
    V = s["v"][ki].float().transpose(1, 2)[:, head]
    if s["k_max"] == 0:
        m = torch.full((len(qi), H, s["q_max"], 1), -math.inf, device=DEV)
        P, l, O = Q[..., :0], torch.zeros_like(m), torch.zeros_like(Q)
    else:
        P = (Q @ K.transpose(-1, -2)).mul_(d ** -0.5).masked_fill_(~km[:, None, None], -math.inf)
        m = P.amax(-1, keepdim=True)
        P = P.sub_(m.clamp(min=-1e30)).exp_()
        l = P.sum(-1, keepdim=True)
        P = P.div_(l.clamp(min=1e-30))
        O = P @ V
    rows = qi[qm]
    out = torch.zeros(N, H, d, dtype=torch.bfloat16, device=DEV)
    out[rows] = O.transpose(1, 2)[qm].to(torch.bfloat16)
    if not train:
        return {"out": out}
    lse = torch.full((H, N), -math.inf, device=DEV)
    lse[:, rows] = (m + l.log())[..., 0].transpose(1, 2)[qm].t()
    dO = (s["dout"][qi].float() * qm[..., None, None]).transpose(1, 2)
    dV = P.transpose(-1, -2) @ dO
    dS = (dO @ V.transpose(-1, -2)).sub_((dO * O).sum(-1, keepdim=True)).mul_(P)
    dQ, dK = dS @ K * d ** -0.5, dS.transpose(-1, -2) @ Q * d ** -0.5
    dq = torch.zeros_like(s["q"])
    dq[rows] = dQ.transpose(1, 2)[qm].to(dq.dtype)
    shared = lambda x: x.unflatten(1, (Hk, -1)).sum(2).transpose(1, 2)[km].to(torch.bfloat16)  # noqa: E731
    dk, dv = (torch.zeros(L, Hk, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dk[ki[km]], dv[ki[km]] = shared(dK), shared(dV)
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


# ----------------------------------------------------------------------------- the framework's calls
def _own(s):
    import learned_token_group_b200 as moga
    op = s["c"]["op"]
    if op.startswith("norm"):
        where = dict(table=s["table"], axes=s["axes"], grid=s["grid"], positions=s["pos"], eps=EPS, halves=s["c"]["halves"])
        if op == "norm":
            if s["pos"] is not None and s["ws"] is None:
                s["ws"] = moga.workspace(256, DEV)
            q, k = moga.qk_norm_rope(s["q"], s["k"], s["w_q"], s["w_k"], ws=s["ws"], **where)
            return {"q": q, "k": k}
        g = moga.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["w_q"], s["w_k"], ws=s["ws"], **where)
        s["ws"] = g["ws"]
        return {n: g[n] for n in ("dq", "dk", "dw_q", "dw_k")}
    seg = dict(q_offsets=s["q_off"], kv_offsets=s["kv_off"], kv_lens=s["kv_len"])
    if s["ws"] is None:  # a program keeps one workspace for its calls
        need = moga.cross_attn_workspace_size(s["q"], s["k"], segments=s["c"]["S"], backward=op == "cross_train")
        s["ws"] = moga.workspace(need, DEV)
    if op == "cross":
        return {"out": moga.cross_attn(s["q"], s["k"], s["v"], ws=s["ws"], **seg)}
    out, lse = moga.cross_attn(s["q"], s["k"], s["v"], ws=s["ws"], return_lse=True, **seg)
    g = moga.cross_attn_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, ws=s["ws"], **seg)
    return {"out": out, "lse": lse, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"]}


def run(state):
    if own:
        return _own(state)
    op = state["c"]["op"]
    if op == "norm":
        return _plain_norm(state)
    if op == "norm_back":
        return _plain_norm_back(state)
    return _plain_cross(state, op == "cross_train")


def work(case):
    c = case
    N, H, Hk, d = c["N"], c["H"], c["Hk"], c["d"]
    if c["op"].startswith("norm"):
        e = 2 if c["dtype"] == "bf16" else 4
        n = N * (H + Hk) * d
        pos = {"grid": 0, "list": 12 * N, "none": 0}[c["pos"]]
        table = 0 if c["pos"] == "none" else min(_rows(c), N * 3) * d * 4
        if c["op"] == "norm":
            return {"bytes": n * (e + 2) + pos + table, "flops": 10 * n}
        return {"bytes": n * (2 * e + 2) + pos + table, "flops": 22 * n}
    qs, ks = _split(c)
    pairs = sum(a * b for (_, a), (_, b) in zip(qs, ks))
    keys = sum(b for _, b in ks)
    if c["op"] == "cross":
        return {"bytes": 2 * d * (2 * N * H + 2 * keys * Hk), "flops": 4 * pairs * H * d}
    return {"bytes": 2 * d * (4 * N * H + 2 * keys * Hk + 2 * c["L"] * Hk) + 4 * N * H, "flops": 14 * pairs * H * d}


# ----------------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    N, H, Hk, d = c["N"], c["H"], c["Hk"], c["d"]
    if c["op"].startswith("norm"):
        return _exact_norm(s)
    out = torch.zeros(N, H, d, dtype=torch.float64, device=DEV)
    lse = torch.full((H, N), -math.inf, dtype=torch.float64, device=DEV)
    dq, dk, dv = torch.zeros_like(out), *(torch.zeros(c["L"], Hk, d, dtype=torch.float64, device=DEV) for _ in range(2))
    for (q0, nq), (k0, nk) in zip(*_split(c)):
        if nq == 0 or nk == 0:
            continue
        for h in range(H):
            g = h // (H // Hk)
            k, v = s["k"][k0:k0 + nk, g].double(), s["v"][k0:k0 + nk, g].double()
            step = max(1, (1 << 28) // nk)
            for a in range(q0, q0 + nq, step):
                r = slice(a, min(a + step, q0 + nq))
                q = s["q"][r, h].double()
                x = torch.einsum("id,jd->ij", q, k) / math.sqrt(d)
                e = torch.logsumexp(x, 1)
                p = torch.exp(x - e[:, None])
                out[r, h], lse[h, r] = p @ v, e
                if c["op"] == "cross_train":
                    do = s["dout"][r, h].double()
                    dp = torch.einsum("id,jd->ij", do, v)
                    ds = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(d)
                    dq[r, h] = ds @ k
                    dk[k0:k0 + nk, g] += ds.t() @ q
                    dv[k0:k0 + nk, g] += p.t() @ do
    if c["op"] == "cross":
        return {"out": out}
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _exact_norm(s):
    c = s["c"]
    N, d, half = c["N"], c["d"], c["d"] // 2
    turn = torch.ones(N, 1, half, dtype=torch.complex128, device=DEV)
    if c["pos"] != "none":
        if s["pos"] is not None:
            p = s["pos"].double()
        else:
            p = torch.cartesian_prod(*(torch.arange(v, device=DEV) for v in s["grid"]))[:N].double()
        axis, freq = _freqs(c)
        phase = p[:, axis] * torch.tensor(freq, dtype=torch.float64, device=DEV)
        turn = torch.polar(torch.ones_like(phase), phase)[:, None]
    first = torch.arange(half, device=DEV) * (1 if c["halves"] else 2)
    second = first + (half if c["halves"] else 1)

    def rotate(z, by):
        y = torch.complex(z[..., first], z[..., second]) * by
        o = torch.empty_like(z)
        o[..., first], o[..., second] = y.real, y.imag
        return o

    def length(x):
        return torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)

    if c["op"] == "norm":
        return {n: rotate(s[n].double() / length(s[n].double()) * s["w_" + n].double(), turn) for n in ("q", "k")}
    got = {}
    for n in ("q", "k"):
        x, w = s[n].double(), s["w_" + n].double()
        dz = rotate(s["d" + n].double(), turn.conj())
        u = length(x)
        got["dw_" + n] = (dz * x / u).sum((0, 1))
        got["d" + n] = dz * w / u - x * (dz * w * x).sum(-1, keepdim=True) / (d * u ** 3)
    return got
