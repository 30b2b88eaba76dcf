"""The operators of a transformer over volume tokens, as cases to time and compare.

Three operators, each in a plain form (elementary torch operations in 32
bits, rounded once at the end) and as the library's entry points:

* rope: rotary positions with the three axes (z, y, x) of a volume's tokens;
* attention: scores capped by a tanh, biased by the distance of two tokens,
  masked by document (several volumes packed in one sequence) or causally
  with a visible prefix;
* linear: act(x W^T + b) + r, the matrix product with its epilogue.
"""
import math

import torch

own = False  # True: run() calls the library; False: the plain form

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one point's token: what a query of the displacement at a single point pays, all latency
        dict(name="rope_point", op="rope", way="fwd", type="bf16", B=1, d=1, h=1, w=1, Hq=16, Hk=4, D=128,
             n0=21, n1=21, n2=22, interleaved=False, fused=False),
        # two 160 x 192 x 224 volumes in patches of 8, q and k as views of one projection's output
        dict(name="rope_volume", op="rope", way="fwd", type="bf16", B=2, d=20, h=24, w=28, Hq=16, Hk=16, D=64,
             n0=10, n1=11, n2=11, interleaved=False, fused=True),
        # gradients in 32 bits: odd grid, interleaved pairs, the last 8 of 80 channels unrotated
        dict(name="rope_grad", op="rope", way="bwd", type="f32", B=3, d=11, h=13, w=9, Hq=12, Hk=12, D=80,
             n0=12, n1=12, n2=12, interleaved=True, fused=False),
        # the displacement asked at one point of each of four volumes, over the volume's cached tokens
        dict(name="attn_point", op="attn", way="fwd", type="bf16", B=4, Sq=1, Sk=13440, Hq=16, Hk=4, D=128,
             h=24, w=28, cap=0.0, bias=True, docs=0, causal=False, prefix=0),
        # attention inside 7^3 windows: many short odd sequences
        dict(name="attn_windows", op="attn", way="fwd", type="f16", B=216, Sq=343, Sk=343, Hq=8, Hk=8, D=32,
             h=7, w=7, cap=0.0, bias=True, docs=0, causal=False, prefix=0),
        # a whole 160 x 192 x 224 volume in patches of 8, every token against every token
        dict(name="attn_volume", op="attn", way="fwd", type="bf16", B=1, Sq=13440, Sk=13440, Hq=16, Hk=16, D=64,
             h=24, w=28, cap=0.0, bias=True, docs=0, causal=False, prefix=0),
        # training on packed crops of unequal size with padding at the end, shared key heads, capped scores
        dict(name="attn_packed_train", op="attn", way="train", type="bf16", B=2, Sq=4096, Sk=4096, Hq=16, Hk=4, D=128,
             h=16, w=16, cap=30.0, bias=False, docs=5, causal=False, prefix=0),
        # training a token-by-token decoder of displacements behind a visible prefix of image tokens, odd length
        dict(name="attn_prefix_train", op="attn", way="train", type="f16", B=3, Sq=1681, Sk=1681, Hq=12, Hk=12, D=64,
             h=12, w=14, cap=0.0, bias=True, docs=0, causal=True, prefix=345),
        # one token through the wide layer of a block: the weights' bytes and latency
        dict(name="linear_point", op="linear", way="fwd", type="bf16", M=1, K=1024, N=4096, act="gelu", bias=True,
             residual=True),
        # a volume's tokens through the wide layer of a block
        dict(name="linear_volume", op="linear", way="fwd", type="bf16", M=13440, K=1024, N=4096, act="gelu", bias=True,
             residual=False),
        # training step of the narrowing layer, with the block's residual
        dict(name="linear_project_train", op="linear", way="train", type="bf16", M=13440, K=4096, N=1024, act="none",
             bias=True, residual=True),
        # training step of a patch embedding: two 5^3 patches per token, nothing a multiple of 8
        dict(name="linear_patch_train", op="linear", way="train", type="f16", M=4099, K=250, N=771, act="silu",
             bias=True, residual=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "attn", "attn", "linear", "linear"))
    if op == "rope":
        D = 8 * rng.randint(4, 16)
        R = rng.choice((D // 2, max(3, D // 2 - rng.randint(0, 6))))
        n0 = rng.randint(1, R - 2)
        n1 = rng.randint(1, R - n0 - 1)
        Hk = rng.choice((1, 2, 4, 8, 12))
        return dict(op="rope", way=rng.choice(("fwd", "bwd")), type=rng.choice(("f32", "f16", "bf16")),
                    B=rng.randint(1, 3), d=_log(rng, 1, 20), h=_log(rng, 1, 24), w=_log(rng, 1, 28),
                    Hq=Hk * rng.choice((1, 2, 4) if Hk < 8 else (1,)), Hk=Hk, D=D, n0=n0, n1=n1, n2=R - n0 - n1,
                    interleaved=rng.random() < 0.5, fused=rng.random() < 0.5)
    if op == "attn":
        way = rng.choice(("fwd", "train", "point"))
        D = rng.choice((32, 64, 64, 80, 96, 128, 128))
        Hk = rng.choice((1, 2, 4, 8))
        Hq = Hk * rng.choice((1, 2, 4) if Hk < 8 else (1, 2))
        h, w = rng.randint(3, 24), rng.randint(3, 28)
        c = dict(op="attn", way="fwd" if way == "point" else way, type=rng.choice(("f16", "bf16")), Hq=Hq, Hk=Hk, D=D,
                 h=h, w=w, cap=rng.choice((0.0, 0.0, 30.0)), bias=rng.random() < 0.6, causal=rng.random() < 0.4,
                 docs=0, prefix=0)
        if way == "point":
            c.update(B=rng.randint(1, 8), Sq=rng.randint(1, 8), Sk=_log(rng, 100, 13440))
        else:
            S = _log(rng, 64, 6000)
            B = rng.choice((1, 2, 3))
            c.update(B=B, Sq=S, Sk=S, docs=rng.choice((0, 0, 3, 7)))
        if c["causal"]:
            c["prefix"] = rng.choice((0, rng.randint(1, c["Sk"])))
        return c
    M, K, N = _log(rng, 1, 13440), _log(rng, 64, 4096), _log(rng, 64, 4096)
    return dict(op="linear", way=rng.choice(("fwd", "train")), type=rng.choice(("f16", "bf16")), M=M, K=K, N=N,
                act=rng.choice(("none", "gelu", "silu")), bias=rng.random() < 0.8, residual=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _padded(gen, rows, cols, dtype, scale=1.0):
    """[rows][cols] normal values in rows that start on 16 bytes."""
    ld = -(-cols // 8) * 8
    return (torch.randn((rows, ld), generator=gen, device="cuda") * scale).to(dtype)[:, :cols]


def _grid_positions(index, h, w):
    """(z, y, x) of tokens in raster order, slices twice as far apart as rows."""
    return torch.stack((2.0 * (index // (h * w)), ((index // w) % h).float(), (index % w).float()), -1).contiguous()


def _document_lengths(S, docs):
    """Unequal lengths and the padding left at the end (about S / 40 tokens)."""
    pad = S // 40
    total = docs * (docs + 1) // 2
    ends = [(S - pad) * (i * (i + 1) // 2) // total for i in range(docs + 1)]
    return [b - a for a, b in zip(ends, ends[1:])]


def _prepare_rope(c, gen):
    dtype = TYPES[c["type"]]
    B, S, Hq, Hk, D = c["B"], c["d"] * c["h"] * c["w"], c["Hq"], c["Hk"], c["D"]
    if c["fused"]:
        x = torch.randn((B, S, Hq + 2 * Hk, D), generator=gen, device="cuda").to(dtype)
        q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hk]
    else:
        q = torch.randn((B, S, Hq, D), generator=gen, device="cuda").to(dtype)
        k = torch.randn((B, S, Hk, D), generator=gen, device="cuda").to(dtype)
    pos = _grid_positions(torch.arange(S, device="cuda"), c["h"], c["w"])
    pos = pos + torch.rand(3, generator=gen, device="cuda")  # where the crop begins
    sections = (c["n0"], c["n1"], c["n2"])
    freq = torch.cat([100.0 ** (-torch.arange(n, dtype=torch.float32) / n) for n in sections]).cuda()
    axis = torch.cat([torch.full((n,), a, dtype=torch.int64) for a, n in enumerate(sections)]).cuda()
    return dict(q=q, k=k, pos=pos, freq=freq, axis=axis, sections=sections)


def _prepare_attn(c, gen):
    dtype = TYPES[c["type"]]
    B, Sq, Sk, Hq, Hk, D = c["B"], c["Sq"], c["Sk"], c["Hq"], c["Hk"], c["D"]

    def normal(S, H):
        return torch.randn((B, S, H, D), generator=gen, device="cuda").to(dtype)

    s = dict(q=normal(Sq, Hq), k=normal(Sk, Hk), v=normal(Sk, Hk), scale=D ** -0.5)
    s["go"] = normal(Sq, Hq) if c["way"] == "train" else None
    index = torch.arange(Sk, device="cuda")
    s["doc"] = None
    if c["docs"]:
        lengths = _document_lengths(Sk, c["docs"])
        ids = torch.full((Sk,), -1, dtype=torch.int32)
        first = torch.zeros((Sk,), dtype=torch.int64)
        at = 0
        for i, n in enumerate(lengths):
            ids[at:at + n], first[at:at + n] = i, at
            at += n
        s["doc"] = ids.cuda().expand(B, Sk).contiguous()
        index = index - first.cuda()
    s["pos_q"] = s["pos_k"] = s["slopes"] = None
    if c["bias"]:
        s["pos_k"] = _grid_positions(index, c["h"], c["w"])
        if Sq == Sk:
            s["pos_q"] = s["pos_k"]
        else:  # points anywhere in the volume
            top = s["pos_k"].amax(0)
            s["pos_q"] = torch.rand((B, Sq, 3), generator=gen, device="cuda") * top
        head = torch.arange(1, Hq + 1, device="cuda", dtype=torch.float32)
        s["slopes"] = (2.0 ** (-8.0 * head / Hq))[:, None] * torch.tensor([1.0, 0.75, 0.75], device="cuda")
    s["prefix"] = torch.full((B,), c["prefix"], dtype=torch.int32, device="cuda") if c["prefix"] else None
    return s


def _prepare_linear(c, gen):
    dtype = TYPES[c["type"]]
    M, K, N = c["M"], c["K"], c["N"]
    return dict(x=_padded(gen, M, K, dtype), w=_padded(gen, N, K, dtype, K ** -0.5),
                bias=torch.randn((N,), generator=gen, device="cuda").to(dtype) if c["bias"] else None,
                residual=_padded(gen, M, N, dtype) if c["residual"] else None,
                gy=_padded(gen, M, N, dtype) if c["way"] == "train" else None)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    make = {"rope": _prepare_rope, "attn": _prepare_attn, "linear": _prepare_linear}[case["op"]]
    state = make(case, gen)
    state["case"] = case
    return state


# ------------------------------------------------------------- plain forms
def _plain_rope_one(x, cos, sin, R, interleaved):
    x32 = x.float()
    if interleaved:
        a, b = x32[..., 0:2 * R:2], x32[..., 1:2 * R:2]
    else:
        a, b = x32[..., :R], x32[..., R:2 * R]
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((turned, x32[..., 2 * R:]), -1).to(x.dtype)


def _plain_rope(s):
    c = s["case"]
    angle = s["pos"][:, s["axis"]] * s["freq"]
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    if c["way"] == "bwd":
        sin = -sin
    R = sum(s["sections"])
    return (_plain_rope_one(s["q"], cos, sin, R, c["interleaved"]),
            _plain_rope_one(s["k"], cos, sin, R, c["interleaved"]))


def _visible(c, s):
    """[B or 1][1][Sq][Sk] truth values, or None where every pair is visible."""
    Sq, Sk = c["Sq"], c["Sk"]
    seen = None
    if c["causal"]:
        i = torch.arange(Sq, device="cuda")[:, None] + (Sk - Sq)
        j = torch.arange(Sk, device="cuda")[None]
        seen = (j <= i)[None, None]
        if s["prefix"] is not None:
            seen = seen | (j[None, None] < s["prefix"][:, None, None, None])
    if s["doc"] is not None:
        d = s["doc"]
        same = ((d[:, :, None] == d[:, None]) & (d >= 0)[:, :, None])[:, None]
        seen = same if seen is None else seen & same
    return seen


def _plain_attn(s):
    c = s["case"]
    B, Sq, Sk, Hq, Hk, D = c["B"], c["Sq"], c["Sk"], c["Hq"], c["Hk"], c["D"]
    G = Hq // Hk
    rows = lambda t: t.float().transpose(1, 2).reshape(B, Hk, G * Sq, D)  # noqa: E731
    q = rows(s["q"])
    k, v = s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2)
    a = (q @ k.transpose(2, 3)) * s["scale"]
    t = None
    if c["cap"]:
        t = torch.tanh(a / c["cap"])
        a = c["cap"] * t
    a = a.view(B, Hq, Sq, Sk)
    if c["bias"]:
        pq, pk, m = s["pos_q"], s["pos_k"], s["slopes"]
        pq = pq if pq.dim() == 3 else pq[None]
        far = (pq[:, :, None] - pk[None, None]).abs()[:, None]
        a = a - (m[:, 0, None, None] * far[..., 0] + m[:, 1, None, None] * far[..., 1] + m[:, 2, None, None] * far[..., 2])
    seen = _visible(c, s)
    if seen is not None:
        a = a.masked_fill(~seen, -math.inf)
    top = a.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(a - top)
    del a
    p = (p / p.sum(-1, keepdim=True).clamp_min(1e-38)).view(B, Hk, G * Sq, Sk)
    o = p @ v
    back = lambda x, H: x.view(B, H, -1, D).transpose(1, 2).to(s["q"].dtype).contiguous()  # noqa: E731
    if c["way"] == "fwd":
        return back(o, Hq)
    go = rows(s["go"])
    gv = p.transpose(2, 3) @ go
    delta = (go * o).sum(-1, keepdim=True)
    ds = p * (go @ v.transpose(2, 3) - delta)
    del p
    if t is not None:
        ds = ds * (1 - t * t)
    ds = ds * s["scale"]
    return back(o, Hq), back(ds @ k, Hq), back(ds.transpose(2, 3) @ q, Hk), back(gv, Hk)


def _plain_linear(s):
    c = s["case"]
    dtype = s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    if c["act"] == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        y = z * cdf
    elif c["act"] == "silu":
        cdf = 1 / (1 + torch.exp(-z))
        y = z * cdf
    else:
        y = z
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y.to(dtype)
    if c["way"] == "fwd":
        return y
    gz = s["gy"].float()
    if c["act"] == "gelu":
        gz = gz * (cdf + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    elif c["act"] == "silu":
        gz = gz * (cdf * (1 + z * (1 - cdf)))
    grads = ((gz @ w).to(dtype), (gz.t() @ x).to(dtype))
    return (y,) + grads + ((gz.sum(0).to(dtype),) if s["bias"] is not None else ())


# ------------------------------------------------------------- the library
def _own_rope(s):
    from voxel_grid_sampler_gb300 import ffdp
    c = s["case"]
    call = ffdp.ffdp_rope_fwd if c["way"] == "fwd" else ffdp.ffdp_rope_bwd
    return call(s["q"], s["pos"], s["freq"], s["sections"], c["interleaved"], s["k"])


def _own_attn(s):
    from voxel_grid_sampler_gb300 import ffdp
    c = s["case"]
    p = ffdp.attention_params(s["scale"], cap=c["cap"], causal=c["causal"])
    more = dict(pos_q=s["pos_q"], pos_k=s["pos_k"], slopes=s["slopes"], doc_q=s["doc"], doc_k=s["doc"],
                prefix=s["prefix"])
    if c["way"] == "fwd":
        return ffdp.ffdp_attention_fwd(s["q"], s["k"], s["v"], p, want_lse=False, **more)[0]
    o, lse = ffdp.ffdp_attention_fwd(s["q"], s["k"], s["v"], p, **more)
    return (o,) + tuple(ffdp.ffdp_attention_bwd(s["q"], s["k"], s["v"], o, lse, s["go"], p, **more))


def _own_linear(s):
    from voxel_grid_sampler_gb300 import ffdp
    c = s["case"]
    train = c["way"] == "train"
    y, z = ffdp.ffdp_linear_fwd(s["x"], s["w"], s["bias"], s["residual"], c["act"], want_z=train)
    if not train:
        return y
    gx, gw, gb = ffdp.ffdp_linear_bwd(s["x"], s["w"], z, s["gy"], c["act"], want_gb=s["bias"] is not None)
    return (y, gx, gw) + ((gb,) if gb is not None else ())


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "attn": _own_attn, "linear": _own_linear}[op](state)
    return {"rope": _plain_rope, "attn": _plain_attn, "linear": _plain_linear}[op](state)


# -------------------------------------------------------------------- work
def _pairs(c):
    """Visible (query, key) pairs of one head of one sequence."""
    Sq, Sk = c["Sq"], c["Sk"]
    lengths = _document_lengths(Sk, c["docs"]) if c["docs"] else None
    if not c["causal"]:
        return sum(n * n for n in lengths) if lengths else Sq * Sk
    count = 0
    at = 0
    for n in lengths or [Sk]:
        for j in range(n):  # queries of this document that see key at + j
            if lengths is None:
                count += Sq if j < c["prefix"] else max(0, min(Sq, Sk - j))
            else:
                count += n if at + j < c["prefix"] else n - j
        at += n
    return count


def work(case):
    c = case
    el = 4 if c.get("type") == "f32" else 2
    if c["op"] == "rope":
        S = c["d"] * c["h"] * c["w"]
        H = c["Hq"] + c["Hk"]
        R = c["n0"] + c["n1"] + c["n2"]
        return {"bytes": 2 * c["B"] * S * H * c["D"] * el + 12 * S + 4 * R, "flops": 6 * c["B"] * S * H * R}
    if c["op"] == "attn":
        q = c["B"] * c["Sq"] * c["Hq"] * c["D"] * el
        k = c["B"] * c["Sk"] * c["Hk"] * c["D"] * el
        flops = c["B"] * c["Hq"] * _pairs(c) * c["D"]
        if c["way"] == "fwd":
            return {"bytes": 2 * q + 2 * k, "flops": 4 * flops}
        return {"bytes": 4 * q + 4 * k, "flops": 14 * flops}  # q, go, o, gq; k, v, gk, gv
    M, K, N = c["M"], c["K"], c["N"]
    bytes_ = el * (M * K + N * K + M * N * (2 if c["residual"] else 1) + (N if c["bias"] else 0))
    if c["way"] == "fwd":
        return {"bytes": bytes_, "flops": 2 * M * N * K}
    return {"bytes": bytes_ + el * (M * N + M * K + N * K + (N if c["bias"] else 0)), "flops": 6 * M * N * K}


# ------------------------------------------------------------ in 64 bits
def _exact_rope(c, s):
    def turn(x):
        x = x.double()
        out = x.clone()
        R = sum(s["sections"])
        k = 0
        for a, n in enumerate(s["sections"]):
            for _ in range(n):
                t = (s["pos"][:, a].double() * s["freq"][k].double())[None, :, None]
                t = -t if c["way"] == "bwd" else t
                i, j = (2 * k, 2 * k + 1) if c["interleaved"] else (k, k + R)
                out[..., i] = x[..., i] * torch.cos(t) - x[..., j] * torch.sin(t)
                out[..., j] = x[..., j] * torch.cos(t) + x[..., i] * torch.sin(t)
                k += 1
        return out

    return turn(s["q"]), turn(s["k"])


def _exact_attn(c, s):
    B, Sq, Sk, Hq, Hk = c["B"], c["Sq"], c["Sk"], c["Hq"], c["Hk"]
    train = c["way"] == "train"
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    gq = torch.zeros_like(o)
    gk = torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda")
    gv = torch.zeros_like(gk)
    j = torch.arange(Sk, device="cuda")
    i = torch.arange(Sq, device="cuda")
    for b in range(B):
        hidden = torch.zeros((Sq, Sk), dtype=torch.bool, device="cuda")
        if c["causal"]:
            hidden |= (j[None] > i[:, None] + Sk - Sq) & (j[None] >= c["prefix"])
        if s["doc"] is not None:
            d = s["doc"][b]
            hidden |= (d[:, None] != d[None]) | (d[:, None] < 0)
        for h in range(Hq):
            q, k, v = s["q"][b, :, h].double(), s["k"][b, :, h * Hk // Hq].double(), s["v"][b, :, h * Hk // Hq].double()
            e = torch.mm(q, k.T) * s["scale"]
            if c["cap"]:
                slope = torch.cosh(e / c["cap"]).pow(-2)
                e = torch.tanh(e / c["cap"]) * c["cap"]
            if c["bias"]:
                pq = s["pos_q"][b] if s["pos_q"].dim() == 3 else s["pos_q"]
                for a in range(3):
                    e -= s["slopes"][h, a].double() * (pq[:, a].double()[:, None] - s["pos_k"][:, a].double()[None]).abs()
            e[hidden] = -math.inf
            p = torch.softmax(e, -1)
            del e
            p[hidden.all(-1)] = 0.0
            o[b, :, h] = torch.mm(p, v)
            if train:
                go = s["go"][b, :, h].double()
                g = h * Hk // Hq
                gv[b, :, g] += torch.mm(p.T, go)
                dp = torch.mm(go, v.T)
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * s["scale"]
                if c["cap"]:
                    ds *= slope
                gq[b, :, h] = torch.mm(ds, k)
                gk[b, :, g] += torch.mm(ds.T, q)
    return (o, gq, gk, gv) if train else o


def _exact_linear(c, s):
    x, w = s["x"].double(), s["w"].double()
    z = torch.mm(x, w.T)
    if s["bias"] is not None:
        z += s["bias"].double()
    # act and its derivative
    if c["act"] == "gelu":
        phi = torch.special.ndtr(z)
        y, slope = z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    elif c["act"] == "silu":
        g = torch.sigmoid(z)
        y, slope = z * g, g + z * g * (1 - g)
    else:
        y, slope = z.clone(), torch.ones_like(z)
    if s["residual"] is not None:
        y += s["residual"].double()
    if c["way"] == "fwd":
        return y
    gz = s["gy"].double() * slope
    out = (y, torch.mm(gz, w), torch.mm(gz.T, x))
    return out + ((gz.sum(0),) if s["bias"] is not None else ())


def exact(case, seed):
    state = prepare(case, seed)
    with torch.no_grad():
        return {"rope": _exact_rope, "attn": _exact_attn, "linear": _exact_linear}[case["op"]](case, state)
