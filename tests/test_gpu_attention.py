"""Attention over volume tokens against the float64 form: head layouts,
lengths from one token, odd sizes, masks that leave rows empty, strides,
garbage in masked places, gradients against the formula and differences."""
import math

import pytest
import torch

import token_reference as ref

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def ffdp():
    from voxel_grid_sampler_gb300 import build, ffdp as f
    build.build()
    return f


def _inputs(seed, B, Sq, Sk, Hq, Hk, D, dtype, axes=0, docs=0, prefix=None):
    g = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    t = dict(q=rnd(B, Sq, Hq, D), k=rnd(B, Sk, Hk, D), v=rnd(B, Sk, Hk, D), go=rnd(B, Sq, Hq, D))
    more = {}
    if axes:
        more["pos_k"] = torch.randint(0, 12, (Sk, axes), generator=g, device="cuda").float()
        more["pos_q"] = more["pos_k"] if Sq == Sk else torch.rand((B, Sq, axes), generator=g, device="cuda") * 12
        more["slopes"] = torch.rand((Hq, axes), generator=g, device="cuda")
    if docs:
        ids = lambda n: torch.sort(torch.randint(-1, docs, (B, n), generator=g, device="cuda"), 1)[0].int()  # noqa: E731
        more["doc_k"] = ids(Sk)
        more["doc_q"] = more["doc_k"] if Sq == Sk else ids(Sq)
    if prefix is not None:
        more["prefix"] = torch.tensor([(prefix + 7 * b) for b in range(B)], dtype=torch.int32, device="cuda")
    return t, more


def _check(ffdp, t, more, cap=0.0, causal=False, train=True, scale=None):
    q, k, v, go = t["q"], t["k"], t["v"], t["go"]
    scale = q.shape[3] ** -0.5 if scale is None else scale
    scale, cap = (float(torch.tensor(x, dtype=torch.float32)) for x in (scale, cap))
    p = ffdp.attention_params(scale, cap, causal)
    want = ref.attention(q, k, v, scale, cap, go=go if train else None, causal=causal, **more)
    o, lse = ffdp.ffdp_attention_fwd(q, k, v, p, **more)
    ref.within(o, *want["o"], "o")
    ref.within(lse, *want["lse"], "lse")
    if not train:
        return o, lse
    got = ffdp.ffdp_attention_bwd(q, k, v, o, lse, go, p, **more)
    for n, x in zip(("gq", "gk", "gv"), got):
        ref.within(x, *want[n], n)
    assert not ffdp.device_error()
    return (o, lse) + tuple(got)


SHAPES = [
    (1, 1, 1, 1, 1, 8), (2, 1, 300, 8, 2, 128), (1, 2, 1, 2, 2, 16), (2, 127, 129, 2, 1, 64), (1, 128, 128, 3, 3, 64),
    (1, 129, 257, 2, 2, 128), (3, 343, 343, 4, 4, 32), (1, 256, 384, 4, 2, 80), (2, 5, 1000, 6, 3, 96),
    (1, 400, 70, 2, 2, 40), (1, 33, 4000, 4, 1, 128), (1, 640, 640, 1, 1, 120),
]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("B,Sq,Sk,Hq,Hk,D", SHAPES)
def test_every_pair_visible(ffdp, B, Sq, Sk, Hq, Hk, D, dtype):
    _check(ffdp, *_inputs(Sq + Sk, B, Sq, Sk, Hq, Hk, D, dtype))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("axes", [1, 2, 3])
@pytest.mark.parametrize("B,Sq,Sk,Hq,Hk,D", [(2, 343, 343, 4, 2, 64), (2, 3, 500, 8, 2, 128), (1, 130, 270, 2, 1, 32)])
def test_distance_bias(ffdp, B, Sq, Sk, Hq, Hk, D, axes, dtype):
    _check(ffdp, *_inputs(axes, B, Sq, Sk, Hq, Hk, D, dtype, axes=axes))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("B,Sq,Sk,Hq,Hk,D", [(1, 200, 333, 2, 2, 64), (2, 4, 700, 4, 4, 128)])
def test_capped_scores(ffdp, B, Sq, Sk, Hq, Hk, D, dtype):
    t, more = _inputs(3, B, Sq, Sk, Hq, Hk, D, dtype, axes=2)
    _check(ffdp, t, {}, cap=2.0)
    _check(ffdp, t, more, cap=20.0, scale=1.0)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("prefix", [None, 0, 1, 130, 10000])
@pytest.mark.parametrize("B,Sq,Sk", [(2, 300, 300), (1, 129, 400), (2, 300, 140), (2, 2, 600), (1, 1, 50)])
def test_causal_and_prefix(ffdp, B, Sq, Sk, prefix, dtype):
    # Sq > Sk leaves the first rows without a key
    _check(ffdp, *_inputs(5, B, Sq, Sk, 4, 2, 64, dtype, prefix=prefix), causal=True)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("docs,causal", [(1, False), (4, False), (4, True), (40, False)])
@pytest.mark.parametrize("B,Sq,Sk", [(2, 500, 500), (2, 130, 700), (2, 3, 700)])
def test_documents_with_padding(ffdp, B, Sq, Sk, docs, causal, dtype):
    _check(ffdp, *_inputs(docs, B, Sq, Sk, 4, 2, 64, dtype, axes=3, docs=docs), causal=causal)


def test_documents_in_any_order(ffdp):
    t, more = _inputs(9, 2, 300, 300, 2, 2, 64, BF16, docs=5)
    g = torch.Generator("cuda").manual_seed(1)
    more["doc_k"] = more["doc_q"] = more["doc_k"][:, torch.randperm(300, generator=g, device="cuda")].contiguous()
    _check(ffdp, t, more)


def test_all_padding_gives_zero(ffdp):
    t, more = _inputs(10, 2, 140, 140, 2, 1, 64, F16, docs=1)
    more["doc_q"] = more["doc_k"] = torch.full_like(more["doc_k"], -1)
    o, lse, gq, gk, gv = _check(ffdp, t, more)
    for x in (o, gq, gk, gv):
        assert not x.any()
    assert bool((lse == -math.inf).all())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf")])
def test_what_is_masked_has_no_effect(ffdp, poison, dtype):
    # padding holds garbage: rows of q, k, v and go
    t, more = _inputs(11, 2, 300, 300, 4, 2, 64, dtype, axes=3, docs=3)
    pad = more["doc_k"] < 0
    assert bool(pad.any())
    for x in t.values():
        x[pad] = poison
    want = _check_poisoned(ffdp, t, more, pad)
    for x in want:
        assert bool(torch.isfinite(x.float()).all())


def _check_poisoned(ffdp, t, more, pad):
    q, k, v, go = t["q"], t["k"], t["v"], t["go"]
    clean = {n: x.masked_fill(pad[:, :, None, None], 0.0) for n, x in t.items()}
    scale = float(torch.tensor(q.shape[3] ** -0.5, dtype=torch.float32))
    want = ref.attention(clean["q"], clean["k"], clean["v"], scale, go=clean["go"], **more)
    p = ffdp.attention_params(scale)
    o, lse = ffdp.ffdp_attention_fwd(q, k, v, p, **more)
    got = (o,) + tuple(ffdp.ffdp_attention_bwd(q, k, v, o, lse, go, p, **more))
    for n, x in zip(("o", "gq", "gk", "gv"), got):
        ref.within(x, *want[n], n)
    return got


@pytest.mark.parametrize("Sq", [260, 2])
def test_keys_behind_the_causal_line_may_hold_anything(ffdp, Sq):
    # and another document's NaN stays in that document
    t, more = _inputs(12, 1, Sq, 260, 2, 2, 64, BF16)
    q, k, v, go = t["q"], t["k"], t["v"], t["go"]
    scale = 0.125
    p = ffdp.attention_params(scale, causal=True)
    want = ref.attention(q, k, v, scale, causal=True)
    n = 257 if Sq == 260 else 259            # rows before the first that sees the poisoned key
    k[:, 258:], v[:, 258:] = float("nan"), float("nan")
    if Sq == 2:
        k[:, 258], v[:, 258] = t["k"][:, 0], t["v"][:, 0]
        want = ref.attention(q, torch.where(torch.isnan(k), 0, k), torch.where(torch.isnan(v), 0, v), scale, causal=True)
        n = 1
    o, lse = ffdp.ffdp_attention_fwd(q, k, v, p)
    ref.within(o[:, :n], want["o"][0][:, :n], want["o"][1][:, :n])
    assert bool(torch.isnan(o[:, -1]).all())
    docs = (torch.arange(260, device="cuda") >= 200).int()
    t, _ = _inputs(13, 1, 260, 260, 2, 2, 64, BF16)
    q, k, v, go = t["q"], t["k"], t["v"], t["go"]
    want = ref.attention(q, k, v, scale, go=go, doc_q=docs, doc_k=docs)
    for x in (k, v, q, go):
        x[:, 230] = float("nan")
    p = ffdp.attention_params(scale)
    o, lse = ffdp.ffdp_attention_fwd(q, k, v, p, doc_q=docs, doc_k=docs)
    got = (o,) + tuple(ffdp.ffdp_attention_bwd(q, k, v, o, lse, go, p, doc_q=docs, doc_k=docs))
    for name, x in zip(("o", "gq", "gk", "gv"), got):
        ref.within(x[:, :200], want[name][0][:, :200], want[name][1][:, :200], name)
        assert bool(torch.isnan(x[:, 200:].float()).all()), name


def test_layouts(ffdp):
    # views of one projection, heads before tokens, padded rows; outputs likewise
    B, S, D = 2, 200, 64
    t, more = _inputs(14, B, S, S, 8, 4, D, BF16)
    want = ref.attention(t["q"], t["k"], t["v"], 0.125, go=t["go"])
    qkv = torch.cat([t["q"], t["k"], t["v"]], 2)
    q, k, v = qkv[:, :, :8], qkv[:, :, 8:12], qkv[:, :, 12:]
    p = ffdp.attention_params(0.125)
    hf = lambda x: x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)  # noqa: E731
    for q, k, v, go in ((q, k, v, t["go"]), tuple(hf(t[n]) for n in ("q", "k", "v", "go"))):
        out = torch.full((B, 8, S, 72), 7.0, dtype=BF16, device="cuda")
        o, lse = ffdp.ffdp_attention_fwd(q, k, v, p, o=out[..., :64].permute(0, 2, 1, 3))
        assert bool((out[..., 64:] == 7.0).all())
        ref.within(o, *want["o"], "o")
        grads = torch.full((B, S, 16, 64), 7.0, dtype=BF16, device="cuda")
        g = ffdp.ffdp_attention_bwd(q, k, v, o, lse, go, p, gq=grads[:, :, :8], gk=grads[:, :, 8:12], gv=grads[:, :, 12:])
        for n, x in zip(("gq", "gk", "gv"), g):
            ref.within(x, *want[n], n)


def test_offsets_past_32_bits(ffdp):
    t, more = _inputs(15, 2, 2, 200, 2, 1, 64, F16)
    big = torch.zeros(2 ** 31 + 32768, dtype=F16, device="cuda")
    k = big.as_strided((2, 200, 1, 64), (2 ** 31, 64, 64, 1))
    v = big.as_strided((2, 200, 1, 64), (2 ** 31, 64, 64, 1), 16384)
    k.copy_(t["k"]), v.copy_(t["v"])
    t["k"], t["v"] = k, v
    _check(ffdp, t, more)


def test_empty_lengths(ffdp):
    p = ffdp.attention_params(0.125)
    t, _ = _inputs(16, 2, 5, 0, 2, 1, 64, F16)
    o, lse = ffdp.ffdp_attention_fwd(t["q"], t["k"], t["v"], p)
    assert not o.any() and bool((lse == -math.inf).all())
    gq, gk, gv = ffdp.ffdp_attention_bwd(t["q"], t["k"], t["v"], o, lse, t["go"], p)
    assert not gq.any() and gk.shape == (2, 0, 1, 64)
    t, _ = _inputs(17, 2, 0, 5, 2, 1, 64, F16)
    o, lse = ffdp.ffdp_attention_fwd(t["q"], t["k"], t["v"], p)
    assert o.shape == (2, 0, 2, 64)
    gq, gk, gv = ffdp.ffdp_attention_bwd(t["q"], t["k"], t["v"], o, lse, t["go"], p)
    assert not gk.any() and not gv.any()


def test_same_bits_twice_and_on_another_stream(ffdp):
    t, more = _inputs(18, 2, 300, 300, 4, 2, 64, BF16, axes=3, docs=3)
    a = _check(ffdp, t, more)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = _check(ffdp, t, more)
    s.synchronize()
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    t, more = _inputs(19, 2, 1, 5000, 8, 2, 128, BF16, axes=3)
    a, b = _check(ffdp, t, more, train=False), _check(ffdp, t, more, train=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_large_scores_and_growing_maxima(ffdp):
    # maxima that rise tile by tile by far more than exp can hold, and scores that differ by thousands
    t, more = _inputs(20, 1, 200, 1000, 2, 2, 64, BF16)
    t["k"] *= torch.linspace(0.1, 30.0, 1000, device="cuda")[None, :, None, None].to(BF16)
    _check(ffdp, t, more, train=False, scale=1.0)


@pytest.mark.parametrize("cap,causal", [(0.0, False), (5.0, True)])
def test_gradients_against_differences(ffdp, cap, causal):
    # <g, e> against central differences of the float64 form along e
    t, more = _inputs(21, 1, 40, 50, 4, 2, 32, F16, axes=3)
    scale = 0.25
    p = ffdp.attention_params(scale, cap, causal)
    o, lse = ffdp.ffdp_attention_fwd(t["q"], t["k"], t["v"], p, **more)
    got = ffdp.ffdp_attention_bwd(t["q"], t["k"], t["v"], o, lse, t["go"], p, **more)
    want = ref.attention(t["q"], t["k"], t["v"], scale, cap, go=t["go"], causal=causal, **more)
    ref.U[torch.float64], ref.FLOOR[torch.float64] = 2.0 ** -53, 0.0
    x64 = {n: ref.d(t[n]) for n in ("q", "k", "v")}
    for n, g in zip(("q", "k", "v"), got):
        e = torch.randn(t[n].shape, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
        f = lambda h: (ref.d(t["go"]) * ref.attention(  # noqa: E731
            *({**x64, n: x64[n] + h * e}[m] for m in ("q", "k", "v")), scale, cap, causal=causal, **more)["o"][0]).sum()
        num = float((f(1e-4) - f(-1e-4)) / 2e-4)
        bound = float((want["g" + n][1] * e.abs()).sum()) + 1e-6 * abs(num)
        assert abs(float((ref.d(g) * e).sum()) - num) <= bound, n


@pytest.mark.parametrize("scale", [-0.2, 0.0])
@pytest.mark.parametrize("Sq", [2, 150])
def test_negative_and_zero_scale(ffdp, scale, Sq):
    t, more = _inputs(22, 2, Sq, 200, 4, 2, 64, BF16, axes=2, docs=2)
    _check(ffdp, t, more, scale=scale)
    _check(ffdp, t, more, scale=scale, cap=1.5)


@pytest.mark.parametrize("Sq,Hq", [(130, 1), (1, 8), (12, 2)])
def test_very_long_keys(ffdp, Sq, Hq):
    # more key tiles than one work item lists, and than a backward CTA keeps codes for
    t, more = _inputs(23, 1, Sq, 270001, Hq, 1, 32, F16, axes=1)
    more["slopes"] *= 0.01
    _check(ffdp, t, more, causal=True, train=Sq == 12)


@pytest.mark.parametrize("G,Sq", [(1, 16), (4, 4), (16, 1), (17, 1), (3, 21), (128, 1), (5, 64)])
def test_few_rows_in_every_packing(ffdp, G, Sq):
    # 16 rows per key head, just above, tiles of several heads that fill 128 rows or do not
    t, more = _inputs(24, 2, Sq, 333, 2 * G, 2, 72, BF16, axes=3, docs=2)
    _check(ffdp, t, more, train=G < 16, causal=True, cap=10.0)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("kind", ["all", "bias", "causal", "documents", "one", "nan"])
@pytest.mark.parametrize("Sq,D", [(100, 64), (300, 32), (257, 40)])
def test_odd_number_of_query_tiles(ffdp, Sq, D, kind, dtype):
    # enough heads that the keys are not split over CTAs; the last tile of each
    # head has a CTA to itself
    bias, docs = kind == "bias", {"documents": 6, "one": 1, "nan": 2}.get(kind, 0)
    t, more = _inputs(Sq, 2, Sq, 530, 80, 80, D, dtype, axes=3 if bias else 0, docs=docs)
    if kind == "one":  # a single visible key in a single tile, and sequences without any
        more["doc_q"] = torch.zeros_like(more["doc_q"])
        more["doc_k"] = torch.full_like(more["doc_k"], -1)
        more["doc_k"][0, 400] = 0
    if kind != "nan":
        _check(ffdp, t, more, causal=kind == "causal", train=False)
        return
    # garbage in the keys that no row sees
    more["doc_q"] = torch.zeros_like(more["doc_q"])
    hidden = (more["doc_k"] != 0)[:, :, None, None]
    o, lse = _check(ffdp, t, more, train=False)
    p = ffdp.attention_params(float(torch.tensor(D ** -0.5, dtype=torch.float32)))
    o2, lse2 = ffdp.ffdp_attention_fwd(t["q"], t["k"].masked_fill(hidden, float("nan")),
                                       t["v"].masked_fill(hidden, float("inf")), p, **more)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("Sq,Sk,docs,causal,cap", [(100, 100, 7, True, 0.0), (30, 30, 0, False, 0.0), (31, 40, 0, True, 3.0),
                                                   (300, 300, 40, False, 0.0)])
def test_gradients_of_rows_with_few_keys(ffdp, Sq, Sk, docs, causal, cap, dtype):
    # two roundings of one size (dS, the result) are sqrt(2) of one; the rounding
    # of o must not add a third: that is 1.6 and more on these inputs
    t, more = _inputs(Sq, 3, Sq, Sk, 4, 2, 64, dtype, axes=2 if docs == 7 else 0, docs=docs)
    if docs:
        more["doc_k"] = more["doc_q"] = (torch.arange(Sq, device="cuda") * docs // Sq).int().expand(3, Sq).contiguous()
    q, k, v, go = t["q"], t["k"], t["v"], t["go"]
    o, lse, gq, gk, gv = _check(ffdp, t, more, cap=cap, causal=causal)
    scale = float(torch.tensor(64 ** -0.5, dtype=torch.float32))
    want = ref.attention(q, k, v, scale, cap, go=go, causal=causal, **more)
    for n, x in (("gq", gq), ("gk", gk)):
        w = want[n][0].double().cpu()
        off, own = ((y.double() - w).norm() for y in (x.cpu(), w.to(dtype)))
        assert off <= 1.55 * own, (n, float(off / own))


@pytest.mark.parametrize("B", [3, 600])
@pytest.mark.parametrize("causal", [False, True])
def test_documents_of_few_and_many_sequences(ffdp, B, causal):
    # work is ordered by length up to 1024 units, taken as it comes above
    t, more = _inputs(B, B, 150, 150, 2, 1, 16, F16, docs=5)
    _check(ffdp, t, more, causal=causal)


@pytest.mark.parametrize("axes", [0, 3])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_query_tiles_of_a_pair_that_see_different_keys(ffdp, D, axes):
    # the pair's first query tile lies in a short document, the second reaches
    # into a long one: the first skips many key tiles in the middle of the walk
    t, more = _inputs(D, 2, 1954, 1954, 8, 8, D, BF16, axes=axes)
    ids = torch.full((1954,), -1, dtype=torch.int32, device="cuda")
    for i, (a, b) in enumerate(((0, 317), (317, 952), (952, 1905))):
        ids[a:b] = i
    more["doc_q"] = more["doc_k"] = ids.expand(2, 1954).contiguous()
    _check(ffdp, t, more)
