"""act(x w^T + b) + r and its gradients against the float64 form: one row to
many, odd sizes, padded rows, every activation, optional parts."""
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


def _matrix(g, rows, cols, dtype, scale=1.0, pad=0):
    ld = -(-cols // 8) * 8 + pad
    return (torch.randn((rows, ld), generator=g, device="cuda") * scale).to(dtype)[:, :cols]


def _inputs(seed, M, K, N, dtype, pad=0):
    g = torch.Generator("cuda").manual_seed(seed)
    return dict(x=_matrix(g, M, K, dtype, pad=pad), w=_matrix(g, N, K, dtype, K ** -0.5, pad=pad),
                b=torch.randn(N, generator=g, device="cuda").to(dtype), r=_matrix(g, M, N, dtype, pad=pad),
                gy=_matrix(g, M, N, dtype, pad=pad))


def _check(ffdp, t, act, bias=True, residual=True, train=True):
    x, w, gy = t["x"], t["w"], t["gy"]
    b, r = t["b"] if bias else None, t["r"] if residual else None
    want = ref.linear(x, w, b, r, act)
    y, z = ffdp.ffdp_linear_fwd(x, w, b, r, act, want_z=True)
    ref.within(y, *want["y"], "y")
    assert (z is None) == (act == "none")
    if z is not None:
        ref.within(z, *want["z"], "z")
    if not train:
        return y
    want = ref.linear_grads(x, w, z, gy, act)
    got = ffdp.ffdp_linear_bwd(x, w, z, gy, act)
    for n, a in zip(("gx", "gw", "gb"), got):
        ref.within(a, *want[n], n)
    assert not ffdp.device_error()
    return (y,) + got


SHAPES = [(1, 64, 64), (1, 1, 1), (2, 250, 771), (7, 1024, 512), (16, 333, 129), (17, 64, 4096), (64, 96, 40),
          (100, 8, 8), (128, 256, 128), (129, 257, 130), (300, 1000, 260), (1000, 40, 24), (4099, 250, 771), (33, 5000, 65)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_shapes(ffdp, M, K, N, dtype):
    _check(ffdp, _inputs(M + K, M, K, N, dtype), "gelu")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("M", [3, 200])
def test_epilogues(ffdp, M, act, bias, residual, dtype):
    _check(ffdp, _inputs(5, M, 72, 136, dtype), act, bias, residual)


def test_padded_rows_are_neither_read_nor_written(ffdp):
    for M in (4, 150):
        t = _inputs(6, M, 50, 70, BF16, pad=16)
        for n in ("x", "w", "r", "gy"):
            full = t[n].as_strided((t[n].shape[0], t[n].stride(0)), (t[n].stride(0), 1))
            full[:, t[n].shape[1]:] = float("nan")
        y = torch.full((M, 88), 7.0, dtype=BF16, device="cuda")
        gx = torch.full((M, 72), 7.0, dtype=BF16, device="cuda")
        gw = torch.full((70, 72), 7.0, dtype=BF16, device="cuda")
        z = torch.full((M, 88), 7.0, dtype=BF16, device="cuda")
        ffdp.ffdp_linear_fwd(t["x"], t["w"], t["b"], t["r"], "silu", y=y[:, :70], z=z[:, :70])
        ref.within(y[:, :70], *ref.linear(t["x"], t["w"], t["b"], t["r"], "silu")["y"])
        ffdp.ffdp_linear_bwd(t["x"], t["w"], z[:, :70], t["gy"], "silu", gx=gx[:, :50], gw=gw[:, :50])
        want = ref.linear_grads(t["x"], t["w"], z[:, :70], t["gy"], "silu")
        ref.within(gx[:, :50], *want["gx"])
        ref.within(gw[:, :50], *want["gw"])
        for m, n in ((y, 70), (z, 70), (gx, 50), (gw, 50)):
            assert bool((m[:, n:] == 7.0).all())


def test_residual_in_place_and_parts_of_the_backward(ffdp):
    t = _inputs(7, 150, 64, 136, F16)
    want = ref.linear(t["x"], t["w"], t["b"], t["r"], "gelu")["y"]
    y = t["r"].clone()
    ffdp.ffdp_linear_fwd(t["x"], t["w"], t["b"], y, "gelu", y=y)
    ref.within(y, *want)
    want = ref.linear_grads(t["x"], t["w"], t["gy"], t["gy"], "none")
    for part in ("gx", "gw", "gb"):
        got = ffdp.ffdp_linear_bwd(t["x"], t["w"], None, t["gy"], want_gx=part == "gx", want_gw=part == "gw",
                                   want_gb=part == "gb")
        for n, a in zip(("gx", "gw", "gb"), got):
            assert (a is None) == (n != part)
            if a is not None:
                ref.within(a, *want[n])


def test_no_rows(ffdp):
    t = _inputs(8, 0, 64, 40, BF16)
    y, z = ffdp.ffdp_linear_fwd(t["x"], t["w"], t["b"], t["r"], "gelu", want_z=True)
    assert y.shape == (0, 40)
    gx, gw, gb = ffdp.ffdp_linear_bwd(t["x"], t["w"], z, t["gy"], "gelu")
    assert gx.shape == (0, 64) and not gw.any() and not gb.any()


def test_non_finite_values_reach_their_own_rows_only(ffdp):
    t = _inputs(9, 200, 64, 136, BF16)
    want = ref.linear(t["x"], t["w"], t["b"], None, "gelu")["y"]
    t["x"][130, 5] = float("nan")
    y, _ = ffdp.ffdp_linear_fwd(t["x"], t["w"], t["b"], None, "gelu")
    keep = [i for i in range(200) if i != 130]
    ref.within(y[keep], want[0][keep], want[1][keep])
    assert bool(torch.isnan(y[130]).all())


def test_same_bits_twice_and_on_another_stream(ffdp):
    t = _inputs(10, 3000, 136, 72, BF16)
    a = _check(ffdp, t, "silu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = _check(ffdp, t, "silu")
    s.synchronize()
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_offsets_past_32_bits(ffdp):
    # rows 2^22 elements apart: the last of 600 starts past 2^31 elements
    t = _inputs(11, 600, 24, 40, F16)
    x = torch.zeros(600 * 2 ** 22, dtype=F16, device="cuda").as_strided((600, 24), (2 ** 22, 1))
    x.copy_(t["x"])
    t["x"] = x
    _check(ffdp, t, "none")


@pytest.mark.parametrize("act", ["gelu", "silu", "none"])
def test_gradients_against_differences(ffdp, act):
    t = _inputs(12, 30, 40, 24, F16)
    y, z = ffdp.ffdp_linear_fwd(t["x"], t["w"], t["b"], None, act, want_z=True)
    gx, gw, gb = ffdp.ffdp_linear_bwd(t["x"], t["w"], z, t["gy"], act)
    x, w, b, gy = (ref.d(t[n]) for n in ("x", "w", "b", "gy"))
    z64 = x @ w.T + b
    want = ref.linear_grads(t["x"], t["w"], z64, t["gy"], act)
    # z is rounded to float16 between the passes: gz moves by at most |gy| |act''| u |z|, |act''| < 1
    ez = gy.abs() * ref.U[F16] * z64.abs() * (act != "none")
    more = {"gx": ez @ w.abs(), "gw": ez.T @ x.abs(), "gb": ez.sum(0)}
    f = lambda x, w, b: (gy * ref.act(act, x @ w.T + b)[0]).sum()  # noqa: E731
    for n, g, at in (("gx", gx, 0), ("gw", gw, 1), ("gb", gb, 2)):
        e = torch.randn(g.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(2))
        arg = lambda h: [v + h * e if i == at else v for i, v in enumerate((x, w, b))]  # noqa: E731
        num = float((f(*arg(1e-4)) - f(*arg(-1e-4))) / 2e-4)
        bound = float(((want[n][1] + more[n]) * e.abs()).sum()) + 1e-6 * abs(num)
        assert abs(float((ref.d(g) * e).sum()) - num) <= bound, n
