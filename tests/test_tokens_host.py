"""Host-side checks of the token operators' entry points (no GPU needed):
refusals before anything is enqueued, workspaces, and the float64 reference's
own gradients against central differences."""
import ctypes

import pytest
import torch

import token_reference as ref


@pytest.fixture(scope="module")
def lib():
    from voxel_grid_sampler_gb300 import build, ffdp
    build.build()
    return ffdp.lib()


nogpu = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only validation checks")
fake, odd = 0x10000, 0x10004   # never dereferenced: every call below is refused


def _rope(lib, **kw):
    from voxel_grid_sampler_gb300 import ffdp
    a = dict(batch=2, tokens=5, head_dim=32, axes=3, sections=(4, 4, 8), heads=2, dt=1, x=fake, n=1, pos=fake, freq=fake)
    a.update(kw)
    v = ffdp.ffdp_heads(a["x"], 320, 64, 32)
    t = (ffdp.ffdp_rope_tensor * 3)(*[ffdp.ffdp_rope_tensor(v, v, a["heads"])] * 3)
    p = ffdp.ffdp_rope_params(a["batch"], a["tokens"], a["head_dim"], a["axes"], (ctypes.c_int * 3)(*a["sections"]), 0)
    return lib.ffdp_rope_fwd(t, a["n"], a["dt"], ctypes.byref(p), a["pos"], 0, a["freq"], None)


@nogpu
@pytest.mark.parametrize("bad", [dict(dt=3), dict(axes=0), dict(axes=4), dict(sections=(8, 8, 8)), dict(sections=(0, 0, 0)),
                                 dict(sections=(-1, 4, 4)), dict(head_dim=2048), dict(heads=0), dict(x=None),
                                 dict(x=0x10001), dict(n=0), dict(n=4), dict(pos=None), dict(freq=None),
                                 dict(batch=-1), dict(batch=1 << 20, tokens=1 << 20)])
def test_rope_refuses(lib, bad):
    n0 = lib.ffdp_launch_count()
    assert _rope(lib, **bad) == 1
    assert lib.ffdp_last_error() and lib.ffdp_launch_count() == n0


def _attention(lib, back=False, **kw):
    from voxel_grid_sampler_gb300 import ffdp
    a = dict(batch=2, q_len=5, k_len=7, q_heads=4, k_heads=2, head_dim=64, scale=0.1, cap=0.0, causal=0, dt=2, q=fake,
             stride=256, lse=fake, ws=fake, ws_bytes=1 << 30, bias=None)
    a.update(kw)
    p = ffdp.ffdp_attention_params(*(a[n] for n in ("batch", "q_len", "k_len", "q_heads", "k_heads", "head_dim", "scale",
                                                    "cap", "causal")))
    v = lambda ptr: ffdp.ffdp_heads(ptr, 4096, a["stride"], 64)  # noqa: E731
    bias = None
    if a["bias"] is not None:
        b = ffdp.ffdp_attention_bias()
        for n, x in a["bias"].items():
            setattr(b, n, x)
        bias = ctypes.byref(b)
    if back:
        return lib.ffdp_attention_bwd(v(a["q"]), v(fake), v(fake), v(fake), a["lse"], v(fake), v(fake), v(fake), v(fake),
                                      a["dt"], ctypes.byref(p), bias, a["ws"], a["ws_bytes"], None)
    return lib.ffdp_attention_fwd(v(a["q"]), v(fake), v(fake), v(fake), a["lse"], a["dt"], ctypes.byref(p), bias, a["ws"],
                                  a["ws_bytes"], None)


@nogpu
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("bad", [
    dict(dt=0), dict(dt=3), dict(head_dim=12), dict(head_dim=136), dict(head_dim=0), dict(q_heads=3), dict(k_heads=0),
    dict(q_len=-1), dict(k_len=1 << 25), dict(scale=float("nan")), dict(cap=-1.0), dict(cap=float("inf")), dict(q=None),
    dict(q=odd), dict(stride=100), dict(stride=32), dict(stride=0), dict(bias=dict(pos_q=fake)),
    dict(bias=dict(slopes=fake, axes=3)), dict(bias=dict(slopes=fake, axes=4, pos_q=fake, pos_k=fake)),
    dict(bias=dict(doc_q=fake)), dict(bias=dict(prefix=fake)), dict(bias=dict(doc_q=0x10001, doc_k=fake))])
def test_attention_refuses(lib, bad, back):
    n0 = lib.ffdp_launch_count()
    assert _attention(lib, back, **bad) == 1
    assert lib.ffdp_last_error() and lib.ffdp_launch_count() == n0


@nogpu
def test_attention_workspace_and_lse(lib):
    assert _attention(lib, ws=None) == 3 and _attention(lib, ws_bytes=8) == 3
    assert _attention(lib, True, lse=None) == 1
    assert _attention(lib, True, ws_bytes=256) == 3
    from voxel_grid_sampler_gb300 import ffdp
    p = ffdp.ffdp_attention_params(2, 5, 7, 4, 3, 64, 0.1, 0.0, 0)
    assert lib.ffdp_attention_workspace_bytes(ctypes.byref(p), 0) == 0


def _linear(lib, back=False, **kw):
    from voxel_grid_sampler_gb300 import ffdp
    a = dict(rows=5, inn=16, out=24, act=2, dt=1, x=fake, ldx=16, w=fake, ldw=16, b=fake, z=fake, y=fake, ldy=24, ws=fake,
             ws_bytes=1 << 30)
    a.update(kw)
    p = ffdp.ffdp_linear_params(a["rows"], a["inn"], a["out"], a["act"])
    if back:
        return lib.ffdp_linear_bwd(a["x"], a["ldx"], a["w"], a["ldw"], a["z"], 24, a["y"], a["ldy"], fake, 16, fake, 16,
                                   a["b"], a["dt"], ctypes.byref(p), a["ws"], a["ws_bytes"], None)
    return lib.ffdp_linear_fwd(a["x"], a["ldx"], a["w"], a["ldw"], a["b"], None, 0, a["y"], a["ldy"], a["z"], 24, a["dt"],
                               ctypes.byref(p), a["ws"], a["ws_bytes"], None)


@nogpu
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("bad", [dict(dt=0), dict(dt=5), dict(rows=-1), dict(inn=0), dict(out=0), dict(rows=1 << 31), dict(act=4),
                                 dict(act=-1), dict(x=None), dict(x=odd), dict(ldx=17), dict(ldx=8), dict(w=None),
                                 dict(ldw=12), dict(y=None), dict(y=odd), dict(ldy=25), dict(b=odd), dict(z=odd)])
def test_linear_refuses(lib, bad, back):
    n0 = lib.ffdp_launch_count()
    assert _linear(lib, back, **bad) == 1
    assert lib.ffdp_last_error() and lib.ffdp_launch_count() == n0


@nogpu
def test_linear_backward_needs_its_activation_and_workspace(lib):
    assert _linear(lib, True, z=None) == 1
    assert _linear(lib, True, ws=None) == 3 and _linear(lib, True, ws_bytes=8) == 3


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    from voxel_grid_sampler_gb300 import ffdp
    x = torch.zeros(1, 2, 3, 8, dtype=torch.float16)
    for call in (lambda: ffdp.ffdp_rope_fwd(x, torch.zeros(2, 1), torch.zeros(4), (4,)),
                 lambda: ffdp.ffdp_attention_fwd(x, x, x, ffdp.attention_params(1.0)),
                 lambda: ffdp.ffdp_linear_fwd(x[0, 0], x[0, 0])):
        with pytest.raises(ffdp.FfdpError) as e:
            call()
        assert e.value.status == 1


@pytest.mark.parametrize("cap,causal,docs", [(0.0, False, False), (3.0, True, False), (0.0, False, True)])
def test_reference_gradients_are_the_derivatives(cap, causal, docs, monkeypatch):
    monkeypatch.setitem(ref.U, torch.float64, 2.0 ** -53)
    monkeypatch.setitem(ref.FLOOR, torch.float64, 0.0)
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x = dict(q=rnd(2, 6, 4, 8), k=rnd(2, 9, 2, 8), v=rnd(2, 9, 2, 8))
    go = rnd(2, 6, 4, 8)
    more = dict(pos_q=rnd(6, 2), pos_k=rnd(9, 2), slopes=rnd(4, 2).abs(), causal=causal)
    if docs:
        more.update(doc_q=torch.tensor([0, 0, 1, 1, -1, 2]), doc_k=torch.tensor([0, 1, 1, 0, -1, 1, 0, 0, 3]))
    out = ref.attention(x["q"], x["k"], x["v"], 0.4, cap, go=go, **more)
    for n in x:
        e = rnd(*x[n].shape)
        f = lambda h: (go * ref.attention(*({**x, n: x[n] + h * e}[m] for m in "qkv"), 0.4, cap, **more)["o"][0]).sum()  # noqa: E731
        num = (f(1e-5) - f(-1e-5)) / 2e-5
        assert abs(float((out["g" + n][0] * e).sum() - num)) <= 1e-6 * (1 + abs(float(num))), n
