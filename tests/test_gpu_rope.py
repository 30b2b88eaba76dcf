"""Rotary positions with one to three axes against the float64 form: types,
pair layouts, sections, odd head sizes, strides, views, in place, long angles."""
import pytest
import torch

import token_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ffdp():
    from voxel_grid_sampler_gb300 import build, ffdp as f
    build.build()
    return f


def _case(seed, B, S, H, D, sections, dtype, reach=30.0, batched=False):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn((B, S, H, D), generator=g, device="cuda").to(dtype)
    pos = torch.rand(((B,) if batched else ()) + (S, len(sections)), generator=g, device="cuda") * reach
    freq = torch.cat([50.0 ** (-torch.arange(n, dtype=torch.float32) / max(n, 1)) for n in sections]).cuda()
    return x, pos, freq


CASES = [
    (1, 1, 1, 8, (4,)), (2, 13, 3, 64, (10, 11, 11)), (3, 7, 5, 80, (12, 12, 12)), (1, 31, 2, 128, (21, 21, 22)),
    (2, 9, 4, 24, (3, 2)), (1, 5, 1, 2, (1,)), (2, 17, 2, 40, (1, 0, 19)), (1, 6, 70, 96, (16, 16, 16)),
    (1, 3, 2, 1024, (200, 100, 212)), (1, 11, 3, 18, (3, 3, 2)),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,S,H,D,sections", CASES)
def test_turn_and_turn_back(ffdp, B, S, H, D, sections, interleaved, dtype):
    x, pos, freq = _case(S, B, S, H, D, sections, dtype, batched=B == 2)
    ref.within(ffdp.ffdp_rope_fwd(x, pos, freq, sections, interleaved), *ref.rope(x, pos, freq, sections, interleaved))
    ref.within(ffdp.ffdp_rope_bwd(x, pos, freq, sections, interleaved),
               *ref.rope(x, pos, freq, sections, interleaved, -1.0))


def test_long_angles_keep_their_accuracy(ffdp):
    x, pos, freq = _case(3, 1, 64, 2, 64, (16, 16), torch.float32, reach=20000.0)
    ref.within(ffdp.ffdp_rope_fwd(x, pos, freq, (16, 16)), *ref.rope(x, pos, freq, (16, 16), False))


def test_backward_is_the_gradient(ffdp):
    # <gx, e> = d/dt <g, turn(x + t e)>, by central differences of the float64 form
    x, pos, freq = _case(4, 2, 9, 3, 32, (5, 6, 5), torch.float32)
    g, e = torch.randn_like(x), torch.randn_like(x)
    gx = ffdp.ffdp_rope_bwd(g, pos, freq, (5, 6, 5), True)
    f = lambda t: (ref.d(g) * _turn64(ref.d(x) + t * ref.d(e), pos, freq)).sum()  # noqa: E731
    num = (f(1e-3) - f(-1e-3)) / 2e-3
    assert abs(float((ref.d(gx) * ref.d(e)).sum() - num)) <= 1e-5 * float(g.norm() * e.norm())


def _turn64(x, pos, freq):
    ref.U[torch.float64], ref.FLOOR[torch.float64] = 2.0 ** -53, 0.0
    return ref.rope(x, pos, freq, (5, 6, 5), True)[0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_views_pairs_of_tensors_and_in_place(ffdp, dtype):
    sections = (10, 11, 11)
    qkv, pos, freq = _case(5, 2, 21, 16, 64, sections, dtype)
    q, k = qkv[:, :, :8], qkv[:, :, 8:12]
    want = [ref.rope(t, pos, freq, sections, False) for t in (q, k)]
    y, y2 = ffdp.ffdp_rope_fwd(q, pos, freq, sections, False, k)
    ref.within(y, *want[0])
    ref.within(y2, *want[1])
    heads_first = q.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)   # [B][H][S][D] in memory
    ref.within(ffdp.ffdp_rope_fwd(heads_first, pos, freq, sections), *want[0])
    # in place, and a view at an odd offset (element-aligned only); v is untouched
    before = qkv.clone()
    ffdp.ffdp_rope_fwd(q, pos, freq, sections, False, k, q, k)
    ref.within(q, *want[0])
    ref.within(k, *want[1])
    assert torch.equal(qkv[:, :, 12:], before[:, :, 12:])
    odd = torch.empty(before.numel() + 1, dtype=dtype, device="cuda")[1:].view(before.shape)
    odd.copy_(before)
    ref.within(ffdp.ffdp_rope_fwd(odd[:, :, :8], pos, freq, sections), *want[0])
    # the unrotated tail of an in-place call stays
    x, pos, freq = _case(6, 1, 5, 2, 48, (4, 4, 8), dtype)
    want = ref.rope(x, pos, freq, (4, 4, 8), True)
    ffdp.ffdp_rope_fwd(x, pos, freq, (4, 4, 8), True, y=x)
    ref.within(x, *want)


def test_offsets_past_32_bits(ffdp):
    sections = (4, 4)
    big = torch.zeros(2 ** 31 + 4096, dtype=torch.float16, device="cuda")
    x = big.as_strided((2, 3, 2, 16), (2 ** 31, 32, 16, 1))
    src, pos, freq = _case(7, 2, 3, 2, 16, sections, torch.float16)
    x.copy_(src)
    ref.within(ffdp.ffdp_rope_fwd(x, pos, freq, sections), *ref.rope(src, pos, freq, sections, False))


def test_empty_and_other_stream(ffdp):
    x, pos, freq = _case(8, 2, 5, 3, 32, (8, 8), torch.float16)
    assert ffdp.ffdp_rope_fwd(x[:0], pos, freq, (8, 8)).shape == (0, 5, 3, 32)
    assert ffdp.ffdp_rope_fwd(x[:, :0], pos[:0], freq, (8, 8)).shape == (2, 0, 3, 32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = ffdp.ffdp_rope_fwd(x, pos, freq, (8, 8))
    s.synchronize()
    ref.within(y, *ref.rope(x, pos, freq, (8, 8), False))
