"""The registration network over volume tokens: its displacement and parameter
gradients against the same network in float64 (torch autograd, CPU), and a few
training steps on a shifted pair."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ffdp():
    from voxel_grid_sampler_gb300 import build, ffdp as f
    build.build()
    return f


def _reference(net, params, F, M):
    """u of the network in float64, from leaf parameters."""
    lin = lambda n, x: x @ params[n + ".w"].T + params[n + ".b"]  # noqa: E731
    gelu = torch.nn.functional.gelu
    p, (d, h, w) = net.patch, net.grid
    both = torch.stack((F, M)).double().reshape(2, d, p, h, p, w, p).permute(1, 3, 5, 0, 2, 4, 6).reshape(d * h * w, -1)
    x = gelu(lin("embed", both))
    pos, freq, slopes = net.pos.cpu().double(), net.freq.cpu().double(), net.slopes.cpu().double()
    axis = torch.cat([torch.full((n,), a) for a, n in enumerate(net.sections)])
    t = pos[:, axis] * freq
    cos, sin = torch.cos(t)[:, None], torch.sin(t)[:, None]
    far = (pos[:, None] - pos[None]).abs()
    bias = -torch.einsum("ha,ija->hij", slopes, far)
    hq, hk, D = net.heads, net.key_heads, net.head_dim

    def turn(x):
        R = D // 2
        a, b = x[..., :R], x[..., R:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)

    for i in range(net.blocks):
        qkv = lin("%d.qkv" % i, x).view(-1, hq + 2 * hk, D)
        q, k, v = turn(qkv[:, :hq]), turn(qkv[:, hq:hq + hk]), qkv[:, hq + hk:]
        k, v = k.repeat_interleave(hq // hk, 1), v.repeat_interleave(hq // hk, 1)
        s = torch.einsum("ihd,jhd->hij", q, k) * D ** -0.5 + bias
        o = torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v).reshape(x.shape[0], -1)
        x = lin("%d.out" % i, o) + x
        x = lin("%d.down" % i, gelu(lin("%d.up" % i, x))) + x
    c = lin("head", x).reshape(1, d, h, w, 3).permute(0, 4, 1, 2, 3)
    return torch.nn.functional.interpolate(c, size=net.dims, mode="trilinear", align_corners=True)[0].permute(1, 2, 3, 0)


def test_displacement_and_gradients(ffdp):
    # about 40 roundings to float16 (2^-11) lie between a parameter's gradient
    # and du, each with a gain of about one: 2 % in the 2-norm at most
    from voxel_grid_sampler_gb300.learned import VolumeNetwork
    g = torch.Generator().manual_seed(5)
    F, M = torch.rand((24, 32, 40), generator=g), torch.rand((24, 32, 40), generator=g)
    du = torch.randn((24, 32, 40, 3), generator=g)
    net = VolumeNetwork(F.shape, patch=8, width=96, heads=4, key_heads=2, dtype=torch.float16)
    net.params = {n: (t if n.endswith("w") else t + 0.1 * torch.randn(t.shape, generator=g).cuda().half())
                  for n, t in net.params.items()}
    u = net.forward(F.cuda(), M.cuda())
    grads = net.backward(du.cuda())
    leaves = {n: t.cpu().double().requires_grad_() for n, t in net.params.items()}
    want = _reference(net, leaves, F, M)
    (want * du.double()).sum().backward()
    rel = lambda a, b: float((a.cpu().double() - b).norm() / b.norm())  # noqa: E731
    assert rel(u, want.detach()) <= 0.02
    assert set(grads) == set(leaves)
    for n, t in leaves.items():
        assert rel(grads[n], t.grad) <= 0.02, (n, rel(grads[n], t.grad))


def test_training_lowers_the_objective(ffdp):
    from voxel_grid_sampler_gb300 import synth
    from voxel_grid_sampler_gb300.learned import VolumeNetwork
    g = torch.Generator().manual_seed(6)
    F = synth.gaussian_smooth(torch.rand((32, 40, 48), generator=g), 4.0)
    F = (F - F.min()) / (F.max() - F.min())
    M = torch.roll(F, 2, 2).contiguous().cuda()
    F = F.cuda()
    objective = ffdp.objective_params(0.0, 1.0, 32, (0.0, 1.0), (0.0, 1.0), 5)
    net = VolumeNetwork(F.shape, patch=8, width=96, heads=4, key_heads=2)
    losses = [float(net.train_step(F, M, objective, 0.02)[0]) for _ in range(25)]
    assert min(losses) < losses[0] - 0.02, losses
    assert not ffdp.device_error()
