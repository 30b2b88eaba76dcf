"""A registration network over volume tokens, trained through the objective.

Instead of optimising the displacement u itself, a small network computes it
from the pair: patches of F and M become tokens, blocks of attention (rotary
positions and a distance bias over the tokens' (z, y, x) grid) and of linear
layers follow, and the last layer gives every token a displacement.  The coarse
field becomes u through ffdp_sample_channels_fwd, ffdp_objective grades it, and
du goes back the same way: the gradient of the coarse field, then each layer's.

    python -m voxel_grid_sampler_gb300.learned     # fit one synthetic pair

Every product, attention and rotation runs in the library; torch holds the
memory, cuts patches, adds gradients and applies the plain gradient step.
"""
from __future__ import annotations

import torch

from . import ffdp


class VolumeNetwork:
    """Predicts a displacement for volumes of shape `dims`, a multiple of `patch` along every axis."""

    def __init__(self, dims, patch=8, width=128, heads=4, key_heads=2, blocks=2, dtype=torch.bfloat16, seed=0,
                 device="cuda"):
        self.dims, self.patch, self.heads, self.key_heads = tuple(dims), patch, heads, key_heads
        if any(n % patch for n in self.dims):
            raise ValueError("dims must be multiples of patch")
        self.grid = tuple(n // patch for n in self.dims)
        self.head_dim = width // heads
        gen = torch.Generator(device).manual_seed(seed)

        def weight(out, fan_in, scale=1.0):
            return (torch.randn((out, fan_in), generator=gen, device=device) * (scale * fan_in ** -0.5)).to(dtype)

        def bias(out):
            return torch.zeros(out, dtype=dtype, device=device)

        features, qkv = 2 * patch ** 3, (heads + 2 * key_heads) * self.head_dim
        self.params = {"embed.w": weight(width, features), "embed.b": bias(width)}
        for i in range(blocks):
            self.params.update({
                "%d.qkv.w" % i: weight(qkv, width), "%d.qkv.b" % i: bias(qkv),
                "%d.out.w" % i: weight(width, width, 0.5), "%d.out.b" % i: bias(width),
                "%d.up.w" % i: weight(4 * width, width), "%d.up.b" % i: bias(4 * width),
                "%d.down.w" % i: weight(width, 4 * width, 0.5), "%d.down.b" % i: bias(width)})
        self.params.update({"head.w": weight(3, width, 0.01), "head.b": bias(3)})
        self.blocks = blocks
        z, y, x = (torch.arange(n, device=device, dtype=torch.float32) for n in self.grid)
        self.pos = torch.stack(torch.meshgrid(z, y, x, indexing="ij"), -1).reshape(-1, 3).contiguous()
        n = self.head_dim // 2
        self.sections = (n // 3, n // 3, n - 2 * (n // 3))
        self.freq = torch.cat([100.0 ** (-torch.arange(s, dtype=torch.float32) / s) for s in self.sections]).to(device)
        # half of the heads look near, half far; slopes per (head, axis)
        slope = torch.tensor([2.0 ** (-4.0 * (h + 1) / heads) for h in range(heads)], device=device)
        self.slopes = slope[:, None].expand(heads, 3).contiguous()
        self.attention = ffdp.attention_params(self.head_dim ** -0.5)
        self.bias = dict(pos_q=self.pos, pos_k=self.pos, slopes=self.slopes)
        self.identity = ffdp.transform()

    # ------------------------------------------------------------- forward
    def _tokens(self, F, M):
        p, (d, h, w) = self.patch, self.grid
        both = torch.stack((F, M)).reshape(2, d, p, h, p, w, p).permute(1, 3, 5, 0, 2, 4, 6)
        return both.reshape(d * h * w, 2 * p ** 3).to(self.params["embed.w"].dtype)

    def _linear(self, name, x, residual=None, act="none"):
        w, b = self.params[name + ".w"], self.params[name + ".b"]
        y, z = ffdp.ffdp_linear_fwd(x, w, b, residual, act, want_z=True)
        self._tape.append((name, x, z, act))
        return y

    def _qkv(self, t):
        """(1, tokens, heads, head_dim) views of queries, keys and values."""
        hq, hk = self.heads, self.key_heads
        t = t.view(1, -1, hq + 2 * hk, self.head_dim)
        return t[:, :, :hq], t[:, :, hq:hq + hk], t[:, :, hq + hk:]

    def forward(self, F, M):
        """u (D, H, W, 3) float32 for volumes F and M; keeps what backward needs."""
        self._tape, self._saved = [], []
        x = self._linear("embed", self._tokens(F, M), act="gelu")
        for i in range(self.blocks):
            q, k, v = self._qkv(self._linear("%d.qkv" % i, x))
            ffdp.ffdp_rope_fwd(q, self.pos, self.freq, self.sections, False, k, q, k)  # in place
            o, lse = ffdp.ffdp_attention_fwd(q, k, v, self.attention, **self.bias)
            self._saved.append((q, k, v, o, lse))
            x = self._linear("%d.out" % i, o.view(o.shape[1], -1), x)
            x = self._linear("%d.down" % i, self._linear("%d.up" % i, x, act="gelu"), x)
        self.coarse = self._linear("head", x).float().reshape(self.grid + (3,)).contiguous()
        return ffdp.ffdp_sample_channels_fwd(self.coarse, self.dims, None, self.identity)

    # ------------------------------------------------------------ backward
    def _back(self, gy, grads):
        name, x, z, act = self._tape.pop()
        gx, grads[name + ".w"], grads[name + ".b"] = ffdp.ffdp_linear_bwd(x, self.params[name + ".w"], z, gy, act)
        return gx

    def backward(self, du):
        """Gradients of the parameters from du = dL/du of the last forward call."""
        dV = ffdp.ffdp_sample_channels_bwd(self.coarse, None, self.identity, du, want_du=False)[3]
        grads, dtype = {}, self.params["head.w"].dtype
        scale = float(dV.abs().max().clamp_min(1e-30))  # keeps small gradients in the 16-bit types' range
        g = torch.empty_strided((self.pos.shape[0], 3), (8, 1), dtype=dtype, device=dV.device).copy_(dV.reshape(-1, 3) / scale)
        g = self._back(g, grads)
        for i in reversed(range(self.blocks)):
            g = g + self._back(self._back(g, grads), grads)          # down, up, and the residual
            q, k, v, o, lse = self._saved.pop()
            go = self._back(g, grads).view(o.shape)
            gqkv = torch.empty(q.shape[1], (self.heads + 2 * self.key_heads) * self.head_dim, dtype=dtype, device=dV.device)
            gq, gk, gv = self._qkv(gqkv)
            ffdp.ffdp_attention_bwd(q, k, v, o, lse, go, self.attention, gq=gq, gk=gk, gv=gv, **self.bias)
            ffdp.ffdp_rope_bwd(gq, self.pos, self.freq, self.sections, False, gk, gq, gk)
            g = g + self._back(gqkv, grads)
        self._back(g, grads)
        return {n: t.float() * scale for n, t in grads.items()}

    def train_step(self, F, M, objective, lr):
        """One step of normalised gradient descent on the objective of (F, M o u); returns its loss[3]."""
        u = self.forward(F, M)
        loss, du, _, _ = ffdp.ffdp_objective(F, M, u, self.identity, objective)
        grads = self.backward(du)
        norm = torch.sqrt(sum(g.square().sum() for g in grads.values())).clamp_min(1e-30)
        for n, g in grads.items():
            self.params[n] = (self.params[n].float() - lr * g / norm).to(self.params[n].dtype)
        return loss


def main(steps=60):
    from . import synth
    g = torch.Generator().manual_seed(1)
    F = synth.gaussian_smooth(torch.rand((64, 64, 64), generator=g), 4.0)
    F = (F - F.min()) / (F.max() - F.min())
    M = torch.roll(F, (1, 2), (1, 2)).contiguous().cuda()  # F, one and two voxels away
    F = F.cuda()
    objective = ffdp.objective_params(1.0, 1.0, 32, (0.0, 1.0), (0.0, 1.0), 5)
    net = VolumeNetwork(F.shape, patch=8, width=96, heads=4, key_heads=2)
    for i in range(steps):
        loss = net.train_step(F, M, objective, 0.02)
        if i % 10 == 0 or i == steps - 1:
            print("step %3d  objective %.5f  (-MI %.5f, -LNCC %.5f)" % ((i,) + tuple(loss.tolist())))


if __name__ == "__main__":
    main()
