"""One decoder layer trained for a few steps: the framework's operators as they are used together.

    python examples/decoder_layer.py [--steps N] [--small]

The neck's feature maps are normalised and activated where they lie
(GroupNormActFunction), every instance gathers its key points' features from
all cameras and scales (DeformableAggregationFunction), and the instances then
attend to each other and to the instances of past frames with a learned bias by
the number of frames between them (DifferentialAttentionFunction). The data is
random; the layer learns to reproduce a fixed target.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import deformable_view_feature_gb300 as da  # noqa: E402


class DecoderLayer(torch.nn.Module):
    def __init__(self, channels, groups, heads, scales, points, cams, buckets=8, reach=16):
        super().__init__()
        self.heads, self.width = heads, channels // heads // 2
        self.norm_groups, self.groups = channels // 8, groups
        self.sample_shape = (points, cams, scales, groups)
        self.gamma = torch.nn.Parameter(torch.ones(scales, channels))
        self.beta = torch.nn.Parameter(torch.zeros(scales, channels))
        self.weigh = torch.nn.Linear(channels, points * cams * scales * groups)
        self.gathered = torch.nn.Linear(channels, channels)
        self.q, self.k, self.v, self.out = (torch.nn.Linear(channels, channels, bias=False) for _ in range(4))
        # lam = exp(a0 . b0) - exp(a1 . b1) + 0.5 of each head's own vectors.
        self.lam_a, self.lam_b = (torch.nn.Parameter(torch.randn(2, heads, self.width) * 0.1) for _ in range(2))
        self.bias_table = torch.nn.Parameter(torch.zeros(buckets, heads))
        self.register_buffer("bucket_map", da.relative_buckets(buckets, reach))

    def forward(self, feat, spatial_shape, level_start_index, location, instances, history, frames):
        """instances [B, A, C], history [B, N, C] with frames [B, N] int32
        (0 now, -1 the frame before, ...)."""
        B, A, C = instances.shape
        feat = da.GroupNormActFunction.apply(feat, spatial_shape, level_start_index, self.gamma, self.beta,
                                             self.norm_groups, 1e-5, "silu")
        points, cams, scales, groups = self.sample_shape
        weights = self.weigh(instances).reshape(B, A, -1, groups).softmax(2).reshape(B, A, points, cams, scales, groups)
        seen = da.DeformableAggregationFunction.apply(feat, spatial_shape, level_start_index, location, weights)
        x = instances + self.gathered(seen)
        keys = torch.cat([x, history], 1)
        pos_k = torch.cat([torch.zeros(B, A, dtype=torch.int32, device=x.device), frames], 1)
        pos_q = torch.zeros(B, A, dtype=torch.int32, device=x.device)
        lam = (self.lam_a * self.lam_b).sum(-1).exp()
        lam = lam[0] - lam[1] + 0.5
        q, k = (m(t).to(torch.bfloat16).reshape(B, -1, self.heads, 2, self.width) for m, t in ((self.q, x), (self.k, keys)))
        v = self.v(keys).to(torch.bfloat16).reshape(B, -1, self.heads, 2 * self.width)
        y = da.DifferentialAttentionFunction.apply(q, k, v, lam, self.bias_table, self.bucket_map, pos_q, pos_k, None, None,
                                                   False, None)
        return x + self.out(y.reshape(B, A, C).float())


def train(steps=5, small=False, lr=3.0, seed=0):
    """Trains the layer on random data; returns the losses."""
    dev = torch.device("cuda")
    torch.manual_seed(seed)
    B, K, shapes, C, A, P, N = (1, 2, [(16, 24), (8, 12)], 64, 40, 4, 60) if small else \
        (2, 6, [(64, 176), (32, 88), (16, 44), (8, 22)], 256, 900, 13, 1200)
    spatial_shape = torch.tensor([shapes] * K, dtype=torch.int32)
    sizes = torch.tensor([h * w for h, w in shapes] * K)
    level_start_index = (sizes.cumsum(0) - sizes).to(torch.int32).reshape(K, len(shapes))
    layer = DecoderLayer(C, 8, 4, len(shapes), P, K).to(dev)
    feat = torch.randn(B, int(sizes.sum()), C, device=dev)
    location = torch.rand(B, A, P, K, 2, device=dev)
    instances, target = torch.randn(B, A, C, device=dev), torch.randn(B, A, C, device=dev)
    history = torch.randn(B, N, C, device=dev)
    frames = -(1 + torch.arange(N, device=dev, dtype=torch.int32) * 4 // N).expand(B, N).contiguous()
    losses = []
    for _ in range(steps):
        out = layer(feat, spatial_shape, level_start_index, location, instances, history, frames)
        loss = (out - target).square().mean()
        layer.zero_grad(set_to_none=True)
        loss.backward()
        with torch.no_grad():
            for p in layer.parameters():
                p -= lr * p.grad
        losses.append(float(loss.detach()))
    assert all(math.isfinite(x) for x in losses)
    return losses, layer


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=5)
    ap.add_argument("--small", action="store_true", help="a toy size")
    a = ap.parse_args()
    da.build.build()
    for i, x in enumerate(train(a.steps, a.small)[0]):
        print(f"step {i}: loss {x:.4f}")
