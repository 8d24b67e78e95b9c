"""A decoder layer for serving: attention over the paged NVFP4 cache, then the
routed MoE layer.

Runs prompts in chunks, forks a sequence into samples, decodes, ends some
sequences and compacts the cache:

    python examples/decoder_layer.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixture_experts_layer_fwd_gb300 import KV4Cache, MoELayer, moe_sync_status  # noqa: E402


def rms(x: torch.Tensor) -> torch.Tensor:
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class DecoderLayer:
    """x + attention(norm(x)), then x + MoE(norm(x)); random weights."""

    def __init__(self, cache: KV4Cache, index: int, H: int, Hq: int, E: int, k: int, I: int, seed: int = 0):
        dev, Hkv, D = cache.device, cache.Hkv, cache.D
        g = torch.Generator(dev).manual_seed(seed + index)
        w = lambda *s: (torch.randn(*s, generator=g, device=dev) * s[-1] ** -0.5).bfloat16()  # noqa: E731
        self.cache, self.index, self.heads = cache, index, (Hq, Hkv, D)
        self.w_qkv, self.w_o = w((Hq + 2 * Hkv) * D, H), w(H, Hq * D)
        self.wq, self.wk = (1 + 0.1 * w(D)).contiguous(), (1 + 0.1 * w(D)).contiguous()
        self.w_router = w(E, H)
        self.moe = MoELayer(H, E, k, I, 0, w(E, 2 * I, H), w(E, H, I))

    def attention(self, x: torch.Tensor, cos_sin: torch.Tensor) -> torch.Tensor:
        Hq, Hkv, D = self.heads
        qkv = rms(x) @ self.w_qkv.T
        q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split((Hq * D, Hkv * D, Hkv * D), 1))
        y = self.cache.attend(self.index, q, k, v, cos_sin, wq=self.wq, wk=self.wk)
        return x + y.flatten(1) @ self.w_o.T

    def __call__(self, x: torch.Tensor, cos_sin: torch.Tensor) -> torch.Tensor:
        x = self.attention(x, cos_sin)
        n = rms(x)
        return x + self.moe(n, (n @ self.w_router.T).float())


def rotation(positions: int, D: int, device, base: float = 1e6) -> torch.Tensor:
    a = torch.arange(positions, device=device).unsqueeze(1) * base ** (-torch.arange(0, D, 2, device=device) / D)
    return torch.cat((a.cos(), a.sin()), 1).float().contiguous()


def main() -> None:
    dev = torch.device("cuda")
    H, Hq, Hkv, D, layers, rows = 512, 8, 2, 64, 2, 6
    scale = torch.full((layers, Hkv), 6.0 / 2688.0, device=dev)
    cache = KV4Cache(layers, num_pages=64, rows=rows, max_pages=16, Hkv=Hkv, D=D, g_k=scale, g_v=scale)
    model = [DecoderLayer(cache, i, H, Hq, E=8, k=2, I=512) for i in range(layers)]
    cos_sin = rotation(1024, D, dev)
    g = torch.Generator(dev).manual_seed(1)

    def step(counts):
        x = torch.randn(sum(counts), H, generator=g, device=dev).bfloat16()
        cache.extend(counts)
        for layer in model:
            x = layer(x, cos_sin)
        return x

    step([300, 130, 0, 0, 0, 0])          # two prompts
    step([200, 1, 0, 0, 0, 0])            # the first one's next chunk beside the second one's first new token
    cache.fork([0, 0, 1], [2, 3, 4])      # samples of both
    for _ in range(4):
        y = step([1, 1, 1, 1, 1, 0])
    cache.free([0, 3])
    cache.compact()
    y = step([0, 1, 1, 0, 1, 0])
    if moe_sync_status() != 0:
        raise RuntimeError("a cache call reported an error")
    print("lengths", cache.lens.tolist(), "pages in use", int((cache.refs > 0).sum()), "output norm %.3f" % y.float().norm())


if __name__ == "__main__":
    main()
