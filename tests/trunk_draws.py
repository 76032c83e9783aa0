"""Seeded inputs of the trunk operators made on the GPU, for sizes at which host inputs would take too
long, and the comparison with float64 results there.

Tolerances as in test_trunk_gpu.py: |x - y| <= tol max|y|, bf16 results plus 2^-8 |y|."""
from __future__ import annotations

import torch


class Draw:
    """Seeded inputs on the GPU, in the type that holds them."""

    def __init__(self, seed, dtype="f32"):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype = torch.float32 if dtype == "f32" else torch.bfloat16

    def normal(self, *shape, std=1.0, mean=0.0, dtype=None):
        v = torch.randn(*shape, generator=self.g, device="cuda") * std + mean
        return v.to(dtype or self.dtype)

    def f32(self, *shape, **k):
        return self.normal(*shape, dtype=torch.float32, **k)

    def uniform(self, *shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=self.g, device="cuda") * (hi - lo) + lo

    def lengths(self, B, K, *first):
        """B lengths from 0 to K, the given ones first."""
        n = torch.randint(0, K + 1, (B,), generator=self.g, device="cuda", dtype=torch.int32)
        for i, v in enumerate(first[:B]):
            n[i] = v
        return n


def check(got, want, tol, name=""):
    assert got.shape == want.shape, name
    x, bound = got.double(), tol * want.abs().max()
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * want.abs()
    err = (x - want).abs()
    assert bool((err <= bound).all()), \
        f"{name}: worst error {err.max().item():.3g}, max|y| {want.abs().max().item():.3g}"


def doubles(t):
    return {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in t.items()}


def norm_inputs(rows, n, dtype, seed):
    d = Draw(seed, dtype)
    return dict(x=d.normal(rows, n, std=1.5, mean=0.3), w=d.f32(n, std=0.2, mean=1.0),
                b=d.f32(n, std=0.2), dy=d.normal(rows, n), residual=d.normal(rows, n, std=2.0),
                ds=d.normal(rows, n))


def scan_inputs(K, B, D, N, G, dtype, seed):
    d = Draw(seed, dtype)
    steps = torch.exp(d.uniform(D, lo=-6.9, hi=-2.3))  # 1e-3 to 0.1 after softplus
    A = -torch.arange(1.0, N + 1, device="cuda") * d.uniform(D, N, lo=0.9, hi=1.1)
    return dict(x=d.normal(K, B, D), dt=d.normal(K, B, D, std=0.5), z=d.normal(K, B, D),
                dy=d.normal(K, B, D), Bm=d.normal(K, B, G, N), Cm=d.normal(K, B, G, N), A=A,
                skip=d.f32(D, std=0.2, mean=1.0), dt_bias=torch.log(torch.expm1(steps)),
                h0=d.f32(B, D, N, std=0.1), dh_last=d.f32(B, D, N))
