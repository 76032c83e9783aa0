"""Seeded inputs of the trunk operators' tests, as float64 arrays that the tested type holds
exactly (bf16 inputs are rounded to bf16 first)."""
from __future__ import annotations

import numpy as np

import oracle.trunk as ot


def hold(v, dtype):
    """float64 values that fp32 or bf16 holds exactly."""
    return ot.bf16(v) if dtype == "bf16" else np.asarray(v).astype(np.float32).astype(np.float64)


def norm_inputs(rows, n, dtype, seed, mean=0.3):
    g = np.random.default_rng(seed)
    f32 = lambda v: hold(v, "f32")  # noqa: E731
    return dict(x=hold(g.normal(mean, 1.5, (rows, n)), dtype), w=f32(g.normal(1, 0.2, n)),
                b=f32(g.normal(0, 0.2, n)), dy=hold(g.normal(0, 1, (rows, n)), dtype),
                residual=hold(g.normal(0, 2, (rows, n)), dtype),
                ds=hold(g.normal(0, 1, (rows, n)), dtype))


def conv_inputs(K, B, D, W, dtype, seed):
    g = np.random.default_rng(seed)
    return dict(x=hold(g.normal(0, 1, (K, B, D)), dtype), w=hold(g.uniform(-.5, .5, (D, W)), "f32"),
                bias=hold(g.normal(0, .1, D), "f32"), x0=hold(g.normal(0, 1, (B, W - 1, D)), dtype),
                du=hold(g.normal(0, 1, (K, B, D)), dtype))


def scan_inputs(K, B, D, N, G, dtype, seed):
    g = np.random.default_rng(seed)
    rows, bc = (K, B, D), (K, B, G, N)
    act = lambda *s, std=1.0: hold(g.normal(0, std, s), dtype)  # noqa: E731
    return dict(x=act(*rows), dt=act(*rows, std=0.5), Bm=act(*bc), Cm=act(*bc), z=act(*rows),
                dy=act(*rows), A=hold(-np.arange(1, N + 1) * g.uniform(.9, 1.1, (D, N)), "f32"),
                skip=hold(g.normal(1, .2, D), "f32"),
                dt_bias=hold(np.log(np.expm1(np.exp(g.uniform(np.log(1e-3), np.log(.1), D)))), "f32"),
                h0=hold(g.normal(0, .1, (B, D, N)), "f32"),
                dh_last=hold(g.normal(0, 1, (B, D, N)), "f32"))
