"""Inputs of the gated block's tests, as float64 numpy arrays whose values the activations' type
holds exactly."""
import numpy as np

import oracle.trunk as ot


def rounded(v, dtype):
    return ot.bf16(v) if dtype == "bf16" else v.astype(np.float32).astype(np.float64)


def rms_inputs(rows, n, dtype, seed):
    r = np.random.default_rng(seed)
    i = {k: rounded(r.normal(size=(rows, n)), dtype) for k in ("x", "residual", "dy", "ds")}
    i["w"] = rounded(r.normal(1.0, 0.2, size=n), "f32")
    i["s"] = rounded(i["x"] + i["residual"], dtype)
    return i


def gated_inputs(K, B, D, dtype, seed, ends=None):
    r = np.random.default_rng(seed)
    i = {k: rounded(r.normal(size=(K, B, D)), dtype) for k in ("x", "f", "z", "dy")}
    i["bias"] = rounded(r.uniform(-1.0, 4.0, size=D), "f32")
    i["h0"] = rounded(r.normal(size=(B, D)), "f32")
    i["dh_last"] = rounded(r.normal(size=(B, D)), "f32")
    i["ends"] = np.full(B, K) if ends is None else np.asarray(ends)
    return i


def weights4_inputs(M, N, K, group, dtype, seed):
    r = np.random.default_rng(seed)
    return dict(codes=r.integers(0, 256, size=(N, (K + 1) // 2), dtype=np.uint8),
                scales=ot.bf16(r.uniform(0.002, 0.02, size=(N, -(-K // group)))),
                x=rounded(r.normal(size=(M, K)), dtype))
