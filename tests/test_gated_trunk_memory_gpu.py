"""What a layer adds to the memory of a trunk of gated blocks that keeps its activations in 8 bits: the
codes and scales of the stream and of x, f and z, the recurrence's states, and small vectors."""
import pytest

pytestmark = pytest.mark.gpu

K, B, D, E, C = 64, 64, 256, 512, 32


def grown(layers):
    """Bytes held once the trunk is made (and most on the way there), and once a step has run, beyond
    what was held before: as they were asked for, since what the allocator rounds them up to (by up to a
    megabyte of a block that it does not split) depends on what ran before."""
    import gc

    import torch

    from recurrent_cfc_cell_gb300.gated_block import GatedTrunk, make_gated_params

    params = make_gated_params(layers, D, E, C)
    r = lambda *n: torch.randn(*n, device="cuda")  # noqa: E731
    s, h0, ts, dH = r(K, B, D), r(B, C), torch.rand(K, B, device="cuda"), r(K, B, C)
    gc.collect()
    torch.cuda.synchronize()

    def held(which="current"):
        return torch.cuda.memory_stats()["requested_bytes.all." + which]

    start = held()
    torch.cuda.reset_peak_memory_stats()
    trunk = GatedTrunk(K, B, params, keep8=True)
    made, peak = held() - start, held("peak") - start
    for _ in range(2):
        trunk.forward(s, h0, ts)
        grads = trunk.backward(dH)
    torch.cuda.synchronize()
    assert len(grads["layers"]) == layers
    return made, peak, held() - start


def test_a_layer_adds_what_it_keeps():
    from recurrent_cfc_cell_gb300 import _lib

    rows = K * B
    kept = rows * (D + 3 * E) * 33 // 32  # codes and their scales
    kept += rows // 8 * E * 4 + rows * 4  # states and the norm's rstd
    work = _lib.rmsnorm_workspace_bytes(rows, D) + _lib.gated_workspace_bytes(K, B, E, True)
    grads = (4 * E * D + 2 * E + 2 * D + B * E + B * E) * 4  # of the weights, biases and states; h
    slack = 64 << 10  # what a layer may hold besides
    (made2, peak2, ran2), (made6, peak6, ran6) = grown(2), grown(6)
    most = kept + work + grads + slack
    assert (made6 - made2) / 4 <= most
    assert (peak6 - peak2) / 4 <= most
    assert (ran6 - ran2) / 4 <= most
    assert most < 1.6 * kept  # the bound means something
