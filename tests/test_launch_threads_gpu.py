"""Host threads that run the same kernels at different sizes at the same time, each on a stream of its own:
no call fails because another one needed less shared memory."""
import pytest

pytestmark = pytest.mark.gpu


def steps_of(name):
    """A step that takes little shared memory and one that takes much of the same kernel."""
    import torch

    from recurrent_cfc_cell_gb300 import build, trunk

    build.build()
    r = lambda *n: torch.randn(*n, device="cuda")  # noqa: E731
    if name == "gated":
        # One warp of a run each, and eight.
        return [trunk.GatedStep(K, 2, 64, train=True).bind(
            r(K, 2, 64), r(K, 2, 64), None, r(K, 2, 64), dy=r(K, 2, 64)) for K in (8, 64)]
    if name == "matvec":
        # Both more than 48 KB: rows of 24 and 32 columns of a CTA.
        w = trunk.Weights4.of(r(64, 4096), 128)
        return [trunk.MatvecStep(M, w, torch.bfloat16).bind(r(M, 4096).bfloat16()) for M in (26, 32)]
    # Rows that wait in a ring, of 272 and 512 threads.
    rng = torch.tensor([1, 2], device="cuda")
    return [trunk.DropoutNormStep(8, n, 0.1).bind(r(8, n), r(8, n), rng, r(n), r(n), r(8, n), r(8, n))
            for n in (4104, 8192)]


@pytest.mark.parametrize("name", ["gated", "matvec", "dropnorm"])
def test_threads_of_different_sizes(name):
    import threading

    import torch

    steps, errors = steps_of(name), []
    for s in steps:
        s.run()
    torch.cuda.synchronize()
    first = [{k: v.clone() for k, v in s.outputs().items()} for s in steps]

    def work(step):
        try:
            stream = torch.cuda.Stream()
            for n in range(4000):
                step.run(stream)
                if n % 100 == 99:
                    stream.synchronize()
        except Exception as e:  # noqa: BLE001 (told below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in steps]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for a, s in zip(first, steps):
        assert all(torch.equal(a[k], v) for k, v in s.outputs().items())
