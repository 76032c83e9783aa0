"""What the trunk block's calls return stays what it was."""
import pytest
import torch

from test_block_gpu import OUT_TOL

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from recurrent_cfc_cell_gb300 import build

    build.build()
    torch.backends.cuda.matmul.allow_tf32 = False


def test_tokens_kept_by_the_caller():
    """Every token's result, collected as it was returned, against the prompt in one piece."""
    from recurrent_cfc_cell_gb300.block import TrunkServe, make_params

    K, B, D, E, N = 6, 3, 24, 48, 8
    P = make_params(D, E, N, 16, seed=7)
    s = torch.randn(K, B, D, generator=torch.Generator().manual_seed(8)).cuda()
    whole = TrunkServe(B, P).prompt(s)
    serve = TrunkServe(B, P)
    got = torch.stack([serve.token(s[t]) for t in range(K)])
    assert (got - whole).abs().max() <= OUT_TOL * whole.abs().max()
