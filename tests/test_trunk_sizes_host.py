"""Sizes at and beyond what the trunk operators' C entry points hold in an int, on the host."""
import pytest

from recurrent_cfc_cell_gb300 import _lib, build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


@pytest.mark.parametrize("n", [1, 8, 60, 256, 1024, 5000, 8192])
def test_workspace_of_the_most_rows(n):
    """From some number of rows on the grid is full and the workspace stays the same, up to the
    largest int."""
    full = _lib.layernorm_workspace_bytes(10**8, n)
    assert full > 0
    for rows in (2**31 - 64, 2**31 - 2, 2**31 - 1):
        assert _lib.layernorm_workspace_bytes(rows, n) == full


BIG = 2**32 + 4  # 4 in an int


def test_sizes_beyond_an_int_are_refused():
    """Not taken modulo 2^32, by the workspace calls and by every entry point (whose tensors are
    looked at for their sizes first)."""
    import torch

    refused = pytest.raises(ValueError, match="32-bit")
    for call, good in ((_lib.layernorm_workspace_bytes, (4, 8)),
                       (_lib.conv_workspace_bytes, (2, 4, 8, 4, 0)),
                       (_lib.scan_workspace_bytes, (4, 2, 8, 4, 1, 0, True)),
                       (_lib.scan_states_bytes, (4, 2, 8, 4, 1, 0))):
        call(*good)
        for k in range(len(good) - (2 if call is _lib.scan_workspace_bytes else 1)):
            with refused:
                call(*(BIG if j == k else v for j, v in enumerate(good)))
    one, par = torch.zeros(1, 1), torch.zeros(1)
    x = one.expand(BIG, 1)
    for args in ((_lib.cfc_layernorm_forward, x, par, par, x, one),
                 (_lib.cfc_layernorm_backward, x, x, par, one, x, par, par),
                 (_lib.cfc_dropout_forward, x, None, par, 0.5, x),
                 (_lib.cfc_dropout_backward, x, par, 0.5, x),
                 (_lib.cfc_dropout_layernorm_forward, x, None, par, 0.5, par, par, x, x, one),
                 (_lib.cfc_dropout_layernorm_backward, x, None, x, par, 0.5, par, one, x, None, par,
                  par)):
        with refused:
            args[0].prepare(*args[1:])
    for shape in ((BIG, 1, 1), (1, BIG, 1), (1, 1, BIG)):
        x = torch.zeros(1, 1, 1).expand(shape)
        bc = torch.zeros(1, 1, 1, 1).expand(*shape[:2], 1, 1)
        with refused:
            _lib.cfc_conv_forward.prepare(x, torch.zeros(1, 2), x)
        with refused:
            _lib.cfc_conv_backward.prepare(x, x, torch.zeros(1, 2), x, one, par)
        with refused:
            _lib.cfc_scan_forward.prepare(x, x, one, bc, bc, x)
        with refused:
            _lib.cfc_scan_backward.prepare(x, x, x, one, bc, bc, one, x, x, one, bc, bc)
        if shape[0] == 1:
            with refused:
                _lib.cfc_conv_step.prepare(x[0], torch.zeros(1, 2), x, x, x[0])
            with refused:
                _lib.cfc_scan_step.prepare(x[0], x[0], one, bc[0], bc[0], x, x, x[0])
    with refused:
        _lib.cfc_scan_forward.prepare(*(torch.zeros(1, 1, 1),) * 2, one,
                                      *(torch.zeros(1, 1, 1, 1).expand(1, 1, BIG, 1),) * 2, x)
