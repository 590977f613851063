"""Where the balance takes one launch (no workspace) and where two: up to 64 rows a
sequence and 384 groups of 64 logits."""

import pytest

from quantized_moe_amd import chord as C


@pytest.mark.parametrize("E,rows", [(1, 64), (64, 64), (256, 64), (384, 64), (385, 54), (512, 48), (1000, 24), (1024, 24)])
def test_rows_of_one_launch(E, rows):
    for n_seq in (1, 8):
        need = C.chord_moe_balance_workspace_bytes
        assert need(n_seq * rows, E, 1, n_seq) == 0
        assert need(n_seq * (rows + 1), E, 1, n_seq) > 0
