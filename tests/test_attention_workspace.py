"""CPU tests of the attention's workspace: it holds the parts of as many workgroups
as its shape can have on the card's 256 CUs, and no more."""

import pytest

import dspark_verify_scheduling_amd as dv


@pytest.mark.parametrize("gamma,hq,hkv,D,per_cu,rows", [
    (1, 8, 8, 64, 2, 16), (64, 64, 1, 64, 2, 128), (8, 32, 8, 128, 3, 48), (15, 32, 8, 128, 3, 64),
    (16, 32, 8, 128, 2, 80), (64, 40, 5, 128, 2, 128), (6, 8, 1, 256, 1, 64), (64, 64, 1, 256, 1, 128)])
@pytest.mark.parametrize("B", [0, 1, 300])
def test_size_is_that_of_the_parts(gamma, hq, hkv, D, per_cu, rows, B):
    parts = 2 * 256 * per_cu * rows
    got = dv.dspark_tree_attention_workspace_size(B, gamma, hq, hkv, D)
    need = 8 * (B + 1) + parts * 4 * (D + 2)  # unit sums; maxima, sums and outputs
    assert need <= got < need + 4 * 256
