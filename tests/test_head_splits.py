"""The splits of the LM head's dX GEMM, checked on the CPU for the library's own choices: unit u of a
launch is piece u // tiles of tile u % tiles, fills [s·L/S, (s + 1)·L/S), and its fp32 slot is u.  So
the pieces cover every fill of every tile once, none is empty, and the slots stay within the
workspace, for all rows and for any number of rows that distillation keeps."""
import pytest

import qlora_linear_b200 as q


def cdiv(a, b):
    return (a + b - 1) // b


@pytest.mark.parametrize("M,D,V", [(1, 4096, 128256), (129, 328, 4096), (300, 64, 256), (1001, 1000, 50008),
                                   (2048, 4096, 128256), (4096, 4096, 128256), (16384, 4096, 128256), (20000, 64, 8),
                                   (700, 8192, 131072)])
def test_pieces_cover_every_fill_within_the_workspace(M, D, V):
    L = cdiv(V, 128)
    for rows in sorted({M, M - 1, M // 2, 257, 256, 1, 0}):
        if not 0 <= rows <= M:
            continue
        S, units = q.lora_testing_head_splits(M, D, V, rows)
        tiles = cdiv(rows, 256) * cdiv(D, 256)
        assert 1 <= S <= min(64, L)
        if S > 1:
            assert tiles * S <= units
        cuts = [s * L // S for s in range(S + 1)]
        assert cuts[0] == 0 and cuts[-1] == L and all(a < b for a, b in zip(cuts, cuts[1:]))
    _, units = q.lora_testing_head_splits(M, D, V, M)
    assert q.head_bwd_workspace_bytes(M, D, V, 1, 0) >= units * 256 * 256 * 4


def test_choices():
    # 128 tiles in 4 pieces are 6.9 waves of the 74 pairs instead of 1.7; many waves stay whole
    assert q.lora_testing_head_splits(2048, 4096, 128256, 2048)[0] == 4
    assert q.lora_testing_head_splits(16384, 4096, 128256, 16384)[0] == 1
    # few kept rows of a large batch spread over the pairs as well
    assert q.lora_testing_head_splits(16384, 4096, 128256, 200)[0] > 4
    assert q.lora_testing_head_splits(1, 0, 8, 1)[0] == -1 and q.lora_testing_head_splits(4, 8, 8, 5)[0] == -1
