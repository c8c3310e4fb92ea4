"""Workspace sizes of the operators for shapes that their calls refuse."""
import pytest

import __graft_entry__
import tree_speculative_decoding_04_b200 as tv


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return tv.load()


@pytest.mark.parametrize("B,M,V", [(0, 3, 100), (-1, 3, 100), (1, -1, 100), (1, 3, 0), (1, 256, 100),
                                   (1, 2 ** 31 - 1, 100), (1, 3, 262145), (1, 3, 2 ** 31 - 1)])
def test_sampling_needs_no_workspace_for_a_shape_that_is_refused(lib, B, M, V):
    assert lib.tree_accept_sample_workspace_size(B, M, V) == 0


@pytest.mark.parametrize("B,M,V", [(1, 0, 1), (4096, 255, 262144)])
def test_sampling_workspace_grows_with_the_rows(lib, B, M, V):
    # 8 * 384 listed tokens of 8 bytes, 1024 bins of 8 and a state of 44 bytes to a row; 4 bytes for 128 tokens and 16 for
    # 1024; eight parts, each rounded up by 256 to 511 bytes
    rows = B * (M + 1)
    exact = rows * (8 * 384 * 8 + 1024 * 8 + 44 + 4 * -(-V // 128) + 16 * -(-V // 1024))
    assert exact + 8 * 256 <= lib.tree_accept_sample_workspace_size(B, M, V) <= exact + 8 * 511


@pytest.mark.parametrize("M,Hkv,window", [(2 ** 31 - 1, 2, 0), (256, 2, 0), (3, 3, 0), (3, 2, -1)])
def test_scored_attention_needs_no_workspace_for_a_shape_that_is_refused(lib, M, Hkv, window):
    assert lib.tree_attention_scored_workspace_size(1, M, 4, Hkv, 64, 1 << 20, window) == 0
