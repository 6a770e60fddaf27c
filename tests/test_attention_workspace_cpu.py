"""Sizes of the attention's workspaces: bounded for wide heads, without a GPU."""
import pytest

import equivariant_gnn_message_gb300 as eq

MB = 1 << 20
PART_MB = 65  # 64 and a block's rounding


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__

    __graft_entry__.build()


def _align(n):
    return (n + 15) // 16 * 16


@pytest.mark.parametrize("E", [1025, 40_000, 65_536, 1 << 20, 1 << 30])
@pytest.mark.parametrize("H,D,Dv", [(8, 32, 128), (16, 64, 588), (128, 128, 128), (64, 256, 1024)])
def test_parts_of_wide_heads_are_bounded(E, H, D, Dv):
    assert 0 < eq.eqmp_edge_attention_workspace_size(E, H, Dv) <= PART_MB * MB
    edges = _align(E * H * 8) + _align(1000 * H * 4)
    assert 0 < eq.eqmp_edge_attention_backward_workspace_size(1000, E, E, H, D, Dv) - edges <= PART_MB * MB


def test_parts_at_the_limits():
    """Eight blocks, whatever a part takes."""
    assert eq.eqmp_edge_attention_workspace_size(1 << 30, 1024, 1024) == 2 * 8 * 1024 * 1026 * 4
    assert eq.eqmp_edge_attention_workspace_size(1024, 1024, 1024) == 0


def test_ordinary_graphs_have_up_to_2048_blocks():
    for E, block in ((1025, 32), (65_536, 32), (65_537, 64), (1_909_372, 960)):
        assert eq.eqmp_edge_attention_workspace_size(E, 8, 128) == 2 * -(-E // block) * 8 * 130 * 4
