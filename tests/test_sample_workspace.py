"""The workspace of kda_sample, on the CPU: what its sections need, and the refusal of one byte less."""
import ctypes

import pytest

from test_sample_abi import ALIAS, L, SAMPLE, WORKSPACE, P, call  # noqa: F401  (L: a fixture)

TILE = 4 + 16 * 4 + 8      # the largest logit of a tile of 1024, of each of its 16 groups, and the sum of its weights
ROW = 3 * 8 + 8 + 4 + 4    # what the last pass takes of a row


@pytest.mark.parametrize("R,V", [(1, 1), (1, 1024), (3, 1025), (4, 1000), (7, 5000), (256, 160000), (2048, 500), (192, 50021),
                                 (3, 1 << 22)])
def test_it_holds_every_section_and_one_byte_less_is_refused(L, R, V):  # noqa: F811
    tiles = (V + 1023) // 1024
    size = L.kda_sample_workspace_size(R, V)
    # (sections begin at multiples of 16 bytes: up to 12 and 8 between them)
    assert R * (tiles * TILE + ROW) <= size <= R * (tiles * TILE + ROW) + 20
    ask = lambda n: call(L.kda_sample, SAMPLE, dict(R=R, V=V, token=P(1), size=ctypes.c_size_t(n)))  # noqa: E731
    assert ask(size - 1) == WORKSPACE and ask(size - TILE) == WORKSPACE
    assert ask(size) == ALIAS      # (past the size: what the call is refused for in the end)
