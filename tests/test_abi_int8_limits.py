"""Borders of the sizes that the int8 MoE layer takes, without a GPU."""

import os

import pytest

from block_diffusion_lm_tq4_amd import _lib

E_SHAPE, E_WS = 2, 4
FAKE = 0x10000          # a non-null, 256-byte aligned address that is never touched


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libtq4.so is not built (run __graft_entry__.build())")
    return _lib.lib()


def test_moe_row_tile_limit(L):
    """t * topk / 256 + n_experts row tiles: 65534 are taken, 65535 are not."""
    e, topk, n1, k = 8, 8, 32, 32
    t = (65534 - e + 1) * 256 // topk - 1
    size = L.tq4_moe_grouped_int8_workspace_size
    assert size(t, topk, e, n1, k) > 0 and size(t + 1, topk, e, n1, k) == 0

    def call(tokens):
        return L.tq4_moe_grouped_int8(FAKE, tokens, k, FAKE, FAKE, topk, e, FAKE, n1, FAKE, FAKE,
                                      None, 0, None)

    assert call(t) == E_WS and call(t + 1) == E_SHAPE
