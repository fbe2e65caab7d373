"""The workspaces of the drafted step's operators: sizes, and refusals of missing, short or misaligned ones."""
import ctypes

import pytest

from latent_mixture_experts_bf16_amd import binding as B
from test_drafted_cpu import FAKE, F32, T, _cache, _says


def _attend(ws, bytes_, rows=2, heads=4):
    return B.lib().moe_tree_attend(ctypes.byref(_cache()), rows, FAKE, 64 * heads, heads, FAKE, None, 0.1, FAKE + 0x300000,
                                   64 * heads, ws, bytes_, None)


def test_attend_workspace():
    need = B.lib().moe_tree_attend_workspace(ctypes.byref(_cache()), 2, 4)
    assert need > 0
    _says(_attend(None, need), "MOE_ERR_INVALID_ARG", "workspace: NULL")
    _says(_attend(FAKE + 8, need), "MOE_ERR_LAYOUT", "workspace: not 16-byte")
    _says(_attend(FAKE, need - 1), "MOE_ERR_SHAPE", f"{need} needed")
    # more queries to a key head never need less
    assert all(B.lib().moe_tree_attend_workspace(ctypes.byref(_cache()), r, 4) <=
               B.lib().moe_tree_attend_workspace(ctypes.byref(_cache()), 4 * r, 4) for r in (1, 5, 20, 100, 5000))


@pytest.mark.parametrize("over", [{}, dict(q=None, ut=None)])
def test_verify_workspace(over):
    need = B.lib().moe_draft_verify_workspace(4, 2, 1000)
    assert need > 0
    z = T(FAKE, F32, [4, 1000])

    def call(ws, bytes_, ut=FAKE, q=FAKE):
        return B.lib().moe_draft_verify(ctypes.byref(z), FAKE, FAKE, 2, None, ut, FAKE, q, 1000, None, FAKE, FAKE, FAKE, FAKE,
                                        FAKE, ws, bytes_, None)

    _says(call(None, need, **over), "MOE_ERR_INVALID_ARG", "workspace: NULL")
    _says(call(FAKE + 4, need, **over), "MOE_ERR_LAYOUT", "workspace: not 16-byte")
    _says(call(FAKE, need - 1, **over), "MOE_ERR_SHAPE", f"{need} needed")
    assert B.lib().moe_draft_verify_workspace(4, 2, 1 << 20) > need
