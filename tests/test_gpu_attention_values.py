"""GPU parity of the attention operators where queries, scales or values are far from ordinary: rows
of a tile that differ by orders of magnitude, infinities and NaN that some rows see and others do
not.  Each case names the kernel that it is meant for."""
import pytest
import torch

import qkv_attention_prolog_gb300 as pkg
from tests.attention_util import D, SCALE, ragged, to_dev
from tests.test_gpu_attention import _check_paged

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
FEW = 256 + 2 * 504 * 16 * (D + 2) * 4                # workspaces: parts of few rows, of key tiles
TILES = 256 + 2 * 160 * 2 * 128 * (D + 2) * 4


@pytest.fixture(scope="module", autouse=True)
def _build():
    import __graft_entry__
    __graft_entry__.build()


def _takes(d, max_new, size):
    """The call is the one of the kernel that the case is meant for."""
    a = pkg.make_paged_attention_args(d, max_new, SCALE)
    assert pkg.mlap_paged_attention_get_workspace_size(a) == size


# new tokens, Nq, Nk, workspace: a tile of eight rows, of sixteen, of 128
SHAPES = [(1, 16, 2, FEW), (4, 8, 2, FEW), (70, 8, 2, TILES)]


# ---------------------------------------------------------------------------------------- queries
@pytest.mark.parametrize("new,Nq,Nk,size", SHAPES)
@pytest.mark.parametrize("up", [3e35, 3e-33])
def test_paged_queries_at_the_ends_of_the_range(new, Nq, Nk, size, up):
    # products with the codes that a 32-bit sum of them as they are would not hold (the largest a sum
    # of 128 of 127 * 1.3e36), and small ones; scores as usual
    t = ragged([new, new], [90, 333], 16, Nk, Nq, BF, seed=63)
    t["q"] = (t["q"].float() * up).to(BF)
    t["k_scale"] = t["k_scale"] * (1.0 / up)
    assert bool(torch.isfinite(t["q"]).all()) and float(t["k_scale"].min()) > 1.2e-38
    _takes(to_dev(t), new, size)
    _check_paged(t, new)
