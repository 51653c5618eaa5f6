"""GPU parity of the attention operators where queries, scales or values are far from ordinary: rows
of a tile that differ by orders of magnitude, infinities and NaN that some rows see and others do
not.  Each case names the kernel that it is meant for."""
import numpy as np
import pytest
import torch

import oracle
import qkv_attention_prolog_gb300 as pkg
from tests.attention_util import (D, SCALE, assert_within, attn_tolerance, prompts, ragged, run_paged,
                                  run_window, to_dev)
from tests.gpu_util import f64
from tests.test_gpu_attention import _check_paged

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
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


def _oracle_paged(t, scale=SCALE, window=0, sinks=0):
    with np.errstate(invalid="ignore"):
        return oracle.paged_attention(f64(t["q"]), t["k_cache"].numpy(), t["v_cache"].numpy(),
                                      t["k_scale"].numpy(), t["v_scale"].numpy(),
                                      t["cu_seqlens"].numpy(), t["context_lens"].numpy(),
                                      t["block_table"].numpy(), scale, window, sinks)


def _keys(t):
    return int((t["context_lens"] + t["cu_seqlens"].diff()).max())


# new tokens, Nq, Nk, workspace: a tile of eight rows, of sixteen, of 128
SHAPES = [(1, 16, 2, FEW), (4, 8, 2, FEW), (70, 8, 2, TILES)]


# ---------------------------------------------------------------------------------------- queries
@pytest.mark.parametrize("new,Nq,Nk,size", SHAPES)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("loud", [float("inf"), float("nan"), 2.0 ** 40, 2.0 ** 13])
def test_paged_rows_do_not_depend_on_each_other(new, Nq, Nk, size, dtype, loud):
    # one row of a tile holds an infinity, a NaN or values far above the others': the others' outputs
    # are those of their own scores
    if loud == 2.0 ** 40 and dtype == FP:
        pytest.skip("no fp16 value")
    t = ragged([new, new], [90, 333], 16, Nk, Nq, dtype, seed=61)
    ordinary = f64(t["q"]).copy()
    if np.isfinite(loud):
        t["q"][0, 1] = (t["q"][0, 1].float() * loud).to(dtype)
    else:
        t["q"][0, 1, 9] = loud
    ordinary[0, 1] = 0.0
    ref = _oracle_paged(t)
    d = to_dev(t)
    _takes(d, new, size)
    assert run_paged(d, new) == 0
    kmax = 127.0 * float(t["k_scale"].max())
    tol = attn_tolerance(ref, None, np.abs(ordinary).max() * kmax * D * SCALE, dtype, FP, _keys(t))
    rows = slice(0, int(t["cu_seqlens"][-1]))
    got, want, tol = f64(d["out"])[rows].copy(), ref["out"][rows].copy(), tol[rows]
    assert np.isnan(got[0, 1]).all() if not np.isfinite(loud) else np.isfinite(got[0, 1]).all()
    got[0, 1] = want[0, 1] = tol[0, 1] = 0.0
    assert_within(got, want, tol, "the other rows")


@pytest.mark.parametrize("new,Nq,Nk,size", SHAPES)
@pytest.mark.parametrize("dtype,big", [(BF, 2.0 ** 60), (FP, 60000.0)])
def test_paged_elements_of_a_row_that_differ_widely(new, Nq, Nk, size, dtype, big):
    # a channel of q far above the others meets keys whose codes are all 0 there: it adds nothing
    t = ragged([new, new], [90, 333], 16, Nk, Nq, dtype, seed=62)
    t["q"][:, :, 70] = 0.0
    top = float(np.abs(f64(t["q"])).max())
    t["q"][:, :, 70] = big
    t["k_cache"][..., 70] = 0
    ref = _oracle_paged(t)
    d = to_dev(t)
    _takes(d, new, size)
    assert run_paged(d, new) == 0
    kmax = 127.0 * float(t["k_scale"].max())
    tol = attn_tolerance(ref, None, top * kmax * D * SCALE, dtype, FP, _keys(t))
    rows = slice(0, int(t["cu_seqlens"][-1]))
    assert_within(f64(d["out"])[rows], ref["out"][rows], tol[rows], "out")


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


# ----------------------------------------------------------------------------------------- scales
@pytest.mark.parametrize("new,ctx,window,size", [(2, 95, 81, FEW), (12, 90, 85, FEW), (20, 90, 85, TILES)])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("name", ["k_scale", "v_scale"])
def test_paged_bad_scale_between_the_rows_of_a_tile(new, ctx, window, size, dtype, name):
    # page 6 holds positions 96..111, which a tile's later rows alone see; page 0's last position
    # leaves the window of its later rows
    for bad, page in ((float("nan"), 6), (float("inf"), 6), (-float("inf"), 6), (float("nan"), 0)):
        t = ragged([new, new], [ctx, 33], 16, 2, 8, dtype, seed=64)
        t[name][t["block_table"][0, page]] = bad
        _takes(to_dev(t), new, size)
        _check_paged(t, new, window if page == 0 else 0, 0, nonfinite=True)


@pytest.mark.parametrize("new,size", [(1, FEW), (12, FEW), (20, TILES)])
@pytest.mark.parametrize("name", ["k_scale", "v_scale"])
@pytest.mark.parametrize("page", [0, 700, 1249])
def test_paged_bad_scale_of_one_head_in_one_part(new, size, name, page):
    # of a context that several blocks share: the rows of the other head join parts without it
    for bad in (float("nan"), float("inf")):
        t = ragged([new], [20000], 16, 2, 8, BF, seed=65)
        t[name][t["block_table"][0, page], 1] = bad
        _takes(to_dev(t), new, size)
        _check_paged(t, new, nonfinite=True)


# ------------------------------------------------------------------------------- rows of no token
def _loud(rows, loud):
    return rows.normal_(generator=torch.Generator(device="cuda").manual_seed(3)).mul_(1e4) if loud else rows.zero_()


@pytest.mark.parametrize("kind", ["window", "paged"])
def test_rows_of_no_token_do_not_reach_the_others_bits(kind):
    # groups of three heads fill 126 of a tile's 128 rows: the last two hold what an earlier call (of
    # whole tiles) left in shared memory, and those behind a sequence's end whatever lies behind it
    Nk, sms = 8, torch.cuda.get_device_properties(0).multi_processor_count
    if kind == "window":
        full, t = to_dev(prompts([256] * 24, Nk, Nk, BF, seed=70)), prompts([1000, 1333], Nk, 3 * Nk, BF, seed=71, pad=100)
        run, longest, rows_full = run_window, 1333, 256
    else:
        full = to_dev(ragged([256] * 24, [900] * 24, 64, Nk, Nk, BF, seed=72))
        t = ragged([150] * 20, [1500 - 11 * b for b in range(20)], 64, Nk, 3 * Nk, BF, seed=73, pad=100)
        run, longest, rows_full = run_paged, 150, 256
        _takes(to_dev(t), longest, TILES)
    assert 24 * Nk > sms                              # a block of 256 rows for each SM
    d = to_dev(t)
    end = int(t["cu_seqlens"][-1])
    got = []
    for loud in (False, True, False, True):
        _loud(full["q"], loud)
        _loud(d["q"][end:], loud)
        assert run(full, rows_full) == 0
        assert run(d, longest) == 0
        got.append(d["out"][:end].clone())
    for other in got[1:]:
        assert torch.equal(got[0].view(torch.int16), other.view(torch.int16))
