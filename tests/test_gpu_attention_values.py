"""GPU parity of the attention operators where queries, scales or values are far from ordinary: rows
of a tile that differ by orders of magnitude, infinities and NaN that some rows see and others do
not.  Each case names the kernel that it is meant for."""
import numpy as np
import pytest
import torch

import oracle
import qkv_attention_prolog_gb300 as pkg
from tests.attention_util import (D, SCALE, assert_within, attn_tolerance, prompts, ragged, run_append,
                                  run_paged, run_window, to_dev, workspace)
from tests.gpu_util import f64
from tests.test_gpu_attention import _check_paged, _max_dot

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
@pytest.mark.parametrize("dtype,loud", [(BF, float("inf")), (BF, float("nan")), (BF, 2.0 ** 40), (BF, 2.0 ** 13),
                                        (FP, float("inf")), (FP, float("nan")), (FP, 2.0 ** 13)])
def test_paged_rows_do_not_depend_on_each_other(new, Nq, Nk, size, dtype, loud):
    # one row of a tile holds an infinity, a NaN or values far above the others': the others' outputs
    # are those of their own scores
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


# ------------------------------------------------------------------------------- places of tensors
@pytest.mark.parametrize("new", [1, 12, 70])
def test_lengths_tables_and_scales_of_longer_tensors(new):
    # a batch's part that begins anywhere: appended and attended over as if it were alone
    t = ragged([new, new], [300, 77], 16, 1, 4, BF, seed=74, width=37)
    want, got = to_dev(t), to_dev(t)
    for name, lead in (("cu_seqlens", 1), ("context_lens", 3), ("block_table", 1), ("k_scale", 3), ("v_scale", 1)):
        x = want[name].reshape(-1)
        got[name] = torch.cat([x.new_full((lead,), 99), x])[lead:].view(want[name].shape)
        assert got[name].data_ptr() % 16 != 0 and got[name].is_contiguous()
    for d in (want, got):
        assert run_append(d, 4, 1, new) == 0
        assert run_paged(d, new) == 0
    for name in ("q_out", "out", "k_cache", "v_cache", "k_scale", "v_scale"):
        assert torch.equal(want[name], got[name]), name
    p = prompts([40, 90], 1, 4, BF, seed=75)
    want, got = to_dev(p), to_dev(p)
    got["cu_seqlens"] = torch.cat([want["cu_seqlens"][:1], want["cu_seqlens"]])[1:]
    assert run_window(want, 90) == 0 and run_window(got, 90) == 0
    assert torch.equal(want["out"], got["out"])


def test_paged_batch_in_two_calls_on_slices():
    # single tokens and a prompt's chunk, each by the kernel meant for it, into one output
    t = ragged([1, 1, 1, 70], [900, 4, 333, 200], 16, 2, 8, FP, seed=76, width=61)
    ref = _oracle_paged(t)
    d = to_dev(t)
    for lo, hi, new, size in ((0, 3, 1, FEW), (3, 4, 70, TILES)):
        part = dict(d, cu_seqlens=d["cu_seqlens"][lo:hi + 1], context_lens=d["context_lens"][lo:hi],
                    block_table=d["block_table"][lo:hi])
        _takes(part, new, size)
        assert run_paged(part, new) == 0
    tol = attn_tolerance(ref, None, np.abs(f64(t["q"])).max() * 127.0 * float(t["k_scale"].max()) * D * SCALE, FP, FP,
                         _keys(t))
    rows = int(t["cu_seqlens"][-1])
    assert_within(f64(d["out"])[:rows], ref["out"][:rows], tol[:rows], "out")
    assert bool((d["out"][rows:] == 7).all())


# ------------------------------------------------------------------------------ values of prompts
def _check_window_kinds(t, max_new, window=0, sinks=0):
    """Finite outputs within the tolerance; where the oracle has a NaN or an infinity, the same one."""
    with np.errstate(invalid="ignore"):
        ref = oracle.window_attention(f64(t["q"]), f64(t["k"]), f64(t["v"]), t["cu_seqlens"].numpy(), SCALE,
                                      window, sinks, out=f64(t["out"]))
    d = to_dev(t)
    assert run_window(d, max_new, window, sinks) == 0
    got, want = f64(d["out"]), ref["out"]
    ok = np.isfinite(want)
    odd = np.where(ok, 0.0, want)
    assert np.array_equal(np.where(np.isfinite(got), 0.0, got), odd, equal_nan=True)
    fin = lambda x: np.nan_to_num(f64(x), nan=0, posinf=0, neginf=0)
    with np.errstate(invalid="ignore"):
        tol = attn_tolerance(ref, None, _max_dot(fin(t["q"]), fin(t["k"])), t["q"].dtype, t["q"].dtype, max_new)
    rows = int(t["cu_seqlens"][-1])
    tol[rows:] = 0
    assert_within(np.where(ok, got, 0), np.where(ok, want, 0), np.where(ok, tol, 0), "out")
    first = d["out"].clone()
    assert run_window(d, max_new, window, sinks) == 0
    assert torch.equal(first.view(torch.int16), d["out"].view(torch.int16))
    return ok[:rows]


KINDS = [float("nan"), float("inf"), -float("inf")]
ODD = [  # new, Nq, Nk, window, sinks
    ([260, 140], 3, 1, 0, 0),
    ([260, 140], 3, 1, 70, 3),
    ([500], 1, 1, 100, 17),                           # one head a tile: the most tokens
    ([500], 1, 1, 300, 9),
    ([700], 2, 2, 33, 650),                           # sinks beyond the windows of most rows
    ([90, 7, 33], 64, 2, 20, 4),
    ([1, 2, 130], 8, 2, 1, 0),
    ([2100, 40], 3, 1, 0, 0),                         # items in parts
    ([2300], 2, 1, 1700, 40),
    ([1 + b * 7 % 40 for b in range(300)], 2, 1, 16, 2),
]


@pytest.mark.parametrize("new,Nq,Nk,window,sinks", ODD)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_window_values_that_are_not_finite(new, Nq, Nk, window, sinks, dtype):
    # single elements here and there, some channels of some rows stay finite
    t = prompts(new, Nk, Nq, dtype, seed=66, pad=40)
    g = torch.Generator().manual_seed(1)
    total = sum(new)
    for n in ("q", "k", "v"):
        t[n][total:] = float("nan")
    for kind in KINDS:
        for _ in range(max(1, total // 90)):
            at = [int(torch.randint(0, m, (1,), generator=g)) for m in (total, Nk, D)]
            t["v"][at[0], at[1], at[2]] = kind
    ok = _check_window_kinds(t, max(new), window, sinks)
    assert ok.any() and not ok.all()


@pytest.mark.parametrize("new,Nq,Nk,window,sinks", ODD[:5] + ODD[7:9])
def test_window_channels_and_stretches_that_are_not_finite(new, Nq, Nk, window, sinks):
    t = prompts(new, Nk, Nq, BF, seed=67)
    t["v"][:, 0, 5] = float("nan")                    # everywhere: each row sees its own
    t["v"][:, 0, 6] = float("inf")
    t["v"][::2, 0, 127] = float("-inf")
    _check_window_kinds(t, max(new), window, sinks)
    t["v"][new[0] // 2:new[0] // 2 + 60] = float("inf")
    t["v"][new[0] - 9:] = float("nan")
    _check_window_kinds(t, max(new), window, sinks)
    t["v"][:] = float("nan")
    assert not _check_window_kinds(t, max(new), window, sinks).any()


@pytest.mark.parametrize("new,Nq,Nk,window,sinks", ODD[:5] + ODD[7:9])
def test_window_keys_and_queries_that_are_not_finite(new, Nq, Nk, window, sinks):
    t = prompts(new, Nk, Nq, FP, seed=68)
    t["k"][new[0] // 3, 0, 9] = float("nan")
    t["k"][new[0] // 2, 0, 8] = float("inf")          # a weight of 0, or no finite one
    t["k"][new[0] - 2, 0, 8] = float("-inf")
    t["q"][5, 0, 0] = float("nan")
    t["v"][new[0] // 4, 0, 3] = float("nan")
    ok = _check_window_kinds(t, max(new), window, sinks)
    assert ok.any() and not ok.all()


def test_window_more_items_than_marks():
    # 160 short prompts of 256 heads: 269 items for each of 152 blocks, which keeps 256 marks
    Nk = 256
    t = prompts([1 + b % 3 for b in range(160)], Nk, Nk, FP, seed=77)
    g = torch.Generator().manual_seed(2)
    for _ in range(60):
        row, head, ch = (int(torch.randint(0, m, (1,), generator=g)) for m in (t["v"].shape[0] - 2, Nk, D))
        t["v"][row, head, ch] = float("nan")
    t["v"][2, :, 7] = float("inf")                    # (the second prompt's last token, in every head)
    ok = _check_window_kinds(t, 3)
    assert ok.any() and not ok.all()


def _window_ms(t, max_new, window=0, sinks=0):
    d = to_dev(t)
    a = pkg.make_window_attention_args(d, max_new, SCALE, window, sinks)
    ws = workspace(pkg.mlap_window_attention_get_workspace_size(a))
    best = float("inf")
    for _ in range(4):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        pkg.mlap_window_attention_execute(a, ws)
        end.record()
        torch.cuda.synchronize()
        best = min(best, start.elapsed_time(end))
    assert pkg.mlap_check_errors(ws) == 0
    return best


@pytest.mark.parametrize("name,first,last,value", [
    ("k", 0, 1, "nan"), ("v", 0, 1, "nan"), ("v", 0, 2000, "nan"), ("v", 1000, 4000, "nan"), ("v", 0, 4096, "inf")])
def test_window_time_does_not_hang_on_what_is_not_finite(name, first, last, value):
    # A second turn of an item costs the first one's time, clearing a tile about as long again, and a
    # row's look at the keys around its own, 127 of them, 128 channels each, about 75 us beside the call's
    # 55: five times the call, whatever V holds.  Rows worked out key by key, 4096 of 8 heads, are a
    # hundred times that.
    t = prompts([4096], 2, 8, BF, seed=69)
    clean = _window_ms(t, 4096)
    t[name][first:last] = float(value)
    assert _window_ms(t, 4096) < 12 * clean
