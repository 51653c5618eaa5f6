"""Attention operators without a GPU: phase-1 validation through the C ABI, the binding's own checks,
and pins of the float64 oracle."""
import ctypes

import numpy as np
import pytest
import torch

import __graft_entry__
import oracle
import qkv_attention_prolog_gb300 as pkg
from qkv_attention_prolog_gb300 import _lib
from tests.test_abi_host import Fake

NULL, SHAPE, DTYPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5
BF, FP, I8, I64, F32 = torch.bfloat16, torch.float16, torch.int8, torch.int64, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()
    return _lib.load()


def _tensors(T=9, B=2, Nq=8, Nk=2, D=128, bs=16, num=5, width=2, dtype=BF):
    return {
        "qkv": Fake((T, (Nq + 2 * Nk) * D), dtype), "cos": Fake((T, D), dtype),
        "sin": Fake((T, D), dtype), "q_out": Fake((T, Nq, D), dtype), "q": Fake((T, Nq, D), dtype),
        "k": Fake((T, Nk, D), dtype), "v": Fake((T, Nk, D), dtype), "out": Fake((T, Nq, D), dtype),
        "cu_seqlens": Fake((B + 1,), I64), "context_lens": Fake((B,), I64),
        "block_table": Fake((B, width), I64), "k_cache": Fake((num, bs, Nk, D), I8),
        "v_cache": Fake((num, bs, Nk, D), I8), "k_scale": Fake((num, Nk), F32),
        "v_scale": Fake((num, Nk), F32)}


OPS = {"kv_append": (_lib.mlap_kv_append_args_t, _lib._APPEND_TENSORS),
       "paged_attention": (_lib.mlap_paged_attention_args_t, _lib._PAGED_TENSORS),
       "window_attention": (_lib.mlap_window_attention_args_t, _lib._WINDOW_TENSORS)}


def _block(op, t, **kw):
    cls, names = OPS[op]
    a = cls()
    for n in names:
        setattr(a, n, t[n].desc() if t.get(n) is not None else _lib.tensor_desc(None))
    given = dict(Nq=8, Nk=2, max_new=4, epsilon=1e-6, window=0, sinks=0, softmax_scale=0.1)
    given.update(kw)
    for n, v in given.items():
        if any(n == f[0] for f in cls._fields_):
            setattr(a, n, v)
    return a


def _status(op, t, **kw):
    a, out = _block(op, t, **kw), ctypes.c_size_t()
    fn = getattr(_lib.load(), f"mlap_{op}_get_workspace_size")
    st = fn(ctypes.byref(a), ctypes.byref(out))
    if st:
        assert _lib.load().mlap_last_error().decode()
    return st, out.value


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_valid_calls_size_the_workspace(op, dtype):
    for t in (_tensors(dtype=dtype), _tensors(T=0, dtype=dtype), _tensors(B=0, dtype=dtype),
              _tensors(bs=48, num=0, dtype=dtype), _tensors(width=0, dtype=dtype)):
        st, size = _status(op, t, cache_mode=b"PA_BSND")
        assert st == 0, _lib.load().mlap_last_error()
        assert size >= 256 and size % 256 == 0


PAGE_REFUSALS = [
    ("context_lens", Fake((3,), I64), SHAPE), ("context_lens", Fake((2,), I8), DTYPE),
    ("block_table", Fake((3, 2), I64), SHAPE), ("block_table", Fake((2,), I64), SHAPE),
    ("block_table", Fake((2, 2), F32), DTYPE),
    ("block_table", Fake((2, (1 << 26) + 1), I64), UNSUPPORTED),
    ("k_cache", Fake((5, 16, 2, 128), BF), DTYPE), ("v_cache", Fake((4, 16, 2, 128), I8), SHAPE),
    ("v_cache", Fake((5, 16, 1, 128), I8), SHAPE),
    ("k_scale", Fake((5, 2), BF), DTYPE), ("v_scale", Fake((5, 3), F32), SHAPE),
    ("k_scale", None, NULL), ("cu_seqlens", None, NULL), ("cu_seqlens", Fake((2, 3), I64), SHAPE),
    ("cu_seqlens", Fake((3,), F32), DTYPE),
]


@pytest.mark.parametrize("op", ["kv_append", "paged_attention"])
@pytest.mark.parametrize("name,value,code", PAGE_REFUSALS)
def test_refusals_of_pages(op, name, value, code):
    t = _tensors()
    t[name] = value
    got = _status(op, t)[0]
    if value is None:
        a = _block(op, t)
        src = _tensors()[name].desc()
        src.data = None
        setattr(a, name, src)
        out = ctypes.c_size_t()
        got = getattr(_lib.load(), f"mlap_{op}_get_workspace_size")(ctypes.byref(a), ctypes.byref(out))
    assert got == code, _lib.load().mlap_last_error()


@pytest.mark.parametrize("op", ["kv_append", "paged_attention"])
def test_refusals_of_page_sizes(op):
    for bs in (8, 24, 0, 1 << 20):
        assert _status(op, _tensors(bs=bs))[0] == UNSUPPORTED, bs
    assert _status(op, _tensors(), cache_mode=b"PA_NZ")[0] == UNSUPPORTED
    t = _tensors()
    t["k_cache"], t["v_cache"] = Fake((5, 16, 2, 64), I8), Fake((5, 16, 2, 64), I8)
    assert _status(op, t)[0] == UNSUPPORTED


def test_refusals_of_append():
    for name, value, code in [
            ("qkv", Fake((9, 12 * 128), F32), DTYPE), ("qkv", Fake((9, 12 * 128 + 1), BF), SHAPE),
            ("qkv", Fake((9, 12 * 64), BF), UNSUPPORTED), ("qkv", Fake((3, 3, 12 * 128), BF), SHAPE),
            ("cos", Fake((9, 64), BF), SHAPE), ("sin", Fake((9, 128), FP), DTYPE),
            ("q_out", Fake((9, 8, 128), FP), DTYPE), ("q_out", Fake((8, 8, 128), BF), SHAPE),
            ("gamma_k", Fake((128,), BF), NULL), ("gamma_q", Fake((128,), BF), NULL)]:
        t = _tensors()
        t[name] = value
        assert _status("kv_append", t)[0] == code, (name, _lib.load().mlap_last_error())
    t = _tensors()
    t["gamma_q"], t["gamma_k"] = Fake((128,), BF), Fake((128,), BF)
    assert _status("kv_append", t)[0] == 0
    t["gamma_k"] = Fake((128,), FP)
    assert _status("kv_append", t)[0] == DTYPE
    assert _status("kv_append", _tensors(), epsilon=-1.0)[0] == SHAPE
    assert _status("kv_append", _tensors(), epsilon=float("nan"))[0] == SHAPE
    assert _status("kv_append", _tensors(), max_new=0)[0] == SHAPE
    assert _status("kv_append", _tensors(), max_new=-1)[0] == SHAPE
    assert _status("kv_append", _tensors(), Nk=0)[0] == SHAPE
    t = _tensors(Nq=7)
    assert _status("kv_append", t, Nq=7)[0] == SHAPE              # Nq not a multiple of Nk
    t = _tensors(Nq=0)
    assert _status("kv_append", t, Nq=0)[0] == 0                  # an empty q_out is no tensor
    t["q_out"] = Fake((9, 8, 128), BF)
    assert _status("kv_append", t, Nq=0)[0] == UNSUPPORTED
    t = _tensors()
    t["q_out"].addr = t["qkv"].addr + 128
    assert _status("kv_append", t)[0] == UNSUPPORTED              # in place: heads move


@pytest.mark.parametrize("op", ["paged_attention", "window_attention"])
def test_refusals_of_attention(op):
    for name, value, code in [
            ("q", Fake((9, 8, 128), F32), DTYPE), ("q", Fake((9, 8 * 128), BF), SHAPE),
            ("q", Fake((9, 8, 64), BF), UNSUPPORTED), ("q", Fake((9, 7, 128), BF), SHAPE),
            ("out", Fake((9, 8, 128), FP), DTYPE), ("out", Fake((8, 8, 128), BF), SHAPE)]:
        t = _tensors()
        t[name] = value
        if name == "q" and value.shape == (9, 7, 128):
            t["out"] = Fake((9, 7, 128), BF)
        assert _status(op, t)[0] == code, (name, _lib.load().mlap_last_error())
    for kw in (dict(window=-1), dict(sinks=-1), dict(softmax_scale=float("inf")),
               dict(softmax_scale=float("nan")), dict(max_new=0)):
        assert _status(op, _tensors(), **kw)[0] == SHAPE, kw
    assert _status(op, _tensors(), window=1 << 62, sinks=1 << 62)[0] == 0
    t = _tensors()
    t["out"] = t["q"]
    assert _status(op, t)[0] == UNSUPPORTED
    t = _tensors()
    t["q"].addr += 8
    assert _status(op, t)[0] == UNSUPPORTED                       # 16-byte alignment
    t = _tensors(Nq=258)
    assert _status(op, t)[0] == UNSUPPORTED                       # 129 heads share one of k
    t = _tensors(Nq=256)
    t["out"].addr += 1 << 30                                      # (clear of the large q)
    assert _status(op, t)[0] == 0


def test_refusals_of_window_attention():
    for name, value, code in [
            ("k", Fake((9, 2, 128), FP), DTYPE), ("v", Fake((9, 4, 128), BF), SHAPE),
            ("v", Fake((8, 2, 128), BF), SHAPE), ("k", Fake((9, 256), BF), SHAPE),
            ("k", Fake((9, 3, 128), BF), SHAPE)]:
        t = _tensors()
        t[name] = value
        assert _status("window_attention", t)[0] == code, name
    t = _tensors()
    t["out"].addr = t["v"].addr
    assert _status("window_attention", t)[0] == UNSUPPORTED


@pytest.mark.parametrize("op", OPS)
def test_execute_checks_the_workspace_before_device_work(op):
    fn = getattr(_lib.load(), f"mlap_{op}_execute")
    a = _block(op, _tensors())
    size = _status(op, _tensors())[1]
    assert fn(ctypes.byref(a), None, 1 << 30, None) == WORKSPACE
    assert fn(ctypes.byref(a), 4096, size - 1, None) == WORKSPACE
    assert fn(ctypes.byref(a), 4096 + 64, size, None) == WORKSPACE
    assert fn(None, 4096, size, None) == NULL
    empty = _block(op, _tensors(T=0))
    assert fn(ctypes.byref(empty), None, 0, None) == 0            # nothing to do
    none = _block(op, _tensors(B=0))
    assert fn(ctypes.byref(none), None, 0, None) == 0


def test_binding_refuses_tensors_that_are_not_on_one_cuda_device():
    z = torch.zeros(4, 8, 128, dtype=BF)
    with pytest.raises(ValueError, match="CUDA device"):
        pkg.make_window_attention_args({"q": z, "k": z, "v": z, "out": z,
                                        "cu_seqlens": torch.zeros(2, dtype=I64)}, 4, 0.1)


# ------------------------------------------------------------------------------------ oracle pins
def test_pin_visible():
    assert oracle.attention.visible(5, 0, 0).tolist() == [0, 1, 2, 3, 4, 5]
    assert oracle.attention.visible(5, 2, 0).tolist() == [4, 5]
    assert oracle.attention.visible(5, 2, 1).tolist() == [0, 4, 5]
    assert oracle.attention.visible(1, 8, 9).tolist() == [0, 1]


def test_pin_equal_scores_average_the_visible_values():
    rng = np.random.default_rng(0)
    q = np.zeros((7, 2, 128))
    k, v = rng.standard_normal((2, 7, 1, 128))
    o = oracle.window_attention(q, k, v, [1, 6], 0.3, window=2, sinks=1)["out"]
    np.testing.assert_allclose(o[1], np.repeat(v[1], 2, 0))
    np.testing.assert_allclose(o[5, 1], (v[1, 0] + v[4, 0] + v[5, 0]) / 3)
    assert (o[0] == 0).all() and (o[6] == 0).all()                # rows of no sequence


def test_pin_one_key_dominates():
    q = np.ones((2, 1, 128))
    k = np.stack([np.full((1, 128), 2.0), np.full((1, 128), -2.0)])
    v = np.stack([np.full((1, 128), 5.0), np.full((1, 128), 9.0)])
    o = oracle.window_attention(q, k, v, [0, 2], 1.0)["out"]
    np.testing.assert_allclose(o[1], 5.0)


def test_pin_paged_equals_dense_over_the_dequantised_rows():
    rng = np.random.default_rng(1)
    kc, vc = rng.integers(-127, 128, (2, 4, 16, 2, 128)).astype(np.int8)
    ks, vs = rng.random((2, 4, 2)) * 0.02
    table = np.array([[2, 0, 3]])
    n = 40
    deq = lambda c, s: (c * s[:, None, :, None])[table[0]].reshape(-1, 2, 128)[:n]
    q = rng.standard_normal((n, 4, 128))
    dense = oracle.window_attention(q, deq(kc, ks), deq(vc, vs), [0, n], 0.1, 9, 2)["out"]
    paged = oracle.paged_attention(q, kc, vc, ks, vs, [0, n], [0], table, 0.1, 9, 2)["out"]
    np.testing.assert_allclose(paged, dense)
    last = oracle.paged_attention(q[-1:], kc, vc, ks, vs, [0, 1], [n - 1], table, 0.1, 9, 2)["out"]
    np.testing.assert_allclose(last[0], dense[-1])


def test_pin_append_holds_every_value_within_half_a_step():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((20, 4 * 128))
    one, zero = np.ones((20, 128)), np.zeros((20, 128))
    z8, zf = np.zeros((3, 16, 1, 128), np.int8), np.full((3, 1), 99.0)
    r = oracle.kv_append(x, one, zero, [0, 20], [5], np.array([[2, 0]]), z8, z8, zf * 0 + 0.5, zf, 2, 1)
    # the page holds five earlier rows: its k scale stays at least 0.5 and v's at 99
    assert r["k_scale"][2, 0] == 0.5 and r["v_scale"][2, 0] == 99.0
    top = np.abs(x[11:, 2 * 128:3 * 128]).max() / 127
    assert r["k_scale"][0, 0] == top and r["k_scale"][1, 0] == 0.5
    got = r["k_cache"][0, :9, 0] * r["k_scale"][0, 0]
    assert np.abs(got - x[11:, 2 * 128:3 * 128]).max() <= top / 2 * (1 + 1e-12)
    np.testing.assert_array_equal(r["q_out"], x.reshape(20, 4, 128)[:, :2])
    assert len(r["written"]) == 20


def test_pin_append_rotates_k_and_q_but_not_v():
    x = np.zeros((1, 3 * 128))
    x[0, 0], x[0, 128 + 64], x[0, 256] = 1.0, 1.0, 1.0
    c, s = np.full((1, 128), 0.6), np.full((1, 128), 0.8)
    z8, zf = np.zeros((1, 16, 1, 128), np.int8), np.zeros((1, 1))
    r = oracle.kv_append(x, c, s, [0, 1], [0], np.array([[0]]), z8, z8, zf, zf, 1, 1)
    assert r["q_out"][0, 0, 0] == 0.6 and r["q_out"][0, 0, 64] == 0.8
    k = r["k_cache"][0, 0, 0] * r["k_scale"][0, 0]
    assert k[0] == pytest.approx(-0.8) and k[64] == pytest.approx(0.6, abs=0.8 / 254)
    assert (r["v_cache"][0, 0, 0][:2] == [127, 0]).all()


@pytest.mark.parametrize("op", ["kv_append", "paged_attention"])
def test_refuses_more_pages_than_32_bits_count(op):
    assert _status(op, _tensors(num=1 << 31))[0] == UNSUPPORTED
    assert _status(op, _tensors(num=(1 << 31) - 1))[0] == 0


def test_workspaces_of_the_attention_calls():
    # the header alone; parts of few rows; parts of key tiles (from 49 rows, or few long prompts)
    def size(op, max_new, B=2, **kw):
        t = _tensors(T=6000, B=B)
        t["out"].addr += 1 << 40                      # (apart from the other tensors)
        st, n = _status(op, t, max_new=max_new, **kw)
        assert st == 0
        return n

    few, many = size("paged_attention", 12), size("paged_attention", 13)
    # two slots for each of 504 stretches and 16 rows, or of 160 and two tiles of 128 rows: O, m and l
    assert few == 256 + 2 * 504 * 16 * (128 + 2) * 4
    assert many == 256 + 2 * 160 * 2 * 128 * (128 + 2) * 4
    assert _status("kv_append", _tensors())[1] == 256
    assert size("window_attention", 900) == 256
    assert size("window_attention", 5000) == many
    assert size("window_attention", 5000, window=200) == 256
    assert size("window_attention", 5000, B=100) == 256


@pytest.mark.parametrize("op", OPS)
def test_lengths_tables_and_scales_begin_at_any_element(op):
    names = set(OPS[op][1])
    for name, size in (("cu_seqlens", 8), ("context_lens", 8), ("block_table", 8), ("k_scale", 4),
                       ("v_scale", 4)):
        if name not in names:
            continue
        t = _tensors()
        t[name].addr += size                          # as context_lens[1:] of a longer batch
        assert _status(op, t)[0] == 0, (name, _lib.load().mlap_last_error())
        t[name].addr += size // 2
        assert _status(op, t)[0] == UNSUPPORTED, name
    for name in names & {"q", "k", "v", "qkv", "cos", "sin", "out", "q_out", "k_cache", "v_cache"}:
        t = _tensors()
        t[name].addr += 8
        assert _status(op, t)[0] == UNSUPPORTED, name


@pytest.mark.parametrize("op", ["paged_attention", "window_attention"])
def test_refuses_scales_beyond_32_bits(op):
    # fp32 ends below 3.41e38, and the kernels count in powers of two: 2.36e38 * log2(e)
    for scale in (1e300, -1e39, 2.4e38):
        assert _status(op, _tensors(), softmax_scale=scale)[0] == SHAPE, scale
    for scale in (2.3e38, -2.3e38, 1e-300, 0.0):
        assert _status(op, _tensors(), softmax_scale=scale)[0] == 0, scale
