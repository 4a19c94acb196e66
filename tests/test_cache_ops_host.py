"""Host side of the 4-bit latent cache, the reading back of rows, the
accumulated attention weights and the eviction: formats and refusals (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from indexed_sparse_attention_lightning_b200 import _abi, build
from indexed_sparse_attention_lightning_b200 import workloads as W
from tests.test_abi import FAKE, good_cache, good_query, new_tokens

FP4 = {"kv_rope": FAKE, "kv_scale": FAKE}
FORMATS = {"mxfp4": _abi.SA_MXFP4, "nvfp4": _abi.SA_NVFP4}


@pytest.fixture(scope="module")
def L():
    build.build()
    return _abi.lib()


# ----------------------------------------------------------------- formats ---

def _rows(seed, n=64, d=64):
    """Rows over many magnitudes, with all-zero and single-valued groups, ties
    between neighbouring codes and subnormal scales among them."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, d)) * np.exp2(rng.integers(-12, 12, (n, 1)))
    x = x.astype(np.float32)
    x[0] = 0.0
    x[1, :] = 0.0
    x[1, 5] = -3.75
    x[2, ::2] = np.float32(1e-3)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], dtype=np.float32)
    x[3] = np.tile(np.concatenate([ties, -ties]), d // 16)
    x[4] = x[3] * np.float32(2.0 ** -9)
    x[5] = np.float32(2.0 ** -140)
    x[6] = -np.float32(3.0e38)
    x[7, :16] = np.float32(7.5)
    return x


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_the_two_quantisers_agree(fmt):
    """The generator's (thresholds) and the oracle's (nearest by search)."""
    x = _rows(1)
    codes, scales = W.quantize_fp4(x, fmt)
    want_codes, want_scales = oracle.quantize_fp4(x, fmt)
    assert np.array_equal(scales, want_scales)
    assert np.array_equal(codes, want_codes)
    assert np.array_equal(W.fp4_value(codes, scales, fmt), oracle.fp4_decode(fmt, codes, scales))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_quantisation_error_is_half_a_step(fmt):
    """|x - v| is at most half the distance of the neighbouring e2m1 values at
    x's own size, and at most 2 scales (MXFP4: 8 against 6) or the e4m3 scale's
    rounding where the largest values saturate."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((200, 64)).astype(np.float32)
    codes, scales = oracle.quantize_fp4(x, fmt)
    v = oracle.fp4_decode(fmt, codes, scales)
    s = np.repeat(oracle.fp4_scale_decode(fmt, scales), oracle.FP4_GROUP[fmt], axis=-1)
    q = np.abs(x) / s
    step = np.where(q < 2, 0.5, np.where(q < 4, 1.0, 2.0))
    inside = q <= 6
    assert np.all(np.abs(x - v)[inside] <= (step * s / 2)[inside] * (1 + 1e-6))
    assert np.all(q < (8 if fmt == "mxfp4" else 6 * (1 + 2 ** -4) * (1 + 1e-6)))
    assert np.array_equal(np.abs(v)[~inside], (6 * s)[~inside].astype(np.float32))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_workload_rows_decode_to_what_was_quantised(fmt):
    sp = W.WorkloadSpec(name="w4", seed=5, batch=2, seq_len=("list", (70, 129)), h_index=8,
                        heads=16, kv_dtype=fmt)
    wl = W.make_workload(sp)
    assert wl.kv.shape == (wl.num_pages, 64, 256) and wl.kv.dtype == np.uint8
    v = W.fp4_value(wl.kv, wl.kv_scale, fmt)
    used = np.zeros((wl.num_pages, 64), bool)
    for b, n in enumerate(wl.seq_len):
        s = np.arange(n)
        used[wl.page_table[b, s // 64], s % 64] = True
    assert np.all(np.isfinite(v[used])) and np.all(np.isnan(v[~used]))  # poison elsewhere
    assert 0.9 < v[used].std() < 1.1
    out, lse = oracle.sparse_attn(wl, np.array([[0, 5, 69], [1, 128, -1]], np.int32))
    assert np.all(np.isfinite(out)) and np.all(np.isfinite(lse))


# ---------------------------------------------------------------- refusals ---

def ws_size(L, c, q, k=256, uses=_abi.SA_WS_DECODE):
    return L.sa_workspace_size(ctypes.byref(c), None if q is None else ctypes.byref(q), k, uses)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_4_bit_cache_argument_checks(L, fmt):
    dt = {"kv_dtype": FORMATS[fmt], **FP4}
    assert ws_size(L, good_cache(**dt), good_query()) > 0
    for bad in ({"kv_scale": None}, {"kv_rope": None}, {"kv_scale": FAKE + 8},
                {"kv_rope": FAKE + 2}, {"kv_scale_tokens": 1, "kv_scale_dims": 32},
                {"d_latent": 48}, {"d_latent": 40}, {"d_rope": 36}):
        assert ws_size(L, good_cache(**{**dt, **bad}), good_query()) == 0, bad
    assert ws_size(L, good_cache(**{**dt, "d_rope": 0, "kv_rope": None}), good_query()) > 0
    # the names belong to the latent cache: neither index keys nor a query take them
    assert ws_size(L, good_cache(index_dtype=FORMATS[fmt]), good_query()) == 0
    assert ws_size(L, good_cache(**dt), good_query(q_dtype=FORMATS[fmt])) == 0
    t = new_tokens()
    assert L.sa_append_tokens(ctypes.byref(good_cache(**dt)), ctypes.byref(t), FAKE, 8,
                              None) == _abi.SA_ERR_WORKSPACE     # accepted up to the workspace


def read(L, c, n=3, seq=FAKE, pos=FAKE, out=FAKE, dt=_abi.SA_BF16, ws=FAKE, nb=8):
    return L.sa_read_tokens(ctypes.byref(c), n, seq, pos, out, dt, ws, nb, None)


def test_read_tokens_refusals(L):
    c = good_cache()
    assert read(L, c) == _abi.SA_ERR_WORKSPACE                   # all else in order
    assert read(L, c, ws=None) == _abi.SA_ERR_WORKSPACE
    assert read(L, c, n=-1) == _abi.SA_ERR_INVALID_ARG
    for k in ("seq", "pos", "out"):
        assert read(L, c, **{k: None}) == _abi.SA_ERR_INVALID_ARG
    assert read(L, c, out=FAKE + 4) == _abi.SA_ERR_INVALID_ARG
    assert read(L, c, dt=_abi.SA_E4M3) == _abi.SA_ERR_UNSUPPORTED
    assert read(L, good_cache(page_size=32)) == _abi.SA_ERR_UNSUPPORTED


def weigh(L, c, q, idx=FAKE, k=100, lse=FAKE, acc=FAKE, decay=1.0, out=FAKE, ld=256, ws=FAKE,
          nb=8):
    return L.sa_accumulate_weights(ctypes.byref(c), ctypes.byref(q), idx, k, lse, acc, decay, out,
                                   ld, ws, nb, None)


def test_accumulate_weights_refusals(L):
    c, q = good_cache(), good_query(q_index=None, w=None, q_index_scale=None)
    need = ws_size(L, c, q, 100, _abi.SA_WS_WEIGHTS)
    assert need >= 256 + 3 * 4 * 2 * 100
    assert weigh(L, c, q) == _abi.SA_ERR_WORKSPACE               # all else in order
    assert weigh(L, c, q, nb=need - 1) == _abi.SA_ERR_WORKSPACE
    assert weigh(L, c, q, ws=FAKE + 16, nb=need) == _abi.SA_ERR_WORKSPACE
    assert weigh(L, c, q, acc=None) == _abi.SA_ERR_WORKSPACE     # acc_in may be absent
    for bad in ({"idx": None}, {"lse": None}, {"out": None}, {"k": 0}, {"k": -5}, {"ld": 0},
                {"ld": 255}, {"decay": float("nan")}, {"decay": float("inf")},
                {"acc": FAKE + 4}, {"acc": FAKE - 4 * (2 * 256 - 1)}):
        assert weigh(L, c, q, **bad) == _abi.SA_ERR_INVALID_ARG, bad
    assert weigh(L, c, good_query(q=None)) == _abi.SA_ERR_INVALID_ARG
    assert weigh(L, c, good_query(sm_scale=float("nan"))) == _abi.SA_ERR_INVALID_ARG
    assert weigh(L, good_cache(num_pages=1 << 25), q) == _abi.SA_ERR_UNSUPPORTED
    assert ws_size(L, c, q, 0, _abi.SA_WS_WEIGHTS) == 0


def evict(L, c, d, acc=FAKE, ld=256, budget=128, first=4, last=64, acc_out=FAKE << 1, ld_out=128,
          src_pos=FAKE, ws=FAKE, nb=8):
    return L.sa_evict_tokens(ctypes.byref(c), acc, ld, budget, first, last, ctypes.byref(d),
                             acc_out, ld_out, src_pos, ws, nb, None)


def test_evict_tokens_refusals(L):
    c, d = good_cache(), good_cache(seq_len=FAKE << 1, page_table=FAKE << 1)
    need = ws_size(L, c, None, 128, _abi.SA_WS_EVICT)
    assert need >= 256 + 4 * 2 * 128
    assert ws_size(L, c, None, 0, _abi.SA_WS_EVICT) == 0
    assert evict(L, c, d) == _abi.SA_ERR_WORKSPACE               # all else in order
    assert evict(L, c, d, nb=need - 1) == _abi.SA_ERR_WORKSPACE
    assert evict(L, c, d, acc_out=None, ld_out=0, src_pos=None) == _abi.SA_ERR_WORKSPACE
    for bad in ({"acc": None}, {"ld": 0}, {"budget": 0}, {"first": -1}, {"last": -1},
                {"first": 65}, {"budget": 257}, {"ld_out": 127}, {"acc_out": FAKE},
                {"acc_out": FAKE + 4 * (2 * 256 - 1)}, {"acc_out": FAKE - 4 * (2 * 128 - 1)},
                {"first": 2 ** 31 - 1, "last": 2 ** 31 - 1}):
        assert evict(L, c, d, **bad) == _abi.SA_ERR_INVALID_ARG, bad
    assert evict(L, c, d, acc_out=FAKE + 4 * 2 * 256) == _abi.SA_ERR_WORKSPACE
    for other in ({"seq_len": FAKE}, {"seq_len": FAKE + 4}, {"seq_len": FAKE - 4}, {"batch": 3}, {"d_latent": 256}, {"d_rope": 32},
                  {"d_index": 64}, {"index_dtype": _abi.SA_BF16}, {"kv_dtype": _abi.SA_F32},
                  {"max_pages": 1}):
        bad_dst = good_cache(**{"seq_len": FAKE << 1, "page_table": FAKE << 1, **other})
        assert evict(L, c, bad_dst) == _abi.SA_ERR_INVALID_ARG, other
    e4 = {"kv_dtype": _abi.SA_E4M3, **FP4}
    for tile, want in (((0, 0), _abi.SA_ERR_UNSUPPORTED), ((16, 128), _abi.SA_ERR_UNSUPPORTED),
                       ((1, 128), _abi.SA_ERR_WORKSPACE)):
        t = {"kv_scale_tokens": tile[0], "kv_scale_dims": tile[1]}
        assert evict(L, good_cache(**e4, **t),
                     good_cache(**e4, **t, seq_len=FAKE << 1)) == want, tile
    assert evict(L, good_cache(num_pages=1 << 25), d) == _abi.SA_ERR_UNSUPPORTED
    assert evict(L, c, good_cache(seq_len=FAKE << 1, num_pages=1 << 25)) == \
        _abi.SA_ERR_UNSUPPORTED


@pytest.mark.parametrize("fmt", [{}, {"kv_dtype": _abi.SA_MXFP4, **FP4}])
def test_attention_refuses_an_output_its_stores_cannot_reach(L, fmt):
    c, q = good_cache(**fmt), good_query()
    ws = _abi.SA_ERR_WORKSPACE                                   # all else in order
    for out, k, want in ((FAKE, 2048, ws), (FAKE + 8, 2048, _abi.SA_ERR_INVALID_ARG),
                         (FAKE + 2, 1, _abi.SA_ERR_INVALID_ARG), (FAKE + 8, 2049, ws)):
        assert L.sa_sparse_mla_attn(ctypes.byref(c), ctypes.byref(q), FAKE, k, out,
                                    _abi.SA_BF16, None, FAKE, 8, None) == want
        assert L.sa_decode(ctypes.byref(c), ctypes.byref(q), k, None, out, _abi.SA_BF16, None,
                           FAKE, 8, None) == want
    few = good_query(heads=16)                                   # the CUDA-core kernel
    assert L.sa_sparse_mla_attn(ctypes.byref(c), ctypes.byref(few), FAKE, 64, FAKE + 8,
                                _abi.SA_BF16, None, FAKE, 8, None) == ws


def test_new_names_are_bound():
    assert _abi.DTYPES["mxfp4"] == 4 and _abi.DTYPES["nvfp4"] == 5
    assert torch.uint8 is not None and len(set(_abi.EXPORTS)) == len(_abi.EXPORTS)


# ------------------------------------------------- values that are not finite ---

def rows_not_finite(d=64):
    """(rows, which groups of 16 hold a NaN or an infinity)."""
    x = _rows(9, n=12, d=d)
    bad = [(0, 3, np.nan), (1, 20, -np.nan), (2, 40, np.inf), (3, 63, -np.inf), (4, 0, np.nan),
           (4, 1, np.inf), (8, 15, np.nan), (8, 16, np.nan)]
    for r, c, v in bad:
        x[r, c] = v
    x[9, 16:32] = np.nan                                  # nothing else in the group
    x[10, 32:48] = -np.inf
    return x, ~np.isfinite(x).reshape(12, d // 16, 16).all(axis=-1)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_a_group_that_is_not_finite_reads_back_as_nan(fmt):
    x, bad = rows_not_finite()
    if fmt == "mxfp4":
        bad = np.repeat(bad.reshape(12, -1, 2).any(axis=-1), 2, axis=1)
    for quantize in (W.quantize_fp4, oracle.quantize_fp4):
        codes, scales = quantize(x, fmt)
        v = oracle.fp4_decode(fmt, codes, scales)
        assert np.array_equal(np.isnan(v).reshape(12, -1, 16).any(axis=-1), bad)
        assert np.array_equal(np.isnan(v).reshape(12, -1, 16).all(axis=-1), bad)
        clean = np.where(np.repeat(bad, 16, axis=1), np.float32(0), x)
        want_codes, want_scales = quantize(clean, fmt)     # the other groups as ever
        at = np.repeat(bad, 8, axis=1)
        assert np.array_equal(codes[~at], want_codes[~at]) and np.all(codes[at] == 0)
        group_bad = bad if fmt == "nvfp4" else bad[:, ::2]
        assert np.array_equal(scales[~group_bad], want_scales[~group_bad])
        assert np.all(scales[group_bad] == (255 if fmt == "mxfp4" else 0x7F))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "mxfp4"])
@pytest.mark.parametrize("n_q", [1, 3, 74, 75, 300])
def test_workspace_of_the_weights_follows_the_selections(L, n_q, fmt):
    """Rows, positions and weights are 12 bytes an entry.  CTAs that share a query make
    a list of rows each only where that is short: 148 lists of 9216 entries at most
    (a query whose tiles are split takes at most as many CTAs as there are SMs)."""
    kv = {"bf16": {}, "e4m3": {"kv_dtype": _abi.SA_E4M3, **FP4, "kv_scale_tokens": 1,
                               "kv_scale_dims": 128},
          "mxfp4": {"kv_dtype": _abi.SA_MXFP4, **FP4}}[fmt]
    c = good_cache(**kv, max_pages=1 << 14, num_pages=1 << 14)
    for k in (64, 2304, 9216, 9217, 100000, 1 << 20):
        q = good_query(n_q=n_q, max_visible=1 << 20)
        need = ws_size(L, c, q, k, _abi.SA_WS_WEIGHTS)
        starts = n_q * (4 + 4 * ((1 << 20) // 256 + 1))
        entries = 12 * n_q * (k + 63)
        assert entries - 12 * n_q * 63 < need <= entries + starts + 148 * 9216 * 4 + 6 * 256
