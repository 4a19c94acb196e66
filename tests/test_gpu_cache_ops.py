"""GPU tests of the 4-bit latent cache, the reading back of rows, the
accumulated attention weights and the eviction, against plain 64-bit forms.

Tolerances are bounds, not observations.  With eps = 2^-24 (fp32 half step; the
tensor cores may truncate, so sums count 2 eps an addition) a logit z = sm *
sum_d q_d k_d of D products is off by at most dz = 2 eps (D + 2) sm sum |q_d k_d|
+ 4 eps |z|.  A weight exp(z - lse) is then off by a factor within exp(+-(dz +
2^-21)) (2^-21: the exponential itself and its argument's rounding).  The
attention output also rounds each weight to bf16 (2^-8, half a step) before the
product with v and itself to the output type.  For the accumulated weights a
value of an e4m3 latent (code times fp32 scale) enters as two bf16: the second
holds what the first left, at most 2^-8 of the value, to half a step, 2^-8, so
at most 2^-16 sm sum |q_d k_d| is missing from a logit.
"""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
from indexed_sparse_attention_lightning_b200 import _abi, api
from indexed_sparse_attention_lightning_b200 import workloads as W
from tests import parity
from tests.test_cache_ops_host import _rows, rows_not_finite

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
OK = (_abi.SA_OK, 0)


def make(kv, lens, seed=3, **kw):
    kw.setdefault("h_index", 8)
    if kv == "f32":
        kw.setdefault("q_dtype", "f32")
    sp = W.WorkloadSpec(name=f"ops_{kv}", seed=seed, batch=len(lens),
                        seq_len=("list", tuple(int(n) for n in lens)), kv_dtype=kv, **kw)
    return W.make_workload(sp)


def values(wl):
    """The latent pool's rows in float64 [pages * 64, d_latent + d_rope]."""
    sp = wl.spec
    n = wl.num_pages * 64
    if sp.kv_dtype in ("f32", "bf16"):
        return oracle.decode(sp.kv_dtype, wl.kv).reshape(n, -1)
    rope = oracle.decode("bf16", wl.kv_rope).reshape(n, -1)
    if sp.kv_dtype == "e4m3":
        st, sd = sp.kv_tile
        sc = np.repeat(np.repeat(wl.kv_scale.astype(np.float64), st, axis=1), sd, axis=2)
        lat = oracle.decode("e4m3", wl.kv).reshape(n, -1) * sc.reshape(n, -1)
    else:
        lat = oracle.fp4_decode(sp.kv_dtype, wl.kv, wl.kv_scale).astype(np.float64).reshape(n, -1)
    return np.concatenate([lat, rope], axis=1)


def q_values(wl):
    return oracle.decode(wl.spec.q_dtype, wl.q)


def row_of(wl, b, pos):
    pos = np.asarray(pos)
    return wl.page_table[b, pos // 64].astype(np.int64) * 64 + pos % 64


def selection(wl, K, seed, holes=False, order="ascending"):
    """[n_q, K] distinct visible positions, -1 padded."""
    rng = np.random.default_rng(seed)
    idx = np.full((wl.n_q, K), -1, dtype=np.int32)
    for t in range(wl.n_q):
        V = int(wl.visible[t])
        s = np.sort(rng.choice(V, size=min(K, V), replace=False))
        if order == "shuffled":
            s = rng.permutation(s)
        idx[t, :s.size] = s
        if holes:
            idx[t, rng.random(K) < 0.2] = -1
    return idx


def upload(wl, idx):
    cache, queries = api.upload(wl)
    return cache, queries, torch.from_numpy(idx).cuda()


def logits(wl, t, sel):
    """(z, bound of its error) [heads, len(sel)] of query t."""
    kv = values(wl)[row_of(wl, int(wl.q_seq[t]), sel)]
    q, sm = q_values(wl)[t], wl.spec.softmax_scale
    z = (q @ kv.T) * sm
    size = (np.abs(q) @ np.abs(kv).T) * abs(sm)
    dz = 2 * EPS * (kv.shape[1] + 2) * size + 4 * EPS * np.abs(z)
    if wl.spec.kv_dtype == "e4m3":
        dz = dz + 2.0 ** -16 * size
    return z, dz, kv


# ------------------------------------------------------- write and read back ---

def _layout(wl):
    sp = wl.spec
    return {"page_table": wl.page_table, "page_size": 64, "num_pages": wl.num_pages,
            "index_dtype": sp.index_dtype, "kv_dtype": sp.kv_dtype, "d_latent": sp.d_latent,
            "kv_scale_dims": sp.kv_tile[1]}


def _pools(wl):
    return {k: getattr(wl, k) for k in ("k_index", "k_index_scale", "kv", "kv_rope", "kv_scale")}


def _device_pools(cache):
    out = {}
    for k in ("k_index", "k_index_scale", "kv", "kv_rope", "kv_scale"):
        t = getattr(cache, k)
        out[k] = None if t is None else t.cpu().numpy()
    return out


def _bytes(a):
    return np.ascontiguousarray(a).view(np.uint8)


def same_bytes(got, want, what=""):
    for k, a in want.items():
        if a is not None:
            assert np.array_equal(_bytes(got[k]), _bytes(a)), f"{what}{k}"


@pytest.mark.parametrize("inp", ["bf16", "f32"])
@pytest.mark.parametrize("dims", [(512, 64), (64, 16), (96, 8)])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_append_and_read_4_bits_exactly(fmt, dims, inp):
    dl, dr = dims
    wl = make(fmt, (200, 1, 1000), d_latent=dl, d_rope=dr, heads=16)
    cache, _ = api.upload(wl)
    rng = np.random.default_rng(11)
    n = 150
    seq = rng.integers(0, 3, n).astype(np.int32)
    pos = np.empty(n, np.int32)
    for b in range(3):
        m = seq == b
        pos[m] = rng.choice(64 * int((wl.page_table[b] >= 0).sum()), m.sum(), replace=False)
    seq[-4:] = [-1, 3, 0, 1]
    pos[-4:] = [0, 0, -1, 64 * wl.max_pages]
    x = np.concatenate([np.resize(_rows(4, n=60, d=dl), (n, dl)),
                        rng.standard_normal((n, dr)).astype(np.float32)], axis=1)
    if inp == "bf16":
        t = torch.from_numpy(x).to(torch.bfloat16)
        x = t.float().numpy()
    else:
        t = torch.from_numpy(x)
    seq_t, pos_t = torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda()
    ws = api.append_tokens(cache, seq_t, pos_t, kv=t.cuda())
    assert api.device_status(ws) == (_abi.SA_ERR_DEVICE_FAULT, _abi.SA_DETAIL_BAD_POSITION)
    want, skipped = oracle.append_tokens(_pools(wl), _layout(wl), seq, pos, None, x)
    assert len(skipped) == 4
    same_bytes(_device_pools(cache), want)

    now = dataclasses.replace(wl, **want)
    rows = values(now)
    for out_dtype in ("bf16", "f32"):
        back, ws = api.read_tokens(cache, seq_t, pos_t, out_dtype=out_dtype)
        assert api.device_status(ws) == (_abi.SA_ERR_DEVICE_FAULT, _abi.SA_DETAIL_BAD_POSITION)
        exp = np.zeros((n, dl + dr))
        for i in range(n - 4):
            exp[i] = rows[row_of(now, seq[i], pos[i])]
        exp = torch.from_numpy(exp).to(back.dtype)
        assert torch.equal(back.cpu(), exp)


@pytest.mark.parametrize("kv,tile", [("f32", (0, 0)), ("bf16", (0, 0)), ("e4m3", (0, 0)),
                                     ("e4m3", (1, 128)), ("nvfp4", (0, 0))])
def test_read_tokens_of_every_pool(kv, tile):
    wl = make(kv, (130, 67), heads=16, kv_scale_tile=tile)
    cache, _ = api.upload(wl)
    seq = np.array([0, 1, 0, 0, 1, 0], np.int32)
    pos = np.array([129, 0, 64, 64, 66, 0], np.int32)     # one of them twice
    out, ws = api.read_tokens(cache, torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda(),
                              out_dtype="f32")
    assert api.device_status(ws) == OK
    exp = np.stack([values(wl)[row_of(wl, b, p)] for b, p in zip(seq, pos)])
    # e4m3 x fp32 scale is one fp32 product: half a step; the others are exact
    assert np.all(np.abs(out.cpu().numpy() - exp) <= EPS * np.abs(exp) * (kv == "e4m3"))
    half, _ = api.read_tokens(cache, torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda())
    assert torch.equal(half, out.to(torch.bfloat16))
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert api.read_tokens(cache, none, none)[0].shape == (0, wl.spec.d_latent + wl.spec.d_rope)


@pytest.mark.parametrize("n", [2048, 2049, 8001])
@pytest.mark.parametrize("inp", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_append_and_read_many_tokens(fmt, inp, n):
    """Several tokens a warp, ragged at the end, with bad ones among them."""
    wl = make(fmt, (2500, 64, 8000), d_latent=64, d_rope=8, heads=16)
    cache, _ = api.upload(wl)
    rng = np.random.default_rng(12)
    every = np.concatenate([[(b, p) for p in range(64 * int((wl.page_table[b] >= 0).sum()))]
                            for b in range(3)])
    pick = every[rng.permutation(len(every))[:n]].astype(np.int32)
    seq, pos = pick[:, 0].copy(), pick[:, 1].copy()
    bad = rng.random(n) < 0.01
    bad[[0, n - 1]] = True
    seq[bad] = 3
    x = np.concatenate([np.resize(_rows(5, n=300, d=64), (n, 64)),
                        rng.standard_normal((n, 8)).astype(np.float32)], axis=1)
    t = torch.from_numpy(x).to(torch.bfloat16 if inp == "bf16" else torch.float32)
    seq_t, pos_t = torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda()
    ws = api.append_tokens(cache, seq_t, pos_t, kv=t.cuda())
    assert api.device_status(ws) == (_abi.SA_ERR_DEVICE_FAULT, _abi.SA_DETAIL_BAD_POSITION)
    want, skipped = oracle.append_tokens(_pools(wl), _layout(wl), seq, pos, None,
                                         t.float().numpy())
    assert len(skipped) == bad.sum()
    same_bytes(_device_pools(cache), want)
    rows = values(dataclasses.replace(wl, **want))
    exp = np.zeros((n, 72))
    for i in np.flatnonzero(~bad):
        exp[i] = rows[row_of(wl, seq[i], pos[i])]
    for out_dtype in ("bf16", "f32"):
        back, ws = api.read_tokens(cache, seq_t, pos_t, out_dtype=out_dtype)
        assert api.device_status(ws) == (_abi.SA_ERR_DEVICE_FAULT, _abi.SA_DETAIL_BAD_POSITION)
        assert torch.equal(back.cpu(), torch.from_numpy(exp).to(back.dtype))


@pytest.mark.parametrize("inp", ["bf16", "f32"])
def test_nvfp4_codes_next_to_every_border(inp):
    """For each scale byte the values on, and next to, each border between two codes,
    and the largest values that take this byte."""
    scales = oracle.fp4_scale_decode("nvfp4", np.arange(1, 127, dtype=np.uint8)).astype(np.float64)
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    step = 2.0 ** -8 if inp == "bf16" else 2.0 ** -24
    dtype = torch.bfloat16 if inp == "bf16" else torch.float32
    near = (borders[:, None] * (1 + step * np.arange(-3, 4))[None]).ravel()
    tops = [(1 + step * k) * 6 for k in range(-4, 5)]
    rows = []
    for i, top in enumerate(tops):
        signs = np.where((np.arange(near.size) + i) % 2, -1.0, 1.0)
        x = (signs * near)[None] * scales[:, None]
        x = np.concatenate([x, np.zeros((x.shape[0], -x.shape[1] % 15))], axis=1)
        g = x.reshape(len(scales), -1, 15)
        lead = np.broadcast_to((top * scales)[:, None, None], g.shape[:2] + (1,))
        rows.append(np.concatenate([lead, g], axis=2).reshape(len(scales), -1))
    x = torch.from_numpy(np.concatenate(rows).astype(np.float32)).to(dtype)  # [n, 64]
    assert x.shape[1] == 64
    n = x.shape[0]
    wl = make("nvfp4", (n,), d_latent=64, d_rope=8, heads=16)
    cache, _ = api.upload(wl)
    x = torch.cat([x, torch.zeros((n, 8), dtype=dtype)], dim=1)
    seq, pos = np.zeros(n, np.int32), np.arange(n, dtype=np.int32)
    ws = api.append_tokens(cache, torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda(),
                           kv=x.cuda())
    assert api.device_status(ws) == OK
    want, _ = oracle.append_tokens(_pools(wl), _layout(wl), seq, pos, None, x.float().numpy())
    same_bytes(_device_pools(cache), want)


def test_status_words_need_no_clearing():
    """A call sets its status whatever the workspace held, on short and on long
    calls, after garbage and after an error."""
    wl = make("mxfp4", (5000, 300), heads=16, d_latent=64, d_rope=8)
    cache, _ = api.upload(wl)
    acc = torch.rand((2, 5000), device="cuda")
    spare = sorted(set(range(wl.num_pages)) - set(wl.page_table.ravel().tolist()))[:2]
    dst = dataclasses.replace(
        cache, page_table=torch.tensor(spare, dtype=torch.int32, device="cuda").reshape(2, 1),
        seq_len=torch.zeros(2, dtype=torch.int32, device="cuda"))
    bad_dst = dataclasses.replace(dst, page_table=dst.page_table + wl.num_pages)
    need = max(api.workspace_size(cache, None, 64, u) for u in (_abi.SA_WS_APPEND,
                                                                 _abi.SA_WS_EVICT))
    ws = api.workspace(need)
    bad_page = (_abi.SA_ERR_DEVICE_FAULT, _abi.SA_DETAIL_BAD_PAGE)
    bad_pos = (_abi.SA_ERR_DEVICE_FAULT, _abi.SA_DETAIL_BAD_POSITION)
    for n in (0, 1, 2048, 2049, 4000):
        seq = torch.zeros(n, dtype=torch.int32, device="cuda")
        pos = torch.arange(n, dtype=torch.int32, device="cuda")
        off = seq.clone()
        off[n // 2:] = 2
        kv = torch.randn((n, 72), device="cuda")
        keys = torch.randn((n, wl.spec.d_index), device="cuda")
        for garbage in (True, False):
            calls = [lambda s: api.append_tokens(cache, s, pos, kv=kv, ws=ws),
                     lambda s: api.read_tokens(cache, s, pos, ws=ws),
                     lambda s: api.append_tokens(cache, s, pos, k_index=keys, kv=kv, ws=ws),
                     lambda s: api.append_tokens(cache, s, pos, k_index=keys, ws=ws)]
            for call in calls:
                for s, want in ((seq, OK), (off, bad_pos if n else OK), (seq, OK)):
                    if garbage:
                        ws.fill_(0xA5)
                    call(s)
                    assert api.device_status(ws) == want
    for d, want in ((dst, OK), (bad_dst, bad_page), (dst, OK)):
        for garbage in (True, False):
            if garbage:
                ws.fill_(0xA5)
            api.evict_tokens(cache, acc, 64, d, 1, 1, ws=ws)
            assert api.device_status(ws) == want


def test_read_tokens_reports_a_bad_page():
    wl = make("mxfp4", (130,), heads=16)
    wl.page_table[0, 1] = wl.num_pages
    cache, _ = api.upload(wl)
    pos = torch.tensor([3, 64, 129], dtype=torch.int32, device="cuda")
    out, ws = api.read_tokens(cache, torch.zeros_like(pos), pos)
    assert api.device_status(ws) == (_abi.SA_ERR_DEVICE_FAULT, _abi.SA_DETAIL_BAD_PAGE)
    assert torch.all(out[1] == 0) and torch.all(torch.isfinite(out.float()))


# ---------------------------------------------------------------- attention ---

def check_attention(wl, idx, out, lse, out_dtype):
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    half = 2.0 ** -8 if out_dtype == "bf16" else EPS
    for t in range(wl.n_q):
        sel = idx[t][idx[t] >= 0]
        if sel.size == 0:
            assert np.all(o[t] == 0) and np.all(l[t] == -np.inf)
            continue
        z, dz, kv = logits(wl, t, sel)
        m = z.max(axis=1, keepdims=True)
        e = np.exp(z - m)
        w = e / e.sum(axis=1, keepdims=True)
        v = kv[:, :wl.spec.d_latent]
        ref = w @ v
        worst = dz.max() + 2.0 ** -21
        # weights off by exp(+-worst) in the numerator and the sum, and rounded to bf16
        room = (np.expm1(2 * worst) + 2.0 ** -8 + 4 * EPS * sel.size) * (w @ np.abs(v))
        assert np.all(np.abs(o[t] - ref) <= room + half * (np.abs(ref) + room) + 1e-30)
        ref_l = (m + np.log(e.sum(axis=1, keepdims=True)))[:, 0]
        assert np.all(np.abs(l[t] - ref_l) <= worst + 2 * EPS * (sel.size + np.abs(ref_l)) + 1e-6)


ATTN = [  # heads, d_latent, d_rope, lengths, K
    (128, 512, 64, (1, 64, 65, 700), 2048),
    (128, 512, 64, (3000, 2047), 1500),
    (128, 512, 64, (500, 1, 129), 1),
    (16, 512, 64, (1, 300), 130),
    (5, 64, 16, (77, 200), 33),
]


@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,dl,dr,lens,K", ATTN)
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_attention_over_4_bits(fmt, heads, dl, dr, lens, K, out_dtype):
    wl = make(fmt, lens, heads=heads, d_latent=dl, d_rope=dr, top_k=K)
    for holes, order in ((False, "ascending"), (True, "shuffled")):
        idx = selection(wl, K, 7, holes, order)
        if holes:
            idx[0] = -1                       # a query with nothing selected
        cache, queries, idx_t = upload(wl, idx)
        ws = api.workspace(api.workspace_size(cache, queries, K, _abi.SA_WS_ATTN))
        out, lse = api.sparse_mla_attn(cache, queries, idx_t, K, out_dtype=out_dtype, ws=ws)
        assert api.device_status(ws) == OK
        check_attention(wl, idx, out, lse, out_dtype)


@pytest.mark.parametrize("sm_scale", [-0.05, 0.0, -0.0, 4.0])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_attention_over_4_bits_with_other_softmax_scales(fmt, sm_scale):
    wl = make(fmt, (900, 65), heads=128, sm_scale=sm_scale)
    idx = selection(wl, 300, 7, holes=True)
    cache, queries, idx_t = upload(wl, idx)
    out, lse = api.sparse_mla_attn(cache, queries, idx_t, 300, out_dtype="f32")
    check_attention(wl, idx, out, lse, "f32")


@pytest.mark.parametrize("fmt", ["mxfp4", "bf16", "e4m3"])
def test_attention_with_many_queries_into_fp32(fmt):
    """No key splits, fp32 output at a 16-byte boundary that is no 32-byte one."""
    wl = make(fmt, (400,), heads=128, queries=("prefill", 300, 100), top_k=130)
    idx = selection(wl, 130, 8)
    cache, queries, idx_t = upload(wl, idx)
    flat = torch.full((100 * 128 * 512 + 8,), 7.0, device="cuda")
    out = flat[4:-4].view(100, 128, 512)
    assert out.data_ptr() % 32 == 16
    got, lse = api.sparse_mla_attn(cache, queries, idx_t, 130, out=out, out_dtype="f32")
    assert torch.all(flat[:4] == 7) and torch.all(flat[-4:] == 7)
    half, _ = api.sparse_mla_attn(cache, queries, idx_t, 130)
    assert torch.equal(half, got.to(torch.bfloat16))
    if fmt != "e4m3":        # its rows are rounded to bf16 before the product
        check_attention(wl, idx, got, lse, "f32")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_attention_over_4_bits_with_many_queries(fmt):
    """More (query, half) pairs than SMs: no key splits."""
    wl = make(fmt, (1400,), heads=128, queries=("prefill", 1300, 100), top_k=700)
    idx = selection(wl, 700, 8)
    cache, queries, idx_t = upload(wl, idx)
    out, lse = api.sparse_mla_attn(cache, queries, idx_t, 700)
    check_attention(wl, idx, out, lse, "bf16")


def test_attention_over_mxfp4_scales_of_every_size():
    """Group scales from 2^-100 to 2^30 within a row: values leave bf16's
    normal range on neither side, and the tiny groups vanish in fp32 sums."""
    wl = make("mxfp4", (200, 90), heads=128, top_k=128)
    rng = np.random.default_rng(4)
    sc = rng.integers(27, 120, wl.kv_scale.shape).astype(np.uint8)
    sc[..., 3] = 130
    wl = dataclasses.replace(wl, kv_scale=sc)
    wl = dataclasses.replace(wl, spec=dataclasses.replace(wl.spec, sm_scale=1e-3))
    idx = selection(wl, 128, 9)
    cache, queries, idx_t = upload(wl, idx)
    out, lse = api.sparse_mla_attn(cache, queries, idx_t, 128, out_dtype="f32")
    check_attention(wl, idx, out, lse, "f32")


@pytest.mark.parametrize("lo,hi", [(4, 40), (120, 137), (130, 150), (127, 200), (0, 252)])
def test_mxfp4_scales_beyond_the_usual(lo, hi):
    """Scales 2^(lo - 127) .. 2^(hi - 128), mixed within rows and between the rows of a
    tile, with logits of order one: values small, on both sides of the one-product
    bound, and far past it (6 x 2^124 is the largest, below fp32's 2^128)."""
    wl = make("mxfp4", (400, 90), heads=128, top_k=200)
    rng = np.random.default_rng(4)
    sc = rng.integers(lo, hi, wl.kv_scale.shape).astype(np.uint8)
    one = rng.random(sc.shape[:2]) < 0.3                     # rows of one small scale
    sc[one] = max(lo, min(hi - 1, 126))
    wl = dataclasses.replace(wl, kv_scale=sc)
    sm = float(np.float32(0.05 * 2.0 ** (127 - max(hi, 120))))
    wl = dataclasses.replace(wl, spec=dataclasses.replace(wl.spec, sm_scale=sm))
    idx = selection(wl, 200, 9)
    cache, queries, idx_t = upload(wl, idx)
    out, lse = api.sparse_mla_attn(cache, queries, idx_t, 200, out_dtype="f32")
    check_attention(wl, idx, out, lse, "f32")
    check_weights(wl, idx, acc=np.zeros((2, 400), np.float32))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_fused_decode_over_4_bits(fmt):
    """sa_decode selects and attends like the oracle, and like its own steps."""
    wl = make(fmt, (1500, 2048, 2049, 6000, 70), h_index=64)
    K = 2048
    cache, queries = api.upload(wl)
    idx = torch.full((wl.n_q, K), -7, dtype=torch.int32, device="cuda")
    ws = api.workspace(api.workspace_size(cache, queries, K, _abi.SA_WS_DECODE))
    out, lse, _ = api.decode(cache, queries, K, idx=idx, ws=ws)
    assert api.device_status(ws) == OK
    sel = idx.cpu().numpy()
    parity.check_topk(sel, oracle.index_scores(wl), wl.visible, K)
    check_attention(wl, sel, out, lse, "bf16")
    out2, lse2 = api.sparse_mla_attn(cache, queries, idx, K)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


# ------------------------------------------------------ accumulated weights ---

def weights_ref(wl, idx, lse, acc, decay):
    """(sums, bound of their error), float64 like acc."""
    ref = acc.astype(np.float64) * decay
    tol = 2 * EPS * np.abs(ref)
    for b, n in enumerate(wl.seq_len):
        ref[b, n:] = acc[b, n:]
        tol[b, n:] = 0
    for t in range(wl.n_q):
        sel = idx[t][idx[t] >= 0]
        if sel.size == 0:
            continue
        b = int(wl.q_seq[t])
        z, dz, _ = logits(wl, t, sel)
        l = lse[t].astype(np.float64)[:, None]
        p = np.where(np.isneginf(l), 0.0, np.exp(z - l))
        np.add.at(ref[b], sel, p.sum(axis=0))
        room = (p * np.expm1(dz + 2.0 ** -21 + 4 * EPS * np.abs(np.where(np.isinf(l), 0, l)))
                ).sum(axis=0) + 2 * EPS * wl.spec.heads * p.sum(axis=0)
        np.add.at(tol[b], sel, room)
    return ref, tol + 2 * EPS * (wl.n_q + 2) * np.abs(ref)


def check_weights(wl, idx, decay=1.0, acc=None, inplace=False, ld=None, lse=None):
    K = idx.shape[1]
    cache, queries, idx_t = upload(wl, idx)
    if lse is None:
        _, lse_t = api.sparse_mla_attn(cache, queries, idx_t, K)
    else:
        lse_t = torch.from_numpy(lse).cuda()
    lse = lse_t.cpu().numpy()
    ld = ld or int(wl.seq_len.max())
    rng = np.random.default_rng(17)
    base = rng.random((len(wl.seq_len), ld)).astype(np.float32) if acc is None else acc
    acc_t = torch.from_numpy(base).cuda()
    out_t = acc_t if inplace else torch.full_like(acc_t, -3.0)
    ws = api.workspace(api.workspace_size(cache, queries, K, _abi.SA_WS_WEIGHTS))
    got = api.accumulate_weights(cache, queries, idx_t, K, lse_t, acc_t, decay=decay, out=out_t,
                                 ws=ws)
    assert got is out_t and api.device_status(ws) == OK
    ref, tol = weights_ref(wl, idx, lse, base, decay)
    out = out_t.double().cpu().numpy()
    for b, n in enumerate(wl.seq_len):
        assert np.all(np.abs(out[b, :n] - ref[b, :n]) <= tol[b, :n])
        assert np.all(out[b, n:] == (base[b, n:] if inplace else -3.0))   # left as it was
    return out_t


WEIGH = [("bf16", (0, 0)), ("e4m3", (1, 128)), ("e4m3", (0, 0)), ("mxfp4", (0, 0)),
         ("nvfp4", (0, 0)), ("f32", (0, 0))]


@pytest.mark.parametrize("kv,tile", WEIGH)
def test_weights_of_a_decode_step(kv, tile):
    wl = make(kv, (1, 64, 700, 1300), heads=128, kv_scale_tile=tile)
    check_weights(wl, selection(wl, 600, 5))
    check_weights(wl, selection(wl, 600, 6, holes=True, order="shuffled"), decay=0.5,
                  inplace=True, ld=1400)


@pytest.mark.parametrize("sm_scale", [-0.05, 0.0])
@pytest.mark.parametrize("kv", ["bf16", "e4m3", "mxfp4"])
def test_weights_with_other_softmax_scales(kv, sm_scale):
    wl = make(kv, (900, 65), heads=128, sm_scale=sm_scale)
    check_weights(wl, selection(wl, 300, 7, holes=True))


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
def test_weights_of_more_queries_than_sms(kv):
    """Every CTA takes all of a query's rows; K of one row, of whole tiles, and odd."""
    wl = make(kv, (400,), heads=128, queries=("prefill", 240, 160))
    for K in (1, 64, 193):
        check_weights(wl, selection(wl, K, 6, order="shuffled" if K == 64 else "ascending"))


@pytest.mark.parametrize("heads", [128, 16])
@pytest.mark.parametrize("kv", ["bf16", "nvfp4", "e4m3"])
def test_weights_of_long_selections(kv, heads):
    """More entries than a CTA's threads look up in one step."""
    wl = make(kv, (5300, 700), heads=heads)
    check_weights(wl, selection(wl, 5000, 6, holes=True))


@pytest.mark.parametrize("kv", ["bf16", "nvfp4", "e4m3"])
def test_weights_of_selections_that_take_many_steps(kv):
    """Longer than the weights kernel looks up itself: a kernel in front does."""
    wl = make(kv, (10500, 9217, 40), heads=128)
    idx = selection(wl, 10000, 6, holes=True)
    idx[1, :300] = idx[1, 300:600]                # repeated entries, and in no order
    check_weights(wl, idx, decay=0.5)
    check_weights(wl, selection(wl, 9217, 7), inplace=True)


@pytest.mark.parametrize("heads,dl,dr", [(1, 64, 16), (7, 96, 8), (20, 512, 64), (130, 32, 0)])
def test_weights_of_other_shapes(heads, dl, dr):
    wl = make("nvfp4", (50, 400), heads=heads, d_latent=dl, d_rope=dr)
    check_weights(wl, selection(wl, 100, 5, holes=True))


@pytest.mark.parametrize("order", ["ascending", "shuffled"])
@pytest.mark.parametrize("kv", ["bf16", "mxfp4"])
def test_weights_of_a_prompts_last_queries(kv, order):
    """Many queries of one sequence meet at the same positions; the result is
    the same bits on every run."""
    wl = make(kv, (5000,), heads=128, queries=("prefill", 4900, 100))
    idx = selection(wl, 300, 6, order=order)
    idx[:, :20] = np.arange(20)[None]            # positions that every query selects
    idx[3] = -1
    first = check_weights(wl, idx, decay=0.9)
    assert torch.equal(first, check_weights(wl, idx, decay=0.9))


def test_weights_of_mixed_queries_and_repeated_entries():
    """Two queries of one sequence, none of another; an entry that occurs twice
    counts twice, next to its twin or not."""
    wl = make("bf16", (300, 200, 100), heads=128)
    wl = dataclasses.replace(wl, q_seq=np.array([2, 0, 2], np.int32),
                             q_pos=np.array([99, 150, 40], np.int32))
    idx = np.full((3, 70), -1, np.int32)
    idx[0, :6] = [5, 5, 7, 90, 90, 99]
    idx[1, :5] = [150, 3, 150, 0, 3]
    idx[2, 64:70] = [40, 5, 0, 1, 2, 3]
    check_weights(wl, idx)


def test_weights_of_one_query_sum_to_the_heads():
    wl = make("mxfp4", (2500, 1), heads=128)
    idx = selection(wl, 2048, 5)
    cache, queries, idx_t = upload(wl, idx)
    _, lse = api.sparse_mla_attn(cache, queries, idx_t, 2048)
    out = api.accumulate_weights(cache, queries, idx_t, 2048, lse, None)
    # lse and the weights see the same logits: what is left are the rounded sums
    assert torch.allclose(out.double().sum(1), torch.full((2,), 128.0, device="cuda",
                                                          dtype=torch.float64), rtol=2e-5, atol=0)
    assert torch.all(out[1, 1:] == 0)


@pytest.mark.parametrize("K", [1, 700])
@pytest.mark.parametrize("heads", [128, 16])
@pytest.mark.parametrize("kv,tile", [("bf16", (0, 0)), ("nvfp4", (0, 0)), ("e4m3", (0, 0)),
                                     ("e4m3", (1, 128))])
def test_weights_of_a_query_against_the_attentions_lse(kv, tile, heads, K):
    """With the attention's own lse a query's weights sum to `heads`.  The tensor-core
    attention rounds an e4m3 value (code times scale) to bf16, 2^-8 of it, and its lse
    belongs to the rounded rows, so there a head's sum is off by a factor within
    exp(+-d), d the largest 2^-8 sm sum |q_d k_d| over the latent dims of its rows.
    Both sides' own errors as in check_attention and weights_ref."""
    wl = make(kv, (2500, 900), heads=heads, kv_scale_tile=tile, sm_scale=0.1)
    idx = selection(wl, K, 5)
    cache, queries, idx_t = upload(wl, idx)
    _, lse = api.sparse_mla_attn(cache, queries, idx_t, K)
    got = api.accumulate_weights(cache, queries, idx_t, K, lse, None).double().sum(1).cpu().numpy()
    l = lse.double().cpu().numpy()
    for t in range(2):
        sel = idx[t][idx[t] >= 0]
        _, dz, kv_rows = logits(wl, t, sel)
        dl = wl.spec.d_latent
        size = (np.abs(q_values(wl)[t][:, :dl]) @ np.abs(kv_rows[:, :dl]).T) * 0.1
        d = 2.0 ** -8 * size.max(axis=1) if kv == "e4m3" and heads == 128 else 0.0
        own = dz.max(axis=1) + 2.0 ** -21 + 2 * EPS * (sel.size + np.abs(l[t])) + 1e-6   # the lse's
        own = own + dz.max(axis=1) + 2.0 ** -21 + 4 * EPS * np.abs(l[t])         # the weights'
        room = np.expm1(d + own).sum() + 4 * EPS * heads * heads
        assert abs(got[t] - heads) <= room


def test_weights_with_infinite_lse_and_no_queries():
    wl = make("bf16", (128, 128), heads=128)
    idx = selection(wl, 40, 3)
    lse = np.full((2, 128), 2.0, np.float32)
    lse[0, ::2] = -np.inf
    lse[1] = np.inf
    out = check_weights(wl, idx, acc=np.zeros((2, 128), np.float32), lse=lse)
    assert torch.all(out[1] == 0)
    cache, _ = api.upload(wl)
    queries = api.DeviceQueries(
        q_seq=torch.empty(0, dtype=torch.int32, device="cuda"),
        q_pos=torch.empty(0, dtype=torch.int32, device="cuda"), max_visible=0, q_index=None,
        q_index_scale=None, w=None, h_index=8, q_dtype="bf16",
        q=torch.empty((0, 128, 576), dtype=torch.bfloat16, device="cuda"), heads=128, sm_scale=1.0)
    acc = torch.rand((2, 128), device="cuda")
    got = api.accumulate_weights(cache, queries, torch.empty((0, 5), dtype=torch.int32,
                                                             device="cuda"), 5,
                                 torch.empty((0, 128), device="cuda"), acc, decay=0.25,
                                 out=torch.zeros_like(acc))
    assert torch.equal(got, acc * 0.25)


def test_weights_report_bad_data_and_skip_it():
    wl = make("bf16", (300, 200), heads=128)
    idx = selection(wl, 40, 3)
    idx[0, 39] = 300                                            # past the query
    cache, queries, idx_t = upload(wl, idx)
    lse = torch.full((2, 128), 3.0, device="cuda")
    ws = api.workspace(api.workspace_size(cache, queries, 40, _abi.SA_WS_WEIGHTS))
    got = api.accumulate_weights(cache, queries, idx_t, 40, lse, None, ws=ws)
    assert api.device_status(ws) == (_abi.SA_ERR_DEVICE_FAULT, _abi.SA_DETAIL_BAD_INDEX)
    idx[0, 39] = -1
    assert torch.equal(got, api.accumulate_weights(cache, queries, torch.from_numpy(idx).cuda(),
                                                   40, lse, None))
    # a sequence longer than the sums' rows is written up to their end
    long = make("bf16", (300, 200), heads=128)
    long = dataclasses.replace(long, q_seq=np.array([1], np.int32), q_pos=np.array([199], np.int32),
                               q=long.q[1:], w=long.w[1:], q_index=long.q_index[1:],
                               q_index_scale=long.q_index_scale[1:])
    cache, queries, idx_t = upload(long, idx[1:])
    buf = torch.full((4, 256), 5.0, device="cuda")
    ws = api.workspace(api.workspace_size(cache, queries, 40, _abi.SA_WS_WEIGHTS))
    api.accumulate_weights(cache, queries, idx_t, 40, lse[1:], buf[1:3], out=buf[1:3], decay=0.0,
                           ws=ws)
    assert api.device_status(ws) == (_abi.SA_ERR_DEVICE_FAULT, _abi.SA_DETAIL_BAD_POSITION)
    assert torch.all(buf[0] == 5) and torch.all(buf[3] == 5) and torch.all(buf[1] == 0)
    assert torch.all(buf[2, 200:] == 5) and torch.equal(buf[2, :200], got[1, :200])


# ------------------------------------------------------------------- evict ---

def keep_ref(n, acc, budget, first, last):
    if n <= budget:
        return np.arange(n)
    mid = np.arange(first, n - last)
    a = np.where(np.isnan(acc[mid]), np.inf, acc[mid].astype(np.float64))
    isnan = np.isnan(acc[mid])
    order = np.lexsort((mid, -a, ~isnan))        # NaN first, then by value, ties by position
    best = mid[order[:budget - first - last]]
    return np.sort(np.concatenate([np.arange(first), best, np.arange(n - last, n)]))


def evict_case(wl, acc, budget, first, last, spare=1, ld_extra=3):
    """Run an eviction into fresh pages of the same pools and check everything."""
    B = len(wl.seq_len)
    per = -(-budget // 64)
    rng = np.random.default_rng(2)
    fresh = rng.permutation(B * per).astype(np.int32).reshape(B, per) + wl.num_pages
    dst_table = np.full((B, per + spare), -1, np.int32)
    dst_table[:, :per] = fresh
    total = wl.num_pages + B * per
    grown = {}
    for k, a in _pools(wl).items():
        if a is not None:
            pad = np.full((B * per,) + a.shape[1:], 7, dtype=a.dtype)
            grown[k] = np.concatenate([a, pad])
    big = dataclasses.replace(wl, num_pages=total, **grown)
    cache, _ = api.upload(big)
    dst = dataclasses.replace(
        cache, page_table=torch.from_numpy(dst_table).cuda(),
        seq_len=torch.full((B,), -9, dtype=torch.int32, device="cuda"))
    acc_out = torch.full((B, budget + ld_extra), 9.0, device="cuda")
    ws = api.workspace(api.workspace_size(cache, None, budget, _abi.SA_WS_EVICT))
    src_pos = api.evict_tokens(cache, torch.from_numpy(acc).cuda(), budget, dst,
                               keep_first=first, keep_last=last, acc_out=acc_out, ws=ws)
    assert api.device_status(ws) == OK
    want = {k: v.copy() for k, v in grown.items()}
    pos = src_pos.cpu().numpy()
    lens = dst.seq_len.cpu().numpy()
    sums = acc_out.cpu().numpy()
    for b in range(B):
        keep = keep_ref(int(wl.seq_len[b]), acc[b], budget, first, last)
        assert lens[b] == keep.size
        assert np.array_equal(pos[b, :keep.size], keep) and np.all(pos[b, keep.size:] == -1)
        assert np.array_equal(sums[b, :keep.size], acc[b, keep], equal_nan=True)
        assert np.all(sums[b, keep.size:] == 0)
        i = np.arange(keep.size)
        to = dst_table[b, i // 64].astype(np.int64) * 64 + i % 64
        for v in want.values():
            flat = v.reshape((total * 64,) + v.shape[2:])
            flat[to] = flat[row_of(wl, b, keep)]
    # every byte of every pool: the kept rows moved, all others as they were
    same_bytes(_device_pools(cache), want)
    assert np.array_equal(cache.seq_len.cpu().numpy(), wl.seq_len)
    return big, dst, pos


EVICT = [("bf16", "e4m3", {}), ("f32", "f32", {}), ("e4m3", "e4m3", {"kv_scale_tile": (1, 128)}),
         ("e4m3", "bf16", {"kv_scale_tile": (1, 16)}), ("mxfp4", "mxfp8", {}),
         ("nvfp4", "e4m3", {}), ("nvfp4", "mxfp8", {"d_latent": 96, "d_rope": 8, "d_index": 32}),
         ("bf16", "bf16", {"d_latent": 33, "d_rope": 6, "d_index": 16})]


@pytest.mark.parametrize("kv,index,kw", EVICT, ids=[f"{a}-{b}-{i}" for i, (a, b, _) in
                                                     enumerate(EVICT)])
def test_evict_moves_the_right_rows(kv, index, kw):
    wl = make(kv, (1, 100, 128, 129, 1000, 2500), heads=16, index_dtype=index, **kw)
    rng = np.random.default_rng(5)
    acc = rng.standard_normal((6, 2500)).astype(np.float32)
    acc[:, rng.random(2500) < 0.6] = 0.0                    # ties
    evict_case(wl, acc, 128, 3, 40)


def test_evict_scales_that_start_at_any_float():
    """Four fp32 scales a row, their pools 4 bytes off a 16-byte boundary."""
    wl = make("e4m3", (400, 90), heads=16, kv_scale_tile=(1, 128))
    acc = np.random.default_rng(9).random((2, 400)).astype(np.float32)
    cache, _ = api.upload(wl)
    flat = torch.empty(cache.kv_scale.numel() + 1, device="cuda")
    odd = flat[1:].view(cache.kv_scale.shape)
    odd.copy_(cache.kv_scale)
    assert odd.data_ptr() % 16 == 4
    out = torch.zeros_like(flat)[1:].view(odd.shape)
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda").reshape(2, 2)
    dst = dataclasses.replace(cache, page_table=table, seq_len=lens,
                              k_index=torch.zeros_like(cache.k_index),
                              k_index_scale=torch.zeros_like(cache.k_index_scale),
                              kv=torch.zeros_like(cache.kv),
                              kv_rope=torch.zeros_like(cache.kv_rope), kv_scale=out)
    api.evict_tokens(dataclasses.replace(cache, kv_scale=odd), torch.from_numpy(acc).cuda(), 100,
                     dst, 1, 10)
    assert lens.tolist() == [100, 90]
    rows = out.view(-1, 4).cpu().numpy()
    scales = wl.kv_scale.reshape(-1, 4)
    for b, keep in enumerate((keep_ref(400, acc[0], 100, 1, 10), np.arange(90))):
        assert np.array_equal(rows[128 * b:128 * b + keep.size], scales[row_of(wl, b, keep)])


@pytest.mark.parametrize("budget,first,last", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (64, 32, 32),
                                               (65, 0, 0), (200, 200, 0), (999, 10, 10),
                                               (1000, 0, 5), (4000, 7, 9), (1500, 0, 0)])
def test_evict_budgets(budget, first, last):
    wl = make("mxfp4", (1000, 3000, 64, 4100), heads=16)
    acc = np.random.default_rng(6).random((4, 4100)).astype(np.float32)
    evict_case(wl, acc, budget, first, last)


def test_evict_special_sums():
    """Equal sums everywhere, infinities, NaN, signed zeros, lowest values."""
    wl = make("nvfp4", (500, 500, 500, 500, 500), heads=16)
    acc = np.zeros((5, 500), np.float32)
    acc[1, 100:110] = np.inf
    acc[1, 300:] = -np.inf
    acc[2, 50::7] = np.nan
    acc[2, 60] = -np.nan
    acc[2, 61] = np.inf
    acc[3, ::2] = -0.0
    acc[4] = np.finfo(np.float32).min
    acc[4, 400:] = np.float32(1e-45)
    evict_case(wl, acc, 130, 2, 5)


def test_evict_long_sequences():
    wl = make("mxfp4", (70001, 33000), heads=16, d_latent=64, d_rope=8)
    rng = np.random.default_rng(8)
    acc = np.exp(rng.standard_normal((2, 70001))).astype(np.float32)
    acc[rng.random(acc.shape) < 0.7] = 0
    evict_case(wl, acc, 9001, 64, 1000)


@pytest.mark.parametrize("lens,width", [((5000, 900), 16 * 48 * 1024 + 128),
                                        ((9, 50000) + 78 * (150,), 50000)])
def test_evict_without_keys_in_shared_memory(lens, width):
    """Rows of sums too wide for the shared memory of a sequence's CTAs: sixteen of
    them for two sequences, one for eighty."""
    wl = make("mxfp4", lens, heads=16, d_latent=64, d_rope=8, d_index=32)
    pages = -(-width // 64)
    table = np.full((len(lens), pages), -1, np.int32)
    table[:, :wl.max_pages] = wl.page_table
    wl = dataclasses.replace(wl, page_table=table)
    acc = np.random.default_rng(8).standard_normal((len(lens), width)).astype(np.float32)
    acc[:, ::3] = 0
    evict_case(wl, acc, 130, 4, 30)


def test_evict_short_sequences_may_keep_their_pages():
    wl = make("bf16", (90, 400, 100), heads=16)
    acc = np.random.default_rng(9).random((3, 400)).astype(np.float32)
    cache, _ = api.upload(wl)
    table = np.full((3, 2), -1, np.int32)
    table[0], table[2] = wl.page_table[0, :2], wl.page_table[2, :2]
    spare = [p for p in range(wl.num_pages) if p not in set(wl.page_table.ravel())]
    table[1] = spare[:2]
    dst = dataclasses.replace(cache, page_table=torch.from_numpy(table).cuda(),
                              seq_len=torch.zeros(3, dtype=torch.int32, device="cuda"))
    before = _device_pools(cache)
    src_pos = api.evict_tokens(cache, torch.from_numpy(acc).cuda(), 100, dst, 1, 10)
    assert dst.seq_len.tolist() == [90, 100, 100]
    keep = keep_ref(400, acc[1], 100, 1, 10)
    assert np.array_equal(src_pos.cpu().numpy()[1], keep)
    for k, a in before.items():
        if a is not None:
            flat = a.reshape((-1,) + a.shape[2:])
            i = np.arange(100)
            flat[table[1, i // 64].astype(np.int64) * 64 + i % 64] = flat[row_of(wl, 1, keep)]
    same_bytes(_device_pools(cache), before)


@pytest.mark.parametrize("what", ["src_page", "dst_page", "length", "negative", "sums"])
def test_evict_skips_a_bad_sequence_whole(what):
    wl = make("bf16", (300, 400, 200), heads=16)
    acc = np.random.default_rng(9).random((3, 400)).astype(np.float32)
    per = 2
    table = np.arange(3 * per, dtype=np.int32).reshape(3, per) + wl.num_pages
    grown = {k: None if a is None else np.concatenate(
        [a, np.full((3 * per,) + a.shape[1:], 7, a.dtype)]) for k, a in _pools(wl).items()}
    lens = wl.seq_len.copy()
    pt = wl.page_table.copy()
    detail = _abi.SA_DETAIL_BAD_POSITION
    if what == "src_page":
        pt[1, 3], detail = -1, _abi.SA_DETAIL_BAD_PAGE
    elif what == "dst_page":
        table[1, 1], detail = wl.num_pages + 6, _abi.SA_DETAIL_BAD_PAGE
    elif what == "length":
        lens[1] = 64 * pt.shape[1] + 1
    elif what == "negative":
        lens[1] = -1
    elif what == "sums":
        acc = np.ascontiguousarray(acc[:, :399])
    big = dataclasses.replace(wl, num_pages=wl.num_pages + 6, seq_len=lens, page_table=pt, **grown)
    cache, _ = api.upload(big)
    dst = dataclasses.replace(cache, page_table=torch.from_numpy(table).cuda(),
                              seq_len=torch.full((3,), 5, dtype=torch.int32, device="cuda"))
    acc_out = torch.full((3, 128), 4.0, device="cuda")
    ws = api.workspace(api.workspace_size(cache, None, 100, _abi.SA_WS_EVICT))
    src_pos = api.evict_tokens(cache, torch.from_numpy(acc).cuda(), 100, dst, 4, 8,
                               acc_out=acc_out, ws=ws)
    assert api.device_status(ws) == (_abi.SA_ERR_DEVICE_FAULT, detail)
    assert dst.seq_len.tolist() == [100, 0, 100]
    assert torch.all(src_pos[1] == -1) and torch.all(acc_out[1] == 0)
    got = _device_pools(cache)
    want = {k: None if a is None else a.copy() for k, a in grown.items()}
    for b in (0, 2):
        keep = keep_ref(int(lens[b]), acc[b], 100, 4, 8)
        assert np.array_equal(src_pos[b].cpu().numpy(), keep)
        i = np.arange(100)
        for a in want.values():
            if a is not None:
                flat = a.reshape((-1,) + a.shape[2:])
                flat[table[b, i // 64].astype(np.int64) * 64 + i % 64] = flat[row_of(wl, b, keep)]
    same_bytes(got, want)


# ------------------------------------------------------------ used together ---

@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_a_long_sequence_written_read_weighed_and_shrunk(fmt):
    """A prompt enters a 4-bit cache, two decode steps attend to it and add up
    their weights, the cache shrinks, and a step over the shrunk cache sees
    exactly the kept tokens."""
    K, budget, first, last = 256, 320, 8, 64
    lens = np.array([1000, 300, 1500])
    wl = make(fmt, lens, h_index=64, heads=128, top_k=K)
    rng = np.random.default_rng(21)
    # the prompt's rows through the library instead of the generator's
    seq = np.repeat(np.arange(3), lens).astype(np.int32)
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    x = torch.from_numpy(rng.standard_normal((seq.size, 576)).astype(np.float32)).bfloat16()
    cache, queries = api.upload(wl)
    api.append_tokens(cache, torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda(),
                      kv=x.cuda())
    pools, _ = oracle.append_tokens(_pools(wl), _layout(wl), seq, pos, None, x.float().numpy())
    wl = dataclasses.replace(wl, **pools)
    same_bytes(_device_pools(cache), pools)

    acc = torch.zeros((3, 1500), device="cuda")
    ref, tol = np.zeros((3, 1500)), np.zeros((3, 1500))
    for step in range(2):
        idx = torch.empty((3, K), dtype=torch.int32, device="cuda")
        _, lse, _ = api.decode(cache, queries, K, idx=idx)
        api.accumulate_weights(cache, queries, idx, K, lse, acc)
        sel = idx.cpu().numpy()
        r, e = weights_ref(wl, sel, lse.cpu().numpy(), ref.astype(np.float32), 1.0)
        ref, tol = r, tol + e
    sums = acc.cpu().numpy()
    assert np.all(np.abs(sums - ref) <= tol + 1e-6 * ref)

    big, dst, kept = evict_case(wl, sums, budget, first, last)
    small = dataclasses.replace(
        big, page_table=dst.page_table.cpu().numpy(), seq_len=dst.seq_len.cpu().numpy(),
        q_pos=(dst.seq_len.cpu().numpy() - 1).astype(np.int32), **{
            k: v for k, v in _device_pools(dst).items() if v is not None})
    small = dataclasses.replace(small, kv_rope=small.kv_rope.view(np.uint16))
    queries.q_pos = torch.from_numpy(small.q_pos).cuda()
    queries.max_visible = int(small.q_pos.max()) + 1
    idx = torch.empty((3, K), dtype=torch.int32, device="cuda")
    out, lse, _ = api.decode(dst, queries, K, idx=idx)
    sel = idx.cpu().numpy()
    parity.check_topk(sel, oracle.index_scores(small), small.visible, K)
    check_attention(small, sel, out, lse, "bf16")
    # position i of the shrunk cache is the kept token's old row
    full = values(wl)
    for b in range(3):
        n = int(small.seq_len[b])
        assert np.array_equal(values(small)[row_of(small, b, np.arange(n))],
                              full[row_of(wl, b, kept[b, :n])])


def test_captured_and_replayed_on_another_stream():
    """One graph of the whole chain, replayed after its inputs changed in place,
    gives the eager calls' results; two graphs with workspaces of their own may
    be replayed at once."""
    K, budget = 200, 128
    wl = make("nvfp4", (900, 400), h_index=64, heads=128, top_k=K)
    per = budget // 64
    grown = {k: None if a is None else np.concatenate(
        [a, np.full((4 * per,) + a.shape[1:], 7, a.dtype)]) for k, a in _pools(wl).items()}
    big = dataclasses.replace(wl, num_pages=wl.num_pages + 4 * per, **grown)
    cache, queries = api.upload(big)
    seq = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    pos = torch.tensor([899, 399], dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    new = torch.randn(2, 576, device="cuda", generator=gen).bfloat16()

    def buffers(k):
        table = np.arange(2 * per, dtype=np.int32).reshape(2, per) + wl.num_pages + 2 * per * k
        dst = dataclasses.replace(cache, page_table=torch.from_numpy(table).cuda(),
                                  seq_len=torch.zeros(2, dtype=torch.int32, device="cuda"))
        f = dict(device="cuda")
        uses = ((queries, K, _abi.SA_WS_DECODE), (queries, K, _abi.SA_WS_WEIGHTS),
                (None, budget, _abi.SA_WS_EVICT), (None, 0, _abi.SA_WS_APPEND))
        return dict(dst=dst, acc=torch.zeros((2, 900), **f), acc_out=torch.zeros((2, budget), **f),
                    out=torch.empty((2, 128, 512), dtype=torch.bfloat16, **f),
                    lse=torch.empty((2, 128), **f),
                    idx=torch.empty((2, K), dtype=torch.int32, **f),
                    src_pos=torch.empty((2, budget), dtype=torch.int32, **f),
                    back=torch.empty((2, 576), dtype=torch.bfloat16, **f),
                    ws=[api.workspace(api.workspace_size(cache, q, n, u)) for q, n, u in uses])

    def chain(m):
        api.append_tokens(cache, seq, pos, kv=new, ws=m["ws"][3])
        api.read_tokens(cache, seq, pos, out=m["back"], ws=m["ws"][3])
        api.decode(cache, queries, K, out=m["out"], lse=m["lse"], idx=m["idx"], ws=m["ws"][0])
        api.accumulate_weights(cache, queries, m["idx"], K, m["lse"], None, out=m["acc"],
                               ws=m["ws"][1])
        api.evict_tokens(cache, m["acc"], budget, m["dst"], 2, 30, acc_out=m["acc_out"],
                         src_pos=m["src_pos"], ws=m["ws"][2])

    def results(m):
        torch.cuda.synchronize()
        keys = ("acc", "acc_out", "out", "lse", "idx", "src_pos", "back")
        return {**{k: m[k].clone() for k in keys}, "len": m["dst"].seq_len.clone(),
                "kv": cache.kv[m["dst"].page_table.long()].clone(),
                "scale": cache.kv_scale[m["dst"].page_table.long()].clone()}

    def same(a, b):
        for k in a:
            assert torch.equal(a[k], b[k]), k

    a, b = buffers(0), buffers(1)
    graphs, side = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for m, st in zip((a, b), side):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            chain(m)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            chain(m)
        graphs.append(g)
    want = buffers(0)
    for seed in (5, 6):
        gen.manual_seed(seed)
        new.copy_(torch.randn(2, 576, device="cuda", generator=gen).bfloat16())
        queries.q.copy_(torch.randn(2, 128, 576, device="cuda", generator=gen).bfloat16()
                        .view(torch.int16))
        torch.cuda.synchronize()
        for g, st in zip(graphs, side):
            with torch.cuda.stream(st):
                g.replay()
        got = [results(a), results(b)]
        chain(want)
        ref = results(want)
        same(got[0], ref)
        same(got[1], ref)
    del graphs


def test_binding_refuses_what_the_library_would_misread():
    wl = make("mxfp4", (200, 100), heads=128)
    idx = selection(wl, 50, 3)
    cache, queries, idx_t = upload(wl, idx)
    lse = torch.zeros((2, 128), device="cuda")
    acc = torch.zeros((2, 256), device="cuda")
    dst = dataclasses.replace(cache, seq_len=torch.zeros(2, dtype=torch.int32, device="cuda"))

    def refused(f, *a, **k):
        with pytest.raises(api.SaError):
            f(*a, **k)

    refused(api.accumulate_weights, cache, queries, idx_t, 50, lse, acc[:, :200])    # strided
    refused(api.accumulate_weights, cache, queries, idx_t, 50, lse, acc[:, :100].contiguous())
    refused(api.accumulate_weights, cache, queries, idx_t, 50, lse, acc.double())
    refused(api.accumulate_weights, cache, queries, idx_t, 50, lse.cpu(), acc)
    refused(api.accumulate_weights, cache, queries, idx_t.long(), 50, lse, acc)
    refused(api.accumulate_weights, cache, queries, idx_t, 50, lse, acc, out=acc[:1])
    refused(api.accumulate_weights, cache, queries, idx_t, 50, lse, acc, decay=float("nan"))
    refused(api.evict_tokens, cache, acc, 64, cache)                 # the same lengths
    refused(api.evict_tokens, cache, acc, 64, dst, 40, 40)
    refused(api.evict_tokens, cache, acc[:1], 64, dst)
    refused(api.evict_tokens, cache, acc.t(), 64, dst)
    refused(api.evict_tokens, cache, acc, 64, dst, acc_out=acc)
    refused(api.evict_tokens, cache, acc, 64, dst, acc_out=torch.zeros((2, 63), device="cuda"))
    refused(api.evict_tokens, cache, acc, 0, dst)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    refused(api.read_tokens, cache, pos, pos.long())
    refused(api.read_tokens, cache, pos, pos, out=torch.zeros((2, 576), device="cuda",
                                                              dtype=torch.float16))
    refused(api.read_tokens, cache, pos, pos[:1])


# ------------------------------------------------- values that are not finite ---

@pytest.mark.parametrize("inp", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_values_that_are_not_finite_stay_visible(fmt, inp):
    wl = make(fmt, (12, 12), d_latent=64, d_rope=8, heads=16)
    cache, _ = api.upload(wl)
    x = torch.from_numpy(np.concatenate([rows_not_finite()[0], np.ones((12, 8), np.float32)],
                                        axis=1))
    x = x.to(torch.bfloat16 if inp == "bf16" else torch.float32)
    seq, pos = np.zeros(12, np.int32), np.arange(12, dtype=np.int32)
    seq_t, pos_t = torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda()
    ws = api.append_tokens(cache, seq_t, pos_t, kv=x.cuda())
    assert api.device_status(ws) == OK
    want, _ = oracle.append_tokens(_pools(wl), _layout(wl), seq, pos, None, x.float().numpy())
    same_bytes(_device_pools(cache), want)
    rows = values(dataclasses.replace(wl, **want))[row_of(wl, 0, pos)]
    assert np.isnan(rows).any() and not np.isnan(rows).all(axis=1).any()
    for out_dtype in ("bf16", "f32"):
        back, _ = api.read_tokens(cache, seq_t, pos_t, out_dtype=out_dtype)
        exp = torch.from_numpy(rows).to(back.dtype)
        assert torch.equal(torch.isnan(back.cpu()), torch.isnan(exp))
        assert torch.equal(torch.nan_to_num(back.cpu()), torch.nan_to_num(exp))


@pytest.mark.parametrize("inp", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_a_poisoned_token_poisons_the_attention_that_selects_it(fmt, inp):
    wl = make(fmt, (70, 70), heads=128)
    idx = selection(wl, 70, 4)
    cache, queries, idx_t = upload(wl, idx)
    before, _ = api.sparse_mla_attn(cache, queries, idx_t, 70)
    x = torch.ones((1, 576), dtype=torch.bfloat16 if inp == "bf16" else torch.float32,
                   device="cuda")
    x[0, 77] = float("nan")
    at = torch.tensor([1], dtype=torch.int32, device="cuda")
    api.append_tokens(cache, at, at + 65, kv=x)
    out, _ = api.sparse_mla_attn(cache, queries, idx_t, 70)
    assert torch.isnan(out[1]).all() and torch.equal(out[0], before[0])
    idx_t[1][idx_t[1] == 66] = -1                          # not selected: not seen
    out, _ = api.sparse_mla_attn(cache, queries, idx_t, 70)
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("log2_t", [-4, 2])
def test_a_tensor_scale_is_folded_into_query_and_output(log2_t):
    """NVFP4 rows of another size: the latent is appended times 1 / T, the query's
    latent dims and the output are multiplied by T.  T is a power of two and the e4m3
    scales stay normal (amax / 6 of 16 values N(0, 1) lies above 2^-4), so every step
    is the same but for exponents."""
    wl = make("nvfp4", (300, 200), heads=128)
    idx = selection(wl, 120, 5)
    cache, queries, idx_t = upload(wl, idx)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    x = torch.randn((500, 576), device="cuda", generator=gen).bfloat16()
    seq = torch.tensor([0] * 300 + [1] * 200, dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(300), torch.arange(200)]).int().cuda()
    t = 2.0 ** log2_t
    got = []
    for stored, query, back in ((1.0, 1.0, 1.0), (1.0, 1.0, 1.0), (t, 1.0, 1.0), (t, t, t)):
        kv, q = x.clone(), queries.q.view(torch.bfloat16).clone()
        kv[:, :512] /= stored                       # times 1 / T and back: both exact
        q[..., :512] *= query
        api.append_tokens(cache, seq, pos, kv=kv)
        mine = dataclasses.replace(queries, q=q)
        out, lse = api.sparse_mla_attn(cache, mine, idx_t, 120)
        sums = api.accumulate_weights(cache, mine, idx_t, 120, lse, None)
        rows, _ = api.read_tokens(cache, seq, pos)
        rows[:, :512] *= back
        got.append((out * back, lse, sums, rows))
    for a, b in zip(got[0], got[1]):
        assert torch.equal(a, b)
    for a, b in zip(got[0], got[3]):
        assert torch.equal(a, b)
    assert not torch.equal(got[0][1], got[2][1])
