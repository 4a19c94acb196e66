"""What a long-lived cache needs, as cases that can be measured: four operators.

* ``attend`` -- sparse MLA attention over selected rows of a latent cache held
  in 4 bits (``mxfp4``: e2m1 codes, one E8M0 scale per 32 dims; ``nvfp4``: e2m1
  codes, one e4m3 scale per 16 dims; the rope stays bf16);
* ``write``  -- new rows quantised into such a cache, and read back from it as
  the values it then stands for;
* ``weigh``  -- the attention weight that every selected position received,
  summed over the heads and queries and added to each sequence's running sums;
* ``evict``  -- per sequence the first and the last tokens and, between them,
  those of the largest accumulated weight, moved in order to fresh pages.

``run`` computes each in its plain form (elementary torch operations in 32
bits) or, with ``own``, through the library's entry points.  ``exact`` computes
the floating outputs in 64 bits from the definitions.
"""
import math

import numpy as np
import torch

own = False

PAGE, DL, DR, HEADS, DI = 64, 512, 64, 128, 128
D = DL + DR
SM_SCALE = 1.0 / math.sqrt(D)
GROUP = {"mxfp4": 32, "nvfp4": 16}


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # one decode step of a loaded server: 64 sequences, 16-32K tokens each
        dict(name="attend_mxfp4_b64_32k", op="attend", kv="mxfp4", mode="decode", n_q=64,
             lo=16384, hi=32768, top_k=2048, holes=False),
        # two very long sequences: few rows of a large cache, so the keys are split
        dict(name="attend_nvfp4_b2_256k", op="attend", kv="nvfp4", mode="decode", n_q=2,
             lo=262144, hi=262144, top_k=2048, holes=False),
        # a chunk of a prompt: consecutive queries of one sequence
        dict(name="attend_nvfp4_chunk512", op="attend", kv="nvfp4", mode="chunk", n_q=512,
             lo=32768, hi=32768, top_k=2048, holes=False),
        # a few short conversations, one of them with nothing selected: latency
        dict(name="attend_mxfp4_b3_short", op="attend", kv="mxfp4", mode="decode", n_q=3,
             lo=1, hi=777, top_k=500, holes=True),
        # the new tokens of one decode step
        dict(name="write_mxfp4_step64", op="write", kv="mxfp4", n=64, seqs=64, inp="bf16"),
        # prompts entering the cache, packed, of different lengths
        dict(name="write_nvfp4_prompt40k", op="write", kv="nvfp4", n=40001, seqs=7, inp="bf16"),
        # the weights of one decode step over the ordinary bf16 cache
        dict(name="weigh_bf16_b64_32k", op="weigh", kv="bf16", mode="decode", n_q=64,
             lo=16384, hi=32768, top_k=2048, decay=1.0, holes=False),
        # the last queries of a prompt, whose weights decide what is kept of it
        dict(name="weigh_mxfp4_window256", op="weigh", kv="mxfp4", mode="chunk", n_q=256,
             lo=30000, hi=30000, top_k=2048, decay=1.0, holes=False),
        # a few sequences in an e4m3 cache, older weights fading: latency
        dict(name="weigh_e4m3_b3", op="weigh", kv="e4m3", mode="decode", n_q=3,
             lo=1500, hi=5000, top_k=1000, decay=0.97, holes=True),
        # a full server shrinks every sequence to 4096 tokens
        dict(name="evict_bf16_b64_4k", op="evict", kv="bf16", batch=64, lo=16384, hi=32768,
             budget=4096, first=4, last=512),
        # two long documents to an eighth of their tokens, 4-bit cache
        dict(name="evict_mxfp4_b2_256k", op="evict", kv="mxfp4", batch=2, lo=262144, hi=262144,
             budget=32768, first=64, last=4096),
        # short conversations, some of them under the budget already: latency
        dict(name="evict_nvfp4_b5_short", op="evict", kv="nvfp4", batch=5, lo=300, hi=2500,
             budget=601, first=1, last=100),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "write", "weigh", "weigh", "evict"])
    if op in ("attend", "weigh"):
        mode = rng.choice(["decode", "chunk"])
        kvs = ["mxfp4", "nvfp4"] if op == "attend" else ["mxfp4", "nvfp4", "bf16", "e4m3"]
        n_q = _log(rng, 1, 64) if mode == "decode" else _log(rng, 2, 400)
        hi = _log(rng, 50, 32768)
        if mode == "chunk":
            hi = max(hi, n_q)
        c = dict(op=op, kv=rng.choice(kvs), mode=mode, n_q=n_q,
                 lo=hi if mode == "chunk" else rng.randint(1, hi), hi=hi,
                 top_k=_log(rng, 1, 2048), holes=rng.random() < 0.4)
        if op == "weigh":
            c["decay"] = rng.choice([0.0, 1.0, round(rng.uniform(0.5, 1.0), 3)])
        return c
    if op == "write":
        n = _log(rng, 1, 40000)
        return dict(op=op, kv=rng.choice(["mxfp4", "nvfp4"]), n=n, seqs=rng.randint(1, min(n, 70)),
                    inp=rng.choice(["bf16", "f32"]))
    batch, hi = _log(rng, 1, 48), _log(rng, 100, 32768)
    budget = max(2, int(hi * rng.uniform(0.05, 0.7)))
    budget = min(budget, 4096 * 48 // batch, 32768)
    first = rng.randint(0, budget // 4)
    return dict(op=op, kv=rng.choice(["mxfp4", "nvfp4", "bf16", "e4m3"]), batch=batch,
                lo=rng.randint(1, hi), hi=hi, budget=budget, first=first,
                last=rng.randint(0, budget // 2))


# ------------------------------------------------------------------ inputs ---

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _lengths(lo, hi, n, seed):
    return np.random.default_rng(seed).integers(lo, hi + 1, size=n).astype(np.int64)


def _tables(lens, gen, seed, extra=0):
    """Page table of sequences of these lengths (unused slots -1), pages in
    random order, and the number of pages (`extra` unowned ones at the end)."""
    pages = (lens + PAGE - 1) // PAGE
    order = np.random.default_rng(seed + 1).permutation(int(pages.sum()))
    table = np.full((len(lens), int(pages.max())), -1, dtype=np.int32)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = order[at:at + p]
        at += p
    return torch.from_numpy(table).cuda(), int(pages.sum()) + extra


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _e2m1_codes(x):
    """Values -> 4-bit codes: nearest e2m1 value, ties to the even code, at most 6."""
    a = x.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8)
         + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8)
         + (a > 5.0).to(torch.uint8))
    return c + 8 * torch.signbit(x).to(torch.uint8)


def _quantise(x, kv):
    """fp32 rows [n, 512] -> (codes uint8 [n, 256], scale bytes uint8 [n, 512 / group])."""
    g = GROUP[kv]
    v = x.view(x.shape[0], DL // g, g)
    amax = v.abs().amax(-1)
    if kv == "mxfp4":   # 2^(floor(log2 amax) - 2); 1 for a group of zeros
        e = torch.frexp(amax).exponent - 1 - 2
        byte = torch.where(amax > 0, (e + 127).clamp(0, 254), torch.full_like(e, 127))
        scale = torch.ldexp(torch.ones_like(amax, dtype=torch.float64), byte - 127).float()
        byte = byte.to(torch.uint8)
    else:               # e4m3(amax / 6), at most 448; 1 for a group of zeros
        s = torch.where(amax > 0, amax / 6.0, torch.ones_like(amax)).clamp(max=448.0)
        s8 = s.to(torch.float8_e4m3fn)
        scale, byte = s8.float(), s8.view(torch.uint8)
    q = v / scale[..., None]
    q = torch.where(scale[..., None] > 0, q, torch.zeros_like(q))
    c = _e2m1_codes(q).view(x.shape[0], DL // 2, 2)
    return c[..., 0] + 16 * c[..., 1], byte


def _pools(kv, n_pages, gen):
    """Latent pools of a cache whose rows are N(0, 1)."""
    n = n_pages * PAGE
    p = {"kv_rope": None, "kv_scale": None}
    if kv == "bf16":
        p["kv"] = torch.randn(n, D, device="cuda", dtype=torch.bfloat16, generator=gen)
        return p
    p["kv_rope"] = torch.randn(n, DR, device="cuda", dtype=torch.bfloat16, generator=gen)
    width, groups = (DL, 4) if kv == "e4m3" else (DL // 2, DL // GROUP[kv])
    p["kv"] = torch.empty(n, width, device="cuda", dtype=torch.uint8)
    p["kv_scale"] = torch.empty(n, groups, device="cuda",
                                dtype=torch.float32 if kv == "e4m3" else torch.uint8)
    for r in range(0, n, 1 << 17):
        x = torch.randn(min(1 << 17, n - r), DL, device="cuda", generator=gen)
        if kv == "e4m3":
            v = x.view(-1, 4, 128)
            s = v.abs().amax(-1) / 448.0
            p["kv"][r:r + x.shape[0]] = ((v / s[..., None]).clamp(-448, 448)
                                         .to(torch.float8_e4m3fn).view(torch.uint8).view(-1, DL))
        else:
            codes, s = _quantise(x, kv)
            p["kv"][r:r + x.shape[0]] = codes
        p["kv_scale"][r:r + x.shape[0]] = s
    return p


def _index_pools(n_pages, gen, real):
    """Index keys (e4m3 with one scale per token); placeholders where no call reads them."""
    n = n_pages * PAGE if real else PAGE
    k = torch.randint(0, 126, (n, DI), device="cuda", dtype=torch.uint8, generator=gen)
    k += 128 * torch.randint(0, 2, (n, DI), device="cuda", dtype=torch.uint8, generator=gen)
    return {"k_index": k, "k_index_scale": torch.rand(n, device="cuda", generator=gen) + 0.5}


def _cache(s, table, seq_len, n_pages):
    from indexed_sparse_attention_lightning_b200 import api
    return api.DeviceCache(
        page_table=table, seq_len=seq_len, num_pages=n_pages, index_dtype="e4m3",
        k_index=s["k_index"], k_index_scale=s["k_index_scale"], kv_dtype=s["kv_dtype"],
        kv=s["kv"], kv_rope=s["kv_rope"], kv_scale=s["kv_scale"], d_index=DI, d_latent=DL,
        d_rope=DR, kv_scale_tile=(1, 128) if s["kv_dtype"] == "e4m3" else (0, 0))


def _attention_state(c, seed):
    gen = _gen(seed)
    n_q, K = c["n_q"], c["top_k"]
    decode = c["mode"] == "decode"
    lens = _lengths(c["lo"], c["hi"], n_q if decode else 1, seed)
    table, n_pages = _tables(lens, gen, seed)
    s = dict(c, kv_dtype=c["kv"], page_table=table, n_pages=n_pages, max_visible=int(lens.max()),
             seq_len=torch.from_numpy(lens.astype(np.int32)).cuda())
    s.update(_pools(c["kv"], n_pages, gen))
    s.update(_index_pools(n_pages, gen, False))
    if decode:
        q_seq, q_pos = np.arange(n_q), lens - 1
    else:
        q_seq, q_pos = np.zeros(n_q, np.int64), lens[0] - n_q + np.arange(n_q)
    s["q_seq"] = torch.from_numpy(q_seq.astype(np.int32)).cuda()
    s["q_pos"] = torch.from_numpy(q_pos.astype(np.int32)).cuda()
    s["q"] = torch.randn(n_q, HEADS, D, device="cuda", dtype=torch.bfloat16, generator=gen)
    # K distinct visible positions each, ascending, padded with -1
    V = s["max_visible"]
    k = min(K, V)
    idx = torch.full((n_q, K), -1, device="cuda", dtype=torch.int32)
    for t in range(0, n_q, 64):
        u = torch.rand(min(64, n_q - t), V, device="cuda", generator=gen)
        u.masked_fill_(torch.arange(V, device="cuda")[None] > s["q_pos"][t:t + 64, None], -1.0)
        top = u.topk(k, dim=1)
        pos = torch.where(top.values >= 0, top.indices, 1 << 30).sort(dim=1).values
        idx[t:t + 64, :k] = torch.where(pos < 1 << 30, pos, -1).int()
    if c["holes"]:   # entries left out anywhere, and a query with none at all
        idx[torch.rand(n_q, K, device="cuda", generator=gen) < 0.1] = -1
        idx[n_q // 2] = -1
    s["idx"] = idx
    s["out"] = torch.empty(n_q, HEADS, DL, device="cuda", dtype=torch.bfloat16)
    s["lse"] = torch.empty(n_q, HEADS, device="cuda")
    return s, gen


def _queries(s):
    from indexed_sparse_attention_lightning_b200 import api
    return api.DeviceQueries(
        q_seq=s["q_seq"], q_pos=s["q_pos"], max_visible=s["max_visible"], q_index=None,
        q_index_scale=None, w=None, h_index=64, q_dtype="bf16", q=s["q"], heads=HEADS,
        sm_scale=SM_SCALE)


def _prepare_attend(c, seed):
    s, _ = _attention_state(c, seed)
    if own:
        from indexed_sparse_attention_lightning_b200 import _abi, api
        s["cache"] = _cache(s, s["page_table"], s["seq_len"], s["n_pages"])
        s["queries"] = _queries(s)
        s["ws"] = api.workspace(api.workspace_size(s["cache"], s["queries"], c["top_k"],
                                                   _abi.SA_WS_ATTN))
    return s


def _prepare_weigh(c, seed):
    s, gen = _attention_state(c, seed)
    s["lse"] = _lse(_scores(s, *_rows(s)))
    shape = (s["seq_len"].numel(), c["hi"])
    s["acc"] = torch.rand(shape, device="cuda", generator=gen).exponential_(generator=gen)
    past = torch.arange(shape[1], device="cuda")[None] >= s["seq_len"][:, None]
    s["acc"][past] = 0.0
    s["acc_out"] = torch.zeros(shape, device="cuda")
    if own:
        from indexed_sparse_attention_lightning_b200 import _abi, api
        s["cache"] = _cache(s, s["page_table"], s["seq_len"], s["n_pages"])
        s["queries"] = _queries(s)
        s["ws"] = api.workspace(api.workspace_size(s["cache"], s["queries"], c["top_k"],
                                                   _abi.SA_WS_WEIGHTS))
    return s


def _prepare_write(c, seed):
    gen = _gen(seed)
    rng = np.random.default_rng(seed)
    # `n` tokens over `seqs` sequences at least one each, ending at a random old length
    cuts = np.sort(rng.choice(np.arange(1, c["n"]), size=c["seqs"] - 1, replace=False))
    new = np.diff(np.concatenate([[0], cuts, [c["n"]]]))
    old = rng.integers(0, 200, size=c["seqs"])
    lens = old + new
    table, n_pages = _tables(lens, gen, seed)
    s = dict(c, kv_dtype=c["kv"], page_table=table, n_pages=n_pages,
             seq_len=torch.from_numpy(old.astype(np.int32)).cuda())
    s.update(_pools(c["kv"], n_pages, gen))
    s.update(_index_pools(n_pages, gen, False))
    s["seq"] = torch.from_numpy(np.repeat(np.arange(c["seqs"]), new).astype(np.int32)).cuda()
    s["pos"] = torch.from_numpy(np.concatenate(
        [np.arange(o, o + n) for o, n in zip(old, new)]).astype(np.int32)).cuda()
    x = torch.randn(c["n"], D, device="cuda", generator=gen)
    x *= torch.exp2(torch.rand(c["n"], 1, device="cuda", generator=gen) * 6 - 3)
    s["x"] = x.to(torch.bfloat16) if c["inp"] == "bf16" else x
    s["back"] = torch.empty(c["n"], D, device="cuda", dtype=torch.bfloat16)
    if own:
        from indexed_sparse_attention_lightning_b200 import api
        s["cache"] = _cache(s, s["page_table"], s["seq_len"], s["n_pages"])
        s["ws"] = api.workspace(256)
    return s


def _prepare_evict(c, seed):
    gen = _gen(seed)
    lens = _lengths(c["lo"], c["hi"], c["batch"], seed)
    dst_pages = (c["budget"] + PAGE - 1) // PAGE
    table, n_pages = _tables(lens, gen, seed, extra=c["batch"] * dst_pages)
    s = dict(c, kv_dtype=c["kv"], page_table=table, n_pages=n_pages,
             src_pages=n_pages - c["batch"] * dst_pages,
             seq_len=torch.from_numpy(lens.astype(np.int32)).cuda())
    s.update(_pools(c["kv"], n_pages, gen))
    s.update(_index_pools(n_pages, gen, True))
    fresh = np.random.default_rng(seed + 2).permutation(c["batch"] * dst_pages) + s["src_pages"]
    s["dst_table"] = torch.from_numpy(fresh.astype(np.int32).reshape(c["batch"], -1)).cuda()
    s["dst_len"] = torch.zeros(c["batch"], device="cuda", dtype=torch.int32)
    # running sums: most positions were never selected, a few took most of the weight
    shape = (c["batch"], c["hi"])
    acc = torch.empty(shape, device="cuda").log_normal_(0.0, 1.5, generator=gen)
    s["acc"] = acc * (torch.rand(shape, device="cuda", generator=gen) < 0.3)
    s["acc_out"] = torch.empty(c["batch"], c["budget"], device="cuda")
    s["src_pos"] = torch.empty(c["batch"], c["budget"], device="cuda", dtype=torch.int32)
    if own:
        from indexed_sparse_attention_lightning_b200 import _abi, api
        s["cache"] = _cache(s, s["page_table"], s["seq_len"], n_pages)
        s["dst"] = _cache(s, s["dst_table"], s["dst_len"], n_pages)
        s["ws"] = api.workspace(api.workspace_size(s["cache"], None, c["budget"],
                                                   _abi.SA_WS_EVICT))
    return s


def prepare(case, seed):
    return {"attend": _prepare_attend, "weigh": _prepare_weigh, "write": _prepare_write,
            "evict": _prepare_evict}[case["op"]](case, seed)


# ------------------------------------------------------------- plain forms ---

def _values(s, rows):
    """Latent + rope of physical rows, as fp32 [..., 576]."""
    if s["kv_dtype"] == "bf16":
        return s["kv"][rows].float()
    rope = s["kv_rope"][rows].float()
    code, scale = s["kv"][rows], s["kv_scale"][rows]
    if s["kv_dtype"] == "e4m3":
        lat = code.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(128, dim=-1)
        return torch.cat([lat, rope], -1)
    nib = torch.stack([code & 15, code >> 4], -1).flatten(-2).int()
    mag = torch.tensor(E2M1, device="cuda")[nib & 7]
    val = torch.where(nib >= 8, -mag, mag)
    if s["kv_dtype"] == "mxfp4":
        sc = torch.exp2(scale.double() - 127.0).float()
    else:
        sc = scale.view(torch.float8_e4m3fn).float()
    return torch.cat([val * sc.repeat_interleave(GROUP[s["kv_dtype"]], dim=-1), rope], -1)


def _rows(s):
    """Physical rows of the selected positions, and which entries hold one."""
    have = s["idx"] >= 0
    pos = s["idx"].clamp(min=0).long()
    page = s["page_table"][s["q_seq"].long()[:, None], pos // PAGE].long()
    return torch.where(have, page * PAGE + pos % PAGE, 0), have


def _scores(s, rows, have):
    z = torch.matmul(s["q"].float(), _values(s, rows).transpose(1, 2)) * SM_SCALE
    return z.masked_fill(~have[:, None], -math.inf)


def _lse(z):
    m = z.amax(-1)
    m0 = torch.where(m == -math.inf, 0.0, m)
    return m0 + torch.log(torch.exp(z - m0[..., None]).sum(-1))


def _plain_attend(s):
    rows, have = _rows(s)
    kv = _values(s, rows)
    z = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * SM_SCALE
    z = z.masked_fill(~have[:, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(z - m)
    l = e.sum(-1, keepdim=True)
    out = torch.matmul(e, kv[..., :DL]) / torch.where(l > 0, l, 1.0)
    return out.to(torch.bfloat16), (m + torch.log(l)).squeeze(-1)


def _plain_weigh(s):
    rows, have = _rows(s)
    z = _scores(s, rows, have)
    lse = s["lse"][..., None]
    p = torch.where(lse == -math.inf, 0.0, torch.exp(z - lse))
    w = p.sum(1)
    acc = s["acc"].double() * s["decay"]
    at = s["q_seq"].long()[:, None] * acc.shape[1] + s["idx"].clamp(min=0).long()
    acc.view(-1).scatter_add_(0, at[have], w[have].double())
    live = torch.arange(acc.shape[1], device="cuda")[None] < s["seq_len"][:, None]
    return torch.where(live, acc.float(), s["acc_out"])


def _plain_write(s):
    row = (s["page_table"][s["seq"].long(), s["pos"].long() // PAGE].long() * PAGE
           + s["pos"].long() % PAGE)
    x = s["x"].float()
    s["kv"][row], s["kv_scale"][row] = _quantise(x[:, :DL].contiguous(), s["kv_dtype"])
    s["kv_rope"][row] = x[:, DL:].to(torch.bfloat16)
    return _values(s, row).to(torch.bfloat16)


def _keep(s):
    """Per sequence the kept positions, ascending, -1 behind them: [batch, budget]."""
    n, budget = s["seq_len"].long()[:, None], s["budget"]
    V = s["acc"].shape[1]
    at = torch.arange(V, device="cuda")[None]
    a = s["acc"].masked_fill((at < s["first"]) | (at >= n - s["last"]) | (n <= budget), math.inf)
    a = a.masked_fill(at >= n, -math.inf)
    best = a.sort(dim=1, descending=True, stable=True).indices[:, :budget]
    best = torch.where(best < n, best, 1 << 30).sort(dim=1).values
    best = torch.where(best < 1 << 30, best, -1)
    pad = torch.full((n.shape[0], max(0, budget - V)), -1, device="cuda", dtype=torch.int64)
    return torch.cat([best, pad], 1)


def _plain_evict(s):
    pos = _keep(s)
    b, i = torch.nonzero(pos >= 0, as_tuple=True)
    p = pos[b, i]
    src = s["page_table"][b, p // PAGE].long() * PAGE + p % PAGE
    dst = s["dst_table"][b, i // PAGE].long() * PAGE + i % PAGE
    s["kv"][dst] = s["kv"][src]
    if s["kv_dtype"] != "bf16":
        s["kv_rope"][dst] = s["kv_rope"][src]
        s["kv_scale"][dst] = s["kv_scale"][src]
    s["k_index"][dst] = s["k_index"][src]
    s["k_index_scale"][dst] = s["k_index_scale"][src]
    s["dst_len"].copy_((pos >= 0).sum(1).int())
    s["src_pos"].copy_(pos.int())
    kept = torch.gather(s["acc"], 1, pos.clamp(min=0))
    s["acc_out"].copy_(torch.where(pos >= 0, kept, 0.0))
    return _evicted(s)


def _evicted(s):
    """The fresh pages as they are now, and what else the pass wrote.  Rows are
    moved, not computed: 4-bit ones go out as the bytes that were moved."""
    new = slice(s["src_pages"] * PAGE, None)
    out = {"src_pos": s["src_pos"], "len": s["dst_len"], "acc": s["acc_out"],
           "k_index": s["k_index"][new].view(torch.float8_e4m3fn),
           "k_index_scale": s["k_index_scale"][new]}
    kv = s["kv"][new]
    out["kv"] = kv.view(torch.float8_e4m3fn) if s["kv_dtype"] == "e4m3" else kv
    if s["kv_dtype"] != "bf16":
        out["kv_rope"], out["kv_scale"] = s["kv_rope"][new], s["kv_scale"][new]
    return out


def run(state):
    s = state
    if not own:
        return {"attend": _plain_attend, "weigh": _plain_weigh, "write": _plain_write,
                "evict": _plain_evict}[s["op"]](s)
    from indexed_sparse_attention_lightning_b200 import api
    if s["op"] == "attend":
        return api.sparse_mla_attn(s["cache"], s["queries"], s["idx"], s["top_k"], out=s["out"],
                                   lse=s["lse"], ws=s["ws"])
    if s["op"] == "weigh":
        return api.accumulate_weights(s["cache"], s["queries"], s["idx"], s["top_k"], s["lse"],
                                      s["acc"], decay=s["decay"], out=s["acc_out"], ws=s["ws"])
    if s["op"] == "write":
        api.append_tokens(s["cache"], s["seq"], s["pos"], kv=s["x"], ws=s["ws"])
        api.read_tokens(s["cache"], s["seq"], s["pos"], out=s["back"], ws=s["ws"])
        return s["back"]
    api.evict_tokens(s["cache"], s["acc"], s["budget"], s["dst"], keep_first=s["first"],
                     keep_last=s["last"], acc_out=s["acc_out"], src_pos=s["src_pos"], ws=s["ws"])
    return _evicted(s)


# ------------------------------------------------------------ work, 64 bits ---

def _row_bytes(kv):
    return {"bf16": 2 * D, "e4m3": DL + 2 * DR + 16, "mxfp4": DL // 2 + 2 * DR + DL // 32,
            "nvfp4": DL // 2 + 2 * DR + DL // 16}[kv]


def work(case):
    c, row = case, _row_bytes(case["kv"])
    if c["op"] in ("attend", "weigh"):
        mean = (c["lo"] + c["hi"]) / 2
        sel = min(c["top_k"], mean) * (0.9 if c["holes"] else 1.0)
        # rows that are read: each query's own, or those of one sequence that any query selected
        n_rows = c["n_q"] * sel
        if c["mode"] == "chunk":
            n_rows = mean * (1.0 - (1.0 - sel / mean) ** c["n_q"])
        moved = n_rows * row + c["n_q"] * (4 * c["top_k"] + HEADS * (2 * D + 4))
        if c["op"] == "attend":
            return {"bytes": moved + c["n_q"] * HEADS * 2 * DL,
                    "flops": 2.0 * c["n_q"] * HEADS * sel * (D + DL)}
        seqs = c["n_q"] if c["mode"] == "decode" else 1
        return {"bytes": moved + seqs * mean * 8, "flops": 2.0 * c["n_q"] * HEADS * sel * D}
    if c["op"] == "write":   # in, into the cache, out of it, back
        return {"bytes": c["n"] * (D * (2 if c["inp"] == "bf16" else 4) + 2 * row + 2 * D),
                "flops": 0.0}
    kept = c["batch"] * min(c["budget"], (c["lo"] + c["hi"]) / 2)
    return {"bytes": kept * 2 * (row + DI + 4) + c["batch"] * (c["lo"] + c["hi"]) / 2 * 4
            + c["batch"] * c["budget"] * 8, "flops": 0.0}


def _exact_row(s, rows):
    """One query's selected rows in 64 bits, decoded value by value."""
    if s["kv_dtype"] == "bf16":
        return s["kv"][rows].double()
    rope = s["kv_rope"][rows].double()
    if s["kv_dtype"] == "e4m3":
        lat = s["kv"][rows].view(torch.float8_e4m3fn).double().view(-1, 4, 128)
        return torch.cat([(lat * s["kv_scale"][rows].double()[..., None]).view(-1, DL), rope], 1)
    byte, g = s["kv"][rows].long(), GROUP[s["kv_dtype"]]
    lat = torch.empty(byte.shape[0], DL, device="cuda", dtype=torch.float64)
    for half in (0, 1):
        n = byte // 16 if half else byte % 16
        e, m = (n // 2) % 4, (n % 2).double()
        # e = 0: m / 2; else 2^(e - 1) (1 + m / 2)
        v = torch.where(e == 0, m / 2, torch.exp2(e.double() - 1) * (1 + m / 2))
        lat[:, half::2] = torch.where(n >= 8, -v, v)
    sb = s["kv_scale"][rows]
    sc = (torch.exp2(sb.double() - 127) if s["kv_dtype"] == "mxfp4"
          else sb.view(torch.float8_e4m3fn).double())
    lat = (lat.view(-1, DL // g, g) * sc[..., None]).view(-1, DL)
    return torch.cat([lat, rope], 1)


def _exact_selected(s):
    table, idx = s["page_table"].cpu().numpy(), s["idx"].cpu().numpy()
    q_seq = s["q_seq"].cpu().numpy()
    for t in range(s["n_q"]):
        pos = idx[t][idx[t] >= 0].astype(np.int64)
        rows = table[q_seq[t]][pos // PAGE].astype(np.int64) * PAGE + pos % PAGE
        kv = _exact_row(s, torch.from_numpy(rows).cuda())
        yield t, int(q_seq[t]), torch.from_numpy(pos).cuda(), kv, \
            (s["q"][t].double() @ kv.T) * SM_SCALE


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "attend":
        out = torch.zeros(s["n_q"], HEADS, DL, device="cuda", dtype=torch.float64)
        lse = torch.full((s["n_q"], HEADS), -math.inf, device="cuda", dtype=torch.float64)
        for t, _, pos, kv, z in _exact_selected(s):
            if pos.numel():
                out[t] = torch.softmax(z, -1) @ kv[:, :DL]
                lse[t] = torch.logsumexp(z, -1)
        return out, lse
    if s["op"] == "weigh":
        acc = s["acc"].double() * s["decay"]
        for t, b, pos, _, z in _exact_selected(s):
            if pos.numel():
                acc[b, pos] += torch.exp(z - s["lse"][t].double()[:, None]).sum(0)
        live = torch.arange(acc.shape[1], device="cuda")[None] < s["seq_len"][:, None]
        return torch.where(live, acc, s["acc_out"].double())
    if s["op"] == "write":
        x = s["x"].double().cpu().numpy()
        g = GROUP[s["kv_dtype"]]
        v = x[:, :DL].reshape(-1, DL // g, g)
        amax = np.abs(v).max(-1)
        if s["kv_dtype"] == "mxfp4":
            sc = np.where(amax > 0, 2.0 ** (np.floor(np.log2(np.where(amax > 0, amax, 1.0))) - 2),
                          1.0)
        else:   # the scale and the quotients are defined in fp32, like every code of the cache
            s32 = np.where(amax > 0, (amax / 6.0).astype(np.float32), np.float32(1.0))
            sc = (torch.from_numpy(np.minimum(s32, np.float32(448))).to(torch.float8_e4m3fn)
                  .double().numpy())
        with np.errstate(divide="ignore", invalid="ignore"):
            q = np.where(sc[..., None] > 0, v / sc[..., None], 0.0).astype(np.float32)
        values = np.array(E2M1)
        even = np.array([0.25, 1.25, 2.5, 5.0], np.float32)   # borders whose lower code is even
        up = np.searchsorted((values[1:] + values[:-1]) / 2, np.abs(q), side="right")
        up = up - np.isin(np.abs(q), even)
        lat = np.copysign(values[up], q) * sc[..., None]
        # the rope is rounded to bf16 when it is stored
        rope = s["x"][:, DL:].to(torch.bfloat16).double().cpu().numpy()
        return torch.from_numpy(np.concatenate([lat.reshape(-1, DL), rope], 1))
    return None
