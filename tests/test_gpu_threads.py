"""GPU test of calls from two host threads at once, each with its own stream,
workspace and outputs, and with sizes that need different shared memory."""
import threading

import pytest
import torch

from indexed_sparse_attention_lightning_b200 import _abi, api
from tests.test_gpu_cache_ops import make, selection, upload

pytestmark = pytest.mark.gpu


def evictions(max_pages):
    """80 sequences, one CTA each, with keys in shared memory for what a row of
    their page table could hold."""
    wl = make("f32", [100] * 80, heads=2, d_latent=16, d_rope=0)
    cache, _, _ = upload(wl, selection(wl, 1, 1))
    acc = torch.rand((80, 64 * max_pages), device="cuda")
    wide = torch.full((80, max_pages), -1, dtype=torch.int32, device="cuda")
    wide[:, :cache.page_table.shape[1]] = cache.page_table
    cache.page_table = wide
    fresh = torch.arange(80, dtype=torch.int32, device="cuda").reshape(80, 1) + wl.num_pages
    cache.num_pages += 80
    for k in ("k_index", "k_index_scale", "kv"):
        t = getattr(cache, k)
        setattr(cache, k, torch.cat([t, t[:80]]))
    dst = api.DeviceCache(**{**vars(cache), "page_table": fresh,
                             "seq_len": torch.zeros(80, dtype=torch.int32, device="cuda")})
    ws = api.workspace(api.workspace_size(cache, None, 64, _abi.SA_WS_EVICT))
    out = torch.zeros((80, 64), dtype=torch.int32, device="cuda")
    return lambda: api.evict_tokens(cache, acc, 64, dst, 1, 1, src_pos=out, ws=ws)


def others(dl, heads, h_index, d_index, ranks):
    wl = make("f32", (150, 90), heads=heads, d_latent=dl, d_rope=16, h_index=h_index,
              d_index=d_index, index_dtype="f32")
    cache, queries, idx = upload(wl, selection(wl, 40, 3))
    use = (_abi.SA_WS_ATTN, _abi.SA_WS_WEIGHTS, _abi.SA_WS_INDEXER)
    ws = api.workspace(max(api.workspace_size(cache, queries, 40, u) for u in use))
    out = torch.empty((2, heads, dl), device="cuda")
    lse = torch.empty((2, heads), device="cuda")
    sums, scores = torch.zeros((2, 150), device="cuda"), torch.zeros((2, 150), device="cuda")
    score = torch.rand((ranks, 2, 40), device="cuda")
    pos = torch.arange(ranks * 80, dtype=torch.int32, device="cuda").view(ranks, 2, 40)
    lo, hi = (torch.full((2,), v, dtype=torch.int32, device="cuda") for v in (0, 1000))
    best = [torch.empty((2, 40), dtype=torch.int32, device="cuda") for _ in range(2)]

    def call():
        api.sparse_mla_attn(cache, queries, idx, 40, out=out, lse=lse, out_dtype="f32", ws=ws)
        api.accumulate_weights(cache, queries, idx, 40, lse, None, out=sums, ws=ws)
        api.indexer_score(cache, queries, scores=scores, ws=ws)
        api.merge_candidates(score, pos, 40, lo, hi, *best)
        return torch.cat([t.float().flatten() for t in (out, lse, sums, scores, *best)])

    return call


@pytest.mark.parametrize("small,large", [
    (lambda: evictions(4), lambda: evictions(768)),
    (lambda: others(32, 16, 4, 16, 2), lambda: others(512, 16, 128, 256, 600)),
], ids=["evict", "others"])
def test_two_threads_with_different_sizes(small, large, monkeypatch):
    """The library's calls are recorded once and repeated without the binding, so
    that both threads are inside the library most of the time."""
    lib = _abi.lib()
    streams = [torch.cuda.Stream() for _ in range(2)]
    calls = [small(), large()]
    want = [c().clone() for c in calls]
    torch.cuda.synchronize()
    recorded = [[], []]

    class Recorder:
        def __getattr__(self, name):
            f = getattr(lib, name)

            def call(*args):
                kept.append((f, args))
                return f(*args)
            return call

    monkeypatch.setattr(_abi, "lib", Recorder)
    for kept, c, s in zip(recorded, calls, streams):
        with torch.cuda.stream(s):
            c()
    monkeypatch.undo()
    start, bad = threading.Barrier(2), []

    def work(mine):
        start.wait()
        for _ in range(1500):
            for f, args in mine:
                status = f(*args)
                if status != _abi.SA_OK:
                    bad.append((f.__name__, status))

    threads = [threading.Thread(target=work, args=(r,)) for r in recorded]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, (len(bad), set(bad))
    for c, w in zip(calls, want):
        assert torch.equal(c(), w)
