"""GPU tests of the Python binding's own part: calls on another stream than the
current one, with the buffers that the binding makes itself, and outputs off the
boundary that the kernels store to."""
import pytest
import torch

from indexed_sparse_attention_lightning_b200 import _abi, api
from tests.test_gpu_cache_ops import make, selection, upload

pytestmark = pytest.mark.gpu


def test_calls_on_a_stream_of_their_own():
    """The current stream has work in front, and after the call takes and fills
    memory as large as what the call has dropped: neither reaches its results."""
    wl = make("bf16", (3000, 2500, 700), heads=128, h_index=64)
    idx = selection(wl, 600, 5)
    cache, queries, idx_t = upload(wl, idx)
    _, lse = api.sparse_mla_attn(cache, queries, idx_t, 600)
    acc = torch.rand((3, 3000), device="cuda")
    spare = torch.arange(9, dtype=torch.int32, device="cuda").reshape(3, 3) + wl.num_pages

    def grown():
        c, _, _ = upload(wl, idx)
        c.kv = torch.cat([c.kv, torch.zeros_like(c.kv[:9])])
        c.k_index = torch.cat([c.k_index, torch.zeros_like(c.k_index[:9])])
        c.k_index_scale = torch.cat([c.k_index_scale, torch.zeros_like(c.k_index_scale[:9])])
        c.num_pages += 9
        d = api.DeviceCache(**{**vars(c), "page_table": spare,
                               "seq_len": torch.zeros(3, dtype=torch.int32, device="cuda")})
        return c, d

    def everything(stream):
        c, d = grown()
        torch.cuda.synchronize()
        sizes = [api.workspace_size(c, queries, 600, u) for u in
                 (_abi.SA_WS_WEIGHTS, _abi.SA_WS_EVICT, _abi.SA_WS_DECODE, _abi.SA_WS_ATTN)]
        sizes += [4 * 3 * wl.max_visible]
        out = []
        for call in (lambda: api.accumulate_weights(cache, queries, idx_t, 600, lse, None,
                                                    stream=stream),
                     lambda: api.evict_tokens(c, acc, 192, d, 4, 30, stream=stream),
                     lambda: api.sparse_mla_attn(cache, queries, idx_t, 600, stream=stream)[0],
                     lambda: api.decode(cache, queries, 600, stream=stream)[0]):
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
                torch.cuda._sleep(4_000_000)            # about 2 ms
            out.append(call())
            for n in sizes:
                torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
            if stream is not None:
                torch.cuda.current_stream().wait_stream(stream)
        torch.cuda.synchronize()
        return out + [c.kv, d.seq_len]

    want = everything(None)
    side = torch.cuda.Stream()
    for _ in range(3):
        for got, exp in zip(everything(side), want):
            assert torch.equal(got, exp)


def test_results_outlive_the_callers_use():
    """A result made on another stream, dropped while the caller's stream still has
    to read it: the next one made there does not overwrite it."""
    wl = make("bf16", (900, 300), heads=128)
    idx = selection(wl, 200, 5)
    cache, queries, idx_t = upload(wl, idx)
    _, lse = api.sparse_mla_attn(cache, queries, idx_t, 200)
    want = api.accumulate_weights(cache, queries, idx_t, 200, lse, None)
    other = 2 * want
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        got = api.accumulate_weights(cache, queries, idx_t, 200, lse, None, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(2_000_000)
        copy = got.clone()
        del got
        with torch.cuda.stream(side):
            torch.empty_like(other).copy_(other)
        torch.cuda.synchronize()
        assert torch.equal(copy, want)


@pytest.mark.parametrize("n,heads", [(2, 128), (90, 128), (2, 16)])   # split keys, whole, CUDA cores
@pytest.mark.parametrize("out_dtype,off", [("bf16", 4), ("bf16", 1), ("f32", 1), ("f32", 2)])
def test_outputs_that_start_anywhere(n, heads, out_dtype, off):
    wl = make("bf16", [200 + i for i in range(n)], heads=heads, h_index=64)
    idx = selection(wl, 150, 5)
    cache, queries, idx_t = upload(wl, idx)
    dtype = torch.bfloat16 if out_dtype == "bf16" else torch.float32
    want = [api.sparse_mla_attn(cache, queries, idx_t, 150, out_dtype=out_dtype)[0],
            api.decode(cache, queries, 150, out_dtype=out_dtype)[0]]
    for i, exp in enumerate(want):
        room = torch.full((exp.numel() + 16,), 7.0, dtype=dtype, device="cuda")
        out = room[off:off + exp.numel()].view(exp.shape)
        assert out.data_ptr() % 16 != 0
        if i == 0:
            got, _ = api.sparse_mla_attn(cache, queries, idx_t, 150, out=out, out_dtype=out_dtype)
        else:
            got, _, _ = api.decode(cache, queries, 150, out=out, out_dtype=out_dtype)
        assert got is out and torch.equal(out, exp)
        assert torch.all(room[:off] == 7) and torch.all(room[off + exp.numel():] == 7)


def test_skipped_work_is_seen_without_a_workspace_of_ones_own():
    wl = make("mxfp4", (300, 200), heads=128)
    idx = selection(wl, 50, 3)
    bad = idx.copy()
    bad[1, 7] = 200                                     # not yet there
    cache, queries, idx_t = upload(wl, idx)
    bad_t = torch.from_numpy(bad).cuda()
    _, lse = api.sparse_mla_attn(cache, queries, idx_t, 50)
    acc = torch.rand((2, 300), device="cuda")
    ok, fault = (_abi.SA_OK, 0), _abi.SA_ERR_DEVICE_FAULT
    for i, want in ((idx_t, ok), (bad_t, (fault, _abi.SA_DETAIL_BAD_INDEX))):
        out, ws = api.accumulate_weights(cache, queries, i, 50, lse, acc, return_ws=True,
                                         out=torch.zeros_like(acc))
        assert api.device_status(ws) == want
        assert torch.equal(out, api.accumulate_weights(cache, queries, i, 50, lse, acc,
                                                       out=torch.zeros_like(acc)))
    pages = torch.arange(2, dtype=torch.int32, device="cuda").reshape(2, 1) + wl.num_pages
    for c, want in ((cache, (fault, _abi.SA_DETAIL_BAD_PAGE)), (None, ok)):
        if c is None:                                   # the pages exist now
            cache.num_pages += 2
            for k in ("k_index", "k_index_scale", "kv", "kv_rope", "kv_scale"):
                t = getattr(cache, k)
                setattr(cache, k, torch.cat([t, t[:2]]))
        dst = api.DeviceCache(**{**vars(cache), "page_table": pages,
                                 "seq_len": torch.zeros(2, dtype=torch.int32, device="cuda")})
        pos, ws = api.evict_tokens(cache, acc, 64, dst, return_ws=True)
        assert api.device_status(ws) == want
        assert dst.seq_len.tolist() == ([0, 0] if want != ok else [64, 64])
        assert torch.equal(pos, api.evict_tokens(cache, acc, 64, dst))
