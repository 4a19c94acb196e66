"""The Python binding's own part, with the library and CUDA replaced by
stand-ins: which stream its buffers are made on (no GPU)."""
import types

import pytest
import torch

from indexed_sparse_attention_lightning_b200 import _abi, api

MAIN, SIDE = (types.SimpleNamespace(cuda_stream=h, device="cpu") for h in (1, 2))


class Made(torch.Tensor):
    """A tensor that the binding allocated; remembers record_stream()."""

    def record_stream(self, stream):
        self.__dict__.setdefault("recorded", []).append(stream)


class World:
    """The current stream, the tensors made and the streams launched on."""

    def __init__(self, monkeypatch):
        self.current, self.made, self.launched = MAIN, [], []
        world = self

        class On:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                self.before, world.current = world.current, self.stream

            def __exit__(self, *exc):
                world.current = self.before

        class Lib:
            def __getattr__(self, name):
                def call(*args):
                    if name == "sa_workspace_size":
                        return 4096
                    world.launched.append(next(a for a in reversed(args) if isinstance(a, int)))
                    return _abi.SA_OK
                return call

        def making(f):
            def make(*args, **kwargs):
                t = f(*args, **kwargs).as_subclass(Made)
                world.made.append((t, world.current))
                return t
            return make

        lib = Lib()
        monkeypatch.setattr(torch.cuda, "stream", On)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: world.current)
        monkeypatch.setattr(_abi, "lib", lambda: lib)
        monkeypatch.setattr(api, "_need", lambda *a, **k: None)
        monkeypatch.setattr(api, "_need_rows", lambda *a, **k: None)
        monkeypatch.setattr(api, "_need_here", lambda *a, **k: None)
        monkeypatch.setattr(api, "_stream", lambda s: (s or world.current).cuda_stream)
        for name in ("empty", "zeros", "full"):
            monkeypatch.setattr(torch, name, making(getattr(torch, name)))


def given():
    """Inputs of every entry point, made before the stand-ins."""
    i32 = dict(dtype=torch.int32)
    cache = api.DeviceCache(
        page_table=torch.zeros((2, 4), **i32), seq_len=torch.zeros(2, **i32), num_pages=8,
        index_dtype="e4m3", k_index=torch.zeros(1), k_index_scale=torch.zeros(1),
        kv_dtype="bf16", kv=torch.zeros(1), kv_rope=None, kv_scale=None, d_index=128,
        d_latent=512, d_rope=64)
    queries = api.DeviceQueries(
        q_seq=torch.zeros(2, **i32), q_pos=torch.zeros(2, **i32), max_visible=200,
        q_index=torch.zeros(1), q_index_scale=torch.zeros(1), w=torch.zeros(1), h_index=64,
        q_dtype="bf16", q=torch.zeros(1), heads=128, sm_scale=0.04)
    idx, lse, sums = torch.zeros((2, 8), **i32), torch.zeros((2, 128)), torch.zeros((2, 256))
    n = torch.zeros(2, **i32)
    score = torch.zeros((3, 2, 8))
    return {
        "indexer_score": (cache, queries), "topk": (lse, n, 8, 128),
        "sparse_mla_attn": (cache, queries, idx, 8), "decode": (cache, queries, 8),
        "local_candidates": (cache, queries, 8, n),
        "merge_candidates": (score, score.int(), 8, n, n),
        "combine_partials": (torch.zeros((3, 2, 4, 16)), torch.zeros((3, 2, 4))),
        "quantize_index_query": (torch.zeros((2, 64, 128)),), "append_tokens": (cache, n, n),
        "read_tokens": (cache, n, n),
        "accumulate_weights": (cache, queries, idx, 8, lse, None),
        "evict_tokens": (cache, sums, 64, cache),
    }


@pytest.mark.parametrize("name", sorted(given()))
def test_buffers_belong_to_the_stream_of_the_call(name, monkeypatch):
    """What the binding allocates or fills, it does on the stream that the kernels
    run on: on another one nothing would order the two, and a workspace dropped on
    return would be given away while they still use it.  What it returns is known
    to be used on the caller's stream too."""
    args = given()[name]
    world = World(monkeypatch)
    got = getattr(api, name)(*args, stream=SIDE)
    assert world.made and all(stream is SIDE for _, stream in world.made)
    assert world.launched == [SIDE.cuda_stream] and world.current is MAIN
    for t in got if isinstance(got, tuple) else (got,):
        if isinstance(t, Made):
            assert t.recorded == [MAIN]
    if isinstance(got, Made):                           # the caller's own are the caller's
        own = got.clone()
        own.recorded = []
        out = {"indexer_score": "scores", "topk": "idx", "accumulate_weights": "out",
               "evict_tokens": "src_pos", "append_tokens": "ws"}[name]
        assert getattr(api, name)(*args, **{out: own}, stream=SIDE) is own
        assert own.recorded == []
        world.launched.pop()

    world.made.clear()
    got = getattr(api, name)(*args)                     # on the current stream: nothing to tell
    assert world.made and all(stream is MAIN for _, stream in world.made)
    assert world.launched == [SIDE.cuda_stream, MAIN.cuda_stream]
    assert not any(hasattr(t, "recorded") for t, _ in world.made)
