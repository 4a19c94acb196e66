"""The Python binding's own part, with the library and CUDA replaced by
stand-ins: which stream its buffers are made on, which device a call runs on
(no GPU)."""
import dataclasses
import types

import pytest
import torch

from indexed_sparse_attention_lightning_b200 import _abi, api

MAIN, SIDE, FAR = (types.SimpleNamespace(cuda_stream=h, device=torch.device("cuda", d))
                   for h, d in ((1, 0), (2, 0), (3, 1)))


class Placed(torch.Tensor):
    """A tensor that says which GPU it is on."""

    def get_device(self):
        return self.on


def placed(t, device=0):
    t = t.as_subclass(Placed)
    t.on = device
    return t


class Made(Placed):
    """One that the binding allocated; remembers record_stream()."""

    def record_stream(self, stream):
        self.__dict__.setdefault("recorded", []).append(stream)


class World:
    """The current device and stream, the tensors made, and the streams and devices
    launched on."""

    def __init__(self, monkeypatch):
        self.device, self.current, self.made, self.launched, self.ran_on = 0, MAIN, [], [], []
        world = self

        class On:
            def __init__(self, where):
                self.at = (where, world.current) if isinstance(where, int) else \
                    (where.device.index, where)

            def __enter__(self):
                self.before = world.device, world.current
                world.device, world.current = self.at

            def __exit__(self, *exc):
                world.device, world.current = self.before

        class Lib:
            def __getattr__(self, name):
                def call(*args):
                    if name == "sa_workspace_size":
                        return 4096
                    if name == "sa_status_string":
                        return b""
                    world.launched.append(next(a for a in reversed(args) if isinstance(a, int)))
                    world.ran_on.append(world.device)
                    return _abi.SA_OK
                return call

        def making(f):
            def make(*args, **kwargs):
                t = f(*args, **kwargs).as_subclass(Made)
                t.on = world.device
                world.made.append((t, world.current))
                return t
            return make

        lib = Lib()
        monkeypatch.setattr(torch.cuda, "stream", On)
        monkeypatch.setattr(torch.cuda, "device", On)
        monkeypatch.setattr(api, "_device", lambda: world.device)
        monkeypatch.setattr(api, "_raw_stream", lambda device: world.current.cuda_stream)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: world.current)
        monkeypatch.setattr(_abi, "lib", lambda: lib)
        monkeypatch.setattr(api, "_need", lambda *a, **k: None)
        monkeypatch.setattr(api, "_need_rows", lambda *a, **k: None)
        for name in ("empty", "zeros", "full"):
            monkeypatch.setattr(torch, name, making(getattr(torch, name)))


def given(on=0):
    """Inputs of every entry point on GPU `on`, made before the stand-ins."""
    def zeros(*shape, dtype=torch.int32):
        return placed(torch.zeros(shape, dtype=dtype), on)

    f32 = dict(dtype=torch.float32)
    cache = api.DeviceCache(
        page_table=zeros(2, 4), seq_len=zeros(2), num_pages=8, index_dtype="e4m3",
        k_index=zeros(1), k_index_scale=zeros(1), kv_dtype="bf16", kv=zeros(1), kv_rope=None,
        kv_scale=None, d_index=128, d_latent=512, d_rope=64)
    queries = api.DeviceQueries(
        q_seq=zeros(2), q_pos=zeros(2), max_visible=200, q_index=zeros(1),
        q_index_scale=zeros(1), w=zeros(1), h_index=64, q_dtype="bf16", q=zeros(1), heads=128,
        sm_scale=0.04)
    idx, lse, sums, n = zeros(2, 8), zeros(2, 128, **f32), zeros(2, 256, **f32), zeros(2)
    score = zeros(3, 2, 8, **f32)
    return {
        "indexer_score": (cache, queries), "topk": (lse, n, 8, 128),
        "sparse_mla_attn": (cache, queries, idx, 8), "decode": (cache, queries, 8),
        "local_candidates": (cache, queries, 8, n),
        "merge_candidates": (score, zeros(3, 2, 8), 8, n, n),
        "combine_partials": (zeros(3, 2, 4, 16, **f32), zeros(3, 2, 4, **f32)),
        "quantize_index_query": (zeros(2, 64, 128, **f32),), "append_tokens": (cache, n, n),
        "read_tokens": (cache, n, n),
        "accumulate_weights": (cache, queries, idx, 8, lse, None),
        "evict_tokens": (cache, sums, 64, cache),
    }


# a tensor that each takes besides its first arguments
EXTRA = {"indexer_score": "scores", "topk": "idx", "sparse_mla_attn": "out", "decode": "ws",
         "local_candidates": "pos", "merge_candidates": "idx_local", "combine_partials": "lse",
         "quantize_index_query": "scale", "append_tokens": "ws", "read_tokens": "out",
         "accumulate_weights": "out", "evict_tokens": "src_pos"}


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
        own.on, own.recorded = 0, []
        assert getattr(api, name)(*args, **{EXTRA[name]: own}, stream=SIDE) is own
        assert own.recorded == []
        world.launched.pop()

    world.made.clear()
    got = getattr(api, name)(*args)                     # on the current stream: nothing to tell
    assert world.made and all(stream is MAIN for _, stream in world.made)
    assert world.launched == [SIDE.cuda_stream, MAIN.cuda_stream]
    assert not any(hasattr(t, "recorded") for t, _ in world.made)


@pytest.mark.parametrize("name", sorted(given()))
def test_a_call_runs_on_the_device_of_its_tensors(name, monkeypatch):
    args = given(on=1)[name]
    near, far = placed(torch.zeros((2, 256))), placed(torch.zeros((2, 256)), 1)
    world = World(monkeypatch)
    f = getattr(api, name)
    f(*args)
    assert world.ran_on == [1] and world.device == 0
    assert world.made and all(t.on == 1 for t, _ in world.made)
    f(*args, stream=FAR)
    assert world.ran_on == [1, 1] and world.launched[1] == FAR.cuda_stream
    assert (world.device, world.current) == (0, MAIN)
    f(*args, **{EXTRA[name]: far})
    assert world.ran_on == [1, 1, 1]
    for bad in ({EXTRA[name]: near}, {"stream": SIDE}):     # of another device
        with pytest.raises(api.SaError):
            f(*args, **bad)
    assert world.ran_on == [1, 1, 1] and world.device == 0


def test_a_status_is_read_on_the_device_of_its_workspace(monkeypatch):
    ws = placed(torch.zeros(256), 1)
    world = World(monkeypatch)
    monkeypatch.setattr(api, "_raw_stream", lambda device: 100 + device)

    class Lib:
        def sa_device_status(self, p, n, stream, detail):
            assert stream == 101
            return 0

    monkeypatch.setattr(_abi, "lib", lambda: Lib())
    assert api.device_status(ws) == (0, 0) and world.device == 0


def test_arrays_that_are_too_short_are_refused(monkeypatch):
    """The kernels read an entry of seq_len per sequence (an eviction writes the
    destination's) and one of q_pos per query."""
    args = given()
    short = placed(torch.zeros(1, dtype=torch.int32))
    flat = placed(torch.zeros(8, dtype=torch.int32))
    World(monkeypatch)
    cache, queries, idx, _, lse, _ = args["accumulate_weights"]
    sums = args["evict_tokens"][1]
    cut = dataclasses.replace(cache, seq_len=short)
    wrong = dataclasses.replace(cache, page_table=flat)
    for call in (lambda: api.evict_tokens(cache, sums, 64, cut),
                 lambda: api.evict_tokens(cut, sums, 64, cache),
                 lambda: api.evict_tokens(cache, sums, 64, wrong),
                 lambda: api.accumulate_weights(cut, queries, idx, 8, lse, None),
                 lambda: api.accumulate_weights(
                     cache, dataclasses.replace(queries, q_pos=short), idx, 8, lse, None),
                 lambda: api.read_tokens(wrong, flat, flat),
                 lambda: api.read_tokens(cache, flat, flat, out_dtype="f16")):
        with pytest.raises(api.SaError):
            call()
    # buffers of a larger capacity are fine
    api.evict_tokens(cache, sums, 64, dataclasses.replace(cache, seq_len=flat))


def test_a_cache_need_only_look_like_one(monkeypatch):
    """Any object with a cache's fields and struct(), on another stream too."""
    cache, seq, pos = given()["read_tokens"]
    like = types.SimpleNamespace(**vars(cache), struct=cache.struct)
    World(monkeypatch)
    for stream in (None, SIDE):
        out, _ = api.read_tokens(like, seq, pos, stream=stream)
        assert out.shape == (2, 576)
