"""The binding of the paged cache without a GPU: tensors on the CPU, in a cache that has no handle."""
import contextlib
import gc
import weakref

import pytest
import torch

import mxfp4_moe_expert_gb300 as pkg


def bare(kv_heads=2, head_dim=64, num_streams=8):
    """A KvCache whose tensors are on the CPU and that makes no library call by itself."""
    c = pkg.KvCache.__new__(pkg.KvCache)
    c.handle, c.device, c._index, c.dtype = None, torch.device("cpu"), -1, torch.bfloat16
    c.kv_heads, c.head_dim, c.num_streams = kv_heads, head_dim, num_streams
    c._layouts, c._pairs, c._ws, c._ws_bytes, c._ws_kept = {}, {}, None, {}, []
    c._i32, c._f32, c._u8, c._mask_types = torch.int32, torch.float32, torch.uint8, (torch.int64, torch.uint64)
    return c


def rows(S, B, H=2, D=64):
    return torch.zeros((S, B, H, D), dtype=torch.bfloat16)


@pytest.mark.parametrize("S,B", [(4, 1), (1, 5), (4, 3)])
def test_tokens_that_share_memory_are_refused(S, B):
    """A token broadcast over streams or positions has a stride of zero, which the library takes for contiguous rows."""
    c, whole = bare(), rows(S, B)
    wide = rows(1, 1).expand(S, B, 2, 64)
    near = torch.zeros(4096, dtype=torch.bfloat16).as_strided((S, B, 2, 64), (B * 64, 64, 64, 1))   # rows that overlap
    for t in (wide, near):
        with pytest.raises(ValueError, match="tokens"):
            c._rows("q", t)
        with pytest.raises(ValueError, match="tokens"):
            c._pair(t, t)
        with pytest.raises(ValueError, match="tokens|stride"):
            c._pair(whole, t)
    assert not c._pairs and c._rows("q", whole) == (S, B, 2, 64, 128)


def test_a_single_token_may_have_any_stride():
    c = bare()
    assert c._rows("q", rows(1, 1).expand(1, 1, 2, 64)) == (1, 1, 2, 64, 128)
    assert c._pair(rows(1, 1), rows(4, 4)[:1, :1]) == (1, 1, 128)
    assert c._rows("q", rows(3, 4)[:0])[:2] == (0, 4) and c._rows("q", rows(3, 4)[:, :0])[:2] == (3, 0)


class OnGpu:
    """A CPU tensor that says that it is on a GPU."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_pools_whose_pages_share_memory_are_refused():
    one = torch.zeros((1, 2, 16, 64), dtype=torch.bfloat16)
    page = 2 * 16 * 64
    for t in (one.expand(5, 2, 16, 64), torch.zeros(5 * page, dtype=one.dtype).as_strided((5, 2, 16, 64), (page // 2, 1024, 64, 1))):
        with pytest.raises(ValueError, match="pages"):
            pkg.KvCache(layers=[(OnGpu(t), OnGpu(t))], num_streams=1, max_pages=1)


class FakeLibrary:
    def __init__(self):
        self.attends = []

    def moe_mxfp4_cache_attend(self, handle, state, layer, args, ws, n, stream):
        self.attends.append((stream, ws, n))
        return 0


@pytest.fixture
def streams(monkeypatch):
    """The stream that torch has as current (7 at first), and the one that each new tensor was made on."""
    now, made = [7], []

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, device=None: ptr)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: 0)
    for name in ("empty", "zeros"):
        plain = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, plain=plain, **kw: (made.append(now[-1]), plain(*a, **kw))[1])
    return now, made


@pytest.mark.parametrize("stream", [None, 7, 99, 0])
@pytest.mark.parametrize("lengths", [False, True])
def test_what_attend_makes_is_made_on_the_stream_of_the_call(stream, lengths, streams):
    """A fill on another stream may land after the kernels, and memory of another stream may still be in use there."""
    now, made = streams
    c = bare()
    c._lib, c._state_ptr = FakeLibrary(), 16
    c._current_stream = lambda index: now[-1]
    c.attend_bytes = lambda S, B, H: 1000
    q = rows(3, 2)
    made.clear()
    c.attend(0, q, lengths=torch.ones(3, dtype=torch.int32) if lengths else None, stream=stream)
    on = 7 if stream is None else stream
    assert made == [on] * 3 and now == [7]            # out, lse, the workspace
    assert c._lib.attends[0][0] == on


def test_a_workspace_elsewhere_or_in_pieces_is_refused():
    c = bare()
    c._lib, c._state_ptr, c._current_stream = FakeLibrary(), 16, lambda index: 7
    q, other = rows(3, 2), OnGpu(torch.zeros(1024, dtype=torch.uint8))
    other.get_device = lambda: 0                     # (the cache's own device here is -1, the CPU)
    for ws in (other, torch.zeros(2048, dtype=torch.uint8)[::2], torch.zeros((4, 512), dtype=torch.uint8).T):
        with pytest.raises(ValueError, match="workspace"):
            c.attend(0, q, workspace=ws)
    ws = torch.zeros(1024, dtype=torch.uint8)
    c.attend(0, q, workspace=ws)
    assert c._lib.attends == [(7, ws.data_ptr(), 1024)]


def test_kept_workspaces_stay_a_small_multiple_of_what_is_needed():
    """Captured graphs may hold a workspace's address, so none is given back: a batch that grows stream by stream must
    not leave one behind for every size."""
    c = bare()
    c._lib, c._state_ptr, c._current_stream = FakeLibrary(), 16, lambda index: 7
    c.attend_bytes = lambda S, B, H: 1000 + 100 * S
    for S in range(1, 101):
        c.attend(0, rows(S, 1))
    need = c.attend_bytes(100, 1, 2)
    assert all(n >= c.attend_bytes(S + 1, 1, 2) and ws % 256 == 0 for S, (_, ws, n) in enumerate(c._lib.attends))
    assert sum(ws.numel() for ws in c._ws_kept) <= 4 * need
    held = {ws.data_ptr() for ws in c._ws_kept}
    assert {ws for _, ws, _ in c._lib.attends} <= held


def test_pools_stay_alive_whatever_becomes_of_the_list(monkeypatch):
    monkeypatch.setattr(pkg, "moe_mxfp4_cache_create", lambda cfg, layers: (0, 1))
    monkeypatch.setattr(pkg, "moe_mxfp4_cache_state_bytes", lambda cache: (0, 4096))
    monkeypatch.setattr(pkg, "moe_mxfp4_cache_destroy", lambda cache: None)
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    layers = [[OnGpu(torch.zeros((5, 2, 16, 64), dtype=torch.bfloat16)) for _ in range(2)] for _ in range(2)]
    refs = [weakref.ref(t) for kv in layers for t in kv]
    c = pkg.KvCache(layers=layers, num_streams=2, max_pages=3)
    layers[1].pop()
    layers.clear()
    gc.collect()
    assert all(r() is not None for r in refs)
    c.close()
