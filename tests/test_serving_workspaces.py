"""The workspaces that the binding gives to serving calls without one: whose they are, and on which stream they are
zeroed."""
import ctypes

import pytest
import torch

import int4_weight_only_gemm_gb300 as w


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


@pytest.fixture
def fresh(monkeypatch):
    """No workspaces from calls before."""
    monkeypatch.setattr(w, "_stream_workspaces", {})


def attention_of(lens, heads, kv_heads, seed=0):
    """A call without a workspace, by output: call(**more) -> out."""
    g = torch.Generator("cuda").manual_seed(seed)
    page, d, columns = 16, 128, max(-(-(p + n) // 16) for p, n in lens)
    pages = columns * len(lens)
    q = torch.randn(sum(n for _, n in lens), heads, d, generator=g, device="cuda").to(torch.bfloat16)
    kc, vc = torch.randn(2, pages, kv_heads, page, d, generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(len(lens), columns)
    starts = [0]
    for _, n in lens:
        starts.append(starts[-1] + n)
    args = (q, kc, vc, table, i32(starts), i32([p + n for p, n in lens]), max(n for _, n in lens))
    need = w.w4a16_paged_attention_workspace_bytes(q.shape[0], len(lens), heads, kv_heads, d, args[-1])
    return (lambda **more: w.w4a16_paged_attention(*args, **more)), need


# ---------------------------------------------------------------------------
# the default stream
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("handle", [0, 1])
def test_the_default_stream_has_no_external_stream(monkeypatch, handle):
    monkeypatch.setattr(torch.cuda, "default_stream", lambda index: ("default", index))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: ("external", h, device))
    assert w._stream_of(0, handle) == ("default", 0)
    assert w._stream_of(0, 0x7f00) == ("external", 0x7f00, 0)


@pytest.mark.gpu
def test_first_and_growing_call_zero_on_the_default_stream(fresh, monkeypatch):
    small, _ = attention_of([(2000, 1), (50, 1)], 8, 2)
    large, need = attention_of([(2500, 1)] * 4 + [(700, 200)], 16, 4, seed=1)
    ws = w.new_workspace(need)
    want = small(workspace=ws), large(workspace=ws)
    torch.cuda.synchronize()
    entered, real = [], torch.cuda.stream
    monkeypatch.setattr(torch.cuda, "stream", lambda s: (entered.append(s.cuda_stream), real(s))[1])
    with real(torch.cuda.default_stream()):
        a = torch.randn(4096, 4096, device="cuda")
        for _ in range(8):  # long work ahead of the calls
            a = a @ a * 1e-3
        got = [small(), large(), small(), large()]
    torch.cuda.synchronize()
    assert entered and set(entered) == {0}
    for i, x in enumerate(got):
        assert torch.equal(x, want[i % 2])


# ---------------------------------------------------------------------------
# captures
# ---------------------------------------------------------------------------

class FakeLibrary:
    """What the binding asks of the library to find a call's workspace."""
    capture = 0

    def w4a16_stream_capture_id(self, stream):
        return self.capture


@pytest.fixture
def fake(monkeypatch, fresh):
    lib = FakeLibrary()
    monkeypatch.setattr(w, "_capture_workspaces", {})
    monkeypatch.setattr(w, "load_library", lambda: lib)
    monkeypatch.setattr(w, "_zeroed", lambda nbytes, index, handle: torch.zeros(max(nbytes, 65536), dtype=torch.uint8))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: lib.capture != 0)
    return lib


@pytest.mark.parametrize("stream", [None, "given"])
def test_a_capture_takes_no_eager_buffer(fake, stream):
    get = lambda n=100, handle=0x70: w._serving_workspace(n, 0, stream, handle)  # noqa: E731
    eager = get()
    assert get() is eager and get(handle=0x80) is not eager
    fake.capture = 5
    first = get()
    assert first is not eager and get() is first and get(handle=0x80) is not first
    assert get(100000).numel() >= 100000
    fake.capture = 6
    second = get()
    assert second is not first and second is not eager
    fake.capture = 0
    assert get() is eager


@pytest.mark.gpu
def test_graph_of_a_warmed_stream_beside_its_calls(fresh):
    """A graph captured on a stream with a workspace, replayed on another while the first one runs calls of its own."""
    small, _ = attention_of([(2000, 1), (50, 1), (700, 30)], 8, 2)
    want = small()
    torch.cuda.synchronize()
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    out = torch.zeros_like(want)
    with torch.cuda.stream(s):
        small()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        small(out=out)
        small(out=out)
        assert len(w._capture_workspaces) == 1
    eager = w._stream_workspaces[(0, s.cuda_stream)]
    eager[:65536].fill_(1)  # nothing of the graph reads it
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert (eager[:65536] == 1).all()
    eager[:65536].zero_()
    torch.cuda.synchronize()
    for _ in range(50):
        with torch.cuda.stream(other):
            graph.replay()
        got = small(stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(out, want)


@pytest.mark.gpu
def test_capture_id():
    s = torch.cuda.Stream()
    lib = w.load_library()
    assert lib.w4a16_stream_capture_id(s.cuda_stream) == 0 == lib.w4a16_stream_capture_id(0)
    ids = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            ids.append(lib.w4a16_stream_capture_id(s.cuda_stream))
            torch.zeros(4, device="cuda")
    assert 0 not in ids and ids[0] != ids[1]
    assert lib.w4a16_stream_capture_id(s.cuda_stream) == 0


# ---------------------------------------------------------------------------
# after a timeout
# ---------------------------------------------------------------------------

def test_buffers_go_after_a_timeout(fake):
    fake.w4a16_last_device_status = lambda stream: fake.status
    get = lambda: w._serving_workspace(100, 0, None, 0x70)  # noqa: E731
    first = get()
    for status, kept in ((w.W4A16_OK, True), (w.W4A16_ECUDA, True), (w.W4A16_ETIMEOUT, False)):
        fake.status = status
        assert w.w4a16_last_device_status(0) == status
        assert (get() is first) == kept


@pytest.mark.gpu
def test_attention_after_a_timeout(fresh):
    """The wait that runs out is the self-test's; the buffer's counters stand for what a kernel that gave up leaves."""
    small, _ = attention_of([(2000, 1), (50, 1), (700, 30)], 8, 2)
    want = small().clone()
    torch.cuda.synchronize()
    (spoilt,) = w._stream_workspaces.values()
    spoilt[:65536].fill_(1)
    assert w.load_library().w4a16_selftest_wait_timeout(ctypes.c_longlong(20_000_000), None) == 0  # 20 ms
    assert w.w4a16_last_device_status() == w.W4A16_ETIMEOUT
    assert torch.equal(small(), want)
    assert w.w4a16_last_device_status() == w.W4A16_OK


# ---------------------------------------------------------------------------
# what is kept
# ---------------------------------------------------------------------------

def test_what_the_binding_keeps_is_bounded(fake):
    """A larger call takes the place of its stream's buffer, streams that come and go do not pile up."""
    import gc
    import weakref
    buffers = []
    for i in range(40):
        buffers.append(weakref.ref(w._serving_workspace(65536 << (i % 8), 0, None, 0x70)))
    gc.collect()
    assert len({id(b()) for b in buffers if b() is not None}) == 1
    for i in range(500):
        w._serving_workspace(100, 0, None, 0x1000 + 16 * i)
    assert len(w._stream_workspaces) == 64 and (0, 0x1000 + 16 * 499) in w._stream_workspaces


def test_sizes_kept_are_bounded(monkeypatch):
    monkeypatch.setattr(w, "_need_cache", {})
    for i in range(10000):
        assert w._remember(("gemm", i), 2 * i) == 2 * i
        assert len(w._need_cache) <= 4096


@pytest.mark.gpu
def test_sizes_asked_once_for_all_steps(fresh, monkeypatch):
    monkeypatch.setattr(w, "_need_cache", {})
    for lens in ([(20, 1)], [(30, 1)] * 5, [(9, 1), (800, 1)]):
        attention_of(lens, 8, 2)[0]()
    assert len(w._need_cache) == 1


@pytest.mark.gpu
def test_workspaces_that_are_none(fresh):
    """Host memory, or every other byte of a buffer, is not handed to a kernel."""
    small, need = attention_of([(20, 1)], 8, 2)
    logits, noise = torch.randn(3, 5000, device="cuda"), torch.ones(3, 5000, device="cuda")
    k = i32([5, 5, 5])
    for bad in (torch.zeros(max(need, 1 << 20), dtype=torch.uint8), w.new_workspace(1 << 21)[::2], 0):
        with pytest.raises(ValueError):
            small(workspace=bad)
        with pytest.raises(ValueError):
            w.w4a16_sample(logits, noise, top_k=k, workspace=bad)
