"""A layer with a stream of its own: the buffers it makes are ordered with the
calls that use them, and a workspace that was handed out stays.

The CPU tests run DeviceLayer's host code over fake streams that log every
fill, wait and call; the GPU tests hold the current stream back so that work
left unordered would show in the results.
"""

import contextlib
import types

import numpy as np
import pytest
import torch

from block_sparse_attention_kv_b200 import build as absp_build
from block_sparse_attention_kv_b200 import synth
from oracle import cache_oracle as CO

LAYER, CURRENT = "layer", "current"


class FakeStream:
    def __init__(self, name, log):
        self.name, self.log, self.cuda_stream = name, log, 7

    def wait_stream(self, other):
        self.log.append(("wait", self.name, other.name))


class FakeCuda:
    """torch.cuda's streams, with a log of (event, stream, detail)."""

    def __init__(self, monkeypatch, abi, capturing=False):
        self.log, self.keep = [], []
        self.layer, self.current = FakeStream(LAYER, self.log), FakeStream(CURRENT, self.log)
        self.now = self.current
        cuda = torch.cuda

        @contextlib.contextmanager
        def stream(s):
            old, self.now = self.now, self.now if s is None else s
            yield
            self.now = old

        monkeypatch.setattr(cuda, "stream", stream)
        monkeypatch.setattr(cuda, "current_stream", lambda device=None: self.now)
        monkeypatch.setattr(cuda, "is_current_stream_capturing", lambda: capturing)
        zeros, empty, full, zeros_like = torch.zeros, torch.empty, torch.full, torch.zeros_like
        for name, f in (("zeros", zeros), ("empty", empty), ("full", full), ("zeros_like", zeros_like)):
            def made(*a, _f=f, **kw):
                t = _f(*a, **kw)
                self.keep.append(t)
                self.log.append(("made", self.now.name, t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()))
                return t
            monkeypatch.setattr(torch, name, made)

        def use(*tensors):
            for t in tensors:
                if t is not None:
                    self.log.append(("use", LAYER, t.data_ptr()))

        monkeypatch.setattr(abi, "absp_full_decode",
                            lambda kv, q, wi, wo, out, ws, st: use(wo, out, ws))
        monkeypatch.setattr(abi, "absp_shared_decode",
                            lambda kv, q, n, wi, wo, out, ws, st: use(wo, out, ws))
        monkeypatch.setattr(abi, "absp_evict",
                            lambda kv, wi, k, p, r, dst, wo, kept, lens, ws, st: use(wo, kept, ws))
        monkeypatch.setattr(abi, "absp_build_centroids", lambda kv, ws, st: use(ws))
        monkeypatch.setattr(abi, "absp_quantize_centroids", lambda kv, ws, c, st: use(ws, c.codes))
        monkeypatch.setattr(abi, "absp_decode_step", lambda kv, c, q, b, out, ws, st: use(out, ws))
        monkeypatch.setattr(abi, "absp_check_device_error", lambda ws, st: (use(ws), (0, 0))[1])

    def assert_ordered(self):
        """Every use on the layer's stream comes behind the making of its buffer."""
        uses = 0
        for i, e in enumerate(self.log):
            if e[0] != "use":
                continue
            uses += 1
            j, owner = [(j, m[1]) for j, m in enumerate(self.log[:i])
                        if m[0] == "made" and m[2] <= e[2] < max(m[3], m[2] + 1)][-1]
            if owner != LAYER:
                assert ("wait", LAYER, CURRENT) in self.log[j:i], ("use before its buffer is filled", e)
        assert uses


@pytest.fixture(scope="module")
def lib():
    absp_build.build()
    from block_sparse_attention_kv_b200 import abi, pipeline
    return abi, pipeline


def _data(device="cpu", lens=(300, 90), shared=64, seed=5):
    w = synth.custom("streams", len(lens), 8, 2, list(lens), [16, 32], 256, seed=seed)
    d = synth.make_layer(w, 0, device)
    d.page_table[1:, :shared // 16] = d.page_table[:1, :shared // 16]
    if device == "cpu":     # the layer checks want pools on 256 bytes, as device memory is
        d = synth.replace(d, plan=None, k_pages=_aligned(d.k_pages), v_pages=_aligned(d.v_pages))
    return d


def _aligned(t):
    buf = torch.empty(t.numel() + 128, dtype=t.dtype)
    off = (-buf.data_ptr()) % 256 // t.element_size()
    return buf[off:off + t.numel()].view(t.shape).copy_(t)


def _calls(dl):
    dl.full_decode()
    w = dl.new_weights()
    dl.full_decode(weights=w)
    dl.full_decode(shared_tokens=64)
    dl.full_decode(weights=w, shared_tokens=64)
    dl.full_decode()
    dl.evict(w, 40, protect=16)
    dl.build_centroids()
    dl.decode_step()


def test_uses_come_behind_fills(lib, monkeypatch):
    abi, pipeline = lib
    d = _data()
    f = FakeCuda(monkeypatch, abi)
    monkeypatch.setattr(pipeline, "_as_stream", lambda stream, device: stream)
    _calls(pipeline.DeviceLayer(d, stream=f.layer))
    f.assert_ordered()
    # what a caller does next on its own stream comes behind the weights' fill
    made = [i for i, e in enumerate(f.log) if e[0] == "made" and e[1] == LAYER]
    assert not made or ("wait", CURRENT, LAYER) in f.log


@pytest.mark.parametrize("capturing", [False, True])
def test_a_workspace_in_use_is_never_dropped(lib, monkeypatch, capturing):
    abi, pipeline = lib
    d = _data()
    dl = None
    FakeCuda(monkeypatch, abi)
    dl = pipeline.DeviceLayer(d, stream=None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    import weakref
    seen = []
    w = dl.new_weights()
    for kw in ({}, {"weights": w}, {"shared_tokens": 64}, {"weights": w, "shared_tokens": 64}, {}):
        dl.full_decode(**kw)
        need = abi.absp_full_workspace_size(dl.kv, kw.get("shared_tokens", 0), "weights" in kw)
        assert dl.full_ws.numel() >= need
        seen.append((dl.full_ws.data_ptr(), weakref.ref(dl.full_ws)))
        assert all(r() is not None for _, r in seen)
    if capturing:     # nothing that a graph fills serves another call
        assert len({p for p, _ in seen}) == len(seen)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
        dl.full_decode()
        assert dl.full_ws.data_ptr() not in {p for p, _ in seen}
    else:             # the largest call's workspace serves the smaller ones
        dl.full_decode(weights=w, shared_tokens=64)
        big = dl.full_ws.data_ptr()
        dl.full_decode(weights=w, shared_tokens=64)
        assert dl.full_ws.data_ptr() == big and len({p for p, _ in seen}) <= 4


def test_check_reads_every_workspace_of_the_layer(lib, monkeypatch):
    abi, pipeline = lib
    d = _data()
    FakeCuda(monkeypatch, abi)
    dl = pipeline.DeviceLayer(d)
    words = {}

    def read(ws, stream):                 # reads a workspace's error word and clears it
        return words.pop(ws.data_ptr(), (abi.ABSP_OK, 0))

    monkeypatch.setattr(abi, "absp_check_device_error", read)
    dl.check()
    dl.full_decode()
    small = dl.full_ws
    dl.full_decode(shared_tokens=64)
    assert dl.full_ws.data_ptr() != small.data_ptr()
    for ws in (dl.ws, small, dl.full_ws):  # a fault from before the layer grew among them
        words[ws.data_ptr()] = (abi.ABSP_ERR_DEVICE_FAULT, 3)
        with pytest.raises(abi.AbspError) as e:
            dl.check()
        assert e.value.status == abi.ABSP_ERR_DEVICE_FAULT
        dl.check()
    for ws in (dl.ws, small, dl.full_ws):  # none is cleared unread
        words[ws.data_ptr()] = (abi.ABSP_ERR_TIMEOUT, 1)
    for _ in range(3):
        with pytest.raises(abi.AbspError):
            dl.check()
    dl.check()
    words[small.data_ptr()] = (abi.ABSP_ERR_DEVICE_FAULT, 0)
    dl.check(dl.full_ws)                  # one workspace alone
    assert words


# -------------------------------------------------------------------- GPU --

def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _hold_current():
    """Keeps the current stream busy for some 30 ms."""
    torch.cuda._sleep(60_000_000)


def _dirty(nbytes):
    """Memory of this size that the current stream has used and freed, all ones."""
    for _ in range(4):
        torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("given", ["stream", "handle", "holder"])
@pytest.mark.parametrize("wide", [False, True])
def test_side_stream_results(lib, given, wide):
    abi, pipeline = lib
    d = _data("cuda", (900, 700, 330), 256)
    if wide:
        pad = torch.full((3, 600 - d.page_table.shape[1]), -1, dtype=torch.int32, device="cuda")
        d = synth.replace(d, plan=None, page_table=torch.cat([d.page_table, pad], 1).contiguous())
    table, lens = d.page_table.cpu().numpy(), [900, 700, 330]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    _dirty(64 << 20)
    _hold_current()
    holder = types.SimpleNamespace(cuda_stream=st.cuda_stream)
    dl = pipeline.DeviceLayer(d, stream={"stream": st, "handle": st.cuda_stream, "holder": holder}[given])
    q, kp, vp = _f64(d.q), _f64(d.k_pages), _f64(d.v_pages)
    total = np.zeros((3, 2, d.page_table.shape[1] * 16))
    w = None
    for i, (shared, weigh) in enumerate([(0, False), (256, False), (0, True), (256, True), (0, False)]):
        if weigh and w is None:
            _hold_current()
            w = dl.new_weights()
        _dirty(32 << 20)
        _hold_current()                       # a fill on this stream would come late
        dl.full_decode(weights=w if weigh else None, shared_tokens=shared)
        st.synchronize()
        out, ww, ob, wb = CO.attention(q, kp, vp, table, lens, shared)
        got = _f64(dl.out)
        assert (np.abs(got - out) <= ob).all(), i
        torch.cuda.synchronize()              # what came late has come
        dl.check(dl.full_ws)
        if weigh:
            total[:, :, shared:] += ww[:, :, shared:]
            assert np.allclose(w.cpu().numpy(), total, rtol=1e-5, atol=1e-30)
    before = w.cpu().numpy().copy()
    bits = lambda t: t.view(torch.int16).cpu().numpy()  # noqa: E731
    want = CO.evict(before, lens, 400, 256, 64, bits(d.k_pages), bits(d.v_pages), table, table, before)
    _hold_current()
    kept = dl.evict(w, 400, protect=256, recent=64)
    torch.cuda.synchronize()
    for got, exp in zip((bits(d.k_pages), bits(d.v_pages), w.cpu().numpy(), kept.cpu().numpy(),
                         d.seq_lens.cpu().numpy()), want):
        assert np.array_equal(got, exp)


@pytest.mark.gpu
def test_default_stream_by_its_handle(lib):
    abi, pipeline = lib
    d = _data("cuda")
    dl = pipeline.DeviceLayer(d, stream=0)
    dl.full_decode()
    a = dl.out.clone()
    other = pipeline.DeviceLayer(d)
    other.full_decode()
    dl.check(dl.full_ws)
    assert torch.equal(a.view(torch.int16), other.out.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("warm", [False, True])
def test_a_graph_outlives_a_growing_layer(lib, warm):
    """A captured call goes on working while the layer meets larger calls."""
    abi, pipeline = lib
    d = _data("cuda", (900, 700, 330), 256)
    pad = torch.full((3, 600 - d.page_table.shape[1]), -1, dtype=torch.int32, device="cuda")
    d = synth.replace(d, plan=None, page_table=torch.cat([d.page_table, pad], 1).contiguous())
    st = torch.cuda.Stream()
    dl = pipeline.DeviceLayer(d, stream=st)
    st.synchronize()
    torch.cuda.synchronize()
    ref = torch.zeros_like(d.q)
    if warm:
        dl.full_decode(out=ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        dl.full_decode()
    graph_ws = dl.full_ws
    dl.full_decode(out=ref)                      # an eager call before any replay
    st.synchronize()
    dl.check(dl.full_ws)
    w = dl.new_weights()
    for shared in (0, 256, 0, 256):
        dl.full_decode(weights=w, shared_tokens=shared)
        dl.check(dl.full_ws)
        _dirty(64 << 20)                         # freed memory would be written over
        torch.cuda.synchronize()
        dl.out.fill_(3.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g.replay()
        st.synchronize()
        assert torch.equal(dl.out.view(torch.int16), ref.view(torch.int16))
        dl.check(graph_ws)


@pytest.mark.gpu
def test_check_raises_a_fault_of_the_whole_cache_call(lib):
    abi, pipeline = lib
    d = _data("cuda")
    dl = pipeline.DeviceLayer(d)
    dl.full_decode()
    dl.check()
    page = int(d.page_table[1, 4])
    d.page_table[1, 4] = 1 << 20
    dl.full_decode()
    dl.full_decode(weights=dl.new_weights(), shared_tokens=64)   # another workspace, the same fault
    for _ in range(2):
        with pytest.raises(abi.AbspError) as e:
            dl.check()
        assert e.value.status == abi.ABSP_ERR_DEVICE_FAULT
    dl.check()
    d.page_table[1, 4] = page
    dl.full_decode()
    dl.check()
