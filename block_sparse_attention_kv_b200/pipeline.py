"""Device buffers + ABI calls for one layer (no arithmetic of its own).

`DeviceLayer` owns the centroid store and the workspaces of one paged layer
and exposes the five steps of the sparse path and the whole-cache calls
(exact decode, shared prefix, eviction); tests, the smoke check and the
benchmark all drive the library through it.
"""

from __future__ import annotations

import torch

from . import abi


def _as_stream(stream, device):
    """torch's Stream for a stream argument: a Stream, a raw handle (0: the
    legacy default stream), an object that holds one as `cuda_stream`, or None."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    handle = stream if isinstance(stream, int) else stream.cuda_stream
    if handle == 0:
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(handle, device=device)


class DeviceLayer:
    def __init__(self, data, budget: int = None, stream=None, block_size=None,
                 fmt: int = abi.ABSP_CENTROIDS_INT4):
        """`data` is a synth.LayerData on a CUDA device; `block_size`
        overrides its per-KV-head block-size table (same cache, other
        blocking).  Calls run on `stream` (None: the current one).  Buffers
        that the layer makes are ordered with it; a caller's own work on other
        streams, and tensors it passes or reads, are the caller's to order.
        One call of a layer at a time: its calls share workspaces."""
        self.data = data
        self.device = data.q.device
        self.budget = int(budget if budget is not None else data.budget)
        self.block_size = list(data.block_size if block_size is None else block_size)
        self.kv = abi.LayerKV(data.seq_lens, data.page_table, data.k_pages, data.v_pages,
                              self.block_size, data.num_q_heads)
        self.cent = abi.alloc_centroids(self.kv, self.device, fmt)
        self.build_ws = None
        dws = abi.absp_decode_workspace_size(self.kv, self.budget)
        self.ws = abi.alloc_workspace(dws, self.device)
        self.kmax = abi.absp_select_capacity(self.kv, self.budget)
        S, Hkv = data.num_seqs, data.num_kv_heads
        self.sel = torch.full((S, Hkv, self.kmax), -1, dtype=torch.int32, device=self.device)
        self.sel_count = torch.zeros((S, Hkv), dtype=torch.int32, device=self.device)
        self.out = torch.zeros_like(data.q)
        self.stream = stream
        self._on = _as_stream(stream, self.device)
        self._behind_current()
        self.full_ws = None       # workspace of the last full_decode
        self._full = []           # the layer's workspaces of full_decode,
        self._graph_full = []     # and those that one captured call uses alone

    def _behind_current(self):
        """The layer's stream waits for what the current stream holds, the
        fills of buffers just made among it."""
        if self._on is not None:
            cur = torch.cuda.current_stream(self.device)
            if cur != self._on:
                self._on.wait_stream(cur)

    def _workspace(self, nbytes: int) -> torch.Tensor:
        """A workspace made, filled and one day reused on the layer's stream."""
        with torch.cuda.stream(self._on):
            return abi.alloc_workspace(nbytes, self.device)

    def _full_workspace(self, nbytes: int) -> torch.Tensor:
        """A workspace of at least `nbytes`.  One that was handed out is never
        dropped: calls in flight and captured graphs go on using it.  In a
        capture that finds none, the fill would be part of the graph, so that
        call gets one of its own."""
        for ws in self._full:
            if ws.numel() >= nbytes:
                return ws
        with torch.cuda.stream(self._on):
            captured = torch.cuda.is_current_stream_capturing()
        ws = self._workspace(nbytes)
        (self._graph_full if captured else self._full).append(ws)
        return ws

    # -- steps 1-2 --------------------------------------------------------
    def build_centroids(self, keep_ws: bool = False, fused: bool = False):
        """Steps 1-2: the separate build and quantize calls, or with `fused`
        the single call; both give the same bits."""
        if self.build_ws is None:
            self.build_ws = self._workspace(abi.absp_build_workspace_size(self.kv))
        if fused:
            abi.absp_build_quantize_centroids(self.kv, self.build_ws, self.cent, self.stream)
        else:
            abi.absp_build_centroids(self.kv, self.build_ws, self.stream)
            abi.absp_quantize_centroids(self.kv, self.build_ws, self.cent, self.stream)
        self.check(self.build_ws)
        if not keep_ws:
            self.build_ws = None

    # -- steps 3-5 --------------------------------------------------------
    def score_select(self, q=None, flags: int = 0):
        q = self.data.q if q is None else q
        if flags:
            abi.absp_score_select_ex(self.kv, self.cent, q, self.budget, self.sel,
                                     self.sel_count, self.ws, flags, self.stream)
        else:
            abi.absp_score_select(self.kv, self.cent, q, self.budget, self.sel,
                                  self.sel_count, self.ws, self.stream)

    def sparse_decode(self, q=None, out=None):
        abi.absp_sparse_decode(self.kv, self.data.q if q is None else q, self.sel,
                               self.sel_count, self.budget, self.out if out is None else out,
                               self.ws, self.stream)

    def decode_step(self, q=None, out=None, flags: int = 0):
        q = self.data.q if q is None else q
        out = self.out if out is None else out
        if flags:
            abi.absp_decode_step_ex(self.kv, self.cent, q, self.budget, out, self.ws, flags,
                                    self.stream)
        else:
            abi.absp_decode_step(self.kv, self.cent, q, self.budget, out, self.ws, self.stream)

    def decode_step_host(self, q_host, out_host, flags: int = 0):
        if flags:
            abi.absp_decode_step_host_ex(self.kv, self.cent, q_host, self.budget, out_host,
                                         self.ws, flags, self.stream)
        else:
            abi.absp_decode_step_host(self.kv, self.cent, q_host, self.budget, out_host,
                                      self.ws, self.stream)

    # -- the whole cache: exact attention, accumulated weights, eviction ------
    def new_weights(self) -> torch.Tensor:
        """Accumulated attention weights of the layer's tokens, all zero, on
        the layer's stream and the current one."""
        d = self.data
        with torch.cuda.stream(self._on):
            w = torch.zeros((d.num_seqs, d.num_kv_heads, self.kv.c.max_pages_per_seq * abi.PAGE_SIZE),
                            dtype=torch.float32, device=self.device)
        if self._on is not None:
            cur = torch.cuda.current_stream(self.device)
            if cur != self._on:
                cur.wait_stream(self._on)
        return w

    def full_decode(self, q=None, out=None, weights=None, shared_tokens: int = 0):
        """Exact attention over every cached token; `weights` (new_weights)
        accumulates the step's attention weights in place.  shared_tokens:
        length of the prefix whose pages all sequences share.  A call of its
        kind ahead of a graph capture lets the captured ones share the layer's
        workspace, which check() reads."""
        need = abi.absp_full_workspace_size(self.kv, shared_tokens, weights is not None)
        self.full_ws = self._full_workspace(need)
        q = self.data.q if q is None else q
        out = self.out if out is None else out
        if shared_tokens:
            abi.absp_shared_decode(self.kv, q, shared_tokens, weights, weights, out, self.full_ws,
                                   self.stream)
        else:
            abi.absp_full_decode(self.kv, q, weights, weights, out, self.full_ws, self.stream)

    def evict(self, weights, keep: int, protect: int = 0, recent: int = 0) -> torch.Tensor:
        """Cut every sequence to `keep` tokens in place: its pages, its
        weights and data.seq_lens.  Returns the positions that stayed, [S][Hkv][keep]
        (-1 behind the last).  The centroids are stale afterwards
        (build_centroids)."""
        d = self.data
        kept = torch.empty((d.num_seqs, d.num_kv_heads, keep), dtype=torch.int32, device=self.device)
        self._behind_current()    # `kept` may be memory that the current stream still uses
        ws = self._workspace(abi.absp_evict_workspace_size(self.kv, keep))
        abi.absp_evict(self.kv, weights, keep, protect, recent, d.page_table, weights, kept,
                       d.seq_lens, ws, self.stream)
        self.check(ws)
        return kept

    # -- device-side faults ------------------------------------------------
    def check(self, ws=None):
        """Waits for the layer's calls and raises a fault that one of them
        reported: in `ws`, or in any workspace of the layer's decode and
        full_decode calls (one fault per call of check; the others stay to be
        read).  Not among them: the workspace of a full_decode that was
        captured before the layer had one, whose error word each replay
        starts anew (`full_ws` after the capture; check(that) after a replay)."""
        for w in [self.ws, *self._full] if ws is None else [ws]:
            st, detail = abi.absp_check_device_error(w, self.stream)
            if st != abi.ABSP_OK:
                raise abi.AbspError(st, f"device fault (unit {detail})")

    # -- views of the centroid store ----------------------------------------
    def codes_of(self, s: int, h: int, n: int) -> torch.Tensor:
        """Centroid rows of (sequence s, KV head h): [n][64] packed INT4
        codes, or [n][256] bytes of bf16 centroids."""
        rb = 256 if self.cent.format == abi.ABSP_CENTROIDS_BF16 else 64
        r0 = abi.absp_centroid_row_offset(self.kv, s, h)
        return self.cent.codes[r0 * rb:(r0 + n) * rb].view(n, rb)

    def params_of(self, s: int, h: int):
        Hkv = self.data.num_kv_heads
        i = (s * Hkv + h) * 128
        return self.cent.scale[i:i + 128], self.cent.zp[i:i + 128]
