"""User-facing API: one object that owns the caches and workspace of a batch of
sequences and runs the hot path chunk by chunk through the C ABI.

``SparseGQA.forward`` (one call: a decode step or one chunk) and ``prefill``
(all chunks) take device tensors; ``forward_host`` takes pinned host tensors
and copies them in and the result out (the end-to-end path).  ``evict`` drops
the blocks with the least accumulated attention weight.  All arithmetic runs
in ``libsgqa.so``.

With ``kv_dtype="e4m3"`` K and V are held in 8 bits: the caches ``k`` and ``v``
give way to ``kv8``, ``kv_scale`` and ``tail``, and every call takes the K/V rows
of its own positions (``k=``, ``v=``), which it appends.  ``track_weights``
accumulates each block's attention weight in ``acc`` along the way.
"""
from __future__ import annotations

import contextlib

import torch

from . import binding as Bd


def _on(stream):
    """Context in which torch's own work runs on the given stream, or the current one."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


class SparseGQA:
    def __init__(self, params: Bd.Params, num_seqs: int, capacity: int, chunk: int, device,
                 keep_merged_f32: bool = False, kv_dtype: str = "bf16", track_weights: bool = False):
        if kv_dtype not in ("bf16", "e4m3"):
            raise ValueError(f"kv_dtype must be 'bf16' or 'e4m3', not {kv_dtype!r}")
        if track_weights and kv_dtype != "e4m3":
            raise ValueError("attention weights are accumulated over the 8-bit cache (kv_dtype='e4m3') only")
        if kv_dtype == "e4m3" and (params.block_size != 8 or capacity % 8):
            raise ValueError("kv_dtype='e4m3' needs block_size 8 and a capacity that is a multiple of 8")
        self.p = params
        self.kv_dtype = kv_dtype
        self.S = num_seqs
        self.cap = capacity
        self.chunk = chunk
        self.device = torch.device(device)
        G, D, Di, B = params.num_kv_groups, params.head_dim, params.idx_dim, params.block_size
        in_dt = torch.float32 if params.merge_in_f32 else torch.bfloat16
        self.kp = torch.empty((num_seqs, capacity, Di), dtype=in_dt, device=device)
        self.c = torch.empty((num_seqs, capacity, Di), dtype=in_dt, device=device)
        self.acc = None
        if kv_dtype == "e4m3":
            blocks = capacity // B
            self.kv8 = torch.zeros((num_seqs, blocks, G, 2, B, D), dtype=torch.uint8, device=device)
            self.kv_scale = torch.ones((num_seqs, blocks, G, 2), dtype=torch.float32, device=device)
            self.tail = torch.zeros((num_seqs, 2, B, G, D), dtype=torch.bfloat16, device=device)
            if track_weights:
                self.acc = torch.zeros((num_seqs, blocks), dtype=torch.int64, device=device)
        else:
            self.k = torch.empty((num_seqs, capacity, G, D), dtype=torch.bfloat16, device=device)
            self.v = torch.empty((num_seqs, capacity, G, D), dtype=torch.bfloat16, device=device)
        self.store = torch.zeros((num_seqs, capacity // B, Di), dtype=torch.uint8, device=device)
        self.merged = (torch.zeros((num_seqs, capacity // B, Di), dtype=torch.float32, device=device)
                       if keep_merged_f32 else None)
        alloc = Bd.alloc_workspace_q8 if kv_dtype == "e4m3" else Bd.alloc_workspace
        self.ws = alloc(params, num_seqs, chunk, capacity, device)
        self.evicted = 0        # blocks of a sequence evicted so far
        self.pos_count = 0      # slots whose original block number `pos` holds
        self.pos = self._evict_ws = None
        # 8-bit cache: tokens it holds after the last call; None: not known (nothing called yet, a cache filled by
        # hand, a captured call), and where a call begins is not checked
        self.length = None

    def _check_tail(self, at):
        """The 8-bit cache's incomplete block is quantised from its BF16 rows; tail holds those of one block only."""
        if at % 8 and self.length is not None and not (at // 8 == self.length // 8 and at <= self.length):
            raise ValueError(f"position {at} lies inside a block whose rows are not in tail, which holds those of positions "
                             f"{self.length // 8 * 8} to {self.length - 1}: go back to a multiple of 8 and append from there "
                             "(or set .length, if the cache was filled outside these calls)")

    def forward(self, q_pos0, q, idx_q, idx_w, sel, sel_count, out, cache_len=None, stream=None, gate=None, k=None,
                v=None):
        """One call of the hot path for queries [q_pos0, q_pos0 + nq) (nq <= chunk).

        Every tensor is contiguous with the layouts of include/sgqa.h; gate
        ([S, nq, G*Hg] bf16 logits) applies the head-wise sigmoid output gate.
        With the 8-bit cache k and v ([S, nq, G, D] bf16) are the call's own
        rows, and the cache holds q_pos0 + nq tokens after it.  A call may take
        back tokens (drafts that were not accepted) by a smaller q_pos0: one
        inside the block that the last call ended in, or a multiple of 8, from
        which that block's rows are given again; others are refused.  Tracked
        weights keep what the tokens taken back have added.
        """
        nq = q.shape[1]
        if self.kv_dtype == "e4m3":
            if k is None or v is None:
                raise ValueError("the 8-bit cache takes the call's K/V rows: forward(..., k=, v=)")
            if cache_len is not None and cache_len != q_pos0 + nq:
                raise ValueError("the 8-bit cache ends with the call's own rows: cache_len is q_pos0 + nq")
            if nq:
                self._check_tail(q_pos0)
            before, self.length = self.length, None
            Bd.sgqa_forward_q8(self.p, self.S, q_pos0, nq, q, idx_q, idx_w, self.cap, self.kp, self.c, k, v, self.tail,
                               self.kv8, self.kv_scale, self.merged, self.store, sel, sel_count, out, self.ws, gate=gate,
                               acc=self.acc, stream=stream)
            if nq == 0:
                self.length = before
            elif not (self.device.type == "cuda" and torch.cuda.is_current_stream_capturing()):
                self.length = q_pos0 + nq
            return
        if k is not None or v is not None:
            raise ValueError("with BF16 caches the call's K/V rows are already in .k and .v")
        clen = self.cap if cache_len is None else cache_len
        if gate is None:
            Bd.sgqa_forward(self.p, self.S, q_pos0, nq, q, idx_q, idx_w, self.cap, clen, self.kp, self.c, self.k,
                            self.v, self.merged, self.store, sel, sel_count, out, self.ws, stream)
        else:
            Bd.sgqa_forward_gated(self.p, self.S, q_pos0, nq, q, idx_q, idx_w, self.cap, clen, self.kp, self.c,
                                  self.k, self.v, self.merged, self.store, sel, sel_count, gate, out, self.ws, stream)

    def reset(self, stream=None):
        """Forget the accumulated weights and evictions: the next call starts new sequences at position 0.
        The weights are cleared on the given stream, which should be the calls' (default: the current one)."""
        self.evicted = self.pos_count = 0
        self.length = None
        if self.acc is not None:
            with _on(stream):
                self.acc.zero_()

    def evict(self, cache_len, keep, first=0, recent=0, acc=None, stream=None):
        """Keep `keep` of the complete blocks of cache_len tokens; returns the new cache length.

        The blocks with the largest accumulated weight stay (acc: [S, capacity / B]
        int64, rearranged in place; where weights are tracked it is those), and in any
        case the `first` first and `recent` last blocks of the sequence.  The
        next call's q_pos0 is the returned length.  The counts that go with an
        eviction are the host's: a captured one is replayed once at most.
        """
        B = self.p.block_size
        if acc is not None and self.acc is not None and acc is not self.acc:
            raise ValueError("evict goes by the tracked weights here: with others those would keep the blocks' old slots")
        acc = self.acc if acc is None else acc
        if acc is None:
            raise ValueError("evict needs accumulated weights: track_weights or acc=")
        if self.kv_dtype == "e4m3":
            self._check_tail(cache_len)
        if self.pos is None:
            # on the call's stream: memory that another stream's work still uses is not handed to it
            with _on(stream):
                self._evict_ws = Bd.alloc_evict_workspace(self.p, self.S, self.cap, self.device)
                self.pos = torch.empty((self.S, self.cap // B), dtype=torch.int32, device=self.device)
        kv = [self.kv8, self.kv_scale] if self.kv_dtype == "e4m3" else [self.k, self.v]
        arrays = kv + [self.store] + ([self.merged] if self.merged is not None else [])
        n = cache_len // B
        Bd.sgqa_evict(self.p, self.S, self.cap, cache_len, keep, first, recent, acc, self.pos,
                      self.pos_count, self.evicted, acc, self.pos, arrays, self._evict_ws,
                      tail_arrays=[self.kp, self.c], stream=stream)
        self.evicted += n - keep
        self.pos_count = keep
        if self.length is not None:
            self.length = keep * B + cache_len % B
        return keep * B + cache_len % B

    def prefill(self, q, idx_q, idx_w, out, sel=None, sel_count=None, q_pos0=0, stream=None, gate=None, k=None, v=None):
        """Chunked prefill of all queries in q ([S, N, G*Hg, D]); caches already hold their K/V
        (the 8-bit cache takes all rows as k and v, [S, N, G, D], and appends them chunk by chunk).

        A chunk of a batch of several sequences is not contiguous in q: it is
        copied into a contiguous tensor before the call.
        """
        S, N = q.shape[0], q.shape[1]
        if self.device.type != "cuda":  # host-side use (tests with a stand-in library)
            self._prefill_chunks(q, idx_q, idx_w, out, sel, sel_count, q_pos0, stream, gate, S, N, k, v)
            return
        st = torch.cuda.current_stream(self.device) if stream is None else stream
        with torch.cuda.stream(st):  # the chunk copies run on the calls' stream
            self._prefill_chunks(q, idx_q, idx_w, out, sel, sel_count, q_pos0, st, gate, S, N, k, v)

    def _prefill_chunks(self, q, idx_q, idx_w, out, sel, sel_count, q_pos0, stream, gate, S, N, k, v):
        G, topk = self.p.num_kv_groups, self.p.topk
        for c0 in range(0, N, self.chunk):
            n = min(self.chunk, N - c0)
            s_sel = sel[:, c0:c0 + n] if sel is not None and S == 1 else torch.empty(
                (S, n, G, topk), dtype=torch.int32, device=self.device)
            s_cnt = sel_count[:, c0:c0 + n] if sel_count is not None and S == 1 else torch.empty(
                (S, n, G), dtype=torch.int32, device=self.device)
            o = out[:, c0:c0 + n] if S == 1 else torch.empty((S, n) + tuple(out.shape[2:]),
                                                             dtype=out.dtype, device=self.device)
            rows = {x: t[:, c0:c0 + n].contiguous() for x, t in (("k", k), ("v", v)) if t is not None}
            self.forward(q_pos0 + c0, q[:, c0:c0 + n].contiguous(), idx_q[:, c0:c0 + n].contiguous(),
                         idx_w[:, c0:c0 + n].contiguous(), s_sel, s_cnt, o, stream=stream,
                         gate=None if gate is None else gate[:, c0:c0 + n].contiguous(), **rows)
            if S != 1:
                out[:, c0:c0 + n] = o
                if sel is not None:
                    sel[:, c0:c0 + n] = s_sel
                if sel_count is not None:
                    sel_count[:, c0:c0 + n] = s_cnt

    def forward_host(self, host: dict, out_host: torch.Tensor, stream=None):
        """End to end from pinned host memory: copy the inputs in, run, copy the output out.

        host holds pinned tensors with the cache layouts (kp, c, k, v) and the query
        layouts (q, idx_q, idx_w) of a full prefill; out_host receives [S, N, G*Hg, D].
        The copies are pipelined with the chunks: chunk c needs only the cache
        positions before its last query and its own queries, so while chunk c
        runs, chunk c+1's inputs are copied in on one stream and chunk c-1's
        output is copied out on another (the two PCIe directions run at once).
        Work is enqueued only; the given stream (default: the current one) waits
        for the last copy out.  Returns (bytes copied host->device, bytes copied
        device->host).
        """
        cur = torch.cuda.current_stream(self.device) if stream is None else stream
        if not hasattr(self, "_copy_streams"):
            self._copy_streams = (torch.cuda.Stream(device=self.device), torch.cuda.Stream(device=self.device))
        h2d_s, d2h_s = self._copy_streams
        S, N = host["q"].shape[0], host["q"].shape[1]
        G, k = self.p.num_kv_groups, self.p.topk
        # copied straight into the caches, and rows that a call takes (the 8-bit cache's K/V among them)
        cached, rows = (("kp", "c"), ("q", "idx_q", "idx_w", "k", "v")) if self.kv_dtype == "e4m3" else \
            (("kp", "c", "k", "v"), ("q", "idx_q", "idx_w"))
        with torch.cuda.stream(cur):  # the buffers belong to the calls' stream (and the two copy streams below)
            dq = {n: torch.empty(host[n].shape, dtype=host[n].dtype, device=self.device) for n in rows}
            out = torch.empty(out_host.shape, dtype=out_host.dtype, device=self.device)
            sel = torch.empty((S, self.chunk, G, k), dtype=torch.int32, device=self.device)
            cnt = torch.empty((S, self.chunk, G), dtype=torch.int32, device=self.device)
        h2d_s.wait_stream(cur)
        d2h_s.wait_stream(cur)
        for c0 in range(0, N, self.chunk):
            n = min(self.chunk, N - c0)
            with torch.cuda.stream(h2d_s):
                for s in range(S):
                    for name in cached:
                        getattr(self, name)[s, c0:c0 + n].copy_(host[name][s, c0:c0 + n], non_blocking=True)
                    for name in rows:
                        dq[name][s, c0:c0 + n].copy_(host[name][s, c0:c0 + n], non_blocking=True)
                ready = torch.cuda.Event()
                ready.record(h2d_s)
            cur.wait_event(ready)
            with torch.cuda.stream(cur):  # the chunk's own copies run on the calls' stream
                o = out[:, c0:c0 + n] if S == 1 else torch.empty((S, n) + tuple(out.shape[2:]), dtype=out.dtype,
                                                                 device=self.device)
                if S == 1 or n == self.chunk:
                    c_sel, c_cnt = sel[:, :n], cnt[:, :n]
                else:  # a short last chunk of several sequences: contiguous scratch of its own
                    c_sel = torch.empty((S, n, G, k), dtype=torch.int32, device=self.device)
                    c_cnt = torch.empty((S, n, G), dtype=torch.int32, device=self.device)
                self.forward(c0, dq["q"][:, c0:c0 + n].contiguous(), dq["idx_q"][:, c0:c0 + n].contiguous(),
                             dq["idx_w"][:, c0:c0 + n].contiguous(), c_sel, c_cnt, o, stream=cur,
                             **{x: dq[x][:, c0:c0 + n].contiguous() for x in rows[3:]})
                if S != 1:
                    out[:, c0:c0 + n] = o
            done = torch.cuda.Event()
            done.record(cur)
            d2h_s.wait_event(done)
            with torch.cuda.stream(d2h_s):
                for s in range(S):
                    out_host[s, c0:c0 + n].copy_(out[s, c0:c0 + n], non_blocking=True)
        for t in list(dq.values()) + [out, sel, cnt]:
            t.record_stream(h2d_s)
            t.record_stream(d2h_s)
        cur.wait_stream(d2h_s)
        h2d = sum(host[n].numel() * host[n].element_size() for n in ("kp", "c", "k", "v", "q", "idx_q", "idx_w"))
        return h2d, out_host.numel() * out_host.element_size()
