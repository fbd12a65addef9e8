"""PRR decode state for one attention layer: device buffers, streams and the step call.

Torch is used for device memory, streams, events and CUDA graphs only; every step of
the path (summaries, selection, speculation, repair, merge, EMA prediction) runs in
libprr_b200.so through the C ABI.
"""
from __future__ import annotations

import contextlib
import dataclasses
from typing import Optional

import torch

from . import _abi
from ._abi import Dims


class PRRDecoder:
    """Caller-owned state of the PRR decode step (PRR abstract / method summary: EMA
    predictor, speculative attention overlapped with selection, repair + LSE merge).

    Buffers (row-major), with S = selections per sequence (Hkv; Hq under per-head
    selection):  k_cache/v_cache [B][Hkv][cap][d] bf16, seq_lens [B] int32,
    summ [B][Hkv][maxnb][2][d] bf16, ema [B][S][maxnb] fp64, pred double buffer
    [2][B][S][P] int32, sel/missed [B][S][K], n_missed [B][S], keep [B][S][P],
    speculative partials [B][Hq][P](+[d]) fp32, out [B][Hq][d] fp32, lse [B][Hq] fp32.
    """

    def __init__(self, dims: Dims, device: Optional[torch.device] = None,
                 block_table: Optional[torch.Tensor] = None, rep_offsets: Optional[torch.Tensor] = None,
                 empty: bool = False):
        """dims.pages > 0 makes the KV cache a paged pool [pages][Hkv][bs][d];
        `block_table` (int32 [B][maxnb], page of block j of sequence b) then defaults to
        block j of sequence b in page b*maxnb + j; with `empty` no sequence holds a page,
        and reserve() hands them out.  The representative-key selector
        takes `rep_offsets` (uint8 [B][Hkv][maxnb][n_rep], offsets of each block's
        representative tokens inside the block).  Both are copied: reserve(), fork(),
        release() and compact() write the decoder's own."""
        if not torch.cuda.is_available():
            raise RuntimeError("PRRDecoder needs a CUDA device")
        _abi.load()
        self.device = torch.device(device or "cuda")
        dev = self.device
        B, Hq, Hkv, d, cap, K, P = dims.B, dims.Hq, dims.Hkv, dims.d, dims.cap_tokens, dims.K, dims.P
        S = dims.sel_heads  # selections per sequence (per-unit arrays are [B][S][...])
        maxnb = dims.maxnb
        self.block_table = None
        self.page_refs = None
        if empty and (dims.pages == 0 or block_table is not None):
            raise ValueError("empty starts a paged cache without a block table")
        if dims.pages > 0:
            if empty:
                block_table = torch.full((B, maxnb), -1, dtype=torch.int32)
            elif block_table is None:
                block_table = torch.arange(B * maxnb, dtype=torch.int32).view(B, maxnb)
            self.block_table = block_table.to(device=dev, dtype=torch.int32, copy=True).contiguous()
            self.table_host = self.block_table.cpu().numpy()
            self.page_refs = self._count_refs(dims.pages).to(dev)
            dims = dataclasses.replace(dims, block_table=self.block_table.data_ptr())
            self.k_cache = torch.zeros((dims.pages, Hkv, dims.bs, d), dtype=torch.bfloat16, device=dev)
        else:
            self.k_cache = torch.zeros((B, Hkv, cap, d), dtype=torch.bfloat16, device=dev)
        self.rep_offsets = None
        if dims.selector == "representative":
            if rep_offsets is None or tuple(rep_offsets.shape) != (B, Hkv, maxnb, dims.n_rep):
                raise ValueError("the representative selector needs rep_offsets [B][Hkv][maxnb][n_rep]")
            self.rep_offsets = rep_offsets.to(device=dev, dtype=torch.uint8, copy=True).contiguous()
            dims = dataclasses.replace(dims, rep_offsets=self.rep_offsets.data_ptr())
        self.dims = dims
        self.v_cache = torch.zeros_like(self.k_cache)
        self.seq_lens = torch.zeros((B,), dtype=torch.int32, device=dev)
        self.summ = torch.zeros((B, Hkv, maxnb, 2, d), dtype=torch.bfloat16, device=dev)
        self.ema = torch.zeros((B, S, maxnb), dtype=torch.float64, device=dev)
        self.pred_buf = torch.full((2, B, S, max(P, 1)), -1, dtype=torch.int32, device=dev)
        self.sel = torch.full((B, S, K), -1, dtype=torch.int32, device=dev)
        self.missed = torch.full((B, S, K), -1, dtype=torch.int32, device=dev)
        self.n_missed = torch.zeros((B, S), dtype=torch.int32, device=dev)
        self.keep = torch.zeros((B, S, max(P, 1)), dtype=torch.uint8, device=dev)
        self.part_m = torch.zeros((B, Hq, max(P, 1)), dtype=torch.float32, device=dev)
        self.part_l = torch.zeros((B, Hq, max(P, 1)), dtype=torch.float32, device=dev)
        self.part_O = torch.zeros((B, Hq, max(P, 1), d), dtype=torch.float32, device=dev)
        # Per-step I/O in two contiguous buffers, so that a caller moves each direction
        # with one copy: io_in = [q | k_new | v_new] (bf16), io_out = [out | lse] (fp32).
        nq, nkv = B * Hq * d, B * Hkv * d
        self.io_in = torch.zeros((nq + 2 * nkv,), dtype=torch.bfloat16, device=dev)
        self.q = self.io_in[:nq].view(B, Hq, d)
        self.k_new = self.io_in[nq:nq + nkv].view(B, Hkv, d)
        self.v_new = self.io_in[nq + nkv:].view(B, Hkv, d)
        self.io_out = torch.zeros((B * Hq * (d + 1),), dtype=torch.float32, device=dev)
        self.out = self.io_out[:B * Hq * d].view(B, Hq, d)
        self.lse = self.io_out[B * Hq * d:].view(B, Hq)
        nbytes = _abi.prr_workspace_bytes(dims)
        if nbytes == 0:
            raise ValueError(f"unsupported dims {dims}")
        self.ws = torch.zeros((nbytes,), dtype=torch.uint8, device=dev)
        lo, hi = torch.cuda.Stream.priority_range()
        self.select_stream = torch.cuda.Stream(device=dev, priority=hi)
        self.spec_stream = torch.cuda.Stream(device=dev, priority=lo)
        # stream-ordering events of the step (torch creates a handle on first record)
        self.step_events = {name: torch.cuda.Event() for name in _abi.STEP_EVENTS}
        for ev in self.step_events.values():
            ev.record(self.select_stream)
        self.parity = 0  # which pred buffer holds Pred_t
        self.fused_parity = 0  # control-word copy of the next fused launch
        self.trace = None      # optional per-item timeline of fused launches (enable_trace)
        self.stats = None      # optional step counters (enable_stats)
        self.serve_ws = None   # workspace of the calls around the step (_serving)
        self.serve_captured = False  # a captured graph works in it
        self.serve_kept = []   # earlier ones that captured graphs work in
        if empty and P > 0:    # what the zero state predicts, of the blocks that the sequence then has
            self.pred_buf.copy_(torch.arange(P, dtype=torch.int32, device=dev))

    def _count_refs(self, pages: int) -> torch.Tensor:
        """How many table entries hold each page (int32 [pages], on the host)."""
        held = self.table_host[(self.table_host >= 0) & (self.table_host < pages)]
        return torch.from_numpy(held.reshape(-1)).long().bincount(minlength=pages).to(torch.int32)

    # ------------------------------------------------------------------ views
    @property
    def pred(self) -> torch.Tensor:
        return self.pred_buf[self.parity]

    @property
    def pred_next(self) -> torch.Tensor:
        return self.pred_buf[1 - self.parity]

    def buffers(self, parity: Optional[int] = None, append: bool = False) -> _abi.PrrStepBuffers:
        """Step buffers; with `append` the step also appends the token held in the
        decoder's k_new / v_new buffers (it then advances seq_lens itself)."""
        par = self.parity if parity is None else parity
        b = _abi.PrrStepBuffers()
        b.q, b.k_cache, b.v_cache = self.q.data_ptr(), self.k_cache.data_ptr(), self.v_cache.data_ptr()
        b.seq_lens, b.summ, b.ema = self.seq_lens.data_ptr(), self.summ.data_ptr(), self.ema.data_ptr()
        b.pred, b.pred_next = self.pred_buf[par].data_ptr(), self.pred_buf[1 - par].data_ptr()
        b.sel, b.missed, b.n_missed = self.sel.data_ptr(), self.missed.data_ptr(), self.n_missed.data_ptr()
        b.keep = self.keep.data_ptr()
        b.part_m, b.part_l, b.part_O = self.part_m.data_ptr(), self.part_l.data_ptr(), self.part_O.data_ptr()
        b.out, b.lse = self.out.data_ptr(), self.lse.data_ptr()
        if append:
            b.k_new, b.v_new = self.k_new.data_ptr(), self.v_new.data_ptr()
        b.trace = self.trace.data_ptr() if self.trace is not None else None
        b.stats = self.stats.data_ptr() if self.stats is not None else None
        return b

    def events(self, timing: Optional[dict] = None) -> _abi.PrrStepEvents:
        """Step events; `timing` maps names of _abi.TIMING_MARKS to timing-enabled
        torch events that have been recorded once (so that their handles exist)."""
        e = _abi.PrrStepEvents()
        for name, ev in self.step_events.items():
            setattr(e, name, ev.cuda_event)
        for name, ev in (timing or {}).items():
            if name not in _abi.TIMING_MARKS:
                raise ValueError(f"unknown timing mark {name}")
            setattr(e, name, ev.cuda_event)
        return e

    def fused_items(self, sms: Optional[int] = None) -> dict:
        """Work items of one fused launch, in ticket (and trace record) order: selection
        chunks, finishers, predictor updates, speculative slots, repair items and merges."""
        d = self.dims
        chunk = min(128, max(32, -(-(-(-d.units * d.maxnb // 512)) // 32) * 32))
        rep = min(d.K, max(4, -(-1024 // d.units)))
        return {"sel": d.units * -(-d.maxnb // chunk), "finish": d.units, "ema": d.units, "spec": d.units * d.P,
                "repair": d.units * rep, "combine": d.units * d.group}

    def enable_trace(self, on: bool = True) -> None:
        """Record start/end times of every work item of the fused launches."""
        self.trace = torch.zeros((sum(self.fused_items().values()), 4), dtype=torch.int64,
                                 device=self.device) if on else None

    def trace_summary(self) -> dict:
        """Timeline of the last traced fused launch, per item kind (see summarize_trace)."""
        if self.trace is None:
            raise RuntimeError("tracing is off: call enable_trace() before the step")
        return summarize_trace(self.trace.cpu().numpy())

    STAT_NAMES = ("tie_mask_units", "key_search_units", "take_all_units", "spec_attended",
                  "spec_skipped", "repaired", "reserved6", "reserved7")

    def enable_stats(self, on: bool = True) -> None:
        """Count, over the following steps, which finisher path each unit took and how
        many speculative and repair blocks were attended or skipped (int64 [8] on the
        device, added to by the kernels; read it with stats_dict)."""
        self.stats = torch.zeros((8,), dtype=torch.int64, device=self.device) if on else None

    def stats_dict(self) -> dict:
        if self.stats is None:
            raise RuntimeError("counters are off: call enable_stats() before the steps")
        return dict(zip(self.STAT_NAMES, (int(x) for x in self.stats.cpu().tolist())))


    # ------------------------------------------------------------------ setup
    def load_context(self, b: int, h: int, k: torch.Tensor, v: torch.Tensor) -> None:
        """Write tokens [0, n) of sequence b, KV head h (k, v: [n][d] bf16 on the device)
        into the cache, through the block table when the cache is paged (whose blocks
        must have their pages)."""
        n, bs = k.shape[0], self.dims.bs
        if self.block_table is None:
            self.k_cache[b, h, :n].copy_(k)
            self.v_cache[b, h, :n].copy_(v)
            return
        nbk = -(-n // bs)
        pages = self.block_table[b, :nbk].long()
        if bool(((pages < 0) | (pages >= self.dims.pages)).any()):  # (-1 as an index would name the pool's last page)
            raise ValueError(f"sequence {b} has no pages for {n} tokens: reserve() them first")
        pad = nbk * bs - n  # rows past n in the last page are never read
        kp = torch.nn.functional.pad(k, (0, 0, 0, pad)).view(nbk, bs, -1)
        vp = torch.nn.functional.pad(v, (0, 0, 0, pad)).view(nbk, bs, -1)
        self.k_cache[pages, h] = kp
        self.v_cache[pages, h] = vp

    def prefill(self, k: Optional[torch.Tensor], v: Optional[torch.Tensor], n0) -> None:
        """Start decoding after an initial context: optionally copy it in (k, v
        [B][Hkv][n][d] bf16 with n >= every length, contiguous caches only; else
        load_context wrote it), set the sequence lengths (n0: one length, or one per
        sequence), build all block summaries, reset the EMA and predict from the zero
        state."""
        d = self.dims
        lens = [int(n0)] * d.B if isinstance(n0, int) else [int(x) for x in n0]
        if len(lens) != d.B or min(lens) < 1 or max(lens) > d.cap_tokens:
            raise ValueError(f"need {d.B} lengths in [1, {d.cap_tokens}], got {lens}")
        if k is not None:
            if self.block_table is not None:
                raise ValueError("prefill copies k/v into a contiguous cache only: fill a paged one with load_context")
            if v is None or k.shape != v.shape or k.dim() != 4 or k.shape[2] < max(lens):
                raise ValueError("k and v must both be [B][Hkv][n][d] with n >= every sequence length")
        self._after_caller(self.select_stream)  # k/v (or load_context's writes) come from the caller's stream
        with torch.cuda.stream(self.select_stream):
            if k is not None:
                n = k.shape[2]
                self.k_cache[:, :, :n].copy_(k)
                self.v_cache[:, :, :n].copy_(v)
            self.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
            self.ema.zero_()
            self.pred_buf.fill_(-1)
            _abi.prr_workspace_init(self.ws, self.select_stream)
            zeros = torch.zeros((d.B,), dtype=torch.int32, device=self.device)
            ends = torch.tensor(lens, dtype=torch.int32, device=self.device)
            _abi.prr_update_summaries(d, self.k_cache, zeros, ends, None, max(lens), self.summ, self.ws,
                                      self.select_stream)
            self.parity = 0
            if d.P > 0:
                _abi.prr_ema_predict(d, self.ema, None, self.seq_lens, self.pred_buf[0], self.ws,
                                     self.select_stream)
        self.select_stream.synchronize()

    # ------------------------------------------------------------------ checkpoint / resume
    def checkpoint(self) -> dict:
        """Host copies of the state a decode step carries to the next one: the caches,
        sequence lengths, block summaries, EMA state and the current prediction Pred_t
        (and the block table of a paged cache, and the representatives' offsets, which
        fork() copies).  The workspace holds nothing that outlives a step, so it is not
        part of the state."""
        self.select_stream.synchronize()
        ck = {"k_cache": self.k_cache.cpu(), "v_cache": self.v_cache.cpu(), "seq_lens": self.seq_lens.cpu(),
              "summ": self.summ.cpu(), "ema": self.ema.cpu(), "pred": self.pred.cpu()}
        if self.block_table is not None:
            ck["block_table"] = self.block_table.cpu()
        if self.rep_offsets is not None:
            ck["rep_offsets"] = self.rep_offsets.cpu()
        return ck

    def restore(self, ck: dict) -> None:
        """Load a checkpoint() into this decoder (same dims): the next step continues
        exactly where the checkpointed decoder stopped.  (A checkpoint of before it held
        the representatives' offsets leaves this decoder's as they are.)"""
        self._after_caller(self.select_stream)
        with torch.cuda.stream(self.select_stream):
            for name in ("k_cache", "v_cache", "seq_lens", "summ", "ema"):
                getattr(self, name).copy_(ck[name])
            if self.block_table is not None:
                self.block_table.copy_(ck["block_table"])
                self.table_host = ck["block_table"].numpy().copy()
                self.page_refs.copy_(self._count_refs(self.dims.pages))
            if self.rep_offsets is not None and "rep_offsets" in ck:
                self.rep_offsets.copy_(ck["rep_offsets"])
            self.parity, self.fused_parity = 0, 0
            self.pred_buf[0].copy_(ck["pred"])
            _abi.prr_workspace_init(self.ws, self.select_stream)
        self.select_stream.synchronize()

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> None:
        """Write the step's token (k_new/v_new [B][Hkv][d] bf16) and advance seq_lens, on
        `stream` (default: the step stream, ordered after the caller's current stream)."""
        st = stream or self.select_stream
        self._after_caller(st)
        _abi.prr_append_kv(self.dims, k_new, v_new, self.seq_lens, self.k_cache, self.v_cache, self.ws, st)

    # ------------------------------------------------------------------ the step
    def _after_caller(self, st) -> None:
        """Order `st` after the caller's current stream, on which the step's input
        tensors were produced (a no-op when the caller already runs on `st`)."""
        cur = torch.cuda.current_stream(self.device)
        if cur != st:
            st.wait_stream(cur)

    def step(self, q: Optional[torch.Tensor] = None, timing: Optional[dict] = None,
             swap: bool = True, append: bool = False) -> None:
        """One decode step on the state's streams (q [B][Hq][d] bf16 is copied into the
        step's query buffer first when given).  Swaps Pred_t / Pred_{t+1} afterwards."""
        if q is not None:
            self._after_caller(self.select_stream)
            with torch.cuda.stream(self.select_stream):
                self.q.copy_(q)
        _abi.prr_decode_step(self.dims, self.buffers(append=append), self.ws, self.select_stream,
                             self.spec_stream, self.events(timing))
        if swap and self.dims.P > 0:
            self.parity ^= 1

    def step_fused(self, q: Optional[torch.Tensor] = None, stream=None, swap: bool = True,
                   parity: Optional[int] = None, k_new: Optional[torch.Tensor] = None,
                   v_new: Optional[torch.Tensor] = None, append: bool = False) -> None:
        """The same step as one persistent launch on `stream` (default: select_stream).
        With k_new / v_new ([B][Hkv][d] bf16, copied into the decoder's token buffers)
        or `append`, the launch also appends the step's token (no separate append)."""
        st = stream or self.select_stream
        if q is not None or k_new is not None:
            self._after_caller(st)
        with torch.cuda.stream(st):
            if q is not None:
                self.q.copy_(q)
            if k_new is not None:
                self.k_new.copy_(k_new)
                self.v_new.copy_(v_new)
        par = self.fused_parity if parity is None else parity
        _abi.prr_decode_step_fused(self.dims, self.buffers(append=append or k_new is not None), self.ws, par, st)
        if parity is None:
            self.fused_parity ^= 1
        if swap and self.dims.P > 0:
            self.parity ^= 1

    # ------------------------------------------------------------------ around the step
    # Prompts and pages.  These run on the step stream, after the caller's current stream;
    # the caller's stream then waits for them, so their results can be used on it at once.
    # They share one workspace: replays of captured ones, too, run one after another.

    @contextlib.contextmanager
    def _serving(self, rows: int = 1):
        """The serving workspace, large enough for `rows` packed rows (allocated when a
        call first needs it, or more of it), with the step stream current.  One that a
        captured graph works in is kept as long as the decoder, whatever comes after it."""
        cur = torch.cuda.current_stream(self.device)
        self._after_caller(self.select_stream)
        with torch.cuda.stream(self.select_stream):
            need = _abi.prr_serving_workspace_bytes(self.dims, max(rows, 1))
            if need == 0:
                raise ValueError(f"unsupported number of rows {rows}")
            capturing = torch.cuda.is_current_stream_capturing()
            if self.serve_ws is None or self.serve_ws.numel() < need:
                if capturing:
                    raise RuntimeError("the serving workspace has to grow: make a call of this size before the capture")
                ws = torch.zeros((need,), dtype=torch.uint8, device=self.device)
                if self.serve_captured:
                    self.serve_kept.append(self.serve_ws)
                elif self.serve_ws is not None:
                    ws[:4] = self.serve_ws[:4]  # the status word
                self.serve_ws, self.serve_captured = ws, False
            self.serve_captured |= capturing
            yield self.serve_ws
        if cur != self.select_stream:
            cur.wait_stream(self.select_stream)

    def _ints(self, x) -> torch.Tensor:
        return torch.as_tensor(x, dtype=torch.int32).to(self.device).contiguous()

    def cache_buffers(self) -> _abi.PrrCacheBuffers:
        """The paged cache and the state that goes with its sequences (prr_cache_* calls),
        with the prediction that is current now: a step makes it the other one."""
        if self.page_refs is None:
            raise ValueError("pages are shared, reserved and moved in a paged cache only (dims.pages > 0)")
        return _abi.cache_buffers(self.k_cache, self.v_cache, self.block_table, self.page_refs, self.seq_lens, self.summ,
                                  self.ema, self.pred if self.dims.P > 0 else None, self.rep_offsets)

    def reserve(self, want_lens) -> None:
        """Give every sequence b pages for want_lens[b] tokens (int32 [B]); it keeps those it holds."""
        with self._serving() as ws:
            _abi.prr_cache_reserve(self.dims, self._ints(want_lens), self.cache_buffers(), ws)

    def fork(self, parents, children) -> None:
        """Make the empty sequences children[i] copies of parents[i]: shared pages, a copy
        of the partly filled last one, and the summaries, EMA state and prediction."""
        with self._serving() as ws:
            _abi.prr_cache_fork(self.dims, self._ints(parents), self._ints(children), self.cache_buffers(), ws)

    def release(self, seqs) -> None:
        """Give back the pages of the sequences; their slots are empty afterwards."""
        with self._serving() as ws:
            _abi.prr_cache_release(self.dims, self._ints(seqs), self.cache_buffers(), ws)

    def compact(self):
        """Move the live pages to the front of the pool.  Returns (remap [pages], n_live [1]) on the device."""
        with self._serving() as ws:
            remap = torch.empty((self.dims.pages,), dtype=torch.int32, device=self.device)
            n_live = torch.empty((1,), dtype=torch.int32, device=self.device)
            _abi.prr_cache_compact(self.dims, self.cache_buffers(), remap, n_live, ws)
        return self._lent(remap), self._lent(n_live)

    def _lent(self, t: torch.Tensor) -> torch.Tensor:
        t.record_stream(torch.cuda.current_stream(self.device))
        return t

    def append_prompt(self, k_rows: torch.Tensor, v_rows: torch.Tensor, q_begin) -> None:
        """Append packed rows k_rows / v_rows [rows][Hkv][d] bf16 behind the sequences'
        tokens (sequence b: rows q_begin[b] .. q_begin[b+1]), with their block summaries."""
        with self._serving() as ws:
            _abi.prr_append_prompt(self.dims, k_rows, v_rows, self._ints(q_begin), self.seq_lens, self.k_cache,
                                   self.v_cache, self.summ, ws)

    def attend_prompt(self, q: torch.Tensor, q_begin, out: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None):
        """Causal attention of packed rows q [rows][Hq][d] bf16, the newest rows of their
        sequences (appended before).  Returns (out [rows][Hq][d] bf16, lse [rows][Hq] fp32)."""
        with self._serving(q.shape[0]) as ws:
            out, lse = self._attend_outputs(q, out, lse)
            _abi.prr_attend_prompt(self.dims, q, self._ints(q_begin), self.seq_lens, self.k_cache, self.v_cache, out, lse, ws)
        return self._lent(out), self._lent(lse)

    def attend_shared(self, q: torch.Tensor, members, group_begin, shared_blocks, out: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None):
        """Attention of q [B][Hq][d] bf16 over all tokens of each sequence, in groups whose
        first shared_blocks[g] blocks are the same and read once.  Returns (out, lse)."""
        with self._serving() as ws:
            out, lse = self._attend_outputs(q, out, lse)
            _abi.prr_attend_shared(self.dims, q, self._ints(members), self._ints(group_begin), self._ints(shared_blocks),
                                   self.seq_lens, self.k_cache, self.v_cache, out, lse, ws)
        return self._lent(out), self._lent(lse)

    def _attend_outputs(self, q, out, lse):
        d = self.dims
        if out is None:
            out = torch.zeros((q.shape[0], d.Hq, d.d), dtype=torch.bfloat16, device=self.device)
        if lse is None:
            lse = torch.zeros((q.shape[0], d.Hq), dtype=torch.float32, device=self.device)
        return out, lse

    def device_status(self) -> int:
        """Device status code of the steps, or if that is 0 of the calls around them, captured
        ones included (prr_workspace_init clears the one that reported: ws, serve_ws or one of serve_kept)."""
        for ws in (self.ws, self.serve_ws, *self.serve_kept):
            code = 0 if ws is None else _abi.prr_get_device_status(ws)
            if code:
                break
        return code


KINDS = {1: "sel", 2: "spec", 3: "repair", 4: "ema", 5: "combine", 6: "finish"}


def summarize_trace(trace) -> dict:
    """Per item kind of one fused launch: how many items ran, when the first and last
    started and the last ended (microseconds after the earliest start), and the p50 /
    mean / max item duration; "finisher" repeats the count and durations of the top-K
    finisher items.  `trace` is the [records][4] array of prr_step_buffers (start ns,
    end ns, SM << 32 | CTA index, kind)."""
    import numpy as np
    tr = np.asarray(trace, dtype=np.int64)
    ran = tr[:, 0] > 0
    if not ran.any():
        return {}
    t0 = tr[ran, 0].min()
    out = {"end_us": float((tr[ran, 1].max() - t0) / 1e3)}
    kinds = tr[:, 3] & 0xFFFFFFFF
    fin = ran & (kinds == 6)
    if fin.any():
        f = (tr[fin, 1] - tr[fin, 0]) / 1e3
        out["finisher"] = {"n": int(len(f)), "dur_p50_us": float(np.median(f)), "dur_max_us": float(f.max())}
    for code, kind in KINDS.items():
        seg = tr[ran & (kinds == code)]
        if len(seg) == 0:
            out[kind] = {"n": 0}
            continue
        st = (seg[:, 0] - t0) / 1e3
        en = (seg[:, 1] - t0) / 1e3
        dur = en - st
        out[kind] = {"n": int(len(seg)), "start_min_us": float(st.min()), "start_max_us": float(st.max()),
                     "end_max_us": float(en.max()), "dur_p50_us": float(np.median(dur)),
                     "dur_mean_us": float(dur.mean()), "dur_max_us": float(dur.max()),
                     "sms": int(len(np.unique(seg[:, 2] >> 32)))}
    return out
