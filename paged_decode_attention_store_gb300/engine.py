"""PagedKVCache: the per-step driver a caller uses (one GPU, one process).

It owns a KV buffer in the mini-sglang layout (2, layers, pages, page_size,
kv_heads, head_dim), the C++ host bookkeeping and the device table, and
issues one decode step as the pages describe it:

1. host bookkeeping appends one token per request (a fresh page on a page
   boundary, lazy copy-on-write of a shared tail page, chapter 15 of
   silicon_compiler_from_scratch, section "The model");
2. the new table entries go to the device in one scatter (mini-sglang code
   series, part 4, with the page->token expansion done on the device for a
   raw-location table), copied-on-write pages are copied;
3. store_cache writes the new K/V rows of every layer to their slots;
4. paged_decode_attention reads each request's window through the table.

Host->device traffic per step is the table writes and slots (from pinned
staging buffers); everything else stays on the device.
"""

from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import binding as kb

_DT = {"bf16": (torch.bfloat16, kb.KVP_BF16), "f32": (torch.float32, kb.KVP_F32)}


def _align32(n):
    return (n + 31) // 32 * 32


def _on_axes(positions, rope):
    """Positions [n] as a plan takes them: those of text, the same on every axis."""
    return positions if rope.axes == 1 else positions.expand(rope.axes, -1).contiguous()


class PagedKVCache:
    def __init__(self, num_pages, page_size, kv_heads, head_dim, num_layers, dtype="bf16", max_requests=256,
                 table_mode="block", max_seq_len=None, free_stack=None, device="cuda", zero=True):
        self.P, self.Hkv, self.D, self.layers = page_size, kv_heads, head_dim, num_layers
        self.num_pages = num_pages
        self.tdt, kdt = _DT[dtype]
        self.mode = table_mode
        self.raw = table_mode == "raw"
        self.dev = torch.device(device)
        extra = 1 if self.raw else 0  # dummy page of the raw-location layout
        alloc = torch.zeros if zero else torch.empty
        self._make_pool(alloc, num_pages + extra, kdt)
        self.host = kb.HostPageTable(num_pages, page_size, max_requests, free_stack)
        self.max_requests = max_requests
        max_seq_len = max_seq_len or num_pages * page_size
        if self.raw:
            cols = _align32(min(max_seq_len, num_pages * page_size))
            self.table = torch.zeros((max_requests + 1, cols), dtype=torch.int32, device=self.dev)
            self.table[max_requests].fill_(num_pages * page_size)  # dummy row -> dummy page
        else:
            cols = -(-max_seq_len // page_size)
            self.table = torch.full((max_requests, cols), -1, dtype=torch.int32, device=self.dev)
        self.table_mode = kb.KVP_RAW_LOCATIONS if self.raw else kb.KVP_BLOCK_TABLE
        self._ws = {}
        self._steps = {}
        self.lengths = np.zeros(max_requests, np.int64)  # tokens appended, per request (the caller's count)
        self.copies = 0
        self.h2d_bytes = 0  # bytes this driver has copied host -> device

    def _make_pool(self, alloc, pages, kdt):
        self.kv = alloc((2, self.layers, pages, self.P, self.Hkv, self.D), dtype=self.tdt, device=self.dev)
        self.pool = kb.Pool(self.kv, self.P, kdt)

    # -- host-side staging -------------------------------------------------
    def _to_device(self, flat):
        # A fresh pinned block per call: torch's caching host allocator does
        # not hand it out again before the asynchronous copy has completed.
        host = torch.from_numpy(np.ascontiguousarray(flat, dtype=np.int32)).pin_memory()
        self.h2d_bytes += 4 * host.numel()
        return host.to(self.dev, non_blocking=True)

    def _write_table(self, writes):
        if not writes:
            return
        r, c, v = zip(*writes)
        d = self._to_device(list(r) + list(c) + list(v))
        n = len(writes)
        kb.page_table_write(self.table, d[:n], d[n:2 * n], d[2 * n:], expand=self.P if self.raw else 1,
                            error_word=self.pool.error_word)

    # -- request lifecycle ---------------------------------------------------
    def new(self, rid):
        self.host.new(rid)
        self.lengths[rid] = 0

    def fork(self, src, dst):
        self._write_table(self.host.fork(src, dst))
        self.lengths[dst] = self.lengths[src]

    def release(self, rid):
        self.host.release(rid)
        self.lengths[rid] = 0

    def trim(self, rid, keep_from, sinks=0):
        """Release the pages below keep_from (except the first ceil(sinks / P));
        returns the number of table writes."""
        writes = self.host.trim(rid, keep_from, sinks=sinks)
        self._write_table(writes)
        return len(writes)

    def append(self, rids):
        """Host bookkeeping for one token per entry; returns the slots on the device.

        Also leaves the counts of this call's table writes and copies in
        ``last_writes`` / ``last_copies``."""
        r = np.ascontiguousarray(rids, dtype=np.int32)
        n = int(r.shape[0])
        buf = np.empty(6 * max(n, 1), np.int32)  # slots, table writes (rows, cols, values), copy pairs
        slots, tw, cow = buf[:n], buf[n:4 * n].reshape(3, n), buf[4 * n:6 * n].reshape(2, n)
        nw, nc = self.host.append_into(r, slots, tw, cow)
        self.lengths += np.bincount(r, minlength=self.lengths.shape[0])
        self.last_writes, self.last_copies = nw, nc
        dev = self._to_device(np.concatenate((slots, tw[:, :nw].ravel(), cow[:, :nc].ravel())))
        if nw:
            kb.page_table_write(self.table, dev[n:n + nw], dev[n + nw:n + 2 * nw], dev[n + 2 * nw:n + 3 * nw],
                                expand=self.P if self.raw else 1, error_word=self.pool.error_word)
        if nc:
            o = n + 3 * nw
            kb.copy_pages(self.pool, dev[o:o + nc], dev[o + nc:o + 2 * nc])
            self.copies += nc
        return dev[:n]

    def store(self, layer, k, v, out_loc):
        kb.store_cache(self.pool, layer, k, v, out_loc)

    def rotary_store(self, layer, q, k, v, positions, out_loc, rope, q_out=None):
        """Rotary positions of q and k and the store of the rotated k and of v
        in one launch; returns the rotated q (``q_out``, or q itself when it
        is None). ``positions`` int32 [n] on the device, ``rope`` a
        binding.RotaryPlan; q [n, Hq, D], k/v [n, Hkv, D] may be views of one
        projection's output."""
        q_out = q if q_out is None else q_out
        kb.rotary_store_cache(self.pool, layer, q, k, v, positions, out_loc, rope, q_out)
        return q_out

    def workspace(self, batch, num_q_heads):
        key = (batch, num_q_heads)
        if key not in self._ws:
            self._ws[key] = kb.alloc_workspace(self.pool, batch, num_q_heads, device=self.dev)
        return self._ws[key]

    def attend(self, layer, q, context_lens, window, scale, out, table_rows=None, sinks=0):
        ws = self.workspace(q.shape[0], q.shape[1])
        kb.paged_decode_attention(self.pool, layer, q, self.table, self.table_mode, context_lens, window, scale,
                                  out, ws, table_rows=table_rows, sinks=sinks)

    def store_and_attend(self, layer, q, k, v, out_loc, context_lens, window, scale, out, table_writes=None,
                         table_rows=None, sinks=0):
        """store_cache + paged_decode_attention of one layer in one launch;
        ``out_loc[b]`` must be the slot of request b's newest position, and
        ``table_writes`` (rows, cols, vals device tensors) may only add the
        pages of this step's new tokens."""
        ws = self.workspace(q.shape[0], q.shape[1])
        kb.store_cache_and_attention(self.pool, layer, q, k, v, out_loc, self.table, self.table_mode, context_lens,
                                     window, scale, out, ws, table_rows=table_rows, table_writes=table_writes,
                                     sinks=sinks)

    def verify(self, layer, q, context_lens, window, scale, out, table_rows=None, sinks=0):
        """Multi-token verify: q/out [B, M, Hq, D], query j of request b at
        position context_lens[b] - M + j (the M newest tokens, stored)."""
        B, M, Hq = q.shape[0], q.shape[1], q.shape[2]
        key = ("verify", B, M, Hq)
        if key not in self._ws:
            self._ws[key] = kb.alloc_verify_workspace(self.pool, B, M, Hq, device=self.dev)
        kb.paged_verify_attention(self.pool, layer, q, self.table, self.table_mode, context_lens, window, scale,
                                  out, self._ws[key], table_rows=table_rows, sinks=sinks)

    def rewind(self, rid, n):
        """Drop the newest n tokens of a request (rejected drafts); returns
        the number of pages given back."""
        writes = self.host.rewind(rid, n)
        self._write_table(writes)
        self.lengths[rid] -= n
        return len(writes)

    def prefill(self, layer, q, context_lens, window, scale, out, q_lens=None, table_rows=None, sinks=0):
        """Chunked prefill: q/out [B, C, Hq, D], query j of request b at
        position context_lens[b] - q_lens[b] + j (the chunk's rows stored)."""
        kb.paged_prefill_attention(self.pool, layer, q, self.table, self.table_mode, context_lens, window, scale,
                                   out, q_lens=q_lens, table_rows=table_rows, sinks=sinks)

    def prefill_step(self, rids, q, k, v, out, window, scale, sinks=0):
        """One chunked-prefill step for ``rids``, all layers: append each
        request's C new tokens (host bookkeeping, table writes, copy-on-write),
        store their K/V and attend them at once. ``q``/``out`` [layers][B, C,
        Hq, D], ``k``/``v`` [layers][B * C, Hkv, D] (request-major), on the host
        (pinned) or the device; returns when ``out`` holds the results."""
        self._multi_step("prefill", rids, q, k, v, out, window, scale, sinks)

    def verify_step(self, rids, q, k, v, out, window, scale, sinks=0):
        """One speculative-decoding verify step for requests ``rids`` (ids =
        table rows), all layers: append the M drafted tokens of each request
        (host bookkeeping, table writes, copy-on-write), store their K/V rows
        and verify them. ``q``/``out`` [layers][B, M, Hq, D] and ``k``/``v``
        [layers][B * M, Hkv, D] (request-major) on the host (pinned) or the
        device. Returns when ``out`` holds the results; the caller then
        rewinds the rejected drafts with :meth:`rewind`."""
        self._multi_step("verify", rids, q, k, v, out, window, scale, sinks)

    def _multi_step(self, kind, rids, q, k, v, out, window, scale, sinks):
        B, M = q[0].shape[0], q[0].shape[1]
        main = torch.cuda.current_stream(self.dev)
        staged = None
        if not q[0].is_cuda:
            # host inputs: every layer's q/k/v go up on a side stream right away,
            # while the host bookkeeping below runs; layer l's store waits for
            # layer l's copies only
            side = self._steps.get("multi_h2d")
            if side is None:
                side = self._steps["multi_h2d"] = torch.cuda.Stream(self.dev)
            side.wait_stream(main)
            staged = []
            with torch.cuda.stream(side):
                for layer in range(self.layers):
                    xs = tuple(x[layer].to(self.dev, non_blocking=True) for x in (q, k, v))
                    for t in xs:
                        t.record_stream(main)
                    ev = torch.cuda.Event()
                    ev.record(side)
                    staged.append((xs, ev))
                    self.h2d_bytes += sum(x[layer].numel() * x[layer].element_size() for x in (q, k, v))
        r = np.ascontiguousarray(rids, dtype=np.int32)
        ctx = self.lengths[r] + M
        out_loc = self.append(np.repeat(r, M))
        bound = self._bound_of(ctx)
        lens = self._to_device(ctx)
        rows = self._to_device(r)
        host_out = not out[0].is_cuda
        for layer in range(self.layers):
            if staged is None:
                qd, kd, vd = (x[layer] for x in (q, k, v))
            else:
                (qd, kd, vd), ev = staged[layer]
                main.wait_event(ev)
            self.store(layer, kd, vd, out_loc)
            od = torch.empty_like(qd) if host_out else out[layer]
            if kind == "verify":
                self.verify(layer, qd, lens, window, scale, od, table_rows=rows, sinks=sinks, **bound)
            else:
                self.prefill(layer, qd, lens, window, scale, od, table_rows=rows, sinks=sinks, **bound)
            if host_out:
                out[layer].copy_(od, non_blocking=True)
        torch.cuda.current_stream(self.dev).synchronize()

    def _bound_of(self, lengths):
        """What a step's attention is told of its requests' lengths."""
        return {}

    def check(self):
        """Raise if a device-side error was recorded since the last check."""
        e = kb.kvp_sync_error(self.pool)
        if e != 0:
            raise kb.KvpError(e, "device")

    def _append_and(self, work, rids, B, C, window, sinks):
        """A step of B distinct requests, C new tokens each: append, then ``work(lens, rows, positions, out_loc)`` (int32 on
        the device: contexts and table rows [B], positions and slots [B * C]), then the pages that the window leaves are
        released. A step that is refused leaves the lengths and pages as they were, but for a copy of a shared last page."""
        r = np.ascontiguousarray(rids, dtype=np.int32)
        if len(r) != B or len(np.unique(r)) != B:
            raise ValueError(f"step takes {B} distinct requests, got {list(map(int, r))}")
        before = self.lengths[r].copy()
        out_loc = self.append(np.repeat(r, C))
        try:
            flat = np.concatenate((before + C, r, (before[:, None] + np.arange(C)).ravel()))
            d = self._to_device(flat)
            work(d[:B], d[B:2 * B], d[2 * B:], out_loc)
        except Exception:
            for rid in r[::-1]:  # the last page taken goes back first
                self.rewind(int(rid), C)
            raise
        if window and window > 0:
            for i, rid in enumerate(r):
                self.trim(int(rid), max(0, int(before[i]) + C + 1 - (window - sinks)), sinks=sinks)

    def _slots_in_order(self, rids):
        """The slots of requests ``rids`` in logical order, int64 [total], and their offsets int32 [len(rids) + 1]. A
        request that a window has taken pages from has no such rows left (ValueError). Waits for the GPU, to see that."""
        r = np.ascontiguousarray(rids, dtype=np.int32)
        lens = self.lengths[r]
        some = lens > 0
        n = int(some.sum())
        d = self._to_device(np.concatenate((lens[some], r[some], [0], np.cumsum(lens))))
        start = d[2 * n:]
        if n == 0:
            return torch.empty(0, dtype=torch.int64, device=self.dev), start
        slots = torch.empty((n, int(lens.max())), dtype=torch.int32, device=self.dev)
        kb.gather_indices(self.pool, self.table, self.table_mode, d[:n], 0, slots, table_rows=d[n:2 * n])
        live = torch.arange(slots.shape[1], device=self.dev)[None, :] < d[:n, None]
        slots = slots[live].long()
        if bool((slots < 0).any()):
            kb.kvp_sync_error(self.pool)  # what the gather recorded of it
            raise ValueError("a request's first pages are released")
        return slots, start

    # -- one decode step, host buffers in and out ----------------------------
    def decode_step(self, rids, q, k, v, out, window, scale, sinks=0):
        """One decode step for the requests ``rids`` (one token each; request
        id = table row), through the native kvp_decode_step.

        ``q`` [layers][B, Hq, D], ``k``/``v`` [layers][B, Hkv, D] and ``out``
        [layers][B, Hq, D] are lists of tensors, all on the host (pinned) or
        all on the device. With several layers, host inputs are copied per
        layer on a side stream and each layer's store + attention waits only
        for its own inputs, and each output is copied back on another side
        stream as soon as its layer is done; a single layer copies on the
        step's own stream. Returns when ``out`` holds the results.
        """
        L = kb.lib()
        n = len(rids)
        Hq = q[0].shape[1]
        st = self._step_state(n, Hq)
        rids = np.ascontiguousarray(rids, dtype=np.int32)
        stream = torch.cuda.current_stream(self.dev)
        slot = st["ring"][st["next"]]
        st["next"] ^= 1
        slot["event"].synchronize()  # its previous copy has finished reading it
        host_io = not q[0].is_cuda
        vp = ctypes.c_void_p
        arr = lambda ts: (vp * self.layers)(*[t.data_ptr() for t in ts])  # noqa: E731
        ready = done = None
        if host_io:
            qd, kd, vd = st["in"]
            od = st["out"]
            qp, kp, vpp, op = st["in_p"][0], st["in_p"][1], st["in_p"][2], st["out_p"]
            side = self.layers > 1  # overlap the per-layer copies with the other layers' kernels
            cs = st["h2d"] if side else stream
            if side:
                st["h2d"].wait_stream(stream)  # the previous step's kernels are done with the buffers
            with torch.cuda.stream(cs):
                for layer in range(self.layers):
                    qd[layer].copy_(q[layer], non_blocking=True)
                    kd[layer].copy_(k[layer], non_blocking=True)
                    vd[layer].copy_(v[layer], non_blocking=True)
                    if side:
                        st["ready"][layer].record(cs)
            self.h2d_bytes += sum(t[i].numel() * t[i].element_size() for t in (q, k, v) for i in range(self.layers))
            if side:
                ready, done = st["ready_p"], st["done_p"]
        else:
            side = False
            qp, kp, vpp, op = arr(q), arr(k), arr(v), arr(out)
        info = kb.StepInfo()
        ws = self.workspace(n, Hq)
        kb._check(L.kvp_decode_step(self.host.handle, self.pool.handle, vp(self.table.data_ptr()), self.table.shape[0],
                                    self.table.shape[1], self.table_mode, rids.ctypes.data_as(vp), n,
                                    int(window or 0), int(sinks), Hq, float(scale), qp, kp, vpp, op, ready,
                                    done, vp(slot["host"].data_ptr()), vp(st["dev"].data_ptr()), st["cap"],
                                    vp(ws.data_ptr()), ws.numel(), vp(stream.cuda_stream), ctypes.byref(info)),
                  "kvp_decode_step")
        slot["event"].record(stream)
        self.h2d_bytes += 4 * info.meta_ints
        self.last_writes, self.last_copies, self.last_trims = info.n_table_writes, info.n_copies, info.n_trim_writes
        self.copies += info.n_copies
        np.add.at(self.lengths, rids, 1)
        if host_io:
            if side:
                with torch.cuda.stream(st["d2h"]):
                    for layer in range(self.layers):
                        st["d2h"].wait_event(st["done"][layer])
                        out[layer].copy_(od[layer], non_blocking=True)
                st["d2h"].synchronize()
            else:
                for layer in range(self.layers):
                    out[layer].copy_(od[layer], non_blocking=True)
        stream.synchronize()  # the step's outputs are in `out`
        return 4 * info.meta_ints

    def _step_state(self, n, Hq):
        key = (n, Hq)
        st = self._steps.get(key)
        if st is not None:
            return st
        cap = 8 * n + 3 * (4 * n + 64)
        ring = []
        for _ in range(2):
            host = torch.zeros(cap, dtype=torch.int32, pin_memory=True)
            ev = torch.cuda.Event()
            ev.record(torch.cuda.current_stream(self.dev))
            ring.append({"host": host, "event": ev})
        ready = [torch.cuda.Event() for _ in range(self.layers)]
        done = [torch.cuda.Event() for _ in range(self.layers)]
        for e in ready + done:  # torch creates the CUDA event at its first record
            e.record(torch.cuda.current_stream(self.dev))
        vp = ctypes.c_void_p
        st = {
            "cap": cap, "ring": ring, "next": 0,
            "dev": torch.empty(cap, dtype=torch.int32, device=self.dev),
            "in": [[torch.empty((n, Hq, self.D), dtype=self.tdt, device=self.dev) for _ in range(self.layers)],
                   [torch.empty((n, self.Hkv, self.D), dtype=self.tdt, device=self.dev) for _ in range(self.layers)],
                   [torch.empty((n, self.Hkv, self.D), dtype=self.tdt, device=self.dev) for _ in range(self.layers)]],
            "out": [torch.empty((n, Hq, self.D), dtype=self.tdt, device=self.dev) for _ in range(self.layers)],
            "h2d": torch.cuda.Stream(self.dev), "d2h": torch.cuda.Stream(self.dev),
            "ready": ready, "done": done,
            "ready_p": (vp * self.layers)(*[e.cuda_event for e in ready]),
            "done_p": (vp * self.layers)(*[e.cuda_event for e in done]),
        }
        st["in_p"] = [(vp * self.layers)(*[t.data_ptr() for t in ts]) for ts in st["in"]]
        st["out_p"] = (vp * self.layers)(*[t.data_ptr() for t in st["out"]])
        torch.cuda.synchronize(self.dev)
        self._steps[key] = st
        return st


class PagedLatentCache(PagedKVCache):
    """A paged cache of latent rows [latent | shared rotated key part], one per
    token for all heads, with the page bookkeeping of :class:`PagedKVCache`
    (new, fork, append with copy-on-write, trim, rewind, release).

    A step appends its tokens (:meth:`append`), then per layer writes their
    rows and rotates the queries' key part (:meth:`store`) and attends in the
    latent space (:meth:`attend`: decode, multi-token verify and chunks). Long
    prompts are cheaper in expanded form: project :meth:`rows` up and call
    :func:`binding.latent_prefill_attention`. All calls of a cache share a
    workspace: they, and replays of graphs that hold them, run one after another
    on the GPU (calls that overlap take their own:
    :func:`binding.paged_latent_attention`)."""

    def __init__(self, num_pages, page_size, latent_dim, rope_dim, num_layers, dtype="bf16", max_requests=256,
                 table_mode="block", max_seq_len=None, free_stack=None, device="cuda", zero=True):
        self.latent_dim, self.rope_dim = latent_dim, rope_dim
        super().__init__(num_pages, page_size, 1, latent_dim + rope_dim, num_layers, dtype=dtype,
                         max_requests=max_requests, table_mode=table_mode, max_seq_len=max_seq_len,
                         free_stack=free_stack, device=device, zero=zero)
        self._need, self._largest = {}, 0

    def _make_pool(self, alloc, pages, kdt):
        self.kv = alloc((self.layers, pages, self.P, self.D), dtype=self.tdt, device=self.dev)
        self.pool = kb.LatentPool(self.kv, self.latent_dim, kdt)

    def store(self, layer, q_pe, latent, k_pe, positions, out_loc, rope, q):
        """Write the tokens' rows and the rotated ``q_pe`` into the tail of the
        absorbed queries ``q`` [n, Hq, latent_dim + rope_dim], in one launch.
        ``q_pe`` and ``q`` None: only the store (the rows of a prompt)."""
        kb.rotary_store_latent(self.pool, layer, q_pe, latent, k_pe, positions, out_loc, rope,
                               None if q is None else q[..., self.latent_dim:])

    def workspace(self, batch, num_q_heads, chunk=1):
        """The cache's workspace, for calls of this shape among others: one that grows. Outgrown ones are kept, as a
        captured graph may hold them: a pool has half a dozen sizes, 10 to 40 MB, whatever the batches and chunks."""
        key = (batch, num_q_heads, chunk)
        need = self._need.get(key)
        if need is None:
            need = self._need[key] = kb.paged_latent_attention_workspace_size(self.pool, batch, chunk, num_q_heads)
        if need > self._largest:
            self._ws[need] = torch.empty(need, dtype=torch.uint8, device=self.dev)
            self._largest = need
        return self._ws[self._largest]

    def attend(self, layer, q, context_lens, window, scale, out, q_lens=None, table_rows=None, sinks=0):
        """Absorbed attention: q [B, C, Hq, latent_dim + rope_dim], out [B, C,
        Hq, latent_dim]; query j of request b sits at position context_lens[b]
        - q_lens[b] + j (its rows stored)."""
        ws = self.workspace(q.shape[0], q.shape[2], q.shape[1])
        kb.paged_latent_attention(self.pool, layer, q, self.table, self.table_mode, context_lens, window, scale, out,
                                  ws, q_lens=q_lens, table_rows=table_rows, sinks=sinks)

    def step(self, rids, q, q_pe, latent, k_pe, rope, out, window, scale, sinks=0):
        """One step for requests ``rids``, all layers, C new tokens each (C = 1:
        decode): append, then per layer store and attend. Per-layer device
        tensors: ``q`` [B, C, Hq, latent_dim + rope_dim] (absorbed; the tails are
        filled from ``q_pe`` [B, C, Hq, rope_dim] rotated), ``latent`` [B * C,
        latent_dim], ``k_pe`` [B * C, rope_dim] (request-major), ``out`` [B, C,
        Hq, latent_dim]. With a window, the pages it leaves are released
        afterwards. A step that is refused leaves the lengths and pages as they
        were, but that a shared last page may have been copied. Asynchronous on
        the current stream."""
        B, C, Hq, W = q[0].shape

        def work(lens, rows, positions, out_loc):
            positions = _on_axes(positions, rope)
            for layer in range(self.layers):
                self.store(layer, q_pe[layer].view(B * C, Hq, self.rope_dim), latent[layer], k_pe[layer], positions,
                           out_loc, rope, q[layer].view(B * C, Hq, W))
                self.attend(layer, q[layer], lens, window, scale, out[layer], table_rows=rows, sinks=sinks)

        self._append_and(work, rids, B, C, window, sinks)

    def rows(self, layer, rids):
        """The stored rows of requests ``rids`` in logical order, [total,
        latent_dim + rope_dim], and their offsets int32 [len(rids) + 1]: what
        the projections of the expanded form take. A request that a window
        has taken pages from has no such rows left (ValueError). Waits for the
        GPU, to see that; not for capture into a graph."""
        slots, start = self._slots_in_order(rids)
        return self.kv[layer].view(-1, self.D)[slots], start

    def _unsupported(self, what):
        raise TypeError(f"{what} reads separate K and V: a latent cache uses store, attend and step")

    def rotary_store(self, *args, **kwargs):
        self._unsupported("rotary_store")

    def store_and_attend(self, *args, **kwargs):
        self._unsupported("store_and_attend")

    def verify(self, *args, **kwargs):
        self._unsupported("verify")

    def prefill(self, *args, **kwargs):
        self._unsupported("prefill")

    def _multi_step(self, kind, *args, **kwargs):
        self._unsupported(kind + "_step")

    def decode_step(self, *args, **kwargs):
        self._unsupported("decode_step")


class PagedFp4Cache(PagedKVCache):
    """A paged cache of K and V in four bits (binding.Fp4Pool: a code of four
    bits an entry, a scale for 16 of them), with the page bookkeeping of
    :class:`PagedKVCache` (new, fork, append with copy-on-write, trim, rewind,
    release). ``dtype`` is that of queries, keys, values and outputs;
    ``k_scale`` and ``v_scale`` (powers of two, one or one a layer) place the
    range of the scales.

    :meth:`rotary_store` or :meth:`store` round a step's keys and values as they
    are stored; :meth:`attend`, :meth:`verify` and :meth:`prefill` read them in
    place; :meth:`step` is a whole step. All calls of a cache share a workspace:
    they, and replays of graphs that hold them, run one after another on the GPU
    (calls that overlap take their own: :func:`binding.paged_fp4_attention`)."""

    def __init__(self, num_pages, page_size, kv_heads, head_dim, num_layers, dtype="bf16", max_requests=256,
                 table_mode="block", max_seq_len=None, free_stack=None, device="cuda", zero=True, k_scale=1.0, v_scale=1.0):
        self.k_scale, self.v_scale = k_scale, v_scale
        super().__init__(num_pages, page_size, kv_heads, head_dim, num_layers, dtype=dtype, max_requests=max_requests,
                         table_mode=table_mode, max_seq_len=max_seq_len, free_stack=free_stack, device=device, zero=zero)
        self._need, self._largest = {}, 0

    def _make_pool(self, alloc, pages, kdt):
        self.pool = kb.kv_fp4_pool_create(pages, self.P, self.Hkv, self.D, kdt, self.layers, self.k_scale, self.v_scale,
                                          device=self.dev, zero=alloc is torch.zeros)
        self.codes, self.block_scales = self.pool.codes, self.pool.scales

    def store(self, layer, k, v, out_loc):
        """k, v [n, Hkv, D] as they are, rounded to four bits."""
        kb.store_cache_fp4(self.pool, layer, k, v, out_loc)

    def rotary_store(self, layer, q, k, v, positions, out_loc, rope, q_out=None):
        """Rotary positions of q and k and the store of the rotated k and of v
        in four bits, in one launch; returns the rotated q (``q_out``, or q
        itself when it is None). As :meth:`PagedKVCache.rotary_store`."""
        q_out = q if q_out is None else q_out
        kb.rotary_store_fp4(self.pool, layer, q, k, v, positions, out_loc, rope, q_out)
        return q_out

    def workspace(self, batch, num_q_heads, chunk=1, max_context=1):
        """The cache's workspace, for calls of this shape among others: one that grows, by powers of two. Outgrown ones are
        kept, as a captured graph may hold them: all together they are no larger than the last."""
        key = (batch, num_q_heads, chunk, max_context)
        need = self._need.get(key)
        if need is None:
            if len(self._need) > 4096:
                self._need.clear()
            need = self._need[key] = kb.paged_fp4_attention_workspace_size(self.pool, batch, chunk, num_q_heads, max_context)
        if need > self._largest:
            self._largest = 1 << (need - 1).bit_length()
            self._ws[self._largest] = torch.empty(self._largest, dtype=torch.uint8, device=self.dev)
        return self._ws[self._largest]

    def _bound_of(self, lengths):
        """A bound of these lengths, in steps of 256: the workspace of a chunk holds as many rows a request."""
        return {"max_context": max(1, -(-int(lengths.max()) // 256)) * 256}

    def attend(self, layer, q, context_lens, window, scale, out, q_lens=None, table_rows=None, sinks=0, max_context=None):
        """Attention over the stored rows: q, out [B, Hq, D] (one token a
        request) or [B, C, Hq, D], query j of request b at position
        context_lens[b] - q_lens[b] + j (q_lens None: C). ``max_context``: a
        bound of context_lens; None: the length of the cache's longest request
        so far, in steps of 256 (a graph that is replayed with longer contexts
        gives theirs; short requests beside a long one theirs, as chunks need a
        workspace of as many rows a request). :meth:`step`, prefill_step and
        verify_step give that of their own requests."""
        if q.dim() == 3:
            q, out = q[:, None], out[:, None]
        if max_context is None:
            max_context = self._bound_of(self.lengths)["max_context"]
        ws = self.workspace(q.shape[0], q.shape[2], q.shape[1], max_context)
        kb.paged_fp4_attention(self.pool, layer, q, self.table, self.table_mode, context_lens, window, scale, out, ws,
                               q_lens=q_lens, table_rows=table_rows, sinks=sinks, max_context=max_context)

    def verify(self, layer, q, context_lens, window, scale, out, table_rows=None, sinks=0, max_context=None):
        self.attend(layer, q, context_lens, window, scale, out, table_rows=table_rows, sinks=sinks, max_context=max_context)

    def prefill(self, layer, q, context_lens, window, scale, out, q_lens=None, table_rows=None, sinks=0, max_context=None):
        self.attend(layer, q, context_lens, window, scale, out, q_lens=q_lens, table_rows=table_rows, sinks=sinks,
                    max_context=max_context)

    def _check_step(self, q, k, v, rope, out, window, scale, sinks, positions, max_context):
        """Refuses what a layer would refuse, before tokens are appended (an append may copy a shared page, which stays) and
        before the first layer turns its q in place."""
        B, C, Hq, D = shape = q[0].shape
        if scale != scale or sinks < 0 or (window and 0 < window <= sinks):
            raise ValueError(f"scale, window and sinks cannot be {scale}, {window} and {sinks}")
        index = self.pool.device_index
        if rope is not None:
            if positions is not None and kb._positions_of(positions, index, rope.axes)[1] != B * C:
                raise ValueError(f"positions must be those of {B * C} tokens, got {tuple(positions.shape)}")
            if rope.rotary_dim > self.D or rope.attn_factor != rope.attn_factor:
                raise ValueError(f"the plan turns {rope.rotary_dim} entries of {self.D}, by {rope.attn_factor}")
            if rope.rotary_dim and rope.freqs.get_device() != index:
                kb._elsewhere(rope.freqs, index, "the plan's frequencies")
        self.workspace(B, Hq, C, max_context)
        native = kb._native()
        if native is not None and native.step(self.pool.dtype, index, self.layers, q, out, k, v, B, C, Hq, self.Hkv, self.D):
            return
        for layer in range(self.layers):
            for t, name in ((q[layer], "q"), (out[layer], "out")):
                kb._on(t, index, self.tdt, name)
                if t.shape != shape or D != self.D or t.data_ptr() % 16:
                    raise ValueError(f"{name} must be [{B}, {C}, {Hq}, {self.D}] on 16 bytes in every layer, got {tuple(t.shape)}")
            for t, name in ((k[layer], "k"), (v[layer], "v")):
                kb._rows_view(t, index, self.tdt, name, B * C, self.Hkv, self.D)

    def step(self, rids, q, k, v, rope, out, window, scale, sinks=0, positions=None):
        """One step for requests ``rids``, all layers, C new tokens each (C = 1:
        decode): append, then per layer rotate, store and attend. Per-layer
        device tensors: ``q`` (rotated in place) and ``out`` [B, C, Hq, D],
        ``k``, ``v`` [B * C, Hkv, D] (request-major). ``positions``: int32 [B * C],
        or [axes, B * C] for a plan of several axes; None: the tokens' places in
        their requests, on every axis. ``rope`` None: q and k as they are. With a
        window, the pages it leaves are released afterwards. A step that is
        refused leaves the lengths and pages as they were, and every layer's q.
        Asynchronous on the current stream."""
        B, C, Hq, D = q[0].shape
        bound = self._bound_of(self.lengths[np.ascontiguousarray(rids, dtype=np.int32)] + C)
        self._check_step(q, k, v, rope, out, window, scale, sinks, positions, bound["max_context"])

        def work(lens, rows, places, out_loc):
            pos = positions
            if rope is not None and pos is None:
                pos = _on_axes(places, rope)
            for layer in range(self.layers):
                if rope is None:
                    self.store(layer, k[layer], v[layer], out_loc)
                else:
                    self.rotary_store(layer, q[layer].view(B * C, Hq, D), k[layer], v[layer], pos, out_loc, rope)
                self.attend(layer, q[layer], lens, window, scale, out[layer], table_rows=rows, sinks=sinks, **bound)

        self._append_and(work, rids, B, C, window, sinks)

    def rows(self, layer, rids):
        """K and V of requests ``rids`` in logical order, [total, Hkv, D] each,
        as the values that the four bits stand for, and their offsets int32
        [len(rids) + 1]. A request that a window has taken pages from has no
        such rows left (ValueError). Waits for the GPU, to see that; not for
        capture into a graph."""
        slots, start = self._slots_in_order(rids)
        k, v = (torch.empty((slots.numel(), self.Hkv, self.D), dtype=self.tdt, device=self.dev) for _ in range(2))
        kb.load_cache_fp4(self.pool, layer, slots.to(torch.int32), k, v)
        return k, v, start

    def store_and_attend(self, *args, **kwargs):
        raise TypeError("a four-bit cache stores, then attends: store or rotary_store, then attend, or step")

    def decode_step(self, *args, **kwargs):
        raise TypeError("a four-bit cache steps through step (or prefill_step and verify_step for host tensors)")


class DevicePagedKVCache:
    """A paged KV cache whose page bookkeeping lives on the device (kvp_dev_*).

    The same layout as :class:`PagedKVCache` (mini-sglang's 6-axis buffer, a
    block table or a raw-location table); the free list, reference counts
    and lengths are device arrays, so a decode step (:meth:`decode_step`)
    makes no host decision and copies nothing to the device but q/k/v.
    Request ids are table rows. Lengths are not mirrored on the host: the
    caller knows its own schedule.
    """

    def __init__(self, num_pages, page_size, kv_heads, head_dim, num_layers, dtype="bf16", max_requests=256,
                 table_mode="block", max_seq_len=None, free_stack=None, device="cuda", zero=True):
        self.P, self.Hkv, self.D, self.layers = page_size, kv_heads, head_dim, num_layers
        self.num_pages = num_pages
        self.tdt, kdt = _DT[dtype]
        self.raw = table_mode == "raw"
        self.dev = torch.device(device)
        extra = 1 if self.raw else 0
        alloc = torch.zeros if zero else torch.empty
        self.kv = alloc((2, num_layers, num_pages + extra, page_size, kv_heads, head_dim), dtype=self.tdt,
                        device=self.dev)
        self.pool = kb.Pool(self.kv, page_size, kdt)
        max_seq_len = max_seq_len or num_pages * page_size
        if self.raw:
            cols = _align32(min(max_seq_len, num_pages * page_size))
            self.table = torch.zeros((max_requests + 1, cols), dtype=torch.int32, device=self.dev)
            self.table[max_requests].fill_(num_pages * page_size)  # dummy row -> dummy page
        else:
            cols = -(-max_seq_len // page_size)
            self.table = torch.full((max_requests, cols), -1, dtype=torch.int32, device=self.dev)
        self.table_mode = kb.KVP_RAW_LOCATIONS if self.raw else kb.KVP_BLOCK_TABLE
        self.pages = kb.DevicePages(num_pages, page_size, max_requests, self.table, self.table_mode,
                                    free_stack=free_stack, device=self.dev)
        self.may_share = False  # set by fork: appends may then copy shared tail pages
        self._ws = {}
        self._scratch = {}
        self._staging = {}
        self._ptrs = {}

    def _i32(self, xs):
        return torch.as_tensor(list(xs), dtype=torch.int32).to(self.dev, non_blocking=True)

    def new(self, rids):
        self.pages.new(self._i32(rids))

    def append(self, rids, counts=None):
        """Append counts[i] rows (default one) to each request; returns the
        slots of the new rows on the device (request-major), after copying
        any shared tail page."""
        n = len(rids)
        total = n if counts is None else int(sum(counts))
        out_loc = torch.empty(max(total, 1), dtype=torch.int32, device=self.dev)
        cow = torch.empty((2, n), dtype=torch.int32, device=self.dev)
        n_cow = torch.zeros(1, dtype=torch.int32, device=self.dev)
        self.pages.append(self._i32(rids), out_loc, cow[0], cow[1], n_cow,
                          counts=None if counts is None else self._i32(counts))
        if self.may_share:
            kb.copy_pages_device_count(self.pool, cow[0], cow[1], n_cow)
        return out_loc[:total]

    def store(self, layer, k, v, out_loc):
        kb.store_cache(self.pool, layer, k, v, out_loc)

    def fork(self, src, dst):
        self.pages.fork(self._i32(src), self._i32(dst))
        self.may_share = True

    def trim(self, rids, window, sinks=0):
        self.pages.trim(self._i32(rids), window=window, sinks=sinks)

    def release(self, rids):
        self.pages.release(self._i32(rids))

    def rewind(self, rids, n_back):
        """Drop the newest n_back[i] rows of each request (rejected drafts)."""
        self.pages.rewind(self._i32(rids), self._i32(n_back))

    def workspace(self, batch, num_q_heads, num_q_tokens=1):
        key = (batch, num_q_heads, num_q_tokens)
        if key not in self._ws:
            self._ws[key] = (kb.alloc_workspace(self.pool, batch, num_q_heads, device=self.dev) if num_q_tokens == 1
                             else kb.alloc_verify_workspace(self.pool, batch, num_q_tokens, num_q_heads,
                                                            device=self.dev))
        return self._ws[key]

    def verify(self, layer, q, context_lens, window, scale, out, table_rows=None, sinks=0):
        """Multi-token verify attention: q/out [B, M, Hq, D] (the M newest tokens, stored)."""
        ws = self.workspace(q.shape[0], q.shape[2], q.shape[1])
        kb.paged_verify_attention(self.pool, layer, q, self.table, self.table_mode, context_lens, window, scale,
                                  out, ws, table_rows=table_rows, sinks=sinks)

    def attend(self, layer, q, context_lens, window, scale, out, table_rows=None, sinks=0):
        ws = self.workspace(q.shape[0], q.shape[1])
        kb.paged_decode_attention(self.pool, layer, q, self.table, self.table_mode, context_lens, window, scale,
                                  out, ws, table_rows=table_rows, sinks=sinks)

    def decode_step(self, rids, q, k, v, out, window, scale, sinks=0):
        """One decode step, all layers, through kvp_decode_step_device.
        ``rids``: device int32 [B]; q/k/v/out: per-layer DEVICE tensors
        ([B, Hq, D] and [B, Hkv, D]). Asynchronous: nothing is synchronised."""
        n, Hq = rids.numel(), q[0].shape[1]
        scratch = self._scratch.get(n)
        if scratch is None:
            scratch = self._scratch[n] = torch.zeros(4 * n + 1, dtype=torch.int32, device=self.dev)
        ws = self.workspace(n, Hq)
        vp = ctypes.c_void_p
        arr = lambda ts: (vp * self.layers)(*[t.data_ptr() for t in ts])  # noqa: E731
        stream = torch.cuda.current_stream(self.dev)
        kb._check(kb.lib().kvp_decode_step_device(
            self.pages.handle, self.pool.handle, vp(self.table.data_ptr()), self.table.shape[0], self.table.shape[1],
            self.table_mode, vp(rids.data_ptr()), n, int(window or 0), int(sinks), Hq, float(scale), arr(q), arr(k),
            arr(v), arr(out), None, None, vp(scratch.data_ptr()), int(self.may_share), vp(ws.data_ptr()),
            ws.numel(), vp(stream.cuda_stream)), "kvp_decode_step_device")

    def _ptr_array(self, ts):
        """ctypes array of the tensors' data pointers, cached by their addresses."""
        key = tuple(t.data_ptr() for t in ts)
        arr = self._ptrs.get(key)
        if arr is None:
            if len(self._ptrs) > 256:
                self._ptrs.clear()
            arr = self._ptrs[key] = (ctypes.c_void_p * len(ts))(*key)
        return arr

    def decode_step_host(self, rids, q, k, v, out, window, scale, sinks=0):
        """One decode step with HOST buffers (pinned): ``q``/``k``/``v``/``out``
        are per-layer host tensors; inputs are copied to device staging, the
        step runs with the bookkeeping on the device, outputs come back. One
        native call (kvp_decode_step_device_io); returns when ``out`` holds
        the results. ``rids``: device int32 [B]."""
        n, Hq = rids.numel(), q[0].shape[1]
        key = (n, Hq)
        stage = self._staging.get(key)
        if stage is None:
            mk = lambda t: torch.empty(t.shape, dtype=t.dtype, device=self.dev)  # noqa: E731
            stage = self._staging[key] = ([mk(t) for t in q], [mk(t) for t in k], [mk(t) for t in v],
                                          [mk(t) for t in out], torch.zeros(4 * n + 1, dtype=torch.int32,
                                                                            device=self.dev))
        qd, kd, vd, od, scratch = stage
        ws = self.workspace(n, Hq)
        vp = ctypes.c_void_p
        pa = self._ptr_array
        stream = torch.cuda.current_stream(self.dev)
        kb._check(kb.lib().kvp_decode_step_device_io(
            self.pages.handle, self.pool.handle, vp(self.table.data_ptr()), self.table.shape[0], self.table.shape[1],
            self.table_mode, vp(rids.data_ptr()), n, int(window or 0), int(sinks), Hq, float(scale), pa(q), pa(k),
            pa(v), pa(out), pa(qd), pa(kd), pa(vd), pa(od), vp(scratch.data_ptr()), int(self.may_share),
            vp(ws.data_ptr()), ws.numel(), vp(stream.cuda_stream)), "kvp_decode_step_device_io")

    def verify_step_host(self, rids, q, k, v, n_back, out, window, scale, sinks=0):
        """One speculative-decoding verify step with HOST buffers (pinned),
        the page bookkeeping on the device: the M drafts of every request are
        appended, stored and verified at once, then each request's rejected
        drafts (``n_back``: host int32 [B], 0..M) are rewound. ``q``/``out``
        per-layer host tensors [B, M, Hq, D], ``k``/``v`` [B * M, Hkv, D]
        (request-major); ``rids``: device int32 [B]. One native call
        (kvp_verify_step_device_io); returns when ``out`` holds the results."""
        n, M, Hq = rids.numel(), q[0].shape[1], q[0].shape[2]
        key = ("verify", n, M, Hq)
        stage = self._staging.get(key)
        if stage is None:
            mk = lambda t: torch.empty(t.shape, dtype=t.dtype, device=self.dev)  # noqa: E731
            stage = self._staging[key] = ([mk(t) for t in q], [mk(t) for t in k], [mk(t) for t in v],
                                          [mk(t) for t in out], torch.zeros(n * M + 4 * n + 1, dtype=torch.int32,
                                                                            device=self.dev))
        qd, kd, vd, od, scratch = stage
        ws = self.workspace(n, Hq, M)
        nb = np.ascontiguousarray(n_back, dtype=np.int32)
        if nb.shape != (n,):
            raise ValueError("n_back must hold one count per request")
        vp = ctypes.c_void_p
        pa = self._ptr_array
        stream = torch.cuda.current_stream(self.dev)
        kb._check(kb.lib().kvp_verify_step_device_io(
            self.pages.handle, self.pool.handle, vp(self.table.data_ptr()), self.table.shape[0], self.table.shape[1],
            self.table_mode, vp(rids.data_ptr()), n, M, int(window or 0), int(sinks), Hq, float(scale), pa(q), pa(k),
            pa(v), nb.ctypes.data_as(vp), pa(out), pa(qd), pa(kd), pa(vd), pa(od), vp(scratch.data_ptr()),
            int(self.may_share), vp(ws.data_ptr()), ws.numel(), vp(stream.cuda_stream)), "kvp_verify_step_device_io")

    def check(self):
        """Raise if a device-side error was recorded since the last check."""
        for e, what in ((kb.kvp_sync_error(self.pool), "device"), (self.pages.sync_error(), "device pages")):
            if e != 0:
                raise kb.KvpError(e, what)
