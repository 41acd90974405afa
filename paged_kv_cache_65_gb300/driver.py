"""Drive a pool through the C ABI from an operation script.

``DeviceRun`` replays ``("append", seq, n, value_seed)``, ``("fork", p, c)``
and ``("release", seq)`` operations against a ``PagedKVCache`` (host block
manager calls plus the slot-write and copy-on-write kernels), and runs decode
steps in the order "PagedAttention 的块表与碎片控制" §10 prescribes: reserve
the batch's slots on the host, upload metadata, copy shared tails, write the
new tokens, attend.  Values come from a caller-supplied function; nothing
here computes any part of the method.
"""

from __future__ import annotations

import numpy as np
import torch

from .cache import DeviceTables, PagedKVCache


class TableRun:
    """Prefill rounds and decode steps of requests whose block tables live on
    the device (``DeviceTables``): every call appends the requests' tokens to
    their rows, writes the new K/V and attends, with no host reservation, no
    upload and no synchronisation, so a captured step can be replayed.

    ``rows``: int32 device tensor of table rows (-1: a padding entry); new K/V
    ``[L, n_tokens, H_kv, D_h]`` and q ``[L, n_tokens, H_q, D_h]`` device
    tensors of the pool's input dtype, the batch's tokens in row order."""

    def __init__(self, cache: PagedKVCache, n_q_heads, n_rows, max_blocks, n_blocks, max_batch,
                 max_tokens=0):
        self.c, self.n_q_heads, self.mb = cache, n_q_heads, max_blocks
        self.t = DeviceTables.from_pool(cache, n_rows, max_blocks, n_blocks)
        dev, mt = cache.k.device, max(max_tokens, max_batch)
        i32 = dict(dtype=torch.int32, device=dev)
        self.slots = torch.empty(mt, dtype=torch.int64, device=dev)
        self.positions = torch.empty(mt, **i32)
        self.start = torch.empty(max_batch + 1, **i32)
        self.table = torch.empty((max_batch, max_blocks), **i32)
        self.lens = torch.empty(max_batch, **i32)
        u8 = dict(dtype=torch.uint8, device=dev)
        self._ws = torch.empty(cache.paged_tables_workspace_bytes(max_batch), **u8)
        self._attn = torch.empty(cache.paged_decode_workspace_bytes(max_batch, n_q_heads), **u8)
        stage = cache.paged_prefill_staging_bytes(max_batch, max_blocks) if max_tokens else 0
        self._stage = torch.empty(stage, **u8) if stage else None

    def _append(self, rows, counts, n_tokens, q, k_new, v_new, out, stream):
        n, c = rows.numel(), self.c
        if n > self.lens.numel() or n_tokens > self.slots.numel():
            raise ValueError("more rows or tokens than the run was made for")
        kv = (c.L, n_tokens, c.H, c.D)
        if (rows.dtype != torch.int32 or (counts is not None and (
                counts.dtype != torch.int32 or counts.numel() != n))):
            raise TypeError("rows and counts: int32, one count per row")
        if tuple(k_new.shape) != kv or tuple(v_new.shape) != kv or \
                tuple(q.shape) != (c.L, n_tokens, self.n_q_heads, c.D) or out.shape != q.shape or \
                not all(x.is_contiguous() for x in (q, k_new, v_new, out, rows)):
            raise ValueError("k_new, v_new [L, tokens, H_kv, D_h], q, out [L, tokens, H_q, D_h], "
                             "contiguous")
        self.c.paged_tables_append(self.t, rows, counts, n, n_tokens, self.slots, self.positions,
                                   self.start, self.table, self.lens, workspace=self._ws,
                                   stream=stream)
        return n

    def prefill(self, rows, counts, max_chunk, q, k_new, v_new, out, stream=None):
        """Append ``counts`` tokens (int32, at most ``max_chunk`` each) to the
        rows and attend them over their contexts; ``out [L, n_tokens, H_q,
        D_h]``, rows past the last token left as they were."""
        c, n_tok = self.c, k_new.shape[1]
        if self._stage is None and c.paged_prefill_staging_bytes(1, self.mb):
            raise ValueError("a run without max_tokens has no staging for prefill")
        n = self._append(rows, counts, n_tok, q, k_new, v_new, out, stream)
        c.reshape_and_cache(-1, k_new, v_new, self.slots, n_tok, stream)
        for layer in range(c.L):
            c.paged_prefill_attention_staged(layer, q[layer], self.n_q_heads, self.table, self.mb,
                                             self.start, self.lens, n, out[layer], self._stage,
                                             max_chunk=max_chunk, stream=stream)
        return out

    def step(self, rows, q, k_new, v_new, out, stream=None):
        """One decode step: a token for every listed row, padding entries last;
        ``out [L, n, H_q, D_h]``, zeros for padding entries."""
        c = self.c
        n = self._append(rows, None, rows.numel(), q, k_new, v_new, out, stream)
        c.reshape_and_cache(-1, k_new, v_new, self.slots, n, stream)
        for layer in range(c.L):
            c.paged_decode_attention(layer, q[layer], self.n_q_heads, self.table, self.mb,
                                     self.lens, n, out[layer], self._attn, 0.0, stream)
        return out

    def release(self, rows, stream=None):
        self.c.paged_tables_release(self.t, rows, rows.numel(), self._ws, stream)

    def close(self):
        """Give the ring's blocks back to the pool."""
        self.c.block_free(self.t.held)


def to_device(x: np.ndarray, dtype: str, device) -> torch.Tensor:
    """Input elements (float32, or bfloat16 bit patterns as uint16) to a
    device tensor of the pool's input dtype (bfloat16 for FP8 pools), bit for
    bit."""
    if dtype == "f32":
        return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(device)
    t = torch.from_numpy(np.ascontiguousarray(x).view(np.int16))
    return t.to(device).view(torch.bfloat16)


def to_host_bits(t: torch.Tensor) -> np.ndarray:
    if t.dtype == torch.bfloat16:
        return t.view(torch.int16).cpu().numpy().view(np.uint16)
    return t.cpu().numpy()


class DeviceRun:
    def __init__(self, cache: PagedKVCache, n_q_heads: int, stream=None):
        self.c = cache
        self.n_q_heads = n_q_heads
        self.stream = stream
        self.dev = cache.k.device
        self.lengths: dict[int, int] = {}
        self.build_cows = []
        self._ws = None
        self._stage_ws = None

    # -------------------------------------------------------------- build
    def apply(self, op, values_fn) -> None:
        kind = op[0]
        c = self.c
        if kind == "append":
            _, seq, n, vseed = op
            slots, pairs = c.seq_append_tokens(seq, n)
            if len(pairs):
                self.build_cows.extend(tuple(p) for p in pairs)
                d_pairs = torch.from_numpy(np.ascontiguousarray(pairs)).to(self.dev)
                c.cow_copy(d_pairs, len(pairs), self.stream)
            if n:
                k, v = values_fn(vseed, n)  # [L, n, H_kv, D_h] stored elements
                dk = to_device(k, c.dtype, self.dev)
                dv = to_device(v, c.dtype, self.dev)
                ds = torch.from_numpy(slots).to(self.dev)
                c.reshape_and_cache(-1, dk, dv, ds, n, self.stream)
            self.lengths[seq] = self.lengths.get(seq, 0) + n
        elif kind == "fork":
            c.seq_fork(op[1], op[2])
            self.lengths[op[2]] = self.lengths[op[1]]
        elif kind == "release":
            c.seq_release(op[1])
            self.lengths.pop(op[1], None)
        else:
            raise ValueError(kind)

    # -------------------------------------------------------------- steps
    def reserve(self, seq_ids):
        slots, pairs = self.c.seq_append_slots(seq_ids)
        for s in seq_ids:
            self.lengths[s] = self.lengths.get(s, 0) + 1
        return slots, pairs

    def max_blocks(self, seq_ids) -> int:
        B = self.c.B
        return max(1, max(-(-self.lengths[s] // B) for s in seq_ids))

    def workspace(self, n_seq: int) -> torch.Tensor:
        nbytes = self.c.paged_decode_workspace_bytes(n_seq, self.n_q_heads)
        if self._ws is None or self._ws.numel() < nbytes:
            self._ws = torch.empty(nbytes, dtype=torch.uint8, device=self.dev)
        return self._ws

    def write(self, slots, pairs, k_new: np.ndarray, v_new: np.ndarray) -> None:
        c = self.c
        if len(pairs):
            d_pairs = torch.from_numpy(np.ascontiguousarray(pairs)).to(self.dev)
            c.cow_copy(d_pairs, len(pairs), self.stream)
        dk = to_device(k_new, c.dtype, self.dev)
        dv = to_device(v_new, c.dtype, self.dev)
        ds = torch.from_numpy(np.ascontiguousarray(slots)).to(self.dev)
        c.reshape_and_cache(-1, dk, dv, ds, len(slots), self.stream)

    def tables(self, seq_ids, max_blocks=None):
        mb = max_blocks or self.max_blocks(seq_ids)
        table, lens = self.c.seq_block_table(seq_ids, mb)
        return (torch.from_numpy(table).to(self.dev), torch.from_numpy(lens).to(self.dev), mb)

    def attend(self, layer, q_dev, d_table, max_blocks, d_lens, n_seq, out=None,
               out_dtype=torch.float32):
        c = self.c
        if out is None:
            out = torch.empty((n_seq, self.n_q_heads, c.D), dtype=out_dtype, device=self.dev)
        c.paged_decode_attention(layer, q_dev, self.n_q_heads, d_table, max_blocks, d_lens, n_seq,
                                 out, self.workspace(n_seq), 0.0, self.stream)
        return out

    def plan(self, seq_ids, max_blocks, min_shared_tokens=0):
        """Host plan of the sharing-aware pass and its device copy."""
        buf, ws_bytes = self.c.paged_decode_plan(seq_ids, self.n_q_heads, max_blocks,
                                                 min_shared_tokens)
        return buf, torch.from_numpy(buf).to(self.dev), ws_bytes

    def attend_planned(self, layer, q_dev, d_table, max_blocks, h_plan, d_plan, ws_bytes,
                       out=None, out_dtype=torch.float32):
        c = self.c
        n_seq = int(q_dev.shape[0])
        if out is None:
            out = torch.empty((n_seq, self.n_q_heads, c.D), dtype=out_dtype, device=self.dev)
        if self._ws is None or self._ws.numel() < ws_bytes:
            self._ws = torch.empty(ws_bytes, dtype=torch.uint8, device=self.dev)
        c.paged_decode_attention_planned(layer, q_dev, self.n_q_heads, d_table, max_blocks, d_plan,
                                         h_plan, out, self._ws, 0.0, self.stream)
        return out

    def step(self, seq_ids, q: np.ndarray, k_new: np.ndarray, v_new: np.ndarray, planned=False):
        """q ``[n_seq, H_q, D_h]`` (or ``[L, n_seq, H_q, D_h]``), new K/V
        ``[L, n_seq, H_kv, D_h]``.  Returns slots, pairs and float32 outputs
        ``[L, n_seq, H_q, D_h]`` on the device."""
        slots, pairs = self.reserve(seq_ids)
        self.write(slots, pairs, k_new, v_new)
        d_table, d_lens, mb = self.tables(seq_ids)
        L = self.c.L
        qd = to_device(q, self.c.dtype, self.dev)
        outs = []
        if planned:
            h_plan, d_plan, ws_bytes = self.plan(seq_ids, mb)
        for layer in range(L):
            ql = qd[layer] if qd.dim() == 4 else qd
            if planned:
                outs.append(self.attend_planned(layer, ql, d_table, mb, h_plan, d_plan, ws_bytes))
            else:
                outs.append(self.attend(layer, ql, d_table, mb, d_lens, len(seq_ids)))
        return slots, pairs, torch.stack(outs)

    def prefill_step(self, chunks, q: np.ndarray, k_new: np.ndarray, v_new: np.ndarray,
                     out_dtype=None, max_chunk=None, scheduled=False):
        """A chunked-prefill round: for each ``(seq, c)`` of ``chunks`` reserve
        ``c`` slots, copy any shared tail, write the chunk's K/V (all layers),
        then attend the chunk's queries over the sequence's context.  ``q``
        ``[n_tok, H_q, D_h]`` (chunks in order), ``k_new, v_new [L, n_tok,
        H_kv, D_h]``.  ``scheduled`` launches the work items heaviest first
        (``paged_prefill_schedule``).  Returns the outputs ``[L, n_tok, H_q,
        D_h]``."""
        import torch

        c = self.c
        seqs = [s for s, _ in chunks]
        t = 0
        for seq, n in chunks:
            if n:
                slots, pairs = c.seq_append_tokens(seq, n)
                if len(pairs):
                    d_pairs = torch.from_numpy(np.ascontiguousarray(pairs)).to(self.dev)
                    c.cow_copy(d_pairs, len(pairs), self.stream)
                dk = to_device(np.ascontiguousarray(k_new[:, t:t + n]), c.dtype, self.dev)
                dv = to_device(np.ascontiguousarray(v_new[:, t:t + n]), c.dtype, self.dev)
                c.reshape_and_cache(-1, dk, dv, torch.from_numpy(slots).to(self.dev), n,
                                    self.stream)
            self.lengths[seq] = self.lengths.get(seq, 0) + n
            t += n
        d_table, d_lens, mb = self.tables(seqs)
        starts = np.zeros(len(chunks) + 1, dtype=np.int32)
        starts[1:] = np.cumsum([n for _, n in chunks])
        d_starts = torch.from_numpy(starts).to(self.dev)
        qd = to_device(q, c.dtype, self.dev)
        dt = out_dtype or torch.float32
        mc = max_chunk if max_chunk is not None else max([n for _, n in chunks] + [0])
        if scheduled:
            sched = c.paged_prefill_schedule(starts, d_lens.cpu().numpy(), self.n_q_heads)
            d_sched = torch.from_numpy(sched).to(self.dev)
        outs = []
        staged = c.dtype in ("fp8_e4m3", "q4_0")  # through a 16-bit copy
        if staged:
            nbytes = c.paged_prefill_staging_bytes(len(chunks), mb)
            if self._stage_ws is None or self._stage_ws.numel() < nbytes:
                self._stage_ws = torch.empty(nbytes, dtype=torch.uint8, device=self.dev)
        for layer in range(c.L):
            out = torch.zeros((int(starts[-1]), self.n_q_heads, c.D), dtype=dt, device=self.dev)
            if staged:
                c.paged_prefill_attention_staged(
                    layer, qd, self.n_q_heads, d_table, mb, d_starts, d_lens, len(chunks), out,
                    self._stage_ws, max_chunk=0 if scheduled else mc,
                    d_sched=d_sched if scheduled else None,
                    n_items=len(sched) if scheduled else 0, stream=self.stream)
            elif scheduled:
                c.paged_prefill_attention_scheduled(layer, qd, self.n_q_heads, d_table, mb,
                                                    d_starts, d_lens, len(chunks), d_sched,
                                                    len(sched), out, 0.0, self.stream)
            else:
                c.paged_prefill_attention(layer, qd, self.n_q_heads, d_table, mb, d_starts,
                                          d_lens, len(chunks), mc, out, 0.0, self.stream)
            outs.append(out)
        return torch.stack(outs)

