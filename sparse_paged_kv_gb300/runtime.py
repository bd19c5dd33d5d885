"""Device buffers of one Locks decode layer, held in torch CUDA tensors.

``LocksLayer`` owns the paged K/V pools, the block table, the summary pool and
the workspaces of one attention layer and calls the C-ABI entry points on
them.  PyTorch only provides memory and streams; every step runs in the
library's kernels.
"""
from __future__ import annotations

import contextlib
import dataclasses
import math
from typing import Optional

import numpy as np

from . import binding as B


def complete_page_blocks(block_table: np.ndarray, seq_lens: np.ndarray, page_size: int) -> np.ndarray:
    """Physical blocks of every complete page (host arrays in, int32 out)."""
    out = []
    for b, t in enumerate(seq_lens.tolist()):
        n_complete = int(t) // page_size
        out.append(block_table[b, :n_complete])
    return np.concatenate(out).astype(np.int32) if out else np.zeros(0, np.int32)


class RopeTable:
    """Rotary frequencies of one model, on the device: the rates of the pairs as fractions of a
    turn per position, the layout of the pairs and the factor on cos and sin.  `scaling` is
    "none", "linear", "ntk", "llama3" or "yarn" (see locks_rope_frequencies)."""

    LAYOUTS = {"half": B.LOCKS_ROPE_HALF, "interleaved": B.LOCKS_ROPE_INTERLEAVED}
    SCALINGS = {"none": B.LOCKS_ROPE_SCALE_NONE, "linear": B.LOCKS_ROPE_SCALE_LINEAR,
                "ntk": B.LOCKS_ROPE_SCALE_NTK, "llama3": B.LOCKS_ROPE_SCALE_LLAMA3,
                "yarn": B.LOCKS_ROPE_SCALE_YARN}

    def __init__(self, rotary_dim: int, theta: float = 10000.0, layout: str = "half",
                 scaling: str = "none", factor: float = 1.0, low_freq_factor: float = 1.0,
                 high_freq_factor: float = 4.0, original_positions: float = 8192.0,
                 beta_fast: float = 32.0, beta_slow: float = 1.0, device: str = "cuda"):
        import ctypes

        import torch
        if layout not in self.LAYOUTS or scaling not in self.SCALINGS:
            raise ValueError(f"layout one of {sorted(self.LAYOUTS)}, scaling one of "
                             f"{sorted(self.SCALINGS)} expected")
        spec = B.locks_rope_spec_t(rotary_dim, self.SCALINGS[scaling], theta, factor,
                                   low_freq_factor, high_freq_factor, original_positions,
                                   beta_fast, beta_slow)
        turns, self.mscale = B.rope_frequencies(spec)
        self.rotary_dim, self.layout = rotary_dim, layout
        self.turns = torch.from_numpy(turns.view(np.int64)).to(device)
        self._c = B.locks_rope_table_t(self.turns.data_ptr(), rotary_dim, self.LAYOUTS[layout],
                                       self.mscale)
        self.ref = ctypes.byref(self._c)


class LocksLayer:
    def __init__(self, cfg: B.LocksConfig, budget_tokens: int, device: str = "cuda"):
        import torch
        self.torch = torch
        self.cfg = cfg
        self.budget = int(budget_tokens)
        self.k = cfg.page_budget(self.budget)
        self.device = device
        d = device
        self.rec_bytes = B.summary_record_bytes(cfg)
        if self.rec_bytes == 0:
            raise B.LocksError("locks_summary_record_bytes", B.LOCKS_ERR_UNSUPPORTED, "unsupported cfg")
        self.summaries = torch.zeros((cfg.num_blocks, cfg.n_kv_heads, self.rec_bytes),
                                     dtype=torch.uint8, device=d)
        self.ws_select = torch.zeros(max(1, B.select_workspace_bytes(cfg, self.budget)),
                                     dtype=torch.uint8, device=d)
        self.ws_sparse = torch.zeros(max(1, B.decode_workspace_bytes(cfg, self.k)),
                                     dtype=torch.uint8, device=d)
        self.ws_dense = torch.zeros(max(1, B.decode_workspace_bytes(cfg, cfg.max_pages)),
                                    dtype=torch.uint8, device=d)
        self.selected = torch.full((cfg.batch, cfg.n_kv_heads, self.k), -1, dtype=torch.int32, device=d)
        self.out = torch.zeros((cfg.batch, cfg.n_q_heads, cfg.head_dim), dtype=torch.bfloat16, device=d)
        self.out_lse = torch.zeros((cfg.batch, cfg.n_q_heads), dtype=torch.float32, device=d)
        self.out_dense = torch.zeros_like(self.out)
        self.out_dense_lse = torch.zeros_like(self.out_lse)
        self.status = torch.zeros(1, dtype=torch.int32, device=d)
        self.q = self.k_cache = self.v_cache = self.block_table = self.seq_lens = None

    # ---- inputs -------------------------------------------------------------
    def load_inputs(self, inputs) -> "LocksLayer":
        """Copy seeded host inputs (workloads.LocksInputs) into device memory."""
        torch = self.torch
        d = self.device

        def bf16(a):
            return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to(d).view(torch.bfloat16)

        self.q = bf16(inputs.q)
        self.k_cache = bf16(inputs.k_cache)
        self.v_cache = bf16(inputs.v_cache)
        self.block_table = torch.from_numpy(inputs.block_table).to(d)
        self.seq_lens = torch.from_numpy(inputs.seq_lens).to(d)
        self.host_block_table = inputs.block_table
        self.host_seq_lens = inputs.seq_lens
        return self

    @classmethod
    def from_inputs(cls, inputs, summary_dtype: int = B.LOCKS_SUMMARY_F32,
                    budget_tokens: Optional[int] = None) -> "LocksLayer":
        w = inputs.workload
        cfg = B.LocksConfig.from_workload(w, summary_dtype)
        return cls(cfg, w.budget_tokens if budget_tokens is None else budget_tokens).load_inputs(inputs)

    def sharing_inputs(self, summary_dtype: int) -> "LocksLayer":
        """A layer over the same device inputs (q, K/V pools, block table,
        sequence lengths) with its own summary pool of another record type."""
        cfg = dataclasses.replace(self.cfg, summary_dtype=int(summary_dtype))
        other = LocksLayer(cfg, self.budget, self.device)
        for name in ("q", "k_cache", "v_cache", "block_table", "seq_lens", "host_block_table",
                     "host_seq_lens"):
            setattr(other, name, getattr(self, name))
        return other

    # ---- calls ----------------------------------------------------------------
    def build(self, block_ids=None, tail_energy=None, status=None, max_sweeps: int = 0):
        torch = self.torch
        if block_ids is None:
            ids = complete_page_blocks(self.host_block_table, self.host_seq_lens, self.cfg.page_size)
            block_ids = torch.from_numpy(ids).to(self.device)
        if block_ids.numel() == 0:
            return block_ids
        B.locks_build_summaries(self.cfg, self.k_cache, block_ids, self.summaries,
                                tail_energy=tail_energy, status=status, max_sweeps=max_sweeps)
        return block_ids

    def select(self, page_lse=None, page_share=None, stream=None):
        B.locks_select(self.cfg, self.q, self.summaries, self.block_table, self.seq_lens,
                       self.budget, self.selected, self.ws_select, page_lse=page_lse,
                       page_share=page_share, status=self.status, stream=stream)

    def sparse_decode(self, stream=None):
        B.locks_sparse_decode(self.cfg, self.q, self.k_cache, self.v_cache, self.block_table,
                              self.seq_lens, self.selected, self.k, self.out, self.ws_sparse,
                              out_lse=self.out_lse, status=self.status, stream=stream)

    def dense_decode(self, stream=None):
        B.locks_dense_decode(self.cfg, self.q, self.k_cache, self.v_cache, self.block_table,
                             self.seq_lens, self.out_dense, self.ws_dense,
                             out_lse=self.out_dense_lse, status=self.status, stream=stream)

    def step(self, stream=None):
        """One sparse decode step: selection, then attention over the selected pages."""
        self.select(stream=stream)
        self.sparse_decode(stream=stream)

    def capture_step(self):
        """A CUDA graph of one sparse decode step (selection, then attention)
        over this layer's buffers.  replay() runs it on the current stream and
        reads q, seq_lens and block_table as they are at replay time.  The
        step runs once outside the capture first, so one-time launch set-up
        (kernel attributes, the cluster-size query) never happens inside it."""
        torch = self.torch
        cur = torch.cuda.current_stream(self.device)
        side = torch.cuda.Stream(device=self.device)
        side.wait_stream(cur)
        with torch.cuda.stream(side):
            self.step()
        cur.wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph

    def append(self, k_new, v_new, completed=None, stream=None):
        """Write each sequence's new token (k_new, v_new: bf16 [batch][H_kv][d]
        on the device) at position seq_lens[b], advance seq_lens, and store in
        `completed` (int32 [batch]) the block of each page the token completed
        (-1 for none)."""
        B.locks_append_kv(self.cfg, k_new, v_new, self.k_cache, self.v_cache, self.block_table,
                          self.seq_lens, completed=completed, status=self.status, stream=stream)

    def build_completed(self, completed, status=None, stream=None):
        """Summaries of the blocks listed in `completed` (entries < 0 skipped)."""
        B.locks_build_completed(self.cfg, self.k_cache, completed, self.summaries, status=status,
                                stream=stream)

    # ---- diagnostics ------------------------------------------------------------
    def host_records(self, blocks, h: int):
        """(mu, V, C) of the given physical blocks for KV head h (float64, host)."""
        raw = self.summaries[self.torch.as_tensor(np.asarray(blocks), device=self.device).long(), h]
        return B.unpack_records(raw.cpu().numpy(), self.cfg)

    def alloc_page_lse(self):
        c = self.cfg
        return self.torch.full((c.batch, c.n_q_heads, c.max_pages), float("nan"),
                               dtype=self.torch.float32, device=self.device)

    def alloc_page_share(self):
        c = self.cfg
        return self.torch.full((c.batch, c.n_kv_heads, c.max_pages), float("nan"),
                               dtype=self.torch.float32, device=self.device)


class QuantCache:
    """The quantised paged cache of one attention layer: pools of e4m3, int8 or
    int4 records, their block table and lengths, and the buffers of a decode
    step.  Queries and keys are rotated by `rope` (a RopeTable, or None) as
    tokens are written; attention reads the codes.

    With `budget_tokens` the steps attend only the pages that the Locks
    selection keeps: summaries are built from complete pages read back out of
    the cache (what the attention will see of them), and each step selects
    before it attends.  The selection's limits then hold: pages of 64 or 16, 1,
    2, 4 or 8 query heads a KV head, and 2 to 256 pages of budget."""

    def __init__(self, cfg: B.LocksKvConfig, block_table, rope: Optional[RopeTable] = None,
                 budget_tokens: int = 0, rank: int = 8,
                 summary_dtype: int = B.LOCKS_SUMMARY_F32, device: str = "cuda"):
        import torch
        self.torch, self.cfg, self.rope, self.device = torch, cfg, rope, device
        rec = B.kv_record_bytes(cfg)
        if rec == 0:
            raise B.LocksError("locks_kv_record_bytes", B.LOCKS_ERR_UNSUPPORTED, "unsupported cfg")

        def zeros(*shape, dtype=torch.uint8):
            return torch.zeros(shape, dtype=dtype, device=device)

        self.k_pool = zeros(cfg.num_blocks, cfg.n_kv_heads, rec)
        self.v_pool = zeros(cfg.num_blocks, cfg.n_kv_heads, rec)
        self.block_table = torch.as_tensor(np.asarray(block_table, np.int32)).to(device)
        self.seq_lens = zeros(cfg.batch, dtype=torch.int32)
        self.positions = zeros(cfg.batch, dtype=torch.int32)    # of a step's tokens
        self.workspace = zeros(max(1, B.kv_decode_workspace_bytes(cfg)))
        rows = (cfg.batch, cfg.n_q_heads, cfg.head_dim)
        self.q = zeros(*rows, dtype=torch.bfloat16)             # rotated query of a step
        self.out = zeros(*rows, dtype=torch.bfloat16)
        self.out_lse = zeros(*rows[:2], dtype=torch.float32)
        self.completed = torch.full((cfg.batch,), -1, dtype=torch.int32, device=device)
        self.status = zeros(1, dtype=torch.int32)
        self.selected = None
        if budget_tokens:
            self.budget = int(budget_tokens)
            self.locks_cfg = B.LocksConfig(
                batch=cfg.batch, n_q_heads=cfg.n_q_heads, n_kv_heads=cfg.n_kv_heads,
                head_dim=cfg.head_dim, page_size=cfg.page_size, rank=rank,
                max_pages=cfg.max_pages, num_blocks=cfg.num_blocks, summary_dtype=summary_dtype)
            summary = B.summary_record_bytes(self.locks_cfg)
            if summary == 0:
                raise B.LocksError("locks_summary_record_bytes", B.LOCKS_ERR_UNSUPPORTED,
                                   "unsupported cfg")
            k = self.locks_cfg.page_budget(self.budget)
            if not 2 <= k <= 256:      # here, and not by a step that has written its token
                raise B.LocksError("locks_select", B.LOCKS_ERR_UNSUPPORTED,
                                   f"budget_tokens {budget_tokens}: 2 to 256 pages expected")
            # one record row more than blocks: where "no page" entries of a step's list go
            self.summaries = zeros(cfg.num_blocks + 1, cfg.n_kv_heads, summary)
            self.ws_select = zeros(max(1, B.select_workspace_bytes(self.locks_cfg, self.budget)))
            self.selected = torch.full((cfg.batch, cfg.n_kv_heads, k), -1, dtype=torch.int32,
                                       device=device)

    # ---- writing ----------------------------------------------------------------
    def write(self, q, k, v, token_seq, token_pos, q_out=None, completed=None, stream=None):
        """Tokens of prompts or chunks of them: k, v (and q, rotated into q_out) bf16
        [tokens][heads][d], slices of one projection's output allowed; token_seq, token_pos
        int32 [tokens] on the device.  Raises seq_lens to cover them."""
        B.locks_kv_write(self.cfg, k, v, token_pos, self.k_pool, self.v_pool, self.block_table,
                         token_seq=token_seq, rope=self.rope, q=q, q_out=q_out,
                         seq_lens=self.seq_lens, completed=completed, status=self.status,
                         stream=stream)

    def append(self, q, k, v, stream=None):
        """One token per sequence at its current length: q rotated into self.q, the blocks of
        pages it completed in self.completed (-1 for none)."""
        with self._on(stream):
            self.positions.copy_(self.seq_lens)
        B.locks_kv_write(self.cfg, k, v, self.positions, self.k_pool, self.v_pool,
                         self.block_table, rope=self.rope, q=q, q_out=self.q,
                         seq_lens=self.seq_lens, completed=self.completed, status=self.status,
                         stream=stream)

    def read(self, block_ids, values: bool = True, stream=None):
        """(keys, values) of the listed blocks as bf16 pages [blocks][H_kv][page_size][d]."""
        c, n = self.cfg, block_ids.numel()
        with self._on(stream):
            out = [self.torch.zeros((n, c.n_kv_heads, c.page_size, c.head_dim),
                                    dtype=self.torch.bfloat16, device=self.device)
                   for _ in range(2 if values else 1)]
        B.locks_kv_read(c, self.k_pool, self.v_pool if values else None, block_ids, out[0],
                        out[1] if values else None, status=self.status, stream=stream)
        return (out[0], out[1]) if values else out[0]

    # ---- attention ----------------------------------------------------------------
    def attend(self, q=None, selected=None, window: int = 0, stream=None):
        """Attention of q (self.q where it is None) over the cache, into self.out and
        self.out_lse: every page, the pages in `selected`, or the last `window` positions."""
        B.locks_kv_decode(self.cfg, self.q if q is None else q, self.k_pool, self.v_pool,
                          self.block_table, self.seq_lens, self.out, self.workspace,
                          selected=selected, window=window, out_lse=self.out_lse,
                          status=self.status, stream=stream)

    def step(self, q, k, v, window: int = 0, stream=None):
        """One decode step: rotate and write each sequence's token, select pages (with a
        budget), attend."""
        self.append(q, k, v, stream=stream)
        if self.selected is not None:
            B.locks_select(self.locks_cfg, self.q, self.summaries, self.block_table, self.seq_lens,
                           self.budget, self.selected, self.ws_select, status=self.status,
                           stream=stream)
        self.attend(selected=self.selected, window=window, stream=stream)

    def capture_step(self, q, k, v, window: int = 0):
        """A CUDA graph of step() over these buffers: fill q, k, v and replay.  The step runs
        once before the capture, on the sequences as they are, and is taken back: every buffer
        of a step holds what it held (a list of completed pages that is still to be built, for
        one), but the token's slots in the pools, which the first replay writes again, and the
        bits in status."""
        torch = self.torch
        held = [(x, x.clone()) for x in (self.seq_lens, self.completed, self.positions, self.q,
                                         self.out, self.out_lse, self.selected) if x is not None]
        cur = torch.cuda.current_stream(self.device)
        side = torch.cuda.Stream(device=self.device)
        side.wait_stream(cur)
        with torch.cuda.stream(side):
            self.step(q, k, v, window)
        cur.wait_stream(side)
        for x, before in held:
            x.copy_(before)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step(q, k, v, window)
        return graph

    # ---- summaries ------------------------------------------------------------------
    def build(self, block_ids, pages_at_once: int = 1024, stream=None):
        """Summaries of complete pages (int32 block ids on the device; entries < 0 are
        skipped, those past the pool also flagged in status), from their keys as the cache
        holds them."""
        if self.selected is None:
            raise ValueError("a QuantCache made without budget_tokens keeps no summaries")
        torch, c = self.torch, self.locks_cfg
        with self._on(stream):
            for at in range(0, block_ids.numel(), pages_at_once):
                ids = block_ids[at:at + pages_at_once].contiguous()
                n = ids.numel()
                cfg = dataclasses.replace(c, num_blocks=n)
                pages = self.read(ids, values=False)
                made = torch.zeros((n, *self.summaries.shape[1:]), dtype=torch.uint8,
                                   device=self.device)
                # (the read has flagged the ids past the pool, which the copy below must not see)
                there = (ids >= 0) & (ids < c.num_blocks)
                slots = torch.where(there, torch.arange(n, dtype=torch.int32, device=self.device), -1)
                B.locks_build_completed(cfg, pages, slots, made)
                self.summaries.index_copy_(0, torch.where(there, ids, c.num_blocks).long(), made)

    def build_completed(self, stream=None):
        """Summaries of the pages that the last append completed; needed before the next
        step selects.  The list stays on the device."""
        self.build(self.completed, stream=stream)

    def _on(self, stream):
        """Torch's work on `stream`: a torch stream, a cudaStream_t as an integer, or None."""
        if stream is None:
            return contextlib.nullcontext()
        cuda = self.torch.cuda
        if isinstance(stream, int):
            stream = cuda.ExternalStream(stream) if stream else cuda.default_stream()
        return cuda.stream(stream)


class DecodeLoop:
    """Decode steps of one layer as an engine runs them, with no host round
    trip: each step appends the new token (current stream), builds the
    summary of any page that token completed on a side stream, then selects
    and decodes.  A page completed at step s becomes a selection candidate at
    step s + 1, so its build overlaps step s's selection and decode, and step
    s + 1's selection waits for it (section 4 "Build": one build per
    finalised page, off the critical path).  Two `completed` buffers
    alternate, so a step's append never overwrites the list the previous
    step's build may still be reading."""

    def __init__(self, layer: LocksLayer, host_lengths=None):
        """host_lengths: optional int array of the sequences' current lengths
        as the caller tracks them (an engine knows them: it allocates a block
        for each page a sequence starts).  With them, a step in which no
        sequence completes a page launches no build; which blocks are built
        is still decided on the device, from the `completed` list."""
        import torch
        self.torch = torch
        self.layer = layer
        self.side = torch.cuda.Stream(device=layer.device)
        self.completed = [torch.full((layer.cfg.batch,), -1, dtype=torch.int32,
                                     device=layer.device) for _ in range(2)]
        self.appended = torch.cuda.Event()
        self.built = None             # event: the previous step's build is done
        self.steps = 0
        self.host_lengths = None if host_lengths is None else np.array(host_lengths, dtype=np.int64)

    def step(self, k_new, v_new, page_lse=None, page_share=None):
        torch = self.torch
        L = self.layer
        cur = torch.cuda.current_stream(L.device)
        done = self.completed[self.steps & 1]
        L.append(k_new, v_new, completed=done, stream=cur)
        crosses = True
        if self.host_lengths is not None:
            crosses = bool(((self.host_lengths + 1) % L.cfg.page_size == 0).any())
            self.host_lengths += 1
        built = None
        if crosses:
            self.appended.record(cur)
            self.side.wait_event(self.appended)
            L.build_completed(done, stream=self.side)
            built = torch.cuda.Event()
            built.record(self.side)
        if self.built is not None:
            cur.wait_event(self.built)
        self.built = built
        L.select(page_lse=page_lse, page_share=page_share, stream=cur)
        L.sparse_decode(stream=cur)
        self.steps += 1

    def finish(self):
        """Make the current stream wait for the last step's build."""
        if self.built is not None:
            self.torch.cuda.current_stream(self.layer.device).wait_event(self.built)
