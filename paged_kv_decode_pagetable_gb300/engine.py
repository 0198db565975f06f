"""One layer's decode step and a continuous-batching driver over the C ABI.

The step follows the write-then-attend order of "unsloth: compare
main...flex-moe-qwen3" · flex_gemma4_moe.py · attention forward: per-head
q/k RMSNorm, RoPE, the paged write of the new K/V, then attention over keys
0..pos. By default the whole step is one fused libpkv kernel (plus the split
combine); the three separate kernels remain available. Everything runs on
the caller's stream with fixed shapes, so a step can be captured in a CUDA
graph (the pages capture the decode step per batch bucket,
capture_decode_cudagraph).

The driver applies a schedule of finished / admitted requests to the
PageTable the way the pages' generate loop does (free on finish, assign a
new request, grow capacity by reserve before each decode step) and yields
the per-step batch_idx / input_pos / seq_lens.
"""
from __future__ import annotations

import dataclasses

import numpy as np
import torch

from . import (NoPagesError, NoSlotError, PageTable, PKV_ERR_TIMEOUT, _stream, kv_append,
               kv_append_q8, kv_copy_pages, paged_decode_attn, paged_decode_attn_q8,
               paged_decode_attn_q8_workspace, paged_decode_attn_splits,
               paged_decode_attn_workspace, paged_decode_step, paged_decode_step_ex,
               pkv_read_error_word, pt_get_stream, qk_norm_rope, qkv_norm_rope)


@dataclasses.dataclass(frozen=True)
class LayerSpec:
    head_dim: int
    theta: float
    window: int = 0
    qk_norm: bool = False
    rope: bool = True
    rotary_dims: int = 0      # 0: all of head_dim; fewer: Gemma-4 proportional RoPE
    v_norm: bool = False      # Gemma-4 gain-free RMSNorm of the value
    k_eq_v: bool = False      # Gemma-4 K=V: the value is the raw k projection

    @property
    def gemma_options(self) -> bool:
        return bool(self.rotary_dims) or self.v_norm or self.k_eq_v


def alloc_cache(Hkv: int, n_pages: int, page_size: int, D: int, device, fill: str = "zeros"):
    """K and V caches, bf16 [Hkv][n_pages * page_size][D]."""
    shape = (Hkv, n_pages * page_size, D)
    if fill == "randn":
        k = torch.randn(shape, dtype=torch.bfloat16, device=device)
        v = torch.randn(shape, dtype=torch.bfloat16, device=device)
    else:
        k = torch.zeros(shape, dtype=torch.bfloat16, device=device)
        v = torch.zeros(shape, dtype=torch.bfloat16, device=device)
    return k, v


def alloc_cache_q8(Hkv: int, n_pages: int, page_size: int, D: int, device,
                   scale_block: int = 16):
    """K and V caches in 8 bits with a scale per kv head and scale_block tokens:
    (k, v, k_scale, v_scale), e4m3 [Hkv][n_pages * page_size][D] and fp32
    [Hkv][n_pages * page_size / scale_block], zeroed."""
    rows = n_pages * page_size
    k, v = (torch.zeros((Hkv, rows, D), dtype=torch.uint8, device=device)
            .view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.zeros((Hkv, rows // scale_block), device=device) for _ in range(2))
    return k, v, ks, vs


class AttnWorkspaceQ8:
    """Workspace of the 8-bit cache's attention: sized by the heads alone, zeroed
    once."""

    def __init__(self, Hq, Hkv, D, device):
        self.buf = torch.zeros(paged_decode_attn_q8_workspace(Hq, Hkv, D), dtype=torch.uint8,
                               device=device)

    def reset(self):
        """Zeroes it again (on the current stream), as after a call that reported
        PKV_ERR_TIMEOUT."""
        self.buf.zero_()


class AttnWorkspace:
    """Split mode and workspace for one (B, Hq, Hkv, D, table, window) shape.

    num_splits 0 is the automatic, length-balanced mode; the workspace is
    sized for the most parts a row can be cut into in that mode. It starts
    zeroed: a zero partial word is one not yet written in the current call
    (each call clears what it read, leaving the workspace zero)."""

    def __init__(self, B, Hq, Hkv, D, max_pages_per_seq, page_size, window, device,
                 num_splits: int = 0):
        self.splits = num_splits
        self.max_parts = num_splits or paged_decode_attn_splits(B, Hkv, D, max_pages_per_seq,
                                                                page_size, window)
        n = paged_decode_attn_workspace(B, Hq, D, self.max_parts)
        self.buf = torch.zeros(n, dtype=torch.uint8, device=device) if n else None

    def reset(self):
        """Zeroes it again (on the current stream), as after a call that reported
        PKV_ERR_TIMEOUT."""
        if self.buf is not None:
            self.buf.zero_()


def decode_layer_step(spec: LayerSpec, pt: PageTable, k_cache, v_cache, q, k, v, batch_idx,
                      input_pos, seq_lens, out, ws: AttnWorkspace, gamma_q=None, gamma_k=None,
                      eps: float = 1e-6, scale: float | None = None, err=None, stream=None,
                      table=None, fused: bool = True, k_scale=None, v_scale=None):
    """One layer's decode step: q/k norm + RoPE, K/V append, attention.

    k_scale and v_scale given: the caches are 8-bit ones (alloc_cache_q8) and ws an
    AttnWorkspaceQ8; the step is then the chain qk_norm_rope (qkv_norm_rope) ->
    kv_append_q8 -> paged_decode_attn_q8, whatever `fused` is (q and k are rotated in place).

    err: an int32 word for the kernels' error bits. After PKV_ERR_TIMEOUT the workspace
    must be reset (ws.reset()) before its next use.

    fused (default, rotary layers): one paged_decode_step(_ex) call; q, k and
    v are read only and seq_lens must equal input_pos + 1 (the kernel derives
    it). Otherwise the chain qk_norm_rope (qkv_norm_rope with the Gemma-4
    options) -> kv_append -> paged_decode_attn, which rotates q and k (and
    normalises v) in place; both give the same bits.

    `pt` supplies the table geometry (n_slots, max_pages_per_seq, page_size,
    n_pages) and, unless `table` is given, the device table itself."""
    table = pt.dev_table if table is None else table
    scale = scale if scale is not None else spec.head_dim ** -0.5
    gq = gamma_q if spec.qk_norm else None
    gk = gamma_k if spec.qk_norm else None
    if spec.gemma_options and not spec.rope:
        raise ValueError("rotary_dims, v_norm and k_eq_v need a rotary layer")
    q8 = k_scale is not None
    if q8 != (v_scale is not None):
        raise ValueError("give both k_scale and v_scale, or neither")
    if fused and spec.rope and not q8:
        if spec.gemma_options:
            paged_decode_step_ex(q, k, v, gq, gk, batch_idx, input_pos, spec.theta, eps,
                                 spec.rotary_dims or None, spec.v_norm, spec.k_eq_v, table,
                                 pt.n_slots, pt.max_pages_per_seq, pt.page_size, pt.n_pages,
                                 k_cache, v_cache, spec.window, scale, ws.splits, ws.buf, out,
                                 err, stream=stream)
        else:
            paged_decode_step(q, k, v, gq, gk, batch_idx, input_pos, spec.theta, eps, table,
                              pt.n_slots, pt.max_pages_per_seq, pt.page_size, pt.n_pages,
                              k_cache, v_cache, spec.window, scale, ws.splits, ws.buf, out,
                              err, stream=stream)
        return
    if spec.k_eq_v:
        v = k.clone()        # the raw k row, before k is rotated in place
    if spec.gemma_options:
        qkv_norm_rope(q, k, v if spec.v_norm else None, gq, gk, input_pos, spec.theta, eps,
                      spec.rotary_dims or None, stream=stream)
    elif spec.rope:
        qk_norm_rope(q, k, gq, gk, input_pos, spec.theta, eps, stream=stream)
    if q8:
        kv_append_q8(k, v, batch_idx, input_pos, table, pt.n_slots, pt.max_pages_per_seq,
                     pt.page_size, pt.n_pages, k_cache, v_cache, k_scale, v_scale, err,
                     stream=stream)
        paged_decode_attn_q8(q, k_cache, v_cache, k_scale, v_scale, table, pt.n_slots,
                             pt.max_pages_per_seq, pt.page_size, pt.n_pages, batch_idx, seq_lens,
                             spec.window, scale, ws.buf, out, err, stream=stream)
        return
    kv_append(k, v, batch_idx, input_pos, table, pt.n_slots, pt.max_pages_per_seq,
              pt.page_size, pt.n_pages, k_cache, v_cache, err, stream=stream)
    paged_decode_attn(q, k_cache, v_cache, table, pt.n_slots, pt.max_pages_per_seq,
                      pt.page_size, pt.n_pages, batch_idx, seq_lens, spec.window, scale,
                      ws.splits, ws.buf, out, err, stream=stream)


@dataclasses.dataclass
class StepMeta:
    batch_idx: np.ndarray      # int32 [B] slot of each row
    input_pos: np.ndarray      # int32 [B] position of the token appended
    seq_lens: np.ndarray       # int32 [B] input_pos + 1
    admitted: list             # [(lane, slot, prompt_len)] new this step


class RolloutDriver:
    """Applies a workloads.RolloutSchedule to a PageTable (host allocator)."""

    def __init__(self, pt: PageTable, schedule):
        self.pt = pt
        self.sched = schedule
        self.slots = []
        self.length = []
        self.t = 0
        first = []
        for lane, r in enumerate(schedule.first):
            s = pt.assign(r.prompt_len + 1)
            self.slots.append(s)
            self.length.append(r.prompt_len)
            first.append((lane, s, r.prompt_len))
        self.pending = first

    def next_step(self) -> StepMeta:
        t = self.t
        admitted = self.pending
        self.pending = []
        for lane in self.sched.finish[t]:
            self.pt.free(self.slots[lane])
        for lane, r in self.sched.start[t]:
            s = self.pt.assign(r.prompt_len + 1)
            self.slots[lane] = s
            self.length[lane] = r.prompt_len
            admitted.append((lane, s, r.prompt_len))
        pos = np.array(self.length, dtype=np.int32)
        for lane in range(self.sched.lanes):
            self.pt.reserve(self.slots[lane], int(pos[lane]) + 1)
            self.length[lane] += 1
        self.t += 1
        return StepMeta(np.array(self.slots, dtype=np.int32), pos, pos + 1, admitted)


# --------------------------------------------------------------------------
# Batch buckets and the continuous-batching scheduler
# --------------------------------------------------------------------------

def bucket_ladder(max_bs: int) -> list:
    """The pages' CUDA-graph batch buckets (capture_decode_cudagraph):
    1, 2, 4, 8, then every multiple of 16 up to max_bs."""
    return [b for b in [1, 2, 4, 8] if b <= max_bs] + list(range(16, max_bs + 1, 16))


def bucket_for(B: int, ladder: list) -> int:
    """Smallest bucket holding B rows (a decode batch is padded up to it)."""
    for b in ladder:
        if b >= B:
            return b
    raise ValueError(f"batch {B} exceeds the largest bucket {ladder[-1]}")


@dataclasses.dataclass
class Sequence:
    rid: int
    prompt_len: int
    max_new_tokens: int
    generated: int = 0
    slot: int = -1
    finished: bool = False

    @property
    def total_length(self) -> int:
        return self.prompt_len + self.generated


def _after(stream: int, other: int) -> None:
    """What `stream` is given from here on waits for what `other` has been given."""
    def of(handle):
        return torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()

    done = torch.cuda.Event()
    done.record(of(other))
    of(stream).wait_event(done)


def _move_pages(pt: PageTable, caches, move, stream):
    """Calls `move`, which changes the table and returns page pairs, and copies them. The
    copy has to stand behind the table's upload and before the next append or attention,
    and the pages it writes may still be read: it runs on the table's stream, behind all
    that `stream` (None: the current one) has been given, and what `stream` is given
    afterwards waits for it."""
    kv_copy_pages(caches, pt.n_pages, [])   # refuses them before anything changes
    use = _stream(stream) or 0
    own = use if pt.dev_table is None else pt_get_stream(pt.handle)
    if own != use:
        _after(own, use)
    pairs = move()
    kv_copy_pages(caches, pt.n_pages, pairs, stream=own)
    if own != use:
        _after(use, own)
    return pairs


class ContinuousBatcher:
    """The scheduling of the pages' generate loop ("unsloth: compare
    main...flex-moe-qwen3" · flex_gemma4_moe.py · generate) over a PageTable:

      * admission (prefill first): while the head of the waiting queue fits
        (can_reserve(total_length)), give it a slot reserved for its whole
        length; an admitted batch is prefilled and the loop starts over;
      * decode: each running sequence keeps its capacity or grows it by
        reserve; when it cannot, it goes back to the front of the queue and
        the newest running sequence is preempted (its slot and pages freed,
        it returns to the front of the waiting queue, keeping its tokens);
      * every prefill or decode appends one token; a sequence that reaches
        max_new_tokens finishes and frees its slot.

    The model work is supplied by prefill(batch) and decode(batch) callbacks
    (each gets the Sequence list; decode rows are in running order). events
    records ("prefill" | "decode", [rids]), ("preempt", rid) and ("finish",
    rid) in order."""

    def __init__(self, pt: PageTable, sequences, prefill=None, decode=None):
        import collections
        self.pt = pt
        self.waiting = collections.deque(sequences)
        self.running = collections.deque()
        self.done = []
        self.events = []
        self._prefill = prefill
        self._decode = decode

    def _finish_if_done(self, s: Sequence) -> bool:
        if s.generated >= s.max_new_tokens:
            s.finished = True
            self.done.append(s)
            self.pt.free(s.slot)
            self.events.append(("finish", s.rid))
            s.slot = -1
            return True
        return False

    def step(self) -> bool:
        """One pass of the loop; False once nothing is waiting or running."""
        if not (self.waiting or self.running):
            return False
        batch = []
        while self.waiting and self.pt.can_reserve(self.waiting[0].total_length):
            s = self.waiting.popleft()
            s.slot = self.pt.assign(s.total_length)
            batch.append(s)
        if batch:
            self.events.append(("prefill", [s.rid for s in batch]))
            if self._prefill:
                self._prefill(batch)
            for s in batch:
                s.generated += 1
                if not self._finish_if_done(s):
                    self.running.append(s)
            return True
        decode_batch = []
        while self.running:
            s = self.running.popleft()
            if self.pt.capacity(s.slot) >= s.total_length:
                decode_batch.append(s)
            elif self.pt.can_reserve(s.total_length, s.slot):
                self.pt.reserve(s.slot, s.total_length)
                decode_batch.append(s)
            else:
                self.running.appendleft(s)
                newest = self.running.pop()
                self.waiting.appendleft(newest)
                self.pt.free(newest.slot)
                newest.slot = -1
                self.events.append(("preempt", newest.rid))
        if not decode_batch:
            return True
        self.events.append(("decode", [s.rid for s in decode_batch]))
        if self._decode:
            self._decode(decode_batch)
        for s in decode_batch:
            s.generated += 1
            if not self._finish_if_done(s):
                self.running.append(s)
        return True

    def fork(self, s: Sequence, rids, caches, stream=None) -> list:
        """Adds a sample of the running sequence `s` for each of `rids` (the group
        of a prompt, called once it is prefilled): each starts with the tokens s
        has, on a slot that shares its full pages. `caches` lists every tensor the
        pages live in (K and V of all layers; with 8-bit caches their scales
        too); the partly filled pages are copied in one call. Samples that find
        no slot or page wait to be admitted like any other sequence. Returns the
        new sequences. `stream` (None: the current one) is the one that appends
        to and reads the caches, besides the page table's: both see the samples'
        pages in order."""
        if s not in self.running:
            raise ValueError(f"sequence {s.rid} is not running")
        rids = list(rids)
        cached = s.total_length - 1      # the last token is appended by the next decode
        new = []

        def move():
            pairs = []
            for rid in rids:
                f = Sequence(rid, s.prompt_len, s.max_new_tokens, s.generated)
                try:
                    slots, copies = self.pt.fork(s.slot, cached)
                    f.slot = slots[0]
                    pairs += copies.tolist()
                    self.running.append(f)
                    self.events.append(("fork", s.rid, rid))
                except (NoSlotError, NoPagesError):
                    self.waiting.append(f)
                new.append(f)
            return pairs

        _move_pages(self.pt, caches, move, stream)
        return new

    def run(self, max_steps: int = 100000) -> list:
        for _ in range(max_steps):
            if not self.step():
                return self.done
        raise RuntimeError("scheduler did not drain")


def compact_cache(pt: PageTable, caches, stream=None) -> int:
    """Moves the used pages to the front of the caches; returns how many moved. `stream`
    (None: the current one) is the one that appends to and reads the caches, besides the
    page table's: both see the pages move in order."""
    return len(_move_pages(pt, caches, pt.compact, stream))


class DecodeGraphs:
    """One CUDA graph of the decode layer step per batch bucket, as the pages'
    capture_decode_cudagraph does (graphs over static buffers, replayed after
    copying the step's inputs in). A batch of B rows replays the smallest
    bucket >= B; rows B.. of the bucket are padding rows on slot 0 (the
    reserved slot: no keys, zero output, their append lands in the reserved
    page 0; an 8-bit cache skips it). The page table is read through
    pt.dev_table, which the host allocator updates between steps. With k_scale
    and v_scale the caches are 8-bit ones."""

    def __init__(self, spec: LayerSpec, pt: PageTable, k_cache, v_cache, Hq: int, max_bs: int,
                 device, gamma_q=None, gamma_k=None, eps: float = 1e-6, ladder=None,
                 k_scale=None, v_scale=None):
        self.spec, self.pt, self.kc, self.vc = spec, pt, k_cache, v_cache
        self.ks, self.vs = k_scale, v_scale
        self.gq, self.gk, self.eps = gamma_q, gamma_k, eps
        self.ladder = ladder or bucket_ladder(max_bs)
        Hkv, D = k_cache.shape[0], k_cache.shape[2]
        bf = dict(dtype=torch.bfloat16, device=device)
        i32 = dict(dtype=torch.int32, device=device)
        self.q = torch.zeros((max_bs, Hq, D), **bf)
        self.k = torch.zeros((max_bs, Hkv, D), **bf)
        self.v = torch.zeros((max_bs, Hkv, D), **bf)
        self.out = torch.zeros((max_bs, Hq, D), **bf)
        self.batch_idx = torch.zeros(max_bs, **i32)
        self.input_pos = torch.zeros(max_bs, **i32)
        self.seq_lens = torch.ones(max_bs, **i32)
        self.err = torch.zeros(1, **i32)
        if k_scale is None:
            self.ws = {b: AttnWorkspace(b, Hq, Hkv, D, pt.max_pages_per_seq, pt.page_size,
                                        spec.window, device) for b in self.ladder}
        else:
            self.ws = {b: AttnWorkspaceQ8(Hq, Hkv, D, device) for b in self.ladder}
        self.graphs = {}
        for b in reversed(self.ladder):
            self._call(b)                  # eager first use of every kernel
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                self._call(b)
            self.graphs[b] = g
        torch.cuda.synchronize()

    def _call(self, b):
        decode_layer_step(self.spec, self.pt, self.kc, self.vc, self.q[:b], self.k[:b],
                          self.v[:b], self.batch_idx[:b], self.input_pos[:b],
                          self.seq_lens[:b], self.out[:b], self.ws[b], self.gq, self.gk,
                          self.eps, err=self.err, k_scale=self.ks, v_scale=self.vs)

    def errors(self) -> int:
        """The error bits of the steps since the last look, on the current stream,
        which it waits for. Clears them, and after PKV_ERR_TIMEOUT (a step's output
        is then unspecified) the workspaces, which the next step needs zero."""
        bits = pkv_read_error_word(self.err)
        if bits:
            self.err.zero_()
        if bits & PKV_ERR_TIMEOUT:
            for w in self.ws.values():
                w.reset()
        return bits

    def step(self, q, k, v, batch_idx, input_pos):
        """Device tensors for B rows; returns the B rows of the output (a view
        of the static buffer, valid until the next step). What a step could not
        do is told by errors()."""
        B = q.shape[0]
        b = bucket_for(B, self.ladder)
        self.q[:B].copy_(q)
        self.k[:B].copy_(k)
        self.v[:B].copy_(v)
        self.batch_idx[:B].copy_(batch_idx)
        self.input_pos[:B].copy_(input_pos)
        self.seq_lens[:B].copy_(input_pos + 1)
        self.batch_idx[B:b].zero_()
        self.input_pos[B:b].zero_()
        self.seq_lens[B:b].fill_(1)
        self.graphs[b].replay()
        return self.out[:B]
