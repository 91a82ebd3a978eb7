"""Memory-budgeted continuous batching over one attention layer (synthetic).

The job-level claim of the pages ([News], "结果": up to 7.83x throughput at
batch 32 against BF16 KV; [Blog], serving paragraphs) comes from memory: at a
fixed KV budget INT2 history holds about 7x more requests than BF16 history, so
more of them decode together.  This module is the loop that turns a page budget
into a batch:

* a request arrives with a cached prefix (a full prefix hit, imported as stored
  KV) and generates ``gen`` tokens; it is admitted, first come first served,
  once the pool holds every history page it will ever need
  (ceil(max(prefix + gen - 320, 0) / 64));
* active requests sit in batch slots 0..n-1; each iteration runs one decode
  step for all of them (append the new token, demote the oldest recent one,
  attend) through the C ABI: ``oscar_decode_step`` for INT2,
  ``oscar_append_bf16_history`` + ``oscar_decode_bf16_history`` for the BF16
  baseline, or ``oscar_append_kv8`` + ``oscar_decode_kv8`` for 8-bit history
  (about 3.6x the INT2 bytes at 8-bit accuracy), there optionally with a budget:
  a request whose history exceeds it by 256 tokens loses the blocks that got the
  least attention (``oscar_evict_kv8``), and pages it no longer needs go back to
  the pool; with 8-bit history the tokens may also come as a layer's projections,
  which ``oscar_rope`` turns into queries, keys and values: the prefix is then a
  prompt that is attended in chunks as it is cached (``oscar_prefill_kv8``);
* a finished request returns its pages; the last active request moves into
  its slot so the batch stays dense.

Host bookkeeping only: every step of the attention runs in the library's
kernels.  One layer, synthetic tokens: it measures the memory-bound batching
effect, not a model.
"""
from __future__ import annotations

import contextlib
import dataclasses
import time

from . import oscar

HISTORY_FREE = 320  # sink 64 + recent 256 tokens live outside the history pages


def pages_needed(prefix: int, gen: int, page: int = 64) -> int:
    """History pages a request needs by the end of its generation."""
    hist = max(prefix + gen - HISTORY_FREE, 0)
    return (hist + page - 1) // page


KV8_KINDS = {"e4m3": 0, "int8": 1}  # DeviceBackend formats with 8-bit history: their oscar_kv8_type


def kv8_history(n: int) -> int:
    """History tokens of a request with 8-bit history after n tokens, without eviction."""
    return -(-max(n - HISTORY_FREE, 0) // 16) * 16


def pages_needed_kv8(prefix: int, gen: int, page: int = 64, budget=None) -> int:
    """History pages a request with 8-bit history needs at its fullest: the
    prefix, then all tokens or, with a budget, what a step can leave before the
    eviction that follows it."""
    grown = kv8_history(prefix + gen)
    if budget is not None:
        grown = min(grown, max(kv8_history(prefix), budget + 256) + 16)
    return -(-max(kv8_history(prefix), grown) // page)


class PagePool:
    """Free list of the pool's page ids."""

    def __init__(self, num_pages: int):
        self.num_pages = num_pages
        self._free = list(range(num_pages - 1, -1, -1))

    @property
    def available(self) -> int:
        return len(self._free)

    def alloc(self, n: int):
        if n > len(self._free):
            return None
        return [self._free.pop() for _ in range(n)]

    def release(self, ids):
        self._free.extend(reversed(ids))


@dataclasses.dataclass
class Request:
    rid: int
    prefix: int
    gen: int
    done: int = 0          # tokens generated so far
    pages: list = None
    admitted_step: int = -1
    finished_step: int = -1


class Scheduler:
    """Admission, slots and retirement, independent of the device (testable on CPU).

    The backend receives: ``admit(slot, req)`` (pages in req.pages),
    ``step(slots)`` (active requests in slot order) and ``move(src, dst)``
    (copy slot src's device state into slot dst).  A backend that evicts also
    has ``kept_pages(slot)``: how many of the request's pages it still needs; the
    others return to the pool after the step.  need(prefix, gen) is the number of
    pages to hold for a request."""

    def __init__(self, pool: PagePool, max_batch: int, backend, max_pages_per_req: int, need=pages_needed):
        self.need = need
        self.pool = pool
        self.max_batch = max_batch
        self.backend = backend
        self.max_pages = max_pages_per_req
        self.active = []   # slot i holds active[i]
        self.waiting = []
        self.finished = []
        self.steps = 0

    def submit(self, req: Request):
        if self.need(req.prefix, req.gen) > min(self.max_pages, self.pool.num_pages):
            raise ValueError(f"request {req.rid} can never fit the pool")
        self.waiting.append(req)

    def _admit(self):
        while self.waiting and len(self.active) < self.max_batch:
            req = self.waiting[0]
            ids = self.pool.alloc(self.need(req.prefix, req.gen))
            if ids is None:
                break  # first come, first served: later requests wait too
            self.waiting.pop(0)
            req.pages = ids
            req.admitted_step = self.steps
            slot = len(self.active)
            self.active.append(req)
            self.backend.admit(slot, req)

    def _retire(self):
        slot = 0
        while slot < len(self.active):
            req = self.active[slot]
            if req.done < req.gen:
                slot += 1
                continue
            req.finished_step = self.steps
            self.pool.release(req.pages)
            self.finished.append(req)
            last = len(self.active) - 1
            if slot != last:
                self.backend.move(last, slot)
                self.active[slot] = self.active[last]
            self.active.pop()

    def _shrink(self):
        kept_pages = getattr(self.backend, "kept_pages", None)
        if kept_pages is None:
            return
        for slot, req in enumerate(self.active):
            kept = kept_pages(slot)
            if kept < len(req.pages):
                self.pool.release(req.pages[kept:])
                req.pages = req.pages[:kept]

    def run(self, max_steps: int = 1 << 30):
        self._admit()
        while (self.active or self.waiting) and self.steps < max_steps:
            if not self.active:
                raise RuntimeError("nothing admitted: the pool is too small for the next request")
            self.backend.step(self.active)
            for req in self.active:
                req.done += 1
            self.steps += 1
            self._shrink()
            self._retire()
            self._admit()
        return self.finished


class DeviceBackend:
    """One layer's cache on the GPU, driven through the C ABI.

    draw(req) -> (K, V, Q): the request's synthetic stream, K and V bf16
    [Hkv][prefix + gen][128] and Q bf16 [gen][Hq][128] device tensors.  At
    admission the prefix is imported and the request's future tokens are
    copied into its batch slot's buffers; a step then gathers every active
    slot's next token with one indexed read per operand and runs one
    pre-marshalled library call.  fmt is "int2", "bf16", "e4m3" or "int8".

    budget (8-bit history only): history tokens a request may keep; the block
    weights decay by `decay` a step.  on_evict(active), if given, runs right
    before an eviction.

    rope (8-bit history only): dict(table=oscar.make_rope(..)) and, for heads
    that are normalised, gamma_q, gamma_k and eps.  Then draw(req) -> the rows of
    the request's projections, bf16 [prefix + gen][Hq + 2 Hkv][128]: the prefix
    is a prompt, attended and cached in chunks of prompt_chunk tokens
    (on_prompt(req, first, out), if given, gets each chunk's attention
    [T][Hq][128] before the chunk is cached), and a step turns every slot's next
    row by its position, which an eviction does not change."""

    def __init__(self, fmt, ctx, cfg, cache, draw, on_step=None, time_steps=False, max_gen=64, budget=None,
                 decay=1.0, on_evict=None, rope=None, prompt_chunk=512, on_prompt=None):
        import torch

        if fmt not in ("int2", "bf16", *KV8_KINDS):
            raise ValueError(f"unknown history format {fmt!r}")
        self.kind = KV8_KINDS.get(fmt)
        if budget is not None and (self.kind is None or budget < 0):
            raise ValueError("a budget needs 8-bit history and is not negative")
        if rope is not None and (self.kind is None or prompt_chunk < 1):
            raise ValueError("projections need 8-bit history and chunks of a token or more")
        self.budget, self.on_evict = budget, on_evict
        self.rope, self.prompt_chunk, self.on_prompt = rope, prompt_chunk, on_prompt
        self.lens = {}  # slot -> [tokens, history tokens] (8-bit history; the device follows the same rule)
        self.kept = {}  # slot -> pages the request holds
        self.weights = None

        self.fmt, self.ctx, self.cfg, self.cache = fmt, ctx, cfg, cache
        self.draw, self.on_step = draw, on_step
        B, Hq, Hkv = cfg.max_batch, cfg.num_q_heads, cfg.num_kv_heads
        dev = cache["seq_lens"].device
        self.dev = dev
        self.out = torch.empty(B, Hq, 128, dtype=torch.bfloat16, device=dev)
        self.scratch = oscar.alloc_scratch(cfg, dev) if self.kind is None else oscar.alloc_scratch_kv8(cfg, dev)
        if rope is not None:
            self.chunk_scratch = oscar.alloc_scratch_kv8(cfg, dev, prefill=True)
            self.place = torch.zeros(B, dtype=torch.int32, device=dev)  # position of each slot's next token
        self.gen_cap = 0
        self._grow(max_gen)
        self.pos = torch.zeros(B, dtype=torch.long, device=dev)  # next token of each slot
        self.slots = torch.arange(B, device=dev)
        if self.kind is None:
            self.call = oscar.bind_step_any_batch(ctx, 0, cache, self.out, None, self.scratch,
                                                  bf16_history=(fmt == "bf16"))
        else:
            if budget is not None:
                self.weights = oscar.alloc_weights_kv8(cfg, dev)
            self.call = oscar.bind_step_kv8(ctx, cache, self.kind, self.out, None, self.scratch, self.weights, decay)
        self.step_events = [] if time_steps else None
        self.import_events = [] if time_steps else None

    def _grow(self, gen):
        """Slot buffers for up to `gen` future tokens per request, keeping the
        tokens already held."""
        import torch

        B, Hq, Hkv = self.cfg.max_batch, self.cfg.num_q_heads, self.cfg.num_kv_heads
        heads = (Hkv, Hkv, Hq) if self.rope is None else (Hq + 2 * Hkv,)
        bufs = [torch.zeros(B, gen, H, 128, dtype=torch.bfloat16, device=self.dev) for H in heads]
        if self.gen_cap:
            for new, old in zip(bufs, self.held):
                new[:, :self.gen_cap] = old
        self.held = bufs
        if self.rope is None:
            self.kbuf, self.vbuf, self.qbuf = bufs
        else:
            self.rows, = bufs
        self.gen_cap = gen

    def _view(self, slot):
        v = dict(self.cache)
        for key in ("page_table", "sink_k", "sink_v", "ring_k", "ring_v", "seq_lens", "hist_lens"):
            v[key] = self.cache[key][slot:slot + 1]
        return v

    def admit(self, slot, req):
        import torch

        if req.gen > self.gen_cap:
            self._grow(req.gen)
        P, n = req.prefix, req.gen
        if self.rope is not None:
            rows = self.draw(req)
            self.rows[slot, :n] = rows[P:P + n]
            self.place[slot] = 0
        else:
            K, V, Q = self.draw(req)
            self.kbuf[slot, :n] = K[:, P:P + n].permute(1, 0, 2)
            self.vbuf[slot, :n] = V[:, P:P + n].permute(1, 0, 2)
            self.qbuf[slot, :n] = Q[:n]
        self.pos[slot] = 0
        row = self.cache["page_table"][slot]
        row.fill_(-1)
        if req.pages:
            # pinned and non-blocking: a pageable copy would wait for all queued GPU work
            ids = torch.tensor(req.pages, dtype=torch.int32)
            if row.is_cuda:
                ids = ids.pin_memory()
            row[:len(req.pages)].copy_(ids, non_blocking=row.is_cuda)
        self.cache["seq_lens"][slot] = 0
        self.cache["hist_lens"][slot] = 0
        self.lens[slot] = [P, kv8_history(P)]
        self.kept[slot] = len(req.pages)
        if P:
            view = self._view(slot)
            if self.rope is None:
                by_token = self.kind is not None  # [1][P][Hkv][128]; else [1][Hkv][P][128]
                Kp = (K[:, :P].transpose(0, 1) if by_token else K[:, :P]).unsqueeze(0).contiguous()
                Vp = (V[:, :P].transpose(0, 1) if by_token else V[:, :P]).unsqueeze(0).contiguous()
            w = self.weights[slot:slot + 1] if self.weights is not None else None
            if self.rope is not None:
                self._prompt(slot, req, rows, view, w)
                return
            with self._timed(self.import_events):
                if self.kind is not None:
                    oscar.oscar_append_kv8(self.ctx, view, self.kind, Kp, Vp, P, 1, weights=w)
                elif self.fmt == "int2":
                    oscar.oscar_import_tokens(self.ctx, 0, view, Kp, Vp, 1, P)
                else:
                    oscar.oscar_import_bf16_history(self.ctx, view, Kp, Vp, 1, P)

    @contextlib.contextmanager
    def _timed(self, events):
        """Events around what is launched inside, added to the list (None: not timed)."""
        import torch

        if events is not None:
            ev = (torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
            ev[0].record()
        yield
        if events is not None:
            ev[1].record()
            events.append(ev)

    def _turn(self, rows, place, T, batch):
        """Queries, keys and values [batch][T][..][128] of projection rows; the first token of each is at `place`."""
        import torch

        Hq, Hkv, r = self.cfg.num_q_heads, self.cfg.num_kv_heads, self.rope
        q, k, v = (torch.empty(batch, T, H, 128, dtype=torch.bfloat16, device=self.dev) for H in (Hq, Hkv, Hkv))
        oscar.oscar_rope(self.ctx, r["table"], rows, place, T, q, k, v, batch, r.get("gamma_q"), r.get("gamma_k"),
                         r.get("eps", 1e-6))
        return q, k, v

    def _prompt(self, slot, req, rows, view, weights):
        """Caches the request's prompt, each chunk after its attention."""
        import torch

        place = self.place[slot:slot + 1]
        for at in range(0, req.prefix, self.prompt_chunk):
            T = min(self.prompt_chunk, req.prefix - at)
            with self._timed(self.import_events):
                q, k, v = self._turn(rows[at:at + T].unsqueeze(0), place, T, 1)
                out = torch.empty_like(q)
                oscar.oscar_prefill_kv8(self.ctx, view, self.kind, q, k, v, T, out, None, self.chunk_scratch, 1)
            if self.on_prompt is not None:
                self.on_prompt(req, at, out[0])
            with self._timed(self.import_events):
                oscar.oscar_append_kv8(self.ctx, view, self.kind, k, v, T, 1, weights=weights)
                place += T

    def export(self, slot):
        """The cached keys and values of a slot (8-bit history), bf16 [Hkv][n][128] in cache
        order, as the imports of the other caches take them."""
        import torch

        if self.kind is None:
            raise ValueError("only a cache with 8-bit history is read back")
        n = self.lens[slot][0]
        K, V = (torch.empty(self.cfg.num_kv_heads, n, 128, dtype=torch.bfloat16, device=self.dev) for _ in range(2))
        oscar.oscar_read_kv8(self.ctx, self._view(slot), self.kind, 0, n, K, V, 1)
        return K, V

    def move(self, src, dst):
        for key in ("page_table", "sink_k", "sink_v", "ring_k", "ring_v", "seq_lens", "hist_lens"):
            self.cache[key][dst].copy_(self.cache[key][src])
        for buf in (*self.held, self.pos):
            buf[dst].copy_(buf[src])
        if self.rope is not None:
            self.place[dst].copy_(self.place[src])
        if self.weights is not None:
            self.weights[dst].copy_(self.weights[src])
        self.lens[dst] = self.lens.pop(src)
        self.kept[dst] = self.kept.pop(src)

    def step(self, active):
        n = len(active)
        sl, ps = self.slots[:n], self.pos[:n]
        if self.rope is not None:
            rows = self.rows[sl, ps].unsqueeze(1)
        else:
            k = self.kbuf[sl, ps]
            v = self.vbuf[sl, ps]
            q = self.qbuf[sl, ps]
        with self._timed(self.step_events):
            if self.rope is not None:
                q, k, v = self._turn(rows, self.place[:n], 1, n)
                q = q[:, 0]
                self.place[:n] += 1
            self.call(k.data_ptr(), v.data_ptr(), q.data_ptr(), n)
        self.pos[:n] += 1
        if self.on_step is not None:
            self.on_step(active, q, self.out[:n])
        if self.kind is not None:
            self._follow(active)

    def _follow(self, active):
        """The host's account of the lengths after a step, and the eviction when due."""
        n = len(active)
        due = False
        for slot in range(n):
            ln = self.lens[slot]
            ln[0] += 1
            ln[1] = max(ln[1], kv8_history(ln[0]))
            due |= self.budget is not None and ln[1] - self.budget >= 256
        if not due:
            return
        if self.on_evict is not None:
            self.on_evict(active)
        oscar.oscar_evict_kv8(self.ctx, self.cache, self.weights, self.budget, self.scratch, n)
        for slot, req in enumerate(active):
            ln = self.lens[slot]
            gone = max(ln[1] - self.budget, 0) // 256 * 256
            if gone:
                ln[0] -= gone
                ln[1] -= gone
                self.kept[slot] = min(self.kept[slot], self._pages(slot, req))
                self.cache["page_table"][slot, self.kept[slot]:] = -1

    def _pages(self, slot, req):
        """Pages the request may still fill, from its present state on."""
        L, H = self.lens[slot]
        grown = kv8_history(L + req.gen - req.done)
        if self.budget is not None:
            grown = min(grown, max(H, self.budget + 256) + 16)
        return -(-max(H, grown) // self.cfg.page_size)

    def kept_pages(self, slot):
        return self.kept[slot]


def step_seconds(backend):
    """Device time of the decode steps (append + attention, from projections
    their positions too; not the gathering of the slots' tokens), summed, when the
    backend was made with time_steps=True."""
    return sum(a.elapsed_time(b) for a, b in backend.step_events) * 1e-3


def import_seconds(backend):
    """Device time of the prefix imports, summed (time_steps=True); from
    projections that of the prompts: positions, attention and append of each
    chunk, without on_prompt."""
    return sum(a.elapsed_time(b) for a, b in backend.import_events) * 1e-3


def run_job(backend, pool_pages, max_batch, max_pages_per_req, requests, need=pages_needed):
    """Runs the requests to completion; returns (finished, steps, seconds)."""
    import torch

    sched = Scheduler(PagePool(pool_pages), max_batch, backend, max_pages_per_req, need)
    for r in requests:
        sched.submit(r)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    done = sched.run()
    torch.cuda.synchronize()
    return done, sched.steps, time.perf_counter() - t0
