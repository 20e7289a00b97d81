"""Serving a batch of requests of changing lengths from paged 4-bit caches.

A scheduler step is one call of ``begin`` (which requests bring how many tokens: one for a decode
step, a few for drafts, a chunk of a prompt) and then, for each layer in order, one of ``attend``
with that step's packed queries, keys and values.  ``finish`` gives the pages of ended requests
back.  The page plan is made once per step and shared by all layers; everything between the
host's ``begin`` and the outputs runs on the device, so a step with fixed sizes can be captured
into a CUDA graph, and replayed between steps of other sizes.  A session's calls and replays share
its lengths, tables and workspace: they run one after the other, on one stream or ordered streams.
This module only holds the tensors and orders the calls.
"""
from __future__ import annotations

from . import kvq as K


class PagedSession:
    """Caches of `layers` layers, and the block tables, lengths and free list of `requests`."""

    def __init__(self, cfg, layers: int, requests: int, rope=None, freqs=None, device="cuda"):
        """cfg: make_paged_cfg.  rope, freqs: make_rope_cfg and its frequencies; without them
        queries and keys are taken as they come."""
        import torch
        self.cfg, self.rope, self.freqs, self.requests = cfg, rope, freqs, requests
        self.caches = [K.PagedCache(cfg, device=device) for _ in range(layers)]
        i32 = dict(dtype=torch.int32, device=self.caches[0].device)
        self.lens = torch.zeros(requests, **i32)
        self.table = torch.full((requests, cfg.max_pages), -1, **i32)
        self.free = torch.arange(cfg.num_pages - 1, -1, -1, **i32)  # page 0 is handed out first
        self.n_free = torch.full((1,), cfg.num_pages, **i32)
        self.cu = torch.zeros(requests + 1, **i32)
        self.slots = self.positions = None  # of the step that began last
        self._held, self._outgrown = {}, []

    def _room(self, name, n: int, dtype):
        """n entries that begin() may use until the session ends.  One that has become too small is
        kept, since a captured step goes on using it; sizes at least double, so all that is kept is
        no more than what is in use."""
        import torch
        t = self._held.get(name)
        if t is None or t.numel() < n:
            if t is not None:
                self._outgrown.append(t)
                n = max(n, 2 * t.numel())
            t = self._held[name] = torch.empty(n, dtype=dtype, device=self.lens.device)
        return t

    def begin(self, n_new, tokens: int, max_q: int, max_len: int = 0) -> None:
        """The step's page plan.  n_new: int32 [requests] on the device, the tokens that each
        request brings; tokens: their sum (or more); max_q: the most that one brings; max_len: an
        upper bound of the lengths after the step (0: what the block table can hold).  A request
        that the plan refuses (see kvq_page_plan and status()) keeps its length; its outputs of
        this step say nothing."""
        import torch
        self.slots = self._room("slots", max(tokens, 16), torch.int32)[:tokens]
        self.positions = self._room("positions", max(tokens, 16), torch.int32)[:tokens]
        self.max_q = max(max_q, 1)  # a step may be without tokens
        self.max_len = max_len or self.cfg.max_pages * self.cfg.page_tokens
        need = K.kvq_paged_attention_workspace(self.cfg, self.requests, tokens, self.max_q,
                                               self.max_len)
        self.workspace = self._room("workspace", max(need, 16), torch.uint8)
        K.kvq_page_plan(self.caches[0], self.lens, n_new, self.table, self.free, self.n_free,
                        self.cu, self.lens, self.n_free, self.slots, self.positions)

    def attend(self, layer: int, q, k, v, sm_scale: float, out, positions=None, window: int = 0,
               lse=None) -> None:
        """Rotate q and k in place, store k and v, and attend: out [tokens, Hq, D].  q, k, v:
        [tokens, heads, D], request by request, rows as far apart as the projection leaves them.
        positions: int32 [axes, tokens] where the rotation has several axes."""
        if self.slots is None:
            raise ValueError("PagedSession.attend: no step has begun")
        cache = self.caches[layer]
        if self.rope is not None:
            K.kvq_rope(self.rope, q, k, self.positions if positions is None else positions,
                       self.freqs, q, k)
        K.kvq_paged_append(cache, k, v, self.slots)
        K.kvq_paged_attention(cache, q, self.cu, self.lens, self.table, self.max_q, self.max_len,
                              sm_scale, out, self.workspace, window=window, lse=lse)

    def finish(self, done) -> None:
        """done: int32 [requests] on the device, not 0 where a request has ended."""
        K.kvq_page_release(self.caches[0], self.lens, done, self.table, self.free, self.n_free)

    def status(self) -> int:
        """KVQ_STATUS_* bits of all layers (waits for the stream)."""
        bits = 0
        for c in self.caches:
            bits |= K.kvq_paged_get_status(c)
        return bits
