"""The attention half of a decoder layer, composed from the C-ABI calls.

[norm ->] projection (grouped GEMM with one expert: FP4 weights) -> cache slots ->
head norms + rotation + cache write -> attention (whole prompts, or one token per
request behind a shared prefix) -> output projection -> residual [with the block's
norm, gate and scale, and the next block's norm].  With ``MoELayer`` on its output
that is a decoder layer; the pages' model has such a pair per layer.  Buffers are
allocated once (the attention's workspace grows with the context, in doublings).

The cache is paged, its rows bf16 or held in 4 bits (NVFP4).  Every request owns the
pages of its own tokens; a prefix that all requests share is kept once and lies before
each request's own tokens (positions count from the prefix's start).  The host keeps the
lengths that it hands out and so knows how many pages a step takes; tables, slots and
positions are built on the GPU.

prompt() reads the first tokens of requests 0 .. n - 1 together, decode() adds one token
to each of requests 0 .. B - 1, extend() adds tokens to any requests, behind a prefix or
what they hold already (a second turn, a prompt in pieces, a request that enters while
others decode).  fork() lets requests go on as copies of another, release() ends requests
and gives their pages back, compact() moves the pages in use to the front of the pool.
"""
from __future__ import annotations

import dataclasses
from typing import Optional, Sequence

import torch

from . import (Fp4Cache, Weights, attn_decode, attn_decode_fp4, attn_decode_fp4_workspace_bytes, attn_decode_workspace_bytes,
               attn_prompt, block_norm, combine, grouped_gemm, kv_compact, kv_fork, kv_free_pages, kv_gather, kv_gather_fp4,
               kv_slots, qk_norm_rope, qk_norm_rope_fp4)


@dataclasses.dataclass
class AttentionWeights:
    qkv: Weights                              # [1, (q_heads + kv_heads) * k_dim + kv_heads * v_dim, hidden]
    out: Weights                              # [1, hidden, q_heads * v_dim]
    q_norm: Optional[torch.Tensor] = None     # float32 [k_dim]; None: no norm
    k_norm: Optional[torch.Tensor] = None
    # The residual stream's norms, float32 [hidden] (None: none).  in_norm: x is the stream, and the projection reads its
    # norm.  post_norm, gate (float32 [hidden]) and residual_scale: of the half's output before the residual is added.
    # next_norm: prompt(), extend() and decode() return (h, norm of h), the norm before the next half.
    in_norm: Optional[torch.Tensor] = None
    post_norm: Optional[torch.Tensor] = None
    gate: Optional[torch.Tensor] = None
    residual_scale: float = 1.0
    next_norm: Optional[torch.Tensor] = None


class AttentionLayer:
    def __init__(self, weights: AttentionWeights, q_heads: int, kv_heads: int, k_dim: int, v_dim: int,
                 cos_sin: torch.Tensor, num_pages: int, page_size: int, max_requests: int, max_context: int,
                 max_tokens: int, interleaved: bool = False, eps: float = 1e-6, device="cuda", cache: str = "bf16",
                 k_global: float = 1.0, v_global: float = 1.0):
        """``cache``: "bf16" or "nvfp4" (k_global and v_global are then its global scales).  ``cos_sin``: float32
        [positions, rotated dims] (cosines, then sines), a row for each position that a token takes: the prefix's length
        and the longest request's own together.  ``max_context``: most tokens of a request, the prefix not counted (and
        most of the prefix); ``max_tokens``: most tokens of one step."""
        self.w, self.cos_sin, self.interleaved, self.eps = weights, cos_sin, interleaved, eps
        self.q_heads, self.kv_heads, self.k_dim, self.v_dim = q_heads, kv_heads, k_dim, v_dim
        self.page_size, self.max_requests, self.max_tokens = page_size, max_requests, max_tokens
        self.blocks = -(-max_context // page_size)
        dev, bf16, i32 = torch.device(device), torch.bfloat16, torch.int32
        H, n = weights.out.packed.shape[1], weights.qkv.packed.shape[1]
        want = (1, (q_heads + kv_heads) * k_dim + kv_heads * v_dim, H // 2), (1, H, q_heads * v_dim // 2)
        got = tuple(weights.qkv.packed.shape), tuple(weights.out.packed.shape)
        if got != want:                       # the projections read rows of their weights' width
            raise ValueError(f"packed weights of the projections are {got[0]} and {got[1]}, these heads need {want[0]} "
                             f"and {want[1]}")
        if cache == "bf16":
            self.fp4 = None
            self.k_cache = torch.zeros((num_pages, page_size, kv_heads, k_dim), dtype=bf16, device=dev)
            self.v_cache = torch.zeros((num_pages, page_size, kv_heads, v_dim), dtype=bf16, device=dev)
            self.buffers = self.k_cache, self.v_cache
        elif cache == "nvfp4":
            if page_size < 16:
                raise ValueError(f"pages of a 4-bit cache hold at least 16 tokens (got {page_size})")
            if cos_sin is not None and cos_sin.shape[1] % 32:
                raise ValueError(f"a 4-bit cache needs a multiple of 32 rotated dims (got {cos_sin.shape[1]})")
            self.fp4 = Fp4Cache.zeros(num_pages, page_size, kv_heads, k_dim, v_dim, k_global, v_global, dev)
            self.buffers = self.fp4.buffers
        else:
            raise ValueError(f"cache is \"bf16\" or \"nvfp4\" (got {cache!r})")
        # one row per request, the last for the prefix
        self.table = torch.full((max_requests + 1, self.blocks), -1, dtype=i32, device=dev)
        self.pool = torch.arange(num_pages, dtype=i32, device=dev)
        self.free = self.pool                 # the free list: a part of pool once pages have come back
        self.lens = torch.zeros(max_requests + 1, dtype=i32, device=dev)
        self.new = torch.zeros(max_requests + 1, dtype=i32, device=dev)
        self.host_lens = [0] * (max_requests + 1)
        self.taken = 0                        # entries of the free list handed out
        # The pages that each row holds, by numbers of the host's own: rows that share pages have the same ones.
        self.held = [[] for _ in range(max_requests + 1)]
        self.pages_made = 0
        T = max_tokens
        self.slots, self.positions = (torch.empty(T, dtype=i32, device=dev) for _ in range(2))
        self.cu = torch.zeros(max_requests + 2, dtype=i32, device=dev)
        self.counts = torch.zeros(3, dtype=i32, device=dev)
        self.qkv = torch.empty((T, n), dtype=bf16, device=dev)
        self.q = torch.empty((T, q_heads, k_dim), dtype=bf16, device=dev)
        self.k = torch.empty((T, kv_heads, k_dim), dtype=bf16, device=dev)
        self.a = torch.empty((T, q_heads, v_dim), dtype=bf16, device=dev)
        self.o, self.y = (torch.empty((T, H), dtype=bf16, device=dev) for _ in range(2))
        self.offsets = {}                     # expert offsets [0, T] of the one-expert projections
        self.rows = torch.arange(T, dtype=i32, device=dev)
        self.ones = torch.ones((T, 1), dtype=torch.float32, device=dev)
        self.ws = torch.empty(16, dtype=torch.uint8, device=dev)
        w = weights
        self.with_norms = any(v is not None for v in (w.post_norm, w.gate, w.next_norm)) or w.residual_scale != 1.0
        for name in ("in_norm", "post_norm", "gate", "next_norm"):
            v = getattr(w, name)
            if v is not None and (tuple(v.shape) != (H,) or v.dtype != torch.float32):
                raise ValueError(f"{name} must be a float32 tensor ({H},) (got {tuple(v.shape)}, {v.dtype})")
        self.xn = torch.empty((T, H), dtype=bf16, device=dev) if w.in_norm is not None else None
        self.z = torch.empty((T, H), dtype=bf16, device=dev) if w.next_norm is not None else None

    @property
    def prefix_len(self) -> int:
        return self.host_lens[-1]

    def _one(self, T: int) -> torch.Tensor:
        if T not in self.offsets:
            self.offsets[T] = torch.tensor([0, T], dtype=torch.int32, device=self.free.device)
        return self.offsets[T]

    def _check_rows(self, **rows: Optional[torch.Tensor]):
        """The step's rows are read and written whole: bf16 [tokens, hidden], contiguous, 16-byte aligned, on the
        layer's device.  Looked at before anything of the step is done."""
        T = rows["x"].shape[0]
        for name, t in rows.items():
            if t is not None and (t.dtype != torch.bfloat16 or tuple(t.shape) != (T, self.o.shape[1])
                                  or not t.is_contiguous() or t.device != self.o.device or t.data_ptr() % 16):
                raise ValueError(f"{name} must be a contiguous bfloat16 tensor, 16-byte aligned, ({T}, {self.o.shape[1]}) on "
                                 f"{self.o.device} (got {tuple(t.shape)}, {t.dtype}, {t.device})")

    def _tokens(self, x: torch.Tensor, new: Sequence[int], first: int, base: int):
        """Projection, slots, norm + rotation + cache write of the step's tokens: requests first .. of the table bring
        ``new`` tokens each.  -> (q, k, v) of the step."""
        T, n = x.shape[0], len(new)
        if T < 1 or T != sum(new) or min(new) < 0 or T > self.max_tokens:
            raise ValueError(f"{T} tokens for requests that bring {sum(new)} (1 to {self.max_tokens})")
        page = self.page_size
        old = self.host_lens[first:first + n]
        if any(c + m > self.blocks * page for c, m in zip(old, new)):
            raise ValueError("a request grows over max_context")
        if self.cos_sin is not None and base + max(c + m for c, m in zip(old, new) if m) > self.cos_sin.shape[0]:
            raise ValueError(f"a token's position is past the {self.cos_sin.shape[0]} rows of cos_sin")
        more = [-(-(c + m) // page) - -(-c // page) for c, m in zip(old, new)]
        self._check_free(sum(more))
        if self.w.in_norm is not None:
            x = block_norm(x, self.w.in_norm, eps=self.eps, want_h=False, y=self.xn[:T])[1]
        qkv = grouped_gemm(x, self.w.qkv, None, self._one(T), T, out=self.qkv[:T])
        nq, nk = self.q_heads * self.k_dim, self.kv_heads * self.k_dim
        q = qkv[:, :nq].unflatten(1, (self.q_heads, self.k_dim))
        k = qkv[:, nq:nq + nk].unflatten(1, (self.kv_heads, self.k_dim))
        v = qkv[:, nq + nk:].unflatten(1, (self.kv_heads, self.v_dim))
        lens = self.lens[first:first + n]
        kv_slots(lens, self.new[first:first + n], self.free[self.taken:], self.table[first:first + n], page, T,
                 base, self.slots, self.positions, self.cu, self.counts)
        lens.add_(self.new[first:first + n])
        self.taken += sum(more)
        for i, m in enumerate(new):
            self.host_lens[first + i] += m
            if more[i]:
                self.held[first + i] += self._new_pages(more[i])
        if self.fp4 is None:
            qk_norm_rope(q, k, self.positions, self.cos_sin, self.w.q_norm, self.w.k_norm, self.eps, self.interleaved, v,
                         self.k_cache, self.v_cache, self.slots, q_out=self.q[:T], k_out=self.k[:T])
        else:
            qk_norm_rope_fp4(q, k, v, self.positions, self.cos_sin, self.fp4, self.slots, self.w.q_norm, self.w.k_norm, self.eps,
                             self.interleaved, q_out=self.q[:T], k_out=self.k[:T])
        return self.q[:T], self.k[:T], v

    def _check_free(self, need: int):
        if self.taken + need > self.free.numel():
            raise ValueError(f"{need} pages needed, {self.free.numel() - self.taken} free")

    def _new_pages(self, n: int) -> list:
        self.pages_made += n
        return list(range(self.pages_made - n, self.pages_made))

    def _in_use(self) -> int:
        return len(set().union(*self.held))

    def _finish(self, x: torch.Tensor, residual: Optional[torch.Tensor], y: Optional[torch.Tensor]):
        T = x.shape[0]
        plain = residual is None and not self.with_norms
        o = y if plain and y is not None else self.o[:T]
        grouped_gemm(self.a[:T].flatten(1), self.w.out, None, self._one(T), T, out=o)
        if plain:
            return o
        y = self.y[:T] if y is None else y
        if not self.with_norms:
            return combine(o, self.rows[:T], self.ones[:T], residual, y=y)
        w = self.w
        h, z = block_norm(o, w.next_norm, residual, w.post_norm, w.gate, w.residual_scale, self.eps, h=y,
                          y=None if self.z is None else self.z[:T])
        return h if z is None else (h, z)

    def prompt(self, x: torch.Tensor, lens: Sequence[int], residual: Optional[torch.Tensor] = None, prefix: bool = False,
               y: Optional[torch.Tensor] = None) -> torch.Tensor:
        """First tokens of requests 0 .. len(lens) - 1, packed: x bf16 [sum(lens), hidden].  ``prefix``: of the shared
        prefix instead (one length).  Behind a prefix a request starts with ``extend`` or ``decode``."""
        self._check_rows(x=x, residual=residual, y=y)
        first = self.max_requests if prefix else 0
        if len(lens) > (1 if prefix else self.max_requests) or any(self.host_lens[first:first + len(lens)]):
            raise ValueError("prompt() takes the first tokens of at most max_requests requests")
        if not prefix and self.prefix_len:
            raise ValueError("prompt() of requests behind a prefix: use extend() or decode()")
        if prefix and any(self.host_lens):
            raise ValueError("the prefix comes before the first tokens of any request: theirs are rotated without it")
        self.new[first:first + len(lens)] = torch.tensor(list(lens), dtype=torch.int32).to(self.new.device)
        q, k, v = self._tokens(x, lens, first, 0)
        cu = self.cu[:len(lens) + 1]
        attn_prompt(q, k, v, cu, cu, out=self.a[:x.shape[0]])
        return self._finish(x, residual, y)

    def extend(self, x: torch.Tensor, requests: Sequence[int], lens: Sequence[int], residual: Optional[torch.Tensor] = None,
               y: Optional[torch.Tensor] = None) -> torch.Tensor:
        """``lens`` more tokens of ``requests`` (ascending), packed: x bf16 [sum(lens), hidden].  They see the prefix, what
        their request holds and one another; keys and values are read back from the cache."""
        self._check_rows(x=x, residual=residual, y=y)
        requests = list(requests)
        if (len(requests) != len(lens) or not requests or sorted(set(requests)) != requests or requests[0] < 0
                or requests[-1] >= self.max_requests):
            raise ValueError(f"requests must ascend within 0 .. {self.max_requests - 1}, with a length for each")
        n = requests[-1] + 1
        new = [0] * n
        for r, m in zip(requests, lens):
            new[r] = m
        base = self.prefix_len
        self.new[:n] = torch.tensor(new, dtype=torch.int32).to(self.new.device)
        q, _, _ = self._tokens(x, new, 0, base)
        cu_k = [0]
        for r, m in enumerate(new):
            cu_k.append(cu_k[-1] + (base + self.host_lens[r] if m else 0))
        at = torch.tensor(cu_k, dtype=torch.int32).to(self.new.device)
        prefix = dict(prefix_table=self.table[-1], prefix_len=base)
        if self.fp4 is None:
            k, v = kv_gather(self.k_cache, self.v_cache, self.table[:n], at, cu_k[-1], **prefix)
        else:
            k, v = kv_gather_fp4(self.fp4, self.table[:n], at, cu_k[-1], **prefix)
        attn_prompt(q, k, v, self.cu[:n + 1], at, out=self.a[:x.shape[0]])
        return self._finish(x, residual, y)

    def decode(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None) -> torch.Tensor:
        """One token of each of requests 0 .. B - 1: x bf16 [B, hidden]."""
        self._check_rows(x=x, residual=residual, y=y)
        B = x.shape[0]
        if not 1 <= B <= self.max_requests:
            raise ValueError(f"{B} requests, at least 1 and at most {self.max_requests}")
        self.new[:B].fill_(1)
        q, _, _ = self._tokens(x, [1] * B, 0, self.prefix_len)
        longest, prefix = max(self.host_lens[:B], default=0), self.prefix_len
        size = attn_decode_workspace_bytes if self.fp4 is None else attn_decode_fp4_workspace_bytes
        need = size(B, prefix, longest, self.q_heads, self.kv_heads, self.k_dim, self.v_dim)
        if self.ws.numel() < need:
            self.ws = torch.empty(2 * need, dtype=torch.uint8, device=x.device)
        keys = (self.table[:B], self.lens, longest, self.table[-1], prefix)
        if self.fp4 is None:
            attn_decode(q, self.k_cache, self.v_cache, *keys, workspace=self.ws, out=self.a[:B])
        else:
            attn_decode_fp4(q, self.fp4, *keys, workspace=self.ws, out=self.a[:B])
        return self._finish(x, residual, y)

    def fork(self, parent: int, children: Sequence[int]):
        """Requests ``children``, which hold nothing, go on as ``parent`` does: they share its whole pages, and each gets a
        copy of a last page that is not full."""
        children = list(children)
        rows = [parent, *children]
        if min(rows) < 0 or max(rows) >= self.max_requests or len(set(rows)) != len(rows):
            raise ValueError(f"parent and children must be different requests of 0 .. {self.max_requests - 1}")
        if any(self.host_lens[c] for c in children):
            raise ValueError("a child holds tokens: release() it first")
        n, page = self.host_lens[parent], self.page_size
        need = len(children) if n % page else 0
        self._check_free(need)
        if not children:
            return
        dev = self.new.device
        ids = torch.tensor(rows, dtype=torch.int32).to(dev)
        kv_fork(self.table, self.lens, ids[:1].expand(len(children)).contiguous(), ids[1:],
                self.free[self.taken:], page, self.buffers, counts=self.counts[:2])
        self.taken += need
        for c in children:
            self.host_lens[c] = n
            self.held[c] = self.held[parent][:n // page] + (self._new_pages(1) if need else [])

    def release(self, requests: Sequence[int]):
        """Requests end: what only they hold is free again.  (Pools of up to 2^20 pages, as for compact().)"""
        requests = list(requests)
        if any(not 0 <= r < self.max_requests for r in requests):
            raise ValueError(f"requests are 0 .. {self.max_requests - 1}")
        if not requests:
            return
        lens, pages = self.lens.clone(), self.pool.numel()
        lens[torch.tensor(requests).to(lens.device)] = 0
        # (refused, for one of pools past its 2^20 pages, it leaves the layer as it was)
        kv_free_pages(self.table, lens, self.page_size, pages, free_pages=self.pool, counts=self.counts[:2])
        self.lens.copy_(lens)
        for r in requests:
            self.host_lens[r], self.held[r] = 0, []
        self.taken, self.free = 0, self.pool[:pages - self._in_use()]

    def compact(self) -> int:
        """Moves the pages in use to the front of the pool.  -> their number: the pool's pages from there on are free."""
        kv_compact(self.table, self.lens, self.page_size, self.buffers, out_table=self.table, counts=self.counts[:2])
        n, pages = self._in_use(), self.pool.numel()
        self.taken, self.free = 0, self.pool[:pages - n]
        self.free.copy_(torch.arange(n, pages, dtype=torch.int32, device=self.free.device))
        return n
