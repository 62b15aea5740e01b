"""The attention half of a decoder layer, composed from the C-ABI calls.

projection (grouped GEMM with one expert: FP4 weights) -> cache slots -> head
norms + rotation + cache write -> attention (whole prompts, or one token per
request behind a shared prefix) -> output projection -> residual.  With
``MoELayer`` on its output that is a decoder layer; the pages' model has such a
pair per layer.  Buffers are allocated once (the attention's workspace grows with
the context, in doublings).

The cache is paged.  Every request owns the pages of its own tokens; a prefix
that all requests share is kept once and lies before each request's own tokens
(positions count from the prefix's start).  The host keeps the lengths that it
hands out and so knows how many pages a step takes; tables, slots and positions
are built on the GPU.

One generation of requests: prompt() reads the first tokens of requests 0 .. n - 1
together, decode() adds one token to each of requests 0 .. B - 1.  A request does not
enter while others decode, gives no pages back, and takes no second prompt (attention
of a prompt on keys in the cache is not built); behind a prefix its tokens come by
decode() alone.
"""
from __future__ import annotations

import dataclasses
from typing import Optional, Sequence

import torch

from . import (Weights, attn_decode, attn_decode_workspace_bytes, attn_prompt, combine, grouped_gemm, kv_slots,
               qk_norm_rope)


@dataclasses.dataclass
class AttentionWeights:
    qkv: Weights                              # [1, (q_heads + kv_heads) * k_dim + kv_heads * v_dim, hidden]
    out: Weights                              # [1, hidden, q_heads * v_dim]
    q_norm: Optional[torch.Tensor] = None     # float32 [k_dim]; None: no norm
    k_norm: Optional[torch.Tensor] = None


class AttentionLayer:
    def __init__(self, weights: AttentionWeights, q_heads: int, kv_heads: int, k_dim: int, v_dim: int,
                 cos_sin: torch.Tensor, num_pages: int, page_size: int, max_requests: int, max_context: int,
                 max_tokens: int, interleaved: bool = False, eps: float = 1e-6, device="cuda"):
        """``cos_sin``: float32 [positions, rotated dims] (cosines, then sines), a row for each position that a token
        takes: the prefix's length and the longest request's own together.  ``max_context``: most tokens of a request,
        the prefix not counted (and most of the prefix); ``max_tokens``: most tokens of one step."""
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
        self.k_cache = torch.zeros((num_pages, page_size, kv_heads, k_dim), dtype=bf16, device=dev)
        self.v_cache = torch.zeros((num_pages, page_size, kv_heads, v_dim), dtype=bf16, device=dev)
        # one row per request, the last for the prefix
        self.table = torch.full((max_requests + 1, self.blocks), -1, dtype=i32, device=dev)
        self.free = torch.arange(num_pages, dtype=i32, device=dev)
        self.lens = torch.zeros(max_requests + 1, dtype=i32, device=dev)
        self.new = torch.zeros(max_requests + 1, dtype=i32, device=dev)
        self.host_lens = [0] * (max_requests + 1)
        self.taken = 0                        # pages handed out
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
        if self.cos_sin is not None and base + max(c + m for c, m in zip(old, new)) > self.cos_sin.shape[0]:
            raise ValueError(f"a token's position is past the {self.cos_sin.shape[0]} rows of cos_sin")
        need = sum(-(-(c + m) // page) - -(-c // page) for c, m in zip(old, new))
        if self.taken + need > self.free.numel():
            raise ValueError(f"{need} pages needed, {self.free.numel() - self.taken} free")
        qkv = grouped_gemm(x, self.w.qkv, None, self._one(T), T, out=self.qkv[:T])
        nq, nk = self.q_heads * self.k_dim, self.kv_heads * self.k_dim
        q = qkv[:, :nq].unflatten(1, (self.q_heads, self.k_dim))
        k = qkv[:, nq:nq + nk].unflatten(1, (self.kv_heads, self.k_dim))
        v = qkv[:, nq + nk:].unflatten(1, (self.kv_heads, self.v_dim))
        lens = self.lens[first:first + n]
        kv_slots(lens, self.new[first:first + n], self.free[self.taken:], self.table[first:first + n], page, T, base,
                 self.slots, self.positions, self.cu, self.counts)
        lens.add_(self.new[first:first + n])
        self.taken += need
        for i, m in enumerate(new):
            self.host_lens[first + i] += m
        qk_norm_rope(q, k, self.positions, self.cos_sin, self.w.q_norm, self.w.k_norm, self.eps, self.interleaved, v,
                     self.k_cache, self.v_cache, self.slots, q_out=self.q[:T], k_out=self.k[:T])
        return self.q[:T], self.k[:T], v

    def _finish(self, x: torch.Tensor, residual: Optional[torch.Tensor], y: Optional[torch.Tensor]):
        T = x.shape[0]
        o = self.o[:T] if residual is not None or y is None else y
        grouped_gemm(self.a[:T].flatten(1), self.w.out, None, self._one(T), T, out=o)
        if residual is None:
            return o
        return combine(o, self.rows[:T], self.ones[:T], residual, y=self.y[:T] if y is None else y)

    def prompt(self, x: torch.Tensor, lens: Sequence[int], residual: Optional[torch.Tensor] = None, prefix: bool = False,
               y: Optional[torch.Tensor] = None) -> torch.Tensor:
        """First tokens of requests 0 .. len(lens) - 1, packed: x bf16 [sum(lens), hidden].  ``prefix``: of the shared
        prefix instead (one length).  Behind a prefix a request starts with ``decode`` steps."""
        self._check_rows(x=x, residual=residual, y=y)
        first = self.max_requests if prefix else 0
        if len(lens) > (1 if prefix else self.max_requests) or any(self.host_lens[first:first + len(lens)]):
            raise ValueError("prompt() takes the first tokens of at most max_requests requests")
        if not prefix and self.prefix_len:
            raise ValueError("prompt() of requests behind a prefix: use decode()")
        if prefix and any(self.host_lens):
            raise ValueError("the prefix comes before the first tokens of any request: theirs are rotated without it")
        self.new[first:first + len(lens)] = torch.tensor(list(lens), dtype=torch.int32).to(self.new.device)
        q, k, v = self._tokens(x, lens, first, 0)
        cu = self.cu[:len(lens) + 1]
        attn_prompt(q, k, v, cu, cu, out=self.a[:x.shape[0]])
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
        need = attn_decode_workspace_bytes(B, prefix, longest, self.q_heads, self.kv_heads, self.k_dim, self.v_dim)
        if self.ws.numel() < need:
            self.ws = torch.empty(2 * need, dtype=torch.uint8, device=x.device)
        attn_decode(q, self.k_cache, self.v_cache, self.table[:B], self.lens, longest, self.table[-1], prefix,
                    workspace=self.ws, out=self.a[:B])
        return self._finish(x, residual, y)
