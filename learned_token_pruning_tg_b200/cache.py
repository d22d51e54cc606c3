"""The decode cache in 8 bits: KVCacheQ8 holds one layer's keys and values for a batch of sequences.

After a pruned prefill the layers above the gate keep the kept tokens' keys, each with its gate score as a
logit bias (aiproducthub.cn article, paragraph 事件详情).  A decoding program then, for every new token,

    lengths += 1                                  # one tensor may serve every layer
    cache.append(k, v, s=score)                   # the token's own key and value
    cache.decode(q, out, gain=gain, tau=tau, accumulate=True)

and, when a cache is full, moves the tokens that gathered the most attention into a smaller one:

    cache.evict_into(other, budget, sink=4, recent=512)

All work is the library's kernels on the current stream; nothing synchronises.  Every call can be captured in
a CUDA graph (call `reserve` first) and replayed as the sequences grow, since lengths are read on the device.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import tokengate as tg

FORMATS = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


class KVCacheQ8:
    """Buffers, handle and workspace of one 8-bit cache.  Calls on one cache must not run at the same time
    (they share its workspace); caches of their own do not disturb one another."""

    def __init__(self, batch: int, capacity: int, Hkv: int, d_h: int, fmt: str = "e4m3", bias: bool = True,
                 weights: bool = True, lengths: Optional[torch.Tensor] = None, device="cuda"):
        """An empty cache of `capacity` tokens a sequence (rounded up to a multiple of 32).  lengths: an
        int32 [batch] tensor to use instead of one of its own."""
        if fmt not in FORMATS:
            raise ValueError(f"fmt must be one of {sorted(FORMATS)}, got {fmt!r}")
        cap = -(-capacity // tg.TG_CACHE_BLOCK) * tg.TG_CACHE_BLOCK
        new = lambda dt, *shape: torch.zeros(*shape, dtype=dt, device=device)  # noqa: E731
        codes = [new(torch.uint8, batch, cap, Hkv, d_h).view(FORMATS[fmt]) for _ in range(2)]
        scales = [new(torch.float32, batch, cap // tg.TG_CACHE_BLOCK, Hkv) for _ in range(2)]
        self._wrap(tg.CacheQ8(*codes, *scales, new(torch.int32, batch) if lengths is None else lengths,
                              s=new(torch.float32, batch, cap) if bias else None,
                              w=new(torch.float32, batch, cap) if weights else None))

    @classmethod
    def over(cls, k, v, k_scale, v_scale, lengths, s=None, w=None) -> "KVCacheQ8":
        """A cache over tensors that the caller has (see tokengate.CacheQ8 for their shapes)."""
        self = cls.__new__(cls)
        self._wrap(tg.CacheQ8(k, v, k_scale, v_scale, lengths, s=s, w=w))
        return self

    def _wrap(self, handle: tg.CacheQ8):
        self.handle = handle
        for name in ("k", "v", "k_scale", "v_scale", "lengths", "s", "w", "batch", "capacity", "Hkv", "d_h"):
            setattr(self, name, getattr(handle, name))
        self._workspace, self._retired, self._room = None, [], {}
        self.reserve()

    def reserve(self, n_q: int = 0, Hq: int = 0, accumulate: bool = False) -> torch.Tensor:
        """The workspace, large enough for decode calls of this shape: call it before capturing them."""
        key = (n_q, Hq, accumulate)
        if key not in self._room:
            n = tg.tg_cache_workspace_bytes(self.handle, n_q, Hq, accumulate)
            if n == 0:
                raise tg.TokenGateError("tg_cache_workspace_bytes", tg.TG_ERR_UNSUPPORTED)
            if self._workspace is None or self._workspace.numel() < n:
                if torch.cuda.is_current_stream_capturing():
                    raise RuntimeError("call reserve() before capturing a decode of this shape")
                workspace = torch.empty(n, dtype=torch.uint8, device=self.handle.device)
                workspace[:256].zero_()                     # the status word; the rest is written before it is read
                if self._workspace is not None:
                    self._retired.append(self._workspace)   # a captured graph may still use it, and its status stays
                self._workspace = workspace
            self._room[key] = n
        return self._workspace

    def append(self, k: torch.Tensor, v: torch.Tensor, s: Optional[torch.Tensor] = None,
               counts: Optional[torch.Tensor] = None) -> "KVCacheQ8":
        """tg_cache_append_q8: k, v [B, n, Hkv, d_h] bf16 become the last tokens of every sequence; `lengths`
        hold the tokens after the append."""
        tg.tg_cache_append_q8(self.handle, k, v, self._workspace, s, counts)
        return self

    def decode(self, q: torch.Tensor, out: Optional[torch.Tensor] = None, gain: Optional[torch.Tensor] = None,
               tau: float = 1.0, lse: Optional[torch.Tensor] = None, accumulate: bool = False,
               max_len: int = 0) -> torch.Tensor:
        """tg_gated_decode_q8: attention of the last n_q tokens' queries q [B, n_q, Hq, d_h] over the cache."""
        shape = q.shape
        if len(shape) != 4:
            raise ValueError("q must be [B, n_q, Hq, d_h]")
        ws = self.reserve(shape[1], shape[2], accumulate)
        return tg.tg_gated_decode_q8(self.handle, q, torch.empty_like(q) if out is None else out, ws, gain, tau,
                                     accumulate, max_len, lse)

    def read(self, k_out: torch.Tensor, v_out: torch.Tensor, first: int = 0):
        """tg_cache_read_q8: tokens from `first` on as bf16 into k_out, v_out [B, n, Hkv, d_h]."""
        return tg.tg_cache_read_q8(self.handle, k_out, v_out, first=first)

    def evict_into(self, dst: "KVCacheQ8", budget: int, sink: int = 0, recent: int = 0,
                   kept: Optional[torch.Tensor] = None, max_len: int = 0) -> torch.Tensor:
        """tg_cache_evict_q8: what stays of every sequence into dst, whose lengths (a tensor of its own, or one that it shares
        with other layers' targets) are written; returns the kept slots [B, budget]."""
        if kept is None:
            kept = torch.empty(self.batch, budget, dtype=torch.int32, device=self.handle.device)
        return tg.tg_cache_evict_q8(self.handle, dst.handle, kept, self._workspace, budget, sink=sink, recent=recent,
                                    max_len=max_len)

    def device_status(self) -> int:
        """Raw TG_STATUS_* bits of the calls so far, graphs captured on an earlier workspace among them (synchronises)."""
        status = 0
        with torch.cuda.device(self.handle.device):
            for workspace in (*self._retired, self._workspace):
                status |= tg.tg_device_status(workspace)
        return status
