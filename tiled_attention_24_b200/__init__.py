"""Fused tiled attention forward for NVIDIA B200 (sm_100a).

The compute lives in ``libtiledattn.so`` (CUDA kernels behind a C ABI, see
``include/tiledattn.h``); this package is its thin ctypes binding plus a few
conveniences that allocate outputs with torch and call the same entry points.
"""
from __future__ import annotations

import contextlib
import math

import torch

from ._binding import (AttnError, LIB_PATH, attn_check_status, attn_debug_counters, attn_decode,  # noqa: F401
                       attn_decode_gqa, attn_decode_noalloc, attn_decode_workspace_bytes, attn_fp4_scores,
                       attn_fwd, attn_fwd_fp8, attn_fwd_gqa, attn_fwd_varlen, attn_decode_varlen, attn_quantize_fp8, attn_quantize_int4, attn_bwd, attn_bwd_fp8p, attn_bwd_workspace_bytes,
                       attn_fwd_fp4, attn_fwd_int8, attn_int8_scores, attn_nvfp4_codes_bytes,
                       attn_nvfp4_sf_bytes, attn_quantize_int8, attn_quantize_nvfp4, attn_set_wait_limit_ns,
                       attn_status_string, attn_version, attn_watchdog_selftest, load,
                       attn_kv4_append, attn_kv4_read, attn_decode_kv4, attn_decode_kv4_splits,
                       attn_decode_kv4_workspace_bytes, attn_key_weights, attn_key_weights_workspace_bytes,
                       attn_kv4_evict, attn_kv4_evict_workspace_bytes)

__all__ = ["load", "attn_fwd", "attn_decode", "attn_decode_workspace_bytes", "attn_check_status",
           "attn_set_wait_limit_ns", "attn_watchdog_selftest", "attn_version", "attn_status_string",
           "AttnError", "forward", "decode", "quantize_int8", "forward_int8",
           "attn_quantize_int8", "attn_fwd_int8", "attn_int8_scores", "attn_decode_noalloc",
           "attn_quantize_nvfp4", "attn_fwd_fp4", "attn_fp4_scores", "quantize_nvfp4", "forward_fp4",
           "attn_fwd_gqa", "attn_decode_gqa", "attn_quantize_int4", "quantize_int4", "forward_int4",
           "attn_bwd", "attn_bwd_fp8p", "attn_bwd_workspace_bytes", "backward",
           "attn_quantize_fp8", "attn_fwd_fp8", "quantize_fp8", "forward_fp8", "hadamard_signs",
           "attn_fwd_varlen", "attn_decode_varlen", "forward_varlen", "decode_varlen",
           "attn_kv4_append", "attn_kv4_read", "attn_decode_kv4", "attn_decode_kv4_splits",
           "attn_decode_kv4_workspace_bytes", "attn_key_weights", "attn_key_weights_workspace_bytes",
           "attn_kv4_evict", "attn_kv4_evict_workspace_bytes", "KV4Cache", "decode_kv4", "key_weights",
           "attn_debug_counters", "DIRECT_P", "QUANT_AFTER_EXP"]

DIRECT_P, QUANT_AFTER_EXP = 0, 1


def forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
            scale: float | None = None, stream=None):
    """Allocate O (bf16) and LSE (fp32) and run ``attn_fwd`` (``attn_fwd_gqa``
    when k/v have fewer heads than q: grouped-query attention)."""
    B, H, Nq, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    if k.shape[1] != H:
        attn_fwd_gqa(q, k, v, o, lse, causal, scale, stream)
    else:
        attn_fwd(q, k, v, o, lse, causal, scale, stream)
    return o, lse


def backward(q, k, v, o, lse, dout, causal: bool = False, scale: float | None = None, stream=None,
             p_fp8: bool = False):
    """Allocate dq, dk, dv (bf16) and the row-statistic workspace, run ``attn_bwd``
    (``attn_bwd_fp8p`` with ``p_fp8``: P in e4m3 for dV) (o, lse: the
    forward's outputs for the same arguments)."""
    B, H, Nq, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty(max(16, attn_bwd_workspace_bytes(B, H, Nq)), dtype=torch.uint8, device=q.device)
    (attn_bwd_fp8p if p_fp8 else attn_bwd)(q, k, v, o, dout, lse, dq, dk, dv, causal, scale, ws, stream)
    return dq, dk, dv


def decode(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float | None = None,
           num_splits: int = 16, workspace: torch.Tensor | None = None, stream=None):
    """Allocate O, LSE (and a workspace if none is given) and run ``attn_decode``
    (``attn_decode_gqa`` when k/v have fewer heads than q)."""
    B, H, _, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if workspace is None:
        nbytes = attn_decode_workspace_bytes(B, H, d, num_splits)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, 1), dtype=torch.float32, device=q.device)
    if k.shape[1] != H:
        attn_decode_gqa(q, k, v, o, lse, scale, num_splits, workspace, stream)
    else:
        attn_decode(q, k, v, o, lse, scale, num_splits, workspace, stream)
    return o, lse


def forward_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, causal: bool = False,
                   scale: float | None = None, stream=None):
    """Packed variable-length forward (q [total_q,H,d], k/v [total_k,Hkv,d],
    cu_seqlens int32 [B+1] on the device).  Returns (o [total_q,H,d], lse [H,total_q])."""
    total_q, H, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.zeros_like(q)
    lse = torch.full((H, total_q), float("-inf"), dtype=torch.float32, device=q.device)
    attn_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, causal, scale, stream)
    return o, lse


def decode_varlen(q, k, v, seqlens_k, scale: float | None = None, num_splits: int = 16, stream=None):
    """Decode with a cache length per batch entry (seqlens_k int32 [B] on the device)."""
    B, H, _, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    ws = torch.empty(attn_decode_workspace_bytes(B, H, d, num_splits), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, 1), dtype=torch.float32, device=q.device)
    attn_decode_varlen(q, k, v, o, lse, seqlens_k, scale, num_splits, ws, stream)
    return o, lse


def quantize_int8(x: torch.Tensor, per_head: bool = False, stream=None):
    """INT8 symmetric quantisation (per token row, or per (batch, head))."""
    B, H, N, d = x.shape
    xq = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    xs = torch.empty((B, H) if per_head else (B, H, N), dtype=torch.float32, device=x.device)
    attn_quantize_int8(x, xq, xs, per_head, stream)
    return xq, xs


def forward_int8(q, k, v, causal: bool = False, scale: float | None = None, stream=None):
    """Quantise bf16 q, k (per token) and v (per head) and run the INT8 forward.
    Returns (o fp32, lse fp32)."""
    B, H, Nq, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    qi, qs = quantize_int8(q, False, stream)
    ki, ks = quantize_int8(k, False, stream)
    vi, vs = quantize_int8(v, True, stream)
    o = torch.empty((B, H, Nq, d), dtype=torch.float32, device=q.device)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    attn_fwd_int8(qi, qs, ki, ks, vi, vs, o, lse, causal, scale, stream)
    return o, lse


def quantize_int4(x: torch.Tensor, stream=None):
    """Token-level INT4 quantisation (codes in [-7, 7], int8 containers)."""
    B, H, N, d = x.shape
    xq = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    xs = torch.empty((B, H, N), dtype=torch.float32, device=x.device)
    attn_quantize_int4(x, xq, xs, stream)
    return xq, xs


def forward_int4(q, k, v, causal: bool = False, scale: float | None = None, stream=None):
    """INT4 q, k (per token), INT8 v (per head), through the INT8 forward.
    Returns (o fp32, lse fp32)."""
    B, H, Nq, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    qi, qs = quantize_int4(q, stream)
    ki, ks = quantize_int4(k, stream)
    vi, vs = quantize_int8(v, True, stream)
    o = torch.empty((B, H, Nq, d), dtype=torch.float32, device=q.device)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    attn_fwd_int8(qi, qs, ki, ks, vi, vs, o, lse, causal, scale, stream)
    return o, lse


def hadamard_signs(d: int, seed: int = 0, device="cuda"):
    """Seeded random sign vector (fp32, +-1) of the FP8 rotation H_d diag(signs)."""
    g = torch.Generator().manual_seed(int(seed))
    s = torch.randint(0, 2, (d,), generator=g, dtype=torch.int64) * 2 - 1
    return s.to(torch.float32).to(device)


def quantize_fp8(x: torch.Tensor, mode: int, signs: torch.Tensor | None = None, stream=None):
    """e4m3 codes (uint8) and fp32 scales of a bf16 [B,H,N,d] tensor: mode 0 per
    token row (rotated first when ``signs`` is given), mode 1 per channel."""
    B, H, N, d = x.shape
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scales = torch.empty((B, H, N) if mode == 0 else (B, H, d), dtype=torch.float32, device=x.device)
    attn_quantize_fp8(x, codes, scales, mode, signs, stream)
    return codes, scales


def forward_fp8(q, k, v, causal: bool = False, scale: float | None = None, rotate: bool = True,
                signs: torch.Tensor | None = None, stream=None):
    """Quantise bf16 q, k (per token, rotated by H_d diag(signs) unless
    ``rotate`` is False) and v (per channel) to e4m3 and run the FP8 forward.
    Returns (o fp32, lse fp32)."""
    B, H, Nq, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if rotate and signs is None:
        signs = hadamard_signs(d, 0, q.device)
    sg = signs if rotate else None
    qc, qs = quantize_fp8(q, 0, sg, stream)
    kc, ks = quantize_fp8(k, 0, sg, stream)
    vc, vs = quantize_fp8(v, 1, None, stream)
    o = torch.empty((B, H, Nq, d), dtype=torch.float32, device=q.device)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    attn_fwd_fp8(qc, qs, kc, ks, vc, vs, o, lse, causal, scale, rotate, stream)
    return o, lse


def quantize_nvfp4(x: torch.Tensor, mode: int, stream=None):
    """NVFP4 codes + tiled scales of a bf16 [B,H,N,128] tensor (mode 0: Q/K,
    mode 1: V, written transposed)."""
    B, H, N, d = x.shape
    codes = torch.empty(attn_nvfp4_codes_bytes(B, H, N, d, mode), dtype=torch.uint8, device=x.device)
    sf = torch.empty(attn_nvfp4_sf_bytes(B, H, N, d, mode), dtype=torch.uint8, device=x.device)
    attn_quantize_nvfp4(x, codes, sf, mode, stream)
    return codes, sf


def forward_fp4(q, k, v, causal: bool = False, scale: float | None = None, p_mode: int = DIRECT_P, stream=None):
    """Quantise bf16 q, k, v to NVFP4 and run the FP4 forward.  Returns (o fp32, lse fp32)."""
    B, H, Nq, d = q.shape
    Nkv = k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    qc, qs = quantize_nvfp4(q, 0, stream)
    kc, ks = quantize_nvfp4(k, 0, stream)
    vc, vs = quantize_nvfp4(v, 1, stream)
    o = torch.empty((B, H, Nq, d), dtype=torch.float32, device=q.device)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    attn_fwd_fp4(qc, qs, kc, ks, vc, vs, o, lse, B, H, Nq, Nkv, causal, scale, p_mode, stream)
    return o, lse


class KV4Cache:
    """A 4-bit key/value cache: codes kc, vc (uint8 [B,Hkv,capacity,d/2]) with scales ks,
    vs (bf16 [B,Hkv,capacity,d/32]), the live slots seqlens and next token positions
    next_pos of each sequence (int32 [B]) and, with ``track``, the accumulated
    attention weights and the positions per slot that an eviction goes by.

    ``capacity`` is rounded up to a multiple of 16.  The host keeps an upper bound of
    the lengths, so that an append that fits needs no synchronisation; where the bound
    has no room left, the lengths are read (one synchronisation), and an append that
    does not fit is refused.

    An append, ``reset`` or ``evict`` captured into a graph moves the lengths at every
    replay, unseen by the host: from then on they are read at every append outside a graph.
    A replayed append whose tokens find no room keeps what fits and counts the others in
    ``dropped`` (int32 [B]); an append outside a graph is refused from then on, until
    ``reset`` empties those sequences."""

    def __init__(self, B: int, Hkv: int, capacity: int, d: int, device="cuda", track: bool = True):
        if B < 1 or Hkv < 1 or capacity < 1 or d not in (64, 128):
            raise ValueError(f"B, Hkv, capacity must be positive and d 64 or 128, got {B}, {Hkv}, {capacity}, {d}")
        capacity = -(-capacity // 16) * 16
        self.B, self.Hkv, self.capacity, self.d = B, Hkv, capacity, d
        z = lambda shape, dtype: torch.zeros(shape, dtype=dtype, device=device)  # noqa: E731
        self.kc, self.vc = (z((B, Hkv, capacity, d // 2), torch.uint8) for _ in range(2))
        self.ks, self.vs = (z((B, Hkv, capacity, d // 32), torch.bfloat16) for _ in range(2))
        self.seqlens, self.next_pos = z((B,), torch.int32), z((B,), torch.int32)
        self.weights = z((B, Hkv, capacity), torch.float32) if track else None
        self.positions = z((B, Hkv, capacity), torch.int32) if track else None
        self.dropped = z((B,), torch.int32)
        self.length_bound = 0
        self._in_graph = False  # whether a graph may move the lengths

    def append(self, k: torch.Tensor, v: torch.Tensor, counts: torch.Tensor | None = None, stream=None):
        """Append n tokens (k, v bf16 [B,Hkv,n,d]) to every sequence, or the first
        ``counts[b]`` (int32 [B], 0 to n) of them."""
        n = k.shape[2]
        captured = self._capturing(stream)
        bound = self.capacity if captured else self._bound_after(n, counts, stream)
        attn_kv4_append(k, v, self.kc, self.ks, self.vc, self.vs, self.seqlens, counts, self.weights, self.positions,
                        self.next_pos if self.positions is not None else None, stream)
        with _stream_context(stream, k.device):
            by = n if counts is None else counts.clamp(0, n)
            self.next_pos.add_(by)
            if captured:
                room = self.capacity - self.seqlens
                self.dropped.add_((by - room).clamp_(min=0))
                by = torch.minimum(room, torch.full_like(room, n) if counts is None else by)
            self.seqlens.add_(by)
        self.length_bound = bound

    def _bound_after(self, n, counts, stream):
        """Upper bound of the lengths after an append of n tokens; ValueError where they do not fit."""
        if self.length_bound + n <= self.capacity and not self._in_graph:
            return self.length_bound + n
        with _stream_context(stream, self.seqlens.device):
            after = self.seqlens + (n if counts is None else counts.clamp(0, n))
            most, dropped = torch.stack((after.max(), self.dropped.max())).tolist()
        if dropped:
            raise ValueError("tokens of an append in a replayed graph found no room (see dropped): reset those sequences")
        if most > self.capacity:
            raise ValueError(f"{n} more tokens may not fit: a sequence would need {most} of {self.capacity} slots")
        return most

    def _capturing(self, stream):
        """Whether calls on the stream go into a graph now; the cache then no longer trusts its bound."""
        with _stream_context(stream, self.seqlens.device):
            captured = self.seqlens.is_cuda and torch.cuda.is_current_stream_capturing()
        self._in_graph |= captured
        return captured

    def reset(self, sequences: torch.Tensor | None = None, stream=None):
        """Empty the given sequences (bool [B] on the cache's device; default: all), for
        requests that have ended: their next token goes to slot 0, at position 0."""
        captured = self._capturing(stream)
        with _stream_context(stream, self.seqlens.device):
            for t in (self.seqlens, self.next_pos, self.dropped):
                t.zero_() if sequences is None else t.masked_fill_(sequences, 0)
        if sequences is None and not captured:
            self.length_bound = 0

    def read(self, n: int | None = None, stream=None):
        """(k, v) of the first n slots (default: the length bound; once a graph may have
        moved the lengths, the longest one, read from the device) as bf16 [B,Hkv,n,d]."""
        if n is None:
            n = self.length_bound
            if self._capturing(stream):
                raise ValueError("in a graph n has to be given: the lengths are not known to the host")
            if self._in_graph:
                with _stream_context(stream, self.seqlens.device):
                    n = int(self.seqlens.max())
        out = []
        with _stream_context(stream, self.kc.device):
            for c, s in ((self.kc, self.ks), (self.vc, self.vs)):
                x = torch.empty((self.B, self.Hkv, n, self.d), dtype=torch.bfloat16, device=c.device)
                attn_kv4_read(c, s, x, None, stream)
                out.append(x)
        return tuple(out)

    def evict(self, n_keep: int, n_recent: int = 0, stream=None):
        """Keep at most n_keep slots per (batch, cache head): the n_recent newest tokens,
        then those of the largest accumulated weight.  Returns the old slot of each
        kept one, int32 [B,Hkv,n_keep] (-1 where a sequence is shorter)."""
        if self.weights is None:
            raise ValueError("this cache does not track weights: nothing to evict by")
        if not 1 <= n_keep <= self.capacity:
            raise ValueError(f"n_keep must be from 1 to {self.capacity}, got {n_keep}")
        captured = self._capturing(stream)
        with _stream_context(stream, self.kc.device):
            kept = torch.empty((self.B, self.Hkv, n_keep), dtype=torch.int32, device=self.kc.device)
            ws = torch.empty(attn_kv4_evict_workspace_bytes(self.B, self.Hkv, self.capacity, n_keep),
                             dtype=torch.uint8, device=self.kc.device)
            attn_kv4_evict(self.kc, self.ks, self.vc, self.vs, self.weights, self.positions, self.seqlens,
                           self.next_pos, self.weights, self.positions, kept, n_recent, ws, stream)
            self.seqlens.clamp_(max=n_keep)
        if not captured:
            self.length_bound = min(self.length_bound, n_keep)
        return kept


def _stream_context(stream, device):
    """torch's own small operations (allocation, lengths) on the stream of the kernels."""
    if device.type != "cuda":
        return contextlib.nullcontext()
    if stream is None:
        return torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def decode_kv4(q: torch.Tensor, cache: KV4Cache, scale: float | None = None, num_splits: int | None = None,
               workspace: torch.Tensor | None = None, track: bool | None = None, stream=None):
    """Allocate O, LSE (and a workspace if none is given) and run ``attn_decode_kv4`` over
    the cache; its weights grow by this step's unless ``track`` is False."""
    B, Hq, _, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    weights = cache.weights if track is None or track else None
    if track and weights is None:
        raise ValueError("this cache does not track weights")
    if num_splits is None:
        num_splits = attn_decode_kv4_splits(B, Hq, cache.Hkv, cache.capacity, d)
    with _stream_context(stream, q.device):
        if workspace is None:
            nbytes = attn_decode_kv4_workspace_bytes(B, Hq, cache.Hkv, cache.capacity, d, num_splits, weights is not None)
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        o = torch.empty_like(q)
        lse = torch.empty((B, Hq, 1), dtype=torch.float32, device=q.device)
        attn_decode_kv4(q, cache.kc, cache.ks, cache.vc, cache.vs, o, lse, cache.seqlens, scale, num_splits,
                        workspace, weights, stream)
    return o, lse


def key_weights(q: torch.Tensor, k: torch.Tensor, lse: torch.Tensor, causal: bool = False, scale: float | None = None,
                out: torch.Tensor | None = None, seqlens: torch.Tensor | None = None, accumulate: bool = False,
                stream=None):
    """Attention weight each key of a prompt received, fp32 [B,Hkv,Nkv] (or the first Nkv
    entries of the rows of ``out``, for instance a cache's weights).  ``seqlens`` (int32
    [B]): a padded batch; without ``causal``, lse then has to leave the padding's keys out,
    which ``forward`` does not."""
    B, Hq, Nq, d = q.shape
    Hkv, Nkv = k.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    with _stream_context(stream, q.device):
        if out is None:
            out = torch.empty((B, Hkv, Nkv), dtype=torch.float32, device=q.device)
        ws = torch.empty(max(16, attn_key_weights_workspace_bytes(B, Hq, Hkv, Nq, Nkv, d)), dtype=torch.uint8,
                         device=q.device)
        attn_key_weights(q, k, lse, out, causal, scale, ws, seqlens, accumulate, stream)
    return out
