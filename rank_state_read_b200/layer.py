"""One recurrent layer on the GPU: a plan plus the caller-owned device tensors.

Plumbing only (allocation with torch, the decode / flush call order of the C ABI);
the arithmetic runs in libsketchssm's kernels.
"""
from __future__ import annotations

from typing import Optional, Sequence

import numpy as np
import torch

from ._binding import (Plan, sketchssm_decode, sketchssm_decode_rows, sketchssm_delta_chunk, sketchssm_delta_step,
                       sketchssm_dense_decode, sketchssm_flush, sketchssm_flush_rows, sketchssm_gated_norm,
                       sketchssm_prefill, sketchssm_step)


def _dev(x, device) -> torch.Tensor:
    if isinstance(x, torch.Tensor):
        return x.to(device=device, dtype=torch.float32).contiguous()
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(device)


def _new(like: torch.Tensor, stream) -> torch.Tensor:
    """A packed tensor of ``like``'s shape and type for work on ``stream``.  Its memory comes from that
    stream's pool, so no other stream's work on it is pending, and is not handed out again before what
    the current stream does with the tensor is done."""
    if stream is None:
        return torch.empty(like.shape, dtype=like.dtype, device=like.device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    with torch.cuda.stream(stream):
        t = torch.empty(like.shape, dtype=like.dtype, device=like.device)
    t.record_stream(torch.cuda.current_stream(like.device))
    return t


class SketchLayer:
    """State S, sketch Y, key/value buffers and output y of one layer at a fixed batch.

    Protocol (include/sketchssm.h): flush(0) once to form the first sketch, then
    decode(pos) for pos = 0 .. W-1, flush(W), and again from pos = 0.

    A call that takes ``gate`` returns the gated norm of the read in the gate's type and shape
    instead of the read itself (which ``out`` still gets).
    """

    def __init__(self, kind: str, *, batch: int, heads: int, qk_heads: int, key_dim: int,
                 value_dim: int, window: int, groups: int, rank_cap: int, rank: Sequence[int],
                 omega, S0=None, norm_weight=None, norm_eps: float = 1e-6, norm_gate: str = "silu",
                 device="cuda", stream=None):
        omega_t = _dev(omega, device)
        self.plan = Plan(kind, batch=batch, heads=heads, qk_heads=qk_heads, key_dim=key_dim,
                         value_dim=value_dim, window=window, groups=groups,
                         basis_rows=omega_t.shape[1], rank_cap=rank_cap, rank=rank, stream=stream)
        sh = self.plan.shapes
        z = lambda name: torch.zeros(sh[name], dtype=torch.float32, device=device)
        self.kind = kind
        self.omega = omega_t
        self.S = z("S") if S0 is None else _dev(S0, device)
        self.Y = z("Y")
        self.kbuf, self.vbuf, self.abuf = z("kbuf"), z("vbuf"), z("abuf")
        self.bbuf = None if kind == "mamba2" else z("bbuf")
        self.y = z("y")
        self.window = window
        # the gated norm behind the read (``gate=`` of the calls below): Gated DeltaNet and KDA
        # norm each head, then gate; Mamba-2 gates, then norms the heads of each basis group
        self.norm_weight = None if norm_weight is None else _dev(norm_weight, device)
        self.norm_eps, self.norm_gate = norm_eps, norm_gate

    def gated_norm(self, y: torch.Tensor, gate: torch.Tensor, out=None, stream=None) -> torch.Tensor:
        """The layer's gated norm of a read y [rows][H][V]: of the gate's type and shape (or ``out``)."""
        if self.norm_weight is None:
            raise ValueError("the layer was made without norm_weight")
        d = self.plan.desc
        out = _new(gate, stream) if out is None else out
        groups = d.groups if self.kind == "mamba2" else d.heads
        shape = (y.shape[0], groups, d.heads * d.value_dim // groups)
        sketchssm_gated_norm(y.view(shape), gate.view(shape), self.norm_weight, out.view(shape), eps=self.norm_eps,
                             activation=self.norm_gate, gate_first=self.kind == "mamba2", stream=stream)
        return out

    def _read(self, y, gate, stream) -> torch.Tensor:
        return y if gate is None else self.gated_norm(y, gate, stream=stream)

    def flush(self, n: int, stream=None) -> None:
        sketchssm_flush(self.plan, self.S, self.omega, self.kbuf, self.vbuf, self.abuf, self.bbuf, n,
                        self.Y, stream)

    def decode(self, pos: int, q, k, v, a, beta: Optional[torch.Tensor] = None, out=None,
               stream=None, gate=None) -> torch.Tensor:
        y = self.y if out is None else out
        sketchssm_decode(self.plan, pos, q, k, v, a, beta, self.kbuf, self.vbuf, self.abuf, self.bbuf,
                         self.Y, self.omega, self.S, y, stream)
        return self._read(y, gate, stream)

    def dense_decode(self, pos: int, q, k, v, a, beta: Optional[torch.Tensor] = None, out=None,
                     stream=None, gate=None) -> torch.Tensor:
        y = self.y if out is None else out
        sketchssm_dense_decode(self.plan, pos, q, k, v, a, beta, self.kbuf, self.vbuf, self.abuf,
                               self.bbuf, self.S, y, stream)
        return self._read(y, gate, stream)

    def decode_rows(self, pos: torch.Tensor, q, k, v, a, beta: Optional[torch.Tensor] = None, out=None,
                    stream=None, gate=None) -> torch.Tensor:
        """Decode with a buffer position per batch row (pos: int32 [B] on the device)."""
        y = self.y if out is None else out
        sketchssm_decode_rows(self.plan, pos, q, k, v, a, beta, self.kbuf, self.vbuf, self.abuf, self.bbuf,
                              self.Y, self.omega, self.S, y, stream)
        return self._read(y, gate, stream)

    def flush_rows(self, n_tokens: torch.Tensor, stream=None) -> None:
        """Flush each batch row's first n_tokens[b] buffered tokens (int32 [B] on the device)."""
        sketchssm_flush_rows(self.plan, self.S, self.omega, self.kbuf, self.vbuf, self.abuf, self.bbuf,
                             n_tokens, self.Y, stream)

    def standard_step(self, q, k, v, a, beta: Optional[torch.Tensor] = None, out=None,
                      stream=None, gate=None) -> torch.Tensor:
        """The per-step recurrent decode (no buffer): S updated in place, y = S^T q."""
        y = self.y if out is None else out
        sketchssm_step(self.plan, q, k, v, a, beta, self.S, y, stream)
        return self._read(y, gate, stream)

    def prefill(self, k, v, a, beta: Optional[torch.Tensor] = None, stream=None) -> None:
        """Prefill handoff: the prompt (token-major k [B][T][Hqk][K], v [B][T][H][V],
        a [B][T][H] or KDA [B][T][H][K], beta [B][T][H]) applied to S, then Y formed
        from the new state; decoding continues at pos = 0."""
        sketchssm_prefill(self.plan, int(k.shape[1]), k, v, a, beta, self.S, self.omega, self.Y, stream)

    def prompt(self, cu: torch.Tensor, q, k, v, a, beta, slot=None, out=None, gate=None, *, normalize_qk=False,
               scale: float = 1.0, stream=None) -> torch.Tensor:
        """Packed prompts with their outputs (Gated DeltaNet): sequence i, tokens cu[i] .. cu[i+1]-1,
        continues batch row slot[i] (None: row i); then the sketches are formed, those of all batch
        rows, once a call (0.67 ms at 512 rows of 32 heads of 128).  q, k [N][Hqk][K] and v [N][H][V]
        of one type, a, beta [N][H] fp32; returns y [N][H][V] of that type (normed and gated with
        ``gate``).  The rows' decoding continues at pos = 0."""
        y = _new(v, stream) if out is None else out
        sketchssm_delta_chunk(self.plan, cu, q, k, v, a, beta, self.S, y, slot=slot, normalize_qk=normalize_qk,
                              scale=scale, stream=stream)
        self.flush(0, stream)
        return self._read(y, gate, stream)

    def step(self, q, k, v, a, beta, slot=None, out=None, gate=None, *, normalize_qk=False, scale: float = 1.0,
             stream=None) -> torch.Tensor:
        """One token for each row i on the state of batch row slot[i] (None: row i), without buffer or
        sketch (Gated DeltaNet): standard_step for tokens of any type and any choice of rows."""
        y = _new(v, stream) if out is None else out
        sketchssm_delta_step(self.plan, q, k, v, a, beta, self.S, y, slot=slot, normalize_qk=normalize_qk, scale=scale,
                             stream=stream)
        return self._read(y, gate, stream)

    def close(self) -> None:
        self.plan.close()
