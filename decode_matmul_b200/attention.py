"""Layer stack with its attention: the four phases of every layer, with the
rotated keys and values appended to a paged cache after phase 0 and the
attention of the new tokens over that cache as phase 1's input.

Where `tq_layer_stack` hands alpha * q straight to phase 1 (its k and v
outputs only stand in for attention), one layer here is

    y   = q|k|v of RHT(h)                          tq_layer_phase, phase 0
    y  += adapters of each token on q, k, v        tq_lora (optional)
    q'  = rotated q; cache <- rotated k, v         tq_kv_append
    a   = attention of q' over the cache           tq_attn (bf16)
    h   = phases 1, 2, 3 of a                      tq_layer_phase

Every call is enqueued on the current stream and none synchronises, so a
decode step can be captured in a CUDA graph (after `buffers`, or an earlier
step of as many tokens): positions, sequences and adapters are read on the
device, and a replay with new values in the same tensors is the next step.
"""
from __future__ import annotations

import math

PHASE_OPS = (("q", "k", "v"), ("o",), ("gate", "up"), ("down",))


class AttentionStack:
    """layers: one dict per layer of DeviceWeights (q, k, v, o, gate, up,
    down), of the same sizes in every layer.  caches: one KvCache per layer (all with the same heads).  freq:
    float64 [rot/2] rotation frequencies (None: no rotation).  scale: of the
    scores (None: head_dim ** -0.5).  window: of the attention (0: all keys).
    adapters: None, or one dict per layer of Lora by op name ("q", "k", "v"),
    bfloat16, over the phase's unrotated input."""

    def __init__(self, layers, caches, freq=None, interleaved: bool = False, scale=None, window: int = 0,
                 adapters=None):
        import torch

        from . import OPS, _need, layer_struct
        if not layers or len(caches) != len(layers) or (adapters is not None and len(adapters) != len(layers)):
            raise ValueError("one cache (and one dict of adapters) per layer is needed")
        c, w = caches[0], layers[0]
        self.q_heads, rest = divmod(w["q"].n, c.head_dim)
        if rest or self.q_heads % c.kv_heads:
            raise ValueError(f"{w['q'].n} query features do not make groups of heads of {c.head_dim}")
        kv, hidden, inter = c.kv_heads * c.head_dim, w["q"].k, w["gate"].n
        want = dict(q=(w["q"].n, hidden), k=(kv, hidden), v=(kv, hidden), o=(hidden, w["q"].n), gate=(inter, hidden),
                    up=(inter, hidden), down=(hidden, inter))
        for L, cache in zip(layers, caches):
            for op in OPS:
                if (L[op].n, L[op].k) != want[op]:
                    raise ValueError(f"{op}: {L[op].n} x {L[op].k}, but the stack's heads and first layer make it "
                                     f"{want[op][0]} x {want[op][1]}")
            if (cache.kv_heads, cache.head_dim, cache.q_dtype, cache.device) != (c.kv_heads, c.head_dim, c.q_dtype, c.device):
                raise ValueError("the caches of a stack have the same heads, type of queries and device")
            if any(t.device != c.device for op in OPS for t in (L[op].codes, L[op].scales, L[op].codebook)):
                raise ValueError(f"the weights of a stack are on its caches' device, {c.device}")
        for A, L in zip(adapters or (), layers):
            for op, lora in A.items():
                if op not in PHASE_OPS[0] or (lora.n, lora.k) != (L[op].n, L[op].k):
                    raise ValueError(f"adapter on {op!r}: only q, k and v, of their projection's size")
                if lora.a.dtype != torch.bfloat16 or lora.device != c.device:
                    raise ValueError(f"adapter on {op!r}: bfloat16 on {c.device} is needed, got {lora.a.dtype} on {lora.device}")
        if freq is not None:
            _need(freq, "freq", torch.float64, (freq.numel(),), c.device)
            if freq.numel() % 8 or 2 * freq.numel() > c.head_dim:
                raise ValueError(f"freq: {freq.numel()} frequencies, a multiple of 8 and at most half of {c.head_dim} are needed")
        if not 0 <= window < 2 ** 31 or (scale is not None and not math.isfinite(scale)):
            raise ValueError(f"window {window} has to be 0 to 2^31 - 1 and scale {scale} finite")
        self.layers, self.caches, self.freq, self.interleaved, self.window = layers, caches, freq, interleaved, window
        self.scale = c.head_dim ** -0.5 if scale is None else scale
        self.adapters = adapters
        self.device = c.device
        self.structs = [layer_struct(L) for L in layers]
        self._buf = {}    # sets of buffers by the most tokens they take
        self._views = {}  # their first m rows, by m

    def buffers(self, m: int) -> dict:
        """The workspace and activation buffers of steps of m tokens (kept; the last layer's values stay in them
        after a step: y, q, attn and the phases' handoffs).  Steps of up to 16, of 17 to 32, 33 to 64, ... tokens share
        one set, of which a step uses the first m rows (so that all sets together are at most twice the largest,
        however many numbers of tokens there are), so those follow one another on one stream.  A captured step's must
        exist before the capture, from an earlier step or this call: what a capture clears is clear only when it is
        replayed."""
        import torch

        from . import tq_attn_workspace, tq_layer_phase_workspace, tq_lora_workspace, workspace
        if m in self._views:
            return self._views[m]
        most = max(16, 1 << (m - 1).bit_length())
        if most not in self._buf:
            n = max(tq_attn_workspace(c, m, self.q_heads) for c in self.caches)  # refuses too many tokens
            with torch.cuda.device(self.device):  # on whose current stream the workspace is cleared
                if torch.cuda.is_current_stream_capturing():
                    raise RuntimeError(f"buffers({m}) has to be called before a step of {m} tokens is captured")
                # (the phases of all layers have the same sizes; fewer tokens can need more)
                n = max([n] + [tq_layer_phase_workspace(self.structs[0], p, i) for p in range(4)
                               for i in range(most // 2 + 1 if most > 16 else 1, most + 1)]
                        + [tq_lora_workspace(a, most) for A in self.adapters or () for a in A.values()])
                w, c, dev = self.layers[0], self.caches[0], self.device

                def bits(width):
                    return torch.empty((most, width), dtype=torch.int16, device=dev)

                heads = (most, self.q_heads, c.head_dim)
                self._buf[most] = dict(
                    ws=workspace(n, dev), y=torch.empty((most, sum(w[o].n for o in PHASE_OPS[0])), device=dev),
                    q=torch.empty(heads, dtype=c.q_dtype, device=dev),
                    attn=torch.empty(heads, dtype=torch.bfloat16, device=dev),
                    hand=[bits(w["q"].n), bits(w["o"].n), bits(w["gate"].n), bits(w["down"].n)])
        b = self._buf[most]
        self._views[m] = dict(ws=b["ws"], hand=[t[:m] for t in b["hand"]], **{k: b[k][:m] for k in ("y", "q", "attn")})
        return self._views[m]

    def forward(self, h, pos, seed: int, seq=None, adapter=None, out=None):
        """One step of m new tokens.  h: int16 (bf16 bits) [m][hidden]; pos: int32 [m], the tokens' positions (-1 = a
        padded row); seq: int32 [m], their rows of the block tables (None: token t is sequence t); adapter: int32 [m]
        (-1 = none), needed with adapters.  Writes the caches and returns the last hidden state, int16 [m][hidden]
        (`out` if given, which may be h; else a new tensor).  An index out of range shows in
        tq_workspace_status(buffers(m)["ws"])."""
        import torch

        from . import _need, tq_attn, tq_kv_append, tq_layer_phase, tq_lora, tq_stack_phase_seed
        if self.adapters is not None and adapter is None:
            raise ValueError("adapter: int32 [m] is needed, since the stack has adapters")
        m = h.shape[0]
        if h.dtype != torch.int16 or h.dim() != 2 or h.shape[1] != self.layers[0]["q"].k or not h.is_contiguous() or h.device != self.device:
            raise ValueError(f"h: contiguous int16 [m][{self.layers[0]['q'].k}] on {self.device} is needed")
        if out is None:
            out = torch.empty_like(h)
        elif out.dtype != h.dtype or out.shape != h.shape or not out.is_contiguous() or out.device != h.device:
            raise ValueError(f"out: like h, contiguous int16 {tuple(h.shape)} on {self.device}, is needed")
        # all of them before the first launch: a step that is refused has written no cache
        for name, t in (("pos", pos), ("seq", seq), ("adapter", adapter if self.adapters is not None else None)):
            if t is not None:
                _need(t, name, torch.int32, (m,), self.device)
        rows = min(c.pages.shape[0] for c in self.caches)
        if seq is None and m > rows:
            raise ValueError(f"{m} tokens without seq, but the block tables have {rows} rows")
        if m == 0:
            return out
        b = self.buffers(m)
        ws, y, hand = b["ws"], b["y"], b["hand"]
        with torch.cuda.device(self.device):
            x = h
            for l, (s, w, cache) in enumerate(zip(self.structs, self.layers, self.caches)):
                tq_layer_phase(s, 0, x, tq_stack_phase_seed(seed, l, 0), y, hand[0], ws)
                col = 0
                for op in PHASE_OPS[0]:
                    lora = self.adapters[l].get(op) if self.adapters is not None else None
                    if lora is not None:
                        tq_lora(lora, x.view(torch.bfloat16), adapter, y[:, col:col + w[op].n], ws=ws)
                    col += w[op].n
                tq_kv_append(cache, y, self.q_heads, pos, self.freq, self.interleaved, seq, b["q"], ws)
                tq_attn(cache, b["q"], pos, self.scale, seq, self.window, b["attn"], ws=ws)
                x = b["attn"].view(torch.int16).view(m, -1)
                for p in (1, 2, 3):
                    to = out if p == 3 and l + 1 == len(self.layers) else hand[p]
                    tq_layer_phase(s, p, x, tq_stack_phase_seed(seed, l, p), None, to, ws)
                    x = to
        return out
