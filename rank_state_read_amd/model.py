"""A model's recurrent layers decoded one token at a time.

The Nemotron Nano 9B v2 calibration card ("SketchSSM calibration: Nemotron
Nano 9B v2 (BF16 weights)", "Contents") lists 27 recurrent layers, each with
its own group-shared basis (the basis array is (27, 8, 79, 128), with the model
layer index of each entry in ``layer_ids``).  Every such layer keeps its own
state cache, sketch and window; one decode token passes through all of them in
turn.  ``SketchModel`` holds those layers (``SketchLayer`` objects, one per
recurrent layer, all with the same window length) and runs that loop over the
C entry points: at window position 0 .. W-2 each layer's read, at W-1 each
layer's last read fused into its flush.  All layers share one window phase,
since every layer sees every token.  ``prefill`` runs the sequences' prompts
through the layers first.  A layer with a gated norm (``set_norm``) returns the
normed output; its token inputs hold the gate ``z``, unless the norm has none.
A layer without one returns its y.  A norm with a skip
``D`` (Mamba-2: y = S^T q + D x) takes the token's ``x``; without that key it takes
``v``, which is x only where no step size is in it (a layer whose heads share keys
holds dt in v = dt x).

Only the recurrent part of a layer is here: the projections that produce a
layer's q, k, v, decay and beta from the previous layer's output are not part of
the decode path this library implements, so the caller supplies each layer's
token inputs.  No arithmetic happens in this module.
"""
from __future__ import annotations

from typing import Dict, List, Optional, Sequence

import torch

from .binding import GATE
from .layer import SketchLayer


class SketchModel:
    def __init__(self, layers: Sequence[SketchLayer], layer_ids: Optional[Sequence[int]] = None):
        if not layers:
            raise ValueError("a model needs at least one recurrent layer")
        W = layers[0].W
        if any(L.W != W for L in layers):
            raise ValueError("all layers must share one window length")
        self.layers: List[SketchLayer] = list(layers)
        self.layer_ids = list(range(len(layers))) if layer_ids is None else [int(i) for i in layer_ids]
        if len(self.layer_ids) != len(self.layers):
            raise ValueError("one layer id per layer")
        self.W = W
        self.pos = 0

    def start(self, stream=None):
        """Form every layer's first sketch from its current state (after a
        prefill) and restart the window at position 0."""
        for L in self.layers:
            L.flush(0, stream=stream)
        self.pos = 0

    def prefill(self, tokens: Sequence[Dict[str, Optional[torch.Tensor]]], offsets: torch.Tensor, max_len: int,
                stream=None) -> List[torch.Tensor]:
        """The prompts of all sequences through every layer, from empty states:
        tokens offsets[b] .. offsets[b+1]-1 of layer i's packed inputs
        ``tokens[i]`` are sequence b's, at most max_len of them.  Writes every state
        and first sketch, restarts the window and returns the layers' outputs
        for all tokens."""
        self._check_tokens(tokens)
        if offsets.numel() != self.layers[0].B + 1:
            raise ValueError("one prompt per sequence")
        out = []
        for L, d in zip(self.layers, tokens):
            y = L.prefill(offsets, max_len, d["q"], d["k"], d["v"], d["a"], d.get("beta"), stream=stream)
            out.append(self._normed(L, y, d, stream))
        self.start(stream)
        return out

    def _check_tokens(self, tokens):
        """Before any layer's state or window changes."""
        if len(tokens) != len(self.layers):
            raise ValueError("one token input per layer")
        for i, (L, d) in enumerate(zip(self.layers, tokens)):
            norm = getattr(L, "norm", None)
            if norm is not None and (d.get("z") is None) != (norm[2] in ("none", GATE["none"])):
                raise ValueError(f"layer {i}: " + ("no gate z for its gated norm" if d.get("z") is None else
                                                   "a gate z, and its norm takes none"))

    @staticmethod
    def _normed(L, y, d, stream):
        z = d.get("z")
        if getattr(L, "norm", z) is None:  # (a layer type of another kind without that attribute: by its tokens)
            return y
        return L.gated_norm(y, z, d["v"] if d.get("x") is None else d["x"], stream=stream)

    def decode_step(self, tokens: Sequence[Dict[str, Optional[torch.Tensor]]], stream=None) -> List[torch.Tensor]:
        """One token through every layer.  ``tokens[i]`` holds layer i's device
        inputs (``q``, ``k``, ``v``, ``a`` and, for the delta rule, ``beta``);
        returns the layers' output buffers (each layer's ``y``, overwritten by
        the next step; of a layer with a norm, a new tensor of the normed output)."""
        self._check_tokens(tokens)
        last = self.pos == self.W - 1
        out = []
        for L, d in zip(self.layers, tokens):
            if last:
                y = L.read_flush(d["q"], d["k"], d["v"], d["a"], d.get("beta"), stream=stream)
            else:
                y = L.read(self.pos, d["q"], d["k"], d["v"], d["a"], d.get("beta"), stream=stream)
            out.append(self._normed(L, y, d, stream))
        self.pos = (self.pos + 1) % self.W
        return out
