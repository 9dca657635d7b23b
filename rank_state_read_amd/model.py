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

Drafted tokens are verified by ``tree_read``: trees of tokens of listed rows, read
over what every layer holds; ``tree_accept`` keeps the accepted paths.  Rows then
stand at window positions of their own, which the caller keeps in a device array
(``flush_seq`` empties the windows of listed rows); the common position of
``decode_step`` is for batches that move in step.  ``cache_store`` and
``cache_load`` copy rows' states of all layers to an 8-bit cache and back.

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

    # -- rows at window positions of their own -----------------------------------
    def tree_read(self, tokens: Sequence[Dict[str, Optional[torch.Tensor]]], parents: torch.Tensor,
                  offsets: torch.Tensor, max_nodes: int, pos: Optional[torch.Tensor] = None,
                  rows: Optional[torch.Tensor] = None, stream=None) -> List[torch.Tensor]:
        """Trees of drafted tokens through every layer: nodes offsets[i] .. offsets[i+1]-1 of layer j's packed inputs
        ``tokens[j]`` are sequence i's, ``parents`` each one's parent within its tree (-1: none), ``pos`` every row's
        held-back tokens.  Returns the layers' (normed) outputs of all nodes; no layer changes."""
        self._check_tokens(tokens)
        out = []
        for L, d in zip(self.layers, tokens):
            y = L.tree_read(offsets, max_nodes, parents, d["q"], d["k"], d["v"], d["a"], d.get("beta"), pos=pos, rows=rows,
                            stream=stream)
            out.append(self._normed(L, y, d, stream))
        return out

    def tree_accept(self, tokens: Sequence[Dict[str, Optional[torch.Tensor]]], parents: torch.Tensor,
                    offsets: torch.Tensor, accepted: torch.Tensor, pos: torch.Tensor,
                    rows: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """The path to node accepted[i] of each tree goes to every layer's window; returns the rows' held-back tokens
        then.  ``tokens``, ``parents``, ``offsets``, ``pos`` and ``rows`` as they were read."""
        if len(tokens) != len(self.layers):
            raise ValueError("one token input per layer")
        new_pos = None
        for L, d in zip(self.layers, tokens):
            new_pos = L.tree_accept(offsets, parents, accepted, d["k"], d["v"], d["a"], d.get("beta"), pos=pos, rows=rows,
                                    new_pos=new_pos, stream=stream)
        return new_pos

    def flush_seq(self, rows: torch.Tensor, n_tokens: torch.Tensor, stream=None):
        """Every layer's flush of the listed rows, which hold n_tokens tokens back (0 .. W)."""
        for L in self.layers:
            L.flush_seq(rows, n_tokens, stream=stream)

    def new_cache(self, n_slots: int, format: str = "i8", stream=None) -> list:
        """An empty cache of states per layer, for calls on `stream`."""
        given = {} if stream is None else {"stream": stream}
        return [L.new_cache(n_slots, format, **given) for L in self.layers]

    def cache_store(self, caches: Sequence, rows: torch.Tensor, slots: torch.Tensor, stream=None):
        """Every layer's states of the listed rows (their windows flushed before) to slots of its cache."""
        if len(caches) != len(self.layers):
            raise ValueError("one cache per layer")
        for L, c in zip(self.layers, caches):
            L.cache_store(c, rows, slots, stream=stream)

    def cache_load(self, caches: Sequence, slots: torch.Tensor, rows: torch.Tensor, stream=None):
        """Slots (negative: the zero state) back to the listed rows of every layer, with their first sketches.  The rows'
        positions are the caller's: 0 from here on, since what a row held back before does not follow its new state."""
        if len(caches) != len(self.layers):
            raise ValueError("one cache per layer")
        none = self.layers[0].zeros_like(rows, stream)
        for L, c in zip(self.layers, caches):
            L.cache_load(c, slots, rows, stream=stream)
            L.flush_seq(rows, none, stream=stream)
