"""What a speculative serving step needs beside the paged cache: the rotation of
queries and keys (skv_rotary) and the verification of drafted trees
(skv_tree_verify)."""
from __future__ import annotations

import ctypes as C

import torch

from . import _binding as B
from .api import _after_current
from .paged import _F32, _I32, _I64, _Status, _check_words, _stream_of

_PROBS = {torch.float32: B.SKV_PROB_F32, torch.bfloat16: B.SKV_PROB_BF16}

# 2^192 / (2 pi), rounded down
_TURN = 0x28BE60DB9391054A7F09D5F47D4D377036D8A5664F10E410


def _turns(freq) -> list:
    """Each frequency (radians per position) in units of 2^-64 of a turn, modulo 1, as a signed word."""
    out = []
    for f in freq:
        num, den = float(f).as_integer_ratio()
        t = (num * _TURN // den >> 127) + 1 >> 1
        t &= (1 << 64) - 1
        out.append(t - (1 << 64) if t >> 63 else t)
    return out


class Rotary:
    """Norms and rotation of query and key heads (skv_rotary), on the GPU.

    inv_freq: radians per position of each of the rot_dim / 2 frequencies (numbers; a tensor's are
    taken as they are), rot_dim a multiple of 16 up to head_dim; q_norm, k_norm: the weights
    [head_dim] of the heads' norms, or None for none; axes: for each frequency the axis of positions that it
    follows (default: one axis), interleaved: pairs (2 j, 2 j + 1) instead of
    (j, j + rot_dim / 2); amplitude: factor of the rotated channels."""

    def __init__(self, head_dim: int, inv_freq, q_norm: torch.Tensor | None = None, k_norm: torch.Tensor | None = None,
                 eps: float = 1e-6, axes=None, interleaved: bool = False, amplitude: float = 1.0, device="cuda"):
        freq = inv_freq.tolist() if isinstance(inv_freq, torch.Tensor) else list(inv_freq)
        if any(not abs(float(f)) < float("inf") for f in freq):
            raise ValueError("inv_freq must be finite")
        self.head_dim, self.rot_dim = int(head_dim), 2 * len(freq)
        axes = None if axes is None else [int(x) for x in (axes.tolist() if isinstance(axes, torch.Tensor) else axes)]
        if axes is not None and (len(axes) != len(freq) or any(not 0 <= x < 16 for x in axes)):
            raise ValueError("axes must name an axis (0 to 15) for each frequency")
        self.n_axes = max(axes) + 1 if axes else 1
        for w in (q_norm, k_norm):
            if w is not None and (w.dim() != 1 or w.numel() != self.head_dim or not w.is_floating_point()):
                raise ValueError(f"q_norm and k_norm must be floating-point tensors [{self.head_dim}]")
        self.turns = torch.tensor(_turns(freq), dtype=_I64).to(device)
        self.axes = None if axes is None else torch.tensor(axes, dtype=torch.uint8).to(device)
        self.q_norm, self.k_norm = (None if w is None else w.detach().to(device, _F32, copy=True).contiguous() for w in (q_norm, k_norm))
        if not self.turns.is_cuda:
            raise ValueError("a Rotary lives on a GPU")
        self._device = self.turns.device.index
        at = lambda t: None if t is None else t.data_ptr()                       # noqa: E731
        self._c = B.skv_rotary(B.SKV_FORMAT_VERSION, self.head_dim, self.rot_dim, self.n_axes, bool(interleaved), eps, amplitude,
                               at(self.turns), at(self.axes), at(self.q_norm), at(self.k_norm))
        self._ref = C.byref(self._c)
        B.check("skv_rotary_check", B.lib().skv_rotary_check(self._ref))
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self._device).synchronize()


class Verifier(_Status):
    """Verification of the drafted trees of n_requests requests over a vocabulary (skv_tree_verify)."""

    def __init__(self, n_requests: int, vocab: int, device="cuda"):
        self.n_requests, self.vocab = int(n_requests), int(vocab)
        self._new_status(device)
        if not self.status.is_cuda:
            raise ValueError("a Verifier lives on a GPU")
        self._settle()

    def _probs(self, t, n):
        """The kind of whole rows of probabilities, and their stride."""
        kind = _PROBS.get(t.dtype)
        if kind is None or t.shape != (n, self.vocab) or t.get_device() != self._device:
            raise ValueError(f"probabilities must be float32 or bfloat16 tensors [{n}][{self.vocab}] on cuda:{self._device}")
        down, across = t.stride()
        if across != 1 or (n > 1 and down < self.vocab):
            raise ValueError("probabilities must be whole rows")
        return kind, down

    def verify_into(self, probs, tokens, cu_new, uniform, accepted, rows, next_tokens, parents=None, draft_probs=None,
                    distinct: bool = False, slots=None, kept=None, ctx_len=None, ctx_out=None, stream=None):
        """Enqueue skv_tree_verify. probs, draft_probs (or None: the draft's tokens are its best): float32 or
        bf16 [n_rows][vocab], of one type, one row per node, node 0 of a request its last certain token;
        tokens, parents (node numbers; None: chains): int32 [n_rows]; uniform: float32
        [n_rows] in [0, 1), node 0's for the next token; distinct: siblings were drawn without
        replacement. Out: accepted and next_tokens int32 [n_requests], rows int32 [n_rows], and with
        slots (int64 [n_rows]) kept, with ctx_len (int32 [n_requests]) ctx_out."""
        n, dev = tokens.numel(), self._device
        kind, stride = self._probs(probs, n)
        draft, draft_stride = None, 0
        if draft_probs is not None:
            draft_kind, draft_stride = self._probs(draft_probs, n)
            if draft_kind != kind:
                raise ValueError("probs and draft_probs must have one type")
            draft = draft_probs.data_ptr()
        _check_words("tokens and rows", _I32, n, dev, tokens, rows)
        _check_words("uniform", _F32, n, dev, uniform)
        _check_words("cu_new", _I32, self.n_requests + 1, dev, cu_new)
        _check_words("accepted and next_tokens", _I32, self.n_requests, dev, accepted, next_tokens)
        if parents is not None:
            _check_words("parents", _I32, n, dev, parents)
            parents = parents.data_ptr()
        if (slots is None) != (kept is None) or (ctx_len is None) != (ctx_out is None):
            raise ValueError("slots come with kept, ctx_len with ctx_out")
        if slots is not None:
            _check_words("slots and kept", _I64, n, dev, slots, kept)
            slots, kept = slots.data_ptr(), kept.data_ptr()
        if ctx_len is not None:
            _check_words("ctx_len and ctx_out", _I32, self.n_requests, dev, ctx_len, ctx_out)
            ctx_len, ctx_out = ctx_len.data_ptr(), ctx_out.data_ptr()
        rc = B.lib().skv_tree_verify(kind, probs.data_ptr(), stride, draft, draft_stride, self.vocab, bool(distinct), n, self.n_requests,
                                     cu_new.data_ptr(), tokens.data_ptr(), parents, uniform.data_ptr(), slots, ctx_len,
                                     accepted.data_ptr(), rows.data_ptr(), kept, ctx_out, next_tokens.data_ptr(), self._status,
                                     _stream_of(stream, dev))
        B.check("skv_tree_verify", rc)

    def verify(self, probs, tokens, cu_new, uniform, parents=None, draft_probs=None, distinct: bool = False, slots=None, ctx_len=None,
               stream=None):
        """verify_into new tensors, waited for and checked: (accepted, rows, next_tokens), and kept with
        slots, and ctx_out with ctx_len. rows and kept are -1 outside every request."""
        accepted, nxt = torch.empty((2, self.n_requests), dtype=_I32, device=tokens.device).unbind()
        rows = torch.full_like(tokens, -1)
        kept = None if slots is None else torch.full_like(slots, -1)
        ctx_out = None if ctx_len is None else torch.empty_like(ctx_len)
        _after_current(stream)
        self.verify_into(probs, tokens, cu_new, uniform, accepted, rows, nxt, parents, draft_probs, distinct, slots, kept, ctx_len, ctx_out,
                         stream)
        self.check_status("skv_tree_verify", stream)
        return tuple(t for t in (accepted, rows, nxt, kept, ctx_out) if t is not None)
