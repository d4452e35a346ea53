"""The output head of a merge's candidates.

A round leaves several flat parameter vectors that could be published: the
global, its EMA, the uniform average, averages of snapshots.  They are compared
by the cross-entropy of a probe's tokens (DiffuRefill-1B technical report,
section "The final stretch", Table 5; model card, "Training progress"), and the
published one answers with token confidences (model card, "Decoding
configuration").  ``Head`` is the last stage of both for one candidate: its
views into the flat buffer (final norm weight and tied embedding, by the
layout), its buffers, and the library's calls on torch's current stream.  The
layers below it, which give the residual stream, are the caller's.

    head = Head(synth.DIFFUREFILL_1B, global_, max_rows=2048)
    a = head.score(x, residual, targets)         # from the fp32 embedding
    head.publish()                               # lay the embedding out in 4 bits
    a = head.answer(x, residual, top_k=8)        # from the published one

Results are views of the head's buffers: the next call on it writes over them.
All buffers, workspaces included, are taken when the head is built and the
published embedding when it is first published; they stay where they are, so
calls may be captured into a graph.  Calls on one head go in one stream's order
(one head for each stream otherwise, and for graphs that may run at once), and a
head outlives the work that uses it.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import dlhead as dh
from . import dlmerge as dl
from . import synth


class Answer(NamedTuple):
    logits: torch.Tensor                       # rows x vocab, fp32
    logprobs: Optional[torch.Tensor]           # rows (None without targets)
    entropy: torch.Tensor                      # rows
    stats: torch.Tensor                        # rows x 2: largest logit, log of the sum
    top_ids: Optional[torch.Tensor]            # rows x top_k
    top_logprobs: Optional[torch.Tensor]       # rows x top_k


class Head:
    """Final RMS norm and tied embedding of one candidate, for up to max_rows
    tokens a call.  `flat` is the candidate's fp32 parameter vector; the views
    follow it (a round that closes in place changes what the head says), the
    published 4-bit embedding does not until the next publish()."""

    def __init__(self, layout: synth.Layout, flat: torch.Tensor, max_rows: int,
                 eps: float = 1e-5):
        names = dict(layout.tensors)
        if "final_norm.weight" not in names or "embed" not in names:
            raise ValueError(f"{layout.name}: no RMS norm and tied embedding at its end")
        if (flat.dtype != torch.float32 or flat.numel() != layout.n_params or
                not flat.is_contiguous()):
            raise ValueError("flat: the layout's parameters in float32 required, contiguous")
        flat = flat.view(-1)
        if max_rows < 1:
            raise ValueError("max_rows must be at least 1")
        self.width = names["final_norm.weight"]
        self.vocab = names["embed"] // self.width
        off = layout.offset_of("final_norm.weight")
        self.weight = flat[off:off + self.width]
        off = layout.offset_of("embed")
        self.embed = flat[off:off + names["embed"]].view(self.vocab, self.width)
        self.eps, self.max_rows, dev = eps, max_rows, flat.device
        self._blocks = (self.width + 31) // 32
        self._packed = self._scales = None

        def new(*shape, dtype=torch.float32):
            return torch.empty(*shape, dtype=dtype, device=dev)

        self._h = new(max_rows, self.width)
        self._h8 = new(max_rows, self.width, dtype=torch.float8_e4m3fn)
        self._h8_scales = new(max_rows, self._blocks, dtype=torch.uint8)
        self._inv = new(max_rows)
        self._logits = new(max_rows, self.vocab)
        self._logprobs, self._entropy, self._stats = new(max_rows), new(max_rows), new(max_rows, 2)
        self._ids = new(max_rows * dh.DL_MAX_TOP, dtype=torch.int64)
        self._top = new(max_rows * dh.DL_MAX_TOP)
        need = max(dh.dl_logprobs_workspace_bytes(r, self.vocab,
                                                  min(dh.DL_MAX_TOP, self.vocab))
                   for r in range(1, min(max_rows, 512) + 1))
        self._ws = new(max(need, 256), dtype=torch.uint8)
        # (a graph that captured score() keeps this address, so no call may replace it)
        need = max(dl.dl_matmul_workspace_bytes(r, self.vocab, self.width)
                   for r in range(1, max_rows + 1))
        self._product_ws = new(max(need, 256), dtype=torch.uint8)

    def publish(self) -> None:
        """Lays the embedding, as it is now, out in 4 bits."""
        if self._packed is None:
            packed, scales = dh.dl_w4_bytes(self.vocab, self.width)
            dev = self.embed.device
            self._packed = torch.empty(packed, dtype=torch.uint8, device=dev)
            self._scales = torch.empty(scales, dtype=torch.uint8, device=dev)
        dh.dl_w4_quantize(self.embed, self.vocab, self.width, self._packed, self._scales)

    def _rows(self, x: torch.Tensor, top_k: int = 0) -> int:
        if not 0 <= top_k <= min(dh.DL_MAX_TOP, self.vocab):
            raise ValueError(f"top_k: 0 to {min(dh.DL_MAX_TOP, self.vocab)} required, got {top_k}")
        if x.dim() != 2 or x.shape[1] != self.width or x.shape[0] > self.max_rows:
            raise ValueError(f"x: at most {self.max_rows} x {self.width} required, got "
                             f"{tuple(x.shape)}")
        return x.shape[0]

    def answer(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
               targets: Optional[torch.Tensor] = None, top_k: int = 0) -> Answer:
        """The published head's answer for the residual stream x (+ residual),
        in bf16 or fp32: norm in 8 bits with block scales, 4-bit product
        (DL_MAX_VECTORS tokens a pass), log probabilities.  (With more bits in
        the stream: dl_rmsnorm to bf16 and dl_w4_matvec.)"""
        if self._packed is None:
            raise RuntimeError("publish() first")
        rows = self._rows(x, top_k)
        dh.dl_rmsnorm(x, rows, self.width, self.weight, self._h8, eps=self.eps,
                      residual=residual, scales=self._h8_scales,
                      scale_kind=dh.DL_SCALE_BLOCK32)
        for r in range(0, rows, dh.DL_MAX_VECTORS):
            n = min(dh.DL_MAX_VECTORS, rows - r)
            dh.dl_w4_matvec(self._packed, self._scales, self.vocab, self.width, self._h8[r:r + n],
                            n, self._logits[r:r + n], x_scales=self._h8_scales[r:r + n],
                            x_scale_kind=dh.DL_SCALE_BLOCK32)
        return self._read(rows, targets, top_k)

    def score(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
              targets: Optional[torch.Tensor] = None, top_k: int = 0,
              sum_: Optional[torch.Tensor] = None) -> Answer:
        """The same from the candidate's own fp32 embedding (dl_matmul_f32).
        sum_, if given, receives x + residual (backward() wants it)."""
        rows = self._rows(x, top_k)
        dh.dl_rmsnorm(x, rows, self.width, self.weight, self._h, eps=self.eps,
                      residual=residual, sum_=sum_, inv_rms=self._inv)
        if rows > 0:
            # The bytes it is told of decide how the product is cut: those of these rows, so
            # that max_rows does not change the bits.
            dl.dl_matmul_f32(dl.DL_NT, self._h, self.width, self.embed, self.width, rows,
                             self.vocab, self.width, self._logits, self.vocab,
                             workspace=self._product_ws,
                             workspace_bytes=dl.dl_matmul_workspace_bytes(rows, self.vocab,
                                                                          self.width))
        return self._read(rows, targets, top_k)

    def _read(self, rows: int, targets: Optional[torch.Tensor], top_k: int) -> Answer:
        ids = top = None
        if top_k > 0:
            ids = self._ids[:rows * top_k].view(rows, top_k)
            top = self._top[:rows * top_k].view(rows, top_k)
        logprobs = None if targets is None else self._logprobs[:rows]
        dh.dl_logprobs(self._logits, rows, self.vocab, targets, logprobs, self._entropy,
                       self._stats, top_k, ids, top, workspace=self._ws)
        return Answer(self._logits[:rows], logprobs, self._entropy[:rows], self._stats[:rows],
                      ids, top)

    def loss_gradient(self, answer: Answer, targets: torch.Tensor, dlogprobs: torch.Tensor,
                      dentropy: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The gradient in answer's logits of sum(dlogprobs * logprobs) +
        sum(dentropy * entropy), written over them."""
        rows = answer.logits.shape[0]
        dh.dl_logprobs_backward(answer.logits, rows, self.vocab, targets, answer.stats, dlogprobs,
                                answer.logits,
                                entropy=None if dentropy is None else answer.entropy,
                                dentropy=dentropy)
        return answer.logits

    def backward(self, dy: torch.Tensor, sum_: torch.Tensor, dx: torch.Tensor,
                 dweight: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> None:
        """The norm's gradients for the gradient dy of its output, after the
        score() that left sum_ (or took it as x).  dy = dlogits x embedding is
        the caller's product: for n rows, dl_matmul_f32(DL_TN,
        dlogits.t().contiguous(), n, embed, width, n, width, vocab, dy, width)."""
        rows = self._rows(sum_)
        dh.dl_rmsnorm_backward(dy, sum_, rows, self.width, self.weight, self._inv, dx,
                               dweight=dweight, workspace=workspace)
