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
    head.publish(bits=8)                         # or in 8: for whole probes at once

``LossHead`` is the same stage where only the log probabilities are wanted, and
their gradients: it holds no logits.

    loss = LossHead.of(synth.DIFFUREFILL_1B, global_, max_rows=16384)
    a = loss.score(x, residual, targets, sum_=s)
    loss.backward(s, targets, dlogprobs, dx, dembed, dweight)

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


class Loss(NamedTuple):
    logprobs: Optional[torch.Tensor]           # rows (None without targets)
    entropy: torch.Tensor                      # rows
    stats: torch.Tensor                        # rows x 2: largest logit, log of the sum


def _views(layout: synth.Layout, flat: torch.Tensor):
    """(final norm weight, tied embedding) in a flat fp32 parameter vector."""
    names = dict(layout.tensors)
    if "final_norm.weight" not in names or "embed" not in names:
        raise ValueError(f"{layout.name}: no RMS norm and tied embedding at its end")
    if (flat.dtype != torch.float32 or flat.numel() != layout.n_params or
            not flat.is_contiguous()):
        raise ValueError("flat: the layout's parameters in float32 required, contiguous")
    flat = flat.view(-1)
    width = names["final_norm.weight"]
    off = layout.offset_of("final_norm.weight")
    weight = flat[off:off + width]
    off = layout.offset_of("embed")
    return weight, flat[off:off + names["embed"]].view(names["embed"] // width, width)


class Head:
    """Final RMS norm and tied embedding of one candidate, for up to max_rows
    tokens a call.  `flat` is the candidate's fp32 parameter vector; the views
    follow it (a round that closes in place changes what the head says), the
    published 4-bit embedding does not until the next publish()."""

    def __init__(self, layout: synth.Layout, flat: torch.Tensor, max_rows: int,
                 eps: float = 1e-5):
        self.weight, self.embed = _views(layout, flat)
        if max_rows < 1:
            raise ValueError("max_rows must be at least 1")
        self.vocab, self.width = self.embed.shape
        self.eps, self.max_rows, dev = eps, max_rows, flat.device
        self._blocks = (self.width + 31) // 32
        self._packed = self._scales = self._codes = self._code_scales = None
        self._bits = 0                           # of the published form

        def new(*shape, dtype=torch.float32):
            return torch.empty(*shape, dtype=dtype, device=dev)

        self._h = new(max_rows, self.width)
        self._h8 = new(max_rows, self.width, dtype=torch.float8_e4m3fn)
        self._h8_scales = new(max_rows, self._blocks, dtype=torch.uint8)
        self._h8_scales128 = new(max_rows, (self.width + 127) // 128, dtype=torch.uint8)
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

    def publish(self, bits: int = 4) -> None:
        """Lays the embedding, as it is now, out in 4 bits (with a scale for each
        32 weights) or in 8 (for each 128 x 128): what answer() then goes by."""
        dev = self.embed.device
        if bits == 4:
            if self._packed is None:
                packed, scales = dh.dl_w4_bytes(self.vocab, self.width)
                self._packed = torch.empty(packed, dtype=torch.uint8, device=dev)
                self._scales = torch.empty(scales, dtype=torch.uint8, device=dev)
            dh.dl_w4_quantize(self.embed, self.vocab, self.width, self._packed, self._scales)
        elif bits == 8:
            if self._codes is None:
                self._codes = torch.empty(self.vocab, self.width, dtype=torch.float8_e4m3fn,
                                          device=dev)
                self._code_scales = torch.empty((self.vocab + 127) // 128,
                                                (self.width + 127) // 128, dtype=torch.uint8,
                                                device=dev)
            dh.dl_e4m3_quantize(self.embed, self.vocab, self.width, self._codes,
                                self._code_scales, dh.DL_SCALE_TILE128)
        else:
            raise ValueError(f"bits: 4 or 8 required, got {bits}")
        self._bits = bits

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
        in bf16 or fp32.  In 4 bits: norm in 8 bits with block scales, 4-bit
        product (DL_MAX_VECTORS tokens a pass), log probabilities.  In 8: norm in
        8 bits with a scale for each 128, one product for all tokens.  (With more
        bits in the stream: dl_rmsnorm to bf16 and dl_w4_matvec.)"""
        if self._bits == 0:
            raise RuntimeError("publish() first")
        rows = self._rows(x, top_k)
        four = self._bits == 4
        dh.dl_rmsnorm(x, rows, self.width, self.weight, self._h8, eps=self.eps,
                      residual=residual,
                      scales=self._h8_scales if four else self._h8_scales128,
                      scale_kind=dh.DL_SCALE_BLOCK32 if four else dh.DL_SCALE_BLOCK128)
        if four:
            for r in range(0, rows, dh.DL_MAX_VECTORS):
                n = min(dh.DL_MAX_VECTORS, rows - r)
                dh.dl_w4_matvec(self._packed, self._scales, self.vocab, self.width,
                                self._h8[r:r + n], n, self._logits[r:r + n],
                                x_scales=self._h8_scales[r:r + n],
                                x_scale_kind=dh.DL_SCALE_BLOCK32)
        else:
            dh.dl_e4m3_matmul(self._codes, self._code_scales, self.vocab, self.width, self._h8,
                              self._h8_scales128, rows, self._logits)
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


class LossHead:
    """Final RMS norm and embedding where the logits themselves are not wanted: a
    long probe's log probabilities, a training step's loss and gradients, for up to
    max_rows tokens a call.  weight: width fp32; embed: vocab x width in fp32 or bf16
    (products are then of bf16 numbers, the norm's output rounded to them), a view of
    the caller's parameters that the head follows."""

    def __init__(self, weight: torch.Tensor, embed: torch.Tensor, max_rows: int,
                 eps: float = 1e-5):
        if embed.dim() != 2 or embed.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("embed: a matrix in float32 or bfloat16 required")
        self.vocab, self.width = embed.shape
        if weight.shape != (self.width,) or weight.dtype != torch.float32:
            raise ValueError(f"weight: {self.width} elements in float32 required")
        if max_rows < 1:
            raise ValueError("max_rows must be at least 1")
        self.weight, self.embed, self.eps, self.max_rows = weight, embed, eps, max_rows
        dev = embed.device

        def new(*shape, dtype=torch.float32):
            return torch.empty(*shape, dtype=dtype, device=dev)

        self._h = new(max_rows, self.width, dtype=embed.dtype)
        self._dh = new(max_rows, self.width, dtype=embed.dtype)
        self._inv = new(max_rows)
        self._logprobs, self._entropy, self._stats = new(max_rows), new(max_rows), new(max_rows, 2)
        need = max(dh.dl_head_workspace_bytes(r, self.vocab, self.width, embed.dtype, True)
                   for r in range(1, max_rows + 1))
        self._ws = new(max(need, 256), dtype=torch.uint8)
        self._scored = None              # (rows, address of their sums) that the buffers are of
        need = dh.dl_rmsnorm_workspace_bytes(max_rows, self.width)      # (fewer rows need no more)
        self._norm_ws = new(max(need, 256), dtype=torch.uint8)

    @classmethod
    def of(cls, layout: synth.Layout, flat: torch.Tensor, max_rows: int, eps: float = 1e-5):
        """A candidate's, over its flat fp32 parameter vector."""
        return cls(*_views(layout, flat), max_rows, eps)

    def _rows(self, x: torch.Tensor, name: str) -> int:
        if x.dim() != 2 or x.shape[1] != self.width or x.shape[0] > self.max_rows:
            raise ValueError(f"{name}: at most {self.max_rows} x {self.width} required, got "
                             f"{tuple(x.shape)}")
        return x.shape[0]

    def score(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
              targets: Optional[torch.Tensor] = None,
              sum_: Optional[torch.Tensor] = None) -> Loss:
        """Log probabilities of the targets and entropies for the residual stream x (+
        residual), in fp32 or bf16; sum_, if given, receives x + residual (backward()
        wants it)."""
        rows = self._rows(x, "x")
        self._scored = None
        dh.dl_rmsnorm(x, rows, self.width, self.weight, self._h, eps=self.eps, residual=residual,
                      sum_=sum_, inv_rms=self._inv)
        logprobs = None if targets is None else self._logprobs[:rows]
        dh.dl_head_logprobs(self._h, self.embed, rows, self.vocab, self.width, targets, logprobs,
                            entropy=self._entropy, stats=self._stats, workspace=self._ws)
        left = x if residual is None else sum_
        self._scored = rows, None if left is None else left.data_ptr()
        return Loss(logprobs, self._entropy[:rows], self._stats[:rows])

    def backward(self, sum_: torch.Tensor, targets: torch.Tensor, dlogprobs: torch.Tensor,
                 dx: torch.Tensor, dembed: Optional[torch.Tensor] = None,
                 dweight: Optional[torch.Tensor] = None,
                 dentropy: Optional[torch.Tensor] = None,
                 dsum: Optional[torch.Tensor] = None) -> None:
        """The gradients of sum(dlogprobs * logprobs) + sum(dentropy * entropy) (and of
        what gave dsum), after the score() of these targets that left sum_ (or took it
        as x): dx in the stream, dembed, dweight, each written.  The stream has to be of
        the embedding's type.  The norm's output and the statistics are that score()'s, so
        no other may come between: sum_ has to be the last one's tensor.  (The host's order
        is what is checked: a graph that holds a score() brings its own backward().)"""
        rows = self._rows(sum_, "sum")
        if sum_.dtype != self.embed.dtype:
            raise ValueError(f"sum: {sum_.dtype}, and the embedding {self.embed.dtype}")
        if self._scored is None:
            raise RuntimeError("score() first")
        scored, at = self._scored
        if rows != scored or (rows > 0 and at is not None and sum_.data_ptr() != at):
            raise ValueError(f"sum: not what the last score(), of {scored} rows, left or took")
        dh.dl_head_logprobs_backward(self._h, self.embed, rows, self.vocab, self.width, targets,
                                     self._stats, dlogprobs, dx=self._dh, dembed=dembed,
                                     entropy=None if dentropy is None else self._entropy,
                                     dentropy=dentropy, workspace=self._ws)
        dh.dl_rmsnorm_backward(self._dh, sum_, rows, self.width, self.weight, self._inv, dx,
                               dsum=dsum, dweight=dweight, workspace=self._norm_ws)
