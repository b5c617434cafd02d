"""The ends of a language model's training step around its NVFP4 linear layers, as
torch modules: the token embedding, the output head with its loss, and gradient
clipping.  The recipe leaves them in BF16 ("Pretraining Large Language Models with
NVFP4", summary page, recipe paragraph); every step runs in the library's HIP
kernels, on the current stream.  There is no CPU path.

  x = ScaledEmbedding(vocab, hidden, scale)(ids)           [.., hidden] BF16
  ... NVFP4Linear layers, norms, attention ...
  loss = CrossEntropyHead(hidden, vocab)(x, targets)       mean over the targets
  loss.backward()
  norm = clip_grad_norm(model.parameters(), 1.0)

The head's loss and its gradients come from one call in the forward pass: the logits
are never stored in FP32 (16-bit values in a bounded workspace, during the call) and
never computed twice; backward multiplies the stored gradients by the incoming one,
which rounds them to BF16 once more unless it is a power of two.  Targets outside 0 .. vocab - 1 (padding, -100) are
left out.
"""
from __future__ import annotations

import math
from typing import Iterable, Optional, Union

import torch
from torch.autograd.function import once_differentiable

from . import (NVFP4_SUMSQ_WORDS, clip_grads, embed, embed_grad, grad_sumsq, linear_ce,
               linear_ce_grad, scale_grads)


class EmbeddingFunction(torch.autograd.Function):
    """scale * weight[ids]; ids of any shape (int32 or int64), weight [vocab][dim]
    bf16 or float32.  The gradient has the weight's type, each row an FP32 sum in
    token order (the same bits every time)."""

    @staticmethod
    def forward(ctx, ids: torch.Tensor, weight: torch.Tensor, scale: float,
                dtype: Optional[torch.dtype] = None):
        flat = ids.reshape(-1).contiguous()
        ctx.save_for_backward(flat)
        ctx.scale, ctx.vocab, ctx.dtype = scale, weight.shape[0], weight.dtype
        return embed(flat, weight, scale, dtype).view(*ids.shape, weight.shape[1])

    @staticmethod
    @once_differentiable
    def backward(ctx, dy: torch.Tensor):
        (flat,) = ctx.saved_tensors
        if not ctx.needs_input_grad[1]:
            return None, None, None, None
        dy = dy.reshape(-1, dy.shape[-1])
        if dy.stride(1) != 1 or dy.stride(0) < dy.shape[1]:
            dy = dy.contiguous()   # expanded or transposed gradients
        return None, embed_grad(flat, dy, ctx.vocab, ctx.scale, ctx.dtype), None, None


def _total(x: torch.Tensor) -> torch.Tensor:
    """The sum of a vector.  A torch sum over more than about 10^5 values is joined by
    several workgroups through a counter that a memset clears; a captured graph does not
    repeat that reliably (the mean of 300007 losses was 0 from the second replay on), so a
    long vector is summed in rows first."""
    while x.numel() > 32768:
        whole = x.numel() // 512 * 512
        x = torch.cat((x[:whole].view(-1, 512).sum(1), x[whole:]))
    return x.sum()


def _reduce(loss: torch.Tensor, targets: torch.Tensor, vocab: int,
            row_weight: Optional[torch.Tensor]) -> torch.Tensor:
    """The weighted sum, or the mean over the tokens that have a target."""
    live = (targets >= 0) & (targets < vocab)
    if row_weight is None:
        return _total(loss) / _total(live).clamp(min=1)
    term = loss * row_weight
    counts = live & (row_weight != 0)   # a weight of 0 masks a loss that is not finite too
    if row_weight.requires_grad and torch.is_grad_enabled():
        counts = counts | (live & (term == 0))   # a finite one is the derivative by its weight
    return _total(torch.where(counts, term, torch.zeros_like(term)))


class LinearCrossEntropyFunction(torch.autograd.Function):
    """The loss of the head z = x weight^T, FP32: the sum over tokens of
    row_weight * loss, or the mean over the tokens that have a target (row_weight
    None; 0 if none has).  x [T][dim], weight [vocab][dim], both bf16.  Differentiable
    by x, weight and row_weight."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                row_weight: Optional[torch.Tensor], piece_tokens: int):
        loss, _, dx, dw = linear_ce_grad(x, weight, targets, row_weight, piece_tokens)
        # a token's loss (0 without a target) is the derivative by its weight; what is not
        # asked for is not kept until the backward pass (dw is as large as the weight)
        need = ctx.needs_input_grad
        ctx.save_for_backward(dx if need[0] else None, dw if need[1] else None,
                              loss if need[3] else None)
        return _reduce(loss, targets, weight.shape[0], row_weight)

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss: torch.Tensor):
        dx, dw, loss = ctx.saved_tensors
        dloss = dloss.float().reshape(1).contiguous()
        scaled = iter(scale_grads([g for g in (dx, dw) if g is not None], dloss))
        return (None if dx is None else next(scaled), None if dw is None else next(scaled), None,
                None if loss is None else loss * dloss, None)


class TokenLossFunction(torch.autograd.Function):
    """The loss of each token, FP32 [T] (0 without a target).  Its gradient takes
    the products again, weighted by the incoming one."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                piece_tokens: int):
        ctx.save_for_backward(x, weight, targets)
        ctx.piece_tokens = piece_tokens
        return linear_ce(x, weight, targets)[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss: torch.Tensor):
        x, weight, targets = ctx.saved_tensors
        _, _, dx, dw = linear_ce_grad(x, weight, targets, dloss.float().contiguous(),
                                      ctx.piece_tokens)
        return dx, dw, None, None


def _operand(x: torch.Tensor) -> torch.Tensor:
    """A bf16 matrix as the products take it: rows that start on 16 bytes.  A piece of a flat
    buffer may start anywhere; it is copied then."""
    if x.dim() == 2 and x.shape[1] % 8 == 0 and (
            x.data_ptr() % 16 or (x.shape[0] > 1 and x.stride(0) % 8)):
        return x.clone(memory_format=torch.contiguous_format)
    return x


def linear_cross_entropy(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                         row_weight: Optional[torch.Tensor] = None, reduction: str = "mean",
                         piece_tokens: int = 0) -> torch.Tensor:
    """Softmax cross entropy of the logits x weight^T without the logits.
    x [.., dim] and weight [vocab][dim] bf16, targets [..] int32 or int64; targets
    outside 0 .. vocab - 1 do not count.  reduction "mean" (over the targets),
    "sum" (of row_weight * loss, row_weight [..] float32 or all 1) or "none" (each
    token's loss, shaped like targets).  piece_tokens bounds the workspace (0: 2
    bytes for each token and word, 4 GiB at most).  x and weight are copied in a call
    where their rows do not start on 16 bytes (a piece of a flat buffer)."""
    if reduction not in ("mean", "sum", "none"):
        raise ValueError(f"reduction {reduction!r} is none of mean, sum, none")
    if row_weight is not None and reduction != "sum":
        raise ValueError("row_weight goes with reduction 'sum'")
    if x.shape[:-1] != targets.shape:
        raise ValueError(f"x {tuple(x.shape)} and targets {tuple(targets.shape)} do not match")
    flat = targets.reshape(-1).contiguous()
    rows = _operand(x.reshape(-1, x.shape[-1]).contiguous())
    weight = _operand(weight)
    train = torch.is_grad_enabled() and (x.requires_grad or weight.requires_grad)
    if reduction == "none":
        if not train:
            return linear_ce(rows, weight, flat)[0].view(targets.shape)
        return TokenLossFunction.apply(rows, weight, flat, piece_tokens).view(targets.shape)
    if reduction == "sum" and row_weight is None:
        row_weight = torch.ones(flat.numel(), dtype=torch.float32, device=x.device)
    if row_weight is not None:
        row_weight = row_weight.reshape(-1).contiguous()
        if row_weight.numel() != flat.numel():
            raise ValueError("one row weight for each target")
    if not train:
        return _reduce(linear_ce(rows, weight, flat)[0], flat, weight.shape[0], row_weight)
    return LinearCrossEntropyFunction.apply(rows, weight, flat, row_weight, piece_tokens)


class ScaledEmbedding(torch.nn.Module):
    """Token embedding with a factor (1, or sqrt(dim) where the table is shared with
    the head)."""

    def __init__(self, vocab: int, dim: int, scale: float = 1.0, device=None,
                 dtype: torch.dtype = torch.bfloat16):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.empty(vocab, dim, dtype=dtype, device=device))
        torch.nn.init.normal_(self.weight, std=1.0 / math.sqrt(dim))
        self.scale = scale

    def forward(self, ids: torch.Tensor) -> torch.Tensor:
        return EmbeddingFunction.apply(ids, self.weight, self.scale, torch.bfloat16)


class CrossEntropyHead(torch.nn.Module):
    """Output head and loss.  weight: a bf16 parameter to share (a tied embedding)."""

    def __init__(self, dim: int, vocab: int, device=None,
                 weight: Optional[torch.nn.Parameter] = None):
        super().__init__()
        if weight is None:
            weight = torch.nn.Parameter(
                torch.empty(vocab, dim, dtype=torch.bfloat16, device=device))
            torch.nn.init.normal_(weight, std=1.0 / math.sqrt(dim))
        elif weight.shape != (vocab, dim):
            raise ValueError(f"weight must be [{vocab}][{dim}]")
        elif weight.dtype != torch.bfloat16:
            raise ValueError(f"weight must be bf16 to be shared with a head, not {weight.dtype}")
        self.weight = weight

    def forward(self, x: torch.Tensor, targets: torch.Tensor, **kw) -> torch.Tensor:
        return linear_cross_entropy(x, self.weight, targets, **kw)


def _in_memory_order(g: torch.Tensor) -> torch.Tensor:
    """The gradient with its dimensions in the order of memory: a transposed parameter's is
    contiguous so, and neither a norm nor a factor minds the order."""
    if g.is_contiguous():
        return g
    return g.permute(sorted(range(g.dim()), key=g.stride, reverse=True))


def clip_grad_norm(parameters: Union[torch.Tensor, Iterable[torch.Tensor]], max_norm: float,
                   group=None) -> torch.Tensor:
    """Clip the gradients of parameters (or of one) in place to a global 2-norm of max_norm;
    returns the norm (float32 [1], on the GPU, not waited for; 0 without gradients).  group: a process
    group over which the parameters are sharded; the squares of all its ranks
    count (one all-reduce of 4 KiB)."""
    if isinstance(parameters, torch.Tensor):   # iterating over it would give its rows
        parameters = (parameters,)
    grads = [_in_memory_order(p.grad) for p in parameters if p.grad is not None]
    partials = None
    if group is not None:
        # a rank without gradients takes part in the sum all the same
        partials = (grad_sumsq(grads) if grads else
                    torch.zeros(NVFP4_SUMSQ_WORDS, dtype=torch.float64, device="cuda"))
        torch.distributed.all_reduce(partials, group=group)
    if not grads:
        return (torch.zeros(1, device="cuda") if partials is None
                else partials.sum().sqrt().float().reshape(1))
    return clip_grads(grads, max_norm, partials=partials)
