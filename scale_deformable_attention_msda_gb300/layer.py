"""Multi-scale deformable attention layer: the projections around the operator.

The msda-triton course, ch. 1 ("The idea: attend to a few learned
locations" and "The equation, term by term"), describes the layer: a linear
layer on the query features predicts K sampling offsets per head and level,
another predicts the attention weights (softmax-normalised over levels and
points), the value is projected per head, and W_m projects the heads' output.
The deformops README ("Multi-scale deformable attention") gives the call
shape: layer(query, reference, value, spatial_shapes, level_start_index).

The four projections are ordinary dense matmuls (torch.nn.Linear, i.e.
cuBLAS); the sampling, the softmax over the L*K logits and their backward run
in libmsda's fused-softmax kernels. Offsets are in pixels of each level: the
sampling location of (q, m, l, k) is reference[q, l] + offset / (W_l, H_l).

A detector's encoder or decoder layer ends this sublayer in
norm(input + sublayer(input)). With norm=True the layer does so itself: the
residual is added on the way into libmsda's layer norm, forward and backward.
With dropout=p the sublayer's output goes through dropout first.

A decoder layer begins with attention of the queries among themselves:
MultiHeadAttention is that sublayer, in the same form.
"""
from __future__ import annotations

import copy
import math

import torch
from torch import nn

from . import binding


class LayerNorm(nn.Module):
    """Layer norm over the last dimension, of x + residual where a residual is given
    (libmsda's kernels; binding.layer_norm). return_sum: (normalised, x + residual), what a
    pre-norm stack passes on. weight and bias start at one and zero. Under autocast x and a
    residual of another type (a projection's 16-bit output beside a float32 stream) are both
    taken in the type that holds both."""

    def __init__(self, dim: int, eps: float = 1e-5, bias: bool = True):
        super().__init__()
        self.dim, self.eps = dim, eps
        self.weight = nn.Parameter(torch.ones(dim))
        self.bias = nn.Parameter(torch.zeros(dim)) if bias else None

    def forward(self, x, residual=None, return_sum: bool = False):
        weight, bias = self.weight, self.bias
        if residual is not None and residual.dtype != x.dtype and torch.is_autocast_enabled("cuda"):
            dtype = torch.promote_types(x.dtype, residual.dtype)
            x, residual = x.to(dtype), residual.to(dtype)
            weight, bias = weight.to(dtype), None if bias is None else bias.to(dtype)
        return binding.layer_norm(x, weight, bias, residual=residual, eps=self.eps,
                                  return_sum=return_sum)


class Dropout(nn.Module):
    """Dropout of libmsda's counter-based generator (binding.dropout), in training; of x, or
    of x on its way into residual + x. `state` holds the generator's seed, drawn
    from torch's, and the number of the next draw, and is advanced on the device at each call
    in training: a captured step draws anew each time it is replayed. A forward that is run
    again for its backward (activation checkpointing) has to draw what it drew first: there
    give the call a `counter` that `next` returned outside of what is run again. Without one
    the second run is refused. A copy of the module
    (copy.deepcopy, of which a decoder's layers are made) has a seed of its own; one that is
    pickled or loaded continues where the stored one was.

    `state` is stored and moved with the module but is not among its buffers, which
    DistributedDataParallel makes those of rank 0: ranks draw from seeds of their own, if
    torch's generators were seeded differently on them. Where they were not, or where all
    ranks loaded one state, call reseed with a seed of the rank's."""

    def __init__(self, p: float = 0.1):
        super().__init__()
        if not 0.0 <= p <= 1.0:
            raise ValueError("a dropout probability lies between 0 and 1")
        self.p = p
        self.state = self._new_state()

    @staticmethod
    def _new_state():
        seed = torch.randint(-2 ** 63, 2 ** 63 - 1, (), dtype=torch.int64)
        return torch.stack([seed, torch.zeros_like(seed)])

    @torch.no_grad()
    def reseed(self, seed=None):
        """Start a generator of `seed`, 64 bits, drawn from torch's unless given."""
        if seed is None:
            self.state.copy_(self._new_state())
        else:
            self.state.copy_(torch.tensor([(int(seed) + 2 ** 63) % 2 ** 64 - 2 ** 63, 0]))

    def _apply(self, fn, recurse=True):
        super()._apply(fn, recurse)
        self.state = fn(self.state)
        return self

    def _save_to_state_dict(self, destination, prefix, keep_vars):
        super()._save_to_state_dict(destination, prefix, keep_vars)
        destination[prefix + "state"] = self.state

    def _load_from_state_dict(self, state_dict, prefix, local_metadata, strict, missing_keys,
                              unexpected_keys, error_msgs):
        key = prefix + "state"
        super()._load_from_state_dict({k: v for k, v in state_dict.items() if k != key}, prefix, local_metadata,
                                      strict, missing_keys, unexpected_keys, error_msgs)
        given = state_dict.get(key)
        if given is None:
            if strict:
                missing_keys.append(key)
        elif given.shape != (2,) or given.dtype != torch.int64:
            error_msgs.append(f"{key} is {given.dtype} of shape {tuple(given.shape)}: two int64 are expected")
        elif local_metadata.get("assign_to_params_buffers", False):
            self.state = given
        else:
            with torch.no_grad():
                self.state.copy_(given)

    def __setstate__(self, state):
        super().__setstate__(state)
        if "state" in self._buffers:             # modules pickled while it was one
            self.state = self._buffers.pop("state")

    def __deepcopy__(self, memo):
        copied = self.__class__.__new__(self.__class__)
        memo[id(self)] = copied
        copied.__setstate__(copy.deepcopy(self.__dict__, memo))
        copied.reseed()
        return copied

    def extra_repr(self):
        return f"p={self.p}"

    def next(self):
        """The counter of the next draw, two int64 on the state's device, for calls that are to
        draw the same."""
        if torch._C._current_graph_task_id() != -1:          # autograd runs a backward pass on this thread
            raise RuntimeError("dropout in a forward that is run again for its backward would draw another mask: "
                               "give both runs one counter (Dropout.next)")
        return binding.dropout_next(self.state)

    def forward(self, x, residual=None, counter=None):
        if residual is not None and residual.dtype != x.dtype and torch.is_autocast_enabled("cuda"):
            dtype = torch.promote_types(x.dtype, residual.dtype)
            x, residual = x.to(dtype), residual.to(dtype)
        if not self.training or self.p == 0.0:
            return x if residual is None else residual + x
        return binding.dropout(x, self.p, self.next() if counter is None else counter, residual=residual)


class MultiHeadAttention(nn.Module):
    """Attention of a detector's decoder: query (B, Q, dim) over key and value (B, S, dim) ->
    (B, Q, dim), through projections of their own and binding.attention. key: the query unless
    given; value: the key unless given (a decoder adds the queries' positions to query and key
    and not to value). mask: bool, broadcasts to (B, num_heads, Q, S), true where a query may
    attend; a query with no key gets the output projection of zeros. kv_heads: key heads, each
    shared by num_heads / kv_heads query heads. dropout: of the output; counter: its draw's,
    where the layer's own next one will not do (see Dropout). norm=True: the result
    is LayerNorm(residual + output), residual the query unless given."""

    def __init__(self, dim: int = 256, num_heads: int = 8, kv_heads: int | None = None,
                 dropout: float = 0.0, norm: bool = False):
        super().__init__()
        kv_heads = num_heads if kv_heads is None else kv_heads
        if min(dim, num_heads, kv_heads) < 1 or dim % num_heads != 0 or num_heads % kv_heads != 0:
            raise ValueError("dim must be divisible by num_heads, num_heads by kv_heads")
        if dim // num_heads % 8 != 0 or dim // num_heads > 128:
            raise ValueError(f"{dim // num_heads} channels a head: multiples of 8 up to 128 are supported")
        self.dim, self.num_heads, self.kv_heads = dim, num_heads, kv_heads
        self.head_dim = dim // num_heads
        self.query_proj = nn.Linear(dim, dim)
        self.key_proj = nn.Linear(dim, kv_heads * self.head_dim)
        self.value_proj = nn.Linear(dim, kv_heads * self.head_dim)
        self.output_proj = nn.Linear(dim, dim)
        self.dropout = Dropout(dropout) if dropout > 0.0 else None
        self.norm = LayerNorm(dim) if norm else None
        self.reset_parameters()

    @torch.no_grad()
    def reset_parameters(self):
        for proj in (self.query_proj, self.key_proj, self.value_proj, self.output_proj):
            nn.init.xavier_uniform_(proj.weight)
            nn.init.zeros_(proj.bias)

    def forward(self, query, key=None, value=None, mask=None, residual=None, counter=None):
        if residual is not None and self.norm is None:
            raise ValueError("a residual is added by a layer made with norm=True")
        if counter is not None and self.dropout is None:
            raise ValueError("a counter is for the draws of a layer made with dropout")
        key = query if key is None else key
        value = key if value is None else value
        B, Q, _ = query.shape
        q = self.query_proj(query).view(B, Q, self.num_heads, self.head_dim)
        k = self.key_proj(key).view(B, key.shape[1], self.kv_heads, self.head_dim)
        v = self.value_proj(value).view(B, value.shape[1], self.kv_heads, self.head_dim)
        out = self.output_proj(binding.attention(q, k, v, mask=mask))
        if self.dropout is not None:
            out = self.dropout(out) if counter is None else self.dropout(out, counter=counter)
        if self.norm is None:
            return out
        return self.norm(out, residual=query if residual is None else residual)


class MultiScaleDeformableAttention(nn.Module):
    """query (B, Q, dim), reference (B, Q, L, 2) or (B, Q, 2) normalised (x, y),
    value (B, S, dim), spatial_shapes (L, 2) int64 (H, W), level_start_index
    (L,) int64 -> (B, Q, dim). dim = num_heads * head_dim. norm=True: the output
    is LayerNorm(residual + attention), residual (B, Q, dim) the query unless
    given (a query with its position added is not what the layer adds to).
    dropout: of the output projection's result, in training; counter: its draw's,
    where the layer's own next one will not do (see Dropout)."""

    def __init__(self, dim: int = 256, num_heads: int = 8, num_levels: int = 4,
                 num_points: int = 4, accum: int = binding.MSDA_ACC_FP32_BUFFER,
                 norm: bool = False, dropout: float = 0.0):
        super().__init__()
        if dim % num_heads != 0:
            raise ValueError("dim must be divisible by num_heads")
        self.dim, self.num_heads = dim, num_heads
        self.num_levels, self.num_points = num_levels, num_points
        self.head_dim = dim // num_heads
        self.accum = accum
        self.sampling_offsets = nn.Linear(dim, num_heads * num_levels * num_points * 2)
        self.attention_weights = nn.Linear(dim, num_heads * num_levels * num_points)
        self.value_proj = nn.Linear(dim, dim)
        self.output_proj = nn.Linear(dim, dim)
        self.output_dropout = Dropout(dropout) if dropout > 0.0 else None
        self.norm = LayerNorm(dim) if norm else None
        self.ends_in_norm = norm         # a subclass may have a norm of its own under that name
        self.reset_parameters()

    @torch.no_grad()
    def reset_parameters(self):
        # Offsets start on a ring of directions, one per head, growing with the
        # point index; logits start at zero (uniform weights).
        nn.init.zeros_(self.sampling_offsets.weight)
        theta = torch.arange(self.num_heads, dtype=torch.float32) * (2.0 * math.pi / self.num_heads)
        grid = torch.stack([theta.cos(), theta.sin()], -1)
        grid = grid / grid.abs().max(-1, keepdim=True)[0]
        grid = grid.view(self.num_heads, 1, 1, 2).repeat(1, self.num_levels, self.num_points, 1)
        grid = grid * torch.arange(1, self.num_points + 1, dtype=torch.float32).view(1, 1, -1, 1)
        self.sampling_offsets.bias.copy_(grid.reshape(-1))
        nn.init.zeros_(self.attention_weights.weight)
        nn.init.zeros_(self.attention_weights.bias)
        nn.init.xavier_uniform_(self.value_proj.weight)
        nn.init.zeros_(self.value_proj.bias)
        nn.init.xavier_uniform_(self.output_proj.weight)
        nn.init.zeros_(self.output_proj.bias)

    def forward(self, query, reference, value, spatial_shapes, level_start_index, residual=None,
                counter=None):
        norm = getattr(self, "norm", None)
        # layers pickled before the mark: those with a norm of this module's were made with it
        if not getattr(self, "ends_in_norm", isinstance(norm, LayerNorm)):
            norm = None
        if residual is not None and norm is None:
            raise ValueError("a residual is added by a layer made with norm=True")
        drop = getattr(self, "output_dropout", None)     # layers pickled before it have none
        if counter is not None and not isinstance(drop, Dropout):
            raise ValueError("a counter is for the draws of a layer made with dropout")
        B, Q, _ = query.shape
        S = value.shape[1]
        M, L, K, D = self.num_heads, self.num_levels, self.num_points, self.head_dim
        v = self.value_proj(value).view(B, S, M, D)
        off = self.sampling_offsets(query).view(B, Q, M, L, K, 2)
        logits = self.attention_weights(query).view(B, Q, M, L, K)
        wh = spatial_shapes.flip(-1).to(off.dtype)                      # (L, 2) = (W, H)
        if reference.dim() == 3:
            reference = reference[:, :, None, :].expand(B, Q, L, 2)
        loc = reference[:, :, None, :, None, :].to(off.dtype) + off / wh[None, None, None, :, None, :]
        out = binding.multi_scale_deformable_attention(v, spatial_shapes, level_start_index, loc,
                                                       logits, accum=self.accum, softmax=True)
        out = self.output_proj(out)
        if isinstance(drop, Dropout):
            out = drop(out, counter=counter)
        if norm is None:
            return out
        return norm(out, residual=query if residual is None else residual)
