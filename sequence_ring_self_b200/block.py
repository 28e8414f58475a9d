"""The Transformer block under sequence parallelism: linear layers on the rank's rows around
Ring Self-Attention.

"Sequence Parallelism: Making 4D Parallelism Possible" (review page, Abstract) splits the
whole block by the sequence: every device holds a chunk of the rows, its linear layers (the
query/key/value projection, the output projection and the two layers of the MLP) work on those
rows alone with the weights every device holds, and only self-attention exchanges data, around
the ring. On rank r with rows X_r [c, hidden] (B = 1: the block's rows are one sequence's):

    [Q; K; V] = X_r Wqkv^T + bqkv               written as [3H, c, d] for attention
    O_r       = RingSelfAttention(Q, K, V)       the ring (sequence_ring_self_b200.ring)
    Y_r       = O_r Wo^T + bo + X_r              O read from [H, c, d] as [c, H d]
    Z_r       = GELU(Y_r W1^T + b1) W2^T + b2 + Y_r

The linear layers run in the library's tensor-core kernel (rsa_linear); the head split of the
projection and the head merge of the attention output are part of its tensor maps, so no copy
is made between the layers. Layer normalisation is not part of the linear layers and is left
out; dropout is absent, as in the attention. With norm weights or rotary frequencies given, the
queries and keys pass through rows.qk_norm_rope between the projection and the attention, at
their positions in the whole sequence (rank r's chunk starts at r c).

``model_forward`` and ``model_loss`` put the blocks between the token embedding (rows.embed) and
the output projection with the distillation loss (rows.distill): a rank's share of evaluating a
model, in which again only the attention exchanges data.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import ring as ringmod
from . import rows, rsa


@dataclass
class BlockWeights:
    """Weights of one block, replicated on every rank: wqkv [3 H d, hidden], wo [hidden, H d],
    w1 [ffn, hidden], w2 [hidden, ffn] (bf16, out x in); biases fp32."""
    wqkv: torch.Tensor
    bqkv: torch.Tensor
    wo: torch.Tensor
    bo: torch.Tensor
    w1: torch.Tensor
    b1: torch.Tensor
    w2: torch.Tensor
    b2: torch.Tensor
    heads: int
    head_dim: int
    # norm of queries and keys (fp32 [d]) and rotary frequencies (fp32 [rot / 2]); all None: neither
    wq_norm: torch.Tensor | None = None
    wk_norm: torch.Tensor | None = None
    freq: torch.Tensor | None = None
    norm_eps: float = 1e-6
    interleaved: bool = False


@dataclass
class ModelWeights:
    """A model around the blocks: table [V, hidden] and head [Vp, hidden] (bf16; Vp >= vocab rows,
    a multiple of 64), the embedding's scale."""
    table: torch.Tensor
    blocks: list
    head: torch.Tensor
    vocab: int
    scale: float = 1.0


def gpu_linear(x, w, bias=None, residual=None, gelu=False, x_kin=None, y_kin=None):
    """The block's linear layer on the GPU (rsa_linear)."""
    return rsa.linear(x, w, bias, residual, gelu, x_kin=x_kin, y_kin=y_kin)


def gpu_qk_norm_rope(q, k, wts: BlockWeights, pos0: int):
    """The block's norm and rotation of queries and keys on the GPU (rsa_qk_norm_rope)."""
    return rows.qk_norm_rope(q, k, wts.wq_norm, wts.wk_norm, wts.freq, pos0=pos0,
                             eps=wts.norm_eps, interleaved=wts.interleaved)


def block_forward(x, wts: BlockWeights, causal: bool = False, ring=None, comp=None,
                  lin=gpu_linear, qk=gpu_qk_norm_rope):
    """One rank's block forward on its rows x [c, hidden]. Returns (Z [c, hidden], parts) with
    parts the intermediate tensors (qkv [3H, c, d], the attention state, Y, the MLP hidden)."""
    H, d = wts.heads, wts.head_dim
    qkv = lin(x, wts.wqkv, wts.bqkv, y_kin=d)                  # [3H, c, d]
    q, k, v = (qkv[i * H:(i + 1) * H].unsqueeze(0) for i in range(3))  # [1, H, c, d] views
    if wts.wq_norm is not None or wts.wk_norm is not None or wts.freq is not None:
        ring = ring or ringmod.DistRing()
        q, k = qk(q, k, wts, ring.rank * x.shape[0])
    st = ringmod.attention(q, k.contiguous(), v.contiguous(), causal, ring=ring, comp=comp)
    y = lin(st.o[0], wts.wo, wts.bo, x, x_kin=d)               # [c, hidden]
    h = lin(y, wts.w1, wts.b1, gelu=True)                       # [c, ffn]
    z = lin(h, wts.w2, wts.b2, y)                               # [c, hidden]
    return z, {"qkv": qkv, "attn": st, "y": y, "h": h}


def model_forward(ids, wts: ModelWeights, causal: bool = True, ring=None, comp=None,
                  lin=gpu_linear, qk=gpu_qk_norm_rope, embed=rows.embed):
    """One rank's logits [c, vocab] for its chunk of the tokens, ids [c] (ids outside the
    vocabulary are padding): embedding, blocks, output projection. A view of the projection's
    padded columns."""
    x = embed(ids, wts.table, wts.scale)
    for b in wts.blocks:
        x, _ = block_forward(x, b, causal, ring=ring, comp=comp, lin=lin, qk=qk)
    return lin(x, wts.head)[:, :wts.vocab]


def model_loss(ids, index, teacher, wts: ModelWeights, temperature: float = 1.0,
               causal: bool = True, ring=None, comp=None):
    """One rank's distillation loss per token [c] (fp32) against a teacher's top logits for the
    same tokens: index [c, K], teacher [c, K] (rows.distill). Their mean over a sequence is the
    sum over its ranks divided by its tokens."""
    z = model_forward(ids, wts, causal, ring=ring, comp=comp)
    return rows.distill(z, index, teacher, temperature)[0]
