"""Python binding of the row-local operators around Ring Self-Attention (``include/rsa_rows.h``).

Under sequence parallelism ("Sequence Parallelism: Making 4D Parallelism Possible", review page,
Abstract) every rank holds a chunk of the rows and only self-attention exchanges data. These
are the parts of a decoder's training step that work on a rank's rows alone, next to
``rsa.linear``:

* ``embed`` / ``embed_backward`` / ``Embedding``: the rows that enter the first block,
  ``scale * table[ids]``, and the gradient of the table by sorted tokens;
* ``qk_norm_rope`` / ``qk_norm_rope_backward`` / ``QKNormRope``: between the query/key/value
  projection and the attention, the RMS norm of every head's row and its rotation by the row's
  position (a rank's chunk starts at ``pos0 = rank * c``), one pass over queries and keys;
* ``distill`` / ``distill_backward`` / ``distill_step`` / ``Distill``: the loss against a
  teacher's top logits and its gradient.

Argument marshalling only, as in ``rsa``: the computation runs in the library's kernels, without
a fallback. With ``stream`` given, outputs and workspaces are allocated for that stream and the
inputs are kept until it has passed the call; ordering the stream after the inputs' producers
and its results before their readers is the caller's part, as everywhere in PyTorch. Workspaces
are allocated per call unless one is passed; calls that may overlap on the GPU (two streams, two
captured graphs) need one each. The functions can be captured into a CUDA graph; capture the
``*_backward`` functions rather than the autograd engine.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from . import rsa

MAX_K = 1024  # RSA_DISTILL_MAX_K

_INDEX = {torch.int64: 1, torch.int32: 0}
_DT = {torch.bfloat16: rsa.RSA_BF16, torch.float32: rsa.RSA_F32}
_S12, _S18 = ctypes.c_longlong * 12, ctypes.c_longlong * 18


def _call(name, device, stream, tensors, written, body):
    """Runs ``body(lib, stream handle)`` with the tensors' device current and, where `stream` is
    not the current one, with its allocations made for `stream`. `body` returns the status code
    and the result. The tensors given as outputs, `written`, count as modified in place, so that
    autograd does not take them for what it saved."""
    lib = rsa._lib or rsa.load_library()
    if stream is None and device.index == torch.cuda.current_device():
        # the current stream's handle, without building a Stream object around it
        rc, out = body(lib, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        here = torch.cuda.current_stream(device)
        s = stream if stream is not None else here
        if s.device != device:
            raise ValueError(f"stream on {s.device}, expected {device} (the tensors' device)")
        with torch.cuda.device(device), torch.cuda.stream(s):
            rc, out = body(lib, s.cuda_stream)
        if s != here:
            for t in tensors:
                if t is not None:
                    t.record_stream(s)
    if rc != rsa.RSA_OK:
        raise rsa.RSAError(rc, name)
    for t in written:
        if t is not None:
            increment_version(t)
    return out


def _on_gpu(*tensors):
    """Tensors of one call live on one CUDA device; returns it."""
    device = tensors[0].device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, got {device}")
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"tensor on {t.device}, expected {device} (the first tensor's device)")
    return device


def _shaped(name, t, shape, dtype):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _given_workspace(workspace, device):
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {device}")
    return workspace


@lru_cache(maxsize=None)
def _qk_workspace(d):
    return int(rsa.load_library().rsa_qk_norm_rope_workspace_size(d))


@lru_cache(maxsize=256)
def _embed_workspace(n, V, D):
    return int(rsa.load_library().rsa_embed_workspace_size(n, V, D))


def _nbytes(t):
    return t.numel() * t.element_size()


def _int32(*sizes):
    """Sizes that the library takes as 32-bit numbers."""
    if not 0 <= min(sizes) <= max(sizes) <= 0x7fffffff:
        raise ValueError(f"a size among {sizes} is outside [0, 2^31)")


def _dtype(t):
    dt = _DT.get(t.dtype)
    return rsa._dtype_code(t.dtype) if dt is None else dt  # which says what is wrong


def _addr(t):
    return None if t is None else t.data_ptr()


def _like(t):
    return torch.empty_like(t, memory_format=torch.contiguous_format)


# ----------------------------------------------------------------- norm and rotation


def _qk_checked(q, k, wq, wk, freq, positions, *same):
    """Checks what both passes share; `same` are the tensors shaped like q and k in turn, or None.
    Returns the device and, as the C call has them, the positions, the sizes and the type."""
    dt = _dtype(q)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("queries and keys must be [B, heads, L, d]")
    qs, ks = q.shape, k.shape
    B, Hq, L, d = qs
    if k.dtype != q.dtype:
        raise TypeError(f"keys must be {q.dtype}, got {k.dtype}")
    if ks[0] != B or ks[2] != L or ks[3] != d:
        raise ValueError("queries and keys must agree in B, L and d")
    _int32(B, Hq, ks[1], L, d)
    device = _on_gpu(q, k, wq, wk, freq, positions, *same)
    if d > 1 and (q.stride(3) != 1 or k.stride(3) != 1):
        raise ValueError("rows of d elements must be contiguous")
    for i, t in enumerate(same):
        if t is None:
            continue
        if t.shape != (ks if i & 1 else qs) or t.dtype != q.dtype:
            _shaped("a tensor like the " + ("keys" if i & 1 else "queries"), t, ks if i & 1 else qs, q.dtype)
        if t.stride(3) != 1 and d > 1:
            raise ValueError("rows of d elements must be contiguous")
    for w in (wq, wk):
        if w is not None and (w.dtype != torch.float32 or w.shape != (d,) or not w.is_contiguous()):
            _shaped("a norm's weight", w, (d,), torch.float32)
            raise ValueError("a norm's weight must be contiguous")
    rot = 0
    if freq is not None:
        if freq.dtype != torch.float32 or freq.dim() != 1 or not freq.is_contiguous():
            raise ValueError("freq must be contiguous fp32 [rot / 2]")
        rot = 2 * freq.numel()
    pos, pos64, pos_sb = None, 0, 0
    if positions is not None:
        pos64 = _INDEX.get(positions.dtype)
        if pos64 is None:
            raise TypeError("positions must be int64 or int32")
        two = positions.dim() == 2
        if positions.shape != ((B, L) if two else (L,)) or (L > 1 and positions.stride(-1) != 1):
            raise ValueError("positions must be [L] or [B, L] with contiguous rows")
        pos, pos_sb = positions.data_ptr(), positions.stride(0) if two and B > 1 else 0
    return device, (_addr(freq), pos, pos64, pos_sb), (B, Hq, ks[1], L, d, rot), dt


def qk_norm_rope(q, k, wq, wk, freq, *, pos0: int = 0, positions=None, eps: float = 1e-6,
                 interleaved: bool = False, out_q=None, out_k=None,
                 stream: torch.cuda.Stream | None = None):
    """RMS norm of every row of q [B, Hq, L, d] and k [B, Hk, L, d] over d, times wq / wk (fp32
    [d], None for 1), then rotation of the first 2 * len(freq) elements by position * freq, in
    pairs (i, i + len(freq)) or, with `interleaved`, (2i, 2i + 1). Positions are pos0 + row, or
    `positions` (int, [L] or [B, L]). freq None or empty: the norm alone.

    bf16 or fp32, d in {32, 64, 128}. Rows must be contiguous and 16-byte aligned, the other
    strides are free: views of the projection's output, or of the ring's key buffer as out_k.
    out_q=q, out_k=k work in place. Returns (q', k'), contiguous unless given."""
    device, pos, sizes, dt = _qk_checked(q, k, wq, wk, freq, positions, out_q, out_k)

    def body(lib, s):
        oq = _like(q) if out_q is None else out_q
        ok = _like(k) if out_k is None else out_k
        st = _S12(*(q.stride()[:3] + k.stride()[:3] + oq.stride()[:3] + ok.stride()[:3]))
        rc = lib.rsa_qk_norm_rope(q.data_ptr(), k.data_ptr(), oq.data_ptr(), ok.data_ptr(), st,
                                  _addr(wq), _addr(wk), *pos, int(pos0), *sizes,
                                  bool(interleaved), float(eps), dt, s)
        return rc, (oq, ok)

    return _call("rsa_qk_norm_rope", device, stream, (q, k, wq, wk, freq, positions, out_q, out_k),
                 (out_q, out_k), body)


def qk_norm_rope_backward(q, k, dq_out, dk_out, wq, wk, freq, *, pos0: int = 0, positions=None,
                          eps: float = 1e-6, interleaved: bool = False, dq=None, dk=None,
                          need_weights: bool = True, workspace=None,
                          stream: torch.cuda.Stream | None = None):
    """Gradients of ``qk_norm_rope`` from its inputs q, k and its outputs' gradients. Returns
    (dq, dk, dwq, dwk): dq, dk like q, k (dq=dq_out or dq=q work in place), dwq, dwk fp32 [d]
    (None where the weight is None, or without need_weights). The workspace, if given, holds
    ``qk_norm_rope_workspace_size(d)`` bytes."""
    device, pos, sizes, dt = _qk_checked(q, k, wq, wk, freq, positions, dq_out, dk_out, dq, dk)

    def body(lib, s):
        d = sizes[4]
        gq = _like(q) if dq is None else dq
        gk = _like(k) if dk is None else dk
        dwq = dwk = ws = None
        if need_weights and (wq is not None or wk is not None):
            ws = (torch.empty(max(_qk_workspace(d), 256), dtype=torch.uint8, device=device)
                  if workspace is None else _given_workspace(workspace, device))
            dwq = None if wq is None else torch.empty_like(wq)
            dwk = None if wk is None else torch.empty_like(wk)
        st = _S18(*(q.stride()[:3] + k.stride()[:3] + dq_out.stride()[:3] + dk_out.stride()[:3]
                    + gq.stride()[:3] + gk.stride()[:3]))
        rc = lib.rsa_qk_norm_rope_backward(
            q.data_ptr(), k.data_ptr(), dq_out.data_ptr(), dk_out.data_ptr(), gq.data_ptr(),
            gk.data_ptr(), st, _addr(wq), _addr(wk), _addr(dwq), _addr(dwk), *pos, int(pos0),
            *sizes, bool(interleaved), float(eps), dt, _addr(ws), 0 if ws is None else _nbytes(ws), s)
        return rc, (gq, gk, dwq, dwk)

    return _call("rsa_qk_norm_rope_backward", device, stream,
                 (q, k, dq_out, dk_out, wq, wk, freq, positions, dq, dk, workspace), (dq, dk), body)


def qk_norm_rope_workspace_size(d: int) -> int:
    """Workspace bytes of ``qk_norm_rope_backward``."""
    n = _qk_workspace(int(d))
    if n == 0:
        raise rsa.RSAError(rsa.RSA_ERR_UNSUPPORTED, "rsa_qk_norm_rope_workspace_size")
    return n


def _vector_rows(t):
    """Rows the kernels can read: contiguous, 16-byte aligned."""
    if t.numel() == 0:
        return True
    vec = 16 // t.element_size()
    return (t.stride(-1) == 1 and t.data_ptr() % 16 == 0
            and all(n == 1 or s % vec == 0 for n, s in zip(t.shape[:-1], t.stride()[:-1])))


class QKNormRope(torch.autograd.Function):
    """autograd wrapper: ``QKNormRope.apply(q, k, wq, wk, freq, positions, pos0, eps,
    interleaved)`` -> (q', k'). Gradients for q, k, wq and wk. Queries, keys and gradients whose rows
    are not contiguous and 16-byte aligned are copied."""

    @staticmethod
    def forward(ctx, q, k, wq, wk, freq, positions=None, pos0=0, eps=1e-6, interleaved=False):
        if ctx.needs_input_grad[4]:
            raise ValueError("freq has no gradient here; detach it")
        q, k = (t if t.dim() != 4 or _vector_rows(t) else t.contiguous() for t in (q, k))
        ctx.save_for_backward(q, k, wq, wk, freq, positions)
        ctx.rest = dict(pos0=pos0, eps=eps, interleaved=interleaved)
        return qk_norm_rope(q, k, wq, wk, freq, positions=positions, **ctx.rest)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, wq, wk, freq, positions = ctx.saved_tensors
        dq_out, dk_out = (t if _vector_rows(t) else t.contiguous() for t in (dq_out, dk_out))
        dq, dk, dwq, dwk = qk_norm_rope_backward(
            q, k, dq_out, dk_out, wq, wk, freq, positions=positions,
            need_weights=any(ctx.needs_input_grad[2:4]), **ctx.rest)
        return dq, dk, dwq, dwk, None, None, None, None, None


# ----------------------------------------------------------------- embedding


def _ids_checked(ids):
    i64 = _INDEX.get(ids.dtype)
    if i64 is None:
        raise TypeError("ids must be int64 or int32")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    return i64


def _ld(t):
    """Elements between the rows of [rows, D]; rows must be contiguous."""
    if t.shape[1] > 1 and t.numel() and t.stride(1) != 1:
        raise ValueError("rows must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _flat(name, t, D):
    """[..., D] as [rows, D] without a copy."""
    if t.dim() == 2:
        return t
    try:
        return t.view(-1, D) if D else t.new_empty((t.numel(), 0))
    except RuntimeError:
        raise ValueError(f"{name}: the leading dimensions must be viewable as one") from None


def embed(ids, table, scale: float = 1.0, *, out=None, stream: torch.cuda.Stream | None = None):
    """``scale * table[ids]``: ids int64 or int32 of any shape, contiguous, table [V, D] bf16 or fp32
    (rows contiguous, any distance apart). An id outside [0, V) gives a row of zeros. Returns
    [*ids.shape, D] in the table's type."""
    i64, dt, n = _ids_checked(ids), _dtype(table), ids.numel()
    if table.dim() != 2:
        raise ValueError("table must be [V, D]")
    V, D = table.shape
    _int32(V, D, n)
    device = _on_gpu(table, ids, out)
    shape = (*ids.shape, D)
    if out is not None:
        _shaped("out", out, shape, table.dtype)
    ld = _ld(table)

    def body(lib, s):
        o = table.new_empty(shape) if out is None else out
        ldo = D if out is None else _ld(_flat("out", o, D))
        rc = lib.rsa_embed(ids.data_ptr(), i64, table.data_ptr(), ld, o.data_ptr(), ldo, n, V, D,
                           float(scale), dt, s)
        return rc, o

    return _call("rsa_embed", device, stream, (ids, table, out), (out,), body)


def embed_backward(ids, dout, num_rows: int, scale: float = 1.0, *, dtable=None,
                   accumulate: bool = False, workspace=None,
                   stream: torch.cuda.Stream | None = None):
    """Gradient of ``embed``'s table [num_rows, D] from dout [*ids.shape, D]: the rows of dout
    summed by id in fp32, times scale. The order of the sums is fixed. dtable: where it goes,
    in dout's type or fp32; with accumulate it is added to, and rows without a token are left as
    they are. The workspace, if given, holds ``embed_workspace_size`` bytes."""
    i64, dt, n = _ids_checked(ids), _dtype(dout), ids.numel()
    if dout.dim() < 1 or dout.shape[:-1] != ids.shape:
        raise ValueError("dout must be [*ids.shape, D]")
    if accumulate and dtable is None:
        raise ValueError("accumulate needs the table's gradient to add to")
    V, D = int(num_rows), dout.shape[-1]
    _int32(V, D, n)
    device = _on_gpu(dout, ids, dtable)
    if dtable is not None:
        _shaped("dtable", dtable, (V, D),
                torch.float32 if dtable.dtype == torch.float32 else dout.dtype)
    g = _flat("dout", dout, D)
    ld = _ld(g)

    def body(lib, s):
        dtab = dout.new_empty((V, D)) if dtable is None else dtable
        ws = (torch.empty(max(_embed_workspace(n, V, D), 256), dtype=torch.uint8, device=device)
              if workspace is None else _given_workspace(workspace, device))
        rc = lib.rsa_embed_backward(ids.data_ptr(), i64, g.data_ptr(), ld, dtab.data_ptr(),
                                    D if dtable is None else _ld(dtab), n, V, D, float(scale),
                                    bool(accumulate), dt, _DT[dtab.dtype], ws.data_ptr(),
                                    _nbytes(ws), s)
        return rc, dtab

    return _call("rsa_embed_backward", device, stream, (ids, dout, dtable, workspace), (dtable,), body)


def embed_workspace_size(n: int, num_rows: int, D: int) -> int:
    """Workspace bytes of ``embed_backward`` for n tokens (0: none needed)."""
    _int32(int(n), int(num_rows), int(D))
    return _embed_workspace(int(n), int(num_rows), int(D))


class Embedding(torch.autograd.Function):
    """autograd wrapper: ``Embedding.apply(ids, table, scale)`` -> rows. ids may be strided (a copy
    is made)."""

    @staticmethod
    def forward(ctx, ids, table, scale=1.0):
        ids = ids.contiguous()
        ctx.save_for_backward(ids)
        ctx.scale, ctx.V = scale, table.shape[0]
        return embed(ids, table, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        (ids,) = ctx.saved_tensors
        return None, embed_backward(ids, dout.contiguous(), ctx.V, ctx.scale), None


# ----------------------------------------------------------------- distillation


def _distill_checked(logits, index, teacher, temperature, *more):
    dt, tdt, i64 = _dtype(logits), _dtype(teacher), _INDEX.get(index.dtype)
    if i64 is None:
        raise TypeError("index must be int64 or int32")
    shape = logits.shape
    if len(shape) < 2 or index.dim() != len(shape) or index.shape[:-1] != shape[:-1]:
        raise ValueError("logits [..., V] and index [..., K] must agree in their rows")
    if teacher.shape != index.shape:
        raise ValueError("teacher must have index's shape [..., K]")
    if not index.is_contiguous() or not teacher.is_contiguous():
        raise ValueError("index and teacher must be contiguous")
    device = _on_gpu(logits, index, teacher, *more)
    V, K = shape[-1], index.shape[-1]
    z = _flat("logits", logits, V)
    n = z.shape[0]
    _int32(n, V, K)
    head = (z.data_ptr(), _ld(z), index.data_ptr(), i64, teacher.data_ptr(), tdt)
    return device, shape[:-1], head, (n, V, K, float(temperature), dt)


def _as_rows(t):
    """t, copied if its rows are not contiguous and the same distance apart."""
    try:
        if t.dim() > 1:
            _ld(_flat("t", t, t.shape[-1]))
        return t
    except ValueError:
        return t.contiguous()


def _rows_of(name, t, shape):
    """fp32 values of the rows: 1 (elements apart) for a contiguous tensor of the rows' shape, 0
    for an expanded one or a single value for all rows."""
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be fp32, got {t.dtype}")
    if t.dim() and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} or be a single value")
    if t.dim() and t.is_contiguous():
        return 1
    if any(n > 1 and s != 0 for n, s in zip(t.shape, t.stride())):
        raise ValueError(f"{name} must be contiguous or one value expanded")
    return 0


def _given_rows(name, t, shape):
    if t is not None:
        _shaped(name, t, shape, torch.float32)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def distill(logits, index, teacher, temperature: float = 1.0, *, loss=None, stats=None,
            stream: torch.cuda.Stream | None = None):
    """Distillation loss of each row of the student's logits [..., V] against the teacher's K
    largest logits: index [..., K] (int64 or int32; outside [0, V): an empty slot) and teacher
    [..., K] (bf16 or fp32; -inf: an empty slot), both contiguous; the rows of the logits are
    contiguous and the same distance apart. With p = softmax(teacher / temperature) over the
    slots and q = softmax(logits / temperature): temperature^2 * sum p (ln p - ln q). A row of
    empty slots has loss 0. With K = 1 this is the cross entropy with index as the label, times
    temperature^2. Returns (loss [...] fp32, stats [..., 2] fp32 = (max logit,
    ln sum exp((z - max) / temperature)))."""
    device, shape, head, sizes = _distill_checked(logits, index, teacher, temperature, loss, stats)
    _given_rows("loss", loss, shape)
    _given_rows("stats", stats, (*shape, 2))

    def body(lib, s):
        lo = torch.empty(shape, dtype=torch.float32, device=device) if loss is None else loss
        sa = lo.new_empty((*shape, 2)) if stats is None else stats
        return lib.rsa_distill(*head, lo.data_ptr(), sa.data_ptr(), *sizes, s), (lo, sa)

    return _call("rsa_distill", device, stream, (logits, index, teacher, loss, stats),
                 (loss, stats), body)


def _gradient(logits, dlogits):
    """The gradient's tensor, its address and the distance of its rows."""
    if dlogits is None:
        out = _like(logits)
        return out, out.data_ptr(), out.shape[-1]
    _shaped("dlogits", dlogits, logits.shape, logits.dtype)
    return dlogits, dlogits.data_ptr(), _ld(_flat("dlogits", dlogits, dlogits.shape[-1]))


def distill_backward(logits, index, teacher, stats, dloss, temperature: float = 1.0, *,
                     dlogits=None, stream: torch.cuda.Stream | None = None):
    """Gradient of ``distill``'s logits, dloss * temperature * (q - p), from its stats. dloss:
    fp32, of the rows' shape, or a single value for all rows. dlogits=logits works in place."""
    device, shape, head, sizes = _distill_checked(logits, index, teacher, temperature, stats,
                                                  dloss, dlogits)
    _given_rows("stats", stats, (*shape, 2))
    step = _rows_of("dloss", dloss, shape)

    def body(lib, s):
        out, at, ld = _gradient(logits, dlogits)
        return lib.rsa_distill_backward(*head, stats.data_ptr(), dloss.data_ptr(), step, at, ld,
                                        *sizes, s), out

    return _call("rsa_distill_backward", device, stream,
                 (logits, index, teacher, stats, dloss, dlogits), (dlogits,), body)


def distill_step(logits, index, teacher, dloss, temperature: float = 1.0, *, loss=None,
                 dlogits=None, stream: torch.cuda.Stream | None = None):
    """``distill`` and ``distill_backward`` in one pass over the logits, for a training loop that
    knows the rows' weights dloss beforehand (a mean's 1 / rows). Returns (loss, dlogits);
    dlogits=logits replaces the logits."""
    device, shape, head, sizes = _distill_checked(logits, index, teacher, temperature, dloss, loss,
                                                  dlogits)
    _given_rows("loss", loss, shape)
    step = _rows_of("dloss", dloss, shape)

    def body(lib, s):
        lo = torch.empty(shape, dtype=torch.float32, device=device) if loss is None else loss
        out, at, ld = _gradient(logits, dlogits)
        return lib.rsa_distill_step(*head, dloss.data_ptr(), step, lo.data_ptr(), at, ld, *sizes,
                                    s), (lo, out)

    return _call("rsa_distill_step", device, stream,
                 (logits, index, teacher, dloss, loss, dlogits), (loss, dlogits), body)


class Distill(torch.autograd.Function):
    """autograd wrapper: ``Distill.apply(logits, index, teacher, temperature)`` -> loss per row.
    Gradient for the logits alone. Strided index and teacher are copied, and so are logits whose
    rows are not the same distance apart, as ``logits[:, :-1]`` of several sequences: there, an
    index of -1 in the last position (a row without a slot has no loss and no gradient) saves the
    copy."""

    @staticmethod
    def forward(ctx, logits, index, teacher, temperature=1.0):
        if ctx.needs_input_grad[2]:
            raise ValueError("the teacher has no gradient here; detach it")
        logits, index, teacher = _as_rows(logits), index.contiguous(), teacher.contiguous()
        loss, stats = distill(logits, index, teacher, temperature)
        ctx.save_for_backward(logits, index, teacher, stats)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        logits, index, teacher, stats = ctx.saved_tensors
        if not dloss.is_contiguous() and any(s != 0 for s in dloss.stride()):
            dloss = dloss.contiguous()
        return distill_backward(logits, index, teacher, stats, dloss, ctx.temperature), None, None, None
