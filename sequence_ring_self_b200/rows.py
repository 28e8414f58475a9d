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

import torch
from torch.autograd.function import once_differentiable

from . import rsa

MAX_K = 1024  # RSA_DISTILL_MAX_K

_INDEX = {torch.int64: 1, torch.int32: 0}


def _call(name, device, stream, tensors, body):
    """Runs ``body(lib, stream handle)`` with the tensors' device current and, where `stream` is
    not the current one, with its allocations made for `stream`. `body` returns the status code
    and the result."""
    lib = rsa.load_library()
    if device.index == torch.cuda.current_device() and stream is None:
        rc, out = body(lib, torch.cuda.current_stream(device).cuda_stream)
    else:
        s = stream if stream is not None else torch.cuda.current_stream(device)
        if s.device != device:
            raise ValueError(f"stream on {s.device}, expected {device} (the tensors' device)")
        other = s != torch.cuda.current_stream(device)
        with torch.cuda.device(device), torch.cuda.stream(s):
            rc, out = body(lib, s.cuda_stream)
        if other:
            for t in tensors:
                if t is not None:
                    t.record_stream(s)
    if rc != rsa.RSA_OK:
        raise rsa.RSAError(rc, name)
    return out


def _on_gpu(*named):
    """Tensors of one call live on one CUDA device; returns it."""
    device = named[0][1].device
    for name, t in named:
        if t is not None:
            if not t.is_cuda:
                raise ValueError(f"{name} must be on a CUDA device")
            if t.device != device:
                raise ValueError(f"{name} is on {t.device}, expected {device}")
    return device


def _shaped(name, t, shape, dtype):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _given_workspace(workspace, device):
    if not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {device}")
    return workspace


def _nbytes(t):
    return t.numel() * t.element_size()


def _int32(**sizes):
    """Sizes that the library takes as 32-bit numbers."""
    for name, n in sizes.items():
        if not 0 <= n <= 0x7fffffff:
            raise ValueError(f"{name} = {n} is outside [0, 2^31)")


def _addr(t):
    return None if t is None else t.data_ptr()


# ----------------------------------------------------------------- norm and rotation


def _qk_checked(q, k, wq, wk, freq, positions, rest, outputs):
    """Checks what both passes share; `rest` and `outputs` are (name, tensor or None, like q)."""
    rsa._dtype_code(q.dtype)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("queries and keys must be [B, heads, L, d]")
    B, Hq, L, d = q.shape
    if k.dtype != q.dtype:
        raise TypeError(f"keys must be {q.dtype}, got {k.dtype}")
    if k.shape[0] != B or k.shape[2:] != q.shape[2:]:
        raise ValueError("queries and keys must agree in B, L and d")
    _int32(B=B, Hq=Hq, Hk=k.shape[1], L=L, d=d)
    device = _on_gpu(("q", q), ("k", k), ("wq", wq), ("wk", wk), ("freq", freq),
                     ("positions", positions), *((n, t) for n, t, _ in rest + outputs))
    for name, t, like_q in rest + outputs:
        if t is not None:
            _shaped(name, t, q.shape if like_q else k.shape, q.dtype)
    for name, t in [("q", q), ("k", k)] + [(n, t) for n, t, _ in rest + outputs]:
        if t is not None and not _vector_rows(t):
            raise ValueError(f"{name}: rows must be contiguous and start on 16-byte boundaries")
    for name, w in (("wq", wq), ("wk", wk)):
        if w is not None:
            _shaped(name, w, (d,), torch.float32)
            if not w.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
    if freq is not None:
        if freq.dtype != torch.float32 or freq.dim() != 1 or not freq.is_contiguous():
            raise ValueError("freq must be contiguous fp32 [rot / 2]")
    pos_sb = 0
    if positions is not None:
        if positions.dtype not in _INDEX:
            raise TypeError("positions must be int64 or int32")
        if tuple(positions.shape) not in ((L,), (B, L)) or (L > 1 and positions.stride(-1) != 1):
            raise ValueError("positions must be [L] or [B, L] with contiguous rows")
        pos_sb = positions.stride(0) if positions.dim() == 2 and B > 1 else 0
    return device, pos_sb


def _vector_rows(t):
    """Rows the kernels can read: contiguous, 16-byte aligned."""
    if t.numel() == 0:
        return True
    vec = 16 // t.element_size()
    shape, stride = t.shape, t.stride()
    return (stride[-1] == 1 and t.data_ptr() % 16 == 0
            and all(n == 1 or s % vec == 0 for n, s in zip(shape[:-1], stride[:-1])))


def _strides(*ts):
    return (ctypes.c_longlong * (3 * len(ts)))(*(s for t in ts for s in t.stride()[:3]))


def _qk_tail(q, k, freq, positions, pos_sb, pos0, eps, interleaved):
    B, Hq, L, d = q.shape
    rot = 0 if freq is None else 2 * freq.numel()
    return (_addr(freq), _addr(positions), _INDEX[positions.dtype] if positions is not None else 0,
            pos_sb, int(pos0), B, Hq, k.shape[1], L, d, rot, int(bool(interleaved)), float(eps),
            rsa._dtype_code(q.dtype))


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
    device, pos_sb = _qk_checked(q, k, wq, wk, freq, positions, [],
                                 [("out_q", out_q, True), ("out_k", out_k, False)])

    def body(lib, s):
        oq = torch.empty(q.shape, dtype=q.dtype, device=device) if out_q is None else out_q
        ok = torch.empty(k.shape, dtype=k.dtype, device=device) if out_k is None else out_k
        rc = lib.rsa_qk_norm_rope(_addr(q), _addr(k), _addr(oq), _addr(ok), _strides(q, k, oq, ok),
                                  _addr(wq), _addr(wk),
                                  *_qk_tail(q, k, freq, positions, pos_sb, pos0, eps, interleaved), s)
        return rc, (oq, ok)

    return _call("rsa_qk_norm_rope", device, stream, (q, k, wq, wk, freq, positions, out_q, out_k),
                 body)


def qk_norm_rope_backward(q, k, dq_out, dk_out, wq, wk, freq, *, pos0: int = 0, positions=None,
                          eps: float = 1e-6, interleaved: bool = False, dq=None, dk=None,
                          need_weights: bool = True, workspace=None,
                          stream: torch.cuda.Stream | None = None):
    """Gradients of ``qk_norm_rope`` from its inputs q, k and its outputs' gradients. Returns
    (dq, dk, dwq, dwk): dq, dk like q, k (dq=dq_out or dq=q work in place), dwq, dwk fp32 [d]
    (None where the weight is None, or without need_weights). The workspace, if given, holds
    ``qk_norm_rope_workspace_size(d)`` bytes."""
    device, pos_sb = _qk_checked(q, k, wq, wk, freq, positions,
                                 [("dq_out", dq_out, True), ("dk_out", dk_out, False)],
                                 [("dq", dq, True), ("dk", dk, False)])

    def body(lib, s):
        d = q.shape[3]
        gq = torch.empty(q.shape, dtype=q.dtype, device=device) if dq is None else dq
        gk = torch.empty(k.shape, dtype=k.dtype, device=device) if dk is None else dk
        want = [w is not None and need_weights for w in (wq, wk)]
        dws, ws = [None, None], None
        if any(want):
            n = lib.rsa_qk_norm_rope_workspace_size(d)
            ws = (torch.empty(max(n, 256), dtype=torch.uint8, device=device) if workspace is None
                  else _given_workspace(workspace, device))
            dws = [torch.empty(d, dtype=torch.float32, device=device) if w else None for w in want]
        rc = lib.rsa_qk_norm_rope_backward(
            _addr(q), _addr(k), _addr(dq_out), _addr(dk_out), _addr(gq), _addr(gk),
            _strides(q, k, dq_out, dk_out, gq, gk), _addr(wq), _addr(wk), _addr(dws[0]),
            _addr(dws[1]), *_qk_tail(q, k, freq, positions, pos_sb, pos0, eps, interleaved),
            _addr(ws), 0 if ws is None else _nbytes(ws), s)
        return rc, (gq, gk, dws[0], dws[1])

    return _call("rsa_qk_norm_rope_backward", device, stream,
                 (q, k, dq_out, dk_out, wq, wk, freq, positions, dq, dk, workspace), body)


def qk_norm_rope_workspace_size(d: int) -> int:
    """Workspace bytes of ``qk_norm_rope_backward``."""
    n = rsa.load_library().rsa_qk_norm_rope_workspace_size(int(d))
    if n == 0:
        raise rsa.RSAError(rsa.RSA_ERR_UNSUPPORTED, "rsa_qk_norm_rope_workspace_size")
    return int(n)


class QKNormRope(torch.autograd.Function):
    """autograd wrapper: ``QKNormRope.apply(q, k, wq, wk, freq, positions, pos0, eps,
    interleaved)`` -> (q', k'). Gradients for q, k, wq and wk."""

    @staticmethod
    def forward(ctx, q, k, wq, wk, freq, positions=None, pos0=0, eps=1e-6, interleaved=False):
        if ctx.needs_input_grad[4]:
            raise ValueError("freq has no gradient here; detach it")
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
    if ids.dtype not in _INDEX:
        raise TypeError("ids must be int64 or int32")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    return _INDEX[ids.dtype]


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
    """``scale * table[ids]``: ids int64 or int32 of any shape, table [V, D] bf16 or fp32 (rows
    contiguous, any distance apart). An id outside [0, V) gives a row of zeros. Returns
    [*ids.shape, D] in the table's type."""
    i64 = _ids_checked(ids)
    dt = rsa._dtype_code(table.dtype)
    if table.dim() != 2:
        raise ValueError("table must be [V, D]")
    V, D = table.shape
    _int32(V=V, D=D, tokens=ids.numel())
    device = _on_gpu(("table", table), ("ids", ids), ("out", out))
    shape = (*ids.shape, D)
    if out is not None:
        _shaped("out", out, shape, table.dtype)
    ld = _ld(table)

    def body(lib, s):
        o = torch.empty(shape, dtype=table.dtype, device=device) if out is None else out
        flat = o if o.dim() == 2 else _flat("out", o, D)
        rc = lib.rsa_embed(_addr(ids), i64, _addr(table), ld, _addr(flat), _ld(flat), ids.numel(),
                           V, D, float(scale), dt, s)
        return rc, o

    return _call("rsa_embed", device, stream, (ids, table, out), body)


def embed_backward(ids, dout, num_rows: int, scale: float = 1.0, *, dtable=None,
                   accumulate: bool = False, workspace=None,
                   stream: torch.cuda.Stream | None = None):
    """Gradient of ``embed``'s table [num_rows, D] from dout [*ids.shape, D]: the rows of dout
    summed by id in fp32, times scale. The order of the sums is fixed. dtable: where it goes,
    in dout's type or fp32; with accumulate it is added to, and rows without a token are left as
    they are. The workspace, if given, holds ``embed_workspace_size`` bytes."""
    i64 = _ids_checked(ids)
    dt = rsa._dtype_code(dout.dtype)
    if tuple(dout.shape[:-1]) != tuple(ids.shape) or dout.dim() < 1:
        raise ValueError("dout must be [*ids.shape, D]")
    if accumulate and dtable is None:
        raise ValueError("accumulate needs the table's gradient to add to")
    V, D = int(num_rows), dout.shape[-1]
    _int32(num_rows=V, D=D, tokens=ids.numel())
    device = _on_gpu(("dout", dout), ("ids", ids), ("dtable", dtable))
    if dtable is not None:
        _shaped("dtable", dtable, (V, D),
                torch.float32 if dtable.dtype == torch.float32 else dout.dtype)
    g = _flat("dout", dout, D)
    ld = _ld(g)

    def body(lib, s):
        dtab = torch.empty((V, D), dtype=dout.dtype, device=device) if dtable is None else dtable
        n = lib.rsa_embed_workspace_size(ids.numel(), V, D)
        ws = (torch.empty(max(n, 256), dtype=torch.uint8, device=device) if workspace is None
              else _given_workspace(workspace, device))
        rc = lib.rsa_embed_backward(_addr(ids), i64, _addr(g), ld, _addr(dtab), _ld(dtab),
                                    ids.numel(), V, D, float(scale), int(bool(accumulate)), dt,
                                    rsa._dtype_code(dtab.dtype), _addr(ws), _nbytes(ws), s)
        return rc, dtab

    return _call("rsa_embed_backward", device, stream, (ids, dout, dtable, workspace), body)


def embed_workspace_size(n: int, num_rows: int, D: int) -> int:
    """Workspace bytes of ``embed_backward`` for n tokens (0: none needed)."""
    _int32(n=n, num_rows=num_rows, D=D)
    return int(rsa.load_library().rsa_embed_workspace_size(int(n), int(num_rows), int(D)))


class Embedding(torch.autograd.Function):
    """autograd wrapper: ``Embedding.apply(ids, table, scale)`` -> rows."""

    @staticmethod
    def forward(ctx, ids, table, scale=1.0):
        ctx.save_for_backward(ids)
        ctx.scale, ctx.V = scale, table.shape[0]
        return embed(ids, table, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        (ids,) = ctx.saved_tensors
        return None, embed_backward(ids, dout.contiguous(), ctx.V, ctx.scale), None


# ----------------------------------------------------------------- distillation


def _distill_checked(logits, index, teacher, temperature, rest):
    dt, tdt = rsa._dtype_code(logits.dtype), rsa._dtype_code(teacher.dtype)
    if index.dtype not in _INDEX:
        raise TypeError("index must be int64 or int32")
    if logits.dim() < 2 or index.dim() != logits.dim() or index.shape[:-1] != logits.shape[:-1]:
        raise ValueError("logits [..., V] and index [..., K] must agree in their rows")
    if teacher.shape != index.shape:
        raise ValueError("teacher must have index's shape [..., K]")
    if not index.is_contiguous() or not teacher.is_contiguous():
        raise ValueError("index and teacher must be contiguous")
    device = _on_gpu(("logits", logits), ("index", index), ("teacher", teacher), *rest)
    V, K = logits.shape[-1], index.shape[-1]
    z = _flat("logits", logits, V)
    _int32(rows=z.shape[0], V=V, K=K)
    return device, z, (z.shape[0], V, K, float(temperature), dt), (_INDEX[index.dtype], tdt)


def _rows_of(name, t, shape):
    """fp32 values of the rows, as (tensor, stride 0 or 1): a tensor of the rows' shape, an
    expanded one, or a single value for all rows."""
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be fp32, got {t.dtype}")
    if t.dim() == 0 or all(n == 1 or s == 0 for n, s in zip(t.shape, t.stride())):
        if t.dim() and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {tuple(shape)} or be a single value")
        return 0
    _shaped(name, t, shape, torch.float32)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous or one value expanded")
    return 1


def distill(logits, index, teacher, temperature: float = 1.0, *, loss=None, stats=None,
            stream: torch.cuda.Stream | None = None):
    """Distillation loss of each row of the student's logits [..., V] against the teacher's K
    largest logits: index [..., K] (int64 or int32; outside [0, V): an empty slot) and teacher
    [..., K] (bf16 or fp32; -inf: an empty slot). With p = softmax(teacher / temperature) over the
    slots and q = softmax(logits / temperature): temperature^2 * sum p (ln p - ln q). A row of
    empty slots has loss 0. With K = 1 this is the cross entropy with index as the label.
    Returns (loss [...] fp32, stats [..., 2] fp32 = (max logit, ln sum exp((z - max) / T)))."""
    device, z, sizes, kinds = _distill_checked(logits, index, teacher, temperature,
                                               [("loss", loss), ("stats", stats)])
    shape = logits.shape[:-1]
    for name, t, sh in (("loss", loss, shape), ("stats", stats, (*shape, 2))):
        if t is not None:
            _shaped(name, t, sh, torch.float32)
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
    ld = _ld(z)

    def body(lib, s):
        lo = torch.empty(shape, dtype=torch.float32, device=device) if loss is None else loss
        sa = torch.empty((*shape, 2), dtype=torch.float32, device=device) if stats is None else stats
        rc = lib.rsa_distill(_addr(z), ld, _addr(index), kinds[0], _addr(teacher), kinds[1],
                             _addr(lo), _addr(sa), *sizes, s)
        return rc, (lo, sa)

    return _call("rsa_distill", device, stream, (logits, index, teacher, loss, stats), body)


def _dlogits(logits, z, dlogits, device):
    """The gradient's tensor and its [rows, V] view: the given one, or a new one."""
    if dlogits is None:
        dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=device)
    return dlogits, _flat("dlogits", dlogits, z.shape[1])


def distill_backward(logits, index, teacher, stats, dloss, temperature: float = 1.0, *,
                     dlogits=None, stream: torch.cuda.Stream | None = None):
    """Gradient of ``distill``'s logits, dloss * temperature * (q - p), from its stats. dloss:
    fp32, of the rows' shape, or a single value for all rows. dlogits=logits works in place."""
    device, z, sizes, kinds = _distill_checked(logits, index, teacher, temperature,
                                               [("stats", stats), ("dloss", dloss),
                                                ("dlogits", dlogits)])
    shape = logits.shape[:-1]
    _shaped("stats", stats, (*shape, 2), torch.float32)
    if not stats.is_contiguous():
        raise ValueError("stats must be contiguous")
    step = _rows_of("dloss", dloss, shape)
    if dlogits is not None:
        _shaped("dlogits", dlogits, logits.shape, logits.dtype)
    ld = _ld(z)

    def body(lib, s):
        out, flat = _dlogits(logits, z, dlogits, device)
        rc = lib.rsa_distill_backward(_addr(z), ld, _addr(index), kinds[0], _addr(teacher),
                                      kinds[1], _addr(stats), _addr(dloss), step, _addr(flat),
                                      _ld(flat), *sizes, s)
        return rc, out

    return _call("rsa_distill_backward", device, stream,
                 (logits, index, teacher, stats, dloss, dlogits), body)


def distill_step(logits, index, teacher, dloss, temperature: float = 1.0, *, loss=None,
                 dlogits=None, stream: torch.cuda.Stream | None = None):
    """``distill`` and ``distill_backward`` in one pass over the logits, for a training loop that
    knows the rows' weights dloss beforehand (a mean's 1 / rows). Returns (loss, dlogits);
    dlogits=logits replaces the logits."""
    device, z, sizes, kinds = _distill_checked(logits, index, teacher, temperature,
                                               [("dloss", dloss), ("loss", loss),
                                                ("dlogits", dlogits)])
    shape = logits.shape[:-1]
    step = _rows_of("dloss", dloss, shape)
    if loss is not None:
        _shaped("loss", loss, shape, torch.float32)
        if not loss.is_contiguous():
            raise ValueError("loss must be contiguous")
    if dlogits is not None:
        _shaped("dlogits", dlogits, logits.shape, logits.dtype)
    ld = _ld(z)

    def body(lib, s):
        lo = torch.empty(shape, dtype=torch.float32, device=device) if loss is None else loss
        out, flat = _dlogits(logits, z, dlogits, device)
        rc = lib.rsa_distill_step(_addr(z), ld, _addr(index), kinds[0], _addr(teacher), kinds[1],
                                  _addr(dloss), step, _addr(lo), _addr(flat), _ld(flat), *sizes, s)
        return rc, (lo, out)

    return _call("rsa_distill_step", device, stream,
                 (logits, index, teacher, dloss, loss, dlogits), body)


class Distill(torch.autograd.Function):
    """autograd wrapper: ``Distill.apply(logits, index, teacher, temperature)`` -> loss per row.
    Gradient for the logits alone."""

    @staticmethod
    def forward(ctx, logits, index, teacher, temperature=1.0):
        if ctx.needs_input_grad[2]:
            raise ValueError("the teacher has no gradient here; detach it")
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
