"""Refusals of the row-local operators, without a GPU: the C entry points check their arguments
before anything is launched, and the binding checks tensors before it calls them."""
import ctypes
import math

import pytest
import torch

import rows_oracle as ro
from sequence_ring_self_b200 import build, rows, rsa

FAKE = 0x100000  # a 16-byte-aligned non-null pointer that is never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = rsa.RSA_ERR_INVALID_ARG, rsa.RSA_ERR_UNSUPPORTED, rsa.RSA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build.build()
    return rsa.load_library()


def far(i):
    return FAKE + (i << 24)


def strides_of(B, H, L, d):
    return [H * L * d, L * d, d]


def qk(lib, backward=False, B=2, Hq=4, Hk=2, L=8, d=64, rot=64, dt=rsa.RSA_BF16, eps=1e-6, w=FAKE,
       dw=FAKE, freq=FAKE, pos=None, pos_sb=0, ptrs=None, strides=None, ws=FAKE, ws_bytes=1 << 20):
    n = 6 if backward else 4
    p = [far(i) for i in range(n)]
    for i, v in (ptrs or {}).items():
        p[i] = v
    st = [x for i in range(n) for x in strides_of(B, Hk if i & 1 else Hq, L, d)]
    for i, v in (strides or {}).items():
        st[i] = v
    st = (ctypes.c_longlong * len(st))(*st)
    tail = (freq, pos, 1, pos_sb, 0, B, Hq, Hk, L, d, rot, 0, eps, dt)
    if backward:
        return lib.rsa_qk_norm_rope_backward(*p, st, w, w, dw, dw, *tail, ws, ws_bytes, None)
    return lib.rsa_qk_norm_rope(*p, st, w, w, *tail, None)


@pytest.mark.parametrize("backward", [False, True])
def test_qk_refusals(lib, backward):
    call = lambda **kw: qk(lib, backward, **kw)
    last = 5 if backward else 3
    for bad in (dict(B=-1), dict(L=-1), dict(Hq=0), dict(Hk=0), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=math.nan), dict(rot=-16), dict(rot=128), dict(freq=0), dict(freq=FAKE + 2),
                dict(pos=FAKE + 4), dict(pos_sb=-1, pos=FAKE), dict(w=FAKE + 1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(d=96, rot=0), dict(d=256, rot=0), dict(d=128, rot=8), dict(rot=24), dict(dt=7),
                dict(B=1 << 16, L=1 << 16)):
        assert call(**bad) == UNSUPPORTED, bad
    for i in range(last + 1):
        assert call(ptrs={i: 0}) == INVALID
        assert call(ptrs={i: far(i) + 8}) == INVALID
    assert call(strides={0: -64}) == INVALID                     # negative
    assert call(strides={2: 68}) == INVALID                      # rows off 16-byte boundaries
    assert call(strides={3 * last + 2: 32}) == INVALID           # written rows that overlap
    assert call(strides={3 * last: 0}) == INVALID                # a broadcast output
    assert call(strides={3 * last: 64}) == INVALID               # a batch inside another's rows
    assert call(ptrs={last: far(last - 1)}) == INVALID           # both outputs in one place
    assert call(ptrs={last: far(0)}) == INVALID                  # keys over the queries' input
    assert call(ptrs={last: far(1)}, strides={3 * last: 4096}) == INVALID  # in place, other layout
    if backward:
        assert call(dw=FAKE + 2) == INVALID
        assert call(ws=FAKE + 16) == INVALID and call(ws=0) == INVALID
        assert call(ws_bytes=lib.rsa_qk_norm_rope_workspace_size(64) - 1) == WORKSPACE
    assert lib.rsa_qk_norm_rope_workspace_size(96) == 0
    assert call(B=0, **(dict(dw=None) if backward else {})) == rsa.RSA_OK  # nothing to do
    assert qk(lib, backward, strides=None, ptrs={}, L=0, **(dict(dw=None) if backward else {})) == rsa.RSA_OK


def emb(lib, n=10, V=100, D=64, ids=far(0), table=far(1), out=far(2), ld=64, ldo=64, dt=rsa.RSA_BF16):
    return lib.rsa_embed(ids, 1, table, ld, out, ldo, n, V, D, 1.0, dt, None)


def embb(lib, n=10, V=100, D=64, ids=far(0), table=far(2), out=far(1), ld=64, ldo=64, dt=rsa.RSA_BF16,
         dt_table=None, ws=FAKE, ws_bytes=1 << 30, acc=0):
    return lib.rsa_embed_backward(ids, 1, out, ldo, table, ld, n, V, D, 1.0, acc, dt,
                                  dt if dt_table is None else dt_table, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [emb, embb])
def test_embed_refusals(lib, call):
    for bad in (dict(n=-1), dict(V=0), dict(V=-3), dict(D=-1), dict(ids=0), dict(table=0), dict(out=0),
                dict(ids=far(0) + 4), dict(table=far(1) + 1), dict(out=far(2) + 1), dict(ld=63),
                dict(table=far(3), out=far(3))):
        assert call(lib, **bad) == INVALID, bad
    for bad in (dict(V=0x7fffffff), dict(D=(1 << 20) + 1, ld=1 << 21, ldo=1 << 21),
                dict(n=1 << 30, D=1 << 20, ld=1 << 20, ldo=1 << 20), dict(dt=5)):
        assert call(lib, **bad) == UNSUPPORTED, bad
    assert call(lib, D=0) == rsa.RSA_OK
    assert lib.rsa_embed_workspace_size(0, 10, 8) == 0 == lib.rsa_embed_workspace_size(10, 0, 8)


def test_embed_backward_refusals(lib):
    assert emb(lib, ldo=63) == INVALID and emb(lib, n=0) == rsa.RSA_OK
    assert embb(lib, ldo=-1) == INVALID
    assert embb(lib, dt=rsa.RSA_F32, dt_table=rsa.RSA_BF16) == UNSUPPORTED
    assert embb(lib, ws=0) == INVALID and embb(lib, ws=FAKE + 16) == INVALID
    assert embb(lib, ws_bytes=lib.rsa_embed_workspace_size(10, 100, 64) - 1) == WORKSPACE
    assert embb(lib, n=0, acc=1) == rsa.RSA_OK


def dist(lib, kind, z=far(0), ld=100, index=far(1), teacher=far(2), tdt=rsa.RSA_F32, loss=far(3),
         stats=far(4), dloss=far(5), step=1, dz=far(6), ldd=100, n=4, V=100, K=8, tau=1.0, dt=rsa.RSA_BF16):
    head = (z, ld, index, 1, teacher, tdt)
    if kind == "forward":
        return lib.rsa_distill(*head, loss, stats, n, V, K, tau, dt, None)
    if kind == "backward":
        return lib.rsa_distill_backward(*head, stats, dloss, step, dz, ldd, n, V, K, tau, dt, None)
    return lib.rsa_distill_step(*head, dloss, step, loss, dz, ldd, n, V, K, tau, dt, None)


@pytest.mark.parametrize("kind", ["forward", "backward", "step"])
def test_distill_refusals(lib, kind):
    call = lambda **kw: dist(lib, kind, **kw)
    for bad in (dict(n=-1), dict(V=0), dict(K=0), dict(tau=0.0), dict(tau=-1.0), dict(tau=math.nan),
                dict(tau=math.inf), dict(tau=1e-19), dict(tau=1e19), dict(z=0), dict(z=far(0) + 1), dict(index=0), dict(index=far(1) + 4),
                dict(teacher=0), dict(teacher=far(2) + 2), dict(ld=-1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(K=1025), dict(V=0x7fffffff), dict(n=1 << 27), dict(dt=9), dict(tdt=9)):
        assert call(**bad) == UNSUPPORTED, bad
    if kind != "backward":
        assert call(loss=0) == INVALID and call(loss=far(3) + 2) == INVALID
    if kind != "step":
        assert call(stats=0) == INVALID and call(stats=far(4) + 4) == INVALID
    if kind != "forward":
        for bad in (dict(dloss=0), dict(step=2), dict(step=-1), dict(dz=0), dict(ldd=99),
                    dict(dz=far(0), ldd=128)):
            assert call(**bad) == INVALID, bad
    assert call(n=0) == rsa.RSA_OK


def test_binding_refuses_before_it_calls():
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    w, f = torch.ones(64), torch.ones(32)
    with pytest.raises(ValueError, match="CUDA"):
        rows.qk_norm_rope(x, x, w, w, f)
    with pytest.raises(TypeError):
        rows.qk_norm_rope(x.half(), x.half(), w, w, f)
    with pytest.raises(TypeError):
        rows.qk_norm_rope(x, x.float(), w, w, f)
    with pytest.raises(ValueError, match="agree"):
        rows.qk_norm_rope(x, x[:, :, :3], w, w, f)
    with pytest.raises(ValueError):
        rows.qk_norm_rope(x[0], x[0], w, w, f)
    ids, table = torch.zeros(3, dtype=torch.int64), torch.zeros(5, 8)
    with pytest.raises(ValueError, match="CUDA"):
        rows.embed(ids, table)
    with pytest.raises(TypeError):
        rows.embed(ids.to(torch.int16), table)
    with pytest.raises(TypeError):
        rows.embed(ids, table.half())
    with pytest.raises(ValueError):
        rows.embed(ids, table[0])
    with pytest.raises(ValueError, match="dout"):
        rows.embed_backward(ids, torch.zeros(4, 8), 5)
    with pytest.raises(ValueError, match="accumulate"):
        rows.embed_backward(ids, torch.zeros(3, 8), 5, accumulate=True)
    with pytest.raises(ValueError, match="size"):
        rows.embed_backward(ids, torch.zeros(3, 8), 1 << 31)
    z, i, t = torch.zeros(3, 9), torch.zeros(3, 2, dtype=torch.int64), torch.zeros(3, 2)
    with pytest.raises(ValueError, match="CUDA"):
        rows.distill(z, i, t)
    with pytest.raises(TypeError):
        rows.distill(z, i.float(), t)
    with pytest.raises(ValueError, match="rows"):
        rows.distill(z, i[:2], t[:2])
    with pytest.raises(ValueError, match="teacher"):
        rows.distill(z, i, t[:, :1])
    with pytest.raises(TypeError):
        rows.distill(z.double(), i, t)


def test_autograd_wrappers_copy_what_the_functions_refuse():
    """Strided ids, slots and rows pass the wrappers and are refused by the functions (here both end
    at the check for a GPU)."""
    ids, table = torch.zeros(2, 5, dtype=torch.int64)[:, :-1], torch.zeros(5, 8)
    z, i, t = torch.zeros(2, 5, 9)[:, :-1], torch.zeros(2, 5, 3, dtype=torch.int64)[:, 1:], torch.zeros(2, 5, 3)[:, 1:]
    with pytest.raises(ValueError, match="contiguous"):
        rows.embed(ids, table)
    with pytest.raises(ValueError, match="CUDA"):
        rows.Embedding.apply(ids, table)
    with pytest.raises(ValueError, match="contiguous"):
        rows.distill(z, i, t)
    with pytest.raises(ValueError, match="CUDA"):
        rows.Distill.apply(z, i, t)


def test_plain_forms_against_differentiation():
    """The plain gradients that the GPU is held against agree with differentiating the plain
    forward passes (fp64, so to about 1e-12)."""
    g = torch.Generator().manual_seed(0)
    ro.HALF.setdefault(torch.float64, 0.0)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    freq = torch.tensor([1.0, 0.3, 0.05, 0.01, 0.7, 0.2, 0.9, 0.11])
    pos = torch.tensor([[3, 100, 70000]])
    for inter in (False, True):
        x, w, dy = rnd(2, 3, 3, 32), rnd(32), rnd(2, 3, 3, 32)
        # differentiate a copy of the forward pass
        xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
        n = xg / torch.sqrt((xg * xg).mean(-1, keepdim=True) + 1e-6) * wg
        cos, sin = ro._angles(freq, pos)
        (ro._rotate(n, cos, sin, 16, inter) * dy).sum().backward()
        y, _ = ro.qk_norm_rope(x, w, freq, pos, 1e-6, inter)
        assert torch.allclose(y, ro._rotate(n, cos, sin, 16, inter).detach(), atol=1e-12)
        dx, _, dw, _ = ro.qk_norm_rope_backward(x, w, freq, pos, dy, 1e-6, inter)
        assert torch.allclose(dx, xg.grad, atol=1e-11) and torch.allclose(dw, wg.grad, atol=1e-11)
    z, index, teacher = rnd(5, 40) * 3, torch.randint(0, 40, (5, 6), generator=g), rnd(5, 6)
    index[0, 3:] = -1
    index[1] = 40
    index[2, 4] = index[2, 1]
    dloss = torch.rand(5, generator=g, dtype=torch.float64)
    zg = z.clone().requires_grad_()
    live = (index >= 0) & (index < 40)
    for r in range(5):
        if live[r].any():
            s = live[r]
            lp = torch.log_softmax(teacher[r, s] / 1.3, 0)
            lq = torch.log_softmax(zg[r] / 1.3, 0)[index[r, s]]
            (1.69 * (lp.exp() * (lp - lq)).sum() * dloss[r]).backward()
    dz, _ = ro.distill_backward(z, index, teacher, dloss, 1.3)
    assert torch.allclose(dz, zg.grad, atol=1e-11) and (dz[1] == 0).all()
