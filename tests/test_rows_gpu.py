"""The row-local operators on the GPU against their plain fp64 forms (rows_oracle), at the sizes,
layouts and masks where they can go wrong; and a run of them together around the attention."""
import math

import pytest
import torch

import rows_oracle as ro
from sequence_ring_self_b200 import build, rows, rsa

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    build.build()
    rsa.load_library()
    torch.cuda.set_device(0)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dt=F32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dt).cuda()


def same(a, b):
    """Equal bit for bit, NaN included."""
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ----------------------------------------------------------------- norm and rotation


def qk_case(seed, B, Hq, Hk, L, d, dt, rot=None, weights=True, positions=None, layout="plain"):
    g = gen(seed)
    rot = d if rot is None else rot
    if layout == "projection":  # [B, Hq + 2 Hk, L, d], as rsa_linear writes it
        qkv = randn(g, B, Hq + 2 * Hk, L, d, dt=dt, scale=2.0)
        q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    elif layout == "rows":      # [B, L, heads, d]
        q = randn(g, B, L, Hq, d, dt=dt, scale=2.0).transpose(1, 2)
        k = randn(g, B, L, Hk, d, dt=dt, scale=2.0).transpose(1, 2)
    else:
        q, k = randn(g, B, Hq, L, d, dt=dt, scale=2.0), randn(g, B, Hk, L, d, dt=dt, scale=2.0)
    w = [1 + randn(g, d, scale=0.3), 1 + randn(g, d, scale=0.3)] if weights else [None, None]
    freq = None
    if rot:
        i = torch.arange(rot // 2, dtype=torch.float64)
        freq = torch.exp(-math.log(10000.0) * 2 * i / rot).float().cuda()
    pos = None
    if positions:
        it = torch.int64 if "64" in positions else torch.int32
        shape = (B, L) if "batch" in positions else (L,)
        pos = torch.randint(-5000, 1 << 22, shape, generator=g).to(it).cuda()
    dy = randn(g, B, Hq, L, d, dt=dt), randn(g, B, Hk, L, d, dt=dt)
    return q, k, w, freq, pos, dy


QK = [
    # B, Hq, Hk, L, d, dt, rot, interleaved, weights, positions, pos0, layout
    (1, 1, 1, 1, 64, BF16, None, False, True, None, 0, "plain"),
    (4, 16, 16, 1, 128, BF16, None, False, True, "batch64", 0, "projection"),
    (2, 3, 5, 37, 64, BF16, None, False, True, None, 12345, "rows"),
    (1, 12, 2, 513, 64, BF16, 32, False, True, "row32", 0, "projection"),
    (3, 5, 1, 130, 128, BF16, 64, True, True, "batch32", 0, "plain"),
    (1, 33, 7, 65, 32, BF16, None, True, False, None, 4000000, "rows"),
    (2, 2, 2, 300, 32, BF16, 16, False, True, None, 3, "plain"),
    (1, 4, 4, 1000, 128, F32, None, False, True, None, 7, "projection"),
    (3, 6, 2, 77, 64, F32, 32, True, True, "batch64", 0, "rows"),
    (2, 1, 3, 129, 32, F32, None, True, True, "row64", 0, "plain"),
    (1, 2, 2, 50, 128, F32, 96, False, False, None, 0, "plain"),
    (2, 3, 3, 40, 64, BF16, 0, False, True, None, 0, "plain"),
    (2, 16, 4, 4096, 64, BF16, None, False, True, None, 8192, "projection"),
]


@pytest.mark.parametrize("case", QK, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_qk_norm_rope_and_its_gradient(case):
    B, Hq, Hk, L, d, dt, rot, inter, weights, positions, pos0, layout = case
    q, k, w, freq, pos, dy = qk_case(1, B, Hq, Hk, L, d, dt, rot, weights, positions, layout)
    kw = dict(pos0=pos0, positions=pos, eps=1e-6, interleaved=inter)
    y = rows.qk_norm_rope(q, k, *w, freq, **kw)
    grads = rows.qk_norm_rope_backward(q, k, *dy, *w, freq, **kw)
    at = ro.positions_of(L, pos0, pos)
    for s, x in enumerate((q, k)):
        ref, bound = ro.qk_norm_rope(x, w[s], freq, at, 1e-6, inter)
        ro.check(y[s], ref, bound, f"y[{s}]")
        dx, dx_bound, dw, dw_bound = ro.qk_norm_rope_backward(x, w[s], freq, at, dy[s], 1e-6, inter)
        ro.check(grads[s], dx, dx_bound, f"dx[{s}]")
        if weights:
            ro.check(grads[2 + s], dw, dw_bound, f"dw[{s}]")
        else:
            assert grads[2 + s] is None


def test_qk_gradient_against_differences():
    """The gradient's product with a direction against central differences of the fp64 form: the
    differences are off by about h^2 times a third derivative, here far below 1e-6."""
    q, k, w, freq, pos, dy = qk_case(5, 2, 3, 2, 9, 32, F32, 16, True, "batch64")
    grads = rows.qk_norm_rope_backward(q, k, *dy, *w, freq, positions=pos, interleaved=True)
    g, h = gen(6), 1e-5
    at = ro.positions_of(9, 0, pos)
    for s, x in enumerate((q, k)):
        f = lambda x, wt: (ro.qk_norm_rope(x, wt, freq, at, 1e-6, True)[0] * ro.f64(dy[s])).sum()
        x64, w64 = ro.f64(x), ro.f64(w[s])
        # the oracle takes any type whose half step it knows; fp64 inputs stay fp64
        ro.HALF.setdefault(torch.float64, 0.0)
        for arg, got in ((0, grads[s]), (1, grads[2 + s])):
            v = torch.randn(got.shape, generator=g, dtype=torch.float64)
            up = f(x64 + h * v, w64) if arg == 0 else f(x64, w64 + h * v)
            down = f(x64 - h * v, w64) if arg == 0 else f(x64, w64 - h * v)
            slope = (up - down) / (2 * h)
            size = (ro.f64(got).abs() * v.abs()).sum()
            assert abs((ro.f64(got) * v).sum() - slope) <= 1e-5 * size


def test_qk_positions_at_the_end_of_the_range():
    """Positions near +-2^31: their angles, off by less than 1e-6 each way, stay within the bound."""
    q, k, w, freq, _, dy = qk_case(8, 1, 2, 2, 64, 64, F32)
    pos = torch.cat([torch.arange(32) + (1 << 31) - 32, torch.arange(32) - (1 << 31)]).cuda()
    at = ro.positions_of(64, 0, pos)
    y = rows.qk_norm_rope(q, k, *w, freq, positions=pos)[0]
    ref, bound = ro.qk_norm_rope(q, w[0], freq, at, 1e-6, False)
    ro.check(y, ref, bound, "y")
    # (pos0 reaches as far: its rows are the positions pos0 + row)
    y0 = rows.qk_norm_rope(q, k, *w, freq, pos0=(1 << 31) - 64)[0]
    y1 = rows.qk_norm_rope(q, k, *w, freq, positions=torch.arange(64, device="cuda") + (1 << 31) - 64)[0]
    assert same(y0, y1)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_qk_in_place_and_into_a_ring_buffer(dt):
    """In place gives the same bits; a rank's keys written into their chunk of the ring's full
    buffer leave the other chunks as they were."""
    B, H, c, d, P, r = 2, 3, 70, 64, 3, 1
    q, k, w, freq, pos, dy = qk_case(2, B, H, H, c, d, dt, layout="projection")
    y = rows.qk_norm_rope(q, k, *w, freq, pos0=r * c)
    full = torch.full((B, H, P * c, d), 7.0, dtype=dt, device="cuda")
    mine = full[:, :, r * c:(r + 1) * c]
    oq, ok = rows.qk_norm_rope(q, k, *w, freq, pos0=r * c, out_k=mine)
    assert ok is mine and same(oq, y[0]) and same(mine, y[1])
    assert (full[:, :, :r * c] == 7).all() and (full[:, :, (r + 1) * c:] == 7).all()
    grads = rows.qk_norm_rope_backward(q, k, *dy, *w, freq, pos0=r * c)
    dq, dk = dy[0].clone(), dy[1].clone()
    inplace = rows.qk_norm_rope_backward(q, k, dq, dk, *w, freq, pos0=r * c, dq=dq, dk=dk)
    assert inplace[0] is dq and all(same(a, b) for a, b in zip(inplace, grads))
    over_x = rows.qk_norm_rope_backward(q2 := q.clone(), k, *dy, *w, freq, pos0=r * c, dq=q2)
    assert all(same(a, b) for a, b in zip(over_x, grads))
    q3, k3 = q.clone(), k.clone()
    rows.qk_norm_rope(q3, k3, *w, freq, pos0=r * c, out_q=q3, out_k=k3)
    assert same(q3, y[0]) and same(k3, y[1])


def test_qk_rows_stand_alone():
    """A row of zeros gives zeros; a NaN or an infinity stays in its row."""
    q, k, w, freq, _, dy = qk_case(3, 1, 2, 2, 20, 64, BF16)
    y0 = rows.qk_norm_rope(q, k, *w, freq)[0]
    g0 = rows.qk_norm_rope_backward(q, k, *dy, *w, freq)[0]
    q = q.clone()
    q[0, 0, 3] = 0
    q[0, 1, 4, 5] = NAN
    q[0, 0, 6, 0] = INF
    y = rows.qk_norm_rope(q, k, *w, freq)[0]
    g = rows.qk_norm_rope_backward(q, k, *dy, *w, freq)[0]
    assert (y[0, 0, 3] == 0).all() and torch.isfinite(g[0, 0, 3]).all()
    assert torch.isnan(y[0, 1, 4]).all() and torch.isnan(y[0, 0, 6]).any()
    for t, t0 in ((y, y0), (g, g0)):
        keep = torch.ones(2, 20, dtype=torch.bool, device="cuda")
        keep[0, 3] = keep[1, 4] = keep[0, 6] = False
        assert same(t[0][keep], t0[0][keep])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_qk_rows_whose_squares_overflow(dt, inter):
    """Rows of finite numbers: where the sum of squares passes the largest fp32 number, zeros, and
    zero gradients that leave the weights' alone; where only the products with weights, factors or
    gradients could pass it, the formula's values."""
    q, k, w, freq, pos, dy = qk_case(9, 1, 3, 3, 40, 64, dt, positions="row64")
    w = [t.abs() + 1 for t in w]
    most = torch.finfo(dt).max
    gone = {2: 1e20, 5: most, 7: -most, 11: 3e19}  # row: its size
    for s, (x, g) in enumerate(zip((q, k), dy)):
        for l, size in gone.items():
            x[0, s, l] = size
        x[0, s, 13, ::3] = most      # (some of the row)
        x[0, 2, 17] *= 3e17          # 64 squares of at most 1e37 each
        x[0, 2, 18] *= 3e17
        x[0, 1, 23] *= 1e17
        g[0, 2, 18] *= 1e24          # and products of 1e42
        g[0, 1, 24] *= 1e30
    out = [(x[0, s, l]) for s, x in enumerate((q, k)) for l in (*gone, 13)]
    assert all(torch.isfinite(t).all() and torch.isinf((t.float() ** 2).sum()) for t in out)
    assert all(torch.isfinite((x[0, 2, 17:19].float() ** 2).sum(-1)).all() for x in (q, k))
    y = rows.qk_norm_rope(q, k, *w, freq, positions=pos, interleaved=inter)
    grads = rows.qk_norm_rope_backward(q, k, *dy, *w, freq, positions=pos, interleaved=inter)
    at = ro.positions_of(40, 0, pos)
    for s, x in enumerate((q, k)):
        keep = torch.ones(3, 40, dtype=torch.bool)
        keep[s, [*gone, 13]] = False
        x0, g0 = x.clone(), dy[s].clone()
        x0[0][~keep.cuda()], g0[0][~keep.cuda()] = 0, 0
        ref, bound = ro.qk_norm_rope(x0, w[s], freq, at, 1e-6, inter)
        ro.check(y[s], ref, bound, f"y[{s}]")
        dx, dx_bound, dw, dw_bound = ro.qk_norm_rope_backward(x0, w[s], freq, at, g0, 1e-6, inter)
        ro.check(grads[s], dx, dx_bound, f"dx[{s}]")
        ro.check(grads[2 + s], dw, dw_bound, f"dw[{s}]")
        assert (y[s][0][~keep.cuda()] == 0).all() and (grads[s][0][~keep.cuda()] == 0).all()


@pytest.mark.parametrize("eps", [1e-40, 1e-30, 1.0])
def test_qk_eps_of_any_size(eps):
    """A row of zeros beside ordinary ones: dx = eps^(-1/2) u, whose square root's square may pass
    the largest fp32 number."""
    eps = float(torch.tensor(eps))  # as the kernel has it
    q, k, w, freq, _, dy = qk_case(10, 1, 2, 1, 9, 64, F32)
    q[0, 1, 4] = 0
    y = rows.qk_norm_rope(q, k, *w, freq, eps=eps)[0]
    dx, _, dw, _ = rows.qk_norm_rope_backward(q, k, *dy, *w, freq, eps=eps)
    at = ro.positions_of(9, 0, None)
    ref, bound = ro.qk_norm_rope(q, w[0], freq, at, eps, False)
    ro.check(y, ref, bound, "y")
    ref, bound, dw_ref, dw_bound = ro.qk_norm_rope_backward(q, w[0], freq, at, dy[0], eps, False)
    ro.check(dx, ref, bound, "dx")
    ro.check(dw, dw_ref, dw_bound, "dw")


def test_qk_without_rows():
    q = torch.empty(2, 3, 0, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    yq, yk = rows.qk_norm_rope(q, q, w, w, None)
    assert yq.shape == q.shape and yk.shape == q.shape
    _, _, dwq, dwk = rows.qk_norm_rope_backward(q, q, q, q, w, w, None)
    assert (dwq == 0).all() and (dwk == 0).all()


def test_qk_broadcast_inputs_and_gradients():
    """Keys shared by a whole batch (stride 0) are read as such; autograd's expanded gradients
    are taken, and the gradient of the shared keys adds up over the batch."""
    B, Hq, Hk, L, d = 3, 4, 2, 11, 64
    q, k1, w, freq, _, _ = qk_case(4, B, Hq, Hk, L, d, F32)
    k1 = k1[:1].clone()
    y = rows.qk_norm_rope(q, k1.expand(B, -1, -1, -1), *w, freq)[1]
    one = rows.qk_norm_rope(q, k1.repeat(B, 1, 1, 1), *w, freq)[1]
    assert same(y, one)
    qg, kg = q.clone().requires_grad_(), k1.clone().requires_grad_()
    wg = [t.clone().requires_grad_() for t in w]
    yq, yk = rows.QKNormRope.apply(qg, kg.expand(B, -1, -1, -1), *wg, freq)
    (yq.sum() + 2 * yk.sum()).backward()
    at = ro.positions_of(L, 0, None)
    ones = torch.ones_like(q)
    dq, bq, dwq, bwq = ro.qk_norm_rope_backward(q, w[0], freq, at, ones, 1e-6, False)
    dk, bk, dwk, bwk = ro.qk_norm_rope_backward(k1.repeat(B, 1, 1, 1), w[1], freq, at,
                                                torch.full((B, Hk, L, d), 2.0), 1e-6, False)
    ro.check(qg.grad, dq, bq, "dq")
    ro.check(kg.grad, dk.sum(0, keepdim=True), bk.sum(0, keepdim=True)
             + 3 * 2.0 ** -24 * dk.abs().sum(0, keepdim=True), "dk")
    ro.check(wg[0].grad, dwq, bwq, "dwq")
    ro.check(wg[1].grad, dwk, bwk, "dwk")


def test_qk_backward_is_the_same_every_time():
    q, k, w, freq, _, dy = qk_case(7, 2, 16, 4, 2048, 128, BF16)
    a = rows.qk_norm_rope_backward(q, k, *dy, *w, freq)
    for _ in range(3):
        assert all(same(x, y) for x, y in zip(a, rows.qk_norm_rope_backward(q, k, *dy, *w, freq)))


# ----------------------------------------------------------------- embedding


@pytest.mark.parametrize("V,D,dt", [(1, 8, BF16), (100, 64, BF16), (33, 7, BF16), (1000, 1001, F32),
                                    (500, 768, BF16), (64, 4, F32), (70000, 33, BF16), (9, 2048, F32)])
@pytest.mark.parametrize("n", [1, 5, 130, 2049])
def test_embed(n, V, D, dt):
    g = gen(n * 7 + V)
    table = randn(g, V, D, dt=dt)
    ids = torch.randint(0, V, (n,), generator=g)
    if n > 4:
        ids[1], ids[3] = -1, V
        ids[4] = -(1 << 40)
    scale = 0.37
    for it in (torch.int64, torch.int32):
        i = ids.clamp(-(1 << 31), (1 << 31) - 1).to(it).cuda()
        ref, bound = ro.embed(i, table, scale)
        ro.check(rows.embed(i, table, scale), ref, bound, f"embed {it}")


def test_embed_layouts():
    """Rows apart, rows off 16-byte boundaries, ids of two dimensions; what lies between the rows
    is left alone."""
    g = gen(11)
    wide = randn(g, 50, 96, dt=BF16)
    ids = torch.randint(-1, 51, (3, 21), generator=g).cuda()
    for lo, D in ((0, 64), (8, 64), (1, 64), (5, 31)):
        table = wide[:, lo:lo + D]
        ref, bound = ro.embed(ids, table, 2.0)
        ro.check(rows.embed(ids, table, 2.0), ref, bound, f"table {lo}")
        for olo in (0, 3):
            buf = torch.full((63, 90), 5.0, dtype=BF16, device="cuda")
            out = buf[:, olo:olo + D]
            rows.embed(ids.view(-1), table, 2.0, out=out)
            ro.check(out, ref.view(63, D), bound.view(63, D), f"out {olo}")
            assert (buf[:, :olo] == 5).all() and (buf[:, olo + D:] == 5).all()
    assert rows.embed(ids[:0], wide).shape == (0, 21, 96)


def tokens(g, n, V, kind):
    if kind == "one":            # a single id
        return torch.full((n,), V // 2, dtype=torch.int64)
    if kind == "few":
        return torch.randint(0, min(V, 3), (n,), generator=g) * ((V - 1) // max(1, min(V, 3) - 1) if V > 1 else 1)
    if kind == "text":           # frequencies like 1 / (v + 10), some padding
        u = torch.rand(n, generator=g, dtype=torch.float64)
        ids = (10 * torch.exp(u * math.log((V + 10) / 10)) - 10).long().clamp(0, V - 1)
        ids[torch.rand(n, generator=g) < 0.05] = -1
        return ids
    return torch.randint(0, V, (n,), generator=g)


@pytest.mark.parametrize("n,V,D,kind", [
    (1, 1, 8, "even"), (1, 30000, 64, "even"), (7, 5, 33, "even"), (31, 100, 64, "few"),
    (33, 3, 256, "one"), (1021, 503, 101, "text"), (8192, 50, 64, "text"), (8193, 30000, 72, "text"),
    (20000, 70000, 40, "text"), (20000, 700, 2056, "few"), (5000, 1, 16, "one"),
    (40000, 2000, 128, "one"), (3000, 2100000, 8, "even"), (140000, 900, 8, "text"),
    (600, 40, 1, "text")])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_embed_backward(n, V, D, kind, dt):
    g = gen(n + V)
    ids = tokens(g, n, V, kind)
    dout = randn(g, n, D, dt=dt)
    for it in (torch.int64, torch.int32):
        i = ids.to(it).cuda()
        got = rows.embed_backward(i, dout, V, 1.7)
        assert got.dtype == dt
        ref, bound = ro.embed_backward(i, dout, V, 1.7, dt)
        ro.check(got, ref, bound, f"dtable {it}")
        assert same(got, rows.embed_backward(i, dout, V, 1.7))  # the same bits every time


@pytest.mark.parametrize("dt,table_dt", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("lo,D", [(0, 64), (8, 48), (3, 61), (1, 17)])
def test_embed_backward_into_a_given_table(dt, table_dt, lo, D):
    """Adding to a gradient, and writing one, inside a wider tensor: rows without a token keep
    their values when adding and get zeros when writing; columns next to it stay."""
    g = gen(D)
    n, V = 700, 300
    ids = tokens(g, n, V, "text")
    ids[ids == 17] = 18
    ids = ids.cuda()
    wide = randn(g, n, 80, dt=dt)
    dout = wide[:, lo:lo + D]
    for accumulate in (True, False):
        buf = randn(g, V, 96, dt=table_dt)
        before = buf.clone()
        dtable = buf[:, lo:lo + D]
        rows.embed_backward(ids, dout, V, 0.3, dtable=dtable, accumulate=accumulate)
        ref, bound = ro.embed_backward(ids, dout, V, 0.3, table_dt,
                                       before[:, lo:lo + D] if accumulate else None)
        untouched = torch.ones(V, dtype=torch.bool)
        untouched[ids.cpu()[ids.cpu() >= 0]] = False
        assert untouched[17]
        if accumulate:
            assert same(dtable[untouched.cuda()], before[:, lo:lo + D][untouched.cuda()])
        else:
            assert (dtable[untouched.cuda()] == 0).all()
        ro.check(dtable, ref, bound, f"accumulate {accumulate}")
        assert same(buf[:, :lo], before[:, :lo]) and same(buf[:, lo + D:], before[:, lo + D:])


def test_embed_backward_edges():
    """No tokens, only padding (whose gradients may hold anything), no columns."""
    z = torch.zeros(0, dtype=torch.int64, device="cuda")
    out = rows.embed_backward(z, torch.empty(0, 24, dtype=BF16, device="cuda"), 10)
    assert out.shape == (10, 24) and (out == 0).all()
    keep = torch.full((10, 24), 3.0, dtype=BF16, device="cuda")
    rows.embed_backward(z, torch.empty(0, 24, dtype=BF16, device="cuda"), 10, dtable=keep, accumulate=True)
    assert (keep == 3).all()
    ids = torch.tensor([-1, 10, -100, 1 << 40], device="cuda")
    bad = torch.full((4, 24), NAN, dtype=F32, device="cuda")
    assert (rows.embed_backward(ids, bad, 10) == 0).all()
    ids[1] = 4
    bad[1] = 1
    out = rows.embed_backward(ids, bad, 10, 2.0)
    assert (out[4] == 2).all() and (out[:4] == 0).all() and (out[5:] == 0).all()
    assert rows.embed_backward(ids, bad[:, :0], 10).shape == (10, 0)
    # one gradient row for all tokens (stride 0)
    one = torch.ones(1, 24, device="cuda")
    out = rows.embed_backward(torch.zeros(50, dtype=torch.int64, device="cuda"), one.expand(50, 24), 2)
    assert (out[0] == 50).all() and (out[1] == 0).all()


def test_autograd_takes_shifted_and_unaligned_inputs():
    """The wrappers on slices of a batch of sequences (tokens and logits without the last position,
    labels without the first) and on rows off 16-byte boundaries: the same bits, forward and
    backward, as on contiguous copies."""
    g = gen(22)
    B, L, V, K, d = 3, 14, 333, 5, 64

    def both_ways(fn, views, grads_of):
        out = []
        for copy in (False, True):
            base = [t.clone().requires_grad_(i in grads_of) for i, (t, _) in enumerate(views)]
            args = [v(b) for b, (_, v) in zip(base, views)]
            if copy:
                args = [a.contiguous() if a is not None else a for a in args]
            y = fn(*args)
            y = y if isinstance(y, tuple) else (y,)
            gy = [randn(gen(23 + i), *t.shape, dt=t.dtype) for i, t in enumerate(y)]
            torch.autograd.backward(y, gy)
            out.append([t.detach() for t in y] + [base[i].grad for i in grads_of])
        assert len(out[0]) == len(out[1]) and all(same(a, b) for a, b in zip(*out))

    ids = torch.randint(-1, 51, (B, L), generator=g).cuda()
    both_ways(lambda i, t: rows.Embedding.apply(i, t, 2.0),
              [(ids, lambda t: t[:, :-1]), (randn(g, 50, 24), lambda t: t)], (1,))
    z, index = randn(g, B, L, V), torch.randint(-1, V, (B, L, K), generator=g).cuda()
    for cut in (lambda t: t[:, :-1], lambda t: t.transpose(1, 2)[:, :, :-1].transpose(1, 2), lambda t: t[:1, :-1]):
        both_ways(lambda *a: rows.Distill.apply(*a, 2.0),
                  [(z, cut), (index, lambda t: t[:, 1:][:cut(z).shape[0]]),
                   (randn(g, B, L, K), lambda t: t[:, 1:][:cut(z).shape[0]])], (0,))
    both_ways(lambda *a: rows.Distill.apply(*a, 2.0),
              [(randn(g, V, L), lambda t: t.T), (index[0].clone(), lambda t: t), (randn(g, L, K), lambda t: t)], (0,))
    freq, w = torch.rand(32, generator=g).cuda(), randn(g, d)
    for dt in (BF16, F32):
        both_ways(lambda q, k, w: rows.QKNormRope.apply(q, k, w, None, freq, None, 5),
                  [(randn(g, B, 2, L, d + 1, dt=dt), lambda t: t[..., 1:]),
                   (randn(g, B, 2, L, d + 1, dt=dt), lambda t: t[..., :d]), (w, lambda t: t)], (0, 1, 2))
        both_ways(lambda q, k: rows.QKNormRope.apply(q, k, None, None, freq),
                  [(randn(g, B, 2, d, L, dt=dt), lambda t: t.transpose(2, 3)),
                   (randn(g, B, 2, L, d, dt=dt), lambda t: t)], (0, 1))


def test_outputs_written_in_place_are_known_to_autograd():
    """A tensor that an operator overwrites counts as modified: a backward pass that saved it refuses
    to run on the new contents."""
    z, index, teacher, dloss = distill_case(24, 6, 100, 4, F32)
    leaf = z.clone().requires_grad_()
    logits = leaf * 1
    loss = rows.Distill.apply(logits, index, teacher, 1.0)
    rows.distill_step(logits.detach(), index, teacher, dloss, dlogits=logits.detach())
    with pytest.raises(RuntimeError, match="inplace"):
        loss.sum().backward()
    q, k, w, freq, _, dy = qk_case(25, 1, 2, 2, 9, 64, F32)
    table, ids, dout = randn(gen(26), 10, 8), torch.arange(5, device="cuda"), randn(gen(27), 5, 8)
    out, dtable, lo, st = dout.clone(), table.clone(), dloss.clone(), torch.empty(6, 2, device="cuda")
    stats = rows.distill(z, index, teacher)[1]
    calls = [
        ((q, k), lambda: rows.qk_norm_rope(q, k, *w, freq, out_q=q, out_k=k)),
        ((dy[0], dy[1]), lambda: rows.qk_norm_rope_backward(q, k, *dy, *w, freq, dq=dy[0], dk=dy[1])),
        ((out,), lambda: rows.embed(ids, table, out=out)),
        ((dtable,), lambda: rows.embed_backward(ids, dout, 10, dtable=dtable, accumulate=True)),
        ((lo, st), lambda: rows.distill(z, index, teacher, loss=lo, stats=st)),
        ((z,), lambda: rows.distill_backward(z, index, teacher, stats, dloss, dlogits=z)),
        ((z, lo), lambda: rows.distill_step(z, index, teacher, dloss, dlogits=z, loss=lo))]
    read = [index, teacher, dloss, stats, ids, table, dout, *w, freq]
    before = [t._version for t in read]
    for written, call in calls:
        versions = [t._version for t in written]
        call()
        assert all(t._version > v for t, v in zip(written, versions))
    assert [t._version for t in read] == before


def test_embedding_autograd_and_differences():
    """The operator is linear in the table, so a difference is exact up to rounding."""
    g = gen(21)
    table = randn(g, 40, 24).requires_grad_()
    ids = torch.randint(-1, 41, (4, 9), generator=g).cuda()
    dout = randn(g, 4, 9, 24)
    y = rows.Embedding.apply(ids, table, 1.5)
    (y * dout).sum().backward()
    v = torch.randn(40, 24, generator=g, dtype=torch.float64)
    up, down = (ro.embed(ids, (ro.f64(table) + s * v).float(), 1.5)[0] for s in (0.5, -0.5))
    slope = ((up - down) * ro.f64(dout)).sum()
    size = (ro.f64(table.grad).abs() * v.abs()).sum()
    assert abs((ro.f64(table.grad) * v).sum() - slope) <= 1e-5 * size
    y.detach_()
    table.grad = None
    rows.Embedding.apply(ids, table, 1.0).sum().backward()  # an expanded gradient
    ref, bound = ro.embed_backward(ids, torch.ones(36, 24), 40, 1.0, F32)
    ro.check(table.grad, ref, bound, "expanded")


# ----------------------------------------------------------------- distillation


def distill_case(seed, n, V, K, dt, index_dt=torch.int64, teacher_dt=F32, pad=True):
    """Rows with all, some or no slots; slots out of range, with the teacher at -inf, and with the
    same index; logits in entries not in use at the type's lowest value or at -inf."""
    g = gen(seed)
    z = torch.randn(n, V, generator=g) * 3
    index = torch.randint(0, max(1, V - V // 8), (n, K), generator=g)
    teacher = torch.randn(n, K, generator=g) * 2
    z.scatter_add_(1, index, torch.full((n, K), 2.0))
    if pad:
        if V >= 16:
            z[:, V - V // 8:] = torch.finfo(dt).min
            z[::2, V - 1] = -INF
        for r in range(n):
            if r % 5 == 1:
                index[r, K // 2:] = -1
            elif r % 5 == 2:
                index[r] = torch.tensor([-1, V, -100])[r % 3]
                teacher[r] = NAN
            elif r % 5 == 3 and K > 1:
                teacher[r, ::2] = -INF
                index[r, 1::2] = index[r, 1]  # the same entry again and again
    return (z.to(dt).cuda(), index.to(index_dt).cuda(), teacher.to(teacher_dt).cuda(),
            torch.rand(n, generator=g).cuda())


DISTILL = [
    # n, V, K, dt, index, teacher, temperature
    (1, 1, 1, F32, torch.int64, F32, 1.0),
    (3, 2, 1, BF16, torch.int64, F32, 1.0),
    (11, 7, 3, BF16, torch.int32, BF16, 2.0),
    (6, 1000, 20, F32, torch.int64, F32, 0.5),
    (5, 1001, 1, BF16, torch.int64, BF16, 1.0),
    (7, 4099, 33, BF16, torch.int64, F32, 2.0),
    (2, 50001, 64, BF16, torch.int32, F32, 1.0),
    (1, 131072, 128, BF16, torch.int64, F32, 1.0),
    (6, 50001, 20, F32, torch.int64, F32, 1.0),
    (400, 1536, 8, BF16, torch.int64, F32, 1.0),
    (300, 8200, 700, F32, torch.int64, F32, 2.0),
    (4, 9000, 1024, BF16, torch.int64, BF16, 1.0),
    (640, 32768, 64, BF16, torch.int64, F32, 2.0),
]


@pytest.mark.parametrize("case", DISTILL, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_distill(case):
    n, V, K, dt, idt, tdt, tau = case
    z, index, teacher, dloss = distill_case(n + V, n, V, K, dt, idt, tdt)
    loss, stats = rows.distill(z, index, teacher, tau)
    ref, bound, sref, sbound = ro.distill(z, index, teacher, tau)
    ro.check(loss, ref, bound, "loss")
    ro.check(stats, sref, sbound, "stats")
    dref, dbound = ro.distill_backward(z, index, teacher, dloss, tau)
    ro.check(rows.distill_backward(z, index, teacher, stats, dloss, tau), dref, dbound, "dlogits")
    sl, sd = rows.distill_step(z, index, teacher, dloss, tau)
    ro.check(sl, ref, bound, "step's loss")
    ro.check(sd, dref, dbound, "step's dlogits")
    for _ in range(2):
        again = rows.distill_step(z, index, teacher, dloss, tau)
        assert same(again[0], sl) and same(again[1], sd)
    # in place
    z1, z2 = z.clone(), z.clone()
    rows.distill_backward(z1, index, teacher, stats, dloss, tau, dlogits=z1)
    assert same(z1, rows.distill_backward(z, index, teacher, stats, dloss, tau))
    assert same(rows.distill_step(z2, index, teacher, dloss, tau, dlogits=z2)[1], sd)


# Several rows per CTA, live and padded ones in turn, through every number of threads: rows that
# shared memory cannot hold whole in one pass (512 threads; 256, 128 and 64 with a little too much for
# their share), and the two passes' ring refilled by CTAs of 64 threads.
DISTILL_MANY = [
    (300, 131072, 128, BF16, 1.0),
    (310, 100003, 33, BF16, 2.0),
    (200, 60001, 20, F32, 1.0),
    (1000, 33501, 20, BF16, 1.0),
    (1100, 8401, 40, F32, 0.5),
    (2400, 8451, 9, BF16, 1.0),
    (2400, 20001, 16, BF16, 1.0),
]


@pytest.mark.parametrize("case", DISTILL_MANY, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_distill_many_rows(case):
    n, V, K, dt, tau = case
    z, index, teacher, dloss = distill_case(n, n, V, K, dt)
    loss, stats = rows.distill(z, index, teacher, tau)
    dz = rows.distill_backward(z, index, teacher, stats, dloss, tau)
    sl, sd = rows.distill_step(z, index, teacher, dloss, tau)
    z1, z2 = z.clone(), z.clone()
    assert same(rows.distill_backward(z1, index, teacher, stats, dloss, tau, dlogits=z1), dz)
    assert same(rows.distill_step(z2, index, teacher, dloss, tau, dlogits=z2)[1], sd)
    for a in range(0, n, 128):
        part = [t[a:a + 128] for t in (z, index, teacher)]
        ref, bound, sref, sbound = ro.distill(*part, tau)
        ro.check(loss[a:a + 128], ref, bound, f"loss from {a}")
        ro.check(sl[a:a + 128], ref, bound, f"step's loss from {a}")
        ro.check(stats[a:a + 128], sref, sbound, f"stats from {a}")
        ref, bound = ro.distill_backward(*part, dloss[a:a + 128], tau)
        ro.check(dz[a:a + 128], ref, bound, f"dlogits from {a}")
        ro.check(sd[a:a + 128], ref, bound, f"step's dlogits from {a}")


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("lo,dlo", [(0, 0), (1, 1), (3, 0), (5, 2)])
def test_distill_layouts(dt, lo, dlo):
    """A padded vocabulary's view (rows apart, off 16-byte boundaries), gradients laid out alike
    or otherwise; what lies between the rows stays."""
    n, V, K = 9, 999, 12
    z, index, teacher, dloss = distill_case(77, n, V, K, dt)
    wide = torch.full((n, 1040), 50.0, dtype=dt, device="cuda")
    wide[:, lo:lo + V] = z
    view = wide[:, lo:lo + V]
    loss, stats = rows.distill(view, index, teacher, 1.5)
    ref, bound, _, _ = ro.distill(z, index, teacher, 1.5)
    ro.check(loss, ref, bound, "loss")
    dref, dbound = ro.distill_backward(z, index, teacher, dloss, 1.5)
    for step in (False, True):
        buf = torch.full((n, 1040), 9.0, dtype=dt, device="cuda")
        out = buf[:, dlo:dlo + V]
        if step:
            rows.distill_step(view, index, teacher, dloss, 1.5, dlogits=out)
        else:
            rows.distill_backward(view, index, teacher, stats, dloss, 1.5, dlogits=out)
        ro.check(out, dref, dbound, f"dlogits step={step}")
        assert (buf[:, :dlo] == 9).all() and (buf[:, dlo + V:] == 9).all()
    one = dloss[3]
    dref, dbound = ro.distill_backward(z, index, teacher, one.expand(n), 1.5)
    ro.check(rows.distill_backward(view, index, teacher, stats, one, 1.5), dref, dbound, "one value")


def test_distill_special_rows():
    """A row of the type's lowest value is uniform; a row of -inf and a row with a NaN give NaN
    and stay alone; a padded row is not read; mass on an entry at -inf is an infinite loss."""
    n, V, K = 8, 2000, 4
    for dt in (BF16, F32):
        z, index, teacher, dloss = distill_case(3, n, V, K, dt, pad=False)
        base = rows.distill(z, index, teacher)[0]
        low = torch.finfo(dt).min
        z = z.clone()
        z[0] = low
        z[1] = -INF
        z[2, 700] = NAN
        z[3] = NAN
        index[3] = -1
        z[4, index[4, 0]] = -INF
        z[5, :1500] = -INF
        index[5] = 1500 + torch.arange(K, device="cuda")
        loss, stats = rows.distill(z, index, teacher)
        assert same(loss[6:], base[6:])
        assert torch.isnan(loss[1]) and torch.isnan(loss[2]) and loss[3] == 0 and loss[4] == INF
        keep = torch.tensor([0, 3, 4, 5, 6, 7], device="cuda")
        zk = z[keep].clone()
        zk[1] = 0
        ref, bound, sref, sbound = ro.distill(zk, index[keep], teacher[keep], 1.0)
        ro.check(loss[keep], ref, bound, "loss")
        ro.check(stats[keep], sref, sbound, "stats")
        dref, dbound = ro.distill_backward(zk, index[keep], teacher[keep], dloss[keep], 1.0)
        for d in (rows.distill_backward(z, index, teacher, stats, dloss),
                  rows.distill_step(z, index, teacher, dloss)[1]):
            ro.check(d[keep], dref, dbound, "dlogits")
            assert torch.isnan(d[1]).all() and torch.isnan(d[2]).all()
    # a NaN or an infinity among the teacher's live slots
    teacher[6, 1] = NAN
    teacher[7, 0] = INF
    loss, _ = rows.distill(z, index, teacher)
    assert torch.isnan(loss[6]) and torch.isnan(loss[7]) and not torch.isnan(loss[0])


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("tau", [0.5, 1.0, 2.0])
def test_distill_slot_at_the_lowest_value(dt, tau):
    """The teacher gives mass to an entry that holds the type's lowest value (an entry not in
    use): the loss is about tau p 3.4e38, which fp32 holds."""
    z, index, teacher, dloss = distill_case(12, 6, 900, 5, dt, pad=False)
    for r in range(5):
        index[r] = torch.arange(5) * 7 + r
        z[r, index[r, r]] = torch.finfo(dt).min
    teacher[:] = torch.tensor([0.2, 0.1, 0.0, -0.1, 0.3])
    ref, bound, _, _ = ro.distill(z, index, teacher, tau)
    assert (ref[:5] > 1e36).all() and (ref < 3e38).all()
    loss, stats = rows.distill(z, index, teacher, tau)
    ro.check(loss, ref, bound, "loss")
    sl, d = rows.distill_step(z, index, teacher, dloss, tau)
    ro.check(sl, ref, bound, "step's loss")
    dref, dbound = ro.distill_backward(z, index, teacher, dloss, tau)
    ro.check(d, dref, dbound, "step's dlogits")
    ro.check(rows.distill_backward(z, index, teacher, stats, dloss, tau), dref, dbound, "dlogits")


def test_distill_is_cross_entropy_with_one_slot():
    z, index, _, dloss = distill_case(9, 50, 777, 1, F32, pad=False)
    loss, _ = rows.distill(z, index, torch.zeros(50, 1, device="cuda"))
    z64 = ro.f64(z)
    ref = torch.logsumexp(z64, 1) - z64.gather(1, index.cpu())[:, 0]
    assert (ro.f64(loss) - ref).abs().max() <= 1e-5


def test_distill_autograd_and_differences():
    """Gradient along a direction against central differences of the fp64 loss."""
    n, V, K, tau, h = 6, 300, 9, 1.7, 1e-5
    z, index, teacher, dloss = distill_case(31, n, V, K, F32, pad=False)
    ro.HALF.setdefault(torch.float64, 0.0)
    zg = z.clone().requires_grad_()
    loss = rows.Distill.apply(zg, index, teacher, tau)
    (loss * dloss).sum().backward()
    v = torch.randn(n, V, generator=gen(32), dtype=torch.float64)
    up, down = (ro.distill((ro.f64(z) + s * h * v), index, teacher, tau)[0] for s in (1, -1))
    slope = ((up - down) * ro.f64(dloss)).sum() / (2 * h)
    got = ro.f64(zg.grad)
    assert abs((got * v).sum() - slope) <= 1e-5 * (got.abs() * v.abs()).sum()
    zg.grad = None
    rows.Distill.apply(zg.view(2, 3, V), index.view(2, 3, K), teacher.view(2, 3, K), tau).mean().backward()
    ref, bound = ro.distill_backward(z, index, teacher, torch.full((n,), 1 / 6), tau)
    ro.check(zg.grad, ref, bound, "mean")


def test_distill_without_rows():
    z = torch.empty(0, 100, dtype=BF16, device="cuda")
    i = torch.empty(0, 4, dtype=torch.int64, device="cuda")
    t, d = torch.empty(0, 4, device="cuda"), torch.empty(0, device="cuda")
    loss, stats = rows.distill(z, i, t)
    assert loss.shape == (0,) and stats.shape == (0, 2)
    assert rows.distill_step(z, i, t, d)[1].shape == (0, 100)
    assert rows.distill_backward(z, i, t, stats, d).shape == (0, 100)


# ----------------------------------------------------------------- streams, graphs, together


def all_ops(seed):
    """Inputs of every operator and a function that runs them all, as (inputs, run)."""
    q, k, w, freq, pos, dy = qk_case(seed, 2, 4, 2, 200, 64, BF16, layout="projection")
    z, index, teacher, dloss = distill_case(seed, 20, 5000, 16, BF16)
    g = gen(seed)
    table, dout = randn(g, 900, 128, dt=BF16), randn(g, 3000, 128, dt=BF16)
    ids = tokens(g, 3000, 900, "text").cuda()
    inputs = [q, k, *w, *dy, z, index, teacher, dloss, table, dout, ids]

    def run(stream=None):
        kw = dict(stream=stream)
        out = [*rows.qk_norm_rope(q, k, *w, freq, **kw),
               *rows.qk_norm_rope_backward(q, k, *dy, *w, freq, **kw),
               rows.embed(ids, table, 2.0, **kw), rows.embed_backward(ids, dout, 900, 2.0, **kw)]
        loss, stats = rows.distill(z, index, teacher, 2.0, **kw)
        return [*out, loss, stats, rows.distill_backward(z, index, teacher, stats, dloss, 2.0, **kw),
                *rows.distill_step(z, index, teacher, dloss, 2.0, **kw)]

    return inputs, run


def test_operators_on_a_given_stream_and_a_current_one():
    inputs, run = all_ops(41)
    ref = [t.clone() for t in run()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(same(a, b) for a, b in zip(got, ref))
    with torch.cuda.stream(s):
        got = run()
    torch.cuda.current_stream().wait_stream(s)
    assert all(same(a, b) for a, b in zip(got, ref))


def test_operators_at_once_on_two_streams():
    (_, run_a), (_, run_b) = all_ops(42), all_ops(43)
    ref_a, ref_b = [t.clone() for t in run_a()], [t.clone() for t in run_b()]
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(sa):
            a = run_a()
        with torch.cuda.stream(sb):
            b = run_b()
        torch.cuda.synchronize()
        assert all(same(x, y) for x, y in zip(a, ref_a)) and all(same(x, y) for x, y in zip(b, ref_b))


def test_operators_captured_and_replayed_on_new_inputs():
    """Two graphs, replayed at the same time on two streams, each on inputs that changed since
    the capture."""
    cases = [all_ops(s) for s in (44, 45)]
    fresh = [all_ops(s) for s in (46, 47)]
    graphs, outs = [], []
    for _, run in cases:
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        graphs.append(g)
    refs = []
    for (inputs, _), (new, run_new) in zip(cases, fresh):
        refs.append([t.clone() for t in run_new()])
        for a, b in zip(inputs, new):
            a.copy_(b)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, (torch.cuda.Stream(), torch.cuda.Stream())):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for out, ref in zip(outs, refs):
            assert all(same(a, b) for a, b in zip(out, ref))


def test_profile_names_the_kernels():
    _, run = all_ops(48)
    rsa.profile_enable(True)
    try:
        run()
        seen = rsa.profile_read()
    finally:
        rsa.profile_enable(False)
    assert {"qk_norm_rope", "qk_norm_rope_bwd", "qk_dw", "embed", "embed_sort", "embed_grad",
            "embed_join", "distill", "distill_bwd", "distill_step"} <= set(seen)


def test_given_workspaces():
    q, k, w, freq, _, dy = qk_case(50, 1, 2, 2, 33, 64, BF16)
    ws = torch.empty(rows.qk_norm_rope_workspace_size(64), dtype=torch.uint8, device="cuda")
    a = rows.qk_norm_rope_backward(q, k, *dy, *w, freq, workspace=ws)
    assert all(same(x, y) for x, y in zip(a, rows.qk_norm_rope_backward(q, k, *dy, *w, freq)))
    with pytest.raises(rsa.RSAError, match="WORKSPACE"):
        rows.qk_norm_rope_backward(q, k, *dy, *w, freq, workspace=ws[:-256])
    ids, dout = tokens(gen(1), 999, 70, "text").cuda(), randn(gen(2), 999, 48)
    ws = torch.full((rows.embed_workspace_size(999, 70, 48) + 256,), 0xff, dtype=torch.uint8, device="cuda")
    ref = rows.embed_backward(ids, dout, 70)
    for _ in range(2):
        assert same(rows.embed_backward(ids, dout, 70, workspace=ws[:-256]), ref)
        assert (ws[-256:] == 0xff).all()
    with pytest.raises(rsa.RSAError, match="WORKSPACE"):
        rows.embed_backward(ids, dout, 70, workspace=ws[:-512])


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements into a tensor: the last ones of 4.3 GB of queries, table, gradient
    and logits, against the same rows by themselves."""
    far = (1 << 31) + 4096
    buf = torch.empty(far + 4096, dtype=BF16, device="cuda")
    x, k, dy = randn(gen(70), 2, 1, 5, 64, dt=BF16), randn(gen(71), 2, 1, 5, 64, dt=BF16), randn(gen(72), 2, 1, 5, 64, dt=BF16)
    w, freq = torch.ones(64, device="cuda"), torch.rand(32, generator=gen(73)).cuda()
    q = buf.as_strided((2, 1, 5, 64), (far, 320, 64, 1))
    q.copy_(x)
    assert same(rows.qk_norm_rope(q, k, w, w, freq)[0], rows.qk_norm_rope(x, k, w, w, freq)[0])
    ref = rows.qk_norm_rope_backward(x, k, dy, dy, w, w, freq)
    got = rows.qk_norm_rope_backward(q, k, dy, dy, w, w, freq, dq=q)
    assert all(same(a, b) for a, b in zip(got, ref))
    # a table and its gradient: 2^25 + 64 rows of 64
    V = far // 64 + 60
    table = buf[:V * 64].view(V, 64)
    ids = torch.tensor([V - 1, 3, V - 2, V - 1], device="cuda")
    table[ids] = x.view(10, 64)[:4]
    assert same(rows.embed(ids, table, 2.0), rows.embed(torch.arange(4, device="cuda"), table[ids].clone(), 2.0))
    rows.embed_backward(ids, dy.view(10, 64)[:4], V, dtable=table)
    small = rows.embed_backward(torch.tensor([2, 0, 1, 2], device="cuda"), dy.view(10, 64)[:4], 3)
    assert same(table[[V - 1, 3, V - 2]], small[[2, 0, 1]]) and (table[V - 3] == 0).all() and (table[:3] == 0).all()
    # logits: the last of 65536 rows of 32768, the others without a slot
    V = 32768
    n = buf.numel() // V
    z = buf[:n * V].view(n, V)
    zs, index, teacher, dloss = distill_case(74, 3, V, 9, BF16, pad=False)
    z[n - 3:] = zs
    many = torch.full((n, 9), -1, device="cuda")
    many[n - 3:] = index
    t = torch.zeros(n, 9, device="cuda")
    t[n - 3:] = teacher
    d = torch.zeros(n, device="cuda")
    d[n - 3:] = dloss
    loss, stats = rows.distill(z, many, t)
    ref, bound, _, _ = ro.distill(zs, index, teacher, 1.0)
    ro.check(loss[n - 3:], ref, bound, "loss")
    rows.distill_step(z, many, t, d, dlogits=z)
    dref, dbound = ro.distill_backward(zs, index, teacher, dloss, 1.0)
    ro.check(z[n - 3:], dref, dbound, "dlogits")
    assert (z[:n - 3] == 0).all()


def test_a_row_of_more_than_2_30_logits():
    """Sizes whose bytes pass 32 bits, on one row: the sum in fp64, piece by piece, and the gradient's
    values at both ends and at the slots."""
    V = (1 << 30) + 77
    z = torch.empty(1, V, dtype=BF16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    index = torch.tensor([[5, V - 1, 1 << 29]], device="cuda")
    teacher = torch.tensor([[1.0, 2.0, 0.5]], device="cuda")
    m = float(z.max())
    total = sum(float(torch.exp(z[0, a:a + (1 << 26)].double() - m).sum()) for a in range(0, V, 1 << 26))
    lse = m + math.log(total)
    p = torch.softmax(teacher.cpu().double(), 1)
    zj = z[0, index[0]].double().cpu()
    want = float((p * (torch.log(p) - (zj - lse))).sum())
    one = torch.ones(1, device="cuda")
    loss, stats = rows.distill(z, index, teacher)
    sl, d = rows.distill_step(z, index, teacher, one)
    db = rows.distill_backward(z, index, teacher, stats, one)
    # an exponent of at most 16 in fp32 and V / 2^11 additions per thread of like terms
    assert abs(float(loss) - want) <= 1e-4 and abs(float(sl) - want) <= 1e-4
    for g in (d, db):
        at = torch.cat([torch.arange(3), torch.arange(V - 3, V), index[0].cpu()])
        ref = torch.exp(z[0, at.cuda()].double().cpu() - lse)
        for j in range(3):
            ref[at == index[0, j].item()] -= p[0, j]
        assert ((g[0, at.cuda()].double().cpu() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-4 * ref.abs() + 1e-15).all()
        assert abs(float(g.double().sum())) <= 2e-3


def test_rows_of_the_most_logits():
    """The largest vocabulary, V = 2^31 - 2, of which a row's last columns lie within a block of 2^31:
    a row without a slot and one with three, of a single row of equal logits that is read for both.
    q = 1 / V; what lies before and behind the gradient stays."""
    V, n, pad = (1 << 31) - 2, 2, 4096
    z = torch.zeros(1, V, dtype=BF16, device="cuda").expand(n, V)
    index = torch.tensor([[-1, -1, -1], [0, V - 1, V // 2]], device="cuda")
    teacher, one = torch.zeros(n, 3, device="cuda"), torch.ones(n, device="cuda")
    buf = torch.empty(pad + n * V + pad, dtype=BF16, device="cuda")
    d = buf[pad:pad + n * V].view(n, V)
    # sums of like terms, at most 2^21 of them in a thread: exact before the last few additions
    want = math.log(V / 3)
    loss, stats = rows.distill(z, index, teacher)
    # (and the loss of 20 carries the probabilities' error of 2^-21 of it)
    assert loss[0] == 0 and abs(float(loss[1]) - want) <= 2e-5
    assert (stats[0] == 0).all() and abs(float(stats[1, 1]) - math.log(V)) <= 1e-5
    for step in (False, True):
        buf.fill_(7)
        if step:
            got, _ = rows.distill_step(z, index, teacher, one, dlogits=d)
            assert same(got, loss)
        else:
            rows.distill_backward(z, index, teacher, stats, one, dlogits=d)
        assert (buf[:pad] == 7).all() and (buf[-pad:] == 7).all()
        for a in range(0, V, 1 << 28):
            assert (d[0, a:a + (1 << 28)] == 0).all()
        at = index[1].sort().values
        assert ((d[1, at].double() + 1 / 3).abs() <= 2.0 ** -8 / 3 + 1e-6).all()
        d[1, at] = d[1, 1].clone()
        assert abs(float(d[1, 1]) * V - 1) <= 2.0 ** -8 + 1e-4
        for a in range(0, V, 1 << 28):
            assert (d[1, a:a + (1 << 28)] == d[1, 1]).all()


def test_embed_at_the_ends_of_its_range():
    """The most rows (V = 2^31 - 2, of one element), the widest (D = 2^20) and millions of tokens."""
    V, pad = (1 << 31) - 2, 4096
    ids = torch.tensor([V - 1, 0, V, V - 1, -1, 5, V // 2, V - 2], device="cuda")
    buf = torch.full((pad + V + pad,), 7.0, dtype=BF16, device="cuda")
    table = buf[pad:pad + V].view(V, 1)
    dout = torch.arange(1, 9, device="cuda").to(BF16)[:, None]
    rows.embed_backward(ids, dout, V, 2.0, dtable=table)
    assert (buf[:pad] == 7).all() and (buf[-pad:] == 7).all()
    want = [10.0, 4.0, 0.0, 10.0, 0.0, 12.0, 14.0, 16.0]
    assert rows.embed(ids, table)[:, 0].tolist() == want
    live = torch.tensor([0, 1, 5, 6, 7], device="cuda")
    table[ids[live]] = 0
    assert all((table[a:a + (1 << 28)] == 0).all() for a in range(0, V, 1 << 28))
    # (one more time, added to what is there)
    rows.embed_backward(ids, dout, V, 2.0, dtable=table, accumulate=True)
    assert rows.embed(ids, table)[:, 0].tolist() == want
    del buf, table
    D = 1 << 20
    wide = randn(gen(28), 5, D, dt=BF16)
    ids = torch.tensor([4, 2, 4, 7], device="cuda")
    assert same(rows.embed(ids, wide)[:3], wide[[4, 2, 4]])
    ref, bound = ro.embed_backward(ids, wide[:4], 5, 1.0, BF16)
    ro.check(rows.embed_backward(ids, wide[:4], 5), ref, bound, "wide")
    # whole numbers, whose sums are exact in fp32
    n, V, D = 5_000_001, 1003, 4
    ids = torch.randint(-3, V + 3, (n,), generator=gen(29)).cuda()
    dout = torch.randint(-3, 4, (n, D), generator=gen(30)).float().cuda()
    got = rows.embed_backward(ids, dout, V)
    ok = (ids >= 0) & (ids < V)
    ref = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, ids[ok], dout[ok].double())
    assert torch.equal(got.double(), ref)


def test_qk_of_many_rows():
    """2^22 + 5 rows of one head, and 3000 heads of a few rows: every row as in a call of its own."""
    w, freq = 1 + randn(gen(31), 32, scale=0.2), torch.rand(8, generator=gen(32)).cuda()
    L = (1 << 22) + 5
    x, dy = (torch.randn(1, 1, L, 32, generator=torch.Generator("cuda").manual_seed(s), device="cuda").to(BF16)
             for s in (33, 34))
    y = rows.qk_norm_rope(x, x, w, w, freq, pos0=3)[0]
    dx = rows.qk_norm_rope_backward(x, x, dy, dy, w, w, freq, pos0=3)[0]
    for a, b in ((0, 9), (L // 2, L // 2 + 17), (L - 5, L)):
        cut = [t[:, :, a:b].contiguous() for t in (x, dy)]
        assert same(y[:, :, a:b], rows.qk_norm_rope(cut[0], cut[0], w, w, freq, pos0=3 + a)[0])
        assert same(dx[:, :, a:b], rows.qk_norm_rope_backward(cut[0], cut[0], cut[1], cut[1], w, w, freq, pos0=3 + a)[0])
    x, dy = randn(gen(35), 2, 3000, 3, 32, dt=F32), randn(gen(36), 2, 3000, 3, 32, dt=F32)
    y = rows.qk_norm_rope(x, x[:, :1], w, None, freq)[0]
    g = rows.qk_norm_rope_backward(x, x[:, :1], dy, dy[:, :1], w, None, freq)
    at = ro.positions_of(3, 0, None)
    ref, bound = ro.qk_norm_rope(x, w, freq, at, 1e-6, False)
    ro.check(y, ref, bound, "y")
    dx, db, dw, wb = ro.qk_norm_rope_backward(x, w, freq, at, dy, 1e-6, False)
    ro.check(g[0], dx, db, "dx")
    ro.check(g[2], dw, wb, "dw")
    assert g[3] is None


def test_numbers_of_other_types():
    """numpy's numbers, where a Python number is meant."""
    import numpy as np

    q, k, w, freq, _, _ = qk_case(75, 1, 1, 1, 5, 64, F32)
    assert same(rows.qk_norm_rope(q, k, *w, freq, pos0=np.int64(3), eps=np.float32(1e-5))[0],
                rows.qk_norm_rope(q, k, *w, freq, pos0=3, eps=float(np.float32(1e-5)))[0])
    z, index, teacher, _ = distill_case(76, 3, 50, 2, F32)
    assert same(rows.distill(z, index, teacher, np.float32(2))[0], rows.distill(z, index, teacher, 2)[0])


def test_a_training_step_of_the_operators_together():
    """tokens -> embed -> projection -> norm and rotation -> ring attention -> projection ->
    distillation, forward and backward in fp32 through the autograd wrappers, against the same
    model in fp64 by differentiation of the plain form. fp32 arithmetic through five layers of
    sums of at most 256 terms: 1e-4 of each gradient's largest value is far above its rounding."""
    B, H, L, d, V, K, N, tau = 2, 2, 96, 64, 500, 10, 4, 2.0
    hid = H * d
    g = gen(60)
    ids = tokens(g, B * L, V, "text").view(B, L)
    index = torch.randint(0, V, (B, L, K), generator=g)
    index[0, :7] = -1
    teacher = torch.randn(B, L, K, generator=g)
    params = {"table": torch.randn(V, hid, generator=g) * 0.1,
              "wqkv": torch.randn(3 * hid, hid, generator=g) * hid ** -0.5,
              "wq": 1 + 0.1 * torch.randn(d, generator=g), "wk": 1 + 0.1 * torch.randn(d, generator=g),
              "head": torch.randn(V, hid, generator=g) * hid ** -0.5}
    freq = torch.exp(-math.log(10000.0) * 2 * torch.arange(d // 2, dtype=torch.float64) / d).float()
    scale = 3.0

    def model(p, own):
        if own:
            x = rows.Embedding.apply(ids.cuda(), p["table"], scale)
        else:
            live = (ids >= 0)[..., None]
            x = torch.where(live, p["table"][ids.clamp(0)] * scale, 0.0)
        qkv = (x @ p["wqkv"].T).view(B, L, 3, H, d).permute(2, 0, 3, 1, 4)
        if own:
            q, k = rows.QKNormRope.apply(qkv[0], qkv[1], p["wq"], p["wk"], freq.cuda(), None, 11)
            o = rsa.RingSelfAttention.apply(q, k, qkv[2].contiguous(), N, True)
        else:
            cos, sin = ro._angles(freq, torch.arange(11, 11 + L)[None])
            q, k = (ro._rotate(t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w, cos, sin, d, False)
                    for t, w in ((qkv[0], p["wq"]), (qkv[1], p["wk"])))
            s = q @ k.transpose(-1, -2) / math.sqrt(d)
            s = s.masked_fill(torch.triu(torch.ones(L, L, dtype=torch.bool), 1), -INF)
            o = torch.softmax(s, -1) @ qkv[2]
        z = (x + o.transpose(1, 2).reshape(B, L, hid)) @ p["head"].T
        if own:
            loss = rows.Distill.apply(z, index.cuda(), teacher.cuda(), tau)
        else:
            live = index >= 0
            used = live.any(-1)
            lp = torch.log_softmax(torch.where(used[..., None], teacher, 0.0).double() / tau, -1)
            lq = (torch.log_softmax(z / tau, -1)).gather(-1, index.clamp(0))
            loss = torch.where(used, tau * tau * (lp.exp() * (lp - lq)).sum(-1), 0.0)
        return loss

    prec = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        mine = {n: t.clone().cuda().requires_grad_() for n, t in params.items()}
        loss = model(mine, True)
        loss.mean().backward()
    finally:
        torch.backends.cuda.matmul.allow_tf32 = prec
    plain = {n: t.double().requires_grad_() for n, t in params.items()}
    ref = model(plain, False)
    ref.mean().backward()
    assert (ro.f64(loss) - ref.detach()).abs().max() <= 1e-4 * ref.detach().abs().max()
    for n in params:
        want = plain[n].grad
        assert (ro.f64(mine[n].grad) - want).abs().max() <= 1e-4 * want.abs().max(), n
