"""Plain fp64 forms of the row-local operators (include/rsa_rows.h), on the CPU, with the error
each output may carry: half a step of its type for the one rounding at the end, plus what fp32
arithmetic on the way can lose. The fp32 terms are written out beside each bound."""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def f64(t):
    return t.detach().to("cpu", torch.float64)


def positions_of(L, pos0, positions):
    return torch.arange(pos0, pos0 + L)[None] if positions is None else positions.cpu().reshape(-1, L)


def _rotate(n, cos, sin, rot, interleaved, back=False):
    if back:
        sin = -sin
    a, b = (n[..., 0:rot:2], n[..., 1:rot:2]) if interleaved else (n[..., :rot // 2], n[..., rot // 2:rot])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((ya, yb), -1).flatten(-2) if interleaved else torch.cat((ya, yb), -1)
    return torch.cat((y, n[..., rot:]), -1)


def _pair_size(n, rot, interleaved):
    """|a| + |b| of each element's pair (|n| where nothing is rotated)."""
    m = n.abs()
    one = torch.ones_like(m[..., :rot // 2])
    a, b = (m[..., 0:rot:2], m[..., 1:rot:2]) if interleaved else (m[..., :rot // 2], m[..., rot // 2:rot])
    s = a + b
    y = torch.stack((s, s), -1).flatten(-2) if interleaved else torch.cat((s, s), -1)
    assert one.shape == s.shape
    return torch.cat((y, m[..., rot:]), -1)


def _angles(freq, pos):
    a = pos.double()[:, None, :, None] * f64(freq)
    return torch.cos(a), torch.sin(a)


def qk_norm_rope(x, w, freq, pos, eps, interleaved):
    """(y, bound): y in fp64. Bound: the sum of squares has at most 13 roundings of 2^-24 behind
    each term, half of it after the root; rsqrtf, the weight, the cosine (sincospif within 2^-22,
    its argument rounded to 2^-24 of half a turn) and the products add up to less than 2^-19 of
    |n_a| + |n_b|."""
    x64 = f64(x)
    rot = 0 if freq is None else 2 * freq.numel()
    n = x64 / torch.sqrt((x64 * x64).mean(-1, keepdim=True) + eps)
    if w is not None:
        n = n * f64(w)
    y = n
    if rot:
        cos, sin = _angles(freq, pos)
        y = _rotate(n, cos, sin, rot, interleaved)
    return y, HALF[x.dtype] * y.abs() + 2.0 ** -19 * _pair_size(n, rot, interleaved) + 1e-37


def qk_norm_rope_backward(x, w, freq, pos, dy, eps, interleaved):
    """(dx, bound, dw, bound): with U >= |u| from the pairs' sizes, dx = r (u - xhat mean(u xhat))
    carries at most 2^-18 r (U + |xhat| mean(U |xhat|)); a weight's gradient adds up N terms of
    size D |xhat|, each off by 2^-19 and behind fewer than 128 roundings of 2^-24 more."""
    x64, g = f64(x), f64(dy)
    rot = 0 if freq is None else 2 * freq.numel()
    r = 1 / torch.sqrt((x64 * x64).mean(-1, keepdim=True) + eps)
    dn, size = g, _pair_size(g, rot, interleaved)
    if rot:
        cos, sin = _angles(freq, pos)
        dn = _rotate(g, cos, sin, rot, interleaved, back=True)
    w64 = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else f64(w)
    u, xhat = dn * w64, x64 * r
    dx = r * (u - xhat * (u * xhat).mean(-1, keepdim=True))
    U = size * w64.abs()
    scale = r * (U + xhat.abs() * (U * xhat.abs()).mean(-1, keepdim=True))
    dw = (dn * xhat).sum((0, 1, 2))
    dw_bound = (2.0 ** -19 + 2.0 ** -17) * (size * xhat.abs()).sum((0, 1, 2)) + 1e-37
    return dx, HALF[x.dtype] * dx.abs() + 2.0 ** -18 * scale + 1e-37, dw, dw_bound


def embed(ids, table, scale):
    """One product in fp32 (2^-24), one rounding."""
    V = table.shape[0]
    ids = ids.cpu().long()
    live = ((ids >= 0) & (ids < V))[..., None]
    y = torch.where(live, f64(table)[torch.where(live[..., 0], ids, 0)] * scale, 0.0)
    return y, (HALF[table.dtype] * (1 + 2.0 ** -10) + 2.0 ** -23) * y.abs() + 1e-37


def embed_backward(ids, dout, V, scale, out_dtype, start=None):
    """A row that adds up c tokens has c roundings of 2^-24 of the sum of magnitudes at most."""
    ids, g = ids.cpu().long().reshape(-1), f64(dout).reshape(-1, dout.shape[-1])
    live = (ids >= 0) & (ids < V)
    ids, g = ids[live], g[live]
    out = torch.zeros(V, g.shape[1], dtype=torch.float64).index_add_(0, ids, g) * scale
    size = torch.zeros_like(out).index_add_(0, ids, g.abs()) * abs(scale)
    c = torch.zeros(V, dtype=torch.float64).index_add_(0, ids, torch.ones(len(ids), dtype=torch.float64))
    if start is not None:
        out, size = out + f64(start), size + f64(start).abs()
    return out, HALF[out_dtype] * (1 + 2.0 ** -10) * out.abs() + (c[:, None] + 3) * 2.0 ** -24 * size + 1e-37


def _teacher(index, teacher, V, tau):
    index, t = index.cpu().long(), f64(teacher)
    live = (index >= 0) & (index < V) & (t != -math.inf)
    t = torch.where(live, t / tau, -math.inf)
    m = t.amax(-1, keepdim=True)
    used = live.any(-1)
    t = torch.where(live, t - torch.where(used[..., None], m, 0.0), -math.inf)
    p = torch.where(live, torch.exp(t), 0.0)
    total = torch.where(used, p.sum(-1), 1.0)[..., None]
    p = p / total
    lnp = torch.where(live, t - torch.log(total), 0.0)
    return torch.where(live, index, 0), live, used, p, lnp, torch.where(live, -t, 0.0)


def distill(logits, index, teacher, tau):
    """(loss, bound, stats, bound). An exponent x = (z - m) / tau in fp32 carries 2^-22 |x|, an
    exponential 2^-22 more, the sum of V of them V / 512 + 32 roundings at most. So ln q is off by
    less than e = 2^-21 (1 + |x_j|) + (V / 512 + 32) 2^-24 + 2^-21 max over the mass' exponents,
    which the row's own entropy-weighted |x| gives, and p by 2^-20 (1 + |t_j|) of itself."""
    z, V = f64(logits), logits.shape[-1]
    index, live, used, p, lnp, t = _teacher(index, teacher, V, tau)
    m = z.amax(-1)
    x = (z - m[..., None]) / tau
    e = torch.exp(x)
    S = e.sum(-1)
    logsum = torch.log(S)
    xj = x.gather(-1, index)
    lnq = xj - logsum[..., None]
    loss = tau * tau * torch.where(p > 0, p * (lnp - lnq), 0.0).sum(-1)
    mass = torch.where(e > 0, e * x.abs(), 0.0).sum(-1) / S  # mean |x| under q
    sum_err = (V / 512 + 32) * 2.0 ** -24 + 2.0 ** -21 * (1 + mass)
    term = torch.where(p > 0, p * ((1 + lnp.abs() + lnq.abs()) * (1 + t) * 2.0 ** -19
                                   + 2.0 ** -21 * xj.abs()), 0.0).sum(-1)
    bound = tau * tau * (term + sum_err) + 2.0 ** -22 * loss.abs()
    stats = torch.stack((m, logsum), -1)
    stats_bound = torch.stack((0 * m, sum_err + 2.0 ** -22 * logsum.abs()), -1)
    zero = torch.zeros_like(loss)
    loss, bound = torch.where(used, loss, zero), torch.where(used, bound, zero)
    return (loss, bound, torch.where(used[..., None], stats, 0.0),
            torch.where(used[..., None], stats_bound, 0.0))


def distill_backward(logits, index, teacher, dloss, tau):
    """(dz, bound): q and p off by what `distill` says, the difference rounded once."""
    z, V = f64(logits), logits.shape[-1]
    index, live, used, p, lnp, t = _teacher(index, teacher, V, tau)
    x = (z - z.amax(-1, keepdim=True)) / tau
    e = torch.exp(x)
    S = e.sum(-1, keepdim=True)
    q = e / S
    mass = torch.where(e > 0, e * x.abs(), 0.0).sum(-1, keepdim=True) / S
    sum_err = (V / 512 + 32) * 2.0 ** -24 + 2.0 ** -20 * (1 + mass)
    g = (f64(dloss) * tau).expand(z.shape[:-1])[..., None]
    dz = torch.where(q >= 0, q, q).scatter_add(-1, index, torch.where(live, -p, 0.0)) * g
    q_err = torch.where(q > 0, q * (2.0 ** -20 * (1 + x.abs()) + sum_err), 0.0)
    p_err = torch.zeros_like(q).scatter_add(-1, index, torch.where(live, p * (1 + t) * 2.0 ** -19, 0.0))
    bound = HALF[logits.dtype] * (1 + 2.0 ** -10) * dz.abs() + g.abs() * (q_err + p_err) + 1e-37
    zero = torch.zeros_like(dz)
    return torch.where(used[..., None], dz, zero), torch.where(used[..., None], bound, zero)


def check(got, ref, bound, name):
    got = f64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{name}: NaN in other places"
    same = got == ref  # infinities among them
    bad = ~nan & ~same & ~((got - ref).abs() <= bound)
    if bad.any():
        i = torch.where(bad, ((got - ref).abs() / bound).nan_to_num(posinf=1e30), 0.0).argmax()
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} out of bounds; worst at {int(i)}: "
                             f"{got.flatten()[i]:.9g} for {ref.flatten()[i]:.9g}, bound {bound.flatten()[i]:.3g}")
