"""The row-local operators around ring attention, as cases to measure: norm and rotation of
queries and keys, embedding lookup and its gradient, distillation from a teacher's top logits.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the calls of
``sequence_ring_self_b200.rows``. Shapes are the repository's workloads (BERT-shaped B=8 H=12
L=512 d=64; GPT-style B=4 H=16 L=4096 d=64; long B=1 H=16 L=16384 d=128, whole or a rank's chunk of
it) with vocabularies of generic sizes, plus odd ones.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------- the cases


def listed():
    return [
        # the next token of four sequences being extended: latency, far positions
        _qk("qk one token", "fwd", B=4, Hq=16, Hk=16, L=1, d=128, explicit=True),
        # one rank's chunk of the long sequence, q and k as views of the projection's output
        _qk("qk rank chunk", "fwd", B=1, Hq=16, Hk=16, L=2048, d=128, pos0=3 * 2048),
        # the whole long sequence, training
        _qk("qk long backward", "bwd", B=1, Hq=16, Hk=16, L=16384, d=128),
        # odd length, shared key heads, part of each head rotated in neighbouring pairs, fp32
        _qk("qk odd backward", "bwd", B=3, Hq=6, Hk=2, L=777, d=64, rot=32, dt="f32",
            interleaved=True, explicit=True),
        # four new tokens
        _embed("embed four tokens", "fwd", T=4, V=32768, D=2048),
        # a GPT-style batch
        _embed("embed batch", "fwd", T=16384, V=50001, D=1024),
        # the long sequence's tokens, training
        _embed("embed long backward", "bwd", T=16384, V=32768, D=2048),
        # a small odd table in fp32, 32-bit ids, some of them padding
        _embed("embed odd backward", "bwd", T=1021, V=5003, D=1001, dt="f32", ids="i32", pad=0.1),
        # a few rows to score, fp32, odd vocabulary
        _distill("distill few rows", "fwd", T=6, V=50001, K=20, dt="f32", temperature=1.0),
        # evaluating a student on a BERT-shaped batch
        _distill("distill forward", "fwd", T=4096, V=32768, K=64, temperature=1.0),
        # training with an odd vocabulary and padded rows
        _distill("distill odd backward", "bwd", T=1000, V=50001, K=33, temperature=2.0, pad=0.1),
        # loss and gradient in one pass, a large vocabulary
        _distill("distill step", "step", T=4096, V=131072, K=128, temperature=2.0),
    ]


def _qk(name, what, B, Hq, Hk, L, d, rot=None, dt="bf16", pos0=0, interleaved=False,
        explicit=False):
    return {"name": name, "op": "qk", "what": what, "B": B, "Hq": Hq, "Hk": Hk, "L": L, "d": d,
            "rot": d if rot is None else rot, "dt": dt, "pos0": pos0, "interleaved": interleaved,
            "explicit": explicit}


def _embed(name, what, T, V, D, dt="bf16", ids="i64", pad=0.0):
    return {"name": name, "op": "embed", "what": what, "T": T, "V": V, "D": D, "dt": dt,
            "ids": ids, "pad": pad}


def _distill(name, what, T, V, K, temperature, dt="bf16", pad=0.0):
    return {"name": name, "op": "distill", "what": what, "T": T, "V": V, "K": K, "dt": dt,
            "temperature": temperature, "pad": pad}


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["qk", "embed", "distill"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op == "qk":
        d = rng.choice([32, 64, 128])
        Hk = rng.choice([1, 2, 5, 8, 12, 16])
        Hq = Hk * rng.choice([1, 1, 2, 4])
        B = _spread(rng, 1, 16)
        L = _spread(rng, 1, max(1, min(16384, 40_000_000 // (B * Hq * d))))
        c = _qk("", rng.choice(["fwd", "bwd"]), B, Hq, Hk, L, d,
                rng.choice([d, d, d // 2]), dt, rng.choice([0, L, 7 * L]),
                rng.random() < 0.4, rng.random() < 0.4)
    elif op == "embed":
        D = _spread(rng, 33, 2048)
        D = rng.choice([D, -(-D // 8) * 8, -(-D // 64) * 64])
        V = _spread(rng, 1000, 60000)
        T = _spread(rng, 1, 32768)
        c = _embed("", rng.choice(["fwd", "bwd", "bwd"]), T, V, D, dt, rng.choice(["i64", "i32"]),
                   rng.choice([0.0, 0.1]))
    else:
        V = _spread(rng, 1000, 131072)
        V = rng.choice([V, -(-V // 128) * 128])
        T = _spread(rng, 1, max(1, min(4096, 400_000_000 // V)))
        c = _distill("", rng.choice(["fwd", "bwd", "step"]), T, V, _spread(rng, 1, 256),
                     rng.choice([0.5, 1.0, 2.0]), dt, rng.choice([0.0, 0.1]))
    del c["name"]
    return c


# ---------------------------------------------------------------------------- the inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape, scale=1.0, dt=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dt)


def _tokens(g, c):
    """Token ids with the frequencies of text (id v about as often as 1 / (v + 10)); a share of
    them -1, which stands for padding."""
    T, V = c["T"], c["V"]
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
    ids = (10.0 * torch.exp(u * math.log((V + 10.0) / 10.0)) - 10.0).long().clamp_(0, V - 1)
    if c["pad"]:
        ids[torch.rand(T, generator=g, device="cuda") < c["pad"]] = -1
    return ids.to(torch.int32 if c["ids"] == "i32" else torch.int64)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    dt = _DT[c["dt"]]
    s = {"case": c}
    if c["op"] == "qk":
        B, Hq, Hk, L, d = c["B"], c["Hq"], c["Hk"], c["L"], c["d"]
        # as the q/k/v projection writes them: heads of q, k and v, one after the other
        qkv = _randn(g, B, Hq + 2 * Hk, L, d, scale=1.5, dt=dt)
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        s["wq"] = 1.0 + _randn(g, d, scale=0.2)
        s["wk"] = 1.0 + _randn(g, d, scale=0.2)
        i = torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64)
        s["freq"] = torch.exp(-math.log(10000.0) * 2.0 * i / c["rot"]).float()
        s["positions"] = None
        if c["explicit"]:
            start = torch.randint(0, 1 << 20, (B, 1), generator=g, device="cuda")
            s["positions"] = start + torch.arange(L, device="cuda")
        if c["what"] == "bwd":
            s["dq_out"] = _randn(g, B, Hq, L, d, dt=dt)
            s["dk_out"] = _randn(g, B, Hk, L, d, dt=dt)
    elif c["op"] == "embed":
        s["ids"] = _tokens(g, c)
        s["scale"] = math.sqrt(c["D"])
        if c["what"] == "fwd":
            s["table"] = _randn(g, c["V"], c["D"], scale=0.02, dt=dt)
        else:
            s["dout"] = _randn(g, c["T"], c["D"], scale=0.1, dt=dt)
    else:
        T, V, K = c["T"], c["V"], c["K"]
        z = torch.empty(T, V, device="cuda", dtype=dt)
        z.normal_(0.0, 2.0, generator=g)
        # the teacher's K tokens of each row, the likeliest first; the last three entries of the
        # vocabulary are never among them
        U = V - 3
        step = 2 * torch.randint(1, max(2, U // (2 * K) - 1), (T, 1), generator=g, device="cuda") - 1
        first = torch.randint(0, U, (T, 1), generator=g, device="cuda")
        index = (first + step * torch.arange(K, device="cuda")) % U
        teacher = 9.0 - 1.2 * torch.log1p(torch.arange(K, device="cuda").float()) \
            + _randn(g, T, K, scale=0.5)
        z.scatter_(1, index, (teacher + _randn(g, T, K)).to(dt))
        if c["pad"]:
            # rows of padding, rows with fewer tokens, entries of the vocabulary not in use
            r = torch.rand(T, 1, generator=g, device="cuda")
            live = torch.where(r < c["pad"], 0.0, torch.where(r < 0.5, K, K * r))
            index = torch.where(torch.arange(K, device="cuda") < live, index, -1)
            z[:, U:] = torch.finfo(dt).min
        s["logits"], s["index"], s["teacher"] = z, index, teacher
        s["dloss"] = torch.rand(T, generator=g, device="cuda") / T
        if c["what"] == "bwd":
            s["stats"] = _distill_rows(z, index, teacher, c["temperature"])[1]
    return s


# ---------------------------------------------------------------------------- one pass


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    from sequence_ring_self_b200 import rows

    c = s["case"]
    if c["op"] == "qk":
        kw = dict(pos0=c["pos0"], positions=s["positions"], eps=1e-6, interleaved=c["interleaved"])
        if c["what"] == "fwd":
            return rows.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["freq"], **kw)
        return rows.qk_norm_rope_backward(s["q"], s["k"], s["dq_out"], s["dk_out"], s["wq"],
                                          s["wk"], s["freq"], **kw)
    if c["op"] == "embed":
        if c["what"] == "fwd":
            return rows.embed(s["ids"], s["table"], s["scale"])
        return rows.embed_backward(s["ids"], s["dout"], c["V"], s["scale"])
    args = (s["logits"], s["index"], s["teacher"])
    if c["what"] == "fwd":
        return rows.distill(*args, c["temperature"])
    if c["what"] == "bwd":
        return rows.distill_backward(*args, s["stats"], s["dloss"], c["temperature"])
    return rows.distill_step(*args, s["dloss"], c["temperature"])


def _plain(s):
    c = s["case"]
    if c["op"] == "qk":
        cos, sin = _angles(s)
        if c["what"] == "fwd":
            return tuple(_norm_rope(x, w, cos, sin, c) for x, w in
                         ((s["q"], s["wq"]), (s["k"], s["wk"])))
        dq, dwq = _norm_rope_backward(s["q"], s["wq"], s["dq_out"], cos, sin, c)
        dk, dwk = _norm_rope_backward(s["k"], s["wk"], s["dk_out"], cos, sin, c)
        return dq, dk, dwq, dwk
    if c["op"] == "embed":
        ids = s["ids"].long()
        live = (ids >= 0) & (ids < c["V"])
        ids = torch.where(live, ids, 0)
        if c["what"] == "fwd":
            x = s["table"][ids].float() * s["scale"]
            return torch.where(live[:, None], x, 0.0).to(s["table"].dtype)
        x = torch.where(live[:, None], s["dout"].float(), 0.0)
        dtable = torch.zeros(c["V"], c["D"], device=x.device).index_add_(0, ids, x)
        return (dtable * s["scale"]).to(s["dout"].dtype)
    args = (s["logits"], s["index"], s["teacher"])
    if c["what"] == "bwd":
        return _distill_grad(*args, s["stats"], s["dloss"], c["temperature"])
    loss, stats = _distill_rows(*args, c["temperature"])
    if c["what"] == "fwd":
        return loss, stats
    return loss, _distill_grad(*args, stats, s["dloss"], c["temperature"])


def _angles(s):
    c = s["case"]
    pos = s["positions"]
    if pos is None:
        pos = c["pos0"] + torch.arange(c["L"], device="cuda")[None]
    a = pos[:, None, :, None].double() * s["freq"].double()
    return torch.cos(a).float(), torch.sin(a).float()


def _pairs(x, c):
    """The two members of each rotated pair, and what is left as it is."""
    r = c["rot"]
    if c["interleaved"]:
        return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]
    return x[..., :r // 2], x[..., r // 2:r], x[..., r:]


def _joined(a, b, rest, c):
    if c["interleaved"]:
        return torch.cat((torch.stack((a, b), -1).flatten(-2), rest), -1)
    return torch.cat((a, b, rest), -1)


def _norm_rope(x, w, cos, sin, c):
    xf = x.float()
    n = xf * torch.rsqrt((xf * xf).mean(-1, keepdim=True) + 1e-6) * w
    a, b, rest = _pairs(n, c)
    return _joined(a * cos - b * sin, b * cos + a * sin, rest, c).to(x.dtype)


def _norm_rope_backward(x, w, dy, cos, sin, c):
    a, b, rest = _pairs(dy.float(), c)
    dn = _joined(a * cos + b * sin, b * cos - a * sin, rest, c)
    xf = x.float()
    r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + 1e-6)
    xhat = xf * r
    u = dn * w
    dx = r * (u - xhat * (u * xhat).mean(-1, keepdim=True))
    dw = (dn * xhat).sum((0, 1, 2), dtype=torch.float64).float()
    return dx.to(x.dtype), dw


def _teacher(index, teacher, V, tau):
    """Live slots, the teacher's probabilities over them and their logarithms."""
    live = (index >= 0) & (index < V) & (teacher != -math.inf)
    t = torch.where(live, teacher.float() / tau, -math.inf)
    m = t.amax(1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(t - m)
    total = e.sum(1, keepdim=True)
    total = torch.where(total == 0, 1.0, total)
    return live, e / total, t - m - torch.log(total)


def _distill_rows(z, index, teacher, tau):
    live, p, logp = _teacher(index, teacher, z.shape[1], tau)
    used = live.any(1)
    zf = z.float()
    m = zf.amax(1)
    logsum = torch.log(torch.exp((zf - m[:, None]) / tau).sum(1))
    logq = (zf.gather(1, torch.where(live, index, 0)) - m[:, None]) / tau - logsum[:, None]
    loss = tau * tau * torch.where(p > 0, p * (logp - logq), 0.0).sum(1)
    stats = torch.stack((m, logsum), 1)
    return torch.where(used, loss, 0.0), torch.where(used[:, None], stats, 0.0)


def _distill_grad(z, index, teacher, stats, dloss, tau):
    live, p, _ = _teacher(index, teacher, z.shape[1], tau)
    g = (tau * dloss)[:, None]
    d = torch.exp((z.float() - stats[:, :1]) / tau - stats[:, 1:]) * g
    d.scatter_add_(1, torch.where(live, index, 0), -g * p)
    return torch.where(live.any(1, keepdim=True), d, 0.0).to(z.dtype)


# ---------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "qk":
        pos = s["positions"]
        pos = torch.arange(c["pos0"], c["pos0"] + c["L"], device="cuda") if pos is None else pos
        angle = torch.einsum("...l,i->...li", pos.double(), s["freq"].double())
        turn = torch.polar(torch.ones_like(angle), angle)
        turn = turn[None, None] if turn.dim() == 2 else turn[:, None]
        outs, grads = [], []
        for x, w, dy in ((s["q"], s["wq"], s.get("dq_out")), (s["k"], s["wk"], s.get("dk_out"))):
            x, w = x.double(), w.double()
            if dy is None:
                outs.append(_exact_rows(x, w, turn, c))
                continue
            x.requires_grad_(), w.requires_grad_()
            grads.append(torch.autograd.grad(_exact_rows(x, w, turn, c), (x, w), dy.double()))
        return tuple(outs) if outs else tuple(grads[j][i] for i in (0, 1) for j in (0, 1))
    if c["op"] == "embed":
        V, ids = c["V"], s["ids"].long()
        ids = torch.where((ids < 0) | (ids >= V), V, ids)  # one row more, for what is outside
        if c["what"] == "fwd":
            rows = torch.cat((s["table"].double(), torch.zeros(1, c["D"], device="cuda").double()))
            return rows[ids] * s["scale"]
        dtable = torch.zeros(V + 1, c["D"], device="cuda", dtype=torch.float64)
        return dtable.index_put_((ids,), s["dout"].double(), accumulate=True)[:V] * s["scale"]
    # distillation: the definition row by row, its gradient by differentiation
    T, V, tau = c["T"], c["V"], c["temperature"]
    loss, stats = [], []
    dz = torch.empty(T, V, device="cuda", dtype=torch.float64) if c["what"] != "fwd" else None
    for a in range(0, T, 512):
        z = s["logits"][a:a + 512].double().requires_grad_(dz is not None)
        index, t = s["index"][a:a + 512], s["teacher"][a:a + 512].double()
        live = (index >= 0) & (index < V) & (t > -math.inf)
        used = live.any(1)
        # the teacher as a distribution over its slots, nothing where a row has none
        logits_t = torch.where(live, t, -1e300) / tau
        logp = torch.where(live, torch.log_softmax(logits_t, 1), 0.0)
        p = torch.where(live, logp.exp(), 0.0)
        logq = torch.gather(z / tau - torch.logsumexp(z / tau, 1, keepdim=True), 1,
                            torch.where(live, index, 0))
        one = torch.where(used, tau * tau * (p * (logp - torch.where(live, logq, 0.0))).sum(1), 0.0)
        m = z.detach().amax(1)
        rest = torch.logsumexp((z.detach() - m[:, None]) / tau, 1)
        loss.append(one.detach())
        stats.append(torch.stack((m, rest), 1) * used[:, None])
        if dz is not None:
            dz[a:a + 512] = torch.autograd.grad(one, z, s["dloss"][a:a + 512].double())[0]
    if c["what"] == "fwd":
        return torch.cat(loss), torch.cat(stats)
    return dz if c["what"] == "bwd" else (torch.cat(loss), dz)


def _exact_rows(x, w, turn, c):
    """Normalised rows whose pairs, as complex numbers, are multiplied by the unit `turn`."""
    r = c["rot"]
    n = x / torch.sqrt(torch.sum(x ** 2, -1, keepdim=True) / c["d"] + 1e-6) * w
    body = n[..., :r]
    shape = (r // 2, 2) if c["interleaved"] else (2, r // 2)
    body = body.unflatten(-1, shape)
    body = body if c["interleaved"] else body.transpose(-1, -2)
    body = torch.view_as_real(torch.view_as_complex(body.contiguous()) * turn)
    body = body if c["interleaved"] else body.transpose(-1, -2)
    return torch.cat((body.flatten(-2), n[..., r:]), -1)


# ---------------------------------------------------------------------------- what it cannot do without


def work(case):
    c = case
    e = 2 if c["dt"] == "bf16" else 4
    if c["op"] == "qk":
        n = c["B"] * (c["Hq"] + c["Hk"]) * c["L"] * c["d"]
        small = 4 * c["rot"] // 2 + 8 * c["d"] + (8 * c["B"] * c["L"] if c["explicit"] else 0)
        if c["what"] == "fwd":
            return {"bytes": 2 * n * e + small, "flops": 8 * n}
        return {"bytes": 3 * n * e + small + 8 * c["d"], "flops": 18 * n}
    if c["op"] == "embed":
        T, V, D = c["T"], c["V"], c["D"]
        ids = T * (8 if c["ids"] == "i64" else 4)
        if c["what"] == "bwd":
            return {"bytes": (T + V) * D * e + ids, "flops": 2 * T * D}
        # the distinct rows that T draws of the tokens' frequencies are expected to meet
        v = np.arange(V, dtype=np.float64)
        share = np.log((v + 11.0) / (v + 10.0)) / math.log((V + 10.0) / 10.0)
        rows = float(np.sum(-np.expm1(T * (1 - c["pad"]) * np.log1p(-np.minimum(share, 0.999999)))))
        return {"bytes": (rows + T) * D * e + ids, "flops": T * D}
    T, V, K = c["T"], c["V"], c["K"]
    slots = T * K * 12
    used = T * (1 - c["pad"])
    if c["what"] == "fwd":
        return {"bytes": used * V * e + slots + 12 * T, "flops": 4 * used * V}
    if c["what"] == "bwd":
        return {"bytes": (used + T) * V * e + slots + 12 * T, "flops": 4 * used * V}
    return {"bytes": (used + T) * V * e + slots + 8 * T, "flops": 8 * used * V}
