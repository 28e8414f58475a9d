"""The row-local operators on the framework's own path: the block with norm and rotation of its
queries and keys, and the model around it (block.model_forward, block.model_loss).

* CPU: gloo ranks run the block with fp64 stand-ins; what is checked is that every rank rotates
  its rows by their positions in the whole sequence, and that a block without norm weights and
  frequencies is what it was.
* GPU (`-m gpu`): a whole model on one rank against the same model in fp64."""
import datetime
import math
import os

import numpy as np
import pytest
import torch
import torch.multiprocessing as mp

import rows_oracle as ro
from sequence_ring_self_b200 import block, ring
from sequence_ring_self_b200.inputs import normals, round_to_bf16

from test_sp_block import BF16_MAXABS, BF16_RELL2, _free_port, _weights, block_inputs, fp64_linear, oracle_block
from test_sp_ring import Fp64Steps

FREQ = (1.0, 0.21)
SHAPE = dict(L=32, hidden=16, H=2, d=4, ffn=24)


def fp64_qk(q, k, wts, pos0):
    """The norm and rotation in fp64, from the oracle's pieces."""
    rot = 2 * len(wts.freq)
    cos, sin = ro._angles(wts.freq, torch.arange(pos0, pos0 + q.shape[2])[None])
    return tuple(ro._rotate(x / torch.sqrt((x * x).mean(-1, keepdim=True) + wts.norm_eps) * w, cos, sin,
                            rot, wts.interleaved)
                 for x, w in ((q, wts.wq_norm), (k, wts.wk_norm)))


def with_norm(wts, d):
    wts.wq_norm, wts.wk_norm = torch.linspace(0.5, 1.5, d), torch.linspace(1.2, 0.8, d)
    wts.freq = torch.tensor(FREQ)
    return wts


def _worker(rank, world, port, out):
    os.environ.update(RANK=str(rank), WORLD_SIZE=str(world), MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    import torch.distributed as dist

    dist.init_process_group("gloo", timeout=datetime.timedelta(seconds=60))
    try:
        s = SHAPE
        w = block_inputs(s["L"], s["hidden"], s["H"], s["d"], s["ffn"], seed=910)
        c = s["L"] // world
        wts = with_norm(_weights(w, s["H"], s["d"], lambda a, bias=False: torch.from_numpy(a.copy())), s["d"])
        x = torch.from_numpy(w["x"][rank * c:(rank + 1) * c].copy())
        z, _ = block.block_forward(x, wts, True, ring=ring.DistRing(), comp=Fp64Steps(), lin=fp64_linear,
                                   qk=fp64_qk)
        out.put((rank, z.numpy()))
    finally:
        dist.destroy_process_group()


def run_ranks(world):
    ctx = mp.get_context("spawn")
    q, port = ctx.Queue(), _free_port()
    procs = [ctx.Process(target=_worker, args=(r, world, port, q)) for r in range(world)]
    for p in procs:
        p.start()
    res = dict(q.get(timeout=180) for _ in range(world))
    for p in procs:
        p.join(timeout=60)
        assert p.exitcode == 0
    return np.concatenate([res[r] for r in range(world)])


def test_every_rank_rotates_by_the_position_in_the_sequence():
    np.testing.assert_allclose(run_ranks(2), run_ranks(1), rtol=0, atol=1e-10)


def fp64_embed(ids, table, scale):
    live = (ids >= 0) & (ids < len(table))
    return torch.where(live[:, None], table[torch.where(live, ids, 0)] * scale, 0.0)


def _model_worker(rank, world, port, out):
    os.environ.update(RANK=str(rank), WORLD_SIZE=str(world), MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    import torch.distributed as dist

    dist.init_process_group("gloo", timeout=datetime.timedelta(seconds=60))
    try:
        s, V, Vp = SHAPE, 45, 48
        to = lambda a, bias=False: torch.from_numpy(a.copy())
        blocks = [with_norm(_weights(block_inputs(s["L"], s["hidden"], s["H"], s["d"], s["ffn"], seed=940 + i),
                                     s["H"], s["d"], to), s["d"]) for i in range(2)]
        blocks[1].freq = None  # the norm alone, and further down neither
        blocks.append(_weights(block_inputs(s["L"], s["hidden"], s["H"], s["d"], s["ffn"], seed=942), s["H"],
                               s["d"], to))
        g = torch.Generator().manual_seed(5)
        wts = block.ModelWeights(table=torch.randn(V, s["hidden"], generator=g, dtype=torch.float64), blocks=blocks,
                                 head=torch.randn(Vp, s["hidden"], generator=g, dtype=torch.float64), vocab=V,
                                 scale=1.5)
        ids = torch.randint(-1, V + 1, (s["L"],), generator=g)
        c = s["L"] // world
        z = block.model_forward(ids[rank * c:(rank + 1) * c], wts, ring=ring.DistRing(), comp=Fp64Steps(),
                                lin=fp64_linear, qk=fp64_qk_or_norm, embed=fp64_embed)
        out.put((rank, z.numpy()))
    finally:
        dist.destroy_process_group()


def fp64_qk_or_norm(q, k, wts, pos0):
    """fp64_qk for a block that may have no frequencies."""
    if wts.freq is not None:
        return fp64_qk(q, k, wts, pos0)
    return tuple(x / torch.sqrt((x * x).mean(-1, keepdim=True) + wts.norm_eps) * w
                 for x, w in ((q, wts.wq_norm), (k, wts.wk_norm)))


def run_model_ranks(world):
    ctx = mp.get_context("spawn")
    q, port = ctx.Queue(), _free_port()
    procs = [ctx.Process(target=_model_worker, args=(r, world, port, q)) for r in range(world)]
    for p in procs:
        p.start()
    res = dict(q.get(timeout=180) for _ in range(world))
    for p in procs:
        p.join(timeout=60)
        assert p.exitcode == 0
    return np.concatenate([res[r] for r in range(world)])


def test_a_model_on_several_ranks_has_the_logits_of_one():
    """Tokens in chunks over gloo ranks: embedding, blocks and head on the rank's rows, every row's
    logits as on one rank, without the head's padded columns."""
    one = run_model_ranks(1)
    assert one.shape == (SHAPE["L"], 45)
    np.testing.assert_allclose(run_model_ranks(2), one, rtol=0, atol=1e-9 * np.abs(one).max())


class _Alone:
    """A ring of one rank, for a block on a whole sequence."""
    rank, world = 0, 1

    def wait(self, handle):
        pass


def test_a_block_without_norm_is_what_it_was(orc):
    s = SHAPE
    w = block_inputs(s["L"], s["hidden"], s["H"], s["d"], s["ffn"], seed=911)
    wts = _weights(w, s["H"], s["d"], lambda a, bias=False: torch.from_numpy(a.copy()))

    def never(*args):
        raise AssertionError("no norm was asked for")

    z, _ = block.block_forward(torch.from_numpy(w["x"]), wts, True, ring=_Alone(), comp=Fp64Steps(),
                               lin=fp64_linear, qk=never)
    np.testing.assert_allclose(z.numpy(), oracle_block(orc, w, s["H"], s["d"], True), rtol=0, atol=1e-10)


@pytest.mark.gpu
def test_model_loss_on_one_rank():
    """Two blocks between embedding and loss, against fp64 on the same bf16 weights; logits within the
    bf16 tolerance of the block's own test, the loss within what such logits can move it:
    tau sum |p - q| |dz| <= 2 tau max |dz|."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from sequence_ring_self_b200 import build

    build.build()
    dev = torch.device("cuda", 0)
    L, hidden, H, d, ffn, V, Vp, K, tau = 256, 128, 2, 64, 256, 500, 512, 12, 2.0
    ws = [block_inputs(L, hidden, H, d, ffn, seed=920 + i) for i in range(2)]
    table = round_to_bf16(normals(930, 0, V * hidden).reshape(V, hidden) * 0.5)
    head = round_to_bf16(normals(931, 0, Vp * hidden).reshape(Vp, hidden) * hidden ** -0.5)
    g = torch.Generator().manual_seed(3)
    ids = torch.randint(0, V, (L,), generator=g)
    ids[5] = -1
    index = torch.randint(0, V, (L, K), generator=g)
    index[:9] = -1
    teacher = torch.randn(L, K, generator=g)
    freq = torch.exp(-math.log(10000.0) * 2 * torch.arange(d // 2, dtype=torch.float64) / d).float()

    def weights(to):
        blocks = []
        for w in ws:
            b = _weights(w, H, d, to)
            b.wq_norm, b.wk_norm, b.freq = torch.linspace(0.5, 1.5, d), torch.linspace(1.2, 0.8, d), freq
            blocks.append(b)
        return block.ModelWeights(table=to(table), blocks=blocks, head=to(head), vocab=V, scale=2.0)

    wts = weights(lambda a, bias=False: torch.from_numpy(np.ascontiguousarray(a)).to(
        torch.float32 if bias else torch.bfloat16).to(dev))
    for b in wts.blocks:
        b.wq_norm, b.wk_norm, b.freq = (t.to(dev) for t in (b.wq_norm, b.wk_norm, b.freq))
    alone = _Alone()
    z = block.model_forward(ids.to(dev), wts, ring=alone)
    loss = block.model_loss(ids.to(dev), index.to(dev), teacher.to(dev), wts, tau, ring=alone)

    plain = weights(lambda a, bias=False: torch.from_numpy(np.ascontiguousarray(a)).double())
    ref = block.model_forward(ids, plain, ring=alone, comp=Fp64Steps(), lin=fp64_linear, qk=fp64_qk,
                              embed=lambda i, t, s: ro.embed(i, t.bfloat16(), s)[0])
    got = z.double().cpu()
    err = (got - ref).abs().max()
    assert err <= BF16_MAXABS * max(1.0, float(ref.abs().max()))
    assert (got - ref).norm() <= 2 * BF16_RELL2 * ref.norm()  # two blocks of what one may be off
    lref, bound, _, _ = ro.distill(ref, index, teacher, tau)
    assert (loss.double().cpu() - lref).abs().max() <= 2 * tau * err + bound.max()
    assert (loss[:9] == 0).all()
