"""Which data-parallel forms take the update with orthogonalised momentum: two gloo ranks on the CPU."""
import multiprocessing as mp

import pytest

import gpt_step_b200 as gs
from gpt_step_b200 import dp

from test_dp_gloo import FakeModel, _batches, _free_port


class MuonModel(FakeModel):
    """The fake model with the package's own clip_muon in front of its whole-array update."""

    def clip_muon(self, step, workspace):
        if self.sharded:
            return gs.GPT2.clip_muon(self, step, workspace)
        self.clip_adamw(step)


def _rank_main(rank, world, port, q, mode):
    import torch.distributed as dist
    dist.init_process_group("gloo", init_method=f"tcp://127.0.0.1:{port}", rank=rank, world_size=world)
    try:
        m = MuonModel()
        d = dp.DataParallel(m, mode=mode)
        m.fwd_bwd(*_batches(0, 0, rank, world))
        try:
            d.sync_grads()
            m.clip_muon(0, None)
            q.put((rank, "updated", d.replicas_agree()))
        except ValueError as e:
            q.put((rank, str(e), None))
    finally:
        dist.destroy_process_group()


@pytest.mark.parametrize("mode", ["zero1", "allreduce"])
def test_sharded_ranks_refuse_the_whole_matrix_update(mode):
    ctx = mp.get_context("spawn")
    q, port = ctx.Queue(), _free_port()
    procs = [ctx.Process(target=_rank_main, args=(r, 2, port, q, mode)) for r in range(2)]
    for p in procs:
        p.start()
    out = sorted(q.get(timeout=120) for _ in procs)
    for p in procs:
        p.join(timeout=60)
        assert p.exitcode == 0
    for _, what, agree in out:
        assert ("sharded over ranks" in what) if mode == "zero1" else (what == "updated" and agree)


def test_one_process_takes_it_in_either_form():
    for mode in ("zero1", "allreduce"):
        m = MuonModel()
        dp.DataParallel(m, mode=mode)
        m.fwd_bwd(*_batches(0, 0, 0, 1))
        m.clip_muon(0, None)
        assert m.sharded is False and m.k == 0
