"""4-bit and bf16 weights of a layer calibrated by two gloo ranks, without a GPU: the rank's buffers that
ask for them are filled, from its rows and the codes it chose, and gathered in row order. The compute
calls go to the stand-in of tests/test_sharded_cpu.py."""
import os

import pytest
import torch
import torch.multiprocessing as mp

from tests import layer_ref as R
from tests.test_sharded_cpu import OracleOps, _free_port, _layer

CASES = {"moe": "full", "mse": "mse"}


class PackingOps(OracleOps):
    def lhcal_pack_weights(self, w, g, codes, packed):
        n = R.pack(w.float(), codes, g)
        packed.copy_((n[..., ::2] | n[..., 1::2] << 4).to(torch.uint8))

    def lhcal_apply_scales(self, w, g, codes, wq=None, wq16=None, amax=None):
        n = R.pack(w.float(), codes, g)
        q = torch.tensor(R.E2M1, dtype=torch.float64)[n & 7] * R.block_scale(codes, g).repeat_interleave(16, -1)
        wq16.copy_(torch.where(n >= 8, -q, q).float().to(torch.bfloat16))


def _worker(rank, world, port, out):
    import datetime

    import torch.distributed as dist

    from scale_calibration_lh_b200 import sharded as S

    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=world, timeout=datetime.timedelta(seconds=120))
    try:
        ops = PackingOps()
        for case, mode in CASES.items():
            layer = _layer(case)
            bf16 = layer.dtype == "bf16"
            x = torch.from_numpy(layer.x_f32()).to(torch.bfloat16 if bf16 else torch.float32)
            w = torch.from_numpy(layer.w_f32()).to(torch.bfloat16 if bf16 else torch.float32)
            t0, t1 = S.token_range(layer.tokens, rank, world)
            r0, r1 = S.row_range(layer.rows, rank, world)
            offs = ids = None
            if layer.group_offsets is not None:
                offs, ids = S.shard_routing(torch.from_numpy(layer.group_offsets), torch.from_numpy(layer.token_ids), t0, t1)
            b = ops.Buffers(mode, t1 - t0, layer.cin, r1 - r0, layer.groups, ops.BF16 if bf16 else ops.F32, "cpu",
                            want_packed=True, want_wq16=True)
            b.packed.fill_(0xA5)
            b.wq16.fill_(7)
            b, res = S.calibrate_sharded(mode, x[t0:t1], w[:, r0:r1].contiguous(), group_offsets=offs, token_ids=ids,
                                         buffers=b, ops=ops)
            out[(rank, case)] = {"w": w, "g": b.g, "codes": res["codes"], "wq": res["wq"], "packed": res.get("packed"),
                                 "wq16": res.get("wq16"), "own": b.packed, "rows": (r0, r1)}
    finally:
        dist.destroy_process_group()


@pytest.fixture(scope="module")
def results():
    world, port = 2, _free_port()
    ctx = mp.get_context("spawn")
    out = ctx.Manager().dict()
    procs = [ctx.Process(target=_worker, args=(r, world, port, out)) for r in range(world)]
    for p in procs:
        p.start()
    for p in procs:
        p.join(300)
        assert p.exitcode == 0
    return dict(out)


@pytest.mark.parametrize("case", sorted(CASES))
@pytest.mark.parametrize("rank", [0, 1])
def test_ranks_pack_their_rows_and_gather_the_layer(results, case, rank):
    r = results[(rank, case)]
    n = R.pack(r["w"].float(), r["codes"], r["g"])
    assert torch.equal(R.nibbles(r["packed"]), n)
    r0, r1 = r["rows"]
    assert torch.equal(R.nibbles(r["own"]), n[:, r0:r1])
    assert torch.equal(r["wq16"].float(), r["wq"].to(torch.bfloat16).float())
