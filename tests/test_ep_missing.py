"""Choices without an expert: gmm_router_topk gives id -1 where fewer than k
experts are left.  Such a choice sends no row, is counted for no expert, and
leaves its token's other choices as they are; every other id out of range is
refused as before.  On the CPU, the exchange between gloo ranks."""
import os
import socket

import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

from moe_fp8_grouped_b200 import ep


def test_route_puts_missing_choices_last_and_counts_them_nowhere():
    ids = torch.tensor([[2, -1], [1, 2], [-1, 3], [-1, -1]], dtype=torch.int32)
    for P in (1, 2):
        rt = ep.route(ids, E=4, P=P)
        assert rt.order.tolist() == [2, 0, 3, 5, 1, 4, 6, 7]  # stable; the missing ones behind the experts' rows
        assert rt.counts.tolist() == [0, 1, 2, 1]
        assert rt.send_splits == ([4] if P == 1 else [1, 3])
        assert rt.missing.tolist() == [False, True, False, False, True, False, True, True]
    rt = ep.route(ids, E=4, P=2, sync=False)
    assert int(rt.bad) == 0 and rt.counts.tolist() == [0, 1, 2, 1]
    rt = ep.route(ids, E=4, P=1, validate=False)
    assert rt.order.tolist() == [2, 0, 3, 5, 1, 4, 6, 7] and rt.counts.tolist() == [0, 1, 2, 1]
    rt = ep.route(torch.full((3, 2), -1), E=4, P=2)
    assert rt.counts.tolist() == [0, 0, 0, 0] and rt.send_splits == [0, 0]


@pytest.mark.parametrize("bad", [-2, 4, 2 ** 31 - 1, -2 ** 31])
def test_other_ids_out_of_range_are_still_refused(bad):
    ids = torch.tensor([[0, -1], [bad, 1]], dtype=torch.int32)
    for P in (1, 2):
        with pytest.raises(ValueError, match="out of range"):
            ep.route(ids, E=4, P=P)
        assert int(ep.route(ids, E=4, P=P, sync=False).bad) == 1


def _free_port():
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        return s.getsockname()[1]


def _worker(rank, world, port, q):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        E, T, k = 6, 5, 3
        g = torch.Generator().manual_seed(7 + rank)
        ids = torch.randint(-1, E, (T, k), generator=g)
        ids[0] = -1
        if rank == 0:
            ids[:] = -1  # this rank sends nothing at all
        payload = rank * 1000 + torch.arange(T * k)
        rt = ep.route(ids, E, world, sync=False)
        recv_counts, arrive = ep.exchange_counts(rt)
        n = int((ids >= 0).sum())
        assert sum(rt.send_splits) == n
        send = payload[rt.order][:n]
        recv = ep.exchange_rows(send, rt.send_splits, arrive)
        perm, inv, gsz = ep.local_order(recv_counts, sum(arrive))
        back = ep.exchange_rows(recv[perm][inv], arrive, rt.send_splits)
        every = [None] * world
        dist.all_gather_object(every, ids.tolist())
        q.put((rank, recv[perm].tolist(), gsz.tolist(), torch.equal(back, send), every))
    finally:
        dist.destroy_process_group()


def test_missing_choices_do_not_travel():
    world, E = 2, 6
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    port = _free_port()
    procs = [ctx.Process(target=_worker, args=(r, world, port, q)) for r in range(world)]
    for p in procs:
        p.start()
    res = sorted(q.get(timeout=120) for _ in range(world))
    for p in procs:
        p.join(timeout=60)
        assert p.exitcode == 0
    for rank, local, gsz, returned, every in res:
        assert returned
        want = []
        for e in range(rank * E // world, (rank + 1) * E // world):
            rows = [src * 1000 + pos for src in range(world)
                    for pos, x in enumerate(v for row in every[src] for v in row) if x == e]
            assert gsz[e - rank * E // world] == len(rows)
            want += rows
        assert local == want
