"""Block tables and slot maps without a GPU: the oracle's own pins, and every
refusal that hpc_block_table_append / _truncate make before a launch."""
import random

import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from oracle import block_table_ref as R


@pytest.fixture(scope="module", autouse=True)
def _lib():
    hpc.build()
    hpc.load_library()


def test_oracle_by_hand():
    # 60 + 5 tokens cross into a second block, 64 + 1 start one, 10 + 0 nothing
    got, bits = R.append([60, 64, 10], [5, 1, 0], [7, 8, 9, 4], 4, 10,
                         [[0, -1], [1, -1], [2, -1]], 8, 2)
    assert bits == 0
    assert got["table"] == [[0, 4], [1, 9], [2, -1]]
    assert got["slots"] == [60, 61, 62, 63, 256, 576, -1, -1]
    assert got["positions"] == [60, 61, 62, 63, 64, 64, 0, 0]
    assert got["cu"] == [0, 5, 6, 6] and got["lens"] == [65, 65, 10] and got["count"] == 2
    back, bits = R.truncate(got["lens"], [60, 64, 10], got["table"], 10, [7, 8, -1, -1], 2, 2)
    assert bits == 0 and back == dict(free=[7, 8, 9, 4], lens=[60, 64, 10], count=4)


def test_oracle_append_then_truncate_is_identity():
    rng = random.Random(5)
    for _ in range(100):
        B = rng.randint(0, 9)
        old = [rng.randint(0, 200) for _ in range(B)]
        new = [rng.randint(0, 150) for _ in range(B)]
        ids = list(range(200))
        rng.shuffle(ids)
        table = [[ids.pop() for _ in range(R.blocks_of(o))] + [-1] * (6 - R.blocks_of(o))
                 for o in old]
        got, bits = R.append(old, new, ids, len(ids), 200, table, sum(new) + 3, 6)
        assert bits == 0
        live = [s for s in got["slots"] if s >= 0]
        assert len(live) == len(set(live)) == sum(new)  # no slot twice
        free = ids[:got["count"]] + [-1] * (len(ids) - got["count"])
        back, bits = R.truncate(got["lens"], old, got["table"], 200, free, got["count"], 6)
        assert bits == 0 and back == dict(free=ids, lens=old, count=len(ids))


def _i(*x):
    return torch.tensor(x, dtype=torch.int32)


def _append_args():
    return dict(seq_lens=_i(3, 4), new_lens=_i(1, 1), free_blocks=_i(0, 1, 2), free_count=_i(3),
                num_blocks=8, block_table=torch.zeros(2, 4, dtype=torch.int32),
                seq_lens_out=_i(0, 0), cu_q_lens=_i(0, 0, 0), positions=_i(0, 0), slots=_i(0, 0),
                free_count_out=_i(0))


def _truncate_args():
    return dict(seq_lens=_i(3, 4), to_lens=_i(1, 1), block_table=torch.zeros(2, 4, dtype=torch.int32),
                num_blocks=8, free_blocks=_i(0, 1, 2), free_count=_i(3), seq_lens_out=_i(0, 0),
                free_count_out=_i(0))


def _status(fn, args, **change):
    a = {**args, **change}
    try:
        fn(**a, stream=0)  # host tensors: refused before anything could read them
    except hpc.HpcError as e:
        return e.status
    raise AssertionError("not refused")


I, U = hpc.HPC_ERR_INVALID_ARG, hpc.HPC_ERR_UNSUPPORTED


@pytest.mark.parametrize("change", [
    dict(seq_lens=torch.zeros(2)), dict(seq_lens=None), dict(new_lens=_i(1)),
    dict(new_lens=_i(1, 0, 1, 0)[::2]), dict(free_count=_i(1, 2)), dict(num_blocks=-1),
    dict(num_blocks=2**25), dict(block_table=torch.zeros(3, 4, dtype=torch.int32)),
    dict(block_table=torch.zeros(4, 2, dtype=torch.int32).t()),
    dict(block_table=torch.zeros(1, 4, dtype=torch.int32).expand(2, 4)),
    dict(cu_q_lens=_i(0, 0)), dict(slots=_i(0, 0, 0)), dict(positions=torch.zeros(2)),
    dict(seq_lens_out=_i(0)), dict(free_count_out=None)])
def test_append_refusals(change):
    assert _status(hpc.hpc_block_table_append, _append_args(), **change) == I


@pytest.mark.parametrize("change", [
    dict(seq_lens=torch.zeros(2)), dict(to_lens=_i(1)), dict(free_count=None), dict(num_blocks=-1),
    dict(block_table=torch.zeros(1, 4, dtype=torch.int32).expand(2, 4)),
    dict(seq_lens_out=_i(0, 0, 0)), dict(free_blocks=None)])
def test_truncate_refusals(change):
    assert _status(hpc.hpc_block_table_truncate, _truncate_args(), **change) == I


def test_overlaps_are_refused():
    a = _append_args()
    buf = torch.zeros(8, dtype=torch.int32)
    for change in (dict(positions=buf[:2], slots=buf[1:3]), dict(slots=a["seq_lens"]),
                   dict(seq_lens_out=a["new_lens"]), dict(free_count_out=a["free_blocks"][:1]),
                   dict(seq_lens=buf[0:2], seq_lens_out=buf[1:3]),
                   dict(cu_q_lens=a["block_table"].flatten()[:3])):
        assert _status(hpc.hpc_block_table_append, a, **change) == I
        assert "overlap" in hpc.hpc_last_error()
    t = _truncate_args()
    for change in (dict(free_blocks=t["block_table"].flatten()[:3]), dict(seq_lens_out=t["to_lens"]),
                   dict(free_count_out=t["free_blocks"][2:])):
        assert _status(hpc.hpc_block_table_truncate, t, **change) == I


def test_too_many_sequences():
    n = 16385
    z = torch.zeros(n, dtype=torch.int32)
    t = torch.zeros(n, 1, dtype=torch.int32)
    assert _status(hpc.hpc_block_table_append, _append_args(), seq_lens=z, new_lens=z.clone(),
                   block_table=t, seq_lens_out=z.clone(),
                   cu_q_lens=torch.zeros(n + 1, dtype=torch.int32)) == U
    assert _status(hpc.hpc_block_table_truncate, _truncate_args(), seq_lens=z, to_lens=z.clone(),
                   block_table=t, seq_lens_out=z.clone()) == U
