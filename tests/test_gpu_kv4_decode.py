"""hpc_decode_kv4_attn against its definition in 64 bits; the tolerances are those that kv4_util.attend derives."""
import json
import os
import subprocess
import sys

import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from tests.kv4_util import Paged, cu_of, decode, i32

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


LENS = {
    "edges": [1, 0, 63, 64, 65, 127, 128, 129, 0, 8, 7, 3],
    "one": [1],
    "empty": [0, 0, 0],
    "ragged": [700, 1, 2049, 64, 333, 0, 1000],
    "many": [5 + 37 * i % 300 for i in range(90)],
    "long": [9000, 12],
}


def case(name, hkv, q_len, **kw):
    lens = LENS[name]
    return Paged(lens, hkv=hkv, q_rows=len(lens) * q_len, **kw)


@pytest.mark.parametrize("q_len", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("hkv", [1, 2, 3, 8])
@pytest.mark.parametrize("name", ["edges", "ragged"])
def test_parity(name, hkv, q_len):
    c = case(name, hkv, q_len, seed=q_len + 10 * hkv)
    c.check(*decode(c, q_len), cu_of([q_len] * len(c.lens)))


@pytest.mark.parametrize("q_len", [1, 2, 7])
@pytest.mark.parametrize("name", ["one", "empty", "many", "long"])
def test_batches(name, q_len):
    c = case(name, 2, q_len, seed=q_len)
    c.check(*decode(c, q_len), cu_of([q_len] * len(c.lens)))


@pytest.mark.parametrize("q_len", [1, 4])
@pytest.mark.parametrize("sms", [1, 2, 7, 64, 300])
def test_any_number_of_ctas(q_len, sms):
    c = case("ragged", 2, q_len, seed=3)
    c.check(*decode(c, q_len, sms=sms), cu_of([q_len] * len(c.lens)))


@pytest.mark.parametrize("q_len", [1, 3, 8])
def test_one_long_sequence_in_many_pieces(q_len):
    """One pair cut over all CTAs and the pool's chunks: states joined in more than one level."""
    c = Paged([40000], hkv=1, q_rows=q_len, seed=5)
    c.check(*decode(c, q_len), [0, q_len])


@pytest.mark.parametrize("q_len", [1, 2, 5])
@pytest.mark.parametrize("q_scale,spread", [(8.0, 1.0), (40.0, 3.0), (2.0 ** -120, 1.0), (1.0, 300.0)])
def test_sharp_and_flat_scores(q_len, q_scale, spread):
    c = Paged([300, 77, 1500], hkv=1, q_rows=3 * q_len, seed=6, q_scale=q_scale, spread=spread, ks=0.5, vs=0.5)
    c.check(*decode(c, q_len), cu_of([q_len] * 3))


def test_rising_scores():
    """Each key scores higher than the one before, by more and by less than what moves the running maximum."""
    for step in (0.02, 1.0, 7.0):
        c = Paged([500], hkv=1, seed=8, ks=1.0)
        kr = torch.zeros(500, 1, 72, dtype=torch.uint8)
        kr[:, 0, :64] = 0x22  # codes of 1
        kr[:, 0, 64:] = 0x38  # scales of 1
        c.rows[0] = (kr, c.rows[0][1])
        # one element of K grows with the position: codes of 6 times scales; the others are the same
        x = torch.ones(500, 1, 128, dtype=torch.float64)
        x[:, 0, :16] = torch.linspace(0, 440, 500, dtype=torch.float64)[:, None]
        from oracle import kv4_ref
        kr = torch.from_numpy(kv4_ref.rows(x.numpy(), 1.0))
        c.rows[0] = (kr, c.rows[0][1])
        pos = torch.arange(500)
        c.k[c.table[0, pos // 64].long(), :, pos % 64] = kr
        c.q = torch.full((1, 8, 128), step, dtype=torch.bfloat16)
        c.check(*decode(c, 1), [0, 1])


@pytest.mark.parametrize("scale", [1.0, 0.01, 3.5])
def test_explicit_scale(scale):
    c = case("ragged", 1, 1, seed=9)
    c.check(*decode(c, 1, scale=scale), cu_of([1] * len(c.lens)), scale=scale)


@pytest.mark.parametrize("q_len", [1, 6])
def test_same_bits(q_len):
    """A repeated step, permuted blocks, heads outside the blocks, K and V side by side, without lse."""
    c = case("many", 3, q_len, seed=11)
    d = c.device()
    out, lse = decode(c, q_len, d)
    for _ in range(3):
        o2, l2 = decode(c, q_len, d)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    perm = torch.randperm(c.blocks)
    e = dict(d, bt=torch.where(d["bt"] >= 0, torch.argsort(perm).int().cuda()[d["bt"].long().clamp(min=0)], d["bt"]),
             k=d["k"][perm.cuda()].contiguous(), v=d["v"][perm.cuda()].contiguous())
    heads = dict(d, k=d["k"].transpose(0, 1).contiguous().transpose(0, 1), v=d["v"].transpose(0, 1).contiguous().transpose(0, 1))
    both = torch.stack([d["k"], d["v"]], 1)
    for x in (e, heads, dict(d, k=both[:, 0], v=both[:, 1])):
        o2, l2 = decode(c, q_len, x)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    plan = hpc.hpc_decode_kv4_plan_create(len(c.lens), q_len, hpc.hpc_device_sm_count(), 8 * c.hkv)
    o2 = torch.empty_like(out)
    hpc.hpc_decode_kv4_attn(d["q"].view(out.shape), d["k"], d["v"], d["bt"], d["sl"], plan, o2, k_scale=c.ks, v_scale=c.vs)
    assert torch.equal(out, o2)


@pytest.mark.parametrize("q_len", [1, 3])
def test_strided_q_out_lse(q_len):
    c = case("edges", 2, q_len, seed=12)
    d, n = c.device(), len(c.lens)
    out, lse = decode(c, q_len, d)
    q = torch.full((n, q_len + 1, 20, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    o = torch.full((n, q_len + 2, 18, 144), 5.0, dtype=torch.bfloat16, device="cuda")
    s = torch.full((n, q_len, 16, 2), 5.0, device="cuda")
    q[:, 1:, 2:18, :128] = d["q"].view(n, q_len, 16, 128)
    views = q[:, 1:, 2:18, :128], o[:, :q_len, 1:17, 8:136], s[..., 1]
    if q_len == 1:
        views = [x[:, 0] for x in views]
    decode(c, q_len, dict(d, q=views[0]), out=views[1], lse=views[2])
    assert torch.equal(views[1], out) and torch.equal(views[2], lse)
    o[:, :q_len, 1:17, 8:136] = 5.0
    assert (o == 5).all() and (s[..., 0] == 5).all()


def test_nan_stays_in_its_sequence_and_head():
    c = Paged([200, 300, 130], hkv=2, seed=13, q_rows=3)
    good, lse = decode(c, 1)
    ids = c.table[1].long()
    c.k[ids[1], 1, 5, 64:] = 0x7F      # sequence 1, head 1: a key it sees
    c.v[ids[2], 0, 3, 66] = 0x7F       # head 0: 16 elements of a value
    out, l2 = decode(c, 1)
    same = [0, 2]
    assert torch.equal(out[same], good[same]) and torch.equal(l2[same], lse[same])
    assert torch.isnan(out[1, 8:]).all() and torch.isnan(l2[1, 8:]).all()
    assert torch.isnan(out[1, :8, 32:48]).all() and torch.isfinite(out[1, :8, :32]).all() and torch.equal(l2[1, :8], lse[1, :8])


@pytest.mark.parametrize("q_len", [1, 4])
def test_bad_blocks_read_zeros(q_len):
    c = case("ragged", 2, q_len, seed=14)
    d = c.device()
    bt = d["bt"].clone()
    bt[2, 3], bt[2, 4], bt[4, 1] = -1, c.blocks, 2 ** 31 - 1
    plan = hpc.hpc_decode_kv4_plan_create(len(c.lens), q_len, hpc.hpc_device_sm_count(), 16)
    out, lse = decode(c, q_len, dict(d, bt=bt), plan=plan)
    assert hpc.hpc_decode_plan_status(plan) == 2  # HPC_DEVCHK_BAD_BLOCK
    for b, t in ((2, 3), (2, 4), (4, 1)):
        for r in c.rows[b]:
            r[64 * t:64 * t + 64] = 0
    c.check(out, lse, cu_of([q_len] * len(c.lens)))
    short = bt[:, :30].contiguous()
    decode(c, q_len, dict(d, bt=short), plan=plan)
    assert hpc.hpc_decode_plan_status(plan) == 2 | 4  # HPC_DEVCHK_TABLE_TOO_SHORT
    out, lse = decode(c, q_len, d, plan=plan)  # and the plan serves on
    assert hpc.hpc_decode_plan_status(plan) == 0 and torch.isfinite(out).all()


@pytest.mark.parametrize("q_len", [1, 2])
def test_bad_lengths(q_len):
    c = case("ragged", 1, q_len, seed=15)
    d = c.device()
    plan = hpc.hpc_decode_kv4_plan_create(len(c.lens), q_len, hpc.hpc_device_sm_count(), 8)
    for n in (-1, -2 ** 31, 2 ** 31 - 1):
        sl = d["sl"].clone()
        sl[3] = n
        out, lse = decode(c, q_len, dict(d, sl=sl), plan=plan)
        assert hpc.hpc_decode_plan_status(plan) == 1  # HPC_DEVCHK_BAD_LENGTH
        assert (out == 0).all() and (lse == -float("inf")).all()
    c.check(*decode(c, q_len, d, plan=plan), cu_of([q_len] * len(c.lens)))
    assert hpc.hpc_decode_plan_status(plan) == 0


def test_far_offsets_in_a_large_cache():
    """Tiles behind 2^32 bytes of the cache, and a table of more than one window of ids."""
    c = Paged([2500, 90], hkv=1, seed=16, spare=0, q_rows=2)
    n = (1 << 32) // 4608 + 100
    d = c.device()
    big = {}
    for x in ("k", "v"):
        big[x] = torch.empty((n, 1, 64, 72), dtype=torch.uint8, device="cuda")
        big[x][n - c.blocks:] = d[x]
    bt = torch.where(d["bt"] >= 0, d["bt"] + (n - c.blocks), d["bt"])
    c.check(*decode(c, 1, dict(d, **big, bt=bt)), [0, 1, 2])


@pytest.mark.parametrize("q_len", [1, 2])
def test_a_very_long_sequence(q_len):
    """2^26 - 3 positions in one block's values: scores 0, so that out is the mean of V."""
    n = 2 ** 26 - 3
    tiles = (n + 63) // 64
    c = Paged([64], hkv=1, seed=17, vs=1.0, q_rows=q_len, q_scale=0.0)
    block = int(c.table[0, 0])
    table = torch.full((1, tiles), block, dtype=torch.int32, device="cuda")
    d = dict(c.device(), bt=table, sl=i32([n]))
    out, lse = decode(c, q_len, d)
    v = c.values(0)[1][0]
    for t in range(q_len):
        m = n - (q_len - 1 - t)
        ref = (v.sum(0) * (m // 64) + v[:m % 64].sum(0)) / m
        got = out.view(q_len, 8, 128)[t].double()
        # sums of like terms in fp32 lose up to their number of steps; 2^12 tiles a warp, of 4 steps each
        assert ((got - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -9 * v.abs().mean(0)).all()
        assert ((lse.view(q_len, 8)[t].double() - torch.log(torch.tensor(float(m)).double().cuda())).abs() <= 2.0 ** -9).all()


def test_4096_sequences():
    c = Paged([i % 97 for i in range(4096)], hkv=1, q_rows=4096, seed=18)
    c.check(*decode(c, 1), cu_of([1] * 4096))


@pytest.mark.parametrize("q_len", [1, 3])
def test_graph_follows_the_lengths(q_len):
    """One captured step, replayed as the lengths change; a plan of more than the step needs."""
    lens = [700, 64, 0, 1300]
    c = Paged(lens, hkv=2, q_rows=len(lens) * q_len, seed=19)
    d = c.device()
    plan = hpc.hpc_decode_kv4_plan_create(9, 8, hpc.hpc_device_sm_count(), 64)
    out, lse = decode(c, q_len, d, plan=plan)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode(c, q_len, d, plan=plan, out=out, lse=lse)
    rows = c.rows
    for cut in ([0, 0, 0, 0], [1, 63, 0, 500], [690, 64, 0, 1299], [700, 64, 0, 1300]):
        c.lens = [n - x for n, x in zip(lens, cut)]
        c.rows = [(k[:n], v[:n]) for (k, v), n in zip(rows, c.lens)]
        d["sl"].copy_(i32(c.lens))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, lse, cu_of([q_len] * len(lens)))
    assert hpc.hpc_decode_plan_status(plan) == 0


def test_two_plans_on_two_streams():
    a, b = case("many", 2, 1, seed=20), case("ragged", 2, 5, seed=21)
    da, db = a.device(), b.device()
    pa = hpc.hpc_decode_kv4_plan_create(90, 1, hpc.hpc_device_sm_count(), 16)
    pb = hpc.hpc_decode_kv4_plan_create(90, 5, hpc.hpc_device_sm_count(), 16)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        with torch.cuda.stream(sa):
            x = decode(a, 1, da, plan=pa)
        with torch.cuda.stream(sb):
            y = decode(b, 5, db, plan=pb)
        got.append((x, y))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x[0], got[0][0][0]) and torch.equal(y[0], got[0][1][0])
    a.check(*got[-1][0], cu_of([1] * 90))
    b.check(*got[-1][1], cu_of([5] * len(b.lens)))


def test_different_steps_queued_on_one_plan():
    plan = hpc.hpc_decode_kv4_plan_create(90, 8, hpc.hpc_device_sm_count(), 64)
    steps = [(case(n, h, t, seed=22), t) for n, h, t in (("many", 8, 1), ("long", 1, 3), ("edges", 2, 8), ("long", 1, 1), ("one", 8, 2),
                                                         ("empty", 1, 4), ("ragged", 3, 5))]
    devs = [c.device() for c, _ in steps]
    torch.cuda.synchronize()
    got = [decode(c, t, d, plan=plan) for (c, t), d in zip(steps, devs)]
    assert hpc.hpc_decode_plan_status(plan) == 0
    for (c, t), g in zip(steps, got):
        c.check(*g, cu_of([t] * len(c.lens)))


CHILD = r"""
import json, os, sys, time
sys.path.insert(0, sys.argv[1])
import torch
import paged_gqa_decode_hpc_gb300 as hpc
from tests.kv4_util import Paged, cu_of, decode
hpc.load_library()
res = []
for q_len in (1, 4):
    c = Paged([3000, 64, 700], hkv=2, q_rows=3 * q_len, seed=1)
    d = c.device()
    plan = hpc.hpc_decode_kv4_plan_create(3, q_len, hpc.hpc_device_sm_count(), 16)
    os.environ["HPC_DECODE_TEST_WITHHOLD_COPIES"] = "1"
    t0 = time.time()
    decode(c, q_len, d, plan=plan)
    bits = hpc.hpc_decode_plan_status(plan)
    seconds = time.time() - t0
    os.environ["HPC_DECODE_TEST_WITHHOLD_COPIES"] = "0"
    c.check(*decode(c, q_len, d, plan=plan), cu_of([q_len] * 3))
    res.append([bits, seconds, hpc.hpc_decode_plan_status(plan)])
print(json.dumps(res))
"""


def test_copies_that_never_come():
    """The waits give up, the step reports it, and the plan serves the next step."""
    env = dict(os.environ, HPC_DECODE_WAIT_LIMIT_MS="200")
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    for bits, seconds, after in json.loads(r.stdout.strip().splitlines()[-1]):
        assert bits & 8 and after == 0 and seconds < 60


def test_refusals_that_need_a_device():
    c = case("one", 1, 1)
    d = c.device()
    plan = hpc.hpc_decode_kv4_plan_create(1, 1, 152, 8)
    out = torch.empty(1, 8, 128, dtype=torch.bfloat16, device="cuda")

    def refused(**kw):
        a = dict(q=d["q"], k_cache=d["k"], v_cache=d["v"], block_table=d["bt"], seq_lens=d["sl"], plan=plan, out=out)
        with pytest.raises(hpc.HpcError) as e:
            hpc.hpc_decode_kv4_attn(**{**a, **kw}, stream=0)
        return e.value.status
    two = torch.zeros(1, 2, 8, 128, dtype=torch.bfloat16, device="cuda")
    assert refused(q=two, out=torch.empty_like(two)) == hpc.HPC_ERR_INVALID_ARG  # more tokens than the plan's
    assert refused(q=out) == hpc.HPC_ERR_INVALID_ARG                             # out overlaps q
    assert refused(lse=two.view(torch.float32)[0, 0, :, :1].t()[:, :8], q=two[:, 0]) == hpc.HPC_ERR_INVALID_ARG
    assert refused(seq_lens=c.table[0, :1]) == hpc.HPC_ERR_INVALID_ARG           # a tensor of the CPU
    cpu = dict(q=c.q, k_cache=c.k, v_cache=c.v, block_table=c.table, seq_lens=i32(c.lens, "cpu"), out=c.q.clone())
    assert refused(**cpu) == hpc.HPC_ERR_INVALID_ARG                             # all of them
    other = hpc.hpc_decode_plan_create(1, 152, 8)
    assert refused(plan=other) == hpc.HPC_ERR_INVALID_ARG
    with pytest.raises(hpc.HpcError):
        hpc.hpc_decode_plan_export(plan)
    bf = torch.zeros(2, 1, 64, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(hpc.HpcError):
        hpc.hpc_decode_step(d["q"], bf, bf, d["bt"], d["sl"], plan, 152, out)
    with pytest.raises(hpc.HpcError):
        hpc.hpc_decode_prefix_attn(d["q"], bf, bf, d["bt"], d["sl"], d["sl"], plan, out)
