"""What only a step of several new tokens can get wrong: rows of q of very different sizes, strides and orders of q and
out, more sequences than one warp plans, pieces of every length, and that nothing is allocated."""
import json
import os
import subprocess
import sys

import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from tests.kv4_util import Paged, cu_of, decode, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


@pytest.mark.parametrize("q_len", [2, 3, 8])
def test_rows_of_very_different_sizes(q_len):
    """Each row of q has a power of two of its own: small rows beside large ones keep their bits."""
    c = Paged([300, 70], hkv=1, q_rows=2 * q_len, seed=41, q_scale=6.0, ks=0.5)
    big = torch.rand(c.q.shape[:2], generator=torch.Generator().manual_seed(1)) < 0.3
    c.q[big] = c.q[big] * 2.0 ** 70
    c.check(*decode(c, q_len), cu_of([q_len] * 2))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("q_len", [2, 7])
def test_a_row_that_is_not_finite_spoils_no_other(q_len, value):
    c = Paged([500, 129], hkv=2, q_rows=2 * q_len, seed=42)
    want = decode(c, q_len)
    c.q[1, 3, 5] = value
    got = decode(c, q_len)
    other = torch.ones(2, q_len, 16, dtype=torch.bool, device="cuda")
    other[0, 1, 3] = False
    for a, b in zip(got, want):
        a, b = (x.view(other.shape + x.shape[3:]) for x in (a, b))
        assert torch.equal(a[other], b[other]) and a[~other].isnan().any()


@pytest.mark.parametrize("q_len", [2, 4, 8])
def test_orders_of_q_and_out(q_len):
    """q and out with tokens outermost, or heads of a KV head apart; one token's q for all sequences and tokens."""
    n = 3
    c = Paged([200, 65, 900], hkv=2, q_rows=n * q_len, seed=43)
    d = c.device()
    want, lse = decode(c, q_len, d)
    q = d["q"].view(n, q_len, 16, 128)
    moved = q.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.full((q_len, n, 16, 128), float("nan"), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    wide = torch.full((n, q_len, 16, 136), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[..., :128] = q
    for x, o in ((moved, out), (wide[..., :128], torch.full_like(wide, float("nan"))[..., 8:])):
        got, l = decode(c, q_len, dict(d, q=x), out=o)
        assert torch.equal(got, want) and torch.equal(l, lse)
    one = q[:1, :1].expand(n, q_len, 16, 128)
    a = decode(c, q_len, dict(d, q=one.contiguous()))
    b = decode(c, q_len, dict(d, q=one))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_results_that_overlap_are_refused():
    c = Paged([200, 65, 900], hkv=1, q_rows=9, seed=43)
    d, shape = c.device(), (3, 3, 8, 128)
    flat = torch.zeros(9 * 8 * 128, dtype=torch.bfloat16, device="cuda")
    for strides in ((8 * 128, 8 * 128, 128, 1), (0, 8 * 128, 128, 1), (3 * 8 * 128, 8 * 128, 0, 1), (2 * 8 * 128, 8 * 128, 128, 1)):
        with pytest.raises(hpc.HpcError, match="out overlap") as e:
            decode(c, 3, d, out=flat.as_strided(shape, strides))
        assert e.value.status == hpc.HPC_ERR_INVALID_ARG
    for lse in (torch.zeros(3, 3, 1, device="cuda").expand(3, 3, 8), torch.zeros(3, 1, 8, device="cuda").expand(3, 3, 8)):
        with pytest.raises(hpc.HpcError, match="lse overlap"):
            decode(c, 3, d, lse=lse)


@pytest.mark.parametrize("seqs", [257, 800, 4096])
def test_more_sequences_than_a_warp_plans(seqs):
    c = Paged([(i * 37) % 131 for i in range(seqs)], hkv=1, q_rows=2 * seqs, seed=44)
    c.check(*decode(c, 2), cu_of([2] * seqs))


@pytest.mark.parametrize("q_len", [2, 3, 6, 8])
@pytest.mark.parametrize("sms", [1, 3, 31, 152])
def test_pieces_of_every_length(q_len, sms):
    """Batches whose pieces begin and end anywhere, one after another on one plan, each twice for its bits."""
    g = torch.Generator().manual_seed(10 * q_len + sms)
    plan = hpc.hpc_decode_kv4_plan_create(12, q_len, sms, 16)
    for it in range(6):
        n = int(torch.randint(1, 13, (), generator=g))
        top = [65, 130, 700, 2500][it % 4]
        lens = torch.randint(0, top, (n,), generator=g).tolist()
        c = Paged(lens, hkv=2, q_rows=n * q_len, seed=it)
        d = c.device()
        a, b = decode(c, q_len, d, plan=plan), decode(c, q_len, d, plan=plan)
        assert all(torch.equal(x.isnan(), y.isnan()) and torch.equal(x.nan_to_num(), y.nan_to_num()) for x, y in zip(a, b))
        c.check(*a, cu_of([q_len] * n))
        assert hpc.hpc_decode_plan_status(plan) == 0


def test_free_memory_stays():
    calls = []
    for q_len in (1, 2, 4, 6, 8):
        c = Paged([3000, 1, 500], hkv=2, q_rows=3 * q_len, seed=45)
        d, plan = c.device(), hpc.hpc_decode_kv4_plan_create(3, q_len, hpc.hpc_device_sm_count(), 16)
        shape = (3, 16, 128) if q_len == 1 else (3, q_len, 16, 128)
        out, lse = torch.empty(shape, dtype=torch.bfloat16, device="cuda"), torch.empty(shape[:-1], device="cuda")
        calls.append(lambda d=d, plan=plan, out=out, lse=lse, shape=shape: hpc.hpc_decode_kv4_attn(
            d["q"].view(shape), d["k"], d["v"], d["bt"], d["sl"], plan, out, lse))
        cu, o = i32(cu_of([q_len] * 3)), torch.empty_like(d["q"])
        sl = i32([3000, 8, 500])
        calls.append(lambda d=d, sl=sl, cu=cu, o=o: hpc.hpc_extend_kv4_attn(d["q"], d["k"], d["v"], d["bt"], sl, cu, o))
    rope, n = hpc.hpc_rope_init(), 700
    rows = [torch.zeros(n, h, 128, dtype=torch.bfloat16, device="cuda") for h in (16, 2, 2)]
    caches = [torch.zeros(11, 2, 64, 72, dtype=torch.uint8, device="cuda") for _ in range(2)]
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    calls.append(lambda: hpc.hpc_rope_kv4_write(*rows, at, at, rope, rows[0], *caches))
    for call in calls:
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="global"):
        for call in calls:
            call()
    graph.replay()
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    for call in calls[::-1] + calls:
        call()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == before


def test_rows_of_very_different_sizes_in_a_prompt():
    c = Paged([300, 70], hkv=1, q_rows=170, seed=46, q_scale=6.0, ks=0.5)
    big = torch.rand(c.q.shape[:2], generator=torch.Generator().manual_seed(2)) < 0.3
    c.q[big] = c.q[big] * 2.0 ** 70
    d, cu = c.device(), cu_of([100, 70])
    out, lse = torch.empty_like(d["q"]), torch.empty(170, 8, device="cuda")
    hpc.hpc_extend_kv4_attn(d["q"], d["k"], d["v"], d["bt"], d["sl"], i32(cu), out, lse, k_scale=c.ks, v_scale=c.vs)
    c.check(out, lse, cu)


def test_one_token_with_large_scores():
    """The maximum's probability is 1 whatever the scores' size (one power of two for the KV head's rows)."""
    c = Paged([300, 70, 5000], hkv=2, q_rows=3, seed=47, q_scale=2.0 ** 70, ks=0.5)
    c.check(*decode(c, 1), cu_of([1] * 3))


@pytest.mark.parametrize("new,old", [([1, 2, 16], [0, 63, 64]), ([5, 300], [8000, 0]), ([16] * 4, [64 * i for i in range(4)]),
                                     ([700, 1, 90], [100, 6000, 5])])
@pytest.mark.parametrize("hkv", [1, 8])
def test_chunks_whose_rows_see_few_or_many_tiles(new, old, hkv):
    """Both kinds of CTA: two query tiles, and one whose keys two chains share (one tile, an odd one, none of a chain's
    keys visible to some rows)."""
    c = Paged([n + o for n, o in zip(new, old)], hkv=hkv, q_rows=sum(new), seed=48, q_scale=4.0)
    d, cu = c.device(), cu_of(new)
    for _ in range(2):
        out, lse = torch.full_like(d["q"], float("nan")), torch.full(d["q"].shape[:2], float("nan"), device="cuda")
        hpc.hpc_extend_kv4_attn(d["q"], d["k"], d["v"], d["bt"], d["sl"], i32(cu), out, lse, k_scale=c.ks, v_scale=c.vs)
        c.check(out, lse, cu)


CHILD = r"""
import json, os, sys, time
sys.path.insert(0, sys.argv[1])
import torch
import paged_gqa_decode_hpc_gb300 as hpc
from tests.kv4_util import Paged, cu_of, i32
hpc.load_library()
res = []
for new, old in (([3, 20], [500, 0]), ([700, 900], [100, 0])):
    c = Paged([n + o for n, o in zip(new, old)], hkv=8, q_rows=sum(new), seed=1)
    d, cu = c.device(), cu_of(new)
    out, lse, err = torch.empty_like(d["q"]), torch.empty(d["q"].shape[:2], device="cuda"), i32([0])
    call = lambda: hpc.hpc_extend_kv4_attn(d["q"], d["k"], d["v"], d["bt"], d["sl"], i32(cu), out, lse, device_error=err,
                                           k_scale=c.ks, v_scale=c.vs)
    os.environ["HPC_DECODE_TEST_WITHHOLD_COPIES"] = "1"
    t0 = time.time()
    call()
    bits = err.item()
    seconds = time.time() - t0
    os.environ["HPC_DECODE_TEST_WITHHOLD_COPIES"] = "0"
    err.zero_()
    call()
    c.check(out, lse, cu)
    res.append([bits, seconds, err.item()])
print(json.dumps(res))
"""


def test_copies_of_a_prompt_that_never_come():
    """The waits give up, the call reports it, and the next one is served."""
    env = dict(os.environ, HPC_DECODE_WAIT_LIMIT_MS="100")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CHILD, root], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    for bits, seconds, after in json.loads(r.stdout.strip().splitlines()[-1]):
        assert bits & 8 and after == 0 and seconds < 60
