"""hpc_decode_prefix_attn against the fp64 decode oracle, which reads every
sequence through its own block table row.

Tolerances, derived. Scores and row sums are fp32; a score is off by at most
2^-15 at these sizes (128 fp32 products and sums of magnitude below 2^6, the
scale, the exponential's 2^-22), so a probability is within 2^-14 relative.
Probabilities are rounded to bf16 (2^-8) for a bf16 cache and to f16 (2^-11) for
e4m3 before the P V product, which accumulates in fp32; with A = sum p |v| / sum p
that moves the output by at most (2^-8 or 2^-11, plus 2^-14) A. f16 also loses
at most 2^-25 per key below its normal range, with row sums of at least 2^-8:
keys 2^-17 max |v|, below 2^-11 A here. The output's own rounding to bf16 adds
2^-8 |out|. lse: 2^-14, and 2^-22 relative for the logarithm's sum."""
import os

import numpy as np
import pytest
import torch

import oracle
import paged_gqa_decode_hpc_gb300 as hpc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


class Case:
    """Groups of sequences over one cache; slots past every sequence's end, unused blocks and table entries hold
    NaN or ids that no call may read."""

    def __init__(self, groups, q_len=1, hkv=2, fp8=False, seed=0, q_scale=1.0, token_major=False, declared=None):
        """groups: [(prefix length, [length of each sequence])]; declared: the prefix lengths passed to the call."""
        g = torch.Generator().manual_seed(seed)
        self.T, self.hkv, self.fp8 = q_len, hkv, fp8
        self.prefixes = [p for p, _ in groups] if declared is None else declared
        self.lens = [n for _, lens in groups for n in lens]
        self.cu = [0]
        shared, own = [], []
        for p, lens in groups:
            self.cu.append(self.cu[-1] + len(lens))
            shared.append(p // 64)
            own += [max(0, -(-n // 64) - p // 64) for n in lens]
        total = sum(shared) + sum(own) + 2
        perm = torch.randperm(total, generator=g).tolist()
        self.blocks, width = total, max([1] + [-(-n // 64) for n in self.lens])
        self.table = torch.full((len(self.lens), width), -1, dtype=torch.int32)
        b = 0
        for s, (p, lens) in zip(shared, groups):
            ids, perm = perm[:s], perm[s:]
            for n in lens:
                k = -(-n // 64)
                row = ids[:k] + perm[:max(0, k - s)]
                perm = perm[max(0, k - s):]
                self.table[b, :len(row)] = torch.tensor(row, dtype=torch.int32)
                b += 1
        shape = (total, hkv, 64, 128)
        used = torch.zeros(total, 64, dtype=torch.bool)
        for row, n in zip(self.table.tolist(), self.lens):
            for j in range(-(-n // 64)):
                used[row[j], :min(64, n - 64 * j)] = True
        hide = ~used[:, None, :, None].expand(shape)
        if fp8:
            x = torch.randint(0, 256, (2,) + shape, generator=g).to(torch.uint8)
            x[(x & 0x7F) >= 0x50] &= 0x8F  # |value| <= 8 (code 0x50)
            x[hide.expand(2, *shape)] = 0x7F  # NaN
            self.scales = (0.21, 0.17)
        else:
            x = torch.randn((2,) + shape, generator=g).to(torch.bfloat16)
            x[hide.expand(2, *shape)] = float("nan")
            self.scales = (1.0, 1.0)
        self.k, self.v = x[0], x[1]
        self.token_major = token_major
        qs = (len(self.lens), 8 * hkv, 128) if q_len == 1 else (len(self.lens), q_len, 8 * hkv, 128)
        self.q = (torch.randn(qs, generator=g) * q_scale).to(torch.bfloat16)
        self.scale = 128 ** -0.5

    def reference(self):
        q = self.q if self.T > 1 else self.q[:, None]
        lens = torch.tensor(self.lens, dtype=torch.int32)
        kw = dict(num_kv_heads=self.hkv, softmax_scale=self.scale, kv_is_fp8=self.fp8, k_scale=self.scales[0],
                  v_scale=self.scales[1])
        out, lse = oracle.paged_decode_multi(q, self.k, self.v, self.table, lens, **kw)
        size, _ = oracle.paged_decode_multi(q, self.k, self.v & 0x7F if self.fp8 else self.v.abs(), self.table, lens, **kw)
        return [x.reshape(self.q.shape) for x in (out, size)] + [lse.reshape(self.q.shape[:-1])]

    def device(self):
        d = {"q": self.q.cuda(), "bt": self.table.cuda(), "sl": torch.tensor(self.lens, dtype=torch.int32).cuda(),
             "cu": torch.tensor(self.cu, dtype=torch.int32).cuda(),
             "pl": torch.tensor(self.prefixes, dtype=torch.int32).cuda()}
        for n in "kv":
            x = getattr(self, n).cuda()
            d[n] = x.transpose(1, 2).contiguous().transpose(1, 2) if self.token_major else x
        return d

    def run(self, d=None, sms=None, plan=None, expect=0, out=None, lse=None, stream=None, scale=None, **kw):
        d = d or self.device()
        sms = sms or hpc.hpc_device_sm_count()
        p = plan or hpc.hpc_decode_prefix_plan_create(len(self.lens), self.T, sms, 8 * self.hkv)
        out = torch.full(self.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
        lse = torch.full(self.q.shape[:-1], float("nan"), device="cuda") if lse is None else lse
        torch.cuda.synchronize()
        hpc.hpc_decode_prefix_attn(d["q"], d["k"], d["v"], d["bt"], d["sl"], d["pl"], p, out, lse,
                                   **{"cu_groups": d["cu"], **kw}, k_scale=self.scales[0], v_scale=self.scales[1],
                                   stream=stream, softmax_scale=scale)
        assert hpc.hpc_decode_plan_status(p) == expect
        return out, lse

    def check(self, got=None, **kw):
        out, lse = self.run(**kw) if got is None else got
        ref, size, ref_lse = self.reference()
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        tol = 2.0 ** -8 * np.abs(ref) + ((2 * 2.0 ** -11 if self.fp8 else 2.0 ** -8) + 2.0 ** -14) * size
        assert np.isfinite(out).all()
        off = np.abs(out - ref) - tol
        assert (off <= 0).all(), f"{(off > 0).sum()} outputs off, worst {off.max():.2e} at {np.unravel_index(off.argmax(), off.shape)}"
        seen = np.isfinite(ref_lse)
        assert np.array_equal(lse[~seen], ref_lse[~seen])  # -inf
        assert (np.abs(lse[seen] - ref_lse[seen]) <= 2.0 ** -14 + 2.0 ** -22 * np.abs(ref_lse[seen])).all()


SHAPES = {
    "one sequence": [(100, [300])],
    "two": [(128, [130, 200])],
    "not whole blocks": [(200, [201, 260, 330])],
    "17 pairs": [(192, [193 + 7 * i for i in range(17)])],
    "33 pairs": [(640, [640 + 3 * i for i in range(1, 34)])],
    "three tiles": [(320, [330 + i for i in range(70)])],
    "groups": [(64, [70, 64, 190]), (0, [5]), (500, [501] * 20), (1000, [1100, 1700]), (70, [])],
    "no prefix": [(0, [1, 64, 65, 700, 3])],
    "short and empty": [(256, [0, 300, 0, 257, 0]), (128, [0, 0]), (128, [0, 190])],
    "shorter than the prefix": [(512, [100, 600, 513]), (512, [64, 600]), (512, [63, 700])],
    "prefix only": [(256, [256, 256, 256])],
    "long": [(6000, [6001, 6100, 7000])],
}


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hkv", [1, 8])
def test_shapes(name, fp8, hkv):
    Case(SHAPES[name], hkv=hkv, fp8=fp8, seed=len(name)).check()


@pytest.mark.parametrize("q_len", [2, 3, 5, 8])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", ["one sequence", "not whole blocks", "groups", "short and empty", "17 pairs"])
def test_several_new_tokens(q_len, fp8, name):
    groups = [(p, [n + (q_len if n else 0) for n in lens]) for p, lens in SHAPES[name]]
    Case(groups, q_len=q_len, fp8=fp8, seed=q_len).check()


def test_new_tokens_that_see_nothing():
    # sequences shorter than q_len, and lengths that cut into the shared blocks
    Case([(128, [3, 1, 200]), (64, [64, 67, 5]), (64, [71, 72])], q_len=8, seed=1).check()


@pytest.mark.parametrize("sms", [1, 2, 3, 7, 40, 151, 400])
@pytest.mark.parametrize("fp8", [False, True])
def test_any_number_of_ctas(sms, fp8):
    Case([(900, [950, 1000, 1600]), (300, [310] * 18), (0, [129])], hkv=2, fp8=fp8, seed=sms).check(sms=sms)


@pytest.mark.parametrize("hkv", [2, 4, 16])
def test_heads(hkv):
    Case([(256, [300, 400, 257])], hkv=hkv, seed=hkv).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_token_major_cache_and_strided_views(fp8):
    c = Case([(200, [230, 300, 1000])], q_len=2, hkv=2, fp8=fp8, seed=3, token_major=True)
    d = c.device()
    d["q"] = torch.zeros(3, 2, 32, 128, dtype=torch.bfloat16, device="cuda")[:, :, 8:24].copy_(d["q"])
    d["bt"] = torch.full((3, 40), 10**6, dtype=torch.int32, device="cuda")[:, 5:5 + c.table.shape[1]].copy_(d["bt"])
    wide = torch.full((3, 3, 20, 136), 5.0, dtype=torch.bfloat16, device="cuda")
    wide_lse = torch.full((3, 2, 40), 5.0, device="cuda")
    got = c.run(d, out=wide[:, :2, 2:18, :128], lse=wide_lse[:, :, ::2][:, :, :16])
    c.check(got)
    wide[:, :2, 2:18, :128] = 5.0
    wide_lse[:, :, ::2][:, :, :16] = 5.0
    assert (wide == 5).all() and (wide_lse == 5).all()


def test_sharp_and_flat_softmax():
    for q_scale in (0.0, 8.0):
        Case([(1000, [1100, 1300] + [1001] * 16)], seed=4, q_scale=q_scale).check()
        Case([(1000, [1100, 1300] + [1001] * 16)], seed=4, q_scale=q_scale, fp8=True).check()


def test_explicit_scale_one_group_and_no_lse():
    c = Case([(320, [400, 500, 321])], seed=5)
    c.scale = 0.05
    c.check(scale=0.05, cu_groups=None)
    d, plan = c.device(), hpc.hpc_decode_prefix_plan_create(3, 1, 152, 16)
    out = torch.zeros_like(d["q"])
    hpc.hpc_decode_prefix_attn(d["q"], d["k"], d["v"], d["bt"], d["sl"], d["pl"], plan, out, softmax_scale=0.05)
    assert torch.equal(out, c.run(d, scale=0.05, cu_groups=None)[0])


def test_declared_prefix_beyond_the_sequences_or_negative():
    groups = [(256, [257, 300, 260])]
    Case(groups, seed=6, declared=[10**9]).check()   # cut to what every sequence sees: still the same blocks
    c = Case(groups, seed=6, declared=[-5])
    c.check(c.run(expect=hpc.HPC_DEVCHK_BAD_LENGTH))


@pytest.mark.parametrize("cu", [[0, 2, 1, 4], [1, 2, 3, 4], [0, 1, 2, 3], [0, 1, 2, 9], [0, -1, 2, 4]])
def test_groups_that_are_no_partition(cu):
    c = Case([(64, [100, 90]), (64, [80]), (0, [70])], seed=7)
    c.cu = cu
    c.check(c.run(expect=hpc.HPC_DEVCHK_BAD_LENGTH))


def test_bad_lengths_and_blocks():
    c = Case([(128, [200, 190, 130])], seed=8)
    d = c.device()
    d["sl"][1] = -7
    c.lens[1] = 0
    c.check(c.run(d, expect=hpc.HPC_DEVCHK_BAD_LENGTH))
    c = Case([(128, [200, 190, 130])], seed=9)
    for where, bad, bit in (((0, 1), c.blocks, hpc.HPC_DEVCHK_BAD_BLOCK), ((2, 2), -1, hpc.HPC_DEVCHK_BAD_BLOCK)):
        d = c.device()
        d["bt"][where] = bad
        out, _ = c.run(d, expect=bit)
        assert torch.isfinite(out.float()).all()
        assert torch.equal(out[1], c.run()[0][1]) == (where[0] == 2)  # a shared block is everyone's
    d = c.device()
    d["sl"][0] = 64 * d["bt"].shape[1] + 10
    c.run(d, expect=hpc.HPC_DEVCHK_TABLE_TOO_SHORT)


def test_same_bits_again_and_whatever_the_blocks():
    c = Case(SHAPES["three tiles"], hkv=8, seed=10)
    d, plan = c.device(), hpc.hpc_decode_prefix_plan_create(len(c.lens), 1, 152, 64)
    first = c.run(d, plan=plan)
    for _ in range(3):
        again = c.run(d, plan=plan)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    perm = torch.randperm(c.blocks, device="cuda")
    moved = dict(d, k=torch.empty_like(d["k"]), v=torch.empty_like(d["v"]))
    moved["k"][perm], moved["v"][perm] = d["k"], d["v"]
    moved["bt"] = torch.where(d["bt"] >= 0, perm.int()[d["bt"].clamp(min=0).long()], d["bt"])
    again = c.run(moved, plan=plan)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_one_plan_for_different_steps():
    plan = hpc.hpc_decode_prefix_plan_create(80, 4, 152, 64)
    for name, hkv, q_len, fp8 in (("three tiles", 8, 1, False), ("two", 1, 4, True), ("groups", 2, 3, False),
                                  ("one sequence", 8, 1, True), ("short and empty", 4, 2, False)):
        groups = [(p, [n + (q_len if n else 0) for n in lens]) for p, lens in SHAPES[name]]
        c = Case(groups, hkv=hkv, q_len=q_len, fp8=fp8, seed=11)
        c.check(c.run(plan=plan))


def test_captured_steps_follow_the_device_lengths():
    """Two captured graphs with plans of their own on two streams; between replays the lengths and prefixes on the
    device change."""
    s = [torch.cuda.Stream() for _ in range(2)]
    cases = [Case([(320, [400 + 9 * i for i in range(20)])], hkv=2, seed=12, fp8=bool(i)) for i in range(2)]
    ds = [c.device() for c in cases]
    plans = [hpc.hpc_decode_prefix_plan_create(20, 1, 152, 16) for _ in cases]
    outs = [c.run(d, plan=p, stream=st) for c, d, p, st in zip(cases, ds, plans, s)]
    graphs = [torch.cuda.CUDAGraph() for _ in cases]
    for c, d, p, st, (out, lse), g in zip(cases, ds, plans, s, outs, graphs):
        with torch.cuda.graph(g, stream=st):
            hpc.hpc_decode_prefix_attn(d["q"], d["k"], d["v"], d["bt"], d["sl"], d["pl"], p, out, lse,
                                       cu_groups=d["cu"], k_scale=c.scales[0], v_scale=c.scales[1])
    for change in range(3):
        for c, d in zip(cases, ds):
            c.lens = [max(0, n - 37 * change) for n in c.lens]
            c.prefixes = [[320], [100], [10**6]][change]
            d["sl"].copy_(torch.tensor(c.lens, dtype=torch.int32))
            d["pl"].copy_(torch.tensor(c.prefixes, dtype=torch.int32))
        for out, lse in outs:
            out.fill_(float("nan"))
            lse.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, st in zip(graphs, s):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for c, got, p in zip(cases, outs, plans):
            assert hpc.hpc_decode_plan_status(p) == 0
            c.check(got)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prefix,lens,hkv,q_len", [
    (20000, [20010, 20300], 1, 1),           # a pair's states come from more CTAs than are listed at once
    (9000, [9003, 9100, 9500], 1, 4),
    (3000, [3001 + 5 * i for i in range(5)], 4, 1),
    (700, [701 + i for i in range(9)], 8, 1),   # eighths, quarters, halves and whole columns a CTA of the merge
    (700, [701 + i for i in range(13)], 8, 1),
    (700, [701 + i for i in range(18)], 8, 1),
    (700, [701 + i for i in range(29)], 8, 1),
    (700, [701 + i for i in range(47)], 8, 1),
    (700, [701 + i for i in range(48)], 8, 1),
])
def test_states_of_many_parts(prefix, lens, hkv, q_len, fp8):
    Case([(prefix, lens)], q_len=q_len, hkv=hkv, fp8=fp8, seed=prefix + len(lens)).check()


@pytest.mark.parametrize("seqs,hkv", [(2, 1), (100, 2)])
def test_more_parts_than_the_device_has_sms(seqs, hkv):
    # states past those that a CTA of the merge lists beforehand (320 for few pairs, 64 for many)
    Case([(44000, [44001 + 3 * i for i in range(seqs)])], hkv=hkv, seed=44).check(sms=900)


def test_large_batches():
    rng = np.random.default_rng(15)
    # 4096 sequences in 700 groups, some empty, most of one or two blocks; 8 new tokens of 300 sequences
    cuts = np.sort(rng.choice(np.arange(1, 4096), 699, replace=False)).tolist()
    groups = [(int(rng.choice([0, 64, 130])), [int(x) for x in rng.integers(0, 200, b - a)])
              for a, b in zip([0] + cuts, cuts + [4096])]
    groups = [(p, [n if n == 0 or n >= p else p + n for n in lens]) for p, lens in groups]
    Case(groups, hkv=1, seed=16).check()
    Case([(192, [200 + i % 90 for i in range(200)]), (64, [72 + i for i in range(100)])], q_len=8, hkv=1, fp8=True, seed=17).check()


def test_queries_that_are_not_finite_spoil_their_rows_only():
    for fp8 in (False, True):
        c = Case([(256, [300, 260, 400])], seed=18, fp8=fp8)
        clean = c.run()[0]
        c.q[1, 3, 7] = float("nan")
        out, lse = c.run()
        bad = torch.zeros(out.shape[:2], dtype=torch.bool)
        bad[1, 3] = True
        assert torch.isnan(out[1, 3]).all() and torch.isnan(lse[1, 3])
        assert torch.equal(out.cpu()[~bad], clean.cpu()[~bad])


def test_plans_are_not_mixed():
    c = Case([(64, [100, 90])], seed=19)
    d, out = c.device(), torch.zeros(c.q.shape, dtype=torch.bfloat16, device="cuda")
    prefix = hpc.hpc_decode_prefix_plan_create(2, 1, 152, 16)
    other = hpc.hpc_decode_plan_create(2, 152, 16)
    small = [hpc.hpc_decode_prefix_plan_create(1, 1, 152, 16), hpc.hpc_decode_prefix_plan_create(2, 8, 152, 8), other]
    for plan in small:
        with pytest.raises(hpc.HpcError) as e:
            hpc.hpc_decode_prefix_attn(d["q"], d["k"], d["v"], d["bt"], d["sl"], d["pl"], plan, out)
        assert e.value.status == hpc.HPC_ERR_INVALID_ARG
    calls = [lambda: hpc.hpc_decode_step(d["q"], d["k"], d["v"], d["bt"], d["sl"], prefix, 152, out),
             lambda: hpc.hpc_decode_attn(d["q"], d["k"], d["v"], d["bt"], d["sl"], prefix, out),
             lambda: hpc.hpc_decode_plan_device(d["sl"], 152, prefix), lambda: hpc.hpc_decode_plan_update([1, 2], 152, prefix),
             lambda: hpc.hpc_decode_plan_export(prefix), lambda: hpc.hpc_decode_plan_set_timing_events(prefix)]
    for call in calls:
        with pytest.raises(hpc.HpcError):
            call()
    c.check(c.run(d, plan=prefix))


def test_agrees_with_the_decode_step():
    c = Case([(1024, [1100 + i for i in range(24)])], hkv=8, seed=13)
    d = c.device()
    # the step reads unused slots of a last block: give it a clean cache
    d["k"], d["v"] = d["k"].nan_to_num(0.0), d["v"].nan_to_num(0.0)
    out, lse = c.run(d)
    plan = hpc.hpc_decode_plan_create(24, 152, 64)
    ref, ref_lse = torch.empty_like(out), torch.empty_like(lse)
    hpc.hpc_decode_step(d["q"], d["k"], d["v"], d["bt"], d["sl"], plan, 152, ref, ref_lse)
    assert hpc.hpc_decode_plan_status(plan) == 0
    assert ((out.double() - ref.double()).norm() / ref.double().norm()).item() < 2.0 ** -7
    assert (lse - ref_lse).abs().max().item() < 1e-4


def test_copies_that_never_arrive_end_the_call():
    """The failure-path switch withholds every copy: the bounded waits run out (2 s), the status word says so and the
    same plan then serves a normal step."""
    for fp8 in (False, True):
        c = Case(SHAPES["17 pairs"], seed=14, fp8=fp8)
        plan = hpc.hpc_decode_prefix_plan_create(17, 1, 4, 16)
        os.environ["HPC_DECODE_TEST_WITHHOLD_COPIES"] = "1"
        try:
            c.run(plan=plan, expect=hpc.HPC_DEVCHK_TIMEOUT)
        finally:
            del os.environ["HPC_DECODE_TEST_WITHHOLD_COPIES"]
        c.check(c.run(plan=plan))
