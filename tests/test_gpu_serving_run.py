"""A serving loop over one paged cache, made of the calls that belong together:
block tables and slots from lengths, rotary positions with the KV write, prefill
over the table, shared-prefix decode, rejected drafts rolled back, a finished
sequence replaced. The decode step runs as a captured graph whose only inputs
are on the device.

Each stage is held to its own oracle: tables, slots and the stack word for word;
cache rows to the rotary formulas; attention to the fp64 oracle on the cache as
it is, through tables that the oracle built."""
import numpy as np
import pytest
import torch

import oracle
import paged_gqa_decode_hpc_gb300 as hpc
from oracle import block_table_ref as BT
from oracle import prologue_ref as PR
from oracle import rope_ref as RR

pytestmark = pytest.mark.gpu

HKV, HQ, WIDTH, BLOCKS = 2, 16, 12, 64
ROPE = dict(rot_dim=96, interleaved=False, base=5e5, scaling="banded", factor=8.0, original_len=8192, low=1.0, high=4.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    def __init__(self, fp8, seqs, seed):
        self.fp8, self.B, self.gen = fp8, seqs, torch.Generator(device="cuda").manual_seed(seed)
        shape = (BLOCKS, HKV, 64, 128)
        self.caches = [torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") if fp8 else
                       torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.scales = (0.02, 0.015) if fp8 else (1.0, 1.0)
        perm = torch.randperm(BLOCKS, generator=torch.Generator().manual_seed(seed)).tolist()
        self.free, self.count = _i32(perm), _i32([BLOCKS])
        self.table, self.lens = _i32([[-1] * WIDTH] * seqs), _i32([0] * seqs)
        self.err = _i32([0])
        self.rope = hpc.hpc_rope_init(**ROPE)
        self.wq, self.wk = (1 + 0.1 * torch.randn((2, 128), generator=self.gen, device="cuda")).to(torch.bfloat16)
        # the same state, held by the oracle
        self.ref = dict(free=perm, count=BLOCKS, table=self.table.tolist(), lens=[0] * seqs)
        self.rows = {}  # (block, slot) -> (k row, v row) in fp64

    def buffers(self, tokens):
        qkv = torch.randn((tokens, (HQ + 2 * HKV) * 128), generator=self.gen, device="cuda").to(torch.bfloat16)
        return dict(qkv=qkv, new=_i32([0] * self.B), cu=_i32([0] * (self.B + 1)), pos=_i32([0] * tokens),
                    slots=_i32([0] * tokens), q=torch.zeros((tokens, HQ, 128), dtype=torch.bfloat16, device="cuda"))

    def views(self, b):
        t = b["qkv"].view(-1, HQ + 2 * HKV, 128)
        return t[:, :HQ], t[:, HQ:HQ + HKV], t[:, HQ + HKV:]

    def write(self, b):
        """Append b['new'] tokens in place and write their K and V."""
        hpc.hpc_block_table_append(self.lens, b["new"], self.free, self.count, BLOCKS, self.table, self.lens, b["cu"],
                                   b["pos"], b["slots"], self.count, device_error=self.err)
        q, k, v = self.views(b)
        hpc.hpc_rope_kv_write(q, k, v, b["pos"], b["slots"], self.rope, b["q"], *self.caches, q_norm_weight=self.wq,
                              k_norm_weight=self.wk, k_scale=self.scales[0], v_scale=self.scales[1],
                              device_error=self.err)

    def follow(self, b):
        """The oracle's append and rows of the same tokens; the device's are checked against them."""
        r = self.ref
        got, bits = BT.append(r["lens"], b["new"].tolist(), r["free"], r["count"], BLOCKS, r["table"], b["pos"].numel(), WIDTH)
        assert bits == 0 and self.err.item() == 0
        r.update(table=got["table"], lens=got["lens"], count=got["count"])
        assert self.table.tolist() == got["table"] and self.lens.tolist() == got["lens"]
        assert self.count.item() == got["count"] and b["cu"].tolist() == got["cu"]
        assert b["pos"].tolist() == got["positions"] and b["slots"].tolist() == got["slots"]
        n = got["cu"][-1]
        q, k, v = (x.double().cpu().numpy() for x in self.views(b))
        f, mag = RR.frequencies(ROPE["rot_dim"], ROPE["base"], *(ROPE[x] for x in ("scaling", "factor", "original_len", "low", "high")))
        turned = [RR.turn(RR.norm(x[:n], w.double().cpu().numpy(), 1e-6), got["positions"][:n], f, mag, ROPE["rot_dim"], False)
                  for x, w in ((q, self.wq), (k, self.wk))]
        # within a rounding to bf16 and the fp32 error of values below 8
        assert np.all(np.abs(b["q"][:n].double().cpu().numpy() - turned[0]) <= 2.0 ** -8 * np.abs(turned[0]) + 2.0 ** -15)
        for i in range(n):
            s = got["slots"][i]
            self.rows[s // 64, s % 64] = turned[1][i], v[i]

    def check_cache(self):
        """Every row that some sequence holds is the one that was written for it."""
        host = [c.cpu() for c in self.caches]
        for t, n in zip(self.ref["table"], self.ref["lens"]):
            for p in range(n):
                blk, off = t[p // 64], p % 64
                for c, want, scale in zip(host, self.rows[blk, off], self.scales):
                    row = c[blk, :, off]
                    if self.fp8:
                        x = np.array([PR.e4m3_decode(i) for i in row.flatten().tolist()]).reshape(HKV, 128) * np.float64(np.float32(scale))
                        assert np.all(np.abs(x - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * scale + 2.0 ** -15)
                    else:
                        assert np.all(np.abs(row.double().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -15)

    def reference(self, q, counts):
        """Attention of q [tokens][H_q][128], counts[b] last tokens of each sequence."""
        rows, limits = [], []
        for t, n, c in zip(self.ref["table"], self.ref["lens"], counts):
            for i in range(c):
                rows.append(t)
                limits.append(n - c + 1 + i)
        kw = dict(num_kv_heads=HKV, softmax_scale=128 ** -0.5, kv_is_fp8=self.fp8, k_scale=self.scales[0], v_scale=self.scales[1])
        table, lens = torch.tensor(rows, dtype=torch.int32), torch.tensor(limits, dtype=torch.int32)
        k, v = (c.cpu() for c in self.caches)
        out, lse = oracle.paged_decode(q.cpu(), k, v, table, lens, **kw)
        size, _ = oracle.paged_decode(q.cpu(), k, v & 0x7F if self.fp8 else v.abs(), table, lens, **kw)
        return out, lse, size

    def check_attention(self, out, lse, q, counts):
        ref, ref_lse, size = self.reference(q, counts)
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -14) * size  # as in the attention's own tests
        assert np.all(np.abs(out - ref) <= tol)
        assert np.all(np.abs(lse - ref_lse) <= 2.0 ** -14 + 2.0 ** -20 * np.abs(ref_lse))

    def truncate(self, to):
        t = _i32(to)
        hpc.hpc_block_table_truncate(self.lens, t, self.table, BLOCKS, self.free, self.count, self.lens, self.count,
                                     device_error=self.err)
        r = self.ref
        got, bits = BT.truncate(r["lens"], to, r["table"], BLOCKS, r["free"], r["count"], WIDTH)
        assert bits == 0 and self.err.item() == 0
        r.update(free=got["free"], lens=got["lens"], count=got["count"])
        assert self.lens.tolist() == got["lens"] and self.count.item() == got["count"]
        assert self.free.tolist()[:got["count"]] == got["free"][:got["count"]]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q_len", [1, 3])
def test_a_serving_loop(fp8, q_len):
    B, prefix = 6, 150  # two whole blocks are shared, 22 tokens of the prefix are each sequence's own
    s = Server(fp8, B, 7 + q_len)
    # the prefix's whole blocks, through row 0; then every row starts with them
    b = s.buffers(130)
    b["new"][0] = 128
    s.write(b)
    s.follow(b)
    s.table[1:5] = s.table[0]
    s.lens[1:5] = 128
    s.ref["table"] = [list(s.ref["table"][0]) if i < 5 else r for i, r in enumerate(s.ref["table"])]
    s.ref["lens"] = [128] * 5 + [0]
    # prompts: the prefix's rest and something of their own; row 5 is still free
    new = [22 + 3, 22 + 70, 22, 22 + 41, 22 + 108, 0]
    b = s.buffers(sum(new) + 9)
    b["new"].copy_(_i32(new))
    s.write(b)
    s.follow(b)
    out, lse = torch.zeros_like(b["q"]), torch.zeros(b["q"].shape[:2], device="cuda")
    total = sum(new)
    if not fp8:  # prefill reads the unused slots of a last block: give it a clean copy
        hpc.hpc_extend_attn(b["q"][:total], *(c.nan_to_num(0.0) for c in s.caches), s.table, s.lens, b["cu"], out[:total],
                            lse[:total], device_error=s.err)
        s.check_attention(out[:total], lse[:total], b["q"][:total], new)
    # decode steps as one captured graph: append, turn and write, attend
    d = s.buffers(B * q_len)
    groups, prefixes = _i32([0, 5, B]), _i32([prefix, 0])
    plan = hpc.hpc_decode_prefix_plan_create(B, q_len, hpc.hpc_device_sm_count(), HQ)
    shape = (B, HQ, 128) if q_len == 1 else (B, q_len, HQ, 128)
    out, lse = torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(shape[:-1], device="cuda")

    def step():
        s.write(d)
        hpc.hpc_decode_prefix_attn(d["q"].view(shape), *s.caches, s.table, s.lens, prefixes, plan, out, lse,
                                   cu_groups=groups, k_scale=s.scales[0], v_scale=s.scales[1])
    keep = {k: v.clone() for k, v in dict(free=s.free, count=s.count, table=s.table, lens=s.lens).items()}
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step()  # outside the capture first; d['new'] is zero: it only attends
    torch.cuda.synchronize()
    assert all(torch.equal(getattr(s, k), v) for k, v in keep.items())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    assert hpc.hpc_decode_plan_status(plan) == 0
    for it in range(4):
        d["qkv"].copy_(torch.randn(d["qkv"].shape, generator=s.gen, device="cuda"))
        if it == 2:  # row 2 finishes; row 5 starts with a prompt of its own length
            s.truncate([n if i != 2 else 128 for i, n in enumerate(s.ref["lens"])])
            s.lens[2] = s.ref["lens"][2] = 0
            p = s.buffers(90)
            p["new"][5] = 77
            s.write(p)
            s.follow(p)
        live = [n > 0 for n in s.ref["lens"]]
        d["new"].copy_(_i32([q_len * x for x in live]))
        graph.replay()
        torch.cuda.synchronize()
        assert hpc.hpc_decode_plan_status(plan) == 0
        s.follow(d)
        if all(live):
            s.check_attention(out.view(-1, HQ, 128), lse.view(-1, HQ), d["q"], [q_len] * B)
        else:
            # the rows that append packed, sequence after sequence; the last ones are left over
            assert not live[5] or not live[2]
            n = q_len * sum(live)
            order = [i for i in range(B) if live[i]]
            q = torch.zeros(shape, dtype=torch.bfloat16, device="cuda").view(B, q_len, HQ, 128)
            q[order] = d["q"][:n].view(len(order), q_len, HQ, 128)
            hpc.hpc_decode_prefix_attn(q.view(shape), *s.caches, s.table, s.lens, prefixes, plan, out, lse, cu_groups=groups,
                                       k_scale=s.scales[0], v_scale=s.scales[1])
            assert hpc.hpc_decode_plan_status(plan) == 0
            o, l = out.view(B, q_len, HQ, 128), lse.view(B, q_len, HQ)
            s.check_attention(o[order].flatten(0, 1), l[order].flatten(0, 1), q[order].flatten(0, 1),
                              [q_len * x for x in live])
            dead = [i for i in range(B) if not live[i]]
            assert (o[dead] == 0).all() and (l[dead] == float("-inf")).all()
        if q_len > 1:  # drafts: all but the first one or two are rejected
            s.truncate([max(0, n - (it + i) % q_len) for i, n in enumerate(s.ref["lens"])])
    s.check_cache()
