"""The serving loop over a cache held in 4 bits: block tables and slots from lengths, rotary positions with the 4-bit
write, prompts in chunks over the table, decode steps of one and of several tokens as one captured graph, rejected
drafts rolled back, a finished sequence replaced. Tables, slots and the stack are held to the oracle word for word, V's
rows bit for bit, K's to half a step of their codes, attention to the reference in 64 bits on the cache as it is."""
import numpy as np
import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from oracle import kv4_ref
from tests.kv4_util import UB, attend
from tests.test_gpu_serving_run import BLOCKS, HKV, HQ, Server, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


class Server4(Server):
    def __init__(self, seqs, seed):
        super().__init__(False, seqs, seed)
        self.caches = [torch.full((BLOCKS, HKV, 64, 72), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.scales = (0.02, 0.7)

    def write(self, b):
        hpc.hpc_block_table_append(self.lens, b["new"], self.free, self.count, BLOCKS, self.table, self.lens, b["cu"],
                                   b["pos"], b["slots"], self.count, device_error=self.err)
        q, k, v = self.views(b)
        hpc.hpc_rope_kv4_write(q, k, v, b["pos"], b["slots"], self.rope, b["q"], *self.caches, q_norm_weight=self.wq,
                               k_norm_weight=self.wk, k_scale=self.scales[0], v_scale=self.scales[1], device_error=self.err)

    def check_cache(self):
        k, v = (c.cpu().numpy() for c in self.caches)
        held = set()
        for t, n in zip(self.ref["table"], self.ref["lens"]):
            for p in range(n):
                blk, off = t[p // 64], p % 64
                held.add((blk, off))
                want_k, want_v = self.rows[blk, off]
                assert np.array_equal(v[blk, :, off], kv4_ref.rows(want_v, self.scales[1]))
                row = k[blk, :, off]
                # half the widest step of the codes, 1 of a scale; at most 3 * 2^-9 of the tensor's where that is 0
                unit = np.repeat(kv4_ref.units(row[:, 64:].astype(np.int64), self.scales[0]), 16, -1)
                err = np.abs(kv4_ref.values(row, self.scales[0]) - want_k)
                assert np.all(err <= np.where(unit > 0, unit, 3 * 2.0 ** -9 * self.scales[0]) * (1 + 2.0 ** -10) + 2.0 ** -15)
        return held

    def check_attention(self, out, lse, q, counts):
        cache = [c.cpu().numpy() for c in self.caches]
        at = 0
        for t, n, c in zip(self.ref["table"], self.ref["lens"], counts):
            if c == 0:
                continue
            pos = np.arange(n)
            kv = [torch.from_numpy(kv4_ref.values(x[np.array(t)[pos // 64], :, pos % 64], s)).cuda()
                  for x, s in zip(cache, self.scales)]
            see = torch.arange(n - c + 1, n + 1, device="cuda")
            for h in range(HKV):
                hs = slice(8 * h, 8 * h + 8)
                ref, rl, bound, bl = attend(q[at:at + c, hs].double(), kv[0][:, h], kv[1][:, h], see, 128 ** -0.5)
                bound = bound + UB * (ref.abs() + bound)
                assert ((out[at:at + c, hs].double() - ref).abs() <= bound).all()
                assert ((lse[at:at + c, hs].double() - rl).abs() <= bl).all()
            at += c


@pytest.mark.parametrize("q_len", [1, 2, 5])
def test_a_serving_loop(q_len):
    B = 5
    s = Server4(B, 30 + q_len)

    def prompts(new):  # a chunk of some sequences' prompts, padded rows behind it
        b = s.buffers(sum(new) + 7)
        b["new"].copy_(_i32(new))
        s.write(b)
        s.follow(b)
        out, lse = torch.zeros_like(b["q"]), torch.full(b["q"].shape[:2], 7.0, device="cuda")
        n = sum(new)
        hpc.hpc_extend_kv4_attn(b["q"][:n], *s.caches, s.table, s.lens, b["cu"], out[:n], lse[:n], k_scale=s.scales[0],
                                v_scale=s.scales[1], device_error=s.err)
        torch.cuda.synchronize()
        assert s.err.item() == 0 and (out[n:] == 0).all() and (lse[n:] == 7).all()
        s.check_attention(out[:n], lse[:n], b["q"][:n], new)
    prompts([1, 130, 64, 0, 77])
    prompts([40, 0, 63, 200, 1])
    d = s.buffers(B * q_len)
    plan = hpc.hpc_decode_kv4_plan_create(B, q_len, hpc.hpc_device_sm_count(), HQ)
    shape = (B, HQ, 128) if q_len == 1 else (B, q_len, HQ, 128)
    out, lse = torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(shape[:-1], device="cuda")

    def attention(q):
        hpc.hpc_decode_kv4_attn(q, *s.caches, s.table, s.lens, plan, out, lse, k_scale=s.scales[0], v_scale=s.scales[1])

    def step():
        s.write(d)
        attention(d["q"].view(shape))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step()  # outside the capture first; d['new'] is zero: it only attends
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for it in range(4):
        d["qkv"].copy_(torch.randn(d["qkv"].shape, generator=s.gen, device="cuda"))
        if it == 2:  # row 2 finishes, and starts again with another prompt after the next step
            s.truncate([n if i != 2 else 0 for i, n in enumerate(s.ref["lens"])])
        if it == 3:
            prompts([0, 0, 90, 0, 0])
        live = [n > 0 for n in s.ref["lens"]]
        d["new"].copy_(_i32([q_len * x for x in live]))
        graph.replay()
        torch.cuda.synchronize()
        assert hpc.hpc_decode_plan_status(plan) == 0
        s.follow(d)
        order = [i for i in range(B) if live[i]]
        n = q_len * len(order)
        if n < B * q_len:  # append packed the rows, sequence after sequence
            q = torch.zeros((B, q_len, HQ, 128), dtype=torch.bfloat16, device="cuda")
            q[order] = d["q"][:n].view(len(order), q_len, HQ, 128)
            attention(q.view(shape))
            assert hpc.hpc_decode_plan_status(plan) == 0
        o, l = out.view(B, q_len, HQ, 128), lse.view(B, q_len, HQ)
        s.check_attention(o[order].flatten(0, 1), l[order].flatten(0, 1), d["q"][:n], [q_len * x for x in live])
        dead = [i for i in range(B) if not live[i]]
        assert (o[dead] == 0).all() and (l[dead] == float("-inf")).all()
        if q_len > 1:  # all but the first few drafts are rejected
            s.truncate([max(0, n - (it + i) % q_len) for i, n in enumerate(s.ref["lens"])])
    held = s.check_cache()
    # slots that were never written still hold what they held
    unwritten = [(b, o) for b in range(BLOCKS) for o in range(64) if (b, o) not in s.rows]
    assert unwritten and not held & set(unwritten)
    b, o = torch.tensor(unwritten).T
    assert all((c.cpu()[b, :, o] == 255).all() for c in s.caches)
