"""hpc_rope_kv_write against the fp64 formulas.

Tolerances, derived: the kernel works in fp32 on exact bf16 inputs. cos and
sin are within 2^-22 absolute (an ulp of each plus the angle's), the norm's
factor within 2^-21 relative (a 128-term sum, a square root, a reciprocal and
two products), so a turned element is within 2^-19 (|a| + |b|) of the formula
(four products and a sum on top). Rounding to bf16 adds 2^-8 of the value; to
e4m3, 2^-4 of the value or, below 2^-6, half a subnormal step (2^-10), both
times the scale.
"""
import numpy as np
import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from oracle import prologue_ref as PR
from oracle import rope_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


SCALINGS = {"none": {}, "linear": dict(factor=4.0), "base": dict(factor=8.0),
            "banded": dict(factor=8.0, original_len=8192, low=1.0, high=4.0),
            "ramp": dict(factor=16.0, original_len=4096, low=1.0, high=32.0)}


class Case:
    def __init__(self, n, hq=8, hkv=1, rot_dim=128, interleaved=False, scaling="none", base=1e4, normed=False,
                 fp8=False, q_fp8=False, pos_hi=5000, seed=0, token_major=False, wdtype=torch.bfloat16):
        g = torch.Generator().manual_seed(seed)
        self.n, self.hq, self.hkv, self.fp8 = n, hq, hkv, fp8
        self.rot_dim, self.interleaved, self.kw, self.base = rot_dim, interleaved, dict(scaling=scaling, **SCALINGS[scaling]), base
        self.blocks = n // 64 + 3
        self.qkv = torch.randn(n, (hq + 2 * hkv) * 128, generator=g).to(torch.bfloat16)
        self.pos = torch.randint(0, pos_hi, (n,), generator=g).to(torch.int32)
        self.slots = torch.randperm(self.blocks * 64, generator=g)[:n].to(torch.int32)
        self.w = [(1 + 0.2 * torch.randn(128, generator=g)).to(wdtype) for _ in range(2)] if normed else [None, None]
        shape = (self.blocks, 64, hkv, 128) if token_major else (self.blocks, hkv, 64, 128)
        c = [torch.randn(shape, generator=g).to(torch.bfloat16) for _ in range(2)]
        if fp8:
            c = [torch.randint(0, 120, shape, generator=g).to(torch.uint8) for _ in range(2)]
        self.caches = [x.transpose(1, 2) if token_major else x for x in c]
        self.scales = (0.011, 0.013) if fp8 else (1.0, 1.0)
        self.q_scale = 0.02 if q_fp8 else None

    def rows(self, qkv):
        n, hq, hkv = self.n, self.hq, self.hkv
        return (qkv[:, :hq * 128].view(n, hq, 128), qkv[:, hq * 128:(hq + hkv) * 128].view(n, hkv, 128),
                qkv[:, (hq + hkv) * 128:].view(n, hkv, 128))

    def reference(self):
        q, k, v = (x.double().numpy() for x in self.rows(self.qkv))
        f, mag = R.frequencies(self.rot_dim, self.base, **self.kw)
        out = []
        for x, w in ((q, self.w[0]), (k, self.w[1])):
            x = R.norm(x, None if w is None else w.double().numpy(), 1e-6)
            y = R.turn(x, self.pos.tolist(), f, mag, self.rot_dim, self.interleaved)
            i = np.arange(128)
            r = self.rot_dim
            partner = np.where(i >= r, i, i ^ 1 if self.interleaved else np.where(i < r // 2, i + r // 2, i - r // 2))
            out.append((y, 2.0 ** -19 * mag * (np.abs(x) + np.abs(x[..., partner]))))
        return out[0], out[1], (v, np.zeros_like(v))

    def run(self, in_place=False, stream=None, err=None):
        qkv = self.qkv.cuda()
        q, k, v = self.rows(qkv)
        # a cache keeps its layout on the device
        caches = [x.transpose(1, 2).contiguous().cuda().transpose(1, 2) if not x.is_contiguous() else x.cuda()
                  for x in self.caches]
        q_out = q if in_place else torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        q8 = torch.full(q.shape, 3, dtype=torch.uint8, device="cuda") if self.q_scale else None
        rope = hpc.hpc_rope_init(self.rot_dim, self.interleaved, self.base, **self.kw)
        wq, wk = (None if w is None else w.cuda() for w in self.w)
        args = (q, k, v, self.pos.cuda(), self.slots.cuda(), rope, q_out, *caches)
        kw = dict(q_norm_weight=wq, k_norm_weight=wk, eps=1e-6, q_out_fp8=q8, q_fp8_scale=self.q_scale or 1.0,
                  k_scale=self.scales[0], v_scale=self.scales[1], device_error=err)
        torch.cuda.synchronize()
        hpc.hpc_rope_kv_write(*args, **kw, stream=stream)
        torch.cuda.synchronize()
        if in_place:  # only the q rows may change
            assert torch.equal(qkv[:, self.hq * 128:].cpu(), self.qkv[:, self.hq * 128:])
        return q_out.cpu(), None if q8 is None else q8.cpu(), [c.cpu() for c in caches]

    def check(self, got, live=None):
        q_out, q8, caches = got
        live = np.ones(self.n, bool) if live is None else live
        (q, q_slack), *kv = self.reference()
        x = q_out.double().numpy()
        assert np.all(np.abs(x - q)[live] <= (2.0 ** -8 * np.abs(q) + q_slack)[live])
        if q8 is not None:
            self.check_e4m3(q8.numpy()[live], q[live], q_slack[live], self.q_scale)
        block, off = self.slots.numpy() // 64, self.slots.numpy() % 64
        for i, (ref, slack) in enumerate(kv):
            c, c0 = caches[i].clone(), self.caches[i]
            rows = c[block[live], :, off[live]]
            if self.fp8:
                self.check_e4m3(rows.numpy(), ref[live], slack[live], self.scales[i])
                if i == 1:  # v is only rounded: every byte is the nearest one
                    codes = [PR.e4m3_encode(y / np.float64(np.float32(self.scales[1]))) for y in ref[live][:40].ravel()]
                    assert rows[:40].numpy().ravel().tolist() == codes
            else:
                y = rows.double().numpy()
                assert np.all(np.abs(y - ref[live]) <= (2.0 ** -8 * np.abs(ref) * (i == 0) + slack)[live])
            c[block[live], :, off[live]] = c0[block[live], :, off[live]]
            assert torch.equal(c, c0)  # every other slot as it was

    @staticmethod
    def check_e4m3(code, ref, slack, scale):
        value = np.array([PR.e4m3_decode(i) for i in range(256)])[code] * np.float64(np.float32(scale))
        top = 448.0 * scale
        ref = np.clip(ref, -top, top)
        assert np.all(np.abs(value - ref) <= 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 * scale + slack)


@pytest.mark.parametrize("rot_dim", [2, 4, 16, 20, 48, 64, 90, 96, 112, 126, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_part_of_the_head(rot_dim, interleaved):
    c = Case(37, rot_dim=rot_dim, interleaved=interleaved, seed=rot_dim)
    c.check(c.run())


@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("rot_dim,interleaved", [(128, False), (64, True), (44, False)])
def test_scalings_at_far_positions(scaling, rot_dim, interleaved):
    c = Case(50, scaling=scaling, rot_dim=rot_dim, interleaved=interleaved, base=5e5, pos_hi=1 << 24, seed=3)
    c.pos[:4] = torch.tensor([0, 1, (1 << 24) - 1, (1 << 24) - 2])
    c.check(c.run())


@pytest.mark.parametrize("n", [1, 2, 3, 16, 17, 151, 305, 700])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (64, 8), (16, 16), (3, 1)])
def test_sizes_and_heads(n, hq, hkv):
    if n * hq > 12000:
        pytest.skip("the plain reference is slow")
    c = Case(n, hq, hkv, normed=n % 2 == 1, seed=n)
    c.check(c.run(in_place=n % 3 == 0))


@pytest.mark.parametrize("hq,hkv", [(128, 2), (200, 4)])
def test_more_rows_than_a_pass(hq, hkv):
    c = Case(400, hq, hkv, rot_dim=8, normed=True, seed=1)  # 16 x 5 rows per pass of one CTA
    c.check(c.run())


@pytest.mark.parametrize("n", [1250, 2000, 3100])  # CTAs a token: 1 or 2 with the layout's residents
@pytest.mark.parametrize("interleaved,rot_dim", [(False, 128), (True, 64), (False, 60)])
def test_a_token_does_not_depend_on_its_batch(n, interleaved, rot_dim):
    def part(c, a, b):
        d = Case(1, 44, 4)
        d.__dict__.update(c.__dict__, n=b - a, qkv=c.qkv[a:b], pos=c.pos[a:b], slots=c.slots[a:b])
        return d
    c = Case(n, 44, 4, rot_dim=rot_dim, interleaved=interleaved, fp8=True, q_fp8=True, seed=n)
    q, q8, caches = c.run()
    first = part(c, 0, 40)
    small = first.run()
    first.check(small)
    block, off = c.slots // 64, c.slots % 64
    for a, b in ((0, 40), (40, 47), (n - 300, n)):
        sq, sq8, sc = part(c, a, b).run()
        assert torch.equal(sq, q[a:b]) and torch.equal(sq8, q8[a:b])
        for x, y in zip(sc, caches):
            assert torch.equal(x[block[a:b], :, off[a:b]], y[block[a:b], :, off[a:b]])


@pytest.mark.parametrize("interleaved,rot_dim", [(False, 128), (True, 80), (False, 60)])
@pytest.mark.parametrize("normed", [False, True])
def test_fp8(interleaved, rot_dim, normed):
    c = Case(70, 16, 2, rot_dim=rot_dim, interleaved=interleaved, normed=normed, fp8=True, q_fp8=True, seed=5,
             wdtype=torch.float32)
    c.check(c.run())


@pytest.mark.parametrize("scale", [4.0 / 448, 1.0 / 112, 0.01, 1.0, 0.25, 3.0, 1.0 / 3, 0.0117, 700.0, 2.0 ** -40, 3e37, 1e-37])
def test_e4m3_rounds_the_exact_quotient(scale):
    """Every finite bf16 magnitude around the e4m3 range, ties included: each byte is the nearest one."""
    codes = torch.arange(0, 0x7F80).to(torch.int16).view(torch.bfloat16)
    s = np.float64(np.float32(scale))
    keep = (codes.double() / s > 2.0 ** -11) & (codes.double() / s < 1000)
    v = torch.cat([codes[keep], -codes[keep], torch.tensor([0.0, -0.0, float("inf"), float("-inf")], dtype=torch.bfloat16)])
    n = -(-v.numel() // 128)
    rows = torch.zeros(n * 128, dtype=torch.bfloat16)
    rows[:v.numel()] = v[torch.randperm(v.numel(), generator=torch.Generator().manual_seed(1))]
    rows = rows.view(n, 1, 128).cuda()
    cache = torch.zeros((2, n // 64 + 1, 1, 64, 128), dtype=torch.uint8, device="cuda")
    q8 = torch.zeros(rows.shape, dtype=torch.uint8, device="cuda")
    hpc.hpc_rope_kv_write(rows, rows.clone(), rows.clone(), torch.zeros(n, dtype=torch.int32, device="cuda"),
                          torch.arange(n, dtype=torch.int32, device="cuda"), hpc.hpc_rope_init(rot_dim=2), rows.clone(),
                          cache[0], cache[1], q_out_fp8=q8, q_fp8_scale=scale, k_scale=scale, v_scale=scale)
    ref = [PR.e4m3_encode(x / s) for x in rows.double().cpu().numpy().ravel()]
    assert cache[1].flatten()[:n * 128].tolist() == ref  # v
    # position 0 turns nothing: q and k are the same rows (0 * inf spoils a pair that holds one)
    fine = torch.isfinite(rows).view(-1, 2).all(1).repeat_interleave(2).cpu()
    for got in (cache[0].flatten()[:n * 128], q8.flatten()):
        same = got.cpu() == torch.tensor(ref, dtype=torch.uint8)
        same |= (rows.cpu().flatten() == 0)  # the sign of a zero
        assert same[fine].all()


@pytest.mark.parametrize("fp8", [False, True])
def test_token_major_cache(fp8):
    c = Case(90, 16, 4, fp8=fp8, token_major=True, seed=6)
    c.check(c.run())


def test_padding_and_bad_tokens():
    c = Case(20, 16, 2, normed=True, q_fp8=True, seed=7)
    live = np.ones(20, bool)
    c.slots[[3, 19]] = -1
    c.pos[3] = -9                        # padding is not looked at
    c.pos[5], c.pos[6] = -1, 1 << 24     # positions out of range: skipped
    live[[3, 5, 6, 19]] = False
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = c.run(err=err)
    c.check(got, live)
    assert err.item() == hpc.HPC_DEVCHK_BAD_LENGTH
    assert (got[0][~live].float() == 7).all() and (got[1][~live] == 3).all()
    # a slot past the cache: q is turned, the cache stays
    c = Case(4, seed=8)
    keep = c.slots[2].clone()
    c.slots[2] = c.blocks * 64
    err.zero_()
    q_out, _, caches = c.run(err=err)
    assert err.item() == hpc.HPC_DEVCHK_BAD_BLOCK
    live = np.array([True, True, False, True])
    c.slots[2] = keep
    (q, slack), _, _ = c.reference()
    assert np.all(np.abs(q_out.double().numpy() - q) <= 2.0 ** -8 * np.abs(q) + slack)
    c.check((q_out, None, caches), live)


def test_values_that_are_not_finite_stay_in_their_pair():
    c = Case(3, rot_dim=64, seed=9)
    q = c.rows(c.qkv)[0]
    q[1, 2, 5] = float("inf")     # paired with 37
    q[1, 3, 100] = float("nan")   # past the turned part
    q[2, 0, 127] = float("-inf")
    q_out, _, _ = c.run()
    bad = ~torch.isfinite(q_out)
    assert sorted(map(tuple, bad.nonzero().tolist())) == [(1, 2, 5), (1, 2, 37), (1, 3, 100), (2, 0, 127)]
    assert q_out[2, 0, 127] == float("-inf")


@pytest.mark.parametrize("rot_dim,interleaved", [(44, False), (64, True), (128, False)])
def test_values_that_are_not_finite_in_every_layout(rot_dim, interleaved):
    c = Case(3, rot_dim=rot_dim, interleaved=interleaved, seed=12)
    q, k, v = c.rows(c.qkv)
    q[1, 2, 6], k[2, 0, 3], v[0, 0, 9] = float("inf"), float("nan"), float("nan")
    q[0, 4, 127] = float("-inf")
    q_out, _, caches = c.run()
    mate = (lambda i: i ^ 1) if interleaved else lambda i: i + rot_dim // 2
    far = [(0, 4, 127)] + ([(0, 4, 63)] if rot_dim == 128 else [])
    bad = ~torch.isfinite(q_out)
    assert sorted(map(tuple, bad.nonzero().tolist())) == sorted([(1, 2, 6), (1, 2, mate(6))] + far)
    at = [(int(s) // 64, int(s) % 64) for s in c.slots]
    kept = [[~torch.isfinite(x[b, 0, o]) for b, o in at] for x in caches]
    assert kept[0][2].nonzero().flatten().tolist() == sorted([3, mate(3)]) and not kept[0][0].any() and not kept[0][1].any()
    assert kept[1][0].nonzero().flatten().tolist() == [9] and not kept[1][1].any() and not kept[1][2].any()


@pytest.mark.parametrize("rot_dim,interleaved", [(96, False), (128, False), (64, True), (90, False), (20, False)])
@pytest.mark.parametrize("which", [0, 1])
def test_a_norm_of_q_or_k_only(rot_dim, interleaved, which):
    c = Case(45, 24, 2, rot_dim=rot_dim, interleaved=interleaved, scaling="ramp", normed=True, seed=rot_dim + which)
    c.w[which] = None
    c.check(c.run(in_place=True))


def test_agrees_with_the_decode_prologue():
    """One token per sequence, the whole head, no scaling: the fused decode
    prologue computes the same rows (each within its own fp32 error)."""
    c = Case(40, 64, 8, normed=True, fp8=True, seed=10)
    got = c.run()
    table = (c.slots // 64).view(-1, 1)
    c.slots = (c.slots // 64) * 64 + c.pos % 64
    keep = []
    for i in range(40):  # distinct slots only
        if c.slots[i].item() not in c.slots[:i].tolist():
            keep.append(i)
    c.qkv, c.pos, c.slots, c.n = c.qkv[keep], c.pos[keep] % 64, c.slots[keep], len(keep)
    table = table[keep]
    q_out, _, caches = c.run()
    q, k, v = (x.contiguous().cuda() for x in c.rows(c.qkv))
    ref = torch.empty_like(q)
    kc, vc = (x.cuda() for x in c.caches)
    hpc.hpc_rope_norm_kv_write(q, k, v, (c.pos + 1).cuda(), table.cuda(), c.w[0].cuda(), c.w[1].cuda(), ref, kc, vc,
                               rope_base=1e4, k_scale=c.scales[0], v_scale=c.scales[1])
    assert torch.equal(vc.cpu(), caches[1])
    d = (ref.cpu().double() - q_out.double()).abs()
    assert (d <= 2.0 ** -7 * q_out.double().abs() + 1e-5).all()
    assert (kc.cpu() != caches[0]).float().mean() < 1e-3


def test_captured_and_on_another_stream():
    c = Case(33, 16, 2, normed=True, seed=11)
    s = torch.cuda.Stream()
    eager = c.run(stream=s)
    c.check(eager)
    q, k, v = (x.contiguous().cuda() for x in c.rows(c.qkv))
    caches = [x.cuda() for x in c.caches]
    q_out, pos, slots = torch.zeros_like(q), c.pos.cuda(), c.slots.cuda()
    rope = hpc.hpc_rope_init()
    wq, wk = (w.cuda() for w in c.w)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        hpc.hpc_rope_kv_write(q, k, v, pos, slots, rope, q_out, *caches, q_norm_weight=wq, k_norm_weight=wk)
    rope = None  # the table was copied into the launch
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(q_out.cpu(), eager[0]) and all(torch.equal(a.cpu(), b) for a, b in zip(caches, eager[2]))
