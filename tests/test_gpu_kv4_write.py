"""hpc_rope_kv4_write: V's rows bit for bit, K's within what fp32 leaves open, and nothing else written."""
import math

import numpy as np
import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from oracle import kv4_ref, rope_ref
from tests.kv4_util import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


class Tokens:
    def __init__(self, n, hkv=2, hq=None, blocks=None, seed=0, spread=1.0, positions=None, slots=None):
        g = torch.Generator().manual_seed(seed)
        self.n, self.hkv, self.hq = n, hkv, hq or 8 * hkv
        bf = lambda h: (torch.randn(n, h, 128, generator=g) * spread).to(torch.bfloat16)
        self.q, self.k, self.v = bf(self.hq), bf(hkv), bf(hkv)
        self.blocks = blocks or -(-n // 64) + 2
        self.positions = positions if positions is not None else torch.randint(0, 100000, (n,), generator=g).tolist()
        self.slots = slots if slots is not None else torch.randperm(self.blocks * 64, generator=g)[:n].tolist()
        self.wq, self.wk = (1 + 0.2 * torch.randn(2, 128, generator=g))

    def write(self, rope=None, ks=0.01, vs=0.02, norm=None, bits=0, caches=None, in_place=False):
        dev = lambda x: x.cuda()
        q = dev(self.q)
        out = q if in_place else torch.full_like(q, float("nan"))
        kc, vc = caches or (torch.full((self.blocks, self.hkv, 64, 72), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(2))
        err = i32([0])
        w = {} if norm is None else dict(q_norm_weight=dev(self.wq).to(norm), k_norm_weight=dev(self.wk).to(norm))
        hpc.hpc_rope_kv4_write(q, dev(self.k), dev(self.v), i32(self.positions), i32(self.slots), rope or hpc.hpc_rope_init(), out, kc, vc,
                               k_scale=ks, v_scale=vs, device_error=err, **w)
        assert err.item() == bits
        return out, kc, vc

    def check(self, got, rot_dim=128, interleaved=False, base=1e4, ks=0.01, vs=0.02, norm=None, live=None):
        out, kc, vc = (x.cpu() for x in got)
        live = list(range(self.n)) if live is None else live
        at = torch.tensor([self.slots[i] for i in live], dtype=torch.long)
        pos = [self.positions[i] for i in live]
        # V: the reference's bytes
        v = self.v[live].double().numpy()
        assert np.array_equal(vc[at // 64, :, at % 64].numpy(), kv4_ref.rows(v, vs))
        f, mag = rope_ref.frequencies(rot_dim, base)
        want = {}
        for name, x, w in (("q", self.q, self.wq), ("k", self.k, self.wk)):
            x = x[live].double().numpy()
            if norm is not None:
                x = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * w.to(norm).double().numpy()
            want[name] = rope_ref.turn(x, pos, f, mag, rot_dim, interleaved)
        # q: bf16 of an fp32 value within 2^-20 of the row's largest element
        big = np.abs(want["q"]).max(-1, keepdims=True)
        err = np.abs(out[live].double().numpy() - want["q"])
        assert (err <= 2.0 ** -8 * np.abs(want["q"]) + 2.0 ** -19 * big).all()
        # K: what an element within e of the exact one gives (e: 2^-19 of the row's largest; norm, angle and turn in fp32)
        k = want["k"]
        e = 2.0 ** -19 * np.abs(k).max(-1, keepdims=True)
        code, scale = kv4_ref.split(kc[at // 64, :, at % 64].numpy())
        lo, hi = kv4_ref.scales(np.maximum(np.abs(k) - e, 0), ks), kv4_ref.scales(np.abs(k) + e, ks)
        assert (lo <= scale).all() and (scale <= hi).all()
        value = lambda x: kv4_ref.E2M1[kv4_ref.codes(x, scale, ks) & 7] * np.where(x < 0, -1, 1)
        assert (value(k - e) <= code).all() and (code <= value(k + e)).all()
        exact = kv4_ref.rows(k, ks)
        assert (exact != kc[at // 64, :, at % 64].numpy()).mean() <= 1e-3
        # every other row of the caches is as it was
        rest = torch.ones(self.blocks * 64, dtype=torch.bool)
        rest[at] = False
        for c in (kc, vc):
            assert (c.transpose(1, 2).reshape(self.blocks * 64, self.hkv, 72)[rest] == 0xA5).all()


@pytest.mark.parametrize("n,hkv", [(1, 1), (5, 2), (64, 8), (333, 2), (1531, 1)])
@pytest.mark.parametrize("norm", [None, torch.float32, torch.bfloat16])
def test_sizes(n, hkv, norm):
    t = Tokens(n, hkv, seed=n)
    t.check(t.write(norm=norm), norm=norm)


@pytest.mark.parametrize("rot_dim", [2, 16, 20, 32, 48, 64, 80, 90, 96, 112, 126, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [None, torch.float32])
def test_rotations(rot_dim, interleaved, norm):
    t = Tokens(70, 2, seed=rot_dim)
    got = t.write(rope=hpc.hpc_rope_init(rot_dim, interleaved), norm=norm)
    t.check(got, rot_dim=rot_dim, interleaved=interleaved, norm=norm)


@pytest.mark.parametrize("ts", [2.0 ** -100, 1e-20, 0.001, 1.0, 0.75, 2.0 ** 100])
def test_tensor_scales(ts):
    """Rows of the size that the tensor's scale is for; bf16 holds them all."""
    t = Tokens(200, 2, seed=3, spread=ts * 400)
    t.check(t.write(ks=ts, vs=ts), ks=ts, vs=ts)


@pytest.mark.parametrize("ts", [1.0, 0.5, 0.015625, 1.25, 0.1])
def test_ties(ts):
    """Small whole numbers: with scales of few bits their quotients are midpoints of e2m1, and the largest one's of e4m3."""
    t = Tokens(256, 2, seed=4)
    g = torch.Generator().manual_seed(1)
    t.v = (torch.randint(-40, 41, t.v.shape, generator=g) * 0.25).to(torch.bfloat16)
    t.v[:, :, 0] = torch.randint(1, 257, t.v.shape[:2], generator=g).to(torch.bfloat16)
    t.positions = [0] * 256  # K does not turn: exact too
    t.k = t.v.flip(0).clone()
    _, kc, vc = got = t.write(ks=ts, vs=ts)
    t.check(got, ks=ts, vs=ts)
    at = torch.tensor(t.slots)
    assert np.array_equal(kc.cpu()[at // 64, :, at % 64].numpy(), kv4_ref.rows(t.k.double().numpy(), ts))


def test_every_bf16_magnitude():
    """Rows of one magnitude each, over all positive finite bf16: scales of every size, 0 and saturated ones among them."""
    x = torch.arange(0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    n = -(-x.numel() // 8)
    v = torch.zeros(n * 8, dtype=torch.bfloat16)
    v[:x.numel()] = x
    t = Tokens(n, 1, seed=5)
    g = torch.Generator().manual_seed(2)
    t.v = (v.view(n, 1, 8, 1).float() * (torch.rand(n, 1, 8, 16, generator=g) * 2 - 1)).to(torch.bfloat16)
    t.v[..., 3] = v.view(n, 1, 8)
    t.v = t.v.reshape(n, 1, 128).contiguous()
    for ts in (1.0, 0.3, 2.0 ** -100, 2.0 ** 100):
        _, _, vc = t.write(vs=ts)
        at = torch.tensor(t.slots)
        assert np.array_equal(vc.cpu()[at // 64, :, at % 64].numpy(), kv4_ref.rows(t.v.double().numpy(), ts)), ts


def test_not_finite():
    t = Tokens(6, 1, seed=6)
    t.v[0, 0, 5] = math.nan
    t.v[1, 0, 20] = math.inf
    t.v[2, 0, 40] = -math.inf
    t.k[3, 0, 7] = math.nan
    t.positions = [0] * 6
    _, kc, vc = t.write(ks=1.0, vs=1.0)
    at = torch.tensor(t.slots)
    v = kv4_ref.values(vc.cpu()[at // 64, :, at % 64].numpy(), 1.0)[:, 0]
    k = kv4_ref.values(kc.cpu()[at // 64, :, at % 64].numpy(), 1.0)[:, 0]
    assert np.isnan(v[0, :16]).all() and np.isfinite(v[0, 16:]).all()
    assert v[1, 20] == 2688 and v[2, 40] == -2688 and np.isfinite(v[1:]).all()
    assert np.isnan(k[3, :16]).all() and np.isfinite(k[[0, 1, 2, 4, 5]]).all()


def test_padding_and_bad_tokens():
    t = Tokens(9, 2, seed=7)
    t.slots[1], t.slots[4] = -1, -5
    t.slots[6] = t.blocks * 64 + 3      # past the cache
    t.positions[7], t.positions[8] = -1, 1 << 24
    got = t.write(bits=1 | 2)
    t.check(got, live=[0, 2, 3, 5])
    assert torch.isnan(got[0][[1, 4, 7, 8]]).all() and torch.isfinite(got[0][6]).all()


def test_in_place_and_views():
    """q turned in place; q, k and v slices of one projection; K and V in one buffer; heads outside the blocks."""
    t = Tokens(100, 2, seed=8)
    ref = t.write()
    out, kc, vc = t.write(in_place=True)
    assert torch.equal(out, ref[0]) and torch.equal(kc, ref[1]) and torch.equal(vc, ref[2])
    both = torch.full((t.blocks, 2, 2, 64, 72), 0xA5, dtype=torch.uint8, device="cuda")
    t.write(caches=(both[:, 0], both[:, 1]))
    assert torch.equal(both[:, 0], ref[1]) and torch.equal(both[:, 1], ref[2])
    heads = torch.full((2, 2, t.blocks, 64, 72), 0xA5, dtype=torch.uint8, device="cuda")
    t.write(caches=(heads[0].transpose(0, 1), heads[1].transpose(0, 1)))
    assert torch.equal(heads[0].transpose(0, 1), ref[1]) and torch.equal(heads[1].transpose(0, 1), ref[2])
    qkv = torch.cat([t.q, t.k, t.v], 1).cuda()
    kc, vc = (torch.full((t.blocks, 2, 64, 72), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(2))
    hpc.hpc_rope_kv4_write(qkv[:, :16], qkv[:, 16:18], qkv[:, 18:], i32(t.positions), i32(t.slots), hpc.hpc_rope_init(), qkv[:, :16], kc, vc,
                           k_scale=0.01, v_scale=0.02)
    assert torch.equal(qkv[:, :16], ref[0]) and torch.equal(kc, ref[1]) and torch.equal(vc, ref[2])


def test_groups_of_any_size():
    t = Tokens(50, 3, hq=3, seed=9)   # as many query heads as KV heads
    t.check(t.write())
    t = Tokens(50, 1, hq=64, seed=10)
    t.check(t.write())


def test_no_tokens_and_no_blocks():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(2, 1, 64, 72, dtype=torch.uint8, device="cuda")
    hpc.hpc_rope_kv4_write(z(0, 8, 128), z(0, 1, 128), z(0, 1, 128), i32([]), i32([]), hpc.hpc_rope_init(), z(0, 8, 128), c, c.clone())
    cpu = torch.zeros(2, 1, 64, 72, dtype=torch.uint8)
    with pytest.raises(hpc.HpcError):
        hpc.hpc_rope_kv4_write(z(1, 8, 128), z(1, 1, 128), z(1, 1, 128), i32([0]), i32([0]), hpc.hpc_rope_init(), z(1, 8, 128), cpu, cpu.clone())
