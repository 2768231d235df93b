"""Cases of the 4-bit cache operators and their reference in 64 bits, shared by the GPU tests."""
import math

import numpy as np
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from oracle import kv4_ref

# How far the kernels may be from the exact result, from what they round (u: a half step).
U16, UB = 2.0 ** -11, 2.0 ** -8   # f16 and bf16: relative
SUB16 = 2.0 ** -25                # f16: absolute, below its normal numbers


def i32(x, dev="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def random_rows(shape, ts, g, spread=1.0):
    """Rows [..., 72] of normal values, by the reference's rounding."""
    x = torch.randn(shape + (128,), generator=g).double() * spread
    return torch.from_numpy(kv4_ref.rows(x.numpy(), ts))


def attend(q, k, v, see, scale):
    """One sequence and KV head: q [n, 8, 128], k and v [L, 128], see [n], all float64. Returns out, lse, and the
    bounds of their errors (out's without the last rounding to bf16)."""
    n = k.shape[0]
    s = torch.einsum("igd,nd->ign", q, k) * scale
    hide = torch.arange(n, device=q.device) >= see[:, None]
    s = s.masked_fill(hide[:, None], -math.inf)
    m = s.amax(-1, keepdim=True) if n else torch.full(s.shape[:2] + (1,), -math.inf, dtype=s.dtype, device=s.device)
    p = torch.exp(s - torch.where(m > -math.inf, m, 0.0))
    l = p.sum(-1, keepdim=True)
    w = p / torch.where(l > 0, l, 1.0)
    out = torch.einsum("ign,nd->igd", w, v)
    lse = (m + torch.log(l))[..., 0]
    # scores: 8 sums of 16 exact products in fp32, each step losing at most 2^-21 of what it holds; then an FMA
    # and the exponential, 2^-22 each of score and result
    big = (torch.einsum("igd,nd->ign", q.abs(), k.abs()).masked_fill(hide[:, None], 0).amax(-1) * scale) if n else s.new_zeros(s.shape[:2])
    ds = 8 * 2.0 ** -21 * big + 2.0 ** -20
    mass = torch.einsum("ign,nd->igd", w, v.abs())
    vmax = v.abs().amax() if n else v.new_zeros(())
    # each probability: 2^-11, at least 2^-25 of the row's largest (which weighs at least 1 / n); the states of the
    # warps of a piece: o in f16
    bound = (2 * ds[..., None] + 2 * U16 + 2.0 ** -18) * mass + (n * SUB16) * vmax / torch.where(l > 0, l, 1.0) + SUB16 * vmax
    return out, lse, bound, 2 * ds + 2.0 ** -18 + 2.0 ** -22 * lse.abs()


class Paged:
    """Lengths, a 4-bit cache whose unused slots hold 0xff (NaN scales), a table in random order and q."""

    def __init__(self, lens, hkv=2, ks=0.013, vs=0.7, seed=0, spare=2, spread=1.0, q_rows=1, q_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hkv, self.ks, self.vs = lens, hkv, ks, vs
        have = [-(-n // 64) for n in lens]
        self.blocks = sum(have) + spare
        perm = torch.randperm(self.blocks, generator=g).tolist()
        self.table = torch.full((len(lens), max(have + [1])), -1, dtype=torch.int32)
        self.k, self.v = (torch.full((self.blocks, hkv, 64, 72), 255, dtype=torch.uint8) for _ in range(2))
        at = 0
        self.rows = []
        for b, n in enumerate(lens):
            ids = torch.tensor(perm[at:at + have[b]], dtype=torch.long)
            at += have[b]
            self.table[b, :have[b]] = ids.int()
            kr, vr = random_rows((n, hkv), ks, g, spread), random_rows((n, hkv), vs, g, spread)
            pos = torch.arange(n)
            self.k[ids[pos // 64], :, pos % 64] = kr
            self.v[ids[pos // 64], :, pos % 64] = vr
            self.rows.append((kr, vr))
        self.q = (torch.randn(q_rows, 8 * hkv, 128, generator=g) * q_scale).to(torch.bfloat16)

    def device(self):
        return dict(q=self.q.cuda(), k=self.k.cuda(), v=self.v.cuda(), bt=self.table.cuda(), sl=i32(self.lens))

    def values(self, b):
        """K and V of sequence b as float64 [H_kv, L, 128]."""
        return [torch.from_numpy(kv4_ref.values(r.numpy(), t)).transpose(0, 1).cuda()
                for r, t in zip(self.rows[b], (self.ks, self.vs))]

    def reference(self, cu, scale=128 ** -0.5):
        """(out, lse, bound of out, bound of lse) of rows cu[b] .. cu[b + 1] - 1, each sequence's last positions."""
        n = self.q.shape[0]
        got = [torch.zeros(n, 8 * self.hkv, 128, dtype=torch.float64, device="cuda"),
               torch.full((n, 8 * self.hkv), -math.inf, dtype=torch.float64, device="cuda")]
        got += [torch.zeros_like(got[0]), torch.zeros_like(got[1])]
        q = self.q.cuda().double()
        for b, length in enumerate(self.lens):
            if length <= 0:
                continue
            k, v = self.values(b)
            a, z = cu[b], cu[b + 1]
            see = torch.arange(length - (z - a) + 1, length + 1, device="cuda")
            for h in range(self.hkv):
                hs = slice(8 * h, 8 * h + 8)
                for into, x in zip(got, attend(q[a:z, hs], k[h], v[h], see, scale)):
                    into[a:z, hs] = x
        return got

    def check(self, out, lse, cu, scale=128 ** -0.5):
        ref, rl, bound, bl = self.reference(cu, scale)
        out, lse = out.reshape(ref.shape).double(), lse.reshape(rl.shape).double()
        err = (out - ref).abs()
        bound = bound + UB * (ref.abs() + bound)
        assert (err <= bound).all(), f"out: worst {(err / bound).max().item():.3g} of its bound"
        fin = torch.isfinite(rl)
        assert torch.equal(fin, torch.isfinite(lse)) and (lse[~fin] == -math.inf).all()
        assert ((lse - rl).abs()[fin] <= bl[fin]).all(), f"lse: off by {(lse - rl).abs()[fin].max().item():.3g}"


def decode(c, q_len, d=None, plan=None, sms=None, scale=None, out=None, lse=None, stream=None):
    """One step; q's rows are [B][q_len]. Returns out, lse; the plan's error bits must be 0."""
    d = d or c.device()
    n = len(c.lens)
    shape = (n, 8 * c.hkv, 128) if q_len == 1 else (n, q_len, 8 * c.hkv, 128)
    own = plan is None
    plan = plan or hpc.hpc_decode_kv4_plan_create(max(n, 1), q_len, sms or hpc.hpc_device_sm_count(), 8 * c.hkv)
    out = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    lse = torch.full(shape[:-1], float("nan"), device="cuda") if lse is None else lse
    hpc.hpc_decode_kv4_attn(d["q"].view(shape) if d["q"].numel() == math.prod(shape) else d["q"], d["k"], d["v"], d["bt"], d["sl"],
                            plan, out, lse, softmax_scale=scale, k_scale=c.ks, v_scale=c.vs, stream=stream)
    if own:
        assert hpc.hpc_decode_plan_status(plan) == 0
        plan.destroy()
    return out, lse


def cu_of(lens):
    return np.cumsum([0] + list(lens)).tolist()
