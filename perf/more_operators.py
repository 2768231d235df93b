"""Measured cases of the operators of a paged KV cache held in 4 bits.

A row of such a cache, one token's K or V of one KV head, is 72 bytes: 64 bytes of e2m1 codes (byte i:
element 2i in its low four bits, 2i + 1 in its high ones), then eight e4m3 scales, one for each sixteen
neighbouring elements. An element stands for code * scale * (the tensor's own fp32 scale). Three groups of
calls, as a serving loop makes them one after the other:

* ``write``: optional QK-norm, rotary positions of a ragged batch of tokens, and the write of K and V,
  rounded to 4 bits, into the cache at the step's slots;
* ``decode``: attention of one to eight new tokens of every sequence over the cache;
* ``extend``: attention of ragged new tokens (prompts, chunks of prompts) over the cache that holds them.

``run`` computes each in plain torch operations, or, where ``own`` is true, by the framework's calls.
"""
import math
import random

import torch

own = False

BLOCK = 64
DIM = 128
GROUP = 8  # query heads per KV head
ROW = 72  # bytes of a row: 64 of codes, 8 of scales
SPAN = 16  # elements that share a scale
E4M3_MAX, E2M1_MAX = 448.0, 6.0


def listed():
    return [
        # a handful of short requests, one KV head: latency
        {"name": "decode_tiny", "op": "decode", "kv_heads": 1, "q_len": 1, "seqs": 4, "len_lo": 37, "len_hi": 1000, "long": 0, "empty": 0.0},
        # a chat service's step, some of its places in the batch free
        {"name": "decode_chat", "op": "decode", "kv_heads": 8, "q_len": 1, "seqs": 64, "len_lo": 200, "len_hi": 6000, "long": 0, "empty": 0.1},
        # one very long sequence next to ordinary ones
        {"name": "decode_skewed", "op": "decode", "kv_heads": 8, "q_len": 1, "seqs": 32, "len_lo": 4096, "len_hi": 4096, "long": 131072, "empty": 0.0},
        # a large batch of ragged lengths, few KV heads on this GPU
        {"name": "decode_mixed", "op": "decode", "kv_heads": 2, "q_len": 1, "seqs": 256, "len_lo": 16, "len_hi": 20000, "long": 0, "empty": 0.0},
        # speculative decoding: four draft tokens checked per sequence
        {"name": "decode_drafts", "op": "decode", "kv_heads": 8, "q_len": 4, "seqs": 24, "len_lo": 3000, "len_hi": 9000, "long": 0, "empty": 0.0},
        # the longest drafts, two KV heads, odd lengths
        {"name": "decode_drafts_wide", "op": "decode", "kv_heads": 2, "q_len": 8, "seqs": 13, "len_lo": 9, "len_hi": 30011, "long": 0, "empty": 0.0},
        # a short prompt by itself: latency
        {"name": "extend_prompt", "op": "extend", "kv_heads": 8, "seqs": 1, "new_lo": 512, "new_hi": 512, "old_lo": 0, "old_hi": 0},
        # chunks of long prompts over what is in the cache already
        {"name": "extend_chunks", "op": "extend", "kv_heads": 8, "seqs": 4, "new_lo": 1024, "new_hi": 1024, "old_lo": 8192, "old_hi": 16384},
        # ragged requests, single tokens among them
        {"name": "extend_ragged", "op": "extend", "kv_heads": 2, "seqs": 37, "new_lo": 1, "new_hi": 411, "old_lo": 0, "old_hi": 3000},
        # one new token for each of 64 sequences, with QK-norm: the decode step's prologue
        {"name": "write_decode", "op": "write", "kv_heads": 8, "tokens": 64, "rot_dim": 128, "interleaved": False, "scaling": "none", "norm": True, "pos_hi": 4096},
        # a prefill chunk at far positions, frequencies scaled by wavelength
        {"name": "write_prefill", "op": "write", "kv_heads": 8, "tokens": 8192, "rot_dim": 128, "interleaved": False, "scaling": "banded", "norm": False, "pos_hi": 131072},
        # an odd batch, interleaved pairs on part of the head, positions interpolated, with QK-norm
        {"name": "write_odd", "op": "write", "kv_heads": 4, "tokens": 1531, "rot_dim": 80, "interleaved": True, "scaling": "linear", "norm": True, "pos_hi": 65536},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "extend", "extend", "write", "write"])
    if op == "decode":
        q_len, heads = rng.choice([1, 1, 1, 2, 3, 4, 5, 6, 7, 8]), rng.choice([1, 2, 4, 8, 8])
        seqs = _log(rng, 1, 250 // q_len)
        hi = _log(rng, q_len, min(100000, 1900000 // (seqs * heads * (q_len + 1) // 2)))
        return {"op": "decode", "kv_heads": heads, "q_len": q_len, "seqs": seqs, "len_lo": max(q_len, hi // rng.choice([1, 2, 8, 100])),
                "len_hi": hi, "long": 0, "empty": rng.choice([0.0, 0.0, 0.2])}
    if op == "extend":
        heads = rng.choice([1, 2, 4, 8, 8])
        seqs = _log(rng, 1, 40)
        new = _log(rng, 1, min(2000, 6000 // seqs))
        old = _log(rng, 1, min(16000, 100000 // seqs, 40000000 // (seqs * new)))
        return {"op": "extend", "kv_heads": heads, "seqs": seqs, "new_lo": max(1, new // rng.choice([1, 3, 50])), "new_hi": new,
                "old_lo": rng.choice([0, old // 2, old]), "old_hi": old}
    return {"op": "write", "kv_heads": rng.choice([1, 2, 4, 8]), "tokens": _log(rng, 1, 8000),
            "rot_dim": rng.choice([20, 32, 48, 64, 80, 90, 96, 112, 128]), "interleaved": rng.random() < 0.4,
            "scaling": rng.choice(["none", "linear", "base", "banded", "ramp"]), "norm": rng.random() < 0.5, "pos_hi": _log(rng, 64, 1 << 20)}


def _rng(case):
    """Lengths belong to the case; values come from the seed."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _ceil(a, b=BLOCK):
    return -(-a // b)


def _lens(case):
    """decode: the lengths of the sequences, spread over their logarithm; extend: (new tokens, positions in all)."""
    rng = _rng(case)
    if case["op"] == "decode":
        lens = [0 if rng.random() < case["empty"] else _log(rng, case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]
        lens[0] = case["long"] or lens[0] or case["len_hi"]  # a step has work
        return lens
    new = [_log(rng, case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    return new, [n + rng.randint(case["old_lo"], case["old_hi"]) for n in new]


#: What each way of scaling the frequencies takes: positions trained on, the factor by which they grow, two band limits.
ROPE = {"base": 500000.0, "factor": 8.0, "original_len": 8192, "low": 1.0, "high": 4.0, "fast": 32.0, "slow": 1.0}


def _frequencies(case):
    """Angle per position of each rotated pair, in 64 bits, and the factor on cosine and sine."""
    r, base, f = case["rot_dim"], ROPE["base"], ROPE["factor"]
    how = case["scaling"]
    if how == "base":
        base *= f ** (r / (r - 2.0))
    freq = torch.tensor([base ** (-2.0 * i / r) for i in range(r // 2)], dtype=torch.float64)
    if how == "linear":
        return freq / f, 1.0
    if how == "banded":
        turns = ROPE["original_len"] * freq / (2 * math.pi)  # turns of each pair over the trained positions
        keep = ((turns - ROPE["low"]) / (ROPE["high"] - ROPE["low"])).clamp(0.0, 1.0)
        return freq * keep + freq / f * (1.0 - keep), 1.0
    if how == "ramp":
        def pair(turns):
            return r * math.log(ROPE["original_len"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(0, math.floor(pair(ROPE["fast"]))), min(r - 1, math.ceil(pair(ROPE["slow"])))
        ramp = ((torch.arange(r // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return freq / f * ramp + freq * (1.0 - ramp), 0.1 * math.log(f) + 1.0
    return freq, 1.0


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rows(x, scale):
    """Rows of a 4-bit cache, [..., 128] to uint8 [..., 72]: each sixteen elements get the e4m3 nearest to their
    largest magnitude / (6 * scale), each element the e2m1 nearest to element / (e4m3 * scale), ties to even."""
    ts = torch.tensor(scale, dtype=torch.float32, device=x.device)
    g = x.unflatten(-1, (DIM // SPAN, SPAN))
    small = (g.abs().amax(-1) / (6 * ts)).clamp(max=E4M3_MAX).to(torch.float8_e4m3fn)
    unit = (small.float() * ts).to(g.dtype)[..., None]
    y = torch.where(unit > 0, g / unit, 0).double()
    # midpoints of 0, 0.5, 1, 1.5, 2, 3, 4, 6; those whose even neighbour is the larger one count from themselves on
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=x.device)
    up = torch.tensor([False, True, False, True, False, True, False], device=x.device)
    code = torch.bucketize(y.abs(), torch.where(up, torch.nextafter(mids, torch.zeros_like(mids)), mids)).to(torch.uint8)
    code = (code | ((y < 0).to(torch.uint8) << 3)).flatten(-2)
    return torch.cat([code[..., 0::2] | (code[..., 1::2] << 4), small.view(torch.uint8)], -1)


def _cache(shape, gen):
    """A cache filled with rows of normal values, in parts that keep the 64-bit temporaries small."""
    out = torch.empty(shape + (ROW,), device="cuda", dtype=torch.uint8)
    scale = 5.0 / (E4M3_MAX * E2M1_MAX)
    step = max(1, (1 << 24) // (shape[1] * shape[2] * DIM))
    for i in range(0, shape[0], step):
        x = torch.randn((min(step, shape[0] - i),) + shape[1:] + (DIM,), generator=gen, device="cuda", dtype=torch.float32)
        out[i:i + step] = _rows(x, scale)
    return out, scale


def _table(lens, perm):
    """Rows of block ids, [sequences][most blocks], from a random order of the blocks."""
    have = _i32([_ceil(x) for x in lens]).long()
    cols = torch.arange(max(1, max(_ceil(x) for x in lens)), device="cuda")
    at = (have.cumsum(0) - have)[:, None] + cols
    return torch.where(cols < have[:, None], perm[at.clamp(max=perm.numel() - 1)], 0).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    hkv = case["kv_heads"]
    if case["op"] == "write":
        n = case["tokens"]
        blocks = _ceil(n) + 2
        for name, heads in (("q", GROUP * hkv), ("k", hkv), ("v", hkv)):
            s[name] = torch.randn((n, heads, DIM), generator=gen, device="cuda", dtype=torch.bfloat16)
        # runs of neighbouring positions from random starts, as the tokens of several sequences lie
        run = 1 + torch.randint(0, 400, (1,), generator=gen, device="cuda")
        at = torch.arange(n, device="cuda")
        starts = torch.randint(0, case["pos_hi"], (n,), generator=gen, device="cuda")
        s["positions"] = ((starts[at // run] + at % run) % case["pos_hi"]).to(torch.int32)
        s["slots"] = torch.randperm(blocks * BLOCK, generator=gen, device="cuda")[:n].to(torch.int32)
        s["wq"] = s["wk"] = None
        if case["norm"]:
            s["wq"], s["wk"] = (1 + 0.1 * torch.randn((2, DIM), generator=gen, device="cuda")).to(torch.bfloat16)
        s["freq"], s["magnitude"] = _frequencies(case)
        s["freq"] = s["freq"].cuda()
        s["kv"], s["k_scale"] = _cache((2 * blocks, hkv, BLOCK), gen)
        s["kv"] = s["kv"].view(2, blocks, hkv, BLOCK, ROW)
        s["v_scale"] = s["k_scale"]
        s["q_out"] = torch.empty_like(s["q"])
        # the pair of values that each byte of codes stands for, as two e4m3 in one 16-bit word
        e2m1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device="cuda")
        byte = torch.arange(256, device="cuda")
        s["pairs"] = torch.stack([e2m1[byte & 15], e2m1[byte >> 4]], -1).to(torch.float8_e4m3fn).view(torch.int16)[:, 0].contiguous()
        if own:
            import paged_gqa_decode_hpc_gb300 as hpc
            band = {"banded": ("low", "high"), "ramp": ("slow", "fast")}.get(case["scaling"], ("low", "high"))
            s["rope"] = hpc.hpc_rope_init(rot_dim=case["rot_dim"], interleaved=case["interleaved"], base=ROPE["base"],
                                          scaling=case["scaling"], factor=ROPE["factor"], original_len=ROPE["original_len"],
                                          low=ROPE[band[0]], high=ROPE[band[1]])
        return s
    if case["op"] == "decode":
        lens, t = _lens(case), case["q_len"]
        shape = (len(lens), GROUP * hkv, DIM) if t == 1 else (len(lens), t, GROUP * hkv, DIM)
    else:
        new, lens = _lens(case)
        shape = (sum(new), GROUP * hkv, DIM)
        s["cu"] = _i32([sum(new[:i]) for i in range(len(new) + 1)])
        s["most"] = max(new)
    total = sum(_ceil(x) for x in lens) + 1
    s["tiles"] = sum(_ceil(x) for x in lens)
    s["k"], s["k_scale"] = _cache((total, hkv, BLOCK), gen)
    s["v"], s["v_scale"] = _cache((total, hkv, BLOCK), gen)
    s["table"] = _table(lens, torch.randperm(total, generator=gen, device="cuda"))
    s["lens"] = _i32(lens)
    s["q"] = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(shape[:-1], device="cuda", dtype=torch.float32)
    if own and case["op"] == "decode":
        import paged_gqa_decode_hpc_gb300 as hpc
        s["plan"] = hpc.hpc_decode_kv4_plan_create(len(lens), case["q_len"], hpc.hpc_device_sm_count(), GROUP * hkv)
    return s


def _values(rows, scale):
    """What rows stand for, in 32 bits: uint8 [..., 72] to float [..., 128]."""
    e2m1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=rows.device)
    code = rows[..., :DIM // 2].int()
    x = torch.stack([e2m1[code & 15], e2m1[code >> 4]], -1).flatten(-2)
    small = rows[..., DIM // 2:].contiguous().view(torch.float8_e4m3fn).float() * scale
    return (x.unflatten(-1, (DIM // SPAN, SPAN)) * small[..., None]).flatten(-2)


def _decode(s):
    """Scores, softmax and weighted sum of every 64-token block by itself, then the blocks of a sequence joined."""
    b, hkv, t = s["lens"].numel(), s["case"]["kv_heads"], s["case"]["q_len"]
    lens = s["lens"].long()
    q = s["q"].float().view(b, t, hkv, GROUP, DIM).permute(0, 2, 1, 3, 4).reshape(b, hkv, t * GROUP, DIM)
    have = (lens + BLOCK - 1) // BLOCK
    first = have.cumsum(0) - have
    seq = torch.repeat_interleave(torch.arange(b, device="cuda"), have, output_size=s["tiles"])
    tile = torch.arange(s["tiles"], device="cuda") - first[seq]
    block = s["table"][seq, tile].long()
    score = torch.matmul(q[seq], _values(s["k"][block], s["k_scale"]).transpose(2, 3)) / math.sqrt(DIM)
    seen = (lens[:, None] - (t - 1) + torch.arange(t, device="cuda")).repeat_interleave(GROUP, 1)  # keys that each row sees
    at = tile[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")
    score = score.masked_fill(at[:, None, None, :] >= seen[seq][:, None, :, None], -math.inf)
    top = score.amax(-1)
    p = torch.exp(score - torch.where(top > -math.inf, top, 0.0)[..., None])
    total = p.sum(-1)
    part = torch.matmul(p, _values(s["v"][block], s["v_scale"]))
    cols = torch.arange(s["table"].shape[1], device="cuda")
    mine = cols < have[:, None]
    index = torch.where(mine, first[:, None] + cols, 0)
    tops = torch.where(mine[..., None, None], top[index], -math.inf)
    most = tops.amax(1)
    weight = torch.exp(tops - torch.where(most > -math.inf, most, 0.0)[:, None])
    total = (weight * total[index]).sum(1)
    out = (weight[..., None] * part[index]).sum(1) / torch.where(total > 0, total, 1.0)[..., None]
    lse = most + torch.log(total)
    out = out.view(b, hkv, t, GROUP, DIM).permute(0, 2, 1, 3, 4).reshape(s["q"].shape)
    lse = lse.view(b, hkv, t, GROUP).permute(0, 2, 1, 3).reshape(s["lse"].shape)
    return {"out": out.to(torch.bfloat16), "lse": lse.contiguous()}


def _extend(s):
    """New tokens and positions padded to the longest: one masked softmax over all of them in 32 bits."""
    b, hkv, most = s["lens"].numel(), s["case"]["kv_heads"], s["most"]
    lens, cu = s["lens"].long(), s["cu"].long()
    new = cu[1:] - cu[:-1]
    token = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), token, right=True)
    place = token - cu[seq]
    q = torch.zeros((b, most) + s["q"].shape[1:], device="cuda")
    q[seq, place] = s["q"].float()
    q = q.view(b, most, hkv, GROUP, DIM).permute(0, 2, 3, 1, 4).reshape(b, hkv, GROUP * most, DIM)
    table = s["table"].long()
    n = table.shape[1] * BLOCK
    k = _values(s["k"][table], s["k_scale"]).permute(0, 2, 1, 3, 4).reshape(b, hkv, n, DIM)
    score = torch.matmul(q, k.transpose(2, 3)).view(b, hkv, GROUP, most, n)
    del k
    score /= math.sqrt(DIM)
    seen = (lens - new)[:, None] + 1 + torch.arange(most, device="cuda")
    score.masked_fill_((torch.arange(n, device="cuda") >= seen[..., None])[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = _values(s["v"][table], s["v_scale"]).permute(0, 2, 1, 3, 4).reshape(b, hkv, n, DIM)
    out = torch.matmul(p.view(b, hkv, GROUP * most, n), v).view(b, hkv, GROUP, most, DIM) / total
    lse = (top + torch.log(total))[..., 0]
    out = out.permute(0, 3, 1, 2, 4)[seq, place].reshape(s["q"].shape)
    return {"out": out.to(torch.bfloat16), "lse": lse.permute(0, 3, 1, 2)[seq, place].reshape(s["lse"].shape).contiguous()}


def _norm(x, w):
    x = x.double()
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.double()


def _rotate(x, cos, sin, r, interleaved):
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _seen(s):
    """The caches as the numbers that their codes and scales stand for."""
    codes = s["pairs"][s["kv"][..., :DIM // 2].int()].view(torch.float8_e4m3fn)
    scales = s["kv"][..., DIM // 2:].view(torch.float8_e4m3fn)
    return {"q": s["q_out"], "k_codes": codes[0], "v_codes": codes[1], "k_scales": scales[0], "v_scales": scales[1]}


def _write(s):
    """In 64 bits, because codes change at borders that a rounding in 32 can cross."""
    c = s["case"]
    angle = (s["positions"].double()[:, None] * s["freq"])[:, None]
    cos, sin = torch.cos(angle) * s["magnitude"], torch.sin(angle) * s["magnitude"]
    s["q_out"].copy_(_rotate(_norm(s["q"], s["wq"]), cos, sin, c["rot_dim"], c["interleaved"]))
    k = _rotate(_norm(s["k"], s["wk"]), cos, sin, c["rot_dim"], c["interleaved"])
    block, slot = s["slots"].long() // BLOCK, s["slots"].long() % BLOCK
    s["kv"][0][block, :, slot] = _rows(k, s["k_scale"])
    s["kv"][1][block, :, slot] = _rows(s["v"].double(), s["v_scale"])
    return _seen(s)


def _own(s):
    import paged_gqa_decode_hpc_gb300 as hpc
    op = s["case"]["op"]
    if op == "decode":
        hpc.hpc_decode_kv4_attn(s["q"], s["k"], s["v"], s["table"], s["lens"], s["plan"], s["out"], s["lse"],
                                k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "extend":
        hpc.hpc_extend_kv4_attn(s["q"], s["k"], s["v"], s["table"], s["lens"], s["cu"], s["out"], s["lse"],
                                k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"out": s["out"], "lse": s["lse"]}
    hpc.hpc_rope_kv4_write(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["rope"], s["q_out"], s["kv"][0], s["kv"][1],
                           q_norm_weight=s["wq"], k_norm_weight=s["wk"], eps=1e-6, k_scale=s["k_scale"], v_scale=s["v_scale"])
    return _seen(s)


def run(state):
    if own:
        return _own(state)
    return {"decode": _decode, "extend": _extend, "write": _write}[state["case"]["op"]](state)


def work(case):
    hkv = case["kv_heads"]
    if case["op"] == "decode":
        lens, t = _lens(case), case["q_len"]
        rows = len(lens) * t * GROUP * hkv
        pairs = sum(max(0, x - (t - 1) + i) for x in lens for i in range(t)) * GROUP * hkv
        return {"bytes": sum(lens) * hkv * 2 * ROW + rows * (DIM * 4 + 4) + 4 * sum(_ceil(x) + 1 for x in lens), "flops": 4.0 * DIM * pairs}
    if case["op"] == "extend":
        new, lens = _lens(case)
        pairs = sum(n * (x - n) + n * (n + 1) // 2 for n, x in zip(new, lens)) * GROUP * hkv
        return {"bytes": sum(lens) * hkv * 2 * ROW + sum(new) * GROUP * hkv * (DIM * 4 + 4) + 4 * sum(_ceil(x) + 2 for x in lens), "flops": 4.0 * DIM * pairs}
    n = case["tokens"]
    turned = 3.0 * n * (GROUP + 1) * hkv
    return {"bytes": n * (2 * DIM * (2 * GROUP + 2) * hkv + 2 * ROW * hkv + 8),
            "flops": turned * case["rot_dim"] + (turned * DIM if case["norm"] else 0) + 4.0 * n * hkv * DIM}


def _stands_for(rows, scale):
    """The rows' numbers in 64 bits, from the bits of e2m1 (sign, two of exponent, one of mantissa)."""
    n = torch.stack([rows[..., :64] & 15, rows[..., :64] >> 4], -1).flatten(-2).long()
    e, m = (n >> 1) & 3, (n & 1).double()
    mag = torch.where(e == 0, 0.5 * m, torch.exp2((e - 1).double()) * (1 + 0.5 * m))
    small = rows[..., 64:].contiguous().view(torch.float8_e4m3fn).double() * scale
    return torch.where(n >= 8, -mag, mag) * small.repeat_interleave(SPAN, -1)


def exact(case, seed):
    """The definitions in 64 bits, one sequence, or one head's pairs, at a time."""
    s = prepare(case, seed)
    if case["op"] != "write":
        hkv, lens, rows = case["kv_heads"], s["lens"].tolist(), s["table"].tolist()
        t = case["q_len"] if case["op"] == "decode" else None
        cu = s["cu"].tolist() if t is None else [i * t for i in range(len(lens) + 1)]
        q = s["q"].double().view(-1, hkv, GROUP, DIM)
        out, lse = torch.zeros_like(q), torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            if n == 0:
                continue
            ids = torch.tensor(rows[b][:_ceil(n)], device="cuda")
            k, v = (_stands_for(s[x][ids], s[x + "_scale"]).transpose(1, 2).reshape(-1, hkv, DIM)[:n] for x in ("k", "v"))
            for a in range(cu[b], cu[b + 1], 256):  # some of the new tokens at once
                z = min(a + 256, cu[b + 1])
                see = n - cu[b + 1] + 1 + torch.arange(a, z, device="cuda")
                logit = torch.einsum("ihgd,nhd->ihgn", q[a:z], k) * DIM ** -0.5
                logit[(torch.arange(n, device="cuda") >= see[:, None])[:, None, None].expand_as(logit)] = -math.inf
                lse[a:z] = torch.logsumexp(logit, -1)
                w = torch.exp(logit - lse[a:z][..., None]).nan_to_num(0.0)
                out[a:z] = torch.einsum("ihgn,nhd->ihgd", w, v)
        return {"out": out.view(s["q"].shape), "lse": lse.view(s["lse"].shape)}
    freq, magnitude = _frequencies(case)
    r = case["rot_dim"]
    got = {}
    angle = s["positions"].double()
    for name, w in (("q", s["wq"]), ("k", s["wk"])):
        x = s[name].double()
        if w is not None:
            x = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
        y = x.clone()
        for i, f in enumerate(freq.tolist()):
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
            c, d = (torch.cos(angle * f) * magnitude)[:, None], (torch.sin(angle * f) * magnitude)[:, None]
            y[..., a], y[..., b] = x[..., a] * c - x[..., b] * d, x[..., b] * c + x[..., a] * d
        got[name] = y
    block, slot = torch.div(s["slots"], BLOCK, rounding_mode="floor").long(), (s["slots"] % BLOCK).long()
    rows = s["v"].double()
    amax = rows.abs().view(rows.shape[:-1] + (DIM // SPAN, SPAN)).max(-1).values
    ts = float(torch.tensor(s["v_scale"], dtype=torch.float32))
    small = (amax / float(torch.tensor(6.0 * ts, dtype=torch.float32))).clamp(max=E4M3_MAX).float().to(torch.float8_e4m3fn)
    unit = (small.double() * ts).float().double().repeat_interleave(SPAN, -1)
    y = torch.where(unit > 0, rows / unit, 0.0).clamp(-E2M1_MAX, E2M1_MAX)
    # the nearest multiple of the step that e2m1 has at |y|: 0.5 below 2, then 1, 2 from 4 on (round() takes ties to even)
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    v_codes = _stands_for(torch.cat([s["kv"][1][..., :64], torch.full_like(s["kv"][1][..., 64:], 0x38)], -1), 1.0)  # (0x38: a scale of 1)
    v_codes[block, :, slot] = torch.round(y / step) * step
    k_scales, v_scales = (s["kv"][i][..., 64:].contiguous().view(torch.float8_e4m3fn).double() for i in (0, 1))
    v_scales[block, :, slot] = small.double()
    amax = got["k"].abs().view(rows.shape[:-1] + (DIM // SPAN, SPAN)).max(-1).values
    k_scales[block, :, slot] = (amax / (6.0 * s["k_scale"])).clamp(max=E4M3_MAX)  # what e4m3 rounds
    # K's codes are decisions at borders that its rotation's last bit can cross: held to the plain form's within their type
    return {"q": got["q"], "k_codes": None, "v_codes": v_codes, "k_scales": k_scales, "v_scales": v_scales}
