"""Measured cases of the operators around a paged KV cache whose sequences share a prefix.

Three groups of calls, as a serving loop makes them one after the other:

* ``append`` / ``truncate``: block tables, slot maps and positions of a step, built on the GPU from
  the lengths (new blocks popped from a stack of free ones; a rolled-back or finished sequence's
  blocks pushed again);
* ``rope``: optional QK-norm, rotary positions (half or interleaved pairs, all or part of the head,
  frequencies scaled for long contexts) of a ragged batch of tokens, and the write of K and V into
  the cache at the step's slots;
* ``prefix``: decode attention of groups of sequences whose first blocks are the same ones.

``run`` computes each in plain torch operations, or, where ``own`` is true, by the framework's calls.
"""
import math
import random

import torch

own = False

BLOCK = 64
DIM = 128
GROUP = 8  # query heads per KV head
E4M3_MAX = 448.0


def listed():
    return [
        # a handful of requests behind a short system prompt, one KV head: latency
        {"name": "prefix_tiny", "op": "prefix", "dtype": "bf16", "kv_heads": 1, "q_len": 1, "groups": 1, "seqs": 4,
         "prefix_lo": 200, "prefix_hi": 200, "suffix_lo": 1, "suffix_hi": 40},
        # a chat service: one system prompt, 32 conversations
        {"name": "prefix_chat", "op": "prefix", "dtype": "bf16", "kv_heads": 8, "q_len": 1, "groups": 1, "seqs": 32,
         "prefix_lo": 4096, "prefix_hi": 4096, "suffix_lo": 64, "suffix_hi": 1024},
        # 64 questions on one long document
        {"name": "prefix_document", "op": "prefix", "dtype": "bf16", "kv_heads": 8, "q_len": 1, "groups": 1, "seqs": 64,
         "prefix_lo": 32768, "prefix_hi": 32768, "suffix_lo": 128, "suffix_hi": 2048},
        # several tenants' prompts in one batch, e4m3 cache, ragged group sizes and lengths
        {"name": "prefix_tenants_fp8", "op": "prefix", "dtype": "fp8", "kv_heads": 8, "q_len": 1, "groups": 6, "seqs": 60,
         "prefix_lo": 1000, "prefix_hi": 16000, "suffix_lo": 1, "suffix_hi": 700},
        # speculative decoding: four draft tokens checked per sequence
        {"name": "prefix_drafts", "op": "prefix", "dtype": "bf16", "kv_heads": 8, "q_len": 4, "groups": 1, "seqs": 16,
         "prefix_lo": 8192, "prefix_hi": 8192, "suffix_lo": 100, "suffix_hi": 600},
        # one new token for each of 64 sequences, with QK-norm: the decode step's prologue
        {"name": "rope_decode", "op": "rope", "dtype": "bf16", "kv_heads": 8, "tokens": 64, "rot_dim": 128, "interleaved": False,
         "scaling": "none", "norm": True, "q_fp8": False, "pos_hi": 4096},
        # a prefill chunk at far positions, frequencies scaled by wavelength
        {"name": "rope_prefill", "op": "rope", "dtype": "bf16", "kv_heads": 8, "tokens": 8192, "rot_dim": 128, "interleaved": False,
         "scaling": "banded", "norm": False, "q_fp8": False, "pos_hi": 131072},
        # interleaved pairs on half of the head, e4m3 cache and an e4m3 copy of q, frequencies scaled by dimension
        {"name": "rope_partial_fp8", "op": "rope", "dtype": "fp8", "kv_heads": 8, "tokens": 1531, "rot_dim": 64, "interleaved": True,
         "scaling": "ramp", "norm": False, "q_fp8": True, "pos_hi": 65536},
        # an odd batch, three quarters of the head, positions interpolated
        {"name": "rope_odd", "op": "rope", "dtype": "bf16", "kv_heads": 2, "tokens": 333, "rot_dim": 96, "interleaved": False,
         "scaling": "linear", "norm": True, "q_fp8": False, "pos_hi": 16384},
        # a decode step of 256 sequences: one token each, a new block for every 64th
        {"name": "append_decode", "op": "append", "seqs": 256, "old_lo": 16, "old_hi": 4096, "new_lo": 1, "new_hi": 1},
        # prefill chunks of 512 requests at once, ragged
        {"name": "append_prefill", "op": "append", "seqs": 512, "old_lo": 0, "old_hi": 8192, "new_lo": 1, "new_hi": 2048},
        # rejected drafts and finished requests of a large batch
        {"name": "truncate_batch", "op": "truncate", "seqs": 1024, "len_lo": 1, "len_hi": 8192, "finished": 0.1, "back_hi": 130},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "prefix", "rope", "rope", "append", "truncate"])
    if op == "prefix":
        q_len = rng.choice([1, 1, 1, 2, 3, 5, 8])
        seqs = _log(rng, 1, 60 // q_len)
        groups = min(seqs, rng.choice([1, 1, 2, 3, 5]))
        p = _log(rng, 64, 30000 // groups)
        s = _log(rng, 1, 1800)
        return {"op": "prefix", "dtype": rng.choice(["bf16", "bf16", "fp8"]), "kv_heads": rng.choice([1, 2, 4, 8, 8]),
                "q_len": q_len, "groups": groups, "seqs": seqs,
                "prefix_lo": max(1, p // rng.choice([1, 2, 8])), "prefix_hi": p,
                "suffix_lo": max(1, s // rng.choice([1, 3, 10])) + q_len - 1, "suffix_hi": s + q_len - 1}
    if op == "rope":
        return {"op": "rope", "dtype": rng.choice(["bf16", "fp8"]), "kv_heads": rng.choice([1, 2, 4, 8]),
                "tokens": _log(rng, 1, 8000), "rot_dim": rng.choice([20, 32, 48, 64, 80, 90, 96, 112, 128]),
                "interleaved": rng.random() < 0.4, "scaling": rng.choice(["none", "linear", "base", "banded", "ramp"]),
                "norm": rng.random() < 0.5, "q_fp8": rng.random() < 0.3, "pos_hi": _log(rng, 64, 1 << 20)}
    if op == "append":
        new = _log(rng, 1, 2000)
        return {"op": "append", "seqs": _log(rng, 1, 500), "old_lo": 0, "old_hi": _log(rng, 1, 8000),
                "new_lo": max(0, new // rng.choice([1, 4]) - 1), "new_hi": new}
    return {"op": "truncate", "seqs": _log(rng, 1, 1000), "len_lo": 0, "len_hi": _log(rng, 64, 8000),
            "finished": rng.choice([0.0, 0.1, 0.5]), "back_hi": _log(rng, 1, 500)}


def _rng(case):
    """Lengths belong to the case; values come from the seed."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _ceil(a, b=BLOCK):
    return -(-a // b)


def _prefix_lens(case):
    """(sequences of each group, prefix length of each group, length of each sequence)."""
    rng = _rng(case)
    n, g = case["seqs"], case["groups"]
    cuts = sorted(rng.sample(range(1, n), g - 1)) if g > 1 else []
    sizes = [b - a for a, b in zip([0] + cuts, cuts + [n])]
    prefixes = [rng.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(g)]
    lens = [p + rng.randint(case["suffix_lo"], case["suffix_hi"]) for p, k in zip(prefixes, sizes) for _ in range(k)]
    return sizes, prefixes, lens


def _append_lens(case):
    rng = _rng(case)
    n = case["seqs"]
    return [rng.randint(case["old_lo"], case["old_hi"]) for _ in range(n)], [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(n)]


def _truncate_lens(case):
    rng = _rng(case)
    lens = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]
    return lens, [0 if rng.random() < case["finished"] else max(0, x - rng.randint(0, case["back_hi"])) for x in lens]


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


def _cache(shape, dtype, gen):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    if dtype == "bf16":
        return x, 1.0
    scale = float(x.abs().max()) / E4M3_MAX
    return (x.float() / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "prefix":
        sizes, prefixes, lens = _prefix_lens(case)
        hkv, t = case["kv_heads"], case["q_len"]
        shared = [p // BLOCK for p in prefixes]  # whole blocks are shared, the rest is each sequence's own
        owner = [g for g, k in enumerate(sizes) for _ in range(k)]
        total = sum(shared) + sum(_ceil(x) - shared[g] for x, g in zip(lens, owner))
        perm = torch.randperm(total, generator=gen, device="cuda").tolist()
        at, first, rows = 0, [], []
        for n in shared:
            first.append(perm[at:at + n])
            at += n
        width = max(_ceil(x) for x in lens)
        for x, g in zip(lens, owner):
            n = _ceil(x) - shared[g]
            rows.append(first[g] + perm[at:at + n] + [0] * (width - _ceil(x)))
            at += n
        b = len(lens)
        shape = (b, GROUP * hkv, DIM) if t == 1 else (b, t, GROUP * hkv, DIM)
        s["q"] = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
        s["k"], s["k_scale"] = _cache((total, hkv, BLOCK, DIM), case["dtype"], gen)
        s["v"], s["v_scale"] = _cache((total, hkv, BLOCK, DIM), case["dtype"], gen)
        s["table"], s["lens"] = _i32(rows), _i32(lens)
        s["groups"], s["prefixes"] = _i32([sum(sizes[:i]) for i in range(len(sizes) + 1)]), _i32(prefixes)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(shape[:-1], device="cuda", dtype=torch.float32)
        if own:
            import paged_gqa_decode_hpc_gb300 as hpc
            s["plan"] = hpc.hpc_decode_prefix_plan_create(b, t, hpc.hpc_device_sm_count(), GROUP * hkv)
    elif case["op"] == "rope":
        n, hkv = case["tokens"], case["kv_heads"]
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
        s["k_cache"], s["k_scale"] = _cache((blocks, hkv, BLOCK, DIM), case["dtype"], gen)
        s["v_cache"], s["v_scale"] = _cache((blocks, hkv, BLOCK, DIM), case["dtype"], gen)
        s["q_out"] = torch.empty_like(s["q"])
        s["q_scale"] = 4.0 / E4M3_MAX
        s["q_fp8"] = torch.empty(s["q"].shape, device="cuda", dtype=torch.float8_e4m3fn) if case["q_fp8"] else None
        if own:
            import paged_gqa_decode_hpc_gb300 as hpc
            band = {"banded": ("low", "high"), "ramp": ("slow", "fast")}.get(case["scaling"], ("low", "high"))
            s["rope"] = hpc.hpc_rope_init(rot_dim=case["rot_dim"], interleaved=case["interleaved"], base=ROPE["base"],
                                          scaling=case["scaling"], factor=ROPE["factor"], original_len=ROPE["original_len"],
                                          low=ROPE[band[0]], high=ROPE[band[1]])
    else:
        lens, other = _append_lens(case) if case["op"] == "append" else _truncate_lens(case)
        ends = [a + b for a, b in zip(lens, other)] if case["op"] == "append" else lens
        used = sum(_ceil(x) for x in lens)
        total = sum(_ceil(x) for x in ends) + 64
        perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
        width = max(1, max(_ceil(x) for x in ends))
        cols = torch.arange(width, device="cuda")
        have = _i32([_ceil(x) for x in lens]).long()
        at = (have.cumsum(0) - have)[:, None] + cols
        s["table"] = torch.where(cols < have[:, None], perm[at.clamp(max=total - 1)], torch.full_like(perm[:1], -1)).contiguous()
        s["free"] = torch.cat([perm[used:], torch.full((used,), -1, dtype=torch.int32, device="cuda")])
        s["count"], s["count_out"] = _i32([total - used]), _i32([0])
        s["lens"], s["other"], s["lens_out"] = _i32(lens), _i32(other), _i32([0] * len(lens))
        s["blocks"] = total
        if case["op"] == "append":
            n = sum(other)
            s["cu"] = _i32([0] * (len(lens) + 1))
            s["positions"], s["slots"] = _i32([0] * max(1, n)), _i32([0] * max(1, n))
    return s


def _softmax_attention(s):
    """Every sequence's keys and values gathered through its table, scores, softmax and weighted sum in 32 bits."""
    q, k, v = s["q"].float(), s["k"], s["v"]
    b, hkv, t = s["lens"].numel(), s["case"]["kv_heads"], s["case"]["q_len"]
    q = q.view(b, t, hkv, GROUP, DIM).permute(0, 2, 1, 3, 4).reshape(b, hkv, t * GROUP, DIM)
    table = s["table"].long()
    n = table.shape[1] * BLOCK
    k = k[table].permute(0, 2, 1, 3, 4).reshape(b, hkv, n, DIM).float()
    score = torch.matmul(q, k.transpose(2, 3)) * (s["k_scale"] / math.sqrt(DIM))
    del k
    seen = s["lens"].long()[:, None] - (t - 1) + torch.arange(t, device="cuda")  # keys that each new token sees
    hidden = torch.arange(n, device="cuda") >= seen.repeat_interleave(GROUP, 1)[:, None, :, None]
    score = score.masked_fill_(hidden, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = v[table].permute(0, 2, 1, 3, 4).reshape(b, hkv, n, DIM).float()
    out = torch.matmul(p, v) / total * s["v_scale"]
    lse = (top + torch.log(total))[..., 0]
    out = out.view(b, hkv, t, GROUP, DIM).permute(0, 2, 1, 3, 4).reshape(s["q"].shape)
    lse = lse.view(b, hkv, t, GROUP).permute(0, 2, 1, 3).reshape(s["lse"].shape)
    return {"out": out.to(torch.bfloat16), "lse": lse.contiguous()}


def _rotate(x, cos, sin, r, interleaved):
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    cos, sin = cos[:, None], sin[:, None]
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _norm(x, w):
    x = x.float()
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()


def _to_e4m3(x, scale):
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _rope_write(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["freq"]
    cos, sin = (torch.cos(angle) * s["magnitude"]).float(), (torch.sin(angle) * s["magnitude"]).float()
    q = _rotate(_norm(s["q"], s["wq"]), cos, sin, c["rot_dim"], c["interleaved"])
    k = _rotate(_norm(s["k"], s["wk"]), cos, sin, c["rot_dim"], c["interleaved"])
    block, slot = s["slots"].long() // BLOCK, s["slots"].long() % BLOCK
    if c["dtype"] == "fp8":
        s["k_cache"].view(torch.uint8)[block, :, slot] = _to_e4m3(k, s["k_scale"]).view(torch.uint8)
        s["v_cache"].view(torch.uint8)[block, :, slot] = _to_e4m3(s["v"].float(), s["v_scale"]).view(torch.uint8)
    else:
        s["k_cache"][block, :, slot] = k.to(torch.bfloat16)
        s["v_cache"][block, :, slot] = s["v"]
    got = {"q": q.to(torch.bfloat16), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if c["q_fp8"]:
        got["q_fp8"] = _to_e4m3(q, s["q_scale"])
    return got


def _append(s):
    old, end = s["lens"].long(), s["lens"].long() + s["other"].long()
    cu = torch.zeros_like(s["cu"])
    cu[1:] = s["other"].cumsum(0)
    b0, b1 = (old + BLOCK - 1) // BLOCK, (end + BLOCK - 1) // BLOCK
    off = (b1 - b0).cumsum(0) - (b1 - b0)
    cols = torch.arange(s["table"].shape[1], device="cuda")
    new = (cols >= b0[:, None]) & (cols < b1[:, None])
    at = s["count"].long() - 1 - (off - b0)[:, None] - cols
    table = torch.where(new, s["free"][at.clamp(0, s["free"].numel() - 1)], s["table"])
    token = torch.arange(s["slots"].numel(), device="cuda")
    seq = torch.searchsorted(cu[1:].long(), token, right=True).clamp(max=old.numel() - 1)
    pos = old[seq] + token - cu.long()[seq]
    live = token < cu[-1]
    block = table[seq, (pos // BLOCK).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(live, block * BLOCK + pos % BLOCK, -1)
    return {"table": table, "lens": end.to(torch.int32), "cu": cu, "positions": torch.where(live, pos, 0).to(torch.int32),
            "slots": slots.to(torch.int32), "count": (s["count"] - (b1 - b0).sum()).to(torch.int32)}


def _truncate(s):
    lens, keep = s["lens"].long(), torch.minimum(s["lens"], s["other"]).long()
    b0, b1 = (keep + BLOCK - 1) // BLOCK, (lens + BLOCK - 1) // BLOCK
    n = b1 - b0
    total = n.sum()
    cols = torch.arange(s["table"].shape[1], device="cuda")
    gone = (cols >= b0[:, None]) & (cols < b1[:, None])
    at = s["count"].long() + total - 1 - (n.cumsum(0) - n - b0)[:, None] - cols
    cap = s["free"].numel()
    free = torch.cat([s["free"], s["free"][:1]])  # one place more for the entries that stay
    free.scatter_(0, torch.where(gone, at, cap).flatten(), s["table"].flatten())
    return {"free": free[:cap], "lens": keep.to(torch.int32), "count": (s["count"] + total).to(torch.int32)}


def _own(s):
    import paged_gqa_decode_hpc_gb300 as hpc
    op = s["case"]["op"]
    if op == "prefix":
        hpc.hpc_decode_prefix_attn(s["q"], s["k"], s["v"], s["table"], s["lens"], s["prefixes"], s["plan"], s["out"], s["lse"],
                                   cu_groups=s["groups"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "rope":
        hpc.hpc_rope_kv_write(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["rope"], s["q_out"], s["k_cache"],
                              s["v_cache"], q_norm_weight=s["wq"], k_norm_weight=s["wk"], eps=1e-6, q_out_fp8=s["q_fp8"],
                              q_fp8_scale=s["q_scale"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        got = {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if s["q_fp8"] is not None:
            got["q_fp8"] = s["q_fp8"]
        return got
    if op == "append":
        hpc.hpc_block_table_append(s["lens"], s["other"], s["free"], s["count"], s["blocks"], s["table"], s["lens_out"],
                                   s["cu"], s["positions"], s["slots"], s["count_out"])
        return {"table": s["table"], "lens": s["lens_out"], "cu": s["cu"], "positions": s["positions"], "slots": s["slots"],
                "count": s["count_out"]}
    hpc.hpc_block_table_truncate(s["lens"], s["other"], s["table"], s["blocks"], s["free"], s["count"], s["lens_out"],
                                 s["count_out"])
    return {"free": s["free"], "lens": s["lens_out"], "count": s["count_out"]}


def run(state):
    if own:
        return _own(state)
    return {"prefix": _softmax_attention, "rope": _rope_write, "append": _append, "truncate": _truncate}[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op == "prefix":
        sizes, prefixes, lens = _prefix_lens(case)
        hkv, t = case["kv_heads"], case["q_len"]
        owner = [g for g, k in enumerate(sizes) for _ in range(k)]
        tokens = sum(prefixes) + sum(x - prefixes[g] for x, g in zip(lens, owner))  # each shared one once
        rows = len(lens) * t * GROUP * hkv
        pairs = sum(x - (t - 1) + i for x in lens for i in range(t)) * GROUP * hkv
        return {"bytes": tokens * hkv * DIM * 2 * (2 if case["dtype"] == "bf16" else 1) + rows * (DIM * 4 + 4), "flops": 4.0 * DIM * pairs}
    if op == "rope":
        n, hkv = case["tokens"], case["kv_heads"]
        heads = GROUP * hkv + 2 * hkv
        moved = n * DIM * (2 * heads + 2 * GROUP * hkv + 2 * hkv * (2 if case["dtype"] == "bf16" else 1) + (GROUP * hkv if case["q_fp8"] else 0))
        return {"bytes": moved + 8 * n, "flops": 3.0 * n * (GROUP + 1) * hkv * case["rot_dim"] + (3.0 * n * (GROUP + 1) * hkv * DIM if case["norm"] else 0)}
    if op == "append":
        old, new = _append_lens(case)
        blocks = sum(_ceil(a + b) - _ceil(a) for a, b in zip(old, new))
        part = sum(1 for a, b in zip(old, new) if a % BLOCK and b)
        return {"bytes": 4 * (4 * len(old) + 3 + 2 * blocks + part + 2 * sum(new)), "flops": float(2 * sum(new) + 4 * len(old))}
    lens, to = _truncate_lens(case)
    return {"bytes": 4 * (3 * len(lens) + 2 + 2 * sum(_ceil(a) - _ceil(min(a, b)) for a, b in zip(lens, to))), "flops": float(4 * len(lens))}


def exact(case, seed):
    """The definitions in 64 bits, one sequence, or one head's pairs, at a time."""
    s = prepare(case, seed)
    if case["op"] == "prefix":
        t, hkv = case["q_len"], case["kv_heads"]
        q = s["q"].double().view(-1, t, hkv, GROUP, DIM)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:-1], dtype=torch.float64, device="cuda")
        rows = s["table"].tolist()
        for b, n in enumerate(s["lens"].tolist()):
            ids = torch.tensor(rows[b][:_ceil(n)], device="cuda")
            k, v = (s[x][ids].double().transpose(1, 2).reshape(-1, hkv, DIM)[:n] * s[x + "_scale"] for x in ("k", "v"))
            for i in range(t):
                m = n - (t - 1) + i
                logit = torch.einsum("hgd,nhd->hgn", q[b, i], k[:m]) * DIM ** -0.5
                lse[b, i] = torch.logsumexp(logit, -1)
                out[b, i] = torch.einsum("hgn,nhd->hgd", torch.exp(logit - lse[b, i][..., None]), v[:m])
        return {"out": out.reshape(s["q"].shape), "lse": lse.reshape(s["lse"].shape)}
    if case["op"] == "rope":
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

        def scaled(x, scale):  # what the cache type rounds
            return (x / scale).clamp(-E4M3_MAX, E4M3_MAX)

        caches = {}
        for name, rows in (("k", got["k"]), ("v", s["v"].double())):
            c = s[name + "_cache"].double()
            c[block, :, slot] = scaled(rows, s[name + "_scale"]) if case["dtype"] == "fp8" else rows
            caches[name + "_cache"] = c
        if case["q_fp8"]:
            caches["q_fp8"] = scaled(got["q"], s["q_scale"])
        return {"q": got["q"], **caches}
    return None
