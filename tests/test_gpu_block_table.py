"""hpc_block_table_append / _truncate against the oracle's plain loops: whole
numbers, so every word is equal, error bits included."""
import random

import pytest
import torch

import paged_gqa_decode_hpc_gb300 as hpc
from oracle import block_table_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    hpc.load_library()


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _case(rng, B, old_hi, new_hi, spare=3, pad=0, width_more=1):
    old = [rng.randint(0, old_hi) for _ in range(B)]
    new = [rng.randint(0, new_hi) for _ in range(B)]
    width = max([1] + [R.blocks_of(o + n) for o, n in zip(old, new)]) + width_more
    total = sum(R.blocks_of(o + n) for o, n in zip(old, new)) + spare
    ids = list(range(total))
    rng.shuffle(ids)
    table = [[ids.pop() for _ in range(R.blocks_of(o))] + [-1] * (width - R.blocks_of(o)) for o in old]
    free = ids + [-1] * (total - len(ids))
    return dict(old=old, new=new, table=table, free=free, count=len(ids), blocks=total, width=width,
                cap=sum(new) + pad)


def _table(c):
    return _dev(c["table"]).reshape(len(c["old"]), c["width"])


def _append(c, in_place=False, table=None, stream=None):
    B = len(c["old"])
    lens, count = _dev(c["old"]), _dev([c["count"]])
    table = _table(c) if table is None else table
    out = dict(table=table, lens=lens if in_place else _dev([77] * B), cu=_dev([77] * (B + 1)),
               positions=_dev([77] * c["cap"]), slots=_dev([77] * c["cap"]),
               count=count if in_place else _dev([77]), err=_dev([0]))
    free = _dev(c["free"])
    hpc.hpc_block_table_append(lens, _dev(c["new"]), free, count, c["blocks"], table, out["lens"],
                               out["cu"], out["positions"], out["slots"], out["count"],
                               device_error=out["err"], stream=stream)
    torch.cuda.synchronize()
    assert free.tolist() == c["free"]
    return out


def _check_append(c, out):
    ref, bits = R.append(c["old"], c["new"], c["free"], c["count"], c["blocks"], c["table"],
                         c["cap"], c["width"])
    assert out["err"].item() == bits
    assert out["count"].item() == ref["count"]
    for k in ("table", "lens", "cu", "positions", "slots"):
        assert out[k].tolist() == ref[k], k
    return ref, bits


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,old_hi,new_hi,pad", [
    (0, 0, 0, 0), (0, 0, 0, 5), (1, 0, 1, 0), (1, 200, 300, 0), (3, 64, 0, 2), (7, 130, 1, 0),
    (33, 500, 70, 9), (256, 4096, 1, 0), (1000, 300, 5, 100), (1025, 90, 64, 1), (40, 3000, 2000, 333),
    (5000, 100, 2, 0)])
def test_append(B, old_hi, new_hi, pad, in_place):
    c = _case(random.Random(B + old_hi), B, old_hi, new_hi, pad=pad)
    _check_append(c, _append(c, in_place))


def test_append_largest_batch():
    c = _case(random.Random(1), 16384, 70, 3, pad=7)
    _check_append(c, _append(c))


def test_append_strided_table_keeps_its_gaps():
    c = _case(random.Random(3), 20, 300, 200)
    wide = torch.full((20, c["width"] + 5), 55, dtype=torch.int32, device="cuda")
    view = wide[:, 2:2 + c["width"]]
    view.copy_(_table(c))
    _check_append(c, _append(c, table=view))
    assert (wide[:, :2] == 55).all() and (wide[:, 2 + c["width"]:] == 55).all()


def test_append_into_unaligned_buffers():
    c = _case(random.Random(5), 30, 200, 90, pad=3)
    buf = [_dev([77] * (c["cap"] + 6)) for _ in range(2)]
    B = 30
    out = dict(table=_table(c), lens=_dev([0] * B), cu=_dev([0] * (B + 1)), positions=buf[0][1:1 + c["cap"]],
               slots=buf[1][3:3 + c["cap"]], count=_dev([0]), err=_dev([0]))
    hpc.hpc_block_table_append(_dev(c["old"]), _dev(c["new"]), _dev(c["free"]), _dev([c["count"]]), c["blocks"], out["table"],
                               out["lens"], out["cu"], out["positions"], out["slots"], out["count"], device_error=out["err"])
    _check_append(c, out)
    assert buf[0][0] == 77 and (buf[0][1 + c["cap"]:] == 77).all() and (buf[1][:3] == 77).all() and (buf[1][3 + c["cap"]:] == 77).all()


def _refused(name):
    c = _case(random.Random(9), 12, 200, 100, pad=2)
    if name == "negative length":
        c["old"][5] = -1
    elif name == "negative new":
        c["new"][3] = -4
    elif name == "past int32":
        c["old"][2], c["new"][2] = 2**31 - 5, 100
    elif name == "table too short":
        c["width"] -= 2
        c["table"] = [r[:c["width"]] for r in c["table"]]
    elif name == "too many tokens":
        c["cap"] -= 3
    elif name == "no blocks":
        c["count"] = 2
    elif name == "count past the stack":
        c["count"] = len(c["free"]) + 1
    elif name == "negative count":
        c["count"] = -1
    elif name == "several":
        c["old"][5], c["count"], c["cap"] = -1, 1, 1
    return c


@pytest.mark.parametrize("name", ["negative length", "negative new", "past int32", "table too short",
                                  "too many tokens", "no blocks", "count past the stack",
                                  "negative count", "several"])
@pytest.mark.parametrize("in_place", [False, True])
def test_append_refuses_as_a_whole(name, in_place):
    c = _refused(name)
    _, bits = _check_append(c, _append(c, in_place))
    assert bits


@pytest.mark.parametrize("in_place", [False, True])
def test_append_of_many_tokens_refused(in_place):
    c = _case(random.Random(6), 60, 500, 2000, pad=5)
    assert c["cap"] > 32768
    c["count"] -= 4  # one block too few
    _, bits = _check_append(c, _append(c, in_place))
    assert bits == R.NO_BLOCKS


def test_append_huge_sums_do_not_wrap():
    # 3000 sequences of 2^30 new tokens: the sum passes 2^41
    c = dict(old=[0] * 3000, new=[2**30] * 3000, table=[[-1]] * 3000, free=[0], count=1, blocks=1,
             width=1, cap=4)
    B = 3000
    out = dict(err=_dev([0]), slots=_dev([7] * 4), positions=_dev([7] * 4), cu=_dev([7] * (B + 1)),
               lens=_dev([7] * B), count=_dev([7]))
    hpc.hpc_block_table_append(_dev(c["old"]), _dev(c["new"]), _dev([0]), _dev([1]), 1,
                               _dev(c["table"]), out["lens"], out["cu"], out["positions"],
                               out["slots"], out["count"], device_error=out["err"])
    assert out["err"].item() == R.TABLE_TOO_SHORT | R.CAPACITY | R.NO_BLOCKS
    assert out["slots"].tolist() == [-1] * 4 and out["count"].item() == 1


def test_append_bad_ids():
    c = _case(random.Random(4), 6, 100, 200, spare=0)
    c["free"][c["count"] - 1] = c["blocks"]       # popped first
    c["table"][2][0] = -7                          # partly filled block of sequence 2
    c["old"][2], c["new"][2] = 20, 10
    c["count"] = c["count"]
    ref, bits = _check_append(c, _append(c))
    assert bits in (R.BAD_BLOCK, R.BAD_BLOCK | R.NO_BLOCKS)


def _truncate(c, to, in_place=False):
    lens, count, free = _dev(c["old"]), _dev([c["count"]]), _dev(c["free"])
    lo = lens if in_place else _dev([77] * len(c["old"]))
    co = count if in_place else _dev([77])
    err, table = _dev([0]), _table(c)
    hpc.hpc_block_table_truncate(lens, _dev(to), table, c["blocks"], free, count, lo, co,
                                 device_error=err)
    torch.cuda.synchronize()
    assert table.tolist() == c["table"]
    ref, bits = R.truncate(c["old"], to, c["table"], c["blocks"], c["free"], c["count"], c["width"])
    assert err.item() == bits
    assert free.tolist() == ref["free"] and lo.tolist() == ref["lens"] and co.item() == ref["count"]
    return bits


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,hi", [(0, 0), (1, 1), (1, 700), (9, 64), (256, 4096), (1025, 300), (3000, 65)])
def test_truncate(B, hi, in_place):
    rng = random.Random(B + hi)
    c = _case(rng, B, hi, 0)
    to = [rng.choice([0, rng.randint(0, hi), x, x + 9, 2**31 - 1]) for x in c["old"]]
    assert _truncate(c, to, in_place) == 0


@pytest.mark.parametrize("name", ["negative length", "negative to", "table", "stack", "bad id"])
def test_truncate_refusals(name):
    c = _case(random.Random(8), 10, 400, 0)
    to = [0] * 10
    if name == "negative length":
        c["old"][3] = -5
    elif name == "negative to":
        to[4] = -1
    elif name == "table":
        c["old"][1] = 64 * c["width"] + 1
    elif name == "stack":
        c["free"] = c["free"][:c["count"] + 2]
    else:
        c["old"][0], c["table"][0][0] = 30, c["blocks"] + 3
    assert _truncate(c, to)


def test_steps_in_a_captured_graph_and_on_another_stream():
    """Append one token in place and roll every second sequence back, as two
    graphs of different buffers replayed on two streams at once: each loop's
    state must go its own way, as the oracle's does."""
    rng = random.Random(2)
    loops = []
    for _ in range(2):
        c = _case(rng, 50, 300, 0, spare=60, width_more=3)
        c["new"] = [1] * 50
        c["cap"] = 64
        t = dict(lens=_dev(c["old"]), new=_dev(c["new"]), free=_dev(c["free"]), count=_dev([c["count"]]),
                 table=_table(c), cu=_dev([0] * 51), pos=_dev([0] * 64), slots=_dev([0] * 64),
                 to=_dev([x if i % 2 else 2**31 - 1 for i, x in enumerate(c["old"])]), err=_dev([0]))

        def step(t=t, n=c["blocks"]):
            hpc.hpc_block_table_append(t["lens"], t["new"], t["free"], t["count"], n, t["table"],
                                       t["lens"], t["cu"], t["pos"], t["slots"], t["count"],
                                       device_error=t["err"])
            hpc.hpc_block_table_truncate(t["lens"], t["to"], t["table"], n, t["free"], t["count"],
                                         t["lens"], t["count"], device_error=t["err"])
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        keep = {k: v.clone() for k, v in t.items()}
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()  # before the capture: attributes are set once
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            step()
        for k, v in t.items():
            v.copy_(keep[k])
        loops.append((c, t, g, s))
    torch.cuda.synchronize()
    for _ in range(70):
        for _, _, g, s in loops:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, t, _, _ in loops:
        lens, count, free, table = c["old"], c["count"], c["free"], c["table"]
        to = [x if i % 2 else 2**31 - 1 for i, x in enumerate(c["old"])]
        for _ in range(70):
            a, bits = R.append(lens, c["new"], free, count, c["blocks"], table, 64, c["width"])
            assert bits == 0
            table = a["table"]
            b, bits = R.truncate(a["lens"], to, table, c["blocks"], free, a["count"], c["width"])
            assert bits == 0
            lens, count, free = b["lens"], b["count"], b["free"]
        assert t["lens"].tolist() == lens and t["count"].item() == count and t["err"].item() == 0
        assert t["free"].tolist()[:count] == free[:count]
        for r, row, n in zip(t["table"].tolist(), table, lens):
            assert r[:R.blocks_of(n)] == row[:R.blocks_of(n)]
        assert t["slots"].tolist() == a["slots"]
