"""What a warp's lanes may rely on after a wait that only some of them made (CPU model of the memory order, and the order
of the statements in the kernels' sources). A lane that sees a barrier's phase acquires what its arrivals released; a vote
or a shuffle orders no memory; a warp barrier hands on what any lane has acquired."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_gqa_decode_hpc_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


class Warp:
    def __init__(self):
        self.known = [set() for _ in range(32)]

    def look(self, lane, released):
        self.known[lane] |= released

    def vote(self):
        pass

    def barrier(self):
        every = set().union(*self.known)
        self.known = [set(every) for _ in range(32)]

    def use(self, lanes, needs):
        return all(needs <= self.known[i] for i in lanes)


# the waits on two barriers of kv4_tc_kernel.cu: what either releases, and the lanes that then rely on both
WAITS = {
    "K to f16": ({"ring slot's bytes"}, {"K's columns read by the MMAs"}, range(32)),
    "V to f16": ({"ring slot's bytes"}, {"V's tile read by the MMAs"}, range(32)),
    "scores' MMAs": ({"K's columns"}, {"scores read"}, [0]),
    "values' MMAs": ({"P^T"}, {"V's tile"}, [0]),
    "values' MMAs, by another lane": ({"P^T"}, {"V's tile"}, [31]),
    "softmax": ({"scores"}, {"P^T read by the MMAs"}, range(32)),
}


def two_barriers(a, b, steps):
    w = Warp()
    for lane in range(32):
        w.look(lane, b if lane & 1 else a)
    for step in steps:
        getattr(w, step)()
    return w


def steps_of_wait2():
    """What wait2 does after the lanes' looks, in the order of its statements: the vote lies in wait()."""
    body = re.search(r"auto wait2 = \[&\].*?\n  };", source("kv4_tc_kernel.cu"), re.S).group(0)
    return [{"wait(": "vote", "__syncwarp()": "barrier"}[x] for x in re.findall(r"\bwait\(|__syncwarp\(\)", body)]


@pytest.mark.parametrize("name", WAITS)
def test_a_wait_on_two_barriers_orders_both_for_every_lane(name):
    a, b, lanes = WAITS[name]
    assert two_barriers(a, b, steps_of_wait2()).use(lanes, a | b)


@pytest.mark.parametrize("name", WAITS)
def test_a_vote_alone_does_not(name):
    a, b, lanes = WAITS[name]
    assert not two_barriers(a, b, ["vote"]).use(lanes, a | b)


def test_rows_of_q_are_copied_behind_what_lane_0_has_seen():
    """kv4_decode_kernel.cu: lane 0 waits for a piece's slot, eight lanes copy rows of q into it."""
    body = re.search(r"auto publish = .*?\n    };", source("kv4_decode_kernel.cu"), re.S).group(0)
    before = body[body.index("wait_phase("):body.index("kv4_copy(")]
    steps = [{"__shfl_sync(": "vote", "__syncwarp()": "barrier"}[x] for x in re.findall(r"__shfl_sync\(|__syncwarp\(\)", before)]

    def after(steps):
        w = Warp()
        w.look(0, {"the slot's rows read"})
        for step in steps:
            getattr(w, step)()
        return w.use(range(8), {"the slot's rows read"})
    assert after(steps) and not after(["vote"])


def lanes_that_go_on(guard, turns_at):
    """The lanes that a guard lets through where they read the abort flag one after another and it turns between two."""
    mine = [lane < turns_at for lane in range(32)]
    return sum([all(mine)] * 32 if "__all_sync(" in guard or "any_of(" in guard else mine)


def guards_of_flag(name, start, end):
    """The conditions that read the abort flag between two marks of a source, of code that a whole warp runs."""
    body = source(name)
    body = body[body.index(start):]
    body = body[:body.index(end)]
    return [x for x in re.findall(r"if \((.*)\) (?:\{|break)", body) if "s_abort" in x or "wait_phase(" in x]


def test_the_extend_epilogue_of_two_chains_stays_together():
    """Loads of tensor memory are a whole warp's: all of its lanes make them or none does."""
    guards = guards_of_flag("prefill_kernel.cu", "const float2 other = others[r];", "tmem_ld32(")
    assert len(guards) == 1
    for guard in guards:
        assert all(lanes_that_go_on(guard, t) in (0, 32) for t in range(33))
    assert lanes_that_go_on("ok && !*s_abort", 7) == 7


def test_a_consumer_warp_leaves_together():
    """kv4_decode_kernel.cu: a lane whose wait for a descriptor has run out takes its warp along, for the others would go on
    to shuffles."""
    body = source("kv4_decode_kernel.cu")
    body = body[body.index("regs_inc<C::kRegsConsumer>();"):]
    body = body[:body.index("named_bar_sync(3")]
    ways_out = re.findall(r"if \((.*)\)\s+break;", body)
    assert "fl & kFlagEnd" in ways_out  # (of the descriptor: the same for all)
    ways_out.remove("fl & kFlagEnd")
    assert len(ways_out) == 1
    assert all(lanes_that_go_on(ways_out[0], t) in (0, 32) for t in range(33))


def test_the_warp_that_copies_q_is_together_at_the_last_barrier():
    """kv4_tc_kernel.cu: after an abort lane 0 alone waits for copies under way; the barrier behind is the whole warp's."""
    body = source("kv4_tc_kernel.cu")
    body = body[body.index("for (int j = q_pieces"):]
    assert "lane == 0" in body[:body.index("wait_phase(")]
    assert "__syncwarp()" in body[body.index("wait_phase("):body.index("named_bar_sync(3")]


def test_the_step_kernel_s_warps_leave_together():
    """step_kernel.cu: the same waits, of its consumer and its epilogue warps, behind which shuffles and warp barriers come."""
    body = source("step_kernel.cu")
    for start in ("for (int j = warp - kEpilogueWarp0;;", "const int w = warp;"):
        part = body[body.index(start):]
        part = part[:part.index("named_bar_sync(3")]
        ways_out = [x for x in re.findall(r"if \(([^;{}]*)\)\s+break;", part) if x != "fl & kFlagEnd"]
        assert ways_out
        for guard in ways_out:
            assert all(lanes_that_go_on(guard, t) in (0, 32) for t in range(33)), guard
