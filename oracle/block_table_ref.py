"""ORACLE (test infrastructure only): block tables and slot maps by plain loops.

Only tests/ may use it. A sequence of L tokens holds ceil(L / 64) blocks; new
blocks come off the top of a stack of free ids, sequence by sequence, and a
shortened sequence's blocks go back so that the first one released ends on
top. See hpc_block_table_append / hpc_block_table_truncate in
include/hpc_decode.h for the refusals.
"""
from __future__ import annotations

from typing import List, Tuple

BLOCK = 64
BAD_LENGTH, BAD_BLOCK, TABLE_TOO_SHORT, CAPACITY, NO_BLOCKS = 1, 2, 4, 16, 32


def blocks_of(tokens: int) -> int:
    return -(-tokens // BLOCK)


def append(lens: List[int], new: List[int], free: List[int], count: int, num_blocks: int,
           table: List[List[int]], cap_tokens: int, max_blocks: int) -> Tuple[dict, int]:
    """(outputs, error bits); nothing given is changed."""
    table = [list(r) for r in table]
    bits = CAPACITY if not 0 <= count <= len(free) else 0
    need = tokens = 0
    for o, n in zip(lens, new):
        if o < 0 or n < 0 or o + n > 2**31 - 1:
            bits |= BAD_LENGTH
            continue
        if blocks_of(o + n) > max_blocks:
            bits |= TABLE_TOO_SHORT
        need += blocks_of(o + n) - blocks_of(o)
        tokens += n
    if tokens > cap_tokens:
        bits |= CAPACITY
    if need > count:
        bits |= NO_BLOCKS
    if bits:
        return dict(table=table, lens=list(lens), cu=[0] * (len(lens) + 1), count=count,
                    positions=[0] * cap_tokens, slots=[-1] * cap_tokens), bits
    stack = list(free[:count])
    cu, positions, slots = [0], [], []
    for b, (o, n) in enumerate(zip(lens, new)):
        for j in range(blocks_of(o), blocks_of(o + n)):
            ident = stack.pop()
            if not 0 <= ident < num_blocks:
                bits, ident = bits | BAD_BLOCK, -1
            table[b][j] = ident
        for pos in range(o, o + n):
            ident = table[b][pos // BLOCK]
            ok = 0 <= ident < num_blocks
            bits |= 0 if ok else BAD_BLOCK
            positions.append(pos)
            slots.append(ident * BLOCK + pos % BLOCK if ok else -1)
        cu.append(cu[-1] + n)
    pad = cap_tokens - tokens
    return dict(table=table, lens=[o + n for o, n in zip(lens, new)], cu=cu, count=len(stack),
                positions=positions + [0] * pad, slots=slots + [-1] * pad), bits


def truncate(lens: List[int], to: List[int], table: List[List[int]], num_blocks: int,
             free: List[int], count: int, max_blocks: int) -> Tuple[dict, int]:
    free = list(free)
    bits = CAPACITY if not 0 <= count <= len(free) else 0
    gone = []
    for b, (n, t) in enumerate(zip(lens, to)):
        if n < 0 or t < 0:
            bits |= BAD_LENGTH
            continue
        k = min(n, t)
        if blocks_of(n) > blocks_of(k) and blocks_of(n) > max_blocks:
            bits |= TABLE_TOO_SHORT
        gone += [(b, j) for j in range(blocks_of(k), blocks_of(n))]
    if count + len(gone) > len(free):
        bits |= CAPACITY
    if bits:
        return dict(free=free, lens=list(lens), count=count), bits
    for b, j in reversed(gone):
        ident = table[b][j]
        if not 0 <= ident < num_blocks:
            bits, ident = bits | BAD_BLOCK, -1
        free[count] = ident
        count += 1
    return dict(free=free, lens=[min(n, t) for n, t in zip(lens, to)], count=count), bits
