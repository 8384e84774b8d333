"""The whole streaming loop of every compiled kernel of attention over caches in 4 bits keeps out of scratch memory (CPU): all
blocks of the loop, wherever the compiler has put them, and with all of a tile's matrix instructions in it."""
import re

import pytest

from test_kv_fp4_wait_states import listing  # noqa: F401  (a fixture)


def blocks(lines):
    """Basic blocks [first, last) of a kernel's lines, and the blocks that each can go to."""
    at = {x[:-1]: i for i, x in enumerate(lines) if x.endswith(":")}
    ends = ("s_branch", "s_cbranch", "s_endpgm")
    first = sorted({0} | set(at.values()) | {i + 1 for i, x in enumerate(lines) if x.startswith(ends) and i + 1 < len(lines)})
    index = {i: b for b, i in enumerate(first)}
    spans = [(i, first[b + 1] if b + 1 < len(first) else len(lines)) for b, i in enumerate(first)]
    to = []
    for b, (lo, hi) in enumerate(spans):
        last, go = lines[hi - 1], []
        m = re.match(r"s_c?branch\w*\s+(\.LBB\w+)", last)
        if m:
            go.append(index[at[m[1]]])
        if not last.startswith(("s_branch", "s_endpgm")) and b + 1 < len(spans):
            go.append(b + 1)
        to.append(go)
    return spans, to


def natural_loops(to):
    """Head -> blocks of the loop: those that reach a branch back to the head without passing it, the head before every one of them."""
    n = len(to)
    back = [[] for _ in range(n)]
    for b, go in enumerate(to):
        for x in go:
            back[x].append(b)
    reached, todo = {0}, [0]
    while todo:
        for x in to[todo.pop()]:
            if x not in reached:
                reached.add(x)
                todo.append(x)
    dom = {b: set(reached) for b in reached}
    dom[0] = {0}
    moved = True
    while moved:
        moved = False
        for b in sorted(reached - {0}):
            new = {b} | set.intersection(*[dom[p] for p in back[b] if p in reached])
            if new != dom[b]:
                dom[b], moved = new, True
    loops = {}
    for b in reached:
        for head in to[b]:
            if head in dom[b]:
                body, todo = {head, b}, [b]
                while todo:
                    x = todo.pop()
                    if x == head:
                        continue
                    for p in back[x]:
                        if p in reached and p not in body:
                            body.add(p)
                            todo.append(p)
                loops.setdefault(head, set()).update(body)
    return loops


def streaming_loop(lines):
    """Instructions of the innermost loop that has matrix instructions (with every branch back to its head)."""
    spans, to = blocks(lines)
    of = lambda body: [x for b in sorted(body) for x in lines[spans[b][0]:spans[b][1]]]  # noqa: E731
    found = [of(body) for body in natural_loops(to).values()]
    found = [x for x in found if any(y.startswith("v_mfma") for y in x)]
    return min(found, key=len)


def products(name):
    """Matrix instructions of a tile of 32 positions: both products, of NQ tiles of 16 query heads under NH key heads."""
    D, NQ, NH = (int(x) for x in re.search(r"ELi(\d+)ELi(\d+)ELi(\d+)E", name).groups())
    return NH * NQ * (2 * D // 32 + D // 16)


def test_the_search_takes_a_loop_s_blocks_wherever_they_lie():
    lines = ["s_branch .LBB0_2", ".LBB0_1:", "v_mfma_b", "s_cbranch_scc0 .LBB0_4", ".LBB0_2:", "v_mfma_a", "s_cbranch_vccz .LBB0_5", ".LBB0_3:",
             "s_branch .LBB0_1", ".LBB0_4:", "s_endpgm", ".LBB0_5:", "scratch_store_dword", "s_branch .LBB0_3"]
    got = streaming_loop(lines)
    assert [x for x in got if x.startswith("v_mfma")] == ["v_mfma_b", "v_mfma_a"] and "scratch_store_dword" in got and "s_endpgm" not in got


def test_every_tile_s_products_are_in_the_loop_and_no_scratch_access(listing):  # noqa: F811
    for name, lines in listing.items():
        loop = streaming_loop(lines)
        assert sum(x.startswith("v_mfma") for x in loop) == products(name), name
        assert not [x for x in loop if x.startswith("scratch_")], name
