"""The handshakes between the tensor cores and the softmax warps of the attention over the 4-bit cache, followed on the
CPU through every order that the roles can run in. An mbarrier tells its phases apart by one bit of parity: a phase that
is over twice before a role has looked once is taken for one that is still to come, and the role waits for nothing.

The barriers and parities of each wait and commit are read from the kernel's source; the roles' order of them is here."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_attention_sequence_gb300", "csrc",
                      "cache4_attn_tc.cu")
WARPS = 2  # softmax warps: one that is late and one that is not


def place(text):
    """`&bar[i]` or `bar`: (its name, the index as a function of the tile)."""
    m = re.fullmatch(r"&?(\w+)(?:\[(.*)\])?", text.strip())
    return m.group(1), m.group(2) or "0"


@pytest.fixture(scope="module")
def source():
    with open(SOURCE, encoding="utf-8") as f:
        return f.read()


def wait_of(source, site):
    """((barrier, index), parity) of the wait with that site number."""
    m = re.search(r"pass\(([^;]*?), ([^;]*?), (?:t\.)?abort_flag, %d\)" % site, source)
    return place(m.group(1)), m.group(2)


def commit_of(source, name):
    m = re.search(r"mma_commit_warp\((&?%s(?:\[[^]]*\])?)\)" % name, source)
    return place(m.group(1))


def at(expression, tile):
    return int(eval(expression, {}, {"n": tile, "m": tile}))


def roles(source, pieces):
    """The products' and a softmax warp's steps: ("wait", barrier, parity, phase), ("commit", barrier) when the products
    issued so far are done, ("arrive", barrier)."""
    def wait(site, tile):
        (name, index), parity = wait_of(source, site)
        bar = (name, at(index, tile))
        # which phase of its barrier this is: as many as the tiles before it that have the same place
        phase = sum(at(index, k) == bar[1] for k in range(tile))
        return ("wait", bar, at(parity, tile) & 1, phase)

    def before(site, tile):  # a wait written for tile n that is for tile n - 1's products
        (name, index), parity = wait_of(source, site)
        return ("wait", (name, at(index, tile)), at(parity, tile) & 1, tile - 1)

    def commit(name, tile):
        bar, index = commit_of(source, name)
        return ("commit", (bar, at(index, tile)))
    products, softmax, n = [], [], 0
    for piece, tiles in enumerate(pieces):
        products.append(("wait", ("q_full", 0), piece & 1, piece))
        softmax.append(("arrive", ("q_full", 0)))
        for j in range(tiles):
            products.append(commit("s_full", n))
            if j > 0:
                products += [wait(411, n - 1), commit("pv_done", n - 1)]
            softmax.append(wait(421, n))
            if j > 0:
                softmax.append(before(422, n))
            softmax.append(("arrive", ("p_full", 0)))
            n += 1
        products += [wait(411, n - 1), commit("pv_done", n - 1)]
        softmax.append(before(423, n))
    return products, softmax


def run(source, pieces):
    """Every reachable state; fails on a wait that passes too early and on states that nothing leads out of."""
    products, softmax = roles(source, pieces)
    bars = sorted({s[1] for s in products + softmax})
    number = {b: i for i, b in enumerate(bars)}
    need = [WARPS if b[0] in ("q_full", "p_full") else 1 for b in bars]
    # state: the products' step, commits under way, each warp's step, arrivals at each barrier
    start = (0, (), (0,) * WARPS, (0,) * len(bars))
    seen, todo = {start}, [start]

    def passes(step, arrived):
        _, bar, parity, phase = step
        over = arrived[number[bar]] // need[number[bar]]  # phases that are over
        if (over & 1) == parity:
            return False
        assert over > phase, f"{bar}: phase {phase} passed after {over}"
        return True

    def arrive(arrived, bar):
        i = number[bar]
        return arrived[:i] + (arrived[i] + 1,) + arrived[i + 1:]
    while todo:
        state = todo.pop()
        p, under_way, warps, arrived = state
        out = []
        if p < len(products):
            step = products[p]
            if step[0] == "commit":
                out.append((p + 1, under_way + (step[1],), warps, arrived))
            elif passes(step, arrived):
                out.append((p + 1, under_way, warps, arrived))
        if under_way:
            out.append((p, under_way[1:], warps, arrive(arrived, under_way[0])))
        for w in range(WARPS):
            if warps[w] == len(softmax):
                continue
            step = softmax[warps[w]]
            moved = warps[:w] + (warps[w] + 1,) + warps[w + 1:]
            if step[0] == "arrive":
                out.append((p, under_way, moved, arrive(arrived, step[1])))
            elif passes(step, arrived):
                out.append((p, under_way, moved, arrived))
        if not out:
            stuck = [softmax[w] for w in warps if w < len(softmax)]
            assert p == len(products) and not stuck, (products[p] if p < len(products) else None, stuck)
        for s in out:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return len(seen)


@pytest.mark.parametrize("pieces", [(1,), (2,), (1, 1, 1), (3,), (2, 1, 3), (5, 4), (1, 6, 2)])
def test_no_order_of_the_roles_gets_stuck(source, pieces):
    assert run(source, pieces) > 0


def test_the_model_finds_a_barrier_that_two_tiles_share(source):
    """The model itself: with one barrier for both places of the scores, a warp that looks late waits for ever."""
    shared = re.sub(r"&s_full\[[^]]*\], \(n >> 1\) & 1", "s_full, n & 1", source)
    shared = re.sub(r"&s_full\[[^]]*\]", "s_full", shared)
    with pytest.raises(AssertionError, match="s_full"):
        run(shared, (3,))
