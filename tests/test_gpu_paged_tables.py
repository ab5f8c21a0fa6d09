"""cg_extend_tables against a plain walk over the requests."""
import random

import pytest
import torch

import kv_cache_compression_cachegen_b200 as cg
from kv_cache_compression_cachegen_b200 import torch_api as ta

pytestmark = pytest.mark.gpu
DEV = "cuda"


def walk(held, added, tables, free, taken, P, base, rows):
    """The definition, one token at a time."""
    tables = [list(r) for r in tables]
    slots, positions, starts, lens = [], [], [0], []
    for r, (h, a) in enumerate(zip(held, added)):
        have = -(-h // P)
        for c in range(have, -(-(h + a) // P)):
            tables[r][c] = free[taken]
            taken += 1
        for i in range(a):
            at = h + i
            slots.append(tables[r][at // P] * P + at % P)
            positions.append(base + at)
        starts.append(starts[-1] + a)
        lens.append(h + a)
    pad = rows - len(slots)
    return (tables, slots + [-1] * pad, positions + [-1] * pad, starts, lens, taken)


def make(B, P, max_held, max_added, seed, base=0, pad=5, taken=2):
    r = random.Random(seed)
    held = [r.choice([0, 0, r.randint(0, max_held), P, r.randint(0, max_held) // P * P])
            for _ in range(B)]
    added = [r.choice([0, 1, 1, r.randint(0, max_added)]) for _ in range(B)]
    columns = max(-(-(h + a) // P) for h, a in zip(held, added)) + 2
    have = [-(-h // P) for h in held]
    need = sum(-(-(h + a) // P) - c for h, a, c in zip(held, added, have))
    pages = list(range(sum(have) + need + 3))
    r.shuffle(pages)
    tables = [[pages.pop() for _ in range(c)] + [-1] * (columns - c) for c in have]
    free = [-9] * taken + [pages.pop() for _ in range(need)]
    num_pages = sum(have) + need + 3
    return held, added, tables, free, num_pages, sum(added) + pad


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("B,P,max_held,max_added", [
    (1, 1, 5, 5), (1, 16, 0, 1), (3, 7, 40, 9), (64, 16, 300, 1), (257, 16, 1000, 40),
    (1024, 50, 700, 3), (1025, 16, 100, 2), (5000, 8, 60, 5), (8192, 16, 64, 1),
    (4, 256, 5000, 9000), (2, 16, 10, 70000)])
def test_matches_the_walk(B, P, max_held, max_added):
    held, added, tables, free, num_pages, rows = make(B, P, max_held, max_added, B + P)
    t = ta.PagedTables(B, rows, P, num_pages, DEV)
    bt = i32(tables)
    t.extend(i32(held), i32(added), bt, i32(free), i32([2]), position_base=11)
    torch.cuda.synchronize()
    assert ta.status_of(t.status) == 0
    want = walk(held, added, tables, free, 2, P, 11, rows)
    assert bt.tolist() == want[0]
    assert t.slots.tolist() == want[1]
    assert t.positions.tolist() == want[2]
    assert t.q_starts.tolist() == want[3]
    assert t.kv_lens.tolist() == want[4]
    assert t.taken.tolist() == [want[5]]


@pytest.mark.parametrize("B,P", [(3, 4), (1500, 16)])
def test_steps_in_place(B, P):
    # held is kv_lens and taken is the object's own count: a decode loop, also replayed
    columns, steps = 12, 9
    pages = list(range(B * columns))
    random.Random(1).shuffle(pages)
    t = ta.PagedTables(B, B, P, len(pages), DEV)
    bt = torch.full((B, columns), -1, dtype=torch.int32, device=DEV)
    free, added = i32(pages), i32([1] * B)
    want = ([[-1] * columns for _ in range(B)], None, None, None, [0] * B, 0)
    t.extend(t.kv_lens, added, bt, free)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.extend(t.kv_lens, added, bt, free)
    for _ in range(steps - 1):
        graph.replay()
    torch.cuda.synchronize()
    assert ta.status_of(t.status) == 0
    for _ in range(steps):
        want = walk(want[4], [1] * B, want[0], pages, want[5], P, 0, B)
    assert bt.tolist() == want[0] and t.slots.tolist() == want[1]
    assert t.positions.tolist() == want[2] and t.kv_lens.tolist() == want[4]
    assert t.taken.tolist() == [want[5]]


@pytest.mark.parametrize("B", [5, 2000])
@pytest.mark.parametrize("what,code", [
    ("pages", cg.CG_ERR_CAPACITY), ("columns", cg.CG_ERR_CAPACITY), ("rows", cg.CG_ERR_CAPACITY),
    ("held", cg.CG_ERR_MISMATCH), ("added", cg.CG_ERR_MISMATCH), ("free", cg.CG_ERR_MISMATCH),
    ("entry", cg.CG_ERR_MISMATCH), ("taken", cg.CG_ERR_MISMATCH),
    ("position", cg.CG_ERR_CAPACITY)])
def test_errors_change_nothing(B, what, code):
    P, columns = 16, 8
    held, added = [21] * B, [20] * B  # two pages held, one new each
    pages = list(range(3 * B))
    tables = [[pages.pop(), pages.pop()] + [-1] * (columns - 2) for _ in range(B)]
    free, taken, rows, base = list(pages), 0, 20 * B, 0
    if what == "pages":
        free = free[:-1]
    elif what == "columns":
        added[B - 2] = P * columns
        rows += P * columns
    elif what == "rows":
        rows -= 1
    elif what == "held":
        held[1] = -1
    elif what == "added":
        added[B - 1] = -3
    elif what == "free":
        free[B // 2] = 3 * B
    elif what == "entry":
        tables[B - 1][1] = -1
    elif what == "taken":
        taken = -1
    elif what == "position":
        base = 2 ** 31 - 30
    t = ta.PagedTables(B, rows, P, 3 * B, DEV)
    bt = i32(tables)
    t.extend(i32(held), i32(added), bt, i32(free), i32([taken]), position_base=base)
    torch.cuda.synchronize()
    assert ta.status_of(t.status) == code
    assert bt.tolist() == tables
    assert t.kv_lens.tolist() == held and t.taken.tolist() == [taken]
    assert t.q_starts.tolist() == [0] * (B + 1)
    assert t.slots.tolist() == [-1] * rows and t.positions.tolist() == [-1] * rows


def test_wrapper_refusals():
    t = ta.PagedTables(4, 8, 16, 10, DEV)
    ok = i32([0] * 4)
    with pytest.raises(ValueError):
        t.extend(ok.long(), ok, i32([[-1]] * 4), ok)
    with pytest.raises(ValueError):
        t.extend(ok[:3], ok, i32([[-1]] * 4), ok)
    with pytest.raises(ValueError):
        t.extend(ok, ok, i32([[-1]] * 3), ok)
    with pytest.raises(ValueError):
        t.extend(ok.cpu(), ok, i32([[-1]] * 4), ok)
    with pytest.raises(cg.CacheGenError):
        t.extend(ok, ok, i32([[-1]] * 4), ok, position_base=-1)
