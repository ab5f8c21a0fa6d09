"""Streams and captures: objects made on one stream and first used on another
while the first one is still busy."""
import time

import pytest
import torch

from kv_cache_compression_cachegen_b200 import torch_api as ta
from paged_util import Batch, check_close

pytestmark = pytest.mark.gpu
DEV = "cuda"
BUSY = 600_000_000  # cycles: 0.3 s or more


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.fixture(autouse=True, scope="module")
def _loaded():
    """Every kernel once: loading one may take longer than a stream is kept busy."""
    T, H, D = torch.float16, 2, 64
    t = ta.PagedTables(1, 1, 4, 4, DEV)
    t.extend(t.kv_lens, i32([1]), i32([[-1]]), i32([0]))
    x = torch.zeros(1, H, D, dtype=T, device=DEV)
    pool = torch.zeros(1, 2, 4, 16, H, D, dtype=T, device=DEV)
    ta.rope_table(8, D, DEV)
    ta.PagedAppend((1, H, D), H, T, DEV).append(x, x, x, torch.empty_like(x), pool, 0, None,
                                                t.slots, None)
    b = Batch([30, 7], [1, 1], 8, 2, 128, 16, T, prefix=20)
    q, pool, starts, lens, tables, ptable = b.device()
    call = ta.PagedAttention((1, 2, 128), 8, T, 2, 2, DEV)
    call.run(q, pool, 0, starts, lens, tables, 1, torch.empty_like(q))
    for n in (2, 3):  # the prefix's rows to either kernel
        b = Batch([30] * n, [1] * n, 8, 2, 128, 16, T, prefix=20)
        q, pool, starts, lens, tables, ptable = b.device()
        call = ta.PagedAttention((1, 2, 128), 8, T, n, n, DEV)
        call.run_shared(q, pool, 0, ptable, 20, starts, lens, tables, 1, torch.empty_like(q))
        call.run(q, pool, 0, starts, lens, tables, 1, torch.empty_like(q))
    torch.cuda.synchronize()


def dirty():
    """Blocks of the allocator that hold something else than zeros."""
    blocks = [torch.full((n,), 7, dtype=torch.int32, device=DEV) for n in (1, 64, 4096) * 8]
    torch.cuda.synchronize()
    del blocks


def waits(side):
    """The side stream's work has not run ahead of the current stream's."""
    time.sleep(0.05)
    return not side.query()


def test_tables_made_on_a_busy_stream():
    B, P = 3, 4
    held, added, free = i32([0, 5, 8]), i32([1, 4, 2]), i32(list(range(10, 20)))
    tables = i32([[-1] * 4, [0, 1, -1, -1], [2, 3, -1, -1]])
    side = torch.cuda.Stream()
    dirty()
    torch.cuda._sleep(BUSY)
    call = ta.PagedTables(B, 9, P, 20, DEV)
    call.extend(held, added, tables, free, stream=side)
    assert waits(side)
    torch.cuda.synchronize()
    assert ta.status_of(call.status) == 0
    assert call.kv_lens.tolist() == [1, 9, 10] and call.q_starts.tolist() == [0, 1, 5, 7]
    assert call.taken.tolist() == [3]
    assert tables.tolist() == [[10, -1, -1, -1], [0, 1, 11, -1], [2, 3, 12, -1]]
    assert call.slots.tolist() == [40, 5, 6, 7, 44, 48, 49, -1, -1]


def test_append_and_rope_table_made_on_a_busy_stream():
    T, N, H, D = torch.float16, 5, 2, 64
    x = torch.randn(N, 3 * H, D, device=DEV).to(T)
    pool = torch.zeros(1, 2, 2, 16, H, D, dtype=T, device=DEV)
    q_out = torch.zeros(N, H, D, dtype=T, device=DEV)
    slots = torch.arange(N, device=DEV)
    want = ta.rope_table(40, D, DEV)
    side = torch.cuda.Stream()
    dirty()
    torch.cuda._sleep(BUSY)
    # the table's block may be one that the busy stream still fills
    torch.empty(40 * D, device=DEV).fill_(9.0)
    table = ta.rope_table(40, D, DEV, stream=side)
    call = ta.PagedAppend((1, H, D), H, T, DEV)
    call.append(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], q_out, pool, 0, None, slots, None,
                stream=side)
    assert waits(side)
    torch.cuda.synchronize()
    assert ta.status_of(call.status) == 0
    assert torch.equal(table, want) and torch.equal(q_out, x[:, :H])


@pytest.mark.parametrize("shared", [False, True])
def test_attention_made_on_a_busy_stream(shared):
    H, Hq, D, T = 2, 8, 128, torch.float16
    b = Batch([3000, 700, 90], [1, 1, 1], Hq, H, D, 16, T, seed=3, prefix=200)
    q, pool, starts, lens, tables, ptable = b.device()
    side, out = torch.cuda.Stream(), torch.empty_like(q)
    calls = [ta.PagedAttention((1, H, D), Hq, T, 3, 3, DEV)]
    if shared:  # met, with its first workspace, before that stream is busy
        calls[0].run(q, pool, 0, starts, lens, tables, 1, out, stream=side)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    if shared:  # the first shared call makes a larger workspace
        calls[0].run_shared(q, pool, 0, ptable, 200, starts, lens, tables, 1, out, stream=side)
    else:
        calls.append(ta.PagedAttention((1, H, D), Hq, T, 3, 3, DEV))
        calls[1].run(q, pool, 0, starts, lens, tables, 1, out, stream=side)
    assert waits(side)
    torch.cuda.synchronize()
    assert all(ta.status_of(c.status) == 0 for c in calls)
    if shared:
        want, _, tol = b.oracle()
        check_close(out, want, tol)


def test_made_on_a_busy_stream_and_grown_on_another():
    # the object is made on one stream, its larger workspace on a second, and a third
    # one uses it: all of it is ready there
    H, Hq, D, T = 2, 8, 128, torch.float16
    b = Batch([300, 70], [1, 1], Hq, H, D, 16, T, seed=3, prefix=200)
    q, pool, starts, lens, tables, ptable = b.device()
    out = torch.empty_like(q)
    first, second, third = (torch.cuda.Stream() for _ in range(3))
    torch.cuda.synchronize()
    with torch.cuda.stream(first):
        torch.cuda._sleep(BUSY)
        call = ta.PagedAttention((1, H, D), Hq, T, 2, 2, DEV)
    with torch.cuda.stream(second):
        call.reserve_shared()
    call.run_shared(q, pool, 0, ptable, 200, starts, lens, tables, 1, out, stream=third)
    assert waits(third)
    torch.cuda.synchronize()
    assert ta.status_of(call.status) == 0
    want, _, tol = b.oracle()
    check_close(out, want, tol)


def test_a_captured_call_keeps_its_workspace_when_a_larger_one_is_made():
    # run() captured, then the first run_shared(): the graph still writes where it did
    H, Hq, D, T = 2, 8, 128, torch.float16
    b = Batch([3000, 700, 90], [1, 1, 1], Hq, H, D, 16, T, seed=3)
    c = Batch([30, 64, 5], [1, 1, 1], Hq, H, D, 16, T, seed=4, prefix=160)
    q, pool, starts, lens, tables, _ = b.device()
    q2, pool2, starts2, lens2, tables2, ptable = c.device()
    call = ta.PagedAttention((1, H, D), Hq, T, 3, 3, DEV)
    out, out2 = torch.empty_like(q), torch.empty_like(q2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run(q, pool, 0, starts, lens, tables, 1, out)
    size, first = call.workspace.numel(), call.workspace.data_ptr()
    call.run_shared(q2, pool2, 0, ptable, 160, starts2, lens2, tables2, 1, out2)
    assert call.workspace.data_ptr() != first
    others = [torch.full((size,), 255, dtype=torch.uint8, device=DEV) for _ in range(3)]
    graph.replay()
    torch.cuda.synchronize()
    assert ta.status_of(call.status) == 0
    assert all(bool((x == 255).all()) for x in others)
    want, _, tol = b.oracle()
    check_close(out, want, tol)
    want, _, tol = c.oracle()
    check_close(out2, want, tol)


def test_an_unused_workspace_is_not_kept():
    call = ta.PagedAttention((1, 2, 128), 8, torch.float16, 3, 3, DEV)
    torch.cuda.synchronize()
    held, old = torch.cuda.memory_allocated(), call.workspace.numel()
    call.reserve_shared()
    assert torch.cuda.memory_allocated() - held < call.workspace.numel() - old + (4 << 20)
