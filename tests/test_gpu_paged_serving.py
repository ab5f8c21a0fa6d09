"""The paged calls together, as a server uses them: a document decoded from its
containers into the pool, then a batch of requests behind it, step by step."""
import math

import pytest
import torch

from gpu_util import gen
from kv_cache_compression_cachegen_b200 import Shape
from kv_cache_compression_cachegen_b200 import torch_api as ta
from paged_util import check_close, half_step

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("norm", [False, True])
def test_decode_extend_append_attend(norm):
    L, H, Hq, D, P, C = 2, 2, 8, 64, 16, 128
    doc, B, layer, T = 200, 3, 1, torch.float16
    dtype_u = half_step(T)
    shape = Shape(L, H, D)
    kv = gen(L, H, D, doc, 3)
    enc = ta.encode(kv, C, 1)
    pages = 64
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(0))
    perm = perm.to(torch.int32).to(DEV)
    doc_pages = -(-doc // P)
    table, free = perm[:doc_pages].contiguous(), perm[doc_pages:].contiguous()
    pool = torch.full((L, 2, pages, P, H, D), math.nan, dtype=T, device=DEV)
    status = ta.decode_into_paged(enc.data, enc.stride, shape, C, 1, 2, pool, P, table, doc)
    tables = ta.PagedTables(B, 64, P, pages, DEV, status)
    append = ta.PagedAppend(shape, Hq, T, DEV, status)
    attend = ta.PagedAttention(shape, Hq, T, 64, B, DEV, status)
    rope = ta.rope_table(400, D, DEV)
    bt = torch.full((B, 8), -1, dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    w = [(1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(T) if norm else None
         for _ in range(2)]
    seen_k, seen_v = ([[] for _ in range(B)] for _ in range(2))
    flat = torch.empty_like(kv)
    ta.decode_into(enc.data, enc.stride, shape, C, 1, 2, flat, status)
    torch.cuda.synchronize()
    doc_kv = flat.view(torch.float16)[layer].double().cpu()
    for added in ([5, 0, 33], [1, 1, 1], [1, 20, 1], [1, 1, 1]):
        a = torch.tensor(added, dtype=torch.int32, device=DEV)
        tables.extend(tables.kv_lens, a, bt, free, position_base=doc)
        n = 64  # a padded batch: rows behind the last token are left as they are
        qkv = torch.randn(n, Hq + 2 * H, D, generator=g, device=DEV).to(T)
        q = torch.full((n, Hq, D), 2.0, dtype=T, device=DEV)
        out = torch.full((n, Hq, D), 3.0, dtype=T, device=DEV)
        append.append(qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:], q, pool, layer,
                      tables.positions, tables.slots, rope, w[0], w[1])
        attend.run_shared(q, pool, layer, table, doc, tables.q_starts, tables.kv_lens, bt,
                          max(added), out)
        torch.cuda.synchronize()
        assert ta.status_of(status) == 0
        total = sum(added)
        assert (q[total:] == 2).all() and (out[total:] == 3).all()
        pos = tables.positions[:total].cpu()
        x = qkv[:total].double().cpu()
        c = rope.double().cpu()[pos.long()][:, None]
        cos, sin = c[..., :D // 2], c[..., D // 2:]

        def turn(y, weight):
            if norm:
                y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double().cpu()
            lo, hi = y[..., :D // 2], y[..., D // 2:]
            return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)
        want_q, want_k = turn(x[:, :Hq], w[0]), turn(x[:, Hq:Hq + H], w[1])
        check_close(q[:total], want_q, dtype_u * want_q.abs() * 1.001 + 2.0 ** -18)
        t = 0
        for r, m in enumerate(added):
            for i in range(m):
                # keys as they are stored: rounded once to the pool's type
                seen_k[r].append(want_k[t].to(T).double())
                seen_v[r].append(x[t, Hq + H:])
                k = torch.cat([doc_kv[0], torch.stack(seen_k[r])])
                v = torch.cat([doc_kv[1], torch.stack(seen_v[r])])
                for h in range(Hq):
                    qq = q[t, h].double().cpu()  # the queries as they were stored
                    s = k[:, h // 4] @ qq / math.sqrt(D)
                    p = torch.softmax(s, 0)
                    o, mass = p @ v[:, h // 4], p @ v[:, h // 4].abs()
                    # weights and output half a step each; a key on a rounding's
                    # edge may be stored one step off: its score by 2 u |q| |k| / sqrt(D)
                    edge = float((2 * dtype_u * k[doc:, h // 4].abs() @ qq.abs()).max()) / \
                        math.sqrt(D) * float(p[doc:].max())
                    tol = dtype_u * (o.abs() + mass) + (edge + 2.0 ** -14) * mass
                    check_close(out[t, h], o, tol * 1.01 + 1e-6, f"request {r} token {i}")
                t += 1


def test_two_streams_two_workspaces():
    # two batches at once, each with its own objects, on streams of their own
    H, Hq, D, P, T = 2, 4, 64, 16, torch.bfloat16
    from paged_util import Batch
    batches = [Batch([500, 90], [1, 1], Hq, H, D, P, T, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in batches]
    held = [b.device() for b in batches]
    calls = [ta.PagedAttention((1, H, D), Hq, T, 2, 2, DEV) for _ in batches]
    outs = [torch.empty_like(d[0]) for d in held]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, call, out, s in zip(held, calls, outs, streams):
            q, pool, starts, lens, tables, _ = d
            call.run(q, pool, 0, starts, lens, tables, 1, out, stream=s)
    torch.cuda.synchronize()
    for b, out in zip(batches, outs):
        want, _, tol = b.oracle()
        check_close(out, want, tol)


def test_objects_outlived_by_their_work_on_another_stream():
    # an object made on one stream, used on another and dropped at once: its
    # workspace is not handed out again while that stream still works in it
    from paged_util import Batch
    H, Hq, D, P, T = 2, 8, 128, 16, torch.float16
    b = Batch([3000, 700, 90], [1, 1, 1], Hq, H, D, P, T, seed=3, prefix=200)
    q, pool, starts, lens, tables, ptable = b.device()
    side = torch.cuda.Stream()
    outs = [torch.empty_like(q) for _ in range(8)]
    torch.cuda.synchronize()
    for out in outs:
        call = ta.PagedAttention((1, H, D), Hq, T, 3, 3, DEV)
        call.run_shared(q, pool, 0, ptable, 200, starts, lens, tables, 1, out, stream=side)
        size = call.workspace.numel()
        del call
        torch.empty(size, dtype=torch.uint8, device=DEV).fill_(255)
    torch.cuda.synchronize()
    want, _, tol = b.oracle()
    for out in outs:
        check_close(out, want, tol)


def test_a_step_that_fails_leaves_the_calls_behind_it_without_rows():
    # too few free pages: no table, no pool row and no output row is written
    H, Hq, D, P, T, B = 2, 4, 64, 16, torch.float16, 3
    tables = ta.PagedTables(B, 8, P, 10, DEV)
    append = ta.PagedAppend((1, H, D), Hq, T, DEV)
    attend = ta.PagedAttention((1, H, D), Hq, T, 8, B, DEV)
    pool = torch.full((1, 2, 10, P, H, D), 5.0, dtype=T, device=DEV)
    bt = torch.full((B, 4), -1, dtype=torch.int32, device=DEV)
    free = torch.arange(2, dtype=torch.int32, device=DEV)
    added = torch.ones(B, dtype=torch.int32, device=DEV)
    qkv = torch.randn(8, Hq + 2 * H, D, device=DEV).to(T)
    q, out = (torch.full((8, Hq, D), 3.0, dtype=T, device=DEV) for _ in range(2))
    tables.extend(tables.kv_lens, added, bt, free)
    append.append(qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:], q, pool, 0, tables.positions,
                  tables.slots, ta.rope_table(8, D, DEV))
    attend.run(q, pool, 0, tables.q_starts, tables.kv_lens, bt, 1, out)
    attend.run_shared(q, pool, 0, free, 20, tables.q_starts, tables.kv_lens, bt, 1, out)
    torch.cuda.synchronize()
    assert ta.status_of(tables.status) == 2  # CG_ERR_CAPACITY
    assert ta.status_of(append.status) == 0 and ta.status_of(attend.status) == 0
    assert (pool == 5).all() and (q == 3).all() and (out == 3).all() and (bt == -1).all()
