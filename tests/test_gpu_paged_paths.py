"""Attention calls that take the kernels' other paths: batches whose lines are
summed up by a kernel of their own, prefixes larger than half the L2 cache,
every kind of page against every kind of item, and random batches.  The
reference is attention in 64 bits on the GPU."""
import math
import random

import pytest
import torch

from kv_cache_compression_cachegen_b200 import torch_api as ta
from paged_util import check_close, half_step

pytestmark = pytest.mark.gpu
DEV = "cuda"


def build(lens, added, Hq, H, D, page, dtype, prefix=0, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    counts = [-(-x // page) for x in lens]
    ppages = -(-prefix // page)
    pages = sum(counts) + ppages + 2
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    tables = torch.full((len(lens), max(counts + [1])), -1, dtype=torch.int32, device=DEV)
    at = ppages
    for r, c in enumerate(counts):
        tables[r, :c] = perm[at:at + c]
        at += c
    pool = torch.randn(1, 2, pages, page, H, D, generator=g, device=DEV).to(dtype)
    # what lies behind a request's last token must not matter
    flat = pool.view(2, pages, page, H, D)
    for r, x in enumerate(lens):
        if x % page:
            flat[:, int(tables[r, x // page]), x % page:] = math.nan
    if prefix % page:
        flat[:, int(perm[ppages - 1]), prefix % page:] = math.nan
    starts = [0]
    for a in added:
        starts.append(starts[-1] + a)
    q = torch.randn(starts[-1], Hq, D, generator=g, device=DEV).to(dtype)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)
    return dict(q=q, pool=pool, tables=tables, prefix_table=perm[:ppages].contiguous(),
                starts=i32(starts), lens=i32(lens), page=page, prefix=prefix,
                host=(starts, list(lens), list(added)))


def reference(b, window=0, sinks=0):
    """(out, tolerance): see paged_util.Batch.oracle for the steps it counts."""
    q, page = b["q"], b["page"]
    N, Hq, D = q.shape
    H = b["pool"].shape[4]
    G = Hq // H
    flat = b["pool"][0].reshape(2, -1, H, D)
    u = half_step(q.dtype)
    tiny = 2.0 ** -25 if q.dtype == torch.float16 else 0.0
    outs, tols = [], []
    starts, lens, added = b["host"]

    def rows(table, n):
        j = torch.arange(n, device=DEV)
        return table[(j // page)].long() * page + j % page
    pre = rows(b["prefix_table"], b["prefix"]) if b["prefix"] else None
    for r, (n, kv) in enumerate(zip(added, lens)):
        if n == 0:
            continue
        at = rows(b["tables"][r], kv) if kv else torch.zeros(0, dtype=torch.long, device=DEV)
        j = torch.arange(kv, device=DEV)
        p = kv - n + torch.arange(n, device=DEV)[:, None]
        see = j[None] <= p
        if window:
            see &= (j[None] > p - window) | (j[None] < sinks)
        if pre is not None:
            at = torch.cat([pre, at])
            see = torch.cat([torch.ones(n, b["prefix"], dtype=torch.bool, device=DEV), see], 1)
        if at.numel() == 0:  # nothing to see: zeros
            outs.append(torch.zeros(n, Hq, D, dtype=torch.float64, device=DEV))
            tols.append(torch.zeros_like(outs[-1]))
            continue
        k = flat[0, at].double().repeat_interleave(G, 1)   # [m, Hq, D]
        v = flat[1, at].double().repeat_interleave(G, 1)
        x = q[starts[r]:starts[r + 1]].double()
        s = torch.einsum("nhd,mhd->hnm", x, k) / math.sqrt(D)
        big = torch.einsum("nhd,mhd->hnm", x.abs(), k.abs()) / math.sqrt(D)
        s = s.masked_fill(~see, -math.inf)
        m = s.amax(-1, keepdim=True)
        e = torch.exp(s - torch.where(m > -math.inf, m, torch.zeros_like(m)))
        total = e.sum(-1, keepdim=True)
        w = e / total.clamp(min=1e-300)
        o = torch.einsum("hnm,mhd->nhd", w, v)
        mass = torch.einsum("hnm,mhd->nhd", w, v.abs())
        score = (D + 4) * 2.0 ** -24 * big.masked_fill(~see, 0).amax(-1).T[..., None]
        faint = tiny * torch.einsum("nm,mhd->nhd", see.double(), v.abs()) / \
            total.squeeze(-1).T[..., None].clamp(min=1e-300)
        tol = u * o.abs() + (u + 2 * score + 2.0 ** -20) * mass + faint.clamp(max=1.0)
        outs.append(o)
        tols.append(tol * 1.01 + 1e-7)
    return torch.cat(outs).cpu(), torch.cat(tols).cpu()


def attend(b, window=0, sinks=0):
    q = b["q"]
    N, Hq, D = q.shape
    H = b["pool"].shape[4]
    call = ta.PagedAttention((1, H, D), Hq, q.dtype, N, len(b["host"][1]), DEV)
    out = torch.full_like(q, 3.0)
    most = max(max(b["host"][2]), 1)
    if b["prefix"]:
        call.reserve_shared()
        call.workspace.fill_(255)
        call.run_shared(q, b["pool"], 0, b["prefix_table"], b["prefix"], b["starts"], b["lens"],
                        b["tables"], most, out)
    else:
        call.workspace.fill_(255)
        call.run(q, b["pool"], 0, b["starts"], b["lens"], b["tables"], most, out, window=window,
                 sinks=sinks)
    torch.cuda.synchronize()
    assert ta.status_of(call.status) == 0
    return out


def verify(b, window=0, sinks=0):
    want, tol = reference(b, window, sinks)
    check_close(attend(b, window, sinks), want, tol)


@pytest.mark.parametrize("prefix", [0, 100])
@pytest.mark.parametrize("B", [1023, 1024, 1500])
def test_many_requests(B, prefix):
    # the rows kernel's line passes what a CTA sums up by itself
    r = random.Random(B)
    lens = [r.choice([1, 2, 15, 16, 17, 40]) for _ in range(B)]
    verify(build(lens, [1] * B, 4, 2, 64, 16, torch.float16, prefix, seed=B))


def test_many_chunks():
    # the same of the tile kernel's, with single tokens between
    r = random.Random(5)
    added = [r.choice([1, 1, 3, 30, 90]) for _ in range(1100)]
    lens = [a + r.choice([0, 5, 100]) for a in added]
    verify(build(lens, added, 4, 1, 64, 16, torch.bfloat16, seed=6))


@pytest.mark.parametrize("page", [1, 8, 12, 16, 24, 64, 128, 200])
@pytest.mark.parametrize("D,Hq,H", [(64, 4, 2), (128, 8, 1), (96, 6, 2), (256, 2, 1), (80, 10, 2)])
def test_pages_and_items(page, D, Hq, H):
    # single tokens, a few, chunks of one and of two query tiles, in one call
    added = [1, 3, 40, 129 // (Hq // H) + 1, 300, 1, 0]
    lens = [200, 3, 333, 129 // (Hq // H) + 5, 301, 70, 9]
    b = build(lens, added, Hq, H, D, page, torch.float16, seed=page)
    verify(b)
    verify(b, window=130, sinks=5)


@pytest.mark.parametrize("prefix,page,B,added", [(20000, 16, 70, 1), (16500, 48, 40, 2),
                                                 (17000, 7, 35, 2)])
def test_prefix_larger_than_half_the_cache(prefix, page, B, added):
    r = random.Random(prefix)
    lens = [added + r.choice([0, 1, 30]) for _ in range(B)]
    verify(build(lens, [added] * B, 32, 8, 128, page, torch.float16, prefix, seed=1))


@pytest.mark.parametrize("seed", range(40))
def test_random_batches(seed):
    r = random.Random(1000 + seed)
    Hq, H = r.choice([(8, 2), (4, 4), (5, 1), (12, 3), (16, 1), (24, 8), (7, 7), (64, 1)])
    D = r.choice([16, 32, 48, 64, 80, 112, 128, 128, 192, 256])
    page = r.choice([1, 3, 8, 16, 16, 32, 40, 64, 256])
    dtype = r.choice([torch.float16, torch.bfloat16])
    B = r.randint(1, 9)
    most = r.choice([1, 1, 4, 70, 300])
    added = [r.choice([0, 1, r.randint(1, most)]) for _ in range(B)]
    added[0] = max(1, added[0])
    # more new tokens than tokens, now and then
    lens = [max(0, a + r.choice([-2, 0, 0, 7, r.randint(0, 700)])) if a else r.randint(0, 50)
            for a in added]
    prefix = r.choice([0, 0, r.randint(1, 900)])
    window, sinks = (0, 0) if prefix else r.choice([(0, 0), (1, 0), (33, 2), (128, 129), (500, 0)])
    b = build(lens, added, Hq, H, D, page, dtype, prefix, seed)
    verify(b, window, sinks)


def test_captured_chunks_and_two_streams():
    # the tile kernel's path replayed with other lengths, and two calls at once
    bs = [build([300, 40, 700], [200, 40, 1], 8, 2, 128, 16, torch.float16, 0, s) for s in (1, 2)]
    want = [reference(b) for b in bs]
    calls = [ta.PagedAttention((1, 2, 128), 8, torch.float16, 241, 3, DEV) for _ in bs]
    outs = [torch.empty_like(b["q"]) for b in bs]

    def go(k, stream=None):
        b = bs[k]
        calls[k].run(b["q"], b["pool"], 0, b["starts"], b["lens"], b["tables"], 200, outs[k],
                     stream=stream)
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(10):
        for k in (0, 1):
            go(k, streams[k])
    torch.cuda.synchronize()
    for k in (0, 1):
        check_close(outs[k], *want[k])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(0)
    lens = bs[0]["lens"].clone()
    bs[0]["lens"].copy_(torch.tensor([210, 40, 5]))
    graph.replay()
    short = outs[0].clone()
    bs[0]["lens"].copy_(lens)
    graph.replay()
    torch.cuda.synchronize()
    check_close(outs[0], *want[0])
    assert not torch.equal(short, outs[0])
    again = outs[0].clone()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, outs[0])


def test_keys_not_finite():
    # a key that is not finite makes every row that sees it NaN, and no other
    for bad in (math.nan, math.inf):
        for added, lens in ((1, 200), (100, 200)):
            b = build([lens, lens], [added, added], 4, 2, 64, 16, torch.float16, seed=3)
            p = b["page"]
            for at in (150, 199):
                flat = b["pool"][0]
                flat[0, int(b["tables"][1, at // p]), at % p] = bad
            want, tol = reference(b)
            out = attend(b)
            first = max(0, 150 - (lens - added))
            good = torch.ones(2 * added, dtype=torch.bool)
            good[added + first:] = False
            check_close(out[good.to(DEV)], want[good], tol[good])
            assert torch.isnan(out[~good.to(DEV)]).all()


def test_first_call_captured():
    # nothing has to run before a capture: kernels that no call has used yet
    b = build([41, 50], [1, 3], 4, 2, 48, 16, torch.bfloat16, 0, 9)
    call = ta.PagedAttention((1, 2, 48), 4, torch.bfloat16, 4, 2, DEV)
    out = torch.empty_like(b["q"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run(b["q"], b["pool"], 0, b["starts"], b["lens"], b["tables"], 3, out)
    graph.replay()
    torch.cuda.synchronize()
    check_close(out, *reference(b))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim", [128, 160, 256])
def test_nine_to_sixteen_rows_of_many_channels(dim, dtype):
    # items of 8, 16 and 9 rows a kv head, some cut; then of 16 rows under more tokens
    b = build([700, 130, 1, 2050], [1, 2, 1, 2], 16, 2, dim, 16, dtype, 0, 9)
    call = ta.PagedAttention((1, 2, dim), 16, dtype, 6, 4, DEV)
    out = torch.empty_like(b["q"])
    call.run(b["q"], b["pool"], 0, b["starts"], b["lens"], b["tables"], 2, out)
    check_close(out, *reference(b))
    b = build([700, 130, 90], [3, 1, 2], 15, 3, dim, 16, dtype, 0, 9)
    call = ta.PagedAttention((1, 3, dim), 15, dtype, 6, 3, DEV)
    out = torch.empty_like(b["q"])
    call.run(b["q"], b["pool"], 0, b["starts"], b["lens"], b["tables"], 3, out, window=100)
    check_close(out, *reference(b, window=100))


@pytest.mark.parametrize("prefix", [0, 100])
def test_starts_out_of_order_leave_other_requests_alone(prefix):
    # request 0 and the ones behind it claim the same rows and request 1 has none:
    # the last one's rows are its own, and right
    added, lens = [1500, 0, 30, 1440, 200], [2000, 5, 40, 1500, 700]
    starts = [0, 1500, 30, 60, 1500, 1700]
    b = build(lens, [0, 0, 0, 0, 200], 4, 2, 64, 16, torch.float16, prefix, seed=4)
    want, tol = reference(b)
    q = torch.zeros(1700, 4, 64, dtype=torch.float16, device=DEV)
    q[1500:] = b["q"]
    b.update(q=q, starts=torch.tensor(starts, dtype=torch.int32, device=DEV))
    call = ta.PagedAttention((1, 2, 64), 4, q.dtype, 1700, 5, DEV)
    call.reserve_shared()
    call.workspace.fill_(255)
    out = torch.empty_like(q)
    args = (b["starts"], b["lens"], b["tables"], max(added), out)
    if prefix:
        call.run_shared(q, b["pool"], 0, b["prefix_table"], prefix, *args)
    else:
        call.run(q, b["pool"], 0, *args)
    torch.cuda.synchronize()
    assert ta.status_of(call.status) == 4  # CG_ERR_MISMATCH
    check_close(out[1500:], want, tol)
