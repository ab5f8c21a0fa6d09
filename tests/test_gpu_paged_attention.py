"""cg_attention_paged and cg_attention_shared against attention in 64 bits.

Every place of the pool that no row may see holds NaN, so a product with a
masked key or value shows."""
import pytest
import torch

import kv_cache_compression_cachegen_b200 as cg
from kv_cache_compression_cachegen_b200 import torch_api as ta
from paged_util import DTYPES, Batch, check_close

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run(b, window=0, sinks=0, scale=None, shared=False, max_q=None, with_lse=True):
    q, pool, starts, lens, tables, ptable = b.device()
    L = pool.shape[0]
    call = ta.PagedAttention((L, b.H, b.D), b.Hq, b.dtype, q.shape[0], len(b.lens), DEV)
    # a workspace holds whatever the call before left in it
    if shared:
        call.reserve_shared()
    call.workspace.fill_(255)
    out = torch.full_like(q, 3.0)
    lse = torch.full(q.shape[:2], 5.0, device=DEV) if with_lse else None
    max_q = max_q or max(max(b.added), 1)
    if shared:
        call.run_shared(q, pool, b.layer, ptable, b.prefix, starts, lens, tables, max_q, out,
                        scale=scale, lse=lse)
    else:
        call.run(q, pool, b.layer, starts, lens, tables, max_q, out, window=window, sinks=sinks,
                 scale=scale, lse=lse)
    torch.cuda.synchronize()
    assert ta.status_of(call.status) == 0
    return out.cpu(), None if lse is None else lse.cpu()


def verify(b, window=0, sinks=0, scale=None, shared=False, **kw):
    out, lse = run(b, window, sinks, scale, shared, **kw)
    want, want_lse, tol = b.oracle(window, sinks, scale)
    n = sum(b.added)
    check_close(out[:n], want, tol, "out")
    assert (out[n:] == 3).all(), "rows behind the last request were written"
    seen = want_lse > -float("inf")
    assert torch.equal(lse[:n].double() == -float("inf"), ~seen)
    # scores: fp32 sums of D products; the sum and its logarithm: a few fp32 steps
    bound = 2.0 ** -18 + (b.D + 8) * 2.0 ** -22 * want_lse[seen].abs().clamp(min=4)
    assert ((lse[:n].double()[seen] - want_lse[seen]).abs() <= bound).all()
    assert (lse[n:] == 5).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("Hq,H,D", [(1, 1, 16), (8, 2, 64), (4, 4, 128), (12, 2, 80), (7, 1, 96),
                                    (16, 1, 128), (3, 3, 48), (8, 1, 256), (10, 2, 112),
                                    (34, 2, 64), (2, 1, 240)])
def test_single_tokens(dtype, Hq, H, D):
    b = Batch([1, 2, 17, 64, 65, 200, 333], [1] * 7, Hq, H, D, 16, DTYPES[dtype], seed=D,
              extra_rows=3)
    verify(b)


@pytest.mark.parametrize("page", [1, 5, 16, 64, 100])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (64, 4), (100, 70), (500, 3),
                                          (37, 500), (130, 0)])
def test_window_and_sinks_single_tokens(page, window, sinks):
    lens = [1, 30, 64, 129, 300, 401]

    def unseen(r, j):
        return bool(window) and j <= lens[r] - 1 - window and j >= sinks
    b = Batch(lens, [1] * 6, 8, 2, 64, page, torch.float16, seed=page, unseen=unseen, layers=2,
              layer=1)
    verify(b, window, sinks)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (50, 3), (128, 130), (200, 0)])
@pytest.mark.parametrize("Hq,H,D", [(4, 2, 64), (2, 2, 128), (6, 1, 80), (2, 1, 256)])
def test_chunks(dtype, window, sinks, Hq, H, D):
    lens, added = [5, 300, 70, 150, 9, 261], [5, 40, 70, 1, 0, 130]

    def unseen(r, j):
        first = lens[r] - added[r]
        return bool(window) and j <= first - window and j >= sinks
    b = Batch(lens, added, Hq, H, D, 16, DTYPES[dtype], seed=window, unseen=unseen, extra_rows=2)
    verify(b, window, sinks)


def test_rows_that_see_nothing():
    # more new tokens than tokens in the pool: the first rows stand before the first key
    b = Batch([0, 3, 0, 70], [2, 5, 0, 90], 4, 2, 64, 16, torch.float16)
    verify(b)
    # no row of the whole batch sees anything
    b = Batch([0, 0], [1, 3], 4, 2, 64, 16, torch.bfloat16)
    verify(b)


@pytest.mark.parametrize("lens,added", [([1], [1]), ([5000], [1]), ([3000], [300]),
                                        ([900, 1, 1, 1], [1, 1, 1, 1])])
def test_one_long_request(lens, added):
    verify(Batch(lens, added, 4, 1, 64, 16, torch.float16, seed=3), 0, 0)


@pytest.mark.parametrize("scale_q,scale", [(30.0, None), (1.0, 0.0), (1.0, -0.3), (1.0, 4.0)])
def test_large_and_odd_scales(scale_q, scale):
    # scores far apart: one key holds the weight; and all weights alike
    b = Batch([300, 120], [1, 30], 4, 2, 64, 16, torch.float16, seed=9, scale_q=scale_q)
    verify(b, scale=scale)


def test_values_not_finite_where_only_some_rows_see_them():
    # token 20's key and value are NaN or infinite: the rows before it must not notice
    for bad in (float("nan"), float("inf")):
        lens, added = [40, 90], [40, 60]
        b = Batch(lens, added, 4, 2, 64, 16, torch.float16, seed=5)
        for r, at in ((0, 20), (1, 70)):
            page, row = int(b.tables[r, at // 16]), at % 16
            b.pool[0, :, page, row] = bad
        out, lse = run(b)
        want, _, tol = b.oracle()
        good = torch.zeros(100, dtype=torch.bool)
        good[:20] = True
        good[40:40 + 70 - 30] = True
        check_close(out[good], want[good], tol[good], "rows before")
        assert not torch.isfinite(out[~good].float()).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("prefix,lens,added", [
    (1, [1], [1]), (64, [0, 3], [1, 1]), (100, [1, 20, 65, 130], [1, 1, 1, 1]),
    (333, [7, 0, 30], [7, 0, 3]), (130, [40, 70], [40, 33]), (0, [20, 1], [1, 1]),
    (700, [5] * 40, [1] * 40)])
@pytest.mark.parametrize("Hq,H,D", [(8, 2, 64), (3, 3, 128), (5, 1, 80)])
def test_shared_prefix(dtype, prefix, lens, added, Hq, H, D):
    b = Batch(lens, added, Hq, H, D, 16, DTYPES[dtype], seed=prefix, prefix=prefix, extra_rows=2)
    verify(b, shared=True)


def test_shared_rows_that_see_only_the_prefix():
    b = Batch([0, 2], [3, 4], 4, 2, 64, 7, torch.float16, prefix=50)
    verify(b, shared=True)


def test_shared_equals_separate_tables():
    # the same tokens once shared, once as part of every request's own table
    b = Batch([30, 64, 5], [1, 2, 5], 8, 2, 128, 16, torch.float16, prefix=160, seed=2)
    out, _ = run(b, shared=True)
    q, pool, starts, lens, tables, ptable = b.device()
    both = torch.cat([ptable.expand(3, -1), tables], 1).contiguous()
    call = ta.PagedAttention((1, 2, 128), 8, b.dtype, q.shape[0], 3, DEV)
    want = call.run(q, pool, 0, starts, lens + 160, both, 5, torch.empty_like(q))
    torch.cuda.synchronize()
    # two results within their tolerances of the same values
    _, _, tol = b.oracle()
    check_close(out, want.double().cpu(), 2 * tol, "shared")


def test_strided_rows_and_layers():
    # q and out are columns of wider rows; the pool's middle layer is read
    b = Batch([40, 3, 100], [1, 3, 20], 4, 2, 64, 16, torch.bfloat16, layers=3, layer=1)
    q, pool, starts, lens, tables, _ = b.device()
    wide = torch.full((24, 12, 64), 9.0, dtype=b.dtype, device=DEV)
    wide[:, 4:8] = q
    res = torch.full((24, 6, 64), 9.0, dtype=b.dtype, device=DEV)
    call = ta.PagedAttention((3, 2, 64), 4, b.dtype, 24, 3, DEV)
    call.run(wide[:, 4:8], pool, 1, starts, lens, tables, 20, res[:, 1:5])
    torch.cuda.synchronize()
    want, _, tol = b.oracle()
    check_close(res[:, 1:5], want, tol)
    assert (res[:, 0] == 9).all() and (res[:, 5] == 9).all()


def test_bad_data_is_left_out():
    b = Batch([40, 50, 60], [1, 1, 1], 4, 2, 64, 16, torch.float16)
    q, pool, starts, lens, tables, _ = b.device()
    want, _, tol = b.oracle()

    def attend(starts=starts, lens=lens, tables=tables, max_q=1):
        call = ta.PagedAttention((1, 2, 64), 4, b.dtype, 3, 3, DEV)
        out = torch.full_like(q, 3.0)
        call.run(q, pool, 0, starts, lens, tables, max_q, out)
        torch.cuda.synchronize()
        return out, ta.status_of(call.status)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)
    # a length beyond the table, a negative one, more rows than max_q, rows behind the last
    for kw in (dict(lens=i32([40, 16 * tables.shape[1] + 1, 60])), dict(lens=i32([40, -1, 60]))):
        out, st = attend(**kw)
        assert st == cg.CG_ERR_MISMATCH
        check_close(out[[0, 2]], want[[0, 2]], tol[[0, 2]])
        assert (out[1] == 3).all()
    out, st = attend(starts=i32([0, 1, 2, 9]))
    assert st == cg.CG_ERR_MISMATCH
    check_close(out[:2], want[:2], tol[:2])
    out, st = attend(starts=i32([0, 2, 1, 3]), max_q=2)
    assert st == cg.CG_ERR_MISMATCH
    # a page outside the pool: its tokens are left out, the others stand
    for page in (-1, pool.shape[2], 1 << 30):
        t = tables.clone()
        t[1, 1] = page
        out, st = attend(tables=t)
        assert st == cg.CG_ERR_MISMATCH
        check_close(out[[0, 2]], want[[0, 2]], tol[[0, 2]])
        assert torch.isfinite(out[1].float()).all()


def test_repeats_bit_for_bit_and_captured():
    # the order of every sum is fixed, whatever ran before in the workspace
    b = Batch([700, 33, 260], [1, 1, 1], 8, 2, 128, 16, torch.float16, prefix=300, seed=4)
    q, pool, starts, lens, tables, ptable = b.device()
    call = ta.PagedAttention((1, 2, 128), 8, b.dtype, 3, 3, DEV)
    call.reserve_shared()
    outs = [torch.empty_like(q) for _ in range(4)]

    def both(a, o):
        call.run(q, pool, 0, starts, lens, tables, 1, a, window=200, sinks=4)
        call.run_shared(q, pool, 0, ptable, 300, starts, lens, tables, 1, o)
    both(*outs[:2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(*outs[2:])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    again = [torch.empty_like(q) for _ in range(2)]
    with torch.cuda.graph(graph):
        both(*again)
    call.workspace.fill_(255)
    lens0 = lens.clone()
    lens.copy_(torch.tensor([20, 30, 40]))  # a replay goes by the lengths it finds
    graph.replay()
    short = again[0].clone()
    lens.copy_(lens0)
    graph.replay()
    torch.cuda.synchronize()
    assert ta.status_of(call.status) == 0
    for k in range(2):
        assert torch.equal(outs[k], outs[2 + k]) and torch.equal(outs[k], again[k])
    assert not torch.equal(short, again[0])
    want, _, tol = b.oracle()
    check_close(outs[1], want, tol)


def test_offsets_past_31_bits():
    # pages at the end of a pool whose halves hold more than 2^31 values
    H, D, page = 8, 128, 64
    pages = (1 << 31) // (H * D * page) + 3
    b = Batch([100, 90], [1, 40], 8, H, D, page, torch.float16, seed=8)
    q, small, starts, lens, tables, _ = b.device()
    pool = torch.empty(1, 2, pages, page, H, D, dtype=torch.float16, device=DEV)
    n = small.shape[2]
    pool[:, :, -n:] = small
    tables = torch.where(tables >= 0, tables + pages - n, tables)
    call = ta.PagedAttention((1, H, D), 8, b.dtype, 41, 2, DEV)
    out = call.run(q, pool, 0, starts, lens, tables, 40, torch.empty_like(q))
    torch.cuda.synchronize()
    assert ta.status_of(call.status) == 0
    want, _, tol = b.oracle()
    check_close(out, want, tol)


def test_wrapper_refusals():
    T = torch.float16
    call = ta.PagedAttention((1, 2, 64), 4, T, 5, 2, DEV)
    pool = torch.zeros(1, 2, 4, 16, 2, 64, dtype=T, device=DEV)
    q = torch.zeros(3, 4, 64, dtype=T, device=DEV)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)
    good = dict(q=q, pool=pool, layer=0, q_starts=i32([0, 1, 3]), kv_lens=i32([4, 5]),
                block_tables=i32([[0, 1], [2, 3]]), max_q=2, out=torch.empty_like(q))
    call.run(**good)
    big = torch.zeros(6, 4, 64, dtype=T, device=DEV)
    for name, value in (("q", q.float()), ("q", big), ("out", big[:2]), ("out", q.cpu()),
                        ("q_starts", i32([0, 1])), ("kv_lens", i32([1, 2, 3])),
                        ("kv_lens", i32([4, 5]).long()), ("block_tables", i32([[0, 1]])),
                        ("block_tables", i32([[0, 1], [2, 3]]).T), ("pool", pool[..., :32]),
                        ("lse", torch.zeros(2, device=DEV))):
        with pytest.raises(ValueError):
            call.run(**{**good, name: value})
    for name, value in (("out", q), ("max_q", 0), ("window", -1), ("layer", 1),
                        ("scale", float("nan"))):
        with pytest.raises(cg.CacheGenError):
            call.run(**{**good, name: value})
    with pytest.raises(ValueError):
        call.run_shared(**good, prefix_table=i32([1]), prefix_tokens=17)
    with pytest.raises(ValueError):
        ta.PagedAttention((1, 2, 64), 4, torch.float32, 5, 2, DEV)
    with pytest.raises(cg.CacheGenError):
        ta.PagedAttention((1, 2, 64), 3, T, 5, 2, DEV)
    torch.cuda.synchronize()
