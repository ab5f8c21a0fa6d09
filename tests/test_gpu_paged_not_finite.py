"""Values that are not finite under chunks of rows: rows that do not see them are
right, rows that do show them, and neither takes the time of a fault."""
import math

import pytest
import torch

from kv_cache_compression_cachegen_b200 import torch_api as ta
from paged_util import check_close, half_step
from test_gpu_paged_paths import attend, build, reference

pytestmark = pytest.mark.gpu
DEV = "cuda"


def place(b, r, at):
    """The values of key `at` of request r: [heads, channels]."""
    return b["pool"][0][1, int(b["tables"][r, at // b["page"]]), at % b["page"]]


def verify_with(b, spots, bad, window=0, sinks=0):
    """spots: (request, key, channel or None for all) whose values become `bad`."""
    for r, at, ch in spots:  # the reference has zeros there
        place(b, r, at)[:, slice(None) if ch is None else ch] = 0
    want, tol = reference(b, window, sinks)
    for r, at, ch in spots:
        place(b, r, at)[:, slice(None) if ch is None else ch] = bad
    out = attend(b, window, sinks).cpu()
    starts, lens, added = b["host"]
    good = torch.ones_like(out, dtype=torch.bool)
    for r, at, ch in spots:
        p = lens[r] - added[r] + torch.arange(added[r])
        sees = at <= p
        if window:
            sees &= (at > p - window) | torch.tensor(at < sinks)
        rows = starts[r] + sees.nonzero()[:, 0]
        good[rows, :, slice(None) if ch is None else ch] = False
    check_close(out[good], want[good], tol[good], "values that see nothing bad")
    assert not torch.isfinite(out[~good].float()).any()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("Hq,H,D", [(4, 2, 64), (2, 1, 128), (2, 2, 80), (2, 1, 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 0), (130, 9)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_rows_that_see_and_rows_that_do_not(dtype, Hq, H, D, window, sinks, bad):
    # one channel of an early key, of keys at the window's edges and of new keys
    added, lens = [300, 90, 1, 150], [520, 400, 333, 150]
    spots = [(0, 3, 5), (0, 215, 7), (0, 300, 5), (1, 250, 11), (1, 390, None), (3, 0, 2),
             (3, 149, 3)]
    b = build(lens, added, Hq, H, D, 16, dtype, seed=D)
    verify_with(b, spots, bad, window, sinks)


def test_a_value_that_later_new_tokens_see_behind_long_contexts():
    # 160 items for the SMs, whole each: the first 60 new tokens of each request are
    # computed again over 20,000 keys
    n, B = 100, 40
    b = build([20000 + n] * B, [n] * B, 8, 4, 64, 16, torch.float16, seed=1)
    verify_with(b, [(r, 20060, None) for r in range(0, B, 3)], math.nan)


@pytest.mark.parametrize("what", ["one channel", "values", "keys"])
def test_one_bad_early_token_of_long_contexts(what):
    # every row of a chunk sees it: nothing is computed again, and other requests are
    # right.  Tables go through the same 4,096 keys, 49 times: 160 items of 200,000 keys.
    T, B, H, D, page, n = torch.float16, 40, 4, 64, 16, 100
    unique, keys = 4096, 200000
    g = torch.Generator(device=DEV).manual_seed(2)
    pages = unique // page
    # requests from 20 on have pages of their own, without the bad token
    pool = torch.randn(1, 2, 2 * pages, page, H, D, generator=g, device=DEV).to(T)
    pool[:, :, pages:] = pool[:, :, :pages]
    if what == "one channel":
        pool[0, 1, 0, 5, :, 3] = math.inf
    else:
        pool[0, 0 if what == "keys" else 1, 0, 5] = math.nan

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)
    columns = -(-keys // page)
    first = [c % pages for c in range(columns)]
    tables = i32([first] * 20 + [[pages + c for c in first]] * 20)
    one = torch.randn(n, 2 * H, D, generator=g, device=DEV).to(T)
    q = one.repeat(B, 1, 1)
    call = ta.PagedAttention((1, H, D), 2 * H, T, B * n, B, DEV)
    out = torch.full_like(q, 3.0)
    call.run(q, pool, 0, i32([n * r for r in range(B + 1)]), i32([keys] * B), tables, n, out)
    torch.cuda.synchronize()
    assert ta.status_of(call.status) == 0
    k, v = pool[0, :, pages:].reshape(2, -1, H, D).double().repeat_interleave(2, 2)
    p = keys - n + torch.arange(n, device=DEV)[:, None]
    count = ((p - torch.arange(unique, device=DEV)[None]).div(unique, rounding_mode="floor")
             + 1).double()
    s = torch.einsum("nhd,mhd->hnm", one.double(), k) / math.sqrt(D)
    big = torch.einsum("nhd,mhd->hnm", one.double().abs(), k.abs()).amax(-1) / math.sqrt(D)
    e = torch.exp(s - s.amax(-1, keepdim=True)) * count
    total = e.sum(-1).T[..., None]
    want = torch.einsum("hnm,mhd->nhd", e, v) / total
    mass = torch.einsum("hnm,mhd->nhd", e, v.abs()) / total
    u = half_step(T)
    # as elsewhere, and up to 12,500 products of 16 keys added in fp32, one step
    # of 2^-23 each, in the weighted sum and the sum
    score = (D + 4) * 2.0 ** -24 * big.T[..., None]
    faint = 2.0 ** -25 * torch.einsum("nm,mhd->nhd", count, v.abs()) / total
    tol = u * want.abs() + (u + 2 * score + 2 * 12500 * 2.0 ** -23) * mass + faint
    want, tol = want.cpu(), (tol * 1.01 + 1e-7).cpu()
    out = out.cpu().view(B, n, 2 * H, D)
    for r in range(20, B):
        check_close(out[r], want, tol, f"request {r}")
    for r in range(20):
        if what == "one channel":
            rest = [d for d in range(D) if d != 3]
            check_close(out[r][..., rest], want[..., rest], tol[..., rest], f"request {r}")
            assert not torch.isfinite(out[r][..., 3].float()).any()
        else:
            assert torch.isnan(out[r].float()).all()


def test_rows_computed_again_for_longer_than_a_wait_may_take():
    # 120 rows of request 0 over 900,000 keys: seconds, in which its CTAs' other warps
    # wait.  As above, but the bad value is a new token's that these rows do not see.
    T, B, H, D, page, n = torch.float16, 40, 4, 64, 16, 100
    unique, keys, bad = 4096, 900000, 900000 - 100 + 60
    g = torch.Generator(device=DEV).manual_seed(3)
    pages = unique // page
    pool = torch.randn(1, 2, pages + 1, page, H, D, generator=g, device=DEV).to(T)
    columns = -(-keys // page)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)
    tables = i32([[c % pages for c in range(columns)]] * B)
    pool[:, :, pages] = pool[:, :, bad // page % pages]
    tables[0, bad // page] = pages
    pool[0, 1, pages, bad % page] = math.nan
    one = (4 * torch.randn(n, 2 * H, D, generator=g, device=DEV)).to(T)
    q = one.repeat(B, 1, 1)
    call = ta.PagedAttention((1, H, D), 2 * H, T, B * n, B, DEV)
    out = torch.full_like(q, 3.0)
    call.run(q, pool, 0, i32([n * r for r in range(B + 1)]), i32([keys] * B), tables, n, out)
    torch.cuda.synchronize()
    assert ta.status_of(call.status) == 0
    k, v = pool[0, :, :pages].reshape(2, -1, H, D).double().repeat_interleave(2, 2)
    p = keys - n + torch.arange(n, device=DEV)[:, None]
    count = ((p - torch.arange(unique, device=DEV)[None]).div(unique, rounding_mode="floor")
             + 1).double()
    s = torch.einsum("nhd,mhd->hnm", one.double(), k) / math.sqrt(D)
    big = torch.einsum("nhd,mhd->hnm", one.double().abs(), k.abs()).amax(-1) / math.sqrt(D)
    e = torch.exp(s - s.amax(-1, keepdim=True)) * count
    total = e.sum(-1).T[..., None]
    want = torch.einsum("hnm,mhd->nhd", e, v) / total
    mass = torch.einsum("hnm,mhd->nhd", e, v.abs()) / total
    u = half_step(T)
    score = (D + 4) * 2.0 ** -24 * big.T[..., None]
    faint = 2.0 ** -25 * torch.einsum("nm,mhd->nhd", count, v.abs()) / total
    # fp32 sums: 900,000 single products of half a step of 2^-24 each where a row is
    # computed again, else 56,250 products of 16 keys, 2^-23 each and twice
    tol = u * want.abs() + (u + 2 * score + 2.0 ** -24 * 900000) * mass + faint
    want, tol = want.cpu(), (tol * 1.01 + 1e-7).cpu()
    out = out.cpu().view(B, n, 2 * H, D)
    check_close(out[0, :60], want[:60], tol[:60], "rows before the bad token")
    assert torch.isnan(out[0, 60:].float()).all()
    for r in range(1, B):
        check_close(out[r], want, tol, f"request {r}")
