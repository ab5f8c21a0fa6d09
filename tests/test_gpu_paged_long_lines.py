"""Attention calls whose line of work has more units times CTAs than 32 bits
hold: long contexts of many requests, whose tables share a few pages."""
import math

import pytest
import torch

from kv_cache_compression_cachegen_b200 import torch_api as ta
from paged_util import check_close, half_step

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("shared", [False, True])
def test_more_units_than_32_bits_deal(shared):
    # 223 requests x 64 kv heads x (1,024 units + 1) = 14.63 million units for the
    # rows kernel's CTAs, two an SM.  Every table goes through the same 16 pages
    # 16 times, so each request attends 4,096 different keys with equal counts.
    T, B, H, D, page, pages, times = torch.float16, 223, 64, 16, 256, 16, 16
    prefix = 4 * page if shared else 0
    g = torch.Generator(device=DEV).manual_seed(11)
    pool = torch.randn(1, 2, pages, page, H, D, generator=g, device=DEV).to(T)
    q = torch.randn(B, H, D, generator=g, device=DEV).to(T)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)
    tables = i32([list(range(pages)) * times] * B)
    lens, starts = i32([pages * page * times] * B), i32(list(range(B + 1)))
    call = ta.PagedAttention((1, H, D), H, T, B, B, DEV)
    if shared:
        call.reserve_shared()
    call.workspace.fill_(255)
    out = torch.full_like(q, 3.0)
    lse = torch.full((B, H), 5.0, device=DEV)
    if shared:
        call.run_shared(q, pool, 0, tables[0], prefix, starts, lens, tables, 1, out, lse=lse)
    else:
        call.run(q, pool, 0, starts, lens, tables, 1, out, lse=lse)
    torch.cuda.synchronize()
    assert ta.status_of(call.status) == 0
    k, v = pool[0].reshape(2, -1, H, D).double()
    count = torch.full((pages * page,), float(times), dtype=torch.float64, device=DEV)
    count[:prefix] += 1
    u = half_step(T)
    for h in range(H):
        s = q[:, h].double() @ k[:, h].T / math.sqrt(D)
        big = (q[:, h].double().abs() @ k[:, h].abs().T).amax(-1, keepdim=True) / math.sqrt(D)
        m = s.amax(-1, keepdim=True)
        e = torch.exp(s - m) * count
        total = e.sum(-1, keepdim=True)
        want, mass = e @ v[:, h] / total, e @ v[:, h].abs() / total
        # half a step for the output and for each weight (an fp16 weight below the
        # normal range: 2^-25), the scores' fp32 products, and up to 1,024 products
        # of 16 keys added to a warp's fp32 sums, twice (sum and weighted sum)
        faint = 2.0 ** -25 * (count @ v[:, h].abs()) / total
        score = (D + 4) * 2.0 ** -24 * big
        tol = u * want.abs() + (u + 2 * score + 2.0 ** -12) * mass + faint
        check_close(out[:, h], want.cpu(), (tol * 1.01 + 1e-7).cpu(), f"head {h}")
        exact = (m + torch.log(total)).squeeze(-1)
        assert ((lse[:, h].double() - exact).abs() <= 2.0 ** -11).all()
