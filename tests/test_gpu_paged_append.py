"""cg_append_qkv and cg_rope_table against the formulas in 64 bits."""
import math

import pytest
import torch

import kv_cache_compression_cachegen_b200 as cg
from kv_cache_compression_cachegen_b200 import torch_api as ta
from paged_util import DTYPES, check_close, half_step

pytestmark = pytest.mark.gpu
DEV = "cuda"


def oracle(x, w, eps, table, positions, rot, inter, dtype):
    """(values, tolerance) for rows x [N, heads, D]: half a step of the type for
    the store; 16 fp32 steps (sum of D squares by halves, reciprocal root,
    three products and the rotation's sum) relative to the pair's size."""
    y = x.double()
    if w is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    size = y.abs()
    if rot:
        half = rot // 2
        a = torch.arange(0, rot, 2) if inter else torch.arange(half)
        b = a + 1 if inter else a + half
        c = table.double()[positions.long()][:, None, :half]
        s = table.double()[positions.long()][:, None, half:]
        z, big = y.clone(), size.clone()
        z[..., a] = y[..., a] * c - y[..., b] * s
        z[..., b] = y[..., b] * c + y[..., a] * s
        big[..., a] = big[..., b] = size[..., a] + size[..., b]
        y, size = z, big
    return y, half_step(dtype) * y.abs() * 1.001 + 16 * 2.0 ** -24 * size + 2.0 ** -25


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("N,Hq,H,D,rot,inter,norm,page", [
    (1, 1, 1, 16, 16, 0, 1, 1), (1, 32, 8, 128, 128, 0, 1, 16), (7, 6, 2, 64, 32, 1, 1, 7),
    (33, 8, 8, 80, 80, 0, 0, 16), (9, 4, 4, 80, 40, 0, 1, 16), (5, 4, 1, 96, 6, 0, 1, 3),
    (12, 5, 1, 112, 112, 1, 0, 16), (3, 2, 2, 256, 256, 0, 1, 64), (4, 4, 2, 240, 2, 0, 1, 5),
    (301, 7, 7, 48, 0, 0, 1, 16), (130, 64, 8, 128, 64, 0, 1, 16), (2, 3, 1, 32, 10, 1, 1, 16)])
def test_matches_the_formula(dtype, N, Hq, H, D, rot, inter, norm, page):
    T = DTYPES[dtype]
    g = torch.Generator().manual_seed(N * D + rot)
    qkv = (3 * torch.randn(N, Hq + 2 * H, D, generator=g)).to(T)
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(T) if norm else None for _ in range(2)]
    pages = -(-N // page) + 2
    far = 5000
    pos = torch.randint(0, far, (N,), generator=g, dtype=torch.int32)
    slots = torch.randperm(pages * page, generator=g)[:N]
    rope = ta.rope_table(far, rot, DEV, theta=5e5) if rot else None
    L, layer = 3, 1
    pool = torch.full((L, 2, pages, page, H, D), 7.0, dtype=T, device=DEV)
    call = ta.PagedAppend((L, H, D), Hq, T, DEV)
    dq = qkv.to(DEV)
    q_out = torch.zeros(N, Hq, D, dtype=T, device=DEV)
    wd = [None if x is None else x.to(DEV) for x in w]
    call.append(dq[:, :Hq], dq[:, Hq:Hq + H], dq[:, Hq + H:], q_out, pool, layer,
                pos.to(DEV) if rot else None, slots.to(DEV), rope, wd[0], wd[1], eps=1e-5,
                interleaved=bool(inter))
    torch.cuda.synchronize()
    assert ta.status_of(call.status) == 0
    table = rope.cpu() if rot else None
    want, tol = oracle(qkv[:, :Hq], w[0], 1e-5, table, pos, rot, inter, T)
    check_close(q_out, want, tol, "q")
    rows = pool.cpu().view(L, 2, -1, H, D)
    want, tol = oracle(qkv[:, Hq:Hq + H], w[1], 1e-5, table, pos, rot, inter, T)
    check_close(rows[layer, 0, slots], want, tol, "k")
    assert torch.equal(rows[layer, 1, slots], qkv[:, Hq + H:])
    # nothing else is touched
    rest = torch.ones(pages * page, dtype=torch.bool)
    rest[slots] = False
    assert (rows[layer][:, rest] == 7).all() and (rows[[0, 2]] == 7).all()
    assert torch.equal(dq.cpu(), qkv)
    # in place, rows left out where the slot is negative
    skip = torch.arange(N) % 3 == 1
    part = torch.where(skip, torch.full_like(slots, -1), slots)
    pool2 = torch.full_like(pool, 7.0)
    call.append(dq[:, :Hq], dq[:, Hq:Hq + H], dq[:, Hq + H:], dq[:, :Hq], pool2, layer,
                pos.to(DEV) if rot else None, part.to(DEV), rope, wd[0], wd[1], eps=1e-5,
                interleaved=bool(inter))
    torch.cuda.synchronize()
    assert ta.status_of(call.status) == 0
    got = dq.cpu()
    assert torch.equal(got[skip], qkv[skip])
    assert torch.equal(got[~skip][:, :Hq], q_out.cpu()[~skip])
    assert torch.equal(got[:, Hq:], qkv[:, Hq:])
    rows2 = pool2.cpu().view(L, 2, -1, H, D)
    assert torch.equal(rows2[layer][:, slots[~skip]], rows[layer][:, slots[~skip]])
    assert (rows2[layer][:, slots[skip]] == 7).all()


def test_bad_rows_are_left_out():
    N, H, D, page, pages = 6, 2, 64, 4, 5
    T = torch.float16
    x = torch.randn(N, 3 * H, D, device=DEV).to(T)
    rope = ta.rope_table(50, D, DEV)
    for slot, pos in ((pages * page, 3), (1 << 40, 3), (2, 50), (2, -1)):
        pool = torch.zeros(1, 2, pages, page, H, D, dtype=T, device=DEV)
        q_out = torch.zeros(N, H, D, dtype=T, device=DEV)
        call = ta.PagedAppend((1, H, D), H, T, DEV)
        slots = torch.arange(N, device=DEV) + 7
        positions = torch.arange(N, device=DEV, dtype=torch.int32)
        slots[3], positions[3] = slot, pos
        call.append(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], q_out, pool, 0, positions, slots, rope)
        torch.cuda.synchronize()
        assert ta.status_of(call.status) == cg.CG_ERR_MISMATCH
        assert (q_out[3] == 0).all() and (q_out[[0, 1, 2, 4, 5]] != 0).any(-1).all()
        wrote = (pool.view(2, -1, H * D) != 0).any(-1).nonzero()[:, 1].unique().tolist()
        assert wrote == [7, 8, 9, 11, 12]


def test_rope_table_far_positions():
    # angles of far positions: 64-bit, then one rounding to fp32
    n, rot, theta = 131072, 10, 10000.0
    t = ta.rope_table(n, rot, DEV, theta).cpu().double()
    p = torch.arange(n, dtype=torch.float64)[:, None]
    k = torch.arange(rot // 2, dtype=torch.float64)
    ang = p * theta ** (-2 * k / rot)
    # a few steps of 2^-52 of pow and of an angle up to 2^17, and half a step of fp32
    tol = 2.0 ** -24 * 1.001 + 2.0 ** 17 * 2.0 ** -50
    assert (t[:, :rot // 2] - ang.cos()).abs().max() <= tol
    assert (t[:, rot // 2:] - ang.sin()).abs().max() <= tol


def test_offsets_past_31_bits():
    # the last rows of a pool whose halves hold more than 2^31 values
    H, D, page = 8, 128, 64
    pages = (1 << 31) // (H * D * page) + 2
    T = torch.float16
    pool = torch.empty(1, 2, pages, page, H, D, dtype=T, device=DEV)
    last = pages * page
    pool[0, :, -1] = 0
    x = torch.randn(2, 3 * H, D, device=DEV).to(T)
    q_out = torch.empty(2, H, D, dtype=T, device=DEV)
    call = ta.PagedAppend((1, H, D), H, T, DEV)
    slots = torch.tensor([last - 1, last - 3], device=DEV)
    call.append(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], q_out, pool, 0, None, slots, None)
    torch.cuda.synchronize()
    assert ta.status_of(call.status) == 0
    assert torch.equal(pool[0, 0, -1, [-1, -3]], x[:, H:2 * H])
    assert torch.equal(pool[0, 1, -1, [-1, -3]], x[:, 2 * H:])
    assert torch.equal(q_out, x[:, :H])


def test_wrapper_refusals():
    T = torch.float16
    call = ta.PagedAppend((1, 2, 64), 4, T, DEV)
    pool = torch.zeros(1, 2, 4, 16, 2, 64, dtype=T, device=DEV)
    q, k = (torch.zeros(3, h, 64, dtype=T, device=DEV) for h in (4, 2))
    slots = torch.arange(3, device=DEV)
    good = dict(q=q, k=k, v=k, q_out=q.clone(), pool=pool, layer=0, positions=None, slots=slots,
                rope=None)
    call.append(**good)
    for name, value in (("q", q.float()), ("q", q[:2]), ("k", k.transpose(0, 1)),
                        ("v", k.expand(3, 2, 64)[:, :, ::2]), ("slots", slots.int()),
                        ("slots", slots[:2]), ("pool", pool[:, :1]), ("pool", pool.bfloat16()),
                        ("q_out", q.cpu()), ("rope", torch.zeros(4, device=DEV)),
                        ("q_weight", torch.zeros(64, device=DEV)),
                        ("k_weight", torch.zeros(32, dtype=T, device=DEV))):
        with pytest.raises(ValueError):
            call.append(**{**good, name: value})
    with pytest.raises(cg.CacheGenError):
        call.append(**{**good, "layer": 1})
    torch.cuda.synchronize()
    assert math.isfinite(float(pool.sum()))
