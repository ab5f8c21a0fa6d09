"""What a row or a channel must not notice: the largest finite values, and
channels that are not turned beside ones that are not finite."""
import math

import pytest
import torch

from kv_cache_compression_cachegen_b200 import torch_api as ta
from test_gpu_paged_paths import attend, build, reference
from paged_util import check_close

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_largest_values_of_keys_that_only_later_rows_see(D, dtype):
    # a weight of 2^-125 times bf16's largest value is 8: a hidden key's has to be
    # zero.  One request for each of 32 neighbouring places of the hidden key.
    places, added, held = 32, 80, 64
    lens = [held + added] * places
    b = build(lens, [added] * places, 2, 1, D, 16, dtype, seed=D)
    flat, page = b["pool"][0], b["page"]
    good = torch.zeros(places * added, dtype=torch.bool)
    for r in range(places):
        at = held + 32 + r
        flat[1, int(b["tables"][r, at // page]), at % page] = torch.finfo(dtype).max
        good[r * added:r * added + 32 + r] = True
    want, tol = reference(b)
    out = attend(b).cpu()
    check_close(out[good], want[good], tol[good], "rows before the key")


@pytest.mark.parametrize("inter,rot,D", [(1, 12, 16), (1, 2, 16), (1, 30, 64), (1, 14, 80),
                                         (0, 12, 16), (0, 6, 32), (0, 26, 64)])
def test_channels_behind_the_rotation_pass_unchanged(inter, rot, D):
    # no norm: what is not turned comes out as it went in, whatever its neighbours hold
    T, N, H = torch.float16, 9, 2
    g = torch.Generator(device=DEV).manual_seed(rot)
    x = torch.randn(N, 3 * H, D, generator=g, device=DEV).to(T)
    x[1, :, rot + 1] = math.inf
    x[2, :, rot] = -math.inf
    x[3, :, rot:] = -0.0
    x[4, :, rot + 1] = math.nan
    pool = torch.zeros(1, 2, 2, 16, H, D, dtype=T, device=DEV)
    q_out = torch.zeros(N, H, D, dtype=T, device=DEV)
    call = ta.PagedAppend((1, H, D), H, T, DEV)
    slots = torch.arange(N, device=DEV) + 5
    positions = torch.arange(N, device=DEV, dtype=torch.int32) + 3
    call.append(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], q_out, pool, 0, positions, slots,
                ta.rope_table(50, rot, DEV), interleaved=bool(inter))
    torch.cuda.synchronize()
    assert ta.status_of(call.status) == 0
    got = torch.cat([q_out, pool[0, 0].view(-1, H, D)[slots]], 1)[..., rot:]
    want = x[:, :2 * H, rot:]
    same = (got.view(torch.int16) == want.view(torch.int16)) | (got.isnan() & want.isnan())
    assert same.all(), (~same).nonzero()[0].tolist()
