"""What a row must not notice: the largest finite values of keys it does not see."""
import pytest
import torch

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
