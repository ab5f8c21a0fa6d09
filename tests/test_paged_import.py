"""The torch layer on builds of torch that lack the private names it is fast by."""
import subprocess
import sys
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parents[1]
WITHOUT = """
import torch
for name in NAMES:
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from kv_cache_compression_cachegen_b200 import paged, torch_api
assert torch_api.PagedTables is paged.PagedTables
"""
USE = """
for _ in range(2):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        assert paged._raw_stream(0) == s.cuda_stream and paged._get_device() == 0
assert paged._raw_stream(0) == torch.cuda.current_stream(0).cuda_stream
t = torch_api.PagedTables(1, 2, 4, 4, "cuda")
one = torch.ones(1, dtype=torch.int32, device="cuda")
table = torch.full((1, 1), -1, dtype=torch.int32, device="cuda")
t.extend(t.kv_lens, one, table, one * 3)
torch.cuda.synchronize()
assert torch_api.status_of(t.status) == 0 and t.slots.tolist() == [12, -1]
"""


def run(names, code):
    subprocess.run([sys.executable, "-c", f"NAMES = {names}\n{code}"], cwd=ROOT, check=True,
                   timeout=300)


def test_imports_without_the_private_names():
    run(["_cuda_getCurrentRawStream", "_cuda_getDevice"], WITHOUT)


@pytest.mark.gpu
def test_runs_without_the_private_name_of_the_stream():
    run(["_cuda_getCurrentRawStream"], WITHOUT + USE)  # torch.cuda itself needs the other
