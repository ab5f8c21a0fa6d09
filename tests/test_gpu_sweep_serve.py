"""The serving sweep: a document decoded into the pool and a batch's step behind it."""
import json
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu


def test_serve_sweep_runs():
    run = subprocess.run([sys.executable, "-m", "kv_cache_compression_cachegen_b200.sweep",
                          "--config", "serve", "--warmup", "1", "--reps", "1"],
                         cwd=Path(__file__).resolve().parents[1], capture_output=True, text=True,
                         timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
    line = json.loads(run.stdout.strip().splitlines()[-1])
    assert line["workload"] == "llama2_7b" and line["requests"] == 64
    assert line["own_tokens"] == 301 and line["document_tokens"] == 10752
    assert all(line[k] > 0 for k in ("decode_document_ms", "extend_us", "append_us", "attend_us"))
