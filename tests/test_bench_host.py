"""bench.py refuses more than one GPU before it touches any (no GPU here)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("args,world", [(["--gpus", "2"], "1"), ([], "2"), (["--gpus", "8", "--impl", "reference"], "8"), (["--gpus", "0"], "1")])
def test_bench_is_for_one_gpu(args, world):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--steps", "1", "--warmup", "3", *args], capture_output=True, text=True,
                       env={**os.environ, "WORLD_SIZE": world, "RANK": "0", "LOCAL_RANK": "0"}, timeout=120)
    assert r.returncode == 1 and "one process on one GPU" in r.stderr and not r.stdout
