"""bench.py --streamed --loss counts the bytes of tensors that are there: each
simulated rank has logits of its own, so that the reported rate is not that of
one rank's logits read again from a cache."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RANKS, VOCAB, TOKENS = 8, 50304, 64


@pytest.mark.parametrize("loss,tensors", [("lm", 2), ("distill", 3)])
def test_bytes_of_every_rank(loss, tensors):
    print("bench --streamed --loss", loss, flush=True)
    res = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--streamed", "--workload", "gpt2l",
                          "--tokens", str(TOKENS), "--steps", "1", "--warmup", "1", "--loss", loss],
                         capture_output=True, text=True, timeout=240, cwd=ROOT)
    assert res.returncode == 0, res.stderr[-3000:]
    d = json.loads(res.stdout)
    # bf16 logits and gradients, and the teacher's logits, of RANKS ranks
    assert d["loss_bytes"] == tensors * RANKS * TOKENS * VOCAB * 2
    ms = d["ms"]["loss_only"]["median"]
    assert abs(d["loss_hbm_GBps"] - d["loss_bytes"] / ms / 1e6) <= 1e-3 * d["loss_hbm_GBps"]
