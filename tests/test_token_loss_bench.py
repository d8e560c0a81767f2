"""bench.py --streamed --loss: the losses on the streamed pass.  On the CPU the
refusals; on the GPU a short run of each loss: one JSON line, and the mean loss
that its logits have (normal with deviation 2: ln V + 2 for the language-model
loss against tokens drawn evenly)."""
import json
import math
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run(args, timeout=240):
    return subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--streamed", *args],
                          capture_output=True, text=True, timeout=timeout, cwd=ROOT)


@pytest.mark.parametrize("args", [["--workload", "gpt2l_block", "--loss", "lm"],
                                  ["--workload", "gpt2l", "--producer", "copy", "--loss", "distill"],
                                  ["--workload", "gpt2l", "--loss", "distill", "--top-k", "0"],
                                  ["--workload", "gpt2l", "--loss", "distill", "--top-k", "257"]])
def test_losses_without_a_head_or_a_record_are_refused(args):
    res = _run(args)
    assert res.returncode != 0 and ("--loss" in res.stderr or "--top-k" in res.stderr), res.stderr
    assert res.stdout == ""


@pytest.mark.gpu
@pytest.mark.parametrize("loss", ["lm", "distill"])
def test_loss_line(loss):
    print("bench --streamed --loss", loss, flush=True)
    res = _run(["--workload", "gpt2l", "--tokens", "64", "--steps", "1", "--warmup", "1", "--loss", loss])
    assert res.returncode == 0, res.stderr[-3000:]
    d = json.loads(res.stdout)
    assert d["config"]["loss"] == loss and d["loss_hbm_GBps"] > 0 and d["ms"]["loss_only"]["median"] > 0
    if loss == "lm":
        # ln sum e^l of 50304 normal logits: ln V + 2, its deviation from row
        # to row sqrt((e^4 - 1) / V) = 0.033; the token's logit: 0 +- 2 over 512
        # rows (64 rows of logits, read by 8 ranks): five deviations of the mean
        assert abs(d["mean_loss"] - (math.log(50304) + 2.0)) < 5 * math.hypot(2.0 / math.sqrt(512), 0.033 / 8)
    else:
        # -H(q) + ln sum e^l - sum q l: ln V + 2 less an entropy of at most ln 64
        # and less a mean of the student's logits (independent of the teacher's;
        # deviation at most 2 / sqrt(64 rows))
        assert -math.log(64) - 1.3 < d["mean_loss"] - (math.log(50304) + 2.0) < 1.3
