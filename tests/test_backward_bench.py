"""bench.py --streamed with the losses over sequences, the weight gradients of 8-bit
checkpoints and the embedding gradient.  On the CPU the refusals; on the GPU a short
run of each: one JSON line, and the mean loss that its inputs have."""
import json
import math
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RANKS, VOCAB, TOKENS = 8, 50304, 300


def _run(args, timeout=240):
    return subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--streamed", *args],
                          capture_output=True, text=True, timeout=timeout, cwd=ROOT)


@pytest.mark.parametrize("args", [["--workload", "gpt2l_block", "--loss", "policy"],
                                  ["--workload", "gpt2l", "--producer", "copy", "--loss", "preference"],
                                  ["--workload", "gpt2l", "--loss", "preference", "--tokens", "1"],
                                  ["--workload", "gpt2l", "--producer", "copy", "--embedding"],
                                  ["--workload", "gpt2l_block", "--embedding"]])
def test_passes_without_what_they_need_are_refused(args):
    res = _run(args)
    assert res.returncode != 0 and ("--loss" in res.stderr or "--embedding" in res.stderr), res.stderr
    assert res.stdout == ""


@pytest.mark.gpu
@pytest.mark.parametrize("loss", ["policy", "preference"])
def test_sequence_loss_lines(loss):
    print("bench --streamed --producer act8 --embedding --loss", loss, flush=True)
    res = _run(["--workload", "gpt2l", "--tokens", str(TOKENS), "--steps", "1", "--warmup", "1", "--loss", loss,
                "--producer", "act8", "--embedding"])
    assert res.returncode == 0, res.stderr[-3000:]
    d = json.loads(res.stdout)
    c = d["config"]
    assert c["loss"] == loss and c["producer"] == "act8" and c["embedding_gradient"]
    assert d["producer_tflops"] > 0 and d["ms"]["loss_only"]["median"] > 0
    # the logits read by both passes, and the gradients
    assert d["loss_bytes"] == 3 * RANKS * TOKENS * VOCAB * 2
    if loss == "policy":
        # -A r of 3 sequences of 8 ranks, A normal, r near 1 (deviation 0.1 a token): five
        # deviations of the mean
        assert abs(d["mean_loss"]) < 5 * 1.1 / math.sqrt(3 * RANKS)
    else:
        # ln 2 - h / 2 + ..., h = 0.1 (s_c - s_r), s of 150 log ratios of deviation 0.1
        h = 0.1 * 0.1 * math.sqrt(2 * 150)
        assert abs(d["mean_loss"] - math.log(2)) < 5 * h / 2 / math.sqrt(RANKS) + h * h


@pytest.mark.gpu
def test_producer_of_checkpoints_alone():
    print("bench --streamed --producer act8", flush=True)
    res = _run(["--workload", "gpt2l_block", "--tokens", "64", "--steps", "1", "--warmup", "1", "--producer", "act8"])
    assert res.returncode == 0, res.stderr[-3000:]
    d = json.loads(res.stdout)
    assert d["config"]["producer"] == "act8" and d["producer_tflops"] > 0 and "mean_loss" not in d
