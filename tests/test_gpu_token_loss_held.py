"""Fused token losses on rows that a workgroup holds on the chip, on the GPU, at
the sizes where the kernels' dispatch changes: a vocabulary that just enters a
thread's last chunk, one that fills the workgroup, one past it (the next
workgroup size, or the calls through a workspace).  Tolerances and definitions:
test_gpu_token_loss.py."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import fsdp_sharded_optimizer_flat_amd as z  # noqa: E402
from gpu_common import DEV  # noqa: E402
from test_gpu_token_loss import (DTYPES, MODES, check_distill, check_logprob, check_logprob_grad,  # noqa: E402
                                 gen, make_logits, make_record, matrix, workspace)


def capacity(dtype, threads, chunks):
    """(the vocabulary that a workgroup of `threads` threads of `chunks` 16-byte
    chunks holds wherever its rows start in a 128-byte line, elements of a chunk)"""
    es = torch.finfo(dtype).bits // 8
    w = 16 // es
    return threads * chunks * w - (128 // es - 1), w


def sizes(dtype, threads, chunks):
    most, w = capacity(dtype, threads, chunks)
    last = threads * (chunks - 1) * w      # the elements before a thread's last chunk
    return [last + 1, last + w * threads // 2 + 3, most, most + 1]


def outs(rows, vocab, dtype, stride):
    """Gradients at their logits' places in a line, and at others."""
    return [matrix(rows, vocab, dtype, stride, 1), matrix(rows, vocab, dtype, vocab + 3, 4)]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("threads", [64, 192, 448, 960])
def test_distill_capacities(threads, dtype):
    rows, k = 5, 33
    for n, vocab in enumerate(sizes(dtype, threads, 17)):
        print("distill", threads, vocab, dtype, flush=True)
        stride = vocab + 1 + vocab % 2     # odd: each row at another place
        x = make_logits(rows, vocab, dtype, 900 + n, stride, 1)
        index, value = make_record(x, k, 1.0, 7)
        index[0, 0], index[1, 1], index[2, 2] = vocab - 1, 0, vocab - 2    # the row's ends among the listed
        index[3] = -1                                                      # a padding row
        dl = torch.randn(rows, generator=gen(n), device=DEV)
        real = torch.arange(rows, device=DEV) != 3
        ws, wcheck = workspace(x)
        for name, mode in MODES.items():
            for out, check in outs(rows, vocab, dtype, stride):
                what = f"{vocab} {name}"
                loss = torch.full((rows,), 5.0, device=DEV)
                z.zero_distill_fused(x, index, value, mode, dl, out, loss=loss, workspace=ws)
                torch.cuda.synchronize()
                check(what)
                wcheck()
                check_distill(x[real], index[real], value[real], mode, 1.0, loss[real], dl[real], out[real], what)
                assert float(loss[3]) == 0 and bool((out[3] == 0).all()), what
        y, check = matrix(rows, vocab, dtype, stride, 1)
        y.copy_(x)
        z.zero_distill_fused(y, index, value, mode, dl, y, workspace=ws)
        torch.cuda.synchronize()
        check("in place")
        check_distill(x[real], index[real], value[real], mode, 1.0, None, dl[real], y[real], f"{vocab} in place")


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("threads", [64, 256, 512, 1024])
def test_logprob_capacities(threads, dtype):
    rows = 5
    for n, vocab in enumerate(sizes(dtype, threads, 16)):
        print("logprob", threads, vocab, dtype, flush=True)
        stride = vocab + 1 + vocab % 2
        x = make_logits(rows, vocab, dtype, 950 + n, stride, 1)
        tok = torch.randint(0, vocab, (rows,), generator=gen(n), device=DEV)
        tok[0], tok[1], tok[3] = vocab - 1, 0, -1
        real = tok >= 0
        dl = torch.randn(rows, generator=gen(10 + n), device=DEV)
        dh = torch.randn(rows, generator=gen(20 + n), device=DEV) * 0.1
        ws, wcheck = workspace(x)
        for e in (None, dh):
            for out, check in outs(rows, vocab, dtype, stride):
                what = f"{vocab} entropy {e is not None}"
                lp, h = torch.full((rows,), 5.0, device=DEV), torch.full((rows,), 5.0, device=DEV)
                z.zero_logprob_fused(x, tok, out, d_logprob=dl, d_entropy=e, logprob=lp, entropy=h, workspace=ws)
                torch.cuda.synchronize()
                check(what)
                wcheck()
                check_logprob(x[real], tok[real], 1.0, lp[real], h[real], None, what)
                check_logprob_grad(x[real], tok[real], 1.0, dl[real], None if e is None else e[real], out[real], what)
                assert float(lp[3]) == 0 and float(h[3]) == 0 and bool((out[3] == 0).all()), what
        y, check = matrix(rows, vocab, dtype, stride, 1)
        y.copy_(x)
        z.zero_logprob_fused(y, tok, y, d_logprob=dl, d_entropy=dh, workspace=ws)
        torch.cuda.synchronize()
        check("in place")
        check_logprob_grad(x[real], tok[real], 1.0, dl[real], dh[real], y[real], f"{vocab} in place")
