"""The token losses as a training step uses them, on the GPU: a teacher's record,
the student's loss and gradient, the head's weight gradient, the sharded
optimizer step, the next logits; a bad token that skips the clipped step; and
the calls side by side on streams, host threads and graphs of their own.

The losses are checked against binary64 with the tolerances of
test_gpu_token_loss.py (checked there); the step against the oracle, bit for
bit, from the very buckets the losses' gradients went into."""
import threading

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import oracle  # noqa: E402
import fsdp_sharded_optimizer_flat_amd as z  # noqa: E402
from gpu_common import DEV, assert_same_bf16, assert_same_f32, hyper_args, scalars, to_np  # noqa: E402
from test_gpu_token_loss import (MODES, check_distill, check_logprob, check_logprob_grad,  # noqa: E402
                                 check_top, gen, make_logits, make_record, matrix, ref_logp, workspace)

G, Lc = z.ZERO_GLOBAL, z.ZERO_LOCAL
H = dict(lr=1e-2, b1=0.9, b2=0.95, eps=1e-8, wd=0.1)
N = 4          # simulated ranks
TOKENS = 96    # of each rank
VOCAB, WIDTH = 5003, 64


class Head:
    """A vocabulary head of VOCAB x WIDTH parameters as the one unit of a layout
    over N ranks, every rank's shard on this device."""

    def __init__(self, seed):
        self.numel = [VOCAB * WIDTH]
        self.L = z.zero_pack(N, self.numel)
        g = gen(seed)
        self.master = torch.zeros(self.L.padded, device=DEV)
        self.master[:self.numel[0]] = torch.randn(self.numel[0], generator=g, device=DEV) * 0.3
        self.m, self.v = torch.zeros_like(self.master), torch.zeros_like(self.master)
        self.out = self.master.to(torch.bfloat16).view(torch.int16).clone()
        self.buckets = [torch.zeros(self.L.padded, dtype=torch.bfloat16, device=DEV) for _ in range(N)]
        self.x = [torch.randn(TOKENS, WIDTH, generator=g, device=DEV).to(torch.bfloat16) for _ in range(N)]
        self.teacher = torch.randn(VOCAB, WIDTH, generator=g, device=DEV).to(torch.bfloat16) * 0.4
        self.tokens = [torch.randint(0, VOCAB, (TOKENS,), generator=g, device=DEV) for _ in range(N)]

    def weights(self):   # the gathered bf16 parameters of the last step
        return self.out.view(torch.bfloat16)[:self.numel[0]].view(VOCAB, WIDTH)

    def logits(self, r):
        return torch.mm(self.x[r], self.weights().t())

    def weight_gradient(self, r, d_logits):
        torch.mm(d_logits.t(), self.x[r], out=self.buckets[r][:self.numel[0]].view(VOCAB, WIDTH))

    def oracle_state(self):
        return [to_np(t).copy() for t in (self.master, self.m, self.v, self.out)]


def test_distillation_and_language_model_steps():
    """Ranks 0 and 1 distill (TAIL, RENORM) from records that zero_logprob writes,
    rank 2 has the language-model loss with padding, rank 3 the same with an
    entropy bonus through the separate forward and backward calls; two steps."""
    head = Head(1)
    k = 32
    head.tokens[2][::7] = -1
    want = head.oracle_state()
    losses = []
    for t in (1, 2):
        mean = torch.zeros(N, device=DEV)
        for r in range(N):
            x = head.logits(r)
            d = torch.empty_like(x)
            ws, check = workspace(x, k)
            what = f"step {t} rank {r}"
            if r < 2:
                mode = MODES["tail" if r == 0 else "renorm"]
                y = torch.mm(head.x[r], head.teacher.t())
                index = torch.empty(TOKENS, k, dtype=torch.int32, device=DEV)
                value = torch.empty(TOKENS, k, device=DEV)
                loss = torch.empty(TOKENS, device=DEV)
                dl = torch.full((TOKENS,), 1.0 / TOKENS, device=DEV)
                z.zero_logprob(y, scale=0.5, top_index=index, top_logprob=value, workspace=ws)
                z.zero_distill_fused(x, index, value, mode, dl, d, scale=0.5, loss=loss, workspace=ws)
                torch.cuda.synchronize()
                check_top(y, 0.5, k, index, value, what)
                check_distill(x, index, value, mode, 0.5, loss, dl, d, what)
                mean[r] = loss.mean()
            else:
                tok = head.tokens[r]
                real = tok >= 0
                dl = torch.full((TOKENS,), -1.0 / int(real.sum()), device=DEV)
                lp = torch.empty(TOKENS, device=DEV)
                if r == 2:
                    dh, h = None, None
                    z.zero_logprob_fused(x, tok, d, d_logprob=dl, logprob=lp, workspace=ws)
                else:
                    dh = torch.full((TOKENS,), -0.01 / TOKENS, device=DEV)
                    h, stats = torch.empty(TOKENS, device=DEV), torch.empty(TOKENS, 2, device=DEV)
                    z.zero_logprob(x, tok, logprob=lp, entropy=h, stats=stats, workspace=ws)
                    z.zero_logprob_grad(x, tok, stats, d, d_logprob=dl, d_entropy=dh, entropy=h)
                torch.cuda.synchronize()
                check_logprob(x[real], tok[real], 1.0, lp[real], None if h is None else h[real], None, what)
                check_logprob_grad(x[real], tok[real], 1.0, dl[real], None if dh is None else dh[real],
                                   d[real], what)
                assert bool((lp[~real] == 0).all()) and bool((d[~real] == 0).all()), what
                mean[r] = -lp.sum() / int(real.sum())
            check()
            head.weight_gradient(r, d)
        losses.append(mean)
        z.zero_step_units(head.L, -1, 0, 1, head.buckets, G, float(N), head.master, head.m, head.v, G,
                          head.out, G, scalars(t, H))
        torch.cuda.synchronize()
        oracle.zero_step_all(N, head.numel, [np.ascontiguousarray(to_np(b)) for b in head.buckets],
                             divisor=float(N), clip=1.0, master=want[0], m=want[1], v=want[2], out=want[3],
                             t=t, **hyper_args(H))
        for got, w, name in zip((head.master, head.m, head.v), want, ("master", "m", "v")):
            assert_same_f32(to_np(got), w, f"{name} after step {t}")
        assert_same_bf16(to_np(head.out), want[3], f"out after step {t}")
    assert bool(torch.isfinite(torch.stack(losses)).all())


@pytest.mark.parametrize("fault", ["token", "record"])
def test_a_bad_target_skips_the_clipped_step(fault):
    """A token, or a record's index, past the vocabulary: NaN in its gradient row,
    so in the weight gradient, the norm and the clip coefficient; master, m, v
    and out stay as they were.  With the target mended the same chain steps."""
    head = Head(2)
    L, rank = head.L, 1
    st = [t[L.shard * rank:L.shard * (rank + 1)].contiguous() for t in (head.master, head.m, head.v, head.out)]
    coef = torch.empty(1, device=DEV)
    ss = torch.empty(1, dtype=torch.float64, device=DEV)
    nws = torch.zeros(z.zero_gradnorm_workspace_bytes(L, rank) // 8, dtype=torch.float64, device=DEV)
    red = torch.zeros(L.shard, device=DEV)
    for bad in (True, False):
        for r in range(N):
            x = head.logits(r)
            d = torch.empty_like(x)
            ws = workspace(x)[0]
            w = torch.full((TOKENS,), 1.0 / TOKENS, device=DEV)
            if fault == "token":
                tok = head.tokens[r].clone()
                if bad and r == 2:
                    tok[11] = VOCAB
                z.zero_logprob_fused(x, tok, d, d_logprob=-w, workspace=ws)
            else:
                index, value = make_record(x, 8, 1.0, 3)
                if bad and r == 2:
                    index[11, 5] = VOCAB
                z.zero_distill_fused(x, index, value, MODES["tail"], w, d, workspace=ws)
            assert bool(torch.isnan(d).any()) == (bad and r == 2)
            head.weight_gradient(r, d)
        before = [to_np(t).copy() for t in st]
        z.zero_gradnorm_async(L, rank, head.buckets, G, float(N), red, Lc, nws, ss)
        z.zero_clip_coef_async(ss, 1.0, coef)
        z.zero_step_device_clip(L, rank, [red], Lc, 1.0, *st[:3], Lc, st[3], Lc, scalars(1, H), coef)
        torch.cuda.synchronize()
        same = [np.array_equal(to_np(t).view(np.uint8), b.view(np.uint8)) for t, b in zip(st, before)]
        assert bool(torch.isnan(coef).all()) == bad
        assert all(same) if bad else not any(same), (bad, same)


class Job:
    """All six calls on inputs, outputs and a workspace of its own."""

    def __init__(self, seed, rows, vocab, dtype):
        self.x = make_logits(rows, vocab, dtype, seed)
        self.tok = torch.randint(0, vocab, (rows,), generator=gen(seed), device=DEV)
        self.index, self.value = make_record(self.x, 24, 1.0, seed)
        self.w = torch.rand(rows, generator=gen(seed + 1), device=DEV)
        self.ws = workspace(self.x, 24)[0]
        f = lambda *s: torch.zeros(*s, device=DEV)
        self.o = dict(lp=f(rows), h=f(rows), st=f(rows, 2), i=torch.zeros(rows, 24, dtype=torch.int32, device=DEV),
                      t=f(rows, 24), loss=f(rows), st4=f(rows, 4), loss2=f(rows), lp2=f(rows),
                      **{f"g{n}": torch.zeros_like(self.x) for n in range(4)})

    def run(self, stream=None):
        o, x = self.o, self.x
        z.zero_logprob(x, self.tok, logprob=o["lp"], entropy=o["h"], stats=o["st"], top_index=o["i"],
                       top_logprob=o["t"], workspace=self.ws, stream=stream)
        z.zero_logprob_grad(x, self.tok, o["st"], o["g0"], d_logprob=self.w, d_entropy=self.w,
                            entropy=o["h"], stream=stream)
        z.zero_logprob_fused(x, self.tok, o["g1"], d_logprob=self.w, d_entropy=self.w, logprob=o["lp2"],
                             workspace=self.ws, stream=stream)
        z.zero_distill(x, self.index, self.value, MODES["tail"], loss=o["loss"], stats=o["st4"],
                       workspace=self.ws, stream=stream)
        z.zero_distill_grad(x, self.index, self.value, MODES["tail"], o["st4"], self.w, o["g2"], stream=stream)
        z.zero_distill_fused(x, self.index, self.value, MODES["renorm"], self.w, o["g3"], loss=o["loss2"],
                             workspace=self.ws, stream=stream)

    def take(self):
        """The outputs' bits; the outputs are cleared."""
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in self.o.items()}
        for t in self.o.values():
            t.zero_()
        torch.cuda.synchronize()
        return got


# rows held on the chip and rows that go through the workspace, both types
JOBS = [(31, 40, 30011, torch.bfloat16), (32, 5, 140001, torch.bfloat16), (33, 12, 70001, torch.float32),
        (34, 300, 513, torch.float32)]


def assert_same(got, want, what):
    for n in want:
        assert torch.equal(got[n].view(torch.uint8), want[n].view(torch.uint8)), (what, n)


def test_side_by_side_on_streams_and_threads():
    jobs = [Job(*j) for j in JOBS]
    want = []
    for j in jobs:
        j.run()
        want.append(j.take())
        assert bool(torch.isfinite(want[-1]["g1"].float()).all()) and bool((want[-1]["g1"] != 0).any())
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(3):
        for j, s in zip(jobs, streams):
            j.run(s)
    for j, w in zip(jobs, want):
        assert_same(j.take(), w, "streams")
    errors = []

    def worker(j, s, gate):
        try:
            gate.wait()
            for _ in range(5):
                j.run(s)
        except BaseException as e:   # noqa: BLE001 -- reported below
            errors.append(e)
    gate = threading.Barrier(len(jobs))
    threads = [threading.Thread(target=worker, args=(j, s, gate)) for j, s in zip(jobs, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for j, w in zip(jobs, want):
        assert_same(j.take(), w, "threads")


def test_two_graphs_replayed_together():
    """Graphs with workspaces of their own, replayed at once on two streams with
    eager work between the replays."""
    jobs = [Job(*j) for j in JOBS[1:3]]
    want = []
    for j in jobs:
        j.run()
        want.append(j.take())
    graphs = []
    for j in jobs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            j.run()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in jobs]
    for turn in range(3):
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        for j, w in zip(jobs, want):
            assert_same(j.take(), w, f"turn {turn}")
        jobs[0].run()
        assert_same(jobs[0].take(), want[0], "eager")


def test_columns_of_a_wider_matrix_and_reversed_use():
    """Logits that are a column range of a wider matrix, its other columns
    untouched, and a forward pass whose statistics serve the backward pass of the
    same rows in a copy at another stride."""
    rows, vocab = 33, 2051
    wide = make_logits(rows, 2 * vocab + 5, torch.bfloat16, 77)
    keep = wide.clone()
    x = wide[:, vocab:2 * vocab]
    tok = torch.randint(0, vocab, (rows,), generator=gen(3), device=DEV)
    lp, st = torch.empty(rows, device=DEV), torch.empty(rows, 2, device=DEV)
    z.zero_logprob(x, tok, logprob=lp, stats=st, workspace=workspace(x)[0])
    dl = torch.full((rows,), -1.0, device=DEV)
    d = torch.empty(rows, vocab, dtype=torch.bfloat16, device=DEV)
    z.zero_logprob_grad(x.contiguous(), tok, st, d, d_logprob=dl)
    z.zero_logprob_grad(x, tok, st, x, d_logprob=dl)      # in place, in the wider matrix
    torch.cuda.synchronize()
    y = keep[:, vocab:2 * vocab].contiguous()
    check_logprob(y, tok, 1.0, lp, None, st, "columns")
    check_logprob_grad(y, tok, 1.0, dl, None, d, "columns")
    assert torch.equal(d.view(torch.int16), x.contiguous().view(torch.int16))
    assert torch.equal(wide[:, :vocab], keep[:, :vocab]) and torch.equal(wide[:, 2 * vocab:], keep[:, 2 * vocab:])
    assert bool(torch.isfinite(ref_logp(y, 1.0)).all())


def test_no_rows():
    """Empty batches through the binding: nothing is written, nothing refused."""
    x = torch.empty(0, 500, dtype=torch.bfloat16, device=DEV)
    f, st, st4 = (torch.empty(0, *s, device=DEV) for s in ((), (2,), (4,)))
    tok = torch.empty(0, dtype=torch.int64, device=DEV)
    i, v = torch.empty(0, 5, dtype=torch.int32, device=DEV), torch.empty(0, 5, device=DEV)
    assert z.zero_loss_workspace_bytes(0, 500, 5) == 0
    z.zero_logprob(x, tok, logprob=f, entropy=f, stats=st, top_index=i, top_logprob=v)
    z.zero_logprob_grad(x, tok, st, x, d_logprob=f, d_entropy=f, entropy=f)
    z.zero_logprob_fused(x, tok, x.clone(), d_logprob=f, logprob=f)
    for mode in MODES.values():
        z.zero_distill(x, i, v, mode, loss=f, stats=st4)
        z.zero_distill_grad(x, i, v, mode, st4, f, x)
        z.zero_distill_fused(x, i, v, mode, f, x.clone(), loss=f)
    torch.cuda.synchronize()


def test_rows_of_one_tensor_are_refused():
    """Rows that share memory (an expanded tensor) and columns of a transposed one."""
    x = torch.zeros(1, 500, dtype=torch.bfloat16, device=DEV).expand(4, 500)
    lp, tok = torch.empty(4, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)
    with pytest.raises(z.ZeroError):
        z.zero_logprob(x, tok, logprob=lp)
    with pytest.raises(ValueError):
        z.zero_logprob(torch.zeros(500, 4, device=DEV).t(), tok, logprob=lp)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("vocab", [1, 5, 31, 64, 67, 517, 2049, 9001])
def test_every_place_in_a_cache_line(vocab, dtype):
    """Rows that start at each place of a 128-byte line (an odd stride walks through
    them), gradients at the same places, at others and in place; what lies between
    the rows stays as it was."""
    rows, k = 70, 8
    stride = vocab + 1 + vocab % 2
    x = make_logits(rows, vocab, dtype, 500 + vocab, stride, 3)
    places = {(x[r].data_ptr() // x.element_size()) % (128 // x.element_size()) for r in range(rows)}
    assert len(places) == 128 // x.element_size()
    tok = torch.randint(0, vocab, (rows,), generator=gen(1), device=DEV)
    index, value = make_record(x, k, 1.0, 3)
    w, h = torch.rand(rows, generator=gen(2), device=DEV), torch.rand(rows, generator=gen(3), device=DEV)
    ws = workspace(x, k)[0]
    f = lambda *s: torch.empty(*s, device=DEV)
    lp, ent, st, st4, loss = f(rows), f(rows), f(rows, 2), f(rows, 4), f(rows)
    ti, tv = torch.empty(rows, k, dtype=torch.int32, device=DEV), f(rows, k)
    z.zero_logprob(x, tok, logprob=lp, entropy=ent, stats=st, top_index=ti, top_logprob=tv, workspace=ws)
    z.zero_distill(x, index, value, MODES["tail"], loss=loss, stats=st4, workspace=ws)
    torch.cuda.synchronize()
    check_logprob(x, tok, 1.0, lp, ent, st, "forward")
    check_top(x, 1.0, k, ti, tv, "forward")
    check_distill(x, index, value, MODES["tail"], 1.0, loss, None, None, "forward")
    for out_stride, shift in ((stride, 3), (stride + 2, 4), (vocab, 0)):
        for fused in (False, True):
            what = f"stride {out_stride} shift {shift} fused {fused}"
            out, check = matrix(rows, vocab, dtype, out_stride, shift)
            if fused:
                z.zero_logprob_fused(x, tok, out, d_logprob=w, d_entropy=h, logprob=lp, workspace=ws)
            else:
                z.zero_logprob_grad(x, tok, st, out, d_logprob=w, d_entropy=h, entropy=ent)
            torch.cuda.synchronize()
            check(what)
            check_logprob_grad(x, tok, 1.0, w, h, out, what)
            out, check = matrix(rows, vocab, dtype, out_stride, shift)
            if fused:
                z.zero_distill_fused(x, index, value, MODES["tail"], w, out, loss=loss, workspace=ws)
            else:
                z.zero_distill_grad(x, index, value, MODES["tail"], st4, w, out)
            torch.cuda.synchronize()
            check(what)
            check_distill(x, index, value, MODES["tail"], 1.0, loss if fused else None, w, out, what)
    y, check = matrix(rows, vocab, dtype, stride, 3)
    y.copy_(x)
    z.zero_logprob_fused(y, tok, y, d_logprob=w, d_entropy=h, workspace=ws)
    torch.cuda.synchronize()
    check("in place")
    check_logprob_grad(x, tok, 1.0, w, h, y, "in place")
