"""Token losses, on the GPU: gradients of rows with huge and tiny logits, rows
with a NaN under a mask, batches of which a workgroup takes several rows.
Definitions and the tolerances of ordinary rows: test_gpu_token_loss.py."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import fsdp_sharded_optimizer_flat_amd as z  # noqa: E402
from gpu_common import DEV  # noqa: E402
from test_gpu_token_loss import (DTYPES, LOWEST, MODES, SUM, U, check_distill, check_logprob,  # noqa: E402
                                 check_logprob_grad, close, gen, half_step, make_logits, make_record, matrix,
                                 ref_distill, ref_entropy, ref_logp, workspace)

INF, NAN = math.inf, math.nan


# -- large logits -----------------------------------------------------------------------------
#
# t = (l - m) c where |c m| is large: the difference, the product and c are each
# rounded once, 3 u |t|, where the usual multiply-add has 2 u |t|.  ln2 |t| is at
# most |ln p| + 14 (a sum of 2^20 terms), so p = 2^t / S carries SUM + (3 |ln p| +
# 3 * 14 + 22) u: the last 22 are the exponential, 1 / S, the coefficient's own
# products, and the statistics' rounding (14).  Beyond |ln p| = 200 p is zero in
# binary32, and is flushed to zero below 2^-126.

def p_tol(lp):
    return SUM + (3 * lp.abs().clamp(max=200.0) + 64) * U


def big_logprob_grad(x, tok, scale, dl, dh, got, what):
    lp = ref_logp(x, scale)
    p = lp.exp()
    d, e = (dl.double() * scale)[:, None], (dh.double() * scale)[:, None]
    h = ref_entropy(x, scale)[:, None]
    f = torch.where(p > 0, lp + h, 0.0)
    want = -p * d - e * p * f
    want.scatter_add_(1, tok[:, None], d)
    # the coefficients of p: d, and e (ln p + H), whose terms carry their own
    # rounding and 2 SUM (1 + H) of the entropy beside their product with p
    size = d.abs() + e.abs() * (lp.abs().clamp(max=200.0) + h + 4 * (1 + h))
    tol = half_step(x.dtype) * want.abs() * 1.01 + size * (p * p_tol(lp) + 2.0 ** -125) + 2.0 ** -133
    # the given token's: a difference of two terms, rounded once more
    tol.scatter_add_(1, tok[:, None], 2 * U * d.abs())
    close(got, want, tol, what)


def big_distill_grad(x, index, value, mode, scale, dl, got, what):
    _, grad, size, _, lp = ref_distill(x, index, value, mode, scale)
    w = (dl.double() * scale)[:, None]
    # twice p's: the tail's share and the rest's probability are two such factors
    tol = half_step(x.dtype) * (w * grad).abs() * 1.01 + w.abs() * (size * 2 * p_tol(lp) + 2.0 ** -125) + 2.0 ** -133
    close(got, w * grad, tol, what)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(8, 5003), (8, 37003), (8, 300), (3, 140001)])
def test_gradients_of_large_and_tiny_logits(rows, vocab, dtype):
    """Logits of 1e30, 1e6 and 1e-30, of the type's lowest value alone and beside
    others, scales at their limits: gradients of both losses from the backward
    calls and the fused ones, at their logits' places, at others and in place."""
    tok = torch.arange(rows, device=DEV) * 7
    dl = torch.rand(rows, generator=gen(4), device=DEV) + 0.5
    dh = torch.rand(rows, generator=gen(5), device=DEV) + 0.1
    stride = vocab + 1 + vocab % 2
    for size, scale in ((1e30, 1.0), (1e30, 2.0 ** -20), (1e6, 1.0), (1e-30, 1.0), (30.0, 2.0 ** -20),
                        (1e-4, 2.0 ** 20), (0.0, 0.7)):
        x, _ = matrix(rows, vocab, dtype, stride, 1)
        if size:
            v = torch.randn(rows, vocab, generator=gen(1), device=DEV) * size
            v[1] = -v[1].abs()
            # neighbours of a huge maximum: several tokens share the probability
            v[2, 5:40] = 4 * size
            x.copy_(v)
        else:
            x.fill_(LOWEST[dtype])          # a plateau of the lowest value
            x[1, ::2] = -INF                # half of it masked away
            x[2, 3:90] = 2.0 ** 30          # huge logits beside it
        x[0, 11] = -INF
        what = f"size {size} scale {scale}"
        ws, _ = workspace(x)
        st, h, lp = torch.empty(rows, 2, device=DEV), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        z.zero_logprob(x, tok, scale=scale, logprob=lp, entropy=h, stats=st, workspace=ws)
        index, value = make_record(x, 20, scale, 3)
        index[-1, 1] = index[-1, 0]          # named twice
        inside = torch.gather(x, 1, index.long()) > -INF
        index = torch.where(inside, index, -1)
        for where in ("same", "other", "in place"):
            for fused in (False, True):
                def target():
                    if where == "in place":
                        y, check = matrix(rows, vocab, dtype, stride, 1)
                        y.copy_(x)
                        return y, y, check
                    out, check = matrix(rows, vocab, dtype, *((stride, 1) if where == "same" else (vocab + 3, 4)))
                    return x, out, check
                y, out, check = target()
                if fused:
                    z.zero_logprob_fused(y, tok, out, scale=scale, d_logprob=dl, d_entropy=dh, workspace=ws)
                else:
                    z.zero_logprob_grad(y, tok, st, out, scale=scale, d_logprob=dl, d_entropy=dh, entropy=h)
                torch.cuda.synchronize()
                check(what)
                big_logprob_grad(x, tok, scale, dl, dh, out, f"logprob {what} {where} fused {fused}")
                for name, mode in MODES.items():
                    st4 = torch.empty(rows, 4, device=DEV)
                    y, out, check = target()
                    z.zero_distill(y, index, value, mode, scale=scale, stats=st4, workspace=ws)
                    if fused:
                        z.zero_distill_fused(y, index, value, mode, dl, out, scale=scale, workspace=ws)
                    else:
                        z.zero_distill_grad(y, index, value, mode, st4, dl, out, scale=scale)
                    torch.cuda.synchronize()
                    check(what)
                    big_distill_grad(x, index, value, mode, scale, dl, out, f"{name} {what} {where} fused {fused}")


@pytest.mark.parametrize("rows,vocab", [(8, 300), (8, 5003), (8, 37003), (300, 20011), (3, 140001)])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** 16, 2.0 ** -10])
def test_references_around_the_change_of_formula(rows, vocab, scale):
    """Logits a few nats apart whose binary logarithms c l lie around 2^20, where a
    reference beyond it takes t = (l - m) c and one below it c l - fl(c m): partial
    sums of both kinds meet in a row.  The differences of such logits are exact
    and t is as small as in ordinary rows, so their tolerances hold."""
    base = 2.0 ** 20 / (scale * math.log2(math.e))
    x = (torch.randn(rows, vocab, generator=gen(6), device=DEV, dtype=torch.float64) * 3.0 / scale)
    x[1::2] -= 2 * base                    # to - base below
    x = (x + base).float()
    tok = torch.randint(0, vocab, (rows,), generator=gen(1), device=DEV)
    dl = torch.rand(rows, generator=gen(4), device=DEV) + 0.5
    dh = torch.rand(rows, generator=gen(5), device=DEV) + 0.1
    ws, _ = workspace(x)
    f = lambda *s: torch.empty(*s, device=DEV)
    lp, h, st, st4, loss = f(rows), f(rows), f(rows, 2), f(rows, 4), f(rows)
    index, _ = make_record(x - x.mean(1, keepdim=True), 20, scale, 3)
    value = torch.log_softmax(torch.randn(rows, 20, generator=gen(8), device=DEV), 1) - 0.5
    out = torch.empty_like(x)
    z.zero_logprob(x, tok, scale=scale, logprob=lp, entropy=h, stats=st, workspace=ws)
    check_logprob(x, tok, scale, lp, h, st, "forward")
    z.zero_logprob_grad(x, tok, st, out, scale=scale, d_logprob=dl, d_entropy=dh, entropy=h)
    check_logprob_grad(x, tok, scale, dl, dh, out, "backward")
    z.zero_logprob_fused(x, tok, out, scale=scale, d_logprob=dl, d_entropy=dh, logprob=lp, entropy=h, workspace=ws)
    check_logprob(x, tok, scale, lp, h, None, "fused")
    check_logprob_grad(x, tok, scale, dl, dh, out, "fused")
    for mode in MODES.values():
        z.zero_distill(x, index, value, mode, scale=scale, loss=loss, stats=st4, workspace=ws)
        z.zero_distill_grad(x, index, value, mode, st4, dl, out, scale=scale)
        check_distill(x, index, value, mode, scale, loss, dl, out, f"mode {mode}")
        z.zero_distill_fused(x, index, value, mode, dl, out, scale=scale, loss=loss, workspace=ws)
        check_distill(x, index, value, mode, scale, loss, dl, out, f"mode {mode} fused")


# -- rows without a distribution, under a mask ---------------------------------------------------

MASKED = [(9, 3001), (300, 3001), (9, 40007), (9, 140001)]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", MASKED)
def test_nan_among_the_listed_of_a_masked_row(rows, vocab, dtype):
    """A student whose allowed tokens are all in the record, one of them NaN (kind 1)
    or +inf (2): loss and the whole gradient row are NaN, or zero at a weight of
    zero.  A row of -inf alone (5) has gradient zero; finite neighbours, masked in
    the same way (4) or not, keep theirs."""
    k = 12
    x = make_logits(rows, vocab, dtype, 77)
    index, value = make_record(x, k, 1.0, 5)
    kinds = torch.arange(rows, device=DEV) % 6
    for r in range(rows):
        if r % 6 in (1, 2, 3, 4):            # all others are masked
            keep = x[r, index[r].long()].clone()
            x[r] = -INF
            x[r, index[r].long()] = keep
    hit = index[:, 3].long()
    for kind, v in ((1, NAN), (2, INF), (3, NAN)):
        at = torch.nonzero(kinds == kind)[:, 0]
        x[at, hit[at]] = v
    x[kinds == 5] = -INF
    dl = torch.rand(rows, generator=gen(4), device=DEV) + 0.5
    dl[kinds == 3] = 0.0
    ws, _ = workspace(x)
    for mode in MODES.values():
        loss, st = torch.full((rows,), 5.0, device=DEV), torch.empty(rows, 4, device=DEV)
        z.zero_distill(x, index, value, mode, loss=loss, stats=st, workspace=ws)
        for fused in (False, True):
            out, loss2 = torch.full_like(x, 9.0), loss
            if fused:
                loss2 = torch.full((rows,), 5.0, device=DEV)
                z.zero_distill_fused(x, index, value, mode, dl, out, loss=loss2, workspace=ws)
            else:
                z.zero_distill_grad(x, index, value, mode, st, dl, out)
            torch.cuda.synchronize()
            for kind in (1, 2, 3):
                assert bool(torch.isnan(loss2[kinds == kind]).all()), (mode, fused, kind, "loss")
            for kind in (1, 2):
                assert bool(torch.isnan(out[kinds == kind]).all()), (mode, fused, kind, "gradient")
            assert bool((loss2[kinds == 5] == INF).all())
            assert bool((out[(kinds == 3) | (kinds == 5)] == 0).all())
            f = (kinds == 0) | (kinds == 4)
            if mode == MODES["tail"]:        # a rest without a token: an infinite loss, finite gradients
                f = kinds == 0
                assert bool((loss2[kinds == 4] == INF).all())
                assert bool(torch.isfinite(out[kinds == 4]).all())
            check_distill(x[f], index[f], value[f], mode, 1.0, loss2[f], dl[f], out[f], f"fused {fused}")


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", MASKED)
def test_record_without_a_finite_value(rows, vocab, dtype):
    """Values of -inf only, renormalised: no distribution, so the loss and the
    gradient are zero -- but NaN over a row that holds a NaN or +inf, listed (1) or
    not (2)."""
    x = make_logits(rows, vocab, dtype, 78)
    index, value = make_record(x, 12, 1.0, 5)
    value.fill_(-INF)
    kinds = torch.arange(rows, device=DEV) % 4
    x[kinds == 1, 0] = NAN
    index[kinds == 1, 2] = 0
    x[kinds == 2, vocab - 1] = INF
    index[kinds == 2] = torch.where(index[kinds == 2] == vocab - 1, 1, index[kinds == 2])
    x[kinds == 3] = -INF
    dl = torch.rand(rows, generator=gen(4), device=DEV) + 0.5
    ws, _ = workspace(x)
    bad = (kinds == 1) | (kinds == 2)
    for fused in (False, True):
        loss, st, out = torch.full((rows,), 5.0, device=DEV), torch.empty(rows, 4, device=DEV), torch.full_like(x, 9.0)
        if fused:
            z.zero_distill_fused(x, index, value, MODES["renorm"], dl, out, loss=loss, workspace=ws)
        else:
            z.zero_distill(x, index, value, MODES["renorm"], loss=loss, stats=st, workspace=ws)
            z.zero_distill_grad(x, index, value, MODES["renorm"], st, dl, out)
        torch.cuda.synchronize()
        assert bool(torch.isnan(loss[bad]).all()) and bool((loss[~bad] == 0).all()), fused
        assert bool(torch.isnan(out[bad]).all()) and bool((out[~bad] == 0).all()), fused


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", MASKED)
def test_entropy_gradient_alone_with_padding(rows, vocab, dtype):
    """An entropy term without one of the log probability: padding rows, marked by
    the tokens of the forward and the backward call, have none; without tokens
    every row has one."""
    x = make_logits(rows, vocab, dtype, 79)
    tok = torch.randint(0, vocab, (rows,), generator=gen(1), device=DEV)
    tok[::3] = -5
    real = tok >= 0
    dh = torch.randn(rows, generator=gen(2), device=DEV)
    ws, _ = workspace(x)
    for t, f in ((tok, real), (None, real | True)):
        y = x if t is None else x.masked_fill(~real[:, None], NAN)
        st, h, h2 = (torch.empty(rows, *s, device=DEV) for s in ((2,), (), ()))
        out, out2 = torch.full_like(x, 9.0), torch.full_like(x, 9.0)
        z.zero_logprob(y, t, entropy=h, stats=st, workspace=ws)
        z.zero_logprob_grad(y, t, st, out, d_entropy=dh, entropy=h)
        z.zero_logprob_fused(y, t, out2, d_entropy=dh, entropy=h2, workspace=ws)
        torch.cuda.synchronize()
        for g, e in ((out, h), (out2, h2)):
            check_logprob_grad(x[f], torch.zeros_like(tok)[f], 1.0, None, dh[f], g[f], f"tokens {t is not None}")
            assert bool((g[~f] == 0).all()) and bool((e[~f] == 0).all())


# -- several rows to a workgroup -------------------------------------------------------------------

def resident(threads):
    """Workgroups of fused calls that go through rows, of `threads` threads."""
    return torch.cuda.get_device_properties(DEV).multi_processor_count * (1024 // threads)


def batch(threads, vocab, dtype, seed):
    """Rows enough that each workgroup takes several, of every kind: 0 ordinary,
    1 padding (its logits NaN), 2 all -inf, 3 weight zero over NaN, 4 a bad target,
    5 a NaN, 6 huge logits.  Some workgroups have padding first, last or only."""
    grid = resident(threads)
    rows = 4 * grid + grid // 2 + 3
    r = torch.arange(rows, device=DEV)
    kinds = torch.zeros_like(r)
    draw = torch.rand(rows, generator=gen(seed), device=DEV)
    for kind in range(1, 7):
        kinds[(draw > 0.04 * kind) & (draw <= 0.04 * (kind + 1))] = kind
    own, turn = r % grid, r // grid
    kinds[own == 3] = 1                           # nothing but padding
    kinds[(own == 5) & (turn < 3)] = 1
    kinds[(own == 7) & (turn > 1)] = 1
    kinds[(own == 9)] = 0
    kinds[(own == 9) & (turn % 2 == 1)] = 1
    kinds[(own == 11)] = 6                        # one after another
    kinds[-1] = 0
    stride = vocab + 1 + vocab % 2
    x = make_logits(rows, vocab, dtype, seed, stride, 1)
    x[kinds == 1] = NAN
    x[kinds == 2] = -INF
    x[kinds == 3] = NAN
    x[kinds == 5, vocab // 2] = NAN
    x[kinds == 6] *= 1e30
    return x, kinds, stride


def blocks(rows):
    return [(a, min(a + 256, rows)) for a in range(0, rows, 256)]


def fixed_rows(out, kinds, what):
    """Gradient rows that have no distribution or no target."""
    for kind in (1, 2, 3):
        assert bool((out[kinds == kind] == 0).all()), (what, kind)
    for kind in (4, 5):
        assert bool(torch.isnan(out[kinds == kind]).all()), (what, kind)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("threads,chunks", [(64, 0), (256, 64), (512, 256), (1024, 512)])
def test_logprob_rows_of_one_workgroup(threads, chunks, dtype):
    """chunks: what the next smaller workgroup holds, in threads of 16 chunks."""
    w = 16 // (torch.finfo(dtype).bits // 8)
    vocab = max(chunks * 16 * w + 33, 131)
    x, kinds, stride = batch(threads, vocab, dtype, 40)
    rows = x.shape[0]
    print("logprob", rows, vocab, dtype, flush=True)
    tok = torch.randint(0, vocab, (rows,), generator=gen(1), device=DEV)
    tok[kinds == 1], tok[kinds == 4] = -1, vocab
    dl = torch.rand(rows, generator=gen(2), device=DEV) + 0.5
    dh = torch.rand(rows, generator=gen(3), device=DEV) * 0.1
    dl[kinds == 3], dh[kinds == 3] = 0.0, 0.0
    for e in (None, dh):
        for where in ("same", "other", "in place"):
            what = f"{where} entropy {e is not None}"
            y, check = matrix(rows, vocab, dtype, *((vocab + 3, 4) if where == "other" else (stride, 1)))
            src = x
            if where == "in place":
                y.copy_(x)
                src = y
            lp, h = torch.full((rows,), 5.0, device=DEV), torch.full((rows,), 5.0, device=DEV)
            z.zero_logprob_fused(src, tok, y, d_logprob=dl, d_entropy=e, logprob=lp, entropy=h,
                                 workspace=None)   # held rows need none
            torch.cuda.synchronize()
            check(what)
            fixed_rows(y, kinds, what)
            assert bool((lp[kinds == 1] == 0).all()) and bool((lp[kinds == 2] == -INF).all())
            for a, b in blocks(rows):
                f, g = kinds[a:b] == 0, kinds[a:b] == 6
                c = lambda t: None if t is None else t[a:b][f]
                check_logprob(c(x), c(tok), 1.0, c(lp), c(h), None, f"{what} rows {a}")
                check_logprob_grad(c(x), c(tok), 1.0, c(dl), c(e), c(y), f"{what} rows {a}")
                if bool(g.any()):
                    big_logprob_grad(x[a:b][g], tok[a:b][g], 1.0, dl[a:b][g],
                                     torch.zeros_like(dl[a:b][g]) if e is None else e[a:b][g], y[a:b][g],
                                     f"{what} huge, rows {a}")


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("threads,chunks", [(128, 0), (256, 64), (512, 192), (1024, 448)])
def test_distill_rows_of_one_workgroup(threads, chunks, dtype):
    """chunks: what the next smaller workgroup holds, in threads of 17 chunks."""
    w = 16 // (torch.finfo(dtype).bits // 8)
    vocab = max(chunks * 17 * w + 33, 131)
    x, kinds, stride = batch(threads, vocab, dtype, 50)
    rows, k = x.shape[0], 21
    print("distill", rows, vocab, dtype, flush=True)
    index, value = make_record(x, k, 1.0, 7)
    index[::5, 2] = index[::5, 1]                 # a token named twice
    index[::7, 9:] = -1                           # short records
    index[kinds == 1], index[kinds == 4, 5] = -1, vocab
    dl = torch.rand(rows, generator=gen(2), device=DEV) + 0.5
    dl[kinds == 3] = 0.0
    for name, mode in MODES.items():
        for where in ("same", "other", "in place"):
            what = f"{where} {name}"
            y, check = matrix(rows, vocab, dtype, *((vocab + 3, 4) if where == "other" else (stride, 1)))
            src = x
            if where == "in place":
                y.copy_(x)
                src = y
            loss = torch.full((rows,), 5.0, device=DEV)
            z.zero_distill_fused(src, index, value, mode, dl, y, loss=loss, workspace=None)
            torch.cuda.synchronize()
            check(what)
            fixed_rows(y, kinds, what)
            assert bool((loss[kinds == 1] == 0).all()) and bool((loss[kinds == 2] == INF).all())
            for a, b in blocks(rows):
                f, g = kinds[a:b] == 0, kinds[a:b] == 6
                c = lambda t: t[a:b][f]
                check_distill(c(x), c(index), c(value), mode, 1.0, c(loss), c(dl), c(y), f"{what} rows {a}")
                if bool(g.any()):
                    big_distill_grad(x[a:b][g], index[a:b][g], value[a:b][g], mode, 1.0, dl[a:b][g], y[a:b][g],
                                     f"{what} huge, rows {a}")
