"""The token losses on the GPU against their definitions in binary64: log
probabilities of given tokens (entropy, top alternatives, backward pass) and
distillation from a teacher's top logits, at sizes, alignments and masks where
they can go wrong.

Tolerances (u = 2^-24, half a binary32 step):
  - a logit's binary logarithm t = c l - R: c is rounded once (u |t|) and the
    fused multiply-add once (u |t|); v_exp_f32 is off by 2 u; so 2^t carries
    (2 |t| ln 2 + 2) u.  A row's sum weighs these with the probabilities: |t|
    enters as an entropy, below 20 bits (2^20 tokens), 28 u.  The additions: at
    most 8 in a group, 64 groups a lane, 16 joining steps -- 88 u; a row cut
    for several workgroups has shorter lanes and up to 16 more steps.  The
    lane's reference is moved at most a handful of times, 4 u each.  SUM = 160 u
    covers them.
  - ln p = ln2 (t - log2 S): (2 |ln p| + 2) u from t and the products, SUM from
    S, and log2 S itself (at most 20 in size) 20 u.
  - results: a bf16 gradient is rounded once more, 2^-8 relative
    (half of finfo.eps); binary32 results, u.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import fsdp_sharded_optimizer_flat_amd as z  # noqa: E402
from gpu_common import DEV  # noqa: E402

U = 2.0 ** -24
SUM = 160 * U
INF, NAN = math.inf, math.nan
LOWEST = {torch.bfloat16: torch.finfo(torch.bfloat16).min, torch.float32: torch.finfo(torch.float32).min}
MODES = {"renorm": z.ZERO_DISTILL_RENORM, "tail": z.ZERO_DISTILL_TAIL}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def matrix(rows, vocab, dtype, stride=None, shift=0, fill=-77.0):
    """(rows, vocab) view `shift` elements into an allocation of rows of `stride`
    elements, and a check that nothing outside the view changed."""
    stride = vocab if stride is None else stride
    base = torch.full((shift + rows * stride + 64,), fill, dtype=dtype, device=DEV)
    view = base[shift:shift + rows * stride].view(rows, stride)[:, :vocab]

    def check(what=""):
        left = base.clone()
        left[shift:shift + rows * stride].view(rows, stride)[:, :vocab] = fill
        assert bool((left == fill).all()), f"{what}: written outside the rows"
    return view, check


def make_logits(rows, vocab, dtype, seed, stride=None, shift=0):
    x, _ = matrix(rows, vocab, dtype, stride, shift)
    g = gen(seed)
    for a in range(0, rows, 256):
        b = min(a + 256, rows)
        v = torch.randn(b - a, vocab, generator=g, device=DEV) * 2.5 - 4.0
        v[:, :1] += 9.0
        x[a:b] = v
    return x


def workspace(x, k=0, guard=256):
    n = z.zero_loss_workspace_bytes(x.shape[0], x.shape[1], k)
    w = torch.full((n + guard,), 0x5A, dtype=torch.uint8, device=DEV)

    def check():
        assert bool((w[n:] == 0x5A).all()), "written past the workspace"
    return w[:n] if n else None, check


def close(got, want, tol, what):
    """|got - want| <= tol elementwise, infinities equal, NaN at the same places."""
    g, w = got.double(), want.double()
    assert g.shape == w.shape, what
    assert torch.equal(torch.isnan(g), torch.isnan(w)), f"{what}: NaN places differ"
    same = (g == w) | torch.isnan(w)
    off = torch.where(same, 0.0, (g - w).abs() - tol)
    off = torch.nan_to_num(off, nan=INF)
    bad = off > 0
    if bool(bad.any()):
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} values off, first at {i}: "
                             f"{g[tuple(i)].item()!r} for {w[tuple(i)].item()!r}")


# -- definitions in binary64 -------------------------------------------------------

def ref_logp(x, scale):
    y = x.double() * scale
    m = y.amax(1, keepdim=True)
    return (y - m) - torch.exp(y - m).sum(1, keepdim=True).log()


def xlogx(p, lp):
    return torch.where(p > 0, p * lp, 0.0)


def ref_entropy(x, scale):
    lp = ref_logp(x, scale)
    return -xlogx(lp.exp(), lp).sum(1)


def logp_tol(lp):
    return SUM + (22 + 2 * torch.nan_to_num(lp.abs(), nan=0.0, posinf=0.0)) * U


def check_logprob(x, tokens, scale, logprob, entropy, stats, what):
    """Rows with finite maxima and given tokens inside the vocabulary."""
    lp = ref_logp(x, scale)
    want = lp.gather(1, tokens[:, None])[:, 0]
    close(logprob, want, logp_tol(want), what + " logprob")
    if entropy is not None:
        h = ref_entropy(x, scale)
        # ln2 (log2 S - A / S): A's terms e t carry e's error and their own
        # product, so A / S (an entropy) SUM, twice
        close(entropy, h, 2 * SUM * (1 + h) + 22 * U, what + " entropy")
    if stats is not None:
        m = x.double().amax(1)
        assert torch.equal(stats[:, 0].double(), m), what + " stats max"
        ln = torch.exp((x.double() - m[:, None]) * scale).sum(1).log()
        close(stats[:, 1], ln, SUM + 22 * U, what + " stats ln")


def ref_top(x, k):
    """Indices of the k largest logits, ties to the lowest index (-1: -inf)."""
    v, i = torch.sort(x.float(), dim=1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k]
    i = torch.where(v == -INF, -1, i)
    if i.shape[1] < k:
        i = torch.nn.functional.pad(i, (0, k - i.shape[1]), value=-1)
    return i.to(torch.int32)


def check_top(x, scale, k, index, logprob, what):
    want = ref_top(x, k)
    assert torch.equal(index, want), f"{what}: top indices differ in rows " \
        f"{torch.nonzero((index != want).any(1))[:4, 0].tolist()}"
    lp = torch.where(want >= 0, ref_logp(x, scale).gather(1, want.long().clamp(min=0)), -INF)
    close(logprob, lp, logp_tol(lp), what + " top logprob")


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def grad_tol(p, lp, size, dtype, want):
    """A gradient element of terms p * size: p carries SUM and (2 |ln p| + 24) u
    (t, the statistics' rounding -- at most 20 in size -- and the products)."""
    rel = SUM + (2 * torch.nan_to_num(lp.abs(), posinf=0.0, nan=0.0) + 48) * U
    # p below binary32's normal range is flushed to zero
    return half_step(dtype) * want.abs() * 1.01 + size.abs() * (p * rel + 2.0 ** -125) + 2.0 ** -133


def check_logprob_grad(x, tokens, scale, dl, dh, got, what):
    lp = ref_logp(x, scale)
    p = lp.exp()
    n = x.shape[0]
    zero = torch.zeros(n, 1, device=DEV, dtype=torch.float64)
    d = zero if dl is None else dl.double()[:, None]
    want = -p * d * scale
    size = (d * scale).abs() + 0 * p
    if dl is not None:
        want.scatter_add_(1, tokens[:, None], d * scale)
        # the one-hot element's difference is rounded once more
        size = size.scatter_add(1, tokens[:, None], (d * scale).abs() / (1e-30 + p.gather(1, tokens[:, None])) * U
                                / (SUM + 48 * U))
    if dh is not None:
        e = dh.double()[:, None]
        h = ref_entropy(x, scale)[:, None]
        f = torch.where(p > 0, lp + h, 0.0)
        want = want - e * scale * p * f
        # ln p and H each carry 2 SUM (1 + H) beside their product with p
        size = size + (e * scale).abs() * (torch.nan_to_num(lp.abs(), posinf=0.0) + h + 4 * (1 + h))
    close(got, want, grad_tol(p, lp, size, x.dtype, want), what + " d_logits")


def ref_distill(x, index, value, mode, scale):
    """(loss, d loss / d logits * 1/scale..., pieces for the tolerances)."""
    lp = ref_logp(x, scale)
    p = lp.exp()
    valid = index >= 0
    at = index.long().clamp(min=0)
    val = torch.where(valid, value.double(), -INF)
    if mode == MODES["renorm"]:
        q = torch.softmax(val, 1)
        log_q = torch.log_softmax(val, 1)
        rest = torch.zeros(x.shape[0], 1, dtype=torch.float64, device=DEV)
    else:
        q, log_q = val.exp(), val
        rest = 1.0 - q.sum(1, keepdim=True)
        rest = torch.where(rest < 2.0 ** -20, 0.0, rest)
    seen = torch.zeros_like(lp).scatter_add(1, at, valid.double()) > 0
    rest = torch.where(seen.all(1, keepdim=True), 0.0, rest)
    total = q.sum(1, keepdim=True) + rest
    log_rest = torch.logsumexp(lp.masked_fill(seen, -INF), 1, keepdim=True)
    lpk = lp.gather(1, at)
    loss = torch.where(q > 0, q * (log_q - lpk), 0.0).sum(1, keepdim=True)
    loss = loss + torch.where(rest > 0, rest * (rest.log() - log_rest), 0.0)
    full_q = torch.zeros_like(lp).scatter_add(1, at, torch.where(valid, q, 0.0))
    within = torch.where(seen, 0.0, torch.exp(lp - log_rest)).nan_to_num(nan=0.0)
    grad = total * p - full_q - rest * within
    terms = torch.where(q > 0, q * (lpk.abs() + log_q.abs()), 0.0).sum(1) + \
        torch.where(rest > 0, rest * (log_rest.abs() + rest.log().abs()), 0.0)[:, 0]
    size = total * p + full_q + rest * within
    return loss[:, 0], grad, size, terms.nan_to_num(nan=0.0, posinf=0.0), lp


def check_distill(x, index, value, mode, scale, loss, d_loss, d_logits, what):
    want, grad, size, terms, lp = ref_distill(x, index, value, mode, scale)
    if loss is not None:
        # ln p of the entries and of the rest: SUM each (weights add up to
        # one), the parts' joining in binary64, the result rounded once
        close(loss, want, 2 * SUM + (48 + 4 * terms) * U, what + " loss")
    if d_logits is not None:
        w = (d_loss.double() * scale)[:, None]
        g = grad * w
        rel = 2 * SUM + (4 * torch.nan_to_num(lp.abs(), posinf=0.0) + 96) * U
        tol = half_step(x.dtype) * g.abs() * 1.01 + (w * size).abs() * rel + w.abs() * 2.0 ** -125 + 2.0 ** -133
        close(d_logits, g, tol, what + " d_logits")


def make_record(x, k, scale, seed, noise=1.0):
    """A teacher's top-k record: log probabilities of logits near x."""
    rows, vocab = x.shape
    k_have = min(k, vocab)
    index = torch.full((rows, k), -1, dtype=torch.int32, device=DEV)
    value = torch.zeros(rows, k, device=DEV)
    g = gen(seed)
    for a in range(0, rows, 256):
        b = min(a + 256, rows)
        y = x[a:b].float()
        y = torch.nan_to_num(y, nan=0.0, posinf=50.0, neginf=-1e4).clamp(-1e4, 1e4)
        y = torch.log_softmax((y + noise * torch.randn(y.shape, generator=g, device=DEV)).double() * scale, 1)
        v, i = torch.topk(y, k_have, dim=1)
        index[a:b, :k_have], value[a:b, :k_have] = i.to(torch.int32), v.float()
    return index, value


def run_logprob(x, tokens, scale, k=0, entropy=True):
    n = x.shape[0]
    out = {"logprob": torch.full((n,), 5.0, device=DEV),
           "entropy": torch.full((n,), 5.0, device=DEV) if entropy else None,
           "stats": torch.full((n, 2), 5.0, device=DEV)}
    if k:
        out["top_index"] = torch.full((n, k), -9, dtype=torch.int32, device=DEV)
        out["top_logprob"] = torch.full((n, k), 5.0, device=DEV)
    ws, check = workspace(x, k)
    z.zero_logprob(x, tokens, scale=scale, workspace=ws, **out)
    torch.cuda.synchronize()
    check()
    return out


# -- ordinary rows at many sizes -------------------------------------------------------

# rows, vocab, row stride, elements into the allocation
SIZES = [(1, 1, 1, 0), (2, 2, 5, 1), (3, 7, 7, 0), (5, 8, 8, 1), (4, 9, 9, 0), (6, 63, 64, 3),
         (1, 4099, 4099, 0), (2, 70001, 70001, 1), (7, 1023, 1040, 2), (300, 2049, 2049, 0), (1100, 130, 130, 1),
         (1030, 5003, 5003, 0), (1, 50304, 50304, 0), (3, 50257, 50257, 5), (2, 131073, 131073, 0),
         (1025, 16500, 16512, 0), (1, 1 << 20, 1 << 20, 0), (2, (1 << 20) - 3, (1 << 20) - 3, 1)]
DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,stride,shift", SIZES)
def test_logprob_sizes(rows, vocab, stride, shift, dtype):
    scale = [1.0, 0.7, 2.0][vocab % 3]
    x = make_logits(rows, vocab, dtype, 1000 + vocab, stride, shift)
    tokens = torch.randint(0, vocab, (rows,), generator=gen(1), device=DEV)
    tokens[-1] = vocab - 1
    tokens[0] = 0
    for k in (0, 1, 5, 64, 256):
        o = run_logprob(x, tokens, scale, k)
        check_logprob(x, tokens, scale, o["logprob"], o["entropy"], o["stats"], f"k={k}")
        if k:
            check_top(x, scale, k, o["top_index"], o["top_logprob"], f"k={k}")
    o = run_logprob(x, tokens, scale, 0, entropy=False)
    check_logprob(x, tokens, scale, o["logprob"], None, o["stats"], "no entropy")


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,stride,shift", SIZES)
def test_logprob_gradients(rows, vocab, stride, shift, dtype):
    scale = [1.0, 0.7, 2.0][vocab % 3]
    x = make_logits(rows, vocab, dtype, 2000 + vocab, stride, shift)
    g = gen(3)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    tokens[-1], tokens[0] = vocab - 1, 0
    dl = torch.randn(rows, generator=g, device=DEV)
    dh = torch.randn(rows, generator=g, device=DEV) * 0.1
    fwd = run_logprob(x, tokens, scale)
    for d, e in ((dl, None), (dl, dh), (None, dh)):
        for out_stride, out_shift in ((stride, shift), (vocab + 3, shift + 1)):
            out, check = matrix(rows, vocab, dtype, out_stride, out_shift)
            z.zero_logprob_grad(x, tokens, fwd["stats"], out, scale=scale, d_logprob=d, d_entropy=e,
                                entropy=fwd["entropy"] if e is not None else None)
            torch.cuda.synchronize()
            check("backward")
            check_logprob_grad(x, tokens, scale, d, e, out, "backward")
            out, check = matrix(rows, vocab, dtype, out_stride, out_shift)
            ws, wcheck = workspace(x)
            lp, h = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
            z.zero_logprob_fused(x, tokens, out, scale=scale, d_logprob=d, d_entropy=e, logprob=lp,
                                 entropy=h if e is not None else None, workspace=ws)
            torch.cuda.synchronize()
            check("fused")
            wcheck()
            check_logprob_grad(x, tokens, scale, d, e, out, "fused")
            check_logprob(x, tokens, scale, lp, h if e is not None else None, None, "fused")
    # in place, padding columns left alone
    y, check = matrix(rows, vocab, dtype, stride, shift)
    y.copy_(x)
    z.zero_logprob_fused(y, tokens, y, scale=scale, d_logprob=dl, workspace=workspace(x)[0])
    torch.cuda.synchronize()
    check("in place")
    check_logprob_grad(x, tokens, scale, dl, None, y, "in place")


@pytest.mark.parametrize("mode", sorted(MODES))
@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,stride,shift", SIZES)
def test_distill_sizes(rows, vocab, stride, shift, dtype, mode):
    scale = [1.0, 0.7, 2.0][vocab % 3]
    mode = MODES[mode]
    x = make_logits(rows, vocab, dtype, 3000 + vocab, stride, shift)
    dl = torch.randn(rows, generator=gen(5), device=DEV)
    for k in (1, 8, 100, 256):
        index, value = make_record(x, k, scale, 7)
        ws, wcheck = workspace(x)
        loss, stats = torch.empty(rows, device=DEV), torch.empty(rows, 4, device=DEV)
        z.zero_distill(x, index, value, mode, scale=scale, loss=loss, stats=stats, workspace=ws)
        torch.cuda.synchronize()
        wcheck()
        check_distill(x, index, value, mode, scale, loss, None, None, f"k={k}")
        for out_stride, out_shift in ((stride, shift), (vocab + 3, shift + 1)):
            out, check = matrix(rows, vocab, dtype, out_stride, out_shift)
            z.zero_distill_grad(x, index, value, mode, stats, dl, out, scale=scale)
            torch.cuda.synchronize()
            check("backward")
            check_distill(x, index, value, mode, scale, None, dl, out, f"backward k={k}")
            out, check = matrix(rows, vocab, dtype, out_stride, out_shift)
            loss2 = torch.empty(rows, device=DEV)
            z.zero_distill_fused(x, index, value, mode, dl, out, scale=scale, loss=loss2, workspace=ws)
            torch.cuda.synchronize()
            check("fused")
            wcheck()
            check_distill(x, index, value, mode, scale, loss2, dl, out, f"fused k={k}")
    y, check = matrix(rows, vocab, dtype, stride, shift)
    y.copy_(x)
    z.zero_distill_fused(y, index, value, mode, dl, y, scale=scale, workspace=ws)
    torch.cuda.synchronize()
    check("in place")
    check_distill(x, index, value, mode, scale, None, dl, y, "in place")


# -- rows that can go wrong ---------------------------------------------------------------

# (rows, vocab): a small and a large workgroup per row, and rows cut for several
WIDTHS = [(1100, 3001), (9, 40007), (9, 80021)]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", WIDTHS)
def test_top_of_plateaus(rows, vocab, dtype):
    """Ties go to the lowest index: constant rows, rows of few values, rows that
    rise and fall, and rows whose largest logits are neighbours."""
    g = gen(11)
    ramp = torch.arange(vocab, device=DEV, dtype=torch.float32)
    kinds = [torch.zeros(vocab, device=DEV), torch.full((vocab,), LOWEST[dtype], device=DEV),
             torch.randint(0, 3, (vocab,), generator=g, device=DEV).float(), ramp / 64, -ramp / 64,
             torch.where(ramp < 2000, 5.0 + ramp / 512, 0.0), torch.where(ramp % 7 == 0, -0.0, 0.0),
             torch.where(ramp >= vocab - 300, 3.0, -3.0)]
    x, _ = matrix(rows, vocab, dtype)
    for r in range(rows):
        x[r] = kinds[r % len(kinds)]
    x = x[:max(9, len(kinds))] if rows < 100 else x
    tokens = torch.zeros(x.shape[0], dtype=torch.int64, device=DEV)
    for k in (1, 20, 256):
        o = run_logprob(x, tokens, 1.0, k)
        check_top(x, 1.0, k, o["top_index"], o["top_logprob"], f"k={k}")
        check_logprob(x, tokens, 1.0, o["logprob"], o["entropy"], o["stats"], f"k={k}")


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", WIDTHS)
def test_masked_logits(rows, vocab, dtype):
    """-inf and the type's lowest value in masked places: at the front, almost
    everywhere, everywhere but one token; tokens on masked places."""
    x = make_logits(rows, vocab, dtype, 21)
    for r in range(rows):
        fill = -INF if r % 2 else LOWEST[dtype]
        kind = (r // 2) % 4
        if kind == 0:
            x[r, :vocab // 2] = fill
        elif kind == 1:
            keep = x[r, 100:110].clone()
            x[r] = fill
            x[r, 100:110] = keep
        elif kind == 2:
            x[r] = fill
            x[r, vocab - 1] = 3.0
        else:
            x[r, ::2] = fill
    tokens = torch.full((rows,), vocab - 1, dtype=torch.int64, device=DEV)
    tokens[::3] = 0
    o = run_logprob(x, tokens, 1.0, 20)
    check_logprob(x, tokens, 1.0, o["logprob"], o["entropy"], o["stats"], "masked")
    check_top(x, 1.0, 20, o["top_index"], o["top_logprob"], "masked")
    dl = torch.randn(rows, generator=gen(2), device=DEV)
    dh = torch.randn(rows, generator=gen(3), device=DEV)
    out = torch.empty_like(x)
    z.zero_logprob_grad(x, tokens, o["stats"], out, d_logprob=dl, d_entropy=dh, entropy=o["entropy"])
    check_logprob_grad(x, tokens, 1.0, dl, dh, out, "masked")
    # a teacher under the same mask: its record names allowed tokens only
    index, value = make_record(x, 8, 1.0, 5)
    allowed = x.gather(1, index.long()) > LOWEST[dtype]
    index = torch.where(allowed, index, -1)
    for mode in MODES.values():
        loss, out = torch.empty(rows, device=DEV), torch.empty_like(x)
        z.zero_distill_fused(x, index, value, mode, dl, out, loss=loss, workspace=workspace(x)[0])
        check_distill(x, index, value, mode, 1.0, loss, dl, out, "masked distill")


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", WIDTHS)
def test_rows_without_a_distribution(rows, vocab, dtype):
    """All -inf, NaN, +inf, padding rows (whatever they hold), tokens and indices
    past the vocabulary, weights of zero: each row's own result, its
    neighbours' untouched."""
    x = make_logits(rows, vocab, dtype, 31)
    tokens = torch.randint(0, vocab, (rows,), generator=gen(1), device=DEV)
    kinds = torch.arange(rows, device=DEV) % 9
    x[kinds == 1] = -INF
    x[kinds == 2, vocab // 3] = NAN
    x[kinds == 3, vocab - 1] = INF
    x[kinds == 4] = NAN
    tokens[kinds == 4] = -1                 # padding: its NaN are never read
    tokens[kinds == 5] = vocab              # outside
    tokens[kinds == 6] = 1 << 40
    x[kinds == 7] = NAN                     # weight zero below
    nan = torch.full((rows,), NAN, device=DEV)
    fine = (kinds == 0) | (kinds == 8)
    k = 20
    o = run_logprob(x, tokens, 1.0, k)
    check_logprob(x[fine], tokens[fine], 1.0, o["logprob"][fine], o["entropy"][fine],
                  o["stats"][fine], "neighbours")
    check_top(x[fine], 1.0, k, o["top_index"][fine], o["top_logprob"][fine], "neighbours")

    def rows_are(kind, name, value):
        got = o[name][kinds == kind]
        want = torch.full_like(got, value)
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and \
            bool((got[~torch.isnan(got)] == want[~torch.isnan(want)]).all()), (kind, name, got[:2])
    for kind, lp, ent, idx, top in ((1, -INF, 0.0, -1, -INF), (2, NAN, NAN, -1, NAN), (3, NAN, NAN, -1, NAN),
                                    (4, 0.0, 0.0, -1, -INF), (7, NAN, NAN, -1, NAN)):
        rows_are(kind, "logprob", lp)
        rows_are(kind, "entropy", ent)
        rows_are(kind, "top_index", idx)
        rows_are(kind, "top_logprob", top)
    rows_are(5, "logprob", NAN)
    rows_are(6, "logprob", NAN)
    rows_are(1, "stats", -INF)
    rows_are(4, "stats", 0.0)
    dl = torch.where(kinds == 7, 0.0, 1.5)
    dh = torch.where(kinds == 7, 0.0, 0.25)
    for fused in (False, True):
        out = torch.full_like(x, 9.0)
        if fused:
            z.zero_logprob_fused(x, tokens, out, d_logprob=dl, d_entropy=dh, workspace=workspace(x)[0])
        else:
            z.zero_logprob_grad(x, tokens, o["stats"], out, d_logprob=dl, d_entropy=dh,
                                entropy=o["entropy"])
        check_logprob_grad(x[fine], tokens[fine], 1.0, dl[fine], dh[fine], out[fine], "neighbours")
        for kind in (1, 4, 7):
            assert bool((out[kinds == kind] == 0).all()), kind
        for kind in (2, 3, 5, 6):
            assert bool(torch.isnan(out[kinds == kind]).all()), kind
    # distillation
    x[kinds == 5] = x[kinds == 0][:1]
    x[kinds == 6] = x[kinds == 0][:1]
    index, value = make_record(x, k, 1.0, 5)
    index[kinds == 4] = -3                  # padding
    index[kinds == 5, 3] = vocab
    value[kinds == 6, 7] = NAN
    index[kinds == 8, 5:] = -1              # a short record
    for mode in MODES.values():
        loss, stats = nan.clone(), torch.empty(rows, 4, device=DEV)
        z.zero_distill(x, index, value, mode, loss=loss, stats=stats, workspace=workspace(x)[0])
        check_distill(x[fine], index[fine], value[fine], mode, 1.0, loss[fine], None, None, "neighbours")
        assert bool((loss[kinds == 1] == INF).all()) and bool((loss[kinds == 4] == 0).all())
        for kind in (2, 3, 5, 6, 7):
            assert bool(torch.isnan(loss[kinds == kind]).all()), kind
        for fused in (False, True):
            out = torch.full_like(x, 9.0)
            if fused:
                z.zero_distill_fused(x, index, value, mode, dl, out, workspace=workspace(x)[0])
            else:
                z.zero_distill_grad(x, index, value, mode, stats, dl, out)
            check_distill(x[fine], index[fine], value[fine], mode, 1.0, None, dl[fine], out[fine], "n")
            for kind in (1, 4, 7):
                assert bool((out[kinds == kind] == 0).all()), (kind, fused)
            for kind in (2, 3, 5, 6):
                assert bool(torch.isnan(out[kinds == kind]).all()), (kind, fused)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(1100, 500), (9, 40007), (4, 3)])
def test_distill_records(rows, vocab, dtype):
    """Entries that name a token twice, a record of the whole vocabulary, a
    student that is sure of a listed token (the rest's probability far below
    binary32's), a teacher sure of one token, values of -inf."""
    x = make_logits(rows, vocab, dtype, 41)
    k = min(200, vocab)
    index, value = make_record(x, k, 1.0, 5)
    kinds = torch.arange(rows, device=DEV) % 4
    x[kinds == 0] = x[kinds == 0].float().index_fill(1, torch.tensor([0], device=DEV), 300.0).to(dtype)
    index[kinds == 1, 1] = index[kinds == 1, 0]           # the same token twice
    value[kinds == 2] = -INF
    value[kinds == 2, 0] = 0.0
    dl = torch.rand(rows, generator=gen(9), device=DEV) + 0.5
    for mode in MODES.values():
        loss, out = torch.empty(rows, device=DEV), torch.empty_like(x)
        z.zero_distill_fused(x, index, value, mode, dl, out, loss=loss, workspace=workspace(x)[0])
        check_distill(x, index, value, mode, 1.0, loss, dl, out, f"mode {mode}")
    # no finite value at all: no distribution, nothing to learn
    value.fill_(-INF)
    z.zero_distill_fused(x, index, value, MODES["renorm"], dl, out, loss=loss, workspace=workspace(x)[0])
    assert bool((loss == 0).all()) and bool((out == 0).all())


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_large_and_tiny_logits(dtype):
    """Logits of 1e30 and of 1e-30, negative rows, scales at their limits."""
    rows, vocab = 8, 5000
    tokens = torch.arange(rows, device=DEV) * 7
    for size, scale in ((1e30, 1.0), (1e30, 2.0 ** -20), (1e-30, 1.0), (30.0, 2.0 ** -20),
                        (1e-4, 2.0 ** 20), (2e4, 1.0)):
        x = (torch.randn(rows, vocab, generator=gen(1), device=DEV) * size).to(dtype)
        x[1] = -x[1].abs()
        o = run_logprob(x, tokens, scale, 5)
        lp = ref_logp(x, scale)
        # t's relative error counts here: t runs to millions and beyond
        want = lp.gather(1, tokens[:, None])[:, 0]
        close(o["logprob"], want.float().double(), logp_tol(want), f"size {size} scale {scale}")
        assert torch.equal(o["top_index"], ref_top(x, 5))
        assert torch.equal(o["stats"][:, 0].double(), x.double().amax(1))


# -- gradients against differences -----------------------------------------------------------

def test_gradients_against_differences():
    """Central differences of the binary64 definition along random directions:
    the step's error is h^2/6 times third derivatives (below 4 scale^3 per unit
    direction), 1e-4^2; the kernel's binary32 gradient is off by 1e-5 of its
    size."""
    rows, vocab, k, scale = 6, 700, 16, 0.9
    x = make_logits(rows, vocab, torch.float32, 51)
    tokens = torch.arange(rows, device=DEV) * 100
    index, value = make_record(x, k, scale, 3)
    dl = torch.rand(rows, generator=gen(4), device=DEV) + 0.5
    dh = torch.rand(rows, generator=gen(5), device=DEV)
    ws = workspace(x)[0]
    h = 1e-4

    def objective(y, what):
        if what == "logprob":
            return (dl.double() * ref_logp(y, scale).gather(1, tokens[:, None])[:, 0]).sum() + \
                (dh.double() * ref_entropy(y, scale)).sum()
        return (dl.double() * ref_distill(y, index, value, MODES[what], scale)[0]).sum()

    for what in ("logprob", "renorm", "tail"):
        g = torch.empty_like(x)
        if what == "logprob":
            z.zero_logprob_fused(x, tokens, g, scale=scale, d_logprob=dl, d_entropy=dh, workspace=ws)
        else:
            z.zero_distill_fused(x, index, value, MODES[what], dl, g, scale=scale, workspace=ws)
        for s in range(4):
            d = torch.randn(rows, vocab, generator=gen(60 + s), device=DEV, dtype=torch.float64)
            d[:, :1] *= 10
            diff = (objective(x.double() + h * d, what) - objective(x.double() - h * d, what)) / (2 * h)
            got = (g.double() * d).sum()
            assert abs(float(diff - got)) <= 1e-4 * float((g.double() * d).abs().sum()) + 1e-4, (what, s)


# -- the calls together and around them --------------------------------------------------------

def test_same_bits_again_and_on_another_stream():
    x = make_logits(40, 30011, torch.bfloat16, 61)
    tokens = torch.randint(0, 30011, (40,), generator=gen(1), device=DEV)
    index, value = make_record(x, 50, 1.0, 3)
    dl = torch.rand(40, generator=gen(2), device=DEV)
    side = torch.cuda.Stream()

    def once(stream):
        o = {n: torch.empty(40, device=DEV) for n in ("logprob", "entropy", "loss")}
        o["i"], o["t"] = torch.empty(40, 20, dtype=torch.int32, device=DEV), torch.empty(40, 20, device=DEV)
        o["g"], o["h"] = torch.empty_like(x), torch.empty_like(x)
        ws = workspace(x, 20)[0]
        torch.cuda.synchronize()
        z.zero_logprob(x, tokens, logprob=o["logprob"], entropy=o["entropy"], top_index=o["i"],
                       top_logprob=o["t"], workspace=ws, stream=stream)
        z.zero_logprob_fused(x, tokens, o["g"], d_logprob=dl, workspace=ws, stream=stream)
        z.zero_distill_fused(x, index, value, MODES["tail"], dl, o["h"], loss=o["loss"], workspace=ws,
                             stream=stream)
        torch.cuda.synchronize()
        return o
    a = once(None)
    for stream in (None, side, side):
        b = once(stream)
        for n in a:
            assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)), n


def test_captured_graph():
    """All six calls in one graph, replayed on new inputs with eager work between
    the replays: each replay equals the eager calls."""
    rows, vocab, k = 70, 20021, 40
    x = make_logits(rows, vocab, torch.bfloat16, 71)
    tokens = torch.randint(0, vocab, (rows,), generator=gen(1), device=DEV)
    index, value = make_record(x, k, 1.0, 3)
    dl = torch.rand(rows, generator=gen(2), device=DEV)
    ws = workspace(x, k)[0]
    f = lambda *s: torch.zeros(*s, device=DEV)
    o = {"lp": f(rows), "h": f(rows), "st": f(rows, 2), "i": torch.zeros(rows, k, dtype=torch.int32, device=DEV),
         "t": f(rows, k), "loss": f(rows), "st4": f(rows, 4), "g1": torch.zeros_like(x), "g2": torch.zeros_like(x),
         "g3": torch.zeros_like(x), "g4": torch.zeros_like(x), "lp2": f(rows), "loss2": f(rows)}

    def calls(stream=None):
        z.zero_logprob(x, tokens, logprob=o["lp"], entropy=o["h"], stats=o["st"], top_index=o["i"],
                       top_logprob=o["t"], workspace=ws, stream=stream)
        z.zero_logprob_grad(x, tokens, o["st"], o["g1"], d_logprob=dl, d_entropy=dl, entropy=o["h"],
                            stream=stream)
        z.zero_logprob_fused(x, tokens, o["g2"], d_logprob=dl, logprob=o["lp2"], workspace=ws, stream=stream)
        z.zero_distill(x, index, value, MODES["tail"], loss=o["loss"], stats=o["st4"], workspace=ws,
                       stream=stream)
        z.zero_distill_grad(x, index, value, MODES["tail"], o["st4"], dl, o["g3"], stream=stream)
        z.zero_distill_fused(x, index, value, MODES["renorm"], dl, o["g4"], loss=o["loss2"], workspace=ws,
                             stream=stream)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        calls()
    for step in range(4):
        x.copy_(make_logits(rows, vocab, torch.bfloat16, 80 + step))
        tokens.copy_(torch.randint(0, vocab, (rows,), generator=gen(90 + step), device=DEV))
        calls()
        torch.cuda.synchronize()
        want = {n: t.clone() for n, t in o.items()}
        for t in o.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n in o:
            assert torch.equal(o[n].view(torch.uint8), want[n].view(torch.uint8)), (step, n)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_rows_past_32_bit_offsets(dtype):
    """Rows of a wide buffer: the last ones start past 2^32 elements."""
    rows, vocab, stride = 1030, 700, (1 << 22) + 9
    base = torch.empty(rows * stride, dtype=dtype, device=DEV)
    x = base.view(rows, stride)[:, :vocab]
    x.copy_(make_logits(rows, vocab, dtype, 5))
    tokens = torch.randint(0, vocab, (rows,), generator=gen(1), device=DEV)
    o = run_logprob(x, tokens, 1.0, 5)
    check_logprob(x, tokens, 1.0, o["logprob"], o["entropy"], o["stats"], "wide")
    check_top(x, 1.0, 5, o["top_index"], o["top_logprob"], "wide")
    dl = torch.rand(rows, generator=gen(2), device=DEV)
    index, value = make_record(x, 20, 1.0, 3)
    keep = x.clone()
    z.zero_logprob_fused(x, tokens, x, d_logprob=dl, workspace=workspace(keep)[0])
    check_logprob_grad(keep, tokens, 1.0, dl, None, x, "wide")
    x.copy_(keep)
    z.zero_distill_fused(x, index, value, MODES["tail"], dl, x, workspace=workspace(keep)[0])
    check_distill(keep, index, value, MODES["tail"], 1.0, None, dl, x, "wide")
    del base, x
    torch.cuda.empty_cache()


def test_binding_refuses_mismatched_tensors():
    x = make_logits(4, 100, torch.bfloat16, 1)
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    f = torch.zeros(4, device=DEV)
    i, v = torch.zeros(4, 5, dtype=torch.int32, device=DEV), torch.zeros(4, 5, device=DEV)
    g = torch.zeros(4, 100, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(4, 4, device=DEV)
    bad = [
        lambda: z.zero_logprob(x.half(), t, logprob=f),
        lambda: z.zero_logprob(x.t(), t, logprob=f),
        lambda: z.zero_logprob(x, t.int(), logprob=f),
        lambda: z.zero_logprob(x, t[:3], logprob=f),
        lambda: z.zero_logprob(x, t, logprob=f[:3]),
        lambda: z.zero_logprob(x, t, logprob=f.double()),
        lambda: z.zero_logprob(x, t, top_index=i),
        lambda: z.zero_logprob(x, t, top_index=i, top_logprob=v[:, :4]),
        lambda: z.zero_logprob(x, t, top_index=i.long(), top_logprob=v),
        lambda: z.zero_logprob(x, t.cpu(), logprob=f),
        lambda: z.zero_logprob_fused(x, t, g.float(), d_logprob=f),
        lambda: z.zero_logprob_fused(x, t, g[:, :99], d_logprob=f),
        lambda: z.zero_logprob_grad(x, t, f, g, d_logprob=f),
        lambda: z.zero_distill(x, i[:3], v[:3], 0, loss=f),
        lambda: z.zero_distill_grad(x, i, v, 0, st[:, :2], f, g),
        lambda: z.zero_logprob(make_logits(1, 70001, torch.bfloat16, 1), t[:1], logprob=f[:1],
                               workspace=torch.zeros(8, dtype=torch.uint8, device=DEV)),
    ]
    for n, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError, z.ZeroError)):
            call()
            raise AssertionError(f"call {n} was not refused")
    with pytest.raises(z.ZeroError) as e:
        z.zero_distill(x, i, v, 0, loss=st.view(-1)[:4], stats=st)
    assert e.value.status == z.ZERO_EINVAL
