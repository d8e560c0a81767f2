"""Gradients of policy losses averaged over targets, where the slopes before d_loss
and the mean leave binary32's range and the gradients do not; upstream gradients of
zero.  The same sequences in one launch, within and beyond the positions that a
workgroup holds, and cut into shares.

Tolerance: the gradient of a mean is rounded twice (2^-24 of its value each); where a
first rounding falls below the normal range, by 2^-150 as well, and is then multiplied by
at most 1."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
z = pytest.importorskip("fsdp_sharded_optimizer_flat_amd")
pytestmark = pytest.mark.gpu

import sequence_ref as ref64  # noqa: E402

DEV = "cuda:0"
LOW, HIGH, COEF = 0.2, 0.28, 0.05
BATCHES = {"held": [900, 1, 30], "beyond a workgroup's": [5000, 10, 10], "cut": [40000, 7, 0, 30001],
           "cut, one sequence": [20001]}


def make(seed, lengths, d_loss):
    g = np.random.default_rng(seed)
    off = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
    n = int(off[-1])
    f = lambda a: np.asarray(a, np.float32)
    old = f(-np.exp(g.normal(-1.0, 1.0, n)))
    lp = f(old + g.normal(0, 0.2, n))
    tokens = np.where(g.random(n) < 0.2, -1, 5).astype(np.int64)
    return dict(off=off, n=n, lp=lp, old=old, ref=f(lp + g.normal(0, 0.3, n)), adv=f(g.normal(0, 1, n)),
                tokens=tokens, d_loss=np.full(len(lengths), d_loss, np.float32))


def gradient(d, coef=COEF):
    on = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    b = len(d["off"]) - 1
    out = torch.full((d["n"],), 3.5, device=DEV)
    ws = torch.full((z.zero_sequence_loss_workspace_bytes(d["n"], b),), 255, dtype=torch.uint8, device=DEV)
    z.zero_policy_loss(on(d["lp"]), on(d["old"]), on(d["adv"]), on(d["off"]), tokens=on(d["tokens"]),
                       ref_logprob=on(d["ref"]), per_token=True, clip_low=LOW, clip_high=HIGH, kl_coef=coef,
                       mode=z.ZERO_SEQUENCE_MEAN, d_loss=on(d["d_loss"]), d_logprob=out, workspace=ws)
    return out.cpu().numpy().astype(np.float64)


def check(d, coef=COEF):
    got = gradient(d, coef)
    want = ref64.policy(d["lp"], d["old"], d["ref"], d["adv"], True, d["tokens"], d["off"], LOW, HIGH, coef, "mean",
                        d["d_loss"], np.zeros(d["n"]))[3]
    assert np.abs(want).max(initial=0.0) < 3e38
    assert np.isfinite(got).all(), np.nonzero(~np.isfinite(got))[0][:5]
    # slopes that are small differences of the two terms lose 2^-40 of the larger one
    tol = 2 * 2.0 ** -24 * np.abs(want) * (1 + 2.0 ** -24) + 1e-12 * np.abs(d["d_loss"]).max() * 10 + 2.0 ** -148
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.nonzero(bad)[0][:5], got[bad][:5], want[bad][:5])


def far(d, seed, least, most):
    """Targets here and there whose reference is far more probable, and whose ratio is
    large beside a negative advantage; some beside each other, some at the ends."""
    g = np.random.default_rng(seed)
    at = np.unique(np.concatenate([g.integers(0, d["n"], 12), [0, d["n"] - 1]]))
    d["tokens"][at] = 5
    for i, t in enumerate(at):
        x = np.float32(g.uniform(least, most))
        if i % 2:
            d["ref"][t] = d["lp"][t] + x
        else:
            d["lp"][t] = d["ref"][t] = d["old"][t] + x
            d["adv"][t] = -1.25
    return at


@pytest.mark.parametrize("name", BATCHES)
def test_upstream_of_zero(name):
    """One improbable target in a sequence of weight zero costs nothing."""
    for least, most in ((89.0, 95.0), (95.0, 300.0), (300.0, 700.0)):
        d = make(1, BATCHES[name], 0.0)
        far(d, 2, least, most)
        assert (gradient(d) == 0).all(), (least, most)


@pytest.mark.parametrize("name", BATCHES)
def test_slopes_beyond_the_range(name):
    """d_loss w slope is a binary32 number, slope is not (nor is d_loss slope, where
    only the mean brings it back)."""
    for least, most, d_loss in ((88.8, 95.0, 1e-6), (95.0, 160.0, 1e-37)):
        d = make(3, BATCHES[name], d_loss)
        far(d, 4, least, most)
        check(d)


@pytest.mark.parametrize("name", ["beyond a workgroup's", "cut", "cut, one sequence"])
def test_only_the_mean_brings_a_gradient_back(name):
    """e^89 and e^91 over 4000 targets and more; a prompt beside each of them stays zero."""
    d = make(5, BATCHES[name], 1.0)
    for t, x in ((100, 89.0), (4500, 91.0), (4503, 90.0)):
        d["tokens"][t - 1:t + 2] = [-1, 5, -1]
        d["lp"][t - 1], d["old"][t + 1] = np.nan, np.inf
        d["lp"][t] = d["ref"][t] = d["old"][t] + np.float32(x)
        d["adv"][t] = -1.0
    check(d)


@pytest.mark.parametrize("name", BATCHES)
def test_slopes_below_the_range(name):
    """Slopes of 10^-40 whose digits a large d_loss keeps."""
    d = make(6, BATCHES[name], 1e10)
    d["adv"] = (d["adv"] * np.float32(1e-37)).astype(np.float32) * np.float32(1e-3)
    got = gradient(d, 0.0)
    want = ref64.policy(d["lp"], d["old"], d["ref"], d["adv"], True, d["tokens"], d["off"], LOW, HIGH, 0.0, "mean",
                        d["d_loss"], np.zeros(d["n"]))[3]
    assert (np.abs(got - want) <= 2 * 2.0 ** -24 * np.abs(want) * (1 + 2.0 ** -24) + 2.0 ** -148).all()
    assert np.abs(want).max() > 1e-35


@pytest.mark.parametrize("name", BATCHES)
def test_a_sequence_is_the_same_in_any_batch(name):
    """What a slope without a binary32 value gives does not depend on the batch that its
    sequence is in: infinite where the gradient is, NaN where d_loss is."""
    for d_loss, want in ((1.0, -np.inf), (np.inf, -np.inf), (np.nan, np.nan)):
        d = make(7, BATCHES[name], d_loss)
        at = [0, d["n"] - 1]
        for t in at:
            d["tokens"][t] = 5
            d["ref"][t] = d["lp"][t] + np.float32(250.0)
        got = gradient(d)[at]
        assert np.array_equal(got, np.full(2, want), equal_nan=True), (d_loss, got)
