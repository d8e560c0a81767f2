"""The sequence losses on the GPU against their definition in binary64
(tests/sequence_ref.py).

Tolerances: terms and sums are binary64, so an output is off by its own rounding
(2^-24 of its value), the gradient of a mean by two, and by what binary64 loses: n
terms of magnitudes that add up to S lose at most (n + 8) 2^-53 S, far below
10^-12 S here.  Values below binary32's normal range round to steps of 2^-149."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
z = pytest.importorskip("fsdp_sharded_optimizer_flat_amd")
pytestmark = pytest.mark.gpu

import sequence_ref as ref64  # noqa: E402

DEV = "cuda:0"
HALF = 2.0 ** -24
MODE = {"mean": z.ZERO_SEQUENCE_MEAN, "sum": z.ZERO_SEQUENCE_SUM}
KIND = {"sigmoid": z.ZERO_PREFER_SIGMOID, "hinge": z.ZERO_PREFER_HINGE, "squared": z.ZERO_PREFER_SQUARED}
KEPT = 7.25     # what positions of no sequence hold


def close(got, want, roundings=1, scale=0.0, what=""):
    got, want = got.double().cpu().numpy(), np.asarray(want, np.float64)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), what
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), what
    ok = ~(nan | inf)
    scale = np.broadcast_to(scale, want.shape)[ok]
    tol = roundings * HALF * np.abs(want[ok]) * (1 + HALF) + 1e-12 * scale + 2.0 ** -148
    bad = np.abs(got[ok] - want[ok]) > tol
    assert not bad.any(), (what, np.nonzero(bad)[0][:5], got[ok][bad][:5], want[ok][bad][:5])


def make(seed, lengths, lead=0, tail=0, prompts=0.25):
    """Offsets and values of packed sequences of the given lengths, `lead` positions
    before the first and `tail` behind the last."""
    g = np.random.default_rng(seed)
    off = lead + np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
    n = int(off[-1]) + tail
    lp = -np.exp(g.normal(-1.0, 1.5, n))
    old = lp + g.normal(0, 0.3, n)
    ref = lp + g.normal(0, 0.4, n)
    tokens = g.integers(0, 50304, n)
    tokens[g.random(n) < prompts] = -1
    f = lambda a: np.asarray(a, np.float32)
    return dict(off=off, n=n, lp=f(lp), old=f(old), ref=f(ref), tokens=tokens.astype(np.int64),
                adv=f(g.normal(0, 1, n)), seq_adv=f(g.normal(0, 1, len(lengths))),
                d_loss=f(g.uniform(0.2, 2.0, len(lengths))))


def dev(a, shift=0):
    """On the device; with `shift`, that many elements into an allocation."""
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a))
    buf = torch.empty(t.numel() + shift, dtype=t.dtype, device=DEV)
    buf[shift:] = t.to(DEV)
    return buf[shift:]


def workspace(n, b, fill=255):
    """Filled with NaN bits: a call must not read what it has not written."""
    return torch.full((z.zero_sequence_loss_workspace_bytes(n, b),), fill, dtype=torch.uint8, device=DEV)


def run_policy(d, per_token=True, low=0.2, high=0.28, coef=0.05, mode="mean", with_ref=True,
               with_tokens=True, shift=0, ws=None, grad=True, stream=None):
    b, n = len(d["off"]) - 1, d["n"]
    f = lambda k: torch.full((k,), KEPT, device=DEV)
    o = dict(loss=f(b), kl=f(b) if with_ref else None, clipped=torch.full((b,), -5, dtype=torch.int32, device=DEV),
             d_logprob=f(n + shift)[shift:] if grad else None)
    z.zero_policy_loss(dev(d["lp"], shift), dev(d["old"], shift), dev(d["adv"] if per_token else d["seq_adv"], shift),
                       dev(d["off"]), tokens=dev(d["tokens"], shift) if with_tokens else None,
                       ref_logprob=dev(d["ref"], shift) if with_ref else None, per_token=per_token, clip_low=low,
                       clip_high=high, kl_coef=coef if with_ref else 0.0, mode=MODE[mode],
                       d_loss=dev(d["d_loss"]) if grad else None, workspace=workspace(n, b) if ws is None else ws,
                       stream=stream, **o)
    return o


def check_policy(d, o, per_token=True, low=0.2, high=0.28, coef=0.05, mode="mean", with_ref=True,
                 with_tokens=True, **_):
    want = ref64.policy(d["lp"], d["old"], d["ref"] if with_ref else None, d["adv"] if per_token else d["seq_adv"],
                        per_token, d["tokens"] if with_tokens else None, d["off"], low, high,
                        coef if with_ref else 0.0, mode, d["d_loss"], np.full(d["n"], KEPT))
    # magnitudes of a sequence's terms: |A| r, kl's
    big = 10.0 * max(1.0, np.nanmax(np.abs(np.where(np.isfinite(want[3]), want[3], 0)), initial=0.0)) * d["n"]
    close(o["loss"], want[0], 1, big, "loss")
    if with_ref:
        close(o["kl"], want[1], 1, big, "kl")
    assert np.array_equal(o["clipped"].cpu().numpy(), want[2])
    if o["d_logprob"] is not None:
        close(o["d_logprob"], want[3], 2 if mode == "mean" else 1, 10.0, "d_logprob")


LENGTHS = {"one": [1], "empty": [0], "short": [1, 2, 3, 0, 5, 4, 0, 0, 7], "tile": [255, 256, 257, 1023, 1024, 1025],
           "long": [9001], "uneven": [3, 6000, 1, 0, 700, 12, 2049], "many": [1, 5, 9, 2] * 200,
           "cut": [40000, 7, 0, 30001, 1], "cut evenly": [4096] * 9}


@pytest.mark.parametrize("mode", ["mean", "sum"])
@pytest.mark.parametrize("name", LENGTHS)
def test_policy(name, mode):
    d = make(len(name), LENGTHS[name], lead=3, tail=5)
    for kw in (dict(mode=mode), dict(mode=mode, per_token=False, with_ref=False),
               dict(mode=mode, with_tokens=False, low=1.0, high=float("inf")), dict(mode=mode, coef=0.0, shift=1)):
        check_policy(d, run_policy(d, **kw), **kw)


def crowds():
    """Many positions: one sequence, thousands of short ones, more than a search of
    three levels tells apart."""
    g = np.random.default_rng(3)
    return {"single": [300001], "thousands": g.integers(0, 17, 5000), "swarm": g.integers(0, 3, 70000),
            "gaps": [0] * 70 + [20000] + [0] * 4100 + [5] + [0] * 3}


@pytest.mark.parametrize("name", crowds())
def test_policy_of_many_positions(name):
    d = make(70, crowds()[name], lead=1, tail=2)
    for kw in (dict(mode="mean"), dict(mode="sum", per_token=False, with_ref=False, shift=1)):
        check_policy(d, run_policy(d, **kw), **kw)


@pytest.mark.parametrize("name", crowds())
def test_preference_of_many_positions(name):
    lengths = crowds()[name]
    d = make(71, list(lengths) + [7] * (len(lengths) % 2), lead=1, tail=2)
    for kw in (dict(mode="mean", beta=0.5), dict(mode="sum", with_ref=False, shift=1, kind="squared")):
        check_preference(d, run_preference(d, **kw), **kw)


def test_policy_outputs_alone_and_forward_only():
    d = make(5, LENGTHS["uneven"])
    full = run_policy(d)
    fwd = run_policy(d, grad=False)
    for k in ("loss", "kl", "clipped"):
        assert torch.equal(full[k], fwd[k])
        got = torch.empty_like(full[k])
        z.zero_policy_loss(dev(d["lp"]), dev(d["old"]), dev(d["adv"]), dev(d["off"]), tokens=dev(d["tokens"]),
                           ref_logprob=dev(d["ref"]), per_token=True, clip_high=0.28, kl_coef=0.05,
                           workspace=workspace(d["n"], 7), **{k: got})
        assert torch.equal(got, full[k]), k


def test_policy_masked_positions_hold_anything():
    """Prompts with NaN, infinities and the type's lowest value add nothing."""
    for lengths in (LENGTHS["uneven"], LENGTHS["cut"]):
        d = make(6, lengths, prompts=0.4)
        clean = run_policy(d)
        off = d["tokens"] < 0
        junk = np.array([np.nan, np.inf, -np.inf, np.finfo(np.float32).min], np.float32)
        for k in ("lp", "old", "ref", "adv"):
            d[k][off] = junk[np.arange(off.sum()) % 4]
        dirty = run_policy(d)
        for k in clean:
            assert torch.equal(clean[k], dirty[k]), k
        # an upstream gradient without a value, too
        d["d_loss"][:] = np.inf
        for mode in ("mean", "sum"):
            o = run_policy(d, mode=mode)
            assert bool((o["d_logprob"].cpu()[torch.from_numpy(off)] == 0).all())


def test_policy_no_targets():
    for lengths in (LENGTHS["uneven"], LENGTHS["cut"]):
        d = make(7, lengths)
        d["tokens"][:] = -1
        for mode in ("mean", "sum"):
            o = run_policy(d, mode=mode)
            assert all(bool((o[k] == 0).all()) for k in o)


def test_policy_values_without_one():
    """NaN and infinite log probabilities: the sequence they are in, no other."""
    d = make(8, [50, 60, 70, 80, 90], prompts=0.0)
    nan, inf = np.nan, np.inf
    d["lp"][55] = nan                          # sequence 1
    d["lp"][120] = -inf                        # 2: ratio 0, k infinite
    d["ref"][185] = -inf                       # 3: k infinite
    d["lp"][270], d["adv"][270] = 1000.0, -1.0  # 4: ratio infinite
    o = run_policy(d, mode="sum")
    check_policy(d, o, mode="sum")
    loss = o["loss"].cpu().numpy()
    assert np.isnan(loss[1]) and loss[2] == inf and loss[3] == inf and loss[4] == inf and np.isfinite(loss[0])


def test_policy_at_the_border():
    """Ratios one binary32 step on either side of the clipping border."""
    low, high = 0.2, 0.28
    old = np.float32(-1.0)
    lps, advs = [], []
    for border in (np.log1p(-low), np.log1p(high)):
        x = np.float32(old + border)
        for step in range(-3, 4):
            v = x
            for _ in range(abs(step)):
                v = np.nextafter(v, np.float32(np.sign(step) * 10))
            for a in (-1.5, 0.0, 1.5):
                lps.append(v)
                advs.append(a)
    n = len(lps)
    d = dict(off=np.arange(n + 1, dtype=np.int64), n=n, lp=np.array(lps, np.float32),
             old=np.full(n, old, np.float32), ref=np.array(lps, np.float32), tokens=np.zeros(n, np.int64),
             adv=np.array(advs, np.float32), seq_adv=np.array(advs, np.float32), d_loss=np.ones(n, np.float32))
    o = run_policy(d)
    check_policy(d, o)
    c = o["clipped"].cpu().numpy()
    assert 0 < c.sum() < n


def test_policy_small_divergence_keeps_its_digits():
    """k = exp(x) - 1 - x of x about 10^-4 to its last digits."""
    d = make(9, [300, 400], prompts=0.0)
    d["ref"] = (d["lp"] * np.float32(1 + 2 ** -13)).astype(np.float32)
    o = run_policy(d, mode="sum")
    want = ref64.policy(d["lp"], d["old"], d["ref"], d["adv"], True, None, d["off"], 0.2, 0.28, 0.05, "sum",
                        d["d_loss"], np.zeros(700))[1]
    # expm1(x) - x in binary64 loses |x| 2^-53 a term: below 10^-9 of x^2 / 2
    close(o["kl"], want, 1, 1e3 * want, "kl")


def test_policy_differences():
    """The gradient against differences of the loss (away from the borders)."""
    d = make(10, [40, 60], prompts=0.2)
    o = run_policy(d)
    g = o["d_logprob"].double().cpu().numpy()
    args = lambda lp: ref64.policy(lp, d["old"], d["ref"], d["adv"], True, d["tokens"], d["off"], 0.2, 0.28, 0.05,
                                   "mean", d["d_loss"], np.zeros(100))
    for t in range(0, 100, 7):
        lp = d["lp"].astype(np.float64)
        if abs(abs(lp[t] - d["old"][t]) - 0.23) < 0.03:
            continue
        h = 1e-5
        up, down = lp.copy(), lp.copy()
        up[t] += h
        down[t] -= h
        diff = ((args(up)[0] - args(down)[0]) * d["d_loss"]).sum() / (2 * h)
        assert abs(diff - g[t]) <= 1e-6 * (1 + abs(g[t])), t


def test_policy_offsets_out_of_range_are_clamped():
    d = make(11, [10, 20, 30])
    d["off"] = np.array([-5, 10, 30, 1 << 40], np.int64)
    o = run_policy(d, mode="sum")
    check_policy(d, o, mode="sum")


def run_preference(d, kind="sigmoid", beta=0.1, margin=0.0, smoothing=0.0, mode="sum", with_ref=True,
                   with_tokens=True, shift=0, ws=None, grad=True, stream=None):
    b, n = len(d["off"]) - 1, d["n"]
    f = lambda k: torch.full((k,), KEPT, device=DEV)
    o = dict(loss=f(b // 2), reward=f(b), d_logprob=f(n + shift)[shift:] if grad else None)
    z.zero_preference_loss(dev(d["lp"], shift), dev(d["off"]), tokens=dev(d["tokens"], shift) if with_tokens else None,
                           ref_logprob=dev(d["ref"], shift) if with_ref else None, kind=KIND[kind], beta=beta,
                           margin=margin, smoothing=smoothing, mode=MODE[mode],
                           d_loss=dev(d["d_loss"][:b // 2]) if grad else None,
                           workspace=workspace(n, b) if ws is None else ws, stream=stream, **o)
    return o


def check_preference(d, o, kind="sigmoid", beta=0.1, margin=0.0, smoothing=0.0, mode="sum", with_ref=True,
                     with_tokens=True, **_):
    b = len(d["off"]) - 1
    want = ref64.preference(d["lp"], d["ref"] if with_ref else None, d["tokens"] if with_tokens else None, d["off"],
                            b // 2, kind, beta, margin, smoothing, mode, d["d_loss"], np.full(d["n"], KEPT))
    size = float(np.abs(d["lp"][np.isfinite(d["lp"])]).sum() + 1) * (1 + beta) * (1 + 1 / beta) ** 2
    close(o["loss"], want[0], 1, size, "loss")
    close(o["reward"], want[1], 1, size, "reward")
    if o["d_logprob"] is not None:
        close(o["d_logprob"], want[2], 1, size, "d_logprob")


PAIRS = {"one": [1, 1], "empty": [0, 0, 3, 0], "short": [1, 2, 3, 0, 5, 4, 0, 0, 7, 6],
         "tile": [255, 256, 257, 1023, 1024, 1025], "long": [9001, 20], "many": [1, 5, 9, 2] * 200,
         "cut": [40000, 7, 0, 30001, 1, 512], "cut evenly": [4096] * 10}


@pytest.mark.parametrize("kind", KIND)
@pytest.mark.parametrize("name", PAIRS)
def test_preference(name, kind):
    d = make(20 + len(name), PAIRS[name], lead=2, tail=9)
    for kw in (dict(mode="sum"), dict(mode="mean", beta=2.0, margin=0.3, with_ref=False),
               dict(mode="mean", with_tokens=False, shift=3), dict(mode="sum", grad=False)):
        kw["kind"] = kind
        if kind == "sigmoid" and kw["mode"] == "mean":
            kw["smoothing"] = 0.1
        check_preference(d, run_preference(d, **kw), **kw)


def test_preference_masked_positions_hold_anything():
    for lengths in ([30, 900, 2000, 5], PAIRS["cut"]):
        d = make(31, lengths, prompts=0.5)
        clean = run_preference(d, mode="mean")
        off = d["tokens"] < 0
        for k in ("lp", "ref"):
            d[k][off] = np.array([np.nan, np.inf, -np.inf, np.finfo(np.float32).min],
                                 np.float32)[np.arange(off.sum()) % 4]
        dirty = run_preference(d, mode="mean")
        for k in clean:
            assert torch.equal(clean[k], dirty[k]), k


def test_preference_extremes():
    """Certain pairs, impossible tokens and NaN."""
    d = make(32, [4] * 10, prompts=0.0)
    d["lp"][0] = -np.inf                   # chosen impossible: h = -inf
    d["lp"][4 * 6] = -np.inf               # rejected impossible: h = +inf
    d["lp"][4 * 2] = np.nan
    d["lp"][4 * 3] = -1e6                  # far beyond exp's range
    d["lp"][4 * 9] = -1e6
    o = run_preference(d, with_ref=False)
    loss, g = o["loss"].cpu().numpy(), o["d_logprob"].cpu().numpy()
    up = d["d_loss"]
    assert loss[0] == np.inf and loss[1] == 0 and np.isnan(loss[2])
    assert abs(loss[3] - 1e5) < 1 and loss[4] == 0
    assert np.allclose(g[0:4], -0.1 * up[0], rtol=1e-6) and np.allclose(g[20:24], 0.1 * up[0], rtol=1e-6)
    assert (g[4:8] == 0).all() and (g[24:28] == 0).all()
    assert np.isnan(g[8:12]).all() and np.isnan(g[28:32]).all()


def test_preference_differences():
    d = make(33, [30, 25, 40, 20], prompts=0.2)
    for kind in KIND:
        o = run_preference(d, kind=kind, beta=0.5, mode="mean")
        g = o["d_logprob"].double().cpu().numpy()
        f = lambda lp: (ref64.preference(lp, d["ref"], d["tokens"], d["off"], 2, kind, 0.5, 0.0, 0.0, "mean",
                                         d["d_loss"], np.zeros(d["n"]))[0] * d["d_loss"][:2]).sum()
        for t in range(0, d["n"], 9):
            h = 1e-5
            up, down = d["lp"].astype(np.float64), d["lp"].astype(np.float64)
            up[t] += h
            down[t] -= h
            assert abs((f(up) - f(down)) / (2 * h) - g[t]) <= 1e-6 * (1 + abs(g[t])), (kind, t)


def test_same_bits_on_another_stream_and_in_graphs():
    d, p = make(40, LENGTHS["cut"]), make(41, PAIRS["cut"])
    want, pwant = run_policy(d), run_preference(p)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = run_policy(d)
    side.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]), k
    # one graph of both calls, replayed between eager work on other values
    b, n = len(d["off"]) - 1, d["n"]
    ins = [dev(d[k]) for k in ("lp", "old", "adv", "off", "tokens", "ref", "d_loss")]
    outs = dict(loss=torch.empty(b, device=DEV), kl=torch.empty(b, device=DEV),
                clipped=torch.empty(b, dtype=torch.int32, device=DEV), d_logprob=torch.empty(n, device=DEV))
    pb, pn = len(p["off"]) - 1, p["n"]
    pins = [dev(p["lp"]), dev(p["off"]), dev(p["tokens"]), dev(p["ref"]), dev(p["d_loss"][:pb // 2])]
    pouts = dict(loss=torch.empty(pb // 2, device=DEV), reward=torch.empty(pb, device=DEV),
                 d_logprob=torch.empty(pn, device=DEV))
    w, pw = workspace(n, b), workspace(pn, pb)

    def calls():
        lp, old, adv, off, tok, rf, dl = ins
        z.zero_policy_loss(lp, old, adv, off, tokens=tok, ref_logprob=rf, per_token=True, clip_high=0.28,
                           kl_coef=0.05, d_loss=dl, workspace=w, **outs)
        z.zero_preference_loss(pins[0], pins[1], tokens=pins[2], ref_logprob=pins[3], d_loss=pins[4],
                               workspace=pw, **pouts)
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for turn in range(3):
        d2, p2 = make(50 + turn, LENGTHS["cut"]), make(60 + turn, PAIRS["cut"])
        want, pwant = run_policy(d2), run_preference(p2)
        for t, k in zip(ins, ("lp", "old", "adv", "off", "tokens", "ref", "d_loss")):
            t.copy_(dev(d2[k]))
        for t, k in zip(pins, (p2["lp"], p2["off"], p2["tokens"], p2["ref"], p2["d_loss"][:pb // 2])):
            t.copy_(dev(k))
        for t in [*outs.values(), *pouts.values()]:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for k in outs:
            assert torch.equal(outs[k], want[k]), (turn, k)
        for k in pouts:
            assert torch.equal(pouts[k], pwant[k]), (turn, k)


@pytest.mark.parametrize("b", [2, 300])
def test_no_positions(b):
    """Sequences that are all empty, with every output: torch's tensors of no elements
    have no address."""
    e, off = torch.empty(0, device=DEV), torch.zeros(b + 1, dtype=torch.int64, device=DEV)
    tok, up = torch.empty(0, dtype=torch.int64, device=DEV), torch.ones(b, device=DEV)
    f = lambda n: torch.full((n,), KEPT, device=DEV)
    for per_token in (True, False):
        for mode in MODE.values():
            o = dict(loss=f(b), kl=f(b), clipped=torch.full((b,), 3, dtype=torch.int32, device=DEV))
            z.zero_policy_loss(e, e, e if per_token else up, off, tokens=tok, ref_logprob=e, per_token=per_token,
                               kl_coef=0.1, mode=mode, d_loss=up, d_logprob=e, workspace=workspace(0, b), **o)
            assert all(bool((v == 0).all()) for v in o.values())
    loss, reward = f(b // 2), f(b)
    z.zero_preference_loss(e, off, tokens=tok, ref_logprob=e, d_loss=up[:b // 2], loss=loss, reward=reward,
                           d_logprob=e, workspace=workspace(0, b))
    close(loss, np.full(b // 2, np.log(2.0)))
    assert bool((reward == 0).all())


@pytest.mark.parametrize("lengths", [[30, 20, 25, 10], PAIRS["cut"]])
def test_preference_squared_of_extreme_beta(lengths):
    """The derivative is 2 (h - 1/2) / beta, whatever beta's square is: with a beta of
    10^-170 zero for an upstream of zero, with one of 10^170 twice the difference of the
    log ratios, (h - 1/2) / beta."""
    d = make(34, lengths, prompts=0.2)
    p = len(lengths) // 2
    d["d_loss"][:] = 0.0
    o = run_preference(d, kind="squared", beta=1e-170)
    assert bool((o["d_logprob"] == 0).all()) and bool((o["reward"] == 0).all())
    d["d_loss"][:] = 1.0
    o = run_preference(d, kind="squared", beta=1e170)
    s = [sum(float(d["lp"][t]) - float(d["ref"][t]) for t in q)
         for q in ref64.targets_of(d["off"], d["tokens"], d["n"])]
    size = float(np.abs(d["lp"]).sum())
    want = np.zeros(d["n"])
    for i in range(p):
        for b, sign in ((i, 1.0), (i + p, -1.0)):
            q = ref64.targets_of(d["off"], d["tokens"], d["n"])[b]
            want[q] = sign * 2.0 * (s[i] - s[i + p])
    close(o["loss"], (np.array(s[:p]) - np.array(s[p:])) ** 2, 1, size * size, "loss")
    close(o["d_logprob"], want, 1, size, "d_logprob")
