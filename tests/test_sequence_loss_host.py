"""The sequence-loss entry points on the host: what they refuse, before any
device work (the addresses below are never read).  CPU only."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")
z = pytest.importorskip("fsdp_sharded_optimizer_flat_amd")

N, B = 1000, 6
BASE = 1 << 40
A = {name: BASE + i * (1 << 24) for i, name in enumerate(
    ["logprob", "old", "ref", "advantage", "tokens", "offsets", "d_loss", "loss", "kl", "clipped", "d_logprob",
     "reward", "workspace"])}
EINVAL, ERANGE, EALIGN, ENOSPC = z.ZERO_EINVAL, z.ZERO_ERANGE, z.ZERO_EALIGN, z.ZERO_ENOSPC
INF, NAN = float("inf"), float("nan")


def call(entry, **change):
    a = dict(A, n=N, b=B, per_token=1, low=0.2, high=0.2, coef=0.1, mode=0, kind=0, beta=0.1, margin=0.0,
             smoothing=0.0, wb=1 << 23)
    a.update(change)
    ws = [a["workspace"], a["wb"], None]
    if entry == "zero_policy_loss":
        args = [a["logprob"], a["old"], a["ref"], a["advantage"], a["per_token"], a["tokens"], a["n"], a["offsets"],
                a["b"], a["low"], a["high"], a["coef"], a["mode"], a["d_loss"], a["loss"], a["kl"], a["clipped"],
                a["d_logprob"], *ws]
    else:
        args = [a["logprob"], a["ref"], a["tokens"], a["n"], a["offsets"], a["b"] // 2, a["kind"], a["beta"],
                a["margin"], a["smoothing"], a["mode"], a["d_loss"], a["loss"], a["reward"], a["d_logprob"], *ws]
    return getattr(z.raw_library(), entry)(*args)


BOTH = ["zero_policy_loss", "zero_preference_loss"]


@pytest.mark.parametrize("entry", BOTH)
def test_refused_sizes_and_pointers(entry):
    for change, want in [(dict(n=-1), EINVAL), (dict(b=-2), EINVAL), (dict(mode=2), EINVAL), (dict(mode=-1), EINVAL),
                         (dict(n=1 << 31), ERANGE), (dict(b=(1 << 20) + 2), ERANGE), (dict(offsets=None), EINVAL),
                         (dict(logprob=None), EINVAL), (dict(d_loss=None), EINVAL),
                         (dict(loss=None, kl=None, clipped=None, d_logprob=None, reward=None), EINVAL)]:
        assert call(entry, **change) == want, change


def test_refused_values():
    for change in (dict(low=-0.1), dict(low=1.1), dict(low=NAN), dict(high=-0.1), dict(high=NAN), dict(coef=-1.0),
                   dict(coef=INF), dict(coef=NAN), dict(ref=None), dict(ref=None, kl=None), dict(old=None),
                   dict(advantage=None), dict(per_token=0, advantage=None)):
        assert call("zero_policy_loss", **change) == EINVAL, change
    for change in (dict(kind=3), dict(kind=-1), dict(beta=0.0), dict(beta=-1.0), dict(beta=INF), dict(beta=NAN),
                   dict(margin=INF), dict(margin=NAN), dict(smoothing=-0.1), dict(smoothing=1.5), dict(smoothing=NAN),
                   dict(kind=1, smoothing=0.1), dict(kind=2, smoothing=0.1)):
        assert call("zero_preference_loss", **change) == EINVAL, change


def test_refused_alignment_and_overlap():
    arrays = {"zero_policy_loss": ["logprob", "old", "ref", "advantage", "tokens", "offsets", "d_loss", "loss", "kl",
                                   "clipped", "d_logprob"],
              "zero_preference_loss": ["logprob", "ref", "tokens", "offsets", "d_loss", "loss", "reward",
                                       "d_logprob"]}
    for entry, names in arrays.items():
        for name in names:
            assert call(entry, **{name: A[name] + 2}) == EALIGN, (entry, name)
        outs = [n for n in names if n in ("loss", "kl", "clipped", "d_logprob", "reward")]
        for out in outs:
            for other in names:
                if other != out:
                    assert call(entry, **{out: A[other]}) == EINVAL, (entry, out, other)
        assert call(entry, d_logprob=A["logprob"] + 4 * (N - 1)) == EINVAL


@pytest.mark.parametrize("entry", BOTH)
def test_no_sequences_is_no_work(entry):
    nothing = {k: None for k in A}
    assert call(entry, b=0, n=0, **nothing, wb=0) == z.ZERO_OK
    assert call(entry, b=0) == z.ZERO_OK
    assert call(entry, b=0, mode=5) == EINVAL


@pytest.mark.parametrize("n,b", [(100000, 2), (1 << 20, 300), ((1 << 31) - 1, 1 << 20)])
def test_workspace(n, b):
    need = z.zero_sequence_loss_workspace_bytes(n, b)
    far = {k: BASE + i * (1 << 36) for i, k in enumerate(A)}
    for entry in BOTH:
        if need:
            assert call(entry, **far | dict(n=n, b=b, workspace=None, wb=0)) == EINVAL
            assert call(entry, **far | dict(n=n, b=b, wb=need - 1)) == ENOSPC
            assert call(entry, **far | dict(n=n, b=b, workspace=far["workspace"] + 8, wb=need)) == EALIGN
            assert call(entry, **far | dict(n=n, b=b, workspace=far["logprob"] + 16, wb=need)) == EINVAL
    out = C.c_size_t()
    lib = z.raw_library()
    assert lib.zero_sequence_loss_workspace_bytes(n, b, None) == EINVAL
    for bad, want in [((-1, 1), EINVAL), ((1, -1), EINVAL), ((1 << 31, 1), ERANGE), ((1, (1 << 20) + 1), ERANGE)]:
        assert lib.zero_sequence_loss_workspace_bytes(*bad, C.byref(out)) == want


def test_binding_refuses_host_tensors():
    f, t = torch.zeros(10), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="device tensor"):
        z.zero_policy_loss(f, f, f, t, loss=f)
    with pytest.raises(ValueError, match="device tensor"):
        z.zero_preference_loss(f, t, loss=f)
    with pytest.raises(TypeError):
        z.zero_policy_loss([0.0], f, f, t, loss=f)


def test_a_reference_of_no_positions_may_be_null():
    assert call("zero_policy_loss", b=0, n=0, ref=None) == z.ZERO_OK
    assert call("zero_policy_loss", b=0, n=0, ref=None, kl=None) == z.ZERO_OK
    assert call("zero_policy_loss", n=1, ref=None, coef=0.0) == EINVAL


def test_a_workspace_serves_fewer_positions_and_sequences():
    """Around each change of the tiles (at 1024 tiles a sequence of 2^8, 2^10 ... positions)
    and of the single launch's sizes."""
    most = z.ZERO_MAX_LOSS_ROWS
    for b in (1, 2, 3, 300, 4097, 1 << 20):
        around = {min(most, max(0, n * b + d)) for n in (2048, 1 << 18, 1 << 20, 1 << 22, 1 << 24, 1 << 26, 1 << 28)
                  for d in (-1, 0, 1, b - 1, b, b + 1)} | {0, 1, 16384, 16385, 100000, most}
        last = 0
        for n in sorted(around):
            now = z.zero_sequence_loss_workspace_bytes(n, b)
            assert now >= last, (n, b)
            last = now
    for n in (1000, 5000, 16384, 16385, 1 << 20, 300_000_001, most):
        around = {max(1, min(1 << 20, (n >> k) + d)) for k in (11, 18, 20, 22, 24, 26, 28) for d in (-1, 0, 1)}
        last = 0
        for b in sorted(around | {1, 2, 3, 1 << 20}):
            now = z.zero_sequence_loss_workspace_bytes(n, b)
            assert now >= last, (n, b)
            last = now


@pytest.mark.parametrize("entry", BOTH)
def test_a_workspace_is_enough(entry):
    """A call with what the query says for its sizes or more is not refused for it, but
    for the overlap that it has besides; one with less is."""
    far = {k: BASE + i * (1 << 40) for i, k in enumerate(A)}
    sizes = [(n, b) for n in (0, 1, 2048, 2049, 4098, 4099, 9000, 16383, 16384, 16385, 300000, 524288, 524291, 1 << 21,
                              40_000_000, (1 << 31) - 1) for b in (2, 4, 6, 8, 64, 300, 1 << 20)]
    cut = 0
    for n, b in sizes:
        clash = far | dict(n=n, b=b, kl=far["loss"], reward=far["loss"])
        for most in sizes:
            if most[0] >= n and most[1] >= b:
                wb = z.zero_sequence_loss_workspace_bytes(*most)
                assert call(entry, **clash, wb=wb) == EINVAL, (n, b, most)
        cut += call(entry, **clash, wb=23) == ENOSPC
    assert cut > 20
