"""The token-loss entry points on the host: what they refuse, before any device
work (the addresses below are never read), and the workspace query.  CPU only."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")
z = pytest.importorskip("fsdp_sharded_optimizer_flat_amd")

R, V, K = 4, 100, 5
BASE = 1 << 40
A = {name: BASE + i * (1 << 20) for i, name in enumerate(
    ["logits", "tokens", "logprob", "entropy", "stats", "top_index", "top_logprob", "d_logprob",
     "d_entropy", "d_logits", "loss", "d_loss", "top_value", "workspace"])}
ENOUGH = 1 << 19


def call(entry, **change):
    a = dict(A, dtype=z.ZERO_F32, rows=R, vocab=V, stride=V, scale=1.0, d_stride=V, top_k=K,
             mode=z.ZERO_DISTILL_TAIL, wb=ENOUGH, stream=None)
    a.update(change)
    head = [a["logits"], a["dtype"], a["rows"], a["vocab"], a["stride"], a["scale"]]
    ws = [a["workspace"], a["wb"], a["stream"]]
    rec = [a["top_k"], a["top_index"], a["top_value"], a["mode"]]
    rest = {
        "zero_logprob": [a["tokens"], a["logprob"], a["entropy"], a["stats"], a["top_k"],
                         a["top_index"], a["top_logprob"], *ws],
        "zero_logprob_grad": [a["tokens"], a["stats"], a["entropy"], a["d_logprob"], a["d_entropy"],
                              a["d_logits"], a["d_stride"], a["stream"]],
        "zero_logprob_fused": [a["tokens"], a["d_logprob"], a["d_entropy"], a["logprob"],
                               a["entropy"], a["d_logits"], a["d_stride"], *ws],
        "zero_distill": [*rec, a["loss"], a["stats"], *ws],
        "zero_distill_grad": [*rec, a["stats"], a["d_loss"], a["d_logits"], a["d_stride"], a["stream"]],
        "zero_distill_fused": [*rec, a["d_loss"], a["loss"], a["d_logits"], a["d_stride"], *ws],
    }[entry]
    return getattr(z.raw_library(), entry)(*head, *rest)


FORWARD = ["zero_logprob", "zero_distill"]
GRAD = ["zero_logprob_grad", "zero_distill_grad"]
FUSED = ["zero_logprob_fused", "zero_distill_fused"]
DISTILL = ["zero_distill", "zero_distill_grad", "zero_distill_fused"]
EVERY = FORWARD + GRAD + FUSED
EINVAL, ERANGE, EALIGN, ENOSPC = z.ZERO_EINVAL, z.ZERO_ERANGE, z.ZERO_EALIGN, z.ZERO_ENOSPC


@pytest.mark.parametrize("entry", EVERY)
def test_refused_sizes(entry):
    nan, inf = float("nan"), float("inf")
    for change, want in [
            (dict(dtype=2), EINVAL), (dict(rows=-1), EINVAL), (dict(vocab=0), EINVAL),
            (dict(vocab=-3), EINVAL), (dict(stride=V - 1), EINVAL), (dict(logits=None), EINVAL),
            (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL), (dict(scale=nan), EINVAL),
            (dict(scale=inf), EINVAL), (dict(scale=2.0 ** 21), ERANGE),
            (dict(scale=2.0 ** -21), ERANGE),
            (dict(vocab=z.ZERO_MAX_VOCAB + 1, stride=1 << 21, d_stride=1 << 21), ERANGE),
            (dict(rows=1 << 31), ERANGE), (dict(stride=1 << 62), ERANGE),
            (dict(logits=A["logits"] + 2), EALIGN)]:
        assert call(entry, **change) == want, change


@pytest.mark.parametrize("entry", EVERY)
def test_no_rows_is_no_work(entry):
    assert call(entry, rows=0) == z.ZERO_OK
    assert call(entry, rows=0, logits=None) == z.ZERO_OK
    # tensors of no rows have no address
    nothing = dict(logits=None, tokens=None, logprob=None, entropy=None, stats=None, top_index=None,
                   top_logprob=None, top_value=None, d_logprob=None, d_entropy=None, d_logits=None,
                   loss=None, d_loss=None, workspace=None, wb=0)
    assert set(nothing) - {"wb"} <= set(A)
    assert call(entry, rows=0, **nothing) == z.ZERO_OK
    assert call(entry, rows=0, **{**nothing, "vocab": 0}) == EINVAL


def test_refused_pointers():
    for entry, change in [
            ("zero_logprob", dict(tokens=None)),                          # logprob wants tokens
            ("zero_logprob", dict(top_index=None)), ("zero_logprob", dict(top_logprob=None)),
            ("zero_logprob", dict(top_k=0)), ("zero_logprob", dict(top_k=-1)),
            ("zero_logprob", dict(logprob=None, entropy=None, stats=None, top_k=0, top_index=None,
                                  top_logprob=None)),                     # nothing is wanted
            ("zero_logprob_grad", dict(stats=None)), ("zero_logprob_grad", dict(tokens=None)),
            ("zero_logprob_grad", dict(entropy=None)), ("zero_logprob_grad", dict(d_logits=None)),
            ("zero_logprob_grad", dict(d_logprob=None, d_entropy=None)),
            ("zero_logprob_fused", dict(d_logprob=None, d_entropy=None)),
            ("zero_logprob_fused", dict(tokens=None)), ("zero_logprob_fused", dict(d_logits=None)),
            ("zero_distill", dict(loss=None, stats=None)),
            ("zero_distill_grad", dict(stats=None)), ("zero_distill_grad", dict(d_loss=None)),
            ("zero_distill_grad", dict(d_logits=None)),
            ("zero_distill_fused", dict(d_loss=None)), ("zero_distill_fused", dict(d_logits=None))]:
        assert call(entry, **change) == EINVAL, (entry, change)
    for entry in DISTILL:
        for change in (dict(top_k=0), dict(mode=2), dict(mode=-1), dict(top_index=None),
                       dict(top_value=None)):
            assert call(entry, **change) == EINVAL, (entry, change)
        assert call(entry, top_k=z.ZERO_MAX_TOP + 1) == ERANGE
    assert call("zero_logprob", top_k=z.ZERO_MAX_TOP + 1) == ERANGE
    for entry in GRAD + FUSED:
        assert call(entry, d_stride=V - 1) == EINVAL
        assert call(entry, d_stride=1 << 62) == ERANGE


def test_refused_alignment_and_overlap():
    odd = [("zero_logprob", n) for n in ("tokens", "logprob", "entropy", "stats", "top_index",
                                         "top_logprob")]
    odd += [("zero_logprob_grad", n) for n in ("tokens", "stats", "entropy", "d_logprob",
                                               "d_entropy", "d_logits")]
    odd += [("zero_logprob_fused", n) for n in ("tokens", "d_logprob", "d_entropy", "logprob",
                                                "entropy", "d_logits")]
    odd += [("zero_distill", n) for n in ("top_index", "top_value", "loss", "stats")]
    odd += [("zero_distill_grad", n) for n in ("top_index", "top_value", "stats", "d_loss", "d_logits")]
    odd += [("zero_distill_fused", n) for n in ("top_index", "top_value", "d_loss", "loss",
                                                "d_logits")]
    for entry, name in odd:
        assert call(entry, **{name: A[name] + 2}) == EALIGN, (entry, name)
    # an output over an input, over another output, and a gradient that is
    # neither apart from the logits nor exactly on them
    for entry, change in [
            ("zero_logprob", dict(logprob=A["logits"] + 4 * V)), ("zero_logprob", dict(entropy=A["logprob"])),
            ("zero_logprob", dict(stats=A["tokens"])), ("zero_logprob", dict(top_index=A["top_logprob"])),
            ("zero_logprob_grad", dict(d_logits=A["logits"] + 4)),
            ("zero_logprob_grad", dict(d_logits=A["logits"], d_stride=V + 1)),
            ("zero_logprob_grad", dict(d_logits=A["stats"])),
            ("zero_logprob_fused", dict(d_logits=A["d_logprob"])),
            ("zero_logprob_fused", dict(logprob=A["d_logprob"])),
            ("zero_distill", dict(loss=A["stats"])), ("zero_distill", dict(loss=A["top_value"])),
            ("zero_distill_grad", dict(d_logits=A["top_index"])),
            ("zero_distill_fused", dict(loss=A["d_loss"])),
            ("zero_distill_fused", dict(d_logits=A["logits"] + 4 * V * (R - 1)))]:
        assert call(entry, **change) == EINVAL, (entry, change)


def test_workspace():
    for rows, vocab, k in [(1, 70001, 5), (64, 128256, 20), (1, 1 << 20, 256), (3, 131073, 0)]:
        need = z.zero_loss_workspace_bytes(rows, vocab, k)
        assert need > 0
        # the fused calls keep rows up to about 10^5 elements in registers
        for entry in FORWARD + (FUSED if vocab == 1 << 20 else []):
            big = dict(rows=rows, vocab=vocab, stride=vocab, d_stride=vocab,
                       logits=BASE + (1 << 34), d_logits=BASE + (1 << 36), top_k=max(k, 1))
            if entry == "zero_logprob" and not k:
                big.update(top_k=0, top_index=None, top_logprob=None)
            assert call(entry, **big, workspace=None, wb=0) == EINVAL
            assert call(entry, **big, wb=15) == ENOSPC
            assert call(entry, **big, workspace=A["workspace"] + 8) == EALIGN
            assert call(entry, **dict(big, logits=A["workspace"] - 16), wb=need) == EINVAL
    # enough for many rows: no partial results, only the fused calls' statistics
    assert z.zero_loss_workspace_bytes(4096, 128256, 64) == 4096 * 20
    assert z.zero_loss_workspace_bytes(0, 10, 0) == 0
    lib, b = z.raw_library(), C.c_size_t()
    assert lib.zero_loss_workspace_bytes(1, 1, 0, None) == EINVAL
    for bad, want in [((-1, 1, 0), EINVAL), ((1, 0, 0), EINVAL), ((1, 1, -1), EINVAL),
                      ((1, z.ZERO_MAX_VOCAB + 1, 0), ERANGE), ((1 << 31, 1, 0), ERANGE),
                      ((1, 1, z.ZERO_MAX_TOP + 1), ERANGE)]:
        assert lib.zero_loss_workspace_bytes(*bad, C.byref(b)) == want


def test_binding_refuses_host_and_malformed_tensors():
    x = torch.zeros(R, V)
    t = torch.zeros(R, dtype=torch.int64)
    f = torch.zeros(R)
    with pytest.raises(ValueError, match="device tensor"):
        z.zero_logprob(x, t, logprob=f)
    with pytest.raises(TypeError):
        z.zero_logprob([[0.0]], t, logprob=f)
    with pytest.raises(ValueError, match="two dimensions"):
        z.zero_logprob(torch.zeros(V), t, logprob=f)
    with pytest.raises(ValueError, match="device tensor"):
        z.zero_distill(x, torch.zeros(R, K, dtype=torch.int32), torch.zeros(R, K), 0, loss=f)
