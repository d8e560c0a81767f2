"""The embedding entry points on the host: what they refuse, before any device
work (the addresses below are never read).  CPU only."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")
z = pytest.importorskip("fsdp_sharded_optimizer_flat_amd")

R, V, H = 40, 100, 24
BASE = 1 << 40
A = {n: BASE + i * (1 << 30) for i, n in enumerate(["table", "tokens", "out", "workspace"])}
EINVAL, ERANGE, EALIGN, ENOSPC = z.ZERO_EINVAL, z.ZERO_ERANGE, z.ZERO_EALIGN, z.ZERO_ENOSPC


def call(entry, **change):
    """table: the looked-up table, or the gradient; out: the activations, or their
    gradient."""
    a = dict(A, dtype=z.ZERO_F32, odtype=z.ZERO_BF16, rows=R, vocab=V, hidden=H, stride=H, ostride=H, scale=1.0,
             accumulate=0, wb=1 << 20)
    a.update(change)
    if entry == "zero_embedding":
        args = [a["table"], a["dtype"], a["vocab"], a["hidden"], a["stride"], a["tokens"], a["rows"], a["scale"],
                a["out"], a["odtype"], a["ostride"], None]
    else:
        args = [a["out"], a["odtype"], a["rows"], a["hidden"], a["ostride"], a["tokens"], a["scale"], a["table"],
                a["dtype"], a["vocab"], a["stride"], a["accumulate"], a["workspace"], a["wb"], None]
    return getattr(z.raw_library(), entry)(*args)


@pytest.mark.parametrize("entry", ["zero_embedding", "zero_embedding_grad"])
def test_refused(entry):
    for change, want in [
            (dict(dtype=2), EINVAL), (dict(odtype=-1), EINVAL), (dict(rows=-1), EINVAL), (dict(vocab=0), EINVAL),
            (dict(hidden=0), EINVAL), (dict(stride=H - 1), EINVAL), (dict(ostride=H - 1), EINVAL),
            (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(table=None), EINVAL),
            (dict(tokens=None), EINVAL), (dict(out=None), EINVAL), (dict(rows=1 << 31), ERANGE),
            (dict(vocab=(1 << 20) + 1), ERANGE), (dict(hidden=(1 << 20) + 1, stride=1 << 21, ostride=1 << 21), ERANGE),
            (dict(stride=1 << 60), ERANGE), (dict(ostride=1 << 60), ERANGE), (dict(table=A["table"] + 2), EALIGN),
            (dict(tokens=A["tokens"] + 4), EALIGN), (dict(out=A["out"] + 1), EALIGN),
            (dict(out=A["table"] + 2 * H), EINVAL), (dict(table=A["out"] + 4), EINVAL)]:
        assert call(entry, **change) == want, change


def test_refused_by_the_gradient():
    need = z.zero_embedding_grad_workspace_bytes(R, V, H)
    assert need > 0
    for change, want in [
            (dict(accumulate=2), EINVAL), (dict(rows=(1 << 20) + 1), ERANGE), (dict(workspace=None), EINVAL),
            (dict(wb=need - 1), ENOSPC), (dict(workspace=A["workspace"] + 8), EALIGN), (dict(table=A["tokens"]), EINVAL),
            (dict(workspace=A["tokens"] + 16), EINVAL), (dict(workspace=A["table"] + 16), EINVAL),
            (dict(workspace=A["out"] + 16), EINVAL)]:
        assert call("zero_embedding_grad", **change) == want, change
    assert call("zero_embedding", out=A["tokens"]) == EINVAL


def test_no_rows():
    assert call("zero_embedding", rows=0, out=None, tokens=None) == z.ZERO_OK
    assert call("zero_embedding_grad", rows=0, out=None, tokens=None, workspace=None, wb=0, accumulate=1) == z.ZERO_OK
    assert call("zero_embedding_grad", rows=0, table=None, accumulate=1) == EINVAL


def test_workspace_query():
    lib, b = z.raw_library(), C.c_size_t()
    assert lib.zero_embedding_grad_workspace_bytes(1, 1, 1, None) == EINVAL
    for bad, want in [((-1, 1, 1), EINVAL), ((1, 0, 1), EINVAL), ((1, 1, 0), EINVAL), (((1 << 20) + 1, 1, 1), ERANGE),
                      ((1, (1 << 20) + 1, 1), ERANGE), ((1, 1, (1 << 20) + 1), ERANGE)]:
        assert lib.zero_embedding_grad_workspace_bytes(*bad, C.byref(b)) == want
    assert z.zero_embedding_grad_workspace_bytes(0, 10, 10) == 0
    # more rows never need less
    last = 0
    for rows in list(range(1, 2000, 13)) + [8191, 8192, 8193, 100000, 1 << 20]:
        now = z.zero_embedding_grad_workspace_bytes(rows, 1000, 1280)
        assert now >= last
        last = now


def test_binding_refuses_host_tensors():
    f, t = torch.zeros(10, 4), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="device tensor"):
        z.zero_embedding(f, t, f)
    with pytest.raises(ValueError, match="device tensor"):
        z.zero_embedding_grad(f, t, f)
    with pytest.raises(TypeError):
        z.zero_embedding([[0.0]], t, f)


def test_a_workspace_serves_fewer_rows():
    """Around every change of the sorting and the sums."""
    for hidden in (5, 512, 1280, 8200):
        last = 0
        for rows in (1, 32, 33, 2047, 2048, 2049, 4096, 8191, 8192, 8193, 65535, 65536, 65537, 70000, (1 << 20) - 1, 1 << 20):
            now = z.zero_embedding_grad_workspace_bytes(rows, 1000, hidden)
            assert now >= last, (hidden, rows)
            last = now


@pytest.mark.parametrize("hidden", [1, 5, 512, 513, 1280, 4096, 8200, 1 << 20])
def test_a_workspace_serves_fewer_rows_around_each_change_of_the_segments(hidden):
    """Segments grow where rows times slabs of 512 columns pass 2^14 and 2^16; longer ones
    need fewer parts, which must not show in what the query says."""
    slabs = (hidden + 511) // 512
    around = {w // slabs + d for w in (1 << 14, 1 << 16) for d in (-1, 0, 1, 2)}
    around |= {r for w in (1 << 14, 1 << 16) for r in (w // slabs * 2, w // slabs * 2 + 1)}
    around |= {1, 31, 32, 33, 2048, 2049, 65536, 65537, 1 << 20}
    last = 0
    for rows in sorted(r for r in around if 1 <= r <= z.ZERO_MAX_EMBEDDING_ROWS):
        now = z.zero_embedding_grad_workspace_bytes(rows, 1000, hidden)
        assert now >= last, (hidden, rows)
        last = now
