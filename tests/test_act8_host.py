"""The entry points of the 8-bit activation checkpoints on the host: what they
refuse, before any device work (the addresses below are never read).  CPU only."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")
z = pytest.importorskip("fsdp_sharded_optimizer_flat_amd")

R, O, K = 50, 70, 100
BASE = 1 << 40
A = {n: BASE + i * (1 << 32) for i, n in enumerate(["x", "codes", "scales", "d_y", "d_w", "workspace"])}
EINVAL, ERANGE, EALIGN, ENOSPC = z.ZERO_EINVAL, z.ZERO_ERANGE, z.ZERO_EALIGN, z.ZERO_ENOSPC


def call(entry, **change):
    a = dict(A, dtype=z.ZERO_F32, rows=R, cols=K, stride=K, out=O, ystride=O, wstride=K, accumulate=0, wb=1 << 31)
    a.update(change)
    args = {"zero_act8_pack": [a["x"], a["dtype"], a["rows"], a["cols"], a["stride"], a["codes"], a["scales"], None],
            "zero_act8_unpack": [a["codes"], a["scales"], a["rows"], a["cols"], a["x"], a["dtype"], a["stride"], None],
            "zero_act8_weight_grad": [a["d_y"], a["rows"], a["out"], a["ystride"], a["codes"], a["scales"], a["cols"],
                                      a["d_w"], a["dtype"], a["wstride"], a["accumulate"], a["workspace"], a["wb"],
                                      None]}[entry]
    return getattr(z.raw_library(), entry)(*args)


EVERY = ["zero_act8_pack", "zero_act8_unpack", "zero_act8_weight_grad"]


@pytest.mark.parametrize("entry", EVERY)
def test_refused(entry):
    wide = dict(cols=(1 << 20) + 1, stride=1 << 21, wstride=1 << 21)
    for change, want in [(dict(dtype=2), EINVAL), (dict(rows=-1), EINVAL), (dict(cols=0), EINVAL),
                         (dict(stride=K - 1, wstride=K - 1), EINVAL), (dict(codes=None), EINVAL),
                         (dict(scales=None), EINVAL), (dict(x=None, d_y=None), EINVAL), (dict(rows=1 << 31), ERANGE),
                         (wide, ERANGE), (dict(stride=1 << 60, wstride=1 << 60), ERANGE),
                         (dict(x=A["x"] + 2, d_w=A["d_w"] + 2), EALIGN)]:
        assert call(entry, **change) == want, change


def test_refused_overlap():
    for entry, change in [("zero_act8_pack", dict(codes=A["x"])), ("zero_act8_pack", dict(scales=A["x"] + 7)),
                          ("zero_act8_pack", dict(scales=A["codes"] + R * K - 1)), ("zero_act8_unpack", dict(x=A["codes"])),
                          ("zero_act8_unpack", dict(x=A["scales"])), ("zero_act8_weight_grad", dict(d_w=A["d_y"])),
                          ("zero_act8_weight_grad", dict(d_w=A["codes"])),
                          ("zero_act8_weight_grad", dict(d_w=A["scales"]))]:
        assert call(entry, **change) == EINVAL, (entry, change)


def test_refused_by_the_weight_grad():
    for change, want in [(dict(out=0), EINVAL), (dict(out=(1 << 20) + 1, ystride=1 << 21), ERANGE),
                         (dict(ystride=O - 1), EINVAL), (dict(ystride=1 << 60), ERANGE), (dict(accumulate=2), EINVAL),
                         (dict(d_w=None), EINVAL), (dict(d_y=A["d_y"] + 1), EALIGN)]:
        assert call("zero_act8_weight_grad", **change) == want, change


def test_no_rows():
    for entry in EVERY[:2]:
        assert call(entry, rows=0, x=None, codes=None, scales=None) == z.ZERO_OK
    assert call("zero_act8_weight_grad", rows=0, d_w=None) == EINVAL


@pytest.mark.parametrize("rows,out,cols", [(8192, 1280, 1280), (100000, 64, 64), (16384, 128, 4096)])
def test_workspace(rows, out, cols):
    need = z.zero_act8_weight_grad_workspace_bytes(rows, out, cols)
    sizes = dict(rows=rows, out=out, cols=cols, ystride=out, wstride=cols)
    if need:
        assert call("zero_act8_weight_grad", **sizes, workspace=None, wb=0) == EINVAL
        assert call("zero_act8_weight_grad", **sizes, wb=need - 1) == ENOSPC
        assert call("zero_act8_weight_grad", **sizes, workspace=A["workspace"] + 8) == EALIGN
        for other in ("codes", "scales", "d_y", "d_w"):
            assert call("zero_act8_weight_grad", **sizes, workspace=A[other] + 16, wb=need) == EINVAL
    lib, b = z.raw_library(), C.c_size_t()
    assert lib.zero_act8_weight_grad_workspace_bytes(rows, out, cols, None) == EINVAL
    for bad, want in [((-1, 1, 1), EINVAL), ((1, 0, 1), EINVAL), ((1, 1, 0), EINVAL), ((1 << 31, 1, 1), ERANGE),
                      ((1, (1 << 20) + 1, 1), ERANGE), ((1, 1, (1 << 20) + 1), ERANGE)]:
        assert lib.zero_act8_weight_grad_workspace_bytes(*bad, C.byref(b)) == want


def test_binding_refuses_host_tensors():
    f, q = torch.zeros(10, 64), torch.zeros(10, 64, dtype=torch.uint8)
    s = torch.zeros(10, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensor"):
        z.zero_act8_pack(f, q, s)
    with pytest.raises(ValueError, match="device tensor"):
        z.zero_act8_unpack(q, s, f)
    with pytest.raises(ValueError, match="device tensor"):
        z.zero_act8_weight_grad(f.to(torch.bfloat16), q, s, f)
    with pytest.raises(TypeError):
        z.zero_act8_pack(None, q, s)
