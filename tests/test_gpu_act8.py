"""8-bit activation checkpoints on the GPU against their definition in binary64
(tests/act8_ref.py).

Packing and unpacking are compared without a tolerance: a power of two scales
exactly, and each value is rounded once.  The weight gradient of whole numbers
whose sums stay below 2^24 is exact in binary32 in any order.  Of other values: each of
the R products is exact in binary32, each addition is off by at most 2^-23 of
the partial sums' magnitudes, whose bound is the sum of the products'
magnitudes, and the output is rounded once."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
z = pytest.importorskip("fsdp_sharded_optimizer_flat_amd")
pytestmark = pytest.mark.gpu

import act8_ref  # noqa: E402

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
KEPT = 5.5


def rows_of(n, cols, dtype, stride=None, shift=0, fill=KEPT):
    stride = stride or cols
    buf = torch.full((shift + max(n, 1) * stride + 16,), fill, dtype=dtype, device=DEV)
    return buf, buf[shift:shift + n * stride].view(n, stride)[:, :cols]


def outside(buf, view):
    on = torch.zeros(buf.numel(), dtype=torch.bool, device=DEV)
    on.as_strided(view.shape, view.stride(), view.storage_offset())[...] = True
    return buf[~on]


def checkpoint(rows, cols, shift=0):
    blocks = (cols + 31) // 32
    a, codes = rows_of(rows, cols, torch.uint8, None, shift, 77)
    b, scales = rows_of(rows, blocks, torch.uint8, None, shift, 77)
    return a, codes, b, scales


def same(got, want):
    """Equal values, NaN where NaN is wanted."""
    got, want = got.double().cpu(), want.double()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(nan=0.0, posinf=9e99, neginf=-9e99),
                       want.nan_to_num(nan=0.0, posinf=9e99, neginf=-9e99))


def activations(g, rows, cols, dtype):
    x = torch.randn(rows, cols, generator=g, device=DEV) * torch.exp(torch.randn(cols, generator=g, device=DEV))
    return (x * torch.exp2(torch.randint(-30, 30, (rows, 1), generator=g, device=DEV).float())).to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,stride,shift", [
    (1, 1, None, 0), (2, 31, None, 1), (3, 32, 35, 0), (5, 33, None, 3), (4, 15, 16, 0), (7, 16, 17, 1), (9, 17, None, 1),
    (64, 1280, None, 0), (33, 1283, 1290, 5), (1000, 48, None, 0)])
def test_pack_and_unpack(dtype, rows, cols, stride, shift):
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    _, x = rows_of(rows, cols, TYPES[dtype], stride, shift)
    x.copy_(activations(g, rows, cols, TYPES[dtype]))
    a, codes, b, scales = checkpoint(rows, cols, shift)
    z.zero_act8_pack(x, codes, scales)
    byte, want = act8_ref.pack_values(x)
    assert torch.equal(scales.cpu().long(), byte)
    same(act8_ref.unpack_values(codes, scales).to(DEV), want)
    assert bool((outside(a, codes) == 77).all()) and bool((outside(b, scales) == 77).all())
    for out in TYPES:
        buf, y = rows_of(rows, cols, TYPES[out], stride, shift)
        z.zero_act8_unpack(codes, scales, y)
        same(y, want.to(TYPES[out]))
        assert bool((outside(buf, y) == KEPT).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_pack_special_values(dtype):
    """Zeros, borders of the scale, ties, the smallest and the largest numbers, NaN and
    infinities."""
    t, info = TYPES[dtype], torch.finfo(TYPES[dtype])
    inf, nan = float("inf"), float("nan")
    rows = [[0.0] * 32, [-0.0] * 32, [448.0] + [1.0] * 31, [449.0] + [1.0] * 31, [-896.0, 897.0] * 16,
            [2.0 ** -127] * 32, [info.tiny] * 32, [info.max, -info.max, 1.0, 0.0] * 8, [info.max / 3] * 32,
            [nan] * 32, [inf, -inf, 1.0, nan] * 8, [inf] * 32, [nan, 3.0] * 16,
            [448.0 / 2.0 ** k for k in range(32)], [1.0 + k / 16.0 for k in range(32)],
            [448.0] + [(k + 0.5) * 2.0 ** -9 for k in range(31)], [2.0 ** -133 * k for k in range(32)],
            [448.0 * 2.0 ** -127] * 32, [450.0 * 2.0 ** -127] * 32]
    x = torch.tensor(rows, dtype=torch.float64).to(t).to(DEV)
    _, codes, _, scales = checkpoint(len(rows), 32)
    z.zero_act8_pack(x, codes, scales)
    byte, want = act8_ref.pack_values(x)
    assert torch.equal(scales.cpu().long(), byte)
    same(act8_ref.unpack_values(codes, scales).to(DEV), want)
    y = torch.empty(len(rows), 32, device=DEV)
    z.zero_act8_unpack(codes, scales, y)
    same(y, want.float())


def test_unpack_every_code_and_scale():
    codes = torch.arange(256, dtype=torch.int64).to(torch.uint8).repeat(256, 1).to(DEV)
    scales = torch.arange(256, dtype=torch.int64).to(torch.uint8)[:, None].repeat(1, 8).contiguous().to(DEV)
    want = act8_ref.unpack_values(codes, scales)
    for t in TYPES.values():
        y = torch.empty(256, 256, dtype=t, device=DEV)
        z.zero_act8_unpack(codes, scales, y)
        same(y, want.to(t))


def workspace(rows, out, cols):
    return torch.full((z.zero_act8_weight_grad_workspace_bytes(rows, out, cols),), 255, dtype=torch.uint8, device=DEV)


def whole_numbers(g, rows, out, cols, stride=None, shift=0):
    """d_y in -3 .. 3, x' in whole numbers up to 15 times 2^-2 .. 2: sums times 4 stay
    whole and below 2^24 for fewer than 2^24 / (3 * 120) rows."""
    _, d_y = rows_of(rows, out, torch.bfloat16, stride, shift, fill=float("nan"))
    d_y.copy_(torch.randint(-3, 4, (rows, out), generator=g, device=DEV))
    _, codes, _, scales = checkpoint(rows, cols, shift)
    table = act8_ref.code_values()
    whole = torch.tensor([c for c in range(256) if table[c] == table[c].round() and abs(table[c]) < 16], device=DEV)
    codes.copy_(whole[torch.randint(0, len(whole), (rows, cols), generator=g, device=DEV)])
    scales.copy_(torch.randint(125, 129, scales.shape, generator=g, device=DEV))
    return d_y, codes, scales


SIZES = [(1, 1, 1), (1, 64, 64), (2, 3, 5), (31, 16, 32), (33, 17, 33), (64, 128, 128), (65, 129, 127), (100, 256, 31),
         (127, 40, 300), (128, 130, 257), (257, 512, 96), (500, 72, 640), (1023, 384, 320), (2000, 33, 48),
         (4097, 129, 200)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,out,cols", SIZES)
def test_weight_grad_of_whole_numbers(dtype, rows, out, cols):
    g = torch.Generator(device=DEV).manual_seed(rows * 3 + out)
    for stride, shift, accumulate in ((None, 0, False), (out + 5, 3, True)):
        d_y, codes, scales = whole_numbers(g, rows, out, cols, stride, shift)
        want = d_y.double().T @ act8_ref.unpack_values(codes, scales).to(DEV)
        buf, d_w = rows_of(out, cols, TYPES[dtype], cols + 3 if shift else None, shift)
        if accumulate:
            base = torch.randint(-9, 10, (out, cols), generator=g, device=DEV)
            d_w.copy_(base)
            want = want + base
        z.zero_act8_weight_grad(d_y, codes, scales, d_w, accumulate=accumulate, workspace=workspace(rows, out, cols))
        same(d_w, want.to(TYPES[dtype]).cpu())
        assert bool((outside(buf, d_w) == KEPT).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,out,cols", [(70, 50, 90), (1000, 640, 200), (3000, 300, 520)])
def test_weight_grad(dtype, rows, out, cols):
    g = torch.Generator(device=DEV).manual_seed(rows)
    x = activations(g, rows, cols, torch.float32) * 2.0 ** -8
    _, codes, _, scales = checkpoint(rows, cols)
    z.zero_act8_pack(x, codes, scales)
    d_y = (torch.randn(rows, out, generator=g, device=DEV) * 1e-3).to(torch.bfloat16)
    d_w = torch.empty(out, cols, dtype=TYPES[dtype], device=DEV)
    z.zero_act8_weight_grad(d_y, codes, scales, d_w, workspace=workspace(rows, out, cols))
    v = act8_ref.unpack_values(codes, scales).to(DEV)
    want, size = d_y.double().T @ v, d_y.double().abs().T @ v.abs()
    err = rows * 2.0 ** -23 * size
    assert bool(((d_w.double() - want).abs() <= err + (want.abs() + err) * HALF[dtype]).all())
    # the same bits again
    again = torch.empty_like(d_w)
    z.zero_act8_weight_grad(d_y, codes, scales, again, workspace=workspace(rows, out, cols))
    assert torch.equal(d_w, again)


def test_weight_grad_scales_of_all_sizes():
    """One row: each product alone, for every code and scale bf16 holds exactly."""
    codes = torch.arange(256, dtype=torch.int64).to(torch.uint8).repeat(1, 32).to(DEV)   # 8192 columns
    for byte in range(10, 245, 9):
        scales = torch.full((1, 256), byte, dtype=torch.uint8, device=DEV)
        d_y = torch.tensor([[1.0, -0.5]], dtype=torch.bfloat16, device=DEV)
        d_w = torch.empty(2, 8192, device=DEV)
        z.zero_act8_weight_grad(d_y, codes, scales, d_w, workspace=workspace(1, 2, 8192))
        v = act8_ref.unpack_values(codes, scales)
        same(d_w, torch.cat([v, -0.5 * v]))


def test_weight_grad_nan():
    """A NaN reaches its column (a code, a block's scale) or its row (d_y), nothing else."""
    g = torch.Generator(device=DEV).manual_seed(3)
    d_y, codes, scales = whole_numbers(g, 200, 70, 150)
    codes[150, 37] = 0x7f
    scales[90, 3] = 255
    d_y[199, 11] = float("nan")
    d_w = torch.empty(70, 150, device=DEV)
    z.zero_act8_weight_grad(d_y, codes, scales, d_w, workspace=workspace(200, 70, 150))
    want = torch.zeros(70, 150, dtype=torch.bool, device=DEV)
    want[:, 37] = True
    want[:, 96:128] = True
    want[11] = True
    assert torch.equal(d_w.isnan(), want)


def test_weight_grad_no_rows():
    d_w = torch.full((5, 40), KEPT, dtype=torch.bfloat16, device=DEV)
    args = (torch.empty(0, 5, dtype=torch.bfloat16, device=DEV), torch.empty(0, 40, dtype=torch.uint8, device=DEV),
            torch.empty(0, 2, dtype=torch.uint8, device=DEV), d_w)
    z.zero_act8_weight_grad(*args, accumulate=True, workspace=workspace(0, 5, 40))
    assert bool((d_w == KEPT).all())
    z.zero_act8_weight_grad(*args, workspace=workspace(0, 5, 40))
    assert bool((d_w == 0).all())
    z.zero_act8_pack(torch.empty(0, 40, device=DEV), args[1], args[2])
    z.zero_act8_unpack(args[1], args[2], torch.empty(0, 40, device=DEV))


def test_graph_and_streams():
    g = torch.Generator(device=DEV).manual_seed(8)
    rows, out, cols = 1500, 200, 144
    x = torch.randn(rows, cols, generator=g, device=DEV).to(torch.bfloat16)
    d_y = torch.randn(rows, out, generator=g, device=DEV).to(torch.bfloat16)

    def buffers():
        _, codes, _, scales = checkpoint(rows, cols)
        return codes, scales, torch.empty_like(x), torch.empty(out, cols, device=DEV), workspace(rows, out, cols)

    def calls(codes, scales, y, d_w, ws):
        z.zero_act8_pack(x, codes, scales)
        z.zero_act8_unpack(codes, scales, y)
        z.zero_act8_weight_grad(d_y, codes, scales, d_w, workspace=ws)
        z.zero_act8_weight_grad(d_y, codes, scales, d_w, accumulate=True, workspace=ws)
    mine = buffers()
    calls(*mine)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(*mine)
    for turn in range(3):
        x.copy_(torch.randn(rows, cols, generator=g, device=DEV))
        d_y.copy_(torch.randn(rows, out, generator=g, device=DEV))
        other, side = buffers(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            calls(*other)
        torch.cuda.synchronize()
        for t in mine[2:4]:
            t.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(mine[:4], other[:4]):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """A checkpoint of more than 2^32 elements: its last rows."""
    rows, cols = (1 << 20) + 3, 4128
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[-2:] = torch.arange(cols, device=DEV).remainder(13)
    codes = torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
    scales = torch.empty(rows, cols // 32, dtype=torch.uint8, device=DEV)
    z.zero_act8_pack(x, codes, scales)
    y = torch.full_like(x, 3)
    z.zero_act8_unpack(codes, scales, y)
    assert torch.equal(x, y)
    d_y = torch.ones(rows, 1, dtype=torch.bfloat16, device=DEV)
    d_w = torch.empty(1, cols, device=DEV)
    z.zero_act8_weight_grad(d_y, codes, scales, d_w, workspace=workspace(rows, 1, cols))
    assert torch.equal(d_w[0], 2 * x[-1].float())


def test_more_rows_than_a_launch_holds():
    """Rows of one element take four threads each: more than 2^31 in all."""
    rows = 600_000_011
    x = torch.zeros(rows, 1, dtype=torch.bfloat16, device=DEV)
    at = [0, 1, (1 << 29) - 1, 1 << 29, rows - 2, rows - 1]
    x[at] = torch.tensor([3.0, -5.0, 7.0, 11.0, -13.0, 0.5], dtype=torch.bfloat16, device=DEV)[:, None]
    codes = torch.empty(rows, 1, dtype=torch.uint8, device=DEV)
    scales = torch.empty(rows, 1, dtype=torch.uint8, device=DEV)
    z.zero_act8_pack(x, codes, scales)
    y = torch.ones_like(x)
    z.zero_act8_unpack(codes, scales, y)
    assert torch.equal(y, x)


@pytest.mark.parametrize("rows,out,cols", [(65, 300, 5), (130, 8, 600), (64, 257, 16), (1, 1, 40), (15, 9, 1), (16, 2, 1),
                                           (7, 1, 40), (8, 1, 40), (1, 7, 40), (1, 8, 40), (200, 600, 17)])
def test_weight_grad_at_the_arrays_ends(rows, out, cols):
    """Few columns, so that a tile's chunks reach past many rows and the arrays' ends,
    in arrays that begin anywhere and end with their allocation."""
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    for shift in (0, 1, 2, 5):
        d_y, codes, scales = whole_numbers(g, rows, out, cols)
        a = torch.full((shift + d_y.numel(),), float("nan"), dtype=torch.bfloat16, device=DEV)
        b = torch.full((shift + codes.numel(),), 0x7f, dtype=torch.uint8, device=DEV)
        c = torch.full((shift + scales.numel(),), 255, dtype=torch.uint8, device=DEV)
        views = [t[shift:].view(s.shape) for t, s in ((a, d_y), (b, codes), (c, scales))]
        for v, s in zip(views, (d_y, codes, scales)):
            v.copy_(s)
        want = d_y.double().T @ act8_ref.unpack_values(codes, scales).to(DEV)
        d_w = torch.empty(out, cols, device=DEV)
        z.zero_act8_weight_grad(*views, d_w, workspace=workspace(rows, out, cols))
        same(d_w, want.float().cpu())


def test_weight_grad_no_rows_of_many_elements():
    """More than 2^32 elements of zeros."""
    n = 65600
    d_w = torch.ones(n, n, dtype=torch.bfloat16, device=DEV)
    empty = lambda cols, dtype: torch.empty(0, cols, dtype=dtype, device=DEV)
    z.zero_act8_weight_grad(empty(n, torch.bfloat16), empty(n, torch.uint8), empty(n // 32, torch.uint8), d_w)
    assert not any(bool(rows.any()) for rows in d_w.split(4096))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,out,cols", [(425, 4795, 6872), (355, 3561, 4716), (2050, 4100, 4200)])
def test_weight_grad_whole_and_shared_tiles(dtype, rows, out, cols):
    """Outputs of a little more than whole rounds of tiles: the last tiles' rows are
    shared by several workgroups, the others' are not."""
    g = torch.Generator(device=DEV).manual_seed(rows)
    for accumulate in (False, True):
        d_y, codes, scales = whole_numbers(g, rows, out, cols)
        want = d_y.double().T @ act8_ref.unpack_values(codes, scales).to(DEV)
        buf, d_w = rows_of(out, cols, TYPES[dtype], cols + 3 if accumulate else None, 0)
        if accumulate:
            base = torch.randint(-9, 10, (out, cols), generator=g, device=DEV)
            d_w.copy_(base)
            want = want + base
        ws = workspace(rows, out, cols)
        assert 0 < ws.numel() < 4 * out * cols   # the parts of some tiles only
        z.zero_act8_weight_grad(d_y, codes, scales, d_w, accumulate=accumulate, workspace=ws)
        same(d_w, want.to(TYPES[dtype]).cpu())
        assert bool((outside(buf, d_w) == KEPT).all())
