"""The weight gradient of 8-bit checkpoints where rows of both factors are whole
16-byte chunks at 16-byte addresses, which are read through buffer windows: outputs of
tiles of 256 and of 128, whole and with shared last tiles, added to what is there, with
gaps between the rows of d_y, and rows that end inside a tile.

Behind each factor's last row, and in the gaps of d_y, lie 200 rows of NaN in the same
allocation (more than any tile reaches), so a window that let one of them through would
show.  Whole numbers whose sums stay below 2^24 are exact in binary32 in any order, so
every element has to be equal."""
import pytest

torch = pytest.importorskip("torch")
z = pytest.importorskip("fsdp_sharded_optimizer_flat_amd")
pytestmark = pytest.mark.gpu

import act8_ref  # noqa: E402

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BEHIND, KEPT = 200, 5.5


def rows_before(rows, cols, dtype, fill, stride=None):
    """(rows, cols) at the beginning of an allocation that holds `fill` elsewhere."""
    stride = stride or cols
    return torch.full(((rows + BEHIND) * stride,), fill, dtype=dtype, device=DEV).view(-1, stride)[:rows, :cols]


def factors(g, rows, out, cols, gap):
    """d_y in -3 .. 3, x' in whole numbers up to 15 times 2^-2 .. 2."""
    d_y = rows_before(rows, out, torch.bfloat16, float("nan"), out + gap)
    d_y.copy_(torch.randint(-3, 4, (rows, out), generator=g, device=DEV))
    table = act8_ref.code_values()
    whole = torch.tensor([c for c in range(256) if table[c] == table[c].round() and abs(table[c]) < 16], device=DEV)
    codes = rows_before(rows, cols, torch.uint8, 0x7f)
    codes.copy_(whole[torch.randint(0, len(whole), (rows, cols), generator=g, device=DEV)])
    scales = rows_before(rows, -(-cols // 32), torch.uint8, 255)
    scales.copy_(torch.randint(125, 129, scales.shape, generator=g, device=DEV))
    assert d_y.data_ptr() % 16 == codes.data_ptr() % 16 == 0 and out % 8 == gap % 8 == cols % 16 == 0
    return d_y, codes, scales


def values(codes, scales):
    """act8_ref.unpack_values on the device: whole numbers times powers of two."""
    v = act8_ref.code_values().to(DEV)[codes.int()]
    return v * torch.exp2(scales.double() - 127.0).repeat_interleave(32, 1)[:, :codes.shape[1]]


def parts(rows, out, cols):
    """The workspace in tiles of 256, and whether tiles of 128 could need as much."""
    n = z.zero_act8_weight_grad_workspace_bytes(rows, out, cols)
    steps = -(-rows // 64)

    def may_be(tile, together):
        tiles = -(-out // tile) * -(-cols // tile)
        return any(n == s * t * tile * tile * 4 for s in range(2, steps + 1) for t in (tiles, tiles % together))
    return n, may_be(256, 256), may_be(128, 512)


def check(dtype, rows, out, cols, gap, accumulate):
    g = torch.Generator(device=DEV).manual_seed(rows + out + cols)
    d_y, codes, scales = factors(g, rows, out, cols, gap)
    want = d_y.double().t().contiguous() @ values(codes, scales)
    buf = torch.full((out, cols + 3), KEPT, dtype=TYPES[dtype], device=DEV)
    d_w = buf[:, :cols] if accumulate else torch.full((out, cols), float("nan"), dtype=TYPES[dtype], device=DEV)
    if accumulate:
        base = torch.randint(-9, 10, (out, cols), generator=g, device=DEV)
        d_w.copy_(base)
        want += base
    ws = torch.full((z.zero_act8_weight_grad_workspace_bytes(rows, out, cols),), 255, dtype=torch.uint8, device=DEV)
    z.zero_act8_weight_grad(d_y, codes, scales, d_w, accumulate=accumulate, workspace=ws)
    assert torch.equal(d_w, want.to(TYPES[dtype]))
    assert bool((buf[:, cols:] == KEPT).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gap,accumulate", [(0, False), (8, True)])
@pytest.mark.parametrize("rows,out,cols", [(64, 128, 128), (65, 264, 272), (79, 128, 48), (81, 136, 144), (95, 8, 400),
                                           (97, 512, 16), (257, 512, 96), (1023, 384, 320), (2017, 40, 1040),
                                           (4129, 136, 208)])
def test_small_tiles(dtype, rows, out, cols, gap, accumulate):
    check(dtype, rows, out, cols, gap, accumulate)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gap,accumulate", [(0, False), (16, True)])
@pytest.mark.parametrize("rows", [2000, 2017, 2049, 2063, 2081])
def test_large_tiles(dtype, rows, gap, accumulate):
    """4096 x 4096: 256 whole tiles of 256, one to a compute unit."""
    assert z.zero_act8_weight_grad_workspace_bytes(rows, 4096, 4096) == 0
    check(dtype, rows, 4096, 4096, gap, accumulate)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gap,accumulate", [(0, False), (8, True)])
@pytest.mark.parametrize("rows,out,cols", [(3011, 4104, 4880), (4113, 4872, 4112), (4127, 4360, 8208), (8191, 4104, 4112)])
def test_large_tiles_whole_and_shared(dtype, rows, out, cols, gap, accumulate):
    n, of_256, of_128 = parts(rows, out, cols)
    assert of_256 and not of_128 and 0 < n < 4 * out * cols, n
    check(dtype, rows, out, cols, gap, accumulate)


@pytest.mark.parametrize("out", [5, 8])
def test_scales_below_the_normal_range(out):
    """One row: each product alone.  Values below bf16's normal range are rounded to its
    steps of 2^-133; by the general path (5) and through windows (8)."""
    codes = torch.arange(256, dtype=torch.int64).to(torch.uint8).repeat(1, 32).to(DEV)
    d_y = torch.tensor([[1.0, -0.5, 2.0 ** 20, 2.0 ** -126, 2.0 ** -130, 3.0, 1.0, 1.0][:out]], dtype=torch.bfloat16,
                       device=DEV)
    ws = torch.empty(z.zero_act8_weight_grad_workspace_bytes(1, out, 8192), dtype=torch.uint8, device=DEV)
    for byte in range(16):
        scales = torch.full((1, 256), byte, dtype=torch.uint8, device=DEV)
        d_w = torch.empty(out, 8192, device=DEV)
        z.zero_act8_weight_grad(d_y, codes, scales, d_w, workspace=ws)
        x = act8_ref.unpack_values(codes, scales).to(torch.bfloat16).double()
        want = (d_y[0, :, None].double().cpu() * x).float()
        got = d_w.cpu()
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num()), byte
