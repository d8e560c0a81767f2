"""The embedding lookup and its gradient on the GPU against sums in binary64.

Tolerances: a lookup is one binary32 product (2^-24 of its value) rounded to its
type (2^-8 for bf16).  A gradient row adds n rows in binary32: (n - 1) 2^-24 times
the sum of magnitudes, one product with the scale, one rounding to the table's
type; accumulated, one binary32 addition more."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
z = pytest.importorskip("fsdp_sharded_optimizer_flat_amd")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U32 = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
KEPT = 5.5


def rows_of(n, cols, dtype, stride=None, shift=0, fill=KEPT):
    """(n, cols) with the given row stride, `shift` elements into its allocation."""
    stride = stride or cols
    buf = torch.full((shift + max(n, 1) * stride + 16,), fill, dtype=dtype, device=DEV)
    return buf, buf[shift:shift + n * stride].view(n, stride)[:, :cols]


def workspace(rows, vocab, hidden):
    return torch.full((z.zero_embedding_grad_workspace_bytes(rows, vocab, hidden),), 255, dtype=torch.uint8,
                      device=DEV)


def outside(buf, view):
    """The elements of an allocation that a view does not show."""
    on = torch.zeros(buf.numel(), dtype=torch.bool, device=DEV)
    on.as_strided(view.shape, view.stride(), view.storage_offset())[...] = True
    return buf[~on]


@pytest.mark.parametrize("src", TYPES)
@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("rows,hidden,vocab,stride,shift", [
    (1, 1, 1, None, 0), (3, 7, 11, None, 1), (5, 8, 4, 13, 3), (64, 1280, 1000, None, 0), (9, 1283, 50, 1300, 5),
    (1000, 65, 77, 65, 1), (2, 4096, 128256, None, 0)])
def test_lookup(src, dst, rows, hidden, vocab, stride, shift):
    g = torch.Generator(device=DEV).manual_seed(rows + hidden)
    _, table = rows_of(vocab, hidden, TYPES[src], stride, shift)
    table.copy_(torch.randn(vocab, hidden, generator=g, device=DEV))
    buf, out = rows_of(rows, hidden, TYPES[dst], stride and stride + 2, shift)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    if rows > 4:
        tokens[1], tokens[3] = -1, vocab
    for scale in (1.0, -35.77):
        z.zero_embedding(table, tokens, out, scale=scale)
        want = table[tokens.clamp(0, vocab - 1)].double() * float(np.float32(scale))
        got = out.double()
        if rows > 4:
            assert bool((got[1] == 0).all()) and bool(got[3].isnan().all())
            want[1], got[1], want[3], got[3] = 0, 0, 0, 0
        assert bool(((got - want).abs() <= want.abs() * (HALF[dst] + U32) * (1 + U32)).all())
        assert bool((outside(buf, out) == KEPT).all())


def reference(d_out, tokens, vocab, scale):
    """Sums, sums of magnitudes and counts in binary64."""
    ok = (tokens >= 0) & (tokens < vocab)
    t, x = tokens[ok].cpu(), d_out[ok].double().cpu()
    s = torch.zeros(vocab, d_out.shape[1], dtype=torch.float64).index_add_(0, t, x)
    m = torch.zeros_like(s).index_add_(0, t, x.abs())
    n = torch.bincount(t, minlength=vocab)[:, None]
    f = float(np.float32(scale))
    return (s * f).to(DEV), (m * abs(f)).to(DEV), n.to(DEV)


def check_grad(got, base, want, mags, count, dst):
    got = got.double()
    err = count * U32 * mags + want.abs() * U32
    if base is not None:
        want = want + base.double()
        err = torch.where(count > 0, err + (want.abs() + err) * U32, torch.zeros_like(err))
    tol = err + (want.abs() + err) * HALF[dst] + 2.0 ** -134
    if base is not None:
        assert torch.equal(torch.where(count > 0, 0.0, got), torch.where(count > 0, 0.0, base.double()))
    bad = (got - want).abs() > tol
    assert not bool(bad.any()), (bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())


def token_sets(g, rows, vocab):
    u = torch.rand(rows, generator=g, device=DEV, dtype=torch.float64)
    text = (torch.exp(u * float(np.log(vocab + 1.0))).long() - 1).clamp(0, vocab - 1)
    mixed = torch.randint(-3, vocab + 3, (rows,), generator=g, device=DEV)
    one = torch.full((rows,), vocab - 1, device=DEV)
    none = torch.full((rows,), -1, device=DEV)
    distinct = torch.arange(rows - 1, -1, -1, device=DEV) % vocab
    huge = mixed.clone()
    huge[::2] = (1 << 40) + 1
    return dict(text=text, mixed=mixed, one=one, none=none, distinct=distinct, huge=huge)


@pytest.mark.parametrize("src", TYPES)
@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("rows,hidden,vocab,stride,shift", [
    (1, 1, 1, None, 0), (2, 3, 5, 7, 1), (31, 8, 40, None, 0), (33, 9, 2, None, 3), (64, 40, 300, 41, 1),
    (500, 513, 129, None, 1), (1024, 1280, 600, None, 0), (1025, 72, 128, 80, 0)])
def test_grad(src, dst, rows, hidden, vocab, stride, shift):
    g = torch.Generator(device=DEV).manual_seed(rows * 7 + hidden)
    _, d_out = rows_of(rows, hidden, TYPES[src], stride, shift)
    d_out.copy_(torch.randn(rows, hidden, generator=g, device=DEV))
    for name, tokens in token_sets(g, rows, vocab).items():
        for accumulate, scale in ((False, 1.0), (True, 35.77)):
            buf, d_table = rows_of(vocab, hidden, TYPES[dst], stride and stride + 3, shift)
            if accumulate:
                d_table.copy_(torch.randn(vocab, hidden, generator=g, device=DEV))
            base = d_table.clone()
            z.zero_embedding_grad(d_out, tokens, d_table, scale=scale, accumulate=accumulate,
                                  workspace=workspace(rows, vocab, hidden))
            check_grad(d_table, base if accumulate else None, *reference(d_out, tokens, vocab, scale), dst)
            assert bool((outside(buf, d_table) == KEPT).all()), name


@pytest.mark.parametrize("rows,hidden,vocab", [(8191, 24, 50304), (8192, 16, 999), (8193, 16, 1 << 20),
                                               (16385, 33, 128256), (70001, 8, 2000), (40000, 520, 3)])
def test_grad_of_many_tokens(rows, hidden, vocab):
    """Lists of one, two and more sorted chunks; sums of whole numbers are exact, so
    every element has to be equal, whatever the order."""
    g = torch.Generator(device=DEV).manual_seed(rows)
    d_out = torch.randint(-3, 4, (rows, hidden), generator=g, device=DEV).to(torch.bfloat16)
    ws = workspace(rows, vocab, hidden)
    for name, tokens in token_sets(g, rows, vocab).items():
        d_table = torch.full((vocab, hidden), KEPT, device=DEV)
        z.zero_embedding_grad(d_out, tokens, d_table, workspace=ws)
        ok = (tokens >= 0) & (tokens < vocab)
        want = torch.zeros(vocab, hidden, dtype=torch.float64)
        want.index_add_(0, tokens[ok].cpu(), d_out[ok].double().cpu())
        assert torch.equal(d_table.double().cpu(), want), name


@pytest.mark.parametrize("hidden", [1, 3, 7, 8, 9, 15, 511, 512, 513, 520, 1025])
@pytest.mark.parametrize("dst", TYPES)
def test_grad_of_runs_over_many_segments(dst, hidden):
    """Runs that many segments share, in rows of fewer than eight columns and around a
    wave's 512; whole numbers, so every element has to be equal."""
    g = torch.Generator(device=DEV).manual_seed(hidden)
    rows, vocab = 700, 4
    for accumulate in (False, True):
        tokens = torch.randint(-1, vocab - 1, (rows,), generator=g, device=DEV)
        d_out = torch.randint(-2, 3, (rows, hidden), generator=g, device=DEV).to(torch.bfloat16)
        buf, d_table = rows_of(vocab, hidden, TYPES[dst], hidden + 1, 1)
        d_table.copy_(torch.randint(-8, 9, (vocab, hidden), generator=g, device=DEV))
        want = d_table.double().cpu() if accumulate else torch.zeros(vocab, hidden, dtype=torch.float64)
        ok = tokens >= 0
        want.index_add_(0, tokens[ok].cpu(), d_out[ok].double().cpu())
        z.zero_embedding_grad(d_out, tokens, d_table, accumulate=accumulate, workspace=workspace(rows, vocab, hidden))
        # sums of at most 700 * 2 + 8 < 2^11: bf16 rounds those beyond 2^8
        assert torch.equal(d_table.cpu(), want.to(TYPES[dst]))
        assert bool((outside(buf, d_table) == KEPT).all())


def test_grad_of_the_most_rows():
    """ZERO_MAX_EMBEDDING_ROWS rows: the most sorted chunks that are put together."""
    rows, vocab, hidden = z.ZERO_MAX_EMBEDDING_ROWS, 5003, 2
    g = torch.Generator(device=DEV).manual_seed(6)
    d_out = torch.randint(-2, 3, (rows, hidden), generator=g, device=DEV).to(torch.bfloat16)
    for name in ("text", "mixed", "one"):
        tokens = token_sets(g, rows, vocab)[name]
        d_table = torch.empty(vocab, hidden, device=DEV)
        z.zero_embedding_grad(d_out, tokens, d_table, workspace=workspace(rows, vocab, hidden))
        ok = (tokens >= 0) & (tokens < vocab)
        want = torch.zeros(vocab, hidden, dtype=torch.float64).index_add_(0, tokens[ok].cpu(), d_out[ok].double().cpu())
        assert torch.equal(d_table.double().cpu(), want), name


def test_lookup_of_more_rows_than_a_launch_holds():
    rows, hidden = (1 << 30) + 5, 9      # two threads a row
    table = torch.arange(3 * hidden, device=DEV).view(3, hidden).to(torch.bfloat16)
    tokens = torch.zeros(rows, dtype=torch.int64, device=DEV)
    ends = [0, 1, (1 << 30) - 1, 1 << 30, rows - 1]
    tokens[ends] = torch.tensor([1, 2, 1, 2, 1], device=DEV)
    out = torch.empty(rows, hidden, dtype=torch.bfloat16, device=DEV)
    z.zero_embedding(table, tokens, out)
    assert torch.equal(out[ends], table[tokens[ends]])
    assert torch.equal(out[12345::1 << 20], table[:1].expand(len(range(12345, rows, 1 << 20)), hidden))


def test_grad_orders_equal_tokens_by_row():
    """A token's rows are added from the first to the last: 2^24 + 1 rounds to 2^24
    (ties to even), while 1 - 2^24 is a binary32 number."""
    rows = 20
    for a, b, want in ((2.0 ** 24, 1.0, 0.0), (-2.0 ** 24, 1.0, 1.0)):
        x = torch.zeros(rows, 4, device=DEV)
        x[3], x[7], x[15] = a, b, -a
        tokens = torch.full((rows,), 2, device=DEV)
        tokens[10] = 1
        d = torch.empty(5, 4, device=DEV)
        z.zero_embedding_grad(x, tokens, d, workspace=workspace(rows, 5, 4))
        assert bool((d[2] == want).all())
        x[15], x[3] = b, a
        x[7] = -a
        z.zero_embedding_grad(x, tokens, d, workspace=workspace(rows, 5, 4))
        assert bool((d[2] == b).all())


def test_grad_same_bits_and_no_rows():
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(20000, 136, generator=g, device=DEV)
    tokens = token_sets(g, 20000, 500)["text"]
    ws = workspace(20000, 500, 136)
    first = torch.empty(500, 136, device=DEV)
    z.zero_embedding_grad(x, tokens, first, workspace=ws)
    for _ in range(3):
        again = torch.empty_like(first)
        z.zero_embedding_grad(x, tokens, again, workspace=ws)
        assert torch.equal(first, again)
    none = torch.full((7, 9), KEPT, device=DEV)
    z.zero_embedding_grad(x[:0, :9], tokens[:0], none, accumulate=True)
    assert bool((none == KEPT).all())
    z.zero_embedding_grad(x[:0, :9], tokens[:0], none)
    assert bool((none == 0).all())
    z.zero_embedding(first, tokens[:0], first[:0].clone())


def test_grad_nan_rows():
    """NaN and infinities stay in their token's row and columns."""
    x = torch.ones(100, 20, device=DEV)
    tokens = torch.arange(100, device=DEV) % 10
    x[13, 4], x[25, 6] = float("nan"), float("inf")
    tokens[50] = -1
    x[50] = float("nan")
    d = torch.empty(12, 20, device=DEV)
    z.zero_embedding_grad(x, tokens, d, workspace=workspace(100, 12, 20))
    bad = ~torch.isfinite(d)
    assert bad.nonzero().tolist() == [[3, 4], [5, 6]]
    assert d[0, 0] == 9 and bool((d[1, :4] == 10).all()) and bool((d[10:] == 0).all())


def test_grad_is_the_lookups():
    """<d_out, lookup(W + h E) - lookup(W - h E)> / 2h = <d_table, E>, in whole numbers."""
    g = torch.Generator(device=DEV).manual_seed(9)
    i = lambda *s: torch.randint(-4, 5, s, generator=g, device=DEV).float()
    W, E, d_out = i(30, 18), i(30, 18), i(200, 18)
    tokens = torch.randint(-1, 30, (200,), generator=g, device=DEV)
    up, down, d = torch.empty_like(d_out), torch.empty_like(d_out), torch.empty_like(W)
    z.zero_embedding(W + E, tokens, up, scale=2.0)
    z.zero_embedding(W - E, tokens, down, scale=2.0)
    z.zero_embedding_grad(d_out, tokens, d, scale=2.0, workspace=workspace(200, 30, 18))
    assert float((d_out * (up - down)).sum()) / 2 == float((d * E).sum())


def test_graph_and_streams():
    g = torch.Generator(device=DEV).manual_seed(5)
    rows, hidden, vocab = 9000, 40, 700
    W = torch.randn(vocab, hidden, generator=g, device=DEV)
    x = torch.randn(rows, hidden, generator=g, device=DEV).to(torch.bfloat16)
    tokens = token_sets(g, rows, vocab)["text"]
    out, d = torch.empty(rows, hidden, device=DEV), torch.empty(vocab, hidden, device=DEV)
    ws = workspace(rows, vocab, hidden)

    def calls(out, d, ws):
        z.zero_embedding(W, tokens, out)
        z.zero_embedding_grad(x, tokens, d, workspace=ws)
    calls(out, d, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(out, d, ws)
    for turn in range(3):
        x.copy_(torch.randn(rows, hidden, generator=g, device=DEV))
        tokens.copy_(token_sets(g, rows, vocab)["mixed" if turn % 2 else "text"].clamp(max=vocab - 1))
        out2, d2 = torch.empty_like(out), torch.empty_like(d)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            calls(out2, d2, workspace(rows, vocab, hidden))
        torch.cuda.synchronize()
        out.fill_(1)
        d.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, out2) and torch.equal(d, d2)


def test_offsets_past_32_bits():
    """A table whose last rows lie beyond 2^32 bytes (and 2^31 elements)."""
    vocab, hidden = (1 << 20) - 5, 2051
    table = torch.empty(vocab, hidden, dtype=torch.bfloat16, device=DEV)
    tokens = torch.tensor([vocab - 1, 3, vocab - 1, vocab - 2], device=DEV)
    x = torch.arange(4 * hidden, device=DEV).remainder(7).view(4, hidden).to(torch.bfloat16)
    z.zero_embedding_grad(x, tokens, table, workspace=workspace(4, vocab, hidden))
    assert torch.equal(table[vocab - 1], x[0] + x[2]) and torch.equal(table[vocab - 2], x[3])
    assert torch.equal(table[3], x[1]) and int((table != 0).any(1).sum()) == 3
    out = torch.empty(4, hidden, dtype=torch.bfloat16, device=DEV)
    z.zero_embedding(table, tokens, out)
    assert torch.equal(out, table[tokens])


@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("rows,hidden,vocab,gap", [(1, 1280, 128001, 0), (3000, 701, 120011, 3), (2049, 8200, 23000, 0),
                                                   (20000, 64, 1 << 20, 5), (2500, 5, 1 << 20, 500), (700, 2, 1 << 20, 150)])
def test_grad_of_a_large_table(dst, rows, hidden, vocab, gap):
    """Tables cleared by many workgroups, as one run of elements or row by row (gaps), that
    begin at and off 16 bytes and hold NaN before: whole numbers, so that every sum is exact,
    tokens at both ends of the table, in neighbouring rows and many times."""
    g = torch.Generator(device=DEV).manual_seed(rows + hidden)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    tokens[rows // 2:] = vocab - 1 - torch.arange(rows - rows // 2, device=DEV) // 2
    if rows > 100:
        tokens[:40] = vocab - 700
        tokens[40:44] = torch.tensor([0, -1, vocab, vocab + 9], device=DEV)
    x = torch.randint(-3, 4, (rows, hidden), generator=g, device=DEV).to(torch.bfloat16)
    buf, d_table = rows_of(vocab, hidden, TYPES[dst], hidden + gap, 1 if gap else 0)
    d_table.fill_(float("nan"))
    ok = (tokens >= 0) & (tokens < vocab)
    named, which = tokens[ok].unique(return_inverse=True)
    want = torch.zeros(named.numel(), hidden, device=DEV).index_add_(0, which, x[ok].float())
    ws = workspace(rows, vocab, hidden)
    for _ in range(2):
        z.zero_embedding_grad(x, tokens, d_table, workspace=ws)
        assert torch.equal(d_table[named], want.to(TYPES[dst]))
        others = torch.ones(vocab, dtype=torch.bool, device=DEV)
        others[named] = False
        for part, on in zip(d_table.split(1 << 15), others.split(1 << 15)):
            assert bool((part[on] == 0).all())
        if gap:
            assert bool((outside(buf, d_table) == KEPT).all())
        d_table[:, :].fill_(float("nan"))
