"""A token-loss workspace serves every call on its rows: each entry point and
every number of alternatives up to the one it was asked for.  CPU only (a call
on addresses that overlap is refused after the workspace's size is checked, so
nothing runs)."""
import pytest

z = pytest.importorskip("fsdp_sharded_optimizer_flat_amd")

BASE = 1 << 40


@pytest.mark.parametrize("rows", [1, 2, 3, 17, 64, 257, 300, 1023, 1024, 5000])
@pytest.mark.parametrize("vocab", [1, 5003, 50304, 65537, 70001, 128256, 262145, 1 << 20])
def test_fewer_alternatives_fit_too(rows, vocab):
    bytes_of = [z.zero_loss_workspace_bytes(rows, vocab, k) for k in range(z.ZERO_MAX_TOP + 1)]
    assert bytes_of == sorted(bytes_of)


@pytest.mark.parametrize("rows,vocab,asked", [(1, 1 << 20, 256), (1, 128256, 17), (3, 70001, 17), (300, 1 << 20, 40)])
def test_calls_accept_it(rows, vocab, asked):
    lib = z.raw_library()
    have = z.zero_loss_workspace_bytes(rows, vocab, asked)
    logits, tokens, out = BASE, BASE + (1 << 38), BASE + (1 << 39)
    for k in range(asked + 1):
        top = [out + (1 << 30), out + (1 << 31)] if k else [None, None]
        # the workspace begins inside the logits: EINVAL, where one too small is ENOSPC before that
        got = lib.zero_logprob(logits, z.ZERO_BF16, rows, vocab, vocab, 1.0, tokens, out, None, None, k, *top,
                               logits + 16, have, None)
        assert got == z.ZERO_EINVAL, k
