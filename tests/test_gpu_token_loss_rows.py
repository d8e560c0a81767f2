"""Token losses, on the GPU: rows with a NaN or +inf under a mask.  Definitions and
tolerances: test_gpu_token_loss.py."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import fsdp_sharded_optimizer_flat_amd as z  # noqa: E402
from gpu_common import DEV  # noqa: E402
from test_gpu_token_loss import DTYPES, MODES, check_distill, gen, make_logits, make_record, workspace  # noqa: E402

INF, NAN = math.inf, math.nan


# -- rows without a distribution, under a mask ---------------------------------------------------

MASKED = [(9, 3001), (300, 3001), (9, 40007), (9, 140001)]


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", MASKED)
def test_nan_among_the_listed_of_a_masked_row(rows, vocab, dtype):
    """A student whose allowed tokens are all in the record, one of them NaN (kind 1)
    or +inf (2): loss and the whole gradient row are NaN, or zero at a weight of
    zero.  A row of -inf alone (5) has gradient zero; finite neighbours, masked in
    the same way (4) or not, keep theirs."""
    k = 12
    x = make_logits(rows, vocab, dtype, 77)
    index, value = make_record(x, k, 1.0, 5)
    kinds = torch.arange(rows, device=DEV) % 6
    for r in range(rows):
        if r % 6 in (1, 2, 3, 4):            # all others are masked
            keep = x[r, index[r].long()].clone()
            x[r] = -INF
            x[r, index[r].long()] = keep
    hit = index[:, 3].long()
    for kind, v in ((1, NAN), (2, INF), (3, NAN)):
        at = torch.nonzero(kinds == kind)[:, 0]
        x[at, hit[at]] = v
    x[kinds == 5] = -INF
    dl = torch.rand(rows, generator=gen(4), device=DEV) + 0.5
    dl[kinds == 3] = 0.0
    ws, _ = workspace(x)
    for mode in MODES.values():
        loss, st = torch.full((rows,), 5.0, device=DEV), torch.empty(rows, 4, device=DEV)
        z.zero_distill(x, index, value, mode, loss=loss, stats=st, workspace=ws)
        for fused in (False, True):
            out, loss2 = torch.full_like(x, 9.0), loss
            if fused:
                loss2 = torch.full((rows,), 5.0, device=DEV)
                z.zero_distill_fused(x, index, value, mode, dl, out, loss=loss2, workspace=ws)
            else:
                z.zero_distill_grad(x, index, value, mode, st, dl, out)
            torch.cuda.synchronize()
            for kind in (1, 2, 3):
                assert bool(torch.isnan(loss2[kinds == kind]).all()), (mode, fused, kind, "loss")
            for kind in (1, 2):
                assert bool(torch.isnan(out[kinds == kind]).all()), (mode, fused, kind, "gradient")
            assert bool((loss2[kinds == 5] == INF).all())
            assert bool((out[(kinds == 3) | (kinds == 5)] == 0).all())
            f = (kinds == 0) | (kinds == 4)
            if mode == MODES["tail"]:        # a rest without a token: an infinite loss, finite gradients
                f = kinds == 0
                assert bool((loss2[kinds == 4] == INF).all())
                assert bool(torch.isfinite(out[kinds == 4]).all())
            check_distill(x[f], index[f], value[f], mode, 1.0, loss2[f], dl[f], out[f], f"fused {fused}")


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", MASKED)
def test_record_without_a_finite_value(rows, vocab, dtype):
    """Values of -inf only, renormalised: no distribution, so the loss and the
    gradient are zero -- but NaN over a row that holds a NaN or +inf, listed (1) or
    not (2)."""
    x = make_logits(rows, vocab, dtype, 78)
    index, value = make_record(x, 12, 1.0, 5)
    value.fill_(-INF)
    kinds = torch.arange(rows, device=DEV) % 4
    x[kinds == 1, 0] = NAN
    index[kinds == 1, 2] = 0
    x[kinds == 2, vocab - 1] = INF
    index[kinds == 2] = torch.where(index[kinds == 2] == vocab - 1, 1, index[kinds == 2])
    x[kinds == 3] = -INF
    dl = torch.rand(rows, generator=gen(4), device=DEV) + 0.5
    ws, _ = workspace(x)
    bad = (kinds == 1) | (kinds == 2)
    for fused in (False, True):
        loss, st, out = torch.full((rows,), 5.0, device=DEV), torch.empty(rows, 4, device=DEV), torch.full_like(x, 9.0)
        if fused:
            z.zero_distill_fused(x, index, value, MODES["renorm"], dl, out, loss=loss, workspace=ws)
        else:
            z.zero_distill(x, index, value, MODES["renorm"], loss=loss, stats=st, workspace=ws)
            z.zero_distill_grad(x, index, value, MODES["renorm"], st, dl, out)
        torch.cuda.synchronize()
        assert bool(torch.isnan(loss[bad]).all()) and bool((loss[~bad] == 0).all()), fused
        assert bool(torch.isnan(out[bad]).all()) and bool((out[~bad] == 0).all()), fused
