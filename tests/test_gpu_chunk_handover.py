"""Row tiles of few rows that both softmax warpgroups share (heads of 64, long
contexts), directly before row tiles that the second warpgroup has to itself:
what the second hands to the first has to last until the first has read it.

The batch is made of equal periods, as many for each SM, so that each CTA's run
of row tiles is whole periods: a long single token, then one or two requests of
more rows than a warp holds, which the warpgroups take in turn.  Those may see
nothing, so that their output follows at once.  Tolerances are test_gpu_chunk's;
the definition is formed here, in binary64, for all periods at once."""
import numpy as np
import pytest
import torch

from test_gpu_chunk import BF16, DEV, E4M3, F16, Case, _values

pytestmark = pytest.mark.gpu
PERIODS = 4                                    # of a CTA: each warpgroup's turn comes up twice


def _batch(period, hq, dtype, cache):
    sms = min(torch.cuda.get_device_properties(0).multi_processor_count, 152)
    n = PERIODS * sms
    c = Case(period, hq, 1, 64, 64, dtype, cache, seed=30)
    # one period's pages for all: their queries differ
    rows = sum(new for new, _ in period)
    c.q = _values((rows * n, hq, 64), dtype, torch.Generator(device=DEV).manual_seed(31))
    c.rows, c.period = rows, [int(x) for x in c.ctx]
    c.tables, c.ctx = c.tables.repeat(n, 1), c.ctx.repeat(n)
    starts = [0]
    for new, _ in period * n:
        starts.append(starts[-1] + new)
    c.starts = torch.tensor(starts, dtype=torch.int32, device=DEV)
    return c


def _definition(c, period):
    q = c.q.double().view(-1, c.rows, *c.q.shape[1:])              # [periods, rows, heads, 64]
    r = {"out": torch.zeros_like(q), "spread": torch.zeros_like(q),
         "lse": torch.full(q.shape[:3], -torch.inf, dtype=torch.float64, device=DEV),
         "mag": torch.zeros(q.shape[:3], dtype=torch.float64, device=DEV),
         "seen": torch.zeros(q.shape[:2], dtype=torch.int64, device=DEV)}
    row = 0
    for b, (n, old) in enumerate(period):
        at = [x[c.tables[b].long()].flatten(0, 1)[:, 0].float().double() for x in (c.k, c.v)]
        k, v = at if c.k_scale is None else (at[0] * c.k_scale.double(), at[1] * c.v_scale.double())
        for j in range(n):
            hi = max(old + j + 1, 0)
            if hi > 0:
                x, kk, vv = q[:, row], k[:hi], v[:hi]
                z = c.scale * (x @ kk.T)
                r["lse"][:, row] = torch.logsumexp(z, -1)
                p = torch.softmax(z, -1)
                r["out"][:, row], r["spread"][:, row] = p @ vv, p @ vv.abs()
                r["mag"][:, row] = (c.scale * (x.abs() @ kk.abs().T)).amax(-1)
                r["seen"][:, row] = hi
            row += 1
    r = {name: x.flatten(0, 1).cpu().numpy() for name, x in r.items()}
    r["mine"] = np.ones(len(r["seen"]), dtype=bool)
    return r


@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, BF16), (F16, E4M3)])
@pytest.mark.parametrize("period,hq", [
    ([(1, 2047), (5, -5)], 16),                # 80 rows that see nothing, the turns in turn
    ([(1, 1535), (20, -20), (20, -20)], 4),    # in every period one of each warpgroup
    ([(1, 1536), (5, 0)], 16), ([(1, 1700), (20, 280)], 4)])
def test_second_warpgroups_rows_last_until_read(period, hq, dtype, cache):
    c = _batch(period, hq, dtype, cache)
    # (fewer entries than new tokens: the request's context is 0)
    assert c.period == [n + old for n, old in period]
    out, lse, err = c.run()
    c.check(out, lse, _definition(c, period))
    assert int(err) == 0
    for _ in range(40):
        again, lse2, _ = c.run()
        assert torch.equal(again, out) and torch.equal(lse2, lse)
