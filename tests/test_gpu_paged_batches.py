"""What a batch's arrays may say: rows behind the last sequence, and starts that are out of order."""

import math

import pytest
import torch

from speculative_decoding_draft_kv_gb300 import paged as P
from tests.paged_oracle import World

pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("fmt,dtype", [("f16", "f16"), ("bf16", "bf16"), ("int8", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("lens", [[(3, 40), (1, 90)], [(40, 300), (5, 5)]])
def test_what_rows_behind_the_batch_hold_changes_nothing(fmt, dtype, lens):
    w = World(lens, fmt=fmt, dtype=dtype, spare_rows=37, seed=41)
    cache, batch = w.handles(P)
    rope, norm = P.PagedRope(w.dim, 1e6), torch.rand(w.dim, generator=w.g, device="cuda") + 0.5
    q, k, v = w.randn(w.heads), w.randn(w.kv_heads), w.randn(w.kv_heads)
    # the batch's own places written once, so that only what the calls below write can differ
    P.paged_append(cache, batch, k, v, rope=rope, k_norm=norm)
    pools = [t for t in (w.k, w.v, w.ks, w.vs) if t is not None]
    results = []
    for behind in (0.0, math.nan, math.inf, -3e4):
        for x in (q, k, v):
            x[w.total:] = behind
        qo, o, kr, vr = torch.full_like(q, 7.0), torch.full_like(q, 7.0), torch.full_like(k, 7.0), torch.full_like(v, 7.0)
        lse = torch.full((w.rows, w.heads), 7.0, device="cuda")
        P.paged_append(cache, batch, k, v, rope=rope, k_norm=norm, q=q, q_norm=norm, q_out=qo)
        P.paged_gather(cache, batch, kr, vr)
        P.paged_attend(cache, batch, q, o, lse=lse)
        assert P.paged_device_error() == 0
        for x in (qo, o, kr, vr, lse):
            assert (x[w.total:] == 7.0).all()
        results.append([x.clone() for x in [qo, o, kr, vr, lse] + pools])
    for other in results[1:]:
        assert all(same(a, b) for a, b in zip(results[0], other))


@pytest.mark.parametrize("starts", [[0, 5, 3, 8], [5, 0, 8, 8], [0, 8, 7, 7]])
@pytest.mark.parametrize("many", [0, 40])
def test_starts_that_decrease_stay_within_the_block_table(starts, many):
    """Reported by the attention; whatever the others make of them, they touch no page that the table
    does not name, and no row behind the tensor's."""
    w = World([(3, 40)] * 3 + [(0, 20)] * many, seed=42)
    w.q_start[:4] = torch.tensor(starts, dtype=torch.int32)
    w.q_start[4:] = starts[3]
    cache, batch = w.handles(P, max_q=8)
    q, k, v = w.randn(w.heads), w.randn(w.kv_heads), w.randn(w.kv_heads)
    before, qo = w.k.clone(), torch.full_like(q, 7.0)
    P.paged_append(cache, batch, k, v, rope=P.PagedRope(128), q=q, q_out=qo)
    named = torch.zeros(w.n_pages, dtype=torch.bool, device="cuda")
    named[w.pages[w.pages >= 0].long()] = True
    assert not named.all() and same(before[~named].contiguous(), w.k[~named].contiguous())
    kr, vr = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    P.paged_gather(cache, batch, kr, vr)
    P.paged_device_error()
    o = torch.full_like(q, 7.0)
    P.paged_attend(cache, batch, q, o)
    assert P.paged_device_error() == P.PAGED_ERR_PAGE
