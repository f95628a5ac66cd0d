"""The ring's attention reads each stage of shared memory before the next copy may overwrite it: the same call gives the same bits, by
itself and beside other work, with clusters and with several CTAs on an SM, from either slot format."""

import pytest
import torch

import synth
from tests.ring_harness import GpuRun

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("number,kw", [(2, {}), (2, {"tiles_per_split": 4}), (4, {}), (2, {"kv_format": "q8_0"})], ids=str)
@pytest.mark.parametrize("kind", ["full", "swa"])
def test_the_same_call_gives_the_same_bits(number, kw, kind):
    w = synth.workload(number)
    run = GpuRun(w, swa_window=2048, **kw)
    try:
        for committed in synth.commit_schedule(w, 2)[:2]:
            run.begin_step(committed)
        q, kn, vn = run.inputs(1, 0, run.dev)
        noise, other = torch.ones(1 << 26, device="cuda"), torch.cuda.Stream()
        outs = [torch.empty_like(q) for _ in range(40)]
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            if i % 2:
                with torch.cuda.stream(other):
                    noise.mul_(1.0)
            run.ring.attend(0, kind, q, kn, vn, o)
        torch.cuda.synchronize()
        assert run.ring.device_error() == 0
        bits = [o.view(torch.int32) for o in outs]
        assert all(torch.equal(b, bits[0]) for b in bits[1:])
    finally:
        run.close()
