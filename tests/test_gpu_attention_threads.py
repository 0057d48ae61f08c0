"""Attention called from several threads at once, on streams of their own, with plans
whose kernels are the same and whose LDS sizes differ."""
import threading

import pytest

from tests.attn_cases import make
from tests.gpu_helpers import gpu_available, to_dev, torch_mod
from tests.test_gpu_attention import _packing, _plan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,dim,dtype", [([70, 100], 128, "f16"), ([60, 64], 32, "f32")])
def test_spans_of_different_threads(lens, dim, dtype):
    # more than 64 KB of LDS a work-group, in every thread another number
    if not gpu_available():
        pytest.skip("no GPU")
    torch = torch_mod()
    cases = [make(lens, lens, 2, 2, dim, dtype, True, bias, seed=20) for bias in ("line", "wide")]
    calls, results, errors = [], [None, None], []
    for c in cases:
        d = {n: to_dev(c[n]) for n in ("q", "k", "v", "dout", "table", "map")}
        calls.append((_plan(c), _packing(c), d))
    torch.cuda.synchronize()

    def run(i, repeats, stream):
        try:
            torch.cuda.set_device(0)
            plan, pk, d = calls[i]
            with torch.cuda.stream(stream):
                for _ in range(repeats):
                    o, lse = plan.forward(d["q"], d["k"], d["v"], pk, d["table"], d["map"])
                    grads = plan.backward(d["dout"], d["q"], d["k"], d["v"], o, lse, pk, d["table"], d["map"])
            stream.synchronize()
            results[i] = (o, lse) + grads
        except Exception as e:  # noqa: BLE001 -- raised below, in the test's thread
            errors.append(e)

    alone = []
    for i in range(2):
        run(i, 1, torch.cuda.current_stream())
        alone.append(results[i])
    threads = [threading.Thread(target=run, args=(i, 50, torch.cuda.Stream())) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(alone, results):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
