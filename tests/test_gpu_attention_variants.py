"""Kernel variants of attention that the sizes of test_gpu_attention.py do not reach,
against the plain binary64 form, with the tolerances of that file."""
import numpy as np
import pytest

from tests.attn_cases import ident, make
from tests.gpu_helpers import gpu_available, torch_mod
from tests.test_gpu_attention import _check_forward, _forward, _plan, _run, _same

pytestmark = pytest.mark.gpu

# (lens_q, lens_k, H, Hk, dim, causal, bias, grid)
CASES = [
    # 33 to 64 queries at dimension 128: the second of two waves works
    ([40, 64, 33, 51], [40, 64, 33, 51], 8, 2, 128, True, None, None),
    ([64, 41, 57], [64, 41, 57], 8, 2, 128, True, "line", None),
    ([49, 49, 49], [49, 49, 49], 8, 2, 128, False, "grid", 7),
    ([64, 36], [64, 36], 3, 3, 120, False, "wide", None),
    ([50, 64], [200, 90], 4, 1, 104, True, "line", None),
    # given positions at dimensions above 64, and above 64 tokens
    ([100, 100], [100, 100], 4, 2, 72, False, "grid", 10),
    ([144, 144, 144], [144, 144, 144], 2, 2, 128, False, "grid", 12),
    ([169], [169], 6, 2, 96, False, "grid", 13),
    ([196, 196], [196, 196], 4, 4, 64, False, "grid", 14),
    ([100] * 6, [100] * 6, 256, 256, 128, False, "grid", 10),
    # few queries and grouped heads on positions
    ([9, 9], [9, 9], 8, 2, 128, False, "grid", 3),
]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not gpu_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=ident)
def test_variants_against_plain64(case, dtype):
    print(f"attention {dtype} {ident(case)}", flush=True)
    lq, lk, H, Hk, dim, causal, bias, grid = case
    _run(make(lq, lk, H, Hk, dim, dtype, causal, bias, seed=60 + dim, grid=grid))


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("keys,H,Hk,dim,bias", [([20000], 4, 1, 64, "line"), ([33000, 700], 2, 1, 128, None),
                                                ([70001], 4, 2, 32, "wide")])
def test_many_pieces_of_a_long_cache(keys, H, Hk, dim, bias, dtype):
    # 78 pieces of the keys, and as many as there can be (128)
    print(f"{dtype} {keys} {H}x{Hk} {dim} {bias}", flush=True)
    c = make([1] * len(keys), keys, H, Hk, dim, dtype, True, bias, seed=70)
    plan = _plan(c)
    o, lse = _forward(c, plan)
    alone, none = _forward(c, plan, want_lse=False)
    torch_mod().cuda.synchronize()
    _check_forward(c, o, lse)
    assert none is None and _same((o,), (alone,))


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_a_long_cache_with_most_of_its_keys_hidden(dtype):
    # pieces whose every key is removed by the bias beside one that has all the weight
    c = make([2], [40000], 2, 1, 64, dtype, False, "line", seed=71)
    far = c["map"][0]
    c["table"][far] = -np.inf  # all offsets below -span
    c["table"][c["map"][-1]] = -np.inf
    o, lse = _forward(c)
    torch_mod().cuda.synchronize()
    _check_forward(c, o, lse)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("bias", [None, "line", "grid"])
@pytest.mark.parametrize("dim", [24, 56, 112])
@pytest.mark.parametrize("n,heads", [(30, "shared"), (50, "shared"), (100, "shared"), (70, "many")])
def test_every_width_dimension_and_kind_of_bias(n, heads, dim, bias, dtype):
    # one, two and four waves a work-group, each padded dimension; key pass on 64 keys
    # and, where there are many heads, on 128
    H, Hk, count = (4, 2, 3) if heads == "shared" else (384, 384, 4)
    lens = [n] * count
    if bias != "grid":
        lens[1] -= 11
    if heads == "many":  # the rule of the key pass
        assert max(lens) / 64 <= 0.75 * H * (sum(lens) / 128) * (sum(lens) / 64) / count / 256 * \
            (0.5 if bias == "line" else 1)
    grid = int(np.ceil(np.sqrt(n)))
    _run(make(lens, lens, H, Hk, dim, dtype, bias == "line", bias, seed=n + dim, grid=grid))
