"""Attention on the GPU at values where a score, a sum or a scale can leave the
range or the precision that its neighbours need.  The tolerances are those of
test_gpu_attention.py (u = 2^-24; binary16 outputs and factors 2^-11) with the error
of a score written out: a binary32 sum of dim products, (dim + 8) u times the
largest product of norms, and one rounding of the sum with the bias, u of it."""
import numpy as np
import pytest

from tests import plain64
from tests.attn_cases import make
from tests.gpu_helpers import gpu_available, to_np64, torch_mod
from tests.test_gpu_attention import U, _backward, _forward, _packing, _plain, _plan, _within

pytestmark = pytest.mark.gpu
GRADS = ("dq", "dk", "dv", "dtable")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not gpu_available():
        pytest.skip("no GPU")


def _products(c):
    """Largest scaled sum of magnitudes of a score without its bias."""
    q, k = c["q"].astype(np.float64), c["k"].astype(np.float64)
    return c["scale"] * np.linalg.norm(q, axis=2).max() * np.linalg.norm(k, axis=2).max()


def _check_grads(c, grads, ref, mag, relative, rows=None):
    """relative: the error of a factor p, as a part of it."""
    half = 2.0 ** -11 if c["dtype"] == "f16" else 0.0
    group = c["H"] // c["Hk"]
    n = {"dq": c["max_k"], "dk": c["max_q"] * group, "dv": c["max_q"] * group,
         "dtable": 2 * (c["max_k"] + c["max_q"]) + 512}
    for name, got, r, m in zip(GRADS, grads, ref, mag):
        if r is None:
            continue
        h = 0.0 if name == "dtable" else half
        bound = m * (h + relative + (n[name] + c["dim"] + 64) * U) + h * np.abs(r) + (2.0 ** -25 if h else 1e-30)
        got = to_np64(got)
        if rows is not None:
            if name != "dq":
                continue
            got, r, bound = got[rows], r[rows], bound[rows]
        _within(got, r, bound, name)


# sequences of one tile and longer ones, offsets by index and by given positions
LENGTHS = [([40, 64], "line"), ([40, 150], "line"), ([36, 49], "grid"), ([100, 169], "grid")]


@pytest.mark.parametrize("lens,bias", LENGTHS)
@pytest.mark.parametrize("value", [-1e4, -1e6, -1e9, -1.1e9, -3e9, -1e10, -7e15, -1e30, -3.4028235e38, 3e9])
def test_a_large_bias_on_every_key_of_a_head(value, lens, bias, monkeypatch):
    # the rows of the first head have nothing but the large value: finite, and a mask
    # value that a program may well use.  A binary32 score near it is the value plus
    # what of the product its last place keeps, and its factor is exp(score - lse).
    c = make(lens, lens, 4, 4 if bias == "line" else 2, 32, "f32", False, bias, seed=8, grid=13)
    c["table"][:, 0] = value
    o, lse = _forward(c)
    grads = _backward(c, o, lse)
    torch_mod().cuda.synchronize()
    assert bool(torch_mod().isfinite(o).all()) and bool(torch_mod().isfinite(lse).all())
    for name, g in zip(GRADS, grads):
        assert bool(torch_mod().isfinite(g).all()), name
    # one rounding of each score, and for the row sums one of lse (which is given here)
    error = (c["dim"] + 8) * U * _products(c) + U * (abs(value) + _products(c))
    if abs(value) >= 1e9:  # half a last place is 32, more than any product: the score is the value
        assert _products(c) < 32 and np.float32(value) == c["table"][0, 0]
        error = (c["dim"] + 8) * U * _products(c)
        exact = plain64.scores

        def rounded(*a):
            s, ids = exact(*a)
            return np.where(np.isfinite(s) & (np.abs(s) > 1e8), np.float64(np.float32(s)), s), ids

        monkeypatch.setattr(plain64, "scores", rounded)
        same = np.float64(np.float32(value))
        assert bool((lse[0].double() == same).all())
    ref, mag = plain64.attention_backward(c, c["dout"], c["q"], c["k"], c["v"], to_np64(o), to_np64(lse),
                                          **_plain(c))
    # a factor is off by exp(error) - 1
    _check_grads(c, grads, ref, mag, np.expm1(2 * error) + 16 * U)


@pytest.mark.parametrize("lens,bias", LENGTHS)
@pytest.mark.parametrize("value", [-1e6, -1e9, -3e9, -1e30, -3.4028235e38])
def test_large_finite_biases_hide_offsets(value, lens, bias):
    # every row sees other keys too: what is hidden has a factor of zero
    c = make(lens, lens, 4, 4 if bias == "line" else 2, 32, "f32", False, bias, seed=9, grid=13)
    if bias == "line":
        c["table"][:5] = value
    else:
        c["table"][::2] = value
        c["table"][len(c["table"]) // 2] = 0.5  # a token sees itself
    ordinary = np.where(np.abs(c["table"]) > 1e5, 0, c["table"])
    error = (c["dim"] + 8) * U * (_products(c) + np.abs(ordinary).max())
    o, lse = _forward(c)
    grads = _backward(c, o, lse)
    torch_mod().cuda.synchronize()
    ref, mag = plain64.attention_backward(c, c["dout"], c["q"], c["k"], c["v"], to_np64(o), to_np64(lse),
                                          **_plain(c))
    _check_grads(c, grads, ref, mag, 2 * error + 16 * U)


@pytest.mark.parametrize("dtype,size", [("f16", 400.0), ("f32", 3e3), ("f32", 1e6)])
@pytest.mark.parametrize("lens,Hk", [([40, 64], 4), ([40, 150], 2)])
def test_scores_far_from_zero(lens, Hk, dtype, size):
    # every row has a key that is its only one (the gap to the next is far above a
    # score's last place): its factor is one, however large score and lse are
    c = make(lens, lens, 4, Hk, 32, dtype, False, None, seed=10, std=size)
    n, group = sum(lens), 4 // Hk
    o, lse = _forward(c)
    grads = _backward(c, o, lse)
    torch_mod().cuda.synchronize()
    half = 2.0 ** -11 if dtype == "f16" else 0.0
    dv, dmag, count = np.zeros(c["v"].shape), np.zeros(c["v"].shape), np.zeros((n, Hk), int)
    start = 0
    clear = np.ones((n, 4), bool)
    for length in lens:
        at = slice(start, start + length)
        for h in range(4):
            s = c["q"][at, h].astype(np.float64) @ c["k"][at, h // group].astype(np.float64).T * c["scale"]
            order = np.sort(s, axis=1)
            best = start + s.argmax(axis=1)
            clear[at, h] = order[:, -1] - order[:, -2] > 40 + 4 * (c["dim"] + 8) * U * _products(c)
            np.add.at(dv[:, h // group], best, c["dout"][at, h].astype(np.float64))
            np.add.at(dmag[:, h // group], best, np.abs(c["dout"][at, h].astype(np.float64)))
            np.add.at(count[:, h // group], best, 1)
            keep = clear[at, h]
            _within(to_np64(o)[at, h][keep], c["v"][best, h // group].astype(np.float64)[keep],
                    (half + 8 * U) * np.abs(c["v"][best, h // group].astype(np.float64)[keep]) + 1e-30, "o")
        start += length
    for g in grads[:3]:
        assert bool(torch_mod().isfinite(g).all())
    # a row whose two best keys are close leaves its sequence out of the comparison of
    # dv; there are few of them, since a gap is of the size of the scores
    assert clear.mean() > 0.95
    start = 0
    for length in lens:
        at = slice(start, start + length)
        for g in range(Hk):
            if clear[at, g * group:(g + 1) * group].all():
                bound = dmag[at, g] * (2 * half + (count[at, g].max() + 24) * U) + (2.0 ** -25 if half else 1e-30)
                _within(to_np64(grads[2])[at, g], dv[at, g], bound, "dv")
        start += length


def _dq_reference(c, o, lse):
    ref, mag = plain64.attention_backward(c, c["dout"], c["q"], c["k"], c["v"], to_np64(o), to_np64(lse),
                                          **_plain(c))
    error = (c["dim"] + 8) * U * (_products(c) + (0 if c["table"] is None else np.abs(c["table"]).max()))
    return ref, mag, 2 * error + 16 * U


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("lens", [[40, 60], [40, 150]])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
def test_a_gradient_that_is_not_finite_stays_in_its_query(value, lens, dtype):
    # (in dq; keys and values sum over all queries)
    c = make(lens, lens, 2, 2, 32, dtype, False, "line", seed=11, do_std=40.0)
    o, lse = _forward(c)
    ref, mag, relative = _dq_reference(c, o, lse)
    others = np.ones((sum(lens), 2), bool)
    for token, head in ((5, 0), (33, 1), (sum(lens) - 1, 0)):
        c["dout"][token, head, 3] = value
        others[token, head] = False
    grads = _backward(c, o, lse)
    torch_mod().cuda.synchronize()
    _check_grads(c, grads, ref, mag, relative, rows=others)


@pytest.mark.parametrize("lens", [[40, 60], [40, 150]])
@pytest.mark.parametrize("ratio", [2.0 ** -14, 2.0 ** -22, 2.0 ** -32])
def test_queries_with_small_gradients_beside_large_ones(ratio, lens):
    # in binary16 a query's factors are scaled by its own size
    c = make(lens, lens, 2, 2, 32, "f16", False, "line", seed=12, do_std=8000.0)
    rows = np.arange(sum(lens)) % 5 != 0
    c["dout"][rows] = (c["dout"][rows].astype(np.float64) * ratio).astype(np.float16)
    # keys of 2^7 and queries of 2^-7: gradients of queries far above binary16's last place
    c["q"] = (c["q"].astype(np.float64) / 128).astype(np.float16)
    c["k"] = (c["k"].astype(np.float64) * 128).astype(np.float16)
    c["dout"] = np.clip(c["dout"], -30000, 30000)
    c["v"] = (c["v"].astype(np.float64) / 128).astype(np.float16)
    o, lse = _forward(c)
    ref, mag, relative = _dq_reference(c, o, lse)
    grads = _backward(c, o, lse)
    torch_mod().cuda.synchronize()
    assert np.isfinite(to_np64(grads[0])).all()
    everywhere = np.ones((sum(lens), 2), bool)
    _check_grads(c, grads, ref, mag, relative, rows=everywhere)


# lengths whose tiles begin and end everywhere in the tiles of the packed tokens, with
# sequences of no query among them
RAGGED = [0, 1, 127, 128, 129, 0, 0, 300, 64, 255, 256, 257, 5, 0, 640, 33, 1, 0]


@pytest.mark.parametrize("spare", [0, 1, 400])
@pytest.mark.parametrize("bias", ["line", "grid"])
@pytest.mark.parametrize("lens_q,Hk", [(RAGGED, 2), ([min(n, 64) for n in RAGGED], 1), ([0] * 6 + [130] + [0] * 5, 2)])
def test_table_gradient_of_many_ragged_sequences(lens_q, Hk, bias, spare):
    # spare: tokens after the last sequence; the workspace holds NaN before the call
    torch = torch_mod()
    c = make(lens_q, [n + 3 * (i % 2) for i, n in enumerate(lens_q)], 2, Hk, 16, "f32", bias == "line",
             bias, seed=14, grid=23)
    if bias == "grid":
        rng = np.random.default_rng(3)
        c["pos_q"] = np.concatenate([rng.permutation(676)[:n] for n in lens_q]).astype(np.int32)
        c["pos_k"] = rng.integers(0, 676, c["k"].shape[0]).astype(np.int32)
    plan, n = _plan(c), sum(lens_q)
    o, lse = _forward(c)
    want = to_np64(_backward(c, o, lse)[3])
    longer = dict(c)
    for name in ("q", "dout"):
        longer[name] = np.concatenate([c[name], np.full((spare, 2, 16), 7, np.float32)])
    if c["pos_q"] is not None:
        longer["pos_q"] = np.concatenate([c["pos_q"], np.full(spare, 5, np.int32)])
    ol = torch.full((n + spare, 2, 16), 7.0, device="cuda")
    ol[:n] = o
    ll = torch.full((2, n + spare), 7.0, device="cuda")
    ll[:, :n] = lse
    packing = _packing(longer)
    ws = torch.full((plan.workspace_bytes(packing, n + spare, c["k"].shape[0])[1] // 4,), float("nan"),
                    device="cuda")
    dq = torch.full_like(ol, 7.0)
    got = _backward(longer, ol, ll, plan, workspace=ws, dq=dq)
    torch.cuda.synchronize()
    ref, mag = plain64.attention_backward(c, c["dout"], c["q"], c["k"], c["v"], to_np64(o), to_np64(lse),
                                          **_plain(c))
    error = (c["dim"] + 8) * U * (_products(c) + np.abs(c["table"]).max())
    _check_grads(c, [got[0][:n]] + list(got[1:]), ref, mag, 2 * error + 16 * U)
    assert bool((dq[n:] == 7).all())
    # the sums' places depend on the number of tokens at the end, their order does not
    assert np.abs(to_np64(got[3]) - want).max() <= 2.0 ** -20 * np.abs(want).max()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("lens,room", [([30, 64, 1], 100), ([700, 1500, 2100], 2500)])
def test_caches_with_spare_room(lens, room, dtype):
    # the room behind a cache's tokens is a sequence of its own without queries
    torch = torch_mod()
    c = make([1] * 3, lens, 8, 2, 64, dtype, True, "line", seed=15)
    want = _forward(c)
    d = dict(c, max_k=room)
    for name in ("k", "v"):
        d[name] = np.full((3 * room, 2, 64), np.nan, c[name].dtype)
        for i, n in enumerate(lens):
            d[name][i * room:i * room + n] = c[name][sum(lens[:i]):sum(lens[:i + 1])]
    d["cu_q"] = np.array([0, 1, 1, 2, 2, 3, 3], np.int32)
    d["cu_k"] = np.array([0] + [x for i, n in enumerate(lens) for x in (i * room + n, (i + 1) * room)], np.int32)
    got = _forward(d)
    torch.cuda.synchronize()
    # sums of other pieces of the keys (none of the short caches)
    error = (2.0 ** -10 if dtype == "f16" else 0) + (max(lens) + 64) * U
    mag = plain64.attention(c, c["q"], c["k"], np.abs(c["v"]), **_plain(c))[0]
    assert (np.abs(to_np64(got[0]) - to_np64(want[0])) <= error * mag + 2.0 ** -24).all()
    assert np.abs(to_np64(got[1]) - to_np64(want[1])).max() <= (max(lens) + 64) * U + 8 * U * 20
