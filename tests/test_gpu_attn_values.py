"""Values that are not finite in cached rows that are attended to: the attention gives
what its formula gives, (sum exp(s_t - m) v_t) / l with every weight that binary32
holds counted as what it is."""
import pytest
import torch

import attn_ref as ref
from test_gpu_attn import BF16, F16, F32, Decode

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

INF, NAN = float("inf"), float("nan")
# Scores of the tokens whose values are looked at; all others have REST. e^-80 is the least of the
# weights here and a normal number of binary32.
SCORES, REST = [0.0, -1.5, -20.0, -30.0, -80.0, -INF], -0.375


def make(dtype, n, hq, hk, width, window=0):
    """A sequence of n tokens with those scores in every head, and the tokens' places (from the window's start on)."""
    d = Decode(dtype, [n, 3], hq, hk, width, 16, window=window)
    first = max(0, n - window) if window else 0
    seen = n - first
    places = [first + p for p in (seen // 2, seen - 1, 0, seen // 3, seen // 5, seen // 7)] if seen >= 100 else [first]
    assert len(set(places)) == len(places)
    d.q.zero_()
    d.q[0, :, 0] = 1.0
    d.scale = 1.0
    d.k.fill_(0)
    d.v[torch.isnan(d.v)] = 0
    t = torch.arange(n, device="cuda")
    s = torch.full((n,), REST, device="cuda")
    for p, x in zip(places, SCORES):
        s[p] = x
    at = (d.table[0][t // 16].long(), t % 16)
    k = torch.zeros((n, hk, width), dtype=dtype, device="cuda")
    k[..., 0] = s.to(dtype)[:, None]
    d.k[at] = k
    return d, at, places, s.double().cpu(), first


def run(d):
    out, lse = d.run()
    return out[0], lse[0]


CASES = [(1, 1, 64), (8, 1, 128), (16, 1, 128), (12, 1, 64), (4, 2, 256), (4, 4, 80)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("hq,hk,width", CASES)
@pytest.mark.parametrize("n,window", [(1, 0), (100, 0), (3000, 0), (3000, 700)])
def test_infinite_values_keep_their_sign(dtype, hq, hk, width, n, window):
    d, at, places, s, first = make(dtype, n, hq, hk, width, window)
    want, wlse, tol, ltol = ref.decode(d.q, d.k, d.v, d.table, d.lens_host, d.scale, window)
    out, lse = run(d)
    ref.assert_near(out, want[0], tol[0], "finite")
    base, base_lse = out, lse
    weights = torch.exp(s - s[first:].max())
    special = {}
    dim = 0
    for p in places:  # each of these tokens with +inf and with -inf in a dimension of its own
        for x in (INF, -INF):
            special[dim] = [(p, x)]
            dim += 1
    if len(places) > 1:
        special[dim] = [(places[0], INF), (places[1], -INF)]
        special[dim + 1] = [(places[2], INF), (places[3], INF)]
        special[dim + 2] = [(places[1], NAN)]
        special[dim + 3] = [(places[3], INF), (places[0], NAN)]
        special[dim + 4] = [(places[4], -INF), (places[2], -INF), (places[1], -INF)]
    v = d.v[at].clone()
    for k, marks in special.items():
        for p, x in marks:
            v[p, :, k] = x
    d.v[at] = v
    out, lse = run(d)
    assert torch.equal(lse, base_lse)
    for k, marks in special.items():
        # the definition: weights 0 (scores of -inf) times an infinity are NaN, infinities of both signs are
        expect = sum(float(weights[p]) * x for p, x in marks)
        got = out[:, k].double().cpu()
        ok = torch.isnan(got) if expect != expect else got == expect
        assert bool(ok.all()), f"dimension {k}: {marks}, {expect} is {got.tolist()}"
    others = [k for k in range(width) if k not in special]
    assert torch.equal(out[:, others], base[:, others]), "other dimensions keep their bits"


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n", [1, 100, 3000])
def test_infinite_values_of_one_sequence_stay_there(dtype, n):
    d, at, places, s, first = make(dtype, n, 8, 2, 128)
    good, good_lse = d.run()
    d.v[at[0][0], at[1][0], 0] = INF
    out, lse = d.run()
    assert torch.equal(out[1], good[1]) and torch.equal(lse, good_lse)
    # of the other key-value head's queries neither
    assert torch.equal(out[0, 4:], good[0, 4:])
    assert bool((out[0, :4] == INF).all())


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("hq,hk,width", CASES)
@pytest.mark.parametrize("score", [NAN, INF])
@pytest.mark.parametrize("n", [1, 100, 3000])
def test_scores_that_have_no_weight_make_their_heads_nan(dtype, hq, hk, width, score, n):
    # m = inf gives inf - inf for the token itself, NaN a NaN weight: the sum is NaN, in its key-value head's queries only
    d, at, places, s, first = make(dtype, n, hq, hk, width)
    good, good_lse = d.run()
    for p in {0, n // 2, n - 1}:
        k = d.k[at].clone()
        k[p, 0, 0] = score
        before = d.k[at].clone()
        d.k[at] = k
        out, lse = d.run()
        d.k[at] = before
        group = hq // hk
        assert bool(torch.isnan(out[0, :group]).all()) and bool(torch.isnan(lse[0, :group]).all()), p
        assert torch.equal(out[0, group:], good[0, group:]) and torch.equal(lse[0, group:], good_lse[0, group:]), p
        assert torch.equal(out[1], good[1]) and torch.equal(lse[1], good_lse[1]), p
