"""Table entries of large magnitude in attention with a relative position bias, against the fp64 oracle.

Bounds from the arithmetic, beside those of test_gpu_attn_recompute.py.  With e_s = (d + 16) 2^-23 max(scale |q|.|k|)
for a score, and keys more than 30 below a row's lse left out of account (their probabilities are under 1e-13):
  * the forward rounds x = scale q.k + b to fp32, half a step or 2^-24 |x|, and takes exponentials of differences:
        e_x = e_s + 2^-24 max |x| + 2^-21 (30 + 4);
  * lse is rounded once more: off by e_x + 2^-24 max |lse|;
  * the backward takes b - lse before anything is added to it, so given lse its probabilities are off by
        e_b = e_s + 2^-21 (30 + max |scale q.k| + 4)
    of themselves, with nothing of the entries' size.
"""
import math

import numpy as np
import pytest
import torch

import oracle.tp_oracle as O
from tests.gpu_util import f64
from tests.test_gpu_attn_recompute import BF, Case, _tp, within

pytestmark = pytest.mark.gpu

LIMIT = 131072.0  # entries below -LIMIT hide their keys, entries above LIMIT are reported


def check_large(c, C, lse, dQKV, dtable):
    X, table, u = f64(c.QKV), f64(c.table), c.used()
    sc = c.cfg["scale"] or 1.0 / math.sqrt(c.d)
    big = top = 0.0
    for a, e in zip(c.starts[:-1], c.starts[1:]):
        for j in range(c.H if e > a else 0):
            qc, kc, _ = O.grouped_head_columns(c.d, c.H, c.KV, c.N, j)
            q, k = X[a:e, qc:qc + c.d], X[a:e, kc:kc + c.d]
            big = max(big, sc * np.max(np.abs(q) @ np.abs(k).T))
            top = max(top, sc * np.max(np.abs(q @ k.T)))
    far = np.max(np.abs(table)) + top
    e_s, e_d = (c.d + 16) * 2.0 ** -23 * big, (c.d + 16) * 2.0 ** -23
    e_x = e_s + 2.0 ** -24 * far + 2.0 ** -21 * 34
    e_b = e_s + 2.0 ** -21 * (34 + top)
    assert e_b < 2.0 ** -9
    rC, rlse, A = O.attention_lse(X, c.starts, c.cfg, c.bias, table)
    gC, glse = f64(C), f64(lse)
    within(gC[u], rC[u], BF * np.abs(rC[u]) + (BF + 2 * e_x) * A[u] + 1e-30, "C")
    within(glse[:, u], rlse[:, u], np.full_like(rlse[:, u], e_x + 2.0 ** -24 * far), "lse")
    dX, dT, EX, _ = O.attention_lse_grad(X, c.starts, c.cfg, gC, glse, f64(c.dC), c.bias, table, BF + e_b, e_d)
    within(f64(dQKV)[u], dX[u], BF * np.abs(dX[u]) + EX[u] + 1e-30, "dQKV")
    _, _, _, ET = O.attention_lse_grad(X, c.starts, c.cfg, gC, glse, f64(c.dC), c.bias, table, BF + e_b,
                                       e_d + e_b + 2.0 ** -21)
    within(f64(dtable), dT, ET + 1e-30, "dtable")


SHAPES = [  # lens, query heads, key/value heads, d, causal, bias
    ([1] * 60 + [2] * 20 + [3] * 10, 2, 2, 64, True, dict(num_buckets=8, max_distance=20, bidirectional=False)),
    ([1] * 24 + [2, 5], 4, 2, 128, False, dict(num_buckets=8, max_distance=20, bidirectional=True)),
    ([300, 130], 2, 1, 128, True, dict(num_buckets=16, max_distance=40, bidirectional=False)),
    ([640], 2, 2, 64, False, dict(num_buckets=32, max_distance=128, bidirectional=True)),  # tiles beyond the distance
    ([2100], 1, 1, 128, True, dict(num_buckets=32, max_distance=128, bidirectional=False)),  # clusters of CTAs
]


@pytest.mark.parametrize("entry", [-1e4, -65504.0, -1.3e5, 1e5])
@pytest.mark.parametrize("lens,H,KV,d,causal,bias", SHAPES)
def test_large_finite_entries(lens, H, KV, d, causal, bias, entry):
    """Head 0 sees nothing but entries near `entry`; other heads see it in bucket 0, which is all that a sequence's
    first row sees if causal."""
    c = Case(lens, H, KV, d, 1, causal, bias=bias, seed=300 + d)
    c.table[:, 0] += entry
    c.table[0, 1:] = entry
    C, lse = c.fwd()
    g, t = c.bwd(C, lse)
    assert _tp().tp_get_status() == _tp().TP_OK
    check_large(c, C, lse, g, t)


@pytest.mark.parametrize("low", [float(np.nextafter(np.float32(-LIMIT), np.float32(-np.inf))), -1e6, -1e9,
                                 torch.finfo(torch.float32).min])
@pytest.mark.parametrize("lens,H,KV,d,causal,bias", SHAPES)
def test_entries_below_the_range_hide_keys(lens, H, KV, d, causal, bias, low):
    """As -infinity does, bit for bit, in both directions: also where they are all that a row sees."""
    c = Case(lens, H, KV, d, 1, causal, bias=bias, seed=310 + d)
    outs = []
    for x in (low, -math.inf):
        c.table[:, 0] = x
        c.table[0, 1:] = x
        C, lse = c.fwd()
        outs.append((C, lse) + c.bwd(C, lse))
    assert _tp().tp_get_status() == _tp().TP_OK
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert (outs[0][1][0][torch.from_numpy(c.used())] == -math.inf).all() and (outs[0][3][:, 0] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("high", [float(np.nextafter(np.float32(LIMIT), np.float32(np.inf))), 1e9, math.inf])
def test_entries_above_the_range_are_reported(high, d):
    """Once, by the forward and by the backward; the next call is right."""
    tp = _tp()
    bias = dict(num_buckets=8, max_distance=20, bidirectional=True)
    c = Case([150, 40], 2, 1, d, 1, True, bias=bias, seed=320)
    c.table[0, 1] = LIMIT  # in range
    C, lse = c.fwd()
    g, t = c.bwd(C, lse)
    assert tp.tp_get_status() == tp.TP_OK
    check_large(c, C, lse, g, t)
    c.table[0, 1] = high
    c.fwd()
    assert tp.tp_get_status() == tp.TP_ERR_INVALID and tp.tp_get_status() == tp.TP_OK
    c.bwd(C, lse)
    assert tp.tp_get_status() == tp.TP_ERR_INVALID and tp.tp_get_status() == tp.TP_OK
    c.table[0, 1] = LIMIT
    C2, lse2 = c.fwd()
    assert torch.equal(C, C2) and torch.equal(lse, lse2) and torch.equal(c.bwd(C, lse)[0], g)
