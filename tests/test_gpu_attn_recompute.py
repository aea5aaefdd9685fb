"""GPU parity of attention without stored probabilities (tp_attn_recompute_*)
and of its relative position bias (tp_attn_relbias_*) against the fp64 oracle.

Bounds, element by element, from the arithmetic (half a step of bf16 is 2^-8
of the value; sums and softmax are fp32):
  * a score is a sum of d products; fp32 accumulation, truncating at worst,
    leaves it off by (d + 16) 2^-23 of its sum of magnitudes, and lse and the
    exponent's argument add 2^-21 of their size: P is off by
        e_x = (d + 16) 2^-23 max(scale |q|.|k|) + 2^-21 (max |lse| + max |x| + 4)
    of itself;
  * P and dS are rounded to bf16 as operands: e_p = 2^-8 + e_x (and a second
    order, 2^-8 of that, covered by the factor 1.01);
  * C, dQKV are rounded to bf16 once: 2^-8 of the value.  D and dC.v are fp32
    sums of d products: e_d = (d + 16) 2^-23 of their magnitudes;
  * the table's gradient sums fp32 dS: e_x of |dS| plus the fp32 sums' 2^-21 of
    the magnitudes.
"""
import math

import numpy as np
import pytest
import torch

import oracle.tp_oracle as O
import synthetic_inputs as SI
from tests.gpu_util import f64

pytestmark = pytest.mark.gpu

BF = 2.0 ** -8


def _tp():
    import megatron_tensor_transformer_tp_gb300 as tp
    return tp


class Case:
    """Inputs of one call on the CPU, and what the call gives."""

    def __init__(self, lens, H, KV, d, N, causal, scale=0.0, tail=0, head=0, bias=None, seed=0, packed=None):
        self.lens, self.H, self.KV, self.d, self.N = lens, H, KV, d, N
        starts = [head]
        for n in lens:
            starts.append(starts[-1] + n)
        self.starts, self.T = starts, starts[-1] + tail
        self.packed = (len(set(lens)) > 1 or tail or head) if packed is None else packed
        self.cfg = dict(b=len(lens), s=max(lens), n_heads=H, n_kv_heads=KV, d=d, N=N, causal=causal, scale=scale)
        self.bias = bias
        sc = scale or 1.0 / math.sqrt(d)
        W = (H + 2 * KV) * d
        X = SI.normal(seed, 1, (self.T, W), 1.0, "f32")
        for j in range(H):
            qc = O.grouped_head_columns(d, H, KV, N, j)[0]
            X[:, qc:qc + d] *= 1.5 / (sc * math.sqrt(d))
        self.QKV = X.to(torch.bfloat16)
        self.dC = SI.normal(seed, 2, (self.T, H * d), 1.0, "bf16")
        self.table = SI.normal(seed, 3, (bias["num_buckets"], H), 0.7, "f32") if bias else None

    def device(self):
        self.starts_d = torch.tensor(self.starts, dtype=torch.int64, device="cuda") if self.packed else None
        return self

    def fwd(self, QKV=None, C=None, lse=None, stream=None):
        tp = _tp()
        self.device()
        QKV = self.QKV.cuda() if QKV is None else QKV
        C = torch.full((self.T, self.H * self.d), 7.0, dtype=torch.bfloat16, device="cuda") if C is None else C
        lse = torch.full((self.H, self.T), 7.0, device="cuda") if lse is None else lse
        if self.bias:
            tp.tp_attn_relbias_fwd(QKV, self.cfg, self.bias, self.table.cuda(), C, lse, seq_starts=self.starts_d,
                                   stream=stream)
        else:
            tp.tp_attn_recompute_fwd(QKV, self.cfg, C, lse, seq_starts=self.starts_d, stream=stream)
        return C, lse

    def bwd(self, C, lse, QKV=None, dC=None, dQKV=None, dtable="new", accumulate=False, stream=None):
        tp = _tp()
        QKV = self.QKV.cuda() if QKV is None else QKV
        dC = self.dC.cuda() if dC is None else dC
        if dQKV is None:
            dQKV = torch.full((self.T, QKV.shape[1]), 7.0, dtype=torch.bfloat16, device="cuda")
        if isinstance(dtable, str):
            dtable = torch.full(self.table.shape, 7.0, device="cuda") if self.bias else None
        n = tp.tp_attn_recompute_workspace_size(self.cfg, self.T, self.bias if dtable is not None else None)
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN wherever it is read unwritten
        if self.bias:
            tp.tp_attn_relbias_bwd(QKV, self.cfg, self.bias, self.table.cuda(), C, lse, dC, dQKV, dtable, ws,
                                   accumulate=accumulate, seq_starts=self.starts_d, stream=stream)
        else:
            tp.tp_attn_recompute_bwd(QKV, self.cfg, C, lse, dC, dQKV, ws, seq_starts=self.starts_d, stream=stream)
        return dQKV, dtable

    def used(self):
        m = np.zeros(self.T, dtype=bool)
        m[self.starts[0]:self.starts[-1]] = True
        return m

    def errors(self):
        """(e_x, e_p, e_d) of the module's docstring, and the exact C, lse, sums of P |v|."""
        X, u = f64(self.QKV), self.used()
        table = None if self.table is None else f64(self.table)
        C, lse, A = O.attention_lse(X, self.starts, self.cfg, self.bias, table)
        sc = self.cfg["scale"] or 1.0 / math.sqrt(self.d)
        big = top = 0.0
        for a, e in zip(self.starts[:-1], self.starts[1:]):
            for j in range(self.H if e > a else 0):
                qc, kc, _ = O.grouped_head_columns(self.d, self.H, self.KV, self.N, j)
                q, k = X[a:e, qc:qc + self.d], X[a:e, kc:kc + self.d]
                big = max(big, sc * np.max(np.abs(q) @ np.abs(k).T))
                top = max(top, sc * np.max(np.abs(q @ k.T)))
        top += 0.0 if table is None else np.max(np.abs(table[np.isfinite(table)]))
        e_x = (self.d + 16) * 2.0 ** -23 * big + 2.0 ** -21 * (np.max(np.abs(lse[:, u]), initial=0) + top + 4)
        assert e_x < 2.0 ** -9  # small against bf16's half step, else the bounds say little
        return e_x, BF + e_x, (self.d + 16) * 2.0 ** -23, C, lse, A


def within(got, ref, bound, what):
    if not ref.size:
        return
    over = np.abs(got - ref) - 1.01 * bound
    assert np.isfinite(got).all(), f"{what}: not finite"
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 0, f"{what}{list(map(int, at))}: {got[at]} is {abs(got - ref)[at]:.3e} off {ref[at]}, allowed {bound[at]:.3e}"


def check(c, C, lse, dQKV=None, dtable=None, untouched=7.0):
    u = c.used()
    e_x, e_p, e_d, rC, rlse, A = c.errors()
    gC, glse = f64(C), f64(lse)
    within(gC[u], rC[u], BF * np.abs(rC[u]) + (e_p + e_x) * A[u] + 1e-30, "C")
    within(glse[:, u], rlse[:, u], np.full_like(rlse[:, u], 2 * e_x), "lse")
    if untouched is not None:
        assert (gC[~u] == untouched).all() and (glse[:, ~u] == untouched).all()
    if dQKV is None:
        return
    table = None if c.table is None else f64(c.table)
    dX, dT, EX, ET = O.attention_lse_grad(f64(c.QKV), c.starts, c.cfg, gC, glse, f64(c.dC), c.bias, table, e_p, e_d)
    g = f64(dQKV)
    within(g[u], dX[u], BF * np.abs(dX[u]) + EX[u] + 1e-30, "dQKV")
    if untouched is not None:
        assert (g[~u] == untouched).all()
    if dtable is not None:
        _, _, _, ET = O.attention_lse_grad(f64(c.QKV), c.starts, c.cfg, gC, glse, f64(c.dC), c.bias, table, e_p,
                                           e_d + e_x + 2.0 ** -21)
        within(f64(dtable), dT, ET + 1e-30, "dtable")


def run(c):
    C, lse = c.fwd()
    dQKV, dtable = c.bwd(C, lse)
    assert _tp().tp_get_status() == _tp().TP_OK
    check(c, C, lse, dQKV, dtable)


PLAIN = [  # lens, query heads, key/value heads, d, shards, causal, scale, tail, head
    ([1], 1, 1, 8, 1, True, 0.0, 0, 0),                     # one token
    ([96], 2, 2, 64, 1, True, 0.0, 0, 0),
    ([128], 2, 1, 128, 1, True, 0.0, 0, 0),                 # exactly one tile
    ([129], 1, 1, 128, 1, False, 0.0, 0, 0),                # one row in the last tile
    ([640, 640], 2, 2, 64, 2, True, 0.0, 0, 0),             # even and odd numbers of tiles
    ([512], 4, 1, 128, 1, False, 0.3, 0, 0),                # four query heads a key/value head
    ([700], 8, 2, 96, 2, True, 0.0, 0, 0),
    ([257], 2, 2, 80, 1, True, 0.0, 0, 0),
    ([300, 1, 0, 65, 511, 128, 2], 4, 2, 128, 2, True, 0.0, 37, 0),   # packed, an empty one, unused rows
    ([300, 1, 0, 65, 511, 128, 2], 4, 2, 64, 2, False, 0.0, 37, 5),   # and rows in front
    ([5] * 40, 2, 1, 40, 1, True, 0.0, 3, 0),               # more sequences than a warp has lanes
    ([0, 0, 0], 2, 2, 64, 1, True, 0.0, 9, 0),              # nothing but empty sequences
]


@pytest.mark.parametrize("lens,H,KV,d,N,causal,scale,tail,head", PLAIN)
def test_recompute_parity(lens, H, KV, d, N, causal, scale, tail, head):
    run(Case(lens, H, KV, d, N, causal, scale, tail, head, seed=sum(lens) + d))


BIASED = [  # lens, query heads, key/value heads, d, shards, causal, tail, buckets, max distance, bidirectional
    ([96], 2, 2, 64, 1, True, 0, 32, 128, False),
    ([640], 2, 2, 64, 2, False, 0, 32, 128, True),           # tiles beyond the distance on both sides
    ([640], 2, 1, 128, 1, True, 0, 32, 128, False),          # query heads with a shared key/value head
    ([300, 1, 0, 65, 511], 2, 2, 64, 1, False, 11, 8, 20, True),
    ([513], 1, 1, 72, 1, False, 0, 6, 5, False),             # keys ahead of the query count as distance 0
    ([700], 2, 2, 32, 1, True, 0, 64, 1024, True),           # no distance reaches the end; half the buckets unused
    ([400], 2, 2, 64, 1, False, 0, 256, 300, True),          # more buckets than distances in places
    ([1, 1, 2], 1, 1, 16, 1, True, 0, 2, 2, False),
]


@pytest.mark.parametrize("lens,H,KV,d,N,causal,tail,nb,md,both", BIASED)
def test_relbias_parity(lens, H, KV, d, N, causal, tail, nb, md, both):
    run(Case(lens, H, KV, d, N, causal, 1.0, tail, bias=dict(num_buckets=nb, max_distance=md, bidirectional=both),
             seed=sum(lens) + nb))


# ----------------------------------------------------------------------------
# layouts, neighbours, streams, graphs
# ----------------------------------------------------------------------------
BIAS = dict(num_buckets=16, max_distance=40, bidirectional=False)


@pytest.mark.parametrize("bias", [None, BIAS])
def test_row_pitches_and_offsets(bias):
    """Every buffer a column slice of a wider one: nothing outside the slice is read into a result or written."""
    c = Case([130, 77], 4, 2, 64, 2, True, tail=3, bias=bias, seed=5)
    W, h = c.QKV.shape[1], c.H * c.d

    def wide(t, cols, fill):
        big = torch.full((c.T, cols + 40), fill, dtype=torch.bfloat16, device="cuda")
        v = big[:, 16:16 + cols]
        if t is not None:
            v.copy_(t)
        return big, v

    nan = float("nan")
    _, Q = wide(c.QKV, W, nan)
    bC, C = wide(torch.full((c.T, h), 7.0), h, 3.0)
    _, dC = wide(c.dC, h, nan)
    bdQ, dQ = wide(torch.full((c.T, W), 7.0), W, 3.0)
    lse = torch.full((c.H, c.T), 7.0, device="cuda")
    c.fwd(Q, C, lse)
    dQKV, dtable = c.bwd(C, lse, Q, dC, dQ)
    check(c, C, lse, dQKV, dtable)
    for big, cols in ((bC, h), (bdQ, W)):
        assert (big[:, :16] == 3.0).all() and (big[:, 16 + cols:] == 3.0).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("bias", [None, dict(BIAS, bidirectional=True)])
def test_neighbours_that_are_not_numbers(causal, bias):
    """A sequence's results do not depend on the rows beside it, NaN and infinities among them, bit for bit."""
    c = Case([100, 190, 60], 4, 2, 128, 1, causal, tail=50, head=30, bias=bias, seed=9)
    C, lse = c.fwd()
    g, _ = c.bwd(C, lse)
    a, e = c.starts[1], c.starts[2]
    for bad in (float("nan"), float("inf"), -float("inf")):
        Q, dC, C2 = c.QKV.cuda(), c.dC.cuda(), C.clone()
        for t in (Q, dC, C2):
            t[:a] = bad
            t[e:] = bad
        l2 = lse.clone()
        l2[:, :a] = bad
        l2[:, e:] = bad
        fC, fl = c.fwd(Q)
        assert torch.equal(fC[a:e], C[a:e]) and torch.equal(fl[:, a:e], lse[:, a:e])
        g2, _ = c.bwd(C2, l2, Q, dC)
        assert torch.equal(g2[a:e], g[a:e])


def test_same_sequence_anywhere():
    """Packed, alone, by starts or by one length: the same rows give the same bits."""
    c = Case([300, 300], 2, 1, 64, 1, True, seed=3, packed=False)
    C, lse = c.fwd()
    d = Case([300, 300], 2, 1, 64, 1, True, seed=3, packed=True)
    D, lse2 = d.fwd()
    assert torch.equal(C, D) and torch.equal(lse, lse2)
    g, _ = c.bwd(C, lse)
    g2, _ = d.bwd(C, lse)
    assert torch.equal(g, g2)


@pytest.mark.parametrize("bias", [None, BIAS])
def test_equal_calls_equal_bits(bias):
    c = Case([500, 260, 31], 8, 4, 64, 2, True, bias=bias, seed=4)
    C, lse = c.fwd()
    g, t = c.bwd(C, lse)
    for _ in range(5):
        C2, lse2 = c.fwd()
        g2, t2 = c.bwd(C, lse)
        assert torch.equal(C, C2) and torch.equal(lse, lse2) and torch.equal(g, g2)
        assert t is None or torch.equal(t, t2)


def test_table_gradient_accumulates_or_is_left_out():
    c = Case([200, 90], 2, 2, 64, 1, True, bias=BIAS, seed=6)
    C, lse = c.fwd()
    g, t = c.bwd(C, lse)
    old = torch.randn(t.shape, device="cuda")
    _, t2 = c.bwd(C, lse, dtable=old.clone(), accumulate=True)
    # the kernel adds in fp64 and rounds once
    assert torch.allclose(t2, (old.double() + t.double()).float(), rtol=2.0 ** -22, atol=2.0 ** -22 * float(t.abs().max()))
    g3, _ = c.bwd(C, lse, dtable=None)
    assert torch.equal(g, g3)


def test_zero_bias_is_no_bias():
    """A table of zeros: the scores pass through another multiply-add, whose result rounds the same."""
    c = Case([300], 2, 2, 64, 1, True, scale=0.25, bias=BIAS, seed=8)
    c.table = torch.zeros_like(c.table)
    C, lse = c.fwd()
    d = Case([300], 2, 2, 64, 1, True, scale=0.25, seed=8)
    check(d, C, lse)


@pytest.mark.parametrize("bias", [None, BIAS])
def test_gradient_against_differences(bias):
    """sum(C w) along a random direction: central differences of the fp64 definition against the kernels' gradient.
    C, dQKV are bf16: half a step of each summed value, with random signs at most 4 sqrt(n) of them."""
    c = Case([90, 41], 4, 2, 64, 2, True, bias=bias, seed=12)
    C, lse = c.fwd()
    g, t = c.bwd(C, lse)
    X, w = f64(c.QKV), f64(c.dC)
    table = None if bias is None else f64(c.table)
    rng = np.random.default_rng(0)
    u = rng.standard_normal(X.shape)
    ut = None if bias is None else rng.standard_normal(table.shape)
    h = 1e-4

    def f(s):
        return np.sum(O.attention_lse(X + s * h * u, c.starts, c.cfg, bias,
                                      None if bias is None else table + s * h * ut)[0] * w)

    num = (f(1) - f(-1)) / (2 * h)
    got = np.sum(f64(g) * u) + (0.0 if bias is None else np.sum(f64(t) * ut))
    e_x, e_p, e_d = c.errors()[:3]
    # D from the bf16 C: off by 2^-8 |dC C| a row element
    _, _, EX, ET = O.attention_lse_grad(X, c.starts, c.cfg, f64(C), f64(lse), w, bias, table, e_p, e_d + BF)
    var = np.sum((EX + BF * np.abs(f64(g))) ** 2) + (0.0 if bias is None else np.sum(ET ** 2))
    assert abs(got - num) <= 4 * math.sqrt(var), (got, num, math.sqrt(var))


def test_against_the_stored_probabilities_core():
    """The same sizes through tp_attn_core_fwd / _bwd: both within their bf16 bounds of the oracle, so within
    twice those of each other."""
    tp = _tp()
    c = Case([256, 256], 4, 4, 64, 2, True, seed=21)
    C, lse = c.fwd()
    g, _ = c.bwd(C, lse)
    Q = c.QKV.cuda()
    P = torch.empty(2, 4, 256, 256, dtype=torch.bfloat16, device="cuda")
    C2, l2 = torch.empty_like(C), torch.empty(2, 4, 256, device="cuda")
    ws = torch.empty(tp.tp_attn_core_workspace_size(c.T, 256, 256, 4), dtype=torch.uint8, device="cuda")
    tp.tp_attn_core_fwd(Q, 256, 4, 2, True, P, C2, l2, ws)
    g2 = torch.empty_like(g)
    tp.tp_attn_core_bwd(Q, P, C2, c.dC.cuda(), 256, 4, 2, True, g2, ws)
    assert tp.tp_get_status() == tp.TP_OK
    assert (lse.view(4, 2, 256).transpose(0, 1) - l2).abs().max() < 1e-4
    for x, y in ((C, C2), (g, g2)):
        assert (x.double() - y.double()).abs().max() <= 2e-2 * y.double().abs().max()


@pytest.mark.parametrize("bias", [None, BIAS])
def test_side_stream_and_graph(bias):
    """On another stream than torch's current one; captured, and replayed on new values in the same buffers."""
    c = Case([300, 130], 4, 2, 64, 1, True, bias=bias, seed=14)
    tp = _tp()
    ref = c.fwd()
    rg, rt = c.bwd(*ref)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    C, lse = c.fwd(stream=st)
    st.synchronize()
    assert torch.equal(C, ref[0]) and torch.equal(lse, ref[1])

    Q, dC = torch.zeros_like(c.QKV.cuda()), torch.zeros_like(c.dC.cuda())
    C, lse, dQ = torch.zeros_like(ref[0]), torch.zeros_like(ref[1]), torch.zeros_like(rg)
    dt = torch.zeros_like(rt) if bias else None
    ws = torch.empty(tp.tp_attn_recompute_workspace_size(c.cfg, c.T, bias), dtype=torch.uint8, device="cuda")
    table = c.table.cuda() if bias else None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if bias:
            tp.tp_attn_relbias_fwd(Q, c.cfg, bias, table, C, lse, seq_starts=c.starts_d)
            tp.tp_attn_relbias_bwd(Q, c.cfg, bias, table, C, lse, dC, dQ, dt, ws, seq_starts=c.starts_d)
        else:
            tp.tp_attn_recompute_fwd(Q, c.cfg, C, lse, seq_starts=c.starts_d)
            tp.tp_attn_recompute_bwd(Q, c.cfg, C, lse, dC, dQ, ws, seq_starts=c.starts_d)
    for _ in range(3):
        Q.zero_(), dC.zero_(), C.zero_()
        graph.replay()
        Q.copy_(c.QKV.cuda())
        dC.copy_(c.dC.cuda())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(C, ref[0]) and torch.equal(lse, ref[1]) and torch.equal(dQ, rg)
        assert not bias or torch.equal(dt, rt)
    assert tp.tp_get_status() == tp.TP_OK


def test_two_streams_at_once():
    """Calls that overlap share nothing but what the caller shares."""
    a = Case([700], 4, 2, 128, 1, True, seed=31)
    b = Case([400, 123], 4, 4, 64, 1, False, seed=32)
    ra, rb = a.fwd(), b.fwd()
    ga, gb = a.bwd(*ra)[0], b.bwd(*rb)[0]
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        torch.cuda.synchronize()
        with torch.cuda.stream(sa):
            xa = a.fwd()
            ya = a.bwd(*xa)[0]
        with torch.cuda.stream(sb):
            xb = b.fwd()
            yb = b.bwd(*xb)[0]
        torch.cuda.synchronize()
        assert torch.equal(xa[0], ra[0]) and torch.equal(xb[0], rb[0])
        assert torch.equal(ya, ga) and torch.equal(yb, gb)


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("bias", [None, BIAS])
def test_calls_in_a_row_on_the_same_buffers(bias, few):
    """Training steps: the same buffers with other values, sequences and tables, and no wait in between, give the
    bits of calls apart from each other, each launch waiting for the one before."""
    tp = _tp()
    H, KV, d, T = (2, 1, 128, 1500) if few else (16, 4, 64, 700)
    steps = []
    for k in range(5):
        cut = 100 + 130 * k
        c = Case([cut, T - cut], H, KV, d, 1, True, bias=bias, seed=200 + k, packed=True)
        steps.append(c)
    ws = torch.empty(tp.tp_attn_recompute_workspace_size(steps[0].cfg, T, bias), dtype=torch.uint8, device="cuda")
    dev = [(c.QKV.cuda(), c.dC.cuda(), torch.tensor(c.starts, device="cuda"), c.table.cuda() if bias else None)
           for c in steps]
    buf = [None if x is None else torch.zeros_like(x) for x in dev[0]]
    bf = dict(dtype=torch.bfloat16, device="cuda")
    C, lse, dQ = torch.zeros(T, H * d, **bf), torch.zeros(H, T, device="cuda"), torch.zeros_like(dev[0][0])
    dt = torch.zeros(bias["num_buckets"], H, device="cuda") if bias else None

    def step(k, keep):
        for b, x in zip(buf, dev[k]):
            if b is not None:
                b.copy_(x)
        Q, dC, starts, table = buf
        cfg = dict(steps[k].cfg, s=None)
        if bias:
            tp.tp_attn_relbias_fwd(Q, cfg, bias, table, C, lse, seq_starts=starts)
            tp.tp_attn_relbias_bwd(Q, cfg, bias, table, C, lse, dC, dQ, dt, ws, seq_starts=starts)
        else:
            tp.tp_attn_recompute_fwd(Q, cfg, C, lse, seq_starts=starts)
            tp.tp_attn_recompute_bwd(Q, cfg, C, lse, dC, dQ, ws, seq_starts=starts)
        for o, x in zip(keep, (C, lse, dQ, dt)):
            if o is not None:
                o.copy_(x)

    outs = [[None if x is None else torch.zeros_like(x) for x in (C, lse, dQ, dt)] for _ in range(30)]
    want = [[None if x is None else torch.zeros_like(x) for x in (C, lse, dQ, dt)] for _ in steps]
    tp.tp_debug_set_pdl(0)
    try:
        for k in range(len(steps)):
            step(k, want[k])
            torch.cuda.synchronize()
    finally:
        tp.tp_debug_set_pdl(1)
    for n, keep in enumerate(outs):
        step(n % len(steps), keep)
    torch.cuda.synchronize()
    assert tp.tp_get_status() == tp.TP_OK
    for n, keep in enumerate(outs):
        for x, y in zip(keep, want[n % len(steps)]):
            assert x is None or torch.equal(x, y)


def test_attention_block_as_used():
    """QKV projection, attention without stored probabilities, output projection, and back, with shards: the
    gradients of the weights and of the input against the fp64 oracle's chain."""
    tp = _tp()
    T, h, H, N = 320, 256, 4, 2
    d = h // H
    c = Case([200, 120], H, H, d, N, True, seed=41)
    X = SI.normal(41, 11, (T, h), 1.0, "bf16")
    Wq = [SI.normal(41, 12 + i, (3 * h // N, h), 0.05, "bf16") for i in range(N)]
    Wo = [SI.normal(41, 22 + i, (h, h // N), 0.05, "bf16") for i in range(N)]
    dO = SI.normal(41, 32, (T, h), 1.0, "bf16")
    dev = lambda t: t.cuda().contiguous()  # noqa: E731
    x, wq, wo, do = dev(X), [dev(t) for t in Wq], [dev(t) for t in Wo], dev(dO)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    QKV, O_, C = torch.empty(T, 3 * h, **bf), torch.empty(T, h, **bf), torch.zeros(T, h, **bf)
    tp.tp_attn_proj_fwd(x, wq, None, C, wo, None, QKV, O_, H)          # QKV (the output is taken below)
    c.device()
    lse = torch.empty(H, T, device="cuda")
    tp.tp_attn_recompute_fwd(QKV, c.cfg, C, lse, seq_starts=c.starts_d)
    tp.tp_attn_proj_fwd(x, wq, None, C, wo, None, QKV, O_, H)
    dX, dC, dQKV = torch.empty(T, h, **bf), torch.empty(T, h, **bf), torch.empty(T, 3 * h, **bf)
    dWq = [torch.empty(3 * h // N, h, device="cuda") for _ in range(N)]
    dWo = [torch.empty(h, h // N, device="cuda") for _ in range(N)]
    zero = torch.zeros(T, 3 * h, **bf)
    tp.tp_attn_proj_bwd(zero, do, x, C, wq, wo, dX, dC, dWq, None, dWo, None, H)   # dC, dWo
    ws = torch.empty(tp.tp_attn_recompute_workspace_size(c.cfg, T), dtype=torch.uint8, device="cuda")
    tp.tp_attn_recompute_bwd(QKV, c.cfg, C, lse, dC, dQKV, ws, seq_starts=c.starts_d)
    tp.tp_attn_proj_bwd(dQKV, do, x, C, wq, wo, dX, dC, dWq, None, dWo, None, H)
    assert tp.tp_get_status() == tp.TP_OK
    Xn, Wqn, Won, dOn = f64(X), [f64(t) for t in Wq], [f64(t) for t in Wo], f64(dO)
    rQ, _ = O.attn_proj_fwd(Xn, Wqn, None, np.zeros((T, h)), Won, None)[:2]
    rC, rl, _ = O.attention_lse(rQ, c.starts, c.cfg)
    rO = O.attn_proj_fwd(Xn, Wqn, None, rC, Won, None)[1]
    rdC = np.concatenate([dOn @ w for w in Won], 1)
    rdQ = O.attention_lse_grad(rQ, c.starts, c.cfg, rC, rl, rdC)[0]
    rdX = sum(rdQ[:, i * 3 * h // N:(i + 1) * 3 * h // N] @ Wqn[i] for i in range(N))
    rdW = [rdQ[:, i * 3 * h // N:(i + 1) * 3 * h // N].T @ Xn for i in range(N)]
    # the framework's bar for chains of bf16 intermediates: 2e-2 of the largest value
    for got, ref in [(O_, rO), (dX, rdX)] + list(zip(dWq, rdW)):
        assert np.max(np.abs(f64(got) - ref)) <= 2e-2 * np.max(np.abs(ref))


# ----------------------------------------------------------------------------
# refused or bad calls that reach the device
# ----------------------------------------------------------------------------
def test_bad_sequence_starts_are_reported():
    """Starts that decrease or leave the buffer: the kernels clamp them, write only inside the buffers and report
    TP_ERR_INVALID once."""
    tp = _tp()
    c = Case([100, 100], 2, 2, 64, 1, True, tail=1, seed=51)
    c.device()
    Q = c.QKV.cuda()
    for bad in ([0, 150, 100], [-5, 100, 200], [0, 100, 202], [0, 1 << 40, 200], [-(1 << 62), 0, 1 << 62]):
        c.starts_d = torch.tensor(bad, dtype=torch.int64, device="cuda")
        C, lse = torch.zeros(c.T, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, c.T, device="cuda")
        tp.tp_attn_recompute_fwd(Q, c.cfg, C, lse, seq_starts=c.starts_d)
        assert tp.tp_get_status() == tp.TP_ERR_INVALID
        assert tp.tp_get_status() == tp.TP_OK
        c.bwd(C, lse)
        assert tp.tp_get_status() == tp.TP_ERR_INVALID
    run(Case([100, 100], 2, 2, 64, 1, True, tail=1, seed=51))


def test_no_rows():
    tp = _tp()
    cfg = dict(b=0, s=1, n_heads=2, n_kv_heads=2, d=64, N=1, causal=True)
    e = lambda *s, **k: torch.empty(*s, device="cuda", **k)  # noqa: E731
    bf = torch.bfloat16
    tp.tp_attn_recompute_fwd(e(0, 384, dtype=bf), cfg, e(0, 128, dtype=bf), e(2, 0))
    t = torch.full((16, 2), 5.0, device="cuda")
    tp.tp_attn_relbias_bwd(e(0, 384, dtype=bf), cfg, BIAS, torch.ones(16, 2, device="cuda"), e(0, 128, dtype=bf),
                           e(2, 0), e(0, 128, dtype=bf), e(0, 384, dtype=bf), t, e(0, dtype=torch.uint8))
    torch.cuda.synchronize()
    assert (t == 0).all() and tp.tp_get_status() == tp.TP_OK


@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_a_wait_that_runs_out_returns(which):
    """The copy that the first product waits for is left out: the call ends with TP_ERR_TIMEOUT and the next one
    is right."""
    tp = _tp()
    c = Case([300], 2, 2, 64, 1, True, seed=61)
    C, lse = c.fwd()
    torch.cuda.synchronize()
    tp.tp_debug_set_wait_limit_ms(20)
    try:
        tp.tp_debug_inject_fault(1)
        if which == "fwd":
            c.fwd()
        else:
            c.bwd(C, lse)
        assert tp.tp_get_status() == tp.TP_ERR_TIMEOUT
    finally:
        tp.tp_debug_inject_fault(0)
        tp.tp_debug_set_wait_limit_ms(0)
    run(c)


def test_binding_refuses():
    tp = _tp()
    c = Case([64], 2, 2, 64, 1, True, seed=71).device()
    Q, C, lse = c.QKV.cuda(), torch.zeros(64, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 64, device="cuda")
    ok = lambda **k: tp.tp_attn_recompute_fwd(**{**dict(QKV=Q, cfg=c.cfg, C=C, lse=lse), **k})  # noqa: E731
    ok()
    with pytest.raises(TypeError):
        ok(QKV=Q.float())
    with pytest.raises(TypeError):
        ok(lse=lse.half())
    with pytest.raises(TypeError):
        ok(seq_starts=torch.tensor([0, 64], dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        ok(C=C.cpu())
    with pytest.raises(ValueError):
        ok(C=C[:, :64])
    with pytest.raises(ValueError):
        ok(lse=lse.t())
    with pytest.raises(ValueError):
        ok(QKV=Q.t().contiguous().t())
    with pytest.raises(ValueError):
        ok(seq_starts=torch.tensor([0, 32, 64], device="cuda"))
    with pytest.raises(tp.TPError) as e:
        ok(cfg=dict(c.cfg, s=63))
    assert e.value.status == tp.TP_ERR_INVALID
    with pytest.raises(tp.TPError) as e:
        tp.tp_attn_recompute_bwd(Q, c.cfg, C, lse, C, torch.empty_like(Q), torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == tp.TP_ERR_WORKSPACE
    assert tp.tp_get_status() == tp.TP_OK


# ----------------------------------------------------------------------------
# buckets that hide keys, many sequences
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("low", [float("-inf"), torch.finfo(torch.float32).min])
@pytest.mark.parametrize("d", [64, 128])
def test_buckets_that_hide_keys(low, d):
    """-infinity (or the lowest fp32) in the last bucket: a window of max_distance keys.  The first key tiles of a
    late row are hidden altogether."""
    bias = dict(num_buckets=4, max_distance=60, bidirectional=False)
    c = Case([500, 30], 2, 1, d, 1, True, bias=bias, seed=81)
    c.table[3] = low
    C, lse = c.fwd()
    g, t = c.bwd(C, lse)
    c.table[3] = float("-inf")
    check(c, C, lse, g, t)
    assert (t[3] == 0).all()


@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_no_key(causal):
    """Every bucket of one head hidden: zeros, lse of -infinity, no gradient; the other head is not touched by it."""
    bias = dict(num_buckets=8, max_distance=20, bidirectional=True)
    c = Case([200, 77], 2, 2, 64, 1, causal, bias=bias, seed=82)
    C0, lse0 = c.fwd()
    g0, t0 = c.bwd(C0, lse0)
    c.table[:, 1] = float("-inf")
    C, lse = c.fwd()
    g, t = c.bwd(C, lse)
    assert (C[:, 64:] == 0).all() and (lse[1] == float("-inf")).all() and (t[:, 1] == 0).all()
    cols = lambda j: [slice(x, x + 64) for x in O.grouped_head_columns(64, 2, 2, 1, j)]  # noqa: E731
    for a, b in zip(cols(0), cols(1)):
        assert (g[:, b] == 0).all() and torch.equal(g[:, a], g0[:, a])
    assert torch.equal(C[:, :64], C0[:, :64]) and torch.equal(lse[0], lse0[0]) and torch.equal(t[:, 0], t0[:, 0])


def test_many_sequences():
    """More sequences than a warp holds and than there are SMs, each of its own length, some empty: every one as if
    it were alone."""
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 200, 300)]
    c = Case(lens, 4, 2, 64, 1, True, tail=5, seed=83)
    C, lse = c.fwd()
    g, _ = c.bwd(C, lse)
    check(c, C, lse, g)


@pytest.mark.parametrize("bias", [None, BIAS])
def test_mostly_empty_sequences(bias):
    """Far more sequences than rows."""
    lens = [0] * 20000 + [77] + [0] * 9000 + [300, 1] + [0] * 5000
    c = Case(lens, 2, 1, 64, 1, True, bias=bias, seed=85)
    run(c)


def test_growing_scores():
    """Each key tile's scores lie far above the one before: the exponents' reference moves at every tile."""
    c = Case([640], 1, 1, 64, 1, False, scale=1.0, seed=84)
    X = c.QKV.float()
    X[:, :64] = 1.0 / 64
    X[:, 64:128] = (torch.arange(640) // 128 * 30.0)[:, None] + X[:, 64:128] * 0.5
    c.QKV = X.to(torch.bfloat16)
    C, lse = c.fwd()
    g, _ = c.bwd(C, lse)
    check(c, C, lse, g)


# ----------------------------------------------------------------------------
# few heads and long sequences: clusters of CTAs share a tile's work.  (On 152 SMs
# the forward, dQ, and dK with dV take as many CTAs an item as stands beside.)
# ----------------------------------------------------------------------------
FEW = [  # lens, query heads, key/value heads, d, shards, causal, tail
    ([2100], 1, 1, 128, 1, True, 0),        # 4, 4, 4: the first rows' items have less tiles than CTAs
    ([2100], 1, 1, 64, 1, False, 0),        # 4, 4, 4
    ([600], 8, 1, 128, 1, True, 0),         # 1, 1, 8
    ([600], 6, 1, 64, 1, False, 3),         # 1, 1, 8: 30 query tiles by 8 CTAs
    ([1290], 3, 1, 96, 1, True, 0),         # 4, 4, 8
    ([1700], 2, 2, 40, 2, True, 0),         # 4, 4, 4
    ([2700, 0], 1, 1, 128, 1, False, 130),  # an empty one, rows behind: 4, 4, 4
    ([1800, 900], 2, 1, 72, 1, True, 0),    # 2, 2, 4
    ([2048], 8, 2, 64, 1, True, 0),         # 1, 1, 4
    ([4000], 8, 1, 64, 1, False, 0),        # 1, 1, 4: in more than one round
]


@pytest.mark.parametrize("lens,H,KV,d,N,causal,tail", FEW)
def test_few_heads(lens, H, KV, d, N, causal, tail):
    run(Case(lens, H, KV, d, N, causal, tail=tail, seed=91 + d))


@pytest.mark.parametrize("lens,H,KV,d,causal,nb,md,both", [
    ([2100], 1, 1, 128, True, 32, 128, False),
    ([2100], 1, 1, 64, False, 32, 128, True),
    ([1290], 2, 1, 64, False, 64, 1024, True),
    ([600], 8, 1, 96, True, 8, 20, True),
])
def test_few_heads_with_a_bias(lens, H, KV, d, causal, nb, md, both):
    run(Case(lens, H, KV, d, 1, causal, 1.0, bias=dict(num_buckets=nb, max_distance=md, bidirectional=both), seed=92 + d))


@pytest.mark.parametrize("d", [64, 128])
def test_few_heads_and_hidden_buckets(d):
    """A window of 60 keys: of the CTAs that share a tile, some see no key of a row; and all of them, where every
    bucket is hidden."""
    bias = dict(num_buckets=4, max_distance=60, bidirectional=False)
    c = Case([2000], 1, 1, d, 1, True, bias=bias, seed=93)
    c.table[3] = float("-inf")
    C, lse = c.fwd()
    g, t = c.bwd(C, lse)
    check(c, C, lse, g, t)
    assert (t[3] == 0).all()
    c.table[:] = float("-inf")
    C, lse = c.fwd()
    g, t = c.bwd(C, lse)
    assert (C == 0).all() and (lse == float("-inf")).all() and (g == 0).all() and (t == 0).all()


def test_few_heads_neighbours_bits_and_graph():
    """Rows beside the sequences that are not numbers, equal calls, a table's gradient left out, another stream, and
    a captured graph that is replayed: the same bits."""
    tp = _tp()
    for bias in (None, BIAS):
        c = Case([1150, 1200], 2, 1, 128, 1, True, tail=60, head=20, bias=bias, seed=94)
        C, lse = c.fwd()
        g, t = c.bwd(C, lse)
        for bad in (float("nan"), float("inf")):
            Q, dC, C2, l2 = c.QKV.cuda(), c.dC.cuda(), C.clone(), lse.clone()
            for x in (Q, dC, C2):
                x[:20] = bad
                x[2370:] = bad
            l2[:, :20] = bad
            l2[:, 2370:] = bad
            fC, fl = c.fwd(Q)
            g2, _ = c.bwd(C2, l2, Q, dC)
            assert torch.equal(fC, C) and torch.equal(fl, lse) and torch.equal(g2, g)
        if bias:
            assert torch.equal(c.bwd(C, lse, dtable=None)[0], g)
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            C2, lse2 = c.fwd()
            g2, _ = c.bwd(C2, lse2)
        st.synchronize()
        assert torch.equal(C2, C) and torch.equal(lse2, lse) and torch.equal(g2, g)
    c = Case([2100], 1, 1, 128, 1, True, seed=95)
    C, lse = c.fwd()
    g, _ = c.bwd(C, lse)
    Q, dC, C2, lse2, dQ = c.QKV.cuda(), c.dC.cuda(), torch.zeros_like(C), torch.zeros_like(lse), torch.zeros_like(g)
    ws = torch.empty(tp.tp_attn_recompute_workspace_size(c.cfg, c.T), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tp.tp_attn_recompute_fwd(Q, c.cfg, C2, lse2)
        tp.tp_attn_recompute_bwd(Q, c.cfg, C2, lse2, dC, dQ, ws)
    for _ in range(3):
        C2.zero_(), lse2.zero_(), dQ.zero_()
        graph.replay()
        assert torch.equal(C2, C) and torch.equal(lse2, lse) and torch.equal(dQ, g)
    assert tp.tp_get_status() == tp.TP_OK


@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_few_heads_a_wait_that_runs_out_returns(which):
    tp = _tp()
    c = Case([2100], 1, 1, 128, 1, True, seed=96)
    C, lse = c.fwd()
    torch.cuda.synchronize()
    tp.tp_debug_set_wait_limit_ms(20)
    try:
        tp.tp_debug_inject_fault(1)
        if which == "fwd":
            c.fwd()
        else:
            c.bwd(C, lse)
        assert tp.tp_get_status() == tp.TP_ERR_TIMEOUT
    finally:
        tp.tp_debug_inject_fault(0)
        tp.tp_debug_set_wait_limit_ms(0)
    run(c)
