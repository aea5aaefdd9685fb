"""More sizes of attention without stored probabilities against the fp64 oracle (bounds as in
test_gpu_attn_recompute.py): every head width, long sequences alone and among many short ones, a table of zeros against
no table, and calls with a bias on two streams at once."""
import pytest
import torch

from tests.test_gpu_attn_recompute import BIAS, Case, _tp, check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bias", [None, dict(num_buckets=32, max_distance=128, bidirectional=True)])
@pytest.mark.parametrize("d", [16, 24, 48, 56, 88, 104, 112, 120])
def test_head_widths(d, bias):
    """Widths of whole and half 32-byte stores, in the first and the second half of a row."""
    run(Case([130, 1, 300], 4, 2, d, 2, bias is None, 1.0 if bias else 0.0, tail=5, bias=bias, seed=500 + d))


@pytest.mark.parametrize("lens,H,KV,d,causal,bias", [
    ([4500], 2, 1, 64, True, None),
    ([5001], 1, 1, 128, False, None),
    ([4231], 2, 2, 64, False, dict(num_buckets=32, max_distance=128, bidirectional=True)),
    ([4777], 1, 1, 96, True, dict(num_buckets=64, max_distance=1024, bidirectional=False)),
])
def test_long_sequences(lens, H, KV, d, causal, bias):
    run(Case(lens, H, KV, d, 1, causal, bias=bias, seed=520 + d))


@pytest.mark.parametrize("short", [20, 45])  # with up to 32 sequences long ones go first, beyond in their own order
@pytest.mark.parametrize("bias", [None, BIAS])
def test_one_long_sequence_among_short_ones(short, bias):
    lens = [3, 64, 0, 1, 130] * (short // 5)
    lens.insert(len(lens) // 2, 2500)
    run(Case(lens, 4, 1, 64, 1, True, tail=7, bias=bias, seed=530 + short))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,H,KV,d,same", [
    ([640], 4, 2, 64, True),      # tiles nearer than the largest distance and beyond it
    ([500, 77], 2, 1, 128, True),
    ([2100], 1, 1, 128, False),   # dQ is summed by clusters without a bias and by single CTAs with one
    ([2100], 1, 1, 64, False),
])
def test_a_table_of_zeros_against_no_table(lens, H, KV, d, same, causal):
    """Forward and backward.  The scale is a power of two, so the scores round the same with and without a table:
    equal bits, but for dQ where other CTAs share its sums."""
    bias = dict(num_buckets=16, max_distance=40, bidirectional=True)
    c = Case(lens, H, KV, d, 1, causal, scale=0.25, bias=bias, seed=540 + d)
    c.table = torch.zeros_like(c.table)
    p = Case(lens, H, KV, d, 1, causal, scale=0.25, seed=540 + d)
    assert torch.equal(c.QKV, p.QKV)
    C, lse = c.fwd()
    Cp, lsep = p.fwd()
    assert torch.equal(C, Cp) and torch.equal(lse, lsep)
    g, t = c.bwd(C, lse)
    gp, _ = p.bwd(C, lse)
    check(c, C, lse, g, t)
    check(p, C, lse, gp)
    n = 0 if same else H * d
    assert torch.equal(g[:, n:], gp[:, n:])


def test_calls_with_a_bias_on_two_streams_at_once():
    """Each with its own table, workspace and gradient of the table."""
    cases = [Case([700, 55], 4, 2, 128, 1, True, bias=BIAS, seed=550),
             Case([400, 123], 8, 8, 64, 1, False, bias=dict(num_buckets=32, max_distance=128, bidirectional=True), seed=551)]
    want = []
    for c in cases:
        C, lse = c.fwd()
        want.append((C, lse) + c.bwd(C, lse))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        torch.cuda.synchronize()
        got = []
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                C, lse = c.fwd()
                got.append((C, lse) + c.bwd(C, lse))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert _tp().tp_get_status() == _tp().TP_OK


@pytest.mark.parametrize("bias", [None, BIAS])
def test_a_graph_replayed_on_other_lengths(bias):
    """The starts are read when the graph runs: other lengths, empty ones and unused rows among them."""
    tp = _tp()
    T, H, KV, d = 900, 4, 2, 64
    plans = [[900, 0, 0, 0], [1, 300, 299, 300], [128, 128, 128, 128], [0, 513, 0, 200], [0, 0, 0, 0]]
    cases = [Case(lens, H, KV, d, 2, True, tail=T - sum(lens), bias=bias, seed=560 + i, packed=True)
             for i, lens in enumerate(plans)]
    bf = dict(dtype=torch.bfloat16, device="cuda")
    Q, dC, starts = torch.zeros(T, (H + 2 * KV) * d, **bf), torch.zeros(T, H * d, **bf), torch.zeros(5, dtype=torch.int64, device="cuda")
    C, lse, dQ = torch.zeros(T, H * d, **bf), torch.zeros(H, T, device="cuda"), torch.zeros(T, (H + 2 * KV) * d, **bf)
    table = torch.zeros(bias["num_buckets"], H, device="cuda") if bias else None
    dt = torch.zeros_like(table) if bias else None
    cfg = dict(cases[0].cfg, s=None)
    ws = torch.empty(tp.tp_attn_recompute_workspace_size(cfg, T, bias), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if bias:
            tp.tp_attn_relbias_fwd(Q, cfg, bias, table, C, lse, seq_starts=starts)
            tp.tp_attn_relbias_bwd(Q, cfg, bias, table, C, lse, dC, dQ, dt, ws, seq_starts=starts)
        else:
            tp.tp_attn_recompute_fwd(Q, cfg, C, lse, seq_starts=starts)
            tp.tp_attn_recompute_bwd(Q, cfg, C, lse, dC, dQ, ws, seq_starts=starts)
    for c in cases + cases[:2]:
        Q.copy_(c.QKV), dC.copy_(c.dC), starts.copy_(torch.tensor(c.starts))
        if bias:
            table.copy_(c.table)
        for x in (C, lse, dQ):
            x.fill_(7.0)
        ws.fill_(255)
        graph.replay()
        assert tp.tp_get_status() == tp.TP_OK
        check(c, C, lse, dQ, dt)


@pytest.mark.parametrize("lens,H,KV,d,bias", [([200, 100], 2, 1, 64, None), ([300], 1, 1, 128, BIAS), ([290], 2, 2, 40, None)])
def test_rows_far_apart(lens, H, KV, d, bias):
    """Row pitches of 2^24 elements: addresses beyond 2^32 in every matrix, and the bits of rows close together."""
    c = Case(lens, H, KV, d, 1, True, bias=bias, seed=570)
    C, lse = c.fwd()
    g, t = c.bwd(C, lse)
    pitch = 1 << 24

    def far(x):
        v = torch.empty((c.T - 1) * pitch + x.shape[1], dtype=torch.bfloat16, device="cuda").as_strided(x.shape, (pitch, 1))
        v.copy_(x)
        return v

    Q, dC, C2, dQ = far(c.QKV), far(c.dC), far(torch.zeros_like(C)), far(torch.zeros_like(g))
    lse2 = torch.zeros_like(lse)
    c.fwd(Q, C2, lse2)
    assert torch.equal(C2, C) and torch.equal(lse2, lse)
    _, t2 = c.bwd(C2, lse2, Q, dC, dQ)
    assert torch.equal(dQ, g) and (t is None or torch.equal(t2, t))
    assert _tp().tp_get_status() == _tp().TP_OK
