"""Calls of attention without stored probabilities beside each other: captured and eager ones at the same time,
and the backward's two launches."""
import pytest
import torch

from tests.test_gpu_attn_recompute import Case, _tp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_captured_calls_share_no_counter_with_later_ones(which):
    """A captured call and eager ones take their items from counters.  However many calls lie between, one that runs
    beside the graph has a counter of its own: both leave the bits that they leave alone.

    A long call that takes half of the SMs lets the graph begin on the others; when it ends, the eager call on the
    stream of higher priority takes its place, and the two run side by side."""
    tp = _tp()
    bf = dict(dtype=torch.bfloat16, device="cuda")

    class Job:
        def __init__(self, lens, H, KV, d, causal, seed):
            g = torch.Generator(device="cuda").manual_seed(seed)
            T = sum(lens)
            self.cfg = dict(b=len(lens), s=None, n_heads=H, n_kv_heads=KV, d=d, N=1, causal=causal)
            self.starts = torch.tensor([0] + lens, device="cuda").cumsum(0)
            self.Q = torch.randn(T, (H + 2 * KV) * d, generator=g, device="cuda").to(torch.bfloat16)
            self.dC = torch.randn(T, H * d, generator=g, device="cuda").to(torch.bfloat16)
            self.C, self.lse, self.dQ = torch.zeros(T, H * d, **bf), torch.zeros(H, T, device="cuda"), torch.zeros_like(self.Q)
            n = tp.tp_attn_recompute_workspace_size(self.cfg, T)
            self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")

        def fwd(self):
            tp.tp_attn_recompute_fwd(self.Q, self.cfg, self.C, self.lse, seq_starts=self.starts)

        def bwd(self):
            tp.tp_attn_recompute_bwd(self.Q, self.cfg, self.C, self.lse, self.dC, self.dQ, self.ws, seq_starts=self.starts)

        def outputs(self):
            return (self.C, self.lse) if which == "fwd" else (self.dQ,)

    lens = [3000 - 100 * i for i in range(24)]
    a, b = (Job(lens, 8, 4, 128, True, 400 + i) for i in range(2))
    long_ = Job([9728] + [1] * 100, 1, 1, 128, False, 403)  # 76 long query tiles; more items than SMs
    tiny = Job([1] * 200, 1, 1, 64, True, 402)  # more items than SMs
    want = []
    for x in (a, b):
        x.fwd(), x.bwd()
        want.append([y.clone() for y in x.outputs()])
    call = Job.fwd if which == "fwd" else Job.bwd
    torch.cuda.synchronize()

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a)
    sa, sb, sc = torch.cuda.Stream(), torch.cuda.Stream(priority=-1), torch.cuda.Stream()
    launches = 1 if which == "fwd" else 2
    for _ in range(3):
        # the eager call comes 4096 launches after the captured or the last one
        for _ in range(4096 - launches - 1):
            tiny.fwd()
        for x in (a, b):
            for y in x.outputs():
                y.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(sc):
            long_.fwd()
        with torch.cuda.stream(sa):
            graph.replay()
        with torch.cuda.stream(sb):
            call(b)
        torch.cuda.synchronize()
        for x, w in zip((a, b), want):
            assert all(torch.equal(y, z) for y, z in zip(x.outputs(), w))
    assert tp.tp_get_status() == tp.TP_OK


def test_the_second_launch_may_wait_longer_than_the_limit():
    """The kernel for dK and dV begins on SMs that dQ has left, 88 here, and waits for its last 64 items, 2 ms each:
    no wait with a limit (1 ms here) covers that."""
    tp = _tp()
    T = 6144 * 128
    cfg = dict(b=1, s=T, n_heads=1, n_kv_heads=1, d=64, N=1, causal=False)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(420)
    Q = torch.randn(T, 192, generator=gen, device="cuda").to(torch.bfloat16)
    dC = torch.randn(T, 64, generator=gen, device="cuda").to(torch.bfloat16)
    C, lse = torch.zeros(T, 64, **bf), torch.zeros(1, T, device="cuda")
    ws = torch.empty(tp.tp_attn_recompute_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    tp.tp_attn_recompute_fwd(Q, cfg, C, lse)
    a, b = torch.zeros_like(Q), torch.zeros_like(Q)
    tp.tp_attn_recompute_bwd(Q, cfg, C, lse, dC, a, ws)
    torch.cuda.synchronize()
    tp.tp_debug_set_wait_limit_ms(1)
    try:
        tp.tp_attn_recompute_bwd(Q, cfg, C, lse, dC, b, ws)
        assert tp.tp_get_status() == tp.TP_OK
    finally:
        tp.tp_debug_set_wait_limit_ms(0)
    assert torch.equal(a, b)


@pytest.mark.parametrize("bias", [None, dict(num_buckets=16, max_distance=40, bidirectional=False)])
@pytest.mark.parametrize("lens,d", [([300], 64), ([300, 190], 128), ([2100], 64), ([2100], 128)])
def test_a_wait_of_the_second_launch_runs_out(lens, d, bias):
    """The kernel for dK and dV misses its keys and values, in single CTAs and in clusters: it ends, the call is
    reported, and the next one is right.  Forward calls leave that fault for the backward."""
    tp = _tp()
    c = Case(lens, 1, 1, d, 1, True, bias=bias, seed=430)
    C, lse = c.fwd()
    g, t = c.bwd(C, lse)
    torch.cuda.synchronize()
    tp.tp_debug_set_wait_limit_ms(20)
    try:
        tp.tp_debug_inject_fault(2)
        c.fwd()
        assert tp.tp_get_status() == tp.TP_OK
        g2, t2 = c.bwd(C, lse)
        assert tp.tp_get_status() == tp.TP_ERR_TIMEOUT
    finally:
        tp.tp_debug_inject_fault(0)
        tp.tp_debug_set_wait_limit_ms(0)
    assert torch.equal(g2[:, :d], g[:, :d]) and (t is None or torch.equal(t2, t))  # dQ and the table came first
    g2, t2 = c.bwd(C, lse)
    assert tp.tp_get_status() == tp.TP_OK
    assert torch.equal(g2, g) and (t is None or torch.equal(t2, t))


def test_captured_calls_beyond_the_counters():
    """After 65536 captured launches the following ones have no counter and take their items in a fixed order: the
    same bits.  (This one uses the counters up, so it comes last.)"""
    tp = _tp()
    lens = [700 - 20 * i for i in range(20)]
    c = Case(lens, 16, 4, 64, 1, True, bias=dict(num_buckets=16, max_distance=40, bidirectional=False), seed=410)
    C, lse = c.fwd()
    g, t = c.bwd(C, lse)
    Q, dC, table = c.QKV.cuda(), c.dC.cuda(), c.table.cuda()
    C2, lse2, dQ, dt = torch.zeros_like(C), torch.zeros_like(lse), torch.zeros_like(g), torch.zeros_like(t)
    ws = torch.empty(tp.tp_attn_recompute_workspace_size(c.cfg, c.T, c.bias), dtype=torch.uint8, device="cuda")
    for _ in range(64):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(1024):
                tp.tp_attn_relbias_fwd(Q, c.cfg, c.bias, table, C2, lse2, seq_starts=c.starts_d)
        del graph
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tp.tp_attn_relbias_fwd(Q, c.cfg, c.bias, table, C2, lse2, seq_starts=c.starts_d)
        tp.tp_attn_relbias_bwd(Q, c.cfg, c.bias, table, C2, lse2, dC, dQ, dt, ws, seq_starts=c.starts_d)
    for _ in range(2):
        for x in (C2, lse2, dQ, dt):
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(C2, C) and torch.equal(lse2, lse) and torch.equal(dQ, g) and torch.equal(dt, t)
    assert tp.tp_get_status() == tp.TP_OK
