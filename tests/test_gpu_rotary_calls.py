"""The rotation of queries and keys and their norms among other calls: before and behind attention, captured and
replayed, on streams of their own and beside each other, with launch chaining on and off."""
import numpy as np
import pytest
import torch

import oracle.tp_oracle as O
import synthetic_inputs as SI
from tests.gpu_util import f64
from tests.test_gpu_rotary import Case, _tp

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------
# as they are used: projection, norm and rotation, attention, and back
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("norm", [None, "rms", "layer"])
@pytest.mark.parametrize("lens,H,KV,d,N,n_rot,inter", [([64, 64], 4, 4, 64, 2, 64, False), ([70, 1, 33], 8, 2, 32, 2, 16, True),
                                                       ([130], 4, 1, 128, 1, 128, False), ([40, 25], 4, 2, 40, 2, 40, False)])
def test_between_projection_and_attention(norm, lens, H, KV, d, N, n_rot, inter):
    """QKV = X W^T, its heads normed and rotated, attention of the result; the gradient of QKV from that of the context.
    Against the same in fp64 on the GPU's own QKV, from which the chain of calls begins.

    The rotated heads and their gradient are rounded to bf16 on the way (half a step 2^-8), P and dS once more inside
    the attention: the scores, sums of magnitude up to s = max sum |q k| scale, are off by 2 2^-8 s, so P by that of
    itself.  Each later sum carries those relative errors of its terms; as a whole (2-norm over 2-norm) the outputs are
    within 8 roundings of bf16 and twice the scores' error."""
    tp = _tp()
    g = dict(dtype=torch.bfloat16, device="cuda")
    T, W, h = sum(lens), (H + 2 * KV) * d, 96
    starts = np.cumsum([0] + lens)
    even = len(set(lens)) == 1
    st = None if even else torch.tensor(starts, dtype=torch.int64, device="cuda")
    cfg = dict(b=len(lens), s=max(lens), n_heads=H, n_kv_heads=KV, d=d, N=N, causal=True, scale=0.0)
    rot = tp.tp_rotary_frequencies(n_rot, interleaved=inter)
    nrm = norm and dict(kind=norm, eps=1e-5)
    X, Wt = SI.normal(30, 1, (T, h), 1.0, "bf16").cuda(), SI.normal(30, 2, (W, h), h ** -0.5, "bf16").cuda()
    QKV = (X.float() @ Wt.float().t()).to(torch.bfloat16)
    dC = SI.normal(30, 3, (T, H * d), 1.0, "bf16").cuda()
    gains = [(SI.normal(30, 4 + i, (d,), 0.2, "f32") + 1).cuda() for i in range(2)]
    R, C, lse = torch.empty_like(QKV), torch.empty(T, H * d, **g), torch.empty(H, T, device="cuda")
    dR, dQKV = torch.empty_like(QKV), torch.empty_like(QKV)
    dg = [torch.empty(d, device="cuda") for _ in "qk"]
    ws = torch.empty(tp.tp_attn_recompute_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(tp.tp_qk_norm_rotary_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    if norm:
        tp.tp_qk_norm_rotary_fwd(QKV, cfg, nrm, rot, *gains, R, seq_starts=st)
    else:
        tp.tp_rotary_fwd(QKV, cfg, rot, R, seq_starts=st)
    tp.tp_attn_recompute_fwd(R, cfg, C, lse, seq_starts=st)
    tp.tp_attn_recompute_bwd(R, cfg, C, lse, dC, dR, ws, seq_starts=st)
    if norm:
        tp.tp_qk_norm_rotary_bwd(QKV, cfg, nrm, rot, *gains, dR, dQKV, *dg, ws2, seq_starts=st)
    else:
        tp.tp_rotary_bwd(dR, cfg, rot, dQKV, seq_starts=st)
    assert tp.tp_get_status() == tp.TP_OK
    x, pos = f64(QKV), O.rotary_positions(T, starts)
    ga = dict(zip("qk", [f64(t) for t in gains]))
    r = O.qk_norm_rotary(x, pos, cfg, rot, nrm, ga)
    c, l, _ = O.attention_lse(r, starts, cfg)
    dr = O.attention_lse_grad(r, starts, cfg, c, l, f64(dC))[0]
    dx, wg = O.qk_norm_rotary_grad(x, dr, pos, cfg, rot, nrm, ga)
    top = 0.0
    for j in range(H):
        qc, kc, _ = O.grouped_head_columns(d, H, KV, N, j)
        for a, e in zip(starts[:-1], starts[1:]):
            top = max(top, np.max(np.abs(r[a:e, qc:qc + d]) @ np.abs(r[a:e, kc:kc + d]).T) * d ** -0.5)
    bound = 8 * 2.0 ** -8 + 2 * 2 * 2.0 ** -8 * min(top, 4.0)
    for got, want in ((R, r), (C, c), (dQKV, dx)) + (tuple(zip(dg, (wg["q"], wg["k"]))) if norm else ()):
        off = np.linalg.norm(f64(got) - want) / np.linalg.norm(want)
        assert off <= bound, off
    # gradients against differences of the loss sum(C dC), in fp64, along a random direction
    E = np.random.default_rng(1).standard_normal(x.shape)

    def loss(step):
        return (O.attention_lse(O.qk_norm_rotary(x + step * E, pos, cfg, rot, nrm, ga), starts, cfg)[0] * f64(dC)).sum()

    want = (loss(1e-5) - loss(-1e-5)) / 2e-5
    assert abs((dx * E).sum() - want) <= 1e-5 * np.abs(dx * E).sum()
    assert abs((f64(dQKV) * E).sum() - want) <= bound * np.linalg.norm(dx) * np.linalg.norm(E)


# ----------------------------------------------------------------------------
# captured, on other streams, beside each other
# ----------------------------------------------------------------------------
def _cases():
    return [Case([300, 1, 77], 8, 2, 128, 2, norm="rms", tail=3, seed=40), Case([64] * 3, 4, 4, 64, 4, 32, True, seed=41),
            Case([900], 4, 4, 40, 2, norm="layer", dtype="f32", seed=42), Case([31], 2, 1, 64, 1, 20, norm="rms", seed=43)]


class Job:
    """One case's buffers, and its calls on them."""

    def __init__(self, c):
        self.c, self.X, self.dY = c, c.X.cuda(), c.dY.cuda()
        self.Y, self.dX = torch.zeros_like(self.X), torch.zeros_like(self.X)
        self.dg = [torch.zeros(c.d, device="cuda") for _ in "qk"]
        self.w, self.g = c.where(), c.g()
        self.wsp = c.ws() if c.norm else None

    def run(self, stream=None):
        tp, c = _tp(), self.c
        k = dict(self.w, stream=stream)
        if c.norm:
            tp.tp_qk_norm_rotary_fwd(self.X, c.cfg, c.norm, c.rot, *self.g, self.Y, **k)
            tp.tp_qk_norm_rotary_bwd(self.X, c.cfg, c.norm, c.rot, *self.g, self.dY, self.dX, *self.dg, self.wsp, **k)
        else:
            tp.tp_rotary_fwd(self.X, c.cfg, c.rot, self.Y, **k)
            tp.tp_rotary_bwd(self.dY, c.cfg, c.rot, self.dX, **k)

    def out(self):
        return [self.Y, self.dX] + self.dg

    def clear(self):
        for t in self.out():
            t.fill_(float("nan"))


def _wanted(jobs):
    for j in jobs:
        j.run()
    torch.cuda.synchronize()
    return [[t.clone() for t in j.out()] for j in jobs]


def _same(jobs, want):
    used = [torch.from_numpy(j.c.used).cuda() for j in jobs]
    for j, w, u in zip(jobs, want, used):
        for a, b in zip(j.out()[:2], w[:2]):
            assert torch.equal(a[u], b[u])
        if j.c.norm:
            assert all(torch.equal(a, b) for a, b in zip(j.dg, w[2:]))


def test_captured_and_replayed():
    """One graph of all cases, replayed on inputs, positions and starts that change under it."""
    tp = _tp()
    jobs = [Job(c) for c in _cases()]
    want = _wanted(jobs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for j in jobs:
            j.run()
    for _ in range(3):
        for j in jobs:
            j.clear()
        graph.replay()
        torch.cuda.synchronize()
        _same(jobs, want)
    j = jobs[0]
    j.X.copy_(j.X.flip(0))
    j.w["seq_starts"].copy_(torch.tensor([2, 50, 50, 380]))
    for t in j.out():
        t.fill_(3.0)
    graph.replay()
    got = [t.clone() for t in j.out()]
    assert (got[0][:2] == 3).all() and (got[1][380:] == 3).all()
    j.run()
    assert all(torch.equal(a, b) for a, b in zip(got, j.out()))
    assert tp.tp_get_status() == tp.TP_OK


def test_first_call_of_a_shape_inside_a_capture():
    """Shapes whose kernels never ran before: the device's first call set them up."""
    tp = _tp()
    a = Job(Case([20], 2, 2, 88, 2, 44, norm="layer", seed=44))
    b = Job(Case([20], 2, 2, 88, 2, 6, dtype="f32", seed=45))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run(), b.run()
    for j in (a, b):
        j.clear()
    graph.replay()
    torch.cuda.synchronize()
    got = [[t.clone() for t in j.out()] for j in (a, b)]
    _wanted([a, b])
    _same([a, b], got)
    assert tp.tp_get_status() == tp.TP_OK


def test_streams_and_calls_at_once():
    """On streams of their own, several at the same time; torch's stream and one that is given are the same."""
    tp = _tp()
    jobs = [Job(c) for c in _cases()] + [Job(Case([2000, 1500], 8, 8, 64, 8, norm="rms", seed=46)) for _ in range(2)]
    want = _wanted(jobs)
    streams = [torch.cuda.Stream() for _ in jobs]
    for rep in range(5):
        for j in jobs:
            j.clear()
        torch.cuda.synchronize()
        for i, (j, s) in enumerate(zip(jobs, streams)):
            if (i + rep) % 2:
                j.run(stream=s)
            else:
                with torch.cuda.stream(s):
                    j.run()
        torch.cuda.synchronize()
        _same(jobs, want)
    assert tp.tp_get_status() == tp.TP_OK


def test_launch_chaining_on_and_off():
    """Calls in a row, each on what the one before left, with programmatic launches and without: the same bits."""
    tp = _tp()
    c = Case([256] * 2, 4, 2, 64, 2, norm="rms", seed=47)

    def chain():
        X = c.X.cuda()
        bufs = [torch.empty_like(X) for _ in range(2)]
        for i in range(20):
            c.fwd(X if i == 0 else bufs[(i + 1) % 2], bufs[i % 2])
        dX, dg = c.bwd(dY=bufs[1])
        return bufs[1], dX, *dg

    a = chain()
    tp.tp_debug_set_pdl(0)
    try:
        b = chain()
    finally:
        tp.tp_debug_set_pdl(1)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_equal_calls_give_equal_bits():
    for c in _cases():
        j = Job(c)
        want = _wanted([j])
        for _ in range(3):
            j.clear()
            j.run()
            torch.cuda.synchronize()
            _same([j], want)


def test_profile_names():
    tp = _tp()
    a, b = Job(Case([8], 2, 1, 16, 1, norm="rms")), Job(Case([8], 2, 1, 16, 1))
    tp.tp_profile_reset()
    tp.tp_profile_enable(1)
    try:
        a.run(), b.run()
        torch.cuda.synchronize()
        got = tp.tp_profile_read()
    finally:
        tp.tp_profile_enable(0)
        tp.tp_profile_reset()
    text = str(got)
    for name in ("rotary_fwd", "rotary_bwd", "qk_norm_rotary_fwd", "qk_norm_rotary_bwd"):
        assert name in text, text


def test_binding_checks():
    """What the binding refuses: other devices' and types' tensors, shapes, strides, a workspace that is too small."""
    tp = _tp()
    c = Case([6], 4, 2, 32, 2, norm="rms", seed=48)
    X, Y, w = c.X.cuda(), torch.empty_like(c.X).cuda(), torch.zeros(32, device="cuda")
    f = lambda **k: tp.tp_qk_norm_rotary_fwd(**dict(dict(QKV=X, cfg=c.cfg, norm=c.norm, rot=c.rot, gq=w, gk=w, Out=Y), **k))  # noqa: E731
    f()
    for bad, error in ((dict(Out=Y.float()), TypeError), (dict(Out=Y[:-1]), ValueError), (dict(Out=Y.cpu()), ValueError),
                       (dict(Out=None), TypeError), (dict(Out=Y.t().contiguous().t()), ValueError), (dict(QKV=X[:, :-8]), ValueError),
                       (dict(QKV=X.half()), TypeError), (dict(gq=w[:-1]), ValueError), (dict(gk=w.half()), TypeError),
                       (dict(gq=w.cpu()), ValueError), (dict(positions=torch.zeros(6, dtype=torch.int32, device="cuda")), TypeError),
                       (dict(positions=torch.zeros(5, dtype=torch.int64, device="cuda")), ValueError),
                       (dict(seq_starts=torch.zeros(3, dtype=torch.int64, device="cuda")), ValueError),
                       (dict(rot=dict(c.rot, freq=c.rot["freq"].cuda())), ValueError)):
        with pytest.raises(error):
            f(**bad)
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(tp.TPError) as e:
        tp.tp_qk_norm_rotary_bwd(X, c.cfg, c.norm, c.rot, w, w, Y, torch.empty_like(Y), w.clone(), w.clone(), small)
    assert e.value.status == tp.TP_ERR_WORKSPACE
    assert tp.tp_get_status() == tp.TP_OK
