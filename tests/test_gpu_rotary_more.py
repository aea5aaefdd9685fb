"""More of the rotation of queries and keys and of their norms: what the call just before has written, positions and
frequencies at their ends, every form in place, with the projections and the attention of wide heads."""
import math
import random
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle.tp_oracle as O
import synthetic_inputs as SI
from tests.gpu_util import assert_close, f64
from tests.test_gpu_rotary import NORMS, Case, _tp

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------
# gains that the kernel before writes
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("lens,d,norm", [([40], 64, "rms"), ([3], 512, "layer"), ([900, 700], 128, "rms")])
def test_gains_written_by_the_call_before(lens, d, norm):
    """The optimizer's step of the gains, the forward, the backward, and the next step from the gradients that it left,
    in a row: the same bits as with a wait behind every call and no launch before the last kernel has ended."""
    tp = _tp()
    c = Case(lens, 4, 2, d, 2, norm=norm, seed=60)
    X, dY, w = c.X.cuda(), c.dY.cuda(), c.where()
    hyper = dict(lr=0.05, beta1=0.9, beta2=0.95, eps=1e-8, max_norm=0.0, use_scaler=0, min_scale=1.0, growth_factor=2.0,
                 backoff_factor=0.5, growth_interval=1000, hysteresis=2)

    def chain(wait):
        gains, grads = [g.clone() for g in c.g()], [SI.normal(61, i, (d,), 1.0, "f32").cuda() for i in range(2)]
        groups = [dict(param=p, grad=g, m=torch.zeros_like(p), v=torch.zeros_like(p), weight_decay=0.0)
                  for p, g in zip(gains, grads)]
        state, ows = tp.make_optimizer_state(), torch.empty(tp.tp_adam_step_workspace_size(), dtype=torch.uint8, device="cuda")
        ws, out = c.ws(), [(torch.empty_like(X), torch.empty_like(X)) for _ in range(8)]
        seen = []
        for Y, dX in out:
            for call in (lambda: tp.tp_adam_step(groups, hyper, state, ows),
                         lambda: tp.tp_qk_norm_rotary_fwd(X, c.cfg, c.norm, c.rot, *gains, Y, **w),
                         lambda: tp.tp_adam_step(groups, hyper, state, ows),
                         lambda: tp.tp_qk_norm_rotary_bwd(X, c.cfg, c.norm, c.rot, *gains, dY, dX, *grads, ws, **w)):
                call()
                if wait:
                    torch.cuda.synchronize()
            seen += [Y, dX]
        return seen + gains + grads

    tp.tp_debug_set_pdl(0)
    try:
        want = chain(True)
    finally:
        tp.tp_debug_set_pdl(1)
    assert not torch.equal(want[0], want[2])  # (the gains do move)
    for _ in range(4):
        got = chain(False)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert tp.tp_get_status() == tp.TP_OK


# ----------------------------------------------------------------------------
# blocks whose number an SM's shared memory limits, not their registers
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("lens,H,KV,d,inter,dtype", [([9000, 77], 8, 2, 128, False, "bf16"), ([6000], 8, 2, 128, False, "f32"),
                                                     ([5000], 8, 2, 64, False, "f32"), ([4845], 1, 1, 512, True, "bf16"),
                                                     ([6007], 1, 1, 128, True, "f32")])
def test_fewer_blocks_an_sm(lens, H, KV, d, inter, dtype, norm):
    """Wide tables and stages of fp32: fewer blocks on an SM than their registers allow, many steps a block."""
    Case(lens, H, KV, d, 1, None, inter, norm=norm, dtype=dtype, seed=62).check()


# ----------------------------------------------------------------------------
# angles
# ----------------------------------------------------------------------------
def _pi():
    """pi to 2^-400: 16 arctan(1/5) - 4 arctan(1/239) (Machin) in whole numbers."""
    one = 1 << 420

    def arctan(n):
        total, power, k = 0, one // n, 0
        while power:
            total += (-1) ** k * (power // (2 * k + 1))
            power //= n * n
            k += 1
        return total

    return Fraction(16 * arctan(5) - 4 * arctan(239), one)


@pytest.mark.parametrize("inter", [False, True])
def test_angles_within_their_bound(inter):
    """Frequencies of 2^-70 to 2^20 radians and positions to the ends of int64.  A pair (1, 0) becomes the cosine and the
    sine of its angle, which the header bounds: freq / 2 pi is off by 2^-52 of itself and 2^-64 of a turn, the position
    multiplies that, 2^-32 of a turn is cut off, and cosine and sine are good to 2^-23.  Against the angle in whole
    numbers; pairs that may be off by a radian and more are only finite."""
    tp = _tp()
    rng = random.Random(7)
    two_pi = 2 * _pi()
    freq = [0.0, 2.0 ** 20, math.pi, 2.0 ** -70] + [2.0 ** rng.uniform(-70, 20) for _ in range(252)]
    pos = [0, 1, -1, (1 << 63) - 1, -(1 << 63)] + [rng.choice((-1, 1)) * int(2 ** rng.uniform(0, 62)) for _ in range(59)]
    T, n = len(pos), 2 * len(freq)
    first = slice(0, n, 2) if inter else slice(0, n // 2)
    second = slice(1, n, 2) if inter else slice(n // 2, n)
    X = torch.zeros(T, 3 * n)
    X[:, first] = 1
    Y = torch.empty(T, 3 * n, device="cuda")
    tp.tp_rotary_fwd(X.cuda(), dict(n_heads=1, n_kv_heads=1, d=n, N=1),
                     dict(n_rot=n, interleaved=inter, freq=torch.tensor(freq, dtype=torch.float64)), Y,
                     positions=torch.tensor(pos).cuda())
    Y = Y.double().cpu()
    assert torch.isfinite(Y).all()
    compared = 0
    for t, at in enumerate(pos):
        c, s = Y[t, :n][first].tolist(), Y[t, :n][second].tolist()
        for k, f in enumerate(freq):
            turns = at * Fraction(f) / two_pi
            allowed = 2 * math.pi * (abs(at) * (f / (2 * math.pi) * 2.0 ** -52 + 2.0 ** -64) + 2.0 ** -32) + 2.0 ** -23
            if allowed >= 1:
                continue
            compared += 1
            a = float(turns % 1 * two_pi)  # (fp64 adds less than 2^-50)
            assert abs(c[k] - math.cos(a)) <= allowed and abs(s[k] - math.sin(a)) <= allowed, (at, f)
    assert compared > T * len(freq) // 2


# ----------------------------------------------------------------------------
# in place
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,n_rot,inter", [(96, 96, False), (96, 60, False), (40, 22, False), (64, 26, False), (104, 26, True),
                                           (64, 64, True), (512, 502, False)])
def test_every_form_in_place(d, n_rot, inter, dtype, norm):
    """Vectors of every width, single elements (an odd number of pairs: they go through shared memory) and both layouts,
    over the input and the gradient over the output's: the same bits, gains' gradients too (which rows and heads a block
    takes does not depend on it)."""
    c = Case([50, 3, 200], 8, 4, d, 4, n_rot, inter, 0.5, norm=norm, dtype=dtype, head=1, tail=2, seed=63)
    Y, (dX, dg) = c.fwd(), c.bwd()
    X, D = c.X.cuda(), c.dY.cuda()
    c.fwd(X, X)
    _, dg2 = c.bwd(dY=D, dX=D)
    u = torch.from_numpy(c.used).cuda()
    assert torch.equal(X[u], Y[u]) and torch.equal(D[u], dX[u])
    assert torch.equal(X[~u].cpu(), c.X[~u.cpu()]) and torch.equal(D[~u].cpu(), c.dY[~u.cpu()])
    assert norm is None or all(torch.equal(a, b) for a, b in zip(dg, dg2))
    assert _tp().tp_get_status() == 0


# ----------------------------------------------------------------------------
# with the projections and the attention that stores its probabilities
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("b,s,H,d,N,n_rot,inter", [(1, 136, 2, 512, 2, 512, False), (2, 64, 4, 128, 2, 128, True),
                                                   (1, 72, 4, 64, 4, 32, False)])
def test_between_projection_and_core(b, s, H, d, N, n_rot, inter, norm):
    """tp_attn_proj_fwd, norm and rotation, tp_attn_core_fwd, tp_attn_proj_fwd of its context, and all the way back.
    Against fp64 from the GPU's own QKV on; the projections from what the GPU gave them, at the bf16 bar.

    The rotated heads are rounded to bf16 (half a step 2^-8 each), so a score, a sum of magnitude up to s = max sum |q k| /
    sqrt(d), is off by 2 2^-8 s, and P by that of itself; P, dS, C and the gradients are rounded to bf16 once more each.  As
    a whole (2-norm over 2-norm) outputs are within 8 roundings of bf16 and twice the scores' error."""
    tp = _tp()
    T, h = b * s, H * d
    bf = dict(dtype=torch.bfloat16, device="cuda")
    cfg = dict(b=b, s=s, n_heads=H, n_kv_heads=H, d=d, N=N, causal=True, scale=0.0)
    rot = tp.tp_rotary_frequencies(n_rot, interleaved=inter)
    nrm = norm and dict(kind=norm, eps=1e-5)
    X, dO = SI.normal(64, 1, (T, h), 1.0, "bf16").cuda(), SI.normal(64, 2, (T, h), 1.0, "bf16").cuda()
    Wq = [SI.normal(64, 10 + i, (3 * h // N, h), 0.5 * h ** -0.5, "bf16").cuda() for i in range(N)]
    Wo = [SI.normal(64, 30 + i, (h, h // N), h ** -0.5, "bf16").cuda() for i in range(N)]
    gains = [(SI.normal(64, 5 + i, (d,), 0.1, "f32") + 0.5).cuda() for i in range(2)]
    QKV, R, dR, dQKV = [torch.full((T, 3 * h), float("nan"), **bf) for _ in range(4)]
    C, Out, dX, dC, unused = [torch.zeros(T, h, **bf) for _ in range(5)]
    P = torch.empty(b, H, s, s, **bf)
    f32 = dict(device="cuda")
    dWq, dWo = [torch.empty(3 * h // N, h, **f32) for _ in range(N)], [torch.empty(h, h // N, **f32) for _ in range(N)]
    dg = [torch.empty(d, device="cuda") for _ in "qk"]
    ws = torch.empty(tp.tp_attn_core_workspace_size(T, s, h, H), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(tp.tp_qk_norm_rotary_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    tp.tp_attn_proj_fwd(X, Wq, None, C, Wo, None, QKV, unused, H)
    if norm:
        tp.tp_qk_norm_rotary_fwd(QKV, cfg, nrm, rot, *gains, R)
    else:
        tp.tp_rotary_fwd(QKV, cfg, rot, R)
    tp.tp_attn_core_fwd(R, s, H, N, True, P, C, None, ws)
    tp.tp_attn_proj_fwd(X, Wq, None, C, Wo, None, torch.empty_like(QKV), Out, H)
    # the gradient of the context comes out of the projections' backward, beside what the gradient of QKV gives
    tp.tp_attn_proj_bwd(torch.zeros_like(QKV), dO, X, C, Wq, Wo, dX, dC, dWq, None, dWo, None, H)
    tp.tp_attn_core_bwd(R, P, C, dC, s, H, N, True, dR, ws)
    if norm:
        tp.tp_qk_norm_rotary_bwd(QKV, cfg, nrm, rot, *gains, dR, dQKV, *dg, ws2)
    else:
        tp.tp_rotary_bwd(dR, cfg, rot, dQKV)
    tp.tp_attn_proj_bwd(dQKV, dO, X, C, Wq, Wo, dX, torch.empty_like(dC), dWq, None, dWo, None, H)
    assert tp.tp_get_status() == tp.TP_OK

    wq, wo = [f64(w) for w in Wq], [f64(w) for w in Wo]
    q, o = O.attn_proj_fwd(f64(X), wq, None, f64(C), wo, None)
    assert_close(QKV, q, "bf16", "QKV")
    assert_close(Out, o, "bf16", "O")
    g = O.attn_proj_bwd(f64(dQKV), f64(dO), f64(X), f64(C), wq, wo)
    assert_close(dX, g["dX"], "bf16", "dX")
    assert_close(dC, g["dC"], "bf16", "dC")
    for i in range(N):
        assert_close(dWq[i], g["dWqkv"][i], "bf16", "dWqkv")

    x, pos, dc = f64(QKV), O.rotary_positions(T, s=s), f64(dC)
    ga = dict(zip("qk", [f64(t) for t in gains]))
    r = O.qk_norm_rotary(x, pos, cfg, rot, nrm, ga)
    c, p = O.attention_core(r, s, H, N, True)
    dx, wg = O.qk_norm_rotary_grad(x, O.attention_core_grad(r, p, dc, s, H, N), pos, cfg, rot, nrm, ga)
    top = 0.0
    for j in range(H):
        qc, kc, _, _ = O.attention_head_columns(h, H, N, j)
        for at in range(0, T, s):
            top = max(top, np.max(np.abs(r[at:at + s, qc:qc + d]) @ np.abs(r[at:at + s, kc:kc + d]).T) * d ** -0.5)
    bound = 8 * 2.0 ** -8 + 2 * 2 * 2.0 ** -8 * top
    assert bound < 0.3  # (so that a sign or a head in the wrong place shows)
    for got, want in ((R, r), (C, c), (dQKV, dx)) + (tuple(zip(dg, (wg["q"], wg["k"]))) if norm else ()):
        off = np.linalg.norm(f64(got) - want) / np.linalg.norm(want)
        assert off <= bound, off
    # the gradient along itself against differences of the loss sum(C dC) in fp64
    E = dx / np.linalg.norm(dx)

    def loss(step):
        return (O.attention_core(O.qk_norm_rotary(x + step * E, pos, cfg, rot, nrm, ga), s, H, N, True)[0] * dc).sum()

    want = (loss(1e-4) - loss(-1e-4)) / 2e-4
    assert abs((dx * E).sum() - want) <= 1e-5 * abs(want)
    assert abs((f64(dQKV) * E).sum() - want) <= bound * abs(want)


# ----------------------------------------------------------------------------
# what the profiler counts
# ----------------------------------------------------------------------------
def test_profile_counts():
    """Every entry point under its own name, with its calls and kernel launches."""
    tp = _tp()
    few, many, plain = Case([8], 2, 1, 16, 1, norm="rms"), Case([3000], 2, 1, 16, 1, norm="rms"), Case([8], 2, 1, 16, 1)
    tp.tp_profile_reset()
    tp.tp_profile_enable(1)
    try:
        for c in (few, few, many):
            c.fwd()
            c.bwd()
        many.bwd(dg=(None, None))
        plain.fwd()
        plain.bwd()
        plain.bwd()
        torch.cuda.synchronize()
        got = tp.tp_profile_read()
    finally:
        tp.tp_profile_enable(0)
        tp.tp_profile_reset()
    counts = {k: v[:2] for k, v in got.items() if "rotary" in k}
    # the sum of the gains' gradients is a second launch, but in a call of few rows or without such gradients
    assert counts == {"rotary_fwd": (1, 1), "rotary_bwd": (2, 2), "qk_norm_rotary_fwd": (3, 3), "qk_norm_rotary_bwd": (4, 5)}
