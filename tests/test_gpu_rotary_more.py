"""More of the rotation of queries and keys and of their norms: what the call just before has written, positions and
frequencies at their ends."""
import math
import random
from fractions import Fraction

import pytest
import torch

import synthetic_inputs as SI
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
