"""GPU parity of the rotation of queries and keys by position (tp_rotary_*) and of their norms with it
(tp_qk_norm_rotary_*) against the fp64 oracle.

Bounds, element by element, from the arithmetic; u = 2^-24 is half a step of fp32:
  * cosines and sines are off by 1.6 u (an angle of up to pi / 4 is rounded once, the series' last steps once each, its
    rest is below u / 2, and the turns' 2^-32nds are 0.03 u); the amplitude, a product and a sum round once each: a
    rotated value is off by
        e_c (|x1| + |x2|) m,  e_c = 6 u + |position| max(freq) 2^-52
    (the last term: freq / 2 pi in a double);
  * a sum of squares adds 16 terms a lane and at most 5 levels of lanes: 21 u of itself, half of that after the root,
    rsqrtf 4 u, the mean and eps 2 u: r is off by e_r = 17 u of itself; a mean is off by 22 u of the mean magnitude;
  * the backward's sums over d likewise by 22 u of their magnitudes; the gains' gradients are sums of at most 310 terms in a
    row, then of at most 64: 400 u of the magnitudes;
  * results are rounded once: 2^-8 (bf16), 2^-24 (fp32) of the value.
"""
import numpy as np
import pytest
import torch

import oracle.tp_oracle as O
import synthetic_inputs as SI
from tests.gpu_util import f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _tp():
    import megatron_tensor_transformer_tp_gb300 as tp
    return tp


class Case:
    def __init__(self, lens, H, KV, d, N, n_rot=None, inter=False, amp=1.0, base=10000.0, norm=None, dtype="bf16",
                 head=0, tail=0, positions=None, seed=0, gains=True, packed=None):
        tp = _tp()
        self.H, self.KV, self.d, self.N = H, KV, d, N
        starts = [head]
        for n in lens:
            starts.append(starts[-1] + n)
        self.starts, self.T = starts, starts[-1] + tail
        self.packed = (len(set(lens)) > 1 or tail or head) if packed is None else packed
        self.cfg = dict(b=len(lens), s=max(lens), n_heads=H, n_kv_heads=KV, d=d, N=N)
        n_rot = d if n_rot is None else n_rot
        self.rot = dict(tp.tp_rotary_frequencies(n_rot, base, interleaved=inter), amplitude=amp) if n_rot else None
        self.norm = norm and dict(kind=norm, eps=1e-5)
        W = (H + 2 * KV) * d
        self.X, self.dY = SI.normal(seed, 1, (self.T, W), 1.0, dtype), SI.normal(seed, 2, (self.T, W), 1.0, dtype)
        g = SI.normal(seed, 3, (2, d), 0.3, "f32") + 1
        self.gains = dict(q=g[0].contiguous(), k=g[1].contiguous()) if gains and norm else dict(q=None, k=None)
        self.positions = None if positions is None else torch.tensor(positions, dtype=torch.int64)
        self.pos = O.rotary_positions(self.T, starts) if positions is None else np.array(positions)
        self.used = (np.arange(self.T) >= starts[0]) & (np.arange(self.T) < starts[-1])

    def where(self):
        d = lambda t: None if t is None else t.cuda()  # noqa: E731
        return dict(seq_starts=d(torch.tensor(self.starts)) if self.packed else None, positions=d(self.positions))

    def g(self):
        return [None if self.gains[k] is None else self.gains[k].cuda() for k in "qk"]

    def fwd(self, X=None, Y=None, **k):
        tp = _tp()
        X = self.X.cuda() if X is None else X
        Y = torch.full_like(X, 7.0) if Y is None else Y
        if self.norm:
            tp.tp_qk_norm_rotary_fwd(X, self.cfg, self.norm, self.rot, *self.g(), Y, **self.where(), **k)
        else:
            tp.tp_rotary_fwd(X, self.cfg, self.rot, Y, **self.where(), **k)
        return Y

    def ws(self):
        n = _tp().tp_qk_norm_rotary_workspace_size(self.cfg, self.T)
        return torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN wherever it is read unwritten

    def bwd(self, X=None, dY=None, dX=None, dg="new", accumulate=False, **k):
        tp = _tp()
        dY = self.dY.cuda() if dY is None else dY
        dX = torch.full_like(dY, 7.0) if dX is None else dX
        if not self.norm:
            tp.tp_rotary_bwd(dY, self.cfg, self.rot, dX, **self.where(), **k)
            return dX, (None, None)
        X = self.X.cuda() if X is None else X
        if isinstance(dg, str):
            dg = [torch.full((self.d,), 7.0, device="cuda") for _ in "qk"]
        tp.tp_qk_norm_rotary_bwd(X, self.cfg, self.norm, self.rot, *self.g(), dY, dX, *dg,
                                 self.ws() if dg[0] is not None or dg[1] is not None else None, accumulate=accumulate,
                                 **self.where(), **k)
        return dX, dg

    # -- what comes out, and how far off it may be ------------------------------------------------------------------
    def _rot(self):
        return self.rot or dict(n_rot=0, interleaved=False, freq=[], amplitude=1.0)

    def _off(self, x, e):
        """Bound of the rotation of rows x that are off by e already."""
        n, r = self._rot()["n_rot"], self._rot()
        out = np.array(e)
        if n:
            i, j = (np.arange(0, n, 2), np.arange(1, n, 2)) if r["interleaved"] else (np.arange(n // 2), np.arange(n // 2, n))
            m = abs(r["amplitude"])
            far = np.abs(self.pos[self.used]).max(initial=0) * float(torch.as_tensor(r["freq"]).max()) * 2.0 ** -52
            both = m * ((6 * U + far) * (np.abs(x[:, i]) + np.abs(x[:, j])) + e[:, i] + e[:, j])
            out[:, i], out[:, j] = both, both
        return out

    def _normed(self, x):
        n, r = O.head_norm(x, self.norm["kind"], self.norm["eps"])
        e = 20 * U * np.abs(n)
        if self.norm["kind"] == "layer":
            e = e + 23 * U * np.abs(x).mean(1, keepdims=True) * r * (1 + np.abs(n))
        return n, r, e

    def _gain(self, kind):
        return np.ones(self.d) if self.gains[kind] is None else f64(self.gains[kind])

    def expect_fwd(self):
        X, half = f64(self.X)[self.used], HALF[self.X.dtype]
        pos, Y = self.pos[self.used], np.array(X)
        B = np.zeros_like(X)
        for c, kind in O.qk_heads(self.cfg):
            x, e = X[:, c:c + self.d], np.zeros((len(X), self.d))
            if self.norm:
                x, _, e = self._normed(x)
                x, e = x * self._gain(kind), e * np.abs(self._gain(kind)) + U * np.abs(x * self._gain(kind))
            Y[:, c:c + self.d] = O.rotate_heads(x, pos, self._rot())
            B[:, c:c + self.d] = self._off(x, e) + half * np.abs(Y[:, c:c + self.d])
        return Y, B

    def expect_bwd(self):
        X, D, half = f64(self.X)[self.used], f64(self.dY)[self.used], HALF[self.X.dtype]
        pos, d = self.pos[self.used], self.d
        dX, B = np.array(D), np.zeros_like(D)
        dg, bg = {k: np.zeros(d) for k in "qk"}, {k: np.zeros(d) for k in "qk"}
        for c, kind in O.qk_heads(self.cfg):
            col, dy = slice(c, c + d), D[:, c:c + d]
            dz = O.rotate_heads(dy, pos, self._rot(), back=True)
            ez = self._off(dy, np.zeros_like(dy))
            if not self.norm:
                dX[:, col], B[:, col] = dz, ez + half * np.abs(dz)
                continue
            n, r, en = self._normed(X[:, col])
            dg[kind] += (dz * n).sum(0)
            bg[kind] += (ez * np.abs(n) + np.abs(dz) * en + 402 * U * np.abs(dz * n)).sum(0)
            g = np.abs(self._gain(kind))
            e, ee = dz * self._gain(kind), ez * g + U * np.abs(dz) * g
            mean = lambda v: v.mean(1, keepdims=True)  # noqa: E731
            along = mean(e * n)
            e_along = mean(ee * np.abs(n) + np.abs(e) * en + 24 * U * np.abs(e * n))
            off = ee + np.abs(n) * e_along + en * np.abs(along) + 3 * U * (np.abs(e) + np.abs(n * along))
            dx = e - n * along
            if self.norm["kind"] == "layer":
                dx = dx - mean(e)
                off = off + mean(ee + 24 * U * np.abs(e))
            dX[:, col] = r * dx
            B[:, col] = r * (off + 20 * U * np.abs(dx)) + half * np.abs(dX[:, col])
        return dX, B, dg, bg

    def check(self):
        Y = self.fwd()
        dX, dg = self.bwd()
        assert _tp().tp_get_status() == 0
        u = self.used
        want, B = self.expect_fwd()
        within(f64(Y)[u], want, B, "Out")
        assert (f64(Y)[~u] == 7).all() and (f64(dX)[~u] == 7).all()
        want, B, wg, bg = self.expect_bwd()
        within(f64(dX)[u], want, B, "dQKV")
        if self.norm:
            for k, got in zip("qk", dg):
                within(f64(got), wg[k], bg[k], "dg" + k)
        return Y, dX, dg


def within(got, ref, bound, what):
    if not ref.size:
        return
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - ref) - 1.01 * bound - 1e-37
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 0, f"{what}{list(map(int, at))}: {got[at]} is {abs(got - ref)[at]:.3e} off {ref[at]}, allowed {bound[at]:.3e}"


NORMS = [None, "rms", "layer"]


@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,n_rot", [(128, 128), (64, 64), (128, 64), (512, 512), (256, 32), (8, 8), (8, 2), (40, 40),
                                     (96, 96), (104, 26), (120, 120), (72, 24), (488, 488), (504, 502), (16, 6),
                                     (256, 254), (24, 20), (80, 20), (488, 484), (512, 4)])
def test_widths(d, n_rot, dtype, inter, norm):
    """Head widths of one vector to 64, whole heads and parts of every remainder, both layouts."""
    Case([9, 1, 23], 4, 2, d, 2, n_rot, inter, 1.25, norm=norm, dtype=dtype, tail=3, seed=1).check()


@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("H,KV,N", [(1, 1, 1), (8, 8, 8), (6, 3, 3), (32, 8, 4), (16, 1, 1), (24, 4, 2), (7, 7, 1)])
def test_heads(H, KV, N, norm):
    Case([5, 5], H, KV, 64, N, norm=norm, seed=2).check()


@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("H,KV,N,d", [(2048, 2048, 8, 8), (4088, 8, 8, 16), (4094, 2, 2, 512), (301, 301, 1, 64),
                                      (90, 45, 5, 128)])
def test_many_heads(H, KV, N, d, norm):
    """More heads than a block takes, up to the most, and numbers that do not fill the last block."""
    Case([3], H, KV, d, N, norm=norm, seed=19).check()


@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("lens,head,tail", [([1], 0, 0), ([1], 3, 2), ([2048], 0, 0), ([700, 1, 333, 64], 0, 40),
                                            ([0, 5, 0, 0, 4, 0], 2, 3), ([1] * 200, 0, 1), ([4000, 97, 5000], 0, 0),
                                            ([0], 4, 4), ([3] * 1500, 0, 7)])
def test_lengths(lens, head, tail, norm):
    """Sequences of no token, of one, long ones and many; unused rows before and behind them."""
    Case(lens, 4, 1, 64, 1, norm=norm, head=head, tail=tail, packed=True, seed=3).check()


@pytest.mark.parametrize("b,s", [(1, 1), (3, 5), (2, 4096), (5000, 1), (7, 1303)])
def test_even_sequences(b, s):
    c = Case([s] * b, 2, 2, 32, 2, norm="rms", seed=4)
    assert not c.packed
    Y, dX, dg = c.check()
    c.packed = True  # the same by starts
    for x, y in zip((Y, dX, *dg), (c.fwd(), *[t for g in [c.bwd()] for t in (g[0], *g[1])])):
        assert torch.equal(x, y)


def test_many_sequences():
    """More sequences than a block has threads, 32-fold search in three steps, empty ones between."""
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 4, 40000) * (rng.random(40000) < 0.3)]
    Case(lens, 1, 1, 8, 1, norm="rms", head=5, tail=5, seed=5).check()


@pytest.mark.parametrize("b", [1, 2, 30, 31, 32, 33, 1023, 1024, 1025])
def test_numbers_of_sequences(b):
    """Around what a warp holds at once, and what it finds in one, two and three steps."""
    rng = np.random.default_rng(b)
    lens = [int(x) for x in rng.integers(0, 9, b)]
    lens[-1] += 1
    Case(lens, 2, 2, 16, 2, norm="rms", head=3, tail=2, packed=True, seed=20).check()


@pytest.mark.parametrize("T", [1, 2, 31, 500])
@pytest.mark.parametrize("norm", NORMS)
def test_given_positions(T, norm):
    """Single tokens, each at its own place: positions count, rows and sequences do not."""
    rng = np.random.default_rng(T)
    pos = [int(x) for x in rng.integers(0, 1 << 17, T)]
    Case([1] * T, 8, 2, 128, 2, norm=norm, positions=pos, packed=False, seed=6).check()
    Case([T], 8, 2, 128, 2, 64, True, norm=norm, positions=pos, packed=False, seed=6).check()


def test_positions_inside_sequences():
    """With both, positions turn and starts say which rows are used."""
    Case([3, 4], 2, 1, 16, 1, positions=[9, 8, 7, 100, 0, 0, 3, 5, 1], head=1, tail=1, seed=7).check()


def test_far_positions():
    """Positions up to the ends of int64: a pair's angle goes by the product modulo a turn.  freq = 2 pi j / 2^32 moves
    whole 2^-32nds of a turn, so the exact angle is known in whole numbers."""
    import math
    tp = _tp()
    turns = [1, 3, 1 << 20, (1 << 31) + 5, 12345678, 0, 7, 1 << 30]
    freq = torch.tensor([2 * math.pi * j / 2.0 ** 32 for j in turns], dtype=torch.float64)
    pos = [0, 1, -1, 12345, (1 << 31) + 7, -(1 << 40) + 3, 1 << 52, (1 << 62) + 11, (1 << 63) - 1, -(1 << 63)]
    T, d = len(pos), 16
    X = SI.normal(8, 1, (T, 3 * d), 1.0, "f32").cuda()
    Y = torch.empty_like(X)
    tp.tp_rotary_fwd(X, dict(n_heads=1, n_kv_heads=1, d=d, N=1), dict(n_rot=d, interleaved=False, freq=freq), Y,
                     positions=torch.tensor(pos).cuda())
    x, y = f64(X), f64(Y)
    for t, at in enumerate(pos):
        for k, j in enumerate(turns):
            # freq / 2 pi is j 2^-32 to 2^-53 of itself: far positions multiply that
            slack = abs(at) * j * 2.0 ** -32 * 2.0 ** -51 * 2 * math.pi + abs(at) * 2.0 ** -63 * 2 * math.pi
            if slack > 2.0 ** -20:
                continue
            a = 2 * math.pi * ((at * j) % (1 << 32)) / 2.0 ** 32
            for c in (0, d):
                x1, x2 = x[t, c + k], x[t, c + k + 8]
                tol = (7 * U + slack) * (abs(x1) + abs(x2))
                assert abs(y[t, c + k] - (x1 * math.cos(a) - x2 * math.sin(a))) <= tol
                assert abs(y[t, c + k + 8] - (x1 * math.sin(a) + x2 * math.cos(a))) <= tol
    assert torch.isfinite(Y).all()


@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(norm, dtype):
    """Over the input, and the gradient over the output's: the same bits, value heads and unused rows untouched.  (The
    gains' gradients sum other heads together, as the value heads are not visited: both are within the bounds.)"""
    c = Case([50, 3, 20], 8, 4, 96, 4, 60, norm=norm, dtype=dtype, head=1, tail=2, seed=9)
    Y, (dX, dg) = c.fwd(), c.bwd()
    X = c.X.cuda()
    D = c.dY.cuda()
    assert c.fwd(X, X) is X
    dX2, dg2 = c.bwd(dY=D, dX=D)
    u = torch.from_numpy(c.used).cuda()
    assert torch.equal(X[u], Y[u]) and torch.equal(dX2[u], dX[u])
    assert torch.equal(X[~u].cpu(), c.X[~u.cpu()]) and torch.equal(D[~u].cpu(), c.dY[~u.cpu()])
    if norm:
        _, _, want, bound = c.expect_bwd()
        for k, a, b in zip("qk", dg, dg2):
            within(f64(a), want[k], bound[k], "dg" + k)
            within(f64(b), want[k], bound[k], "dg" + k)


@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("dtype,u,n_rot", [("bf16", 8, 40), ("f32", 4, 40), ("bf16", 8, 22)])
def test_slices_of_wider_buffers(dtype, u, n_rot, norm):
    """Row pitches of their own, multiples of 16 bytes (u elements); what lies between the rows stays."""
    c = Case([30, 11], 4, 2, 40, 2, n_rot, norm=norm, dtype=dtype, tail=1, seed=10)
    Y, (dX, dg) = c.fwd(), c.bwd()
    T, W = c.X.shape

    def wide(t, left, right):
        big = torch.full((T, left + W + right), 5.0, dtype=t.dtype, device="cuda")
        big[:, left:left + W] = t
        return big, big[:, left:left + W]

    _, X = wide(c.X.cuda(), u, 3 * u)
    _, D = wide(c.dY.cuda(), 2 * u, 0)
    bigY, Y2 = wide(torch.full_like(Y, 7.0), u, 5 * u)
    bigG, dX2 = wide(torch.full_like(dX, 7.0), 0, u)
    c.fwd(X, Y2)
    _, dg2 = c.bwd(X, D, dX2)
    assert torch.equal(Y, Y2) and torch.equal(dX, dX2)
    assert (bigY[:, :u] == 5).all() and (bigY[:, u + W:] == 5).all() and (bigG[:, W:] == 5).all()
    if norm:
        assert all(torch.equal(a, b) for a, b in zip(dg, dg2))


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_gains(norm):
    """No gains, one gradient of two, none, and adding to old values."""
    Case([40], 4, 2, 64, 1, norm=norm, gains=False, seed=11).check()
    c = Case([40], 4, 2, 64, 1, norm=norm, seed=11)
    dX, (a, b) = c.bwd()
    one = torch.full((64,), 3.0, device="cuda")
    assert torch.equal(c.bwd(dg=(one, None))[0], dX) and torch.equal(one, a)
    assert torch.equal(c.bwd(dg=(None, one))[0], dX) and torch.equal(one, b)
    assert torch.equal(c.bwd(dg=(None, None))[0], dX)
    old = [torch.randn(64, device="cuda") for _ in "qk"]
    _, new = c.bwd(dg=[t.clone() for t in old], accumulate=True)
    assert torch.equal(new[0], old[0] + a) and torch.equal(new[1], old[1] + b)


def test_norms_alone():
    for kind in ("rms", "layer"):
        for d in (64, 104):
            c = Case([21], 4, 2, d, 2, 0, norm=kind, seed=12)
            assert c.rot is None
            Y, dX, dg = c.check()
            c.rot = dict(n_rot=0, freq=None)
            assert torch.equal(Y, c.fwd()) and torch.equal(dX, c.bwd()[0])


def test_no_rows():
    tp = _tp()
    c = dict(b=0, s=0, n_heads=2, n_kv_heads=1, d=16, N=1)
    r, norm = tp.tp_rotary_frequencies(16), dict(kind="rms", eps=1e-6)
    X = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    dg = [torch.full((16,), 3.0, device="cuda") for _ in "qk"]
    tp.tp_rotary_fwd(X, c, r, X)
    tp.tp_qk_norm_rotary_fwd(X, c, norm, r, None, None, X)
    tp.tp_qk_norm_rotary_bwd(X, c, norm, r, None, None, X, X.clone(), *dg, None, accumulate=True)
    assert all((g == 3).all() for g in dg)
    tp.tp_qk_norm_rotary_bwd(X, c, norm, r, None, None, X, X.clone(), *dg, None)
    assert all((g == 0).all() for g in dg) and tp.tp_get_status() == tp.TP_OK


@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("n_rot,inter", [(32, False), (32, True), (20, False), (24, False), (18, True)])
def test_not_finite(norm, n_rot, inter):
    """NaN and infinities stay in their row, head and kind; a rotation alone keeps them in their pair or column;
    those of unused rows and of values reach nothing."""
    c = Case([30], 4, 2, 64, 2, n_rot, inter, norm=norm, head=2, tail=2, seed=13)
    Y, (dX, dg) = c.fwd(), c.bwd()
    X, D = c.X.cuda(), c.dY.cuda()
    nan, inf = float("nan"), float("inf")
    for t in (X, D):
        t[0], t[-1] = nan, inf  # unused
        t[5, 3 * 64 + 1] = nan  # shard 0: Q0 Q1 K0 V0, a value
    Y2, (dX2, dg2) = c.fwd(X), c.bwd(X, D)
    u = torch.from_numpy(c.used).cuda()
    keep = u[:, None].repeat(1, Y.shape[1])
    keep[5, 3 * 64 + 1] = False
    assert torch.equal(Y[keep], Y2[keep]) and torch.equal(dX[keep], dX2[keep])
    assert norm is None or all(torch.equal(a, b) for a, b in zip(dg, dg2))
    X[7, 64 + 40], X[9, 4], D[7, 64 + 40], D[9, 4] = inf, nan, inf, nan
    Y2, (dX2, _) = c.fwd(X), c.bwd(X, D)
    for a, b in ((Y, Y2), (dX, dX2)):
        if norm:
            keep[7, 64:128] = keep[9, :64] = False
            assert torch.isnan(b[9, :64]).all()
        else:
            keep[7, 64 + 40] = False
            partner = (4 ^ 1) if inter else 4 + n_rot // 2
            keep[9, 4] = keep[9, partner] = False
            assert b[7, 64 + 40] == inf and torch.isnan(b[9, 4]) and torch.isnan(b[9, partner])
        assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_head_of_equal_values(norm):
    """Heads of zeros, and of one value: r is 1 / sqrt(eps) where nothing is left of the head."""
    c = Case([6], 2, 1, 64, 1, norm=norm, seed=14)
    c.X[1] = 0.0
    c.X[2] = 1.0
    c.X[3, :64] = 2.0 ** -60
    c.check()


@pytest.mark.parametrize("starts", [[5, 3, 60], [0, 70, 64], [-5, 20, 64], [0, 20, 65], [0, 1 << 62, 64],
                                    [-(1 << 62), 1 << 62, 3]])
@pytest.mark.parametrize("norm", [None, "rms"])
def test_bad_starts_are_reported(starts, norm):
    """Starts that decrease or leave the buffer: every access stays inside (rows are only compared with them), the
    call is reported, and the next one is right."""
    tp = _tp()
    c = Case([30, 34], 4, 2, 64, 2, norm=norm, packed=True, seed=15)
    want = c.fwd()
    good, c.starts = c.starts, starts
    big = torch.full((64 + 2, c.X.shape[1]), 7.0, dtype=torch.bfloat16, device="cuda")
    c.fwd(Y=big[1:-1])
    assert tp.tp_get_status() == tp.TP_ERR_INVALID
    assert (big[0] == 7).all() and (big[-1] == 7).all()
    c.bwd()
    assert tp.tp_get_status() == tp.TP_ERR_INVALID
    c.starts = good
    assert torch.equal(c.fwd(), want) and tp.tp_get_status() == tp.TP_OK


def test_many_rows():
    """More tiles than blocks in the backward, and rows that do not fill the last tile."""
    Case([40003], 1, 1, 16, 1, norm="rms", seed=16).check()
    Case([30001, 20000], 1, 1, 8, 1, 6, norm="layer", dtype="f32", tail=13, seed=17).check()
    Case([1500000], 1, 1, 8, 1, norm="rms", seed=21).check()
    Case([700001, 3], 2, 1, 8, 1, 4, True, tail=1, seed=22).check()


def test_amplitude_and_frequencies_at_their_ends():
    """An amplitude of 0 counts as 1; frequencies of 0, of whole turns and beyond a turn a position."""
    import math
    tp = _tp()
    c = Case([40], 2, 1, 16, 1, amp=1.0, seed=23)
    Y = c.fwd()
    c.rot["amplitude"] = 0.0
    assert torch.equal(c.fwd(), Y)
    c.rot = dict(c.rot, amplitude=None)
    assert torch.equal(c.fwd(), Y)
    c.rot = dict(c.rot, amplitude=0.25, freq=torch.tensor([0.0, 6.5, 2 * math.pi, 100.0, 1e-300, 1048576.0, 1e-5, math.pi],
                                                          dtype=torch.float64))
    c.check()
    assert tp.tp_get_status() == tp.TP_OK


def test_rows_far_apart():
    """Offsets beyond 2^32 elements: 260 rows 2^24 + 64 elements apart, in one 8.7 GB buffer."""
    c = Case([260], 2, 1, 16, 1, norm="rms", seed=18)
    pitch = (1 << 24) + 64
    buf = torch.empty(260 * pitch, dtype=torch.bfloat16, device="cuda")
    X = buf.as_strided((260, 64), (pitch, 1))
    Y = buf.as_strided((260, 64), (pitch, 1), 64)
    D = buf.as_strided((260, 64), (pitch, 1), 128)
    G = buf.as_strided((260, 64), (pitch, 1), 192)
    X.copy_(c.X)
    D.copy_(c.dY)
    want, (dX, dg) = c.fwd(), c.bwd()
    c.fwd(X, Y)
    _, dg2 = c.bwd(X, D, G)
    assert torch.equal(want, Y) and torch.equal(dX, G) and all(torch.equal(a, b) for a, b in zip(dg, dg2))
