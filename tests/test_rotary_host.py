"""Host-side tests of the rotation of queries and keys by position and of their norms: the oracle's functions against
independent forms, the frequencies, and the entry points' refusals (before the device is touched)."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import megatron_tensor_transformer_tp_gb300 as tp
import oracle.tp_oracle as O

FAKE = 0x100000  # never dereferenced: every refused call fails validation first
L = tp.lib()


# ----------------------------------------------------------------------------
# oracle pins
# ----------------------------------------------------------------------------
def plain_rot(n, inter, amp=1.0, base=100.0):
    return dict(n_rot=n, interleaved=inter, freq=[base ** (-2.0 * k / n) for k in range(n // 2)], amplitude=amp)


def test_hand_made_rotation():
    x = np.array([[1.0, 2.0, 3.0, 4.0, 5.0, 6.0]])
    rot = dict(n_rot=4, interleaved=False, freq=[math.pi / 2, math.pi], amplitude=2.0)
    # pairs (1, 3) by a quarter turn and (2, 4) by half a turn, twice as long; the rest stays
    assert np.allclose(O.rotate_heads(x, [1], rot), [[-6, -4, 2, -8, 5, 6]], atol=1e-12)
    assert np.allclose(O.rotate_heads(x, [1], dict(rot, interleaved=True)), [[-4, 2, -6, -8, 5, 6]], atol=1e-12)
    assert np.allclose(O.rotate_heads(x, [1], rot, back=True), [[6, -4, -2, -8, 5, 6]], atol=1e-12)


def test_hand_made_columns_and_positions():
    # two shards of 2 query heads and 1 key/value head, d = 8: [Q0 Q1 K0 V0 | Q2 Q3 K1 V1]
    assert O.qk_heads(dict(d=8, n_heads=4, n_kv_heads=2, N=2)) == [(0, "q"), (8, "q"), (16, "k"), (32, "q"), (40, "q"),
                                                                   (48, "k")]
    assert O.rotary_positions(6, s=3).tolist() == [0, 1, 2, 0, 1, 2]
    assert O.rotary_positions(7, [1, 1, 4, 6]).tolist() == [-1, 0, 1, 2, 0, 1, -1]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("kind", [None, "rms", "layer"])
@pytest.mark.parametrize("n_rot", [0, 6, 16])
def test_oracle_against_torch(kind, inter, n_rot):
    """Explicit 2 x 2 rotations of every pair, torch's layer_norm, and autograd, in float64."""
    T, cfg = 5, dict(d=16, n_heads=4, n_kv_heads=2, N=2)
    g = torch.Generator().manual_seed(3)
    X = torch.randn(T, 8 * 16, generator=g, dtype=torch.float64, requires_grad=True)
    dY = torch.randn(T, 8 * 16, generator=g, dtype=torch.float64)
    gain = {k: torch.randn(16, generator=g, dtype=torch.float64, requires_grad=True) for k in "qk"}
    pos = [0, 3, 1, 70, 2]
    rot = plain_rot(n_rot, inter, 1.5) if n_rot else dict(n_rot=0, interleaved=inter, freq=[], amplitude=1.0)
    norm = None if kind is None else dict(kind=kind, eps=1e-3)
    parts = []
    for c in range(0, 8 * 16, 16):
        which = "v" if c // 16 % 4 == 3 else "k" if c // 16 % 4 == 2 else "q"
        x = X[:, c:c + 16]
        if which != "v":
            if kind == "layer":
                x = torch.nn.functional.layer_norm(x, (16,), gain[which], None, 1e-3)
            elif kind == "rms":
                x = x / torch.sqrt((x * x).sum(1, keepdim=True) / 16 + 1e-3) * gain[which]
            rows = []
            for t in range(T):
                R = torch.eye(16, dtype=torch.float64)
                for k in range(n_rot // 2):
                    i, j = (2 * k, 2 * k + 1) if inter else (k, k + n_rot // 2)
                    a = pos[t] * rot["freq"][k]
                    R[i, i] = R[j, j] = 1.5 * math.cos(a)
                    R[j, i] = 1.5 * math.sin(a)
                    R[i, j] = -R[j, i]
                rows.append(R @ x[t])
            x = torch.stack(rows)
        parts.append(x)
    Y = torch.cat(parts, 1)
    (Y * dY).sum().backward()
    gains = {k: v.detach().numpy() for k, v in gain.items()}
    assert np.allclose(O.qk_norm_rotary(X.detach().numpy(), pos, cfg, rot, norm, gains), Y.detach().numpy(), atol=1e-12)
    dX, dg = O.qk_norm_rotary_grad(X.detach().numpy(), dY.numpy(), pos, cfg, rot, norm, gains)
    assert np.allclose(dX, X.grad.numpy(), atol=1e-12)
    for k in "qk":
        assert norm is None or np.allclose(dg[k], gain[k].grad.numpy(), atol=1e-12)


def test_gradient_against_differences():
    rng = np.random.default_rng(5)
    cfg, norm, pos = dict(d=8, n_heads=2, n_kv_heads=1, N=1), dict(kind="layer", eps=1e-2), [4, 0, 9]
    rot = plain_rot(6, True, 0.7)
    X, dY = rng.standard_normal((3, 32)), rng.standard_normal((3, 32))
    gains = {k: rng.standard_normal(8) for k in "qk"}
    loss = lambda X, g: (O.qk_norm_rotary(X, pos, cfg, rot, norm, g) * dY).sum()  # noqa: E731
    dX, dg = O.qk_norm_rotary_grad(X, dY, pos, cfg, rot, norm, gains)
    h = 1e-5
    for t in range(3):
        for c in range(32):
            E = np.zeros_like(X)
            E[t, c] = h
            assert abs((loss(X + E, gains) - loss(X - E, gains)) / (2 * h) - dX[t, c]) < 1e-7
    for k in "qk":
        for c in range(8):
            E = np.zeros(8)
            E[c] = h
            up, down = dict(gains, **{k: gains[k] + E}), dict(gains, **{k: gains[k] - E})
            assert abs((loss(X, up) - loss(X, down)) / (2 * h) - dg[k][c]) < 1e-7


# ----------------------------------------------------------------------------
# frequencies
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("kind,more", [("plain", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
                                       ("by_turns", dict(factor=8.0, trained=8192.0, low=1.0, high=4.0)),
                                       ("by_pair", dict(factor=40.0, trained=4096.0)),
                                       ("by_pair", dict(factor=2.0, trained=64.0, low=1.5, high=8.0))])
@pytest.mark.parametrize("n_rot,base", [(4, 10000.0), (64, 10000.0), (128, 500000.0), (20, 10.0), (512, 10000.0)])
def test_frequencies(kind, more, n_rot, base):
    got = tp.tp_rotary_frequencies(n_rot, base, kind, **more)
    want, amp = O.rotary_frequencies(n_rot, base, kind, **more)
    # pow, log and a few products in doubles on both sides
    assert got["freq"].dtype == torch.float64 and np.allclose(got["freq"].numpy(), want, rtol=1e-13, atol=0)
    assert got["amplitude"] == np.float32(amp) and got["n_rot"] == n_rot and got["interleaved"] is False


def test_hand_made_frequencies():
    f = lambda *a, **k: tp.tp_rotary_frequencies(*a, **k)["freq"].tolist()  # noqa: E731
    assert np.allclose(f(4, 100.0), [1, 0.1], rtol=1e-15)
    assert np.allclose(f(4, 100.0, "linear", 4.0), [0.25, 0.025], rtol=1e-15)
    assert np.allclose(f(4, 100.0, "base", 9.0), [1, 1 / 90], rtol=1e-15)  # 100 * 9^2, its root
    # in 20 pi tokens the pairs turn 10 and 1 times
    kw = dict(factor=2.0, trained=20 * math.pi)
    assert np.allclose(f(4, 100.0, "by_turns", low=1.0, high=10.0, **kw), [1, 0.05], rtol=1e-12)
    assert np.allclose(f(4, 100.0, "by_turns", low=1.0, high=19.0, **kw), [0.75, 0.05], rtol=1e-12)
    # 8 pairs a power of ten each: pair k turns 10^(7-k) times; kept to pair 2, interpolated from pair 6
    got = f(16, 1e8, "by_pair", factor=4.0, trained=2e7 * math.pi, low=10.0 * 1.0001, high=1e5 * 0.9999)
    share = [1, 1, 1, 0.75, 0.5, 0.25, 0, 0]
    assert np.allclose(got, [10.0 ** -k * (u + (1 - u) / 4) for k, u in enumerate(share)], rtol=1e-12)


@pytest.mark.parametrize("bad", [dict(n_rot=3), dict(n_rot=0), dict(n_rot=514), dict(base=1.0), dict(base=math.nan),
                                 dict(kind="linear", factor=0.5), dict(kind="linear", factor=math.inf),
                                 dict(kind="base", n_rot=2, factor=2.0), dict(kind="by_turns", factor=2.0),
                                 dict(kind="by_pair", factor=2.0, trained=4096.0, low=4.0, high=4.0),
                                 dict(kind="by_pair", factor=2.0, trained=4096.0, low=0.0),
                                 dict(kind="base", factor=1e300, base=1e300)])
def test_frequencies_refused(bad):
    with pytest.raises(tp.TPError) as e:
        tp.tp_rotary_frequencies(**dict(dict(n_rot=64, base=10000.0), **bad))
    assert e.value.status == tp.TP_ERR_INVALID
    with pytest.raises(ValueError):
        tp.tp_rotary_frequencies(64, kind="other")
    f, a = (ctypes.c_double * 32)(), ctypes.c_float()
    sc = tp.tp_rotary_scaling(64, 5, 10000.0, 2.0, 4096.0, 1.0, 32.0)
    assert L.tp_rotary_frequencies(ctypes.byref(sc), f, ctypes.byref(a)) == tp.TP_ERR_INVALID
    sc.kind = 0
    assert L.tp_rotary_frequencies(None, f, ctypes.byref(a)) == tp.TP_ERR_INVALID
    assert L.tp_rotary_frequencies(ctypes.byref(sc), None, ctypes.byref(a)) == tp.TP_ERR_INVALID
    assert L.tp_rotary_frequencies(ctypes.byref(sc), f, None) == tp.TP_ERR_INVALID
    assert L.tp_rotary_frequencies(ctypes.byref(sc), f, ctypes.byref(a)) == tp.TP_OK


# ----------------------------------------------------------------------------
# refusals
# ----------------------------------------------------------------------------
CFG = dict(T=256, b=2, s=128, n_heads=4, n_kv_heads=2, d=64, N=2, causal=1, scale=0.0)
FREQ = (ctypes.c_double * 256)(*[0.5] * 256)


def cfg(**k):
    return ctypes.byref(tp.tp_attn_config(*[{**CFG, **k}[f] for f, _ in tp.tp_attn_config._fields_]))


def rot(n=64, inter=0, freq=FREQ, amp=1.0):
    return ctypes.byref(tp.tp_rotary_config(n, inter, ctypes.cast(freq, ctypes.c_void_p) if freq else None, amp))


def norm(kind=0, eps=1e-6):
    return ctypes.byref(tp.tp_qk_norm_config(kind, eps))


def turn(c=None, r=None, starts=None, pos=None, x=FAKE, ldx=512, y=FAKE * 2, ldy=512, dt=tp.TP_BF16, **k):
    c = cfg(**k) if c is None else c
    r = rot() if r is None else r
    got = {f(dt, c, r, starts, pos, x, ldx, y, ldy, None) for f in (L.tp_rotary_fwd, L.tp_rotary_bwd)}
    assert len(got) == 1
    return got.pop()


def fwd(n=None, r=None, gq=FAKE, gk=FAKE, starts=None, pos=None, x=FAKE, ldx=512, y=FAKE * 2, ldy=512, dt=tp.TP_BF16,
        **k):
    return L.tp_qk_norm_rotary_fwd(dt, cfg(**k), norm() if n is None else n, rot() if r is None else r, gq, gk, starts,
                                   pos, x, ldx, y, ldy, None)


def bwd(n=None, r=None, gq=FAKE * 8, gk=FAKE * 9, starts=None, pos=None, x=FAKE, ldx=512, dy=FAKE * 2, lddy=512,
        dx=FAKE * 3, lddx=512, dgq=FAKE * 4, dgk=FAKE * 5, ws=FAKE * 6, wsn=1 << 30, dt=tp.TP_BF16, **k):
    return L.tp_qk_norm_rotary_bwd(dt, cfg(**k), norm() if n is None else n, rot() if r is None else r, gq, gk, starts,
                                   pos, x, ldx, dy, lddy, dx, lddx, dgq, dgk, 0, ws, wsn, None)


CALLS = (turn, fwd, bwd)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(T=2 ** 31), dict(n_heads=0), dict(n_kv_heads=0), dict(n_kv_heads=3),
                                 dict(n_heads=6, n_kv_heads=4), dict(N=0), dict(N=9), dict(N=3), dict(d=0),
                                 dict(d=520), dict(b=0), dict(s=0), dict(s=100), dict(b=3), dict(n_heads=1 << 20, n_kv_heads=1 << 20),
                                 dict(n_heads=2050, n_kv_heads=2050, d=8), dict(n_heads=2 ** 31 - 2, n_kv_heads=2),
                                 dict(b=1 << 62, s=4)])
def test_sizes_refused(bad):
    for f in CALLS:
        assert f(**bad) == tp.TP_ERR_INVALID, bad


def test_other_refusals():
    for f in CALLS:
        assert f(dt=7) == tp.TP_ERR_UNSUPPORTED
        assert f(d=60, r=rot(60)) == tp.TP_ERR_ALIGN
        for r in (rot(3), rot(66), rot(-2), rot(64, 0, None), rot(amp=-1.0), rot(amp=math.inf), rot(amp=math.nan)):
            assert f(r=r) == tp.TP_ERR_INVALID
        for v in (-0.1, math.nan, math.inf, 2.0 ** 21):
            assert f(r=rot(64, 1, (ctypes.c_double * 32)(*[0.5] * 31, v))) == tp.TP_ERR_INVALID
        assert f(x=None) == tp.TP_ERR_INVALID
        assert f(ldx=504) == tp.TP_ERR_INVALID and f(ldx=1 << 40) == tp.TP_ERR_INVALID
        assert f(ldx=516) == tp.TP_ERR_ALIGN and f(ldx=514, dt=tp.TP_F32) == tp.TP_ERR_ALIGN
        assert f(x=FAKE + 8) == tp.TP_ERR_ALIGN
        assert f(starts=FAKE + 4) == tp.TP_ERR_ALIGN and f(pos=FAKE + 4) == tp.TP_ERR_ALIGN
        assert f(starts=FAKE, b=0) == tp.TP_ERR_INVALID and f(starts=FAKE, b=(1 << 22) + 1) == tp.TP_ERR_INVALID
        # sequences are given: b and s need not fill the rows (the next check fails)
        assert f(starts=FAKE, b=9, x=FAKE + 8) == tp.TP_ERR_ALIGN
        assert f(pos=FAKE, b=0, s=0, x=FAKE + 8) == tp.TP_ERR_ALIGN
    for f in (turn, fwd):
        assert f(y=None) == tp.TP_ERR_INVALID and f(ldy=504) == tp.TP_ERR_INVALID
        assert f(ldy=516) == tp.TP_ERR_ALIGN and f(y=FAKE * 2 + 8) == tp.TP_ERR_ALIGN
        assert f(y=FAKE, ldy=520) == tp.TP_ERR_INVALID  # in place with another pitch
        assert f(T=0, b=0) == tp.TP_OK
    assert turn(r=rot(0)) == tp.TP_ERR_INVALID
    for g in (L.tp_rotary_fwd, L.tp_rotary_bwd):
        assert g(tp.TP_BF16, cfg(), None, None, None, FAKE, 512, FAKE * 2, 512, None) == tp.TP_ERR_INVALID
        assert g(tp.TP_BF16, None, rot(), None, None, FAKE, 512, FAKE * 2, 512, None) == tp.TP_ERR_INVALID


def test_norm_refusals():
    for f in (fwd, bwd):
        for n in (norm(2), norm(-1), norm(0, 0.0), norm(0, -1.0), norm(1, math.nan), norm(1, math.inf)):
            assert f(n=n) == tp.TP_ERR_INVALID
        assert f(gq=FAKE + 2) == tp.TP_ERR_ALIGN and f(gk=FAKE + 2) == tp.TP_ERR_ALIGN
    assert L.tp_qk_norm_rotary_fwd(tp.TP_BF16, cfg(), None, rot(), None, None, None, None, FAKE, 512, FAKE * 2, 512,
                                   None) == tp.TP_ERR_INVALID
    assert bwd(dy=None) == tp.TP_ERR_INVALID and bwd(dx=None) == tp.TP_ERR_INVALID
    assert bwd(lddy=504) == tp.TP_ERR_INVALID and bwd(lddx=504) == tp.TP_ERR_INVALID
    assert bwd(lddy=516) == tp.TP_ERR_ALIGN and bwd(lddx=516) == tp.TP_ERR_ALIGN
    assert bwd(dy=FAKE * 2 + 8) == tp.TP_ERR_ALIGN and bwd(dx=FAKE * 3 + 8) == tp.TP_ERR_ALIGN
    assert bwd(dx=FAKE) == tp.TP_ERR_INVALID  # over the forward's input
    assert bwd(dx=FAKE * 2, lddx=520) == tp.TP_ERR_INVALID
    assert bwd(dgq=FAKE + 2) == tp.TP_ERR_ALIGN and bwd(dgk=FAKE + 2) == tp.TP_ERR_ALIGN
    assert bwd(dgq=FAKE * 5) == tp.TP_ERR_INVALID  # one buffer for both
    for g in ("dgq", "dgk"):
        for at in (8, 9):
            assert bwd(**{g: FAKE * at}) == tp.TP_ERR_INVALID
    need = L.tp_qk_norm_rotary_workspace_size(cfg())
    assert need > 0
    assert bwd(ws=None) == tp.TP_ERR_WORKSPACE and bwd(wsn=need - 1) == tp.TP_ERR_WORKSPACE
    assert bwd(ws=FAKE + 128) == tp.TP_ERR_ALIGN
    assert bwd(T=0, b=0, dgq=None, dgk=None) == tp.TP_OK
    for bad in (dict(T=0), dict(d=0), dict(d=60), dict(d=520), dict(T=-1)):
        assert L.tp_qk_norm_rotary_workspace_size(cfg(**bad)) == 0
    assert L.tp_qk_norm_rotary_workspace_size(None) == 0


def test_packed_sizes():
    """What the binding packs are the C structs."""
    r = tp.tp_rotary_frequencies(64, interleaved=True)
    want = tp.tp_rotary_config(64, 1, r["freq"].data_ptr(), r["amplitude"])
    assert tp._rotary_cfg(r) == bytes(want) and len(bytes(want)) == 24
    assert tp._rotary_cfg(None) is None
    assert tp._rotary_cfg(dict(n_rot=0, freq=None)) == bytes(tp.tp_rotary_config(0, 0, None, 0.0))
    assert tp._norm_cfg(dict(kind="layer", eps=1e-5)) == bytes(tp.tp_qk_norm_config(1, 1e-5))
    for bad in (dict(r, freq=r["freq"].float()), dict(r, freq=r["freq"][:-1]), dict(r, n_rot=62), dict(r, freq=None),
                dict(r, freq=r["freq"].tolist()), dict(r, freq=torch.ones(64).double()[::2])):
        with pytest.raises(ValueError):
            tp._rotary_cfg(bad)
    with pytest.raises(ValueError):
        tp._norm_cfg(dict(kind="batch", eps=1e-5))
    with pytest.raises(ValueError):
        tp._rotary_sizes(dict(n_heads=1 << 40, n_kv_heads=1, d=64, N=1), 4)


def test_structs_match_the_header(tmp_path):
    src = tmp_path / "layout.c"
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    classes = {c.__name__: c for c in (tp.tp_rotary_config, tp.tp_qk_norm_config, tp.tp_rotary_scaling)}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "tp.h"', 'int main(void) {']
    for name, c in classes.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in c._fields_]
    src.write_text("\n".join(lines + ["return 0; }"]))
    import subprocess
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "l")], check=True)
    out = dict(x.split() for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    for name, c in classes.items():
        assert int(out[name]) == ctypes.sizeof(c)
        for f, _ in c._fields_:
            assert int(out[f"{name}.{f}"]) == getattr(c, f).offset, f


def test_binding_refuses_cpu_tensors():
    c, r = dict(b=1, s=4, n_heads=2, n_kv_heads=1, d=8, N=1), tp.tp_rotary_frequencies(8)
    X = torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        tp.tp_rotary_fwd(X, c, r, torch.empty_like(X))
    with pytest.raises(ValueError, match="2D"):
        tp.tp_rotary_fwd(X[0], c, r, X[0])
    with pytest.raises(TypeError, match="dtype"):
        tp.tp_qk_norm_rotary_fwd(X.half(), c, dict(kind="rms", eps=1e-6), r, None, None, X)
