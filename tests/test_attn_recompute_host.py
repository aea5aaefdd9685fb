"""Host-side tests of attention without stored probabilities and its relative
position bias: the oracle's functions against independent forms, and the
entry points' refusals (before the device is touched)."""
import ctypes
import decimal
import math

import numpy as np
import pytest
import torch

import megatron_tensor_transformer_tp_gb300 as tp
import oracle.tp_oracle as O

FAKE = 0x100000  # never dereferenced: every refused call fails validation first


# ----------------------------------------------------------------------------
# oracle pins
# ----------------------------------------------------------------------------
def test_bucket_hand_made_table():
    # B = 8, E = 4, max 32: steps at 4 * 8^(j/4) = 4, 6.73, 11.31, 19.03
    want = {0: 0, 1: 1, 3: 3, 4: 4, 6: 4, 7: 5, 11: 5, 12: 6, 19: 6, 20: 7, 31: 7, 32: 7, 500: 7}
    for n, u in want.items():
        assert O.relative_bucket(-n, 8, 32, False) == u
        assert O.relative_bucket(-n, 16, 32, True) == u
        assert O.relative_bucket(n, 16, 32, True) == (u + 8 if n else 0)
    assert all(O.relative_bucket(n, 8, 32, False) == 0 for n in range(1, 50))  # ahead of the query


@pytest.mark.parametrize("nb,md,both", [(32, 128, True), (32, 128, False), (6, 5, False), (64, 1024, True),
                                         (256, 300, True), (2, 2, False), (32, 256, False), (24, 48, True)])
def test_bucket_against_60_digit_logarithms(nb, md, both):
    """The formula with its floor taken in 60 digits; a whole number of steps is told apart by whole powers."""
    decimal.getcontext().prec = 60
    B = nb // 2 if both else nb
    E = B // 2
    last = 0
    for n in range(0, md + 20):
        got = O.relative_bucket(-n, nb, md, both)
        assert got >= last
        last = got
        if n < E:
            want = n
        else:
            t = (decimal.Decimal(n) / E).ln() / (decimal.Decimal(md) / E).ln() * (B - E)
            near = int(t.to_integral_value())
            if abs(t - near) < decimal.Decimal("1e-40"):
                assert n ** (B - E) * E ** near == md ** near * E ** (B - E)  # exactly on the border
                t = decimal.Decimal(near)
            want = min(B - 1, E + int(t // 1))
        assert got == want, n
    assert last == B - 1


def test_grouped_columns():
    # two shards of 2 query heads and 1 key/value head, d = 8: [Q0 Q1 K0 V0 | Q2 Q3 K1 V1]
    assert [O.grouped_head_columns(8, 4, 2, 2, j) for j in range(4)] == [(0, 16, 24), (8, 16, 24), (32, 48, 56),
                                                                         (40, 48, 56)]
    for h, H, N in ((64, 4, 2), (96, 6, 3), (32, 2, 1)):
        for j in range(H):
            assert O.grouped_head_columns(h // H, H, H, N, j) == O.attention_head_columns(h, H, N, j)[:3]


def test_attention_lse_is_the_core():
    rng = np.random.default_rng(0)
    X = rng.standard_normal((24, 3 * 32))
    cfg = dict(n_heads=4, n_kv_heads=4, d=8, N=2, causal=True, scale=0.0)
    C, lse, A = O.attention_lse(X, [0, 12, 24], cfg)
    rC, P = O.attention_core(X, 12, 4, 2, True)
    assert np.allclose(C, rC, atol=1e-12) and (A >= np.abs(C) - 1e-12).all()
    dC = rng.standard_normal(C.shape)
    dX = O.attention_lse_grad(X, [0, 12, 24], cfg, C, lse, dC)[0]
    assert np.allclose(dX, O.attention_core_grad(X, P, dC, 12, 4, 2), atol=1e-12)


@pytest.mark.parametrize("causal", [True, False])
def test_attention_lse_against_torch(causal):
    """Shared key/value heads, unequal sequences and the bias: torch's attention with an additive mask and its
    autograd, in float64."""
    H, KV, d, N, starts, T = 4, 2, 8, 2, [1, 8, 8, 19], 21
    bias = dict(num_buckets=8, max_distance=7, bidirectional=True)
    g = torch.Generator().manual_seed(1)
    X = torch.randn(T, (H + 2 * KV) * d, generator=g, dtype=torch.float64, requires_grad=True)
    table = torch.randn(8, H, generator=g, dtype=torch.float64, requires_grad=True)
    dC = torch.randn(T, H * d, generator=g, dtype=torch.float64)
    cfg = dict(n_heads=H, n_kv_heads=KV, d=d, N=N, causal=causal, scale=0.3)
    parts = []
    for a, e in zip(starts[:-1], starts[1:]):
        for j in range(H if e > a else 0):
            q, k, v = (X[a:e, c:c + d] for c in O.grouped_head_columns(d, H, KV, N, j))
            m = table[torch.tensor(O.relative_buckets(e - a, **bias)), j]
            if causal:
                m = m.masked_fill(torch.ones(e - a, e - a).triu(1).bool(), float("-inf"))
            o = torch.nn.functional.scaled_dot_product_attention(q[None], k[None], v[None], attn_mask=m[None], scale=0.3)
            parts.append((a, e, j, o[0]))
    loss = sum((o * dC[a:e, j * d:(j + 1) * d]).sum() for a, e, j, o in parts)
    loss.backward()
    Xn, tn = X.detach().numpy(), table.detach().numpy()
    C, lse, _ = O.attention_lse(Xn, starts, cfg, bias, tn)
    for a, e, j, o in parts:
        assert np.allclose(C[a:e, j * d:(j + 1) * d], o.detach().numpy(), atol=1e-12)
    dX, dT, EX, ET = O.attention_lse_grad(Xn, starts, cfg, C, lse, dC.numpy(), bias, tn, 0.0, 0.0)
    assert np.allclose(dX, X.grad.numpy(), atol=1e-12) and np.allclose(dT, table.grad.numpy(), atol=1e-12)
    assert not EX.any() and not ET.any()


# ----------------------------------------------------------------------------
# refusals
# ----------------------------------------------------------------------------
L = tp.lib()
CFG = dict(T=256, b=2, s=128, n_heads=4, n_kv_heads=2, d=64, N=2, causal=1, scale=0.0)


def cfg(**k):
    c = tp.tp_attn_config(*[{**CFG, **k}[f] for f, _ in tp.tp_attn_config._fields_])
    return ctypes.byref(c)


def bias(nb=32, md=128, both=1):
    return ctypes.byref(tp.tp_relbias_config(nb, md, both))


def fwd(dt=tp.TP_BF16, c=None, starts=None, qkv=FAKE, ld=512, C=FAKE, ldc=256, lse=FAKE, **k):
    return L.tp_attn_recompute_fwd(dt, cfg(**k) if c is None else c, starts, qkv, ld, C, ldc, lse, None)


def bwd(dt=tp.TP_BF16, starts=None, qkv=FAKE, ld=512, C=FAKE, ldc=256, lse=FAKE, dC=FAKE, lddc=256, dq=FAKE,
        lddq=512, ws=FAKE, wsn=1 << 30, **k):
    return L.tp_attn_recompute_bwd(dt, cfg(**k), starts, qkv, ld, C, ldc, lse, dC, lddc, dq, lddq, ws, wsn, None)


def bfwd(b=None, table=FAKE, **k):
    return L.tp_attn_relbias_fwd(tp.TP_BF16, cfg(**k), b, table, None, FAKE, 512, FAKE, 256, FAKE, None)


SIZES = [dict(T=-1), dict(T=1 << 31), dict(T=(1 << 31) - 511, b=1, s=(1 << 31) - 511), dict(b=0),
         dict(b=-1), dict(s=127), dict(s=0), dict(s=-128), dict(b=3),
         dict(n_heads=0), dict(n_kv_heads=0), dict(n_kv_heads=3), dict(N=0), dict(N=9), dict(N=4), dict(d=0),
         dict(d=136), dict(d=-8), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
         dict(b=1 << 40, s=1)]


@pytest.mark.parametrize("bad", SIZES, ids=str)
def test_sizes_refused(bad):
    assert fwd(**bad) == tp.TP_ERR_INVALID
    assert bwd(**bad) == tp.TP_ERR_INVALID
    if not {"b", "s"} & set(bad):
        assert fwd(starts=FAKE, **bad) == tp.TP_ERR_INVALID
        assert L.tp_attn_recompute_workspace_size(cfg(**bad), None) == 0


def test_other_refusals_forward():
    assert L.tp_attn_recompute_fwd(tp.TP_BF16, None, None, FAKE, 512, FAKE, 256, FAKE, None) == tp.TP_ERR_INVALID
    assert fwd(dt=tp.TP_F32) == tp.TP_ERR_UNSUPPORTED
    assert fwd(dt=7) == tp.TP_ERR_UNSUPPORTED
    assert fwd(d=60) == tp.TP_ERR_ALIGN
    for k in ("qkv", "C", "lse"):
        assert fwd(**{k: None}) == tp.TP_ERR_INVALID
    assert fwd(ld=504) == tp.TP_ERR_INVALID and fwd(ldc=248) == tp.TP_ERR_INVALID
    assert fwd(ld=1 << 40) == tp.TP_ERR_INVALID
    assert fwd(ld=516) == tp.TP_ERR_ALIGN and fwd(ldc=260) == tp.TP_ERR_ALIGN
    assert fwd(qkv=FAKE + 8) == tp.TP_ERR_ALIGN and fwd(C=FAKE + 8) == tp.TP_ERR_ALIGN
    assert fwd(lse=FAKE + 2) == tp.TP_ERR_ALIGN and fwd(starts=FAKE + 4) == tp.TP_ERR_ALIGN
    assert fwd(C=FAKE) == tp.TP_ERR_INVALID  # in place
    assert fwd(starts=FAKE, b=(1 << 22) + 1) == tp.TP_ERR_INVALID
    assert fwd(T=0, b=0) == tp.TP_OK


def test_other_refusals_backward():
    for k in ("qkv", "C", "lse", "dC", "dq"):
        assert bwd(**{k: None}) == tp.TP_ERR_INVALID
    assert bwd(lddc=248) == tp.TP_ERR_INVALID and bwd(lddq=504) == tp.TP_ERR_INVALID
    assert bwd(lddc=260) == tp.TP_ERR_ALIGN and bwd(lddq=516) == tp.TP_ERR_ALIGN
    assert bwd(dC=FAKE + 8) == tp.TP_ERR_ALIGN and bwd(dq=FAKE + 8) == tp.TP_ERR_ALIGN
    need = L.tp_attn_recompute_workspace_size(cfg(), None)
    assert need >= 4 * 4 * 256
    assert bwd(ws=None) == tp.TP_ERR_WORKSPACE and bwd(wsn=need - 1) == tp.TP_ERR_WORKSPACE
    assert bwd(ws=FAKE + 128) == tp.TP_ERR_ALIGN
    for i in range(3):  # in place
        assert bwd(qkv=FAKE, C=FAKE + 256, dC=FAKE + 512, dq=FAKE + 256 * i) == tp.TP_ERR_INVALID
    assert bwd(dt=tp.TP_F32) == tp.TP_ERR_UNSUPPORTED
    assert bwd(T=0, b=0) == tp.TP_OK


def test_packed_sizes():
    """What the binding packs are the C structs; numbers that do not fit their fields are refused, not cut."""
    c = dict(b=2, s=128, n_heads=4, n_kv_heads=2, d=64, N=2, causal=True, scale=0.25)
    assert tp._attn_cfg(c, 256) == bytes(tp.tp_attn_config(256, 2, 128, 4, 2, 64, 2, 1, 0.25))
    assert tp._attn_cfg(dict(c, s=None, scale=None, causal=False), 7) == \
        bytes(tp.tp_attn_config(7, 2, 0, 4, 2, 64, 2, 0, 0.0))
    assert tp._bias_cfg(dict(num_buckets=32, max_distance=128, bidirectional=True)) == \
        bytes(tp.tp_relbias_config(32, 128, 1))
    for bad in (dict(n_heads=(1 << 32) + 4), dict(b=1 << 63), dict(d=64.5)):
        with pytest.raises(ValueError):
            tp._attn_cfg(dict(c, **bad), 256)
    # (beyond fp32 is infinite, which the library refuses)
    assert L.tp_attn_recompute_workspace_size(tp._attn_cfg(dict(c, scale=1e300), 256), None) == 0
    with pytest.raises(ValueError):
        tp._bias_cfg(dict(num_buckets=(1 << 32) + 32, max_distance=128, bidirectional=0))


@pytest.mark.parametrize("nb,md,both", [(1, 128, 0), (0, 128, 0), (257, 1000, 0), (33, 128, 1), (2, 128, 1), (32, 16, 0),
                                         (32, 8, 1), (32, 1025, 0), (-4, 128, 0), (32, -1, 1)])
def test_bias_refused(nb, md, both):
    assert bfwd(bias(nb, md, both)) == tp.TP_ERR_INVALID
    assert L.tp_attn_recompute_workspace_size(cfg(), bias(nb, md, both)) == 0


def test_bias_arguments():
    assert bfwd(None) == tp.TP_ERR_INVALID
    assert bfwd(bias(), table=None) == tp.TP_ERR_INVALID
    assert bfwd(bias(), table=FAKE + 2) == tp.TP_ERR_ALIGN
    need = L.tp_attn_recompute_workspace_size(cfg(), bias())
    assert need > L.tp_attn_recompute_workspace_size(cfg(), None)

    def b(dtable=FAKE, wsn=need, dq=FAKE):
        return L.tp_attn_relbias_bwd(tp.TP_BF16, cfg(), bias(), FAKE, None, FAKE, 512, FAKE, 256, FAKE, FAKE, 256, dq,
                                     512, dtable, 0, FAKE, wsn, None)
    assert b(dq=FAKE + 256) == tp.TP_ERR_INVALID  # dtable in place
    assert b(wsn=need - 1) == tp.TP_ERR_WORKSPACE
    assert b(dtable=FAKE + 2) == tp.TP_ERR_ALIGN
