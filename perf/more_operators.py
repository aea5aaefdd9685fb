"""The operators whose cost is followed beside attention: the rotation of queries and keys by their positions, the
norm of every query and key head with that rotation in the same pass, and the gradients of both.

Each case names an operator and its sizes.  ``run`` computes it either through the package's entry points (``own``)
or in elementary torch operations in fp32 (angles in 64 bits), on the same inputs.
"""
import math

import torch

own = False

ROT_FWD, ROT_BWD, NORM_FWD, NORM_BWD = "rotary_fwd", "rotary_bwd", "qk_norm_rotary_fwd", "qk_norm_rotary_bwd"


def _case(name, op, lens, heads, kv, d, N, n_rot=None, inter=False, scaling="none", factor=1.0, layer=False, tail=0,
          dtype="bf16", far=0):
    c = {"op": op, "lens": ",".join(str(x) for x in lens), "heads": heads, "kv_heads": kv, "d": d, "N": N,
         "n_rot": d if n_rot is None else n_rot, "interleaved": bool(inter), "scaling": scaling,
         "factor": float(factor), "tail": tail, "dtype": dtype, "far": far}
    if op in (NORM_FWD, NORM_BWD):
        c["layer"] = bool(layer)
    if name:
        c["name"] = name
    return c


# Lengths of documents packed into one row of training data: one token up to a few thousand.
_PACKED = (1, 2048, 37, 700, 3001, 129, 128, 1500, 64, 2, 911, 3400)


def listed():
    return [
        # the next token of 16 sequences, each at a position of its own, far into contexts that were lengthened
        _case("rotary_fwd_16_tokens_heads32_kv8_d128", ROT_FWD, [1] * 16, 32, 8, 128, 1, scaling="ramp", factor=16.0,
              far=131072),
        # the training step of the h = 4096 model, two sequences of 2048, heads of 128
        _case("rotary_fwd_b2_s2048_heads32_d128", ROT_FWD, [2048] * 2, 32, 32, 128, 2),
        # packed documents of unequal lengths, half of every head rotated in adjacent pairs, unused rows at the end
        _case("rotary_fwd_packed_heads32_kv8_d128_of_it_64", ROT_FWD, _PACKED, 32, 8, 128, 4, n_rot=64, inter=True,
              tail=79),
        # one long document, positions interpolated
        _case("rotary_bwd_s65536_heads8_kv2_d128", ROT_BWD, [65536], 8, 2, 128, 2, scaling="linear", factor=8.0),
        # an fp32 run that another one is checked against
        _case("rotary_bwd_f32_b4_s1024_heads16_d64", ROT_BWD, [1024] * 4, 16, 16, 64, 4, inter=True, dtype="f32"),
        # the next token of 16 sequences
        _case("qk_norm_rotary_fwd_16_tokens_heads32_kv8_d128", NORM_FWD, [1] * 16, 32, 8, 128, 1, far=32768),
        # the training step of the h = 4096 model, forward
        _case("qk_norm_rotary_fwd_b2_s2048_heads32_d128", NORM_FWD, [2048] * 2, 32, 32, 128, 2),
        # packed documents, a head width that is no power of two
        _case("qk_norm_rotary_fwd_packed_heads16_kv4_d96", NORM_FWD, _PACKED, 16, 4, 96, 4, tail=79),
        # a short prompt of a small model, backward: launches and latency
        _case("qk_norm_rotary_bwd_s96_heads8_d64", NORM_BWD, [96], 8, 8, 64, 1, inter=True),
        # the training step of the h = 4096 model, backward; then with its 8 heads of 512 and centred norms
        _case("qk_norm_rotary_bwd_b2_s2048_heads32_d128", NORM_BWD, [2048] * 2, 32, 32, 128, 2),
        _case("qk_norm_rotary_bwd_s2048_heads8_d512_layer", NORM_BWD, [2048], 8, 8, 512, 8, layer=True),
        # one long document, backward
        _case("qk_norm_rotary_bwd_s65536_heads8_kv2_d128", NORM_BWD, [65536], 8, 2, 128, 2, scaling="ramp", factor=8.0),
    ]


_MOST = 65536 * 12 * 128  # values of QKV in the longest listed document


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice((ROT_FWD, ROT_BWD, NORM_FWD, NORM_BWD))
    kv = rng.choice((1, 2, 4, 8, 16, 32))
    heads = min(kv * rng.choice((1, 1, 2, 4)), 32) // kv * kv
    N = rng.choice([n for n in (1, 2, 4, 8) if kv % n == 0])
    d = rng.choice((64, 128, 128, 256, 512, 8 * rng.randint(1, 16)))
    inter = rng.random() < 0.5
    dtype = "bf16" if rng.random() < 0.8 else "f32"
    n_rot = rng.choice((d, d, d // 2 // 2 * 2, 2 * rng.randint(1, d // 2)))
    room = _MOST // (1 if dtype == "bf16" else 2) // ((heads + 2 * kv) * d)  # no more bytes than the longest listed
    scaling = rng.choice(("none", "none", "linear", "ramp"))
    factor = rng.choice((2.0, 8.0, 40.0)) if scaling != "none" else 1.0
    tail = far = 0
    if rng.random() < 0.25:
        lens, far = [1] * _log_int(rng, 1, 512), rng.choice((4096, 131072, 1000000))
    else:
        longest = min(_log_int(rng, 1, 65536), room)
        b = max(1, min(_log_int(rng, 1, 48), room // longest))
        lens = [longest] * b
        if rng.random() < 0.5:
            lens, tail = [longest] + [_log_int(rng, 1, longest) for _ in range(b - 1)], rng.randint(0, 200)
            rng.shuffle(lens)
    return _case(None, op, lens, heads, kv, d, N, n_rot, inter, scaling, factor, rng.random() < 0.3, tail, dtype, far)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _sizes(case):
    lens = [int(x) for x in case["lens"].split(",")]
    starts = [0]
    for x in lens:
        starts.append(starts[-1] + x)
    return lens, starts, starts[-1] + case["tail"]


def _frequencies(n_rot, scaling, factor, base=10000.0, trained=4096):
    """(radians a position of every pair, amplitude)"""
    f = [base ** (-2.0 * k / n_rot) for k in range(n_rot // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling == "ramp":
        # pairs that turn 32 times and more in the trained length keep their frequency, those that turn less than
        # once are interpolated, a ramp over the pairs' numbers lies between
        at = [n_rot * math.log(trained / (r * 2 * math.pi)) / (2 * math.log(base)) for r in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), n_rot - 1)
        t = [min(max((k - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for k in range(n_rot // 2)]
        return [x * (1 - u) + x / factor * u for x, u in zip(f, t)], 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    lens, starts, T = _sizes(case)
    H, kv, d, N = case["heads"], case["kv_heads"], case["d"], case["N"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, dt = "cuda", torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    draw_n = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    W = (H + 2 * kv) * d
    even = case["tail"] == 0 and len(set(lens)) == 1 and not case["far"]
    freq, amplitude = _frequencies(case["n_rot"], case["scaling"], case["factor"])
    freq = torch.tensor(freq, dtype=torch.float64)
    st = {"op": case["op"], "H": H, "kv": kv, "d": d, "N": N, "T": T, "used": starts[-1],
          "freq": freq.to(dev), "rot": {"n_rot": case["n_rot"], "interleaved": case["interleaved"], "freq": freq,
                                        "amplitude": amplitude},
          "starts": None if even or case["far"] else torch.tensor(starts, dtype=torch.int64, device=dev),
          "positions": None, "out": torch.zeros(T, W, dtype=dt, device=dev),
          "cfg": {"b": len(lens), "s": max(lens), "n_heads": H, "n_kv_heads": kv, "d": d, "N": N, "causal": True}}
    if case["far"]:
        st["positions"] = torch.randint(0, case["far"], (T,), generator=g, device=dev)
    if case["op"] != ROT_BWD:
        st["QKV"] = draw_n(T, W).to(dt)
    if case["op"] in (NORM_FWD, NORM_BWD):
        st["norm"] = {"kind": "layer" if case["layer"] else "rms", "eps": 1e-6}
        st["gq"], st["gk"] = 1 + 0.2 * draw_n(d), 1 + 0.2 * draw_n(d)
    if case["op"] in (ROT_BWD, NORM_BWD):
        st["dOut"] = draw_n(T, W).to(dt)
    if case["op"] == NORM_BWD:
        st["dgq"], st["dgk"] = torch.zeros(d, device=dev), torch.zeros(d, device=dev)
        st["ws"] = torch.empty(8192 * d + 4096, dtype=torch.uint8, device=dev)
    return st


# ----------------------------------------------------------------------------
# the plain form
# ----------------------------------------------------------------------------
def _heads(st, X):
    """The used rows as (rows, shards, query and key heads, d) in fp32, and the values' heads as they are."""
    y = X[: st["used"]].view(st["used"], st["N"], -1, st["d"])
    n = (st["H"] + st["kv"]) // st["N"]
    return y[:, :, :n].float(), y[:, :, n:]


def _turn(st, x, back=False):
    """x rotated by its rows' positions; `back`: by the transposed matrix."""
    t = torch.arange(st["used"], device=x.device)
    if st["positions"] is not None:
        pos = st["positions"]
    elif st["starts"] is not None:
        pos = t - st["starts"][torch.searchsorted(st["starts"], t, right=True) - 1]
    else:
        pos = t % st["cfg"]["s"]
    angle = pos.double()[:, None] * st["freq"]
    c = (angle.cos() * st["rot"]["amplitude"]).float()[:, None, None]
    s = (angle.sin() * (-1 if back else 1) * st["rot"]["amplitude"]).float()[:, None, None]
    n = st["rot"]["n_rot"]
    if st["rot"]["interleaved"]:
        a, b = x[..., 0:n:2], x[..., 1:n:2]
        y = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = x[..., : n // 2], x[..., n // 2:n]
        y = torch.cat([a * c - b * s, a * s + b * c], -1)
    return torch.cat([y, x[..., n:]], -1)


def _normed(st, x):
    """(x in units of its head's norm, 1 over that norm, the gains of every head)"""
    if st["norm"]["kind"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = (x.square().mean(-1, keepdim=True) + st["norm"]["eps"]).rsqrt()
    hq, hk = st["H"] // st["N"], st["kv"] // st["N"]
    return x * r, r, torch.cat([st["gq"].expand(hq, -1), st["gk"].expand(hk, -1)])


def _whole(st, x, v):
    st["out"][: st["used"]] = torch.cat([x.to(v.dtype), v], 2).view(st["used"], -1)


def _plain(st):
    op = st["op"]
    if op in (ROT_FWD, ROT_BWD):
        x, v = _heads(st, st["QKV"] if op == ROT_FWD else st["dOut"])
        _whole(st, _turn(st, x, op == ROT_BWD), v)
        return
    x, v = _heads(st, st["QKV"])
    n, r, gain = _normed(st, x)
    if op == NORM_FWD:
        _whole(st, _turn(st, n * gain), v)
        return
    dy, v = _heads(st, st["dOut"])
    dz = _turn(st, dy, True)
    hq = st["H"] // st["N"]
    dg = (dz * n).sum((0, 1))
    st["dgq"].copy_(dg[:hq].sum(0))
    st["dgk"].copy_(dg[hq:].sum(0))
    dn = dz * gain
    dx = dn - n * (dn * n).mean(-1, keepdim=True)
    if st["norm"]["kind"] == "layer":
        dx -= dn.mean(-1, keepdim=True)
    _whole(st, dx * r, v)


def run(state):
    st, op = state, state["op"]
    if own:
        import megatron_tensor_transformer_tp_gb300 as tp
        at = {"seq_starts": st["starts"], "positions": st["positions"]}
        if op == ROT_FWD:
            tp.tp_rotary_fwd(st["QKV"], st["cfg"], st["rot"], st["out"], **at)
        elif op == ROT_BWD:
            tp.tp_rotary_bwd(st["dOut"], st["cfg"], st["rot"], st["out"], **at)
        elif op == NORM_FWD:
            tp.tp_qk_norm_rotary_fwd(st["QKV"], st["cfg"], st["norm"], st["rot"], st["gq"], st["gk"], st["out"], **at)
        else:
            tp.tp_qk_norm_rotary_bwd(st["QKV"], st["cfg"], st["norm"], st["rot"], st["gq"], st["gk"], st["dOut"],
                                     st["out"], st["dgq"], st["dgk"], st["ws"], **at)
    else:
        _plain(st)
    if op == NORM_BWD:
        return {"dQKV": st["out"], "dgq": st["dgq"], "dgk": st["dgk"]}
    return {"dQKV": st["out"]} if op == ROT_BWD else {"Out": st["out"]}


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    lens, _, _ = _sizes(case)
    used, d, size = sum(lens), case["d"], 2 if case["dtype"] == "bf16" else 4
    qk, row = used * (case["heads"] + case["kv_heads"]) * d, used * (case["heads"] + 2 * case["kv_heads"]) * d
    at = 8 * used if case["far"] else 0
    turn = qk * case["n_rot"] // d * 3  # two products and a sum a value
    if case["op"] in (ROT_FWD, ROT_BWD):
        return {"bytes": 2 * row * size + at, "flops": turn}
    if case["op"] == NORM_FWD:
        return {"bytes": 2 * row * size + at + 8 * d, "flops": turn + 4 * qk}
    return {"bytes": (2 * row + qk) * size + at + 16 * d, "flops": turn + 12 * qk}


# ----------------------------------------------------------------------------
# the same in 64 bits: head by head, pairs as complex numbers
# ----------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    lens, starts, T = _sizes(case)
    H, kv, d, N, n = st["H"], st["kv"], st["d"], st["N"], case["n_rot"]
    hq, hk = H // N, kv // N
    used = starts[-1]
    if st["positions"] is not None:
        pos = st["positions"].double()
    else:
        pos = torch.cat([torch.arange(x, device="cuda") for x in lens]).double()
    unit = torch.polar(torch.full((used, n // 2), st["rot"]["amplitude"], dtype=torch.float64, device="cuda"),
                       torch.outer(pos, st["freq"]))
    if case["interleaved"]:
        first, second = torch.arange(0, n, 2, device="cuda"), torch.arange(1, n, 2, device="cuda")
    else:
        first, second = torch.arange(n // 2, device="cuda"), torch.arange(n // 2, n, device="cuda")

    def turned(x, w):
        z = torch.complex(x[:, first], x[:, second]) * w
        y = x.clone()
        y[:, first], y[:, second] = z.real, z.imag
        return y

    src = st["QKV"] if "QKV" in st else st["dOut"]
    out = torch.zeros(T, src.shape[1], dtype=torch.float64, device="cuda")
    dg = {"q": torch.zeros(d, dtype=torch.float64, device="cuda"), "k": torch.zeros(d, dtype=torch.float64, device="cuda")}
    for at in range(N * (hq + 2 * hk)):
        col = slice(at * d, (at + 1) * d)
        inside = at % (hq + 2 * hk)
        x = src[:used, col].double()
        if inside >= hq + hk:
            out[:used, col] = x if case["op"] != NORM_BWD else st["dOut"][:used, col].double()
            continue
        if case["op"] in (ROT_FWD, ROT_BWD):
            out[:used, col] = turned(x, unit if case["op"] == ROT_FWD else unit.conj())
            continue
        which = "q" if inside < hq else "k"
        gain = st["g" + which].double()
        centred = x - x.mean(1, keepdim=True) if case["layer"] else x
        size = torch.sqrt((centred ** 2).sum(1, keepdim=True) / d + st["norm"]["eps"])
        y = centred / size
        if case["op"] == NORM_FWD:
            out[:used, col] = turned(y * gain, unit)
            continue
        dz = turned(st["dOut"][:used, col].double(), unit.conj())
        dg[which] += (dz * y).sum(0)
        e = dz * gain
        along = y * (e * y).sum(1, keepdim=True) / d
        out[:used, col] = (e - along - (e.sum(1, keepdim=True) / d if case["layer"] else 0)) / size
    if case["op"] == NORM_FWD or case["op"] == ROT_FWD:
        return {"Out": out}
    return {"dQKV": out, "dgq": dg["q"], "dgk": dg["k"]} if case["op"] == NORM_BWD else {"dQKV": out}
