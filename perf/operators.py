"""The operators whose cost is followed: softmax attention that keeps no probabilities, its gradient, and both with
a learned relative position bias.

Each case names an operator and its sizes.  ``run`` computes it either through the package's entry points (``own``)
or in elementary torch operations in fp32, on the same inputs.
"""
import math

import torch

own = False

FWD, BWD, BIAS_FWD, BIAS_BWD = "attn_fwd", "attn_bwd", "relbias_fwd", "relbias_bwd"


def _case(name, op, lens, heads, kv, d, N, causal, scale=0.0, tail=0, buckets=32, distance=128, both=False):
    c = {"op": op, "lens": ",".join(str(x) for x in lens), "heads": heads, "kv_heads": kv, "d": d, "N": N,
         "causal": bool(causal), "scale": float(scale), "tail": tail}
    if op in (BIAS_FWD, BIAS_BWD):
        c.update(buckets=buckets, distance=distance, both=bool(both))
    if name:
        c["name"] = name
    return c


# Lengths of documents packed into one row of training data: one token up to a few thousand.
_PACKED = (1, 2048, 37, 700, 3001, 129, 128, 1500, 64, 2, 911, 3400)
_PACKED_SMALL = (300, 1, 65, 511, 128, 200)


def listed():
    return [
        # a short prompt of a small model: launch and latency
        _case("fwd_s96_heads8_d64", FWD, [96], 8, 8, 64, 1, True),
        _case("bwd_s96_heads8_d64", BWD, [96], 8, 8, 64, 1, True),
        # the training step of the h = 4096 model, two sequences of 2048, heads of 128
        _case("fwd_b2_s2048_heads32_d128", FWD, [2048] * 2, 32, 32, 128, 2, True),
        _case("bwd_b2_s2048_heads32_d128", BWD, [2048] * 2, 32, 32, 128, 2, True),
        # packed documents of unequal lengths with shared key/value heads, unused rows behind the last one
        _case("fwd_packed_heads32_kv8_d128", FWD, _PACKED, 32, 8, 128, 4, True, tail=79),
        _case("bwd_packed_heads16_kv4_d96", BWD, _PACKED, 16, 4, 96, 4, True, tail=79),
        # one long document
        _case("fwd_s16384_heads8_kv2_d128", FWD, [16384], 8, 2, 128, 2, True),
        _case("bwd_s16384_heads8_kv2_d128", BWD, [16384], 8, 2, 128, 2, True),
        # an encoder of width 1024: bias of both directions, scores not scaled
        _case("relbias_fwd_b4_s1024_heads16_d64", BIAS_FWD, [1024] * 4, 16, 16, 64, 4, False, 1.0, both=True),
        _case("relbias_bwd_b4_s1024_heads16_d64", BIAS_BWD, [1024] * 4, 16, 16, 64, 4, False, 1.0, both=True),
        # a decoder's packed short documents, and its long training sequences
        _case("relbias_fwd_packed_heads8_d64", BIAS_FWD, _PACKED_SMALL, 8, 8, 64, 2, True, 1.0),
        _case("relbias_bwd_b2_s4096_heads16_d64", BIAS_BWD, [4096] * 2, 16, 16, 64, 2, True, 1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice((FWD, BWD, BIAS_FWD, BIAS_BWD))
    kv = rng.choice((1, 2, 4, 8, 16))
    heads = kv * rng.choice((1, 1, 2, 4))
    heads = min(heads, 32) // kv * kv
    N = rng.choice([n for n in (1, 2, 4, 8) if kv % n == 0])
    d = rng.choice((64, 128, 8 * rng.randint(1, 16)))
    causal = rng.random() < 0.6
    # a token that sees itself alone has no gradient towards its score: the bias's gradient needs longer ones
    longest = _log_int(rng, 16 if op == BIAS_BWD else 1, 8192)
    room = 1.0e9 / (heads * longest * longest)  # no more work than the longest listed sequence
    while room < 1:
        longest = longest * 3 // 4
        room = 1.0e9 / (heads * longest * longest)
    b = max(1, min(_log_int(rng, 1, 48), int(room), 40000 // longest))
    if rng.random() < 0.5:
        lens, tail = [longest] * b, 0
    else:
        lens, tail = [longest] + [_log_int(rng, 1, longest) for _ in range(b - 1)], rng.randint(0, 200)
        rng.shuffle(lens)
    scale = rng.choice((0.0, 1.0))
    buckets = 2 * rng.randint(2, 32)
    distance = rng.choice((buckets + 1 + rng.randint(0, 64), 128, 256))
    return _case(None, op, lens, heads, kv, d, N, causal, scale, tail, buckets, distance, rng.random() < 0.5)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _sizes(case):
    lens = [int(x) for x in case["lens"].split(",")]
    starts = [0]
    for x in lens:
        starts.append(starts[-1] + x)
    return lens, starts, starts[-1] + case["tail"]


def _pack(q, k, v, N):
    """(T, heads, d) tensors as the shard-major (T, (heads + 2 kv) d) buffer."""
    T = q.shape[0]
    return torch.cat([t.reshape(T, N, -1) for t in (q, k, v)], 2).reshape(T, -1).contiguous()


def prepare(case, seed):
    lens, starts, T = _sizes(case)
    H, kv, d, N = case["heads"], case["kv_heads"], case["d"], case["N"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf, dev = torch.bfloat16, "cuda"
    draw_n = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    scale = case["scale"] or 1.0 / math.sqrt(d)
    # queries such that the scaled scores have a standard deviation of 1.5
    q = draw_n(T, H, d) * (1.5 / (scale * math.sqrt(d)))
    k, v, dC = draw_n(T, kv, d), draw_n(T, kv, d), draw_n(T, H * d)
    even = case["tail"] == 0 and len(set(lens)) == 1
    st = {"op": case["op"], "H": H, "kv": kv, "d": d, "N": N, "causal": case["causal"], "scale": scale,
          "b": len(lens), "s": max(lens), "T": T, "used": starts[-1], "even": even,
          "starts": torch.tensor(starts, dtype=torch.int64, device=dev),
          "QKV": _pack(q.to(bf), k.to(bf), v.to(bf), N),
          "C": torch.zeros(T, H * d, dtype=bf, device=dev), "lse": torch.zeros(H, T, device=dev)}
    st["cfg"] = {"b": st["b"], "s": st["s"], "n_heads": H, "n_kv_heads": kv, "d": d, "N": N,
                 "causal": case["causal"], "scale": case["scale"]}
    if case["op"] in (BIAS_FWD, BIAS_BWD):
        st["table"] = draw_n(case["buckets"], H) * 0.5
        st["bias"] = {"num_buckets": case["buckets"], "max_distance": case["distance"], "bidirectional": case["both"]}
    if case["op"] in (BWD, BIAS_BWD):
        # what the forward pass left behind
        C, lse = _plain_fwd(st)
        st["C"][: st["used"]] = C
        st["lse"][:, : st["used"]] = lse
        del C, lse
        st["dC"] = dC.to(bf)
        st["dQKV"] = torch.zeros_like(st["QKV"])
        W = st["QKV"].shape[1]
        # a caller's scratch: 4 bytes a head and row, and 4 bytes a bucket, head and 64 rows
        rows = T // 64 + 2 * st["b"] + 2
        st["ws"] = torch.empty((4 * H * (T + 64) + 4 * H * rows * case.get("buckets", 0) + W * 64 + 65536) // 256 * 256,
                               dtype=torch.uint8, device=dev)
        if "table" in st:
            st["dtable"] = torch.zeros_like(st["table"])
    return st


# ----------------------------------------------------------------------------
# the plain form
# ----------------------------------------------------------------------------
def _token_index(st):
    """Of every token its place in a (b, s) grid, and of every grid place its token and whether it has one."""
    starts, s = st["starts"], st["s"]
    t = torch.arange(st["used"], device=starts.device)
    seq = torch.searchsorted(starts, t, right=True) - 1
    place = seq * s + (t - starts[seq])
    pos = torch.arange(s, device=starts.device)
    token = starts[:-1, None] + pos[None, :]
    valid = token < starts[1:, None]
    return place, torch.where(valid, token, torch.zeros_like(token)), valid


def _heads(st, x, token, valid):
    """(T, heads, d) rows as (b, heads, s, d) in fp32, zeros where there is no token."""
    y = x.float()[token] * valid[:, :, None, None]
    return y.permute(0, 2, 1, 3)


def _split(st):
    T, N, H, kv, d = st["T"], st["N"], st["H"], st["kv"], st["d"]
    q, k, v = st["QKV"].view(T, N, -1).split([H // N * d, kv // N * d, kv // N * d], 2)
    return q.reshape(T, H, d), k.reshape(T, kv, d), v.reshape(T, kv, d)


def _buckets(st):
    """(s, s) bucket of key position j seen from query position i."""
    nb, far, both = st["bias"]["num_buckets"], st["bias"]["max_distance"], st["bias"]["bidirectional"]
    i = torch.arange(st["s"], device="cuda")
    rel = i[None, :] - i[:, None]
    side = torch.zeros_like(rel)
    if both:
        nb //= 2
        side = nb * (rel > 0).long()
        n = rel.abs()
    else:
        n = (-rel).clamp(min=0)
    exact_n = nb // 2
    # in 64 bits; distances whose bucket is a whole number by the formula stay on their side of the border
    t = torch.log(n.clamp(min=1).double() / exact_n) / math.log(far / exact_n) * (nb - exact_n)
    large = (exact_n + torch.floor(t + 1e-9).long()).clamp(max=nb - 1)
    return side + torch.where(n < exact_n, n, large)


def _scores(st, q, k, valid):
    """(b, kv, group, s, s) scaled scores with the bias, minus infinity where a key is not seen."""
    b, H, s, d = q.shape
    kv = st["kv"]
    S = torch.matmul(q.reshape(b, kv, H // kv * s, d), k.transpose(2, 3)).view(b, kv, H // kv, s, s)
    S *= st["scale"]
    if "bias" in st:
        S += st["table"].t()[:, _buckets(st)].view(1, kv, H // kv, s, s)
    i = torch.arange(s, device=q.device)
    seen = valid[:, None, :] & (i[None, None, :] <= i[None, :, None] if st["causal"] else True)
    return S.masked_fill_(~seen[:, None, None], float("-inf"))


def _plain_fwd(st):
    place, token, valid = _token_index(st)
    q, k, v = (_heads(st, x, token, valid) for x in _split(st))
    b, H, s, d = q.shape
    kv = st["kv"]
    S = _scores(st, q, k, valid)
    m = S.amax(-1, keepdim=True)
    E = S.sub_(m).exp_()
    z = E.sum(-1, keepdim=True)
    lse = (m + z.log()).view(b, H, s)
    C = torch.matmul(E.view(b, kv, H // kv * s, s), v).view(b, H, s, d) / z.view(b, H, s, 1)
    C = C.permute(0, 2, 1, 3).reshape(b * s, H * d)[place].to(torch.bfloat16)
    return C, lse.permute(1, 0, 2).reshape(H, b * s)[:, place]


def _plain_bwd(st):
    place, token, valid = _token_index(st)
    q, k, v = (_heads(st, x, token, valid) for x in _split(st))
    b, H, s, d = q.shape
    kv, N = st["kv"], st["N"]
    rows = lambda x: _heads(st, x.view(st["T"], H, d), token, valid)  # noqa: E731
    dC, C = rows(st["dC"]), rows(st["C"])
    lse = (st["lse"][:, token] * valid).permute(1, 0, 2).reshape(b, kv, H // kv, s, 1)
    P = _scores(st, q, k, valid).sub_(lse).exp_()
    P *= valid[:, None, None, :, None]
    D = (dC * C).sum(-1).view(b, kv, H // kv, s, 1)
    gq = lambda x: x.reshape(b, kv, H // kv * s, -1)  # noqa: E731
    dv = torch.matmul(gq(P).transpose(2, 3), gq(dC))
    dS = torch.matmul(gq(dC), v.transpose(2, 3)).view(b, kv, H // kv, s, s).sub_(D).mul_(P)
    del P
    dk = torch.matmul(gq(dS).transpose(2, 3), gq(q)) * st["scale"]
    dq = torch.matmul(gq(dS), k).view(b, H, s, d) * st["scale"]
    back = lambda x: x.permute(0, 2, 1, 3).reshape(b * s, N, -1)[place]  # noqa: E731
    out = {"dQKV": torch.cat([back(dq), back(dk), back(dv)], 2).reshape(st["used"], -1).to(torch.bfloat16)}
    if "bias" in st:
        # sums along the diagonals j - i: rows 2s - 1 wide read with a pitch of 2s put (i, j) in column j - i
        A = dS.sum(0).view(H, s, s)
        A = torch.nn.functional.pad(A, (0, s - 1)).view(H, -1)
        A = torch.nn.functional.pad(A, (0, s)).view(H, s, 2 * s).sum(1, dtype=torch.float64)
        rel = torch.arange(2 * s, device=A.device)
        bk = _buckets(st)
        of = torch.where(rel < s, bk[0, rel.clamp(max=s - 1)], bk[(2 * s - rel).clamp(0, s - 1), 0])
        hot = of[:, None] == torch.arange(st["bias"]["num_buckets"], device=A.device)
        out["dtable"] = torch.matmul(hot.double().t(), A.t()).float()
    return out


def run(state):
    st = state
    bias = "bias" in st
    if own:
        import megatron_tensor_transformer_tp_gb300 as tp
        starts = None if st["even"] else st["starts"]
        if st["op"] == FWD:
            tp.tp_attn_recompute_fwd(st["QKV"], st["cfg"], st["C"], st["lse"], seq_starts=starts)
        elif st["op"] == BIAS_FWD:
            tp.tp_attn_relbias_fwd(st["QKV"], st["cfg"], st["bias"], st["table"], st["C"], st["lse"],
                                   seq_starts=starts)
        elif st["op"] == BWD:
            tp.tp_attn_recompute_bwd(st["QKV"], st["cfg"], st["C"], st["lse"], st["dC"], st["dQKV"], st["ws"],
                                     seq_starts=starts)
        else:
            tp.tp_attn_relbias_bwd(st["QKV"], st["cfg"], st["bias"], st["table"], st["C"], st["lse"], st["dC"],
                                   st["dQKV"], st["dtable"], st["ws"], seq_starts=starts)
    elif st["op"] in (FWD, BIAS_FWD):
        C, lse = _plain_fwd(st)
        st["C"][: st["used"]] = C
        st["lse"][:, : st["used"]] = lse
    else:
        out = _plain_bwd(st)
        st["dQKV"][: st["used"]] = out["dQKV"]
        if bias:
            st["dtable"].copy_(out["dtable"])
    if st["op"] in (FWD, BIAS_FWD):
        return {"C": st["C"], "lse": st["lse"]}
    return {"dQKV": st["dQKV"], "dtable": st["dtable"]} if bias else {"dQKV": st["dQKV"]}


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    lens, _, _ = _sizes(case)
    H, kv, d = case["heads"], case["kv_heads"], case["d"]
    used = sum(lens)
    pairs = sum(x * (x + 1) // 2 if case["causal"] else x * x for x in lens)
    qkv, ctx, row = used * (H + 2 * kv) * d * 2, used * H * d * 2, used * H * 4
    table = 4 * case["buckets"] * H if "buckets" in case else 0
    if case["op"] in (FWD, BIAS_FWD):
        return {"bytes": qkv + ctx + row + table, "flops": 4 * d * pairs * H}
    return {"bytes": 2 * qkv + 2 * ctx + row + 2 * table, "flops": 10 * d * pairs * H}


# ----------------------------------------------------------------------------
# the same in 64 bits: head by head and sequence by sequence, from the definition
# ----------------------------------------------------------------------------
def _exact_bucket(rel, bias):
    """Bucket of one distance key - query, in whole numbers."""
    nb, far = bias["num_buckets"], bias["max_distance"]
    add = 0
    if bias["bidirectional"]:
        nb //= 2
        add, n = (nb if rel > 0 else 0), abs(rel)
    else:
        n = max(-rel, 0)
    e = nb // 2
    if n < e:
        return add + n
    if n >= far:
        return add + nb - 1
    steps = nb - e
    j = 0
    # step j begins at the first n with (n / e)^steps >= (far / e)^j
    while j + 1 < steps and far ** (j + 1) * e ** steps <= n ** steps * e ** (j + 1):
        j += 1
    return add + e + j


def exact(case, seed):
    st = prepare(case, seed)
    lens, starts, T = _sizes(case)
    H, kv, d, N = st["H"], st["kv"], st["d"], st["N"]
    X = st["QKV"].double().view(T, N, -1)
    hq, hk = H // N, kv // N

    def column(x, shard, at):
        return x[:, shard, at * d:(at + 1) * d]

    f64 = dict(dtype=torch.float64, device="cuda")
    fwd = case["op"] in (FWD, BIAS_FWD)
    C, lse = torch.zeros(T, H * d, **f64), torch.zeros(H, T, **f64)
    dX = torch.zeros(T, N, (hq + 2 * hk) * d, **f64)
    bias = st.get("bias")
    if bias:
        smax = max(lens)
        far = torch.tensor([_exact_bucket(r, bias) for r in range(-min(smax, bias["max_distance"]),
                                                                  min(smax, bias["max_distance"]) + 1)], device="cuda")
        half = far.numel() // 2
        dtab = torch.zeros(bias["num_buckets"], H, **f64)
    for h in range(H):
        g = h // (H // kv)
        q = column(X, h // hq, h % hq)
        k, v = column(X, g // hk, hq + g % hk), column(X, g // hk, hq + hk + g % hk)
        for a, n in zip(starts, lens):
            r = slice(a, a + n)
            S = (q[r] @ k[r].t()) * st["scale"]
            if bias:
                i = torch.arange(n, device="cuda")
                of = far[(i[None, :] - i[:, None]).clamp(-half, half) + half]
                S += st["table"].double()[:, h][of]
            if case["causal"]:
                S.masked_fill_(torch.ones(n, n, dtype=torch.bool, device="cuda").triu_(1), float("-inf"))
            if fwd:
                lse[h, r] = torch.logsumexp(S, 1)
                C[r, h * d:(h + 1) * d] = torch.exp(S - lse[h, r, None]) @ v[r]
                continue
            P = S.sub_(st["lse"][h, r, None].double()).exp_()
            dO, O = (st[x][r, h * d:(h + 1) * d].double() for x in ("dC", "C"))
            column(dX, g // hk, hq + hk + g % hk)[r] += P.t() @ dO
            dS = P.mul_((dO @ v[r].t()).sub_((dO * O).sum(1, keepdim=True)))
            column(dX, h // hq, h % hq)[r] += dS @ k[r] * st["scale"]
            column(dX, g // hk, hq + g % hk)[r] += dS.t() @ q[r] * st["scale"]
            if bias:
                # distance by distance through the running sums of each bucket's one-hot rows
                flat, idx = dS.reshape(-1), of.reshape(-1)
                for u in range(bias["num_buckets"]):
                    dtab[u, h] += torch.where(idx == u, flat, torch.zeros((), **f64)).sum()
    if fwd:
        return {"C": C, "lse": lse}
    out = {"dQKV": dX.reshape(T, -1)}
    if bias:
        out["dtable"] = dtab
    return out
