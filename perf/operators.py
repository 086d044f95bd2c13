"""The operators that serve a Gated DeltaNet layer, and the cases they are measured on.

Five operators, each named by a case's "op":

* ``recurrent``  -- the gated delta rule token by token over a pool of states (``gdn_recurrent_fwd``);
* ``prep``       -- the short causal convolution with its state, SiLU, the heads' L2 norm and the two gates
  (``gdn_prep_fwd``): what turns a layer's projections into the delta rule's q, k, v, g and beta;
* ``add_norm``   -- root-mean-square norm with the residual's addition, output in bf16 or in 8 bits with scales
  (``add_rms_norm_fwd``);
* ``gated_norm`` -- the norm of the delta rule's output, gated by SiLU(z) (``gated_rms_norm_fwd``);
* ``copy``       -- slots of the state pools copied or cleared, every layer's pools at once (``gdn_state_copy``).

``run`` computes a case with the framework's operators where ``own`` is true, else with plain torch operations in
fp32.  ``exact`` computes it in fp64, written apart from both.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TAPS = 4       # width of the short convolution
FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": FP8}


# ----------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one user's decode step: one token, 16 heads; the call's latency
        dict(name="recurrent_one", op="recurrent", seqs=1, tokens=1, ragged=False, hk=16, hv=16, d=128, state="f32",
             io="bf16", gated=True, spare=0),
        # a serving batch: one token for each of 64 sequences, two value heads for each key head, states scattered
        # over the pool
        dict(name="recurrent_serve", op="recurrent", seqs=64, tokens=1, ragged=False, hk=16, hv=32, d=128, state="f32",
             io="bf16", gated=True, spare=32),
        # 33 sequences that bring 1 to 8 tokens each (drafted tokens to verify, short follow-ups), states kept in bf16
        dict(name="recurrent_ragged_bf16", op="recurrent", seqs=33, tokens=8, ragged=True, hk=16, hv=16, d=128,
             state="bf16", io="bf16", gated=True, spare=7),
        # the largest batch: 256 sequences of a layer with 64 heads, more state than the caches hold
        dict(name="recurrent_large", op="recurrent", seqs=256, tokens=1, ragged=False, hk=64, hv=64, d=128, state="f32",
             io="bf16", gated=True, spare=64),
        # the serving batch's step before the delta rule: one token each, the convolution's state read and shifted
        dict(name="prep_decode", op="prep", seqs=64, tokens=1, ragged=False, hk=16, hv=32, d=128, io="bf16", bias=False,
             expand=False, spare=32),
        # a packed prefill of nine prompts of uneven length, 16 heads
        dict(name="prep_prefill", op="prep", seqs=9, tokens=6144, ragged=True, hk=16, hv=16, d=128, io="bf16", bias=True,
             expand=False, spare=3),
        # the layer's input norm in decode: 64 rows, output in 8 bits for an 8-bit projection
        dict(name="add_norm_decode_fp8", op="add_norm", rows=64, dim=2048, io="bf16", out="fp8", residual=True),
        # the same in a prefill of four 8192-token sequences, bf16 output
        dict(name="add_norm_prefill", op="add_norm", rows=32768, dim=4096, io="bf16", out="bf16", residual=True),
        # the layer's output norm in decode: 64 tokens of 32 heads, bf16 output
        dict(name="gated_norm_decode", op="gated_norm", rows=64, heads=32, d=128, io="bf16", out="bf16"),
        # the same in a prefill of four 8192-token sequences with 16 heads, output in 8 bits, a scale for each head
        dict(name="gated_norm_prefill_fp8", op="gated_norm", rows=32768, heads=16, d=128, io="bf16", out="fp8"),
        # one prompt's state copied to four samples, in two layers
        dict(name="copy_fork", op="copy", moves=4, fan=4, clear=0, layers=2, slots=16, hk=16, hv=16, d=128, state="f32"),
        # compaction of a server's pools: 61 live states moved down and 19 freed slots cleared, in four layers
        dict(name="copy_compact", op="copy", moves=61, fan=1, clear=19, layers=4, slots=160, hk=16, hv=32, d=128,
             state="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# (key heads, value heads) of a layer, by head dimension
HEADS = {128: ((8, 16), (4, 4), (16, 16), (16, 32), (8, 32), (16, 48), (16, 64), (32, 32), (48, 48), (64, 64), (1, 3), (5, 5)),
         64: ((8, 16), (4, 4), (16, 32), (4, 32), (16, 64), (32, 32), (64, 64), (1, 3), (5, 5))}


def _heads(rng, d, cap):
    """(hk, hv) with at most ``cap`` value heads."""
    return rng.choice([h for h in HEADS[d] if h[1] <= cap])


def draw(rng):
    op = rng.choice(("recurrent", "recurrent", "prep", "add_norm", "gated_norm", "copy"))
    if op == "recurrent":
        d = rng.choice((128, 128, 64))
        seqs = _log_int(rng, 1, 256)
        ragged = rng.random() < 0.4
        tokens = rng.choice((2, 3, 5, 8)) if ragged else rng.choice((1, 1, 1, 4))
        hk, hv = _heads(rng, d, 64 if tokens == 1 else max(4, 64 * 24 // max(24, seqs)))
        return dict(op=op, seqs=seqs, tokens=tokens, ragged=ragged, hk=hk, hv=hv, d=d, state=rng.choice(("f32", "bf16")),
                    io=rng.choice(("bf16", "bf16", "f32")), gated=rng.random() < 0.8, spare=rng.randrange(0, 40))
    if op == "prep":
        d = rng.choice((128, 128, 64))
        if rng.random() < 0.5:  # decode: a token or a few for each sequence
            seqs, tokens, ragged = _log_int(rng, 1, 256), rng.choice((1, 1, 2, 4)), rng.random() < 0.3
        else:
            seqs, ragged = rng.randrange(1, 10), rng.random() < 0.7
            tokens = max(2, _log_int(rng, 16, 32768) // seqs)
        hk, hv = _heads(rng, d, 32 if seqs * tokens < 12000 else 16)
        return dict(op=op, seqs=seqs, tokens=tokens, ragged=ragged, hk=hk, hv=hv, d=d, io=rng.choice(("bf16", "bf16", "f32")),
                    bias=rng.random() < 0.5, expand=rng.random() < 0.4, spare=rng.randrange(0, 20))
    if op == "add_norm":
        # whole groups of 128, a power of two, or a width that no vector divides
        dim = rng.choice((128 * rng.randrange(1, 65, 2), 1 << rng.randrange(7, 14), rng.randrange(65, 8192, 2)))
        rows = _log_int(rng, 1, max(1, min(32768, 32768 * 4096 // dim)))
        return dict(op=op, rows=rows, dim=dim, io=rng.choice(("bf16", "bf16", "f32")), out=rng.choice(("bf16", "fp8")),
                    residual=rng.random() < 0.7)
    if op == "gated_norm":
        heads = rng.choice((4, 8, 16, 32, 64, 3, 5))
        rows = _log_int(rng, 1, 32768 * 16 // max(16, heads))
        return dict(op=op, rows=rows, heads=heads, d=rng.choice((128, 128, 64)), io=rng.choice(("bf16", "bf16", "f32")),
                    out=rng.choice(("bf16", "fp8")))
    d = rng.choice((128, 128, 64))
    hk, hv = _heads(rng, d, 32)
    moves = _log_int(rng, 1, 60)
    clear = rng.randrange(0, 16)
    fan = rng.choice((1, 1, 2, 4))
    return dict(op=op, moves=moves, fan=fan, clear=clear, layers=rng.randrange(1, 5), slots=2 * moves + clear + rng.randrange(1, 20),
                hk=hk, hv=hv, d=d, state=rng.choice(("f32", "bf16")))


def _lengths(case, seed):
    """Tokens of each sequence: ``tokens`` each, or 1 to ``tokens`` spread evenly and rotated by the seed."""
    n, t = case["seqs"], case["tokens"]
    if not case["ragged"]:
        return [t] * n
    every = [1 + (i * (t - 1)) // max(1, n - 1) for i in range(n)]
    return [every[(i * 7 + seed) % n] for i in range(n)] if n % 7 else every[seed % n:] + every[:seed % n]


def _tokens(case):
    return sum(_lengths(case, 0))  # the same for every seed: the lengths only change places


# ---------------------------------------------------------------------------------------------- inputs

def _unit(x):
    return x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)

    def slots_of(n, total):
        return torch.randperm(total, generator=gen, device=DEV)[:n].to(torch.int32)

    s = dict(case=case)
    op = case["op"]
    if op in ("recurrent", "prep"):
        hk, hv, d, io = case["hk"], case["hv"], case["d"], TYPES[case["io"]]
        lengths = _lengths(case, seed)
        n = len(lengths)
        if case["ragged"]:
            shape = (1, sum(lengths))
            cu = [0]
            for x in lengths:
                cu.append(cu[-1] + x)
            s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        else:
            shape = (n, case["tokens"])
            s["cu_seqlens"] = None
        s["longest"] = max(lengths)
        s["slots"] = slots_of(n, n + case["spare"])
    if op == "recurrent":
        s["q"] = _unit(randn(*shape, hk, d)).to(io)
        s["k"] = _unit(randn(*shape, hk, d)).to(io)
        s["v"] = randn(*shape, hv, d).to(io)
        s["beta"] = torch.sigmoid(randn(*shape, hv))
        s["g"] = torch.nn.functional.logsigmoid(randn(*shape, hv) + 2.5) if case["gated"] else None
        s["state"] = (randn(n + case["spare"], hv, d, d) * d ** -0.5).to(TYPES[case["state"]])
    elif op == "prep":
        dim = (2 * hk + hv) * d
        s["x"] = randn(*shape, dim).to(io)
        s["weight"] = (randn(dim, TAPS) * TAPS ** -0.5).to(io)
        s["bias"] = (0.1 * randn(dim)).to(io) if case["bias"] else None
        s["a"], s["b"] = randn(*shape, hv).to(io), randn(*shape, hv).to(io)
        s["A_log"] = torch.log(1.0 + 15.0 * torch.rand(hv, generator=gen, device=DEV))
        s["dt_bias"] = randn(hv) - 4.0
        s["conv_state"] = randn(n + case["spare"], TAPS - 1, dim).to(io)
    elif op == "add_norm":
        io = TYPES[case["io"]]
        s["x"] = randn(case["rows"], case["dim"]).to(io)
        s["residual"] = (3.0 * randn(case["rows"], case["dim"])).to(io) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * randn(case["dim"])).to(io)
    elif op == "gated_norm":
        io = TYPES[case["io"]]
        s["x"] = (0.3 * randn(case["rows"], case["heads"], case["d"])).to(io)
        s["z"] = randn(case["rows"], case["heads"], case["d"]).to(io)
        s["weight"] = (1.0 + 0.2 * randn(case["d"])).to(io)
    else:
        hv, d, p = case["hv"], case["d"], case["slots"]
        dim = (2 * case["hk"] + hv) * d
        s["pools"] = []
        for _ in range(case["layers"]):
            s["pools"].append(randn(p, hv, d, d).to(TYPES[case["state"]]))
            s["pools"].append(randn(p, TAPS - 1, dim).to(torch.bfloat16))
        order = torch.randperm(p, generator=gen, device=DEV).to(torch.int32)
        m, c = case["moves"], case["clear"]
        src = order[:-(-m // case["fan"])].repeat_interleave(case["fan"])[:m]
        s["src_slots"] = torch.cat([src, torch.full((c,), -1, dtype=torch.int32, device=DEV)])
        s["dst_slots"] = order[m:2 * m + c].contiguous()
    return s


# ----------------------------------------------------------------------------------------------- a pass

def run(s):
    op = s["case"]["op"]
    return (_run_own if own else _run_plain)(op, s)


def _run_own(op, s):
    import gdn_chunkwise_ut_gb300 as gdn
    case = s["case"]
    if op == "recurrent":
        o = gdn.gdn_recurrent_fwd(s["q"], s["k"], s["v"], s["beta"], s["state"], g=s["g"], slots=s["slots"],
                                  cu_seqlens=s["cu_seqlens"])
        return {"o": o, "state": s["state"]}
    if op == "prep":
        q, k, v, g, beta = gdn.gdn_prep_fwd(s["x"], s["weight"], s["a"], s["b"], s["A_log"], s["dt_bias"],
                                            s["conv_state"], Hk=case["hk"], Hv=case["hv"], dk=case["d"], dv=case["d"],
                                            bias=s["bias"], slots=s["slots"], cu_seqlens=s["cu_seqlens"],
                                            expand=case["expand"])
        return {"q": q, "k": k, "v": v, "g": g, "beta": beta, "conv_state": s["conv_state"]}
    if op == "add_norm":
        y, scales, residual = gdn.add_rms_norm_fwd(s["x"], s["weight"], s["residual"], out_dtype=TYPES[case["out"]])
        return {"y": y, "scales": scales, "residual": residual}
    if op == "gated_norm":
        y, scales = gdn.gated_rms_norm_fwd(s["x"], s["z"], s["weight"], out_dtype=TYPES[case["out"]])
        return {"y": y, "scales": scales}
    gdn.gdn_state_copy(s["pools"], s["dst_slots"], s["pools"], s["src_slots"])
    return s["pools"]


def _run_plain(op, s):
    return {"recurrent": _plain_recurrent, "prep": _plain_prep, "add_norm": _plain_add_norm,
            "gated_norm": _plain_gated_norm, "copy": _plain_copy}[op](s)


def _plain_recurrent(s):
    case, pool, slots = s["case"], s["state"], s["slots"].long()
    hk, hv, d = case["hk"], case["hv"], case["d"]
    scale = d ** -0.5
    # tokens as [token, head, d], keys and queries for each value head
    q = s["q"].float().reshape(-1, hk, d).repeat_interleave(hv // hk, 1)
    k = s["k"].float().reshape(-1, hk, d).repeat_interleave(hv // hk, 1)
    v = s["v"].float().reshape(-1, hv, d)
    beta = s["beta"].reshape(-1, hv)
    alpha = torch.exp(s["g"].reshape(-1, hv)) if s["g"] is not None else torch.ones_like(beta)
    cu = s["cu_seqlens"]
    if cu is None:
        first = torch.arange(case["seqs"], device=DEV) * case["tokens"]
        count = torch.full_like(first, case["tokens"])
    else:
        first, count = cu[:-1].long(), (cu[1:] - cu[:-1]).long()
    S = pool[slots].float()
    o = torch.empty_like(v)
    for t in range(s["longest"]):
        at = first + torch.clamp(torch.minimum(torch.full_like(count, t), count - 1), min=0)
        live = (t < count).view(-1, 1, 1, 1)
        kt, qt = k[at], q[at]
        Sa = S * alpha[at][..., None, None]
        delta = beta[at][..., None] * (v[at] - (Sa * kt[..., None]).sum(-2))
        S = torch.where(live, Sa + kt[..., None] * delta[..., None, :], S)
        # a sequence that has ended writes its last token's output again: its state has not changed since
        o[at] = scale * (S * qt[..., None]).sum(-2)
    pool.index_copy_(0, slots, S.to(pool.dtype))
    return {"o": o.reshape(s["v"].shape).to(s["v"].dtype), "state": pool}


def _plain_prep(s):
    case, x, pool = s["case"], s["x"], s["conv_state"]
    hk, hv, d = case["hk"], case["hv"], case["d"]
    dim, keep = x.shape[-1], TAPS - 1
    flat = x.reshape(-1, dim).float()
    total, n = flat.shape[0], s["slots"].shape[0]
    cu = s["cu_seqlens"]
    cu = torch.arange(n + 1, device=DEV) * case["tokens"] if cu is None else cu.long()
    # every sequence behind the inputs that its state holds
    seq = torch.searchsorted(cu, torch.arange(total, device=DEV), right=True) - 1
    row = torch.arange(total, device=DEV) + (seq + 1) * keep
    taps = torch.arange(keep, device=DEV)
    before = (cu[:-1] + torch.arange(n, device=DEV) * keep)[:, None] + taps
    after = (cu[1:] + torch.arange(n, device=DEV) * keep)[:, None] + taps
    slots = s["slots"].long()
    line = torch.empty((total + n * keep, dim), device=DEV)
    line[before.reshape(-1)] = pool[slots].float().reshape(-1, dim)
    line[row] = flat
    w = s["weight"].float()
    y = line[row] * w[:, 3] + line[row - 1] * w[:, 2] + line[row - 2] * w[:, 1] + line[row - 3] * w[:, 0]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = y / (1.0 + torch.exp(-y))
    pool.index_copy_(0, slots, line[after.reshape(-1)].reshape(n, keep, dim).to(pool.dtype))
    shape = x.shape[:2]
    q, k, v = (z.reshape(*shape, -1, d) for z in y.split([hk * d, hk * d, hv * d], 1))
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + EPS)
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + EPS)
    if case["expand"]:
        q, k = q.repeat_interleave(hv // hk, 2), k.repeat_interleave(hv // hk, 2)
    u = s["a"].float() + s["dt_bias"]
    g = -torch.exp(s["A_log"]) * torch.where(u > 0, u + torch.log1p(torch.exp(-u.abs())), torch.log1p(torch.exp(-u.abs())))
    beta = 1.0 / (1.0 + torch.exp(-s["b"].float()))
    return {"q": q.to(x.dtype), "k": k.to(x.dtype), "v": v.to(x.dtype), "g": g, "beta": beta, "conv_state": pool}


def _rounded(y, out, group):
    """(y in the output's type, scales or None): in 8 bits, each ``group`` of a row has the scale that takes its largest
    magnitude to the type's largest value."""
    if out != FP8:
        return y.to(out), None
    rows, dim = y.shape[:-1], y.shape[-1]
    groups = -(-dim // group)
    padded = torch.nn.functional.pad(y, (0, groups * group - dim)).reshape(*rows, groups, group)
    top = padded.abs().amax(-1)
    scales = torch.where(top > 0, top / FP8_MAX, torch.ones_like(top))
    small = (padded / scales[..., None]).clamp(-FP8_MAX, FP8_MAX)
    return small.reshape(*rows, groups * group)[..., :dim].to(FP8), scales


def _plain_add_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    y, scales = _rounded(y, TYPES[s["case"]["out"]], 128)
    return {"y": y, "scales": scales, "residual": h.to(s["x"].dtype) if s["residual"] is not None else None}


def _plain_gated_norm(s):
    x, z = s["x"].float(), s["z"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"].float() * (z / (1.0 + torch.exp(-z)))
    y, scales = _rounded(y, TYPES[s["case"]["out"]], s["case"]["d"])
    return {"y": y, "scales": None if scales is None else scales.squeeze(-1)}


def _plain_copy(s):
    src, dst = s["src_slots"].long(), s["dst_slots"].long()
    return [_plain_copy_one(pool, src, dst) for pool in s["pools"]]


def _plain_copy_one(pool, src, dst):
    held = (src >= 0).view(-1, *[1] * (pool.dim() - 1))
    return pool.index_copy_(0, dst, torch.where(held, pool[src.clamp(min=0)], torch.zeros((), dtype=pool.dtype, device=DEV)))


# ------------------------------------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "recurrent":
        e, t = (4 if case["io"] == "f32" else 2), _tokens(case)
        hk, hv, d = case["hk"], case["hv"], case["d"]
        state = case["seqs"] * hv * d * d * (4 if case["state"] == "f32" else 2)
        # q, k, v in, o out; beta and g; the states read and written; the slots
        return {"bytes": 2 * state + t * ((2 * hk + 2 * hv) * d * e + hv * 4 * (2 if case["gated"] else 1)) + 4 * case["seqs"],
                "flops": t * hv * 7 * d * d}
    if op == "prep":
        e, t = (4 if case["io"] == "f32" else 2), _tokens(case)
        hk, hv, d = case["hk"], case["hv"], case["d"]
        dim = (2 * hk + hv) * d
        out = ((2 * hv if case["expand"] else 2 * hk) + hv) * d
        # x in, q, k, v out; a, b in, g, beta out; the convolution's state read and written; its weights
        return {"bytes": t * ((dim + out) * e + hv * (2 * e + 8)) + 2 * case["seqs"] * (TAPS - 1) * dim * e + dim * TAPS * e,
                "flops": t * dim * (2 * TAPS + 6)}
    if op in ("add_norm", "gated_norm"):
        e = 4 if case["io"] == "f32" else 2
        count = case["rows"] * (case["dim"] if op == "add_norm" else case["heads"] * case["d"])
        group = 128 if op == "add_norm" else case["d"]
        out = {"bf16": 2.0, "fp8": 1.0 + 4.0 / group}[case["out"]]
        # add_norm: x in, y out, the residual in and out; gated_norm: x and z in, y out
        extra = (2 if case["residual"] else 0) if op == "add_norm" else 1
        return {"bytes": count * ((1 + extra) * e + out), "flops": 8 * count}
    dim = (2 * case["hk"] + case["hv"]) * case["d"]
    slot = case["hv"] * case["d"] ** 2 * (4 if case["state"] == "f32" else 2) + (TAPS - 1) * dim * 2
    # every source read once, every destination written once
    return {"bytes": case["layers"] * slot * (-(-case["moves"] // case["fan"]) + case["moves"] + case["clear"]), "flops": 0}


# ----------------------------------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    return {"recurrent": _exact_recurrent, "prep": _exact_prep, "add_norm": _exact_norm, "gated_norm": _exact_norm,
            "copy": _exact_copy}[case["op"]](case, s, seed)


def _exact_recurrent(case, s, seed):
    """The definition, S_t = a (I - beta k k^T) S_{t-1} + beta k v^T, o = scale S^T q, a sequence at a time."""
    lengths, hk, hv, d = _lengths(case, seed), case["hk"], case["hv"], case["d"]
    if sum(lengths) > 4096:
        return None
    q, k = (s[n].double().reshape(-1, hk, d) for n in ("q", "k"))
    v, beta = s["v"].double().reshape(-1, hv, d), s["beta"].double().reshape(-1, hv)
    g = None if s["g"] is None else s["g"].double().reshape(-1, hv)
    head = torch.arange(hv, device=DEV) // (hv // hk)
    pool, o, at = s["state"].double(), torch.empty_like(v), 0
    for slot, count in zip(s["slots"].tolist(), lengths):
        S = pool[slot]
        for t in range(at, at + count):
            kt, qt = k[t, head], q[t, head]
            a = torch.ones(hv, device=DEV, dtype=torch.float64) if g is None else g[t].exp()
            kS = torch.bmm(kt[:, None], S)
            S = a[:, None, None] * (S - beta[t][:, None, None] * torch.bmm(kt[:, :, None], kS))
            S = S + torch.bmm(beta[t][:, None, None] * kt[:, :, None], v[t][:, None])
            o[t] = torch.bmm(qt[:, None], S)[:, 0] / math.sqrt(d)
        pool[slot] = S
        at += count
    return {"o": o.reshape(s["v"].shape), "state": pool}


def _exact_prep(case, s, seed):
    """A sequence at a time: its state and its inputs end to end, the convolution as a sum over windows."""
    hk, hv, d, eps = case["hk"], case["hv"], case["d"], EPS
    x = s["x"].double().reshape(-1, s["x"].shape[-1])
    w, pool = s["weight"].double(), s["conv_state"].double()
    y, at = torch.empty_like(x), 0
    for slot, count in zip(s["slots"].tolist(), _lengths(case, seed)):
        line = torch.cat([pool[slot], x[at:at + count]])
        y[at:at + count] = torch.einsum("tdj,dj->td", line.unfold(0, TAPS, 1), w)
        pool[slot] = line[line.shape[0] - (TAPS - 1):]
        at += count
    if s["bias"] is not None:
        y += s["bias"].double()
    y = y * torch.sigmoid(y)
    y = y.reshape(-1, 2 * hk + hv, d)
    qk = y[:, :2 * hk] * ((y[:, :2 * hk] ** 2).sum(-1, keepdim=True) + eps) ** -0.5
    q, k, v = qk[:, :hk], qk[:, hk:], y[:, 2 * hk:]
    if case["expand"]:
        head = torch.arange(hv, device=DEV) // (hv // hk)
        q, k = q[:, head], k[:, head]
    shape = s["x"].shape[:2]
    g = -s["A_log"].double().exp() * torch.logaddexp(s["a"].double() + s["dt_bias"].double(), torch.zeros((), device=DEV, dtype=torch.float64))
    return {"q": q.reshape(*shape, -1, d), "k": k.reshape(*shape, -1, d), "v": v.reshape(*shape, -1, d), "g": g,
            "beta": torch.sigmoid(s["b"].double()), "conv_state": pool}


def _exact_norm(case, s, seed):
    """In 8 bits the exact output is what the stored value times its scale stands for, over that scale: y / scale unrounded."""
    x, w = s["x"].double(), s["weight"].double()
    if case["op"] == "add_norm":
        h = x if s["residual"] is None else x + s["residual"].double()
        y = w * h / ((h ** 2).sum(-1, keepdim=True) / h.shape[-1] + EPS).sqrt()
        group = 128
    else:
        z = s["z"].double()
        y = w * x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * z * torch.sigmoid(z)
        group = case["d"]
    out = {}
    if case["out"] == "fp8":
        parts = y.split(group, -1)
        tops = [p.abs().amax(-1, keepdim=True) / FP8_MAX for p in parts]
        tops = [torch.where(t > 0, t, torch.ones_like(t)) for t in tops]
        y = torch.cat([p / t for p, t in zip(parts, tops)], -1)
        scales = torch.cat(tops, -1)
        out["scales"] = scales if case["op"] == "add_norm" else scales.squeeze(-1)
    else:
        out["scales"] = None
    out["y"] = y
    if case["op"] == "add_norm":
        out["residual"] = h if s["residual"] is not None else None
    return out


def _exact_copy(case, s, seed):
    moved = []
    src, dst = s["src_slots"].tolist(), s["dst_slots"].tolist()
    for pool in s["pools"]:
        p = pool.double()
        new = p.clone()
        for a, b in zip(src, dst):
            new[b] = p[a] if a >= 0 else 0.0
        moved.append(new)
    return moved
