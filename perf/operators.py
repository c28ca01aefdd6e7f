"""The encoder layer's attention operators, as they are timed and compared.

  rotary          rotary positions of the queries and keys of packed rows (half or
                  interleaved pairs, part of the head, scaled for long rows)
  qk_norm_rotary  a norm of every query and key head with the rotation in the same pass
  diff_attention  differential attention: the difference of two softmax maps with a
                  learned weight, and the norm of every head's output

Rows are packed back to back; a token's position is its index in its row.  With `own`
false each operator is computed in elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HEAD = 64  # the head width of the attention's query and key heads; values are twice as wide


# ------------------------------------------------------------------ cases


def _rotary(name, **kw):
    c = dict(op="rotary", dtype="bf16", head_dim=64, q_heads=6, k_heads=6, layout="half", dims=64, theta=160000.0,
             scaling="none", factor=1.0, original=8192, rows=1, shortest=1, longest=1)
    c.update(kw)
    return dict(c, name=name) if name else c


def _norm(name, **kw):
    c = dict(_rotary(name), op="qk_norm_rotary", norm="rms", gains=True)
    c.update(kw)
    return c


def _diff(name, **kw):
    c = dict(op="diff_attention", dtype="bf16", v_dtype="bf16", heads=3, kv_heads=3, window=-1, norm=True,
             depth=4, rows=1, shortest=1, longest=1)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one request of three questions on a 200-token state: latency counts
        _rotary("rotary request", rows=3, shortest=225, longest=300),
        # the long-context batch, positions stretched to four times a trained length of 2048
        _rotary("rotary long rows", rows=16, shortest=8192, longest=8192, scaling="yarn", factor=4.0, original=2048),
        # the throughput batch of ragged rows with half of every head rotated, interleaved pairs
        _rotary("rotary part of head", rows=256, shortest=64, longest=1024, dtype="f16", layout="interleaved",
                dims=32, scaling="ntk", factor=2.0),
        # the validation precision with a head and a rotated part that fit no vector width
        _rotary("rotary fp32 odd", rows=37, shortest=1, longest=777, dtype="f32", head_dim=80, q_heads=5, k_heads=3,
                dims=20, theta=10000.0, scaling="linear", factor=3.0),
        # one request again, norms on
        _norm("norm request", rows=3, shortest=225, longest=300),
        # the throughput batch: 1024 ragged rows
        _norm("norm throughput rows", rows=1024, shortest=64, longest=1024),
        # many query heads on few, wide key heads; layer norms
        _norm("norm wide heads", rows=48, shortest=100, longest=500, dtype="f16", head_dim=128, q_heads=32, k_heads=8,
              layout="interleaved", dims=64, norm="layer", theta=10000.0),
        # one request through a global layer, values in FP16 beside BF16 queries and keys
        _diff("diff request", rows=3, shortest=225, longest=300, v_dtype="f16"),
        # the throughput batch through a global layer
        _diff("diff throughput rows", rows=256, shortest=64, longest=1024),
        # and through a sliding-window layer
        _diff("diff window", rows=256, shortest=64, longest=1024, window=64, v_dtype="f16"),
        # the long-context batch through a global layer
        _diff("diff long rows", rows=16, shortest=8192, longest=8192, v_dtype="f16"),
        # the validation precision, shared key heads
        _diff("diff fp32", rows=24, shortest=64, longest=512, dtype="f32", v_dtype="f32", heads=4, kv_heads=2),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "qk_norm_rotary", "diff_attention"])
    longest = _log_int(rng, 1, 8192)
    shortest = rng.choice([longest, max(1, longest // 2), 1])
    if op == "diff_attention":
        dtype, v = rng.choice([("bf16", "bf16"), ("bf16", "f16"), ("f16", "f16"), ("f32", "f32")])
        kv = rng.choice([1, 2, 3])
        window = rng.choice([-1, -1, 64, 64, rng.randrange(0, 600)])
        pairs = (1 << 30) if dtype != "f32" else (1 << 26)  # row pairs of a case, times heads
        h = kv * rng.choice([1, 1, 2])
        rows = _log_int(rng, 1, max(1, min(1024, 200000 // longest, pairs // (h * longest * longest))))
        return _diff("", rows=rows, shortest=shortest, longest=longest, dtype=dtype, v_dtype=v, heads=h, kv_heads=kv,
                     window=window, norm=rng.random() < 0.8, depth=rng.randrange(0, 22))
    d = rng.choice([32, 64, 64, 64, 80, 96, 128, 256])
    qh, kh = rng.choice([(6, 6), (6, 6), (8, 2), (5, 1), (12, 4)])
    room = 200000 * 12 * 64 // ((qh + kh) * d)
    rows = _log_int(rng, 1, max(1, min(1024, room // longest)))
    scaling = rng.choice(["none", "linear", "ntk", "yarn"])
    kw = dict(rows=rows, shortest=shortest, longest=longest, head_dim=d, q_heads=qh, k_heads=kh,
              dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), layout=rng.choice(["half", "interleaved"]),
              dims=rng.choice([d, d, d // 2, 2 * rng.randrange(2, d // 2 + 1)]), theta=rng.choice([10000.0, 160000.0]),
              scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 7.5]),
              original=rng.choice([1024, 2048, 8192]))
    if op == "rotary":
        return _rotary("", **kw)
    return _norm("", norm=rng.choice(["rms", "layer"]), gains=rng.random() < 0.9, **kw)


def _lengths(case):
    """The rows' lengths: part of the case, not of the seed."""
    r = random.Random(case["rows"] * 10007 + case["shortest"] * 101 + case["longest"])
    return [r.randint(case["shortest"], case["longest"]) for _ in range(case["rows"])]


def work(case):
    lens = _lengths(case)
    T = sum(lens)
    if case["op"] != "diff_attention":
        e = 4 if case["dtype"] == "f32" else 2
        d, h = case["head_dim"], case["q_heads"] + case["k_heads"]
        b = 2 * T * h * d * e + 4 * (len(lens) + 1)
        f = T * h * 3 * case["dims"]
        if case["op"] == "qk_norm_rotary":
            b += 4 * d * 2 if case["gains"] else 0
            f += T * h * d * 4
        return {"bytes": b, "flops": f}
    e, ev = (4 if case[k] == "f32" else 2 for k in ("dtype", "v_dtype"))
    h, g, w = case["heads"], case["kv_heads"], case["window"]

    def pairs(n):
        if w < 0 or w >= n:
            return n * n
        return n * (2 * w + 1) - w * (w + 1)

    f = sum(pairs(n) for n in lens) * h * (2 * 2 * HEAD + 2 * 2 * 2 * HEAD)
    b = T * 2 * HEAD * (2 * h * e + g * e + g * ev) + 4 * (len(lens) + 1)
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = _lengths(case)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    T, dt = cu[-1], DTYPES[case["dtype"]]
    s = dict(case=case, lens=lens, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"))

    def normal(*shape, dtype=dt, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    if case["op"] == "diff_attention":
        h, kv = case["heads"], case["kv_heads"]
        s["q"] = normal(T, 2 * h, HEAD, std=1.3)
        s["k"] = normal(T, 2 * kv, HEAD, std=1.3)
        s["v"] = normal(T, kv, 2 * HEAD, dtype=DTYPES[case["v_dtype"]])
        s["lambdas"] = [normal(HEAD, dtype=torch.float32, std=0.1) for _ in range(4)]
        s["gain"] = 1.0 + 0.1 * normal(2 * HEAD, dtype=torch.float32) if case["norm"] else None
        s["out"] = torch.empty(T, h, 2 * HEAD, dtype=dt, device="cuda")
        return s
    # queries, keys and values lie side by side in a token's row, as the projection writes them
    qh, kh, d = case["q_heads"], case["k_heads"], case["head_dim"]
    packed = normal(T, qh + 2 * kh, d, std=1.5)
    s["q"], s["k"] = packed[:, :qh], packed[:, qh:qh + kh]
    s["q_out"] = torch.empty(T, qh, d, dtype=dt, device="cuda")
    s["k_out"] = torch.empty(T, kh, d, dtype=dt, device="cuda")
    if case["op"] == "qk_norm_rotary":
        s["q_gain"] = 1.0 + 0.1 * normal(d, dtype=torch.float32) if case["gains"] else None
        s["k_gain"] = 1.0 + 0.1 * normal(d, dtype=torch.float32) if case["gains"] else None
    return s


def _lambda_init(depth):
    return 0.8 - 0.6 * math.exp(-0.3 * depth)


EPS = 1e-5


# ------------------------------------------------------------------ the passes


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "diff_attention":
        return _plain_diff(state, case)
    return _plain_rotary(state, case)


def _run_own(s, case):
    import encoder_decision_model_b200 as jd

    stream = torch.cuda.current_stream()
    if case["op"] == "diff_attention":
        l1, m1, l2, m2 = s["lambdas"]
        jd.jd_diff_attention(s["q"], s["k"], s["v"], s["out"], s["cu"], l1, m1, l2, m2, _lambda_init(case["depth"]),
                             norm_gain=s["gain"], norm_eps=EPS, window=case["window"], stream=stream)
        return s["out"]
    rc = jd.rotary_config(case["dims"], case["theta"], layout=case["layout"], scaling=case["scaling"],
                          factor=case["factor"], original_length=case["original"])
    if case["op"] == "rotary":
        jd.jd_rotary(s["q"], s["k"], s["q_out"], s["k_out"], rc, cu_seqlens=s["cu"], stream=stream)
    else:
        jd.jd_qk_norm_rotary(s["q"], s["k"], s["q_out"], s["k_out"], rc, cu_seqlens=s["cu"], norm=case["norm"],
                             eps=EPS, q_gain=s["q_gain"], k_gain=s["k_gain"], stream=stream)
    return s["q_out"], s["k_out"]


def _frequencies(case):
    """Angle per position of every rotated pair, in 64 bits on the host, and the amplitude."""
    r, theta, f = case["dims"], case["theta"], case["factor"]
    if case["scaling"] == "ntk" and r > 2:
        theta = theta * f ** (r / (r - 2))
    inv = theta ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    amplitude = 1.0
    if case["scaling"] == "linear":
        inv = inv / f
    if case["scaling"] == "yarn":
        low, high = (r * math.log(case["original"] / (2 * math.pi * b)) / (2 * math.log(theta)) for b in (32.0, 1.0))
        low, high = max(math.floor(low), 0), min(math.ceil(high), r - 1)
        ramp = ((torch.arange(r // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
        inv = inv * (1 - ramp) + inv / f * ramp
        amplitude = 0.1 * math.log(f) + 1.0 if f > 1 else 1.0
    return inv, amplitude


def _plain_rotary(s, case):
    cu = s["cu"].long()
    T = s["q"].shape[0]
    t = torch.arange(T, device="cuda")
    pos = t - cu[torch.searchsorted(cu, t, right=True) - 1]
    inv, amplitude = _frequencies(case)
    angle = pos.double()[:, None] * inv.to("cuda")[None]  # far positions need 64 bits
    c, si = (amplitude * angle.cos()).float()[:, None], (amplitude * angle.sin()).float()[:, None]
    r = case["dims"]

    def one(x, gain):
        y = x.float()
        if case["op"] == "qk_norm_rotary":
            if case["norm"] == "layer":
                y = y - y.mean(-1, keepdim=True)
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
            if gain is not None:
                y = y * gain
        if case["layout"] == "half":
            a, b = y[..., :r // 2], y[..., r // 2:r]
            turned = torch.cat([a * c - b * si, b * c + a * si], -1)
        else:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
            turned = torch.stack([a * c - b * si, b * c + a * si], -1).flatten(-2)
        return torch.cat([turned, y[..., r:]], -1).to(x.dtype)

    return one(s["q"], s.get("q_gain")), one(s["k"], s.get("k_gain"))


def _plain_diff(s, case):
    h, kv, w = case["heads"], case["kv_heads"], case["window"]
    lens, cu = s["lens"], s["cu"].long()
    l1, m1, l2, m2 = s["lambdas"]
    start = _lambda_init(case["depth"])
    lam = torch.exp((l1 * m1).sum()) - torch.exp((l2 * m2).sum()) + start
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    longest = max(lens)
    at_once = max(1, (1 << 30) // (2 * h * longest * longest))  # rows whose scores are held together
    outs = []
    for r0 in range(0, len(lens), at_once):
        n = len(lens[r0:r0 + at_once])
        L = max(lens[r0:r0 + n])
        first, count = cu[r0:r0 + n, None], cu[r0 + 1:r0 + n + 1, None] - cu[r0:r0 + n, None]
        i = torch.arange(L, device="cuda")
        at = (first + i).clamp(max=q.shape[0] - 1)  # [n, L]
        qr = q[at].view(n, L, h, 2, HEAD).permute(0, 2, 3, 1, 4)
        kr = k[at].view(n, L, kv, 2, HEAD).permute(0, 2, 3, 1, 4)
        vr = v[at].permute(0, 2, 1, 3)
        if kv != h:
            kr, vr = (x.repeat_interleave(h // kv, 1) for x in (kr, vr))
        score = qr @ kr.transpose(-1, -2) * HEAD ** -0.5
        hidden = (i >= count)[:, None, None, None, :]
        if w >= 0:
            hidden = hidden | ((i[:, None] - i[None]).abs() > w)
        # a padded row of a window may see nothing: its values are not kept
        score = score.masked_fill(hidden, float("-inf"))
        score = torch.exp(score - score.amax(-1, keepdim=True))
        p = score / score.sum(-1, keepdim=True)
        d = p[:, :, 0] @ vr - lam * (p[:, :, 1] @ vr)  # [n, h, L, 128]
        if s["gain"] is not None:
            d = d * torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS) * s["gain"] * (1.0 - start)
        tok = torch.arange(sum(lens[:r0]), sum(lens[:r0 + n]), device="cuda")
        row = torch.searchsorted(cu, tok, right=True) - 1
        outs.append(d[row - r0, :, tok - cu[row]].to(s["q"].dtype))
    return torch.cat(outs)


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    """The operators' definition in 64 bits, row by row."""
    s = prepare(case, seed)
    f64 = torch.float64
    bounds = s["cu"].tolist()
    rows = [(a, b) for a, b in zip(bounds, bounds[1:]) if b > a]
    if case["op"] == "diff_attention":
        lq1, lk1, lq2, lk2 = (x.to(f64) for x in s["lambdas"])
        lam = float(torch.dot(lq1, lk1).exp() - torch.dot(lq2, lk2).exp()) + _lambda_init(case["depth"])
        out = torch.zeros(bounds[-1], case["heads"], 2 * HEAD, dtype=f64, device="cuda")
        share = case["heads"] // case["kv_heads"]
        for a, b in rows:
            i = torch.arange(b - a, device="cuda")
            seen = None if case["window"] < 0 else (i[:, None] - i[None, :]).abs() <= case["window"]
            for h in range(case["heads"]):
                value = s["v"][a:b, h // share].to(f64)
                maps = []
                for m in (0, 1):
                    qm, km = s["q"][a:b, 2 * h + m].to(f64), s["k"][a:b, 2 * (h // share) + m].to(f64)
                    z = torch.mm(qm, km.T).div_(math.sqrt(HEAD))
                    if seen is not None:
                        z.masked_fill_(~seen, -math.inf)
                    maps.append(torch.mm(torch.softmax(z, dim=1), value))
                d = maps[0] - lam * maps[1]
                if s["gain"] is not None:
                    d = d / torch.sqrt(d.square().mean(1, keepdim=True) + EPS)
                    d = d * s["gain"].to(f64) * (1.0 - _lambda_init(case["depth"]))
                out[a:b, h] = d
        return out
    r, half = case["dims"], case["dims"] // 2
    freq, base = [], case["theta"]
    if case["scaling"] == "ntk" and r > 2:
        base = base * math.pow(case["factor"], r / (r - 2.0))
    amp = 1.0
    for j in range(half):
        w = math.pow(base, -2.0 * j / r)
        if case["scaling"] == "linear":
            w /= case["factor"]
        if case["scaling"] == "yarn":
            def where(turns):
                return r * math.log(case["original"] / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
            lo, hi = max(0, math.floor(where(32.0))), min(r - 1, math.ceil(where(1.0)))
            t = min(1.0, max(0.0, (j - lo) / max(hi - lo, 0.001)))
            w = (1.0 - t) * w + t * w / case["factor"]
            amp = 0.1 * math.log(case["factor"]) + 1.0 if case["factor"] > 1 else 1.0
        freq.append(w)
    ends = torch.zeros(bounds[-1], dtype=f64, device="cuda")
    for a, b in rows:
        ends[a:b] = torch.arange(b - a, dtype=f64, device="cuda")
    turn = torch.polar(torch.full((bounds[-1], half), amp, dtype=f64, device="cuda"),
                       torch.outer(ends, torch.tensor(freq, dtype=f64, device="cuda")))
    outs = []
    for x, gain in ((s["q"], s.get("q_gain")), (s["k"], s.get("k_gain"))):
        y = x.to(f64).clone()
        if case["op"] == "qk_norm_rotary":
            if case["norm"] == "layer":
                y -= y.mean(dim=-1, keepdim=True)
            y /= torch.sqrt(y.square().mean(dim=-1, keepdim=True) + EPS)
            if gain is not None:
                y *= gain.to(f64)
        if case["layout"] == "half":
            z = torch.complex(y[..., :half], y[..., half:r]) * turn[:, None]
            y[..., :half], y[..., half:r] = z.real, z.imag
        else:
            z = torch.view_as_complex(y[..., :r].reshape(*y.shape[:-1], half, 2).contiguous()) * turn[:, None]
            y[..., :r] = torch.view_as_real(z).flatten(-2)
        outs.append(y)
    return tuple(outs)
