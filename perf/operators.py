"""Workloads of the query/key preparation and of the 4-bit K/V cache, for measurement.

Three families of calls are measured:

``rope``   RMS norm of queries and keys for each head, position rotation, and the append of
           the K/V rows to the cache, in one pass (std_qk_norm_rope)
``kv4``    K/V rows written to a 4-bit cache (std_kv4_append for new rows, std_kv4_quantize
           for rows of the full cache) and read back as values (std_kv4_read)
``attn4``  decode attention over the 4-bit cache (std_kv4_attn)

The 4-bit format: a group of 64 channels of one row has m = bf16(min x), s = bf16(fl32(max x - m) / 15),
codes c = clamp(round_half_even(fl32(x - m) / s), 0, 15) and stands for m + c s.  Codes lie in 32-bit
words of 8 channels, channel 8 j + n of a group in bits [4 n, 4 n + 4) of word j; with two groups
(head dim 128) the words of group 0 and 1 alternate.  Scales are (s, m) pairs for each group.

With ``own`` false, ``run`` computes the plain form with elementary torch operations; with ``own``
true it makes the library's calls.
"""
import math

import torch

own = False

GROUP = 64


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode token of one layer: the call whose latency counts
        dict(name="rope-token", op="rope", dtype="bf16", L=1, lens="16512", rows=1, ragged=False, Hq=28, Hkv=4, d=128,
             rot=128, interleaved=False, axes=1, norm=True, cap=16576),
        # the gamma + 1 verify rows of a padded batch of eight
        dict(name="rope-verify-batch8", op="rope", dtype="bf16", L=1, lens="4096,2011,4087,40,3133,17,0,1001",
             rows=9, ragged=True, Hq=28, Hkv=4, d=128, rot=128, interleaved=False, axes=1, norm=True, cap=4160),
        # a whole video prompt of one layer, with positions on three axes
        dict(name="rope-prompt-33k", op="rope", dtype="bf16", L=1, lens="0", rows=33024, ragged=False, Hq=28, Hkv=4, d=128,
             rot=128, interleaved=False, axes=3, norm=True, cap=33088),
        # fp32 model slice, adjacent pairs rotated, part of the head only, an odd length
        dict(name="rope-prompt-2113-f32", op="rope", dtype="f32", L=1, lens="5", rows=2113, ragged=False, Hq=4, Hkv=2, d=64,
             rot=48, interleaved=True, axes=1, norm=True, cap=2176),
        # the accepted and drafted rows of all layers: the append inside a decode round
        dict(name="kv4-append-28L", op="kv4", mode="append", dtype="bf16", L=28, lens="33024", n="9", Hkv=4, d=128, cap=33088),
        # the 4-bit copy of a prompt, one layer of a short and of a long video
        dict(name="kv4-prompt-16k", op="kv4", mode="quantize", dtype="bf16", L=1, lens="0", n="16512", Hkv=4, d=128, cap=16576),
        dict(name="kv4-prompt-143k", op="kv4", mode="quantize", dtype="bf16", L=1, lens="0", n="143616", Hkv=4, d=128,
             cap=143680),
        # fp32 slice, one query row over a short context
        dict(name="attn4-step-2k-f32", op="attn4", dtype="f32", L=1, lens="2112", rows=1, Hq=4, Hkv=2, d=64, cap=2176),
        # a draft step of one layer
        dict(name="attn4-step-16k", op="attn4", dtype="bf16", L=1, lens="16512", rows=1, Hq=28, Hkv=4, d=128, cap=16576),
        # a draft step of a ragged batch
        dict(name="attn4-step-batch8", op="attn4", dtype="bf16", L=1,
             lens="16384,20011,65536,40000,31337,59999,24242,52001", rows=1, Hq=28, Hkv=4, d=128, cap=65600),
        # a draft step of the whole stack over a long video: the largest
        dict(name="attn4-step-28L-143k", op="attn4", dtype="bf16", L=28, lens="143616", rows=1, Hq=28, Hkv=4, d=128,
             cap=143680),
        # the verify rows of the whole stack over the 4-bit cache alone
        dict(name="attn4-verify-28L-33k", op="attn4", dtype="bf16", L=28, lens="33024", rows=7, Hq=28, Hkv=4, d=128,
             cap=33088),
    ]


def _ints(text):
    """A case holds plain values: the lengths of its sequences are a text."""
    return [int(x) for x in text.split(",")]


def _text(values):
    return ",".join(str(x) for x in values)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "kv4", "attn4", "attn4"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    B = rng.choice([1, 1, 2, 3, 5, 8])
    L = rng.choice([1, 1, 2, 5, 12])
    if op == "rope":
        rows = max(1, min(_log(rng, 1, 16384), 20000 // (L * B)))
        rot = rng.choice([d, d, d, d // 2, d // 4])
        ragged = B > 1
        lens = [_log(rng, 1, min(20000, 100000 // (L * B))) - 1 for _ in range(B)]
        axes = rng.choice([1, 1, 3])
        return dict(op=op, dtype=dtype, L=L, lens=_text(lens), rows=rows, ragged=ragged, Hq=Hkv * rng.choice([1, 2, 4, 7]), Hkv=Hkv,
                    d=d, rot=rot, interleaved=rng.random() < 0.3, axes=axes, norm=rng.random() < 0.7,
                    cap=max(lens) + rows + rng.randrange(50))
    if op == "kv4":
        mode = rng.choice(["append", "quantize"])
        lens = [_log(rng, 1, min(20000, 400000 // (L * B * Hkv))) - 1 for _ in range(B)]
        most = _log(rng, 1, 32) if mode == "append" else max(1, min(_log(rng, 16, 65536), 400000 // (L * B * Hkv)))
        n = [most] * B if mode == "append" else [most] + [rng.randrange(most + 1) for _ in range(B - 1)]
        return dict(op=op, mode=mode, dtype=dtype, L=L, lens=_text(lens), n=_text(n), Hkv=Hkv, d=d,
                    cap=-(-(max(lens) + most) // 16) * 16 + 16 * rng.randrange(4))
    rows = rng.choice([1, 1, 1, 1, 2, 3, 5, 7, 9, 11])
    G = rng.choice([g for g in (1, 2, 3, 4, 6, 7, 8, 16) if g * rows <= 128])
    top = max(16, 2000000 // (L * B * Hkv * (1 if rows == 1 else 4)))
    first = _log(rng, 1, min(65536, top))
    lens = [first] + [_log(rng, 1, first + 1) - 1 for _ in range(B - 1)]
    return dict(op=op, dtype=dtype, L=L, lens=_text(lens), rows=rows, Hq=G * Hkv, Hkv=Hkv, d=d,
                cap=-(-(max(lens) + rows - 1) // 16) * 16 + 16 * rng.randrange(4))


def _eb(case):
    return 4 if case["dtype"] == "f32" else 2


def _valid_rows(case):
    """Rows of each sequence that a ragged (padded) call holds."""
    return [max(0, case["rows"] - 2 * b) if case["ragged"] else case["rows"] for b in range(len(_ints(case["lens"])))]


def work(case):
    L, d, Hkv, eb = case["L"], case["d"], case["Hkv"], _eb(case)
    packed = d // 2 + 4 * (d // GROUP)
    if case["op"] == "rope":
        tokens = L * sum(_valid_rows(case))
        values = tokens * (case["Hq"] + 2 * Hkv) * d
        return {"bytes": 2 * values * eb + 4 * case["axes"] * tokens // L,
                "flops": tokens * (case["Hq"] + Hkv) * (4 * d + 3 * case["rot"])}
    if case["op"] == "kv4":
        rows = 2 * L * Hkv * sum(_ints(case["n"]))
        # values in, 4-bit rows out; and back
        return {"bytes": rows * (2 * d * eb + 2 * packed), "flops": rows * d * 8}
    rows = case["rows"]
    keys = L * Hkv * sum(n + rows - 1 for n in _ints(case["lens"]))
    pairs = L * case["Hq"] * sum(rows * n + rows * (rows - 1) // 2 for n in _ints(case["lens"]))
    return {"bytes": 2 * keys * packed + 2 * L * len(_ints(case["lens"])) * case["Hq"] * rows * d * eb, "flops": 4 * pairs * d}


# --------------------------------------------------------------------------- the 4-bit format in plain torch

def _quantize(x):
    """[..., d] -> codes uint8 [..., d], scales bf16 [..., d / 64, 2] (s, m)."""
    x = x.float()
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    m = g.amin(-1, keepdim=True).to(torch.bfloat16).float()
    s = ((g.amax(-1, keepdim=True) - m) / 15.0).to(torch.bfloat16).float()
    diff = (g - m).double()
    c = torch.where(s > 0, torch.round(diff / s.double()), torch.zeros_like(diff)).clamp_(0, 15).to(torch.uint8)
    return c.reshape(x.shape), torch.cat([s, m], -1).to(torch.bfloat16)


def _pack(c):
    """codes [..., d] -> bytes [..., d / 2] in the cache's order."""
    w = c.reshape(*c.shape[:-1], -1, GROUP // 8, 8).transpose(-3, -2).reshape(*c.shape[:-1], -1, 2)
    return (w[..., 0] | (w[..., 1] << 4)).contiguous()


def _unpack(p):
    """bytes [..., d / 2] -> codes [..., d]."""
    d = 2 * p.shape[-1]
    w = torch.stack([p & 15, p >> 4], -1).reshape(*p.shape[:-1], GROUP // 8, d // GROUP, 8)
    return w.transpose(-3, -2).reshape(*p.shape[:-1], d)


def _values(p, scales, dtype=torch.float32):
    """The values that packed rows stand for, [..., d]."""
    c = _unpack(p).to(dtype).reshape(*scales.shape[:-1], GROUP)
    sc = scales.to(dtype)
    return (sc[..., 1:2] + c * sc[..., 0:1]).reshape(*p.shape[:-1], 2 * p.shape[-1])


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _storage(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _kv_layer(g, case, n):
    """K and V rows of one layer, [B][Hkv][n][d], with a direction that a few keys share and a sink at row 0."""
    B, Hkv, d = len(_ints(case["lens"])), case["Hkv"], case["d"]
    u = _randn(g, B, Hkv, 1, d)
    u = u / u.norm(dim=-1, keepdim=True)
    k = _randn(g, B, Hkv, n, d)
    k += 4 * u * (torch.rand(B, Hkv, n, 1, generator=g, device="cuda") < 0.01)
    if n:
        k[:, :, 0] *= 6 / 4
    return k, _randn(g, B, Hkv, n, d), u


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    st = _storage(case)
    L, B, Hkv, d, cap = case["L"], len(_ints(case["lens"])), case["Hkv"], case["d"], case["cap"]
    s = {"case": case, "len": _int32(_ints(case["lens"]))}
    if case["op"] == "rope":
        rows, Hq = case["rows"], case["Hq"]
        # the projection's output, q, k and v of a token side by side
        s["qkv"] = (_randn(g, L, B, rows, Hq + 2 * Hkv, d) * 1.5 + 0.1).to(st)
        s["q_weight"] = (1 + 0.2 * _randn(g, L, d)).to(st) if case["norm"] else None
        s["k_weight"] = (1 + 0.2 * _randn(g, L, d)).to(st) if case["norm"] else None
        s["eps"] = 1e-6
        half = case["rot"] // 2
        s["inv_freq"] = 1000000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        s["sections"] = [half] if case["axes"] == 1 else [half - 2 * (3 * half // 8), 3 * half // 8, 3 * half // 8]
        # text: the cache position; video: frame, row and column of a patch, after the prompt's start
        if case["axes"] == 1:
            s["pos"] = None
        else:
            r = torch.arange(rows, device="cuda").expand(B, rows)
            s["pos"] = torch.stack([r // 256, r // 16 % 16, r % 16]).to(torch.int32) + s["len"].view(1, B, 1)
            s["pos"] = s["pos"].contiguous()
        s["n_rows"] = _int32(_valid_rows(case)) if case["ragged"] else None
        s["q_out"] = torch.zeros(L, B, Hq, rows, d, dtype=st, device="cuda")
        s["k_cache"] = torch.zeros(L, B, Hkv, cap, d, dtype=st, device="cuda")
        s["v_cache"] = torch.zeros_like(s["k_cache"])
    elif case["op"] == "kv4":
        most = max(_ints(case["n"]))
        s["begin"], s["count"] = s["len"], _int32(_ints(case["n"]))
        rows = cap if case["mode"] == "quantize" else most
        k, v = [], []
        for _ in range(L):
            a, b, _u = _kv_layer(g, case, rows)
            k.append(a.to(st))
            v.append(b.to(st))
        s["k"], s["v"] = torch.stack(k), torch.stack(v)
        s["cache"] = _empty_cache(L, B, Hkv, cap, d)
        s["k_out"] = torch.zeros(L, B, Hkv, most, d, dtype=st, device="cuda")
        s["v_out"] = torch.zeros_like(s["k_out"])
    else:
        rows, G = case["rows"], case["Hq"] // Hkv
        cache = _empty_cache(L, B, Hkv, cap, d)
        n = max(_ints(case["lens"])) + rows - 1
        q = torch.empty(L, B, case["Hq"], rows, d, dtype=st, device="cuda")
        for layer in range(L):
            k, v, u = _kv_layer(g, case, n)
            for name, x in (("k", k), ("v", v)):
                c, sc = _quantize(x.to(st))
                cache[name + "_codes"][layer, :, :, :n] = _pack(c)
                cache[name + "_scales"][layer, :, :, :n] = sc
            q[layer] = (_randn(g, B, case["Hq"], rows, d) + 4 * u.repeat_interleave(G, 1)).to(st)
        s["q"], s["cache"] = q, cache
        s["o"] = torch.zeros_like(q)
    if own:
        from sparse_top_kv_std_b200 import binding as b
        code = b.STD_F32 if case["dtype"] == "f32" else b.STD_BF16
        s["dims"] = b.dims(L, B, case.get("Hq", Hkv), Hkv, d, code, cap, 1)
        if case["op"] == "rope":
            s["rope"] = b.std_rope(s["inv_freq"], sections=s["sections"], interleaved=case["interleaved"])
        elif case["op"] == "attn4":
            s["ws"] = torch.empty(max(16, b.std_kv4_attn_workspace_size(s["dims"], case["rows"], cap)), dtype=torch.uint8,
                                  device="cuda")
    return s


def _empty_cache(L, B, Hkv, cap, d):
    c = {}
    for x in "kv":
        c[x + "_codes"] = torch.zeros(L, B, Hkv, cap, d // 2, dtype=torch.uint8, device="cuda")
        c[x + "_scales"] = torch.zeros(L, B, Hkv, cap, d // GROUP, 2, dtype=torch.bfloat16, device="cuda")
    c["cap"] = cap
    return c


# --------------------------------------------------------------------------- one pass

def run(state):
    return _OWN[state["case"]["op"]](state) if own else _PLAIN[state["case"]["op"]](state)


def _own_rope(s):
    from sparse_top_kv_std_b200 import binding as b
    case = s["case"]
    Hq, Hkv = case["Hq"], case["Hkv"]
    q, k, v = s["qkv"].split([Hq, Hkv, Hkv], dim=3)
    b.std_qk_norm_rope(s["dims"], s["rope"], q, k, v, case["rows"], s["n_rows"], s["q_weight"], s["k_weight"], s["eps"],
                       s["pos"], s["q_out"], s["k_cache"], s["v_cache"], case["cap"], s["len"], 0)
    return s["q_out"], s["k_cache"], s["v_cache"]


def _own_kv4(s):
    from sparse_top_kv_std_b200 import binding as b
    case = s["case"]
    most = max(_ints(case["n"]))
    if case["mode"] == "append":
        b.std_kv4_append(s["dims"], s["cache"], s["len"], 0, s["k"], s["v"], most)
    else:
        b.std_kv4_quantize(s["dims"], s["cache"], s["k"], s["v"], s["begin"], s["count"], most)
    b.std_kv4_read(s["dims"], s["cache"], s["begin"], s["count"], most, s["k_out"], s["v_out"])
    return s["k_out"], s["v_out"]


def _own_attn4(s):
    from sparse_top_kv_std_b200 import binding as b
    b.std_kv4_attn(s["dims"], s["q"], s["case"]["rows"], s["cache"], s["len"], 0, s["o"], s["ws"])
    return s["o"]


_OWN = {"rope": _own_rope, "kv4": _own_kv4, "attn4": _own_attn4}


def _rope_plain(x, w, eps, cos, sin, rot, interleaved):
    """x [rows][H][d] fp32, cos / sin [rows][1][rot / 2]."""
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1)


def _positions(s, b, n):
    """Position of every (row, pair) of sequence b, [n][rot / 2]."""
    half = s["case"]["rot"] // 2
    if s["pos"] is None:
        return (_ints(s["case"]["lens"])[b] + torch.arange(n, device="cuda")).view(n, 1).expand(n, half)
    axis = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(s["sections"], device="cuda"))
    return s["pos"][:, b, :n].t()[:, axis]


def _plain_rope(s):
    case = s["case"]
    st = _storage(case)
    Hq, Hkv = case["Hq"], case["Hkv"]
    q_out, k_cache, v_cache = s["q_out"], s["k_cache"], s["v_cache"]
    for b, n in enumerate(_valid_rows(case)):
        angle = _positions(s, b, n).double() * s["inv_freq"]
        cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
        at = _ints(case["lens"])[b]
        for layer in range(case["L"]):
            q, k, v = s["qkv"][layer, b, :n].split([Hq, Hkv, Hkv], dim=1)
            qw, kw = (s[x][layer] if case["norm"] else None for x in ("q_weight", "k_weight"))
            args = (s["eps"], cos, sin, case["rot"], case["interleaved"])
            q_out[layer, b, :, :n] = _rope_plain(q.float(), qw, *args).to(st).transpose(0, 1)
            k_cache[layer, b, :, at:at + n] = _rope_plain(k.float(), kw, *args).to(st).transpose(0, 1)
            v_cache[layer, b, :, at:at + n] = v.transpose(0, 1)
    return q_out, k_cache, v_cache


def _plain_kv4(s):
    case = s["case"]
    st = _storage(case)
    for b, n in enumerate(_ints(case["n"])):
        at = _ints(case["lens"])[b]
        src = slice(0, n) if case["mode"] == "append" else slice(at, at + n)
        for layer in range(case["L"]):
            for x in "kv":
                c, sc = _quantize(s[x][layer, b, :, src])
                codes, scales = s["cache"][x + "_codes"], s["cache"][x + "_scales"]
                codes[layer, b, :, at:at + n] = _pack(c)
                scales[layer, b, :, at:at + n] = sc
                s[x + "_out"][layer, b, :, :n] = _values(codes[layer, b, :, at:at + n], scales[layer, b, :, at:at + n]).to(st)
    return s["k_out"], s["v_out"]


def _attend(s, layer, b, dtype):
    """Attention of one layer and sequence in `dtype`, [Hq][rows][d]."""
    case = s["case"]
    rows, Hkv, d = case["rows"], case["Hkv"], case["d"]
    G = case["Hq"] // Hkv
    n = _ints(case["lens"])[b] + rows - 1
    if n == 0:
        return torch.zeros(case["Hq"], rows, d, dtype=dtype, device="cuda")
    k, v = (_values(s["cache"][x + "_codes"][layer, b, :, :n], s["cache"][x + "_scales"][layer, b, :, :n], dtype) for x in "kv")
    q = s["q"][layer, b].to(dtype).reshape(Hkv, G * rows, d)
    x = torch.matmul(q, k.transpose(1, 2)) / math.sqrt(d)
    i = torch.arange(rows, device="cuda").repeat(G).view(1, -1, 1)
    seen = torch.arange(n, device="cuda").view(1, 1, -1) < _ints(case["lens"])[b] + i
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
    return o.reshape(case["Hq"], rows, d)


def _plain_attn4(s):
    for layer in range(s["case"]["L"]):
        for b in range(len(_ints(s["case"]["lens"]))):
            s["o"][layer, b] = _attend(s, layer, b, torch.float32).to(s["o"].dtype)
    return s["o"]


_PLAIN = {"rope": _plain_rope, "kv4": _plain_kv4, "attn4": _plain_attn4}


# --------------------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "kv4": _exact_kv4, "attn4": _exact_attn4}[case["op"]](s)


def _exact_rope(s):
    case = s["case"]
    L, B, rows, Hq, Hkv, d, cap = (case["L"], len(_ints(case["lens"])), case["rows"], case["Hq"], case["Hkv"], case["d"], case["cap"])
    half = case["rot"] // 2
    q_out = torch.zeros(L, B, Hq, rows, d, dtype=torch.float64, device="cuda")
    k_out = torch.zeros(L, B, Hkv, cap, d, dtype=torch.float64, device="cuda")
    v_out = torch.zeros_like(k_out)
    lo = torch.arange(half, device="cuda")
    first, second = (2 * lo, 2 * lo + 1) if case["interleaved"] else (lo, lo + half)
    for b, n in enumerate(_valid_rows(case)):
        at = _ints(case["lens"])[b]
        turn = torch.zeros(n, half, dtype=torch.float64, device="cuda")
        start = 0
        for axis, width in enumerate(s["sections"]):
            pos = s["pos"][axis, b, :n].double() if s["pos"] is not None else at + torch.arange(n, device="cuda").double()
            turn[:, start:start + width] = pos[:, None] * s["inv_freq"][start:start + width]
            start += width
        z = torch.polar(torch.ones_like(turn), turn)[:, None]
        for layer in range(L):
            x = s["qkv"][layer, b, :n].double()
            v_out[layer, b, :, at:at + n] = x[:, Hq + Hkv:].transpose(0, 1)
            for part, weight, out, row in ((x[:, :Hq], s["q_weight"], q_out, 0), (x[:, Hq:Hq + Hkv], s["k_weight"], k_out, at)):
                y = part.clone()
                if weight is not None:
                    y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / d + s["eps"]) * weight[layer].double()
                w = torch.complex(y[..., first], y[..., second]) * z
                y[..., first], y[..., second] = w.real, w.imag
                out[layer, b, :, row:row + n] = y.transpose(0, 1)
    return q_out, k_out, v_out


def _exact_kv4(s):
    case = s["case"]
    outs = []
    for x in "kv":
        out = torch.zeros(s[x + "_out"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_ints(case["n"])):
            at = 0 if case["mode"] == "append" else _ints(case["lens"])[b]
            for layer in range(case["L"]):
                for group in range(case["d"] // GROUP):
                    ch = slice(GROUP * group, GROUP * (group + 1))
                    r = s[x][layer, b, :, at:at + n, ch].float()
                    low = r.min(-1, keepdim=True).values.bfloat16().float()
                    step = ((r.max(-1, keepdim=True).values - low) / 15).bfloat16().double()
                    code = ((r - low).double() / step.clamp_min(1e-300)).round().clamp(0, 15)
                    out[layer, b, :, :n, ch] = low.double() + step * code
        outs.append(out)
    return tuple(outs)


def _exact_attn4(s):
    """One key/value head at a time, straight from the nibbles."""
    case = s["case"]
    rows, d, G = case["rows"], case["d"], case["Hq"] // case["Hkv"]
    out = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    ch = torch.arange(d, device="cuda")
    word = (ch % GROUP // 8) * (d // GROUP) + ch // GROUP
    byte, shift = 4 * word + ch % 8 // 2, (4 * (ch % 2)).to(torch.uint8)

    def rows_of(x, layer, b, h, n):
        code = (s["cache"][x + "_codes"][layer, b, h, :n][:, byte] >> shift) & 15
        sc = s["cache"][x + "_scales"][layer, b, h, :n].double()
        return code.double() * sc[:, :, 0].repeat_interleave(GROUP, 1) + sc[:, :, 1].repeat_interleave(GROUP, 1)

    for layer in range(case["L"]):
        for b, n0 in enumerate(_ints(case["lens"])):
            for h in range(case["Hkv"]):
                n = n0 + rows - 1
                if n == 0:
                    continue
                k, v = rows_of("k", layer, b, h, n), rows_of("v", layer, b, h, n)
                for i in range(rows):
                    if n0 + i == 0:
                        continue
                    q = s["q"][layer, b, h * G:(h + 1) * G, i].double()
                    p = torch.softmax(q @ k[:n0 + i].t() * d ** -0.5, -1)
                    out[layer, b, h * G:(h + 1) * G, i] = p @ v[:n0 + i]
    return out
