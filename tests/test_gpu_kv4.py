"""The 4-bit cache on the GPU: rows written and read back, and decode attention over it, against
the fp64 oracle.

Writing is exact: codes, scales and minima are those of the definition, bit for bit, and so are
the values read back (m + c s is one fp32 rounding, then one to bf16).

Attention tolerances.  A tensor-core step adds 16 products to a float32 accumulator; with its
internal alignment it is off by at most 2^-22 of the sum of the magnitudes so far.  A logit takes
d / 16 steps (twice that for fp32 queries) and a few float32 operations:
    dx <= (d / 8 + 8) 2^-22 A,   A = max_j sum_g (sk |q . (a - 8)|_abs + |mk + 8 sk| |q|_abs) / sqrt d
A weight is then off by dx + 2^-20 (relative; ex2 within two units, its argument rounded at
magnitude X = max |x| log2 e: X 2^-24 more).  For bf16 queries p s is rounded to 11 bits (2^-12
relative); fp32 keeps 22.  The sum over n keys runs in at most n / 16 steps of one warp:
    do <= (2 (dx + 2^-20 + X 2^-23) + r + (n / 16 + 16) 2^-22) V,  V = max_c (max (s |b - 8|) + max |m + 8 s|)
with r = 2^-11 (bf16) or 2^-21 (fp32), and the output is rounded to its type (finfo.eps / 2)."""
import numpy as np
import pytest
import torch

from oracle import kv4_oracle as O
from sparse_top_kv_std_b200 import binding as B
from sparse_top_kv_std_b200.kv4 import Kv4Cache
from tests import harness as H

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    B.lib()
    B.std_get_device_error(clear=True)


def _code(dtype):
    return B.STD_F32 if dtype == torch.float32 else B.STD_BF16


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _guarded(cv, L, nB, Hkv, cap, d):
    c = {"cap": cap}
    for x in "kv":
        c[x + "_codes"] = cv.tensor((L, nB, Hkv, cap, d // 2), torch.uint8, fill=0x5a)
        c[x + "_scales"] = cv.tensor((L, nB, Hkv, cap, d // 64, 2), torch.bfloat16, fill=float("nan"))
    return c


def _bits(t):
    return t.view(torch.int16 if t.element_size() == 2 else torch.int32)


def _same(a, b):
    """Equal values, NaN equal to NaN."""
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


# ----------------------------------------------------------------------------- rows in and out

def _rows(kind, shape, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda")
    if kind == "ties":        # many quotients exactly half way
        x = torch.randint(-30, 31, shape, generator=g, device="cuda") * 0.5
        x[..., 0::64] = -15.0
        x[..., 1::64] = 15.0
    elif kind == "offset":
        x = x * 1e-3 + 100
    elif kind == "huge":
        x = x * 3e37
    elif kind == "tiny":      # scales below the smallest normal number
        x = x * 1e-39
    elif kind == "odd":       # constant, one outlier, not finite
        x[..., 0, :] = 1.25
        x[..., 1, :] = 0
        x[..., 1, 3] = 1e6
        x[..., 2, 70 % shape[-1]] = float("inf")
        x[..., 3, 5] = float("nan")
        x[..., 4, 6] = -float("inf")
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["normal", "ties", "offset", "huge", "tiny", "odd"])
def test_append_and_read_are_exact(dtype, d, kind):
    L, nB, Hkv, n, cap = 2, 3, 2, 23, 64
    lens = [0, 5, 38]
    cv = H.Canaries()
    c = _guarded(cv, L, nB, Hkv, cap, d)
    k, v = (_rows(kind, (L, nB, Hkv, n, d), dtype, s) for s in (1, 2))
    dims = B.dims(L, nB, Hkv, Hkv, d, _code(dtype), 1, 1)
    before = {x: t.clone() for x, t in c.items() if x != "cap"}
    B.std_kv4_append(dims, c, _i32(lens), 2, k, v, n)
    k_out, v_out = (cv.tensor(tuple(k.shape), dtype, fill=-3) for _ in "kv")
    B.std_kv4_read(dims, c, _i32([x + 2 for x in lens]), None, n, k_out, v_out)
    cv.check()
    assert B.std_get_device_error() == 0
    for x, src, out in (("k", k, k_out), ("v", v, v_out)):
        codes, s, m = O.kv4_quantize(src.float().cpu().numpy())
        want = O.kv4_values(codes, s, m)
        for b in range(nB):
            at = slice(lens[b] + 2, lens[b] + 2 + n)
            got = c[x + "_codes"][:, b, :, at].cpu().numpy()
            assert (got == O.kv4_pack(codes[:, b])).all()
            sc = c[x + "_scales"][:, b, :, at].float().cpu().numpy()
            assert np.array_equal(sc[..., 0], s[:, b]) and np.array_equal(sc[..., 1], m[:, b], equal_nan=True)
            # other rows as they were
            for name in ("_codes", "_scales"):
                t, t0 = c[x + name], before[x + name]
                t, t0 = (t, t0) if name == "_codes" else (_bits(t), _bits(t0))
                assert torch.equal(t[:, b, :, :at.start], t0[:, b, :, :at.start])
                assert torch.equal(t[:, b, :, at.stop:], t0[:, b, :, at.stop:])
        assert _same(out, torch.from_numpy(want).cuda().float().to(dtype))


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float32, 64)])
@pytest.mark.parametrize("n", [1, 16, 331, 2500])
def test_quantise_from_a_full_cache(dtype, d, n):
    L, nB, Hkv, cap_full, cap = 1, 3, 2, 2600, 2608
    begin, count = [0, 99, 2599 if n == 1 else 17], [n, n // 2, min(n, 1)]
    cv = H.Canaries()
    c = _guarded(cv, L, nB, Hkv, cap, d)
    k, v = (_rows("normal", (L, nB, Hkv, cap_full, d), dtype, s) for s in (3, 4))
    dims = B.dims(L, nB, Hkv, Hkv, d, _code(dtype), cap_full, 1)
    B.std_kv4_quantize(dims, c, k, v, _i32(begin), _i32(count), n)
    out = cv.tensor((L, nB, Hkv, n, d), dtype, fill=-3)
    out_v = cv.tensor((L, nB, Hkv, n, d), dtype, fill=-3)
    B.std_kv4_read(dims, c, _i32(begin), _i32(count), n, out, out_v)
    cv.check()
    assert B.std_get_device_error() == 0
    for src, got in ((k, out), (v, out_v)):
        for b in range(nB):
            rows = src[:, b, :, begin[b]:begin[b] + count[b]].float().cpu().numpy()
            want = torch.from_numpy(O.kv4_values(*O.kv4_quantize(rows))).cuda().float().to(dtype)
            assert torch.equal(got[:, b, :, :count[b]], want)
            assert (got[:, b, :, count[b]:] == -3).all()     # rows behind a sequence's last are left
    # begin NULL and count NULL: the first max_n rows of every sequence
    c2 = Kv4Cache(L, nB, Hkv, cap, d)
    B.std_kv4_quantize(dims, c2, k, v, None, None, n)
    c3 = Kv4Cache(L, nB, Hkv, cap, d)
    B.std_kv4_append(dims, c3, _i32([0] * nB), 0, k[:, :, :, :n].contiguous(), v[:, :, :, :n].contiguous(), n)
    assert all(torch.equal(_bits(c2[x]) if "sc" in x else c2[x], _bits(c3[x]) if "sc" in x else c3[x])
               for x in ("k_codes", "k_scales", "v_codes", "v_scales"))


def test_rows_past_a_capacity_are_skipped_and_flagged():
    L, nB, Hkv, d, cap = 1, 4, 1, 64, 32
    k = _rows("normal", (L, nB, Hkv, 8, d), torch.bfloat16)
    cv = H.Canaries()
    c = _guarded(cv, L, nB, Hkv, cap, d)
    dims = B.dims(L, nB, Hkv, Hkv, d, B.STD_BF16, 8, 1)
    B.std_kv4_append(dims, c, _i32([24, 25, -1, 0]), 0, k, k, 8)
    cv.check()
    assert B.std_get_device_error() == B.STD_DEVERR_CAPACITY
    assert (c["k_codes"][0, 1] == 0x5a).all() and (c["k_codes"][0, 2] == 0x5a).all()
    assert torch.isnan(c["v_scales"][0, 1].float()).all()
    assert not torch.isnan(c["v_scales"][0, 0, 0, 24:].float()).any()
    # the source's capacity and the count's bound count too
    for begin, count in (([0] * 4, [9, 0, 0, 0]), ([0, 1, 0, 0], [8, 8, 0, 0]), ([0] * 4, [0, -1, 0, 0])):
        B.std_kv4_quantize(dims, c, k, k, _i32(begin), _i32(count), 8)
        assert B.std_get_device_error() == B.STD_DEVERR_CAPACITY
    out = cv.tensor((L, nB, Hkv, 8, d), torch.bfloat16, fill=-3)
    B.std_kv4_read(dims, c, _i32([25, 24, 24, 24]), None, 8, out, cv.like(out))
    cv.check()
    assert B.std_get_device_error() == B.STD_DEVERR_CAPACITY
    assert (out[0, 0] == -3).all()


# ----------------------------------------------------------------------------- attention

def _attn_inputs(L, nB, Hq, Hkv, d, rows, lens, off, dtype, seed=0, kind="normal", cap=None, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    n = max(lens) + off + rows - 1
    cap = cap or -(-max(n, 1) // 16) * 16
    k, v = rn(L, nB, Hkv, cap, d), rn(L, nB, Hkv, cap, d)
    q = rn(L, nB, Hq, rows, d) * scale
    if kind == "rising":       # every tile beats the last one's logits: the reference moves on
        k = k + q[:, :, ::Hq // Hkv, :1] * torch.linspace(0, 2, cap, device="cuda").view(1, 1, 1, cap, 1)
    elif kind == "sink":
        k[:, :, :, 0] = 3 * q[:, :, ::Hq // Hkv, 0]
    elif kind == "scales":     # value rows of very different size
        v = v * torch.pow(10.0, torch.randint(-9, 5, (L, nB, Hkv, cap, 1), generator=g, device="cuda").float())
    elif kind == "constant":   # value rows whose scale is 0
        v[:] = v[..., :1]
    cv = H.Canaries()
    c = _guarded(cv, L, nB, Hkv, cap, d)
    dims = B.dims(L, nB, Hq, Hkv, d, _code(dtype), cap, 1)
    q, k, v = (cv.like(t.to(dtype)) for t in (q, k, v))
    used = [x + off + rows - 1 for x in lens]
    B.std_kv4_quantize(dims, c, k, v, None, _i32([min(max(x, 0), cap) for x in used]), cap)
    B.std_get_device_error(clear=True)
    return dims, q, c, cv, cap


def _attend(dims, q, rows, c, cv, lens, off, stream=None):
    o = cv.tensor(tuple(q.shape), q.dtype, fill=-9)
    ws = cv.tensor((max(16, B.std_kv4_attn_workspace_size(dims, rows, c["cap"])),), torch.uint8, fill=0xff)
    B.std_kv4_attn(dims, q, rows, c, _i32(lens) if isinstance(lens, list) else lens, off, o, ws, stream)
    return o


def _parts(c, x):
    codes = O.kv4_unpack(c[x + "_codes"].cpu().numpy())
    sc = c[x + "_scales"].float().cpu().numpy()
    return codes, sc[..., 0], sc[..., 1]


def _want(q, c, lens, off, dtype):
    """Oracle output and tolerance."""
    kc, ks, km = _parts(c, "k")
    vc, vs, vm = _parts(c, "v")
    q = q.double().cpu().numpy()
    L, nB, Hq, rows, d = q.shape
    G, n = Hq // kc.shape[2], max(lens) + off + rows - 1
    first = np.array(lens) + off
    want = O.causal_decode_attn(q, np.nan_to_num(O.kv4_values(kc, ks, km)), np.nan_to_num(O.kv4_values(vc, vs, vm)), first)
    tol = np.zeros(want.shape[:3] + (1, 1))
    for l in range(L):
        for b in range(nB):
            m = max(int(first[b]) + rows - 1, 0)
            if m == 0:
                continue
            for h in range(Hq):
                kv = h // G
                e = lambda t: np.repeat(t[l, b, kv, :m].astype(np.float64), 64, -1)  # noqa: E731
                aq = np.abs(q[l, b, h]).max(0)
                A = ((np.abs(kc[l, b, kv, :m] - 8.0) * e(ks) + np.abs(e(km) + 8 * e(ks))) @ aq).max() / np.sqrt(d)
                V = (np.abs(vc[l, b, kv, :m] - 8.0) * e(vs)).max() + np.abs(e(vm) + 8 * e(vs)).max()
                dx = (d / 8 + 8) * 2.0 ** -22 * A
                X = A * 1.4427
                r = 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -21
                tol[l, b, h] = (2 * (dx + 2.0 ** -20 + X * 2.0 ** -23) + r + (n / 16 + 16) * 2.0 ** -22) * V
    return want, tol + torch.finfo(dtype).eps / 2 * np.abs(want)


def _check(o, q, c, lens, off, dtype):
    want, tol = _want(q, c, lens, off, dtype)
    err = np.abs(o.double().cpu().numpy() - want)
    assert (err <= tol).all(), (float(err.max()), float((err / np.maximum(tol, 1e-300)).max()))


# (Hq, Hkv, d, rows): 1 to 128 query rows of a KV head, one to three rows of 8 and of 16, both dims
SHAPES = [(4, 2, 64, 1), (1, 1, 128, 1), (7, 1, 128, 1), (16, 2, 64, 1), (16, 1, 128, 1), (6, 2, 128, 3), (28, 4, 128, 9),
          (8, 8, 64, 11), (16, 1, 64, 8), (4, 4, 128, 32), (9, 1, 128, 1)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hq,Hkv,d,rows", SHAPES)
def test_head_layouts_and_row_counts(dtype, Hq, Hkv, d, rows):
    lens = [301, 0, 17]
    dims, q, c, cv, _ = _attn_inputs(2, 3, Hq, Hkv, d, rows, lens, 1, dtype, seed=1)
    o = _attend(dims, q, rows, c, cv, lens, 1)
    cv.check()
    assert B.std_get_device_error() == 0
    _check(o, q, c, lens, 1, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 127, 128, 129, 255, 1000, 4099])
@pytest.mark.parametrize("d,rows", [(128, 1), (64, 3)])
def test_lengths(dtype, n, d, rows):
    dims, q, c, cv, _ = _attn_inputs(1, 1, 4, 1, d, rows, [n], 0, dtype, seed=n)
    o = _attend(dims, q, rows, c, cv, [n], 0)
    cv.check()
    assert B.std_get_device_error() == 0
    _check(o, q, c, [n], 0, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_without_keys_are_zero(dtype):
    """Length 0 and no offset: position 0 attends nothing, position i the first i keys."""
    for rows, lens in ((1, [0, 3, 0]), (4, [0, 0, 5])):
        dims, q, c, cv, _ = _attn_inputs(1, 3, 4, 2, 64, rows, lens, 0, dtype, seed=3)
        o = _attend(dims, q, rows, c, cv, lens, 0)
        cv.check()
        assert B.std_get_device_error() == 0
        assert (o[0, 0, :, 0] == 0).all()
        _check(o, q, c, lens, 0, dtype)
    lens = [0, 0]                                # nothing anywhere
    dims, q, c, cv, _ = _attn_inputs(2, 2, 4, 2, 128, 1, lens, 0, dtype, seed=3)
    o = _attend(dims, q, 1, c, cv, lens, 0)
    cv.check()
    assert (o == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind,scale", [("rising", 1.0), ("sink", 1.0), ("scales", 1.0), ("constant", 1.0), ("normal", 8.0),
                                        ("normal", 0.0)])
@pytest.mark.parametrize("Hq,rows", [(7, 1), (5, 7)])
def test_moving_references_and_scales(dtype, kind, scale, Hq, rows):
    lens = [1500, 700]
    dims, q, c, cv, _ = _attn_inputs(1, 2, Hq, 1, 128, rows, lens, 1, dtype, seed=5, kind=kind, scale=scale)
    o = _attend(dims, q, rows, c, cv, lens, 1)
    cv.check()
    assert B.std_get_device_error() == 0
    _check(o, q, c, lens, 1, dtype)


@pytest.mark.parametrize("n", [700, 2112, 30000])
@pytest.mark.parametrize("d,Hq,rows", [(64, 2, 1), (128, 1, 1), (128, 5, 3)])
def test_fp32_results_keep_fp32_accuracy(n, d, Hq, rows):
    """Diffuse attention, where the result is a small difference of large sums.  A fp32 accumulator of a
    tensor core is off by at most 2^-23 of its size a step; over a warp's n / 128 or fewer steps of
    centred codes, whose sums grow like sqrt(n), that is below sqrt(n / 128) 2^-23 of the result, 2e-6
    here; the logits' own rounding (2^-22 of some 30 in each) adds as much, at random."""
    dims, q, c, cv, _ = _attn_inputs(1, 1, Hq, 1, d, rows, [n], 0, torch.float32, seed=n)
    o = _attend(dims, q, rows, c, cv, [n], 0)
    want, _ = _want(q, c, [n], 0, torch.float32)
    err = np.linalg.norm(o.double().cpu().numpy() - want) / np.linalg.norm(want)
    assert err <= 8e-6, err


@pytest.mark.parametrize("dtype,Hq,rows", [(torch.bfloat16, 7, 1), (torch.float32, 2, 1), (torch.bfloat16, 7, 7)])
def test_long_context_split_over_the_device(dtype, Hq, rows):
    lens = [70001, 33333]
    dims, q, c, cv, _ = _attn_inputs(1, 2, Hq, 1, 128, rows, lens, 0, dtype, seed=6)
    o = _attend(dims, q, rows, c, cv, lens, 0)
    cv.check()
    assert B.std_get_device_error() == 0
    _check(o, q, c, lens, 0, dtype)


@pytest.mark.parametrize("rows", [1, 5])
def test_many_short_problems(rows):
    """More units than CTAs, one of them shared between neighbours, and a batch above 32."""
    lens = [(37 * i) % 300 for i in range(70)]
    dims, q, c, cv, _ = _attn_inputs(3, 70, 6, 3, 64, rows, lens, 1, torch.bfloat16, seed=7)
    o = _attend(dims, q, rows, c, cv, lens, 1)
    cv.check()
    assert B.std_get_device_error() == 0
    _check(o, q, c, lens, 1, torch.bfloat16)


@pytest.mark.parametrize("rows", [1, 3])
def test_a_full_cache(rows):
    """The last tile ends inside the cache's last block."""
    for cap in (16, 112, 144):
        lens = [cap - rows + 1, cap - rows]
        dims, q, c, cv, _ = _attn_inputs(1, 2, 4, 2, 128, rows, lens, 0, torch.bfloat16, seed=8, cap=cap)
        o = _attend(dims, q, rows, c, cv, lens, 0)
        cv.check()
        assert B.std_get_device_error() == 0
        _check(o, q, c, lens, 0, torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hq,rows", [(4, 4), (28, 4)])
def test_nan_in_rows_that_are_not_attended(dtype, Hq, rows):
    """Stale rows (codes and scales of any bits) and the later positions' own rows do not reach a
    query that does not attend them; a query that attends a NaN row gets NaN."""
    lens, off = [200, 63], 1
    dims, q, c, cv, cap = _attn_inputs(1, 2, Hq, 2, 64, rows, lens, off, dtype, seed=9, cap=320)
    for b, n in enumerate(lens):
        for x in "kv":
            c[x + "_scales"][:, b, :, n + off + rows - 1:] = float("nan")
            c[x + "_scales"][:, b, :, n + off + rows:n + off + rows + 3] = float("inf")
            c[x + "_codes"][:, b, :, n + off + rows - 1:] = 0xff
    want = _attend(dims, q, rows, c, cv, lens, off)
    _check(want, q, c, lens, off, dtype)
    for x in "kv":                               # position 2's own row, in keys, then in values
        keep = c[x + "_scales"].clone()
        c[x + "_scales"][:, 0, :, 202] = torch.tensor([0.0, float("nan")], device="cuda", dtype=torch.bfloat16)
        o = _attend(dims, q, rows, c, cv, lens, off)
        cv.check()
        assert torch.equal(o[:, 0, :, :2], want[:, 0, :, :2]) and torch.equal(o[:, 1], want[:, 1])
        assert torch.isnan(o[:, 0, :, 2:]).all()
        c[x + "_scales"].copy_(keep)
    assert B.std_get_device_error() == 0


def test_lengths_out_of_range_are_flagged_and_left():
    lens = [30, 49, -1, 46, 1 << 30]
    dims, q, c, cv, _ = _attn_inputs(2, 5, 4, 2, 64, 3, [30, 46, 0, 46, 0], 0, torch.bfloat16, seed=10, cap=48)
    o = _attend(dims, q, 3, c, cv, lens, 0)
    cv.check()
    assert B.std_get_device_error() == B.STD_DEVERR_LENGTH
    for b in (1, 2, 4):
        assert (o[:, b] == -9).all()
    for b in (0, 3):
        _check(o[:, b:b + 1], q[:, b:b + 1], {x: t[:, b:b + 1] if x != "cap" else t for x, t in c.items()}, [lens[b]], 0,
               torch.bfloat16)
    o = _attend(dims, q, 3, c, cv, [-5] * 5, 0)
    cv.check()
    assert B.std_get_device_error() == B.STD_DEVERR_LENGTH and (o == -9).all()


def test_workspace_too_small_is_refused():
    dims, q, c, cv, _ = _attn_inputs(1, 1, 4, 2, 64, 1, [500], 0, torch.bfloat16)
    need = B.std_kv4_attn_workspace_size(dims, 1, c["cap"])
    assert need > 0
    o = torch.zeros_like(q)
    with pytest.raises(B.StdError) as e:
        B.std_kv4_attn(dims, q, 1, c, _i32([500]), 0, o, torch.empty(need - 4, dtype=torch.uint8, device="cuda"))
    assert e.value.code == B.STD_ERR_WORKSPACE
    with pytest.raises(B.StdError):
        B.std_kv4_attn(dims, q, 1, c, _i32([500]), 0, o, None)


def test_calls_repeat_bit_for_bit_on_streams_and_in_graphs():
    lens = [5000, 1234]
    dims, q, c, cv, _ = _attn_inputs(2, 2, 7, 1, 128, 1, lens, 0, torch.bfloat16, seed=11)
    n = _i32(lens)
    want = _attend(dims, q, 1, c, cv, n, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [_attend(dims, q, 1, c, cv, n, 0, stream=side if i % 2 else None) for i in range(6)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graphs = []
    ws = torch.empty(B.std_kv4_attn_workspace_size(dims, 1, c["cap"]), dtype=torch.uint8, device="cuda")
    for _ in range(2):                           # two graphs that share a workspace, replayed in turn
        o = torch.zeros_like(q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            B.std_kv4_attn(dims, q, 1, c, n, 0, o, ws)
        graphs.append((graph, o))
    for graph, o in graphs * 2:
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for _, o in graphs)
    n.sub_(1000)                                 # the lengths are read at replay
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], _attend(dims, q, 1, c, cv, [4000, 234], 0))
    cv.check()


@pytest.mark.parametrize("dtype,Hq,rows", [(torch.bfloat16, 7, 1), (torch.float32, 4, 1), (torch.bfloat16, 5, 7)])
@pytest.mark.parametrize("power", [-40, 40])
def test_values_of_any_stated_size(dtype, Hq, rows, power):
    """Value rows of one constant (scale 0, where weights may grow largest) beside ordinary ones."""
    n = 1500
    dims, q, c, cv, cap = _attn_inputs(1, 1, Hq, 1, 128, rows, [n], 1, dtype, seed=11)
    g = torch.Generator(device="cuda").manual_seed(12)
    v = torch.randn(1, 1, 1, cap, 128, generator=g, device="cuda")
    v[..., ::2, :] = v[..., ::2, :1]
    v = (v * 2.0 ** power).to(dtype)
    B.std_kv4_quantize(dims, c, v, v, None, None, cap)
    keep = c["v_codes"].clone(), c["v_scales"].clone()
    k = torch.randn(1, 1, 1, cap, 128, generator=g, device="cuda").to(dtype)
    B.std_kv4_quantize(dims, c, k, k, None, None, cap)
    c["v_codes"].copy_(keep[0])
    c["v_scales"].copy_(keep[1])
    o = _attend(dims, q, rows, c, cv, [n], 1)
    cv.check()
    assert B.std_get_device_error() == 0
    _check(o, q, c, [n], 1, dtype)


@pytest.mark.parametrize("dtype,Hq,rows", [(torch.bfloat16, 7, 1), (torch.float32, 4, 1), (torch.bfloat16, 5, 7)])
@pytest.mark.parametrize("power", [-100, 100])
def test_queries_of_any_stated_size(dtype, Hq, rows, power):
    """Tiny queries weigh all keys alike, huge ones take the key of the largest logit."""
    n = 500
    dims, q, c, cv, cap = _attn_inputs(1, 1, Hq, 1, 128, rows, [n], 1, dtype, seed=13)
    q.copy_((torch.sign(q.float()) * 2.0 ** power).to(dtype))
    o = _attend(dims, q, rows, c, cv, [n], 1)
    cv.check()
    assert B.std_get_device_error() == 0
    if power < 0:
        _check(o, q, c, [n], 1, dtype)
        return
    kc, ks, km = _parts(c, "k")
    vc, vs, vm = _parts(c, "v")
    K, V = O.kv4_values(kc, ks, km)[0, 0, 0], O.kv4_values(vc, vs, vm)[0, 0, 0]
    sign = np.sign(q.double().cpu().numpy())[0, 0]
    got = o.double().cpu().numpy()[0, 0]
    for h in range(Hq):
        for i in range(rows):
            x = K[:n + 1 + i] @ sign[h, i]
            top = np.argsort(x)[-2:]
            # fp32 sums of 128 terms: a gap that their rounding cannot close decides the key
            if x[top[1]] - x[top[0]] > 2 * (128 / 8 + 8) * 2.0 ** -22 * (np.abs(K).sum(1).max() + 16 * ks.max() * 128):
                assert np.allclose(got[h, i], V[top[1]], rtol=torch.finfo(dtype).eps, atol=2.0 ** -10 * np.abs(V[top[1]]).max())


def test_many_rows_on_two_streams_and_in_graphs():
    lens = [3000, 777]
    dims, q, c, cv, _ = _attn_inputs(2, 2, 6, 1, 128, 9, lens, 1, torch.bfloat16, seed=14)
    n = _i32(lens)
    want = _attend(dims, q, 9, c, cv, n, 1)
    _check(want, q, c, lens, 1, torch.bfloat16)
    side = [torch.cuda.Stream() for _ in range(2)]
    need = B.std_kv4_attn_workspace_size(dims, 9, c["cap"])
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in side]
    outs = [torch.zeros_like(q) for _ in range(8)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):                 # two calls at once, a workspace each
        B.std_kv4_attn(dims, q, 9, c, n, 1, o, ws[i % 2], side[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    o, graph = torch.zeros_like(q), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.std_kv4_attn(dims, q, 9, c, n, 1, o, ws[0])
        n.sub_(600)                              # what follows a call does not reach into it
        B.std_kv4_attn(dims, q, 9, c, n, 1, outs[0], ws[0])
        n.add_(600)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want)
    assert torch.equal(outs[0], _attend(dims, q, 9, c, cv, [2400, 177], 1))
    cv.check()
    assert B.std_get_device_error() == 0


@pytest.mark.parametrize("nB,Hq,rows", [(1024, 2, 1), (333, 5, 5), (33, 3, 6)])
def test_many_sequences(nB, Hq, rows):
    lens = [(37 * b) % 211 for b in range(nB)]
    dims, q, c, cv, cap = _attn_inputs(1, nB, Hq, 1, 64, rows, lens, 0, torch.bfloat16, seed=15)
    o = _attend(dims, q, rows, c, cv, lens, 0)
    cv.check()
    assert B.std_get_device_error() == 0
    _check(o, q, c, lens, 0, torch.bfloat16)
    bad = list(lens)
    bad[nB - 1], bad[7] = cap + 1, -1            # left as they are, the others as before
    p = _attend(dims, q, rows, c, cv, bad, 0)
    cv.check()
    assert B.std_get_device_error(clear=True) == B.STD_DEVERR_LENGTH
    ok = torch.ones(nB, dtype=torch.bool, device="cuda")
    ok[7] = ok[nB - 1] = False
    assert (p[:, ~ok] == -9).all()
    _check(p[:, ok], q[:, ok], {k: (t[:, ok] if torch.is_tensor(t) else t) for k, t in c.items()},
           [x for b, x in enumerate(lens) if b not in (7, nB - 1)], 0, torch.bfloat16)
