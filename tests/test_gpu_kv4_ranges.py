"""Decode attention over the 4-bit cache where query rows, value groups and logits differ much in size:
each row and each group keeps the accuracy that it has alone.

Tolerances.  Of a row r and a key j, in float32: a logit is the sum of d / 16 tensor-core steps (twice that
for fp32 queries), each off by at most 2^-22 of the sum of the magnitudes so far, and a few operations,
    dx_r <= (d / 8 + 8) 2^-22 A_r + 2^-36 max |q_r| max_j sum_c 15 sk / sqrt d
    A_r = max_j sum_c |q_rc| (sk max(a, |a - 8|) + |mk| + |mk + 8 sk|) / sqrt d
(the second term: a query's entry keeps what is above 2^-36 of the row's largest).  A weight is off by
dx + 2^-20 + X 2^-23, X the row's largest logit in log2 units, and, where it enters the tensor cores, by
r = 2^-11 (bf16 queries, 11 bits in weight and sum) or 2^-21 (fp32) of itself and by 2^-32 of the row's
largest p sv of that group.  Sums over n keys run in at most n / 16 steps of a warp:
    do_rc <= (2 (e^(dx + 2^-20 + X 2^-23) - 1) + r + (n / 16 + 16) 2^-22) V_rc + n 2^-32 15 max_j p sv / sum p
    V_rc = sum_j p (15 sv + |mv + 8 sv|) / sum p     (over the row's keys, c's group)
and the output is rounded to its type (finfo.eps / 2)."""
import numpy as np
import pytest
import torch

from oracle import kv4_oracle as O
from sparse_top_kv_std_b200 import binding as B
from tests import harness as H

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float32]
# (Hq of one KV head, rows): 8 query rows, 16, blocks of 16 or of 64, two blocks of 64
HEADS = [(7, 1), (5, 3), (7, 7), (4, 20)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    B.lib()
    B.std_get_device_error(clear=True)


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def _attend(q, k, v, rows, lens, dtype):
    """o of the 4-bit copies of k and v [L][B][Hkv][cap][d], all rows written, and that cache."""
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    L, nB, Hkv, cap, d = k.shape
    cv = H.Canaries()
    c = {"cap": cap}
    for x in "kv":
        c[x + "_codes"] = cv.tensor((L, nB, Hkv, cap, d // 2), torch.uint8, fill=0x5a)
        c[x + "_scales"] = cv.tensor((L, nB, Hkv, cap, d // 64, 2), torch.bfloat16, fill=float("nan"))
    dims = B.dims(L, nB, q.shape[2], Hkv, d, B.STD_F32 if dtype == torch.float32 else B.STD_BF16, cap, 1)
    B.std_kv4_quantize(dims, c, k, v, None, None, cap)
    o = cv.tensor(tuple(q.shape), dtype, fill=-9)
    ws = cv.tensor((max(16, B.std_kv4_attn_workspace_size(dims, rows, cap)),), torch.uint8, fill=0xff)
    B.std_kv4_attn(dims, q, rows, c, torch.tensor(lens, dtype=torch.int32, device="cuda"), 1, o, ws)
    cv.check()
    assert B.std_get_device_error() == 0
    return o.double().cpu().numpy(), q.double().cpu().numpy(), c


def _units(q, c, lens):
    """For every (layer, sequence, KV head): its place in q, the queries [R][d], each row's number of keys, and
    codes, scales and minima of K and V as float64 [n][d]."""
    parts = []
    for x in "kv":
        sc = c[x + "_scales"].double().cpu().numpy()
        wide = lambda t: np.repeat(t, 64, -1)  # noqa: E731
        parts.append((O.kv4_unpack(c[x + "_codes"].cpu().numpy()).astype(np.float64), wide(sc[..., 0]), wide(sc[..., 1])))
    L, nB, Hq, rows, d = q.shape
    Hkv = parts[0][0].shape[2]
    G = Hq // Hkv
    for l in range(L):
        for b in range(nB):
            for h in range(Hkv):
                at = (l, b, slice(h * G, (h + 1) * G))
                keys = np.tile(lens[b] + 1 + np.arange(rows), G)
                n = int(keys.max())
                yield at, q[at].reshape(G * rows, d), keys, [t[l, b, h, :n] for t in parts[0]], [t[l, b, h, :n] for t in parts[1]]


def _logits(Q, keys, K):
    """Logits [R][n] (-inf where not attended), and dx [R]."""
    code, s, m = K
    d = Q.shape[1]
    x = Q @ (m + code * s).T / np.sqrt(d)
    seen = np.arange(x.shape[1])[None] < keys[:, None]
    size = np.abs(Q) @ (s * np.maximum(code, np.abs(code - 8)) + np.abs(m) + np.abs(m + 8 * s)).T / np.sqrt(d)
    A = np.where(seen, size, 0).max(1)
    dx = (d / 8 + 8) * 2.0 ** -22 * A + 2.0 ** -36 * np.abs(Q).max(1) * (15 * s).sum(1).max() / np.sqrt(d)
    return np.where(seen, x, -np.inf), dx


def _r(dtype):
    return 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -21


def _check(o, q, c, lens, dtype, skip=None):
    """Every output against the oracle's, but those of the rows `skip` [rows of a KV head]."""
    worst = 0.0
    for at, Q, keys, K, V in _units(q, c, lens):
        x, dx = _logits(Q, keys, K)
        n = x.shape[1]
        keep = np.ones(len(Q), bool) if skip is None else ~skip
        x, dx = x[keep], dx[keep]
        p = np.exp(x - x.max(1, keepdims=True))
        total = p.sum(1, keepdims=True)
        code, s, m = V
        want = p @ (m + code * s) / total
        size = p @ (15 * s + np.abs(m + 8 * s)) / total
        X = np.where(np.isfinite(x), np.abs(x), 0).max(1) * 1.4427
        rel = 2 * np.expm1(dx + 2.0 ** -20 + X * 2.0 ** -23) + _r(dtype) + (n / 16 + 16) * 2.0 ** -22
        floor = n * 2.0 ** -32 * 15 * np.stack([(p * s[:, g]).max(1) for g in range(s.shape[1])], 1) / total
        tol = rel[:, None] * size + floor + torch.finfo(dtype).eps / 2 * np.abs(want)
        err = np.abs(o[at].reshape(len(Q), -1)[keep] - want)
        assert (err <= tol).all(), (at, float((err / np.maximum(tol, 1e-300)).max()), float(np.nanmax(err)))
        worst = max(worst, float((err / np.maximum(tol, 1e-300)).max()))
    return worst


def _check_largest_logit(o, q, c, lens, dtype, rows=None):
    """Queries so large that float32 logits are far apart: where the largest is further from the next than
    their rounding, the output is that key's values; everywhere it lies among the keys' values."""
    decided = 0
    for at, Q, keys, K, V in _units(q, c, lens):
        x, dx = _logits(Q, keys, K)
        code, s, m = V
        v = m + code * s
        top = np.abs(v).max()
        # weights are rounded, their sum is not: r of the size, and the sums' own rounding
        slack = (_r(dtype) + 2.0 ** -18 + torch.finfo(dtype).eps) * (15 * s + np.abs(m + 8 * s)).max()
        got = o[at].reshape(len(Q), -1)
        for r in range(len(Q)) if rows is None else np.flatnonzero(rows):
            y = v[:keys[r]]
            assert (got[r] >= y.min(0) - slack).all() and (got[r] <= y.max(0) + slack).all(), (at, r, got[r][:4], top)
            a, b = np.argsort(x[r, :keys[r]])[-2:]
            if x[r, b] - x[r, a] > 2 * dx[r] + 60:
                decided += 1
                assert (np.abs(got[r] - v[b]) <= slack).all(), (at, r)
    return decided


# ----------------------------------------------------------------------------- query rows

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,rows", HEADS)
@pytest.mark.parametrize("power", [20, 28, 40, 60])
def test_a_large_query_row_leaves_the_others_alone(dtype, d, G, rows, power):
    """One row of every block of 8 is 2^power times the others, as a row of a padded batch that was never
    written may be: the others' logits keep their bits."""
    lens = [700, 19]
    q = _randn(1, 1, 2, 2 * G, rows, d)
    large = np.arange(G * rows) % 8 == 5
    q.view(2, 2, G * rows, d)[:, :, torch.from_numpy(large).cuda()] *= 2.0 ** power
    o, q, c = _attend(q, _randn(2, 1, 2, 2, 736, d), _randn(3, 1, 2, 2, 736, d), rows, lens, dtype)
    _check(o, q, c, lens, dtype, skip=large)
    assert np.isfinite(o).all()
    if power >= 40:
        assert _check_largest_logit(o, q, c, lens, dtype, rows=large) > 0


@pytest.mark.parametrize("G,rows", HEADS)
def test_rows_of_any_bits_behind_the_valid_ones(G, rows):
    """Query rows that hold anything (the rows behind a short sequence's last) do not reach the others."""
    lens = [500]
    q = _randn(4, 1, 1, G, rows, 128).bfloat16()
    junk = np.arange(G * rows) % 3 == 1
    g = torch.Generator(device="cuda").manual_seed(5)
    bits = torch.randint(-2 ** 15, 2 ** 15, (int(junk.sum()), 128), generator=g, device="cuda").to(torch.int16)
    q.view(G * rows, 128)[torch.from_numpy(junk).cuda()] = bits.view(torch.bfloat16)
    o, q, c = _attend(q, _randn(6, 1, 1, 1, 528, 128), _randn(7, 1, 1, 1, 528, 128), rows, lens, torch.bfloat16)
    _check(o, np.where(np.isfinite(q), q, 0), c, lens, torch.bfloat16, skip=junk)


# ----------------------------------------------------------------------------- sums of weights and minima

def _steps(q_sign, cap, d, height):
    """Keys along q_sign [d] whose logits (for queries q_sign) rise by `height` in log2 units with every tile of 128
    keys, five tiles long, then start again."""
    level = (torch.arange(cap, device="cuda") // 128 % 5).float() * height * np.log(2) / np.sqrt(d)
    return q_sign * level[:, None]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,rows", HEADS[:3])
@pytest.mark.parametrize("power", [20, 36, 40])
def test_constant_values_with_rising_logits(dtype, d, G, rows, power):
    """Value rows of one constant have scale 0, so that no weight times scale ever grows: the sum of weights
    times minima has to stay finite by itself."""
    L, Hkv, n = 6, 8, 2000
    sign = torch.sign(_randn(8, d))
    k = _steps(sign, n + 16 + rows // 16 * 16, d, 45).expand(L, 1, Hkv, -1, d)
    cap = k.shape[3]
    v = (2.0 ** power * (1 + torch.arange(cap, device="cuda") % 7 / 8.)).view(1, 1, 1, cap, 1).expand(L, 1, Hkv, cap, d)
    q = sign.expand(L, 1, G * Hkv, rows, d)
    o, q, c = _attend(q.contiguous(), k.contiguous(), v.contiguous(), rows, [n], dtype)
    _check(o, q, c, [n], dtype)


# ----------------------------------------------------------------------------- groups of values

def _groups(kind, L, nB, Hkv, cap, d, seed):
    """Values and the powers of two of their groups, [..., cap][d / 64]."""
    v = _randn(seed, L, nB, Hkv, cap, d)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    e = torch.zeros(L, nB, Hkv, cap, d // 64, device="cuda")
    if kind == "keys":        # every key and group of a size of its own
        e = torch.randint(-30, 31, e.shape, generator=g, device="cuda").float()
    elif kind == "steps":     # sizes rise and fall with the tiles, in opposite directions
        t = torch.arange(cap, device="cuda") // 128
        e[..., 0] = 12.0 * (t * 3 % 5 - 2)
        e[..., -1] -= 9.0 * (t * 2 % 7 - 3)
    elif kind == "tiny":
        e -= 80
    elif kind == "large":
        e += 37
    else:                     # the second group 2^kind of the first
        e[..., 1] = kind
    return (v.view(*e.shape, 64) * torch.exp2(e)[..., None]).view(v.shape)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("G,rows", HEADS)
@pytest.mark.parametrize("kind", [-12, -16, -24, -40, 24, "keys", "tiny", "large"])
def test_value_groups_of_different_sizes(dtype, G, rows, kind):
    lens = [1100, 77]
    q = _randn(9, 1, 2, 2 * G, rows, 128)
    k, v = _randn(10, 1, 2, 2, 1136, 128), _groups(kind, 1, 2, 2, 1136, 128, 11)
    o, q, c = _attend(q, k, v, rows, lens, dtype)
    _check(o, q, c, lens, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,rows", HEADS[:3])
@pytest.mark.parametrize("height", [0, 7, 45])
def test_sizes_and_logits_that_move_from_tile_to_tile(dtype, d, G, rows, height):
    """Several tiles a CTA: references and the groups' factors move, up and down, while sums are under way."""
    L, Hkv, n = 6, 8, 2000
    sign = torch.sign(_randn(12, d))
    cap = n + 16 + rows // 16 * 16
    k = _steps(sign, cap, d, height) + 0.3 * _randn(13, L, 1, Hkv, cap, d)
    q = sign + 0.3 * _randn(14, L, 1, G * Hkv, rows, d)
    v = _groups("steps", L, 1, Hkv, cap, d, 15)
    o, q, c = _attend(q, k, v, rows, [n], dtype)
    _check(o, q, c, [n], dtype)


@pytest.mark.parametrize("d,G,rows", [(128, 1, 1), (128, 5, 3)])
@pytest.mark.parametrize("kind", [-12, -16, -24])
def test_fp32_accuracy_in_both_groups(d, G, rows, kind):
    """Diffuse attention, the result a small difference of large sums: a fp32 accumulator of centred codes is off by
    sqrt(n / 128) 2^-23 of the result, 5e-7 here, the logits' own rounding (2^-22 of some 30 in each) as much
    as four times that, at random: 8e-6 in norm, in either group."""
    n = 2112
    q, k = _randn(16, 1, 1, G, rows, d), _randn(17, 1, 1, 1, n + 16, d)
    o, q, c = _attend(q, k, _groups(kind, 1, 1, 1, n + 16, d, 18), rows, [n], torch.float32)
    for at, Q, keys, K, V in _units(q, c, [n]):
        x, _ = _logits(Q, keys, K)
        p = np.exp(x - x.max(1, keepdims=True))
        want = p @ (V[2] + V[0] * V[1]) / p.sum(1, keepdims=True)
        got = o[at].reshape(want.shape)
        for g in (slice(0, 64), slice(64, 128)):
            assert np.linalg.norm((got - want)[:, g]) <= 8e-6 * np.linalg.norm(want[:, g])


# ----------------------------------------------------------------------------- large logits

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,rows", HEADS)
@pytest.mark.parametrize("power", [24, 40, 100])
@pytest.mark.parametrize("value_power", [0, 39])
def test_logits_whose_rounding_exceeds_the_exponents(dtype, d, G, rows, power, value_power):
    """Logits far above 2^24, where one unit in the last place is many powers of two: the weights and the reference
    that they are relative to round alike, so the largest logit's weight is finite and not zero."""
    lens = [900, 40]
    q = _randn(19, 1, 2, 2 * G, rows, d) * 2.0 ** power
    k, v = _randn(20, 1, 2, 2, 944, d), _randn(21, 1, 2, 2, 944, d) * 2.0 ** value_power
    o, q, c = _attend(q, k, v, rows, lens, dtype)
    assert np.isfinite(o).all()
    assert _check_largest_logit(o, q, c, lens, dtype) > 0
