"""std_qk_norm_rope against the fp64 oracle.

Tolerance: the result is rounded once to its type (half a step, finfo.eps / 2 of its value).  Before
that, in float32: a sum of up to 128 squares in 8 + 4 additions and four products or quotients
(relative error below 2^-20), an angle reduced in 64 bits and rounded to 32 (2^-23 rad), sine and
cosine within two units, and a rotation of two products: together below 2^-19 of the pair's length,
which is at most sqrt(2) of the row's largest value."""
import numpy as np
import pytest
import torch

from oracle import kv4_oracle as O
from sparse_top_kv_std_b200 import binding as B
from tests import harness as H

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    B.lib()
    B.std_get_device_error(clear=True)


def _f64(t):
    return t.double().cpu().numpy()


def _close(got, want, dtype):
    got = _f64(got)
    want = np.asarray(want)
    top = np.abs(want).max(-1, keepdims=True)
    tol = torch.finfo(dtype).eps / 2 * np.abs(want) + 2.0 ** -19 * 1.5 * top + 1e-30
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) - tol).max())


def _make(L, nB, rows, Hq, Hkv, d, dtype, lens, rot, axes, seed, fused=True, norm=True, ragged=None, cap=None, off=0,
          pos=None, interleaved=False, base=10000.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (3 * rn(L, nB, rows, Hq + 2 * Hkv, d)).to(dtype)
    q, k, v = x.split([Hq, Hkv, Hkv], 3)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    half = rot // 2
    f = base ** (-torch.arange(half, dtype=torch.float64, device="cuda") / max(half, 1))
    sections = [half] if axes == 1 else [half - 2 * (half // 3), half // 3, half // 3][:axes]
    if axes == 2:
        sections = [half - half // 3, half // 3]
    if pos is None and axes > 1:
        pos = torch.randint(0, 200000, (axes, nB, rows), generator=g, device="cuda", dtype=torch.int32)
    return dict(L=L, B=nB, rows=rows, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, q=q, k=k, v=v, f=f, sections=sections,
                interleaved=interleaved, pos=pos, off=off, lens=lens,
                len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                n=ragged, n_rows=None if ragged is None else torch.tensor(ragged, dtype=torch.int32, device="cuda"),
                qw=(1 + 0.3 * rn(L, d)).to(dtype) if norm else None, kw=(1 + 0.3 * rn(L, d)).to(dtype) if norm else None,
                cap=cap or max(lens) + off + rows + 3)


def _run(c, cv=None, parts="qkv", stream=None):
    cv = cv or H.Canaries()
    code = B.STD_F32 if c["dtype"] == torch.float32 else B.STD_BF16
    dims = B.dims(c["L"], c["B"], c["Hq"], c["Hkv"], c["d"], code, c["cap"], 1)
    q_out = cv.tensor((c["L"], c["B"], c["Hq"], c["rows"], c["d"]), c["dtype"], fill=-7)
    kc = cv.tensor((c["L"], c["B"], c["Hkv"], c["cap"], c["d"]), c["dtype"], fill=-7)
    vc = cv.tensor((c["L"], c["B"], c["Hkv"], c["cap"], c["d"]), c["dtype"], fill=-7)
    rope = B.std_rope(c["f"] if len(c["f"]) else None, sections=c["sections"], interleaved=c["interleaved"])
    pick = lambda p, x: x if p in parts else None  # noqa: E731
    B.std_qk_norm_rope(dims, rope, pick("q", c["q"]), pick("k", c["k"]), pick("v", c["v"]), c["rows"], c["n_rows"], c["qw"],
                       c["kw"], 1e-6, c["pos"], pick("q", q_out), pick("k", kc), pick("v", vc), c["cap"], c["len"], c["off"],
                       stream)
    return q_out, kc, vc, cv


def _check(c, q_out, kc, vc, skipped=()):
    for b in range(c["B"]):
        n = c["rows"] if c["n"] is None else c["n"][b]
        if b in skipped:
            n = 0
        at = c["lens"][b] + c["off"]
        if c["pos"] is None:
            pos = at + np.arange(n)[None]
        else:
            pos = c["pos"][:, b, :n].cpu().numpy()
        for l in range(c["L"]):
            args = (1e-6, pos, c["f"].cpu().numpy(), c["sections"], c["interleaved"])
            w = lambda t: None if t is None else _f64(t[l])  # noqa: E731
            if n:
                _close(q_out[l, b, :, :n], O.norm_rope(_f64(c["q"][l, b, :n]), w(c["qw"]), *args).swapaxes(0, 1), c["dtype"])
                _close(kc[l, b, :, at:at + n], O.norm_rope(_f64(c["k"][l, b, :n]), w(c["kw"]), *args).swapaxes(0, 1),
                       c["dtype"])
                assert torch.equal(vc[l, b, :, at:at + n], c["v"][l, b, :n].transpose(0, 1))
            assert (q_out[l, b, :, n:] == -7).all()
            for t in (kc, vc):  # the cache's other rows are as they were
                assert (t[l, b, :, :at] == -7).all() and (t[l, b, :, at + n:] == -7).all()


@pytest.mark.parametrize("d,dtype", [(64, torch.bfloat16), (128, torch.bfloat16), (32, torch.float32), (64, torch.float32),
                                     (96, torch.float32), (128, torch.float32)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,part", [(1, 1), (5, 2), (37, 8)])
def test_types_heads_and_partial_rotation(d, dtype, interleaved, rows, part):
    rot = d // part if (d // part) % (d // 8) == 0 else d // 2
    c = _make(2, 2, rows, 6, 2, d, dtype, [0, 143000], rot, 1, 1, interleaved=interleaved, off=2)
    q, k, v, cv = _run(c)
    cv.check()
    assert B.std_get_device_error() == 0
    _check(c, q, k, v)


@pytest.mark.parametrize("axes", [1, 2, 3])
@pytest.mark.parametrize("fused", [False, True])
def test_position_axes_and_strides(axes, fused):
    c = _make(1, 3, 20, 28, 4, 128, torch.bfloat16, [7, 0, 300], 128, axes, 2, fused=fused,
              pos=None if axes > 1 else torch.randint(-50, 1 << 24, (1, 3, 20), device="cuda", dtype=torch.int32))
    q, k, v, cv = _run(c)
    cv.check()
    _check(c, q, k, v)


def test_no_norm_no_rotation_and_parts():
    c = _make(1, 1, 9, 8, 8, 64, torch.float32, [3], 0, 1, 3, norm=False)
    q, k, v, cv = _run(c)
    cv.check()
    assert torch.equal(q[0, 0], c["q"][0, 0].transpose(0, 1))   # nothing to compute: a transposed copy
    assert torch.equal(k[0, 0, :, 3:12], c["k"][0, 0].transpose(0, 1))
    c = _make(1, 1, 9, 8, 2, 128, torch.bfloat16, [3], 128, 1, 4)
    whole = _run(c)
    for part, i in (("q", 0), ("k", 1), ("v", 2), ("kv", 1)):
        some = _run(c, parts=part)
        some[3].check()
        assert torch.equal(some[i], whole[i])
        for j, name in enumerate("qkv"):
            if name not in part:
                assert (some[j] == -7).all()


def test_many_tokens_take_the_wide_grid_and_agree_with_few():
    """The grid for many tokens (eight a CTA) gives the bits of the grid for few."""
    c = _make(1, 1, 1003, 14, 2, 128, torch.bfloat16, [50], 128, 1, 5)
    q, k, v, cv = _run(c)
    cv.check()
    _check(c, q, k, v)
    one = _make(1, 1, 1003, 14, 2, 128, torch.bfloat16, [50], 128, 1, 5)
    for r in (0, 7, 8, 1002):
        s = dict(one, rows=1, q=c["q"][:, :, r:r + 1].contiguous(), k=c["k"][:, :, r:r + 1].contiguous(),
                 v=c["v"][:, :, r:r + 1].contiguous(), off=r)
        q1, k1, _, _ = _run(s)
        assert torch.equal(q1[:, :, :, 0], q[:, :, :, r]) and torch.equal(k1[:, :, :, 50 + r], k[:, :, :, 50 + r])


@pytest.mark.parametrize("rows", [9, 700])
def test_ragged_batch_leaves_padding_alone(rows):
    n = [rows, 0, rows // 2, 1]
    c = _make(2, 4, rows, 4, 2, 64, torch.bfloat16, [0, 5, 9, 100], 64, 1, 6, ragged=n)
    c["q"][:, 2, n[2]:] = float("nan")
    q, k, v, cv = _run(c)
    cv.check()
    assert B.std_get_device_error() == 0
    _check(c, q, k, v)


def test_device_side_refusals():
    c = _make(1, 3, 8, 4, 2, 64, torch.bfloat16, [0, 20, 3], 64, 1, 7, cap=24)
    q, k, v, cv = _run(c)                       # sequence 1 would pass the capacity
    cv.check()
    assert B.std_get_device_error() == B.STD_DEVERR_CAPACITY
    _check(c, q, k, v, skipped=(1,))
    c = _make(1, 3, 8, 4, 2, 64, torch.bfloat16, [0, 20, 3], 64, 1, 7, cap=40, ragged=[8, 9, -1])
    q, k, v, cv = _run(c)
    cv.check()
    assert B.std_get_device_error() == B.STD_DEVERR_LENGTH
    _check(c, q, k, v, skipped=(1, 2))


def test_zeros_infinities_and_nan_stay_in_their_head():
    c = _make(1, 1, 4, 4, 2, 64, torch.float32, [0], 64, 1, 8, fused=False)
    c["q"][0, 0, 0, 1] = 0
    c["q"][0, 0, 1, 2, 5] = float("inf")
    c["k"][0, 0, 2, 0, 9] = float("nan")
    q, k, v, cv = _run(c)
    cv.check()
    assert (q[0, 0, 1, 0] == 0).all()
    assert not torch.isfinite(q[0, 0, 2, 1]).all() and not torch.isfinite(k[0, 0, 0, 2]).any()
    ok = torch.ones_like(q, dtype=torch.bool)
    ok[0, 0, 2, 1] = False
    assert torch.isfinite(q[ok]).all() and torch.isfinite(k[0, 0, 1, :4]).all()


def test_no_rows_and_another_stream_and_a_graph():
    c = _make(1, 1, 6, 4, 2, 64, torch.bfloat16, [4], 64, 1, 9)
    want = _run(c)
    none = _make(1, 1, 0, 4, 2, 64, torch.bfloat16, [4], 64, 1, 9)
    q, k, v, cv = _run(none)
    cv.check()
    assert (k == -7).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _run(c, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
    graph = torch.cuda.CUDAGraph()
    cv = H.Canaries()
    with torch.cuda.graph(graph):
        got = _run(c, cv)
    c["q"].neg_()
    c["len"].add_(1)                            # the replay reads inputs and lengths anew
    graph.replay()
    again = _run(c)
    torch.cuda.synchronize()
    assert torch.equal(got[0], again[0]) and torch.equal(got[1][:, :, :, 5:11], again[1][:, :, :, 5:11])


@pytest.mark.parametrize("nB,rows,d,dtype", [(300, 1, 128, torch.bfloat16), (700, 3, 64, torch.bfloat16), (130, 5, 32, torch.float32)])
def test_tokens_of_many_sequences_share_a_cta(nB, rows, d, dtype):
    ragged = [(7 * b) % (rows + 1) for b in range(nB)]
    lens = [(5 * b) % 11 for b in range(nB)]
    ragged[3], lens[5] = -1, 1000                # one refused for its rows, one for the capacity, among others
    c = _make(2, nB, rows, 6, 2, d, dtype, [min(x, 11) for x in lens], d, 3, 10, ragged=ragged, cap=11 + rows)
    c["lens"] = lens
    c["len"].copy_(torch.tensor(lens, dtype=torch.int32))
    q, k, v, cv = _run(c)
    cv.check()
    assert B.std_get_device_error(clear=True) == B.STD_DEVERR_CAPACITY | B.STD_DEVERR_LENGTH
    for b in (3, 5):
        assert (q[:, b] == -7).all() and (k[:, b] == -7).all() and (v[:, b] == -7).all()
    lens[5], c["n"][3], c["n"][5] = 0, 0, 0
    _check(c, q, k, v)
