"""The 4-bit cache and the norm/rotation pass without a GPU: the oracle against values worked
out by hand, and the host-side refusals of every entry point."""
import ctypes

import numpy as np
import pytest

from oracle import kv4_oracle as O
from sparse_top_kv_std_b200 import binding as B
from tests.test_abi_cpu import FAKE, no_gpu_only


def test_quantise_by_hand():
    x = np.zeros((1, 64), np.float32)
    x[0, :4] = [-1.0, 14.0, 6.5, 5.5]           # min -1, scale 1: codes 0, 15, 7.5 -> 8, 6.5 -> 6 (ties to even)
    c, s, m = O.kv4_quantize(x)
    assert m[0, 0] == -1 and s[0, 0] == 1
    assert c[0, :5].tolist() == [0, 15, 8, 6, 1]
    assert O.kv4_values(c, s, m)[0, :5].tolist() == [-1, 14, 7, 5, 0]


def test_quantise_constant_and_non_finite_groups():
    x = np.full((3, 64), 2.5, np.float32)
    x[1, 7] = np.nan
    x[2, 7] = np.inf
    c, s, m = O.kv4_quantize(x)
    v = O.kv4_values(c, s, m)
    assert (v[0] == 2.5).all() and np.isnan(v[1]).all() and np.isnan(v[2]).all()


def test_layout_by_hand():
    # d = 64: natural order, low nibble first
    c = np.arange(64, dtype=np.uint8) % 16
    p = O.kv4_pack(c[None])[0]
    assert p[:4].tolist() == [0x10, 0x32, 0x54, 0x76]
    # d = 128: 4-byte words of the two groups alternate
    c = np.concatenate([np.full(64, 1), np.full(64, 2)]).astype(np.uint8)
    p = O.kv4_pack(c[None])[0]
    assert p[:8].tolist() == [0x11] * 4 + [0x22] * 4
    for d in (64, 128):
        c = np.random.default_rng(0).integers(0, 16, (5, d)).astype(np.uint8)
        assert (O.kv4_unpack(O.kv4_pack(c)) == c).all()


def test_rotation_by_hand():
    x = np.array([[[3.0, 4.0, 1.0, 2.0]]])
    pos, f = np.array([[1]]), np.array([np.pi / 2, np.pi])
    assert np.allclose(O.norm_rope(x, None, 0, pos, f, [2], False), [[[-1, -4, 3, -2]]])
    assert np.allclose(O.norm_rope(x, None, 0, pos, f, [2], True), [[[-4, 3, -1, -2]]])
    # two axes: the second pair turns with the second position
    assert np.allclose(O.norm_rope(x, None, 0, np.array([[1], [2]]), f, [1, 1], True), [[[-4, 3, 1, 2]]])
    assert np.allclose(O.norm_rope(x, np.full(4, 2.0), 0, pos * 0, f, [2], True), x * 2 / np.sqrt(7.5))


def test_attention_without_keys_is_zero():
    q = np.ones((1, 2, 2, 2, 4))
    kv = np.ones((1, 2, 1, 3, 4))
    o = O.causal_decode_attn(q, kv, kv, np.array([0, 2]))
    assert (o[0, 0, :, 0] == 0).all() and (o[0, 0, :, 1] == 1).all() and np.allclose(o[0, 1], 1)


# ----------------------------------------------------------------------------- refusals

def _dims(**kw):
    base = dict(L=2, B=1, Hq=28, Hkv=4, d=128, dtype=B.STD_BF16, cap_full=1000, cap_sparse=300)
    base.update(kw)
    return ctypes.byref(B.dims(**base))


def _cache(**kw):
    base = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE, cap=1008)
    base.update(kw)
    return ctypes.byref(B.StdKv4Cache(**base))


def _rope(**kw):
    base = dict(inv_freq=FAKE, rot_dim=128, interleaved=0, n_axes=1, section=(64, 0, 0))
    base.update(kw)
    base["section"] = (ctypes.c_int32 * 3)(*base["section"])
    return ctypes.byref(B.StdRope(**base))


def _call_rope(dims=None, rope=None, **kw):
    a = dict(q=FAKE, qs=4608, k=FAKE, ks=4608, v=FAKE, vs=4608, rows=4, n_rows=None, qw=FAKE, kw=FAKE, eps=1e-6, pos=None,
             qo=FAKE, kc=FAKE, vc=FAKE, cap=1000, len=FAKE, off=0)
    a.update(kw)
    return B.lib().std_qk_norm_rope(_dims() if dims is None else dims, _rope() if rope is None else rope, a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"],
                                    a["rows"], a["n_rows"], a["qw"], a["kw"], a["eps"], a["pos"], a["qo"], a["kc"], a["vc"],
                                    a["cap"], a["len"], a["off"], None)


_INV, _UNS, _CAP, _WS = B.STD_ERR_INVALID_ARG, B.STD_ERR_UNSUPPORTED, B.STD_ERR_CAPACITY, B.STD_ERR_WORKSPACE


@no_gpu_only
@pytest.mark.parametrize("kw,code", [
    (dict(dims=ctypes.POINTER(B.StdDims)()), _INV),
    (dict(dims=_dims(d=96)), _UNS),
    (dict(rope=ctypes.POINTER(B.StdRope)()), _INV),
    (dict(q=None, k=None, v=None), _INV),
    (dict(q=FAKE + 8), _INV),
    (dict(qo=None), _INV),
    (dict(kc=None), _INV),
    (dict(vc=FAKE + 2), _INV),
    (dict(qs=3583), _INV),
    (dict(ks=511), _INV),
    (dict(vs=4609), _INV),
    (dict(qw=FAKE + 4), _INV),
    (dict(eps=-1.0), _INV),
    (dict(eps=float("nan")), _INV),
    (dict(eps=float("inf")), _INV),
    (dict(rows=-1), _INV),
    (dict(off=-1), _INV),
    (dict(len=None), _INV),
    (dict(k=None, v=None, len=None), _INV),                      # positions come from len
    (dict(cap=0), _INV),
    (dict(cap=1 << 31), _INV),
    (dict(rows=1000, off=1), _CAP),
    (dict(rope=_rope(rot_dim=136)), _INV),
    (dict(rope=_rope(rot_dim=-16)), _INV),
    (dict(rope=_rope(rot_dim=72, section=(36, 0, 0))), _UNS),
    (dict(rope=_rope(interleaved=2)), _INV),
    (dict(rope=_rope(inv_freq=None)), _INV),
    (dict(rope=_rope(n_axes=0)), _INV),
    (dict(rope=_rope(n_axes=4), pos=FAKE), _INV),
    (dict(rope=_rope(n_axes=3, section=(32, 16, 16))), _INV),    # axes without positions
    (dict(rope=_rope(n_axes=3, section=(32, 16, 17)), pos=FAKE), _INV),
    (dict(rope=_rope(n_axes=2, section=(80, -16, 0)), pos=FAKE), _INV),
    (dict(pos=FAKE + 2), _INV),
    (dict(n_rows=FAKE + 1), _INV),
    (dict(dims=_dims(L=1 << 15, B=1 << 15)), _INV),
])
def test_norm_rope_refusals(kw, code):
    assert _call_rope(**kw) == code
    assert B.std_last_error() != ""


def _lib():
    return B.lib()


@no_gpu_only
@pytest.mark.parametrize("call,code", [
    (lambda: _lib().std_kv4_append(None, _cache(), FAKE, 0, FAKE, FAKE, 1, None), _INV),
    (lambda: _lib().std_kv4_append(_dims(), None, FAKE, 0, FAKE, FAKE, 1, None), _INV),
    (lambda: _lib().std_kv4_append(_dims(dtype=B.STD_F32, d=96), _cache(), FAKE, 0, FAKE, FAKE, 1, None), _UNS),
    (lambda: _lib().std_kv4_append(_dims(dtype=B.STD_F32, d=32), _cache(), FAKE, 0, FAKE, FAKE, 1, None), _UNS),
    (lambda: _lib().std_kv4_append(_dims(), _cache(cap=1000), FAKE, 0, FAKE, FAKE, 1, None), _INV),
    (lambda: _lib().std_kv4_append(_dims(), _cache(cap=0), FAKE, 0, FAKE, FAKE, 1, None), _INV),
    (lambda: _lib().std_kv4_append(_dims(), _cache(cap=1 << 31), FAKE, 0, FAKE, FAKE, 1, None), _INV),
    (lambda: _lib().std_kv4_append(_dims(), _cache(k_codes=FAKE + 8), FAKE, 0, FAKE, FAKE, 1, None), _INV),
    (lambda: _lib().std_kv4_append(_dims(), _cache(v_scales=None), FAKE, 0, FAKE, FAKE, 1, None), _INV),
    (lambda: _lib().std_kv4_append(_dims(), _cache(), None, 0, FAKE, FAKE, 1, None), _INV),
    (lambda: _lib().std_kv4_append(_dims(), _cache(), FAKE, -1, FAKE, FAKE, 1, None), _INV),
    (lambda: _lib().std_kv4_append(_dims(), _cache(), FAKE, 0, None, FAKE, 1, None), _INV),
    (lambda: _lib().std_kv4_append(_dims(), _cache(), FAKE, 0, FAKE, FAKE, -1, None), _INV),
    (lambda: _lib().std_kv4_append(_dims(), _cache(), FAKE, 1000, FAKE, FAKE, 9, None), _CAP),
    (lambda: _lib().std_kv4_quantize(_dims(), _cache(), FAKE, FAKE + 8, None, None, 10, None), _INV),
    (lambda: _lib().std_kv4_quantize(_dims(), _cache(), FAKE, FAKE, FAKE + 2, None, 10, None), _INV),
    (lambda: _lib().std_kv4_quantize(_dims(), _cache(), FAKE, FAKE, None, FAKE + 2, 10, None), _INV),
    (lambda: _lib().std_kv4_quantize(_dims(), _cache(), FAKE, FAKE, None, None, 1001, None), _CAP),
    (lambda: _lib().std_kv4_quantize(_dims(), _cache(cap=96), FAKE, FAKE, None, None, 97, None), _CAP),
    (lambda: _lib().std_kv4_quantize(_dims(L=1 << 12, B=1 << 12), _cache(), FAKE, FAKE, None, FAKE, 1000, None), _INV),
    (lambda: _lib().std_kv4_read(_dims(), _cache(), None, None, 10, None, FAKE, None), _INV),
    (lambda: _lib().std_kv4_read(_dims(), _cache(), None, None, 1009, FAKE, FAKE, None), _CAP),
    (lambda: _lib().std_kv4_read(_dims(), _cache(), None, None, -1, FAKE, FAKE, None), _INV),
    (lambda: _lib().std_kv4_attn(_dims(), None, 1, _cache(), FAKE, 0, FAKE, FAKE, 1 << 30, None), _INV),
    (lambda: _lib().std_kv4_attn(_dims(), FAKE, 0, _cache(), FAKE, 0, FAKE, FAKE, 1 << 30, None), _INV),
    (lambda: _lib().std_kv4_attn(_dims(), FAKE, 33, _cache(), FAKE, 0, FAKE, FAKE, 1 << 30, None), _INV),
    (lambda: _lib().std_kv4_attn(_dims(), FAKE, 19, _cache(), FAKE, 0, FAKE, FAKE, 1 << 30, None), _UNS),
    (lambda: _lib().std_kv4_attn(_dims(B=1025), FAKE, 1, _cache(), FAKE, 0, FAKE, FAKE, 1 << 30, None), _UNS),
    (lambda: _lib().std_kv4_attn(_dims(), FAKE, 1, _cache(), FAKE, -1, FAKE, FAKE, 1 << 30, None), _INV),
    (lambda: _lib().std_kv4_attn(_dims(), FAKE, 1, _cache(), None, 0, FAKE, FAKE, 1 << 30, None), _INV),
    (lambda: _lib().std_kv4_attn(_dims(), FAKE, 1, _cache(), FAKE, 0, FAKE + 4, FAKE, 1 << 30, None), _INV),
    (lambda: _lib().std_kv4_attn(_dims(L=1 << 14, B=1024), FAKE, 1, _cache(), FAKE, 0, FAKE, FAKE, 1 << 30, None), _UNS),
])
def test_kv4_refusals(call, code):
    assert call() == code
    assert B.std_last_error() != ""


def test_workspace_of_invalid_arguments_is_zero():
    for d, rows, cap in ((B.dims(1, 1, 4, 2, 96, B.STD_F32, 64, 1), 1, 64), (B.dims(1, 1, 4, 2, 64, B.STD_F32, 64, 1), 0, 64),
                         (B.dims(1, 1, 4, 2, 64, B.STD_F32, 64, 1), 1, 60)):
        assert B.std_kv4_attn_workspace_size(d, rows, cap) == 0


def test_binding_refuses_uneven_token_views():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        B._tokens(torch.zeros(1, 2, 3, 4, 64), 1, 2, 4, 64, 0)   # not on the GPU
    for view in (torch.zeros(1, 2, 3, 4, 64), torch.zeros(1, 2, 3, 6, 64)[:, :, :, 1:5], torch.zeros(1, 2, 1, 9, 64)[:, :, :, :4]):
        assert B._tokens(view, 1, 2, 4, 64, -1)[1] == view.stride(2) or view.shape[2] == 1
    for view in (torch.zeros(1, 2, 5, 4, 64)[:, :, :3], torch.zeros(1, 2, 3, 4, 128)[..., :64], torch.zeros(1, 2, 3, 64, 4).mT,
                 torch.zeros(1, 2, 4, 3, 64).transpose(2, 3), torch.zeros(2, 3, 4, 64), torch.zeros(1, 2, 3, 5, 64)):
        with pytest.raises(ValueError):
            B._tokens(view, 1, 2, 4, 64, -1)
    with pytest.raises(ValueError):
        B.std_rope(torch.zeros(32), sections=[32])               # not float64


@no_gpu_only
def test_row_counts_that_pass_31_bits_are_refused():
    one = dict(dims=_dims(L=1, B=1, Hq=4, Hkv=1), k=None, v=None, pos=FAKE)
    for n in (2**31 - 1, 2**31 - 100):
        assert _call_rope(rows=n, **one) == _INV
        for begin in (None, FAKE):
            assert _lib().std_kv4_quantize(_dims(L=1, Hkv=1, Hq=4), _cache(), FAKE, FAKE, begin, FAKE, n, None) == _INV
            assert _lib().std_kv4_read(_dims(L=1, Hkv=1, Hq=4), _cache(), begin, FAKE, n, FAKE, FAKE, None) == _INV
    assert _call_rope(rows=2**28, dims=_dims(L=4, B=4, Hq=4, Hkv=1), k=None, v=None, pos=FAKE) == _INV


def test_binding_checks_rows_devices_and_takes_addresses(monkeypatch):
    torch = pytest.importorskip("torch")
    calls = []
    fake = type("Lib", (), {"std_qk_norm_rope": lambda self, *a: calls.append(a) or 0})()
    monkeypatch.setattr(B, "lib", lambda: fake)
    monkeypatch.setattr(B, "_current_device", lambda: -1)        # what a CPU tensor's get_device() gives
    monkeypatch.setattr(B, "_stream", lambda s: None)
    monkeypatch.setattr(B, "_ptr", lambda x: None if x is None else x.data_ptr())
    d, out = B.dims(1, 2, 4, 2, 64, B.STD_F32, 8, 1), torch.zeros(1)

    def call(q, rows, rope, pos=None):
        B.std_qk_norm_rope(d, rope, q, None, None, rows, None, None, None, 1e-6, pos, out, None, None, 8, None)

    rope = B.std_rope(torch.zeros(32, dtype=torch.float64))
    call(torch.zeros(1, 2, 3, 4, 64), 3, rope)
    for rows in (2, 4):                                          # not the rows that the tensor has
        with pytest.raises(ValueError):
            call(torch.zeros(1, 2, 3, 4, 64), rows, rope)
    call(torch.zeros(1, 2, 0, 4, 64), 0, rope)                   # no rows of several sequences
    call(torch.zeros(1, 2, 3, 4, 64), 3, rope, pos=4096)         # an address, as in the other calls
    assert len(calls) == 3 and calls[2][13] == 4096
    other = B.std_rope(torch.zeros(32, dtype=torch.float64))
    other.device = 1                                             # frequencies on another GPU
    with pytest.raises(ValueError):
        call(torch.zeros(1, 2, 3, 4, 64), 3, other)
