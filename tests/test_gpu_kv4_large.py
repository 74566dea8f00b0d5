"""Caches whose offsets pass 32 bits: the last layers of one call over all of them against a call of their own."""
import pytest
import torch

from sparse_top_kv_std_b200 import binding as B
from sparse_top_kv_std_b200.kv4 import Kv4Cache

pytestmark = pytest.mark.gpu

L, HKV, D = 80, 8, 128


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    if torch.cuda.get_device_properties(0).total_memory < 120 << 30:
        pytest.skip("needs 60 GB")
    B.lib()
    B.std_get_device_error(clear=True)
    yield
    torch.cuda.empty_cache()


def _dims(layers, cap, Hq=HKV, dtype=B.STD_BF16):
    return B.dims(layers, 1, Hq, HKV, D, dtype, cap, 1)


def _last(cache, clone=False):
    return {x: (t[-1:].clone() if clone else t[-1:]) if torch.is_tensor(t) else t for x, t in cache.items()}


def _len(n):
    return torch.tensor([n], dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("G,rows", [(1, 1), (3, 9)])
def test_attention(G, rows):
    cap = 140000                                 # 5.7 GB of codes each
    c = Kv4Cache(L, 1, HKV, cap, D)
    g = torch.Generator(device="cuda").manual_seed(1)
    for x in "kv":
        c[x + "_codes"].random_(0, 256, generator=g)
        c[x + "_scales"][..., 0] = 0.25
        c[x + "_scales"][..., 1] = -2
        assert c[x + "_codes"].numel() > 2 ** 32
    q = torch.randn(L, 1, G * HKV, rows, D, generator=g, device="cuda").bfloat16()
    n = _len(cap - rows + 1)
    out = []
    for dims, qq, cc in ((_dims(L, cap, G * HKV), q, c), (_dims(1, cap, G * HKV), q[-1:].clone(), _last(c, clone=True))):
        o = torch.zeros_like(qq)
        ws = torch.empty(max(16, B.std_kv4_attn_workspace_size(dims, rows, cap)), dtype=torch.uint8, device="cuda")
        B.std_kv4_attn(dims, qq, rows, cc, n, 0, o, ws)
        out.append(o[-1].float())
    assert B.std_get_device_error() == 0
    # (the two calls cut the keys in other places; values are within [-2, 1.75], their mean some 2^-7 of that)
    assert out[1].abs().max() > 0 and (out[0] - out[1]).abs().max() <= 2.0 ** -7 * out[1].abs().max()


def test_rows_of_the_full_cache_and_new_ones():
    cap = 70000                                  # 4.6e9 values, 9.2 GB
    full = torch.zeros(L, 1, HKV, cap, D, dtype=torch.bfloat16, device="cuda")
    assert full.numel() > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(2)
    full[-1] = torch.randn(1, HKV, cap, D, generator=g, device="cuda").bfloat16()
    c, one = Kv4Cache(L, 1, HKV, cap, D), Kv4Cache(1, 1, HKV, cap, D)
    begin, count = _len(cap - 4100), _len(4000)
    B.std_kv4_quantize(_dims(L, cap), c, full, full, begin, count, 4000)
    B.std_kv4_quantize(_dims(1, cap), one, full[-1:].clone(), full[-1:].clone(), begin, count, 4000)
    new = torch.randn(L, 1, HKV, 3, D, generator=g, device="cuda").bfloat16()
    B.std_kv4_append(_dims(L, cap), c, _len(cap - 50), 7, new, new, 3)
    B.std_kv4_append(_dims(1, cap), one, _len(cap - 50), 7, new[-1:].clone(), new[-1:].clone(), 3)
    assert B.std_get_device_error() == 0
    for x in ("k_codes", "v_codes"):
        assert torch.equal(c[x][-1], one[x][0]) and bool(one[x].any())
    for x in ("k_scales", "v_scales"):
        assert torch.equal(c[x][-1].view(torch.int16), one[x][0].view(torch.int16))
    k, v = full, full                            # read back over it: the same values twice
    B.std_kv4_read(_dims(L, cap), c, None, None, cap, k, v)
    k1, v1 = (torch.zeros(1, 1, HKV, cap, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    B.std_kv4_read(_dims(1, cap), one, None, None, cap, k1, v1)
    assert B.std_get_device_error() == 0
    assert torch.equal(k1, v1) and torch.equal(full[-1], k1[0])


def test_norm_and_rotation():
    cap, rows = 70000, 40
    cache = torch.full((L, 1, HKV, cap, D), -7, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randn(L, 1, rows, HKV, D, generator=g, device="cuda").bfloat16()
    w = torch.ones(L, D, dtype=torch.bfloat16, device="cuda")
    rope = B.std_rope(10000.0 ** (-torch.arange(D // 2, dtype=torch.float64, device="cuda") / (D // 2)))
    one = torch.full((1, 1, HKV, cap, D), -7, dtype=torch.bfloat16, device="cuda")
    n = _len(cap - rows - 5)
    B.std_qk_norm_rope(_dims(L, cap), rope, None, k, None, rows, None, None, w, 1e-6, None, None, cache, None, cap, n, 5)
    B.std_qk_norm_rope(_dims(1, cap), rope, None, k[-1:].clone(), None, rows, None, None, w[-1:].clone(), 1e-6, None, None, one,
                       None, cap, n, 5)
    assert B.std_get_device_error() == 0
    assert torch.equal(cache[-1], one[0]) and bool((one[0, 0, :, -rows:] != -7).any())
