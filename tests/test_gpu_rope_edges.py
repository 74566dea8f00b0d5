"""std_qk_norm_rope where the tests of its values do not reach: channels that are not rotated, and every grid of its launch."""
import pytest
import torch

from sparse_top_kv_std_b200 import binding as B
from tests.test_gpu_rope import _check, _make, _run

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    B.lib()
    B.std_get_device_error(clear=True)


@pytest.mark.parametrize("d,dtype", [(64, torch.bfloat16), (128, torch.bfloat16), (32, torch.float32), (96, torch.float32)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotated", [0, 0.5])
@pytest.mark.parametrize("rows", [1, 9])
def test_channels_past_the_rotated_ones_pass_through(d, dtype, interleaved, rotated, rows):
    """Without a norm they are copied, whatever they hold; with one, an infinity makes the others of its head 0
    and itself NaN (x / infinity)."""
    rot = int(d * rotated)
    for norm in (False, True):
        c = _make(1, 1, rows, 4, 2, d, dtype, [3], rot, 1, 1, fused=False, norm=norm, interleaved=interleaved)
        plain = _run(c)
        c["q"][0, 0, 0, 1, rot + 2] = INF
        c["q"][0, 0, 0, 2, rot + 5] = -INF
        c["q"][0, 0, 0, 3, d - 1] = float("nan")
        c["k"][0, 0, 0, 1, d - 2] = INF
        q, k, v, cv = _run(c)
        cv.check()
        if norm:
            for head, ch in ((q[0, 0, 1, 0], rot + 2), (q[0, 0, 2, 0], rot + 5), (k[0, 0, 1, 3], d - 2)):
                others = torch.arange(d, device="cuda") != ch
                assert torch.isnan(head[ch]) and (head[others] == 0).all()
            assert torch.isnan(q[0, 0, 3, 0]).all()
        else:
            for got, want in ((q[0, 0], c["q"][0, 0].transpose(0, 1)), (k[0, 0, :, 3:3 + rows], c["k"][0, 0].transpose(0, 1))):
                a, b = got[..., rot:], want[..., rot:]
                bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
                assert torch.equal(torch.isnan(a), torch.isnan(b))
                assert torch.equal(torch.nan_to_num(a).view(bits), torch.nan_to_num(b).contiguous().view(bits))
                assert torch.isfinite(got[..., :rot]).all()
        # the rotated channels of heads without one, and all other heads, are as before
        assert torch.equal(q[0, 0, 0], plain[0][0, 0, 0]) and torch.equal(k[0, 0, 0], plain[1][0, 0, 0])
        if not norm:
            assert torch.equal(q[..., :rot], plain[0][..., :rot]) and torch.equal(k[..., :rot], plain[1][..., :rot])
    assert B.std_get_device_error() == 0


def test_zeros_keep_their_signs_without_norm_and_rotation():
    c = _make(1, 1, 5, 4, 2, 64, torch.float32, [0], 0, 1, 2, norm=False, fused=False)
    c["q"][..., ::3] = -0.0
    q, _, _, cv = _run(c)
    cv.check()
    assert torch.equal(q[0, 0].view(torch.int32), c["q"][0, 0].transpose(0, 1).contiguous().view(torch.int32))


@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (128, torch.float32), (32, torch.float32)])
@pytest.mark.parametrize("rows", [1, 40])
def test_entries_of_the_largest_stated_size_are_normalised(d, dtype, rows):
    c = _make(1, 2, rows, 4, 2, d, dtype, [3, 0], d, 1, 4, fused=False)
    for x in "qk":
        c[x].mul_(2.0 ** 55)
        c[x][0, 0, 0, 1] = torch.sign(c[x][0, 0, 0, 1].float()).to(dtype) * 2.0 ** 60
        assert c[x].abs().max() == 2.0 ** 60
    q, k, v, cv = _run(c)
    cv.check()
    assert B.std_get_device_error() == 0
    _check(c, q, k, v)


# ----------------------------------------------------------------------------- grids

def _grid(tokens, rows, heads, sms):
    """Tokens of a CTA and whether sequences share CTAs, by the launch's rule."""
    most = sms * (12 if heads > 16 else 6) // 5
    parts = -(-heads // 16)
    if tokens * parts <= most:
        return 1, False
    tok = next((t for t in (2, 4, 8) if tokens <= t * most), 16)
    places = -(-rows // tok) * tok
    return tok, 10 * (places - rows) > places


@pytest.mark.parametrize("dtype,d,Hq,Hkv", [(torch.bfloat16, 128, 14, 2), (torch.bfloat16, 64, 6, 1), (torch.float32, 64, 4, 2)])
@pytest.mark.parametrize("tok", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("axes", [1, 3])
def test_every_number_of_tokens_a_cta(dtype, d, Hq, Hkv, tok, shared, axes):
    """Chunks of a sequence's own with a remainder, and CTAs shared by sequences, of 1 to 16 tokens: padded
    batches, as many tokens as the rule of the launch asks for on this device."""
    if tok == 1 and shared:
        pytest.skip("a CTA of one token is not shared")
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    heads = Hq + 2 * Hkv
    most = sms * (12 if heads > 16 else 6) // 5
    if tok == 1:
        nB, rows = 3, most // -(-heads // 16) // 3
    elif shared:
        rows = {2: 3, 4: 5, 8: 11, 16: 19}[tok]
        nB = (most * tok * 3 // 4) // rows if tok < 16 else most * 9 // rows
    else:
        nB = 2
        rows = (most * tok * 3 // 4 if tok < 16 else most * 9) // nB | 1
    assert _grid(nB * rows, rows, heads, sms) == (tok, shared)
    n = [rows, rows - 1] + [(7 * b) % (rows + 1) for b in range(2, nB)]
    if not shared:
        n[-1] = rows // 2 // tok * tok + 1       # one token in its last chunk
    lens = [(5 * b) % 11 for b in range(nB)]
    c = _make(1, nB, rows, Hq, Hkv, d, dtype, lens, d, axes, 3, ragged=n)
    for b in range(nB):
        for x in "qkv":
            c[x][:, b, n[b]:] = float("nan")     # never read
    q, k, v, cv = _run(c)
    cv.check()
    assert B.std_get_device_error() == 0
    _check(c, q, k, v)
