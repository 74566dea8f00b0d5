"""Decoding with a draft over the 4-bit copy gives the dense model's greedy tokens exactly.

The toy model and the seeds of the top-K draft's losslessness test: ones whose fp64 greedy stream keeps a gap of
0.03 between the first and the second logit, far above the rounding of the verification, so that the streams are
equal, whatever the draft proposes."""
import pytest
import torch

from sparse_top_kv_std_b200 import binding as B
from sparse_top_kv_std_b200.kv4 import Kv4Cache
from tests.test_gpu_lossless import CAP_FULL, CFG, N_TOKENS, _first_diff, _model
from tests.toy_lm import _attn_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.backends.cuda.matmul.allow_tf32 = False
    B.lib()
    B.std_get_device_error(clear=True)


def _decode(m, k_full, v_full, first, gamma):
    """Tokens and the accepted inputs of every round."""
    c, W = m.cfg, m.dev()
    k_full, v_full = k_full.clone(), v_full.clone()
    dims = B.dims(c.L, 1, c.Hq, c.Hkv, c.d, B.STD_BF16, CAP_FULL, 1)
    one = B.dims(1, 1, c.Hq, c.Hkv, c.d, B.STD_BF16, CAP_FULL, 1)
    c4 = Kv4Cache(c.L, 1, c.Hkv, CAP_FULL, c.d)
    ws = torch.empty(max(16, B.std_kv4_attn_workspace_size(one, 1, c4.cap), B.std_attn_workspace_size(one, gamma + 1, CAP_FULL, 0)),
                     dtype=torch.uint8, device="cuda")
    n_ctx = c.nvis + c.T
    length = torch.tensor([n_ctx], dtype=torch.int32, device="cuda")
    B.std_kv4_quantize(dims, c4, k_full, v_full, None, length, CAP_FULL)
    n1 = torch.zeros(1, dtype=torch.int32, device="cuda")
    acc = torch.zeros((1, gamma + 1), dtype=torch.int32, device="cuda")
    out, counts = [first], []
    while len(out) < N_TOKENS:
        drafts = []
        for j in range(gamma):
            x = m.embed([(out + drafts)[-1]], n_ctx + j)
            for l in range(c.L):
                q, k, v = m.qkv(l, x)
                layer = {n: t[l:l + 1] if torch.is_tensor(t) else t for n, t in c4.items()}
                o = torch.empty((1, 1, c.Hq, 1, c.d), dtype=torch.bfloat16, device="cuda")
                B.std_kv4_append(one, layer, length, j, k[None, None].contiguous(), v[None, None].contiguous(), 1)
                B.std_kv4_attn(one, q[None, None].contiguous(), 1, layer, length, j + 1, o, ws)
                x = x + o[0, 0].float().transpose(0, 1).reshape(1, -1) @ W["Wo"][l]
            drafts.append(int(torch.argmax(x[0] @ W["Wlm"])))
        x = m.embed([out[-1]] + drafts, n_ctx)
        for l in range(c.L):
            x = _attn_layer(B, m, l, x, gamma + 1, k_full, v_full, length, 0,
                            lambda d, q, kl, vl, o: B.std_dense_verify_attn(d, q, gamma, kl, vl, length, o, 0, ws))
        dense = torch.argmax(x @ W["Wlm"], -1).to(torch.int32).reshape(1, gamma + 1).contiguous()
        B.std_accept_prefix(1, gamma, torch.tensor([drafts], dtype=torch.int32, device="cuda"), dense, n1, acc)
        B.std_kv4_quantize(dims, c4, k_full, v_full, length, n1, gamma + 1)
        length += n1
        n = int(n1)
        out.extend(acc[0, :n].tolist())
        counts.append(n)
        n_ctx += n
    assert B.std_get_device_error() == 0
    return out[:N_TOKENS], counts


@pytest.mark.parametrize("seed,gamma", [(1, 6), (2, 6), (6, 8), (1, 1), (2, 31)])
def test_the_stream_equals_dense_greedy(seed, gamma):
    m, want, kf, vf, _, first = _model(seed)
    got, counts = _decode(m, kf, vf, first, gamma)
    assert got == want, (_first_diff(got, want), counts)
    assert all(1 <= n <= gamma + 1 for n in counts)
