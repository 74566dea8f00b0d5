"""Norm and rotation, the 4-bit cache and the attention over it, run together as a decoder runs them.

``Kv4Session``: rounds whose draft reads a 4-bit copy of the context, against the oracle on the values
that copy holds.  ``TinyLM``: a random-weight model whose layers go from the fused projection through
std_qk_norm_rope into the caches; its tokens, drafted over the 4-bit copy and verified over the bf16 cache,
are the greedy choices of the dense model (as for the top-K draft: the draft only proposes)."""
import math

import numpy as np
import pytest
import torch

import oracle
import synth
from oracle import kv4_oracle as O
from sparse_top_kv_std_b200 import binding as B
from sparse_top_kv_std_b200.kv4 import Kv4Cache, Kv4Session
from tests import harness as H

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    B.lib()
    B.std_get_device_error(clear=True)
    torch.backends.cuda.matmul.allow_tf32 = False


def _quantised(x):
    """float64 values of the 4-bit copy of bf16 rows (bits as uint16)."""
    return O.kv4_values(*O.kv4_quantize(synth.storage_to_f64(x, "bf16")))


def test_session_rounds_match_the_oracle():
    wl = synth.Workload("kv4", 150, "bf16", 2, 2, 28, 4, 128, (700, 333), 32, 128, 5, 0.02, 0.7, 3)
    x = synth.host_inputs(wl, seed=3)
    s = Kv4Session(wl.L, wl.B, wl.Hq, wl.Hkv, wl.d, B.STD_BF16, wl.cap_full, wl.gamma)
    s.k_full.copy_(H.to_dev(x["k_full"]))
    s.v_full.copy_(H.to_dev(x["v_full"]))
    n = np.array(wl.nvis) + wl.T
    s.start(n)
    kf, vf = H.f64(x["k_full"], wl), H.f64(x["v_full"], wl)
    k4, v4 = np.zeros_like(kf), np.zeros_like(vf)
    for b in range(wl.B):
        k4[:, b, :, :n[b]] = _quantised(x["k_full"][:, b, :, :n[b]])
        v4[:, b, :, :n[b]] = _quantised(x["v_full"][:, b, :, :n[b]])
    for r in range(wl.rounds):
        io = {k: H.to_dev(x[k][r]) for k in ("q_draft", "k_draft", "v_draft", "q_verify", "k_verify", "v_verify")}
        io["draft_tokens"] = torch.from_numpy(x["draft_tokens"][r]).cuda()
        io["dense_tokens"] = torch.from_numpy(x["dense_tokens"][r]).cuda()
        io.update(s.round_outputs())
        s.round(io)
        torch.cuda.synchronize()
        assert B.std_get_device_error() == 0
        kd, vd = k4.copy(), v4.copy()
        for j in range(wl.gamma):
            for b in range(wl.B):
                kd[:, b, :, n[b] + j] = _quantised(x["k_draft"][r][j][:, b, :, 0])
                vd[:, b, :, n[b] + j] = _quantised(x["v_draft"][r][j][:, b, :, 0])
            want = O.causal_decode_attn(H.f64(x["q_draft"][r][j], wl), kd, vd, n + j + 1)
            assert np.abs(io["o_draft"][j].double().cpu().numpy() - want).max() <= H.attn_tol(wl)
        for b in range(wl.B):
            kf[:, b, :, n[b]:n[b] + wl.gamma + 1] = H.f64(x["k_verify"][r][:, b], wl)
            vf[:, b, :, n[b]:n[b] + wl.gamma + 1] = H.f64(x["v_verify"][r][:, b], wl)
        want = oracle.dense_verify_attn(H.f64(x["q_verify"][r], wl), kf, vf, n)
        assert np.abs(io["o_verify"].cpu().numpy() - want).max() <= H.attn_tol(wl)
        n1, acc = oracle.accept_prefix(x["draft_tokens"][r], x["dense_tokens"][r])
        assert io["n_plus_1"].cpu().tolist() == list(n1)
        for b in range(wl.B):
            new = slice(n[b], n[b] + n1[b])
            k4[:, b, :, new] = _quantised(x["k_verify"][r][:, b, :, :n1[b]])
            v4[:, b, :, new] = _quantised(x["v_verify"][r][:, b, :, :n1[b]])
        n = n + n1
        assert s.len_full.cpu().tolist() == n.tolist()
    # the 4-bit copy at the end, read back
    out = torch.zeros((wl.L, wl.B, wl.Hkv, int(n.max()), wl.d), dtype=torch.bfloat16, device="cuda")
    out_v = torch.zeros_like(out)
    B.std_kv4_read(s.dims, s.cache4, None, s.len_full, out.shape[3], out, out_v)
    for b in range(wl.B):
        for got, want in ((out, k4), (out_v, v4)):
            w = torch.from_numpy(want[:, b, :, :n[b]]).cuda().float().bfloat16()
            assert torch.equal(got[:, b, :, :n[b]], w)


class TinyLM:
    """Embedding, L layers (fused projection, norm and rotation, attention, residual), head; random weights."""

    def __init__(self, seed, L=2, Hq=4, Hkv=2, d=64, dm=128, vocab=96):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
        self.L, self.Hq, self.Hkv, self.d = L, Hq, Hkv, d
        self.E = r(vocab, dm)
        self.Wqkv = r(L, dm, (Hq + 2 * Hkv) * d) / math.sqrt(dm)
        self.Wo = r(L, Hq * d, dm) / math.sqrt(Hq * d)
        self.Wlm = 6 * r(dm, vocab) / math.sqrt(dm)
        self.qw = (1.5 + 0.2 * r(L, d)).bfloat16()
        self.kw = (1.5 + 0.2 * r(L, d)).bfloat16()
        self.prompt = torch.randint(0, vocab, (112,), generator=g).cuda()
        self.freq = 10000.0 ** (-torch.arange(d // 2, dtype=torch.float64, device="cuda") / (d // 2))
        self.rope = B.std_rope(self.freq)

    def qkv(self, l, x):
        y = (x @ self.Wqkv[l]).bfloat16().view(1, 1, x.shape[0], self.Hq + 2 * self.Hkv, self.d)
        return y.split([self.Hq, self.Hkv, self.Hkv], dim=3)

    def forward(self, tokens, length, attend, place):
        """Logits of `tokens` at positions length..; place(l, q, k, v, rows) -> rotated q with the rows in the
        caches, attend(l, q, rows) -> [Hq][rows][d]."""
        x = self.E[tokens]
        rows = x.shape[0]
        for l in range(self.L):
            q = place(l, *self.qkv(l, x), rows)
            o = attend(l, q, rows).float()
            x = x + o.transpose(0, 1).reshape(rows, -1) @ self.Wo[l]
        return x @ self.Wlm


class Decoder:
    def __init__(self, m, cap):
        self.m, self.cap = m, cap
        self.k = torch.zeros((m.L, 1, m.Hkv, cap, m.d), dtype=torch.bfloat16, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.c4 = Kv4Cache(m.L, 1, m.Hkv, cap, m.d)
        self.dims = B.dims(1, 1, m.Hq, m.Hkv, m.d, B.STD_BF16, cap, 1)
        self.all = B.dims(m.L, 1, m.Hq, m.Hkv, m.d, B.STD_BF16, cap, 1)
        self.len = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.zero = torch.zeros(1, dtype=torch.int32, device="cuda")
        need = max([B.std_attn_workspace_size(self.dims, r, cap, 0) for r in range(1, 17)] +
                   [B.std_kv4_attn_workspace_size(self.dims, 1, self.c4.cap), 16])
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def layer4(self, l):
        return {x: t[l:l + 1] if torch.is_tensor(t) else t for x, t in self.c4.items()}

    def full(self, tokens):
        """Tokens over the bf16 cache, their rows placed behind it."""
        m = self.m

        def place(l, q, k, v, rows):
            out = torch.empty((1, 1, m.Hq, rows, m.d), dtype=torch.bfloat16, device="cuda")
            B.std_qk_norm_rope(self.dims, m.rope, q, k, v, rows, None, m.qw[l:l + 1], m.kw[l:l + 1], 1e-6, None, out,
                               self.k[l:l + 1], self.v[l:l + 1], self.cap, self.len, 0)
            return out

        def attend(l, q, rows):
            o = torch.empty((1, 1, m.Hq, rows, m.d), device="cuda")
            B.std_dense_verify_attn(self.dims, q, rows - 1, self.k[l:l + 1], self.v[l:l + 1], self.len, o, 0, self.ws)
            return o[0, 0]

        return m.forward(tokens, self.len, attend, place)

    def draft(self, token, j):
        """One token over the 4-bit cache, j rows behind its committed ones."""
        m = self.m
        pos = (self.len + j).view(1, 1, 1)

        def place(l, q, k, v, rows):
            out = torch.empty((1, 1, m.Hq, 1, m.d), dtype=torch.bfloat16, device="cuda")
            row_k, row_v = (torch.empty((1, 1, m.Hkv, 1, m.d), dtype=torch.bfloat16, device="cuda") for _ in "kv")
            B.std_qk_norm_rope(self.dims, m.rope, q, k, v, 1, None, m.qw[l:l + 1], m.kw[l:l + 1], 1e-6, pos, out, row_k,
                               row_v, 1, self.zero, 0)
            B.std_kv4_append(self.dims, self.layer4(l), self.len, j, row_k, row_v, 1)
            return out

        def attend(l, q, rows):
            o = torch.empty((1, 1, m.Hq, 1, m.d), dtype=torch.bfloat16, device="cuda")
            B.std_kv4_attn(self.dims, q, 1, self.layer4(l), self.len, j + 1, o, self.ws)
            return o[0, 0]

        return m.forward(token, self.len, attend, place)

    def prefill(self):
        for i in range(0, len(self.m.prompt), 16):
            logits = self.full(self.m.prompt[i:i + 16])
            self.len += 16
        return int(logits[-1].argmax())


@pytest.mark.parametrize("seed", [0, 1, 2, 3])
@pytest.mark.parametrize("gamma", [1, 4])
def test_tokens_drafted_over_four_bits_are_the_greedy_ones(seed, gamma):
    m = TinyLM(seed)
    n = 48
    d = Decoder(m, 256)
    out = [d.prefill()]
    B.std_kv4_quantize(d.all, d.c4, d.k, d.v, None, d.len, d.cap)
    n1 = torch.zeros(1, dtype=torch.int32, device="cuda")
    acc = torch.zeros((1, gamma + 1), dtype=torch.int32, device="cuda")
    counts = []
    while len(out) < n:
        drafted = []
        for j in range(gamma):
            drafted.append(int(d.draft(torch.tensor([(out + drafted)[-1]], device="cuda"), j)[-1].argmax()))
        dense = d.full(torch.tensor([out[-1]] + drafted, device="cuda")).argmax(-1).to(torch.int32).view(1, -1).contiguous()
        B.std_accept_prefix(1, gamma, torch.tensor([drafted], dtype=torch.int32, device="cuda"), dense, n1, acc)
        B.std_kv4_quantize(d.all, d.c4, d.k, d.v, d.len, n1, gamma + 1)
        d.len += n1
        counts.append(int(n1))
        out += acc[0, :counts[-1]].tolist()
    assert B.std_get_device_error() == 0
    # Every token is the greedy choice of the dense model, one row at a time, after the tokens before it.  Rows
    # verified together and alone differ by the attention's rounding, up to 2e-2 an output; through the output
    # projection (rows of norm 1) and the head (6) that is 0.12 of a logit: a choice within 0.25 of the largest.
    check = Decoder(m, 256)
    assert check.prefill() == out[0]
    for a, b in zip(out, out[1:]):
        logits = check.full(torch.tensor([a], device="cuda"))[-1]
        check.len += 1
        assert logits.max() - logits[b] <= 0.25
    assert sum(counts) / len(counts) > 1.3, counts       # the 4-bit draft is worth having
