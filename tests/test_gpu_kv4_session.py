"""Kv4Session at a cache's end, on streams and in graphs."""
import pytest
import torch

from sparse_top_kv_std_b200 import binding as B
from sparse_top_kv_std_b200.kv4 import Kv4Session

pytestmark = pytest.mark.gpu

L, NB, HQ, HKV, D, CAP, GAMMA = 2, 3, 4, 2, 64, 200, 4


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    B.lib()
    B.std_get_device_error(clear=True)


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def _session(n, stream=None):
    s = Kv4Session(L, NB, HQ, HKV, D, B.STD_BF16, CAP, GAMMA)
    s.k_full.copy_(_randn(1, *s.k_full.shape))
    s.v_full.copy_(_randn(2, *s.v_full.shape))
    torch.cuda.synchronize()
    s.start(n, stream=stream)
    return s


def _io(s, seed, accepted):
    """Inputs of a round in which sequence b's first accepted[b] drafts agree with the dense model."""
    io = dict(zip(("q_draft", "k_draft", "v_draft"),
                  (_randn(seed + i, GAMMA, L, NB, h, 1, D) for i, h in enumerate((HQ, HKV, HKV)))))
    io.update(zip(("q_verify", "k_verify", "v_verify"),
                  (_randn(seed + 9 + i, L, NB, h, GAMMA + 1, D) for i, h in enumerate((HQ, HKV, HKV)))))
    io["draft_tokens"] = torch.zeros(NB, GAMMA, dtype=torch.int32, device="cuda")
    io["dense_tokens"] = torch.tensor([[0] * a + [7] * (GAMMA + 1 - a) for a in accepted], dtype=torch.int32, device="cuda")
    io.update(s.round_outputs())
    return io


def _copy4(s):
    """The values of the 4-bit cache's committed rows."""
    k = torch.zeros(L, NB, HKV, CAP, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    B.std_kv4_read(s.dims, s.cache4, None, s.len_full, CAP, k, v)
    return k, v


def test_a_sequence_without_room_keeps_its_length():
    """Four rows are left where a round takes five: nothing of it is accepted there, whatever the tokens say,
    and the other sequences go on."""
    lens = [100, CAP - GAMMA, 30]
    s = _session(lens)
    before, full = _copy4(s), s.k_full.clone()
    io = _io(s, 10, [2, 1, 4])
    s.round(io)
    torch.cuda.synchronize()
    assert B.std_get_device_error(clear=True) != 0
    assert s.len_full.tolist() == [103, CAP - GAMMA, 35]
    after = _copy4(s)
    for a, b in zip(after, before):
        assert torch.equal(a[:, 1], b[:, 1])
        assert torch.equal(a[:, 0, :, :100], b[:, 0, :, :100]) and torch.equal(a[:, 2, :, :30], b[:, 2, :, :30])
    assert torch.equal(s.k_full[:, 1, :, :CAP - GAMMA], full[:, 1, :, :CAP - GAMMA])
    assert torch.equal(s.k_full[:, 0, :, 100:105], io["k_verify"][:, 0])
    s.round(_io(s, 40, [0, 4, 1]))
    torch.cuda.synchronize()
    assert B.std_get_device_error(clear=True) != 0
    assert s.len_full.tolist() == [104, CAP - GAMMA, 37]


def test_a_round_that_just_fits_is_accepted():
    s = _session([CAP - GAMMA - 1, 5, 0])
    s.round(_io(s, 10, [4, 0, 4]))
    torch.cuda.synchronize()
    assert B.std_get_device_error(clear=True) == 0
    assert s.len_full.tolist() == [CAP, 6, 5]


@pytest.mark.parametrize("handle", [False, True])
def test_rounds_on_another_stream_and_in_a_graph(handle):
    lens, accepted = [100, 61, 0], [2, 4, 0]
    s = _session(lens)
    want = _io(s, 10, accepted)
    s.round(want)
    torch.cuda.synchronize()
    want4 = _copy4(s)

    side = torch.cuda.Stream()
    t = _session(lens, stream=side.cuda_stream if handle else side)
    got = _io(t, 10, accepted)
    side.wait_stream(torch.cuda.current_stream())
    busy = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(side):
        for _ in range(20):                      # the round has to wait for its own stream, not for the current one
            busy.add_(1)
    t.round(got, stream=side.cuda_stream if handle else side)
    side.synchronize()
    assert t.len_full.tolist() == s.len_full.tolist()
    for x in ("o_draft", "o_verify", "n_plus_1", "accepted"):
        assert torch.equal(got[x], want[x])
    assert all(torch.equal(a, b) for a, b in zip(_copy4(t), want4))

    u = _session(lens)
    io = _io(u, 10, accepted)
    graph = torch.cuda.CUDAGraph()
    u.round(io)                                  # (first calls set kernels up)
    u.start(lens)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        u.round(io)
    graph.replay()
    torch.cuda.synchronize()
    assert u.len_full.tolist() == s.len_full.tolist()
    for x in ("o_draft", "o_verify", "n_plus_1", "accepted"):
        assert torch.equal(io[x], want[x])
    assert all(torch.equal(a, b) for a, b in zip(_copy4(u), want4))
    assert B.std_get_device_error(clear=True) == 0


def test_a_handle_of_zero_is_the_default_stream():
    """A round on 0, called while another stream is current, comes after what the default stream holds."""
    s = _session([100, 61, 0])
    io, tokens = _io(s, 10, [0, 0, 0]), _io(s, 10, [2, 4, 0])["dense_tokens"]
    s.round(io, stream=0)                        # (first calls load kernels and take memory, which waits for the device)
    s.start([100, 61, 0])
    side = torch.cuda.Stream()
    busy = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(600):                         # (some 50 ms, well above what the round takes to be launched)
        busy.add_(1)
    io["dense_tokens"].copy_(tokens)
    with torch.cuda.stream(side):
        s.round(io, stream=0)
    torch.cuda.synchronize()
    assert s.len_full.tolist() == [103, 66, 1]
    assert B.std_get_device_error(clear=True) == 0
