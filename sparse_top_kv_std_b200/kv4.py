"""A 4-bit K/V cache on the device, and decoding with a draft that reads one.

``Kv4Cache`` owns the four arrays of a 4-bit cache and is the mapping that ``binding``'s
std_kv4_* calls take.  ``Kv4Session`` runs Sparse-to-Dense rounds whose draft attends a 4-bit
copy of the whole context instead of a top-K subset; verification is over the full cache, so
the output is that of dense decoding:

    s = Kv4Session(L=28, B=1, Hq=28, Hkv=4, d=128, dtype=STD_BF16, cap=..., gamma=8)
    s.k_full[...] = prompt keys; s.v_full[...] = prompt values
    s.start(n)               # committed context = n rows; their 4-bit copy
    s.round(io)              # gamma drafts + verify + accept + commit
"""
from __future__ import annotations

from contextlib import nullcontext
from typing import Dict

import torch

from . import binding as B_
from .session import storage_dtype

ROWS = 16  # a capacity is a multiple of this


class Kv4Cache(dict):
    """k_codes, k_scales, v_codes, v_scales and cap of a cache of at least `cap` rows."""

    def __init__(self, L: int, B: int, Hkv: int, cap: int, d: int, device="cuda"):
        cap = -(-int(cap) // ROWS) * ROWS
        dev = torch.device(device)
        super().__init__(cap=cap)
        for x in "kv":
            self[x + "_codes"] = torch.zeros((L, B, Hkv, cap, d // 2), dtype=torch.uint8, device=dev)
            self[x + "_scales"] = torch.zeros((L, B, Hkv, cap, d // 64, 2), dtype=torch.bfloat16, device=dev)

    @property
    def cap(self) -> int:
        return self["cap"]

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in self.values() if torch.is_tensor(t))


def _on(stream):
    """The context in which torch and the library work on `stream` (a torch stream, a handle, or None: the
    current one)."""
    if stream is None:
        return nullcontext()
    if isinstance(stream, int):  # (ExternalStream(0) would be a stream of its own)
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


class Kv4Session:
    def __init__(self, L: int, B: int, Hq: int, Hkv: int, d: int, dtype: int, cap: int, gamma: int, device="cuda"):
        self.L, self.B, self.Hq, self.Hkv, self.d, self.gamma = L, B, Hq, Hkv, d, gamma
        self.dims = B_.dims(L, B, Hq, Hkv, d, dtype, cap, 1)
        dev, st = torch.device(device), storage_dtype(dtype)
        self.k_full = torch.zeros((L, B, Hkv, cap, d), dtype=st, device=dev)
        self.v_full = torch.zeros_like(self.k_full)
        self.cache4 = Kv4Cache(L, B, Hkv, cap, d, device)
        self.len_full = torch.zeros(B, dtype=torch.int32, device=dev)
        need = max(16, B_.std_kv4_attn_workspace_size(self.dims, 1, self.cache4.cap),
                   B_.std_attn_workspace_size(self.dims, gamma + 1, cap, 0))
        self.ws = torch.empty(need, dtype=torch.uint8, device=dev)

    def start(self, n, stream=None) -> None:
        """Set the committed lengths (n: one for each sequence) and copy their rows to the 4-bit cache."""
        with _on(stream):
            self.len_full.copy_(torch.as_tensor(n, dtype=torch.int32))
            B_.std_kv4_quantize(self.dims, self.cache4, self.k_full, self.v_full, None, self.len_full, self.dims.cap_full)

    def round(self, io: Dict[str, torch.Tensor], stream=None) -> None:
        """io: the tensors of a std_round_io (round_outputs() makes its outputs).  A sequence without room for
        gamma + 1 rows is flagged (STD_DEVERR_*) and its context left as it is."""
        with _on(stream):
            self._round(io)

    def _round(self, io) -> None:
        d, g = self.dims, self.gamma
        for j in range(g):
            B_.std_kv4_append(d, self.cache4, self.len_full, j, io["k_draft"][j], io["v_draft"][j], 1)
            B_.std_kv4_attn(d, io["q_draft"][j], 1, self.cache4, self.len_full, j + 1, io["o_draft"][j], self.ws)
        B_.std_dense_verify_attn_append(d, io["q_verify"], g, self.k_full, self.v_full, self.len_full, io["k_verify"],
                                        io["v_verify"], io["o_verify"], 0, self.ws)
        B_.std_accept_prefix(self.B, g, io["draft_tokens"], io["dense_tokens"], io["n_plus_1"], io["accepted"])
        # the accepted inputs' rows replace the draft's own; what lies behind them is not read again.  The verify
        # has appended nothing to a sequence whose rows would pass the capacity: none of them are accepted.
        fits = (self.len_full >= 0) & (self.len_full <= d.cap_full - (g + 1))
        n = io["n_plus_1"] * fits
        B_.std_kv4_quantize(d, self.cache4, self.k_full, self.v_full, self.len_full, n, g + 1)
        self.len_full += n

    def round_outputs(self) -> Dict[str, torch.Tensor]:
        """o_draft (in the queries' type), o_verify, n_plus_1 and accepted of one round."""
        dev, g = self.k_full.device, self.gamma
        return {"o_draft": torch.zeros((g, self.L, self.B, self.Hq, 1, self.d), dtype=self.k_full.dtype, device=dev),
                "o_verify": torch.zeros((self.L, self.B, self.Hq, g + 1, self.d), dtype=torch.float32, device=dev),
                "n_plus_1": torch.zeros(self.B, dtype=torch.int32, device=dev),
                "accepted": torch.zeros((self.B, g + 1), dtype=torch.int32, device=dev)}
