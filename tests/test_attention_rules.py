"""Attention on the host, without a GPU: which strides of an output are refused
(rows of two CTAs must never meet), and the sizes that the splitting rules give."""
import ctypes
import itertools

import pytest

from chunked_vocab_cross_gb300 import _abi
from chunked_vocab_cross_gb300.build import build

OK = (5, 9)   # the host checks pass; there is no sm_103 device here


@pytest.fixture(scope="module")
def lib():
    build()
    return _abi.lib()


def _attn(**kw):
    a = _abi.LceAttn()
    a.causal, a.scale = 1, 0.125
    a.B, a.Tq, a.Tk, a.Hq, a.Hk, a.D = 1, 100, 100, 4, 2, 64
    for n, h in (("q", 4), ("k", 2), ("v", 2), ("o", 4), ("dO", 4), ("dq", 4), ("dk", 2), ("dv", 2)):
        setattr(a, n, 4096)
        setattr(a, n + "_ts", h * 64)
        setattr(a, n + "_hs", 64)
    a.lse = 4096
    for n, v in kw.items():
        setattr(a, n, v)
    return ctypes.byref(a)


def test_output_rows_that_meet_are_refused(lib):
    for f, outs in ((lib.lce_attention_forward, ("o",)), (lib.lce_attention_backward, ("dq", "dk", "dv"))):
        for n in outs:
            heads = 4 if n in ("o", "dq") else 2
            at = lambda ts, hs: f(_attn(**{n + "_ts": ts, n + "_hs": hs}))  # noqa: E731
            assert at(64, 64) == 2, n                        # head 1 of token 0 is head 0 of token 1
            assert at(64 * heads - 8, 64) == 2 and at(64, 64 * 99) == 2
            assert at(64 * heads, 64) in OK and at(64, 64 * 100) in OK      # token by token, head by head
            assert at(64 * 3 * heads, 64 * 3) in OK and at(128, 64 * 201) in OK
            assert at(128, 64 * 199) in OK                   # heads in each other's gaps
            assert at(128, 64 * 198) == 2
        # inputs may share rows
        assert f(_attn(k_ts=64, k_hs=64, q_ts=64, q_hs=64)) in OK


def test_output_rows_agree_with_a_count(lib):
    """Small layouts of rows of 16: refused exactly where two rows share an element."""
    for T, H, ts, hs in itertools.product((1, 3, 5), (1, 2, 4), *[(8, 16, 24, 32, 40, 64, 80)] * 2):
        cells = [t * ts + h * hs + c for t in range(T) for h in range(H) for c in range(0, 16, 8)]
        apart = len(set(cells)) == len(cells)
        got = lib.lce_attention_forward(_attn(Tq=T, Tk=T, Hq=H, Hk=1, D=16, q_ts=16 * H, q_hs=16, o_ts=ts, o_hs=hs))
        assert (got in OK) == apart and (apart or got == 2), (T, H, ts, hs, got)


def _ranges(lib, Tq, Hq, D, **kw):
    """Ranges that the keys are taken in, from the scratch: each has an o and an lse in fp32."""
    need = lib.lce_attention_forward_workspace_size(_attn(Tq=Tq, Hq=Hq, D=D, cu_q=4096, cu_k=4096, **kw))
    each = Tq * Hq * (D + 1) * 4
    assert need % each == 0
    return max(need // each, 1)


@pytest.mark.parametrize("B,heads,keys", [(1000, (2, 1), 4096), (64, (2, 1), 4096), (64, (32, 8), 4096), (8, (8, 8), 32768)])
def test_a_sequence_without_a_query_does_not_change_the_ranges(lib, B, heads, keys):
    """One-token decoding where a sequence or two have nothing to ask: still a tile of work for each of the others."""
    kw = dict(B=B, Tk=B * keys, Hk=heads[1], causal=0)
    for causal in (0, 1):
        kw["causal"] = causal
        n = _ranges(lib, B, heads[0], 128, **kw)
        assert n == _ranges(lib, B - 1, heads[0], 128, **kw) == _ranges(lib, B // 2 + 1, heads[0], 128, **kw)
    assert _ranges(lib, 1, heads[0], 128, **dict(kw, B=1, Tk=keys)) >= n


@pytest.mark.parametrize("B", [2, 9, 100])
def test_a_sequence_without_a_query_does_not_change_the_shares(lib, B):
    """The backward's scratch over its row statistics: as many shares of dK and dV for B - 1 queries as for B."""
    def shares(Tq, Hq=16):
        ws = lambda h: lib.lce_attention_workspace_size(_attn(Tq=Tq, Tk=200 * B, B=B, Hq=Hq, Hk=h, D=64, cu_q=4096, cu_k=4096))  # noqa: E731
        return ws(1) - ws(Hq)   # with as many key heads as query heads there is nothing to share
    assert shares(B) == shares(B - 1)
