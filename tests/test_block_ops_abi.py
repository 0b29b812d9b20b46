"""The block operators' C entry points without a GPU: struct layouts of the
ctypes mirrors and the host-side argument checks."""
import ctypes
import os
import subprocess
import tempfile

import pytest

from chunked_vocab_cross_gb300 import _abi
from chunked_vocab_cross_gb300.build import INCLUDE, build

OK = (5, 9)   # the host checks pass; there is no sm_103 device here


@pytest.fixture(scope="module")
def lib():
    build()
    return _abi.lib()


@pytest.mark.parametrize("mirror,name", [(_abi.LceAttn, "lce_attn_t"), (_abi.LceNorm, "lce_norm_t")])
def test_struct_layout_matches_c(mirror, name):
    fields = [f[0] for f in mirror._fields_]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "lce.h"\nint main(void) {\n  printf("%zu", sizeof(' + name + "));\n"
    src += "".join(f'  printf(" %zu", offsetof({name}, {f}));\n' for f in fields) + "  return 0; }\n"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        with open(c, "w") as f:
            f.write(src)
        subprocess.run(["gcc", "-I", INCLUDE, "-o", exe, c], check=True)
        vals = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert vals[0] == ctypes.sizeof(mirror)
    assert vals[1:] == [getattr(mirror, f).offset for f in fields]


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
    return ctypes.byref(a), a


@pytest.mark.parametrize("entry", ["lce_attention_forward", "lce_attention_backward"])
def test_attention_host_checks(lib, entry):
    f = getattr(lib, entry)
    run = lambda **kw: f(_attn(**kw)[0])  # noqa: E731
    assert f(None) == 1
    assert run() in OK
    assert run(q=None) == 1 and run(lse=None) == 1 and run(o=None) == 1
    assert run(dtype=3) == 4
    for kw in (dict(D=0), dict(D=136), dict(Hq=3), dict(Hk=0), dict(B=0), dict(Tq=-1), dict(Tk=1 << 30), dict(B=3),
               dict(q_ts=-64), dict(k_hs=1 << 36)):
        assert run(**kw) == 2, kw
    for kw in (dict(D=12), dict(q=4100), dict(k_ts=132), dict(v_hs=4)):
        assert run(**kw) == 3, kw
    assert run(cu_q=4096) == 1                               # offsets of one side only
    assert run(scale=float("nan")) == 10 and run(scale=float("inf")) == 10
    assert run(Tq=0, q=None, o=None, lse=None, dO=None, dq=None) in OK
    if entry.endswith("forward"):
        assert run(o_ts=0) == 2                              # output rows in one place
    else:
        assert run(dq_ts=0) == 2 and run(dk_hs=8) == 2 and run(dv=None) == 1 and run(dO=None) == 1


def test_attention_workspace(lib):
    ws = lambda **kw: lib.lce_attention_workspace_size(_attn(**kw)[0])  # noqa: E731
    assert ws(D=12) == 0 and ws(Hk=3) == 0
    assert 0 < ws() and ws(Tk=1000, B=1) >= ws()
    # row statistics, not probabilities: linear in the tokens
    assert ws(Tq=1 << 20, Tk=1 << 20, Hq=32, Hk=8, D=128) < (1 << 20) * 32 * 128 * 64
    fwd = lambda **kw: lib.lce_attention_forward_workspace_size(_attn(**kw)[0])  # noqa: E731
    assert fwd() == 0 and fwd(Tq=8192, Tk=8192, Hq=32, Hk=8, D=128, B=1) == 0 and fwd(D=12) == 0
    # few rows over long keys: at most 64 ranges of o and lse in fp32
    assert 0 < fwd(Tq=1, Tk=1 << 20, Hq=32, Hk=8, D=128, B=1) <= 64 * 32 * 129 * 4
    # few query heads of one key head: the heads' sums of dK and dV
    assert ws(Tq=1024, Tk=1024, Hq=16, Hk=1, D=128, B=1) > ws(Tq=1024, Tk=1024, Hq=16, Hk=16, D=128, B=1)


def _norm(**kw):
    a = _abi.LceNorm()
    a.N, a.d, a.scale, a.eps = 10, 64, 1.0, 1e-6
    for n in ("x", "b", "w_post", "gate", "w_pre", "r", "n", "rstd_post", "rstd_pre", "dr", "dn", "dx", "db", "dw_post",
              "dgate", "dw_pre"):
        setattr(a, n, 4096)
    for n, v in kw.items():
        setattr(a, n, v)
    return ctypes.byref(a), a


def test_norm_host_checks(lib):
    fwd, bwd = lib.lce_block_norm_forward, lib.lce_block_norm_backward
    for f in (fwd, bwd):
        run = lambda **kw: f(_norm(**kw)[0])  # noqa: E731
        assert f(None) == 1 and run() in OK
        assert run(dtype=2) == 4
        assert run(d=4) == 2 and run(d=16392) == 2 and run(N=-1) == 2
        assert run(d=68) == 3 and run(b=4100) == 3 and run(ld_b=68) == 3
        assert run(rstd_post=None) == 1 and run(rstd_pre=None) == 1 and run(r=None) == 1
        assert run(b=None) == 10 and run(b=None, w_post=None, gate=None, w_pre=None) == 10
        assert run(scale=float("nan")) == 10 and run(eps=-1.0) == 10
        assert run(b=None, w_post=None, gate=None) in OK
    assert fwd(_norm(x=None)[0]) == 1 and fwd(_norm(n=None)[0]) == 1
    for n in ("dn", "dx", "db", "dw_post", "dgate", "dw_pre"):
        assert bwd(_norm(**{n: None})[0]) == 1, n
    assert bwd(_norm(dr=None)[0]) in OK
    ws = lambda **kw: lib.lce_block_norm_workspace_size(_norm(**kw)[0])  # noqa: E731
    assert ws() > 0 and ws(d=12) == 0 and ws(N=1 << 20) == ws(N=1 << 24)   # partial sums do not grow with the rows


def test_clip_host_checks(lib):
    ptr = (ctypes.c_void_p * 2)(4096, 8192)
    n, dt = (ctypes.c_int64 * 2)(10, 20), (ctypes.c_int32 * 2)(0, 1)
    run = lambda count=2, g=ptr, o=None, n=n, dt=dt, m=1.0, e=1e-6, norm=4096: lib.lce_clip_grads(  # noqa: E731
        count, g, o, n, dt, m, e, norm, None, None, 0, None)
    assert run() in OK and run(o=ptr) in OK
    assert run(norm=None) == 1 and run(g=None) == 1 and run(g=(ctypes.c_void_p * 2)(4096, None)) == 1
    assert run(count=-1) == 2 and run(n=(ctypes.c_int64 * 2)(10, -1)) == 2
    assert run(dt=(ctypes.c_int32 * 2)(0, 5)) == 4
    assert run(g=(ctypes.c_void_p * 2)(4097, 8192)) == 3 and run(g=(ctypes.c_void_p * 2)(4096, 8194)) == 3
    assert run(m=-1.0) == 10 and run(m=float("nan")) == 10 and run(e=-1.0) == 10
    assert run(g=(ctypes.c_void_p * 2)(4096, None), n=(ctypes.c_int64 * 2)(10, 0)) in OK
    assert lib.lce_grad_norm(2, ptr, n, dt, 4096, None, 0, None) in OK
    assert lib.lce_grad_norm(2, ptr, n, dt, 4096, 4096, 8, None) in OK + (6,)
    assert lib.lce_clip_workspace_size(2) > 0 and lib.lce_clip_workspace_size(-1) == 0
