"""The recurrent block's C entry points without a GPU: struct layouts of the
ctypes mirrors, host-side argument checks and workspace sizes. (The addresses
are made up: only where nothing can be launched on them.)"""
import ctypes
import os
import subprocess
import tempfile

import pytest

torch = pytest.importorskip("torch")

from chunked_vocab_cross_gb300 import _abi  # noqa: E402
from chunked_vocab_cross_gb300.build import INCLUDE, build  # noqa: E402

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where there is no GPU")
OK = (5, 9)   # the host checks pass; there is no sm_103 device here


@pytest.fixture(scope="module")
def lib():
    build()
    return _abi.lib()


@pytest.mark.parametrize("mirror,name", [(_abi.LceLayerNorm, "lce_layer_norm_t"), (_abi.LceWgrad, "lce_wgrad_t"),
                                         (_abi.LceRecurrence, "lce_recurrence_t")])
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
    assert vals[0] == ctypes.sizeof(mirror) and vals[1:] == [getattr(mirror, f).offset for f in fields]


def _filled(mirror, pointers, values, **kw):
    a = mirror()
    for n in pointers:
        setattr(a, n, 4096)
    for n, v in {**values, **kw}.items():
        setattr(a, n, v)
    return ctypes.byref(a), a


def _ln(**kw):
    return _filled(_abi.LceLayerNorm, ("x", "b", "weight", "bias", "r", "n", "mean", "rstd", "dr", "dn", "dx", "dweight", "dbias"),
                   dict(N=10, d=64, eps=1e-5), **kw)


def test_layer_norm_host_checks(lib):
    fwd, bwd = lib.lce_layer_norm_forward, lib.lce_layer_norm_backward
    packed = dict(codes=4096, exps=4096, ld_codes=64, ld_exps=16)
    for f in (fwd, bwd):
        run = lambda **kw: f(_ln(**kw)[0])  # noqa: E731
        assert f(None) == 1 and run() in OK and run(**packed) in OK
        assert run(dtype=2) == 4
        assert run(d=4) == 2 and run(d=16392) == 2 and run(N=-1) == 2 and run(N=1 << 31) == 2
        assert run(d=68) == 3 and run(weight=4100) == 3
        assert run(weight=None) == 1 and run(mean=None) == 1 and run(rstd=None) == 1 and run(r=None) == 1
        assert run(**{**packed, "exps": None}) == 1
        assert run(**{**packed, "ld_codes": 48}) == 2 and run(**{**packed, "ld_exps": 0}) == 2
        assert run(**{**packed, "ld_codes": 72}) == 3 and run(**{**packed, "codes": 4104}) == 3 and run(**{**packed, "ld_exps": 24}) == 3
    assert fwd(_ln(x=None)[0]) == 1 and fwd(_ln(n=None)[0]) == 1 and fwd(_ln(ld_x=68)[0]) == 3 and fwd(_ln(ld_b=-8)[0]) == 2
    assert fwd(_ln(b=None, r=None)[0]) in OK and fwd(_ln(bias=None)[0]) in OK
    assert fwd(_ln(eps=-1.0)[0]) == 10 and fwd(_ln(eps=float("nan"))[0]) == 10
    assert fwd(_ln(N=0, x=None, b=None, r=None, n=None, mean=None, rstd=None)[0]) in OK
    for n in ("dn", "dx", "dweight"):
        assert bwd(_ln(**{n: None})[0]) == 1, n
    assert bwd(_ln(dr=None, dbias=None)[0]) in OK and bwd(_ln(r=None, **packed)[0]) in OK and bwd(_ln(ld_dn=68)[0]) == 3
    ws = lambda **kw: lib.lce_layer_norm_workspace_size(_ln(**kw)[0])  # noqa: E731
    assert ws() > 0 and ws(d=12) == 0 and ws(N=1 << 20) == ws(N=1 << 24)


def test_pack_host_checks(lib):
    def pack(dtype=0, x=4096, ld=0, N=10, d=200, codes=4096, ldc=208, exps=4096, lde=16):
        return lib.lce_pack8(dtype, x, ld, N, d, codes, ldc, exps, lde, None)

    def unpack(dtype=0, out=4096, ld=0, N=10, d=200, codes=4096, ldc=208, exps=4096, lde=16):
        return lib.lce_unpack8(dtype, codes, ldc, exps, lde, N, d, out, ld, None)

    for run, x in ((pack, "x"), (unpack, "out")):
        assert run() in OK and run(N=0, codes=None, exps=None, **{x: None}) in OK
        assert run(dtype=2) == 4 and run(**{x: None}) == 1 and run(codes=None) == 1 and run(exps=None) == 1
        assert run(N=-1) == 2 and run(d=0) == 2 and run(d=1 << 24) == 2 and run(ldc=192) == 2 and run(lde=0) == 2
        assert run(d=204) == 3 and run(ldc=200) == 3 and run(lde=10) == 3 and run(codes=4104) == 3 and run(ld=204) == 3 and run(**{x: 4098}) == 3
    assert pack(ld=8) in OK and unpack(ld=8) == 2   # rows that overlap may be read, not written


def _wg(**kw):
    return _filled(_abi.LceWgrad, ("dy", "codes", "exps", "dw"), dict(T=100, n=64, k=200, ld_codes=208, ld_exps=112), **kw)


def test_weight_gradient_host_checks(lib):
    run = lambda **kw: lib.lce_packed_wgrad(_wg(**kw)[0])  # noqa: E731
    assert lib.lce_packed_wgrad(None) == 1 and run() in OK and run(dw_dtype=1) in OK and run(dtype=1, dw_dtype=1) in OK
    assert run(dtype=2) == 4 and run(dtype=1, dw_dtype=0) == 4 and run(dw_dtype=2) == 4
    for n in ("dy", "codes", "exps", "dw"):
        assert run(**{n: None}) == 1, n
    assert run(T=-1) == 2 and run(n=0) == 2 and run(k=1 << 24) == 2 and run(n=1 << 23, k=1 << 23) == 2 and run(ld_exps=96) == 2
    assert run(n=68) == 3 and run(k=204) == 3 and run(ld_dy=68) == 3 and run(dy=4104) == 3 and run(dw=4104) == 3
    ws = lambda **kw: lib.lce_packed_wgrad_workspace_size(_wg(**kw)[0])  # noqa: E731
    assert ws(n=68) == 0 and ws(T=0) == 0 and ws(T=8192, n=4096, k=4096) == 0
    assert ws(T=16384, n=256, k=256) > 256 * 256 * 4                                            # few tiles: sums of the splits
    assert ws(T=8192, n=4096, k=4096, dtype=1, dw_dtype=1) == 8192 * 4096 * 6                   # fp32: three bf16 parts
    assert run(workspace=4096, workspace_bytes=16, T=16384, n=256, k=256, ld_codes=256, ld_exps=16384) in OK + (6,)


def _rec(**kw):
    return _filled(_abi.LceRecurrence, ("cu", "x", "g", "state", "kept", "h", "final", "dh", "dfinal", "dx", "dg", "dstate"),
                   dict(B=3, T=100, d=64), **kw)


def test_recurrence_host_checks(lib):
    for f in (lib.lce_recurrence_forward, lib.lce_recurrence_backward):
        run = lambda **kw: f(_rec(**kw)[0])  # noqa: E731
        assert f(None) == 1 and run() in OK and run(state=None, dfinal=None, final=None, dstate=None) in OK
        assert run(dtype=2) == 4 and run(x=None) == 1 and run(g=None) == 1
        assert run(T=-1) == 2 and run(T=1 << 30) == 2 and run(B=0) == 2 and run(d=0) == 2 and run(cu=None) == 2 and run(ld_x=56) == 2
        assert run(d=68) == 3 and run(x=4100) == 3 and run(ld_g=68) == 3 and run(state=4100) == 3
        assert run(cu=None, T=99) in OK and run(T=0, x=None, g=None, h=None, dh=None, dx=None, dg=None, kept=None) in OK
    assert lib.lce_recurrence_forward(_rec(kept=None)[0]) in OK and lib.lce_recurrence_forward(_rec(h=None)[0]) == 1
    for n in ("kept", "dh", "dx", "dg"):
        assert lib.lce_recurrence_backward(_rec(**{n: None})[0]) == 1, n


def test_python_refusals():
    """What the Python forms refuse before any address is taken, on tensors without a GPU."""
    import chunked_vocab_cross_gb300 as lce
    x, w = torch.zeros(4, 64), torch.ones(64)
    for call in (lambda: lce.layer_norm_forward(x, weight=w), lambda: lce.layer_norm_backward(None, x, x, weight=w, mean=w, rstd=w),
                 lambda: lce.pack_activation(x), lambda: lce.packed_weight_grad(x, None), lambda: lce.gated_recurrence_forward(x, x),
                 lambda: lce.PackedActivation(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(1, 4, dtype=torch.int8), torch.float32)):
        with pytest.raises(ValueError, match="no CPU path"):
            call()
    with pytest.raises(ValueError, match="one CUDA device"):
        lce.linear_keep8(x, torch.zeros(8, 64))
    with pytest.raises(ValueError, match="int8"):
        lce.PackedActivation(x, x, torch.float32)
