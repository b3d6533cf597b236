"""Host-side refusals of the few-token operators: every bad argument is answered
before anything is launched (no GPU needed)."""
import ctypes
import os
import subprocess

import pytest
import torch

import combine_send_counts_gb300 as ep

P, BAD = 4096, 4098   # never dereferenced: an aligned and a misaligned address


@pytest.fixture(scope="module")
def lib():
    return ep.load()


def test_quantize(lib):
    q = lambda w=P, N=4, K=256, g=64, q=P, s=P, z=None: lib.ep_w4_quantize(w, N, K, g, q, s, z, None)
    for bad in (dict(N=-1), dict(K=0), dict(K=-64), dict(K=100), dict(g=16), dict(g=0), dict(g=256), dict(K=96, g=64),
                dict(w=None), dict(q=None), dict(s=None), dict(w=BAD), dict(q=BAD), dict(s=P + 1)):
        assert q(**bad) == ep.EP_ERR_INVALID_ARG, bad
    assert q(N=0, w=None) == ep.EP_OK


def test_dequantize(lib):
    d = lambda q=P, s=P, z=None, N=4, K=256, g=64, w=P, o=0: lib.ep_w4_dequantize(q, s, z, N, K, g, w, o, None)
    for bad in (dict(N=-1), dict(K=0), dict(K=100), dict(g=16), dict(w=None), dict(q=None), dict(s=None), dict(w=BAD),
                dict(q=BAD), dict(s=P + 1)):
        assert d(**bad) == ep.EP_ERR_INVALID_ARG, bad
    assert d(o=2) == ep.EP_ERR_UNSUPPORTED
    assert d(N=0, w=None) == ep.EP_OK


def test_matvec(lib):
    m = lambda x=P, M=2, q=P, s=P, z=None, N=4, K=256, g=64, y=P, o=0: lib.ep_w4_matvec(x, M, q, s, z, N, K, g, y, o,
                                                                                      None)
    for bad in (dict(M=-1), dict(N=-1), dict(K=0), dict(K=100), dict(g=16), dict(x=None), dict(q=None), dict(s=None),
                dict(y=None), dict(x=BAD), dict(q=BAD), dict(s=P + 1), dict(y=BAD)):
        assert m(**bad) == ep.EP_ERR_INVALID_ARG, bad
    assert m(o=2) == ep.EP_ERR_UNSUPPORTED
    assert m(M=1 << 20) == ep.EP_ERR_UNSUPPORTED
    assert m(N=1 << 31) == ep.EP_ERR_UNSUPPORTED
    assert m(M=0, x=None) == ep.EP_OK
    assert m(N=0, q=None) == ep.EP_OK


def test_router(lib):
    def r(x=P, T=2, H=64, w=P, wd=0, E=8, b=None, K=2, sc=0, n=1, scale=1.0, i=P, o=P, l=None, ws=P, nb=1 << 20):
        return lib.ep_router_topk(x, T, H, w, wd, E, b, K, sc, n, scale, i, o, l, ws, nb, None)
    for bad in (dict(T=-1), dict(H=0), dict(H=60), dict(E=0), dict(E=8193), dict(K=0), dict(K=9), dict(E=64, K=33),
                dict(sc=2), dict(sc=-1), dict(x=None), dict(w=None), dict(i=None), dict(o=None), dict(ws=None),
                dict(x=BAD), dict(w=BAD), dict(ws=P + 16), dict(nb=8)):
        assert r(**bad) == ep.EP_ERR_INVALID_ARG, bad
    assert r(wd=2) == ep.EP_ERR_UNSUPPORTED
    assert r(T=0, x=None) == ep.EP_OK
    assert ep.ep_router_workspace_size(-1, 8, 8) == 0
    assert ep.ep_router_workspace_size(4, 64, 8) >= 4 * 8 * 4


def matrices(fmt=0, group=0, **kw):
    a = dict(data=P, scale=None if fmt == 0 else P, zero=None, format=fmt, group=group)
    a.update(kw)
    return ep.EPMatrix(a["data"], a["scale"], a["zero"], a["format"], a["group"])


def moe(lib, a=None, b=None, x=P, i=P, w=P, T=2, K=2, H=64, I=64, E=8, El=4, r=1, out=P, o=0, ws=P, nb=1 << 20):
    a, b = a or matrices(), b or matrices()
    return lib.ep_moe_decode(x, i, w, T, K, H, I, E, El, r, ctypes.byref(a), ctypes.byref(b), out, o, ws, nb, None,
                             None)


def test_moe(lib):
    for bad in (dict(T=-1), dict(K=0), dict(K=33), dict(H=0), dict(H=60), dict(I=0), dict(I=60), dict(E=0),
                dict(E=8193, El=1), dict(El=0), dict(El=3), dict(r=-1), dict(r=2), dict(x=None), dict(i=None),
                dict(w=None), dict(out=None), dict(ws=None), dict(x=BAD), dict(out=BAD), dict(ws=P + 16), dict(nb=64),
                dict(a=matrices(data=None)), dict(b=matrices(data=BAD)), dict(a=matrices(scale=P)),
                dict(b=matrices(zero=P)), dict(a=matrices(1, 16), b=matrices(1, 16)),
                dict(a=matrices(1, 128), b=matrices(1, 128)),                      # 128 does not divide 64
                dict(a=matrices(1, 32, scale=None), b=matrices(1, 32)), dict(a=matrices(1, 32, scale=P + 1),
                                                                             b=matrices(1, 32))):
        assert moe(lib, **bad) == ep.EP_ERR_INVALID_ARG, bad
    for bad in (dict(o=2), dict(a=matrices(2), b=matrices(2)), dict(a=matrices(1, 32)), dict(b=matrices(1, 32)),
                dict(a=matrices(1, 32), b=matrices(1, 64)), dict(T=513), dict(H=1 << 20), dict(I=1 << 20)):
        assert moe(lib, **bad) == ep.EP_ERR_UNSUPPORTED, bad
    assert moe(lib, T=0, x=None) == ep.EP_OK
    assert lib.ep_moe_decode(P, P, P, 2, 2, 64, 64, 8, 4, 1, None, None, P, 0, P, 1 << 20, None, None) \
        == ep.EP_ERR_INVALID_ARG
    assert ep.ep_moe_workspace_size(4, 2, 64, 64) > 0 and ep.ep_moe_workspace_size(4, 0, 64, 64) == 0
    with pytest.raises(ep.EPError, match="EP_ERR_UNSUPPORTED"):
        ep._check(moe(lib, T=513), "moe")


def test_matrix_struct_matches_the_header(tmp_path):
    import shutil
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    names = [n for n, _ in ep.EPMatrix._fields_]
    src = tmp_path / "probe.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "ep.h"\nint main(void) {'
                   'printf("%zu", sizeof(ep_matrix));'
                   + "".join(f'printf(" %zu", offsetof(ep_matrix, {n}));' for n in names)
                   + 'printf(" %d %d %d %d %d", EP_W_BF16, EP_W_INT4, EP_SCORE_SOFTMAX, EP_SCORE_SIGMOID, '
                     'EP_MOE_MAX_SLOTS); return 0; }')
    subprocess.run([cc, "-I", inc, str(src), "-o", str(tmp_path / "probe")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "probe")], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [ctypes.sizeof(ep.EPMatrix)] + [getattr(ep.EPMatrix, n).offset for n in names] + \
        [ep.EP_W_BF16, ep.EP_W_INT4, ep.EP_SCORE_SOFTMAX, ep.EP_SCORE_SIGMOID, ep.EP_MOE_MAX_SLOTS]


def w4(lead=(4,), N=8, K=64, group=32, **kw):
    a = dict(q=torch.zeros((*lead, N, K // 2), dtype=torch.uint8),
             scale=torch.zeros((*lead, N, K // group), dtype=torch.bfloat16), zero=None, group=group)
    a.update(kw)
    return ep.W4(a["q"], a["scale"], a["zero"], a["group"])


def test_w4_container():
    w = w4(zero=torch.zeros((4, 8, 2), dtype=torch.uint8))
    assert w.shape == (4, 8, 64) and w[1].shape == (8, 64)
    with pytest.raises(IndexError):
        w[1][0]
    with pytest.raises(TypeError, match="q must be torch.uint8"):
        w4(q=torch.zeros((4, 8, 32)))
    with pytest.raises(TypeError, match="scale must be torch.bfloat16"):
        w4(scale=torch.zeros((4, 8, 2)))
    with pytest.raises(TypeError, match="zero must be torch.uint8"):
        w4(zero=torch.zeros((4, 8, 2)))
    for bad in (dict(group=16), dict(scale=torch.zeros((4, 8, 1), dtype=torch.bfloat16)),
                dict(zero=torch.zeros((4, 8, 1), dtype=torch.uint8)),
                dict(q=torch.zeros((4, 8, 40), dtype=torch.uint8)),
                dict(q=torch.zeros((4, 32, 8), dtype=torch.uint8).transpose(1, 2))):
        with pytest.raises(ValueError):
            w4(**bad)


def test_helpers_refuse_wrong_tensors():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="x must be torch.bfloat16"):
        ep.w4_matvec(x.float(), w4(()))
    with pytest.raises(ValueError, match="shape"):
        ep.w4_matvec(x[:, :32], w4(()))
    with pytest.raises(ValueError, match="one matrix"):
        ep.w4_matvec(x, w4())
    with pytest.raises(ValueError, match="device tensor"):
        ep.w4_matvec(x, w4(()))
    with pytest.raises(TypeError, match="w must be torch.bfloat16"):
        ep.w4_quantize(x.float())
    with pytest.raises(ValueError, match="matrix"):
        ep.w4_quantize(x[0])
    with pytest.raises(TypeError, match="out_dtype"):
        ep.w4_dequantize(w4(), torch.float16)
    with pytest.raises(TypeError, match="w must be torch.bfloat16 or torch.float32"):
        ep.RouterTopk(x.half(), 1)
    with pytest.raises(ValueError, match="scoring"):
        ep.RouterTopk(x, 1, scoring="tanh")
    with pytest.raises(TypeError, match="both"):
        ep.MoeDecode(w4(), x, topk=1)
    with pytest.raises(ValueError, match="stacks"):
        ep.MoeDecode(x, x, topk=1)
    with pytest.raises(ValueError, match="belong together"):
        ep.MoeDecode(w4(N=8, K=64), w4(N=32, K=32), topk=1)
    with pytest.raises(ValueError, match="at most 1024"):
        ep.MoeDecode(w4(N=64, K=64), w4(N=64, K=32), topk=8, max_tokens=129)
