"""Refusals of the operators around the long convolution, on the CPU: the C ABI
before any HIP call, and the Python checks before the library. No call here
reaches a GPU."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIBPATH = os.path.join(ROOT, "subquadratic_sequence_amd", "libhyena.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIBPATH), reason="libhyena.so not built")

OK, INVALID, UNSUPPORTED, WORKSPACE, HIP = 0, 1, 2, 3, 5
INT_MAX, INT_MIN = 2 ** 31 - 1, -2 ** 31


@pytest.fixture(scope="module")
def hy():
    from subquadratic_sequence_amd import hyena
    return hyena


@pytest.fixture(scope="module")
def p():
    buf = ctypes.create_string_buffer(128)
    addr = (ctypes.addressof(buf) + 63) // 64 * 64
    p.keep = buf
    return addr


def done(st):
    """What a call with valid arguments returns: it reaches HIP, which has no device here."""
    return st == HIP


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="valid calls would run")


# ------------------------------------------------- gated linear recurrence


def test_glr_sizes(hy):
    L = hy.lib()
    for f in (L.hyena_glr_workspace_bytes, L.hyena_glr_bwd_workspace_bytes):
        assert f(1, 1, 8, 0) > 0 and f(2, 1 << 20, 256, 1) > 0 and f(1 << 20, 1, 8, 1) > 0
        for bad in [(0, 4, 8, 0), (-1, 4, 8, 0), (1, 0, 8, 0), (1, -5, 8, 0), (1, (1 << 24) + 1, 8, 0), (1, 4, 0, 0),
                    (1, 4, 12, 0), (1, 4, 65544, 0), (1, 4, 8, 2), (1, 4, 8, -1), ((1 << 20) + 1, 4, 8, 0),
                    (1 << 20, 4, 4096, 0), (1 << 10, 1 << 24, 1 << 10, 0), (INT_MAX, INT_MAX, INT_MAX, 0),
                    (INT_MIN, INT_MIN, INT_MIN, 1)]:
            assert f(*bad) == 0, bad
    # a sequence that one workgroup per 64 channels walks alone needs no aggregates
    assert L.hyena_glr_workspace_bytes(1024, 4096, 64, 1) == 256
    assert L.hyena_glr_bwd_workspace_bytes(1, 1000, 64, 1) > 1000 // 64 * 64 * 8


def glr(hy, p, **kw):
    d = dict(B=2, L=5, D=16, dtype=1, v=p, f=p, g=p, v_batch=80, v_row=16, f_batch=80, f_row=16, g_batch=80, g_row=16,
             bias=p, h0=p, reset=p, lens=p, pad_zero=0)
    d.update(kw)
    return ctypes.byref(hy.GlrInputs(*(d[k] for k, _ in hy.GlrInputs._fields_)))


BAD_GLR = [(dict(dtype=2), INVALID), (dict(v=None), INVALID), (dict(f=None), INVALID), (dict(B=0), INVALID),
           (dict(L=0), UNSUPPORTED), (dict(D=12), UNSUPPORTED), (dict(v_row=12), INVALID), (dict(v_row=-16), INVALID),
           (dict(f_batch=4), INVALID), (dict(g_row=-8), INVALID), (dict(v_batch=1 << 40), INVALID)]


@pytest.mark.parametrize("kw,st", BAD_GLR)
def test_glr_inputs_are_refused(hy, p, kw, st):
    L = hy.lib()
    assert L.hyena_glr_fwd(glr(hy, p, **kw), p, 80, 16, p, p, 1 << 30, None) == st
    assert L.hyena_glr_bwd(glr(hy, p, **kw), p, 80, 16, p, p, p, p, 80, 16, p, p, p, 1 << 30, None) == st


def test_glr_outputs_are_refused(hy, p):
    L = hy.lib()
    need, bneed = L.hyena_glr_workspace_bytes(2, 5, 16, 1), L.hyena_glr_bwd_workspace_bytes(2, 5, 16, 1)
    a = glr(hy, p)
    assert L.hyena_glr_fwd(None, p, 80, 16, p, p, need, None) == INVALID
    for y, yb, yr, hl, ws, n, st in [(None, 80, 16, p, p, need, INVALID), (p + 8, 80, 16, p, p, need, INVALID),
                                     (p, 80, 8, p, p, need, INVALID), (p, 72, 16, p, p, need, INVALID),
                                     (p, 80, 20, p, p, need, INVALID), (p, 0, 16, p, p, need, INVALID),
                                     (p, 80, 16, p + 4, p, need, INVALID), (p, 80, 16, p, None, need, INVALID),
                                     (p, 80, 16, p, p, need - 1, WORKSPACE)]:
        assert L.hyena_glr_fwd(a, y, yb, yr, hl, ws, n, None) == st
    args = dict(dy=p, dyb=80, dyr=16, dhl=p, dv=p, df=p, dg=p, db=80, dr=16, dbias=p, dh0=p, ws=p, n=bneed)
    for kw, st in [(dict(dy=None), INVALID), (dict(dv=None), INVALID), (dict(df=p + 2), INVALID),
                   (dict(dg=None), INVALID), (dict(dr=8), INVALID), (dict(db=64), INVALID), (dict(dyr=-16), INVALID),
                   (dict(dbias=p + 4), INVALID), (dict(dh0=p + 4), INVALID), (dict(n=bneed - 1), WORKSPACE)]:
        assert L.hyena_glr_bwd(a, *{**args, **kw}.values(), None) == st, kw
    # dg without g
    assert L.hyena_glr_bwd(glr(hy, p, g=None), *args.values(), None) == INVALID


@no_gpu
def test_glr_valid_calls_reach_hip(hy, p):
    L = hy.lib()
    n = 1 << 20
    assert done(L.hyena_glr_fwd(glr(hy, p), p, 80, 16, p, p, n, None))
    assert done(L.hyena_glr_fwd(glr(hy, p, g=None, bias=None, h0=None, reset=None, lens=None), p, 80, 16, None, p, n, None))
    assert done(L.hyena_glr_fwd(glr(hy, p, v_row=0, v_batch=0), p, 80, 16, p, p, n, None))
    assert done(L.hyena_glr_fwd(glr(hy, p, reset=p + 1), p, 80, 16, p, p, n, None))  # bytes: any address
    assert done(L.hyena_glr_bwd(glr(hy, p), p, 80, 16, None, p, p, p, 80, 16, None, None, p, n, None))
    assert done(L.hyena_glr_step(2, 16, 2, 1, p, 16, p, 16, p, 16, p, None, p, p, p, 16, 0, None))


def test_glr_step_is_refused(hy, p):
    L = hy.lib()
    good = dict(B=2, D=16, S=4, dtype=1, v=p, vr=16, f=p, fr=16, g=p, gr=16, bias=p, slots=p, state=p, out=p, y=p, yr=16,
                pz=0)
    for kw, st in [(dict(B=0), INVALID), (dict(S=0), INVALID), (dict(dtype=3), INVALID), (dict(v=None), INVALID),
                   (dict(state=None), INVALID), (dict(out=p + 8), INVALID), (dict(y=None), INVALID),
                   (dict(slots=p + 1), INVALID), (dict(bias=p + 4), INVALID), (dict(vr=4), INVALID),
                   (dict(yr=8), INVALID), (dict(B=8193), UNSUPPORTED), (dict(D=20), UNSUPPORTED),
                   (dict(S=(1 << 24) + 1), UNSUPPORTED), (dict(slots=None, S=1), INVALID)]:
        assert L.hyena_glr_step(*{**good, **kw}.values(), None) == st, kw


# ---------------------------------------------- gated feed-forward block


def test_ffn_sizes_and_refusals(hy, p):
    L = hy.lib()
    for f in (L.hyena_ffn_workspace_bytes, L.hyena_ffn_bwd_workspace_bytes):
        assert f(1, 8, 8, 0) > 0 and f(1 << 24, 8, 65536, 1) > 0
        for bad in [(0, 8, 8, 0), ((1 << 24) + 1, 8, 8, 0), (1, 4, 8, 0), (1, 8, 12, 0), (1, 65544, 8, 0), (1, 8, 65544, 0),
                    (1, 8, 8, 2), (INT_MAX, INT_MAX, INT_MAX, 0), (INT_MIN, 8, 8, 1)]:
            assert f(*bad) == 0, bad
    n, b = L.hyena_ffn_workspace_bytes(3, 16, 24, 1), L.hyena_ffn_bwd_workspace_bytes(3, 16, 24, 1)
    fwd = dict(M=3, D=16, F=24, dtype=1, act=1, x=p, wi=p, wo=p, y=p, ws=p, n=n)
    bwd = dict(M=3, D=16, F=24, dtype=1, act=1, x=p, wi=p, wo=p, dy=p, dx=p, dwi=p, dwo=p, ws=p, n=b)
    for call, good in ((L.hyena_ffn_fwd, fwd), (L.hyena_ffn_bwd, bwd)):
        for kw, st in [(dict(M=0), INVALID), (dict(dtype=-1), INVALID), (dict(act=3), INVALID), (dict(act=-1), INVALID),
                       (dict(x=None), INVALID), (dict(wi=p + 8), INVALID), (dict(wo=None), INVALID),
                       (dict(ws=None), INVALID), (dict(D=20), UNSUPPORTED), (dict(F=0), UNSUPPORTED),
                       (dict(n=good["n"] - 1), WORKSPACE)]:
            assert call(*{**good, **kw}.values(), None) == st, kw
    for kw in (dict(dy=None), dict(dx=p + 2), dict(dwi=None), dict(dwo=None)):
        assert L.hyena_ffn_bwd(*{**bwd, **kw}.values(), None) == INVALID, kw
    if not torch.cuda.is_available():
        assert done(L.hyena_ffn_fwd(*fwd.values(), None)) and done(L.hyena_ffn_bwd(*bwd.values(), None))


# ------------------------------------------------ group norm, channels last


def test_group_norm_sizes_and_refusals(hy, p):
    L = hy.lib()
    for f in (L.hyena_group_norm_workspace_bytes, L.hyena_group_norm_bwd_workspace_bytes):
        assert f(1, 1, 8, 1, 0) > 0 and f(1 << 24, 1, 64, 64, 1) > 0 and f(2, 1 << 24, 8192, 8192, 1) > 0
        for bad in [(0, 1, 8, 1, 0), (1, 0, 8, 1, 0), (1, 1, 12, 1, 0), (1, 1, 8200, 1, 0), (1, 1, 8, 3, 0), (1, 1, 8, 0, 0),
                    (1, 1, 8, 16, 0), (1, 1, 8, -1, 0), (1, 1, 8, 1, 2), ((1 << 24) + 1, 1, 8, 1, 0),
                    (1, (1 << 24) + 1, 8, 1, 0), (1 << 24, 1, 128, 1, 0), (1 << 12, 1 << 24, 64, 1, 0),
                    (INT_MAX, INT_MAX, INT_MAX, INT_MAX, 0), (INT_MIN, INT_MIN, INT_MIN, INT_MIN, 0)]:
            assert f(*bad) == 0, bad
    n, b = L.hyena_group_norm_workspace_bytes(2, 9, 24, 4, 0), L.hyena_group_norm_bwd_workspace_bytes(2, 9, 24, 4, 0)
    fwd = dict(B=2, S=9, C=24, G=4, dtype=0, act=0, eps=1e-5, x=p, ga=p, be=p, lens=p, pz=0, y=p, mean=p, rstd=p, ws=p, n=n)
    bwd = dict(B=2, S=9, C=24, G=4, dtype=0, act=0, x=p, dy=p, ga=p, be=p, lens=p, mean=p, rstd=p, dx=p, dga=p, dbe=p, ws=p,
               n=b)
    for call, good in ((L.hyena_group_norm_fwd, fwd), (L.hyena_group_norm_bwd, bwd)):
        for kw, st in [(dict(B=0), INVALID), (dict(dtype=2), INVALID), (dict(act=5), INVALID), (dict(x=None), INVALID),
                       (dict(ga=p + 4), INVALID), (dict(lens=p + 2), INVALID), (dict(rstd=p + 4), INVALID),
                       (dict(ws=p + 8), INVALID), (dict(G=5), UNSUPPORTED), (dict(C=20, G=4), UNSUPPORTED),
                       (dict(S=0), UNSUPPORTED), (dict(n=good["n"] - 1), WORKSPACE)]:
            assert call(*{**good, **kw}.values(), None) == st, kw
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert L.hyena_group_norm_fwd(*{**fwd, "eps": eps}.values(), None) == INVALID
    for kw in (dict(mean=None), dict(rstd=None), dict(dy=None), dict(dx=None), dict(dga=p + 4)):
        assert L.hyena_group_norm_bwd(*{**bwd, **kw}.values(), None) == INVALID, kw
    if not torch.cuda.is_available():
        for kw in (dict(), dict(ga=None, be=None, lens=None, mean=None, rstd=None)):
            assert done(L.hyena_group_norm_fwd(*{**fwd, **kw}.values(), None))
        for kw in (dict(), dict(ga=None, be=None, lens=None, dga=None, dbe=None)):
            assert done(L.hyena_group_norm_bwd(*{**bwd, **kw}.values(), None))


# ------------------------------------------------------------ Python checks


def test_python_checks():
    import subquadratic_sequence_amd as hs
    t = torch.zeros
    x = t(2, 5, 16)
    bad = [
        (ValueError, lambda: hs.hyena_glr_fwd(t(5, 16), t(5, 16))),
        (ValueError, lambda: hs.hyena_glr_fwd(x, t(2, 4, 16))),
        (TypeError, lambda: hs.hyena_glr_fwd(x, x.bfloat16())),
        (TypeError, lambda: hs.hyena_glr_fwd(x.half(), x.half())),
        (TypeError, lambda: hs.hyena_glr_fwd(x, None)),
        (ValueError, lambda: hs.hyena_glr_fwd(x, t(2, 16, 5).transpose(1, 2))),
        (ValueError, lambda: hs.hyena_glr_fwd(x, x, bias=t(15))),
        (TypeError, lambda: hs.hyena_glr_fwd(x, x, bias=t(16).double())),
        (ValueError, lambda: hs.hyena_glr_fwd(x, x, h0=t(16, 2).t())),
        (TypeError, lambda: hs.hyena_glr_fwd(x, x, lens=t(2, dtype=torch.int64))),
        (TypeError, lambda: hs.hyena_glr_fwd(x, x, reset=t(2, 5))),
        (ValueError, lambda: hs.hyena_glr_fwd(x, x)),  # not on a GPU
        (ValueError, lambda: hs.hyena_glr_bwd(x, x, x, dh_last=t(2, 15))),
        (ValueError, lambda: hs.hyena_glr_bwd(x, x, x, dp=t(2, 5, 48))),
        (ValueError, lambda: hs.hyena_glr_step(t(4, 16), t(2, 5, 16), t(2, 5, 16))),
        (ValueError, lambda: hs.hyena_glr_step(t(4, 8), t(2, 16), t(2, 16))),
        (TypeError, lambda: hs.hyena_glr_step(t(4, 16), t(2, 16), t(2, 16), slots=t(2))),
        (ValueError, lambda: hs.hyena_ffn_fwd(x, t(16, 48), t(23, 16))),
        (TypeError, lambda: hs.hyena_ffn_fwd(x, t(16, 48).bfloat16(), t(24, 16))),
        (ValueError, lambda: hs.hyena_ffn_fwd(x, t(48, 16).t(), t(24, 16))),
        (TypeError, lambda: hs.hyena_ffn_fwd(x, None, t(24, 16))),
        (ValueError, lambda: hs.hyena_ffn_fwd(x, t(16, 48), t(24, 16))),
        (TypeError, lambda: hs.hyena_ffn_bwd(x, t(16, 48), t(24, 16), None)),
        (ValueError, lambda: hs.hyena_ffn_bwd(x, t(16, 48), t(24, 16), t(2, 5, 8))),
        (ValueError, lambda: hs.hyena_group_norm_fwd(t(16), 4)),
        (ValueError, lambda: hs.hyena_group_norm_fwd(x, 4, gamma=t(8))),
        (ValueError, lambda: hs.hyena_group_norm_fwd(x, 4, mean=t(2, 3))),
        (ValueError, lambda: hs.hyena_group_norm_fwd(t(2, 16, 5).transpose(1, 2), 4)),
        (ValueError, lambda: hs.hyena_group_norm_fwd(x, 4)),
        (ValueError, lambda: hs.hyena_group_norm_bwd(x, x, 4, None, None)),
        (ValueError, lambda: hs.hyena_group_norm_bwd(x, t(2, 5, 8), 4, t(2, 4), t(2, 4))),
    ]
    for i, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            raise AssertionError(f"case {i} was not refused")


def test_outputs_that_are_inputs_are_refused():
    import subquadratic_sequence_amd as hs
    x, h = torch.zeros(2, 5, 16), torch.zeros(2, 16)
    for kw, what in [(dict(h0=h, h_last=h), "h_last may not be h0"), (dict(y=x), "y may not be v")]:
        with pytest.raises(ValueError, match=what):
            hs.hyena_glr_fwd(x, x.clone(), **kw)


def test_unsupported_sizes_raise_the_status():
    from subquadratic_sequence_amd import HyenaError, block
    for query, sizes in [("hyena_glr_workspace_bytes", (1, 4, 12, 0)), ("hyena_ffn_workspace_bytes", (1, 12, 8, 0)),
                         ("hyena_group_norm_workspace_bytes", (1, 1, 16, 3, 0))]:
        with pytest.raises(HyenaError) as e:
            block._need(query, *sizes)
        assert e.value.status == UNSUPPORTED
