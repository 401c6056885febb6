"""Refusals of the sequence operators: argument checks that return before any CUDA call."""
import bit_gemv_gemm_dfssm_b200 as dfssm

A = 1 << 20          # a 16-byte aligned address that is never followed
SHAPE, ARG = dfssm.DFSSM_ERR_UNSUPPORTED_SHAPE, dfssm.DFSSM_ERR_INVALID_ARG


def test_norm_quant_refusals():
    lib = dfssm.lib()

    def call(**kw):
        a = dict(w=A, d=2048, eps=1e-5, rin=A, delta=A, ddt=dfssm.DFSSM_BF16, m=1, rout=A, q=A, sx=A, val=A)
        a.update(kw)
        return lib.dfssm_add_rmsnorm_quant(a["w"], a["d"], a["eps"], a["rin"], a["delta"], a["ddt"], a["m"], a["rout"],
                                           a["q"], a["sx"], a["val"], None)

    for bad in (dict(d=2044), dict(d=0), dict(d=8200), dict(m=0), dict(m=65537), dict(m=-1)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(w=None), dict(rin=A + 4), dict(delta=A + 8), dict(rout=None), dict(q=None), dict(q=A + 8),
                dict(sx=None), dict(sx=A + 4), dict(val=A + 2), dict(eps=-1.0), dict(eps=float("nan")),
                dict(ddt=dfssm.DFSSM_I8)):
        assert call(**bad) == ARG, bad


def test_norm_bwd_refusals():
    lib = dfssm.lib()
    need = dfssm.dfssm_add_rmsnorm_bwd_workspace_bytes(2048, 9)
    assert need >= 4 * 2048

    def call(**kw):
        a = dict(w=A, d=2048, eps=1e-5, r=A, dout=A, kind=dfssm.DFSSM_F32, ds=A, m=9, dr=A, dw=A, ws=A, n=need)
        a.update(kw)
        return lib.dfssm_add_rmsnorm_bwd(a["w"], a["d"], a["eps"], a["r"], a["dout"], a["kind"], a["ds"], a["m"],
                                         a["dr"], a["dw"], a["ws"], a["n"], None)

    for bad in (dict(d=12), dict(d=8200), dict(m=0), dict(m=65537)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(w=None), dict(r=None), dict(r=A + 8), dict(dout=None), dict(dout=A + 2), dict(ds=A + 4),
                dict(dr=None), dict(dw=A + 4), dict(ws=None), dict(ws=A + 4), dict(n=need - 1), dict(n=0),
                dict(eps=float("inf")), dict(kind=dfssm.DFSSM_I8)):
        assert call(**bad) == ARG, bad
    assert lib.dfssm_add_rmsnorm_bwd_workspace_bytes(2048, 9, None) == ARG


def test_xent_refusals():
    lib = dfssm.lib()

    def table(**kw):
        a = dict(table=A, scale=A, vocab=1000, d=256)
        a.update(kw)
        return dfssm.Int8Table(a["table"], a["scale"], a["vocab"], a["d"])

    size = {b: dfssm.dfssm_xent_workspace_bytes(table(), 5, b) for b in (False, True)}

    def fwd(t=None, **kw):
        a = dict(q=A, sx=A, tg=A, m=5, nll=A, lse=A, ws=A, n=size[False])
        a.update(kw)
        return lib.dfssm_xent_fwd(t or table(), a["q"], a["sx"], a["tg"], a["m"], a["nll"], a["lse"], a["ws"], a["n"],
                                  None)

    def bwd(t=None, **kw):
        a = dict(q=A, sx=A, tg=A, lse=A, grad=A, m=5, dh=A, ws=A, n=size[True])
        a.update(kw)
        return lib.dfssm_xent_bwd(t or table(), a["q"], a["sx"], a["tg"], a["lse"], a["grad"], a["m"], a["dh"], a["ws"],
                                  a["n"], None)

    for call in (fwd, bwd):
        for bad in (dict(d=8), dict(d=264), dict(d=8208), dict(vocab=0), dict(vocab=(1 << 24) + 1)):
            assert call(table(**bad)) == SHAPE, bad
        for bad in (dict(table=None), dict(scale=None), dict(table=A + 8), dict(scale=A + 4)):
            assert call(table(**bad)) == ARG, bad
        for m in (0, -3, 65537):
            assert call(m=m) == SHAPE
        for bad in (dict(q=None), dict(q=A + 8), dict(sx=None), dict(sx=A + 2), dict(tg=None), dict(tg=A + 1),
                    dict(lse=None), dict(ws=None), dict(ws=A + 16), dict(n=0)):
            assert call(**bad) == ARG, bad
    assert fwd(n=size[False] - 1) == ARG and fwd(nll=None) == ARG
    assert bwd(n=size[True] - 1) == ARG and bwd(dh=None) == ARG and bwd(dh=A + 8) == ARG and bwd(grad=None) == ARG
    assert lib.dfssm_xent_workspace_bytes(table(), 5, 0, None) == ARG
