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


def test_scan_refusals():
    lib = dfssm.lib()

    def dims(**kw):
        a = dict(nheads=4, ngroups=2, headdim=64, d_state=128)
        a.update(kw)
        return dfssm.ScanDims(a["nheads"], a["ngroups"], a["headdim"], a["d_state"])

    def ins(**kw):
        a = dict(x=A, x_stride=256, b=A, b_stride=256, c=A, c_stride=256, dt=A, dt_stride=4, dt_bias=A, a_log=A, d_skip=A,
                 init_state=A, cu_seqlens=A)
        a.update(kw)
        return dfssm.ScanInputs(*a.values())

    def grads(**kw):
        a = dict(dx=A, dx_stride=256, db=A, db_stride=256, dc=A, dc_stride=256, ddt=A, ddt_stride=4, ddt_bias=A, da_log=A,
                 dd_skip=A, dinit_state=A)
        a.update(kw)
        return dfssm.ScanGrads(*a.values())

    size = {b: dfssm.dfssm_ssm_scan_workspace_bytes(dims(), 100, 3, b) for b in (False, True)}

    def fwd(d=None, i=None, **kw):
        a = dict(total=100, nseq=3, y=A, ld=256, fin=A, ws=A, n=size[False])
        a.update(kw)
        return lib.dfssm_ssm_scan_fwd(d or dims(), i or ins(), a["total"], a["nseq"], a["y"], a["ld"], a["fin"], a["ws"],
                                      a["n"], None)

    def bwd(d=None, i=None, gr=None, **kw):
        a = dict(total=100, nseq=3, dy=A, ld=256, dfin=A, ws=A, n=size[True])
        a.update(kw)
        return lib.dfssm_ssm_scan_bwd(d or dims(), i or ins(), a["total"], a["nseq"], a["dy"], a["ld"], a["dfin"],
                                      gr or grads(), a["ws"], a["n"], None)

    for call in (fwd, bwd):
        for bad in (dict(headdim=32), dict(d_state=64), dict(nheads=0), dict(nheads=1025, ngroups=1), dict(ngroups=3),
                    dict(ngroups=0)):
            assert call(dims(**bad)) == SHAPE, bad
        for bad in (dict(total=0), dict(total=(1 << 22) + 1), dict(nseq=0), dict(nseq=65537)):
            assert call(**bad) == SHAPE, bad
        for bad in (dict(x=None), dict(x=A + 8), dict(x_stride=255), dict(x_stride=248), dict(x_stride=260), dict(b=None),
                    dict(b=A + 2), dict(b_stride=128), dict(c=None), dict(c_stride=1 << 31), dict(dt=None), dict(dt=A + 1),
                    dict(dt_stride=3), dict(dt_bias=None), dict(a_log=A + 2), dict(d_skip=None), dict(init_state=A + 4),
                    dict(cu_seqlens=None), dict(cu_seqlens=A + 2)):
            assert call(i=ins(**bad)) == ARG, bad
        for bad in (dict(ld=248), dict(ld=260), dict(ws=None), dict(ws=A + 16), dict(n=0)):
            assert call(**bad) == ARG, bad
    for bad in (dict(y=None), dict(y=A + 8), dict(fin=A + 8), dict(n=size[False] - 1)):
        assert fwd(**bad) == ARG, bad
    for bad in (dict(dy=None), dict(dy=A + 8), dict(dfin=A + 4), dict(n=size[True] - 1)):
        assert bwd(**bad) == ARG, bad
    for bad in (dict(dx=None), dict(dx=A + 8), dict(dx_stride=264 + 1), dict(db=None), dict(db_stride=192), dict(dc=None),
                dict(dc=A + 4), dict(ddt=None), dict(ddt=A + 1), dict(ddt_stride=3), dict(ddt_bias=None), dict(da_log=None),
                dict(dd_skip=A + 2), dict(dinit_state=A + 8)):
        assert bwd(gr=grads(**bad)) == ARG, bad
    assert lib.dfssm_ssm_scan_fwd(None, ins(), 100, 3, A, 256, A, A, size[False], None) == ARG
    assert lib.dfssm_ssm_scan_fwd(dims(), None, 100, 3, A, 256, A, A, size[False], None) == ARG
    assert lib.dfssm_ssm_scan_workspace_bytes(dims(), 100, 3, 0, None) == ARG


def test_scan_struct_layout_matches_c(tmp_path):
    import ctypes
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "%s"\n'
                    'int main(void) { printf("%%zu %%zu %%zu %%zu %%zu\\n", sizeof(dfssm_scan_dims), sizeof(dfssm_scan_inputs),'
                    ' sizeof(dfssm_scan_grads), offsetof(dfssm_scan_inputs, cu_seqlens),'
                    ' offsetof(dfssm_scan_grads, dinit_state)); return 0; }' % os.path.join(root, "include", "dfssm.h"))
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c99", "-o", str(exe), str(prog)])
    got = [int(v) for v in subprocess.check_output([str(exe)]).split()]
    assert got == [ctypes.sizeof(dfssm.ScanDims), ctypes.sizeof(dfssm.ScanInputs), ctypes.sizeof(dfssm.ScanGrads),
                   dfssm.ScanInputs.cu_seqlens.offset, dfssm.ScanGrads.dinit_state.offset]
