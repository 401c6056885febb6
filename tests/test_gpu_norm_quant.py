"""Residual add + RMS norm with an int8 output, and the norm's gradient, on the GPU against 64 bits.

Tolerances. o is r_new times the factor times w: two products of at most half a step of 2^-24
each, and the factor's error. The sum of squares is an fmaf chain and a tree over at most 8192
terms, all of one sign: a thread adds at most 32 in order and the rest in at most 13 levels, so
its relative error is below 45 2^-24, the factor's below 24 2^-24 (half of it, two more
roundings), and o's below 27 2^-24 < 2^-19 relative. sx is |o| of one element over 127 (one more
rounding): 2^-18. The quantiser's argument x inv is at most 127, off by at most 127 2^-18 < 2^-11
from its 64-bit value, so q may differ by one step only where that value is within 2^-11 of a
midpoint; elsewhere it is equal. val is bf16(sx q): half a step (2^-9 relative to the value's
binade, 2^-8 of the value at most) around sx q, itself off by 2^-18.

The gradient: f g - f^3 c r with c = sum(g r)/d. The terms of c have both signs: its error is
bounded by 45 2^-24 sum|g r|/d. dresid's error is then below 2^-18 (|f g| + f^3 |r| (sum|g r|/d +
|c|) + |dstream|) elementwise; dnorm_w adds m terms (chains of at most ceil(m/444) rows per CTA,
then up to 14 in order and 32 more; m <= 65536) with |error| < (m/444 + 47) 2^-24 sum|dout r f| <
(m/592 + 120) 2^-24 sum|dout r f| for each column.
"""
import numpy as np
import pytest
import torch

import bit_gemv_gemm_dfssm_b200 as dfssm

pytestmark = pytest.mark.gpu
BF16, F32 = dfssm.DFSSM_BF16, dfssm.DFSSM_F32
KIND = {torch.bfloat16: BF16, torch.float32: F32}


def stream():
    return torch.cuda.current_stream().cuda_stream


def ptr(t):
    return 0 if t is None else t.data_ptr()


def inputs(seed, m, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = torch.randn(m, d, device="cuda", generator=g) * (torch.rand(m, 1, device="cuda", generator=g) * 20 + 0.05)
    w = torch.rand(d, device="cuda", generator=g) + 0.5
    x = None if dtype is None else torch.randn(m, d, device="cuda", generator=g).to(dtype)
    return r, w, x, g


def run_q8(r, w, delta, eps, val=True, resid_out=None):
    m, d = r.shape
    ro = torch.full_like(r, float("nan")) if resid_out is None else resid_out
    q = torch.full((m, d), 99, dtype=torch.int8, device="cuda")
    sx = torch.full((m,), float("nan"), device="cuda")
    v = torch.full((m, d), float("nan"), dtype=torch.bfloat16, device="cuda") if val else None
    dfssm.dfssm_add_rmsnorm_quant(ptr(w), d, eps, ptr(r), ptr(delta), KIND[delta.dtype] if delta is not None else BF16, m,
                               ptr(ro), ptr(q), ptr(sx), ptr(v), stream())
    torch.cuda.synchronize()
    return ro, q, sx, v


def check_q8(r, w, delta, eps, got):
    ro, q, sx, v = got
    rn = r if delta is None else r + delta.float()               # one IEEE addition
    assert torch.equal(ro, rn)
    x = rn.double()
    o = x / (x.square().mean(1, keepdim=True) + eps).sqrt() * w.double()
    amax = o.abs().amax(1)
    assert ((sx.double() - amax / 127).abs() <= 2.0 ** -18 * amax / 127).all()
    arg = torch.where(amax[:, None] > 0, o * 127 / amax[:, None].clamp(min=1e-300), torch.zeros_like(o))
    want = torch.round(arg)
    far = (arg - want).abs() < 0.5 - 2.0 ** -11
    assert torch.equal(q.double()[far], want[far])
    assert ((q.double() - arg).abs() <= 0.5 + 2.0 ** -11).all()
    if v is not None:
        assert torch.equal(v, (q.float() * sx[:, None]).to(torch.bfloat16))    # one product, one rounding


@pytest.mark.parametrize("m,d,dtype", [(1, 2048, torch.bfloat16), (3, 8, None), (37, 64, torch.float32),
                                       (33, 72, torch.bfloat16), (9, 256, torch.float32), (17, 264, None),
                                       (5, 512, torch.bfloat16), (8, 1024, torch.bfloat16), (2, 1032, torch.float32),
                                       (7, 2056, torch.bfloat16), (4, 4096, None), (3, 8192, torch.float32),
                                       (65536, 16, torch.bfloat16)])
def test_q8_parity(m, d, dtype):
    r, w, delta, _ = inputs(m * 10007 + d, m, d, dtype)
    check_q8(r, w, delta, 1e-5, run_q8(r, w, delta, 1e-5))


def test_q8_in_place_zero_rows_and_no_values():
    r, w, delta, _ = inputs(3, 6, 520, torch.bfloat16)
    r[2] = 0
    delta[2] = 0
    keep = r.clone()
    got = run_q8(r, w, delta, 0.25, val=False, resid_out=r)
    check_q8(keep, w, delta, 0.25, got)
    assert (got[1][2] == 0).all() and got[2][2] == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_q8_a_token_that_is_not_finite_leaves_the_others_alone(bad):
    for d in (40, 200, 2048):
        r, w, delta, _ = inputs(5, 70, d, torch.bfloat16)
        want = run_q8(r, w, delta, 1e-5)
        r2 = r.clone()
        r2[33, d // 2] = bad
        got = run_q8(r2, w, delta, 1e-5)
        assert not torch.isfinite(got[2][33])
        rest = torch.arange(70, device="cuda") != 33
        for a, b in zip(want[1:], got[1:]):
            assert torch.equal(a[rest], b[rest])


def run_bwd(r, w, dout, dstream, eps, dw=True, dresid=None, ws_bytes=None):
    m, d = r.shape
    dr = torch.full_like(r, float("nan")) if dresid is None else dresid
    out = torch.full((d,), float("nan"), device="cuda") if dw else None
    n = dfssm.dfssm_add_rmsnorm_bwd_workspace_bytes(d, m)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if dw else None     # NaNs: nothing read before written
    dfssm.dfssm_add_rmsnorm_bwd(ptr(w), d, eps, ptr(r), ptr(dout), KIND[dout.dtype], ptr(dstream), m, ptr(dr), ptr(out),
                                ptr(ws), n if dw else 0, stream())
    torch.cuda.synchronize()
    return dr, out


@pytest.mark.parametrize("m,d,dtype,with_stream", [(1, 2048, torch.bfloat16, True), (3, 8, torch.float32, False),
                                                   (700, 64, torch.bfloat16, True), (45, 136, torch.float32, True),
                                                   (9, 512, torch.bfloat16, False), (300, 1000, torch.bfloat16, True),
                                                   (77, 2056, torch.float32, True), (1300, 1032, torch.bfloat16, False),
                                                   (5, 8192, torch.bfloat16, True), (40000, 24, torch.float32, False)])
def test_bwd_parity(m, d, dtype, with_stream):
    eps = 1e-5
    r, w, dout, g = inputs(m * 31 + d, m, d, dtype)
    ds = torch.randn(m, d, device="cuda", generator=g) if with_stream else None
    dr, dw = run_bwd(r, w, dout, ds, eps)
    x, do, w64 = r.double(), dout.double(), w.double()
    f = (x.square().mean(1, keepdim=True) + eps).rsqrt()
    gw = do * w64
    c = (gw * x).mean(1, keepdim=True)
    want = f * gw - f ** 3 * c * x
    room = (f * gw).abs() + f ** 3 * x.abs() * ((gw * x).abs().mean(1, keepdim=True) + c.abs())
    if ds is not None:
        want, room = want + ds.double(), room + ds.double().abs()
    assert ((dr.double() - want).abs() <= 2.0 ** -18 * room).all()
    dww, roomw = (do * x * f).sum(0), (do * x * f).abs().sum(0)
    assert ((dw.double() - dww).abs() <= (m / 592 + 120) * 2.0 ** -24 * roomw).all()


def test_bwd_in_place_without_weights_gradient_and_repeatable():
    r, w, dout, g = inputs(8, 50, 2048, torch.bfloat16)
    ds = torch.randn(50, 2048, device="cuda", generator=g)
    want, dw = run_bwd(r, w, dout, ds, 1e-5)
    again, dw2 = run_bwd(r, w, dout, ds, 1e-5)
    assert torch.equal(want, again) and torch.equal(dw, dw2)
    only, none = run_bwd(r, w, dout, ds, 1e-5, dw=False)
    assert torch.equal(want, only) and none is None
    a = r.clone()
    assert torch.equal(run_bwd(a, w, dout, ds, 1e-5, dresid=a)[0], want)
    b = ds.clone()
    assert torch.equal(run_bwd(r, w, dout, b, 1e-5, dresid=b)[0], want)


def test_bwd_against_differences():
    """<dresid, u> and <dnorm_w, v> against central differences of the 64-bit norm's <dout, o>."""
    m, d, eps = 4, 96, 1e-5
    r, w, dout, g = inputs(12, m, d, torch.float32)
    dr, dw = run_bwd(r, w, dout, None, eps)

    def loss(rr, ww):
        return (dout.double() * rr / (rr.square().mean(1, keepdim=True) + eps).sqrt() * ww).sum()

    u = torch.randn(m, d, device="cuda", generator=g).double()
    v = torch.randn(d, device="cuda", generator=g).double()
    h = 1e-6    # central difference: h^2 truncation, 2^-52 |loss| / h cancellation, both below 1e-8 |terms|
    du = (loss(r.double() + h * u, w.double()) - loss(r.double() - h * u, w.double())) / (2 * h)
    dv = (loss(r.double(), w.double() + h * v) - loss(r.double(), w.double() - h * v)) / (2 * h)
    scale_u, scale_v = (dr.double() * u).abs().sum(), (dw.double() * v).abs().sum()
    assert abs((dr.double() * u).sum() - du) <= 1e-5 * scale_u
    assert abs((dw.double() * v).sum() - dv) <= 1e-5 * scale_v


def test_on_another_stream_and_in_a_graph():
    r, w, delta, _ = inputs(21, 100, 1024, torch.bfloat16)
    m, d = r.shape
    want = run_q8(r, w, delta, 1e-5)
    dwant, dwwant = run_bwd(r, w, delta, None, 1e-5)
    s = torch.cuda.Stream()
    out = [torch.empty_like(t) for t in want]
    dr, dw = torch.empty_like(r), torch.empty_like(w)
    n = dfssm.dfssm_add_rmsnorm_bwd_workspace_bytes(d, m)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def both():
        dfssm.dfssm_add_rmsnorm_quant(ptr(w), d, 1e-5, ptr(r), ptr(delta), BF16, m, *[ptr(t) for t in out], stream())
        dfssm.dfssm_add_rmsnorm_bwd(ptr(w), d, 1e-5, ptr(r), ptr(delta), BF16, 0, m, ptr(dr), ptr(dw), ptr(ws), n,
                                    stream())

    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    s.synchronize()
    for rounds in range(2):
        for a, b in zip(want + (dwant, dwwant), out + [dr, dw]):
            assert torch.equal(a, b)
        if rounds == 0:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                both()
            for t in out + [dr, dw]:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
