"""Cross entropy over the int8 table and its gradient on the GPU against 64 bits.

Tolerances, with L the largest |logit| of the token:
* A logit is an exact integer, converted (half a step, 2^-24) and multiplied three times (by the
  scale, by s_x log2 e, itself rounded): 4 2^-24 relative, so any softmax average of logits is off
  by at most 4 2^-24 L. exp2f is within 2 ulp (2^-22) and the arguments' subtraction within 2^-24 of
  at most 2 L log2 e. The sum over a half tile adds at most 32 + 12 roundings, the joins at most
  3 (2 ceil(V/256)/32 + 6), each 2^-24 relative; log2f 1 ulp, two more operations on lse. In all
    |d lse| <= 2^-24 (8 L + 4 |lse| + 64 + 3 (V/4096 + 8)),
  and nll adds the target's logit (4 2^-24 L) and one subtraction.
* dh: the probabilities carry the errors above as relative errors, d_p = 2^-24 (16 L + 8 |lse| + 80),
  are rounded to fp16 (2^-11; below its normal range by at most 2^-38 max|s|, 2^-25 over K), and the
  fp32 accumulator takes V/16 steps of at most 2^-23 each of the sum of magnitudes S = sum p |s E|;
  the splits add at most 148 2^-24 S. The target's row and the products with grad: 2^-22. The output's
  bf16 rounding: 2^-8 |dh|.
"""
import pytest
import torch

import bit_gemv_gemm_dfssm_b200 as dfssm

pytestmark = pytest.mark.gpu
IGNORE = dfssm.DFSSM_IGNORE_TARGET


def stream():
    return torch.cuda.current_stream().cuda_stream


def inputs(seed, m, v, d, ignored=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    table = torch.randint(-128, 128, (v, d), device="cuda", generator=g, dtype=torch.int8)
    scale = torch.rand(v, device="cuda", generator=g) * 9e-4 + 1e-4
    h = torch.randn(m, d, device="cuda", generator=g)
    amax = h.abs().amax(1)
    q = (h * (127 / amax)[:, None]).round().to(torch.int8)
    # small widths get larger activations, so that the logits spread
    sx = amax / 127 * (2048 / d) ** 0.5
    tg = torch.randint(0, v, (m,), device="cuda", generator=g, dtype=torch.int32)
    tg[torch.rand(m, device="cuda", generator=g) < ignored] = IGNORE
    grad = torch.rand(m, device="cuda", generator=g) + 0.5
    return dict(table=table, scale=scale, q=q, sx=sx, tg=tg, grad=grad)


def ctable(a):
    v, d = a["table"].shape
    return dfssm.Int8Table(a["table"].data_ptr(), a["scale"].data_ptr(), v, d)


def workspace(a, backward, fill=0):
    n = dfssm.dfssm_xent_workspace_bytes(ctable(a), a["q"].shape[0], backward)
    ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    return ws


def fwd(a, ws=None):
    m = a["q"].shape[0]
    ws = workspace(a, False, 255) if ws is None else ws
    nll = torch.full((m,), float("nan"), device="cuda")
    lse = torch.full((m,), float("nan"), device="cuda")
    dfssm.dfssm_xent_fwd(ctable(a), a["q"].data_ptr(), a["sx"].data_ptr(), a["tg"].data_ptr(), m, nll.data_ptr(),
                         lse.data_ptr(), ws.data_ptr(), ws.numel(), stream())
    return nll, lse, ws


def bwd(a, lse, ws=None):
    m, d = a["q"].shape
    ws = workspace(a, True, 255) if ws is None else ws
    dh = torch.full((m, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    dfssm.dfssm_xent_bwd(ctable(a), a["q"].data_ptr(), a["sx"].data_ptr(), a["tg"].data_ptr(), lse.data_ptr(),
                         a["grad"].data_ptr(), m, dh.data_ptr(), ws.data_ptr(), ws.numel(), stream())
    return dh, ws


def logits64(a):
    return (a["q"].double() @ a["table"].double().T) * a["sx"].double()[:, None] * a["scale"].double()[None, :]


def check(a, nll, lse, dh=None):
    m, d = a["q"].shape
    v = a["scale"].numel()
    lg = logits64(a)
    top = lg.abs().amax(1)
    want = torch.logsumexp(lg, 1)
    room = 2.0 ** -24 * (8 * top + 4 * want.abs() + 64 + 3 * (v / 4096 + 8))
    assert ((lse.double() - want).abs() <= room).all()
    on = a["tg"] >= 0
    t0 = a["tg"].clamp(min=0).long()
    hit = lg.gather(1, t0[:, None])[:, 0]
    wn = torch.where(on, want - hit, torch.zeros_like(want))
    assert ((nll.double() - wn).abs() <= room + 2.0 ** -24 * (4 * top + wn.abs())).all()
    assert (nll[~on] == 0).all()
    if dh is None:
        return
    p = torch.exp(lg - lse.double()[:, None])
    e, s = a["table"].double(), a["scale"].double()
    hot = e[t0] * s[t0][:, None]
    gr = torch.where(on, a["grad"].double(), torch.zeros_like(want))[:, None]
    wd = ((p * s) @ e - hot) * gr
    mag = (p * s) @ e.abs()
    dp = 2.0 ** -24 * (16 * top + 8 * want.abs() + 80)[:, None]
    room = 2.0 ** -8 * wd.abs() + gr * (mag * (dp + 2.0 ** -11 + 2.0 ** -23 * (v / 16 + 148)) + 2.0 ** -22 * hot.abs()
                                       + 2.0 ** -38 * s.max() * 128 * v)
    assert ((dh.double() - wd).abs() <= room).all()
    assert (dh[~on] == 0).all()


@pytest.mark.parametrize("m,v,d", [(1, 1000, 256), (3, 1, 16), (2, 300, 16), (5, 128, 144), (128, 256, 128),
                                   (130, 257, 272), (129, 513, 2048), (257, 5000, 400), (64, 2049, 8192),
                                   (2300, 700, 64), (1, 50288, 2048), (16, 50288, 2048)])
def test_parity(m, v, d):
    a = inputs(m * 7 + v + d, m, v, d)
    nll, lse, ws = fwd(a)
    dh, ws2 = bwd(a, lse)
    torch.cuda.synchronize()
    check(a, nll, lse, dh)
    for w in (ws, ws2):
        assert dfssm.dfssm_ssm_read_error(w.data_ptr(), stream()) == (dfssm.DFSSM_OK, 0)


def test_vocabulary_in_pieces_and_repeatable():
    a = inputs(77, 2048, 50288, 256, 0.1)
    nll, lse, ws = fwd(a)
    dh, ws2 = bwd(a, lse)
    torch.cuda.synchronize()
    check(a, nll, lse, dh)
    nll2, lse2, _ = fwd(a, ws)
    dh2, _ = bwd(a, lse2, ws2)
    torch.cuda.synchronize()
    assert torch.equal(nll, nll2) and torch.equal(lse, lse2) and torch.equal(dh, dh2)


def test_peaked_and_flat_rows():
    """One logit far above the others (probability 1), a row of zeros (uniform), a negative scale."""
    a = inputs(5, 6, 700, 512, 0.0)
    a["scale"][3] = -a["scale"][3]
    a["sx"][0] *= 300.0                       # logits in the hundreds: all probability on one row
    a["q"][1] = 0                             # all logits 0
    a["sx"][2] = 0.0
    nll, lse, _ = fwd(a)
    dh, _ = bwd(a, lse)
    torch.cuda.synchronize()
    check(a, nll, lse, dh)


def test_targets_outside_the_vocabulary_are_ignored_and_reported():
    a = inputs(9, 40, 900, 256, 0.0)
    good = {k: v.clone() for k, v in a.items()}
    for i, bad in ((3, 900), (7, -1), (20, 2 ** 31 - 1), (21, -2 ** 31)):
        a["tg"][i] = bad
        good["tg"][i] = IGNORE
    nll, lse, ws = fwd(a)
    dh, ws2 = bwd(a, lse)
    torch.cuda.synchronize()
    check(good, nll, lse, dh)
    for w in (ws, ws2):
        assert dfssm.dfssm_ssm_read_error(w.data_ptr(), stream()) == (dfssm.DFSSM_ERR_DEVICE_CHECK,
                                                                     dfssm.DFSSM_DEVERR_TOKEN_ID)
        assert dfssm.dfssm_ssm_read_error(w.data_ptr(), stream()) == (dfssm.DFSSM_OK, 0)


def test_rows_that_are_not_finite_leave_the_others_alone():
    a = inputs(10, 140, 900, 256, 0.0)
    nll, lse, _ = fwd(a)
    dh, _ = bwd(a, lse)
    b = {k: v.clone() for k, v in a.items()}
    b["sx"][5], b["sx"][130] = float("nan"), float("inf")
    b["tg"][6], b["sx"][6], b["grad"][6] = IGNORE, float("nan"), float("nan")
    nll2, lse2, _ = fwd(b)
    dh2, _ = bwd(b, lse2)
    torch.cuda.synchronize()
    assert not torch.isfinite(nll2[5]) and not torch.isfinite(nll2[130])
    assert nll2[6] == 0 and (dh2[6] == 0).all()
    rest = torch.ones(140, dtype=torch.bool, device="cuda")
    rest[[5, 6, 130]] = False
    assert torch.equal(nll[rest], nll2[rest]) and torch.equal(lse[rest], lse2[rest]) and torch.equal(dh[rest], dh2[rest])


def test_gradient_against_differences():
    a = inputs(11, 6, 400, 96, 0.0)
    nll, lse, _ = fwd(a)
    dh, _ = bwd(a, lse)
    torch.cuda.synchronize()
    h = a["q"].double() * a["sx"].double()[:, None]
    es = a["table"].double() * a["scale"].double()[:, None]
    t0 = a["tg"].long()

    def loss(x):
        lg = x @ es.T
        return ((torch.logsumexp(lg, 1) - lg.gather(1, t0[:, None])[:, 0]) * a["grad"].double()).sum()

    g = torch.Generator(device="cuda").manual_seed(1)
    for _ in range(4):
        u = torch.randn(h.shape, device="cuda", generator=g, dtype=torch.float64)
        step = 1e-5
        slope = (loss(h + step * u) - loss(h - step * u)) / (2 * step)
        # dh's rounding (2^-8 of each entry, 2^-11 of the probabilities before it) and lse's in fp32
        assert abs((dh.double() * u).sum() - slope) <= 2.0 ** -7 * (dh.double() * u).abs().sum()


def test_on_another_stream_and_in_a_graph():
    a = inputs(12, 200, 3000, 512)
    nll, lse, ws = fwd(a)
    dh, ws2 = bwd(a, lse)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        n2, l2, _ = fwd(a, ws)
        d2, _ = bwd(a, l2, ws2)
    s.synchronize()
    assert torch.equal(nll, n2) and torch.equal(lse, l2) and torch.equal(dh, d2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n3, l3, _ = fwd(a, ws)
        d3, _ = bwd(a, l3, ws2)
    other = inputs(13, 200, 3000, 512)
    for k in ("q", "sx", "tg", "grad", "table", "scale"):
        a[k].copy_(other[k])
    graph.replay()
    torch.cuda.synchronize()
    check(a, n3, l3, d3)


def confident(a, left):
    """`a` with a target of probability 1 - left[i] for token i: the token's largest logit, s_x by bisection in 64 bits."""
    m = len(left)
    one = logits64(dict(a, sx=torch.ones(m, device="cuda")))
    tg = one.argmax(1)
    gap = (one - one.amax(1, keepdim=True)).scatter_(1, tg[:, None], float("-inf"))
    lo, hi = torch.zeros(m, dtype=torch.float64, device="cuda"), torch.full((m,), 1e3, dtype=torch.float64, device="cuda")
    want = torch.tensor(left, dtype=torch.float64, device="cuda")
    for _ in range(80):
        mid = (lo + hi) / 2
        rest = torch.exp(torch.logsumexp(gap * mid[:, None], 1))
        more = rest / (1 + rest) > want
        lo, hi = torch.where(more, mid, lo), torch.where(more, hi, mid)
    return dict(a, tg=tg.to(torch.int32), sx=hi.float())


@pytest.mark.parametrize("v,d", [(700, 512), (3000, 64), (50288, 256)])
def test_gradient_of_confident_tokens(v, d):
    """Targets of probability 0.9 to 0.99999: what is left of (p - 1) s E, not what cancels in it, sets the room.

    The other rows as at the head of this file, over S' = their sum of p |s E|. The target's factor expm1(l - lse) is off
    by half a step of its argument, two steps of expm1f and three roundings behind it: below 2^-21 of itself."""
    left = [0.1, 1e-2, 1e-3, 1e-4, 3e-5, 1e-5]
    a = confident(inputs(21 + v, len(left), v, d, 0.0), left)
    _, lse, _ = fwd(a)
    dh, _ = bwd(a, lse)
    torch.cuda.synchronize()
    lg, e, s, t0 = logits64(a), a["table"].double(), a["scale"].double(), a["tg"].long()[:, None]
    x = lg - lse.double()[:, None]
    off = torch.expm1(x.gather(1, t0))                                   # p - 1 of the target
    p = torch.exp(x).scatter_(1, t0, 0.0)
    hot = off * e[t0[:, 0]] * s[t0]
    gr = a["grad"].double()[:, None]
    want = gr * ((p * s) @ e + hot)
    dp = 2.0 ** -24 * (16 * lg.abs().amax(1) + 8 * lse.double().abs() + 80)[:, None]
    room = 2.0 ** -8 * want.abs() + gr * (((p * s) @ e.abs()) * (dp + 2.0 ** -11 + 2.0 ** -23 * (v / 16 + 148))
                                         + 2.0 ** -21 * hot.abs() + 2.0 ** -38 * s.max() * 128 * v)
    err = (dh.double() - want).abs()
    assert (err <= room).all(), [f"{float(r):.3g}" for r in err.norm(dim=1) / want.norm(dim=1)]


@pytest.mark.parametrize("v,d", [(700, 512), (3000, 2048)])
def test_loss_of_confident_tokens_with_large_logits(v, d):
    """Logits in the hundreds (the target's row has a near twin), losses of 1e-1 to 1e-4: the logits' own roundings do
    not reach them.

    The target's logit is the running maximum, bit for bit, so nll is the logarithm of 1 plus the others' share 1 - p,
    which is off by the differences of two logits (16 2^-24 L) and 80 2^-24 of itself; the sums and joins round as at
    the head of this file, 2^-24 of about 1 each; the logarithm and its factor 2^-22 of the loss. lse is the target's
    logit in 64 bits plus that, rounded once."""
    left = [0.1, 1e-2, 1e-3, 3e-4, 1e-4]
    a = inputs(40 + v, len(left), v, d, 0.0)
    top = logits64(dict(a, sx=torch.ones(len(left), device="cuda"))).argmax(1)
    twin = (top + v // 2) % v
    assert torch.cat([top, twin]).unique().numel() == 2 * len(left)
    a["table"][twin] = a["table"][top]
    a["scale"][twin] = a["scale"][top] * (1 - 2.0 ** -6)
    a = confident(a, left)
    nll, lse, _ = fwd(a)
    torch.cuda.synchronize()
    lg, t0 = logits64(a), a["tg"].long()[:, None]
    hit = lg.gather(1, t0)[:, 0]
    rest = torch.exp(torch.logsumexp(lg.scatter(1, t0, float("-inf")) - hit[:, None], 1))
    want = torch.log1p(rest)
    room = 2.0 ** -24 * (rest * (16 * lg.abs().amax(1) + 80) + 64 + 3 * (v / 4096 + 8)) + 2.0 ** -22 * want
    err = (nll.double() - want).abs()
    assert (err <= room).all(), [f"{float(r):.3g}" for r in err / want]
    assert ((lse.double() - (hit + want)).abs() <= room + 2.0 ** -24 * (hit + want).abs()).all()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_scale_that_is_not_finite_shows_in_every_token(bad):
    """... whatever the sign of its row's sums; an s_x in its own token."""
    a = inputs(14, 140, 900, 256)
    a["scale"][300] = bad
    nll, lse, _ = fwd(a)
    dh, _ = bwd(a, lse)
    b = inputs(14, 140, 900, 256)
    b["sx"][7] = bad
    b["tg"][7] = 5
    b["q"][7] = b["q"][7].abs().clamp(1, 127)
    b["table"] = -b["table"].clamp(-127, 127).abs().clamp(min=1)         # every sum of token 7 below 0
    nll2, lse2, _ = fwd(b)
    torch.cuda.synchronize()
    on = a["tg"] >= 0
    assert torch.isnan(lse).all() and torch.isnan(nll[on]).all() and (nll[~on] == 0).all()
    assert torch.isnan(dh[on]).all() and (dh[~on] == 0).all()
    assert torch.isnan(lse2[7]) and torch.isnan(nll2[7]) and torch.isfinite(lse2[8:]).all()


@pytest.mark.parametrize("m,v,d", [(2049, 300, 272), (2300, 33000, 64), (4100, 1000, 16), (4096, 21000, 32)])
def test_token_blocks_of_unequal_size_and_vocabulary_pieces(m, v, d):
    """More tokens than one block holds, the last block short, with one and with two pieces of the vocabulary."""
    a = inputs(m + v, m, v, d)
    nll, lse, _ = fwd(a)
    dh, ws = bwd(a, lse)
    torch.cuda.synchronize()
    check(a, nll, lse, dh)
    assert dfssm.dfssm_ssm_read_error(ws.data_ptr(), stream()) == (dfssm.DFSSM_OK, 0)


@pytest.mark.parametrize("m", [1, 100])
@pytest.mark.parametrize("v", [18944, 18945, 28120, 38000, 80000])
def test_tile_sizes_of_few_tokens(m, v):
    """Vocabularies on both sides of the rule that picks the tiles' rows, one of them exactly one tile per SM."""
    a = inputs(m + v, m, v, 48)
    nll, lse, _ = fwd(a)
    dh, _ = bwd(a, lse)
    torch.cuda.synchronize()
    check(a, nll, lse, dh)
