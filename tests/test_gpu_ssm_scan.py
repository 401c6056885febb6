"""The state recurrence over packed sequences and its gradient on the GPU against 64 bits, token by token.

Tolerances. Every result is a sum of products, and its error is bounded by a factor f times the same
sum of magnitudes (the recurrence run on absolute values):
* x, B, C and dy enter exactly. In y, M and S are one fp16 number each: half a step, 2^-11 of the value,
  added to f for y. Elsewhere the second operand (M, W, S, dS, weighted x and dy) is two fp16 parts, 2^-22 of its value
  (2^-17, two bf16 parts, are allowed); fp32 accumulators round at most 2^-23 per MMA step, at most 32
  steps per chunk and result, 2^-18; a result passes through at most three such products: 2^-15.
* a decay exp(cum_t - cum_s) carries the error of its exponent: the chunk's sums round 2^-24 of at most
  their largest value c (in units of log 2) in at most 8 steps: 2^-21 c; exp2f and the products with dt
  (softplus: 4 ulp) 2^-21. The decay over a whole chunk is taken once per chunk: n_chunks (2^-21 + 2^-21 c')
  with c' <= 24 where the state still counts (2^-24): n_chunks 2^-16 at most, for a token that far back.
  f = 2^-14 + 2^-20 c + 2^-16 n_chunks, for states 2^-16 + the same.
* bf16 results add half a step, 2^-8 of the value.
* fp32 underflow: a decay below 2^-126 (the smallest normal number), or a product with it, is off by up
  to 2^-126 itself. It multiplies a sum of at most 64 x 128 products of two operands below 2^3 each (the
  inputs here): 2^-126 2^13 2^6 < 2^-106 absolute.
The magnitudes of the gradient of dt contain r_t and k_t of the whole chunk (the sums they are taken from).
"""
import pytest
import torch

import bit_gemv_gemm_dfssm_b200 as dfssm

pytestmark = pytest.mark.gpu
P, N, Q = 64, 128, 64
BF = torch.bfloat16


def stream():
    return torch.cuda.current_stream().cuda_stream


def ptr(t):
    return 0 if t is None else t.data_ptr()


def inputs(seed, lens, nh, ng, init=True, gap=0, dt0=(0.001, 0.1), spread=1.0):
    """x, b, c as column blocks of wider rows; `gap` rows of no sequence in front, between and behind."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*s):
        return torch.randn(*s, device="cuda", generator=g)

    def uni(lo, hi, *s):
        return torch.rand(*s, device="cuda", generator=g) * (hi - lo) + lo

    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    total = max(1, cu[-1] + gap)
    a = dict(lens=lens, nh=nh, ng=ng, total=total, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    a["row"] = torch.nn.functional.silu(rnd(total, nh * P + 2 * ng * N + 8)).to(BF)
    a["z"] = (spread * rnd(total, nh + 3)).to(BF)
    a["bias"] = torch.log(torch.expm1(uni(*dt0, nh)))
    a["a_log"] = torch.log(uni(1, 16, nh))
    a["d"] = uni(0.5, 1.5, nh)
    a["init"] = 0.5 * rnd(len(lens), nh, P, N) if init else None
    a["dy"] = rnd(total, nh * P + 16).to(BF)
    a["dfinal"] = rnd(len(lens), nh, P, N) if init else None
    return a


def structs(a):
    nh, ng = a["nh"], a["ng"]
    ld = a["row"].shape[1]
    x = ptr(a["row"])
    ins = dfssm.ScanInputs(x, ld, x + 2 * nh * P, ld, x + 2 * (nh * P + ng * N), ld, ptr(a["z"]) + 4, a["z"].shape[1],
                           ptr(a["bias"]), ptr(a["a_log"]), ptr(a["d"]), ptr(a["init"]), ptr(a["cu"]))
    return dfssm.ScanDims(nh, ng, P, N), ins


def space(dims, a, backward):
    n = dfssm.dfssm_ssm_scan_workspace_bytes(dims, a["total"], len(a["lens"]), backward)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")     # NaNs: nothing is read before it is written
    ws[:256] = 0
    return ws


def run_fwd(a, ws=None, final=True):
    dims, ins = structs(a)
    ws = space(dims, a, False) if ws is None else ws
    nh = a["nh"]
    y = torch.full((a["total"], nh * P + 8), 77.0, dtype=BF, device="cuda")
    fin = torch.full((len(a["lens"]), nh, P, N), float("nan"), device="cuda") if final is True else final
    dfssm.dfssm_ssm_scan_fwd(dims, ins, a["total"], len(a["lens"]), ptr(y), nh * P + 8, ptr(fin), ptr(ws), ws.numel(),
                             stream())
    return y, fin, ws


def run_bwd(a, ws=None):
    dims, ins = structs(a)
    ws = space(dims, a, True) if ws is None else ws
    nh, ng, total = a["nh"], a["ng"], a["total"]
    r = dict(dx=torch.full((total, nh * P + 8), 77.0, dtype=BF, device="cuda"),
             db=torch.full((total, ng * N + 8), 77.0, dtype=BF, device="cuda"),
             dc=torch.full((total, ng * N), 77.0, dtype=BF, device="cuda"),
             ddt=torch.full((total, nh + 1), 77.0, dtype=BF, device="cuda"))
    for k in ("ddt_bias", "da_log", "dd_skip"):
        r[k] = torch.full((nh,), float("nan"), device="cuda")
    r["dinit"] = torch.full((len(a["lens"]), nh, P, N), float("nan"), device="cuda") if a["init"] is not None else None
    gr = dfssm.ScanGrads(ptr(r["dx"]), nh * P + 8, ptr(r["db"]), ng * N + 8, ptr(r["dc"]), ng * N, ptr(r["ddt"]), nh + 1,
                         ptr(r["ddt_bias"]), ptr(r["da_log"]), ptr(r["dd_skip"]), ptr(r["dinit"]))
    dfssm.dfssm_ssm_scan_bwd(dims, ins, total, len(a["lens"]), ptr(a["dy"]), a["dy"].shape[1], ptr(a["dfinal"]), gr,
                             ptr(ws), ws.numel(), stream())
    return r, ws


def split(a, s):
    """64-bit x, b, c (expanded over the heads), v, dy of sequence s."""
    t0, n = int(a["cu"][s]), a["lens"][s]
    nh, ng = a["nh"], a["ng"]
    z = a["row"][t0:t0 + n].double()
    x = z[:, :nh * P].reshape(n, nh, P)
    b = z[:, nh * P:nh * P + ng * N].reshape(n, ng, N).repeat_interleave(nh // ng, 1)
    c = z[:, nh * P + ng * N:nh * P + 2 * ng * N].reshape(n, ng, N).repeat_interleave(nh // ng, 1)
    v = a["z"][t0:t0 + n, 2:2 + nh].double() + a["bias"].double()
    return x, b, c, v, a["dy"][t0:t0 + n, :nh * P].double().reshape(n, nh, P)


def softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(v.clamp(max=30))))


def forward64(x, b, c, dt, decay, d, s0):
    n = x.shape[0]
    s, ys, states = s0, [], [s0]
    for t in range(n):
        s = s * decay[t][:, None, None] + (dt[t][:, None] * x[t])[:, :, None] * b[t][:, None, :]
        ys.append((s * c[t][:, None, :]).sum(-1) + d[:, None] * x[t])
        states.append(s)
    return (torch.stack(ys) if n else x), s, states


def backward64(x, b, c, dt, decay, d, states, dy, ds):
    n = x.shape[0]
    dx, db, dc, k, da, r = [[None] * n for _ in range(6)]
    for t in range(n - 1, -1, -1):
        ds = ds + dy[t][:, :, None] * c[t][:, None, :]
        ub = (ds * b[t][:, None, :]).sum(-1)
        dx[t] = dt[t][:, None] * ub + d[:, None] * dy[t]
        db[t] = (ds * (dt[t][:, None] * x[t])[:, :, None]).sum(1)
        dc[t] = (states[t + 1] * dy[t][:, :, None]).sum(1)
        r[t] = (dc[t] * c[t]).sum(-1)
        k[t] = (ub * x[t]).sum(-1)
        ds = ds * decay[t][:, None, None]
        da[t] = (ds * states[t]).sum((1, 2))
    z = x.new_zeros((0, x.shape[1]))
    st = lambda q, e: torch.stack(q) if n else e  # noqa: E731
    return st(dx, x), st(db, b), st(dc, c), st(k, z), st(da, z), st(r, z), ds


def facts(a, s):
    x, b, c, v, dy = split(a, s)
    dt = softplus(v)
    neg = -torch.exp(a["a_log"].double())
    decay = torch.exp(dt * neg)
    n = x.shape[0]
    c_max = 0.0
    for q in range(0, n, Q):
        c_max = max(c_max, float((dt[q:q + Q] * -neg).sum(0).max()) * 1.4427)
    f = 2.0 ** -14 + 2.0 ** -20 * c_max + 2.0 ** -16 * (n // Q + 1)
    s0 = a["init"][s].double() if a["init"] is not None else x.new_zeros(a["nh"], P, N)
    return x, b, c, v, dy, dt, neg, decay, s0, f


def close(got, want, room, half=0.0):
    err = (got.double() - want).abs()
    lim = room + half * want.abs() + 2.0 ** -106
    assert (err <= lim).all(), f"worst {float((err / lim.clamp(min=1e-300)).max()):.3g} of the bound"


def check_fwd(a, y, fin):
    nh = a["nh"]
    used = torch.zeros(a["total"], dtype=torch.bool, device="cuda")
    for s, n in enumerate(a["lens"]):
        x, b, c, v, dy, dt, neg, decay, s0, f = facts(a, s)
        d = a["d"].double()
        want, end, _ = forward64(x, b, c, dt, decay, d, s0)
        mag, mend, _ = forward64(x.abs(), b.abs(), c.abs(), dt, decay, d.abs(), s0.abs())
        t0 = int(a["cu"][s])
        used[t0:t0 + n] = True
        close(y[t0:t0 + n, :nh * P].reshape(n, nh, P), want, (f + 2.0 ** -11) * mag, 2.0 ** -8)
        if fin is not None:
            close(fin[s], end, (f - 2.0 ** -14 + 2.0 ** -16) * mend)
    assert (y[:, nh * P:] == 77).all() and (y[~used] == 77).all()          # padding columns, rows of no sequence


def check_bwd(a, r):
    nh, ng = a["nh"], a["ng"]
    sums = {k: [0.0, 0.0] for k in ("ddt_bias", "da_log", "dd_skip")}
    used = torch.zeros(a["total"], dtype=torch.bool, device="cuda")
    for s, n in enumerate(a["lens"]):
        x, b, c, v, dy, dt, neg, decay, s0, f = facts(a, s)
        d = a["d"].double()
        t0 = int(a["cu"][s])
        used[t0:t0 + n] = True
        got = []
        for mag in (False, True):
            m = (lambda q: q.abs()) if mag else (lambda q: q)
            _, end, states = forward64(m(x), m(b), m(c), dt, decay, d, m(s0))
            ds = m(a["dfinal"][s].double()) if a["dfinal"] is not None else torch.zeros_like(end)
            got.append(backward64(m(x), m(b), m(c), dt, decay, d, states, m(dy), ds))
        (dx, db, dc, k, da, rr, d0), (mx, mb, mc, mk, ma, mr, m0) = got
        rows = slice(t0, t0 + n)

        def group(q):
            return q.reshape(n, ng, nh // ng, N).sum(2).reshape(n, ng * N)

        close(r["dx"][rows, :nh * P].reshape(n, nh, P), dx, f * mx, 2.0 ** -8)
        close(r["db"][rows, :ng * N], group(db), f * group(mb), 2.0 ** -8)
        close(r["dc"][rows], group(dc), f * group(mc), 2.0 ** -8)
        sig = torch.where(v > 20, torch.ones_like(v), torch.sigmoid(v))
        near = torch.zeros_like(ma)
        for q in range(0, n, Q):
            near[q:q + Q] = (mr + dt * mk)[q:q + Q].sum(0)
        ddt, mdt = (k + neg * da) * sig, (mk - neg * (ma + near)) * sig
        close(r["ddt"][rows, :nh], ddt, f * mdt, 2.0 ** -8)
        for key, val, mag in (("ddt_bias", ddt.sum(0), f * mdt.sum(0)),
                              ("da_log", (da * dt * neg).sum(0), f * ((ma + near) * dt * -neg).sum(0)),
                              ("dd_skip", (dy * x).sum((0, 2)), f * (dy * x).abs().sum((0, 2)))):
            sums[key][0] = sums[key][0] + val
            sums[key][1] = sums[key][1] + mag
        if r["dinit"] is not None:
            close(r["dinit"][s], d0, (f - 2.0 ** -14 + 2.0 ** -16) * m0)
    for key, (val, mag) in sums.items():
        close(r[key], val, mag)
    for key, cols in (("dx", nh * P), ("db", ng * N), ("ddt", nh)):
        assert (r[key][:, cols:] == 77).all()
    for key in ("dx", "db", "dc", "ddt"):
        assert (r[key][~used] == 77).all()


CASES = [([1], 1, 1, True, 0), ([64], 2, 1, False, 0), ([65, 0, 1, 63], 4, 2, True, 5), ([0], 3, 3, True, 2),
         ([5, 1, 0, 17], 64, 1, True, 0), ([130, 300], 6, 1, False, 3), ([200] * 3, 5, 5, True, 0),
         ([3] * 70, 2, 1, False, 1), ([16, 17, 32, 33, 49, 80], 2, 1, True, 0)]


@pytest.mark.parametrize("lens,nh,ng,init,gap", CASES)
def test_forward(lens, nh, ng, init, gap):
    a = inputs(len(lens) * 100 + nh, lens, nh, ng, init, gap)
    y, fin, ws = run_fwd(a)
    torch.cuda.synchronize()
    check_fwd(a, y, fin)
    assert dfssm.dfssm_ssm_read_error(ptr(ws), stream()) == (dfssm.DFSSM_OK, 0)


@pytest.mark.parametrize("lens,nh,ng,init,gap", CASES)
def test_backward(lens, nh, ng, init, gap):
    a = inputs(len(lens) * 100 + nh + 1, lens, nh, ng, init, gap)
    r, ws = run_bwd(a)
    torch.cuda.synchronize()
    check_bwd(a, r)
    assert dfssm.dfssm_ssm_read_error(ptr(ws), stream()) == (dfssm.DFSSM_OK, 0)


@pytest.mark.parametrize("lens,nh,ng,init,gap", [([513], 1, 1, False, 0), ([128, 129, 0, 1, 127, 256], 4, 2, True, 5),
                                                 ([640], 3, 1, True, 1), ([2] * 300, 2, 2, False, 0),
                                                 ([0, 0, 600, 0], 2, 1, True, 600), ([1000] + [1] * 7, 2, 1, True, 0),
                                                 ([40] * 40, 80, 1, True, 0), ([41] * 40, 80, 1, False, 0)])
def test_forward_of_long_calls(lens, nh, ng, init, gap):
    a = inputs(len(lens) * 100 + nh + 2, lens, nh, ng, init, gap)
    y, fin, ws = run_fwd(a)
    torch.cuda.synchronize()
    check_fwd(a, y, fin)
    assert dfssm.dfssm_ssm_read_error(ptr(ws), stream()) == (dfssm.DFSSM_OK, 0)


@pytest.mark.parametrize("lens", [[1500], [700, 513, 512, 1100, 64], [1537, 1536, 3, 2600], [4000]])
def test_sequences_that_are_cut_into_segments(lens):
    a = inputs(5, lens, 2, 1, True, 7)
    y, fin, _ = run_fwd(a)
    r, _ = run_bwd(a)
    torch.cuda.synchronize()
    check_fwd(a, y, fin)
    check_bwd(a, r)


def test_many_sequences_need_the_table():
    a = inputs(6, [41 + i % 60 for i in range(80)], 2, 2, False, 0)
    y, fin, _ = run_fwd(a)
    torch.cuda.synchronize()
    check_fwd(a, y, fin)


@pytest.mark.parametrize("dt0,spread", [((1.0, 30.0), 3.0), ((1e-6, 1e-5), 0.1)])
def test_fast_and_slow_decays(dt0, spread):
    """Decays that leave nothing after one token (dt above softplus's bend), and next to none."""
    a = inputs(7, [150, 40], 4, 1, True, 0, dt0, spread)
    y, fin, _ = run_fwd(a)
    r, _ = run_bwd(a)
    torch.cuda.synchronize()
    check_fwd(a, y, fin)
    check_bwd(a, r)


def test_continuing_a_sequence_equals_the_whole():
    """Two calls, the second from the first one's final state (in place), within both bounds of the whole."""
    a = inputs(8, [200], 3, 1, True)
    first = {**a, "lens": [77], "cu": torch.tensor([0, 77], dtype=torch.int32, device="cuda")}
    y1, fin, _ = run_fwd(first)
    rest = {**a, "lens": [123], "cu": torch.tensor([77, 200], dtype=torch.int32, device="cuda"), "init": fin}
    y2, fin2, _ = run_fwd(rest, final=fin)
    torch.cuda.synchronize()
    y = torch.where((torch.arange(200, device="cuda") < 77)[:, None], y1, y2)
    check_fwd(a, y, fin2)


def test_bad_offsets_are_reported_and_skipped():
    for lens, cu in (([10, 20, 30], [0, 10, 5, 61]), ([10, 20, 30], [-4, 10, 30, 60]), ([60], [0, 1 << 30])):
        a = inputs(9, lens, 2, 1, False)
        a["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        y, fin, ws = run_fwd(a)
        st, bits = dfssm.dfssm_ssm_read_error(ptr(ws), stream())
        assert st == dfssm.DFSSM_ERR_DEVICE_CHECK and bits == dfssm.DFSSM_DEVERR_SEQLENS
        r, ws = run_bwd(a)
        st, bits = dfssm.dfssm_ssm_read_error(ptr(ws), stream())
        assert st == dfssm.DFSSM_ERR_DEVICE_CHECK and bits == dfssm.DFSSM_DEVERR_SEQLENS
    # the sequences around a bad one are computed
    a = inputs(10, [10, 20, 30], 2, 1, False)
    good, _, _ = run_fwd(a)
    a["cu"][3] = 1000
    y, _, _ = run_fwd(a)
    torch.cuda.synchronize()
    assert torch.equal(y[:30], good[:30]) and (y[30:] == 77).all()


def test_offsets_that_overlap_leave_out_what_the_workspace_cannot_hold():
    """The same 700 rows as three sequences (0..700, and back, twice): more chunks than the call's rows can have. What is
    left is whole: the first sequence's results, its parameters' gradients among them."""
    a = inputs(16, [700], 2, 1, False)
    y, _, _ = run_fwd(a)
    r, _ = run_bwd(a)
    b = {**a, "lens": [700, 0, 700, 0, 700], "cu": torch.tensor([0, 700, 0, 700, 0, 700], dtype=torch.int32, device="cuda")}
    y2, _, ws = run_fwd(b, final=None)
    r2, ws2 = run_bwd(b)
    torch.cuda.synchronize()
    assert torch.equal(y, y2)
    for k in r:
        assert r[k] is None or torch.equal(r[k], r2[k]), k
    for w in (ws, ws2):
        st, bits = dfssm.dfssm_ssm_read_error(ptr(w), stream())
        assert st == dfssm.DFSSM_ERR_DEVICE_CHECK and bits == dfssm.DFSSM_DEVERR_SEQLENS


def test_a_sequence_that_is_not_finite_leaves_the_others_alone():
    a = inputs(11, [70, 90, 30], 2, 1, True)
    y, fin, _ = run_fwd(a)
    r, _ = run_bwd(a)
    b = {**a, "row": a["row"].clone(), "dy": a["dy"].clone()}
    b["row"][100, 3] = float("nan")
    b["dy"][120, 5] = float("inf")
    y2, fin2, _ = run_fwd(b)
    r2, _ = run_bwd(b)
    torch.cuda.synchronize()
    rest = torch.ones(190, dtype=torch.bool, device="cuda")
    rest[70:160] = False
    assert torch.equal(y[rest], y2[rest]) and torch.equal(fin[[0, 2]], fin2[[0, 2]])
    for k in ("dx", "db", "dc", "ddt"):
        assert torch.equal(r[k][rest], r2[k][rest])


@pytest.mark.parametrize("lens", [[200, 30], [700, 30]])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_no_finite_value_is_wrong_beside_one_that_is_not(lens, bad):
    """An entry of x, b or c that is not finite: what is finite in the results is what it was without it."""
    a = inputs(15, lens, 2, 1, True)
    y, fin, _ = run_fwd(a)
    r, _ = run_bwd(a)
    for col in (3, 2 * P + 5, 2 * P + N + 7):          # x of head 0, b, c
        e = {**a, "row": a["row"].clone()}
        e["row"][100, col] = bad
        y2, fin2, _ = run_fwd(e)
        r2, _ = run_bwd(e)
        torch.cuda.synchronize()
        for u, v in [(y, y2), (fin, fin2)] + [(r[k], r2[k]) for k in r]:
            kept = torch.isfinite(v)
            assert torch.isfinite(u).all() and torch.equal(u[kept], v[kept])
        assert not torch.isfinite(y2[100]).all() and torch.isfinite(y2[lens[0]:]).all()


def test_gradient_against_differences():
    """sum(dy y) + <dfinal, final> of the 64-bit recurrence along random directions of every input."""
    a = inputs(12, [70], 2, 1, True, 0, (0.01, 0.1))
    r, _ = run_bwd(a)
    torch.cuda.synchronize()
    x, b, c, v, dy, dt, neg, decay, s0, f = facts(a, 0)
    b, c = b[:, :1], c[:, :1]
    raw = a["z"][:70, 2:4].double()
    args = [x, b, c, raw, a["bias"].double(), a["a_log"].double(), a["d"].double(), s0]

    def loss(x, b, c, raw, bias, a_log, d, s0):
        dt = softplus(raw + bias)
        y, end, _ = forward64(x, b.expand(-1, 2, -1), c.expand(-1, 2, -1), dt, torch.exp(-torch.exp(a_log) * dt), d, s0)
        return (dy * y).sum() + (a["dfinal"][0].double() * end).sum()

    got = [r["dx"][:70, :2 * P].reshape(70, 2, P), r["db"][:70, :N].reshape(70, 1, N), r["dc"][:70].reshape(70, 1, N),
           r["ddt"][:70, :2], r["ddt_bias"], r["da_log"], r["dd_skip"], r["dinit"][0]]
    g = torch.Generator(device="cuda").manual_seed(3)
    for i, q in enumerate(got):
        u = torch.randn(args[i].shape, device="cuda", generator=g, dtype=torch.float64)
        h = 1e-6
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + h * u, args[i] - h * u
        slope = (loss(*up) - loss(*dn)) / (2 * h)
        # rounding of the entries to bf16 (2^-8) and the bounds above (below 2^-8 of the entries' own size here)
        assert abs((q.double() * u).sum() - slope) <= 2.0 ** -7 * (q.double() * u).abs().sum(), i


def test_repeatable_on_another_stream_and_in_a_graph():
    a = inputs(13, [300, 17, 1200], 4, 2, True)
    y, fin, ws = run_fwd(a)
    r, ws2 = run_bwd(a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, fin2, _ = run_fwd(a, ws)
        r2, _ = run_bwd(a, ws2)
    s.synchronize()
    assert torch.equal(y, y2) and torch.equal(fin, fin2) and all(torch.equal(r[k], r2[k]) for k in r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, fin3, _ = run_fwd(a, ws)
        r3, _ = run_bwd(a, ws2)
    # other values and other lengths in the same buffers
    b = inputs(14, [1100, 17, 400], 4, 2, True)
    for k in ("row", "z", "bias", "a_log", "d", "init", "dy", "dfinal", "cu"):
        a[k].copy_(b[k])
    graph.replay()
    torch.cuda.synchronize()
    check_fwd(b, y3, fin3)
    check_bwd(b, r3)


@pytest.mark.parametrize("dt0,spread", [((1.0, 30.0), 3.0), ((0.3, 3.0), 1.0), ((1e-6, 1e-5), 0.1)])
def test_fast_and_slow_decays_of_long_calls(dt0, spread):
    """The same in chunks of 128 tokens, whose decays off the diagonal are products of two (a chunk of twice the tokens has
    at most twice the exponent c of two of 64, at 2^-21 of it, within the 2^-20 c of the bound)."""
    a = inputs(17, [700, 0, 131, 300], 4, 2, True, 3, dt0, spread)
    y, fin, _ = run_fwd(a)
    torch.cuda.synchronize()
    check_fwd(a, y, fin)


@pytest.mark.parametrize("lens", [[40, 3, 0, 65], [300, 1, 0, 200], [1700, 30]])
def test_rows_of_no_sequence_reach_no_result(lens):
    """NaN in front of the first sequence and behind the last, in every input: the results are the same bits as beside
    other rows, and the rows are not written."""
    a = inputs(18, lens, 2, 1, True, 150)
    a["cu"] += 70                                        # 70 rows in front, 80 behind
    used = torch.zeros(a["total"], dtype=torch.bool, device="cuda")
    used[70:70 + sum(lens)] = True
    b = {**a, **{k: a[k].clone() for k in ("row", "z", "dy")}}
    for k in ("row", "z", "dy"):
        b[k][~used] = float("nan")
    (y, fin, _), (y2, fin2, _) = run_fwd(a), run_fwd(b)
    (r, _), (r2, _) = run_bwd(a), run_bwd(b)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(fin, fin2) and (y2[~used] == 77).all()
    for k in r:
        assert torch.equal(r[k], r2[k]) and torch.isfinite(r2[k]).all(), k


@pytest.mark.parametrize("lens", [[1, 70, 33], [600, 20]])
def test_tokens_masked_by_the_lowest_step(lens):
    """dt_raw of -Inf and of the type's lowest value: dt is 0, the state passes, the gradient of dt_raw is 0."""
    a = inputs(19, lens, 2, 1, True)
    n = a["total"]
    a["z"][torch.arange(0, n, 3, device="cuda")] = float("-inf")
    a["z"][torch.arange(1, n, 7, device="cuda")] = torch.finfo(BF).min
    y, fin, _ = run_fwd(a)
    r, _ = run_bwd(a)
    torch.cuda.synchronize()
    check_fwd(a, y, fin)
    check_bwd(a, r)
