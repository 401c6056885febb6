"""The sequence operators of the library, as measured: the cases, their inputs, their plain forms.

Six operators of the model's run over a text, next to its linears:

  norm_q8    residual add + RMS norm with an int8 output and one scale per token
  norm_bwd   its gradient (straight through the quantiser)
  xent_fwd   softmax cross entropy over the int8 table, without keeping the logits
  xent_bwd   the gradient with respect to the hidden state it was computed from
  scan_fwd   the Mamba-2 state recurrence over packed sequences of any length
  scan_bwd   its gradient

`run` computes the plain form in torch, in fp32, where `own` is false, and calls the library where it is true.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
HEADDIM, D_STATE = 64, 128
IGNORE = -100
EPS = 1e-5


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode token in front of the LM head of the 2048-channel model: a call's latency
        dict(name="norm_q8_token", op="norm_q8", m=1, d=2048, delta="bf16"),
        # the frame between two blocks over a packed batch of prompts
        dict(name="norm_q8_prompts", op="norm_q8", m=16384, d=2048, delta="bf16"),
        # the gradient of the frame for a short text, an odd width
        dict(name="norm_bwd_short", op="norm_bwd", m=77, d=2056, delta="f32"),
        # the gradient of the frame for a training batch
        dict(name="norm_bwd_batch", op="norm_bwd", m=16384, d=2048, delta="bf16"),
        # the loss of one new token over the whole vocabulary (scoring a continuation)
        dict(name="xent_fwd_token", op="xent_fwd", m=1, vocab=50288, d=2048, ignored=0.0),
        # the loss of a 2048-token text
        dict(name="xent_fwd_text", op="xent_fwd", m=2048, vocab=50288, d=2048, ignored=0.1),
        # the loss's gradient for the 16 answer tokens of a short example
        dict(name="xent_bwd_answer", op="xent_bwd", m=16, vocab=50288, d=2048, ignored=0.0),
        # the loss's gradient for a 2048-token text, prompt tokens ignored
        dict(name="xent_bwd_text", op="xent_bwd", m=2048, vocab=50288, d=2048, ignored=0.1),
        # a few continued conversations: short pieces on top of a carried state, one of a single token, one empty
        dict(name="scan_fwd_continue", op="scan_fwd", lens="5,1,0,17", heads=64, groups=1, init=True),
        # a packed batch of prompts of different lengths
        dict(name="scan_fwd_prompts", op="scan_fwd", lens="2048,1511,4096,777,2049,3967,1900,36", heads=64, groups=1,
             init=False),
        # the gradient over a short ragged batch that goes on from a state
        dict(name="scan_bwd_short", op="scan_bwd", lens="130,1,63", heads=64, groups=1, init=True),
        # the gradient over a training batch
        dict(name="scan_bwd_batch", op="scan_bwd", lens="2048,2048,2048,2048", heads=64, groups=1, init=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_q8", "norm_bwd", "xent_fwd", "xent_bwd", "scan_fwd", "scan_bwd"])
    if op.startswith("norm"):
        # 8 to 8192 channels, a multiple of 8; tokens within the largest listed case's bytes
        d = 8 * _log_int(rng, 1, 1024)
        m = _log_int(rng, 1, min(65536, 16384 * 2048 // d))
        return dict(op=op, m=m, d=d, delta=rng.choice(["bf16", "f32", "none"]))
    if op.startswith("xent"):
        return dict(op=op, m=_log_int(rng, 1, 2048), vocab=_log_int(rng, 1000, 50288), d=16 * _log_int(rng, 8, 128),
                    ignored=rng.choice([0.0, 0.1, 0.5]))
    nseq = _log_int(rng, 1, 16)
    longest = _log_int(rng, 1, 8192 // nseq)
    lens = [longest] + [rng.randint(0 if longest < 64 else longest // 3, longest) for _ in range(nseq - 1)]
    rng.shuffle(lens)
    groups = rng.choice([1, 1, 2, 4])
    return dict(op=op, lens=",".join(map(str, lens)), heads=groups * rng.randint(1, 64 // groups), groups=groups,
                init=rng.choice([True, False]))


# ------------------------------------------------------------------------------- inputs

def _lens(case):
    return [int(v) for v in case["lens"].split(",")]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, device="cuda", generator=g) * (hi - lo) + lo

    op = case["op"]
    st = dict(case=case, op=op)
    if op.startswith("norm"):
        m, d = case["m"], case["d"]
        # the residual stream's rows differ in size from token to token
        st["resid"] = normal(m, d) * uniform(0.05, 20.0, m, 1)
        st["w"] = uniform(0.5, 1.5, d)
        if op == "norm_q8":
            dt = {"bf16": BF16, "f32": F32, "none": None}[case["delta"]]
            st["delta"] = None if dt is None else normal(m, d).to(dt)
        else:
            # the loss's gradient arrives in the type that `delta` names; "none": no gradient on the stream itself
            st["dout"] = normal(m, d).to(F32 if case["delta"] == "f32" else BF16)
            st["dstream"] = None if case["delta"] == "none" else normal(m, d)
    elif op.startswith("xent"):
        m, v, d = case["m"], case["vocab"], case["d"]
        st["table"] = torch.randint(-127, 128, (v, d), device="cuda", generator=g, dtype=torch.int8)
        st["scale"] = uniform(1e-4, 1e-3, v)
        # a normed hidden state, one channel in a hundred 20 times as large, in the layer's int8 form
        h = normal(m, d)
        loud = torch.randperm(d, device="cuda", generator=g)[: max(1, d // 100)]
        h[:, loud] *= 20.0
        amax = h.abs().amax(1)
        st["q"] = (h * (127.0 / amax)[:, None]).round().clamp(-127, 127).to(torch.int8)
        st["sx"] = amax / 127.0
        tg = torch.randint(0, v, (m,), device="cuda", generator=g, dtype=torch.int32)
        off = torch.rand(m, device="cuda", generator=g) < case["ignored"]
        st["targets"] = torch.where(off, torch.full_like(tg, IGNORE), tg)
        if op == "xent_bwd":
            st["lse"] = torch.logsumexp(_logits(st), 1)                 # the forward call's
            st["grad"] = uniform(0.5, 1.5, m) / m                       # weights of a mean over the tokens
    else:
        lens, nh, ng = _lens(case), case["heads"], case["groups"]
        total, nseq = sum(lens), len(lens)
        # the convolution's output rows [x | B | C] and dt as a column block of the in_proj output's rows
        row = nh * HEADDIM + 2 * ng * D_STATE
        st["xbc"] = torch.nn.functional.silu(normal(total, row)).to(BF16)
        st["zdt"] = normal(total, 8 + nh).to(BF16)
        dt0 = uniform(0.001, 0.1, nh)
        st["dt_bias"] = torch.log(torch.expm1(dt0))
        st["a_log"] = torch.log(uniform(1.0, 16.0, nh))
        st["d_skip"] = uniform(0.5, 1.5, nh)
        st["init"] = 0.5 * normal(nseq, nh, HEADDIM, D_STATE) if case["init"] else None
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        st["total"], st["nseq"] = total, nseq
        if op == "scan_bwd":
            st["dy"] = normal(total, nh * HEADDIM).to(BF16)
            st["dfinal"] = normal(nseq, nh, HEADDIM, D_STATE) if case["init"] else None
        # the plain form's plan: every sequence padded to whole chunks, total = the row that stands for padding
        nc = max(1, -(-max(lens) // CHUNK))
        at = torch.arange(nc * CHUNK, device="cuda")[None, :]
        first, n = st["cu"][:-1, None].long(), (st["cu"][1:] - st["cu"][:-1])[:, None].long()
        st["pad"] = torch.where(at < n, first + at, torch.full_like(at, total))
        st["inside"] = st["pad"] < total
    return st


# ------------------------------------------------------------------------------- plain forms

CHUNK = 64


def _logits(st):
    return (st["q"].float() @ st["table"].float().T) * (st["sx"][:, None] * st["scale"][None, :])


def _norm_q8(st):
    r = st["resid"] if st["delta"] is None else st["resid"] + st["delta"].float()
    o = r * torch.rsqrt(r.square().mean(1, keepdim=True) + EPS) * st["w"]
    amax = o.abs().amax(1, keepdim=True)
    q = torch.where(amax > 0, (o * (127.0 / amax)).round().clamp(-127, 127), torch.zeros_like(o))
    sx = amax / 127.0
    return dict(resid=r, sx=sx[:, 0], val=(q * sx).to(BF16))


def _norm_bwd(st):
    r, do = st["resid"], st["dout"].float()
    f = torch.rsqrt(r.square().mean(1, keepdim=True) + EPS)
    gw = do * st["w"]
    dr = f * gw - f.pow(3) * (gw * r).mean(1, keepdim=True) * r
    if st["dstream"] is not None:
        dr = dr + st["dstream"]
    return dict(dresid=dr, dw=(do * r * f).sum(0))


def _xent_fwd(st):
    lg, tg = _logits(st), st["targets"].long()
    lse = torch.logsumexp(lg, 1)
    hit = lg.gather(1, tg.clamp(min=0)[:, None])[:, 0]
    return dict(nll=torch.where(tg >= 0, lse - hit, torch.zeros_like(lse)), lse=lse)


def _xent_bwd(st):
    tg = st["targets"].long()
    p = torch.exp(_logits(st) - st["lse"][:, None])
    hot = torch.zeros_like(p).scatter_(1, tg.clamp(min=0)[:, None], 1.0)
    gr = torch.where(tg >= 0, st["grad"], torch.zeros_like(st["grad"]))
    return dict(dh=(((p - hot) * st["scale"]) @ st["table"].float() * gr[:, None]).to(BF16))


def _decays(a):
    """exp(a_{s+1} + ... + a_t) for t >= s over the last axis, 0 for t < s: [..., t, s]."""
    n = a.shape[-1]
    cum = a.cumsum(-1)
    keep = torch.ones(n, n, dtype=torch.bool, device=a.device).tril()
    return torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(~keep, -math.inf))


def _scan(st, x, b, c, dt_raw, dt_bias, a_log, d_skip, init):
    """The recurrence in chunks, without a loop: x [total, h, p], b and c [total, g, n], dt_raw [total, h]."""
    nh, ng = st["case"]["heads"], st["case"]["groups"]
    nseq, nc = st["nseq"], st["pad"].shape[1] // CHUNK

    def chunks(v):
        v = torch.cat([v, torch.zeros_like(v[:1]) if v.shape[0] else v.new_zeros((1,) + v.shape[1:])])
        return v[st["pad"]].reshape(nseq, nc, CHUNK, *v.shape[1:])

    dt = torch.nn.functional.softplus(dt_raw + dt_bias)
    xc, dtc = chunks(x), chunks(dt)
    bc = chunks(b).repeat_interleave(nh // ng, 3)
    cc = chunks(c).repeat_interleave(nh // ng, 3)
    a = (dtc * -torch.exp(a_log)).permute(0, 3, 1, 2)                    # [seq, h, chunk, t]
    xd = xc * dtc[..., None]
    within = torch.einsum("bcthn,bcshn->bhcts", cc, bc) * _decays(a)
    y = torch.einsum("bhcts,bcshp->bcthp", within, xd)
    cum = a.cumsum(-1)
    left = torch.exp(cum[..., -1:] - cum).permute(0, 2, 3, 1)            # [seq, chunk, t, h]
    own_states = torch.einsum("bcshp,bcshn->bchpn", xd * left[..., None], bc)
    start = init if init is not None else torch.zeros_like(own_states[:, 0])
    states = torch.cat([start[:, None], own_states], 1)                  # what each chunk adds, the start first
    over = _decays(torch.nn.functional.pad(cum[..., -1], (1, 0)))        # [seq, h, to, from]
    states = torch.einsum("bhij,bjhpn->bihpn", over, states)
    y = y + torch.einsum("bcthn,bchpn->bcthp", cc, states[:, :-1]) * torch.exp(cum).permute(0, 2, 3, 1)[..., None]
    y = y + xc * d_skip[:, None]
    y = y.reshape(nseq * nc * CHUNK, nh, HEADDIM)[st["inside"].reshape(-1)]
    return y, states[:, -1]


def _scan_args(st):
    nh, ng, total = st["case"]["heads"], st["case"]["groups"], st["total"]
    di, gn = nh * HEADDIM, ng * D_STATE
    xbc = st["xbc"].float()
    return [xbc[:, :di].reshape(total, nh, HEADDIM), xbc[:, di:di + gn].reshape(total, ng, D_STATE),
            xbc[:, di + gn:].reshape(total, ng, D_STATE), st["zdt"][:, 8:].float(), st["dt_bias"], st["a_log"],
            st["d_skip"], st["init"]]


def _scan_fwd(st):
    y, final = _scan(st, *_scan_args(st))
    return dict(y=y.reshape(st["total"], -1).to(BF16), final=final)


def _scan_bwd(st):
    args = [None if v is None else v.detach().requires_grad_(True) for v in _scan_args(st)]
    y, final = _scan(st, *args)
    outs, grads = [y], [st["dy"].float().reshape(y.shape)]
    if st["dfinal"] is not None:
        outs.append(final)
        grads.append(st["dfinal"])
    got = torch.autograd.grad(outs, [v for v in args if v is not None], grads)
    total = st["total"]
    r = dict(dx=got[0].reshape(total, -1).to(BF16), db=got[1].reshape(total, -1).to(BF16),
             dc=got[2].reshape(total, -1).to(BF16), ddt=got[3].to(BF16), ddt_bias=got[4], da_log=got[5],
             dd_skip=got[6])
    if st["init"] is not None:
        r["dinit"] = got[7]
    return r


# ------------------------------------------------------------------------------- the library's calls

def _kept(st, key, make):
    """A buffer that a program makes once and keeps beside its inputs."""
    if key not in st:
        st[key] = make()
    return st[key]


def _bytes(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def _own(st):
    import bit_gemv_gemm_dfssm_b200 as dfssm

    case, op = st["case"], st["op"]
    stream = torch.cuda.current_stream().cuda_stream

    def ptr(v):
        return 0 if v is None else v.data_ptr()

    if op == "norm_q8":
        m, d, delta = case["m"], case["d"], st["delta"]
        out = _kept(st, "out", lambda: dict(
            resid=torch.empty(m, d, device="cuda"), q=torch.empty(m, d, dtype=torch.int8, device="cuda"),
            sx=torch.empty(m, device="cuda"), val=torch.empty(m, d, dtype=BF16, device="cuda")))
        kind = dfssm.DFSSM_F32 if delta is not None and delta.dtype == F32 else dfssm.DFSSM_BF16
        dfssm.dfssm_add_rmsnorm_quant(ptr(st["w"]), d, EPS, ptr(st["resid"]), ptr(delta), kind, m, ptr(out["resid"]),
                                   ptr(out["q"]), ptr(out["sx"]), ptr(out["val"]), stream)
        return dict(resid=out["resid"], sx=out["sx"], val=out["val"])
    if op == "norm_bwd":
        m, d = case["m"], case["d"]
        size = _kept(st, "size", lambda: dfssm.dfssm_add_rmsnorm_bwd_workspace_bytes(d, m))
        ws = _kept(st, "ws", lambda: _bytes(size))
        out = _kept(st, "out", lambda: dict(dresid=torch.empty(m, d, device="cuda"), dw=torch.empty(d, device="cuda")))
        kind = dfssm.DFSSM_F32 if st["dout"].dtype == F32 else dfssm.DFSSM_BF16
        dfssm.dfssm_add_rmsnorm_bwd(ptr(st["w"]), d, EPS, ptr(st["resid"]), ptr(st["dout"]), kind, ptr(st["dstream"]), m,
                                    ptr(out["dresid"]), ptr(out["dw"]), ptr(ws), size, stream)
        return out
    if op.startswith("xent"):
        m, v, d = case["m"], case["vocab"], case["d"]
        table = _kept(st, "ctable", lambda: dfssm.Int8Table(ptr(st["table"]), ptr(st["scale"]), v, d))
        size = _kept(st, "size", lambda: dfssm.dfssm_xent_workspace_bytes(table, m, op == "xent_bwd"))
        ws = _kept(st, "ws", lambda: _bytes(size))
        if op == "xent_fwd":
            out = _kept(st, "out", lambda: dict(nll=torch.empty(m, device="cuda"), lse=torch.empty(m, device="cuda")))
            dfssm.dfssm_xent_fwd(table, ptr(st["q"]), ptr(st["sx"]), ptr(st["targets"]), m, ptr(out["nll"]),
                                 ptr(out["lse"]), ptr(ws), size, stream)
        else:
            out = _kept(st, "out", lambda: dict(dh=torch.empty(m, d, dtype=BF16, device="cuda")))
            dfssm.dfssm_xent_bwd(table, ptr(st["q"]), ptr(st["sx"]), ptr(st["targets"]), ptr(st["lse"]),
                                 ptr(st["grad"]), m, ptr(out["dh"]), ptr(ws), size, stream)
        return out
    nh, ng, total, nseq = case["heads"], case["groups"], st["total"], st["nseq"]
    di, gn = nh * HEADDIM, ng * D_STATE
    row = di + 2 * gn
    dims = _kept(st, "dims", lambda: dfssm.ScanDims(nh, ng, HEADDIM, D_STATE))
    size = _kept(st, "size", lambda: dfssm.dfssm_ssm_scan_workspace_bytes(dims, total, nseq, op == "scan_bwd"))
    ws = _kept(st, "ws", lambda: _bytes(size))
    ins = _kept(st, "ins", lambda: dfssm.ScanInputs(
        ptr(st["xbc"]), row, ptr(st["xbc"]) + 2 * di, row, ptr(st["xbc"]) + 2 * (di + gn), row, ptr(st["zdt"]) + 16,
        8 + nh, ptr(st["dt_bias"]), ptr(st["a_log"]), ptr(st["d_skip"]), ptr(st["init"]), ptr(st["cu"])))

    def state():
        return torch.empty(nseq, nh, HEADDIM, D_STATE, device="cuda")

    if op == "scan_fwd":
        out = _kept(st, "out", lambda: dict(y=torch.empty(total, di, dtype=BF16, device="cuda"), final=state()))
        dfssm.dfssm_ssm_scan_fwd(dims, ins, total, nseq, ptr(out["y"]), di, ptr(out["final"]), ptr(ws), size, stream)
        return out

    def grads():
        r = dict(dx=torch.empty(total, di, dtype=BF16, device="cuda"), db=torch.empty(total, gn, dtype=BF16, device="cuda"),
                 dc=torch.empty(total, gn, dtype=BF16, device="cuda"), ddt=torch.empty(total, nh, dtype=BF16, device="cuda"),
                 ddt_bias=torch.empty(nh, device="cuda"), da_log=torch.empty(nh, device="cuda"),
                 dd_skip=torch.empty(nh, device="cuda"))
        if st["init"] is not None:
            r["dinit"] = state()
        return r

    out = _kept(st, "out", grads)
    gr = _kept(st, "grads", lambda: dfssm.ScanGrads(
        ptr(out["dx"]), di, ptr(out["db"]), gn, ptr(out["dc"]), gn, ptr(out["ddt"]), nh, ptr(out["ddt_bias"]),
        ptr(out["da_log"]), ptr(out["dd_skip"]), ptr(out.get("dinit"))))
    dfssm.dfssm_ssm_scan_bwd(dims, ins, total, nseq, ptr(st["dy"]), di, ptr(st["dfinal"]), gr, ptr(ws), size, stream)
    return out


def run(st):
    if own:
        return _own(st)
    return {"norm_q8": _norm_q8, "norm_bwd": _norm_bwd, "xent_fwd": _xent_fwd, "xent_bwd": _xent_bwd,
            "scan_fwd": _scan_fwd, "scan_bwd": _scan_bwd}[st["op"]](st)


# ------------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op.startswith("norm"):
        m, d = case["m"], case["d"]
        extra = {"bf16": 2, "f32": 4, "none": 0}[case["delta"]]
        if op == "norm_q8":     # resid, delta, resid', q, the values q stands for, one scale; the weights
            return dict(bytes=m * (d * (4 + extra + 4 + 1 + 2) + 4) + 4 * d, flops=8 * m * d)
        dout, stream = (4, 4) if case["delta"] == "f32" else (2, 4 if case["delta"] == "bf16" else 0)
        return dict(bytes=m * d * (4 + dout + stream + 4) + 8 * d, flops=12 * m * d)
    if op.startswith("xent"):
        m, v, d = case["m"], case["vocab"], case["d"]
        if op == "xent_fwd":
            return dict(bytes=v * (d + 4) + m * (d + 16), flops=2 * m * v * d)
        return dict(bytes=v * (d + 4) + m * (d + 16 + 2 * d), flops=4 * m * v * d)
    lens, nh, ng = _lens(case), case["heads"], case["groups"]
    total, nseq = sum(lens), len(lens)
    rows = 2 * (nh * HEADDIM + 2 * ng * D_STATE + nh)                    # x, B, C, dt of a token
    state = 4 * nseq * nh * HEADDIM * D_STATE
    step = nh * HEADDIM * D_STATE * total
    if op == "scan_fwd":
        return dict(bytes=total * (rows + 2 * nh * HEADDIM) + state * (2 if case["init"] else 1), flops=5 * step)
    return dict(bytes=total * (2 * rows + 2 * nh * HEADDIM) + state * (3 if case["init"] else 0), flops=14 * step)


# ------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm_q8":
        r = st["resid"].double()
        if st["delta"] is not None:
            r = r + st["delta"].double()
        o = r / (r.pow(2).sum(1, keepdim=True) / case["d"] + EPS).sqrt() * st["w"].double()
        top = o.abs().max(1, keepdim=True).values
        step = top / 127
        q = torch.where(top > 0, torch.round(o / step), torch.zeros_like(o))
        return dict(resid=r, sx=step[:, 0], val=q * step)
    if op == "norm_bwd":
        r, do, w, d = st["resid"].double(), st["dout"].double(), st["w"].double(), case["d"]
        ms = r.pow(2).sum(1, keepdim=True) / d + EPS
        dr = (do * w) / ms.sqrt() - r * ((do * w * r).sum(1, keepdim=True) / d) / (ms * ms.sqrt())
        if st["dstream"] is not None:
            dr = dr + st["dstream"].double()
        return dict(dresid=dr, dw=(do * (r / ms.sqrt())).sum(0))
    if op.startswith("xent"):
        m, v, d = case["m"], case["vocab"], case["d"]
        q, sx, sc, tg = st["q"].double(), st["sx"].double(), st["scale"].double(), st["targets"].long()
        on = tg >= 0
        piece = 8192
        if op == "xent_fwd":
            parts = []
            for v0 in range(0, v, piece):
                lg = (q @ st["table"][v0:v0 + piece].double().T) * sx[:, None] * sc[v0:v0 + piece]
                parts.append(torch.logsumexp(lg, 1))
            lse = torch.logsumexp(torch.stack(parts), 0)
            t0 = tg.clamp(min=0)
            hit = (q * st["table"][t0].double()).sum(1) * sx * sc[t0]
            return dict(nll=torch.where(on, lse - hit, torch.zeros_like(lse)), lse=lse)
        dh = torch.zeros(m, d, dtype=torch.float64, device="cuda")
        for v0 in range(0, v, piece):
            e = st["table"][v0:v0 + piece].double()
            lg = (q @ e.T) * sx[:, None] * sc[v0:v0 + piece]
            dh += (torch.exp(lg - st["lse"].double()[:, None]) * sc[v0:v0 + piece]) @ e
        t0 = tg.clamp(min=0)
        dh -= st["table"][t0].double() * sc[t0][:, None]
        return dict(dh=dh * torch.where(on, st["grad"].double(), torch.zeros_like(sx))[:, None])
    return _exact_scan(st, case)


def _exact_scan(st, case):
    """Token by token, all sequences side by side (each step's rows past a sequence's end count for nothing)."""
    lens, nh, ng = _lens(case), case["heads"], case["groups"]
    total, nseq, longest = sum(lens), len(lens), max(lens)
    di, gn, rep = nh * HEADDIM, ng * D_STATE, nh // ng
    n = torch.tensor(lens, device="cuda")
    first = st["cu"][:-1].long()
    v = st["zdt"][:, 8:].double() + st["dt_bias"].double()
    dt = torch.where(v > 20, v, torch.log1p(torch.exp(v)))
    neg = -torch.exp(st["a_log"].double())
    skip = st["d_skip"].double()

    def rows(t):
        live = t < n
        return live, torch.where(live, first + t, torch.zeros_like(first))

    def token(at, live):
        z = st["xbc"][at].double()
        on = live.double()[:, None]
        d = dt[at] * on
        return (z[:, :di].reshape(nseq, nh, HEADDIM), z[:, di:di + gn].reshape(nseq, ng, D_STATE).repeat_interleave(rep, 1),
                z[:, di + gn:].reshape(nseq, ng, D_STATE).repeat_interleave(rep, 1), d, torch.exp(d * neg))

    s = torch.zeros(nseq, nh, HEADDIM, D_STATE, dtype=torch.float64, device="cuda")
    if st["init"] is not None:
        s = st["init"].double()
    back = case["op"] == "scan_bwd"
    y = torch.zeros(total, nh, HEADDIM, dtype=torch.float64, device="cuda")
    dc = torch.zeros(total, ng, D_STATE, dtype=torch.float64, device="cuda")
    ydy = torch.zeros(total, nh, dtype=torch.float64, device="cuda")
    dy = st["dy"].double().reshape(total, nh, HEADDIM) if back else None
    for t in range(longest):
        live, at = rows(t)
        x, b, c, d, keep = token(at, live)
        s = s * keep[..., None, None] + (x * d[..., None])[..., None] * b[:, :, None, :]
        if back:
            dch = torch.einsum("bhpn,bhp->bhn", s, dy[at])
            ydy[at[live]] = (dch * c).sum(-1)[live]
            dc[at[live]] = dch.reshape(nseq, ng, rep, D_STATE).sum(2)[live]
        else:
            yt = torch.einsum("bhpn,bhn->bhp", s, c) + x * skip[:, None]
            y[at[live]] = yt[live]
    if not back:
        return dict(y=y.reshape(total, di), final=s)
    ds = st["dfinal"].double() if st["dfinal"] is not None else torch.zeros_like(s)
    cross = (ds * s).sum((2, 3))                    # gradient of the decays summed from the end: <dS, S> there
    dx = torch.zeros_like(y)
    db, ddt, da = torch.zeros_like(dc), torch.zeros_like(ydy), torch.zeros_like(ydy)
    for t in range(longest - 1, -1, -1):
        live, at = rows(t)
        x, b, c, d, keep = token(at, live)
        on = live.double()[:, None]
        ds = ds + (dy[at] * on[..., None])[..., None] * c[:, :, None, :]
        ub = torch.einsum("bhpn,bhn->bhp", ds, b)
        xub = (ub * x).sum(-1)
        cross = cross + ydy[at] * on - d * xub      # <dS_t, S_t> less what token t itself adds: <dS_t, e^a S_{t-1}>
        dx[at[live]] = (ub * d[..., None] + dy[at] * skip[:, None])[live]
        db[at[live]] = (torch.einsum("bhpn,bhp->bhn", ds, x) * d[..., None]).reshape(nseq, ng, rep, D_STATE).sum(2)[live]
        da[at[live]] = cross[live]
        ddt[at[live]] = xub[live]
        ds = ds * keep[..., None, None]
    ddt = (ddt + neg * da) * torch.sigmoid(v)
    xr = st["xbc"][:, :di].double().reshape(total, nh, HEADDIM)
    r = dict(dx=dx.reshape(total, di), db=db.reshape(total, gn), dc=dc.reshape(total, gn), ddt=ddt, ddt_bias=ddt.sum(0),
             da_log=(da * dt * neg).sum(0), dd_skip=(dy * xr).sum((0, 2)))
    if st["init"] is not None:
        r["dinit"] = ds
    return r
