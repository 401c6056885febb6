"""A training step's and a server's path through the sequence operators, as a model strings them together, on the GPU:
state scan -> residual add, norm and int8 rounding -> cross entropy over the int8 table, and the gradients back through all
three. Every stage is checked against 64 bits on what the stage before it left (the tolerances are those of the
operators' own tests); the whole chain, replayed from a CUDA graph on other inputs, gives the bits of the eager run.
"""
import pytest
import torch

import bit_gemv_gemm_dfssm_b200 as dfssm
import test_gpu_norm_quant as tn
import test_gpu_ssm_scan as ts
import test_gpu_xent as tx

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-5


class Chain:
    """Buffers of one shape; load() fills the inputs, step() launches the chain on the current stream."""

    def __init__(self, seed, lens, nh, ng, vocab):
        self.a = ts.inputs(seed, lens, nh, ng)
        self.x = tx.inputs(seed + 1, self.a["total"], vocab, nh * ts.P)
        d, t = nh * ts.P, self.a["total"]
        g = torch.Generator(device="cuda").manual_seed(seed + 2)
        self.r0 = torch.randn(t, d, device="cuda", generator=g)
        self.w = torch.rand(d, device="cuda", generator=g) + 0.5
        dims, _ = ts.structs(self.a)
        self.ws = [ts.space(dims, self.a, False), tx.workspace(self.x, False), tx.workspace(self.x, True),
                   torch.zeros(dfssm.dfssm_add_rmsnorm_bwd_workspace_bytes(d, t), dtype=torch.uint8, device="cuda"),
                   ts.space(dims, self.a, True)]
        self.out = {}

    def step(self):
        a, x, o, s = self.a, self.x, self.out, ts.stream()
        t, d = self.r0.shape
        y, o["fin"], _ = ts.run_fwd(a, self.ws[0])
        o["y"] = y[:, :d].contiguous()
        o["r1"], x["q"], x["sx"] = torch.empty_like(self.r0), torch.empty_like(x["q"]), torch.empty_like(x["sx"])
        dfssm.dfssm_add_rmsnorm_quant(ts.ptr(self.w), d, EPS, ts.ptr(self.r0), ts.ptr(o["y"]), dfssm.DFSSM_BF16, t,
                                      ts.ptr(o["r1"]), ts.ptr(x["q"]), ts.ptr(x["sx"]), 0, s)
        o["q"], o["sx"] = x["q"], x["sx"]
        o["nll"], o["lse"], _ = tx.fwd(x, self.ws[1])
        o["dh"], _ = tx.bwd(x, o["lse"], self.ws[2])
        o["dr"], o["dw"] = torch.empty_like(self.r0), torch.empty_like(self.w)
        dfssm.dfssm_add_rmsnorm_bwd(ts.ptr(self.w), d, EPS, ts.ptr(o["r1"]), ts.ptr(o["dh"]), dfssm.DFSSM_BF16, 0, t,
                                    ts.ptr(o["dr"]), ts.ptr(o["dw"]), ts.ptr(self.ws[3]), self.ws[3].numel(), s)
        a["dy"] = o["dr"].to(BF)
        o["dy"] = a["dy"]
        grads, _ = ts.run_bwd(a, self.ws[4])
        o.update({"g_" + k: v for k, v in grads.items()})


def check_norm_grad(c):
    r, w, do = c.out["r1"].double(), c.w.double(), c.out["dh"].double()
    f = (r.square().mean(1, keepdim=True) + EPS).rsqrt()
    gw = do * w
    k = (gw * r).mean(1, keepdim=True)
    room = (f * gw).abs() + f ** 3 * r.abs() * ((gw * r).abs().mean(1, keepdim=True) + k.abs())
    assert ((c.out["dr"].double() - (f * gw - f ** 3 * k * r)).abs() <= 2.0 ** -18 * room).all()
    lim = (r.shape[0] / 592 + 120) * 2.0 ** -24 * (do * r * f).abs().sum(0)
    assert ((c.out["dw"].double() - (do * r * f).sum(0)).abs() <= lim).all()


@pytest.mark.parametrize("lens,nh,ng,vocab", [([130, 1, 0, 77], 4, 1, 1000), ([9], 2, 2, 333), ([300, 320], 8, 2, 700)])
def test_training_step(lens, nh, ng, vocab):
    c = Chain(31 + len(lens), lens, nh, ng, vocab)
    c.step()
    torch.cuda.synchronize()
    o, d = c.out, nh * ts.P
    padded = torch.full((c.a["total"], d + 8), 77.0, dtype=BF, device="cuda")
    padded[:, :d] = o["y"]
    ts.check_fwd(c.a, padded, o["fin"])
    tn.check_q8(c.r0, c.w, o["y"], EPS, (o["r1"], o["q"], o["sx"], None))
    tx.check(c.x, o["nll"], o["lse"], o["dh"])
    check_norm_grad(c)
    ts.check_bwd(c.a, {k[2:]: v for k, v in o.items() if k.startswith("g_")})


def test_training_step_from_a_graph():
    lens, nh, ng, vocab = [200, 3, 450], 4, 2, 900
    c = Chain(5, lens, nh, ng, vocab)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.step()
    kept = dict(c.out)
    other = Chain(6, lens, nh, ng, vocab)
    for k in ("row", "z", "bias", "a_log", "d", "init", "dfinal"):
        c.a[k].copy_(other.a[k])
    for k in ("table", "scale", "tg", "grad"):
        c.x[k].copy_(other.x[k])
    c.r0.copy_(other.r0)
    c.w.copy_(other.w)
    for _ in range(2):
        graph.replay()
    other.step()
    torch.cuda.synchronize()
    for k, v in other.out.items():
        assert torch.equal(v, kept[k]), k


def test_two_chains_at_once():
    """Two chains with their own buffers, launched in turn on two streams that nothing orders."""
    args = ([300, 5, 700], 4, 2, 900), ([64] * 9, 4, 1, 2000)
    alone = [Chain(50 + i, *v) for i, v in enumerate(args)]
    for c in alone:
        c.step()
    torch.cuda.synchronize()
    both = [Chain(50 + i, *v) for i, v in enumerate(args)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for c, s in zip(both, streams):
            with torch.cuda.stream(s):
                c.step()
    torch.cuda.synchronize()
    for c, e in zip(both, alone):
        for k, v in e.out.items():
            assert torch.equal(v, c.out[k]), k


def test_server_continues_token_by_token():
    """Two prompts in one call, then three tokens each from the states that call left, each token through the norm and
    the table: every call's states and losses against 64 bits."""
    nh, ng, vocab = 4, 1, 1000
    c = Chain(17, [70, 9], nh, ng, vocab)
    _, fin, _ = ts.run_fwd(c.a, c.ws[0])
    for k in range(3):
        n = Chain(40 + k, [1, 1], nh, ng, vocab)
        for key in ("bias", "a_log", "d"):
            n.a[key] = c.a[key]
        n.a["init"] = fin.clone()
        n.step()
        torch.cuda.synchronize()
        padded = torch.full((2, nh * ts.P + 8), 77.0, dtype=BF, device="cuda")
        padded[:, :nh * ts.P] = n.out["y"]
        ts.check_fwd(n.a, padded, n.out["fin"])
        tn.check_q8(n.r0, n.w, n.out["y"], EPS, (n.out["r1"], n.out["q"], n.out["sx"], None))
        tx.check(n.x, n.out["nll"], n.out["lse"], n.out["dh"])
        # in place: the state that a server keeps
        _, own, _ = ts.run_fwd(dict(n.a, init=fin), n.ws[0], final=fin)
        torch.cuda.synchronize()
        assert torch.equal(own, n.out["fin"])
