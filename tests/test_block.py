"""The operators together, as a decoder block uses them.

Training: x -> norm -> dense gated block -> + x -> norm (the residual added in front of it) -> MoE layer -> + residual,
forward and backward through the library, against the same block in 64 bits on the GPU's own choice of experts.
Serving: residual + norm -> quantiser -> 8-bit product, eager, and captured and replayed.

Tolerance of the training step: every tensor between two operators (n1, a, y1, h, n2, the layer's activations and
pre-activations, and as many gradients on the way back) is rounded to bf16 once, half = 2^-8 of its norm at most; at
most 14 of them lie on the way to any output.  Errors of independent roundings add in squares, so the sum is a bound.
"""
import torch
import pytest

from sparse_mixture_experts_sigmoid_b200 import binding as B
from sparse_mixture_experts_sigmoid_b200.workloads import Workload
from sparse_mixture_experts_sigmoid_b200 import synth

pytestmark = pytest.mark.gpu
HALF = torch.finfo(torch.bfloat16).eps / 2
STEPS = 14


def norm64(x, w, b, eps, rms=False):
    z = x if rms else x - x.mean(1, keepdim=True)
    y = z / torch.sqrt((z * z).mean(1, keepdim=True) + eps) * w
    return y if b is None else y + b


def moe64(x, layer, ids, k):
    """The routed layer in 64 bits on given experts (softmax over the kept logits)."""
    s = torch.softmax(x @ layer["router"].T, 1)
    g = s.gather(1, ids)
    g = g / g.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    for j in range(k):
        for e in range(layer["gate"].shape[0]):
            rows = ids[:, j] == e
            if rows.any():
                xe = x[rows]
                u = xe @ layer["gate"][e].T
                a = u * torch.sigmoid(u) * (xe @ layer["up"][e].T)
                y = y.index_add(0, rows.nonzero()[:, 0], g[rows, j:j + 1] * (a @ layer["down"][e].T))
    return y


@pytest.mark.parametrize("T", [1, 37, 300])
@pytest.mark.parametrize("kind,act", [("layer", "silu"), ("rms", "gelu_tanh")])
def test_block_forward_and_backward(T, kind, act):
    d, h, E, k, he = 128, 384, 4, 2, 192
    w = Workload("block", T=T, d=d, E=E, h=he, k=k, seed=5, weight_std=0.08, router_std=0.2)
    layer = synth.make_layer(w, "cpu").to("cuda")
    g = torch.Generator(device="cuda").manual_seed(T)

    def n(*s, std=1.0, mean=0.0, t=torch.bfloat16):
        return (torch.randn(*s, generator=g, device="cuda") * std + mean).to(t)

    x, dy = n(T, d), n(T, d)
    w1, b1 = n(d, std=0.1, mean=1.0, t=torch.float32), n(d, std=0.1, t=torch.float32)
    w2 = n(d, std=0.1, mean=1.0)
    wg, wu, wd = n(h, d, std=d ** -0.5), n(h, d, std=d ** -0.5), n(d, h, std=h ** -0.5)
    c1 = B.norm_config(T, d, kind=kind, w_dtype="f32")
    c2 = B.norm_config(T, d, kind="rms")
    cf, cm = B.ffn_config(T, d, h, act=act), B.config_of(w)

    n1, _, m1, r1 = B.norm_forward(c1, x, w1, bias=b1, want_stats=True)
    fws = B.alloc_ffn_workspace(cf, train=True)
    y1 = B.ffn_forward_train(cf, n1, wg, wu, wd, fws)
    n2, hh, _, r2 = B.norm_forward(c2, y1, w2, residual=x, want_stats=True)
    layer.x = n2
    mws = B.alloc_train_workspace(cm)
    y2 = B.forward_train(cm, layer, mws)
    ids = B.workspace_views(cm, mws)["ids"].clone().long()

    mg = B.backward(cm, layer, dy, mws)
    dh, dw2, _ = B.norm_backward(c2, hh, w2, None, r2, mg["dx"], dh=dy)          # the residual stream carries dy on
    fg = B.ffn_backward(cf, n1, wg, wu, wd, dh, fws)
    dx, dw1, db1 = B.norm_backward(c1, x, w1, m1, r1, fg["dx"], dh=dh, want_bias=True)
    torch.cuda.synchronize()
    assert B.device_status() == 0

    leaf = {"x": x, "w1": w1, "b1": b1, "w2": w2, "wg": wg, "wu": wu, "wd": wd}
    L = {q: t.double().requires_grad_() for q, t in leaf.items()}
    moe = {q: t.double() for q, t in (("router", layer.w_router), ("gate", layer.w_gate), ("up", layer.w_up),
                                      ("down", layer.w_down))}
    a1 = norm64(L["x"], L["w1"], L["b1"], 1e-5, kind == "rms")
    u = a1 @ L["wg"].T
    act_u = u * torch.sigmoid(u) if act == "silu" else torch.nn.functional.gelu(u, approximate="tanh")
    out1 = (act_u * (a1 @ L["wu"].T)) @ L["wd"].T
    hidden = out1 + L["x"]
    out2 = moe64(norm64(hidden, L["w2"], None, 1e-5, True), moe, ids, k)
    total = ((out2 + hidden) * dy.double()).sum()
    grads = dict(zip(L, torch.autograd.grad(total, list(L.values()))))
    got = {"x": dx, "w1": dw1, "b1": db1, "w2": dw2, "wg": fg["dw_gate"], "wu": fg["dw_up"], "wd": fg["dw_down"]}
    got = {"y2": y2, "h": hh, **got}
    want = {"y2": out2.detach(), "h": hidden.detach(), **grads}
    for q in want:
        err = (got[q].double() - want[q]).norm() / want[q].norm()
        assert err <= STEPS * HALF, f"{q}: {float(err):.2e}"


@pytest.mark.parametrize("T", [1, 50, 400])
def test_serving_norm_quantiser_product(T):
    d, N = 640, 1032
    g = torch.Generator(device="cuda").manual_seed(T)
    x, res = (torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.ones(d, device="cuda", dtype=torch.bfloat16)
    wq, ws = B.quantize_fp8(torch.randn(N, d, generator=g, device="cuda") * 0.05, 128)
    cfg = B.norm_config(T, d, kind="rms")

    def step():
        n, h, _, _ = B.norm_forward(cfg, x, w, residual=res)
        q, s = B.quantize_fp8(n)
        return n, h, q, s, B.gemm_fp8(q, s, wq, ws)

    def holds(n, h, q, s, y):
        assert torch.equal(h, (x.float() + res.float()).to(torch.bfloat16))
        a = q.double() * s.double().repeat_interleave(128, 1)[:, :d]
        b = wq.double() * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :d]
        want = a @ b.T
        tol = HALF * 1.01 * want.abs() + 2.0 ** -17 * (a.abs() @ b.abs().T)
        assert ((y.double() - want).abs() <= tol).all()
        # a code is off by half a step of 2^-3 of the value, or of the smallest code's 2^-9 steps of the scale
        off = (a - n.double()).abs()
        assert (off <= 2.0 ** -4 * n.double().abs() * 1.0001 + 2.0 ** -10 * s.double().repeat_interleave(128, 1)[:, :d]).all()

    holds(*step())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(torch.randn(T, d, generator=g, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    holds(*out)


def test_a_call_given_a_stream_allocates_on_it():
    """Outputs and a workspace of the call's own belong to the given stream: the current stream's next allocation of
    the same size is not handed memory that the call, still running there, had dropped."""
    T, d, h = 300, 512, 640
    g = torch.Generator(device="cuda").manual_seed(7)
    x, w, wg, wd = (torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16) for s in ((T, d), (d,), (h, d), (d, h)))
    ncfg, fcfg = B.norm_config(T, d), B.ffn_config(T, d, h)
    side = torch.cuda.Stream()

    def calls(**kw):
        y, _, mean, rstd = B.norm_forward(ncfg, x, w, want_stats=True, **kw)
        ws = B.alloc_ffn_workspace(fcfg, train=True)
        side.wait_stream(torch.cuda.current_stream())
        f = B.ffn_forward_train(fcfg, x, wg, wg, wd, ws, **kw)
        q, s = B.quantize_fp8(x, **kw)
        p, t = B.quantize_fp8(wg, 128, **kw)
        grads = B.ffn_backward(fcfg, x, wg, wg, wd, f, ws, **kw)
        out = [y, f, B.ffn_forward(fcfg, x, wg, wg, wd, **kw), q, B.gemm_fp8(q, s, p, t, **kw),
               *B.norm_backward(ncfg, x, w, mean, rstd, y, want_bias=True, **kw), *grads.values()]
        torch.cuda.synchronize()
        return out

    want = calls()
    side.wait_stream(torch.cuda.current_stream())
    got = calls(stream=side)
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    del a, b
    while got:
        t = got.pop()
        at, shape, dtype = t.data_ptr(), t.shape, t.dtype
        del t
        assert torch.empty(shape, dtype=dtype, device="cuda").data_ptr() != at
