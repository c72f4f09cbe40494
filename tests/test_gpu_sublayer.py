"""FeedForwardSublayer: dense bf16, dense MXFP8 and MoE sublayers chained along
one residual stream, and a dense stack trained by its own backward passes."""
import pytest
import torch

import oracle as O
from lmoe_inputs import configs as C
from tests import _ffn_reference as R
from tests._harness import built_library, gpu_inputs, make_layer

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def ops():
    built_library()
    import latent_mixture_experts_gb300 as P
    return P


def _dense(d, F, g):
    def rnd(*s, std):
        return (torch.randn(*s, device="cuda", generator=g) * std).bfloat16()
    return {"gate": rnd(F, d, std=d ** -0.5), "up": rnd(F, d, std=d ** -0.5), "down": rnd(d, F, std=F ** -0.5)}


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 16, 130])
def test_dense_then_mxfp8_then_moe(ops, T, stream):
    wl = C.workload("k3_tiny_t16")
    d, F = wl.cfg.d_model, wl.cfg.d_shared_ff
    g = torch.Generator(device="cuda").manual_seed(T)
    norms = [(1 + 0.1 * torch.randn(d, device="cuda", generator=g)).bfloat16() for _ in range(3)]
    W = _dense(d, F, g)
    M = {}
    for n, o, i in (("gate", F, d), ("up", F, d), ("down", d, F)):
        M[n], M[n + "_s"] = R.mx_random((o, i), i ** -0.5, g, "cuda")
    E, _ = gpu_inputs(wl, T=1)
    moe = make_layer(wl, E, max_tokens=T, keep_f32=False)
    subs = [ops.FeedForwardSublayer(norms[0], ops.GatedFFN(W, max_tokens=T), EPS),
            ops.FeedForwardSublayer(norms[1], ops.GatedFFN(M, max_tokens=T), EPS),
            ops.FeedForwardSublayer(norms[2], moe, EPS)]
    x = torch.randn(T, d, device="cuda", generator=g).bfloat16()
    r = torch.randn(T, d, device="cuda", generator=g).to(stream)
    for i, sub in enumerate(subs):
        y, h = sub.forward(x, r)
        nref, href = R.norm(x, r, norms[i], EPS)
        assert torch.equal(h, href)
        if i == 0:
            ref = R.forward(nref, W["gate"], W["up"], W["down"], "situ")[0]
        elif i == 1:
            wg, wu, wd = (R.mx_decode(M[n], M[n + "_s"]) for n in ("gate", "up", "down"))
            q = R.mx_encode(nref)[0]
            a, v, _, _ = R.act_parts(q @ wg.T, q @ wu.T, "situ")
            ref = R.mx_encode(a * v)[0] @ wd.T
        else:
            # the layer on the same norm, rounded as the sublayer passes it on
            n, _, _ = ops.lmoe_add_rms_norm(x, norms[i], EPS, residual=r)
            ref = moe.lmoe_forward(n).to(R.D)
        # norm, hidden and output roundings: three of 2^-8 / sqrt(3) at most, in the root mean square
        assert R.rel_l2(y, ref) <= 2.0 ** -8 * (2 if i == 1 else 1), (i, R.rel_l2(y, ref))
        x, r = y, h
    moe.lmoe_sync_status()
    moe.close()


def test_moe_sublayer_against_the_oracle(ops):
    """The MoE layer behind the norm, as the fp64 oracle computes it from the same norm."""
    wl = C.workload("k3_tiny_t16")
    W, x = gpu_inputs(wl)
    layer = make_layer(wl, W, max_tokens=wl.T, keep_f32=False)
    w = torch.ones(wl.cfg.d_model, device="cuda", dtype=torch.bfloat16)
    r = torch.zeros_like(x)
    y, h = ops.FeedForwardSublayer(w, layer, EPS).forward(x, r)
    n, _, _ = ops.lmoe_add_rms_norm(x, w, EPS, residual=r)
    _, idx, _ = layer.lmoe_forward(n, return_routing=True)
    import numpy as np
    olayer = O.Layer(wl.cfg, O.numpy_inputs({k: v.cpu() for k, v in W.items()}))
    ref = O.forward(olayer, n.cpu().view(torch.int16).numpy().view(np.uint16), idx=idx.cpu().numpy())["delta"]
    got = y.cpu().double().numpy()
    rel = np.sqrt(((got - ref) ** 2).sum(-1) / (ref ** 2).sum(-1))
    assert rel.max() <= 1e-2
    layer.close()


def _loss_grads(P, x, r, target):
    """64-bit loss and gradients of two sublayers (autograd over the plain forward)."""
    leaves = [t.to(R.D).requires_grad_(True) for t in P]
    n0, g0, u0, d0, n1, g1, u1, d1 = leaves

    def sub(a, stream, n, gate, up, down):
        h = stream + a
        y = n * h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
        g, u = y @ gate.T, y @ up.T
        act = 4 * torch.tanh(g / 4) * torch.sigmoid(g) * 25 * torch.tanh(u / 25)
        return act @ down.T, h
    a, h = sub(x.to(R.D), r.to(R.D), n0, g0, u0, d0)
    a, h = sub(a, h, n1, g1, u1, d1)
    loss = ((h + a - target.to(R.D)) ** 2).mean()
    return float(loss), torch.autograd.grad(loss, leaves)


def test_training_a_stack(ops):
    """Two sublayers, fp32 residual stream: gradients against 64-bit autograd, and five optimizer steps that update
    the weights in place lower the loss."""
    T, d, F = 200, 256, 384
    g = torch.Generator(device="cuda").manual_seed(1)
    W = [_dense(d, F, g) for _ in range(2)]
    norms = [torch.ones(d, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    subs = [ops.FeedForwardSublayer(norms[i], ops.GatedFFN(W[i], max_tokens=T, training=True), EPS) for i in range(2)]
    x = torch.randn(T, d, device="cuda", generator=g).bfloat16()
    r = torch.randn(T, d, device="cuda", generator=g)
    target = torch.randn(T, d, device="cuda", generator=g)
    losses = []
    for step in range(5):
        y0, h0, s0 = subs[0].forward_train(x, r)
        y1, h1, s1 = subs[1].forward_train(y0, h0)
        out = h1 + y1.float()
        losses.append(float(((out - target) ** 2).mean()))
        dout = 2 * (out - target) / out.numel()
        b1 = subs[1].backward(dout.bfloat16(), dout, s1)
        b0 = subs[0].backward(b1.dx.bfloat16(), b1.dx, s0)
        if step == 0:
            P = [norms[0], W[0]["gate"], W[0]["up"], W[0]["down"], norms[1], W[1]["gate"], W[1]["up"], W[1]["down"]]
            loss, want = _loss_grads(P, x, r, target)
            assert abs(loss - losses[0]) <= 1e-2 * loss
            got = [b0.norm_w, b0.gate, b0.up, b0.down, b1.norm_w, b1.gate, b1.up, b1.down]
            # a dozen bf16 roundings along the way, each at most 2^-8 / sqrt(3) in the root mean square: 2^-6
            for a, b in zip(got, want):
                assert R.rel_l2(a, b) <= 2.0 ** -6, R.rel_l2(a, b)
        for sub, grad, w in ((subs[0], b0, W[0]), (subs[1], b1, W[1])):
            for n in ("gate", "up", "down"):
                w[n].sub_((20.0 * getattr(grad, n).float()).bfloat16())
            sub.norm_w.sub_((20.0 * grad.norm_w).bfloat16())
    assert losses[-1] < 0.95 * losses[0], losses


def test_blocks_on_streams_of_their_own(ops):
    """Dense, MXFP8 and MoE blocks and the norms, each on a stream of its own at the same time: the bits of the calls
    one after the other."""
    wl = C.workload("k3_tiny_t16")
    d, F = wl.cfg.d_model, 512
    g = torch.Generator(device="cuda").manual_seed(2)
    W = _dense(d, F, g)
    M = {}
    for n, o, i in (("gate", F, d), ("up", F, d), ("down", d, F)):
        M[n], M[n + "_s"] = R.mx_random((o, i), i ** -0.5, g, "cuda")
    E, _ = gpu_inputs(wl, T=1)
    w = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).bfloat16()
    xs = {T: torch.randn(T, d, device="cuda", generator=g).bfloat16() for T in (1, 16, 40, 300, 1100)}
    rs = {T: torch.randn(T, d, device="cuda", generator=g).bfloat16() for T in xs}

    def dense(T):
        block = ops.GatedFFN(W, max_tokens=T, training=True)

        def call():
            y, gg, u = block.lmoe_ffn_forward(xs[T], save=True)
            return (y, *block.lmoe_ffn_backward(xs[T], gg, u, y))
        return call

    def mx(T):
        block = ops.GatedFFN(M, max_tokens=T)
        q, s, _ = ops.lmoe_add_rms_norm(xs[T], w, EPS, out_format="mxfp8")
        return lambda: (block.lmoe_ffn_forward_mx(q, s),)

    def moe(T):
        layer = make_layer(wl, E, max_tokens=T, keep_f32=False)
        return lambda: (layer.lmoe_forward(xs[T]),)

    def norm(T):
        return lambda: ops.lmoe_add_rms_norm_backward(xs[T], rs[T], w, EPS, dh=xs[T])
    calls = [dense(300), dense(16), mx(16), mx(1100), moe(40), norm(1100), dense(1100), mx(1)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(20):
        got = []
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(c())
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
