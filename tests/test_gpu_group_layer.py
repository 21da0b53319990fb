"""The layer with routing by groups, experts in 8 bits and 8-bit activation checkpoints: the chained calls, and its gradients."""
import numpy as np
import pytest
import torch

from oracle import group_route_oracle as O

pytestmark = pytest.mark.gpu


def rel(a, b):
    a, b = a.double(), b.double()
    return float((a - b).norm() / b.norm())


def parts(T, h, E, F, seed=0, shared=False):
    g = torch.Generator().manual_seed(seed)
    mk = lambda *s: (torch.randn(*s, generator=g) / s[-1] ** 0.5).bfloat16().cuda()
    p = dict(w_r=(torch.randn(h, E, generator=g) / h**0.5).bfloat16().cuda(), bias=(torch.randn(E, generator=g) * 0.05).cuda(),
             w_gate=mk(E, F, h), w_up=mk(E, F, h), w_down=mk(E, h, F))
    if shared:
        p["shared"] = (mk(1, F, h), mk(1, F, h), mk(1, h, F))
    return p, torch.randn(T, h, generator=g).bfloat16().cuda()


def layer(T, h, E, k, F, p, **kw):
    from top_routing_dispatch_moe_gb300.layer import MoELayer
    return MoELayer(T=T, h=h, E=E, k=k, F=F, gating=kw.pop("gating", "sigmoid"), cf=kw.pop("cf", 0.0), R=1, alpha=0.01, routing="group",
                    groups=kw.pop("groups", 4), top_groups=2, route_scale=2.5, **p, **kw)


@pytest.mark.parametrize("experts", ["dtype", "int8", "nvfp4"])
@pytest.mark.parametrize("T,E,cf,shared", [(3, 16, 0.0, False), (257, 64, 0.0, True), (200, 32, 1.0, False)])
def test_forward_is_the_chain_of_its_calls(gpu_lib, experts, T, E, cf, shared):
    h, k, F = 128, 4, 96
    p, x = parts(T, h, E, F, T, shared)
    lay = layer(T, h, E, k, F, p, cf=cf, experts=experts)
    y = lay.forward(x).clone()
    torch.cuda.synchronize()
    assert gpu_lib.moe_check_device_error() == gpu_lib.MOE_OK
    r = lay.r_out
    want = O.route(r["logits"].double().cpu().numpy(), p["bias"].cpu().numpy(), k, 4, 2, "sigmoid", 2, True, 2.5)
    np.testing.assert_array_equal(r["topk_ids"].cpu().numpy(), want["ids"])
    np.testing.assert_allclose(r["gates"].cpu().numpy(), want["gates"], rtol=1e-5)
    # the whole layer in 64 bits on the same choice; capacity drops as the dispatch marked them
    X = x.double()
    w = [p[n].double() for n in ("w_gate", "w_up", "w_down")]
    ids, drop = torch.from_numpy(want["ids"]).cuda(), lay.d_out["drop_mask"].bool()
    ref = torch.zeros_like(X)
    for j in range(k):
        e = ids[:, j]
        a = torch.nn.functional.silu(torch.einsum("th,tfh->tf", X, w[0][e])) * torch.einsum("th,tfh->tf", X, w[1][e])
        ref += torch.where(drop[:, j, None], 0.0, torch.einsum("tf,thf->th", a, w[2][e]) * torch.from_numpy(want["gates"][:, j, None]).cuda())
    if shared:
        s = [v[0].double() for v in p["shared"]]
        ref += (torch.nn.functional.silu(X @ s[0].t()) * (X @ s[1].t())) @ s[2].t()
    # bf16: roundings of act, eout and y, 2^-9 rms each at most. 8 bits: a uniform error of a step of amax / 127, amax up to 4 (rows,
    # channels) or 10 (act) times the rms: 0.9 % for x and each weight, 2.3 % for act. 4 bits: 10 % for each of the five.
    assert rel(y, ref) <= {"dtype": 0.01, "int8": 0.05, "nvfp4": 0.35}[experts]
    graph = lay.capture_forward(x)
    lay.y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(lay.y, y)


@pytest.mark.parametrize("gating,renorm", [("sigmoid", True), ("softmax", False)])
@pytest.mark.parametrize("checkpoint", ["dtype", "int8"])
def test_gradients_against_autograd(gpu_lib, gating, renorm, checkpoint):
    T, h, E, k, F = 150, 128, 16, 3, 200
    p, x = parts(T, h, E, F, 5, True)
    lay = layer(T, h, E, k, F, p, gating=gating, renorm=renorm, backward=True, checkpoint=checkpoint)
    lay.forward(x, save=True)
    dy = torch.randn(T, h, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    lay.act.fill_(float("nan")) if checkpoint == "int8" else None      # the backward computes it again
    g = lay.backward(x, dy)
    torch.cuda.synchronize()
    assert gpu_lib.moe_check_device_error() == gpu_lib.MOE_OK and g["d_bias"] is None
    leaves = {"x": x.double(), "W_r": p["w_r"].double(), **{"W_" + n: p["w_" + n].double() for n in ("gate", "up", "down")}}
    leaves = {n: v.clone().requires_grad_(True) for n, v in leaves.items()}
    ids = lay.r_out["topk_ids"].long()
    L = leaves["x"] @ leaves["W_r"]
    s = torch.sigmoid(L) if gating == "sigmoid" else torch.softmax(L, 1)
    c = s.gather(1, ids)
    gates = 2.5 * (c / c.sum(1, keepdim=True) if renorm else c)
    P = (s / s.sum(1, keepdim=True)).mean(0)
    y = torch.zeros(T, h, dtype=torch.float64, device="cuda")
    for j in range(k):
        e = ids[:, j]
        gt, up = (torch.einsum("th,tfh->tf", leaves["x"], leaves[n][e]) for n in ("W_gate", "W_up"))
        y = y + torch.einsum("tf,thf->th", torch.nn.functional.silu(gt) * up, leaves["W_down"][e]) * gates[:, j, None]
    sh = [v[0].double() for v in p["shared"]]
    y = y + (torch.nn.functional.silu(leaves["x"] @ sh[0].t()) * (leaves["x"] @ sh[1].t())) @ sh[2].t()
    loss = (y * dy.double()).sum() + 0.01 * E * (lay.r_out["f"].double() * P).sum()
    want = torch.autograd.grad(loss, list(leaves.values()))
    # bf16 operands of each product (act, d_act, d_gu, eout ...): 2^-9 rms a factor, 1 % in all; the checkpoint's g and u are off by a
    # uniform error of a step of amax / 127, amax up to 4 times the rms: 0.9 % each, of which d_gu and act carry at most twice
    tol = 0.02 if checkpoint == "dtype" else 0.045
    for n, w in zip(leaves, want):
        assert rel(g["d" + n], w) <= tol, (n, rel(g["d" + n], w))


def test_layers_share_the_scratch(gpu_lib):
    from top_routing_dispatch_moe_gb300.layer import MoELayer
    T, h, E, k, F = 100, 64, 8, 2, 72
    ps = [parts(T, h, E, F, i, True) for i in range(2)]
    scratch = torch.full((MoELayer.checkpoint_scratch(T * k, F, T),), float("nan"), dtype=torch.bfloat16, device="cuda")
    dy = torch.randn(T, h, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    alone = []
    for p, x in ps:
        lay = layer(T, h, E, k, F, p, backward=True, checkpoint="int8")
        lay.forward(x, save=True)
        alone.append({n: v.clone() for n, v in lay.backward(x, dy).items() if v is not None})
    lays = [layer(T, h, E, k, F, p, backward=True, checkpoint="int8", scratch=scratch) for p, _ in ps]
    for lay, (_, x) in zip(lays, ps):
        lay.forward(x, save=True)
    scratch.fill_(float("nan"))
    for i in (1, 0):
        g = lays[i].backward(ps[i][1], dy)
        torch.cuda.synchronize()
        for n, v in alone[i].items():
            assert torch.equal(g[n], v), n
    with pytest.raises(ValueError):
        layer(T, h, E, k, F, ps[0][0], backward=True, checkpoint="int8", scratch=scratch[:100])
    assert gpu_lib.moe_check_device_error() == gpu_lib.MOE_OK


def test_refusals(gpu_lib):
    p, x = parts(8, 64, 16, 64)
    for kw in (dict(experts="int4"), dict(gating="softmax_renorm"), dict(experts="int8", backward=True), dict(checkpoint="int8"),
               dict(checkpoint="int4", backward=True),
               dict(checkpoint="int8", backward=True, scratch=torch.empty(1 << 16, dtype=torch.bfloat16))):      # (of the host)
        with pytest.raises(ValueError):
            layer(8, 64, 16, 2, 64, p, **kw)
    for kw in (dict(), dict(experts="int8")):
        with pytest.raises(NotImplementedError):
            layer(8, 64, 16, 2, 64, p, **kw).native_desc()
    with pytest.raises(gpu_lib.MoEError):
        layer(8, 64, 16, 2, 64, p, groups=5).forward(x)
