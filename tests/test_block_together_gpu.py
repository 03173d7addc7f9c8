"""The operators as a block uses them, one after the other, forward and backward,
against the 64-bit form of the whole: a 1D block (norm per token, projection, gated
linear recurrence, projection, norm, feed-forward), its prefill and decoding, and a
grid block (group norm with SiLU, 2D Hyena, feed-forward).

Bars: every stage of the fp32 block is within its own test's bar; through the chain
they are bounded here by 2e-5 of the largest value of each output or gradient (about
a hundred fp32 roundings of intermediate values that do not exceed it by much), in
bf16 by 16 half steps (the stages' outputs are rounded a dozen times on the way)."""
import numpy as np
import pytest
import torch

import oracle
import subquadratic_sequence_amd as hs
from synth import make_nd
from tests import block_ref
from tests.gpu_util import to_dev

pytestmark = pytest.mark.gpu
BAR = {torch.float32: 2e-5, torch.bfloat16: 16 * 2.0 ** -8}


def near(name, got, want, dtype):
    err = (got.double().cpu() - want).abs().max().item() / want.abs().max().item()
    print(f"{name}: {err:.2e}", flush=True)
    assert err <= BAR[dtype], (name, err)


def weights(D, F, G, seed, dtype):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return dict(ga=1 + 0.1 * rnd(D), be=0.1 * rnd(D), wp=(rnd(D, 3 * D) * D ** -0.5).to(dtype),
                bias=torch.rand(D, generator=gen) * 2, wo=(rnd(D, D) * D ** -0.5).to(dtype), ga2=1 + 0.1 * rnd(D),
                be2=0.1 * rnd(D), w_in=(rnd(D, 2 * F) * D ** -0.5).to(dtype), w_out=(rnd(F, D) * F ** -0.5).to(dtype))


def block_ref_1d(x, w, G, reset):
    B, L, D = x.shape
    n, _, _ = block_ref.group_norm(x.reshape(B * L, 1, D), G, w["ga"], w["be"])
    p = n.reshape(B, L, D) @ w["wp"]
    m, _ = block_ref.glr(p[..., :D], p[..., D:2 * D], p[..., 2 * D:], w["bias"], reset=reset)
    r = x + m @ w["wo"]
    n2, _, _ = block_ref.group_norm(r.reshape(B * L, 1, D), 1, w["ga2"], w["be2"])
    return r + block_ref.ffn(n2.reshape(B * L, D), w["w_in"], w["w_out"], "silu")[0].reshape(B, L, D)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sequence_block_trains(dtype):
    B, L, D, F, G = 2, 300, 128, 344, 8
    gen = torch.Generator().manual_seed(0)
    x, dy = (torch.randn(B, L, D, generator=gen).to(dtype) for _ in range(2))
    reset = (torch.rand(B, L, generator=gen) < 0.02).to(torch.uint8)
    w = weights(D, F, G, 1, dtype)
    c = {k: t.cuda() for k, t in w.items()}
    xc, dyc, rc = x.cuda(), dy.cuda(), reset.cuda()
    T = B * L
    f = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    # forward
    m1, r1, m2, r2 = f(T, G), f(T, G), f(T, 1), f(T, 1)
    n = hs.hyena_group_norm_fwd(xc.view(T, D), G, gamma=c["ga"], beta=c["be"], mean=m1, rstd=r1)
    p = (n @ c["wp"]).view(B, L, 3 * D)
    v, fg, g = p[..., :D], p[..., D:2 * D], p[..., 2 * D:]
    m = hs.hyena_glr_fwd(v, fg, g=g, bias=c["bias"], reset=rc)
    r = xc + m @ c["wo"]
    n2 = hs.hyena_group_norm_fwd(r.view(T, D), 1, gamma=c["ga2"], beta=c["be2"], mean=m2, rstd=r2)
    y = r + hs.hyena_ffn_fwd(n2, c["w_in"], c["w_out"]).view(B, L, D)
    # backward
    d_ffn = hs.hyena_ffn_bwd(n2, c["w_in"], c["w_out"], dyc.view(T, D))
    d_n2 = hs.hyena_group_norm_bwd(r.view(T, D), d_ffn["dx"], 1, m2, r2, gamma=c["ga2"], beta=c["be2"])
    dr = dyc + d_n2["dx"].view(B, L, D)
    dm = (dr.view(T, D) @ c["wo"].t().contiguous()).view(B, L, D)
    d_glr = hs.hyena_glr_bwd(v, fg, dm, g=g, bias=c["bias"], reset=rc)
    dn = d_glr["dp"].view(T, 3 * D) @ c["wp"].t().contiguous()
    d_n1 = hs.hyena_group_norm_bwd(xc.view(T, D), dn, G, m1, r1, gamma=c["ga"], beta=c["be"])
    dx = dr + d_n1["dx"].view(B, L, D)
    got = dict(y=y, x=dx, ga=d_n1["dgamma"], be=d_n1["dbeta"], bias=d_glr["dbias"], ga2=d_n2["dgamma"],
               be2=d_n2["dbeta"], w_in=d_ffn["dw_in"], w_out=d_ffn["dw_out"],
               wp=n.t().contiguous() @ d_glr["dp"].view(T, 3 * D))
    wd = {k: t.double().requires_grad_(True) for k, t in w.items()}
    xd = x.double().requires_grad_(True)
    ry = block_ref_1d(xd, wd, G, reset)
    names = ["ga", "be", "bias", "ga2", "be2", "w_in", "w_out", "wp"]
    gr = torch.autograd.grad((ry * dy.double()).sum(), [xd] + [wd[k] for k in names])
    near("y", got["y"], ry.detach(), dtype)
    for k, want in zip(["x"] + names, gr):
        near("d" + k, got[k], want, dtype)


def test_prefill_then_decode():
    # a padded batch is prefilled, then continued token by token: the same as all at once
    B, L, D, F, G, S = 3, 60, 128, 344, 8, 7
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(B, L, D, generator=gen).cuda()
    lens = torch.tensor([20, 33, 41], dtype=torch.int32).cuda()
    slots = torch.tensor([5, 0, 3], dtype=torch.int32).cuda()
    c = {k: t.cuda() for k, t in weights(D, F, G, 4, torch.float32).items()}

    def mix(h, prefill):
        n = hs.hyena_group_norm_fwd(h.reshape(-1, D), G, gamma=c["ga"], beta=c["be"]) @ c["wp"]
        p = n.view(*h.shape[:-1], 3 * D)
        return p[..., :D], p[..., D:2 * D], p[..., 2 * D:]

    def rest(h, m):
        r = h + m @ c["wo"]
        n2 = hs.hyena_group_norm_fwd(r.reshape(-1, D), 1, gamma=c["ga2"], beta=c["be2"])
        return r + hs.hyena_ffn_fwd(n2, c["w_in"], c["w_out"]).view_as(r)

    v, f, g = mix(x, True)
    whole = rest(x, hs.hyena_glr_fwd(v, f, g=g, bias=c["bias"]))
    state, last = torch.zeros(S, D, device="cuda"), torch.empty(B, D, device="cuda")
    m = hs.hyena_glr_fwd(v, f, g=g, bias=c["bias"], lens=lens, h_last=last)
    out = rest(x, m)
    state[slots.long()] = last
    pos = lens.tolist()
    for b in range(B):
        near(f"prefill {b}", out[b, :pos[b]], whole[b, :pos[b]].double().cpu(), torch.float32)
    for step in range(15):
        xt = torch.stack([x[b, pos[b] + step] for b in range(B)])
        vt, ft, gt = mix(xt, False)
        yt = rest(xt, hs.hyena_glr_step(state, vt, ft, g=gt, bias=c["bias"], slots=slots))
        want = torch.stack([whole[b, pos[b] + step] for b in range(B)])
        near(f"step {step}", yt, want.double().cpu(), torch.float32)


def test_grid_block_with_the_2d_operator():
    inp = make_nd(5, 2, 1, 16, 16, 64, N=2)
    x = torch.from_numpy(np.asarray(inp.u, np.float32))
    gen = torch.Generator().manual_seed(6)
    ga, be = 1 + 0.1 * torch.randn(64, generator=gen), 0.1 * torch.randn(64, generator=gen)
    w_in, w_out = torch.randn(64, 176, generator=gen) / 8, torch.randn(88, 64, generator=gen) / 9
    layer = hs.HyenaNDLayer(1, 16, 16, 64, 2)
    hs.hyena_nd_filter_gen(layer, *(to_dev(a) for a in (inp.w1, inp.b1, inp.w2, inp.b2, inp.w3, inp.b3, inp.decay)))
    n = hs.hyena_group_norm_fwd(x.cuda(), 8, gamma=ga.cuda(), beta=be.cuda(), act=hs.ACT_SILU)
    h = hs.hyena_nd_fwd(layer, n, to_dev(inp.w_in), to_dev(inp.dskip), to_dev(inp.gate_a), to_dev(inp.gate_b),
                        to_dev(inp.w_out))
    y = hs.hyena_ffn_fwd(h, w_in.cuda(), w_out.cuda(), act=hs.ACT_GELU)
    rn, _, _ = block_ref.group_norm(x.double().reshape(2, 256, 64), 8, ga.double(), be.double(), name="silu")
    K = oracle.nd_filter(inp.filter_params, 1, 16, 16, 2, 64, circular=False)
    rh = oracle.hyena_nd_fwd(rn.reshape(x.shape).numpy(), inp.w_in, inp.dskip, inp.gate_a, inp.gate_b, inp.w_out, K,
                             conv="fft", circular=False)
    ry, _ = block_ref.ffn(torch.from_numpy(rh).reshape(-1, 64), w_in.double(), w_out.double(), "gelu")
    err = (y.double().cpu().reshape(-1, 64) - ry).abs().max().item() / ry.abs().max().item()
    # the 2D operator's own bar (1e-4 of the largest value), carried through one feed-forward block of gain about 1
    assert err <= 2e-4, err
