"""The channels-last group norm against its 64-bit form.

Bars (u = 2^-24; |xh| <= X, the largest normalised value). Sums run over n terms in
runs of 4 rows and a tree above them, so their relative error is taken as
32 u of the sum of magnitudes. Mean: 32 u avg|x|. Variance: from deviations, each with
the mean's error and its own rounding: relative 64 u (1 + (mean / std)^2 32 u); rstd half
of that. xh: error of the mean times rstd, plus the rstd's, plus 3 u: with r = max|x| rstd
at most (32 r + 64 X) u. y: |gamma| times it, times the slope of the activation (<= 1.13),
plus 4 u |y| and, for the exp2-based tails, 8 u. Gradients: dn carries the slope's error
(second derivative <= 1, times the error of n), m1 and m2 are averages of such terms, and
all are multiplied by rstd: (8 errors of y) rstd max|dy gamma|. Outputs in bf16 add half a
step of their own value."""
import pytest
import torch

import subquadratic_sequence_amd as hs
from tests import block_ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ACT = {"none": hs.ACT_NONE, "silu": hs.ACT_SILU, "gelu": hs.ACT_GELU}
U = 2.0 ** -24


def make(B, S, C, G, dtype, seed=0, affine=True, lens=False, offset=1.0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    d = dict(x=(rnd(B, S, C) * (0.5 + torch.rand(C, generator=gen)) + offset * rnd(C)).to(DT[dtype]),
             dy=rnd(B, S, C).to(DT[dtype]), gamma=1 + 0.3 * rnd(C) if affine else None,
             beta=0.3 * rnd(C) if affine else None,
             lens=torch.randint(0, S + 1, (B,), generator=gen).to(torch.int32) if lens else None)
    return d


def near(name, got, want, bar):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), name
    over = (got - want).abs() - bar
    assert (over <= 0).all(), f"{name}: {over.max().item():.3e} over the bar, max error {(got - want).abs().max():.3e}"


def run(d, G, act, check=True):
    dev = {k: (t.cuda() if t is not None else None) for k, t in d.items()}
    B, S, C = d["x"].shape
    mean, rstd = torch.empty(B, G, device="cuda"), torch.empty(B, G, device="cuda")
    y = hs.hyena_group_norm_fwd(dev["x"], G, gamma=dev["gamma"], beta=dev["beta"], act=ACT[act], lens=dev["lens"],
                                mean=mean, rstd=rstd)
    g = hs.hyena_group_norm_bwd(dev["x"], dev["dy"], G, mean, rstd, gamma=dev["gamma"], beta=dev["beta"],
                                act=ACT[act], lens=dev["lens"])
    if not check:
        return y, mean, rstd, g
    x = d["x"].double().requires_grad_(True)
    ga = (d["gamma"] if d["gamma"] is not None else torch.ones(C)).double().requires_grad_(True)
    be = (d["beta"] if d["beta"] is not None else torch.zeros(C)).double().requires_grad_(True)
    ry, rm, rr = block_ref.group_norm(x, G, ga, be, name=act, lens=d["lens"])
    rdx, rdg, rdb = torch.autograd.grad((ry * d["dy"].double()).sum(), [x, ga, be])
    ry, rm, rr, xd = ry.detach(), rm.detach(), rr.detach(), x.detach()
    cg = C // G
    avg = xd.abs().max().item()
    near("mean", mean, rm, 32 * U * avg)
    ratio = (rm.abs() * rr).max().item() ** 2 * 32 * U
    near("rstd", rstd, rr, 64 * U * (1 + ratio) * rr)
    rs = rr.repeat_interleave(cg, 1)[:, None]
    n = torch.full((B,), S) if d["lens"] is None else d["lens"].long()
    live = (torch.arange(S) < n[:, None])[..., None]
    xh = ((xd - rm.repeat_interleave(cg, 1)[:, None]) * rs * live).abs()
    X, r = xh.max().item(), (avg * rr.max().item() if n.max() > 0 else 0.0)
    err_n = (32 * r + 64 * X + 4) * U * ga.detach().abs().max().item()
    half = block_ref.half_step(d["x"].dtype) if d["x"].dtype == torch.bfloat16 else 0.0
    near("y", y, ry, 1.13 * err_n + (4 * U + half) * ry.abs() + 8 * U)
    size = d["dy"].double().abs().max().item() * ga.detach().abs().max().item()
    e = 8 * (err_n + 8 * U) * size * max(X, 1)
    near("dx", g["dx"], rdx, e * rs * max(X, 1) + half * rdx.abs())
    terms = float(n.sum()) + 1
    near("dbeta", g["dbeta"], rdb, 8 * (err_n + 8 * U) * size * terms)
    near("dgamma", g["dgamma"], rdg, 8 * (err_n + 8 * U) * size * max(X, 1) * terms)


# positions, channels, groups: rows by themselves in every lane split, groups that cut
# vectors, one group, a group per channel, one and many chunks
SHAPES = [(5, 1, 8, 1), (33, 1, 64, 8), (300, 1, 768, 12), (40, 1, 768, 1), (7, 1, 768, 768), (9, 1, 384, 32),
          (70, 1, 24, 1), (5, 1, 8192, 1), (3, 1, 8192, 8192), (6, 1, 4104, 3), (2100, 1, 40, 5),
          (1, 2, 8, 8), (3, 17, 72, 9), (2, 64, 384, 32), (2, 1000, 128, 8), (1, 4097, 320, 10), (1, 5000, 64, 64),
          (2, 3, 8192, 2), (2, 40, 8192, 4096), (600, 5, 64, 4), (2060, 3, 16, 2), (1, 9001, 8, 1), (4, 700, 2056, 8),
          # many samples in one launch and in two, more rows than workgroups
          (130, 40, 64, 8), (100, 300, 32, 4), (140, 2200, 64, 8), (1500, 1, 64, 8)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,S,C,G", SHAPES)
@pytest.mark.parametrize("act,lens", [("none", False), ("silu", True), ("gelu", False)])
def test_forward_and_gradients(B, S, C, G, dtype, act, lens):
    say(f"group_norm B={B} S={S} C={C} G={G} {dtype} {act} lens={lens}")
    run(make(B, S, C, G, dtype, seed=B + S + C + G, lens=lens), G, act)


@pytest.mark.parametrize("B,S,C,G", [(4, 1, 64, 4), (2, 500, 64, 4), (2, 3, 64, 4)])
def test_without_affine_and_far_means(B, S, C, G):
    run(make(B, S, C, G, "f32", seed=7, affine=False), G, "silu")
    # means 300 deviations away: the variance must not come from a difference of large sums
    run(make(B, S, C, G, "f32", seed=8, offset=300.0), G, "none")


@pytest.mark.parametrize("B,S,C,G", [(5, 1, 64, 4), (3, 700, 64, 4), (600, 4, 64, 4)])
def test_constant_and_empty_samples(B, S, C, G):
    d = make(B, S, C, G, "f32", seed=3)
    d["x"][0] = 2.5
    d["lens"] = torch.full((B,), S, dtype=torch.int32)
    d["lens"][1] = 0
    d["lens"][2] = -5
    if B > 3:
        d["lens"][3] = S + 100
    y, mean, rstd, g = run(d, G, "none", check=False)
    inv = torch.full((G,), 1e-5).rsqrt()
    assert torch.equal(mean[0].cpu(), torch.full((G,), 2.5))
    assert torch.allclose(rstd[0].cpu(), inv, rtol=1e-6, atol=0)
    for b in (1, 2):
        assert (mean[b] == 0).all() and torch.allclose(rstd[b].cpu(), inv, rtol=1e-6, atol=0)
        assert (y[b] == 0).all() and (g["dx"][b] == 0).all()
    assert torch.allclose(y[0].cpu(), d["beta"].expand(S, C), rtol=0, atol=1e-6)


@pytest.mark.parametrize("B,S,C,G", [(6, 1, 64, 4), (2, 900, 72, 9), (700, 6, 64, 4)])
def test_padding_never_enters(B, S, C, G):
    d = make(B, S, C, G, "f32", seed=13, lens=True)
    want = run(d, G, "silu", check=False)
    for bad in (float("nan"), float("inf")):
        e = {k: (t.clone() if t is not None else None) for k, t in d.items()}
        pad = torch.arange(S)[None] >= d["lens"][:, None]
        e["x"][pad] = bad
        e["dy"][pad] = bad
        got = run(e, G, "silu", check=False)
        for a, b in zip(want[:3], got[:3]):
            assert torch.equal(a, b)
        for k in want[3]:
            assert torch.equal(want[3][k], got[3][k]), k
        # a given y keeps what it holds there
        y = torch.full((B, S, C), 7.0, device="cuda")
        hs.hyena_group_norm_fwd(e["x"].cuda(), G, gamma=e["gamma"].cuda(), beta=e["beta"].cuda(), act=ACT["silu"],
                                lens=e["lens"].cuda(), y=y)
        assert (y.cpu()[pad] == 7).all() and torch.equal(y.cpu()[~pad], want[0].cpu()[~pad])


def test_in_place_and_grids():
    d = make(2, 4 * 6 * 8, 64, 8, "bf16", seed=17)
    x = d["x"].cuda().view(2, 4, 6, 8, 64)
    mean, rstd = torch.empty(2, 8, device="cuda"), torch.empty(2, 8, device="cuda")
    want = hs.hyena_group_norm_fwd(x, 8, act=hs.ACT_SILU, mean=mean, rstd=rstd)
    dy = d["dy"].cuda().view_as(x)
    g = hs.hyena_group_norm_bwd(x, dy, 8, mean, rstd, act=hs.ACT_SILU)
    dd = dy.clone()
    g2 = hs.hyena_group_norm_bwd(x, dd, 8, mean, rstd, act=hs.ACT_SILU, dx=dd)
    assert g2["dx"] is dd and all(torch.equal(g[k], g2[k]) for k in g)
    xi = x.clone()
    assert hs.hyena_group_norm_fwd(xi, 8, act=hs.ACT_SILU, y=xi) is xi and torch.equal(xi, want)


@pytest.mark.parametrize("B,S,C,G", [(3000, 1, 128, 8), (2, 5000, 128, 8), (1000, 20, 128, 8)])
def test_captured_replayed_and_two_streams(B, S, C, G):
    d = make(B, S, C, G, "bf16", seed=19)
    c = {k: (t.cuda() if t is not None else None) for k, t in d.items()}

    def both():
        mean, rstd = torch.empty(B, G, device="cuda"), torch.empty(B, G, device="cuda")
        y = hs.hyena_group_norm_fwd(c["x"], G, gamma=c["gamma"], beta=c["beta"], act=hs.ACT_GELU, mean=mean, rstd=rstd)
        g = hs.hyena_group_norm_bwd(c["x"], c["dy"], G, mean, rstd, gamma=c["gamma"], beta=c["beta"], act=hs.ACT_GELU)
        return [y, mean, rstd, g["dx"], g["dgamma"], g["dbeta"]]

    want = both()
    torch.cuda.synchronize()
    outs = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            outs.append(both())
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rec = both()
    for i in range(4):
        c["x"].copy_(make(B, S, C, G, "bf16", seed=40 + i)["x"].cuda())
        want = both()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(rec, want))
