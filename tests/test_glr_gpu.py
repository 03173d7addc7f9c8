"""The gated linear recurrence against its 64-bit form.

Bars. With f + bias <= 4 the state forgets at least 1 - a >= 0.0179 a step, so an
error of k 2^-24 a step sums to at most H k 2^-24 max|h|, H = min(L, 56). One step
has the gate (relative error 3 2^-24: exp2, reciprocal, their product), 1 - a (the
same), two products and a sum: k = 8; joining runs multiplies and adds the same
quantities once more. The gradients multiply up to four such factors and run the
scan twice: k = 32. Sums over positions (dbias) add their terms' errors. Outputs in
bf16 add half a step of their own value."""
import pytest
import torch

import subquadratic_sequence_amd as hs
from tests import block_ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(B, L, D, dtype, seed=0, gate=True, bias=True, h0=True, reset=False, lens=False, p_reset=0.05):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    p = rnd(B, L, 3 * D)
    p[..., D:2 * D].clamp_(-2, 2)
    d = dict(p=p.to(DT[dtype]), bias=torch.rand(D, generator=gen) * 2 if bias else None,
             h0=rnd(B, D) if h0 else None, dy=rnd(B, L, D).to(DT[dtype]), dh_last=rnd(B, D),
             reset=(torch.rand(B, L, generator=gen) < p_reset).to(torch.uint8) if reset else None,
             lens=torch.randint(0, L + 1, (B,), generator=gen).to(torch.int32) if lens else None, gate=gate, D=D)
    return d


def blocks(d, dev="cuda"):
    p, D = d["p"].to(dev), d["D"]
    mv = lambda t: None if t is None else t.to(dev)  # noqa: E731
    return dict(v=p[..., :D], f=p[..., D:2 * D], g=p[..., 2 * D:] if d["gate"] else None, bias=mv(d["bias"]),
                h0=mv(d["h0"]), reset=mv(d["reset"]), lens=mv(d["lens"]))


def reference(d, grads=False):
    a = {k: (t.double().requires_grad_(grads) if t is not None and t.is_floating_point() else t)
         for k, t in blocks(d, "cpu").items()}
    y, hl = block_ref.glr(**a)
    if not grads:
        return y, hl
    names = [k for k in ("v", "f", "g", "bias", "h0") if a[k] is not None]
    loss = (y * d["dy"].double()).sum() + (hl * d["dh_last"].double()).sum()
    gr = torch.autograd.grad(loss, [a[k] for k in names], allow_unused=True)
    return {"d" + k: (g if g is not None else torch.zeros_like(a[k])) for k, g in zip(names, gr)}


def check(name, got, want, dtype, k, H, scale=None, terms=1):
    got, want = got.double().cpu(), want
    scale = want.abs().max().item() if scale is None else scale
    bar = k * 2.0 ** -24 * H * terms * max(scale, 1e-30)
    if dtype == torch.bfloat16:
        bar = bar + block_ref.half_step(dtype) * want.abs() * (1 + 2.0 ** -8)
    bad = (got - want).abs() - bar
    assert torch.isfinite(got).all(), name
    assert (bad <= 0).all(), f"{name}: {bad.max().item():.3e} over the bar, max error {(got - want).abs().max():.3e}"


SHAPES = [(1, 1, 8), (2, 2, 64), (3, 63, 72), (2, 64, 64), (1, 65, 320), (2, 127, 8), (1, 129, 136), (3, 1000, 64),
          (1, 4097, 72), (17, 300, 1032)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D", SHAPES)
@pytest.mark.parametrize("masks", ["none", "reset", "lens", "both"])
def test_forward_and_gradients(B, L, D, dtype, masks):
    say(f"glr B={B} L={L} D={D} {dtype} {masks}")
    d = make(B, L, D, dtype, seed=B + L + D, reset=masks in ("reset", "both"), lens=masks in ("lens", "both"))
    a = blocks(d)
    H = min(L, 56)
    hl = torch.empty(B, D, device="cuda")
    y = hs.hyena_glr_fwd(**a, h_last=hl)
    ry, rhl = reference(d)
    check("y", y, ry, DT[dtype], 8, H)
    check("h_last", hl, rhl, torch.float32, 8, H)
    got = hs.hyena_glr_bwd(dy=d["dy"].cuda(), dh_last=d["dh_last"].cuda(), **a)
    want = reference(d, grads=True)
    for n in ("dv", "df", "dg"):
        check(n, got[n], want[n], DT[dtype], 32, H)
    check("dh0", got["dh0"], want["dh0"], torch.float32, 32, H, scale=want["dh0"].abs().max().item() + 1)
    df_max = want["df"].abs().max().item()
    # dbias is a sum of B L terms, each with the error of a df before its rounding, plus the sum's own
    check("dbias", got["dbias"], want["dbias"], torch.float32, 32, H, scale=df_max, terms=B * L)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_gate_bias_state(dtype):
    d = make(2, 333, 72, dtype, seed=5, gate=False, bias=False, h0=False)
    a = blocks(d)
    y = hs.hyena_glr_fwd(a["v"], a["f"])
    ry, _ = reference(d)
    check("y", y, ry, DT[dtype], 8, 56)
    d["dh_last"] = torch.zeros_like(d["dh_last"])
    got = hs.hyena_glr_bwd(a["v"], a["f"], d["dy"].cuda())
    assert "dg" not in got and got["dp"].shape[-1] == 2 * 72
    want = reference(d, grads=True)
    for n in ("dv", "df"):
        check(n, got[n], want[n], DT[dtype], 32, 56)


def test_gradients_against_differences():
    # central differences of the 64-bit form along random directions: the
    # truncation error is of order h^2 = 1e-8 of third derivatives of order 1
    d = make(2, 150, 24, "f32", seed=9, reset=True, lens=True)
    got = hs.hyena_glr_bwd(dy=d["dy"].cuda(), dh_last=d["dh_last"].cuda(), **blocks(d))
    base = {k: (t.double() if t is not None and t.is_floating_point() else t) for k, t in blocks(d, "cpu").items()}

    def loss(args):
        y, hl = block_ref.glr(**args)
        return ((y * d["dy"].double()).sum() + (hl * d["dh_last"].double()).sum()).item()

    gen = torch.Generator().manual_seed(1)
    for k in ("v", "f", "g", "bias", "h0"):
        u = torch.randn(base[k].shape, generator=gen, dtype=torch.float64)
        eps = 1e-4
        num = (loss({**base, k: base[k] + eps * u}) - loss({**base, k: base[k] - eps * u})) / (2 * eps)
        ana = (got["d" + k].double().cpu() * u).sum().item()
        size = (got["d" + k].double().cpu().abs() * u.abs()).sum().item()
        assert abs(num - ana) <= 1e-5 * size, (k, num, ana)


def test_extreme_gates_and_values():
    # gates far in both tails, -inf and +inf among them: a is exactly 0 or 1 there
    v = torch.randn(1, 9, 8)
    f = torch.tensor([-1e4, 1e4, -100.0, 100.0, -90.0, 20.0, -20.0, float("-inf"), float("inf")])[None, :, None]
    f = f.expand(1, 9, 8).contiguous()
    g = torch.tensor([-1e4, 1e4, -100.0, 100.0, 0.0, 50.0, float("-inf"), float("inf"), -3.0])[None, :, None]
    g = g.expand(1, 9, 8).contiguous()
    y = hs.hyena_glr_fwd(v.cuda(), f.cuda())
    ry, _ = block_ref.glr(v.double(), f.double())
    check("y", y, ry, torch.float32, 8, 9)
    z = torch.zeros(1, 9, 8)
    got = hs.hyena_glr_bwd(v.cuda(), f.cuda(), torch.ones(1, 9, 8).cuda(), g=g.clamp(-1e4, 1e4).cuda())
    assert all(torch.isfinite(got[k]).all() for k in ("dv", "df", "dg"))
    y = hs.hyena_glr_fwd(v.cuda(), z.cuda(), g=g.cuda()).cpu()
    assert (y[0, 6] == 0).all() and torch.isinf(y[0, 7]).all()  # silu(-inf) = 0, silu(inf) = inf


@pytest.mark.parametrize("L", [40, 700, 5000])
def test_nothing_crosses_a_reset_or_the_length(L):
    B, D = 2, 72
    d = make(B, L, D, "f32", seed=3, reset=True, lens=True, p_reset=0.0)
    cut, n = L // 3, L - 7
    d["reset"][:, cut] = 1
    d["lens"][:] = n
    clean = blocks(d)
    hl0 = torch.empty(B, D, device="cuda")
    y0 = hs.hyena_glr_fwd(**clean, h_last=hl0)
    dy = d["dy"].cuda()
    g0 = hs.hyena_glr_bwd(dy=dy, dh_last=d["dh_last"].cuda(), **clean)
    # NaN and infinities in the first document and in the padding: the second document is the same to the bit
    for bad in (float("nan"), float("inf")):
        a = blocks(d)
        for k in ("v", "f", "g"):
            a[k] = a[k].clone()
            a[k][:, :cut] = bad
            a[k][:, n:] = bad
        rs = a["reset"].clone()
        rs[:, n:] = 1
        a["reset"] = rs
        dy2 = dy.clone()
        dy2[:, :cut] = bad
        dy2[:, n:] = bad
        hl = torch.empty(B, D, device="cuda")
        y = hs.hyena_glr_fwd(**a, h_last=hl)
        assert torch.equal(y[:, cut:n], y0[:, cut:n]) and torch.equal(hl, hl0)
        assert (y[:, n:] == 0).all()
        g = hs.hyena_glr_bwd(dy=dy2, dh_last=d["dh_last"].cuda(), **a)
        for k in ("dv", "df", "dg"):
            assert torch.equal(g[k][:, cut:n], g0[k][:, cut:n]), k
            assert (g[k][:, n:] == 0).all(), k
    # and a bad second document leaves the first one's gradients alone
    a = blocks(d)
    a["v"] = a["v"].clone()
    a["v"][:, cut:] = float("nan")
    dy2 = dy.clone()
    dy2[:, cut:] = float("nan")
    g = hs.hyena_glr_bwd(dy=dy2, dh_last=d["dh_last"].cuda(), **a)
    for k in ("dv", "df", "dg"):
        assert torch.equal(g[k][:, :cut], g0[k][:, :cut]), k
    assert torch.equal(g["dh0"], g0["dh0"])


def test_outputs_stay_inside_their_rows():
    B, L, D = 3, 131, 72
    d = make(B, L, D, "bf16", seed=4, lens=True)
    a = blocks(d)
    big = torch.full((B + 2, L + 5, D + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    y = big[1:B + 1, 2:L + 2, 8:D + 8]
    hs.hyena_glr_fwd(**a, y=y)
    ref = hs.hyena_glr_fwd(**a)
    live = (torch.arange(L, device="cuda") < a["lens"][:, None])[..., None]
    assert torch.equal(torch.where(live, ref, torch.full_like(ref, 7.0)), y)
    edge = torch.ones_like(big, dtype=torch.bool)
    edge[1:B + 1, 2:L + 2, 8:D + 8] = False
    assert (big[edge] == 7).all()


def test_strides_of_every_input():
    B, L, D = 2, 200, 64
    d = make(B, L, D, "bf16", seed=6)
    a = blocks(d)
    want = hs.hyena_glr_fwd(**{k: (t.contiguous() if t is not None else None) for k, t in a.items()})
    # time-major storage, every other row, one sample for the whole batch
    tm = {k: a[k].transpose(0, 1).contiguous().transpose(0, 1) for k in ("v", "f", "g")}
    assert torch.equal(hs.hyena_glr_fwd(**{**a, **tm}), want)
    wide = torch.empty(B, 2 * L, D, dtype=torch.bfloat16, device="cuda")
    wide[:, ::2] = a["v"]
    assert torch.equal(hs.hyena_glr_fwd(**{**a, "v": wide[:, ::2]}), want)
    one = {k: a[k][:1].expand(B, L, D) for k in ("v", "f", "g")}
    got = hs.hyena_glr_fwd(**{**a, **one})
    assert torch.equal(got, hs.hyena_glr_fwd(**{**a, **{k: t.contiguous() for k, t in one.items()}}))


@pytest.mark.parametrize("B,L,D", [(1, 20000, 64), (2, 3000, 256)])
def test_reproducible_and_batch_invariant_streams(B, L, D):
    d = make(B, L, D, "bf16", seed=11, reset=True)
    a = blocks(d)
    dy = d["dy"].cuda()
    y0, g0 = hs.hyena_glr_fwd(**a), hs.hyena_glr_bwd(dy=dy, **a)
    torch.cuda.synchronize()
    # two calls at once, on two streams
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        y1, g1 = hs.hyena_glr_fwd(**a), hs.hyena_glr_bwd(dy=dy, **a)
    with torch.cuda.stream(s2):
        y2, g2 = hs.hyena_glr_fwd(**a), hs.hyena_glr_bwd(dy=dy, **a)
    torch.cuda.synchronize()
    for y, g in ((y1, g1), (y2, g2)):
        assert torch.equal(y, y0)
        for k in g0:
            assert torch.equal(g[k], g0[k]), k


def test_captured_and_replayed():
    B, L, D = 2, 1500, 128
    d = make(B, L, D, "f32", seed=12, lens=True)
    a = blocks(d)
    dy = d["dy"].cuda()
    hs.hyena_glr_fwd(**a), hs.hyena_glr_bwd(dy=dy, **a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, g = hs.hyena_glr_fwd(**a), hs.hyena_glr_bwd(dy=dy, **a)
    for i in range(4):
        a["v"].copy_(torch.randn(B, L, D, generator=torch.Generator().manual_seed(i)).cuda())
        ye, ge = hs.hyena_glr_fwd(**a), hs.hyena_glr_bwd(dy=dy, **a)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ye)
        for k in ge:
            assert torch.equal(g[k], ge[k]), k


# --------------------------------------------------------------- one position


def step_inputs(B, S, D, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    p = torch.randn(B, 3 * D, generator=gen)
    p[:, D:2 * D].clamp_(-2, 2)
    p = p.to(DT[dtype]).cuda()
    return dict(state=torch.randn(S, D, generator=gen).cuda(), v=p[:, :D], f=p[:, D:2 * D], g=p[:, 2 * D:],
                bias=(torch.rand(D, generator=gen) * 2).cuda())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,S,D", [(1, 1, 8), (3, 5, 72), (16, 24, 768), (300, 400, 64), (2, 2, 4104)])
def test_step(B, S, D, dtype):
    a = step_inputs(B, S, D, dtype, seed=B + D)
    gen = torch.Generator().manual_seed(2)
    slots = torch.randperm(S, generator=gen)[:B].to(torch.int32)
    old = a["state"].clone()
    new = torch.full_like(old, 9.0)
    y = hs.hyena_glr_step(**a, slots=slots.cuda(), state_out=new)
    assert torch.equal(a["state"], old)
    idx = slots.long()
    c = {k: t.double().cpu() for k, t in a.items()}
    ry, rh = block_ref.glr(c["v"][:, None], c["f"][:, None], c["g"][:, None], c["bias"], c["state"][idx])
    check("y", y[:, None], ry, DT[dtype], 8, 1)
    check("state", new[idx.cuda()], rh, torch.float32, 8, 1)
    rest = torch.ones(S, dtype=torch.bool)
    rest[idx] = False
    assert (new.cpu()[rest] == 9).all()
    # in place, default slots
    if S == B:
        y2 = hs.hyena_glr_step(**{**a, "state": old[idx.cuda()].contiguous()})
        assert torch.equal(y2, y)


def test_step_continues_the_scan():
    B, L, D = 2, 70, 64
    d = make(B, L, D, "f32", seed=21)
    a = blocks(d)
    hl = torch.empty(B, D, device="cuda")
    y = hs.hyena_glr_fwd(**a, h_last=hl)
    state = torch.empty(B, D, device="cuda")
    part = {k: (a[k][:, :50] if k in ("v", "f", "g") else a[k]) for k in a}
    hs.hyena_glr_fwd(**part, h_last=state)
    for t in range(50, L):
        yt = hs.hyena_glr_step(state, a["v"][:, t], a["f"][:, t], g=a["g"][:, t], bias=a["bias"])
        check("y_t", yt, y[:, t].double().cpu(), torch.float32, 16, 56, scale=y.abs().max().item())
    check("h_last", state, hl.double().cpu(), torch.float32, 16, 56)


def test_step_shared_and_missing_slots():
    B, S, D = 9, 4, 72
    a = step_inputs(B, S, D, "f32", seed=31)
    slots = torch.tensor([2, -1, 2, 0, 7, 2, 0, -2147483648, 2147483647], dtype=torch.int32)
    y = torch.full((B, D), 5.0, device="cuda")
    state = a["state"].clone()
    hs.hyena_glr_step(**{**a, "state": state}, slots=slots.cuda(), y=y)
    c = {k: t.double().cpu() for k, t in a.items()}
    want, wy = c["state"].clone(), torch.full((B, D), 5.0, dtype=torch.float64)
    for r, s in enumerate(slots.tolist()):
        if 0 <= s < S:
            yy, hh = block_ref.glr(c["v"][r][None, None], c["f"][r][None, None], c["g"][r][None, None], c["bias"],
                                   want[s][None])
            want[s], wy[r] = hh[0], yy[0, 0]
    check("state", state, want, torch.float32, 8, 4)
    check("y", y, wy, torch.float32, 8, 4)
    assert torch.equal(state[[1, 3]], a["state"][[1, 3]])
    fresh = hs.hyena_glr_step(**{**a, "state": a["state"].clone()}, slots=slots.cuda())
    assert torch.equal(fresh, torch.where(y == 5, torch.zeros_like(y), y))
