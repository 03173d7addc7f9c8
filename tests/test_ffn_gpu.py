"""The gated feed-forward block against its 64-bit form.

Whole numbers: with few entries of 1 and -1 a row every intermediate is a small
integer, exact in bf16, and every sum is exact in fp32, so the results equal the
64-bit ones rounded once.

Real numbers (u = 2^-24 and, for bf16, h = 2^-8, else 0): p and q carry K u of the sum of
magnitudes P = |x| |w_in|; the activation's slope is at most 1.13 and its own error
8 u of its size plus, for gelu, 4 u |q|; z = p act(q) is rounded once (h). With Z the
bound of |z|'s error, y is off by Z |w_out|, F u of |z| |w_out|, and its rounding. The
backward's dp, dq follow in the same way, through dz with D u of |dy| |w_out|^T and
dz's own rounding (h); dx and
the weight gradients sum such terms over 2F or M, with as many u and one rounding.
These are sums of worst cases, elementwise."""
import pytest
import torch

import subquadratic_sequence_amd as hs
from tests import block_ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ACT = {"none": hs.ACT_NONE, "silu": hs.ACT_SILU, "gelu": hs.ACT_GELU}
U = 2.0 ** -24

# rows, D, F: one row, single tiles cut everywhere, K tails, more tiles than one, few and many rows
SHAPES = [(1, 8, 8), (1, 64, 64), (3, 72, 40), (8, 768, 2048), (16, 320, 1032), (17, 64, 136), (33, 136, 8),
          (64, 512, 256), (100, 200, 296), (129, 384, 520), (257, 256, 264), (300, 1032, 72), (1000, 96, 640),
          (4099, 128, 136), (700, 768, 2048)]


def sparse(gen, m, n, per, dtype):
    t = torch.zeros(m, n)
    idx = torch.randint(0, n, (m, per), generator=gen)
    return t.scatter_(1, idx, torch.randint(0, 2, (m, per), generator=gen) * 2.0 - 1).to(dtype)


def rounded(t, dtype):
    # the sums are integers below 2^24: exact in fp32, rounded once to the storage type
    assert t.abs().max() < 2 ** 24
    return t.float().to(dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,D,F", SHAPES)
def test_whole_numbers_are_exact(M, D, F, dtype):
    say(f"ffn exact M={M} D={D} F={F} {dtype}")
    gen = torch.Generator().manual_seed(M + D + F)
    x, dy = (sparse(gen, M, D, 3, DT[dtype]) for _ in range(2))
    w_in = torch.randint(-1, 2, (D, 2 * F), generator=gen).to(DT[dtype])
    w_out = torch.randint(-1, 2, (F, D), generator=gen).to(DT[dtype])
    xd, wi, wo, dd = (t.double() for t in (x, w_in, w_out, dy))
    y, z = block_ref.ffn(xd, wi, wo, "none")
    dev = [t.cuda() for t in (x, w_in, w_out)]
    got = hs.hyena_ffn_fwd(*dev, act=hs.ACT_NONE)
    assert torch.equal(got.cpu(), rounded(y, DT[dtype]))
    p, q = (xd @ wi)[:, :F], (xd @ wi)[:, F:]
    dz = dd @ wo.t()
    dpq = torch.cat([dz * q, dz * p], 1)
    g = hs.hyena_ffn_bwd(*dev, dy.cuda(), act=hs.ACT_NONE)
    assert torch.equal(g["dx"].cpu(), rounded(dpq @ wi.t(), DT[dtype]))
    assert torch.equal(g["dw_in"].cpu(), rounded(xd.t() @ dpq, DT[dtype]))
    assert torch.equal(g["dw_out"].cpu(), rounded(z.t() @ dd, DT[dtype]))


def make(M, D, F, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return [t.to(DT[dtype]) for t in (rnd(M, D), rnd(D, 2 * F) * D ** -0.5, rnd(F, D) * F ** -0.5, rnd(M, D))]


def near(name, got, want, bar):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), name
    over = (got - want).abs() - bar
    assert (over <= 0).all(), f"{name}: {over.max().item():.3e} over the bar, max error {(got - want).abs().max():.3e}"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "none"])
@pytest.mark.parametrize("M,D,F", SHAPES)
def test_real_numbers(M, D, F, act, dtype):
    x, w_in, w_out, dy = make(M, D, F, dtype, seed=M + D + F)
    h = block_ref.half_step(DT[dtype]) if dtype == "bf16" else 0.0
    xd, wi, wo = (t.double().requires_grad_(True) for t in (x, w_in, w_out))
    dd = dy.double()
    y, z = block_ref.ffn(xd, wi, wo, act)
    want = torch.autograd.grad((y * dd).sum(), [xd, wi, wo])
    y, z, xd, wi, wo = (t.detach() for t in (y, z, xd, wi, wo))
    got = hs.hyena_ffn_fwd(x.cuda(), w_in.cuda(), w_out.cuda(), act=ACT[act])
    g = hs.hyena_ffn_bwd(x.cuda(), w_in.cuda(), w_out.cuda(), dy.cuda(), act=ACT[act])
    E = (D + 4) * U * (xd.abs() @ wi.abs())  # error of p and q
    pq = xd @ wi
    p, q, ep, eq = pq[:, :F], pq[:, F:], E[:, :F], E[:, F:]
    a = block_ref.act(q, act)
    ea = 1.13 * eq + 8 * U * (a.abs() + q.abs())
    ez = (ep * a.abs() + p.abs() * ea) * (1 + h) + (h + 2 * U) * z.abs()
    near("y", got, y, ez @ wo.abs() + (F + 4) * U * (z.abs() @ wo.abs()) + (h + U) * y.abs() * (1 + h))
    qq = q.clone().requires_grad_(True)
    da = torch.autograd.grad(block_ref.act(qq, act).sum(), qq)[0]
    eda = 1.0 * eq + 8 * U * (1 + q.abs())  # |act''| <= 1
    dz = dd @ wo.t()
    edz = (D + 4) * U * (dd.abs() @ wo.abs().t()) * (1 + h) + (h + U) * dz.abs()
    dp, dq = dz * a, dz * p * da
    edp = (edz * a.abs() + dz.abs() * ea) * (1 + h) + (h + 2 * U) * dp.abs()
    edq = (edz * (p * da).abs() + dz.abs() * (ep * da.abs() + p.abs() * eda)) * (1 + h) + (h + 4 * U) * dq.abs()
    ed, d = torch.cat([edp, edq], 1), torch.cat([dp, dq], 1)

    def bar(e, v, wa, k, ref):
        return e @ wa + (k + 4) * U * (v.abs() @ wa) + (h + U) * ref.abs() * (1 + h)

    near("dx", g["dx"], want[0], bar(ed, d, wi.abs().t(), 2 * F, want[0]))
    near("dw_in", g["dw_in"].t(), want[1].t(), bar(ed.t(), d.t(), xd.abs(), M, want[1].t()))
    near("dw_out", g["dw_out"], want[2], bar(ez.t(), z.t(), dd.abs(), M, want[2]))


def test_gradients_against_differences():
    M, D, F = 40, 64, 72
    x, w_in, w_out, dy = (t.double() for t in make(M, D, F, "f32", seed=1))
    g = hs.hyena_ffn_bwd(*(t.float().cuda() for t in (x, w_in, w_out, dy)), act=hs.ACT_GELU)
    gen = torch.Generator().manual_seed(2)
    for i, k in enumerate(("dx", "dw_in", "dw_out")):
        args = [x, w_in, w_out]
        u = torch.randn(args[i].shape, generator=gen, dtype=torch.float64)
        vals = []
        for s in (1e-4, -1e-4):
            b = list(args)
            b[i] = b[i] + s * u
            vals.append((block_ref.ffn(*b, "gelu")[0] * dy).sum().item())
        num, ana = (vals[0] - vals[1]) / 2e-4, (g[k].double().cpu() * u).sum().item()
        # differences of order 1e-8 in the step, fp32 gradients
        assert abs(num - ana) <= 1e-5 * (g[k].double().cpu().abs() * u.abs()).sum().item(), (k, num, ana)


def test_rows_do_not_mix_and_batches_agree():
    x, w_in, w_out, _ = make(300, 136, 264, "bf16", seed=4)
    xc, wi, wo = x.cuda(), w_in.cuda(), w_out.cuda()
    want = hs.hyena_ffn_fwd(xc, wi, wo)
    assert torch.equal(hs.hyena_ffn_fwd(xc.view(3, 100, 136), wi, wo).view(300, 136), want)
    bad = xc.clone()
    bad[7] = float("nan")
    bad[299] = float("inf")
    got = hs.hyena_ffn_fwd(bad, wi, wo)
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[7] = keep[299] = False
    assert torch.equal(got[keep], want[keep])
    assert not torch.isfinite(got[~keep]).any()


def test_outputs_stay_inside_their_buffers():
    for M, D, F in [(5, 72, 40), (257, 136, 264), (700, 72, 520)]:
        x, w_in, w_out, dy = (t.cuda() for t in make(M, D, F, "bf16", seed=5))
        for make_ws in (hs.hyena_ffn_workspace_bytes, hs.hyena_ffn_bwd_workspace_bytes):
            n = make_ws(M, D, F, hs.HYENA_BF16)
            buf = torch.full((n + 4096,), 77, dtype=torch.uint8, device="cuda")
            ws = buf[2048:2048 + n]
            out = torch.full((M + 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
            if make_ws is hs.hyena_ffn_workspace_bytes:
                y = out[1:M + 1]
                hs.hyena_ffn_fwd(x, w_in, w_out, y=y, ws=ws)
                assert torch.equal(y, hs.hyena_ffn_fwd(x, w_in, w_out))
                assert (out[0] == 7).all() and (out[-1] == 7).all()
            else:
                hs.hyena_ffn_bwd(x, w_in, w_out, dy, ws=ws)
            assert (buf[:2048] == 77).all() and (buf[2048 + n:] == 77).all()


@pytest.mark.parametrize("M,D,F", [(3, 128, 256), (40, 256, 512), (900, 256, 512)])
def test_captured_replayed_and_two_streams(M, D, F):
    x, w_in, w_out, dy = (t.cuda() for t in make(M, D, F, "bf16", seed=6))

    def both():
        y = hs.hyena_ffn_fwd(x, w_in, w_out)
        g = hs.hyena_ffn_bwd(x, w_in, w_out, dy)
        return [y, g["dx"], g["dw_in"], g["dw_out"]]

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
        x.copy_(make(M, D, F, "bf16", seed=50 + i)[0].cuda())
        want = both()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(rec, want))


@pytest.mark.parametrize("M", [1, 64, 100, 1000, 5000])
def test_bf16_gradients_of_the_products_are_rounded_once(M):
    """One row's x is (1, 0, ..), the only one with a gradient, so dw_in[0] = (dp, dq) of that row
    with nothing summed: dp = dz q, dq = dz p. dz arrives to 2^-17 (two bf16 words of 8 bits), its
    sum of D products to D 2^-24: relative 2^-16 in all. The value before its rounding lies so
    close to a tie in about 2^-16 * 2^8 * 2 < 1 % of the elements; a dz rounded to bf16 first
    would differ in a quarter of them."""
    say(f"ffn rounded once M={M}")
    D, F = 72, 1032
    gen = torch.Generator().manual_seed(M)
    x, dy = torch.zeros(M, D), torch.zeros(M, D)
    x[M - 1, 0] = 1
    dy[M - 1] = torch.rand(D, generator=gen) + 0.5  # one sign: no cancellation in dz
    w_in = torch.randn(D, 2 * F, generator=gen)
    w_out = torch.rand(F, D, generator=gen) + 0.5
    x, dy, w_in, w_out = (t.bfloat16() for t in (x, dy, w_in, w_out))
    dz = dy[M - 1].double() @ w_out.double().t()
    p, q = w_in[0, :F].double(), w_in[0, F:].double()
    want = torch.cat([dz * q, dz * p]).bfloat16()
    got = hs.hyena_ffn_bwd(*(t.cuda() for t in (x, w_in, w_out, dy)), act=hs.ACT_NONE)["dw_in"][0].cpu()
    assert (got != want).double().mean() < 0.02


@pytest.mark.parametrize("M", [5, 300])
def test_an_overflowing_dz_stays_infinite(M):
    D, F = 64, 128
    x = torch.ones(M, D, dtype=torch.bfloat16, device="cuda")
    w_in = torch.full((D, 2 * F), 2.0 ** -6, dtype=torch.bfloat16, device="cuda")
    w_out = torch.full((F, D), 2.0 ** 66, dtype=torch.bfloat16, device="cuda")
    dy = torch.full((M, D), 2.0 ** 66, dtype=torch.bfloat16, device="cuda")
    g = hs.hyena_ffn_bwd(x, w_in, w_out, dy, act=hs.ACT_NONE)  # dz = 2^138
    assert torch.isposinf(g["dx"]).all() and torch.isposinf(g["dw_in"]).all()
