"""Measured cases of the operators around the long convolution in a block: the
gated linear recurrence, the gated feed-forward block, and the group norm with
an activation, channels last.

With v, f, g [B][L][D] (columns of one projection), per channel:

  a_t = sigmoid(f_t + bias),  h_t = a_t h_{t-1} + (1 - a_t) v_t,  y_t = h_t silu(g_t)

  reset[b][t] != 0 drops the history at t (a document starts), positions at and
  behind lens[b] hold the state and have no output; the step form takes one
  position per row with its state in a table of slots.

  feed-forward: (p, q) = x W_in, y = (p act(q)) W_out
  group norm:   y = act(gamma (x - mean) rstd + beta), mean and rstd over the
                positions of a sample and the channels of a group

`run` computes them from elementary torch operations in 32 bits, or, with
`own` set, through the framework's entry points.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_DTYPE = {BF16: torch.bfloat16, F32: torch.float32}
_SIZE = {BF16: 2, F32: 4}


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one decoded token for each of 16 running requests
        dict(name="glr_step_bf16_B16_D768", op="glr_step", dtype=BF16, B=16, D=768, slots=24),
        # training and prefill at the 2k language-model context
        dict(name="glr_fwd_bf16_B8_L2k_D768", op="glr_fwd", dtype=BF16, B=8, L=2048, D=768, ragged=False),
        # a padded batch of packed documents, odd lengths, full precision
        dict(name="glr_fwd_f32_B3_L10007_D320_ragged", op="glr_fwd", dtype=F32, B=3, L=10007, D=320, ragged=True),
        # training at the 2k context
        dict(name="glr_bwd_bf16_B8_L2k_D768", op="glr_bwd", dtype=BF16, B=8, L=2048, D=768, ragged=False),
        # training on the 1M nucleotide context: one sample, all parallelism along the sequence
        dict(name="glr_bwd_bf16_L1M_D256", op="glr_bwd", dtype=BF16, B=1, L=1 << 20, D=256, ragged=False),
        # decoding: one token for each of 8 requests
        dict(name="ffn_fwd_bf16_M8_D768", op="ffn_fwd", dtype=BF16, M=8, D=768, F=2048, act="silu"),
        # full precision, odd row count, the exact GELU
        dict(name="ffn_fwd_f32_M4099_D384", op="ffn_fwd", dtype=F32, M=4099, D=384, F=1032, act="gelu"),
        # training at the 2k context, 8 samples
        dict(name="ffn_fwd_bf16_M16k_D768", op="ffn_fwd", dtype=BF16, M=16384, D=768, F=2048, act="silu"),
        dict(name="ffn_bwd_bf16_M16k_D768", op="ffn_bwd", dtype=BF16, M=16384, D=768, F=2048, act="silu"),
        # image grids: norm and SiLU in front of the 2D operator
        dict(name="gn_fwd_f32_B8_64sq_C384", op="gn_fwd", dtype=F32, B=8, S=4096, C=384, G=32, act="silu", ragged=False),
        # volumes: the gradient of the same in 3D
        dict(name="gn_bwd_f32_B2_64cube_C128", op="gn_bwd", dtype=F32, B=2, S=1 << 18, C=128, G=8, act="silu",
             ragged=False),
        # per-token head norm of a mixer's output (every token a sample of one position)
        dict(name="gn_fwd_bf16_tokens_C768", op="gn_fwd", dtype=BF16, B=16384, S=1, C=768, G=12, act="none",
             ragged=False),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["glr_step", "glr_fwd", "glr_bwd", "ffn_fwd", "ffn_bwd", "gn_fwd", "gn_bwd"])
    dtype = rng.choice([BF16, F32])
    if op == "glr_step":
        B = _logint(rng, 1, 512)
        return dict(op=op, dtype=dtype, B=B, D=8 * _logint(rng, 8, 512), slots=B + rng.randint(0, 16))
    if op in ("glr_fwd", "glr_bwd"):
        B, L, D = _logint(rng, 1, 64), _logint(rng, 1, 1 << 18), 8 * _logint(rng, 4, 256)
        while B * L * D > 1 << 26:
            if B > 1:
                B //= 2
            else:
                L //= 2
        return dict(op=op, dtype=dtype, B=B, L=max(L, 1), D=D, ragged=rng.random() < 0.4)
    if op in ("ffn_fwd", "ffn_bwd"):
        D, F = 8 * _logint(rng, 8, 192), 8 * _logint(rng, 16, 512)
        M = _logint(rng, 1, 16384)
        cap = 1.5e9 if dtype == F32 else 2.5e10
        M = max(1, min(M, int(cap / (D * F))))
        return dict(op=op, dtype=dtype, M=M, D=D, F=F, act=rng.choice(["silu", "gelu", "none"]))
    C, B, S = 8 * _logint(rng, 4, 192), _logint(rng, 1, 4096), _logint(rng, 1, 1 << 18)
    while B * S * C > 1 << 26:
        if S > B:
            S //= 2
        else:
            B //= 2
    G = rng.choice([k for k in range(1, 65) if C % k == 0])
    return dict(op=op, dtype=dtype, B=max(B, 1), S=max(S, 1), C=C, G=G, act=rng.choice(["silu", "gelu", "none"]),
                ragged=rng.random() < 0.25)


# ----------------------------------------------------------------- inputs


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = _DTYPE[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=gen, device=dev) * (hi - lo) + lo

    st = dict(case=case)
    op = case["op"]
    if op == "glr_step":
        B, D, S = case["B"], case["D"], case["slots"]
        p = normal(B, 3 * D)
        st.update(v=p[:, :D], f=p[:, D:2 * D], g=p[:, 2 * D:], bias=uniform(D, lo=0.0, hi=6.0),
                  state=normal(S, D, dtype=torch.float32),
                  slots=torch.randperm(S, generator=gen, device=dev)[:B].to(torch.int32))
        st["state_out"] = st["state"].clone()
    elif op in ("glr_fwd", "glr_bwd"):
        B, L, D = case["B"], case["L"], case["D"]
        # one projection's output; its column blocks are the operator's inputs
        p = normal(B, L, 3 * D)
        st.update(v=p[..., :D], f=p[..., D:2 * D], g=p[..., 2 * D:], bias=uniform(D, lo=0.0, hi=6.0),
                  h0=normal(B, D, scale=0.5, dtype=torch.float32), reset=None, lens=None)
        if case["ragged"]:
            st["reset"] = (torch.rand(B, L, generator=gen, device=dev) < 1.0 / 512).to(torch.uint8)
            st["lens"] = torch.randint(L // 2, L + 1, (B,), generator=gen, device=dev).to(torch.int32)
        if op == "glr_fwd":
            st["h_last"] = torch.empty(B, D, device=dev)
        else:
            st.update(dy=normal(B, L, D), dh_last=normal(B, D, dtype=torch.float32))
    elif op in ("ffn_fwd", "ffn_bwd"):
        M, D, F = case["M"], case["D"], case["F"]
        st.update(x=normal(M, D), w_in=normal(D, 2 * F, scale=D ** -0.5), w_out=normal(F, D, scale=F ** -0.5))
        if op == "ffn_bwd":
            st["dy"] = normal(M, D)
    else:
        B, S, C = case["B"], case["S"], case["C"]
        x = torch.randn(B, S, C, generator=gen, device=dev)
        x = x * uniform(C, lo=0.5, hi=2.0) + normal(C, dtype=torch.float32)
        st.update(x=x.to(dt), gamma=1 + 0.2 * normal(C, dtype=torch.float32), beta=0.2 * normal(C, dtype=torch.float32),
                  lens=None)
        if case["ragged"]:
            st["lens"] = torch.randint(0, S + 1, (B,), generator=gen, device=dev).to(torch.int32)
        if op == "gn_bwd":
            # what a training program kept from its forward pass
            m, r = _gn_stats(st["x"].float(), case["G"], st["lens"])
            st.update(dy=normal(B, S, C), mean=m, rstd=r)
        else:
            st.update(mean=torch.empty(B, case["G"], device=dev), rstd=torch.empty(B, case["G"], device=dev))
    return st


# ------------------------------------------------------------- plain forms


def _scan(a, x):
    """h_t = a_t h_{t-1} + x_t along dim 1 (h before the first position zero), by doubling."""
    a, x, k, L = a.clone(), x.clone(), 1, a.shape[1]
    while k < L:
        x[:, k:] += a[:, k:] * x[:, :-k]
        a[:, k:] = a[:, k:] * a[:, :-k]
        k *= 2
    return x


def _glr_gates(st):
    """a (0 at resets, 1 behind the length), the input (1 - a) v (0 behind it), and the mask of the positions."""
    v, f = st["v"].float(), st["f"].float()
    z = f + st["bias"]
    a, c = torch.sigmoid(z), torch.sigmoid(-z)
    live = None
    at = a
    if st["reset"] is not None:
        at = torch.where(st["reset"].bool()[:, :, None], torch.zeros_like(a), a)
    if st["lens"] is not None:
        live = (torch.arange(v.shape[1], device=v.device) < st["lens"][:, None])[:, :, None]
        at = torch.where(live, at, torch.ones_like(at))
    x = c * v
    if live is not None:
        x = x * live
    return v, a, c, at, x, live


def _glr_fwd(st):
    _, _, _, at, x, live = _glr_gates(st)
    x[:, 0] += at[:, 0] * st["h0"]
    h = _scan(at, x)
    g = st["g"].float()
    y = h * (g * torch.sigmoid(g))
    if live is not None:
        y = y * live
    return dict(y=y.to(st["v"].dtype), h_last=h[:, -1].contiguous())


def _glr_bwd(st):
    v, a, c, at, x, live = _glr_gates(st)
    x[:, 0] += at[:, 0] * st["h0"]
    h = _scan(at, x)
    g, dy = st["g"].float(), st["dy"].float()
    if live is not None:
        dy = dy * live
    s = torch.sigmoid(g)
    dg = dy * h * (s * (1 + g * (1 - s)))
    r = dy * (g * s)
    r[:, -1] += st["dh_last"]
    # lam_t = r_t + a_{t+1} lam_{t+1}: the same scan on the reversed sequence
    an = torch.cat([torch.zeros_like(at[:, :1]), at[:, 1:].flip(1)], 1)
    lam = _scan(an, r.flip(1)).flip(1)
    hp = torch.cat([st["h0"][:, None], h[:, :-1]], 1)
    if st["reset"] is not None:
        hp = hp * (st["reset"] == 0)[:, :, None]
    dv = c * lam
    df = a * c * lam * (hp - v)
    if live is not None:
        dv, df = dv * live, df * live
    t = st["v"].dtype
    return dict(dv=dv.to(t), df=df.to(t), dg=dg.to(t), dbias=df.sum((0, 1)), dh0=at[:, 0] * lam[:, 0])


def _glr_step(st):
    v, f, g = st["v"].float(), st["f"].float(), st["g"].float()
    z = f + st["bias"]
    slots = st["slots"].long()
    h = torch.sigmoid(z) * st["state"][slots] + torch.sigmoid(-z) * v
    y = h * (g * torch.sigmoid(g))
    st["state_out"][slots] = h
    return dict(y=y.to(st["v"].dtype), state=st["state_out"])


def _act(q, name):
    if name == "silu":
        return q * torch.sigmoid(q)
    if name == "gelu":
        return 0.5 * q * (1 + torch.erf(q * 0.5 ** 0.5))
    return q


def _dact(q, name):
    if name == "silu":
        s = torch.sigmoid(q)
        return s * (1 + q * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(q * 0.5 ** 0.5)) + q * torch.exp(-0.5 * q * q) * (2 * math.pi) ** -0.5
    return torch.ones_like(q)


def _ffn_fwd(st):
    F, act = st["case"]["F"], st["case"]["act"]
    pq = st["x"].float() @ st["w_in"].float()
    z = pq[:, :F] * _act(pq[:, F:], act)
    return (z @ st["w_out"].float()).to(st["x"].dtype)


def _ffn_bwd(st):
    F, act, t = st["case"]["F"], st["case"]["act"], st["x"].dtype
    x, w_in, w_out, dy = (st[k].float() for k in ("x", "w_in", "w_out", "dy"))
    pq = x @ w_in
    p, q = pq[:, :F], pq[:, F:]
    aq = _act(q, act)
    dz = dy @ w_out.t()
    dpq = torch.cat([dz * aq, dz * p * _dact(q, act)], 1)
    return dict(dx=(dpq @ w_in.t()).to(t), dw_in=(x.t() @ dpq).to(t), dw_out=((p * aq).t() @ dy).to(t))


def _gn_live(x, lens):
    if lens is None:
        return None, x.shape[1]
    live = (torch.arange(x.shape[1], device=x.device) < lens[:, None])[:, :, None, None].to(x.dtype)
    return live, lens.to(x.dtype)[:, None]


def _gn_stats(x, G, lens, eps=1e-5):
    B, S, C = x.shape
    xg = x.view(B, S, G, C // G)
    live, n = _gn_live(x, lens)
    if live is None:
        mean = xg.mean((1, 3))
        var = (xg - mean[:, None, :, None]).square().mean((1, 3))
    else:
        cnt = (n * (C // G)).clamp(min=1)
        mean = (xg * live).sum((1, 3)) / cnt
        var = ((xg - mean[:, None, :, None]).square() * live).sum((1, 3)) / cnt
    return mean, torch.rsqrt(var + eps)


def _gn_fwd(st):
    G, act = st["case"]["G"], st["case"]["act"]
    x = st["x"].float()
    B, S, C = x.shape
    mean, rstd = _gn_stats(x, G, st["lens"])
    xh = ((x.view(B, S, G, C // G) - mean[:, None, :, None]) * rstd[:, None, :, None]).view(B, S, C)
    y = _act(xh * st["gamma"] + st["beta"], act)
    live, _ = _gn_live(x, st["lens"])
    if live is not None:
        y = y * live[..., 0]
    return dict(y=y.to(st["x"].dtype), mean=mean, rstd=rstd)


def _gn_bwd(st):
    G, act = st["case"]["G"], st["case"]["act"]
    x, dy = st["x"].float(), st["dy"].float()
    B, S, C = x.shape
    live, n = _gn_live(x, st["lens"])
    mean, rstd = st["mean"][:, None, :, None], st["rstd"][:, None, :, None]
    xh = ((x.view(B, S, G, C // G) - mean) * rstd).view(B, S, C)
    dn = dy * _dact(xh * st["gamma"] + st["beta"], act)
    if live is not None:
        dn = dn * live[..., 0]
        n = n.clamp(min=1)[:, None, :, None]
    w, xg = (dn * st["gamma"]).view(B, S, G, C // G), xh.view(B, S, G, C // G)
    cnt = n * (C // G)
    m1 = w.sum((1, 3), keepdim=True) / cnt
    m2 = (w * xg).sum((1, 3), keepdim=True) / cnt
    dx = rstd * (w - m1 - xg * m2)
    if live is not None:
        dx = dx * live
    return dict(dx=dx.view(B, S, C).to(st["x"].dtype), dgamma=(dn * xh).sum((0, 1)), dbeta=dn.sum((0, 1)))


_PLAIN = dict(glr_fwd=_glr_fwd, glr_bwd=_glr_bwd, glr_step=_glr_step, ffn_fwd=_ffn_fwd, ffn_bwd=_ffn_bwd,
              gn_fwd=_gn_fwd, gn_bwd=_gn_bwd)


# ------------------------------------------------------ the framework's calls


def _own(st):
    import subquadratic_sequence_amd as hs
    case = st["case"]
    op = case["op"]
    if op == "glr_step":
        y = hs.hyena_glr_step(st["state"], st["v"], st["f"], g=st["g"], bias=st["bias"], slots=st["slots"],
                              state_out=st["state_out"])
        return dict(y=y, state=st["state_out"])
    if op == "glr_fwd":
        y = hs.hyena_glr_fwd(st["v"], st["f"], g=st["g"], bias=st["bias"], h0=st["h0"], reset=st["reset"],
                             lens=st["lens"], h_last=st["h_last"])
        return dict(y=y, h_last=st["h_last"])
    if op == "glr_bwd":
        d = hs.hyena_glr_bwd(st["v"], st["f"], st["dy"], g=st["g"], bias=st["bias"], h0=st["h0"], reset=st["reset"],
                             lens=st["lens"], dh_last=st["dh_last"])
        return {k: d[k] for k in ("dv", "df", "dg", "dbias", "dh0")}
    act = {"none": hs.ACT_NONE, "silu": hs.ACT_SILU, "gelu": hs.ACT_GELU}[case["act"]]
    if op == "ffn_fwd":
        return hs.hyena_ffn_fwd(st["x"], st["w_in"], st["w_out"], act=act)
    if op == "ffn_bwd":
        d = hs.hyena_ffn_bwd(st["x"], st["w_in"], st["w_out"], st["dy"], act=act)
        return {k: d[k] for k in ("dx", "dw_in", "dw_out")}
    if op == "gn_fwd":
        y = hs.hyena_group_norm_fwd(st["x"], case["G"], gamma=st["gamma"], beta=st["beta"], eps=1e-5, act=act,
                                    lens=st["lens"], mean=st["mean"], rstd=st["rstd"])
        return dict(y=y, mean=st["mean"], rstd=st["rstd"])
    d = hs.hyena_group_norm_bwd(st["x"], st["dy"], case["G"], st["mean"], st["rstd"], gamma=st["gamma"],
                                beta=st["beta"], act=act, lens=st["lens"])
    return {k: d[k] for k in ("dx", "dgamma", "dbeta")}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def work(case):
    """Bytes and operations of one pass: every input read once, every output written once."""
    op, e = case["op"], _SIZE[case["dtype"]]
    if op == "glr_step":
        n = case["B"] * case["D"]
        return {"bytes": n * (4 * e + 8) + 4 * case["D"] + 4 * case["B"], "flops": 14 * n}
    if op in ("glr_fwd", "glr_bwd"):
        B, L, D = case["B"], case["L"], case["D"]
        n = B * L * D
        mask = (B * L + 4 * B) if case["ragged"] else 0
        if op == "glr_fwd":
            return {"bytes": 4 * n * e + 8 * B * D + 4 * D + mask, "flops": 14 * n}
        return {"bytes": 7 * n * e + 12 * B * D + 8 * D + mask, "flops": 34 * n}
    if op in ("ffn_fwd", "ffn_bwd"):
        M, D, F = case["M"], case["D"], case["F"]
        if op == "ffn_fwd":
            return {"bytes": (2 * M * D + 3 * D * F) * e, "flops": 6 * M * D * F + 6 * M * F}
        return {"bytes": (3 * M * D + 6 * D * F) * e, "flops": 16 * M * D * F + 16 * M * F}
    B, S, C, G = case["B"], case["S"], case["C"], case["G"]
    n = B * S * C
    if op == "gn_fwd":
        return {"bytes": 2 * n * e + 8 * C + 8 * B * G, "flops": 12 * n}
    return {"bytes": 3 * n * e + 16 * C + 8 * B * G, "flops": 24 * n}


# ------------------------------------------------------------ 64-bit values


def _walk(coef, add, start):
    """The recurrence s_t = coef_t s_{t-1} + add_t from s_{-1} = start, in float64: runs of about sqrt(L)
    positions side by side from zero, position by position, then the runs joined in order."""
    B, L, D = coef.shape
    run = max(1, int(math.sqrt(L)))
    nrun = (L + run - 1) // run
    pad = nrun * run - L
    c = torch.cat([coef, coef.new_ones(B, pad, D)], 1).view(B, nrun, run, D)
    a = torch.cat([add, add.new_zeros(B, pad, D)], 1).view(B, nrun, run, D)
    part, prod = torch.empty_like(a), torch.empty_like(c)
    s, w = torch.zeros_like(a[:, :, 0]), torch.ones_like(c[:, :, 0])
    for i in range(run):
        s = c[:, :, i] * s + a[:, :, i]
        w = c[:, :, i] * w
        part[:, :, i], prod[:, :, i] = s, w
    before, h = [], start
    for j in range(nrun):
        before.append(h)
        h = part[:, j, -1] + prod[:, j, -1] * h
    out = part + prod * torch.stack(before, 1)[:, :, None]
    return out.view(B, nrun * run, D)[:, :L]


def _sig(x):
    return torch.where(x >= 0, 1 / (1 + torch.exp(-x)), torch.exp(x) / (1 + torch.exp(x)))


def _act64(q, name, slope=False):
    if name == "none":
        return torch.ones_like(q) if slope else q
    if name == "silu":
        s = _sig(q)
        return s + q * s * _sig(-q) if slope else q * s
    phi = 0.5 * torch.erfc(-q / math.sqrt(2))
    return phi + q * torch.exp(-q * q / 2) / math.sqrt(2 * math.pi) if slope else q * phi


def exact(case, seed):
    st = prepare(case, seed)
    d = {k: (x.double() if isinstance(x, torch.Tensor) and x.is_floating_point() else x) for k, x in st.items()}
    op = case["op"]
    if op == "glr_step":
        keep, gate = _sig(d["f"] + d["bias"]), _sig(-(d["f"] + d["bias"]))
        idx = d["slots"].long()
        h = keep * d["state"].index_select(0, idx) + gate * d["v"]
        return dict(y=h * _act64(d["g"], "silu"), state=d["state"].index_copy(0, idx, h))
    if op in ("glr_fwd", "glr_bwd"):
        L = case["L"]
        u = d["f"] + d["bias"]
        keep, gate = _sig(u), _sig(-u)
        ones = torch.ones(case["B"], L, 1, dtype=torch.float64, device=u.device)
        start = ones if d["reset"] is None else (d["reset"][:, :, None] == 0).double()
        on = ones
        if d["lens"] is not None:
            on = (torch.arange(L, device=u.device)[None, :, None] < d["lens"][:, None, None]).double()
        coef = keep * start * on + (1 - on)
        h = _walk(coef, gate * d["v"] * on, d["h0"])
        sg = _act64(d["g"], "silu")
        if op == "glr_fwd":
            return dict(y=h * sg * on, h_last=h[:, -1])
        dy = d["dy"] * on
        # backwards in time: lam_t = dy_t sg_t + coef_{t+1} lam_{t+1}, the last from dh_last
        nxt = torch.cat([coef[:, 1:], ones.expand(-1, -1, case["D"])[:, :1]], 1)
        lam = _walk(nxt.flip(1), (dy * sg).flip(1), d["dh_last"]).flip(1)
        prev = torch.cat([d["h0"][:, None], h[:, :-1]], 1) * start
        df = keep * gate * lam * (prev - d["v"]) * on
        return dict(dv=gate * lam * on, df=df, dg=dy * h * _act64(d["g"], "silu", slope=True), dbias=df.sum((0, 1)),
                    dh0=coef[:, 0] * lam[:, 0])
    if op in ("ffn_fwd", "ffn_bwd"):
        F, act = case["F"], case["act"]
        p, q = d["x"] @ d["w_in"][:, :F], d["x"] @ d["w_in"][:, F:]
        z = p * _act64(q, act)
        if op == "ffn_fwd":
            return z @ d["w_out"]
        dz = d["dy"] @ d["w_out"].t()
        dp, dq = dz * _act64(q, act), dz * p * _act64(q, act, slope=True)
        return dict(dx=dp @ d["w_in"][:, :F].t() + dq @ d["w_in"][:, F:].t(),
                    dw_in=torch.cat([d["x"].t() @ dp, d["x"].t() @ dq], 1), dw_out=z.t() @ d["dy"])
    B, S, C, G = case["B"], case["S"], case["C"], case["G"]
    per = C // G
    on = torch.ones(B, S, 1, dtype=torch.float64, device=d["x"].device)
    if d["lens"] is not None:
        on = (torch.arange(S, device=on.device)[None, :, None] < d["lens"][:, None, None]).double()
    count = (on.sum((1, 2)) * per).clamp(min=1)[:, None]

    def spread(t):  # [B, G] -> [B, 1, C]
        return t.repeat_interleave(per, 1)[:, None]

    def pooled(t):  # [B, S, C] -> sums over the positions and a group's channels [B, G]
        return (t * on).sum(1).view(B, G, per).sum(2)

    if op == "gn_fwd":
        mean = pooled(d["x"]) / count
        dev = d["x"] - spread(mean)
        rstd = 1 / torch.sqrt(pooled(dev * dev) / count + 1e-5)
        return dict(y=_act64(dev * spread(rstd) * d["gamma"] + d["beta"], case["act"]) * on, mean=mean, rstd=rstd)
    xh = (d["x"] - spread(d["mean"])) * spread(d["rstd"])
    dn = d["dy"] * _act64(xh * d["gamma"] + d["beta"], case["act"], slope=True) * on
    w = dn * d["gamma"]
    dx = spread(d["rstd"]) * (w - spread(pooled(w) / count) - xh * spread(pooled(w * xh) / count)) * on
    return dict(dx=dx, dgamma=(dn * xh).sum((0, 1)), dbeta=dn.sum((0, 1)))
