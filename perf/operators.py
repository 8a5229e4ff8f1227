"""Cases of the gated delta rule and of layer norm, with their plain forms.

The gated delta rule keeps, per batch row and value head, a real state S in
R^{N x P} (N = dstate, P = headdim, as the complex SSD state) and writes each
token's value at its key, correcting what the state already answers there:

    S' = exp(g_t) S_{t-1}
    S_t = S' + k_t (beta_t (v_t - S'^T k_t))^T
    o_t = scale S_t^T q_t

Key heads may be fewer than value heads (value head h reads key head
h // (H / KH)).  Rows of a padded batch end at `lens`: what lies behind is not
read, and outputs and gradients there are zero.

Operators: delta_forward and delta_backward (a sequence), delta_step (one token
of a decode loop, the state updated in place), layernorm and layernorm_backward
(the normalisation before and after such a mixer).
"""

import math

import torch

from complex_valued_state_gb300 import workloads as wl

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_CHUNK = 64
_EPS = 1e-5


def _calls():
    from complex_valued_state_gb300 import cssd

    return cssd


def listed():
    lay, lng, pam, dec = wl.MAMBA2_LAYER, wl.LONG_SEQ, wl.PAM, wl.DECODE
    return [
        # one sequence being answered: a single token at the width of the PAM layer
        {"name": "step_one", "op": "step", "B": 1, "H": pam.nheads, "KH": pam.nheads, "N": 64, "P": 64, "dtype": "bf16", "pool": 0},
        # the decode workload: 256 sequences answered at once
        {"name": "step_decode", "op": "step", "B": dec.batch, "H": dec.nheads, "KH": dec.nheads, "N": dec.dstate, "P": dec.headdim, "dtype": "bf16", "pool": 0},
        # a server's pool of states, some of its rows active, key heads shared by four value heads
        {"name": "step_pool", "op": "step", "B": 77, "H": 32, "KH": 8, "N": 128, "P": 128, "dtype": "fp16", "pool": 96},
        # one layer over a training batch (mamba2_layer's sizes)
        {"name": "fwd_layer", "op": "fwd", "B": lay.batch, "T": lay.seqlen, "H": lay.nheads, "KH": lay.nheads, "N": lay.dstate, "P": lay.headdim, "dtype": "bf16", "ragged": False, "state": False},
        # a long document taken in one call (long_seq's heads and widths), continued from a state
        {"name": "fwd_long", "op": "fwd", "B": lng.batch, "T": lng.seqlen // 4, "H": lng.nheads, "KH": lng.nheads, "N": lng.dstate, "P": lng.headdim, "dtype": "bf16", "ragged": False, "state": True},
        # prompts of different lengths padded to one batch, key heads shared by two value heads
        {"name": "fwd_prompts", "op": "fwd", "B": 6, "T": 1333, "H": 16, "KH": 8, "N": 128, "P": 128, "dtype": "fp16", "ragged": True, "state": True},
        # gradients of one layer over a training batch
        {"name": "bwd_layer", "op": "bwd", "B": lay.batch, "T": lay.seqlen, "H": lay.nheads, "KH": lay.nheads, "N": lay.dstate, "P": lay.headdim, "dtype": "bf16", "ragged": False, "state": False},
        # gradients at the wide head sizes, key heads shared by two value heads, ragged rows
        {"name": "bwd_wide", "op": "bwd", "B": 4, "T": 1501, "H": 16, "KH": 8, "N": 128, "P": 128, "dtype": "bf16", "ragged": True, "state": True},
        # a small fp32 run, as one trains while looking for a bug
        {"name": "bwd_fp32", "op": "bwd", "B": 2, "T": 515, "H": 12, "KH": 12, "N": 64, "P": 64, "dtype": "fp32", "ragged": False, "state": False},
        # a single prompt in fp32
        {"name": "fwd_fp32", "op": "fwd", "B": 1, "T": 1000, "H": pam.nheads, "KH": pam.nheads, "N": 64, "P": 64, "dtype": "fp32", "ragged": False, "state": False},
        # the norm before that layer over the same tokens (24 heads of 64)
        {"name": "ln_layer", "op": "ln", "R": lay.batch * lay.seqlen, "D": lay.nheads * lay.headdim, "dtype": "bf16", "wdtype": "bf16", "bias": True},
        # its gradients
        {"name": "lnb_layer", "op": "lnb", "R": lay.batch * lay.seqlen, "D": lay.nheads * lay.headdim, "dtype": "bf16", "wdtype": "fp32", "bias": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "fwd", "fwd", "bwd", "bwd", "ln", "lnb"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("ln", "lnb"):
        D = rng.choice([rng.randint(5, 600), 64 * rng.randint(4, 64), 1000 + rng.randint(0, 3000)])
        R = max(1, min(_log(rng, 1, 40000), 24_000_000 // D))
        return {"op": op, "R": R, "D": D, "dtype": dtype, "wdtype": rng.choice([dtype, "fp32"]), "bias": rng.random() < 0.7}
    N, P = rng.choice([(64, 64), (128, 64), (128, 128), (64, 128), (32, 64), (16, 16), (96, 80), (128, 32)])
    KH = rng.choice([1, 2, 3, 4, 8, 12, 16])
    H = KH * rng.choice([1, 1, 2, 4])
    if op == "step":
        B = max(1, min(_log(rng, 1, 256), 60_000_000 // (H * N * P)))
        return {"op": op, "B": B, "H": H, "KH": KH, "N": N, "P": P, "dtype": dtype, "pool": rng.choice([0, B + rng.randint(0, 20)])}
    B = rng.randint(1, 6)
    T = max(1, min(_log(rng, 1, 3000), (150_000 if op == "fwd" else 80_000) // (B * H)))
    return {"op": op, "B": B, "T": T, "H": H, "KH": KH, "N": N, "P": P, "dtype": dtype, "ragged": B > 1 and rng.random() < 0.4, "state": rng.random() < 0.5}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if case["op"] in ("ln", "lnb"):
        R, D = case["R"], case["D"]
        wt = _TYPES[case["wdtype"]]
        s = {"case": case, "x": (normal(R, D) * torch.exp(0.5 * normal(R, 1)) + 0.3 * normal(R, 1)).to(dt),
             "weight": (1 + 0.2 * normal(D)).to(wt), "bias": (0.2 * normal(D)).to(wt) if case["bias"] else None}
        if case["op"] == "lnb":  # the statistics that the forward pass left
            xf = s["x"].double()
            mean = xf.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = ((xf - mean[:, None]).square().mean(1) + _EPS).rsqrt().float()
            s["dy"] = normal(R, D).to(dt)
        return s
    B, H, KH, N, P = (case[k] for k in ("B", "H", "KH", "N", "P"))
    lead = (B,) if case["op"] == "step" else (B, case["T"])

    def unit(*shape):
        x = normal(*shape)
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    # decays: each head forgets at a rate of its own, from 1 to some thousands of tokens
    rate = torch.exp(math.log(5e-4) + (math.log(1.0) - math.log(5e-4)) * torch.rand(H, generator=gen, device="cuda"))
    s = {"case": case, "q": unit(*lead, KH, N), "k": unit(*lead, KH, N), "v": normal(*lead, H, P).to(dt),
         "g": -rate * torch.nn.functional.softplus(1 + normal(*lead, H)), "beta": torch.sigmoid(normal(*lead, H)), "scale": N ** -0.5}
    if case["op"] == "step":
        rows = case["pool"] or B
        s["h"] = 0.3 * normal(rows, H, N, P)
        s["slots"] = torch.randperm(rows, generator=gen, device="cuda")[:B].to(torch.int32) if case["pool"] else None
        return s
    T = case["T"]
    s["lens"] = torch.randint(0, T + 1, (B,), generator=gen, device="cuda").to(torch.int32) if case["ragged"] else None
    s["h0"] = 0.3 * normal(B, H, N, P) if case["state"] else None
    if case["op"] == "bwd":
        s["do"] = normal(B, T, H, P).to(dt)
        s["dh"] = 0.3 * normal(B, H, N, P) if case["state"] else None
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    cssd = _calls()
    op = s["case"]["op"]
    if op == "ln":
        y, mean, rstd = cssd.layernorm(s["x"], s["weight"], s["bias"], eps=_EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "lnb":
        return cssd.layernorm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], want_bias=s["bias"] is not None)
    if op == "step":
        o = cssd.delta_step(s["h"], s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], slots=s["slots"])
        return {"o": o, "h": s["h"]}
    if op == "fwd":
        o, h = cssd.delta_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], h0=s["h0"], lens=s["lens"])
        return {"o": o, "h": h}
    return cssd.delta_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], scale=s["scale"], h0=s["h0"], dh_final=s["dh"], lens=s["lens"])


def _run_plain(s):
    op = s["case"]["op"]
    if op == "ln":
        x = s["x"].float()
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = (c.square().mean(1) + _EPS).rsqrt()
        y = c * rstd[:, None] * s["weight"].float()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    if op == "lnb":
        x, dy = s["x"].float(), s["dy"].float()
        xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
        wdy = dy * s["weight"].float()
        gx = s["rstd"][:, None] * (wdy - wdy.mean(1, keepdim=True) - xh * (wdy * xh).mean(1, keepdim=True))
        out = {"gx": gx.to(s["x"].dtype), "gweight": (dy * xh).sum(0).to(s["weight"].dtype)}
        if s["bias"] is not None:
            out["gbias"] = dy.sum(0).to(s["weight"].dtype)
        return out
    if op == "step":
        return _step_plain(s)
    return _fwd_plain(s) if op == "fwd" else _bwd_plain(s)


def _step_plain(s):
    G = s["case"]["H"] // s["case"]["KH"]
    q, k = (s[n].float().repeat_interleave(G, 1) for n in ("q", "k"))
    h = s["h"] if s["slots"] is None else s["h"][s["slots"].long()]
    h = h * torch.exp(s["g"])[..., None, None]
    e = s["beta"][..., None] * (s["v"].float() - (h * k[..., None]).sum(-2))
    h = h + k[..., None] * e[..., None, :]
    o = s["scale"] * (h * q[..., None]).sum(-2)
    if s["slots"] is None:
        s["h"].copy_(h)
    else:
        s["h"][s["slots"].long()] = h
    return {"o": o.to(s["v"].dtype), "h": s["h"]}


class _Chunks:
    """The sequence cut into chunks [B, H, chunk, token, width], in 32 bits, with the matrices of the chunk form."""

    def __init__(self, s):
        c = s["case"]
        self.B, self.T, self.H, self.KH = c["B"], c["T"], c["H"], c["KH"]
        self.G = self.H // self.KH
        self.nc = -(-self.T // _CHUNK)
        t = torch.arange(self.T, device="cuda")
        self.live = (t < s["lens"][:, None]) if s["lens"] is not None else (t < self.T).expand(self.B, -1)  # [B, T]
        self.q, self.k = (self.cut(s[n].repeat_interleave(self.G, 2)) for n in ("q", "k"))
        self.v = self.cut(s["v"])
        beta, g = self.cut(s["beta"][..., None]), self.cut(s["g"][..., None])
        self.beta = beta
        sums = torch.cumsum(g.double(), 3)
        self.eg = torch.exp(sums).float()  # exp(G_i): decay since the chunk began
        self.ee = torch.exp(sums[..., -1:, :] - sums).float()  # exp(G_end - G_i)
        self.gend = self.eg[..., -1:, :]
        low = torch.ones(_CHUNK, _CHUNK, device="cuda").tril().bool()
        self.m = torch.where(low, torch.exp(torch.where(low, sums - sums.transpose(3, 4), 0.0)), 0.0).float()  # i >= j
        self.strict = self.m * torch.ones(_CHUNK, _CHUNK, device="cuda").tril(-1)
        a = beta * self.strict * (self.k @ self.k.transpose(3, 4))
        self.t = torch.eye(_CHUNK, device="cuda").expand_as(a).clone()  # (I + a)^-1 by forward substitution
        for i in range(1, _CHUNK):
            self.t[..., i, :i] = -(a[..., i : i + 1, :i] @ self.t[..., :i, :i])[..., 0, :]
        self.scale = s["scale"]

    def cut(self, x):
        """[B, T, H, w] -> [B, H, chunk, token, w], zero where no token is."""
        x = torch.where(self.live[:, :, None, None], x.float(), 0.0)
        pad = self.nc * _CHUNK - self.T
        x = torch.cat([x, x.new_zeros(self.B, pad, *x.shape[2:])], 1) if pad else x
        return x.reshape(self.B, self.nc, _CHUNK, self.H, -1).permute(0, 3, 1, 2, 4)

    def join(self, x):
        """[B, H, chunk, token, w] -> [B, T, H, w], zero where no token is."""
        x = x.permute(0, 2, 3, 1, 4).reshape(self.B, self.nc * _CHUNK, self.H, -1)[:, : self.T]
        return torch.where(self.live[:, :, None, None], x, 0.0)

    def scan(self, s):
        """The state entering each chunk, each chunk's writes u, and the last state."""
        h = s["h0"].clone() if s["h0"] is not None else torch.zeros(self.B, self.H, s["case"]["N"], s["case"]["P"], device="cuda")
        states, writes = [], []
        kd = (self.ee * self.k).transpose(3, 4)
        ke = self.eg * self.k
        for c in range(self.nc):
            u = self.t[:, :, c] @ (self.beta[:, :, c] * (self.v[:, :, c] - ke[:, :, c] @ h))
            states.append(h)
            writes.append(u)
            h = self.gend[:, :, c] * h + kd[:, :, c] @ u
        return torch.stack(states, 2), torch.stack(writes, 2), h


def _fwd_plain(s):
    c = _Chunks(s)
    states, u, h = c.scan(s)
    o = c.scale * ((c.eg * c.q) @ states + (c.m * (c.q @ c.k.transpose(3, 4))) @ u)
    return {"o": c.join(o).to(s["v"].dtype), "h": h}


def _bwd_plain(s):
    c = _Chunks(s)
    states, u, h = c.scan(s)
    do = c.cut(s["do"])
    p = c.scale * c.m * (c.q @ c.k.transpose(3, 4))
    direct = p.transpose(3, 4) @ do  # what o asks of u
    kd, qe, ke = c.ee * c.k, c.scale * c.eg * c.q, c.eg * c.k
    dh = s["dh"].clone() if s["dh"] is not None else torch.zeros_like(h)
    after, z = [None] * c.nc, [None] * c.nc  # the gradient of the state leaving each chunk; that of beta (v - ..)
    for i in reversed(range(c.nc)):
        after[i] = dh
        z[i] = c.t[:, :, i].transpose(2, 3) @ (direct[:, :, i] + kd[:, :, i] @ dh)
        dh = c.gend[:, :, i] * dh + qe[:, :, i].transpose(2, 3) @ do[:, :, i] - ke[:, :, i].transpose(2, 3) @ (c.beta[:, :, i] * z[i])
    after, z = torch.stack(after, 2), torch.stack(z, 2)
    dp = c.scale * c.m * (do @ u.transpose(3, 4))
    zu = c.strict * (z @ u.transpose(3, 4))
    zs = z @ states.transpose(3, 4)
    n = -c.beta * zu
    gq = c.scale * c.eg * (do @ states.transpose(3, 4)) + dp @ c.k
    gk = dp.transpose(3, 4) @ c.q + (n + n.transpose(3, 4)) @ c.k - c.beta * c.eg * zs + c.ee * (u @ after.transpose(3, 4))
    gv = c.beta * z
    gbeta = (z * c.v).sum(4) - c.eg[..., 0] * (c.k * zs).sum(4) - (zu * (c.k @ c.k.transpose(3, 4))).sum(4)
    # dL/dg_t is the sum over u >= t of q.gq - v.gv, and what the next state asks of this one
    leaving = torch.cat([states[:, :, 1:], h[:, :, None]], 2)
    r = ((c.q * gq).double().sum(4) - (c.v * gv).double().sum(4)).flip(3).cumsum(3).flip(3)
    gg = r + (leaving * after).double().sum((3, 4))[..., None]

    def shared(x):  # the key heads' gradients sum over the value heads that read them
        return c.join(x).reshape(c.B, c.T, c.KH, c.G, -1).sum(3)

    dt = s["q"].dtype
    return {"gq": shared(gq).to(dt), "gk": shared(gk).to(dt), "gv": c.join(gv).to(dt), "gg": c.join(gg[..., None])[..., 0].float(),
            "gbeta": c.join(gbeta[..., None])[..., 0], "gh0": dh}


def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] in ("ln", "lnb"):
        R, D = case["R"], case["D"]
        w = (4 if case["wdtype"] == "fp32" else 2) * D * (2 if case["bias"] else 1)
        if case["op"] == "ln":
            return {"bytes": 2 * R * D * e + 8 * R + w, "flops": 7 * R * D}
        return {"bytes": 3 * R * D * e + 8 * R + 2 * w, "flops": 12 * R * D}
    B, H, KH, N, P = (case[k] for k in ("B", "H", "KH", "N", "P"))
    rows = B * case.get("T", 1)
    io = rows * (2 * KH * N * e + 2 * H * P * e + 8 * H)  # q, k, v, o, g, beta
    state = 4 * B * H * N * P
    if case["op"] == "step":
        return {"bytes": io + 2 * state, "flops": 7 * rows * H * N * P}
    # the recurrence itself: three products with the state a token (answer, write, read) and the decay
    if case["op"] == "fwd":
        return {"bytes": io + state * (2 if case["state"] else 1), "flops": 7 * rows * H * N * P}
    # the same again, and for the gradients twice as many products
    return {"bytes": rows * (4 * KH * N * e + 3 * H * P * e + 16 * H) + state * (3 if case["state"] else 1), "flops": 21 * rows * H * N * P}


def exact(case, seed):
    """The recurrence itself, token by token in 64 bits; its gradients by the reversed recurrence."""
    s = prepare(case, seed)
    f = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    op = case["op"]
    if op in ("ln", "lnb"):
        return _exact_norm(f, op)
    B, H, KH, N, P = (case[k] for k in ("B", "H", "KH", "N", "P"))
    head = torch.arange(H, device="cuda") // (H // KH)
    if op == "step":
        at = s["slots"].long() if s["slots"] is not None else torch.arange(B, device="cuda")
        S, o = _exact_token(f["h"][at], f["q"][:, head], f["k"][:, head], f["v"], f["g"], f["beta"])[:2]
        h = f["h"].clone()
        h[at] = S
        return {"o": case["N"] ** -0.5 * o, "h": h}
    T = case["T"]
    if op == "bwd" and 8 * T * B * H * N * P > 100e9:
        return None
    S = f["h0"] if f["h0"] is not None else torch.zeros(B, H, N, P, dtype=torch.float64, device="cuda")
    ends = s["lens"].long() if s["lens"] is not None else torch.full((B,), T, device="cuda")
    kept, errs, outs = [S], [], []
    for t in range(T):
        alive = (t < ends)[:, None]
        new, o, e = _exact_token(S, f["q"][:, t][:, head], f["k"][:, t][:, head], f["v"][:, t], f["g"][:, t], f["beta"][:, t])
        S = torch.where(alive[..., None, None], new, S)
        outs.append(torch.where(alive[..., None], o, 0.0))
        if op == "bwd":
            kept.append(S)
            errs.append(e)
    if op == "fwd":
        return {"o": case["N"] ** -0.5 * torch.stack(outs, 1), "h": S}
    z = lambda *w: torch.zeros(B, T, *w, dtype=torch.float64, device="cuda")  # noqa: E731
    r = {"gq": z(KH, N), "gk": z(KH, N), "gv": z(H, P), "gg": z(H), "gbeta": z(H)}
    dS = f["dh"] if f["dh"] is not None else torch.zeros_like(S)
    for t in reversed(range(T)):
        alive = (t < ends)[:, None]
        k, q = f["k"][:, t][:, head], f["q"][:, t][:, head]
        beta, a = f["beta"][:, t], torch.exp(f["g"][:, t])[..., None, None]
        do = case["N"] ** -0.5 * f["do"][:, t]
        D = dS + q[..., :, None] * do[..., None, :]  # the gradient of S_t
        gq = (kept[t + 1] @ do[..., None])[..., 0]
        ke = (k[..., None, :] @ D)[..., 0, :]  # of the write beta e
        gv = beta[..., None] * ke
        decayed = a * kept[t]
        gk = (D @ (beta[..., None] * errs[t])[..., None])[..., 0] - (decayed @ gv[..., None])[..., 0]
        D = D - k[..., :, None] * gv[..., None, :]  # of the decayed state
        put = lambda x, w: torch.where(alive.reshape(B, *[1] * (w - 1)), x, 0.0)  # noqa: E731
        r["gq"][:, t], r["gk"][:, t] = (put(x.reshape(B, KH, H // KH, N).sum(2), 3) for x in (gq, gk))
        r["gv"][:, t] = put(gv, 3)
        r["gbeta"][:, t] = put((errs[t] * ke).sum(-1), 2)
        r["gg"][:, t] = put((D * decayed).sum((-1, -2)), 2)
        dS = torch.where(alive[..., None, None], a * D, dS)
    r["gh0"] = dS
    return r


def _exact_token(S, q, k, v, g, beta):
    S = torch.exp(g)[..., None, None] * S
    e = v - (k[..., None, :] @ S)[..., 0, :]
    S = S + k[..., :, None] * (beta[..., None] * e)[..., None, :]
    return S, (q[..., None, :] @ S)[..., 0, :], e


def _exact_norm(f, op):
    x = f["x"]
    n = x.shape[1]
    if op == "ln":
        mean = x.sum(1) / n
        var = (x * x).sum(1) / n - mean * mean
        rstd = 1 / torch.sqrt(var + _EPS)
        y = (x - mean.unsqueeze(1)) / torch.sqrt(var + _EPS).unsqueeze(1)
        return {"y": torch.addcmul(f["bias"], y, f["weight"]) if f["bias"] is not None else y * f["weight"], "mean": mean, "rstd": rstd}
    xh = (x - f["mean"].unsqueeze(1)) * f["rstd"].unsqueeze(1)
    a = f["dy"] * f["weight"]
    gx = (a - (a.sum(1) / n).unsqueeze(1) - xh * ((a * xh).sum(1) / n).unsqueeze(1)) * f["rstd"].unsqueeze(1)
    out = {"gx": gx, "gweight": torch.einsum("rd,rd->d", f["dy"], xh)}
    if f["bias"] is not None:
        out["gbias"] = f["dy"].sum(0)
    return out
