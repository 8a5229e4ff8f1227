"""Cases of linear attention with a decay for each head, and of the norms before
and after such a block, with their plain forms.

Linear attention keeps, per batch row and value head, a real state S in
R^{N x P} (N = dstate, P = headdim) that decays and takes each token's value at
its key:

    S_t = exp(g_t) S_{t-1} + k_t v_t^T
    o_t = scale S_t^T q_t

The log decay g is one number a head, or one a token and head.  Key heads may
be fewer than value heads (value head h reads key head h // (H / KH)).  Rows of
a padded batch end at `lens`: what lies behind is not read, and outputs and
gradients there are zero.

The norm before a block takes the residual stream with it (s is what is kept):

    s = residual + alpha (scale * x),   y = norm(s) weight + bias

and the norm after a mixer carries the block's gate z, over groups of columns:

    y = (norm(x) weight + bias) silu(z)    or    y = norm(x silu(z)) weight + bias

norm is the root-mean-square norm (no mean is taken off) or the layer norm.

Operators: linattn_forward and linattn_backward (a sequence), linattn_step (one
token of a decode loop, the state updated in place); add_norm, gated_norm and
the gradients of both.
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
    rows, width = lay.batch * lay.seqlen, lay.nheads * lay.headdim
    return [
        # one sequence being answered: a single token at the width of the PAM layer, one decay a head
        {"name": "step_one", "op": "step", "B": 1, "H": pam.nheads, "KH": pam.nheads, "N": 64, "P": 64, "dtype": "bf16", "decay": "head", "pool": 0},
        # the decode workload: 256 rows of a server's pool of states, decays of the tokens
        {"name": "step_decode", "op": "step", "B": dec.batch, "H": dec.nheads, "KH": dec.nheads, "N": dec.dstate, "P": dec.headdim, "dtype": "bf16", "decay": "token", "pool": dec.batch + 32},
        # one layer over a training batch (mamba2_layer's sizes), decays of the tokens
        {"name": "fwd_layer", "op": "fwd", "B": lay.batch, "T": lay.seqlen, "H": lay.nheads, "KH": lay.nheads, "N": lay.dstate, "P": lay.headdim, "dtype": "bf16", "decay": "token", "ragged": False, "state": False},
        # a long document taken in one call (long_seq's heads and widths), continued from a state, one decay a head
        {"name": "fwd_long", "op": "fwd", "B": lng.batch, "T": lng.seqlen // 4, "H": lng.nheads, "KH": lng.nheads, "N": lng.dstate, "P": lng.headdim, "dtype": "bf16", "decay": "head", "ragged": False, "state": True},
        # prompts of different lengths padded to one batch, key heads shared by two value heads
        {"name": "fwd_prompts", "op": "fwd", "B": 6, "T": 1333, "H": 16, "KH": 8, "N": 128, "P": 128, "dtype": "fp16", "decay": "token", "ragged": True, "state": True},
        # gradients of one layer over a training batch
        {"name": "bwd_layer", "op": "bwd", "B": lay.batch, "T": lay.seqlen, "H": lay.nheads, "KH": lay.nheads, "N": lay.dstate, "P": lay.headdim, "dtype": "bf16", "decay": "token", "ragged": False, "state": False},
        # gradients at the wide head sizes, key heads shared by two value heads, ragged rows, learned decays of the heads
        {"name": "bwd_wide", "op": "bwd", "B": 4, "T": 1501, "H": 16, "KH": 8, "N": 128, "P": 128, "dtype": "bf16", "decay": "head", "ragged": True, "state": True},
        # a small fp32 run, as one trains while looking for a bug
        {"name": "bwd_fp32", "op": "bwd", "B": 2, "T": 515, "H": 12, "KH": 12, "N": 64, "P": 64, "dtype": "fp32", "decay": "token", "ragged": False, "state": False},
        # the norm before that layer over the same tokens (24 heads of 64), the residual stream in fp32
        {"name": "add_layer", "op": "add", "R": rows, "D": width, "dtype": "bf16", "rtype": "fp32", "wtype": "bf16", "kind": "rms", "bias": False, "scale": True},
        # its gradients
        {"name": "addb_layer", "op": "addb", "R": rows, "D": width, "dtype": "bf16", "rtype": "fp32", "wtype": "fp32", "kind": "rms", "bias": False, "scale": True},
        # the norm of the mixer's heads under the gate
        {"name": "gated_layer", "op": "gated", "R": rows, "D": width, "group": lay.headdim, "dtype": "bf16", "wtype": "bf16", "kind": "rms", "bias": False, "first": False},
        # gradients of the norm over the whole row, the gate taken in first
        {"name": "gatedb_layer", "op": "gatedb", "R": rows, "D": width, "group": width, "dtype": "bf16", "wtype": "fp32", "kind": "rms", "bias": False, "first": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "fwd", "fwd", "bwd", "bwd", "add", "addb", "gated", "gatedb"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("add", "addb"):
        D = rng.choice([rng.randint(5, 600), 64 * rng.randint(4, 64), 1000 + rng.randint(0, 3000)])
        R = max(1, min(_log(rng, 1, 40000), 12_000_000 // D))
        return {"op": op, "R": R, "D": D, "dtype": dtype, "rtype": rng.choice([dtype, "fp32"]), "wtype": rng.choice([dtype, "fp32"]),
                "kind": rng.choice(["rms", "layer"]), "bias": rng.random() < 0.4, "scale": rng.random() < 0.5}
    if op in ("gated", "gatedb"):
        group = rng.choice([32, 64, 80, 128, 256, rng.randint(5, 600), 64 * rng.randint(4, 40), 1000 + rng.randint(0, 2000)])
        D = group * rng.randint(1, max(1, min(32, 4096 // group)))
        R = max(1, min(_log(rng, 1, 40000), 12_000_000 // D))
        return {"op": op, "R": R, "D": D, "group": group, "dtype": dtype, "wtype": rng.choice([dtype, "fp32"]),
                "kind": rng.choice(["rms", "rms", "layer"]), "bias": rng.random() < 0.3, "first": rng.random() < 0.5}
    N, P = rng.choice([(64, 64), (128, 64), (128, 128), (64, 128), (32, 64), (16, 16), (96, 80), (128, 32)])
    KH = rng.choice([1, 2, 3, 4, 8, 12, 16])
    H = KH * rng.choice([1, 1, 2, 4])
    decay = rng.choice(["token", "head"])
    if op == "step":
        B = max(1, min(_log(rng, 1, 256), 60_000_000 // (H * N * P)))
        return {"op": op, "B": B, "H": H, "KH": KH, "N": N, "P": P, "dtype": dtype, "decay": decay, "pool": rng.choice([0, B + rng.randint(0, 20)])}
    B = rng.randint(1, 6)
    T = max(1, min(_log(rng, 1, 6000), (150_000 if op == "fwd" else 80_000) // (B * H)))
    return {"op": op, "B": B, "T": T, "H": H, "KH": KH, "N": N, "P": P, "dtype": dtype, "decay": decay, "ragged": B > 1 and rng.random() < 0.4, "state": rng.random() < 0.5}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if case["op"] in ("add", "addb", "gated", "gatedb"):
        return _prepare_norm(case, normal, dt)
    B, H, KH, N, P = (case[k] for k in ("B", "H", "KH", "N", "P"))
    lead = (B,) if case["op"] == "step" else (B, case["T"])
    # decays: each head forgets at a rate of its own, from 1 to some thousands of tokens
    rate = torch.exp(math.log(5e-4) + (math.log(1.0) - math.log(5e-4)) * torch.rand(H, generator=gen, device="cuda"))
    g = -rate if case["decay"] == "head" else -rate * torch.nn.functional.softplus(1 + normal(*lead, H))
    s = {"case": case, "q": normal(*lead, KH, N).to(dt), "k": (N ** -0.5 * normal(*lead, KH, N)).to(dt), "v": normal(*lead, H, P).to(dt),
         "g": g, "scale": N ** -0.5}
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


def _prepare_norm(case, normal, dt):
    R, D = case["R"], case["D"]
    wt = _TYPES[case["wtype"]]
    s = {"case": case, "weight": (1 + 0.2 * normal(D)).to(wt), "bias": (0.2 * normal(D)).to(wt) if case["bias"] else None}
    if case["op"] in ("add", "addb"):
        rt = _TYPES[case["rtype"]]
        s["alpha"] = 0.7
        s["scale"] = (0.5 + 0.2 * normal(D)).to(wt) if case["scale"] else None
        s["x"] = (normal(R, D) * torch.exp(0.5 * normal(R, 1))).to(dt)
        stream = (2 * normal(R, D) + 0.3 * normal(R, 1)).to(rt)
        if case["op"] == "add":
            s["residual"] = stream
            return s
        s["s"] = stream  # what the forward pass kept
        s["dy"] = normal(R, D).to(dt)
        s["ds"] = normal(R, D).to(rt)
        h = stream.double().unsqueeze(1)
    else:
        s["x"] = (normal(R, D) * torch.exp(0.5 * normal(R, 1)) + 0.3 * normal(R, 1)).to(dt)
        s["z"] = (2 * normal(R, D)).to(dt)
        if case["op"] == "gated":
            return s
        s["dy"] = normal(R, D).to(dt)
        h = s["x"].double()
        if case["first"]:
            z = s["z"].double()
            h = h * z * torch.sigmoid(z)
        h = h.reshape(R, -1, case["group"])
    # the statistics that the forward pass left
    mean = h.mean(2) if case["kind"] == "layer" else torch.zeros_like(h[..., 0])
    rstd = ((h - mean[..., None]).square().mean(2) + _EPS).rsqrt()
    mean, rstd = (t.squeeze(1) if case["op"] == "addb" else t for t in (mean, rstd))
    s["mean"] = mean.float() if case["kind"] == "layer" else None
    s["rstd"] = rstd.float()
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    cssd = _calls()
    c = s["case"]
    op = c["op"]
    if op == "add":
        y, kept, mean, rstd = cssd.add_norm(s["x"], s["residual"], s["weight"], s["bias"], kind=c["kind"], alpha=s["alpha"], scale=s["scale"], eps=_EPS)
        return {"y": y, "s": kept, "mean": mean, "rstd": rstd}
    if op == "addb":
        return cssd.add_norm_backward(s["dy"], s["ds"], s["x"], s["s"], s["weight"], s["mean"], s["rstd"], alpha=s["alpha"], scale=s["scale"],
                                      want_bias=s["bias"] is not None)
    if op == "gated":
        y, mean, rstd = cssd.gated_norm(s["x"], s["z"], s["weight"], s["bias"], kind=c["kind"], group=c["group"], gate_first=c["first"], eps=_EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "gatedb":
        return cssd.gated_norm_backward(s["dy"], s["x"], s["z"], s["weight"], s["bias"], s["mean"], s["rstd"], group=c["group"], gate_first=c["first"],
                                        want_bias=s["bias"] is not None)
    if op == "step":
        o = cssd.linattn_step(s["h"], s["q"], s["k"], s["v"], s["g"], scale=s["scale"], slots=s["slots"])
        return {"o": o, "h": s["h"]}
    if op == "fwd":
        o, h = cssd.linattn_forward(s["q"], s["k"], s["v"], s["g"], scale=s["scale"], h0=s["h0"], lens=s["lens"])
        return {"o": o, "h": h}
    return cssd.linattn_backward(s["q"], s["k"], s["v"], s["g"], s["do"], scale=s["scale"], h0=s["h0"], dh_final=s["dh"], lens=s["lens"])


def _run_plain(s):
    op = s["case"]["op"]
    if op == "step":
        return _step_plain(s)
    if op in ("fwd", "bwd"):
        return _fwd_plain(s) if op == "fwd" else _bwd_plain(s)
    return {"add": _add_plain, "addb": _addb_plain, "gated": _gated_plain, "gatedb": _gatedb_plain}[op](s)


def _norm_plain(h, kind):
    """h [.., n] in 32 bits -> (normalised, mean or None, rstd)."""
    mean = h.mean(-1) if kind == "layer" else None
    c = h - mean[..., None] if mean is not None else h
    rstd = (c.square().mean(-1) + _EPS).rsqrt()
    return c * rstd[..., None], mean, rstd


def _norm_back_plain(a, hh, rstd, layer):
    """The gradient of h from that of the normalised values."""
    t = a - hh * (a * hh).mean(-1, keepdim=True)
    if layer:
        t = t - a.mean(-1, keepdim=True)
    return t * rstd[..., None]


def _add_plain(s):
    x = s["x"].float()
    if s["scale"] is not None:
        x = x * s["scale"].float()
    kept = (s["residual"].float() + s["alpha"] * x).to(s["residual"].dtype)
    y, mean, rstd = _norm_plain(kept.float(), s["case"]["kind"])
    y = y * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return {"y": y.to(s["x"].dtype), "s": kept, "mean": mean, "rstd": rstd}


def _addb_plain(s):
    dy, h = s["dy"].float(), s["s"].float()
    layer = s["mean"] is not None
    hh = (h - s["mean"][:, None] if layer else h) * s["rstd"][:, None]
    t = s["ds"].float() + _norm_back_plain(dy * s["weight"].float(), hh, s["rstd"], layer)
    x = s["x"].float()
    wt = s["weight"].dtype
    out = {"gresidual": t.to(s["s"].dtype), "gweight": (dy * hh).sum(0).to(wt)}
    if s["scale"] is not None:
        out["gscale"] = (s["alpha"] * (t * x).sum(0)).to(wt)
        t = t * s["scale"].float()
    out["gx"] = (s["alpha"] * t).to(s["x"].dtype)
    if s["bias"] is not None:
        out["gbias"] = dy.sum(0).to(wt)
    return out


def _gated_plain(s):
    c = s["case"]
    x, z = s["x"].float(), s["z"].float()
    gate = z * torch.sigmoid(z)
    h = (x * gate if c["first"] else x).reshape(c["R"], -1, c["group"])
    y, mean, rstd = _norm_plain(h, c["kind"])
    y = y.reshape(c["R"], c["D"]) * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if not c["first"]:
        y = y * gate
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _gatedb_plain(s):
    c = s["case"]
    R, D, layer = c["R"], c["D"], s["mean"] is not None
    x, z, dy, w = s["x"].float(), s["z"].float(), s["dy"].float(), s["weight"].float()
    sg = torch.sigmoid(z)
    gate = z * sg
    slope = sg * (1 + z * (1 - sg))
    h = (x * gate if c["first"] else x).reshape(R, -1, c["group"])
    hh = (h - s["mean"][..., None] if layer else h) * s["rstd"][..., None]
    du = dy if c["first"] else dy * gate
    dh = _norm_back_plain((du * w).reshape(hh.shape), hh, s["rstd"], layer).reshape(R, D)
    hh = hh.reshape(R, D)
    out = {"gweight": (du * hh).sum(0).to(s["weight"].dtype)}
    if s["bias"] is not None:
        out["gbias"] = du.sum(0).to(s["weight"].dtype)
    if c["first"]:
        gx, gz = dh * gate, dh * x * slope
    else:
        u = hh * w
        if s["bias"] is not None:
            u = u + s["bias"].float()
        gx, gz = dh, dy * u * slope
    out["gx"], out["gz"] = gx.to(s["x"].dtype), gz.to(s["z"].dtype)
    return out


def _step_plain(s):
    G = s["case"]["H"] // s["case"]["KH"]
    q, k = (s[n].float().repeat_interleave(G, 1) for n in ("q", "k"))
    h = s["h"] if s["slots"] is None else s["h"][s["slots"].long()]
    h = h * torch.exp(s["g"])[..., None, None] + k[..., None] * s["v"].float()[..., None, :]
    o = s["scale"] * (h * q[..., None]).sum(-2)
    if s["slots"] is None:
        s["h"].copy_(h)
    else:
        s["h"][s["slots"].long()] = h
    return {"o": o.to(s["v"].dtype), "h": s["h"]}


class _Chunks:
    """The sequence cut into chunks [B, H, chunk, token, width], in 32 bits, with the decays between tokens and between chunks (angles of long sums in 64)."""

    def __init__(self, s):
        c = s["case"]
        self.B, self.T, self.H, self.KH, self.N, self.P = (c[k] for k in ("B", "T", "H", "KH", "N", "P"))
        self.G = self.H // self.KH
        self.nc = -(-self.T // _CHUNK)
        t = torch.arange(self.T, device="cuda")
        self.live = (t < s["lens"][:, None]) if s["lens"] is not None else (t < self.T).expand(self.B, -1)  # [B, T]
        self.q, self.k = (self.cut(s[n].repeat_interleave(self.G, 2)) for n in ("q", "k"))
        self.v = self.cut(s["v"])
        g = s["g"].expand(self.B, self.T, self.H)
        sums = torch.cumsum(self.cut(g[..., None]).double(), 3)
        self.eg = torch.exp(sums).float()  # exp(G_i): decay since the chunk began
        self.ee = torch.exp(sums[..., -1:, :] - sums).float()  # exp(G_end - G_i)
        low = torch.ones(_CHUNK, _CHUNK, device="cuda").tril().bool()
        self.m = torch.where(low, torch.exp(torch.where(low, sums - sums.transpose(3, 4), 0.0)), 0.0).float()  # i >= j
        ends = torch.cumsum(sums[..., -1, 0], 2)  # [B, H, chunk]: from the start through each chunk
        begins = torch.cat([torch.zeros_like(ends[..., :1]), ends], 2)  # [B, H, chunk + 1]: up to each chunk, and through the last
        low = torch.ones(self.nc + 1, self.nc, device="cuda").tril(-1).bool()  # chunk c (row) comes after chunk d
        self.between = torch.where(low, torch.exp(torch.where(low, begins[..., :, None] - ends[..., None, :], 0.0)), 0.0).float()
        self.begin = torch.exp(begins).float()
        self.after = torch.exp(ends[..., -1:] - ends).float()  # from the end of each chunk to the last one's
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

    def states(self, s):
        """The state before each chunk, and after the last."""
        new = ((self.ee * self.k).transpose(3, 4) @ self.v).reshape(self.B, self.H, self.nc, -1)
        h = self.between @ new
        if s["h0"] is not None:
            h = h + self.begin[..., None] * s["h0"].reshape(self.B, self.H, 1, -1)
        return h.reshape(self.B, self.H, self.nc + 1, self.N, self.P)


def _fwd_plain(s):
    c = _Chunks(s)
    h = c.states(s)
    o = c.scale * ((c.eg * c.q) @ h[:, :, :-1] + (c.m * (c.q @ c.k.transpose(3, 4))) @ c.v)
    return {"o": c.join(o).to(s["v"].dtype), "h": h[:, :, -1].contiguous()}


def _bwd_plain(s):
    c = _Chunks(s)
    h = c.states(s)
    do = c.cut(s["do"])
    # the gradient of the state after each chunk, and of the first one
    asks = c.scale * (c.eg * c.q).transpose(3, 4) @ do
    back = torch.cat([asks.new_zeros(c.B, c.H, 1, c.N * c.P), asks.reshape(c.B, c.H, c.nc, -1)], 2)
    reach = c.between.transpose(2, 3)  # [chunk d, chunk c]: from the end of d to the start of c
    dS = torch.cat([c.begin[:, :, None, :-1] @ back[:, :, 1:], reach[..., :-1] @ back[:, :, 1:]], 2)
    if s["dh"] is not None:
        dS = dS + torch.cat([c.begin[..., -1:], c.after], 2)[..., None] * s["dh"].reshape(c.B, c.H, 1, -1)
    dS = dS.reshape(c.B, c.H, c.nc + 1, c.N, c.P)
    first, dS = dS[:, :, 0].contiguous(), dS[:, :, 1:]
    dp = c.scale * c.m * (do @ c.v.transpose(3, 4))
    p = c.scale * c.m * (c.q @ c.k.transpose(3, 4))
    gq = c.scale * c.eg * (do @ h[:, :, :-1].transpose(3, 4)) + dp @ c.k
    gk = c.ee * (c.v @ dS.transpose(3, 4)) + dp.transpose(3, 4) @ c.q
    gv = c.ee * (c.k @ dS) + p.transpose(3, 4) @ do
    # dL/dg_t is the sum over u >= t of q.gq - k.gk (in the chunk), and what the next chunk asks of the state
    r = ((c.q * gq).sum(4).double() - (c.k * gk).sum(4).double()).flip(3).cumsum(3).flip(3)
    gg = c.join((r + (h[:, :, 1:].double() * dS.double()).sum((3, 4))[..., None])[..., None])[..., 0]

    def shared(x):  # the key heads' gradients sum over the value heads that read them
        return c.join(x).reshape(c.B, c.T, c.KH, c.G, -1).sum(3)

    dt = s["q"].dtype
    return {"gq": shared(gq).to(dt), "gk": shared(gk).to(dt), "gv": c.join(gv).to(dt), "gg": (gg.sum((0, 1)) if s["g"].dim() == 1 else gg).float(), "gh0": first}


def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    op = case["op"]
    if op in ("add", "addb", "gated", "gatedb"):
        R, D = case["R"], case["D"]
        w = (4 if case["wtype"] == "fp32" else 2) * D
        if op in ("add", "addb"):
            r = 4 if case["rtype"] == "fp32" else 2
            vectors = w * (1 + case["bias"] + case["scale"])
            stats = 4 * R * (2 if case["kind"] == "layer" else 1)
            if op == "add":
                return {"bytes": R * D * (2 * e + 2 * r) + stats + vectors, "flops": 8 * R * D}
            return {"bytes": R * D * ((2 + case["scale"]) * e + 3 * r) + stats + w * (2 + case["bias"] + 2 * case["scale"]), "flops": 16 * R * D}
        stats = 4 * R * (D // case["group"]) * (2 if case["kind"] == "layer" else 1)
        if op == "gated":
            return {"bytes": 3 * R * D * e + stats + w * (1 + case["bias"]), "flops": 12 * R * D}
        return {"bytes": 5 * R * D * e + stats + 2 * w * (1 + case["bias"]), "flops": 28 * R * D}
    B, H, KH, N, P = (case[k] for k in ("B", "H", "KH", "N", "P"))
    rows = B * case.get("T", 1)
    g = 4 * (H if case["decay"] == "head" else rows * H)
    io = rows * (2 * KH * N * e + 2 * H * P * e) + g  # q, k, v, o, g
    state = 4 * B * H * N * P
    if op == "step":
        return {"bytes": io + 2 * state, "flops": 5 * rows * H * N * P}
    # the recurrence itself: the decay, the write and the answer, five operations a state element and token
    if op == "fwd":
        return {"bytes": io + state * (2 if case["state"] else 1), "flops": 5 * rows * H * N * P}
    # the same again, and for the gradients twice as many products
    return {"bytes": rows * (4 * KH * N * e + 3 * H * P * e) + 2 * g + state * (3 if case["state"] else 1), "flops": 15 * rows * H * N * P}


def exact(case, seed):
    """The recurrence itself, token by token in 64 bits; its gradients by the reversed recurrence."""
    s = prepare(case, seed)
    f = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    op = case["op"]
    if op in ("add", "addb"):
        return _exact_add(f, s, op)
    if op in ("gated", "gatedb"):
        return _exact_gated(f, case)
    B, H, KH, N, P = (case[k] for k in ("B", "H", "KH", "N", "P"))
    head = torch.arange(H, device="cuda") // (H // KH)
    if op == "step":
        at = s["slots"].long() if s["slots"] is not None else torch.arange(B, device="cuda")
        S = torch.exp(f["g"])[..., None, None] * f["h"][at] + torch.einsum("bhn,bhp->bhnp", f["k"][:, head], f["v"])
        h = f["h"].clone()
        h[at] = S
        return {"o": N ** -0.5 * torch.einsum("bhn,bhnp->bhp", f["q"][:, head], S), "h": h}
    T = case["T"]
    if op == "bwd" and 8 * T * B * H * N * P > 100e9:
        return None
    S = f["h0"] if f["h0"] is not None else torch.zeros(B, H, N, P, dtype=torch.float64, device="cuda")
    ends = s["lens"].long() if s["lens"] is not None else torch.full((B,), T, device="cuda")
    decay = torch.exp(f["g"].expand(B, T, H))
    kept, outs = [S], []
    for t in range(T):
        alive = (t < ends)[:, None]
        new = torch.addcmul(decay[:, t, :, None, None] * S, f["k"][:, t][:, head][..., :, None], f["v"][:, t][..., None, :])
        S = torch.where(alive[..., None, None], new, S)
        if op == "fwd":
            o = (f["q"][:, t][:, head][..., None, :] @ new)[..., 0, :]
            outs.append(torch.where(alive[..., None], o, 0.0))
        else:
            kept.append(S)
    if op == "fwd":
        return {"o": N ** -0.5 * torch.stack(outs, 1), "h": S}
    z = lambda *w: torch.zeros(B, T, *w, dtype=torch.float64, device="cuda")  # noqa: E731
    r = {"gq": z(KH, N), "gk": z(KH, N), "gv": z(H, P), "gg": z(H)}
    D = f["dh"] if f["dh"] is not None else torch.zeros_like(S)
    for t in reversed(range(T)):
        alive = (t < ends)[:, None]
        k, q = f["k"][:, t][:, head], f["q"][:, t][:, head]
        do = N ** -0.5 * f["do"][:, t]
        X = torch.addcmul(D, q[..., :, None], do[..., None, :])  # the gradient of S_t
        put = lambda x, w: torch.where(alive.reshape(B, *[1] * (w - 1)), x, 0.0)  # noqa: E731
        gq = (kept[t + 1] @ do[..., None])[..., 0]
        gk = (X @ f["v"][:, t][..., None])[..., 0]
        r["gq"][:, t], r["gk"][:, t] = (put(x.reshape(B, KH, H // KH, N).sum(2), 3) for x in (gq, gk))
        r["gv"][:, t] = put((k[..., None, :] @ X)[..., 0, :], 3)
        r["gg"][:, t] = put(decay[:, t] * (X * kept[t]).sum((-1, -2)), 2)
        D = torch.where(alive[..., None, None], decay[:, t, :, None, None] * X, D)
    if case["decay"] == "head":
        r["gg"] = r["gg"].sum((0, 1))
    r["gh0"] = D
    return r


def _exact_stats(h, kind):
    n = h.shape[-1]
    mean = h.sum(-1) / n if kind == "layer" else None
    var = (h * h).sum(-1) / n - (mean * mean if mean is not None else 0)
    return mean, 1 / torch.sqrt(var + _EPS)


def _exact_add(f, s, op):
    wx = f["x"] * f["scale"] if f["scale"] is not None else f["x"]
    if op == "add":
        kept = torch.add(f["residual"], wx, alpha=f["alpha"])
        h = kept.to(s["residual"].dtype).double()  # the norm is of what is kept
        mean, rstd = _exact_stats(h, f["case"]["kind"])
        y = (h if mean is None else h - mean.unsqueeze(1)) * rstd.unsqueeze(1) * f["weight"]
        return {"y": y + f["bias"] if f["bias"] is not None else y, "s": kept, "mean": mean, "rstd": rstd}
    n = f["s"].shape[1]
    hh = (f["s"] - f["mean"].unsqueeze(1) if f["mean"] is not None else f["s"]) * f["rstd"].unsqueeze(1)
    a = f["dy"] * f["weight"]
    t = a - hh * (torch.einsum("rd,rd->r", a, hh) / n).unsqueeze(1)
    if f["mean"] is not None:
        t = t - (a.sum(1) / n).unsqueeze(1)
    t = torch.addcmul(f["ds"], t, f["rstd"].unsqueeze(1))
    out = {"gresidual": t, "gx": f["alpha"] * t, "gweight": torch.einsum("rd,rd->d", f["dy"], hh)}
    if f["scale"] is not None:
        out["gx"] = out["gx"] * f["scale"]
        out["gscale"] = f["alpha"] * torch.einsum("rd,rd->d", t, f["x"])
    if f["bias"] is not None:
        out["gbias"] = f["dy"].sum(0)
    return out


def _exact_gated(f, case):
    R, D, n = case["R"], case["D"], case["group"]
    split = lambda x: x.reshape(R, D // n, n)  # noqa: E731
    x, z = split(f["x"]), split(f["z"])
    w, b = (t.reshape(1, D // n, n) if t is not None else None for t in (f["weight"], f["bias"]))
    sg = 1 / (1 + torch.exp(-z))
    h = x * z * sg if case["first"] else x
    if case["op"] == "gated":
        mean, rstd = _exact_stats(h, case["kind"])
        u = (h if mean is None else h - mean.unsqueeze(2)) * rstd.unsqueeze(2) * w
        u = u if b is None else u + b
        return {"y": (u if case["first"] else u * z * sg).reshape(R, D), "mean": mean, "rstd": rstd}
    dy, rstd = split(f["dy"]), f["rstd"].unsqueeze(2)
    hh = (h if f["mean"] is None else h - f["mean"].unsqueeze(2)) * rstd
    du = dy if case["first"] else dy * z * sg
    a = du * w
    dh = a - hh * ((a * hh).sum(2, keepdim=True) / n)
    if f["mean"] is not None:
        dh = dh - a.sum(2, keepdim=True) / n
    dh = dh * rstd
    u = hh * w if b is None else hh * w + b
    dgate = dh * x if case["first"] else dy * u
    out = {"gx": dh * z * sg if case["first"] else dh, "gz": dgate * (sg + z * sg * (1 - sg))}
    out = {k: v.reshape(R, D) for k, v in out.items()}
    out["gweight"] = torch.einsum("rgn,rgn->gn", du, hh).reshape(D)
    if b is not None:
        out["gbias"] = du.sum(0).reshape(D)
    return out
