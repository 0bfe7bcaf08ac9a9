"""Measured cases of the gated delta rule (a state that is corrected towards
each value instead of only added to), of the group norm with an activation
that follows such a state, and of activations kept in 8 bits for the backward
pass: prompts, gradients and single tokens.

``run`` computes a case in plain torch operations, or, with ``own`` set, by the
calls a program makes of this framework.  Layouts are the framework's: tokens
are rows, channels are contiguous; q and k are [B, L, G, N], v is [B, L, H, P],
states are [B, H, N, P].
"""
import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "f32": torch.float32}
_BLOCK = 64     # values that share a scale in 8 bits
_C = 64         # tokens the plain form of the delta rule takes at a time
_EPS = 1e-5     # of the norms
_QK_EPS = 1e-6  # of the unit length of q and k


# ---------------------------------------------------------------- cases

def listed():
    return [
        # A prompt through a layer of 32 heads over 16 key heads, going on from
        # a cached state, which is returned for decoding.
        dict(name="delta_prompt", op="delta_forward", B=2, L=8192, H=32, G=16, N=128, P=128, dtype="bf16", packed=0,
             state=1),
        # One very long prompt on one rank's few heads: parallel only along
        # the tokens.
        dict(name="delta_prompt_long", op="delta_forward", B=1, L=65536, H=8, G=4, N=128, P=128, dtype="bf16",
             packed=0, state=0),
        # A short chat turn at the 130M layer's heads (24 of 64 columns, one
        # key head), packed from several requests.
        dict(name="delta_turn_packed", op="delta_forward", B=1, L=700, H=24, G=1, N=128, P=64, dtype="bf16",
             packed=5, state=1),
        # A training step's gradients.
        dict(name="delta_train", op="delta_backward", B=2, L=2048, H=32, G=16, N=128, P=128, dtype="bf16", packed=0,
             state=0),
        # Training on packed sequences at the 130M layer's heads.
        dict(name="delta_train_packed", op="delta_backward", B=4, L=2048, H=24, G=1, N=128, P=64, dtype="bf16",
             packed=16, state=0),
        # Odd sizes in fp32, with the gradient of the state that came in.
        dict(name="delta_train_ragged_f32", op="delta_backward", B=2, L=777, H=6, G=3, N=48, P=80, dtype="f32",
             packed=0, state=1),
        # Decoding for 64 streams at once, and for one.
        dict(name="delta_step_64", op="delta_step", B=64, L=1, H=32, G=16, N=128, P=128, dtype="bf16", packed=0,
             state=1),
        dict(name="delta_step_1", op="delta_step", B=1, L=1, H=24, G=1, N=128, P=64, dtype="bf16", packed=0, state=1),
        # The heads' norm and gate over the prompt of a 2.7B layer (80 heads of
        # 64), the gate read in place out of the input projection's rows.
        dict(name="group_norm_prompt", op="group_norm_forward", rows=16384, D=5120, groups=80, zrow=10576,
             dtype="bf16", rms=1, gate="after", shared=1, bias=0),
        # Its gradients in training, from x and gate kept in 8 bits.
        dict(name="group_norm_train_kept8", op="group_norm_backward", rows=8192, D=4096, groups=32, zrow=4096,
             dtype="bf16", rms=1, gate="after", shared=1, bias=0, kept8=1),
        # The convolution's input (5376 of the projection's 10576 columns) put
        # into 8 bits, to be kept for the backward pass.
        dict(name="pack8_projection", op="pack8", rows=16384, D=5376, row=10576, dtype="bf16"),
        # The other way, for one training step's tokens: the same columns of
        # the 130M layer's rows, in place.
        dict(name="unpack8_projection", op="unpack8", rows=8192, D=1792, row=3352, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["delta_forward"] * 4 + ["delta_backward"] * 4 + ["delta_step"] * 2 + ["group_norm_forward"] * 2 +
                    ["group_norm_backward"] * 3 + ["pack8", "unpack8"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("delta"):
        G = rng.choice([1, 1, 2, 3, 4, 8, 16])
        H = G * rng.choice([1, 2, 2, 3, 4])
        N = rng.choice([16, 32, 48, 64, 64, 96, 128, 128, 128, 256])
        P = rng.choice([16, 32, 48, 64, 64, 80, 128, 128, 128, 256])
        if op == "delta_step":
            return dict(op=op, B=_log(rng, 1, 96), L=1, H=H, G=G, N=N, P=P, dtype=dtype, packed=0, state=1)
        most = 3_000_000_000 if op == "delta_forward" else 500_000_000
        B = _log(rng, 1, 6)
        L = _log(rng, 1, max(1, min(30_000 if op == "delta_forward" else 4000, most // (B * H * N * P))))
        return dict(op=op, B=B, L=L, H=H, G=G, N=N, P=P, dtype=dtype, packed=min(rng.choice([0, 0, 3, 9]), L),
                    state=rng.choice([0, 1]))
    if op.endswith("pack8"):
        D = _log(rng, 64, 12000)
        if rng.random() < 0.6:
            D = max(64, D // 64 * 64)
        rows = _log(rng, 1, max(1, 60_000_000 // D))
        return dict(op=op, rows=rows, D=D, row=D + rng.choice([0, 0, 64, 8, 1]), dtype=dtype)
    groups = _log(rng, 1, 80)
    size = rng.choice([16, 32, 64, 64, 80, 100, 128, 128, 192, 256, 37, 512, 1000, 2048])
    groups = max(1, min(groups, 12000 // size))
    D = groups * size
    rows = _log(rng, 1, max(1, 30_000_000 // D))
    c = dict(op=op, rows=rows, D=D, groups=groups, zrow=D + rng.choice([0, 0, 8, 256, 1]), dtype=dtype,
             rms=rng.choice([0, 1, 1]), gate=rng.choice(["after", "after", "first", "none", "self"]),
             shared=rng.choice([0, 1]), bias=rng.choice([0, 1]))
    if op == "group_norm_backward":
        c["kept8"] = rng.choice([0, 1])
    return c


# ---------------------------------------------------------------- inputs

class _Maker:
    def __init__(self, seed):
        self.dev = "cuda" if torch.cuda.is_available() else "cpu"
        self.g = torch.Generator(device=self.dev).manual_seed(seed)

    def randn(self, shape, dtype=torch.float32, scale=1.0):
        t = torch.randn(shape, generator=self.g, device=self.dev, dtype=torch.float32)
        return (t.mul_(scale) if scale != 1.0 else t).to(dtype)

    def rand(self, shape):
        return torch.rand(shape, generator=self.g, device=self.dev, dtype=torch.float32)


def _seq_idx(m, B, L, packed):
    """[B, L] int32: `packed` sequences a row, of random lengths."""
    cuts = (m.rand((B, max(packed - 1, 1))) * L).long().clamp_(0, L - 1)
    idx = torch.zeros((B, L), device=m.dev, dtype=torch.int64)
    if packed > 1:
        idx.scatter_add_(1, cuts, torch.ones_like(cuts))
    return idx.cumsum(1).to(torch.int32).contiguous()


def _activations(m, shape, dtype):
    """Values with a few channels far larger than the others, as projections have them."""
    t = m.randn(shape, scale=0.7)
    return (t * torch.exp(m.randn(shape[-1:], scale=0.5))).to(dtype)


def _to8(x):
    """Plain 8-bit form of rows of values: whole numbers -127 .. 127 and a bf16
    scale for each _BLOCK values, the largest magnitude / 127 rounded up to bf16."""
    D = x.shape[-1]
    nb = -(-D // _BLOCK)
    x = torch.nn.functional.pad(x.float(), (0, nb * _BLOCK - D)).unflatten(-1, (nb, _BLOCK))
    most = x.abs().amax(-1)
    # 127 times a candidate has 15 bits and is exact
    scale = (most / 127).to(torch.bfloat16)
    up = (scale.view(torch.int16) + 1).view(torch.bfloat16)
    scale = torch.where(scale.float() * 127 < most, up, scale)
    s = scale.float()[..., None]
    q = torch.where(s > 0, torch.round(x / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(x))
    return q.to(torch.int8).flatten(-2)[..., :D].contiguous(), scale


def _from8(q, scale):
    D = q.shape[-1]
    return q.float() * scale.float().repeat_interleave(_BLOCK, -1)[..., :D]


def prepare(case, seed):
    m = _Maker(seed)
    c = case
    t = _T[c["dtype"]]
    s = dict(case=dict(c))
    if c["op"] in ("pack8", "unpack8"):
        x = _activations(m, (c["rows"], c["row"]), t)[:, :c["D"]]
        if c["op"] == "pack8":
            s["x"] = x
        else:
            s["q"], s["scale"] = _to8(x)
            s["out"] = torch.empty((c["rows"], c["row"]), device=m.dev, dtype=t)[:, :c["D"]]
        return s
    if c["op"].startswith("group_norm"):
        rows, D, groups = c["rows"], c["D"], c["groups"]
        wn = D // groups if c["shared"] else D
        s["weight"] = 1.0 + m.randn((wn,), scale=0.1)
        s["bias"] = m.randn((wn,), scale=0.1) if c["bias"] else None
        s["x"] = _activations(m, (rows, D), t)
        s["z"] = m.randn((rows, c["zrow"]), t)[:, :D] if c["gate"] in ("after", "first") else None
        if c["op"] == "group_norm_backward":
            s["dy"] = m.randn((rows, D), t)
            # the statistics are the forward's, of the values before they went into 8 bits
            v = s["x"].double()
            if c["gate"] == "first":
                v = v * s["z"].double() * torch.sigmoid(s["z"].double())
            v = v.view(rows, groups, -1)
            mean = None if c["rms"] else v.mean(-1)
            d = v if c["rms"] else v - mean[..., None]
            s["rstd"] = ((d * d).mean(-1) + _EPS).rsqrt().float()
            s["mean"] = None if mean is None else mean.float()
            if c["kept8"]:
                s["x"] = _to8(s["x"])
                s["z"] = None if s["z"] is None else _to8(s["z"])
            if own:
                from mamba_ssd_scan_chunk_amd import ops
                s["workspace"] = torch.empty(max(ops.ssd_group_norm_backward_workspace_bytes(rows, D, groups), 1),
                                             device=m.dev, dtype=torch.uint8)
        return s

    B, L, H, G, N, P = (c[k] for k in "BLHGNP")
    lead = (B,) if c["op"] == "delta_step" else (B, L)
    # q, k and v side by side, as one convolution leaves them
    qkv = m.randn(lead + (2 * G * N + H * P,), t)
    s["q"] = qkv[..., :G * N].unflatten(-1, (G, N))
    s["k"] = qkv[..., G * N:2 * G * N].unflatten(-1, (G, N))
    s["v"] = qkv[..., 2 * G * N:].unflatten(-1, (H, P))
    # the raw decay and writing strength of every head, side by side
    ab = m.randn(lead + (2 * H,), t)
    s["dt"], s["beta"] = ab[..., :H], ab[..., H:]
    s["A"] = -(1.0 + 15.0 * m.rand((H,)))
    dt0 = torch.exp(m.rand((H,)) * (math.log(0.1) - math.log(1e-3)) + math.log(1e-3))
    s["dt_bias"] = (dt0 + torch.log(-torch.expm1(-dt0))).contiguous()
    s["seq_idx"] = _seq_idx(m, B, L, c["packed"]) if c["packed"] else None
    s["h0"] = m.randn((B, H, N, P), scale=0.3) if c["state"] else None
    if c["op"] == "delta_step":
        s["y"] = torch.empty((B, H, P), device=m.dev, dtype=t)
        s["state_out"] = torch.empty_like(s["h0"])
        return s
    if c["op"] == "delta_backward":
        s["dy"] = m.randn((B, L, H, P), t)
        s["dfinal"] = m.randn((B, H, N, P), scale=0.3) if c["state"] else None
    if own:
        from mamba_ssd_scan_chunk_amd import ops
        f = (ops.ssd_delta_rule_workspace_bytes if c["op"] == "delta_forward"
             else ops.ssd_delta_rule_backward_workspace_bytes)
        s["workspace"] = torch.empty(max(f(B, L, H, G, N, P, t), 1), device=m.dev, dtype=torch.uint8)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return _own(s) if own else _PLAIN[s["case"]["op"]](s)


def _own(s):
    from mamba_ssd_scan_chunk_amd import ops
    c = s["case"]
    op = c["op"]
    if op == "delta_forward":
        y, fin = ops.ssd_delta_rule(s["q"], s["k"], s["v"], s["dt"], s["beta"], s["A"], dt_bias=s["dt_bias"],
                                    initial_states=s["h0"], seq_idx=s["seq_idx"], want_final=True,
                                    workspace=s["workspace"])
        return dict(y=y, final=fin)
    if op == "delta_backward":
        r = ops.ssd_delta_rule_backward(s["q"], s["k"], s["v"], s["dt"], s["beta"], s["A"], s["dy"],
                                        dt_bias=s["dt_bias"], initial_states=s["h0"], dfinal=s["dfinal"],
                                        seq_idx=s["seq_idx"], want_dinitial=s["h0"] is not None,
                                        workspace=s["workspace"])
        return {k: r[k] for k in ("dq", "dk", "dv", "ddt", "dbeta", "dA", "ddt_bias", "dinitial") if r[k] is not None}
    if op == "delta_step":
        y = ops.ssd_delta_step(s["q"], s["k"], s["v"], s["dt"], s["beta"], s["A"], s["h0"], dt_bias=s["dt_bias"],
                               y=s["y"], state_out=s["state_out"])
        return dict(y=y, state=s["state_out"])
    if op == "pack8":
        q, scale = ops.ssd_pack8(s["x"])
        return dict(values=q, scale=scale)
    if op == "unpack8":
        return dict(x=ops.ssd_unpack8(s["q"], s["scale"], x=s["out"]))
    how = dict(bias=s["bias"], z=s["z"], groups=c["groups"], rms=bool(c["rms"]), gate_first=c["gate"] == "first",
               silu=c["gate"] == "self")
    if op == "group_norm_forward":
        y, mean, rstd = ops.ssd_group_norm(s["x"], s["weight"], eps=_EPS, **how)
        return dict(y=y, rstd=rstd) if mean is None else dict(y=y, rstd=rstd, mean=mean)
    r = ops.ssd_group_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], workspace=s["workspace"],
                                    **how)
    return {k: r[k] for k in ("dx", "dz", "dweight", "dbias") if r[k] is not None}


# ---- plain forms: elementary torch operations in 32 bits, rounded once at the end

def _plain_pack8(s):
    q, scale = _to8(s["x"])
    return dict(values=q, scale=scale)


def _plain_unpack8(s):
    return dict(x=_from8(s["q"], s["scale"]).to(s["out"].dtype))


def _norm_inputs(s):
    """x and z in 32 bits, from wherever they are kept."""
    get = lambda v: None if v is None else _from8(*v) if isinstance(v, tuple) else v.float()
    return get(s["x"]), get(s["z"])


def _plain_group_norm_forward(s):
    c = s["case"]
    rows, groups = c["rows"], c["groups"]
    x, z = _norm_inputs(s)
    act = None if z is None else z / (1 + torch.exp(-z))
    if c["gate"] == "first":
        x = x * act
    x = x.view(rows, groups, -1)
    mean = None if c["rms"] else x.mean(-1)
    d = x if mean is None else x - mean[..., None]
    rstd = 1 / torch.sqrt((d * d).mean(-1) + _EPS)
    wide = lambda w: w if c["shared"] else w.view(groups, -1)
    y = d * rstd[..., None] * wide(s["weight"])
    if s["bias"] is not None:
        y = y + wide(s["bias"])
    y = y.view(rows, -1)
    if c["gate"] == "after":
        y = y * act
    if c["gate"] == "self":
        y = y / (1 + torch.exp(-y))
    out = dict(y=y.to(_T[c["dtype"]]), rstd=rstd)
    if mean is not None:
        out["mean"] = mean
    return out


def _plain_group_norm_backward(s):
    c = s["case"]
    rows, groups = c["rows"], c["groups"]
    t = _T[c["dtype"]]
    x, z = _norm_inputs(s)
    dy = s["dy"].float()
    out = {}
    if z is not None:
        sg = 1 / (1 + torch.exp(-z))
        act, dact = z * sg, sg * (1 + z * (1 - sg))
    xin = x
    if c["gate"] == "first":
        x = x * act
    wide = lambda w: w if c["shared"] else w.view(groups, -1)
    x = x.view(rows, groups, -1)
    xh = (x if c["rms"] else x - s["mean"][..., None]) * s["rstd"][..., None]
    pre = xh * wide(s["weight"])
    if s["bias"] is not None:
        pre = pre + wide(s["bias"])
    if c["gate"] == "after":
        out["dz"] = (dy * pre.view(rows, -1) * dact).to(t)
        dy = dy * act
    if c["gate"] == "self":
        p = pre.view(rows, -1)
        sp = 1 / (1 + torch.exp(-p))
        dy = dy * (sp * (1 + p * (1 - sp)))
    dy = dy.view(rows, groups, -1)
    v = dy * wide(s["weight"])
    dx = v - xh * (v * xh).mean(-1, keepdim=True)
    if not c["rms"]:
        dx = dx - v.mean(-1, keepdim=True)
    dx = (dx * s["rstd"][..., None]).view(rows, -1)
    if c["gate"] == "first":
        out["dz"] = (dx * xin * dact).to(t)
        dx = dx * act
    out["dx"] = dx.to(t)
    over = (0, 1) if c["shared"] else 0
    out["dweight"] = (dy * xh).sum(over).view(-1)
    if s["bias"] is not None:
        out["dbias"] = dy.sum(over).view(-1)
    return out


def _delta_terms(s):
    """Unit q (scaled) and k of every head [B, L, H, N], v, the raw time step,
    the log decay and the writing strength [B, L, H], all in 32 bits, and the
    factors of the unit lengths."""
    rep = s["case"]["H"] // s["case"]["G"]
    q, k = s["q"].float(), s["k"].float()
    rq = 1 / torch.sqrt((q * q).sum(-1, keepdim=True) + _QK_EPS)
    rk = 1 / torch.sqrt((k * k).sum(-1, keepdim=True) + _QK_EPS)
    heads = lambda x: x.repeat_interleave(rep, -2)
    raw = s["dt"].float() + s["dt_bias"]
    step = torch.where(raw > 20, raw, torch.log1p(torch.exp(raw.clamp(max=20.0))))
    beta = 1 / (1 + torch.exp(-s["beta"].float()))
    return (heads(q * rq) * (s["case"]["N"] ** -0.5), heads(k * rk), s["v"].float(), raw, step, step * s["A"], beta,
            rq, rk)


def _chunks(x, nc):
    """[B, L, H, ..] -> [B, H, nc, C, ..], padded with zeros."""
    L = x.shape[1]
    x = torch.nn.functional.pad(x.movedim(1, -1), (0, nc * _C - L)).movedim(-1, 1)
    return x.unflatten(1, (nc, _C)).movedim(3, 1).contiguous()


def _unchunk(x, L):
    return x.movedim(1, 3).flatten(1, 2)[:, :L]


def _delta_chunks(s):
    """What the chunks have before any state is known.  With E[t,s] = exp(G_t -
    G_s) k_t.k_s (s < t) the corrected values of a chunk obey
    u = beta (X - E u), X = v - exp(G) k S: u = beta (X + R beta X)."""
    c = s["case"]
    q, k, v, raw, step, g, beta, rq, rk = _delta_terms(s)
    L = c["L"]
    nc = -(-L // _C)
    d = dict(nc=nc, L=L, raw=raw, step=step, rq=rq, rk=rk)
    d["q"], d["k"], d["v"], g, d["beta"] = (_chunks(x, nc) for x in (q, k, v, g, beta))
    d["G"] = g.cumsum(-1)
    dev = q.device
    same = torch.ones((1, 1, nc, _C, _C), device=dev, dtype=torch.bool)
    first = last = torch.ones((1, 1, nc, _C), device=dev, dtype=torch.bool)
    if s["seq_idx"] is not None:
        ids = s["seq_idx"]
        st = torch.zeros_like(ids, dtype=torch.bool)
        st[:, 1:] = ids[:, 1:] != ids[:, :-1]
        seg = _chunks(st.float()[..., None], nc).cumsum(-1)
        same = seg[..., :, None] == seg[..., None, :]
        first = seg == 0                                 # of the sequence that came in
        last = seg == seg[..., -1:]                      # of the one that goes on
    low = torch.ones((_C, _C), device=dev, dtype=torch.bool).tril()
    rel = torch.exp((d["G"][..., :, None] - d["G"][..., None, :]).masked_fill(~(low & same), -math.inf))
    d["rel"] = rel
    d["Pm"] = rel * (d["q"] @ d["k"].transpose(-1, -2))
    E = (rel * (d["k"] @ d["k"].transpose(-1, -2))).tril(-1)
    R = -E
    Eb = E * d["beta"][..., None, :]
    for i in range(1, _C):
        R[..., i, :i] -= (Eb[..., i, None, :i] @ R[..., :i, :i])[..., 0, :]
    d["R"] = R
    d["into"] = torch.exp(d["G"]) * first                # of the state that comes in
    d["rest"] = torch.exp(d["G"][..., -1:] - d["G"]) * last
    d["whole"] = d["into"][..., -1]
    return d


def _delta_states(s, d):
    """States at the chunks' starts [B,H,nc,N,P], w and u, the last state."""
    c = s["case"]
    S = s["h0"] if s["h0"] is not None else torch.zeros((c["B"], c["H"], c["N"], c["P"]), device=d["q"].device)
    at, ws = [], []
    kin = d["k"] * d["into"][..., None]
    kout = (d["k"] * d["rest"][..., None]).transpose(-1, -2)
    be = d["beta"][..., None]
    for i in range(d["nc"]):
        at.append(S)
        X = d["v"][:, :, i] - kin[:, :, i] @ S
        w = X + d["R"][:, :, i] @ (be[:, :, i] * X)
        ws.append(w)
        S = d["whole"][:, :, i, None, None] * S + kout[:, :, i] @ (be[:, :, i] * w)
    return torch.stack(at, 2), torch.stack(ws, 2), S


def _plain_delta_forward(s):
    d = _delta_chunks(s)
    S, w, last = _delta_states(s, d)
    y = (d["q"] * d["into"][..., None]) @ S + d["Pm"] @ (d["beta"][..., None] * w)
    return dict(y=_unchunk(y, d["L"]).to(s["v"].dtype), final=last)


def _plain_delta_backward(s):
    c = s["case"]
    B, L, H, G, N, P = (c[k] for k in "BLHGNP")
    t = s["v"].dtype
    d = _delta_chunks(s)
    S, w, last = _delta_states(s, d)
    q, k, be = d["q"], d["k"], d["beta"][..., None]
    into, rest = d["into"][..., None], d["rest"][..., None]
    u = be * w
    dy = _chunks(s["dy"].float(), d["nc"])
    # the chunks back to front, with the gradient of the state each leaves
    D = s["dfinal"] if s["dfinal"] is not None else torch.zeros_like(last)
    own_ = d["Pm"].transpose(-1, -2) @ dy
    qin, kin, kout = (q * into).transpose(-1, -2), (k * into).transpose(-1, -2), k * rest
    Rt = d["R"].transpose(-1, -2)
    leaving, dus = [None] * d["nc"], [None] * d["nc"]
    for i in range(d["nc"] - 1, -1, -1):
        leaving[i] = D
        du = own_[:, :, i] + kout[:, :, i] @ D
        du = du + Rt[:, :, i] @ (be[:, :, i] * du)
        dus[i] = du
        D = d["whole"][:, :, i, None, None] * D + qin[:, :, i] @ dy[:, :, i] - kin[:, :, i] @ (be[:, :, i] * du)
    Dl, du = torch.stack(leaving, 2), torch.stack(dus, 2)
    dw = be * du
    ut = u.transpose(-1, -2)
    dQK = d["rel"] * (dy @ ut)
    dKK = -(d["rel"] * (dw @ ut)).tril(-1)
    St = S.transpose(-1, -2)
    dq = into * (dy @ St) + dQK @ k
    drow = dKK @ k - into * (dw @ St)
    dcol = rest * (u @ Dl.transpose(-1, -2)) + dQK.transpose(-1, -2) @ q + dKK.transpose(-1, -2) @ k
    # the log decay up to a token multiplies what the token reads and divides what later ones read of it
    dG = (q * dq + k * drow - k * dcol).sum(-1)
    end = d["whole"] * (S * Dl).sum((-1, -2)) + (rest * k * (u @ Dl.transpose(-1, -2))).sum((-1, -2))
    dG[..., -1] += end
    dg = dG.flip(-1).cumsum(-1).flip(-1)
    if s["seq_idx"] is not None:
        # not past the end of the token's own sequence
        ids = s["seq_idx"]
        st = torch.zeros_like(ids, dtype=torch.bool)
        st[:, 1:] = ids[:, 1:] != ids[:, :-1]
        seg = _chunks(st.float()[..., None], d["nc"]).cumsum(-1)
        same = (seg[..., :, None] == seg[..., None, :]) & torch.ones((_C, _C), device=seg.device, dtype=torch.bool).triu()
        dg = (same * dG[..., None, :]).sum(-1)
        # nothing comes in at a sequence's start
        dg = dg * (1 - _chunks(st.float()[..., None], d["nc"]))
    dg = _unchunk(dg, L)
    dbeta = _unchunk((du * w).sum(-1), L)
    beta = _unchunk(d["beta"], L)
    draw_ = dg * s["A"] / (1 + torch.exp(-d["raw"]))
    wide = lambda x, r, raw: _unit_grad(_unchunk(x, L).unflatten(2, (G, H // G)).sum(3), raw.float(), r).to(t)
    out = dict(dq=wide(dq * N ** -0.5, d["rq"], s["q"]), dk=wide(drow + dcol, d["rk"], s["k"]),
               dv=_unchunk(dw, L).to(t), ddt=draw_.to(t), dbeta=(dbeta * beta * (1 - beta)).to(t),
               dA=(dg * d["step"]).sum((0, 1)), ddt_bias=draw_.sum((0, 1)))
    if s["h0"] is not None:
        out["dinitial"] = D
    return out


def _unit_grad(d, x, r):
    """The gradient through x r, r = 1 / sqrt(sum x^2 + eps)."""
    xh = x * r
    return r * (d - xh * (xh * d).sum(-1, keepdim=True))


def _plain_delta_step(s):
    one = dict(s)
    for k in ("q", "k", "v", "dt", "beta"):
        one[k] = s[k][:, None]
    q, k, v, raw, step, g, beta, rq, rk = (x[:, 0] for x in _delta_terms(one))
    h = torch.exp(g)[..., None, None] * s["h0"]
    u = beta[..., None] * (v - (k[..., None] * h).sum(-2))
    h = h + k[..., None] * u[..., None, :]
    return dict(y=(q[..., None] * h).sum(-2).to(s["v"].dtype), state=h)


_PLAIN = dict(delta_forward=_plain_delta_forward, delta_backward=_plain_delta_backward, delta_step=_plain_delta_step,
              group_norm_forward=_plain_group_norm_forward, group_norm_backward=_plain_group_norm_backward,
              pack8=_plain_pack8, unpack8=_plain_unpack8)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"].endswith("pack8"):
        n = c["rows"] * c["D"]
        return dict(bytes=(e + 1) * n + 2 * c["rows"] * -(-c["D"] // _BLOCK), flops=4 * n)
    if c["op"].startswith("group_norm"):
        n = c["rows"] * c["D"]
        gated = c["gate"] in ("after", "first")
        par = 4 * (1 + c["bias"]) * (c["D"] // c["groups"] if c["shared"] else c["D"])
        stats = 4 * c["rows"] * c["groups"] * (1 if c["rms"] else 2)
        if c["op"] == "group_norm_forward":
            return dict(bytes=e * n * (3 if gated else 2) + par + stats, flops=(14 if gated else 8) * n)
        xe = 1 + 2 / _BLOCK if c["kept8"] else e
        # dy, x and the gate in; their gradients out
        return dict(bytes=n * (e * (3 if gated else 2) + xe * (2 if gated else 1)) + 2 * par + stats,
                    flops=(30 if gated else 15) * n)
    B, L, H, G, N, P = (c[k] for k in "BLHGNP")
    qk, v, ab, st = 2 * e * B * L * G * N, e * B * L * H * P, 2 * e * B * L * H, 4 * B * H * N * P
    sq = 4 * B * L if c["packed"] else 0
    one = B * L * H * N * P
    if c["op"] == "delta_step":
        return dict(bytes=qk + 2 * v + ab + 8 * H + 2 * st, flops=7 * one)
    if c["op"] == "delta_forward":
        return dict(bytes=qk + 2 * v + ab + 8 * H + st * (1 + c["state"]) + sq, flops=7 * one)
    return dict(bytes=2 * qk + 3 * v + 2 * ab + 16 * H + 3 * c["state"] * st + sq, flops=20 * one)


# ---------------------------------------------------------------- the definitions in 64 bits, token by token

def exact(case, seed):
    s = prepare(case, seed)
    double = lambda v: v.double() if torch.is_tensor(v) and v.is_floating_point() else v
    f = {k: double(v) for k, v in s.items() if k not in ("workspace", "y", "state_out", "out")}
    op = case["op"]
    if op == "pack8":
        return _exact_pack8(f, case)
    if op == "unpack8":
        return dict(x=_exact_values(f["q"], f["scale"]))
    if op.startswith("group_norm"):
        with torch.enable_grad():
            return _exact_group_norm(f, case)
    grads = op == "delta_backward"
    if grads and case["L"] > 5000:
        return None                                      # the tape of single tokens takes too long
    with torch.set_grad_enabled(grads):
        return _exact_delta_grad(f, case) if grads else _exact_delta(f, case)


def _exact_pack8(f, c):
    """The definition: the least bf16 that times 127 reaches the block's largest
    magnitude, and the nearest whole multiple of it, ties to even."""
    x, D = f["x"], c["D"]
    values, scales = torch.empty_like(x), []
    for a in range(0, D, _BLOCK):
        b = x[:, a:a + _BLOCK]
        most = b.abs().max(1).values
        mant, expo = torch.frexp(most / 127)
        sc = torch.ldexp(torch.ceil(mant * 256), expo - 8)  # 8 bits, upwards
        scales.append(sc)
        values[:, a:a + _BLOCK] = torch.where(sc[:, None] > 0, torch.round(b / sc.clamp(min=1e-300)[:, None]), 0.0)
    return dict(values=values.to(torch.int8), scale=torch.stack(scales, 1))


def _exact_values(q, scale):
    D = q.shape[-1]
    which = torch.arange(D, device=q.device) // _BLOCK
    return q.double() * scale.double()[:, which]


def _exact_group_norm(f, c):
    rows, groups, D = c["rows"], c["groups"], c["D"]
    back = c["op"] == "group_norm_backward"
    get = lambda v: None if v is None else _exact_values(*v) if isinstance(v, tuple) else v
    x, z, w, b = get(f["x"]), get(f["z"]), f["weight"], f["bias"]
    leaves = {}
    if back:
        x, w = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
        leaves = dict(dx=x, dweight=w)
        if z is not None:
            z = z.clone().requires_grad_(True)
            leaves["dz"] = z
        if b is not None:
            b = b.clone().requires_grad_(True)
            leaves["dbias"] = b
    xin = x * (z * torch.sigmoid(z)) if c["gate"] == "first" else x
    parts = xin.reshape(rows, groups, D // groups)
    mean = torch.zeros_like(parts[..., 0]) if c["rms"] else parts.mean(2)
    if back:
        # statistics of the values before they went into 8 bits: their own dependence on x
        # enters through sums over what is normalised here
        mean = torch.zeros_like(mean) if c["rms"] else f["mean"]
    var = ((parts - mean[..., None]) ** 2).mean(2)
    rstd = f["rstd"] if back else torch.rsqrt(var + _EPS)
    xh = (parts - mean[..., None]) * rstd[..., None]
    if back:
        xh = _NormValue.apply(xh, parts, rstd, bool(c["rms"]))
    tile = lambda v: v.repeat(groups) if c["shared"] else v
    y = xh.reshape(rows, D) * tile(w)
    if b is not None:
        y = y + tile(b)
    if c["gate"] == "after":
        y = y * (z * torch.sigmoid(z))
    if c["gate"] == "self":
        y = y * torch.sigmoid(y)
    if back:
        got = torch.autograd.grad((y * f["dy"]).sum(), list(leaves.values()))
        return dict(zip(leaves, got))
    out = dict(y=y, rstd=rstd)
    if not c["rms"]:
        out["mean"] = mean
    return out


class _NormValue(torch.autograd.Function):
    """The normalised values as they are, with the derivative of normalisation
    at them: rstd (I - 1 1^T / n - xh xh^T / n), without the ones for rms."""

    @staticmethod
    def forward(ctx, xh, parts, rstd, rms):
        ctx.save_for_backward(xh, rstd)
        ctx.rms = rms
        return xh.clone()

    @staticmethod
    def backward(ctx, g):
        xh, rstd = ctx.saved_tensors
        n = xh.shape[-1]
        d = g - xh * torch.einsum("rgi,rgi->rg", g, xh)[..., None] / n
        if not ctx.rms:
            d = d - g.sum(-1, keepdim=True) / n
        return None, d * rstd[..., None], None, None


def _ex_delta(f, c):
    """Outputs [B, L, H, P] and the last state, one token after the other:
    h <- a h; u = beta (v - k^T h); h <- h + k u^T; y = q^T h."""
    lift = (lambda v: v.unsqueeze(1)) if c["op"] == "delta_step" else (lambda v: v)
    q, k, v, dt, be = (lift(f[n]) for n in ("q", "k", "v", "dt", "beta"))
    B, L, H, P = v.shape
    N, rep = c["N"], H // c["G"]
    q = q / torch.sqrt((q ** 2).sum(-1, keepdim=True) + _QK_EPS) / math.sqrt(N)
    k = k / torch.sqrt((k ** 2).sum(-1, keepdim=True) + _QK_EPS)
    a = torch.exp(f["A"] * torch.logaddexp(dt + f["dt_bias"], torch.zeros_like(dt)))
    be = torch.sigmoid(be)
    q, k = q.repeat_interleave(rep, 2), k.repeat_interleave(rep, 2)
    if f["seq_idx"] is not None:
        new = torch.zeros((B, L, 1), device=v.device, dtype=torch.bool)
        new[:, 1:, 0] = f["seq_idx"][:, 1:] != f["seq_idx"][:, :-1]
        a = a.masked_fill(new, 0.0)
    h = f["h0"] if f["h0"] is not None else v.new_zeros((B, H, N, P))
    # one unbind each: a slice's gradient a token would be a whole tensor of zeros
    ys, rows = [], [x.unbind(1) for x in (q.unsqueeze(-2), k.unsqueeze(-2), v.unsqueeze(-2), a[..., None, None],
                                          be[..., None, None])]
    for qt, kt, vt, at, bt in zip(*rows):
        h = at * h
        u = bt * (vt - kt @ h)
        h = h + kt.transpose(-1, -2) * u
        ys.append(qt @ h)
    return torch.cat(ys, 2).transpose(1, 2), h


def _exact_delta(f, c):
    y, h = _ex_delta(f, c)
    if c["op"] == "delta_step":
        return dict(y=y[:, 0], state=h)
    return dict(y=y, final=h)


def _exact_delta_grad(f, c):
    names = dict(q="dq", k="dk", v="dv", dt="ddt", beta="dbeta", A="dA", dt_bias="ddt_bias")
    if f["h0"] is not None:
        names["h0"] = "dinitial"
    f = dict(f)
    for n in names:
        f[n] = f[n].clone().requires_grad_(True)
    y, h = _ex_delta(f, c)
    loss = (y * f["dy"]).sum()
    if f["dfinal"] is not None:
        loss = loss + (h * f["dfinal"]).sum()
    return dict(zip(names.values(), torch.autograd.grad(loss, [f[n] for n in names])))
