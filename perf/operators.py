"""Cases that measure the training and serving operators around the sketch layer:

  linear attention with a decay per head over a ragged batch of histories
  (forward, backward, one step of a stored state), the norms before and after
  a block with its gate and residual scale (forward, backward), and the global
  gradient norm with clipping.

``run`` computes each in its plain form (elementary torch operations in 32
bits, 64 where sums and powers need them) or, with ``own`` set, by the
library's calls.  ``exact`` is the definition in 64 bits, written apart.
"""

import math

import torch

own = False

F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16
TYPES = {"bf16": BF16, "fp32": F32}


# ---------------------------------------------------------------- cases


def listed():
    return [
        # one user's new session appended to a stored state: the smallest prompt
        dict(name="attn fwd 1x17", op="attn_fwd", dtype="bf16", users=1, longest=17, ragged=False,
             heads=2, dk=64, dv=64, state=True),
        # the headline history batch: 16 users x 100K behaviours, width 128 in two heads
        dict(name="attn fwd 16x100K", op="attn_fwd", dtype="bf16", users=16, longest=100000,
             ragged=False, heads=2, dk=64, dv=64, state=False),
        # ragged histories at the ranking model's width (8 heads x 128)
        dict(name="attn fwd ragged 48x4K w1024", op="attn_fwd", dtype="bf16", users=48,
             longest=4099, ragged=True, heads=8, dk=128, dv=128, state=True),
        # a small training batch, odd lengths, some users empty
        dict(name="attn bwd ragged 5x300", op="attn_bwd", dtype="bf16", users=5, longest=301,
             ragged=True, heads=2, dk=128, dv=64, state=True),
        # a training batch of 10K-row histories at the ranking width
        dict(name="attn bwd 16x10K w1024", op="attn_bwd", dtype="bf16", users=16, longest=10000,
             ragged=False, heads=8, dk=128, dv=128, state=False),
        # one new behaviour for one user
        dict(name="step 1 fp32", op="step", dtype="fp32", users=1, heads=2, dk=64, dv=64),
        # one new behaviour for each user of a serving batch
        dict(name="step 1000 w1024", op="step", dtype="bf16", users=1000, heads=8, dk=128, dv=128),
        # the norms around a block over the sketch rows of the headline batch, fp32
        dict(name="norm fwd 2048x128 fp32", op="norm_fwd", dtype="fp32", res="fp32", rows=2048,
             d=128, kind="layer", gate="silu", post=True, scale=True),
        # the norms around a block over every history row, at the ranking width
        dict(name="norm fwd 200Kx1024", op="norm_fwd", dtype="bf16", res="bf16", rows=200000,
             d=1024, kind="rms", gate="silu", post=True, scale=True),
        # its gradient over history rows of width 128, the residual stream in 32 bits
        dict(name="norm bwd 400Kx128", op="norm_bwd", dtype="bf16", res="fp32", rows=400001,
             d=128, kind="layer", gate="sigmoid", post=True, scale=True),
        # the gradients of a two-layer refinement stack
        dict(name="clip stack", op="clip", dtype="fp32", layers=2, d=128, h=512, extra=128),
        # the gradients of a 24-layer model of width 1024
        dict(name="clip 24 layers w1024", op="clip", dtype="bf16", layers=24, d=1024, h=4096,
             extra=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "step", "norm_fwd", "norm_bwd",
                     "clip"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("attn_fwd", "attn_bwd"):
        heads, dk, dv = rng.randint(1, 8), rng.choice([64, 128]), rng.choice([64, 128])
        rows = _log(rng, 1, 1500 if dtype == "fp32" else 20000)
        most = (200000 if dtype == "fp32" else 1000000) // (rows * heads)
        return dict(op=op, dtype=dtype, users=_log(rng, 1, max(1, min(64, most))), longest=rows,
                    ragged=rng.random() < 0.7, heads=heads, dk=dk, dv=dv,
                    state=rng.random() < 0.5)
    if op == "step":
        return dict(op=op, dtype=dtype, users=_log(rng, 1, 900), heads=rng.randint(1, 8),
                    dk=rng.choice([64, 96, 128]), dv=rng.choice([64, 100, 128]))
    if op in ("norm_fwd", "norm_bwd"):
        d = _log(rng, 8, 8192)
        if rng.random() < 0.5:
            d = (d + 63) // 64 * 64
        return dict(op=op, dtype=dtype, res=rng.choice([dtype, "fp32"]),
                    rows=_log(rng, 1, max(2, min(200000, 50000000 // d))), d=d,
                    kind=rng.choice(["layer", "rms"]),
                    gate=rng.choice(["none", "identity", "sigmoid", "silu"]),
                    post=rng.random() < 0.7, scale=rng.random() < 0.5)
    return dict(op=op, dtype=dtype, layers=rng.randint(1, 12), d=_log(rng, 64, 1024),
                h=_log(rng, 64, 4096), extra=_log(rng, 1, 5000))


# ---------------------------------------------------------------- inputs


def _lengths(case):
    """Rows per user, from the case alone: ragged batches run from empty users to the longest."""
    n, b = case["longest"], case["users"]
    if not case["ragged"]:
        return [n] * b
    return [n if i == 0 else (n * ((i * 0.6180339887) % 1.0) ** 2).__floor__() for i in range(b)]


def _heads_decay(h):
    """log(1 - 2^-(5 + 7 i / (h - 1))): horizons from 32 to 4096 rows over the heads."""
    i = torch.arange(h, dtype=F64)
    return torch.log1p(-torch.exp2(-(5 + 7 * i / max(h - 1, 1)))).to(F32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, dtype=F32, mul=1.0, add=0.0):
        return torch.randn(*shape, generator=gen, device=dev).mul_(mul).add_(add).to(dtype)

    s, op, t = dict(case), case["op"], TYPES[case["dtype"]]
    if op in ("attn_fwd", "attn_bwd"):
        lens = _lengths(case)
        n, b, h, dk, dv = sum(lens), len(lens), case["heads"], case["dk"], case["dv"]
        s.update(lens=lens, offsets=torch.tensor([0] + lens, device=dev).cumsum(0),
                 q=normal(n, h, dk, dtype=t), k=normal(n, h, dk, dtype=t),
                 v=normal(n, h, dv, dtype=t), g=_heads_decay(h).to(dev), mul=dk ** -0.5,
                 s0=normal(b, h, dk, dv, mul=4.0) if case["state"] else None)
        if op == "attn_bwd":
            s.update(do=normal(n, h, dv, dtype=t),
                     ds=normal(b, h, dk, dv) if case["state"] else None)
    elif op == "step":
        b, h, dk, dv = case["users"], case["heads"], case["dk"], case["dv"]
        s.update(q=normal(b, h, dk, dtype=t), k=normal(b, h, dk, dtype=t),
                 v=normal(b, h, dv, dtype=t), g=_heads_decay(h).to(dev), mul=dk ** -0.5,
                 s0=normal(b, h, dk, dv, mul=4.0))
    elif op in ("norm_fwd", "norm_bwd"):
        n, d, tr = case["rows"], case["d"], TYPES[case["res"]]
        s.update(x=normal(n, d, dtype=tr, mul=2.0, add=0.3), y=normal(n, d, dtype=t, add=0.1),
                 gate_in=normal(n, d, dtype=t) if case["gate"] != "none" else None,
                 g1=normal(d, mul=0.2, add=1.0) if case["post"] else None,
                 b1=normal(d, mul=0.1) if case["post"] and case["kind"] == "layer" else None,
                 rs=normal(d, mul=0.1, add=0.5) if case["scale"] else None,
                 g2=normal(d, mul=0.2, add=1.0),
                 b2=normal(d, mul=0.1) if case["kind"] == "layer" else None)
        if op == "norm_bwd":  # x is then the forward's residual output
            s.update(dr=normal(n, d, dtype=tr), du=normal(n, d, dtype=t))
    else:
        d, h = case["d"], case["h"]
        shapes = [(d, d), (d, d), (d, h), (d, h), (h, d), (d,), (d,), (d,), (d,)] * case["layers"]
        shapes.append((case["extra"], d))
        sizes = [math.prod(x) for x in shapes]
        flat, out = normal(sum(sizes), dtype=t, mul=0.01), torch.empty(sum(sizes), dtype=t,
                                                                       device=dev)
        s.update(flat_out=out, max_norm=1.0,
                 grads=[x.view(y) for x, y in zip(flat.split(sizes), shapes)],
                 outs=[x.view(y) for x, y in zip(out.split(sizes), shapes)])
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sketch_attention_compression_b200 as sa
    op = s["op"]
    if op == "attn_fwd":
        o, state, _ = sa.linear_attention_forward(s["q"], s["k"], s["v"], s["g"], s["offsets"],
                                                  s["mul"], initial_state=s["s0"],
                                                  max_rows=max(s["lens"]))
        return {"o": o, "state": state}
    if op == "attn_bwd":
        grads, _ = sa.linear_attention_backward(s["q"], s["k"], s["v"], s["g"], s["offsets"],
                                                s["mul"], s["do"], initial_state=s["s0"],
                                                d_final_state=s["ds"], max_rows=max(s["lens"]))
        return grads
    if op == "step":
        o = sa.linear_attention_step(s["s0"], s["q"], s["k"], s["v"], s["g"], s["mul"])
        return {"o": o, "state": s["s0"]}
    if op == "clip":
        norm = sa.clip_grad_norm(s["grads"], s["max_norm"], out=s["outs"])
        return {"norm": norm, "grads": s["flat_out"]}
    params = dict(gate=s["gate_in"], post_gain=s["g1"], post_bias=s["b1"], res_scale=s["rs"],
                  pre_gain=s["g2"], pre_bias=s["b2"], kind=s["kind"],
                  gate_kind=s["gate"] if s["gate"] != "none" else "identity")
    if op == "norm_fwd":
        r, u = sa.block_norm_forward(s["x"], s["y"], **params)
        return {"residual": r, "normed": u}
    return sa.block_norm_backward(s["x"], s["y"], s["dr"], s["du"], **params)


EPS = 1e-5
CHUNK = 128


class _Chunks:
    """The ragged rows in chunks of CHUNK rows of one user each, zeros behind a user's end."""

    def __init__(self, lens, offsets, g):
        n = offsets[1:] - offsets[:-1]
        per = (n + CHUNK - 1) // CHUNK
        count = sum((x + CHUNK - 1) // CHUNK for x in lens)
        self.rows, self.users, self.g = sum(lens), len(lens), g.double()
        self.user = torch.repeat_interleave(torch.arange(len(lens), device=g.device), per,
                                            output_size=count)
        first = (per.cumsum(0) - per)[self.user]
        r = torch.arange(CHUNK, device=g.device)
        self.pos = (torch.arange(count, device=g.device) - first)[:, None] * CHUNK + r
        self.length = n[self.user][:, None]
        self.valid = self.pos < self.length
        self.index = torch.where(self.valid, self.pos + offsets[self.user][:, None], 0)

    def take(self, x):
        return x[self.index].float() * self.valid[..., None, None]

    def put(self, x, dtype):
        out = torch.empty((self.rows,) + x.shape[2:], dtype=dtype, device=x.device)
        out[self.index[self.valid]] = x[self.valid].to(dtype)
        return out

    def power(self, e):
        """decay ** e per head, (heads, *e.shape); 0 where e is negative."""
        e = e.double()
        return torch.where(e < 0, 0.0, (self.g.view(-1, *([1] * e.dim())) * e.clamp(min=0)).exp()).float()

    def mix(self, a, b, c, ends, reverse):
        """sum over j <= i (or j >= i) of decay^|i-j| (a_i . b_j) c_j, plus the
        decayed share of each user's end state `ends` (users, heads, da, dc)."""
        r = torch.arange(CHUNK, device=a.device)
        dist = r[:, None] - r[None, :]
        w = self.power(-dist if reverse else dist)
        p = torch.einsum("nihd,njhd->nhij", a, b) * w
        out = torch.einsum("nhij,njhd->nihd", p, c)
        wb = self.power(r if reverse else CHUNK - 1 - r)
        local = torch.einsum("hj,njhd,njhe->hnde", wb, b, c)
        m = torch.arange(self.user.numel(), device=a.device)
        gap = (m[None, :] - m[:, None] if reverse else m[:, None] - m[None, :]) - 1
        gap = torch.where(self.user[:, None] == self.user[None, :], gap, -1)
        carry = torch.matmul(self.power(torch.where(gap < 0, -1, gap * CHUNK)),
                             local.flatten(2)).view_as(local)
        wa = self.power(CHUNK - r if reverse else r + 1)
        out += torch.einsum("hi,nihd,hnde->nihe", wa, a, carry)
        if ends is not None:
            we = self.power(self.length - 1 - self.pos if reverse else self.pos + 1)
            out += torch.einsum("hni,nihd,nhde->nihe", we, a, ends[self.user])
        return out

    def sums(self, b, c, ends, reverse):
        """The state behind a user's last row (or the gradient before its first)."""
        w = self.power(torch.where(self.valid, self.pos + 1 if reverse else self.length - 1 - self.pos, -1))
        local = torch.einsum("hnj,njhd,njhe->nhde", w, b, c)
        out = torch.zeros((self.users,) + local.shape[1:], device=b.device)
        out.index_add_(0, self.user, local)
        return out

    def whole(self, n):
        return self.power(n).t()[:, :, None, None]


def _norm(x, kind, gain, bias):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    rstd = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    y = x * rstd * gain
    return y if bias is None else y + bias


def _norm_grad(x, kind, gain, dy):
    """(dx, d gain, d bias) of _norm."""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    rstd = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    hat, dh = x * rstd, dy * gain
    dx = dh - hat * (dh * hat).mean(-1, keepdim=True)
    if kind == "layer":
        dx = dx - dh.mean(-1, keepdim=True)
    return (dx * rstd, (dy * hat).sum(0, dtype=F64).float(), dy.sum(0, dtype=F64).float())


def _gate(z, kind):
    if kind == "identity":
        return z, torch.ones_like(z)
    sig = 1 / (1 + (-z).exp())
    if kind == "sigmoid":
        return sig, sig * (1 - sig)
    return z * sig, sig * (1 + z * (1 - sig))


def _run_plain(s):
    op = s["op"]
    if op in ("attn_fwd", "attn_bwd"):
        c = _Chunks(s["lens"], s["offsets"], s["g"])
        q, k, v, s0, mul = c.take(s["q"]), c.take(s["k"]), c.take(s["v"]), s["s0"], s["mul"]
        n = s["offsets"][1:] - s["offsets"][:-1]
        if op == "attn_fwd":
            o = c.mix(q, k, v, s0, False) * mul
            state = c.sums(k, v, s0, False)
            if s0 is not None:
                state = state + c.whole(n) * s0
            return {"o": c.put(o, s["q"].dtype), "state": state}
        do, ds, t = c.take(s["do"]), s["ds"], s["q"].dtype
        dst = None if ds is None else ds.transpose(2, 3) / mul
        dq = c.mix(do, v, k, None if s0 is None else s0.transpose(2, 3), False) * mul
        dk = c.mix(v, do, q, dst, True) * mul
        dv = c.mix(k, q, do, None if ds is None else ds / mul, True) * mul
        grads = {"dq": c.put(dq, t), "dk": c.put(dk, t), "dv": c.put(dv, t)}
        if s0 is not None:
            grads["d_initial_state"] = c.sums(q, do, None, True) * mul + (
                0.0 if ds is None else c.whole(n) * ds)
        return grads
    if op == "step":
        k, v, q = s["k"].float(), s["v"].float(), s["q"].float()
        s["s0"].mul_(s["g"].exp()[:, None, None]).add_(k[..., :, None] * v[..., None, :])
        o = (q[..., :, None] * s["s0"]).sum(2) * s["mul"]
        return {"o": o.to(s["q"].dtype), "state": s["s0"]}
    if op == "clip":
        norm = torch.stack([x.double().square().sum() for x in s["grads"]]).sum().sqrt()
        mul = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
        [o.copy_(x.float() * mul) for o, x in zip(s["outs"], s["grads"])]
        return {"norm": norm.float(), "grads": s["flat_out"]}
    x, y, t, tr = s["x"].float(), s["y"].float(), s["y"].dtype, s["x"].dtype
    post = y if s["g1"] is None else _norm(y, s["kind"], s["g1"], s["b1"])
    act, slope = (1.0, None) if s["gate_in"] is None else _gate(s["gate_in"].float(), s["gate"])
    rs = 1.0 if s["rs"] is None else s["rs"]
    if op == "norm_fwd":
        r = x + rs * act * post
        return {"residual": r.to(tr), "normed": _norm(r, s["kind"], s["g2"], s["b2"]).to(t)}
    dx, dg2, db2 = _norm_grad(x, s["kind"], s["g2"], s["du"].float())
    dx = dx + s["dr"].float()
    dpost, grads = dx * rs * act, {"d_residual": dx.to(tr), "d_pre_gain": dg2}
    if s["gate_in"] is not None:
        grads["d_gate"] = (dx * rs * post * slope).to(t)
    if s["rs"] is not None:
        grads["d_res_scale"] = (dx * act * post).sum(0, dtype=F64).float()
    if s["b2"] is not None:
        grads["d_pre_bias"] = db2
    if s["g1"] is not None:
        dpost, grads["d_post_gain"], db1 = _norm_grad(y, s["kind"], s["g1"], dpost)
        if s["b1"] is not None:
            grads["d_post_bias"] = db1
    grads["d_block"] = dpost.to(t)
    return grads


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("attn_fwd", "attn_bwd", "step"):
        h, dk, dv, b = case["heads"], case["dk"], case["dv"], case["users"]
        n = b if op == "step" else sum(_lengths(case))
        states = 4 * b * h * dk * dv
        if op == "step":
            return {"bytes": n * h * 2 * (dk + dv) * e + 2 * states, "flops": 6 * n * h * dk * dv}
        # the recurrence: one rank-1 update and one product with the state per output
        if op == "attn_fwd":
            return {"bytes": n * h * 2 * (dk + dv) * e + states * (2 if case["state"] else 1),
                    "flops": 4 * n * h * dk * dv}
        return {"bytes": n * h * (4 * dk + 3 * dv) * e + states * (3 if case["state"] else 0),
                "flops": 10 * n * h * dk * dv}
    if op == "clip":
        d, h = case["d"], case["h"]
        n = case["layers"] * (2 * d * d + 3 * d * h + 4 * d) + case["extra"] * d
        return {"bytes": 2 * n * e, "flops": 3 * n}
    n, d, er = case["rows"], case["d"], 2 if case["res"] == "bf16" else 4
    gates = 0 if case["gate"] == "none" else 1
    params = 4 * d * (1 + case["post"]) * (1 + (case["kind"] == "layer")) + 4 * d * case["scale"]
    if op == "norm_fwd":
        return {"bytes": n * d * (2 * er + (2 + gates) * e) + params, "flops": 16 * n * d}
    return {"bytes": n * d * (3 * er + (3 + 2 * gates) * e) + 2 * params, "flops": 40 * n * d}


# ---------------------------------------------------------------- the definition in 64 bits


def _exact_attention(q, k, v, g, lens, mul, s0):
    """S_t = e^g S_{t-1} + k_t v_t^T, o_t = mul q_t S_t, user by user in blocks of rows."""
    outs, states, at, block = [], [], 0, 256
    for u, n in enumerate(lens):
        s = s0[u] if s0 is not None else torch.zeros(q.shape[1], q.shape[2], v.shape[2], dtype=F64,
                                                     device=q.device)
        for lo in range(at, at + n, block):
            hi = min(lo + block, at + n)
            m = hi - lo
            i = torch.arange(m, dtype=F64, device=q.device)
            qb, kb, vb = (x[lo:hi].transpose(0, 1) for x in (q, k, v))
            gap = (i[:, None] - i[None, :]).clamp(min=0)
            w = torch.tril(torch.exp(g[:, None, None] * gap))
            o = (qb @ kb.transpose(1, 2) * w) @ vb
            o = o + torch.exp(g[:, None] * (i + 1))[..., None] * (qb @ s)
            outs.append(o.transpose(0, 1) * mul)
            s = torch.exp(g * m)[:, None, None] * s + \
                (kb * torch.exp(g[:, None] * (m - 1 - i))[..., None]).transpose(1, 2) @ vb
        states.append(s)
        at += n
    o = torch.cat(outs) if outs else q.new_zeros((0, q.shape[1], v.shape[2]))
    return o, torch.stack(states)


def _exact_block(s):
    """The block's norms, gate and residual, layer or root-mean-square form."""
    def norm(x, gain, bias):
        mean = x.mean(-1, keepdim=True) if s["kind"] == "layer" else 0.0
        var = ((x - mean) ** 2).mean(-1, keepdim=True)
        y = gain * (x - mean) / torch.sqrt(var + EPS)
        return y if bias is None else y + bias

    add = s["y"] if s["g1"] is None else norm(s["y"], s["g1"], s["b1"])
    if s["gate_in"] is not None:
        z = s["gate_in"]
        add = add * {"identity": z, "sigmoid": torch.sigmoid(z),
                     "silu": z * torch.sigmoid(z)}[s["gate"]]
    return (add if s["rs"] is None else add * s["rs"]), norm


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "clip":
        total = math.fsum(float(x.double().square().sum()) for x in s["grads"])
        mul = min(1.0, s["max_norm"] / (math.sqrt(total) + 1e-6))
        out = torch.cat([x.double().reshape(-1) * mul for x in s["grads"]])
        return {"norm": torch.tensor(math.sqrt(total), dtype=F64), "grads": out}
    w = {key: (x.double() if torch.is_tensor(x) and x.is_floating_point() else x)
         for key, x in s.items()}
    if op == "step":
        state = torch.exp(w["g"])[None, :, None, None] * w["s0"] + torch.einsum(
            "bhd,bhe->bhde", w["k"], w["v"])
        return {"o": torch.einsum("bhd,bhde->bhe", w["q"], state) * s["mul"], "state": state}
    if op in ("attn_fwd", "attn_bwd"):
        names = [x for x in ("q", "k", "v", "s0") if w[x] is not None]
        if op == "attn_bwd":
            [w[x].requires_grad_() for x in names]
        o, state = _exact_attention(w["q"], w["k"], w["v"], w["g"], s["lens"], s["mul"], w["s0"])
        if op == "attn_fwd":
            return {"o": o, "state": state}
        loss = (o * w["do"]).sum()
        if w["ds"] is not None:
            loss = loss + (state * w["ds"]).sum()
        got = torch.autograd.grad(loss, [w[x] for x in names], allow_unused=True)
        name = {"q": "dq", "k": "dk", "v": "dv", "s0": "d_initial_state"}
        return {name[x]: y if y is not None else torch.zeros_like(w[x]) for x, y in zip(names, got)}
    if op == "norm_fwd":
        add, norm = _exact_block(w)
        r = w["x"] + add
        return {"residual": r, "normed": norm(r, w["g2"], w["b2"])}
    # the gradient is taken at the given residual output x: r = x + (add - its own value)
    name = {"x": "d_residual", "y": "d_block", "gate_in": "d_gate", "g1": "d_post_gain",
            "b1": "d_post_bias", "rs": "d_res_scale", "g2": "d_pre_gain", "b2": "d_pre_bias"}
    names = [x for x in name if w[x] is not None]
    [w[x].requires_grad_() for x in names]
    add, norm = _exact_block(w)
    r = w["x"] + (add - add.detach())
    loss = (r * w["dr"]).sum() + (norm(r, w["g2"], w["b2"]) * w["du"]).sum()
    got = torch.autograd.grad(loss, [w[x] for x in names])
    return {name[x]: y for x, y in zip(names, got)}
