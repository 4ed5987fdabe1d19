"""What the selective state space block is measured on: its scan, its short convolution, and the norm of its stream.

Eight calls of three operators, each on cases spread over its real range:
  scan_fwd    the selective scan over a prompt (outputs and the last state)
  scan_train  forward and backward pass of a training step
  scan_step   its recurrent form for one token per sequence, states in a pool
  conv_fwd    the short causal convolution over time, one filter per channel (outputs and the last inputs)
  conv_bwd    its backward pass
  conv_step   its form for one token per sequence, the last inputs in a pool
  ln_fwd      a branch added to the residual stream and the stream's rows normalised
  ln_bwd      its backward pass, with the sums for the weight and the bias
``run`` computes them in plain torch operations, or, where ``own`` is true, by the package's entry points;
``exact`` in 64 bits from the definitions.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ---- cases -------------------------------------------------------------------------------------------------


def _scan(name, op, B, T, G, per, N, dtype, gate=True, start=False, ragged=False, softplus=True):
    return dict(name=name, op=op, B=B, T=T, G=G, per=per, N=N, dtype=dtype, gate=gate, start=start, ragged=ragged,
                softplus=softplus)


def _conv(name, op, B, T, D, W, dtype, act="silu", start=False, ragged=False):
    return dict(name=name, op=op, B=B, T=T, D=D, W=W, dtype=dtype, act=act, start=start, ragged=ragged)


def _ln(name, op, N, S, C, x, r, y, rms=False, add=True, ragged=False):
    return dict(name=name, op=op, N=N, S=S, C=C, x=x, r=r, y=y, rms=rms, add=add, ragged=ragged)


def listed():
    return [
        # a short prompt of one user, state carried on: nothing but latency
        _scan("scan_short_prompt", "scan_fwd", 1, 37, 1, 512, 16, "bf16", start=True),
        # a prefill batch: many sequences and channels fill the card
        _scan("scan_batch", "scan_fwd", 8, 4096, 1, 2048, 16, "bf16"),
        # one very long document in a narrow model: parallel over time or not at all
        _scan("scan_long", "scan_fwd", 1, 131072, 1, 1024, 16, "bf16", start=True),
        # a training step's forward and backward pass
        _scan("scan_train_batch", "scan_train", 4, 4096, 1, 2048, 16, "bf16"),
        # a padded batch in fp32, groups of odd widths, a state size that is no power of two, states in and out
        _scan("scan_train_ragged_f32", "scan_train", 3, 517, 3, 100, 9, "f32", gate=False, start=True, ragged=True),
        # one token of each of many users served at once, their states in a pool
        dict(name="scan_step_serving", op="scan_step", B=256, G=1, per=4096, N=16, dtype="bf16", gate=True, pool=320,
             softplus=True),
        # the convolution in front of the scan, for a prefill or training batch
        _conv("conv_batch", "conv_fwd", 8, 4096, 4096, 4, "bf16"),
        # its backward pass over a padded batch of odd lengths in fp32, the last inputs carried in and out
        _conv("conv_ragged_bwd_f32", "conv_bwd", 5, 2011, 1000, 3, "f32", start=True, ragged=True),
        # one token of one user
        dict(name="conv_step_single", op="conv_step", B=1, D=2048, W=4, dtype="bf16", act="silu", pool=4),
        # a block's entry in training: a bf16 branch onto an fp32 stream, normalised for the next projection
        _ln("ln_stream", "ln_fwd", 8, 4096, 2048, "bf16", "f32", "bf16"),
        # its backward pass
        _ln("ln_stream_bwd", "ln_bwd", 4, 4096, 2048, "bf16", "f32", "bf16"),
        # the same of the tokens of a few users, without the mean: latency again
        _ln("ln_rms_tokens", "ln_fwd", 8, 1, 4096, "bf16", "bf16", "bf16", rms=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_train", "scan_train", "scan_step", "conv_fwd", "conv_bwd", "conv_step",
                     "ln_fwd", "ln_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("scan"):
        N = rng.choice([16, 16, 16, 8, 32, 64, rng.randint(1, 64)])
        G = rng.choice([1, 1, 1, 2, 3, 8])
        D = _log_int(rng, 1, 4096)
        if rng.random() < 0.5:
            D = max(64, D // 64 * 64)
        per = max(1, D // G)
        c = dict(op=op, G=G, per=per, N=N, dtype=dtype, gate=rng.random() < 0.7, softplus=rng.random() < 0.85)
        if op == "scan_step":
            B = min(_log_int(rng, 1, 512), max(1, 16_777_216 // (G * per * N)))
            return dict(c, B=B, pool=B + rng.randint(0, B))
        most = (2_000_000_000 if op == "scan_fwd" else 500_000_000) // (1 if dtype == "bf16" else 4)
        B = _log_int(rng, 1, 16)
        T = _log_int(rng, 1, 131072)
        T = max(1, min(T, most // (B * G * per * N)))
        return dict(c, B=B, T=T, start=rng.random() < 0.5, ragged=rng.random() < 0.4)
    if op.startswith("conv"):
        D = _log_int(rng, 1, 8192)
        if rng.random() < 0.6:
            D = max(8, D // 8 * 8)
        W, act = rng.choice([4, 4, 4, 2, 3, 5, 8]), rng.choice(["silu", "silu", "none"])
        B = _log_int(rng, 1, 512 if op == "conv_step" else 16)
        if op == "conv_step":
            return dict(op=op, B=B, D=D, W=W, dtype=dtype, act=act, pool=B + rng.randint(0, B))
        most = 134_217_728 if op == "conv_fwd" else 33_554_432
        T = max(1, min(_log_int(rng, 1, 131072), most // (B * D)))
        return dict(op=op, B=B, T=T, D=D, W=W, dtype=dtype, act=act, start=rng.random() < 0.5, ragged=rng.random() < 0.4)
    most = 67_108_864 if op == "ln_fwd" else 33_554_432
    C = _log_int(rng, 1, 16384)
    if rng.random() < 0.6:
        C = max(8, C // 8 * 8)
    rows = max(1, min(_log_int(rng, 1, 65536), most // C))
    N = rng.randint(1, min(8, rows))
    r = rng.choice([dtype, "f32"])
    return dict(op=op, N=N, S=rows // N, C=C, x=dtype, r=r, y=rng.choice([dtype, "bf16"]), rms=rng.random() < 0.5,
                add=rng.random() < 0.7, ragged=rows // N > 1 and rng.random() < 0.3)


# ---- inputs ------------------------------------------------------------------------------------------------


def _normal(gen, *shape, dtype=torch.float32, mean=0.0, std=1.0):
    x = torch.randn(*shape, device="cuda", generator=gen)
    return x.mul_(std).add_(mean).to(dtype)


def _lengths(gen, n, most, ragged):
    """Lengths of a padded batch: one full row, one empty one where there are three, the rest anywhere."""
    if not ragged:
        return None
    lengths = torch.randint(1, most + 1, (n,), device="cuda", generator=gen, dtype=torch.int32)
    lengths[0] = most
    if n > 2:
        lengths[n // 2] = 0
    return lengths


def _spoil(x, lengths):
    """Behind a row's length a padded batch holds whatever was there."""
    if lengths is not None:
        behind = torch.arange(x.shape[1], device=x.device)[None] >= lengths[:, None]
        x[behind] = float("nan")
    return x


def _slots(gen, B, pool):
    slots = torch.randperm(pool, device="cuda", generator=gen)[:B].to(torch.int32)
    if B > 4:
        slots[B // 2] = -1  # a request that has ended
    return slots


def _prepare_scan(c, gen, dtype):
    """Steps of 0.001 to 0.1 and decay rates around 1 .. N, as such a layer is set up and stays close to."""
    B, G, N = c["B"], c["G"], c["N"]
    D = G * c["per"]
    rates = torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(_normal(gen, D, N, std=0.2))
    step = torch.exp(torch.rand(D, device="cuda", generator=gen) * math.log(100.0) + math.log(0.001))
    st = dict(a=-rates, skip=_normal(gen, D, mean=1.0, std=0.2), softplus=c["softplus"])
    lead = (B,) if c["op"] == "scan_step" else (B, c["T"])
    lengths = None if c["op"] == "scan_step" else _lengths(gen, B, c["T"], c["ragged"])
    rows = lambda *s: _spoil(_normal(gen, *lead, *s, dtype=dtype), lengths)
    st.update(x=rows(D), b=rows(G, N), c=rows(G, N), gate=rows(D) if c["gate"] else None)
    if c["softplus"]:
        st.update(dt=rows(D), dt_bias=torch.log(torch.expm1(step)))
    else:
        st.update(dt=_spoil((step * torch.exp(_normal(gen, *lead, D, std=0.5))).to(dtype), lengths), dt_bias=None)
    if c["op"] == "scan_step":
        state = _normal(gen, c["pool"], D, N)
        st.update(state=state, after=state.clone(), slots=_slots(gen, B, c["pool"]))
        return st
    st.update(lengths=lengths, h0=_normal(gen, B, D, N) if c["start"] else None)
    if c["op"] == "scan_train":
        st.update(dy=rows(D), dh=_normal(gen, B, D, N) if c["start"] else None)
    return st


def _prepare_conv(c, gen, dtype):
    B, D, W = c["B"], c["D"], c["W"]
    st = dict(weight=_normal(gen, D, W, std=W ** -0.5), bias=_normal(gen, D, std=0.2), act=c["act"])
    if c["op"] == "conv_step":
        state = _normal(gen, c["pool"], W - 1, D, dtype=dtype)
        st.update(x=_normal(gen, B, D, dtype=dtype), state=state, after=state.clone(), slots=_slots(gen, B, c["pool"]))
        return st
    lengths = _lengths(gen, B, c["T"], c["ragged"])
    before = lambda: _normal(gen, B, W - 1, D, dtype=dtype) if c["start"] else None
    st.update(x=_spoil(_normal(gen, B, c["T"], D, dtype=dtype), lengths), lengths=lengths, state=before())
    if c["op"] == "conv_bwd":
        st.update(dy=_spoil(_normal(gen, B, c["T"], D, dtype=dtype), lengths), dlast=before())
    return st


def _prepare_ln(c, gen):
    N, S, C = c["N"], c["S"], c["C"]
    lengths = _lengths(gen, N, S, c["ragged"])
    rows = lambda t, **k: _spoil(_normal(gen, N, S, C, dtype=DTYPES[t], **k), lengths)
    st = dict(weight=_normal(gen, C, mean=1.0, std=0.2), bias=_normal(gen, C, std=0.2), lengths=lengths, rms=c["rms"],
              out=DTYPES[c["y"]])
    if c["op"] == "ln_fwd":
        st.update(x=rows(c["x"]), residual=rows(c["r"], mean=0.3, std=2.0) if c["add"] else None)
        return st
    r = rows(c["r"], mean=0.3, std=2.0)
    st.update(r=r, stats=_row_stats(r.double(), c["rms"]).float(), dy=rows(c["y"]), dr=rows(c["r"]) if c["add"] else None,
              branch=DTYPES[c["x"]])
    if lengths is not None:
        behind = torch.arange(S, device="cuda")[None] >= lengths[:, None]
        st["stats"][behind] = torch.tensor([0.0, EPS ** -0.5], device="cuda")
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op.startswith("ln"):
        st = _prepare_ln(case, gen)
    else:
        st = (_prepare_scan if op.startswith("scan") else _prepare_conv)(case, gen, DTYPES[case["dtype"]])
    return dict(st, op=op)


# ---- plain forms -------------------------------------------------------------------------------------------


def _valid(n, T, lengths, device):
    t = torch.arange(T, device=device)
    return torch.ones(n, T, dtype=torch.bool, device=device) if lengths is None else t[None] < lengths[:, None]


def _clean(x, valid):
    """fp32 with zeros behind the lengths."""
    return torch.where(valid.reshape(valid.shape + (1,) * (x.dim() - 2)), x.float(), 0.0)


def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(v.clamp(max=20.0))))


def _silu(v):
    return v * torch.sigmoid(v)


def _silu_slope(v):
    s = torch.sigmoid(v)
    return s * (1 + v * (1 - s))


def _chunk(T):
    """Steps taken one after another; the chunks of a sequence go side by side."""
    return 1 << max(0, math.ceil(math.log2(max(1.0, math.sqrt(T)))))


def _chunks(x, K):
    """[B, T, ...] -> [B, n, K, ...], zeros behind the end."""
    B, T = x.shape[:2]
    n = -(-T // K)
    pad = x.new_zeros(B, n * K - T, *x.shape[2:])
    return torch.cat([x, pad], 1).reshape(B, n, K, *x.shape[2:])


def _joined(local, decay, first, reverse=False):
    """The state before each chunk, from what each adds (local) and keeps (decay) of it; and the one after the last."""
    before, n = torch.empty_like(local), local.shape[1]
    h = torch.zeros_like(local[:, 0]) if first is None else first
    for i in (reversed(range(n)) if reverse else range(n)):
        before[:, i] = h
        h = decay[:, i] * h + local[:, i]
    return before, h


class _Scan:
    """A scan's operands in fp32, [B, n, K, ...]."""

    def __init__(self, st):
        x = st["x"]
        self.B, self.T, self.D = x.shape
        self.G, self.N = st["b"].shape[2:]
        self.valid = _valid(self.B, self.T, st["lengths"], x.device)
        self.K = _chunk(self.T)
        self.a = st["a"]
        self.x = _chunks(_clean(x, self.valid), self.K)
        raw = _clean(st["dt"], self.valid)
        raw = raw if st["dt_bias"] is None else raw + st["dt_bias"]
        self.raw = raw
        dt = _softplus(raw) if st["softplus"] else raw
        self.dt = _chunks(torch.where(self.valid[..., None], dt, 0.0), self.K)
        self.b, self.c = (_chunks(_clean(st[n], self.valid), self.K) for n in "bc")
        self.kept = torch.exp(self.a * self.dt.double().sum(2)[..., None].float())

    def wide(self, m, j):
        """Step j of b or c for every channel: [B, n, D, N]."""
        return m[:, :, j].repeat_interleave(self.D // self.G, dim=2)

    def decay(self, j):
        return torch.exp(self.dt[:, :, j, :, None] * self.a)

    def forward(self, h, each=None):
        u = self.dt * self.x
        for j in range(self.K):
            h = self.decay(j) * h + u[:, :, j, :, None] * self.wide(self.b, j)
            if each is not None:
                each(j, h)
        return h

    def flat(self, x):
        return x.reshape(self.B, -1, *x.shape[3:])[:, :self.T]


def _plain_scan_fwd(st, history=None):
    s = _Scan(st)
    zero = s.x.new_zeros(s.B, s.x.shape[1], s.D, s.N)
    before, last = _joined(s.forward(zero), s.kept, st["h0"])
    y = torch.empty_like(s.x)

    def each(j, h):
        y[:, :, j] = (s.wide(s.c, j) * h).sum(-1)
        if history is not None:
            history.append(h)

    s.forward(before, each)
    y = s.flat(y) + st["skip"] * s.flat(s.x)
    if history is not None:
        history.extend([s, before, y])
    if st["gate"] is not None:
        y = y * _silu(_clean(st["gate"], s.valid))
    return dict(y=y.to(st["x"].dtype), h=last)


def _plain_scan_train(st):
    hs = []
    out = _plain_scan_fwd(st, hs)
    s, before, inner = hs[-3:]
    dtype, skip = st["x"].dtype, st["skip"]
    dy, dgate = _clean(st["dy"], s.valid), None
    if st["gate"] is not None:
        gate = _clean(st["gate"], s.valid)
        dgate = (dy * inner * _silu_slope(gate)).to(dtype)
        dy = dy * _silu(gate)
    dyc = _chunks(dy, s.K)
    g = before.new_zeros(before.shape)
    for j in reversed(range(s.K)):
        g = s.decay(j) * (dyc[:, :, j, :, None] * s.wide(s.c, j) + g)
    g, dh0 = _joined(g, s.kept, st["dh"], reverse=True)
    du, ddt = torch.empty_like(s.x), torch.empty_like(s.x)
    db, dc = torch.empty_like(s.b), torch.empty_like(s.c)
    da = torch.zeros(s.D, s.N, dtype=torch.float64, device=g.device)  # a long sum
    per_group = lambda v: v.reshape(*v.shape[:2], s.G, s.D // s.G, s.N).sum(3)
    for j in reversed(range(s.K)):
        h, u, w = hs[j], dyc[:, :, j, :, None], s.decay(j)
        gh = u * s.wide(s.c, j) + g
        dc[:, :, j] = per_group(u * h)
        db[:, :, j] = per_group(gh * (s.dt[:, :, j] * s.x[:, :, j])[..., None])
        du[:, :, j] = (gh * s.wide(s.b, j)).sum(-1)
        g = w * gh
        moved = g * (hs[j - 1] if j else before)
        ddt[:, :, j] = (moved * s.a).sum(-1) + du[:, :, j] * s.x[:, :, j]
        da += (moved * s.dt[:, :, j, :, None]).sum((0, 1))
    dx = s.flat(du * s.dt) + skip * dy
    ddt = s.flat(ddt)
    if st["softplus"]:
        ddt = ddt * torch.sigmoid(s.raw)
    ddt = torch.where(s.valid[..., None], ddt, 0.0)
    return dict(out, dx=dx.to(dtype), ddt=ddt.to(dtype), da=da.float(), db=s.flat(db).to(dtype), dc=s.flat(dc).to(dtype),
                dskip=(dy * s.flat(s.x)).sum((0, 1)), dgate=dgate,
                ddt_bias=None if st["dt_bias"] is None else ddt.sum((0, 1)), dh0=None if st["h0"] is None else dh0)


def _put(after, slots, rows):
    """The rows of a pool after the step; those of ended requests go to a spare one."""
    spare = torch.cat([after, torch.zeros_like(after[:1])])
    on = slots >= 0
    spare[torch.where(on, slots, after.shape[0]).long()] = torch.where(on.reshape(-1, *[1] * (rows.dim() - 1)), rows, 0.0).to(after.dtype)
    after.copy_(spare[:-1])
    return after


def _plain_scan_step(st):
    x, slots = st["x"].float(), st["slots"]
    D, G = x.shape[1], st["b"].shape[1]
    dt = st["dt"].float()
    dt = dt if st["dt_bias"] is None else dt + st["dt_bias"]
    dt = _softplus(dt) if st["softplus"] else dt
    b, c = (st[n].float().repeat_interleave(D // G, dim=1) for n in "bc")
    h = torch.exp(dt[..., None] * st["a"]) * st["state"][slots.clamp(min=0).long()] + (dt * x)[..., None] * b
    y = (c * h).sum(-1) + st["skip"] * x
    if st["gate"] is not None:
        y = y * _silu(st["gate"].float())
    return dict(y=torch.where(slots[:, None] >= 0, y, 0.0).to(st["x"].dtype), state=_put(st["after"], slots, h))


def _conv_inputs(st):
    """The inputs in fp32 with the W - 1 before them, and the mask of the rows that count."""
    x, W = st["x"], st["weight"].shape[1]
    valid = _valid(x.shape[0], x.shape[1], st["lengths"], x.device)
    first = x.new_zeros(x.shape[0], W - 1, x.shape[2]) if st["state"] is None else st["state"]
    return torch.cat([first.float(), _clean(x, valid)], 1), valid


def _after(x, full, lengths, W):
    """Where in the inputs the last W - 1 of each sequence stand: [B, W - 1, D] indices."""
    L = torch.full((x.shape[0],), x.shape[1], device=x.device) if lengths is None else lengths.long()
    return (L[:, None] + torch.arange(W - 1, device=x.device))[..., None].expand(-1, -1, full.shape[2])


def _plain_conv_fwd(st):
    x, w = st["x"], st["weight"]
    T, W = x.shape[1], w.shape[1]
    full, valid = _conv_inputs(st)
    y = sum(w[:, j] * full[:, j:j + T] for j in range(W)) + st["bias"]
    y = _silu(y) if st["act"] == "silu" else y
    last = full.gather(1, _after(x, full, st["lengths"], W)).to(x.dtype)
    return dict(y=torch.where(valid[..., None], y, 0.0).to(x.dtype), last=last)


def _plain_conv_bwd(st):
    x, w = st["x"], st["weight"]
    T, W = x.shape[1], w.shape[1]
    full, valid = _conv_inputs(st)
    g = _clean(st["dy"], valid)
    if st["act"] == "silu":
        g = g * _silu_slope(sum(w[:, j] * full[:, j:j + T] for j in range(W)) + st["bias"])
    dfull = torch.zeros_like(full)
    for j in range(W):
        dfull[:, j:j + T] += w[:, j] * g
    if st["dlast"] is not None:
        dfull.scatter_add_(1, _after(x, full, st["lengths"], W), st["dlast"].float())
    dweight = torch.stack([(g * full[:, j:j + T]).sum((0, 1)) for j in range(W)], 1)
    dx = torch.where(valid[..., None], dfull[:, W - 1:], 0.0)
    return dict(dx=dx.to(x.dtype), dweight=dweight, dbias=g.sum((0, 1)),
                dstate=None if st["state"] is None else dfull[:, :W - 1].to(x.dtype))


def _plain_conv_step(st):
    x, slots, w = st["x"], st["slots"], st["weight"]
    full = torch.cat([st["state"][slots.clamp(min=0).long()], x[:, None]], 1)
    y = (full.float() * w.T).sum(1) + st["bias"]
    y = _silu(y) if st["act"] == "silu" else y
    return dict(y=torch.where(slots[:, None] >= 0, y, 0.0).to(x.dtype), state=_put(st["after"], slots, full[:, 1:]))


def _row_stats(r, rms):
    """Mean (zero without it) and 1 / sqrt(variance + eps) of each row: [..., 2]."""
    mean = torch.zeros_like(r[..., 0]) if rms else r.mean(-1)
    return torch.stack([mean, torch.rsqrt((r - mean[..., None]).square().mean(-1) + EPS)], -1)


def _plain_ln_fwd(st):
    x, res = st["x"], st["residual"]
    valid = _valid(x.shape[0], x.shape[1], st["lengths"], x.device)
    r = _clean(x, valid)
    r = r if res is None else r + _clean(res, valid)
    stats = _row_stats(r, st["rms"])
    y = (r - stats[..., :1]) * stats[..., 1:] * st["weight"] + st["bias"]
    y = torch.where(valid[..., None], y, 0.0).to(st["out"])
    return dict(y=y, r=None if res is None else r.to(res.dtype), stats=stats)


def _plain_ln_bwd(st):
    r, w, stats = st["r"], st["weight"], st["stats"]
    valid = _valid(r.shape[0], r.shape[1], st["lengths"], r.device)
    hat = torch.where(valid[..., None], (_clean(r, valid) - stats[..., :1]) * stats[..., 1:], 0.0)
    dy = _clean(st["dy"], valid)
    dh = dy * w
    g = dh - hat * (dh * hat).mean(-1, keepdim=True)
    if not st["rms"]:
        g = g - dh.mean(-1, keepdim=True)
    g = g * stats[..., 1:]
    if st["dr"] is not None:
        g = g + _clean(st["dr"], valid)
    return dict(dr=g.to(r.dtype), dx=g.to(st["branch"]), dweight=(dy * hat).sum((0, 1)), dbias=dy.sum((0, 1)))


PLAIN = {"scan_fwd": _plain_scan_fwd, "scan_train": _plain_scan_train, "scan_step": _plain_scan_step,
         "conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd, "conv_step": _plain_conv_step,
         "ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd}


# ---- the package's operators -------------------------------------------------------------------------------


def _own(st):
    import newton_solve_nonlinear_b200 as fw

    op = st["op"]
    if op.startswith("scan"):
        args = [st[n] for n in ("x", "dt", "a", "b", "c")]
        more = {n: st[n] for n in ("skip", "gate", "dt_bias", "softplus")}
        if op == "scan_step":
            y = fw.selective_scan_step(*args, st["state"], slots=st["slots"], out_state=st["after"], **more)
            return dict(y=y, state=st["after"])
        more.update(h0=st["h0"], lengths=st["lengths"])
        if op == "scan_fwd":
            y, h = fw.selective_scan(*args, **more)
            return dict(y=y, h=h)
        y, h, kept = fw.selective_scan(*args, keep=True, **more)
        return dict(fw.selective_scan_backward(*args, st["dy"], dh=st["dh"], kept=kept, **more), y=y, h=h)
    if op == "conv_fwd":
        y, last = fw.causal_conv(st["x"], st["weight"], st["bias"], act=st["act"], state=st["state"], lengths=st["lengths"])
        return dict(y=y, last=last)
    if op == "conv_bwd":
        return fw.causal_conv_backward(st["x"], st["weight"], st["dy"], st["bias"], act=st["act"], state=st["state"],
                                       dlast=st["dlast"], lengths=st["lengths"])
    if op == "conv_step":
        y = fw.causal_conv_step(st["x"], st["weight"], st["state"], st["bias"], act=st["act"], slots=st["slots"],
                                out_state=st["after"])
        return dict(y=y, state=st["after"])
    if op == "ln_fwd":
        y, r, stats = fw.layer_norm(st["x"], st["weight"], st["bias"], residual=st["residual"], rms=st["rms"], eps=EPS,
                                    lengths=st["lengths"], out_dtype=st["out"])
        return dict(y=y, r=None if st["residual"] is None else r, stats=stats)
    return fw.layer_norm_backward(st["r"], st["stats"], st["dy"], st["weight"], st["bias"], dr=st["dr"], rms=st["rms"],
                                  lengths=st["lengths"], dx_dtype=st["branch"])


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---- 64 bits, from the definitions -------------------------------------------------------------------------


def _on(x, lengths):
    """[B, T, 1]: 1 where a token counts, in 64 bits."""
    n = x.shape[0]
    lengths = torch.full((n,), x.shape[1], device=x.device) if lengths is None else lengths
    return (torch.arange(x.shape[1], device=x.device)[None] < lengths[:, None]).double()[..., None]


def _double(x, lengths):
    """64 bits, zeros behind the lengths."""
    if lengths is None:
        return x.double()
    on = _on(x, lengths).bool().reshape(*x.shape[:2], *[1] * (x.dim() - 2))
    return x.double().masked_fill(~on, 0.0)


def _exact_scan_fwd(st):
    """Blocks of tokens, in each of them log2 steps that compose (decay, addition) pairs of ever longer stretches."""
    B, T, D = st["x"].shape
    G, N = st["b"].shape[2:]
    L = st["lengths"]
    a, skip = st["a"].double(), st["skip"].double()
    h = torch.zeros(B, D, N, dtype=torch.float64, device=a.device) if st["h0"] is None else st["h0"].double()
    y = torch.empty(B, T, D, dtype=torch.float64, device=a.device)
    on = _on(st["x"], L)
    most = max(1, (1 << 27) // (B * D * N))
    for t in range(0, T, most):
        cut = lambda v: _double(v, L)[:, t:t + most] if T <= most else _double(v[:, t:t + most], None if L is None else L - t)
        x, dt, b, c = cut(st["x"]), cut(st["dt"]), cut(st["b"]), cut(st["c"])
        n = x.shape[1]
        dt = dt if st["dt_bias"] is None else dt + st["dt_bias"].double()
        dt = (torch.nn.functional.softplus(dt, threshold=40.0) if st["softplus"] else dt) * on[:, t:t + most]
        decay = torch.exp(dt[..., None] * a)
        add = ((dt * x).reshape(B, n, G, D // G, 1) * b[:, :, :, None]).reshape(B, n, D, N)
        add[:, 0] += decay[:, 0] * h
        far = 1
        while far < n:
            add[:, far:] = add[:, far:] + decay[:, far:] * add[:, :-far]
            decay[:, far:] = decay[:, far:] * decay[:, :-far]
            far *= 2
        h = add[:, -1].clone()
        out = (add.reshape(B, n, G, D // G, N) * c[:, :, :, None]).sum(-1).reshape(B, n, D) + skip * x
        if st["gate"] is not None:
            out = out * torch.nn.functional.silu(cut(st["gate"]))
        y[:, t:t + most] = out * on[:, t:t + most]
    return dict(y=y, h=h)


def _exact_scan_train(st):
    """Token by token, the gradients by differentiation; a block of a group's channels at a time."""
    B, T, D = st["x"].shape
    G, N = st["b"].shape[2:]
    per = D // G
    width = max(1, min(per, (1 << 32) // (B * T * N)))
    if T * G * -(-per // width) > 20_000:
        return None
    L, new = st["lengths"], lambda *s: torch.zeros(*s, dtype=torch.float64, device=st["a"].device)
    out = dict(y=new(B, T, D), h=new(B, D, N), dx=new(B, T, D), ddt=new(B, T, D), da=new(D, N), db=new(B, T, G, N),
               dc=new(B, T, G, N), dskip=new(D), dgate=None if st["gate"] is None else new(B, T, D),
               ddt_bias=None if st["dt_bias"] is None else new(D), dh0=None if st["h0"] is None else new(B, D, N))
    on = _on(st["x"], L)
    for g in range(G):
        for lo in range(g * per, (g + 1) * per, width):
            k = slice(lo, min(lo + width, (g + 1) * per))
            leaf = lambda v: None if v is None else v.double().contiguous().requires_grad_()
            cut = lambda v: None if v is None else leaf(_double(v[..., k], L))
            x, raw, gate, dy = cut(st["x"]), cut(st["dt"]), cut(st["gate"]), _double(st["dy"][..., k], L)
            a, skip, bias = leaf(st["a"][k]), leaf(st["skip"][k]), None if st["dt_bias"] is None else leaf(st["dt_bias"][k])
            b, c = leaf(_double(st["b"], L)[:, :, g]), leaf(_double(st["c"], L)[:, :, g])
            h0 = new(B, x.shape[2], N) if st["h0"] is None else st["h0"][:, k].double()
            h0.requires_grad_()
            with torch.enable_grad():
                dt = raw if bias is None else raw + bias
                dt = (torch.nn.functional.softplus(dt, threshold=40.0) if st["softplus"] else dt) * on
                h, u, ys = h0, dt * x, []
                for dt_t, u_t, b_t, c_t in zip(dt.unbind(1), u.unbind(1), b.unbind(1), c.unbind(1)):
                    h = torch.exp(dt_t[..., None] * a) * h + u_t[..., None] * b_t[:, None]
                    ys.append(torch.einsum("bdn,bn->bd", h, c_t))
                y = torch.stack(ys, 1) + skip * x
                y = y if gate is None else y * torch.nn.functional.silu(gate)
                loss = (y * dy * on).sum()
                loss = loss if st["dh"] is None else loss + (h * st["dh"][:, k].double()).sum()
            leaves = [v for v in (x, raw, a, b, c, skip, gate, bias, h0) if v is not None]
            grads = dict(zip(map(id, leaves), torch.autograd.grad(loss, leaves)))
            of = lambda v: grads[id(v)]
            out["y"][..., k], out["h"][:, k] = (y * on).detach(), h.detach()
            out["dx"][..., k], out["ddt"][..., k], out["da"][k], out["dskip"][k] = of(x), of(raw), of(a), of(skip)
            out["db"][:, :, g] += of(b)
            out["dc"][:, :, g] += of(c)
            if gate is not None:
                out["dgate"][..., k] = of(gate)
            if bias is not None:
                out["ddt_bias"][k] = of(bias)
            if st["h0"] is not None:
                out["dh0"][:, k] = of(h0)
    return out


def _exact_scan_step(st):
    x, dt, b, c, state = (st[n].double() for n in ("x", "dt", "b", "c", "state"))
    D, G = x.shape[1], b.shape[1]
    dt = dt if st["dt_bias"] is None else dt + st["dt_bias"].double()
    dt = torch.nn.functional.softplus(dt, threshold=40.0) if st["softplus"] else dt
    after, y = state.clone(), torch.zeros_like(x)
    for row, slot in enumerate(st["slots"].tolist()):
        if slot >= 0:
            u = (dt[row] * x[row]).reshape(G, D // G)
            add = torch.einsum("gd,gn->gdn", u, b[row]).reshape(D, -1)
            after[slot] = torch.exp(dt[row][:, None] * st["a"].double()) * state[slot] + add
            y[row] = torch.einsum("gdn,gn->gd", after[slot].reshape(G, D // G, -1), c[row]).reshape(D) + st["skip"].double() * x[row]
            if st["gate"] is not None:
                y[row] *= torch.nn.functional.silu(st["gate"][row].double())
    return dict(y=y, state=after)


def _exact_conv(st, back):
    x, w, bias = _double(st["x"], st["lengths"]), st["weight"].double(), st["bias"].double()
    B, T, D = x.shape
    W, on = w.shape[1], _on(x, st["lengths"])
    first = torch.zeros(B, W - 1, D, dtype=torch.float64, device=x.device) if st["state"] is None else st["state"].double()
    for v in (x, w, bias, first):
        v.requires_grad_(back)
    with torch.enable_grad():
        full = torch.cat([first, x], 1)
        y = torch.einsum("btdw,dw->btd", full.unfold(1, W, 1), w) + bias
        y = (torch.nn.functional.silu(y) if st["act"] == "silu" else y) * on
        ends = [T] * B if st["lengths"] is None else st["lengths"].tolist()
        last = torch.stack([full[i, n:n + W - 1] for i, n in enumerate(ends)])
    if not back:
        return dict(y=y, last=last)
    loss = (y * _double(st["dy"], st["lengths"])).sum()
    if st["dlast"] is not None:
        loss = loss + (last * st["dlast"].double()).sum()
    dx, dweight, dbias, dstate = torch.autograd.grad(loss, (x, w, bias, first))
    return dict(dx=dx * on, dweight=dweight, dbias=dbias, dstate=None if st["state"] is None else dstate)


def _exact_conv_step(st):
    x, w, state, bias = (st[n].double() for n in ("x", "weight", "state", "bias"))
    after, y = state.clone(), torch.zeros_like(x)
    for row, slot in enumerate(st["slots"].tolist()):
        if slot >= 0:
            full = torch.cat([state[slot], x[row][None]])
            v = torch.einsum("wd,dw->d", full, w) + bias
            y[row] = torch.nn.functional.silu(v) if st["act"] == "silu" else v
            after[slot] = full[1:]
    return dict(y=y, state=after)


def _exact_ln(st, back):
    w, bias, L, rms = st["weight"].double(), st["bias"].double(), st["lengths"], st["rms"]
    if not back:
        r = _double(st["x"], L)
        r = r if st["residual"] is None else r + _double(st["residual"], L)
        if rms:
            mean, var = torch.zeros_like(r[..., 0]), (r * r).mean(-1)
        else:
            var, mean = torch.var_mean(r, -1, correction=0)
        stats = torch.stack([mean, 1 / torch.sqrt(var + EPS)], -1)
        y = ((r - mean[..., None]) * stats[..., 1:] * w + bias) * _on(r, L)
        return dict(y=y, r=None if st["residual"] is None else r, stats=stats)
    # with the statistics as functions of the row; their given values are rounded to fp32, so they enter as they are
    r, dy = _double(st["r"], L), _double(st["dy"], L)
    mean, rstd = (st["stats"][..., i:i + 1].double() for i in (0, 1))
    hat = (r - mean) * rstd * _on(r, L)
    n = r.shape[-1]
    along = torch.einsum("btc,btc,c->bt", dy, hat, w)[..., None] / n
    level = 0.0 if rms else torch.einsum("btc,c->bt", dy, w)[..., None] / n
    g = rstd * (dy * w - level - hat * along) * _on(r, L)
    if st["dr"] is not None:
        g = g + _double(st["dr"], L)
    return dict(dr=g, dx=g, dweight=torch.einsum("btc,btc->c", dy, hat), dbias=dy.sum((0, 1)))


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op.startswith("ln"):
        return _exact_ln(st, op == "ln_bwd")
    if op.startswith("conv"):
        return _exact_conv_step(st) if op == "conv_step" else _exact_conv(st, op == "conv_bwd")
    return {"scan_fwd": _exact_scan_fwd, "scan_train": _exact_scan_train, "scan_step": _exact_scan_step}[op](st)


# ---- what a pass cannot do without -------------------------------------------------------------------------


def work(case):
    """Per state of the scan: an exponential, four products and sums forward, eleven more of them backward."""
    c = case
    e = {"bf16": 2, "f32": 4}
    if c["op"].startswith("ln"):
        n = c["N"] * c["S"] * c["C"]
        x, r, y = e[c["x"]], e[c["r"]], e[c["y"]]
        if c["op"] == "ln_fwd":
            return {"bytes": n * (x + y + (2 * r if c["add"] else 0)), "flops": n * 8}
        return {"bytes": n * (r + y + (r if c["add"] else 0) + r + (x if x != r else 0)), "flops": n * 14}
    s = e[c["dtype"]]
    if c["op"] == "conv_step":
        rows = c["B"] * c["D"]
        return {"bytes": rows * (2 + 2 * (c["W"] - 1)) * s + c["D"] * (c["W"] + 1) * 4, "flops": rows * (2 * c["W"] + 4)}
    if c["op"].startswith("conv"):
        rows, ends = c["B"] * c["T"] * c["D"], c["B"] * (c["W"] - 1) * c["D"] * (2 if c["start"] else 1)
        if c["op"] == "conv_fwd":
            return {"bytes": (2 * rows + ends) * s, "flops": rows * (2 * c["W"] + 4)}
        return {"bytes": (3 * rows + (ends if c["start"] else 0)) * s, "flops": rows * (6 * c["W"] + 8)}
    D = c["G"] * c["per"]
    gate = 1 if c["gate"] else 0
    if c["op"] == "scan_step":
        rows = c["B"]
        return {"bytes": rows * (D * c["N"] * 8 + (D * (3 + gate) + 2 * c["G"] * c["N"]) * s) + D * (c["N"] + 2) * 4,
                "flops": rows * D * c["N"] * 6}
    tokens, h = c["B"] * c["T"], c["B"] * D * c["N"] * 4
    rows, shared = D * (3 + gate), 2 * c["G"] * c["N"]
    if c["op"] == "scan_fwd":
        return {"bytes": tokens * (rows + shared) * s + h * (2 if c["start"] else 1), "flops": tokens * D * c["N"] * 6}
    rows += D * (2 + gate) + D  # dx, ddt, dgate and dy
    return {"bytes": tokens * (rows + 2 * shared) * s + h * (4 if c["start"] else 1), "flops": tokens * D * c["N"] * 28}
