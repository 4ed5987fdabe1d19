"""What the matrix-state recurrence and the group norm are measured on.

Five operators, each on cases spread over its real range:
  la_fwd   linear attention with a decay per head over a prompt (outputs and the final state)
  la_bwd   its backward pass
  la_step  its recurrent form for one token per sequence, states in a pool
  gn_fwd   group norm with an activation or a gate, channels last (outputs and statistics)
  gn_bwd   its backward pass
``run`` computes them in plain torch operations, or, where ``own`` is true, by the package's entry points;
``exact`` in 64 bits from the definitions.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -------------------------------------------------------------------------------------------------


def _la(name, op, B, T, H, Hkv, dk, dv, dtype, ragged=False, start=False, decay="slow"):
    return dict(name=name, op=op, B=B, T=T, H=H, Hkv=Hkv, dk=dk, dv=dv, dtype=dtype, ragged=ragged, start=start,
                decay=decay)


def _step(name, B, H, Hkv, dk, dv, dtype, pool):
    return dict(name=name, op="la_step", B=B, H=H, Hkv=Hkv, dk=dk, dv=dv, dtype=dtype, pool=pool)


def _gn(name, op, N, S, G, cg, dtype, out, act, gate, ragged=False):
    return dict(name=name, op=op, N=N, S=S, G=G, cg=cg, dtype=dtype, out=out, act=act, gate=gate, ragged=ragged)


def listed():
    return [
        # a short prompt of one user: nothing but latency
        _la("fwd_short_prompt", "la_fwd", 1, 37, 4, 4, 64, 64, "bf16", start=True),
        # a training or prefill batch: many sequences and heads fill the card
        _la("fwd_batch", "la_fwd", 8, 8192, 16, 16, 128, 128, "bf16"),
        # one very long document on few heads with shared keys and values: parallel over time or not at all
        _la("fwd_long", "la_fwd", 1, 131072, 8, 2, 64, 64, "bf16", start=True),
        # a padded batch of prompts of odd lengths in fp32, head widths that are no power of two
        _la("fwd_ragged_f32", "la_fwd", 5, 2011, 12, 4, 96, 80, "f32", ragged=True, start=True, decay="mixed"),
        # a training step's backward pass
        _la("bwd_batch", "la_bwd", 4, 4096, 16, 16, 128, 128, "bf16"),
        # a padded batch with shared keys and values, state carried in and out, in fp32
        _la("bwd_ragged_f32", "la_bwd", 3, 517, 6, 3, 48, 64, "f32", ragged=True, start=True, decay="mixed"),
        # one token of one user
        _step("step_single", 1, 8, 8, 64, 64, "bf16", 4),
        # one token of each of many users served at once, their states in a pool
        _step("step_serving", 256, 16, 16, 128, 128, "bf16", 320),
        # each token's heads normalised behind linear attention, gated
        _gn("gn_heads_gated", "gn_fwd", 32768, 1, 16, 128, "bf16", "bf16", "silu", True),
        # the states of a recurrent layer over a whole sequence, handed on in bf16 to the next layer's projection
        _gn("gn_states", "gn_fwd", 16, 65536, 4, 16, "f32", "bf16", "silu", False),
        # the gated heads' backward pass
        _gn("gn_heads_gated_bwd", "gn_bwd", 8192, 1, 16, 128, "bf16", "bf16", "silu", True),
        # the backward pass over a padded batch of sequences
        _gn("gn_states_bwd", "gn_bwd", 8, 1000, 32, 20, "f32", "f32", "gelu", False, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["la_fwd", "la_fwd", "la_bwd", "la_step", "gn_fwd", "gn_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("la_fwd", "la_bwd", "la_step"):
        H = _log_int(rng, 1, 32)
        Hkv = rng.choice([h for h in range(1, H + 1) if H % h == 0])
        if rng.random() < 0.5:
            dk, dv = rng.choice([32, 64, 96, 128]), rng.choice([32, 64, 96, 128])
        else:
            dk, dv = rng.randint(1, 128), rng.randint(1, 128)
        if op == "la_step":
            B = _log_int(rng, 1, 512)
            B = max(1, min(B, 268_435_456 // (H * dk * dv * 4)))
            return dict(op=op, B=B, H=H, Hkv=Hkv, dk=dk, dv=dv, dtype=dtype, pool=B + rng.randint(0, B))
        most = 268_435_456 if op == "la_fwd" else 67_108_864
        B = _log_int(rng, 1, 16)
        T = _log_int(rng, 1, 131072)
        T = max(1, min(T, most // (B * H * (dk + dv)) // (1 if dtype == "bf16" else 8)))
        return dict(op=op, B=B, T=T, H=H, Hkv=Hkv, dk=dk, dv=dv, dtype=dtype, ragged=rng.random() < 0.4,
                    start=rng.random() < 0.5, decay=rng.choice(["slow", "slow", "mixed"]))
    most = 67_108_864 if op == "gn_fwd" else 16_777_216
    G, cg = _log_int(rng, 1, 64), _log_int(rng, 1, 256)
    if rng.random() < 0.5:
        cg = max(8, cg // 8 * 8)
    if rng.random() < 0.5:
        S, N = 1, _log_int(rng, 1, 65536)
    else:
        S, N = _log_int(rng, 2, 65536), _log_int(rng, 1, 32)
        S = max(2, min(S, most // (G * cg)))
    N = max(1, min(N, most // (S * G * cg)))
    return dict(op=op, N=N, S=S, G=G, cg=cg, dtype=dtype, out=rng.choice([dtype, "bf16", "f32"]),
                act=rng.choice(["none", "silu", "gelu"]), gate=rng.random() < 0.4,
                ragged=S > 1 and rng.random() < 0.3)


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c, dtype = case, DTYPES[case["dtype"]]
    st = dict(op=c["op"], case=c)
    if c["op"].startswith("la_"):
        B, H, Hkv, dk, dv = c["B"], c["H"], c["Hkv"], c["dk"], c["dv"]
        if c.get("decay") == "mixed":  # from no decay at all to one that forgets within a token or two
            ld = torch.linspace(0.0, -3.0, H, device="cuda")
        else:  # memories of 32 to 4096 tokens over the heads
            ld = torch.log1p(-torch.exp2(-torch.linspace(5.0, 12.0, H, device="cuda")))
        st.update(log_decay=ld)
        if c["op"] == "la_step":
            state = _normal(gen, c["pool"], H, dk, dv)
            slots = torch.randperm(c["pool"], device="cuda", generator=gen)[:B].to(torch.int32)
            if B > 4:
                slots[B // 2] = -1  # a request that has ended
            st.update(q=_normal(gen, B, H, dk, dtype=dtype), k=_normal(gen, B, Hkv, dk, dtype=dtype),
                      v=_normal(gen, B, Hkv, dv, dtype=dtype), state=state, slots=slots, after=state.clone())
            return st
        T = c["T"]
        lengths = _lengths(gen, B, T, c["ragged"])
        st.update(lengths=lengths)
        for name, h, d in (("q", H, dk), ("k", Hkv, dk), ("v", Hkv, dv)):
            st[name] = _spoil(_normal(gen, B, T, h, d, dtype=dtype), lengths)
        st["s0"] = _normal(gen, B, H, dk, dv) if c["start"] else None
        if c["op"] == "la_bwd":
            st["do"] = _spoil(_normal(gen, B, T, H, dv, dtype=dtype), lengths)
            st["ds"] = _normal(gen, B, H, dk, dv) if c["start"] else None
        return st
    N, S, G, cg = c["N"], c["S"], c["G"], c["cg"]
    C = G * cg
    lengths = _lengths(gen, N, S, c["ragged"])
    x = _spoil(_normal(gen, N, S, C, dtype=dtype, mean=0.3, std=1.5), lengths)
    st.update(x=x, lengths=lengths, groups=G, act=c["act"], out=DTYPES[c["out"]],
              weight=_normal(gen, C, mean=1.0, std=0.2), bias=_normal(gen, C, std=0.2),
              gate=_spoil(_normal(gen, N, S, C, dtype=dtype), lengths) if c["gate"] else None)
    if c["op"] == "gn_bwd":
        st["dy"] = _spoil(_normal(gen, N, S, C, dtype=DTYPES[c["out"]]), lengths)
        st["stats"] = _statistics(x.double(), lengths, G)[2].float()
    return st


# ---- plain forms -------------------------------------------------------------------------------------------

EPS = 1e-5
CHUNK = 256


def _valid(n, T, lengths, device):
    t = torch.arange(T, device=device)
    return torch.ones(n, T, dtype=torch.bool, device=device) if lengths is None else t[None] < lengths[:, None]


def _clean(x, valid):
    """fp32 with zeros behind the lengths."""
    return torch.where(valid.reshape(valid.shape + (1,) * (x.dim() - 2)), x.float(), 0.0)


def _pow(ld, n):
    """decay^n in fp32, [H, *n.shape]; the exponents in 64 bits, as far positions need."""
    ld = ld.double().clamp(min=-1e4)
    return torch.exp(ld.reshape(-1, *([1] * n.dim())) * n.double()).float()


def _causal(q, k, v, ld, s0):
    """sum_{s <= t} decay^(t-s) (q_t . k_s) v_s + decay^(t+1) s0^T q_t for [B, T, H, .] in fp32, by chunks."""
    B, T, H, dk = q.shape
    dv, C = v.shape[-1], min(CHUNK, T)
    n = -(-T // C)
    split = lambda x: torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * C - T)).reshape(B, n, C, H, -1).permute(0, 3, 1, 2, 4)
    q, k, v = split(q), split(k), split(v)
    i, j = torch.arange(C, device=q.device), torch.arange(n, device=q.device)
    gap = i[:, None] - i[None]
    weight = torch.where(gap >= 0, _pow(ld, gap.clamp(min=0)), 0.0)
    o = (q @ k.transpose(-1, -2)).mul_(weight[None, :, None]) @ v
    add = (k * _pow(ld, C - 1 - i)[None, :, None, :, None]).transpose(-1, -2) @ v
    gap = j[:, None] - 1 - j[None]
    weight = torch.where(gap >= 0, _pow(ld, C * gap.clamp(min=0)), 0.0)
    state = (weight[None] @ add.reshape(B, H, n, dk * dv)).reshape(B, H, n, dk, dv)
    if s0 is not None:
        state = state + _pow(ld, C * j)[None, :, :, None, None] * s0[:, :, None]
    o = o + (q * _pow(ld, i + 1)[None, :, None, :, None]) @ state
    return o.permute(0, 2, 3, 1, 4).reshape(B, n * C, H, dv)[:, :T]


def _left(ld, lengths, B, T, device):
    """decay^(L - 1 - t) for t < L, else 0: [B, T, H]; and decay^L: [B, H]."""
    L = torch.full((B,), T, device=device) if lengths is None else lengths.long()
    gap = L[:, None] - 1 - torch.arange(T, device=device)[None]
    w = torch.where(gap >= 0, _pow(ld, gap.clamp(min=0)), 0.0)
    return w.permute(1, 2, 0), _pow(ld, L).transpose(0, 1)


def _heads(x, H):
    return x.repeat_interleave(H // x.shape[2], dim=2)


def _shared(x, Hkv):
    B, T, H, d = x.shape
    return x.reshape(B, T, Hkv, H // Hkv, d).sum(3)


def _plain_la_fwd(st):
    q, k, v, ld, s0 = st["q"], st["k"], st["v"], st["log_decay"], st["s0"]
    B, T, H, dk = q.shape
    valid = _valid(B, T, st["lengths"], q.device)
    k, v = _heads(_clean(k, valid), H), _heads(_clean(v, valid), H)
    o = _causal(_clean(q, valid), k, v, ld, s0).mul_(dk ** -0.5)
    left, whole = _left(ld, st["lengths"], B, T, q.device)
    s = (k * left[..., None]).permute(0, 2, 3, 1) @ v.transpose(1, 2)
    if s0 is not None:
        s = s + whole[..., None, None] * s0
    return dict(o=o.to(q.dtype), s=s)


def _plain_la_bwd(st):
    ld, s0, ds = st["log_decay"], st["s0"], st["ds"]
    B, T, H, dk = st["q"].shape
    Hkv, scale, dtype, dev = st["k"].shape[2], dk ** -0.5, st["q"].dtype, st["q"].device
    valid = _valid(B, T, st["lengths"], dev)
    q, do = _clean(st["q"], valid), _clean(st["do"], valid)
    k, v = _heads(_clean(st["k"], valid), H), _heads(_clean(st["v"], valid), H)
    dq = _causal(do, v, k, ld, None if s0 is None else s0.transpose(-1, -2)).mul_(scale)
    dk_ = _causal(v.flip(1), do.flip(1), q.flip(1), ld, None).flip(1).mul_(scale)
    dv_ = _causal(k.flip(1), q.flip(1), do.flip(1), ld, None).flip(1).mul_(scale)
    left, whole = _left(ld, st["lengths"], B, T, dev)
    far = _pow(ld, torch.arange(1, T + 1, device=dev)).transpose(0, 1)
    ds0 = (q * (far * scale)[None, ..., None]).permute(0, 2, 3, 1) @ do.transpose(1, 2)
    if ds is not None:
        dk_ = dk_ + ((v * left[..., None]).transpose(1, 2) @ ds.transpose(-1, -2)).transpose(1, 2)
        dv_ = dv_ + ((k * left[..., None]).transpose(1, 2) @ ds).transpose(1, 2)
        ds0 = ds0 + whole[..., None, None] * ds
    return dict(dq=dq.to(dtype), dk=_shared(dk_, Hkv).to(dtype), dv=_shared(dv_, Hkv).to(dtype),
                ds0=None if s0 is None else ds0)


def _plain_la_step(st):
    q, k, v, ld = st["q"], st["k"], st["v"], st["log_decay"]
    H, dk = q.shape[1], q.shape[2]
    slots = st["slots"].long()
    active = slots >= 0
    rows = slots.clamp(min=0)
    k, v = k.float().repeat_interleave(H // k.shape[1], dim=1), v.float().repeat_interleave(H // v.shape[1], dim=1)
    s = torch.exp(ld)[None, :, None, None] * st["state"][rows] + k[..., :, None] * v[..., None, :]
    o = (q.float()[..., None, :] @ s).squeeze(-2) * dk ** -0.5
    on = active[:, None, None, None]
    spare = torch.cat([st["after"], torch.zeros_like(st["after"][:1])])  # ended requests write to a spare row
    spare[torch.where(active, rows, spare.shape[0] - 1)] = torch.where(on, s, 0.0)
    st["after"].copy_(spare[:-1])
    return dict(o=torch.where(on[..., 0], o, 0.0).to(q.dtype), state=st["after"])


def _statistics(x, lengths, groups):
    """x [N, S, C] -> normalised x [N, S, G, cg] (zeros behind the lengths), the rows' mask, [N, G, 2] mean and 1/std."""
    N, S, C = x.shape
    valid = _valid(N, S, lengths, x.device)[:, :, None, None]
    xg = torch.where(valid, x.reshape(N, S, groups, -1), 0.0)
    count = valid.sum(1, keepdim=True).clamp(min=1) * (C // groups)
    mean = xg.sum((1, 3), keepdim=True) / count
    diff = torch.where(valid, xg - mean, 0.0)
    rstd = torch.rsqrt(diff.square().sum((1, 3), keepdim=True) / count + EPS)
    return diff * rstd, valid, torch.stack([mean, rstd], -1).reshape(N, groups, 2)


def _act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def _plain_gn_fwd(st):
    x, G = st["x"], st["groups"]
    N, S, C = x.shape
    hat, valid, stats = _statistics(x.float(), st["lengths"], G)
    z = (hat.reshape(N, S, C) * st["weight"] + st["bias"])
    y = _act(z, st["act"]) if st["gate"] is None else z * _act(_clean(st["gate"], valid[:, :, 0, 0]), st["act"])
    return dict(y=torch.where(valid[..., 0], y, 0.0).to(st["out"]), stats=stats)


def _plain_gn_bwd(st):
    x, G, w = st["x"], st["groups"], st["weight"]
    N, S, C = x.shape
    valid = _valid(N, S, st["lengths"], x.device)
    mean, rstd = (st["stats"][..., i].reshape(N, 1, G, 1) for i in (0, 1))
    hat = (_clean(x, valid).reshape(N, S, G, -1) - mean).mul_(rstd)
    hat = torch.where(valid[..., None, None], hat, 0.0).reshape(N, S, C)
    z = hat * w + st["bias"]
    dy = _clean(st["dy"], valid)
    dgate = None
    if st["gate"] is None:
        dz = dy * _act_slope(z, st["act"])
    else:
        gate = _clean(st["gate"], valid)
        dz = dy * _act(gate, st["act"])
        dgate = (dy * z * _act_slope(gate, st["act"])).to(st["gate"].dtype)
    count = valid.sum(1).clamp(min=1).reshape(N, 1, 1, 1) * (C // G)
    dh, hg = (dz * w).reshape(N, S, G, -1), hat.reshape(N, S, G, -1)
    dx = dh - dh.sum((1, 3), keepdim=True) / count - hg * ((dh * hg).sum((1, 3), keepdim=True) / count)
    dx = torch.where(valid[..., None, None], dx * rstd, 0.0).reshape(N, S, C)
    return dict(dx=dx.to(x.dtype), dweight=(dz * hat).sum((0, 1)), dbias=dz.sum((0, 1)), dgate=dgate)


PLAIN = {"la_fwd": _plain_la_fwd, "la_bwd": _plain_la_bwd, "la_step": _plain_la_step, "gn_fwd": _plain_gn_fwd,
         "gn_bwd": _plain_gn_bwd}


# ---- the package's operators -------------------------------------------------------------------------------


def _own(st):
    import newton_solve_nonlinear_b200 as fw

    op = st["op"]
    if op == "la_fwd":
        o, s = fw.linear_attention(st["q"], st["k"], st["v"], st["log_decay"], s0=st["s0"], lengths=st["lengths"])
        return dict(o=o, s=s)
    if op == "la_bwd":
        return fw.linear_attention_backward(st["q"], st["k"], st["v"], st["log_decay"], st["do"], s0=st["s0"],
                                            ds=st["ds"], lengths=st["lengths"])
    if op == "la_step":
        o = fw.linear_attention_step(st["q"], st["k"], st["v"], st["log_decay"], st["state"], slots=st["slots"],
                                     out_state=st["after"])
        return dict(o=o, state=st["after"])
    if op == "gn_fwd":
        y, stats = fw.group_norm(st["x"], st["groups"], st["weight"], st["bias"], gate=st["gate"], act=st["act"],
                                 eps=EPS, lengths=st["lengths"], out_dtype=st["out"])
        return dict(y=y, stats=stats)
    return fw.group_norm_backward(st["x"], st["stats"], st["dy"], st["groups"], st["weight"], st["bias"],
                                  gate=st["gate"], act=st["act"], lengths=st["lengths"])


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---- 64 bits, from the definitions -------------------------------------------------------------------------

ROWS = 2048


def _exact_la(st, back):
    """Token by token sums over all earlier tokens, a block of rows of the [T, T] weights at a time."""
    q, k, v, ld, s0 = st["q"], st["k"], st["v"], st["log_decay"].double(), st["s0"]
    B, T, H, dk = q.shape
    Hkv, dv, scale, dev = k.shape[2], v.shape[3], dk ** -0.5, q.device
    if (3 if back else 1) * B * H * float(T) * T * (dk + dv) > 2e14:
        return None
    zeros = lambda *s: torch.zeros(*s, dtype=torch.float64, device=dev)
    o, s = zeros(B, T, H, dv), zeros(B, H, dk, dv)
    dq, dkk, dvv, ds0 = (zeros(B, T, H, dk), zeros(B, T, Hkv, dk), zeros(B, T, Hkv, dv), zeros(B, H, dk, dv)) if back else [None] * 4
    for b in range(B):
        L = T if st["lengths"] is None else int(st["lengths"][b])
        t = torch.arange(L, device=dev, dtype=torch.float64)
        for h in range(H):
            u = h // (H // Hkv)
            Q, K, V = q[b, :L, h].double(), k[b, :L, u].double(), v[b, :L, u].double()
            end, first = torch.exp((L - 1 - t) * ld[h])[:, None], torch.exp((t + 1) * ld[h])[:, None]
            if back:
                dO = st["do"][b, :L, h].double()
            for a in range(0, L, ROWS):
                z = min(L, a + ROWS)
                gap = t[a:z, None] - t[None, :z]
                W = torch.exp(gap.clamp(min=0) * ld[h]).mul_(gap >= 0)
                if back:
                    P, dP = (Q[a:z] @ K[:z].T).mul_(W), (dO[a:z] @ V[:z].T).mul_(W)
                    dq[b, a:z, h] = scale * dP @ K[:z]
                    dkk[b, :z, u] += scale * dP.T @ Q[a:z]
                    dvv[b, :z, u] += scale * P.T @ dO[a:z]
                else:
                    o[b, a:z, h] = scale * ((Q[a:z] @ K[:z].T).mul_(W) @ V[:z])
            if back:
                ds0[b, h] = scale * (Q * first).T @ dO
                if s0 is not None:
                    dq[b, :L, h] += scale * first * (dO @ s0[b, h].double().T)
                if st["ds"] is not None:
                    dS = st["ds"][b, h].double()
                    dkk[b, :L, u] += end * (V @ dS.T)
                    dvv[b, :L, u] += end * (K @ dS)
                    ds0[b, h] += torch.exp(L * ld[h]) * dS
            else:
                s[b, h] = (K * end).T @ V
                if s0 is not None:
                    o[b, :L, h] += scale * first * (Q @ s0[b, h].double())
                    s[b, h] += torch.exp(L * ld[h]) * s0[b, h].double()
    if back and s0 is None:
        ds0 = None
    return dict(dq=dq, dk=dkk, dv=dvv, ds0=ds0) if back else dict(o=o, s=s)


def _exact_step(st):
    q, k, v, state = (st[n].double() for n in ("q", "k", "v", "state"))
    after, o = state.clone(), torch.zeros(*q.shape[:2], v.shape[2], dtype=torch.float64, device=q.device)
    decay, per = torch.exp(st["log_decay"].double()), q.shape[1] // k.shape[1]
    for b, slot in enumerate(st["slots"].tolist()):
        if slot >= 0:
            kb, vb = k[b].repeat_interleave(per, 0), v[b].repeat_interleave(per, 0)
            after[slot] = decay[:, None, None] * state[slot] + torch.einsum("hi,hj->hij", kb, vb)
            o[b] = torch.einsum("hi,hij->hj", q[b], after[slot]) * q.shape[2] ** -0.5
    return dict(o=o, state=after)


def _exact_gn(st, back):
    x, G, w, bias, act = st["x"].double(), st["groups"], st["weight"].double(), st["bias"].double(), st["act"]
    N, S, C = x.shape
    other = (lambda u: u) if act == "none" else torch.nn.functional.silu if act == "silu" else torch.nn.functional.gelu
    lengths = [S] * N if st["lengths"] is None else st["lengths"].tolist()
    new = lambda *s: torch.zeros(*s, dtype=torch.float64, device=x.device)
    if not back and all(n == S for n in lengths):
        var, mean = torch.var_mean(x.reshape(N, S, G, -1), (1, 3), correction=0)
        stats = torch.stack([mean, (var + EPS).rsqrt()], -1)
        z = ((x.reshape(N, S, G, -1) - mean[:, None, :, None]) * stats[:, None, :, 1, None]).reshape(N, S, C) * w + bias
        return dict(y=other(z) if st["gate"] is None else z * other(st["gate"].double()), stats=stats)
    if not back:
        y, stats = new(N, S, C), new(N, G, 2)
        stats[..., 1] = EPS ** -0.5
        for n, L in enumerate(lengths):
            if L:
                var, mean = torch.var_mean(x[n, :L].reshape(L, G, -1), (0, 2), correction=0)
                stats[n] = torch.stack([mean, (var + EPS).rsqrt()], -1)
                z = ((x[n, :L].reshape(L, G, -1) - mean[:, None]) * stats[n, :, 1, None]).reshape(L, C) * w + bias
                y[n, :L] = other(z) if st["gate"] is None else z * other(st["gate"][n, :L].double())
        return dict(y=y, stats=stats)
    # the gradient of a sum over the rows that count, with the given statistics
    on = torch.arange(S, device=x.device)[None] < torch.tensor(lengths, device=x.device)[:, None]
    clean = lambda u: u.double().masked_fill(~on[..., None], 0.0)
    mean, rstd = (st["stats"][..., i].double().repeat_interleave(C // G, 1)[:, None] for i in (0, 1))
    hat = clean((x - mean) * rstd)
    z, dy = hat * w + bias, clean(st["dy"])
    with torch.enable_grad():
        at = (z if st["gate"] is None else clean(st["gate"])).detach().requires_grad_()
        a = other(at)
        slope, = torch.autograd.grad(a.sum(), at)
    dz = dy * slope if st["gate"] is None else dy * a.detach()
    dgate = None if st["gate"] is None else dy * z * slope
    count = torch.tensor([max(n, 1) * (C // G) for n in lengths], dtype=torch.float64, device=x.device)[:, None, None]
    per = lambda u: (u.sum(1).reshape(N, 1, G, -1).sum(-1) / count).repeat_interleave(C // G, 2)
    dx = clean(rstd * (dz * w - per(dz * w) - hat * per(dz * w * hat)))
    return dict(dx=dx, dweight=(dz * hat).sum((0, 1)), dbias=dz.sum((0, 1)), dgate=dgate)


def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "la_step":
        return _exact_step(st)
    return (_exact_la if st["op"].startswith("la") else _exact_gn)(st, st["op"].endswith("bwd"))


# ---- what a pass cannot do without -------------------------------------------------------------------------


def work(case):
    c = case
    e = {"bf16": 2, "f32": 4}
    if c["op"] == "la_step":
        rows, s = c["B"] * c["H"], c["dk"] * c["dv"]
        io = c["B"] * (c["H"] + c["Hkv"]) * (c["dk"] + c["dv"]) * e[c["dtype"]]
        return {"bytes": rows * s * 8 + io, "flops": rows * s * 5}
    if c["op"].startswith("la"):
        tokens, heads = c["B"] * c["T"], c["H"] * (c["dk"] + c["dv"])
        shared, s = c["Hkv"] * (c["dk"] + c["dv"]), c["B"] * c["H"] * c["dk"] * c["dv"] * 4
        per = c["H"] * c["dk"] * c["dv"] * tokens
        if c["op"] == "la_fwd":
            return {"bytes": tokens * (heads + shared) * e[c["dtype"]] + s * (2 if c["start"] else 1), "flops": 4 * per}
        return {"bytes": tokens * (heads + 2 * shared + c["H"] * c["dk"]) * e[c["dtype"]] + s * (3 if c["start"] else 0),
                "flops": 10 * per}
    n = c["N"] * c["S"] * c["G"] * c["cg"]
    x, y = e[c["dtype"]], e[c["out"]]
    if c["op"] == "gn_fwd":
        return {"bytes": n * (x + y + (x if c["gate"] else 0)), "flops": n * 12}
    return {"bytes": n * (2 * x + y + (2 * x if c["gate"] else 0)), "flops": n * 24}
