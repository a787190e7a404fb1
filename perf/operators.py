"""Workloads of the layer operators around the recurrence: the short causal convolution (la_conv_*),
the selective scan (la_scan_*) and the residual-adding RMS norm with 8-bit output (la_norm_*).

`run` makes one pass through an operator: with `own` false in elementary torch operations in
32 bits (64 for cumulated decays and sums over tokens), with `own` true by the library's calls.
"""
import torch

own = False

CHUNK = 64  # tokens of one chunk of the plain scan


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one generated token for a full serving batch, states in a slot pool
        dict(name="conv_step_b256", op="conv_step", B=256, C=2304, W=4, type="bf16"),
        # serving prefill of packed prompts of 0 to about 1200 tokens, conversation states carried
        dict(name="conv_prefill_packed", op="conv_fwd", packed=True, B=64, T=40686, C=2304, W=4, type="bf16"),
        # training step at the long-sequence shape, forward and backward
        dict(name="conv_train_b8t4096", op="conv_train", B=8, T=4096, C=2304, W=4, type="bf16"),
        # one token of a few interactive conversations: latency
        dict(name="scan_step_b4", op="scan_step", B=4, H=16, G=1, d_k=128, d_v=128, type="bf16"),
        # one token of the serving batch that the decode benchmark has
        dict(name="scan_step_b256", op="scan_step", B=256, H=16, G=1, d_k=128, d_v=128, type="bf16"),
        # one long prompt: few heads and sequences, many tokens
        dict(name="scan_prefill_t32768", op="scan_fwd", packed=False, B=1, T=32768, H=32, G=1, d_k=128, d_v=64, type="bf16"),
        # packed prompts of ragged lengths, conversation states carried
        dict(name="scan_prefill_packed", op="scan_fwd", packed=True, B=64, T=40686, H=16, G=1, d_k=128, d_v=128, type="bf16"),
        # training step at the long-sequence shape
        dict(name="scan_train_b8t4096", op="scan_train", B=8, T=4096, H=16, G=1, d_k=128, d_v=128, type="bf16"),
        # training in full precision at an odd length, two groups of heads
        dict(name="scan_train_f32_t1000", op="scan_train", B=2, T=1000, H=8, G=2, d_k=64, d_v=64, type="f32"),
        # one token's rows, E4M3 output with one scale a row for the next product
        dict(name="norm_step_e4m3_b256", op="norm_fwd", rows=256, d=2048, codec="e4m3", group=0, type="bf16"),
        # a prompt's rows, INT8 output with a scale for each group of 64
        dict(name="norm_prefill_int8", op="norm_fwd", rows=40686, d=4096, codec="int8", group=64, type="bf16"),
        # training step of the norm, forward and backward
        dict(name="norm_train_32768", op="norm_train", rows=32768, d=2048, codec="none", group=0, type="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["conv_step", "conv_fwd", "conv_train", "scan_step", "scan_fwd", "scan_train", "norm_fwd", "norm_train"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        d = 8 * _log(rng, 8, 1024)
        rows = _log(rng, 1, max(1, min(40686, 40686 * 4096 // d // (2 if kind == "f32" else 1))))
        codec = rng.choice(["none", "int8", "e4m3"])
        fits = [0] + [g for g in (16, 32, 64, 128) if d % g == 0]
        return dict(op=op, rows=rows, d=d, codec=codec, group=rng.choice(fits) if codec != "none" else 0, type=kind)
    if op.startswith("conv"):
        C, W = 8 * _log(rng, 8, 1024), rng.choice([2, 3, 4])
        if op == "conv_step":
            return dict(op=op, B=_log(rng, 1, 512), C=C, W=W, type=kind)
        most = 8 * 4096 * 2304 // C // (2 if kind == "f32" else 1)
        if op == "conv_fwd" and rng.random() < 0.5:
            B = _log(rng, 1, 64)
            return dict(op=op, packed=True, B=B, T=_log(rng, 2 * B, max(2 * B, min(40686, most))), C=C, W=W, type=kind)
        B = _log(rng, 1, 8)
        case = dict(op=op, B=B, T=_log(rng, 1, max(1, min(16384, most // B))), C=C, W=W, type=kind)
        return dict(case, packed=False) if op == "conv_fwd" else case
    d_k, d_v = rng.choice([16, 32, 64, 128]), rng.choice([64, 64, 128])
    G = rng.choice([1, 1, 2])
    H = G * _log(rng, 1, 16)
    case = dict(op=op, H=H, G=G, d_k=d_k, d_v=d_v, type=kind)
    if op == "scan_step":
        return dict(case, B=_log(rng, 1, max(1, 256 * 16 // H)))
    most = 8 * 4096 * 16 * 128 // (H * d_v) // (8 if kind == "f32" else 1)
    if op == "scan_fwd" and rng.random() < 0.5:
        B = _log(rng, 1, 64)
        return dict(case, packed=True, B=B, T=_log(rng, 2 * B, max(2 * B, min(40686, most))))
    B = _log(rng, 1, 8)
    case = dict(case, B=B, T=_log(rng, 1, max(1, min(32768 if op == "scan_fwd" else 4096, most // B))))
    return dict(case, packed=False) if op == "scan_fwd" else case


# ----------------------------------------------------------------------------------- inputs
def _type(case):
    return torch.bfloat16 if case["type"] == "bf16" else torch.float32


def _lengths(case, rng):
    """Sequence lengths of a packing of T tokens: ragged, one of them empty where there are many."""
    B, T = case["B"], case["T"]
    w = 0.02 + torch.rand(B, generator=rng, dtype=torch.float64)
    if B > 4:
        w[torch.randint(B, (1,), generator=rng)] = 0.0
    cu = torch.cat([torch.zeros(1, dtype=torch.float64), w.cumsum(0)]) * (T / w.sum())
    cu = cu.round().to(torch.int64)
    cu[-1] = T
    return cu


def prepare(case, seed):
    host = torch.Generator().manual_seed(int(seed))
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    t = _type(case)

    def normal(*shape, scale=1.0, dtype=t):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=gen, device="cuda") * (hi - lo) + lo

    s = dict(case=case, cu=None, longest=0)
    op = case["op"]
    if op.startswith("norm"):
        rows, d = case["rows"], case["d"]
        s.update(x=normal(rows, d), residual=normal(rows, d, scale=3.0), weight=normal(d, scale=0.2, dtype=torch.float32) + 1.0,
                 eps=1e-6)
        if op == "norm_train":
            s.update(dy=normal(rows, d, scale=0.5), dres=normal(rows, d, scale=0.5))
        return s
    B = case["B"]
    if case.get("packed"):
        cu = _lengths(case, host)
        s.update(cu=cu.to(torch.int32).cuda(), longest=int((cu[1:] - cu[:-1]).max()))
    lead = (B,) if op.endswith("_step") else (case["T"],) if case.get("packed") else (B, case["T"])
    if op.endswith("_step"):  # a pool with some free slots; slot 0 is the padding's
        n_slots = B + 1 + B // 8
        s.update(n_slots=n_slots, slots=(torch.randperm(n_slots - 1, generator=host)[:B] + 1).to(torch.int32).cuda())
    if op.startswith("conv"):
        C, W = case["C"], case["W"]
        s.update(x=normal(*lead, C), weight=uniform(-0.5, 0.5, C, W), bias=uniform(-0.5, 0.5, C))
        if op == "conv_step":
            s.update(pool=normal(s["n_slots"], W - 1, C))
        else:
            s.update(state0=normal(B, W - 1, C))
        if op == "conv_train":
            s.update(dy=normal(*lead, C), dstate_T=normal(B, W - 1, C))
        return s
    H, G, d_k, d_v = case["H"], case["G"], case["d_k"], case["d_v"]
    # x, b and c are the slices of one convolution output
    width = H * d_v + 2 * G * d_k
    xbc = normal(*lead, width)
    xbc[..., H * d_v + G * d_k:] *= d_k ** -0.5
    # softplus(dt_bias) spread over 0.001 .. 0.1, decay rates over 1 .. 16
    dt0 = torch.exp(uniform(-6.9, -2.3, H))
    s.update(xbc=xbc, dt=normal(*lead, H), A=-uniform(1.0, 16.0, H), D=normal(H, dtype=torch.float32),
             dt_bias=dt0 + torch.log(-torch.expm1(-dt0)))
    if op == "scan_step":
        s.update(pool=normal(s["n_slots"], H, d_k, d_v, scale=0.1, dtype=torch.float32))
    else:
        s.update(S0=normal(B, H, d_k, d_v, scale=0.1, dtype=torch.float32))
    if op == "scan_train":
        s.update(dy=normal(*lead, H, d_v), dS_T=normal(B, H, d_k, d_v, scale=0.1, dtype=torch.float32))
    return s


def _slices(case, xbc):
    """x [.., H, d_v], b and c [.., G, d_k] of a convolution output [.., H d_v + 2 G d_k]."""
    H, G, d_k, d_v = case["H"], case["G"], case["d_k"], case["d_v"]
    x, b, c = xbc.split([H * d_v, G * d_k, G * d_k], -1)
    return x.unflatten(-1, (H, d_v)), b.unflatten(-1, (G, d_k)), c.unflatten(-1, (G, d_k))


# --------------------------------------------------------------------------------- plain forms
def _pad(packed, cu, longest):
    """[T, ...] packed to [B, longest, ...] with zeros behind each sequence."""
    cu = cu.long()
    at = cu[:-1, None] + torch.arange(longest, device=cu.device)
    live = at < cu[1:, None]
    out = packed[at.clamp(max=max(packed.shape[0] - 1, 0))]
    return out * live.reshape(live.shape + (1,) * (packed.dim() - 1))


def _unpad(padded, cu, total):
    cu = cu.long()
    t = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    return padded[b, t - cu[b]]


def _silu(z):
    return z / (1 + torch.exp(-z))


def _conv_rows(x, state0):
    """Windows [B, T, C, W] of the rows state0 ++ x."""
    W = state0.shape[1] + 1
    return torch.cat([state0, x], 1).unfold(1, W, 1)


def _plain_conv_fwd(s):
    case, t = s["case"], _type(s["case"])
    x, state0 = s["x"].float(), s["state0"].float()
    if s["cu"] is not None:
        x = _pad(x, s["cu"], s["longest"])
        length = (s["cu"][1:] - s["cu"][:-1]).long()
    else:
        length = torch.full((case["B"],), case["T"], device=x.device)
    y = _silu((_conv_rows(x, state0) * s["weight"]).sum(-1) + s["bias"])
    if s["cu"] is not None:
        y = _unpad(y, s["cu"], case["T"])
    at = length[:, None] + torch.arange(case["W"] - 1, device=x.device)
    last = torch.cat([state0, x], 1)[torch.arange(case["B"], device=x.device)[:, None], at]
    return dict(y=y.to(t), state_T=last.to(t))


def _plain_conv_train(s):
    case, t = s["case"], _type(s["case"])
    out = _plain_conv_fwd(s)
    W, T, w = case["W"], case["T"], s["weight"]
    rows = _conv_rows(s["x"].float(), s["state0"].float())
    pre = (rows * w).sum(-1) + s["bias"]
    sig = 1 / (1 + torch.exp(-pre))
    dpre = s["dy"].float() * sig * (1 + pre * (1 - sig))
    zero = torch.zeros_like(dpre[:, :1]).expand(-1, W - 1, -1)
    drows = (torch.cat([zero, dpre, zero], 1).unfold(1, W, 1) * w.flip(1)).sum(-1)
    drows[:, T:] += s["dstate_T"].float()
    out.update(dx=drows[:, W - 1:].to(t), dstate0=drows[:, :W - 1].to(t),
               dweight=(dpre.unsqueeze(-1) * rows).sum((0, 1), dtype=torch.float64).float(),
               dbias=dpre.sum((0, 1), dtype=torch.float64).float())
    return out


def _plain_conv_step(s):
    t = _type(s["case"])
    at = s["slots"].long()
    rows = torch.cat([s["pool"][at], s["x"][:, None]], 1)
    y = _silu((rows.float() * s["weight"].t()).sum(1) + s["bias"])
    s["pool"][at] = rows[:, 1:]
    return dict(y=y.to(t), pool=s["pool"])


def _softplus(z):
    return z.clamp(min=0) + torch.log1p(torch.exp(-z.abs()))


def _chunked(v, n):
    """[B, T, ...] to [B, n, CHUNK, ...], zeros behind the last token."""
    more = n * CHUNK - v.shape[1]
    if more:
        v = torch.cat([v, v.new_zeros(v.shape[0], more, *v.shape[2:])], 1)
    return v.reshape(v.shape[0], n, CHUNK, *v.shape[2:])


def _scan_parts(case, x, z, live, b, c, A, S0):
    """The chunk form's pieces for dense [B, T] inputs in 32 bits: heads before tokens, [B, n, H, CHUNK, ..]."""
    n = max(1, -(-x.shape[1] // CHUNK))
    delta = _softplus(z) * live
    heads = lambda v: _chunked(v, n).transpose(2, 3)  # noqa: E731
    rep = case["H"] // case["G"]
    x, delta = heads(x), heads(delta.unsqueeze(-1)).squeeze(-1)
    bg, cg = heads(b), heads(c)
    cum = (delta.double() * A.double()[:, None]).cumsum(-1)
    later = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=x.device).tril()
    L = torch.exp((cum.unsqueeze(-1) - cum.unsqueeze(-2)).masked_fill(~later, float("-inf")).float())
    gram = (cg @ bg.transpose(-1, -2)).repeat_interleave(rep, 2)
    b, c = bg.repeat_interleave(rep, 2), cg.repeat_interleave(rep, 2)
    end = cum[..., -1:]
    tail = torch.exp((end - cum).float())
    head = torch.exp(cum.float())
    own_state = (b * (tail * delta).unsqueeze(-1)).transpose(-1, -2) @ x
    # carry[i, j]: decay from the end of chunk j - 1 (0: the initial state) to the start of chunk i
    total = torch.cat([torch.zeros_like(end[:, :1, :, 0]), end[..., 0].cumsum(1)], 1).transpose(1, 2)
    upto = torch.ones(n + 1, n + 1, dtype=torch.bool, device=x.device).tril()
    carry = torch.exp((total.unsqueeze(-1) - total.unsqueeze(-2)).masked_fill(~upto, float("-inf")).float())
    parts = torch.cat([S0.unsqueeze(2), own_state.transpose(1, 2)], 2)
    states = (carry @ parts.flatten(-2)).reshape(parts.shape).transpose(1, 2)  # entering chunk i; the last: S_T
    return n, x, delta, b, c, L, gram, head, tail, end, carry, states


def _scan_inputs(s):
    case = s["case"]
    x, b, c = (v.float() for v in _slices(case, s["xbc"]))
    z = s["dt"].float() + s["dt_bias"]
    live = torch.ones_like(z)
    if s["cu"] is not None:
        x, b, c, z, live = (_pad(v, s["cu"], s["longest"]) for v in (x, b, c, z, live))
    return x, b, c, z, live


def _plain_scan(s, backward):
    case, t = s["case"], _type(s["case"])
    x, b, c, z, live = _scan_inputs(s)
    T = x.shape[1]
    n, xc, delta, bc, cc, L, gram, head, tail, end, carry, states = _scan_parts(case, x, z, live, b, c, s["A"], s["S0"])
    M = gram * L * delta.unsqueeze(-2)
    S_in = states[:, :n]
    y = M @ xc + head.unsqueeze(-1) * (cc @ S_in)
    tokens = lambda v: v.transpose(2, 3).flatten(1, 2)[:, :T]  # noqa: E731
    y = tokens(y) + s["D"][:, None] * x
    if s["cu"] is not None:
        y = _unpad(y, s["cu"], case["T"])
    out = dict(y=y.to(t), S_T=states[:, n].contiguous())
    if not backward:
        return out
    G, rep = case["G"], case["H"] // case["G"]
    dy = s["dy"].float()
    dyc = _chunked(dy, n).transpose(2, 3)
    local = (cc * head.unsqueeze(-1)).transpose(-1, -2) @ dyc
    ends = torch.cat([local.transpose(1, 2), s["dS_T"].unsqueeze(2)], 2)
    dstates = (carry.transpose(-1, -2) @ ends.flatten(-2)).reshape(ends.shape).transpose(1, 2)
    dS0, dS = dstates[:, 0], dstates[:, 1:]
    dM = dyc @ xc.transpose(-1, -2)
    groups = lambda v: v.unflatten(2, (G, rep)).sum(3)  # noqa: E731
    dgram = dM * L * delta.unsqueeze(-2)
    from_state = bc @ dS                     # b_s^T dS, [.., CHUNK, d_v]
    dx = M.transpose(-1, -2) @ dyc + (tail * delta).unsqueeze(-1) * from_state
    dc = dgram @ bc + head.unsqueeze(-1) * (dyc @ S_in.transpose(-1, -2))
    db = dgram.transpose(-1, -2) @ cc + (tail * delta).unsqueeze(-1) * (xc @ dS.transpose(-1, -2))
    pairs = gram * L * dM
    inner = tail * (from_state * xc).sum(-1)
    ddelta = pairs.sum(-2) + inner
    dcum = ((pairs * delta.unsqueeze(-2)).sum(-1) + head * ((cc @ S_in) * dyc).sum(-1) - delta * ddelta).double()
    dcum[..., -1] += torch.exp(end[..., 0]) * (S_in * dS).sum((-1, -2)) + (delta * inner).sum(-1)
    drate = dcum.flip(-1).cumsum(-1).flip(-1)
    ddelta = ddelta + s["A"][:, None] * drate.float()
    ddt = tokens(ddelta.unsqueeze(-1)).squeeze(-1) / (1 + torch.exp(-z))
    out.update(dx=(tokens(dx) + s["D"][:, None] * dy).to(t), db=tokens(groups(db)).to(t), dc=tokens(groups(dc)).to(t),
               ddt=ddt.to(t), dA=(drate * delta).sum((0, 1, 3)).float(),
               dD=(dy * x).sum((0, 1, 3), dtype=torch.float64).float(),
               ddt_bias=ddt.sum((0, 1), dtype=torch.float64).float(), dS0=dS0.contiguous())
    return out


def _plain_scan_step(s):
    case, t = s["case"], _type(s["case"])
    at, rep = s["slots"].long(), case["H"] // case["G"]
    x, b, c = (v.float() for v in _slices(case, s["xbc"]))
    b, c = b.repeat_interleave(rep, 1), c.repeat_interleave(rep, 1)
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    S = s["pool"][at] * torch.exp(delta * s["A"])[..., None, None]
    S = S + (delta.unsqueeze(-1) * b).unsqueeze(-1) * x.unsqueeze(-2)
    y = (S * c.unsqueeze(-1)).sum(-2) + s["D"][:, None] * x
    s["pool"][at] = S
    return dict(y=y.to(t), pool=s["pool"])


def _round_e4m3(v):
    """The nearest value of 8 bits with 4 of exponent and 3 of mantissa, ties to even, |v| <= 448."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    # log2 may round up at a power of two's lower neighbour: there the finer step applies
    step = torch.where(v.abs().clamp(min=2.0 ** -6) < step * 8, step / 2, step)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _plain_norm_fwd(s):
    case, t = s["case"], _type(s["case"])
    h = (s["x"].float() + s["residual"].float()).to(t)
    v = h.float()
    y = v / torch.sqrt((v * v).mean(-1, keepdim=True) + s["eps"]) * s["weight"]
    if case["codec"] == "none":
        return dict(res_out=h, y=y.to(t))
    g = y.unflatten(-1, (-1, case["group"] or case["d"]))
    most = 127.0 if case["codec"] == "int8" else 448.0
    scale = g.abs().amax(-1, keepdim=True) / most
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    code = torch.round(g / scale).clamp(-127, 127) if case["codec"] == "int8" else _round_e4m3(g / scale)
    return dict(res_out=h, y=(code * scale).flatten(-2).to(t), scales=scale.squeeze(-1))


def _plain_norm_train(s):
    t = _type(s["case"])
    out = _plain_norm_fwd(s)
    h, dy = out["res_out"].float(), s["dy"].float()
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + s["eps"])
    g = dy * s["weight"]
    dx = s["dres"].float() + r * (g - h * r * r * (g * h).mean(-1, keepdim=True))
    out.update(dx=dx.to(t), dweight=(dy * h * r).sum(0, dtype=torch.float64).float())
    return out


# ------------------------------------------------------------------------------ the library's calls
def _own_conv(s, la):
    case, t = s["case"], _type(s["case"])
    code = la.LA_BF16 if case["type"] == "bf16" else la.LA_F32
    cfg = la.ConvConfig(B=case["B"], T=case.get("T", 1), C=case["C"], width=case["W"], act=la.LA_ACT_SILU, x_dtype=code)
    y = torch.empty_like(s["x"])
    if case["op"] == "conv_step":
        la.la_conv_step(cfg, s["x"], s["weight"], s["bias"], s["pool"], y, slots=s["slots"], n_slots=s["n_slots"])
        return dict(y=y, pool=s["pool"])
    state_T = torch.empty_like(s["state0"])
    la.la_conv_fwd(cfg, s["x"], s["weight"], s["bias"], s["state0"], y, state_T, cu_seqlens=s["cu"])
    out = dict(y=y, state_T=state_T)
    if case["op"] == "conv_train":
        dx, dstate0 = torch.empty_like(s["x"]), torch.empty_like(s["state0"])
        dweight, dbias = torch.empty_like(s["weight"]), torch.empty_like(s["bias"])
        n = la.la_conv_bwd_workspace_bytes(cfg)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        la.la_conv_bwd(cfg, s["x"], s["weight"], s["bias"], s["state0"], s["dy"], s["dstate_T"], dx, dweight, dbias,
                       dstate0, ws, n)
        out.update(dx=dx, dstate0=dstate0, dweight=dweight, dbias=dbias)
    return out


def _own_scan(s, la):
    case, t = s["case"], _type(s["case"])
    code = la.LA_BF16 if case["type"] == "bf16" else la.LA_F32
    width = s["xbc"].shape[-1]
    cfg = la.ScanConfig(B=case["B"], T=case.get("T", 1), H=case["H"], G=case["G"], d_k=case["d_k"], d_v=case["d_v"],
                        softplus=1, x_dtype=code, dt_dtype=code, out_dtype=code, ld_x=width, ld_b=width, ld_c=width)
    x, b, c = _slices(case, s["xbc"])
    y = torch.empty(x.shape, dtype=t, device="cuda")
    if case["op"] == "scan_step":
        la.la_scan_step(cfg, x, s["dt"], s["A"], b, c, s["D"], s["dt_bias"], s["pool"], y, slots=s["slots"],
                        n_slots=s["n_slots"])
        return dict(y=y, pool=s["pool"])
    S_T = torch.empty_like(s["S0"])
    n = la.la_scan_workspace_bytes(cfg)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    la.la_scan_fwd(cfg, x, s["dt"], s["A"], b, c, s["D"], s["dt_bias"], s["S0"], y, S_T, ws, n, cu_seqlens=s["cu"])
    out = dict(y=y, S_T=S_T)
    if case["op"] == "scan_train":
        dx, db, dc = _slices(case, torch.empty_like(s["xbc"]))
        ddt, dS0 = torch.empty_like(s["dt"]), torch.empty_like(s["S0"])
        dA, dD, ddt_bias = (torch.empty_like(s["A"]) for _ in range(3))
        n = la.la_scan_bwd_workspace_bytes(cfg)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        la.la_scan_bwd(cfg, x, s["dt"], s["A"], b, c, s["D"], s["dt_bias"], s["S0"], s["dy"], s["dS_T"], dx, ddt, dA,
                       db, dc, dD, ddt_bias, dS0, ws, n)
        out.update(dx=dx, db=db, dc=dc, ddt=ddt, dA=dA, dD=dD, ddt_bias=ddt_bias, dS0=dS0)
    return out


def _own_norm(s, la):
    case, t = s["case"], _type(s["case"])
    code = la.LA_BF16 if case["type"] == "bf16" else la.LA_F32
    codec = {"none": la.LA_QDQ_NONE, "int8": la.LA_QDQ_INT8_GROUP, "e4m3": la.LA_QDQ_E4M3_TILE}[case["codec"]]
    cfg = la.NormConfig(rows=case["rows"], d=case["d"], eps=s["eps"], qdq=codec, group=case["group"], x_dtype=code,
                        out_dtype=code)
    res_out, y = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    codes = scales = None
    if case["codec"] != "none":
        codes = torch.empty(case["rows"], case["d"], dtype=torch.uint8, device="cuda")
        scales = torch.empty(case["rows"], case["d"] // (case["group"] or case["d"]), device="cuda")
    la.la_norm_fwd(cfg, s["x"], s["residual"], s["weight"], res_out, y, codes, scales)
    out = dict(res_out=res_out, y=y)
    if scales is not None:  # the codes come back as the values that they stand for: y
        out["scales"] = scales
    if case["op"] == "norm_train":
        dx, dweight = torch.empty_like(s["x"]), torch.empty_like(s["weight"])
        n = la.la_norm_bwd_workspace_bytes(cfg)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        la.la_norm_bwd(cfg, res_out, s["weight"], s["dy"], s["dres"], dx, dweight, ws, n)
        out.update(dx=dx, dweight=dweight)
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        import quantized_state_qat_amd as la
        return (_own_conv if op.startswith("conv") else _own_scan if op.startswith("scan") else _own_norm)(state, la)
    if op == "conv_step":
        return _plain_conv_step(state)
    if op == "conv_fwd":
        return _plain_conv_fwd(state)
    if op == "conv_train":
        return _plain_conv_train(state)
    if op == "scan_step":
        return _plain_scan_step(state)
    if op == "norm_fwd":
        return _plain_norm_fwd(state)
    if op == "norm_train":
        return _plain_norm_train(state)
    return _plain_scan(state, op == "scan_train")


# ------------------------------------------------------------------------------------- work
def work(case):
    es = 2 if case["type"] == "bf16" else 4
    op = case["op"]
    if op.startswith("norm"):
        n = case["rows"] * case["d"]
        b, f = 4 * n * es + 4 * case["d"], 6 * n
        if case["codec"] != "none":
            b += n + 4 * (n // (case["group"] or case["d"]))
            f += 4 * n
        if op == "norm_train":
            b += 4 * n * es + 4 * case["d"]
            f += 12 * n
        return dict(bytes=b, flops=f)
    B = case["B"]
    tokens = B if op.endswith("_step") else case["T"] if case.get("packed") else B * case["T"]
    if op.startswith("conv"):
        n, st = tokens * case["C"], B * (case["W"] - 1) * case["C"]
        par = 4 * case["C"] * (case["W"] + 1)
        if op == "conv_train":
            return dict(bytes=5 * n * es + 4 * st * es + 2 * par, flops=n * (6 * case["W"] + 16))
        return dict(bytes=2 * n * es + 2 * st * es + par, flops=n * (2 * case["W"] + 5))
    H, G, N, P = case["H"], case["G"], case["d_k"], case["d_v"]
    st = B * H * N * P
    io, bc = tokens * H * P, tokens * G * N
    fwd = dict(bytes=(2 * io + 2 * bc + tokens * H) * es + 8 * st + 12 * H,
               flops=tokens * H * (4 * N * P) + 2 * io)
    if op == "scan_step":
        return fwd
    fwd["flops"] += CHUNK * tokens * (G * N + H * P)  # half of the pairs within a chunk
    if op == "scan_train":
        fwd["bytes"] += (3 * io + 4 * bc + 2 * tokens * H) * es + 12 * st + 24 * H
        fwd["flops"] += tokens * H * 8 * N * P + CHUNK * tokens * (2 * H * N + 2 * H * P + G * N)
    return fwd


# ---------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    def norm(s):
        case, t = s["case"], _type(s["case"])
        # what is stored in res_out is rounded to its type, and the norm reads the stored values
        res = (s["x"].double() + s["residual"].double())
        h = res.float().to(t).double() if t is torch.bfloat16 else res.float().double()
        w = s["weight"].double()
        var = h.square().sum(1) / case["d"] + s["eps"]
        n = h * w * var.rsqrt()[:, None]
        out = dict(res_out=h)
        if case["codec"] == "none":
            out["y"] = n
        else:
            width = case["group"] or case["d"]
            top = 127 if case["codec"] == "int8" else 448
            parts = n.reshape(case["rows"], case["d"] // width, width)
            sc = parts.abs().max(2).values / top
            sc[sc == 0] = 1
            q = parts / sc[:, :, None]
            if case["codec"] == "int8":
                q = q.round()
            else:
                _, e = torch.frexp(q)
                ulp = torch.ldexp(torch.ones_like(q), (e - 4).clamp(min=-9))
                q = (q / ulp).round() * ulp
            out.update(y=(q * sc[:, :, None]).reshape(n.shape), scales=sc)
        if case["op"] == "norm_train":
            dy = s["dy"].double()
            gw = dy * w
            dot = (gw * h).sum(1) / case["d"]
            out.update(dx=s["dres"].double() + gw * var.rsqrt()[:, None] - h * (dot * var.pow(-1.5))[:, None],
                       dweight=(dy * h * var.rsqrt()[:, None]).sum(0))
        return out

    def conv(s):
        case = s["case"]
        W, B = case["W"], case["B"]
        w, bias = s["weight"].double(), s["bias"].double()
        if case["op"] == "conv_step":
            at = s["slots"].long()
            rows = [s["pool"][at, j].double() for j in range(W - 1)] + [s["x"].double()]
            pre = bias + sum(rows[j] * w[:, j] for j in range(W))
            pool = s["pool"].double()
            for j in range(W - 1):
                pool[at, j] = rows[j + 1]
            return dict(y=pre * torch.sigmoid(pre), pool=pool)
        x = s["x"].double()
        if s["cu"] is not None:
            cu = s["cu"].tolist()
            seqs = [x[cu[i]:cu[i + 1]] for i in range(B)]
        else:
            seqs = [x[i] for i in range(B)]
        ys, last = [], []
        train = case["op"] == "conv_train"
        dxs, ds0, dw, dbias = [], [], torch.zeros_like(w), torch.zeros_like(bias)
        for i, xi in enumerate(seqs):
            full = torch.cat([s["state0"][i].double(), xi])
            T = xi.shape[0]
            pre = bias.expand(T, -1).clone()
            for j in range(W):
                pre += full[j:j + T] * w[:, j]
            sg = torch.sigmoid(pre)
            ys.append(pre * sg)
            last.append(full[T:])
            if train:
                dp = s["dy"][i].double() * (sg + pre * sg * (1 - sg))
                df = torch.zeros_like(full)
                df[T:] += s["dstate_T"][i].double()
                for j in range(W):
                    df[j:j + T] += dp * w[:, j]
                    dw[:, j] += (dp * full[j:j + T]).sum(0)
                dbias += dp.sum(0)
                dxs.append(df[W - 1:])
                ds0.append(df[:W - 1])
        out = dict(y=torch.cat(ys) if s["cu"] is not None else torch.stack(ys), state_T=torch.stack(last))
        if train:
            out.update(dx=torch.stack(dxs), dstate0=torch.stack(ds0), dweight=dw, dbias=dbias)
        return out

    def scan(s):
        """Token by token."""
        case = s["case"]
        H, G = case["H"], case["G"]
        x, b, c = (v.double() for v in _slices(case, s["xbc"]))
        A, D = s["A"].double(), s["D"].double()
        z = s["dt"].double() + s["dt_bias"].double()
        delta = torch.logaddexp(z, torch.zeros_like(z))
        ofgroup = torch.arange(H, device="cuda") // (H // G)
        if case["op"] == "scan_step":
            pool = s["pool"].double()
            at = s["slots"].long()
            S = pool[at] * (delta * A).exp()[:, :, None, None] + (b[:, ofgroup] * delta[:, :, None])[..., None] * x[:, :, None]
            pool[at] = S
            return dict(y=(c[:, ofgroup][:, :, None] @ S)[:, :, 0] + D[:, None] * x, pool=pool)
        B = case["B"]
        if s["cu"] is not None:
            start = s["cu"][:-1].long()
            length = (s["cu"][1:] - s["cu"][:-1]).long()
            steps, total = s["longest"], case["T"]
            y = torch.zeros(total, H, case["d_v"], dtype=torch.float64, device="cuda")
            S = s["S0"].double().clone()
            order = torch.argsort(length, descending=True)   # the sequences still running are a prefix of this order
            running = [int(k) for k in (length[None] > torch.arange(steps, device="cuda")[:, None]).sum(1)]
            Sr = S[order]
            for i in range(steps):
                k = running[i]
                t = start[order[:k]] + i
                Sk = Sr[:k]
                Sk *= (delta[t] * A).exp()[:, :, None, None]
                Sk += (b[t][:, ofgroup] * delta[t][:, :, None])[..., None] * x[t][:, :, None]
                y[t] = (c[t][:, ofgroup][:, :, None] @ Sk)[:, :, 0]
            S[order] = Sr
            return dict(y=y + D[:, None] * x, S_T=S)
        T = case["T"]
        a = (delta * A).exp()
        train = case["op"] == "scan_train"
        y = torch.empty_like(x)
        S = s["S0"].double()
        kept = {}

        def token(S, t):
            return S * a[:, t, :, None, None] + (b[:, t][:, ofgroup] * delta[:, t, :, None])[..., None] * x[:, t, :, None]

        for t in range(T):
            if train and t % 64 == 0:
                kept[t] = S
            S = token(S, t)
            y[:, t] = (c[:, t][:, ofgroup][:, :, None] @ S)[:, :, 0]
        out = dict(y=y + D[:, None] * x, S_T=S)
        if not train:
            return out
        dy = s["dy"].double()
        dS = s["dS_T"].double()
        dx, ddelta, drate = torch.empty_like(x), torch.empty_like(delta), torch.empty_like(delta)
        dbh = torch.empty(*b.shape[:2], G, case["d_k"], dtype=torch.float64, device="cuda")
        dch = torch.empty_like(dbh)
        for t0 in sorted(kept, reverse=True):
            before = [kept[t0]]
            for t in range(t0, min(T, t0 + 64)):
                before.append(token(before[-1], t))
            for t in reversed(range(t0, min(T, t0 + 64))):
                now, prev = before[t - t0 + 1], before[t - t0]
                bt, ct = b[:, t][:, ofgroup], c[:, t][:, ofgroup]
                dch[:, t] = (now @ dy[:, t, :, :, None])[..., 0].reshape(B, G, H // G, -1).sum(2)
                dS = dS + ct[..., None] * dy[:, t, :, None]
                into = (bt[:, :, None] @ dS)[:, :, 0]                       # b^T dS
                dx[:, t] = into * delta[:, t, :, None]
                dbh[:, t] = ((dS @ x[:, t, :, :, None])[..., 0] * delta[:, t, :, None]).reshape(B, G, H // G, -1).sum(2)
                drate[:, t] = (dS * prev).sum((-1, -2)) * a[:, t]
                ddelta[:, t] = (into * x[:, t]).sum(-1)
                dS = dS * a[:, t, :, None, None]
        ddelta = ddelta + A * drate
        ddt = ddelta * torch.sigmoid(z)
        out.update(dx=dx + D[:, None] * dy, db=dbh, dc=dch, ddt=ddt, dA=(drate * delta).sum((0, 1)), dD=(dy * x).sum((0, 1, 3)),
                   ddt_bias=ddt.sum((0, 1)), dS0=dS)
        return out

    s = prepare(case, seed)
    with torch.no_grad():
        return (norm if case["op"].startswith("norm") else conv if case["op"].startswith("conv") else scan)(s)
