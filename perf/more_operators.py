"""Workloads of the operators between two recurrences: the INT8 matrix product with scales for each
token and channel (la_linear_*), and the norms after and before a block with its gate and residual
scale (la_gate_norm_*).

`run` makes one pass through an operator: with `own` false in elementary torch operations in
32 bits (64 for sums over tokens), with `own` true by the library's calls.
"""
import torch

own = False


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token of one conversation through the q, k, v and gate projection of 16 heads of 128: latency
        dict(name="linear_token", op="linear_fwd", M=1, K=2048, N=8192, bias=False, type="bf16"),
        # one token of the serving batch that the decode benchmark has, through the same projection
        dict(name="linear_decode_b256", op="linear_fwd", M=256, K=2048, N=8192, bias=False, type="bf16"),
        # a ragged batch of tokens, an odd number of channels, bias, FP32 output
        dict(name="linear_ragged_f32", op="linear_fwd", M=777, K=1040, N=2305, bias=True, type="f32"),
        # packed prompts of the serving prefill, to the convolution's channels
        dict(name="linear_prefill_packed", op="linear_fwd", M=40686, K=4096, N=2304, bias=False, type="bf16"),
        # training step at the long-sequence shape (8 sequences of 4096), output projection, weight gradients in FP32
        dict(name="linear_train_b8t4096", op="linear_train", M=32768, K=2048, N=2048, bias=True, type="bf16", dw="f32"),
        # training in full precision at an odd length (2 sequences of 1000): 8 heads' q, k, v of 64 and their gates
        dict(name="linear_train_f32_t1000", op="linear_train", M=2000, K=512, N=1552, bias=True, type="f32", dw="f32"),
        # the gated output norm of a few interactive conversations' tokens, codes for the output projection: latency
        dict(name="gate_token_b4", op="gate_fwd", rows=4, d=2048, head=128, act="silu", first=False, post=True,
             residual=False, pre=False, codec="int8", type="bf16"),
        # the gated output norm of packed prompts, 32 heads of 128
        dict(name="gate_prefill_packed", op="gate_fwd", rows=40686, d=4096, head=128, act="silu", first=False, post=True,
             residual=False, pre=False, codec="int8", type="bf16"),
        # behind the output projection: the block's norm, residual scale and addition, the next block's norm, codes
        dict(name="join_prefill_packed", op="gate_fwd", rows=40686, d=2048, head=0, act="none", first=False, post=True,
             residual=True, pre=True, codec="int8", type="bf16"),
        # the same in a training step, forward and backward
        dict(name="join_train_32768", op="gate_train", rows=32768, d=2048, head=0, act="none", first=False, post=True,
             residual=True, pre=True, codec="none", type="bf16"),
        # the gated output norm in a training step, 16 heads of 128 that share the norm's weight
        dict(name="gate_train_32768", op="gate_train", rows=32768, d=2048, head=128, act="sigmoid", first=False, post=True,
             residual=False, pre=False, codec="none", type="bf16"),
        # training in full precision: the gate before the norm, then residual and the next norm
        dict(name="gate_first_train_f32_t1000", op="gate_train", rows=2000, d=512, head=0, act="silu", first=True, post=True,
             residual=True, pre=True, codec="none", type="f32"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["linear_fwd", "linear_fwd", "linear_train", "gate_fwd", "gate_train"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("linear"):
        train = op == "linear_train"
        K, N = 16 * _log(rng, 8, 256 if train else 1024), _log(rng, 48, 4096 if train else 16384)
        most = (32768 * 2048 * 2048 if train else 40686 * 4096 * 2304) // (K * N) // (2 if kind == "f32" else 1)
        case = dict(op=op, M=_log(rng, 1, max(1, min(32768 if train else 40686, most))), K=K, N=N,
                    bias=rng.random() < 0.5, type=kind)
        return dict(case, dw=rng.choice(["f32", "bf16"])) if train else case
    head = rng.choice([0, 0, 16, 32, 64, 128, 256, 512])
    d = head * _log(rng, 1, 4096 // head) if head else 8 * _log(rng, 8, 1024)
    train = op == "gate_train"
    most = (32768 * 2048 if train else 40686 * 4096) // d // (2 if kind == "f32" else 1)
    act = rng.choice(["none", "silu", "silu", "sigmoid"])
    return dict(op=op, rows=_log(rng, 1, max(1, min(32768 if train else 40686, most))), d=d, head=head, act=act,
                first=act != "none" and rng.random() < 0.3, post=rng.random() < 0.8, residual=rng.random() < 0.5,
                pre=rng.random() < 0.5, codec="none" if train else rng.choice(["none", "int8", "e4m3"]), type=kind)


# ----------------------------------------------------------------------------------- inputs
def _type(case, key="type"):
    return torch.bfloat16 if case[key] == "bf16" else torch.float32


def _rows_to_int8(v):
    """Codes and scale of each row, as the norm in front of the product or a weight's layout makes them."""
    scale = v.abs().amax(1) / 127
    return torch.round(v / scale[:, None]).clamp(-127, 127).to(torch.int8), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    t, f32 = _type(case), torch.float32

    def normal(*shape, scale=1.0, dtype=t):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    s = dict(case=case)
    if case["op"].startswith("linear"):
        M, N, K = case["M"], case["N"], case["K"]
        s["xc"], s["xs"] = _rows_to_int8(normal(M, K, dtype=f32))
        s["wc"], s["ws"] = _rows_to_int8(normal(N, K, scale=K ** -0.5, dtype=f32))
        s["bias"] = normal(N, scale=0.1, dtype=f32) if case["bias"] else None
        if case["op"] == "linear_train":
            # a loss's gradient: small, and a few times larger at some tokens than at others
            s["dy"] = (normal(M, N, dtype=f32) * torch.exp(normal(M, 1, dtype=f32)) * 1e-4).to(t)
        return s
    rows, d = case["rows"], case["d"]
    s.update(x=normal(rows, d, scale=0.7), eps=1e-6,
             z=normal(rows, d, scale=1.5) if case["act"] != "none" else None,
             w_post=normal(case["head"] or d, scale=0.2, dtype=f32) + 1.0 if case["post"] else None,
             alpha=normal(d, scale=0.05, dtype=f32) + 0.3 if case["residual"] else None,
             residual=normal(rows, d, scale=3.0) if case["residual"] else None,
             w_pre=normal(d, scale=0.2, dtype=f32) + 1.0 if case["pre"] else None)
    if case["op"] == "gate_train":
        s.update(dy=normal(rows, d, scale=0.5), dh=normal(rows, d, scale=0.5) if case["residual"] else None)
    return s


# --------------------------------------------------------------------------------- plain forms
def _plain_linear(s):
    case, t = s["case"], _type(s["case"])
    xc, wc = s["xc"].float(), s["wc"].float()
    y = (xc @ wc.t()) * s["xs"][:, None] * s["ws"]
    if s["bias"] is not None:
        y = y + s["bias"]
    out = dict(y=y.to(t))
    if case["op"] == "linear_train":
        dy = s["dy"].float()
        out["dx"] = ((dy * s["ws"]) @ wc).to(t)
        out["dweight"] = ((dy * s["xs"][:, None]).t() @ xc).to(_type(case, "dw"))
        out["dbias"] = dy.sum(0, dtype=torch.float64).float()
    return out


def _gate(z, act):
    """The gate and its derivative."""
    sig = 1 / (1 + torch.exp(-z))
    if act == "sigmoid":
        return sig, sig * (1 - sig)
    return z * sig, sig * (1 + z * (1 - sig))


def _round_e4m3(v):
    """The nearest value of 8 bits with 4 of exponent and 3 of mantissa, ties to even, |v| <= 448."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    # log2 may round up at a power of two's lower neighbour: there the finer step applies
    step = torch.where(v.abs().clamp(min=2.0 ** -6) < step * 8, step / 2, step)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _plain_gate(s):
    case, t = s["case"], _type(s["case"])
    head = case["head"] or case["d"]
    heads = lambda v: v.unflatten(-1, (-1, head))  # noqa: E731
    x = s["x"].float()
    gate, slope = _gate(s["z"].float(), case["act"]) if s["z"] is not None else (None, None)
    u = x * gate if case["first"] else x
    n = u
    if case["post"]:
        rms = torch.sqrt((heads(u) * heads(u)).mean(-1, keepdim=True) + s["eps"])
        unit = heads(u) / rms
        n = (unit * s["w_post"]).flatten(-2)
    p = n * gate if gate is not None and not case["first"] else n
    v = s["residual"].float() + s["alpha"] * p if case["residual"] else p
    h = v.to(t)  # stored, and the next norm reads what is stored
    out = dict(h=h) if case["residual"] or case["pre"] else {}
    if case["pre"]:
        hf = h.float()
        row = torch.sqrt((hf * hf).mean(-1, keepdim=True) + s["eps"])
        unit_row = hf / row
        v = unit_row * s["w_pre"]
    if case["codec"] == "none":
        out["y"] = v.to(t)
    else:
        scale = v.abs().amax(-1, keepdim=True) / (127.0 if case["codec"] == "int8" else 448.0)
        scale = torch.where(scale == 0, torch.ones_like(scale), scale)
        code = torch.round(v / scale).clamp(-127, 127) if case["codec"] == "int8" else _round_e4m3(v / scale)
        out.update(y=(code * scale).to(t), scales=scale.squeeze(-1))
    if case["op"] != "gate_train":
        return out
    g = s["dy"].float()
    if case["pre"]:
        out["dw_pre"] = (g * unit_row).sum(0, dtype=torch.float64).float()
        g = g * s["w_pre"]
        g = (g - unit_row * (g * unit_row).mean(-1, keepdim=True)) / row
    if s["dh"] is not None:
        g = g + s["dh"].float()
    if case["residual"]:
        out["dres"] = g.to(t)
        out["dalpha"] = (g * p).sum(0, dtype=torch.float64).float()
        g = g * s["alpha"]
    if gate is not None and not case["first"]:
        out["dz"] = (g * n * slope).to(t)
        g = g * gate
    if case["post"]:
        g = heads(g)
        out["dw_post"] = (g * unit).sum((0, 1), dtype=torch.float64).float()
        g = g * s["w_post"]
        g = ((g - unit * (g * unit).mean(-1, keepdim=True)) / rms).flatten(-2)
    if case["first"]:
        out["dz"] = (g * x * slope).to(t)
        g = g * gate
    out["dx"] = g.to(t)
    return out


# ------------------------------------------------------------------------------ the library's calls
def _own_linear(s, la):
    case, t = s["case"], _type(s["case"])
    code = {torch.bfloat16: la.LA_BF16, torch.float32: la.LA_F32}
    train = case["op"] == "linear_train"
    dwt = _type(case, "dw") if train else torch.float32
    M, N, K = case["M"], case["N"], case["K"]
    cfg = la.LinearConfig(M=M, N=N, K=K, x_dtype=code[t], out_dtype=code[t], w_dtype=la.LA_F32, dw_dtype=code[dwt])
    dev = s["xc"].device
    y = torch.empty(M, N, dtype=t, device=dev)
    la.la_linear_fwd(cfg, s["xc"], s["xs"], s["wc"], s["ws"], s["bias"], y)
    out = dict(y=y)
    if train:
        dx = torch.empty(M, K, dtype=t, device=dev)
        dweight = torch.empty(N, K, dtype=dwt, device=dev)
        dbias = torch.empty(N, device=dev)
        n = la.la_linear_bwd_workspace_bytes(cfg)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        la.la_linear_bwd(cfg, s["xc"], s["xs"], s["wc"], s["ws"], s["dy"], dx, dweight, dbias, ws, n)
        out.update(dx=dx, dweight=dweight, dbias=dbias)
    return out


def _own_gate(s, la):
    case, x = s["case"], s["x"]
    code = la.LA_BF16 if case["type"] == "bf16" else la.LA_F32
    codec = {"none": la.LA_QDQ_NONE, "int8": la.LA_QDQ_INT8_GROUP, "e4m3": la.LA_QDQ_E4M3_TILE}[case["codec"]]
    act = {"none": la.LA_GATE_NONE, "silu": la.LA_GATE_SILU, "sigmoid": la.LA_GATE_SIGMOID}[case["act"]]
    rows, d = case["rows"], case["d"]
    cfg = la.GateNormConfig(rows=rows, d=d, head=case["head"], eps=s["eps"], gate=act, gate_first=int(case["first"]),
                            post=int(case["post"]), pre=int(case["pre"]), qdq=codec, group=0, x_dtype=code,
                            out_dtype=code)
    h = torch.empty_like(x) if case["residual"] or case["pre"] else None
    y = torch.empty_like(x)
    codes = scales = None
    if case["codec"] != "none":
        codes = torch.empty(rows, d, dtype=torch.uint8, device=x.device)
        scales = torch.empty(rows, device=x.device)
    la.la_gate_norm_fwd(cfg, x, s["z"], s["w_post"], s["alpha"], s["residual"], s["w_pre"], h, y, codes, scales)
    out = dict(y=y)
    if h is not None:
        out["h"] = h
    if scales is not None:  # the codes come back as the values that they stand for: y
        out["scales"] = scales
    if case["op"] == "gate_train":
        empty = lambda like, wanted=True: torch.empty_like(like) if wanted and like is not None else None  # noqa: E731
        grads = dict(dx=empty(x), dz=empty(s["z"]), dres=empty(s["residual"]), dw_post=empty(s["w_post"]),
                     dalpha=empty(s["alpha"]), dw_pre=empty(s["w_pre"]))
        n = la.la_gate_norm_bwd_workspace_bytes(cfg)
        ws = torch.empty(n, dtype=torch.uint8, device=x.device)
        la.la_gate_norm_bwd(cfg, x, s["z"], s["w_post"], s["alpha"], h if case["pre"] else None, s["w_pre"], s["dy"],
                            s["dh"], *grads.values(), ws, n)
        out.update((k, v) for k, v in grads.items() if v is not None)
    return out


def run(state):
    linear = state["case"]["op"].startswith("linear")
    if own:
        import quantized_state_qat_amd as la
        return (_own_linear if linear else _own_gate)(state, la)
    return (_plain_linear if linear else _plain_gate)(state)


# ------------------------------------------------------------------------------------- work
def work(case):
    es = 2 if case["type"] == "bf16" else 4
    if case["op"].startswith("linear"):
        M, N, K = case["M"], case["N"], case["K"]
        w = dict(bytes=M * K + N * K + 4 * (M + N) + M * N * es + (4 * N if case["bias"] else 0), flops=2 * M * N * K)
        if case["op"] == "linear_train":
            # dy in; dx, dweight and dbias out
            w["bytes"] += M * N * es + M * K * es + N * K * (2 if case["dw"] == "bf16" else 4) + 4 * N
            w["flops"] += 4 * M * N * K
        return w
    rows, d = case["rows"], case["d"]
    e, gated = rows * d, case["act"] != "none"
    stored = case["residual"] or case["pre"]
    w = dict(bytes=e * es * (2 + gated + case["residual"] + stored) + 4 * d * (case["post"] + case["residual"] + case["pre"]),
             flops=e * (4 * case["post"] + 6 * gated + 2 * case["residual"] + 4 * case["pre"]))
    if case["codec"] != "none":
        w["bytes"] += e + 4 * rows
        w["flops"] += 4 * e
    if case["op"] == "gate_train":
        # dy and dh in; dx, dz and dres out (x, z and h are there from the forward, read once)
        w["bytes"] += e * es * (2 + gated + 2 * case["residual"]) + 4 * d * (case["post"] + case["residual"] + case["pre"])
        w["flops"] += e * (10 * case["post"] + 8 * gated + 4 * case["residual"] + 10 * case["pre"])
    return w


# ---------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64 = {k: v.double() for k, v in s.items() if torch.is_tensor(v)}
    if case["op"].startswith("linear"):
        x, w = f64["xc"] * f64["xs"].unsqueeze(1), f64["wc"] * f64["ws"].unsqueeze(1)
        out = dict(y=torch.mm(x, w.T.contiguous()))
        if case["bias"]:
            out["y"] += f64["bias"]
        if case["op"] == "linear_train":
            out["dx"] = torch.mm(f64["dy"], w)
            out["dweight"] = torch.mm(f64["dy"].T.contiguous(), x)
            out["dbias"] = f64["dy"].sum(0)
        return out
    rows, d, t = case["rows"], case["d"], _type(case)
    width = case["head"] or d
    out = {}
    x = f64["x"]
    act = dact = None
    if case["act"] != "none":
        e = torch.sigmoid(f64["z"])
        act = e if case["act"] == "sigmoid" else f64["z"] * e
        dact = e - e * e if case["act"] == "sigmoid" else e + f64["z"] * (e - e * e)
    inner = x * act if case["first"] else x
    if case["post"]:
        inv = (inner.square().reshape(rows, -1, width).sum(2) / width + s["eps"]).rsqrt().repeat_interleave(width, 1)
        wide = f64["w_post"].repeat(d // width)
        normed = inner * inv * wide
    else:
        normed = inner
    outer = normed if act is None or case["first"] else normed * act
    total = f64["residual"] + f64["alpha"] * outer if case["residual"] else outer
    # what is stored is rounded to its type, and the norm reads the stored values
    held = total.float().to(t).double()
    if case["residual"] or case["pre"]:
        out["h"] = total
    if case["pre"]:
        inv_row = (held.square().sum(1, keepdim=True) / d + s["eps"]).rsqrt()
        total = held * inv_row * f64["w_pre"]
    if case["codec"] == "none":
        out["y"] = total
    else:
        step = total.abs().max(1, keepdim=True).values / (127 if case["codec"] == "int8" else 448)
        step[step == 0] = 1
        q = total / step
        if case["codec"] == "int8":
            q = q.round()
        else:
            _, ex = torch.frexp(q)
            ulp = torch.ldexp(torch.ones_like(q), (ex - 4).clamp(min=-9))
            q = (q / ulp).round() * ulp
        out.update(y=q * step, scales=step[:, 0])
    if case["op"] != "gate_train":
        return out
    grad = f64["dh"] if case["residual"] else torch.zeros_like(x)
    if case["pre"]:
        out["dw_pre"] = (f64["dy"] * held * inv_row).sum(0)
        c = f64["dy"] * f64["w_pre"]
        grad = grad + c * inv_row - held * ((c * held).sum(1, keepdim=True) / d * inv_row ** 3)
    else:
        grad = grad + f64["dy"]
    if case["residual"]:
        out["dres"] = grad
        out["dalpha"] = (grad * outer).sum(0)
        grad = grad * f64["alpha"]
    if act is not None and not case["first"]:
        out["dz"] = grad * normed * dact
        grad = grad * act
    if case["post"]:
        out["dw_post"] = (grad * inner * inv).sum(0).reshape(-1, width).sum(0)
        c = grad * wide
        mean = (c * inner).reshape(rows, -1, width).sum(2).repeat_interleave(width, 1) / width
        grad = c * inv - inner * (mean * inv ** 3)
    if case["first"]:
        out["dz"] = grad * x * dact
        grad = grad * act
    out["dx"] = grad
    return out
