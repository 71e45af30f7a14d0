"""What is measured of the routing with scores and groups, the residual norm, and the selective scan
with its short convolution.

Nine kinds of passes, each through the calls a user makes:
  route / route_bwd  experts of a token from its logits; the logits' gradient
  norm / norm_bwd    root-mean-square norm of x + residual, output in bf16 or in 8 bits; its gradient
  conv / conv_bwd    causal depthwise convolution of a few taps over packed prompts, with SiLU
  scan / scan_bwd    selective state space scan over packed prompts, with the gate
  step               one token for each row of a batch: the convolution, then the scan, caches in place

Definitions.
Routing: s = sigmoid(l) or softmax(l); c = s + bias chooses (l itself without a bias), the group_k groups
  with the largest sum of their group_top best c stay, of those the k largest c (ties: the lowest index;
  compared in 64 bits); w = scale s / sum s over the chosen, or scale s. l = -inf is never chosen before others.
Norm: u = x + residual, y = u weight / sqrt(mean(u^2) + eps); in 8 bits E4M3 with one scale (largest
  magnitude / 448) for each block of a row.
Convolution: p_t = bias + sum_j w[j] x_{t-W+1+j}, y = silu(p); a sequence's state is its last W - 1 inputs.
Scan: dt = softplus(delta + dt_bias), h_t = exp(dt A) h_{t-1} + dt u_t B_t, y = (C_t . h_t + skip u_t) silu(z_t).
"""
import itertools
import math

import torch

own = False

F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
EPS = 1e-6
INF = math.inf


# ------------------------------------------------------------------------- cases

def listed():
    return [
        # a few decoding rows through the layer's 896 experts: the latency of a call
        dict(name="route_decode", kind="route", T=5, E=896, k=16, score="sigmoid", groups=1, group_k=1,
             group_top=2, bias=True, renorm=True, scale=2.5, masked=0, pad=0),
        # the training step's 16384 tokens, experts in 8 groups of which 4 stay, some padded rows
        dict(name="route_train", kind="route", T=16384, E=896, k=16, score="sigmoid", groups=8, group_k=4,
             group_top=2, bias=True, renorm=True, scale=2.5, masked=0, pad=100),
        # the same step with softmax scores that are not renormalised: every logit has a gradient
        dict(name="route_softmax_bwd", kind="route_bwd", T=16384, E=896, k=16, score="softmax", groups=1,
             group_k=1, group_top=1, bias=True, renorm=False, scale=1.0, masked=0, pad=0),
        # a ragged serving batch whose norm's output goes on in 8 bits, residual stream in fp32
        dict(name="norm8_serve", kind="norm", T=777, d=5120, res="f32", out="fp8", block=128),
        # the training step's 16384 tokens of width 4096
        dict(name="norm_train", kind="norm", T=16384, d=4096, res="bf16", out="bf16", block=0),
        dict(name="norm_bwd", kind="norm_bwd", T=16384, d=4096, res="bf16", out="bf16", block=0),
        # prompts of a serving batch packed on one token axis, states resumed; inner width 2 x 4096
        dict(name="conv_packed", kind="conv", lens="1,513,0,2048,129,1000,77,4096", D=8192, W=4, silu=True,
             states=True),
        # the training step's convolution
        dict(name="conv_bwd", kind="conv_bwd", lens="4096,4096,4096,4096", D=8192, W=4, silu=True, states=False),
        # one short prompt on a small model
        dict(name="scan_short", kind="scan", lens="77", D=512, S=16, G=1, gate=True, states=False),
        # the packed prompts again
        dict(name="scan_packed", kind="scan", lens="1,513,0,2048,129,1000,77,4096", D=8192, S=16, G=1, gate=True,
             states=True),
        # the training step's scan
        dict(name="scan_bwd", kind="scan_bwd", lens="4096,4096,4096,4096", D=8192, S=16, G=1, gate=True,
             states=False),
        # a serving batch with empty rows, rows scattered over the caches
        dict(name="step_batch", kind="step", B=61, D=8192, S=16, G=1, W=4, gate=True, silu=True, pad=3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["route", "route_bwd", "norm", "norm_bwd", "conv", "conv_bwd", "scan", "scan_bwd", "scan_bwd",
                       "step"])
    if kind.startswith("route"):
        E, groups = rng.choice([(896, 1), (896, 8), (896, 7), (896, 14), (256, 8), (256, 1), (64, 1), (60, 4), (100, 1),
                                (8, 1), (160, 8), (1024, 32), (1000, 5), (384, 1)])
        size = E // groups
        group_k = rng.randint(1, max(1, groups - 1))
        k = rng.randint(1, max(1, min(32, group_k * size // 2)))
        T = _log(rng, 1, 16384)
        return dict(kind=kind, T=T, E=E, k=k, score=rng.choice(["sigmoid", "softmax"]), groups=groups, group_k=group_k,
                    group_top=rng.choice([1, 2]) if size > 1 else 1, bias=rng.random() < 0.6, renorm=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]), masked=rng.choice([0, 0, size // 8]), pad=rng.choice([0, T // 9]))
    if kind.startswith("norm"):
        d = rng.choice([64, 256, 1000, 1024, 2048, 4096, 5120, 7168, 8192, 12288])
        out = rng.choice(["bf16", "fp8"]) if kind == "norm" else "bf16"
        return dict(kind=kind, T=_log(rng, 1, 16384 * 4096 // max(d, 4096)), d=d, res=rng.choice(["bf16", "f32", "none"]),
                    out=out, block=rng.choice([64, 128, d]) if out == "fp8" else 0)
    D = rng.choice([64, 520, 1024, 1536, 2048, 4096, 5120, 8192])
    dims = dict(D=D, silu=rng.random() < 0.8)
    scan = dict(S=rng.choice([16, 16, 16, 8, 4, 12]), G=rng.choice([1, 1, 2]), gate=rng.random() < 0.8)
    if kind == "step":
        return dict(kind=kind, B=_log(rng, 1, 256), pad=rng.choice([0, 0, 1, 5]), W=rng.choice([4, 4, 3, 2]), **dims, **scan)
    most = 16384 * 8192 // D
    n = rng.choice([1, 1, 2, 4, 7])
    lens = [_log(rng, 1, max(1, min(most // n, 20000))) for _ in range(n)]
    if n > 2 and rng.random() < 0.5:
        lens[rng.randrange(n)] = 0
    case = dict(kind=kind, lens=",".join(map(str, lens)), states=rng.random() < 0.5, D=D)
    return {**case, **scan} if kind.startswith("scan") else {**case, "W": rng.choice([4, 4, 3, 2]), "silu": dims["silu"]}


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _res_bytes(case):
    return dict(none=0, bf16=2, f32=4)[case["res"]]


def work(case):
    kind = case["kind"]
    if kind == "route":
        return {"bytes": case["T"] * (4 * case["E"] + 12 * case["k"]), "flops": 4 * case["T"] * case["E"]}
    if kind == "route_bwd":
        reads = 4 * case["E"] if case["score"] == "softmax" and not case["renorm"] else 0
        return {"bytes": case["T"] * (reads + 4 * case["E"] + 16 * case["k"]), "flops": 4 * case["T"] * case["E"]}
    if kind == "norm":
        n, r = case["T"] * case["d"], _res_bytes(case)
        return {"bytes": n * (2 + 2 * r + (2 if case["out"] == "bf16" else 1 + 4 / case["block"])), "flops": 5 * n}
    if kind == "norm_bwd":
        n, r = case["T"] * case["d"], _res_bytes(case)
        return {"bytes": n * {0: 6, 2: 8, 4: 16}[r], "flops": 10 * n}
    D = case["D"]
    if kind == "step":
        rows = case["B"] - min(case["pad"], case["B"] - 1)
        gs = 2 * case["G"] * case["S"]
        return {"bytes": rows * (D * (8 * case["S"] + 4 * (case["W"] - 1) + 10 + 2 * case["gate"]) + 2 * gs),
                "flops": rows * D * (7 * case["S"] + 2 * case["W"])}
    T, N = sum(_lens(case)), len(_lens(case))
    if kind.startswith("conv"):
        st = 2 * N * (case["W"] - 1) * D if case["states"] else 0
        if kind == "conv":
            return {"bytes": 4 * T * D + 2 * st, "flops": T * D * (2 * case["W"] + 4)}
        return {"bytes": 6 * T * D + 3 * st, "flops": T * D * (6 * case["W"] + 8)}
    S, gs = case["S"], 2 * case["G"] * case["S"]
    st = 4 * N * D * S if case["states"] else 0
    if kind == "scan":
        return {"bytes": T * (D * (6 + 2 * case["gate"]) + 2 * gs) + 2 * st, "flops": T * D * 7 * S}
    return {"bytes": T * (D * (10 + 4 * case["gate"]) + 4 * gs) + 3 * st, "flops": T * D * 22 * S}


# ------------------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    kind = case["kind"]
    if kind.startswith("route"):
        return _prepare_route(case, randn, gen)
    if kind.startswith("norm"):
        return _prepare_norm(case, randn)
    D = case["D"]
    s = dict(case=case)
    if kind == "step":
        B, slots = case["B"], case["B"] + 5
        idx = torch.randperm(slots, generator=gen, device="cuda")[:B].to(torch.int32)
        idx[B - min(case["pad"], B - 1):] = -1
        s.update(idx=idx, lens=[1] * B, conv_state=randn(slots, case["W"] - 1, D).to(BF16),
                 scan_state=0.3 * randn(slots, D, case["S"]))
        _prepare_conv(s, randn, B)
        _prepare_scan(s, randn, B)
        return s
    s["lens"] = lens = _lens(case)
    T, N = sum(lens), len(lens)
    s["cu"] = torch.tensor(list(itertools.accumulate([0] + lens)), dtype=torch.int32, device="cuda")
    s.update(_bounds(lens))
    make, state = (_prepare_conv, lambda: randn(N, case["W"] - 1, D).to(BF16)) if kind.startswith("conv") else (
        _prepare_scan, lambda: 0.3 * randn(N, D, case["S"]))
    s["state_in"] = state() if case["states"] else None
    s["d_state"] = state() if case["states"] and kind.endswith("bwd") else None
    if kind.endswith("bwd"):
        s["dy"] = randn(T, D).to(BF16)
    make(s, randn, T)
    return s


def _prepare_route(case, randn, gen):
    T, E = case["T"], case["E"]
    logits = 1.5 * randn(T, E)
    if case["masked"]:  # experts that are out of service, the same for every token
        logits[:, torch.randperm(E, generator=gen, device="cuda")[:case["masked"]]] = -INF
    logits[T - case["pad"]:] = 0.0  # rows of padding: equal logits
    s = dict(case=case, logits=logits, bias=0.05 * randn(E) if case["bias"] else None)
    if case["kind"] == "route_bwd":
        s["d_w"] = randn(T, case["k"])
        s["idx"], s["w"], s["s"] = _plain_route(s).values()
    if own:
        from sparse_moe_layer_topk_gb300.route import Router
        s["router"] = Router(T, E, case["k"], score=case["score"], groups=case["groups"], group_k=case["group_k"],
                             group_top=case["group_top"], renorm=case["renorm"], scale=case["scale"])
        if case["kind"] == "route_bwd":
            s["router"].forward(s["logits"], s["bias"])
    return s


def _prepare_norm(case, randn):
    T, d = case["T"], case["d"]
    res = dict(bf16=BF16, f32=F32, none=None)[case["res"]]
    x = randn(T, d) * torch.exp(0.3 * randn(T, 1))
    s = dict(case=case, x=x.to(BF16), weight=1.0 + 0.2 * randn(d), residual=None if res is None else (2.0 * randn(T, d)).to(res))
    if case["kind"] == "norm_bwd":
        s["u"] = s["x"] if res is None else (s["x"].float() + s["residual"].float()).to(res)
        s["dy"] = randn(T, d).to(BF16)
        s["d_sum"] = None if res is None else randn(T, d).to(res)
    if own:
        from sparse_moe_layer_topk_gb300.norm import RMSNorm
        s["norm"] = RMSNorm(s["weight"], T, eps=EPS, residual_dtype=res, out=case["out"], block=case["block"],
                            backward=case["kind"] == "norm_bwd")
        if case["kind"] == "norm_bwd":
            s["norm"].forward(s["x"], s["residual"])
    return s


def _prepare_conv(s, randn, T):
    case = s["case"]
    D, W = case["D"], case["W"]
    # the inner activations are one half of a projection's rows
    s["x"] = randn(T, 2 * D).to(BF16)[:, :D]
    s["conv_w"], s["conv_b"] = W ** -0.5 * randn(D, W), 0.1 * randn(D)
    if own:
        from sparse_moe_layer_topk_gb300.scan import CausalConv
        s["conv"] = CausalConv(s["conv_w"], s["conv_b"], T, N=len(s["lens"]), silu=case["silu"],
                               backward=case["kind"] == "conv_bwd")
        if case["kind"] == "conv_bwd":
            s["conv"].forward(s["x"], s["cu"], s["state_in"])


def _prepare_scan(s, randn, T):
    case = s["case"]
    D, S, G = case["D"], case["S"], case["G"]
    # decays 1 .. S a state, time steps spread from 0.001 to 0.1: memories of 1 to 1000 tokens
    s["A"] = -torch.arange(1, S + 1, device="cuda", dtype=F32) * torch.exp(0.1 * randn(D, S))
    dt = torch.exp(torch.sigmoid(1.5 * randn(D)) * math.log(100.0) + math.log(0.001))
    s["dt_bias"] = dt + torch.log(-torch.expm1(-dt))
    s["skip"] = 1.0 + 0.1 * randn(D)
    s["delta"] = (0.5 * randn(T, D)).to(BF16)
    # B and C are slices of one projection's rows, z the second half of the rows that u came from
    bc = randn(T, 32 + 2 * G * S).to(BF16)
    s["B"] = bc[:, 32:32 + G * S].unflatten(1, (G, S))
    s["C"] = bc[:, 32 + G * S:].unflatten(1, (G, S))
    s["z"] = randn(T, 2 * D).to(BF16)[:, D:] if case["gate"] else None
    if case["kind"] != "step":
        s["u"] = torch.nn.functional.silu(randn(T, D)).to(BF16)
    if own:
        from sparse_moe_layer_topk_gb300.scan import SelectiveScan
        s["scan"] = SelectiveScan(s["A"], T, skip=s["skip"], dt_bias=s["dt_bias"], groups=G, N=len(s["lens"]),
                                  max_seqlen=max(s["lens"]), backward=case["kind"] == "scan_bwd")
        if case["kind"] == "scan_bwd":
            s["scan"].forward(s["u"], s["delta"], s["B"], s["C"], s["z"], s["cu"], s["state_in"])


def _bounds(lens):
    """Of the sequences that have tokens: their numbers, first and last tokens; each token's sequence and place."""
    n = torch.tensor(lens, device="cuda")
    start = n.cumsum(0) - n
    live = torch.nonzero(n)[:, 0]
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), n)
    return dict(live=live, first=start[live], last=(start + n - 1)[live], seq=seq,
                place=torch.arange(len(seq), device="cuda") - start[seq], start=start, n=n)


# ------------------------------------------------------------------------- plain forms

def _softmax(x):
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_route(s):
    case, logits = s["case"], s["logits"]
    T, E, k, groups = case["T"], case["E"], case["k"], case["groups"]
    score = torch.sigmoid if case["score"] == "sigmoid" else _softmax
    c = score(logits.double())  # (64 bits: two experts' values may be nearer than 32 bits tell apart)
    if s["bias"] is not None:
        c = c + s["bias"].double()
    out = logits == -INF
    value = torch.where(out, -INF, logits.double() if s["bias"] is None else c)
    if groups > 1:
        best = torch.where(out, -INF, c).view(T, groups, -1).sort(dim=-1, descending=True).values[..., :case["group_top"]]
        total = torch.where(best == -INF, 0.0, best).sum(-1)
        total = torch.where(best[..., 0] == -INF, -INF, total)
        order = total.sort(dim=-1, descending=True, stable=True).indices[:, :case["group_k"]]
        keep = torch.zeros(T, groups, dtype=torch.bool, device="cuda").scatter_(1, order, True)
        value = torch.where(keep.repeat_interleave(E // groups, 1), value, -math.inf)
        # (what is left out of the groups comes behind what is masked in them)
        rank = torch.where(keep.repeat_interleave(E // groups, 1), 0, 1)
        first = rank.sort(dim=-1, stable=True).indices
        idx = first.gather(1, value.gather(1, first).sort(dim=-1, descending=True, stable=True).indices[:, :k])
    else:
        idx = value.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    sel = score(logits).gather(1, idx)
    if not case["renorm"]:
        w = sel * case["scale"]
    elif case["score"] == "softmax":
        w = case["scale"] * _softmax(logits.gather(1, idx))
    else:
        w = case["scale"] * sel / sel.sum(1, keepdim=True)
    return {"idx": idx.int(), "w": w, "s": sel}


def _plain_route_bwd(s):
    case, idx, w, sel, g = s["case"], s["idx"].long(), s["w"], s["s"], s["d_w"]
    softmax = case["score"] == "softmax"
    if case["renorm"]:
        d = w * (g - (w * g).sum(1, keepdim=True) / case["scale"])
        d = d if softmax else d * (1.0 - sel)
    elif not softmax:
        d = g * w * (1.0 - sel)
    else:
        p = _softmax(s["logits"])
        dL = -case["scale"] * p * (g * sel).sum(1, keepdim=True)
        return {"dlogits": dL.scatter_add(1, idx, case["scale"] * sel * g)}
    return {"dlogits": torch.zeros_like(s["logits"]).scatter(1, idx, d)}


def _plain_norm(s):
    case = s["case"]
    u = s["x"].float()
    out = {}
    if s["residual"] is not None:
        u = u + s["residual"].float()
        out["sum"] = u.to(s["residual"].dtype)
    y = u * torch.rsqrt(u.square().mean(1, keepdim=True) + EPS) * s["weight"]
    if case["out"] == "bf16":
        return {**out, "y": y.to(BF16)}
    T, d = y.shape
    b = torch.nn.functional.pad(y, (0, -d % case["block"])).view(T, -1, case["block"])
    scale = b.abs().amax(-1) / 448.0
    codes = (b / torch.where(scale > 0, scale, 1.0)[..., None]).clamp(-448.0, 448.0)
    return {**out, "y8": codes.view(T, -1)[:, :d].to(torch.float8_e4m3fn), "scale": scale}


def _plain_norm_bwd(s):
    u, dy, w = s["u"].float(), s["dy"].float(), s["weight"]
    r = torch.rsqrt(u.square().mean(1, keepdim=True) + EPS)
    n = u * r
    g = dy * w
    dx = r * (g - n * (g * n).mean(1, keepdim=True))
    out = {}
    if s["d_sum"] is not None:
        dx = dx + s["d_sum"].float()
        out["d_residual"] = dx.to(s["d_sum"].dtype)
    return {"dx": dx.to(BF16), **out, "dw": (dy * n).sum(0)}


def _taps(s, W):
    """Rows of [x; states] that each token's taps read, [T, W], and those of the last states, [N, W - 1]."""
    T = len(s["seq"])
    at = s["place"][:, None] - (W - 1) + torch.arange(W, device="cuda")
    own_row = s["start"][s["seq"]][:, None] + at
    taps = torch.where(at >= 0, own_row, T + s["seq"][:, None] * (W - 1) + at + W - 1)
    end = s["n"][:, None] - (W - 1) + torch.arange(W - 1, device="cuda")
    numbers = torch.arange(len(s["n"]), device="cuda")[:, None]
    return taps, torch.where(end >= 0, s["start"][:, None] + end, T + numbers * (W - 1) + end + W - 1)


def _rows_and_states(s, W, D):
    states = s["state_in"] if s["state_in"] is not None else torch.zeros(len(s["lens"]), W - 1, D, dtype=BF16, device="cuda")
    return torch.cat([s["x"], states.flatten(0, 1)])


def _plain_conv(s):
    case = s["case"]
    W = case["W"]
    taps, last = _taps(s, W)
    ext = _rows_and_states(s, W, case["D"])
    p = s["conv_b"] + sum(s["conv_w"][:, j] * ext[taps[:, j]].float() for j in range(W))
    out = {"y": (p * torch.sigmoid(p) if case["silu"] else p).to(BF16)}
    return {**out, "state": ext[last]} if case["states"] else out


def _plain_conv_bwd(s):
    case = s["case"]
    W, T = case["W"], len(s["seq"])
    taps, last = _taps(s, W)
    ext = _rows_and_states(s, W, case["D"])
    dp = s["dy"].float()
    if case["silu"]:
        p = s["conv_b"] + sum(s["conv_w"][:, j] * ext[taps[:, j]].float() for j in range(W))
        sg = torch.sigmoid(p)
        dp = dp * sg * (1.0 + p * (1.0 - sg))
    d = torch.zeros(ext.shape, device="cuda")
    dw = torch.stack([(dp * ext[taps[:, j]].float()).sum(0) for j in range(W)], 1)
    for j in range(W):
        d.index_add_(0, taps[:, j], s["conv_w"][:, j] * dp)
    if s["d_state"] is not None:
        d.index_add_(0, last.flatten(), s["d_state"].float().flatten(0, 1))
    out = {"dx": d[:T].to(BF16), "dw": dw, "db": dp.sum(0)}
    return {**out, "d_state_in": d[T:].view(len(s["lens"]), W - 1, -1).to(BF16)} if case["states"] else out


def _recur(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling; a is 0 where a sequence starts."""
    step = 1
    while step < longest:
        b = torch.cat([b[:step], torch.addcmul(b[step:], a[step:], b[:-step])])
        a = torch.cat([a[:step], a[step:] * a[:-step]]) if 2 * step < longest else a
        step *= 2
    return b


def _wide(x, per):
    """[T, G, S] -> [T, D, S]: each group's row for its channels."""
    return x.float().repeat_interleave(per, 1)


def _parts(s):
    """Channel ranges whose states of all tokens take about 2 GB in 32 bits, none across a group's end."""
    case = s["case"]
    per = case["D"] // case["G"]
    width = max(1, min(per, (1 << 29) // (16 * max(1, sum(s["lens"])))))
    return [(g, c, min(c + width, (g + 1) * per)) for g in range(case["G"]) for c in range(g * per, (g + 1) * per, width)]


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _scan_part(s, g, lo, hi):
    """dt, u, decays, B, C and states after each token of some channels."""
    dt = _softplus(s["delta"][:, lo:hi].float() + s["dt_bias"][lo:hi])
    u, Bm, Cm = s["u"][:, lo:hi].float(), s["B"][:, g:g + 1].float(), s["C"][:, g:g + 1].float()
    a = torch.exp(dt[..., None] * s["A"][lo:hi])
    b = (dt * u)[..., None] * Bm
    if s["state_in"] is not None:
        b[s["first"]] += a[s["first"]] * s["state_in"][s["live"], lo:hi]
    cut = a.clone()
    cut[s["first"]] = 0.0
    return dt, u, a, Bm, Cm, _recur(cut, b, max(s["lens"]))


def _plain_scan(s):
    case = s["case"]
    T, D = len(s["seq"]), case["D"]
    y = torch.empty(T, D, dtype=BF16, device="cuda")
    state = s["state_in"].clone() if case["states"] else None
    for g, lo, hi in _parts(s):
        _, u, _, _, Cm, h = _scan_part(s, g, lo, hi)
        part = (h * Cm).sum(-1) + s["skip"][lo:hi] * u
        if s["z"] is not None:
            z = s["z"][:, lo:hi].float()
            part = part * z * torch.sigmoid(z)
        y[:, lo:hi] = part.to(BF16)
        if state is not None:
            state[s["live"], lo:hi] = h[s["last"]]
    return {"y": y, "state": state} if state is not None else {"y": y}


def _plain_scan_bwd(s):
    case = s["case"]
    T, D, S, G = len(s["seq"]), case["D"], case["S"], case["G"]
    new = lambda *shape: torch.empty(*shape, device="cuda")  # noqa: E731
    du, dd, dz = (torch.empty(T, D, dtype=BF16, device="cuda") for _ in range(3))
    dA, dskip, dbias = new(D, S), new(D), new(D)
    dB, dC = torch.zeros(T, G, S, device="cuda"), torch.zeros(T, G, S, device="cuda")
    d_in = s["d_state"].clone() if s["d_state"] is not None else None
    for g, lo, hi in _parts(s):
        dt, u, a, Bm, Cm, h = _scan_part(s, g, lo, hi)
        dy = s["dy"][:, lo:hi].float()
        if s["z"] is not None:
            z = s["z"][:, lo:hi].float()
            sg = torch.sigmoid(z)
            y = (h * Cm).sum(-1) + s["skip"][lo:hi] * u
            dz[:, lo:hi] = (dy * y * sg * (1.0 + z * (1.0 - sg))).to(BF16)
            dy = dy * z * sg
        x = dy[..., None] * Cm
        if d_in is not None:
            x[s["last"]] += s["d_state"][s["live"], lo:hi]
        after = torch.cat([a[1:], a[:1]])
        after[s["last"]] = 0.0
        dh = _recur(after.flip(0), x.flip(0), max(s["lens"])).flip(0)
        dC[:, g] += (h * dy[..., None]).sum(1)
        dB[:, g] += (dh * (dt * u)[..., None]).sum(1)
        before = torch.cat([h[:1], h[:-1]])
        before[s["first"]] = s["state_in"][s["live"], lo:hi] if s["state_in"] is not None else 0.0
        to_b = (dh * Bm).sum(-1)
        q = dh * a * before
        d_dt = (q * s["A"][lo:hi]).sum(-1) + to_b * u
        dA[lo:hi] = (q * dt[..., None]).sum(0)
        du[:, lo:hi] = (to_b * dt + dy * s["skip"][lo:hi]).to(BF16)
        dskip[lo:hi] = (dy * u).sum(0)
        d_dt = d_dt * torch.sigmoid(s["delta"][:, lo:hi].float() + s["dt_bias"][lo:hi])
        dd[:, lo:hi] = d_dt.to(BF16)
        dbias[lo:hi] = d_dt.sum(0)
        if d_in is not None:
            d_in[s["live"], lo:hi] = (a * dh)[s["first"]]
    out = {"du": du, "ddelta": dd, "dB": dB.to(BF16), "dC": dC.to(BF16), "dA": dA, "dskip": dskip, "d_dt_bias": dbias}
    if s["z"] is not None:
        out["dz"] = dz
    return out if d_in is None else {**out, "d_state_in": d_in}


def _plain_step(s):
    case, keep = s["case"], s["idx"] >= 0
    at = s["idx"].long().clamp(min=0)
    some = keep[:, None]
    window = torch.cat([s["conv_state"][at], s["x"][:, None]], 1)
    p = s["conv_b"] + (window.float() * s["conv_w"].t()).sum(1)
    u = torch.where(some, p * torch.sigmoid(p) if case["silu"] else p, 0.0).to(BF16)
    s["conv_state"][at[keep]] = window[keep, 1:]
    per = case["D"] // case["G"]
    dt = _softplus(s["delta"].float() + s["dt_bias"])[..., None]
    h = torch.exp(dt * s["A"]) * s["scan_state"][at] + dt * u.float()[..., None] * _wide(s["B"], per)
    y = (h * _wide(s["C"], per)).sum(-1) + s["skip"] * u.float()
    if s["z"] is not None:
        y = y * s["z"].float() * torch.sigmoid(s["z"].float())
    s["scan_state"][at[keep]] = h[keep]
    return {"u": u, "y": torch.where(some, y, 0.0).to(BF16), "conv_state": s["conv_state"], "scan_state": s["scan_state"]}


# ------------------------------------------------------------------------- one pass

PLAIN = {"route": _plain_route, "route_bwd": _plain_route_bwd, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd,
         "conv": _plain_conv, "conv_bwd": _plain_conv_bwd, "scan": _plain_scan, "scan_bwd": _plain_scan_bwd,
         "step": _plain_step}


def run(state):
    s, kind = state, state["case"]["kind"]
    return _own(s, kind) if own else PLAIN[kind](s)


def _own(s, kind):
    case = s["case"]
    if kind == "route":
        idx, w = s["router"].forward(s["logits"], s["bias"])
        return {"idx": idx, "w": w, "s": s["router"].topk_s}
    if kind == "route_bwd":
        return {"dlogits": s["router"].backward(s["d_w"])}
    if kind == "norm":
        n = s["norm"]
        y = n.forward(s["x"], s["residual"])
        out = {} if s["residual"] is None else {"sum": n.sum}
        return {**out, "y": y} if case["out"] == "bf16" else {**out, "y8": y, "scale": n.scale}
    if kind == "norm_bwd":
        n = s["norm"]
        dx = n.backward(s["dy"], s["d_sum"])
        out = {} if s["d_sum"] is None else {"d_residual": n.d_residual}
        return {"dx": dx, **out, "dw": n.dw}
    if kind == "conv":
        y = s["conv"].forward(s["x"], s["cu"], s["state_in"], want_state=case["states"])
        return {"y": y, "state": s["conv"].state_out} if case["states"] else {"y": y}
    if kind == "conv_bwd":
        c = s["conv"]
        out = {"dx": c.backward(s["dy"], s["d_state"]), "dw": c.dw, "db": c.db}
        return {**out, "d_state_in": c.d_state_in} if case["states"] else out
    if kind == "scan":
        y = s["scan"].forward(s["u"], s["delta"], s["B"], s["C"], s["z"], s["cu"], s["state_in"], want_state=case["states"])
        return {"y": y, "state": s["scan"].state_out} if case["states"] else {"y": y}
    if kind == "scan_bwd":
        c = s["scan"]
        du, dd, dB, dC, dz = c.backward(s["dy"], s["d_state"])
        out = {"du": du, "ddelta": dd, "dB": dB, "dC": dC, "dA": c.dA, "dskip": c.dskip, "d_dt_bias": c.d_dt_bias}
        out = out if s["z"] is None else {**out, "dz": dz}
        return {**out, "d_state_in": c.d_state_in} if case["states"] else out
    u = s["conv"].step(s["x"], s["conv_state"], s["idx"])
    y = s["scan"].step(u, s["delta"], s["B"], s["C"], s["z"], s["scan_state"], s["idx"])
    return {"u": u, "y": y, "conv_state": s["conv_state"], "scan_state": s["scan_state"]}


# ------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return EXACT[case["kind"]](case, {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
                                      for k, v in s.items()})


def _exact_route(case, s):
    T, E, k, groups = case["T"], case["E"], case["k"], case["groups"]
    l, dead = s["logits"], torch.isinf(s["logits"])
    if case["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-l))
    else:
        p = torch.exp(l - l.max(1, keepdim=True).values)
        p = p / p.sum(1, keepdim=True)
    c = (p + s["bias"] if s["bias"] is not None else p).masked_fill(dead, -INF)
    number = torch.arange(E, device="cuda")
    left = (l if s["bias"] is None else c).masked_fill(dead, -1e300)  # (behind all others, before what is taken)
    if groups > 1:
        rest, total = c.view(T, groups, -1).clone(), 0.0
        for j in range(case["group_top"]):
            top = rest.max(2, keepdim=True)
            total = total + (top.values[..., 0] if j == 0 else top.values[..., 0].clamp(min=-1e300).masked_fill(top.values[..., 0] == -INF, 0.0))
            rest.scatter_(2, top.indices, -INF)
        lower = torch.arange(groups, device="cuda")
        ahead = (total[:, None, :] > total[:, :, None]) | ((total[:, None, :] == total[:, :, None]) & (lower[None, None, :] < lower[None, :, None]))
        left = left.masked_fill((ahead.sum(2) >= case["group_k"]).repeat_interleave(E // groups, 1), -INF)
    chosen = []
    for _ in range(k):
        best = left.max(1, keepdim=True).values
        e = torch.where(left == best, number, E).min(1, keepdim=True).values
        chosen.append(e)
        left = left.scatter(1, e, -INF)
    idx = torch.cat(chosen, 1)
    sel = p.gather(1, idx)
    w = case["scale"] * (sel / sel.sum(1, keepdim=True) if case["renorm"] else sel)
    return {"idx": idx.int(), "w": w, "s": sel}


def _exact_route_bwd(case, s):
    fwd = _exact_route(case, s)
    idx, g = fwd["idx"].long(), s["d_w"]
    l = s["logits"].clone().requires_grad_()
    p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    sel = p.gather(1, idx)
    w = case["scale"] * (sel / sel.sum(1, keepdim=True) if case["renorm"] else sel)
    return {"dlogits": torch.autograd.grad((w * g).sum(), l)[0]}


def _exact_norm(case, s):
    u = s["x"] + (0.0 if s["residual"] is None else s["residual"])
    y = s["weight"] * u / torch.sqrt((u * u).sum(1, keepdim=True) / case["d"] + EPS)
    out = {} if s["residual"] is None else {"sum": u}
    if case["out"] == "bf16":
        return {**out, "y": y}
    scale = torch.stack([y[:, i:i + case["block"]].abs().max(1).values for i in range(0, case["d"], case["block"])], 1) / 448.0
    each = scale.repeat_interleave(case["block"], 1)[:, :case["d"]]
    return {**out, "y8": torch.where(each > 0, y / each, 0.0), "scale": scale}


def _exact_norm_bwd(case, s):
    u, w = s["u"].clone().requires_grad_(), s["weight"].clone().requires_grad_()
    y = w * u / torch.sqrt((u * u).sum(1, keepdim=True) / case["d"] + EPS)
    du, dw = torch.autograd.grad((y * s["dy"]).sum(), (u, w))
    if s["d_sum"] is None:
        return {"dx": du, "dw": dw}
    return {"dx": du + s["d_sum"], "d_residual": du + s["d_sum"], "dw": dw}


def _exact_conv(case, s, grads=False):
    W, D = case["W"], case["D"]
    out = {"y": [], "state": []} if not grads else {"dx": [], "d_state_in": []}
    dw, db = torch.zeros(D, W, dtype=F64, device="cuda"), torch.zeros(D, dtype=F64, device="cuda")
    at = 0
    for i, n in enumerate(s["lens"]):
        before = s["state_in"][i] if s["state_in"] is not None else torch.zeros(W - 1, D, dtype=F64, device="cuda")
        x = torch.cat([before, s["x"][at:at + n]])
        p = (x.unfold(0, W, 1) * s["conv_w"]).sum(-1) + s["conv_b"] if n else x[:0]
        sg = torch.sigmoid(p)
        if not grads:
            out["y"].append(p * sg if case["silu"] else p)
            out["state"].append(x[n:])
        else:
            dp = s["dy"][at:at + n]
            dp = dp * (sg + p * sg * (1.0 - sg)) if case["silu"] else dp
            dx = torch.zeros_like(x)
            for j in range(W if n else 0):
                dx[j:j + n] += dp * s["conv_w"][:, j]
                dw[:, j] += (dp * x[j:j + n]).sum(0)
            db += dp.sum(0)
            if s["d_state"] is not None:
                dx[n:] += s["d_state"][i]
            out["d_state_in"].append(dx[:W - 1])
            out["dx"].append(dx[W - 1:])
        at += n
    if grads:
        res = {"dx": torch.cat(out["dx"]), "dw": dw, "db": db}
        return {**res, "d_state_in": torch.stack(out["d_state_in"])} if case["states"] else res
    return {"y": torch.cat(out["y"]), "state": torch.stack(out["state"])} if case["states"] else {"y": torch.cat(out["y"])}


def _exact_scan(case, s, grads=False):
    """Token by token, the sequences that still have one side by side."""
    D, S, N, lens = case["D"], case["S"], len(s["lens"]), s["lens"]
    T, per = sum(lens), D // case["G"]
    start = [sum(lens[:i]) for i in range(N)]
    order = sorted(range(N), key=lambda i: -lens[i])
    inverse = [order.index(i) for i in range(N)]
    live = [sum(n > t for n in lens) for t in range(max(lens))]
    base = torch.tensor([start[i] for i in order], device="cuda")
    last = torch.tensor([start[i] + lens[i] - 1 for i in order], device="cuda")
    pre = s["delta"] + s["dt_bias"]
    dt = torch.where(pre > 30.0, pre, torch.log1p(torch.exp(pre.clamp(max=30.0))))
    u, A = s["u"], s["A"]
    h = s["state_in"][order] if s["state_in"] is not None else torch.zeros(N, D, S, dtype=F64, device="cuda")
    wide = lambda x: x.repeat_interleave(per, 1)  # noqa: E731
    y = torch.empty(T, D, dtype=F64, device="cuda")
    hs = torch.empty(T, D, S, dtype=F64, device="cuda") if grads else None
    for t, n in enumerate(live):
        at = base[:n] + t
        if grads:
            hs[at] = h[:n]
        h[:n] = torch.exp(dt[at][..., None] * A) * h[:n] + (dt[at] * u[at])[..., None] * wide(s["B"][at])
        y[at] = (h[:n] * wide(s["C"][at])).sum(-1) + s["skip"] * u[at]
    gate = s["z"] * torch.sigmoid(s["z"]) if s["z"] is not None else 1.0
    if not grads:
        return {"y": y * gate, "state": h[inverse]} if case["states"] else {"y": y * gate}
    out = {}
    if s["z"] is not None:
        sg = torch.sigmoid(s["z"])
        out["dz"] = s["dy"] * y * (sg + gate * (1.0 - sg))
    dy = s["dy"] * gate
    X = s["d_state"][order] if s["d_state"] is not None else torch.zeros(N, D, S, dtype=F64, device="cuda")
    du, ddt = torch.empty_like(u), torch.empty_like(u)
    dB, dC = torch.empty_like(s["B"]), torch.empty_like(s["C"])
    dA = torch.zeros_like(A)
    of_group = lambda x: x.unflatten(1, (case["G"], per)).sum(2)  # noqa: E731
    for t, n in enumerate(live):
        at = last[:n] - t
        a = torch.exp(dt[at][..., None] * A)
        Bw, Cw = wide(s["B"][at]), wide(s["C"][at])
        now = a * hs[at] + (dt[at] * u[at])[..., None] * Bw
        dC[at] = of_group(now * dy[at][..., None])
        X[:n] += dy[at][..., None] * Cw
        dB[at] = of_group(X[:n] * (dt[at] * u[at])[..., None])
        da = X[:n] * hs[at] * a
        dA += (da * dt[at][..., None]).sum(0)
        to_b = (X[:n] * Bw).sum(-1)
        ddt[at] = (da * A).sum(-1) + to_b * u[at]
        du[at] = to_b * dt[at] + dy[at] * s["skip"]
        X[:n] *= a
    ddelta = ddt * torch.sigmoid(pre)
    res = {"du": du, "ddelta": ddelta, "dB": dB, "dC": dC, "dA": dA, "dskip": (dy * u).sum(0), "d_dt_bias": ddelta.sum(0), **out}
    return {**res, "d_state_in": X[inverse]} if case["states"] else res


def _exact_step(case, s):
    B, D, W = case["B"], case["D"], case["W"]
    per = D // case["G"]
    u, y = torch.zeros(B, D, dtype=F64, device="cuda"), torch.zeros(B, D, dtype=F64, device="cuda")
    for b, slot in enumerate(s["idx"].tolist()):
        if slot < 0:
            continue
        x = torch.cat([s["conv_state"][slot], s["x"][b][None]])
        s["conv_state"][slot] = x[1:]
        p = s["conv_b"] + sum(x[j] * s["conv_w"][:, j] for j in range(W))
        u[b] = p / (1.0 + torch.exp(-p)) if case["silu"] else p
        v = u[b].to(BF16).double()  # (the scan reads the convolution's output)
        pre = s["delta"][b] + s["dt_bias"]
        dt = torch.log1p(torch.exp(pre))[:, None]
        h = torch.exp(dt * s["A"]) * s["scan_state"][slot] + dt * v[:, None] * s["B"][b].repeat_interleave(per, 0)
        s["scan_state"][slot] = h
        o = (h * s["C"][b].repeat_interleave(per, 0)).sum(-1) + s["skip"] * v
        y[b] = o * s["z"][b] / (1.0 + torch.exp(-s["z"][b])) if s["z"] is not None else o
    return {"u": u, "y": y, "conv_state": s["conv_state"], "scan_state": s["scan_state"]}


EXACT = {"route": _exact_route, "route_bwd": _exact_route_bwd, "norm": _exact_norm, "norm_bwd": _exact_norm_bwd,
         "conv": _exact_conv, "conv_bwd": lambda case, s: _exact_conv(case, s, True), "scan": _exact_scan,
         "scan_bwd": lambda case, s: _exact_scan(case, s, True), "step": _exact_step}
