"""What is measured of the sequence mixer and the optimizer step.

Five kinds of passes, each through the calls a user makes:
  fwd   linear attention with a decay for each state head, chunked form over packed prompts
  bwd   its backward pass
  step  its recurrent form, one token for each row of a batch, state cache updated in place
  adamw one AdamW step over many tensors, states in 32 or 8 bits

Definitions. State head h has the decay lam = exp(log_decay[h]) <= 1 and r query heads a:
  S_t = lam S_{t-1} + k_t v_t^T;  o_t = scale S_t^T q_t
AdamW: c = min(1, max_norm / (|g| + 1e-6)) (1 when max_norm is 0), g' = c g,
  m = b1 m + (1 - b1) g', v = b2 v + (1 - b2) g'^2,
  p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
8-bit states hold m and r = sqrt(v) as E4M3 with one scale (largest magnitude / 448) for each
block of 256 values; they, and bf16 weights without a master copy, are rounded stochastically
with the counter hash below.
"""
import itertools
import math

import torch

own = False

F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
QBLOCK = 256
HYPER = dict(lr=1e-3, b1=0.9, b2=0.95, eps=1e-8, wd=0.1)
STEP0 = 100   # steps the optimizer state has behind it


# ------------------------------------------------------------------------- cases

def listed():
    return [
        # one short prompt on a small model: the latency of a call
        dict(name="fwd_short", kind="fwd", lens="77", Hs=8, r=1, Dk=64, Dv=64, states=False),
        # prompts of a serving batch packed on one token axis, grouped query heads, states resumed
        dict(name="fwd_packed", kind="fwd", lens="1,513,0,2048,129,1000,77,4096", Hs=8, r=4, Dk=128,
             Dv=128, states=True),
        # one long document, d = 4096 as 32 heads of 128
        dict(name="fwd_long", kind="fwd", lens="32768", Hs=32, r=1, Dk=128, Dv=128, states=True),
        # the training step's 16384 tokens, d = 4096 as 32 heads of 128
        dict(name="bwd_train", kind="bwd", lens="4096,4096,4096,4096", Hs=32, r=1, Dk=128, Dv=128,
             states=False),
        # packed documents with odd lengths, grouped heads, narrow keys, states carried
        dict(name="bwd_packed", kind="bwd", lens="1531,64,2,777,1300,255", Hs=16, r=2, Dk=64, Dv=128,
             states=True),
        # one user's token
        dict(name="step_one", kind="step", B=1, Hs=32, r=1, Dk=128, Dv=128, pad=0),
        # a large serving batch
        dict(name="step_batch", kind="step", B=256, Hs=32, r=1, Dk=128, Dv=128, pad=0),
        # an odd batch with empty rows, grouped heads, rows scattered over the cache
        dict(name="step_grouped", kind="step", B=37, Hs=8, r=4, Dk=96, Dv=128, pad=3),
        # the weights of the tiny layer (d 256, l 128, 8 experts) and their norms, fp32
        dict(name="adamw32_small", kind="adamw", sizes="65536,32768,16384,131072,65536,256,256,1",
             p="f32", g="f32", bits=32, master=False, clip=False),
        # 64 experts of the layer (l 1024, f 512) and its projections: bf16 weights with a master copy
        dict(name="adamw32_master", kind="adamw", sizes="67108864,33554432,4194304,4194304,3670016,4096",
             p="bf16", g="f32", bits=32, master=True, clip=True),
        # 128 experts, everything in few bits
        dict(name="adamw8_large", kind="adamw", sizes="134217728,67108864,4194304,4194304,3670016,4096",
             p="bf16", g="bf16", bits=8, master=False, clip=False),
        # odd tensors, fp32 weights, clipped
        dict(name="adamw8_odd", kind="adamw", sizes="1,255,257,100003,999999,31,4099,7654321", p="f32",
             g="f32", bits=8, master=False, clip=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "adamw", "adamw"])
    if kind == "adamw":
        total = _log(rng, 1000, 100_000_000)
        cuts = sorted(rng.random() ** 2 for _ in range(rng.randint(0, 9)))
        sizes = [max(1, int(total * (b - a))) for a, b in zip([0.0] + cuts, cuts + [1.0])]
        p = rng.choice(["f32", "bf16"])
        return dict(kind=kind, sizes=",".join(map(str, sizes)), p=p, g=rng.choice(["f32", "bf16"]),
                    bits=rng.choice([8, 32]), master=p == "bf16" and rng.random() < 0.5,
                    clip=rng.random() < 0.5)
    dims = dict(Hs=rng.choice([1, 2, 3, 5, 8, 16, 24, 32]), r=rng.choice([1, 1, 1, 2, 4]),
                Dk=rng.choice([64, 128, 128, 96, 40]), Dv=rng.choice([64, 128, 128, 96, 72]))
    if kind == "step":
        return dict(kind=kind, B=_log(rng, 1, 256), pad=rng.choice([0, 0, 1, 5]), **dims)
    most = 16384 * 32 // (dims["Hs"] * dims["r"])
    n = rng.choice([1, 1, 2, 4, 7])
    lens = [_log(rng, 1, max(1, min(most // n, 24000))) for _ in range(n)]
    if n > 2 and rng.random() < 0.5:
        lens[rng.randrange(n)] = 0
    return dict(kind=kind, lens=",".join(map(str, lens)), states=rng.random() < 0.5, **dims)


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def work(case):
    if case["kind"] == "adamw":
        n = sum(int(x) for x in case["sizes"].split(","))
        pb, gb = (4 if case["p"] == "f32" else 2), (4 if case["g"] == "f32" else 2)
        per = 2 * pb + gb + (16 if case["bits"] == 32 else 4 + 16 / QBLOCK)
        if case["master"]:
            per += 8 - pb  # the weight is written from its master copy, not read
        return {"bytes": n * per, "flops": 16 * n}
    Hs, Hq, Dk, Dv = case["Hs"], case["Hs"] * case["r"], case["Dk"], case["Dv"]
    if case["kind"] == "step":
        B = case["B"] - min(case["pad"], case["B"] - 1)
        return {"bytes": B * (8 * Hs * Dk * Dv + 2 * (Hq + Hs) * (Dk + Dv)),
                "flops": B * (3 * Hs + 2 * Hq) * Dk * Dv}
    T, N = sum(_lens(case)), len(_lens(case))
    st = 4 * N * Hs * Dk * Dv if case["states"] else 0
    if case["kind"] == "fwd":
        return {"bytes": 2 * T * (Hq + Hs) * (Dk + Dv) + 2 * st, "flops": 2 * T * Dk * Dv * (Hs + Hq)}
    return {"bytes": 2 * T * (2 * Hq * Dk + 2 * Hs * (Dk + Dv) + Hq * Dv) + 3 * st,
            "flops": 2 * T * Dk * Dv * (3 * Hs + 2 * Hq)}


# ------------------------------------------------------------------------- inputs

def _decays(Hs):
    """Slopes spread geometrically over the heads, from a memory of 2 tokens to 2000."""
    h = torch.arange(Hs, dtype=F64)
    return (-0.5 * 1000.0 ** (-h / max(Hs - 1, 1))).to(F32).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    if case["kind"] == "adamw":
        return _prepare_adamw(case, seed, gen)
    Hs, r, Dk, Dv = case["Hs"], case["r"], case["Dk"], case["Dv"]
    Hq = Hs * r
    lens = _lens(case) if "lens" in case else [1] * case["B"]
    T, N = sum(lens), len(lens)
    # one fused projection's output: the three operands are slices of its rows; queries and keys
    # have unit length, as the mixer's head norms leave them
    wq, wk, wv = Hq * Dk, Hs * Dk, Hs * Dv
    qkv = torch.empty(T, wq + wk + wv, dtype=BF16, device="cuda")
    unit = lambda n: torch.nn.functional.normalize(randn(T, n, Dk), dim=-1).reshape(T, n * Dk)  # noqa: E731
    qkv[:, :wq] = unit(Hq) * Dk ** 0.5
    qkv[:, wq:wq + wk] = unit(Hs)
    qkv[:, wq + wk:] = randn(T, wv)
    s = dict(case=case, lens=lens, log_decay=_decays(Hs), scale=Dk ** -0.5,
             q=qkv[:, :wq].unflatten(1, (Hq, Dk)), k=qkv[:, wq:wq + wk].unflatten(1, (Hs, Dk)),
             v=qkv[:, wq + wk:].unflatten(1, (Hs, Dv)))
    if case["kind"] == "step":
        B = case["B"]
        slots = B + 5
        s["state"] = 0.3 * randn(slots, Hs, Dk, Dv)
        idx = torch.randperm(slots, generator=gen, device="cuda")[:B].to(torch.int32)
        idx[B - min(case["pad"], B - 1):] = -1
        s["idx"] = idx
    else:
        s["cu"] = torch.tensor(list(itertools.accumulate([0] + lens)), dtype=torch.int32, device="cuda")
        s["state_in"] = 0.3 * randn(N, Hs, Dk, Dv) if case["states"] else None
        if case["kind"] == "bwd":
            s["dout"] = randn(T, Hq, Dv).to(BF16)
            s["d_state"] = 0.3 * randn(N, Hs, Dk, Dv) if case["states"] else None
    if own:
        from sparse_moe_layer_topk_gb300.linattn import LinearAttention
        s["la"] = LinearAttention(s["log_decay"], T, Dk, Dv, r=r, N=N, max_seqlen=max(lens),
                                  scale=s["scale"], backward=case["kind"] == "bwd")
        if case["kind"] == "bwd":  # the forward that the training step ran before
            s["la"].forward(s["q"], s["k"], s["v"], cu_seqlens=s["cu"], state_in=s["state_in"])
    else:
        s["fwd_rows"] = _rows(lens, False) if "lens" in case else None
        s["rev_rows"] = _rows(lens, True) if case["kind"] == "bwd" else None
    return s


def _prepare_adamw(case, seed, gen):
    sizes = [int(x) for x in case["sizes"].split(",")]
    dt = dict(f32=F32, bf16=BF16)
    s = dict(case=case, seed=seed & 0x7FFFFFFF, step=STEP0, p=[], g=[], m=[], v=[], ms=[], vs=[], master=[])
    for n in sizes:
        randn = lambda: torch.randn(n, generator=gen, device="cuda")  # noqa: E731
        spread = torch.exp(randn())  # entries of very different size, as gradients have
        w = 0.02 * randn()
        m, r = 1e-3 * spread * randn(), 1e-3 * spread * (0.3 + randn().abs())
        s["g"].append((2e-3 * spread * randn()).to(dt[case["g"]]))
        s["p"].append(w.to(dt[case["p"]]))
        if case["master"]:
            s["master"].append(w)
        if case["bits"] == 32:
            s["m"].append(m)
            s["v"].append(r.square())
        else:
            for x, codes, scales in ((m, s["m"], s["ms"]), (r, s["v"], s["vs"])):
                b = _blocks(x)
                sc = b.abs().amax(1) / 448.0
                codes.append((b / sc[:, None]).to(torch.float8_e4m3fn).reshape(-1)[:n].clone())
                scales.append(sc)
        del spread, w, m, r
    if own:
        from sparse_moe_layer_topk_gb300.optim import AdamW
        s["opt"] = opt = AdamW(s["p"], s["g"], lr=HYPER["lr"], betas=(HYPER["b1"], HYPER["b2"]),
                               eps=HYPER["eps"], weight_decay=HYPER["wd"],
                               max_norm=_max_norm(case), state_bits=case["bits"],
                               master=case["master"], seed=s["seed"])
        opt.load_state(STEP0, s["m"], s["v"], s["ms"] or None, s["vs"] or None, s["master"] or None)
    return s


def _max_norm(case):
    return 1.0 if case["clip"] else 0.0


def _blocks(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % QBLOCK)).view(-1, QBLOCK)


# ------------------------------------------------------------------------- the random numbers

MASK = 0xFFFFFFFF


def _mix(x):
    x = x ^ (x >> 16)
    x = (x * 0x45D9F3B5) & MASK
    x = x ^ (x >> 15)
    x = (x * 0x2F7D9D4B) & MASK
    return x ^ (x >> 16)


def _random16(seed, step, tensor, n):
    """Three 16-bit numbers (for m, r and the weight) of each of a tensor's n values."""
    key = _mix((_mix((seed ^ _mix(step)) & MASK) + 0x9E3779B9 * (tensor + 1)) & MASK)
    i = torch.arange(n, device="cuda")
    h = _mix((i & MASK) ^ _mix((i >> 32) + key & MASK))
    return h & 0xFFFF, h >> 16, (((h ^ (h >> 15)) * 0x1B56C4E9) & MASK) >> 16


# ------------------------------------------------------------------------- plain forms

CHUNK = 64


def _rows(lens, backwards):
    """[N, L] token of each place of each sequence (left aligned, length a multiple of the
    chunk), T where there is none."""
    L = max(CHUNK, -(-max(lens) // CHUNK) * CHUNK)
    n = torch.tensor(lens, device="cuda")[:, None]
    start = n.cumsum(0) - n
    j = torch.arange(L, device="cuda")[None]
    return torch.where(j < n, start + (n - 1 - j if backwards else j), int(n.sum()))


def _recur(q, k, v, s, rows, state, first):
    """sum_{j<=i} lam^(i-j) (q_i.k_j) v_j + lam^(i+first) q_i state, in the order of `rows`, summed over
    the group where q has one head for a group of k and v heads; and sum_j lam^(n-1-j) k_j v_j^T,
    lam^n (n: a sequence's length)."""
    Hs = s["case"]["Hs"]
    N, L = rows.shape
    nc = L // CHUNK

    def take(x):  # [N, Hs, group, nc, CHUNK, D] in 32 bits, zeros where there is no token
        x = torch.cat([x.float(), x.new_zeros(1, *x.shape[1:], dtype=F32)])[rows]
        return x.view(N, nc, CHUNK, Hs, -1, x.shape[-1]).permute(0, 3, 4, 1, 2, 5)

    q, k, v = take(q), take(k), take(v)
    ld = s["log_decay"].view(Hs, 1, 1)
    i = torch.arange(CHUNK, device="cuda", dtype=F32)
    gap = i[:, None] - i[None]
    inside = torch.where(gap >= 0, torch.exp(ld * gap.clamp(min=0)), 0.0)[:, None, None]
    out = (q @ k.transpose(-1, -2) * inside) @ v
    out = out.sum(2, keepdim=True) if q.shape[2] == 1 else out
    left = torch.exp(ld * (CHUNK - 1 - i)[:, None])[:, None, None]  # [Hs, 1, 1, CHUNK, 1]
    z = ((k * left).transpose(-1, -2) @ v).sum(2)                   # [N, Hs, nc, Dk, Dv]
    c = torch.arange(nc, device="cuda", dtype=F32)
    between = c[:, None] - 1 - c[None]
    carry = torch.where(between >= 0, torch.exp(ld * CHUNK * between.clamp(min=0)), 0.0)
    before = (carry @ z.flatten(3)).view(z.shape)
    out = out + torch.exp(ld * (i + 1)[:, None])[:, None, None] * (q @ before[:, :, None])
    n = torch.tensor(s["lens"], device="cuda", dtype=F32)[:, None, None]
    if state is not None:
        pos = torch.arange(L, device="cuda", dtype=F32).view(nc, CHUNK, 1) + first
        out = out + torch.exp(ld[..., None, None] * pos) * (q @ state[:, :, None, None])
    flat = out.permute(0, 3, 4, 1, 2, 5).reshape(N * L, -1, out.shape[-1])
    real = rows.flatten() < sum(s["lens"])
    back = flat.new_empty(sum(s["lens"]), *flat.shape[1:])
    back[rows.flatten()[real]] = flat[real]
    w = torch.exp(ld[:, 0] * (n - 1 - torch.arange(L, device="cuda", dtype=F32)).clamp(min=0))
    w = w.view(N, Hs, 1, nc, CHUNK, 1)
    total = ((k * w).flatten(3, 4).transpose(-1, -2) @ v.flatten(3, 4)).sum(2)
    return back, total, torch.exp(ld[:, 0] * n)[..., None]


def _plain_fwd(s):
    S0 = s["state_in"]
    o, total, decay = _recur(s["q"], s["k"], s["v"], s, s["fwd_rows"], S0, 1)
    out = {"o": (s["scale"] * o).to(BF16)}
    if s["case"]["states"]:
        out["state"] = total + decay * S0
    return out


def _plain_bwd(s):
    q, k, v, do, S0, X = s["q"], s["k"], s["v"], s["dout"], s["state_in"], s["d_state"]
    c = s["scale"]
    flip = lambda x: None if x is None else x.transpose(-1, -2)  # noqa: E731
    over = None if X is None else X / c
    dq, _, _ = _recur(do, v, k, s, s["fwd_rows"], flip(S0), 1)
    dv, total, decay = _recur(k, q, do, s, s["rev_rows"], over, 0)
    dk, _, _ = _recur(v, do, q, s, s["rev_rows"], flip(over), 0)
    out = {"dq": (c * dq).to(BF16), "dk": (c * dk).to(BF16), "dv": (c * dv).to(BF16)}
    if X is not None:
        lam = torch.exp(s["log_decay"])[:, None, None]
        n = torch.tensor(s["lens"], device="cuda")[:, None, None, None]
        out["d_state_in"] = torch.where(n > 0, lam * c * total, 0.0) + decay * X
    return out


def _plain_step(s):
    case, keep = s["case"], s["idx"] >= 0
    at = s["idx"].long().clamp(min=0)
    lam = torch.exp(s["log_decay"])[:, None, None]
    S = lam * s["state"][at] + s["k"].float()[..., None] * s["v"].float()[..., None, :]
    q = s["q"].float().unflatten(1, (case["Hs"], case["r"]))
    o = s["scale"] * (q @ S).flatten(1, 2)
    s["state"][at[keep]] = S[keep]
    return {"o": torch.where(keep[:, None, None], o, 0.0).to(BF16), "state": s["state"]}


def _stochastic_e4m3(y, rand16):
    """E4M3 bytes of 0 <= y <= 448: the value's bits below the format's last are added to a random
    number and cut; times 2^-120 the format's subnormals become those of 32-bit floats."""
    bits = (y * 2.0 ** -120).view(torch.int32)
    return ((bits + (rand16 << 4)) >> 20).clamp(max=0x7E)


def _plain_adamw_one(s, t, n, clip, bc1, bc2):
    case, h = s["case"], HYPER
    g = s["g"][t].float() * clip
    if case["bits"] == 32:
        m, v = s["m"][t], s["v"][t]
    else:
        m = (_blocks(s["m"][t].float()) * s["ms"][t][:, None]).flatten()[:n]
        v = (_blocks(s["v"][t].float()) * s["vs"][t][:, None]).flatten()[:n].square()
    m = h["b1"] * m + (1 - h["b1"]) * g
    v = h["b2"] * v + (1 - h["b2"]) * g * g
    p = (s["master"][t] if case["master"] else s["p"][t]).float()
    p = p * (1 - h["lr"] * h["wd"]) - h["lr"] / bc1 * m / (torch.sqrt(v) / math.sqrt(bc2) + h["eps"])
    um, ur, up = _random16(s["seed"], s["step"], t, n) if case["bits"] == 8 or case["p"] == "bf16" else [None] * 3
    if case["bits"] == 32:
        s["m"][t].copy_(m)
        s["v"][t].copy_(v)
    else:
        for x, u, codes, scales in ((m, um, s["m"], s["ms"]), (torch.sqrt(v), ur, s["v"], s["vs"])):
            b = _blocks(x)
            top = b.abs().amax(1)
            y = (b.abs() * (448.0 / top)[:, None]).flatten()[:n]
            code = _stochastic_e4m3(y, u.int()) | ((x < 0).int() << 7)
            codes[t].view(torch.uint8).copy_(code)
            scales[t].copy_(top / 448.0)
    if case["master"]:
        s["master"][t].copy_(p)
    if case["p"] == "bf16" and not case["master"]:
        p = ((p.view(torch.int32) + up.int()) & -65536).view(F32)
    s["p"][t].copy_(p)


def _plain_adamw(s):
    s["step"] += 1
    clip = 1.0
    if s["case"]["clip"]:
        norm = torch.sqrt(sum(g.float().square().sum() for g in s["g"]))
        clip = torch.clamp(_max_norm(s["case"]) / (norm + 1e-6), max=1.0)
    bc1, bc2 = 1 - HYPER["b1"] ** s["step"], 1 - HYPER["b2"] ** s["step"]
    for t, g in enumerate(s["g"]):
        _plain_adamw_one(s, t, g.numel(), clip, bc1, bc2)


# ------------------------------------------------------------------------- one pass

def run(state):
    s, kind = state, state["case"]["kind"]
    if kind == "adamw":
        s["opt"].step() if own else _plain_adamw(s)
        src = s["opt"] if own else None
        out = {"p": s["p"], "m": src.m if own else s["m"], "v": src.v if own else s["v"]}
        if s["case"]["bits"] == 8:
            out["ms"], out["vs"] = (src.m_scale, src.v_scale) if own else (s["ms"], s["vs"])
        if s["case"]["master"]:
            out["master"] = src.master if own else s["master"]
        return out
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step}[kind](s)
    la = s["la"]
    if kind == "fwd":
        want = s["case"]["states"]
        o = la.forward(s["q"], s["k"], s["v"], cu_seqlens=s["cu"], state_in=s["state_in"], want_state=want)
        return {"o": o, "state": la.state_out} if want else {"o": o}
    if kind == "bwd":
        dq, dk, dv = la.backward(s["dout"], d_state_out=s["d_state"])
        out = {"dq": dq, "dk": dk, "dv": dv}
        return out if s["d_state"] is None else {**out, "d_state_in": la.d_state_in}
    return {"o": la.step(s["q"], s["k"], s["v"], s["state"], s["idx"]), "state": s["state"]}


# ------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["kind"] == "adamw":
        return _exact_adamw(case, s)
    if "lens" in case and max(_lens(case)) > 40000:
        return None
    lam = torch.exp(s["log_decay"].double())[:, None, None]
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    Hs, r = case["Hs"], case["r"]
    group = lambda x: x.unflatten(1, (Hs, r))  # noqa: E731
    if case["kind"] == "step":
        state, o = s["state"].double(), torch.zeros(case["B"], Hs * r, case["Dv"], dtype=F64, device="cuda")
        for b, slot in enumerate(s["idx"].tolist()):
            if slot >= 0:
                state[slot] = lam * state[slot] + k[b][:, :, None] * v[b][:, None, :]
                o[b] = s["scale"] * torch.einsum("hrk,hkv->hrv", group(q)[b], state[slot]).flatten(0, 1)
        return {"o": o, "state": state}
    lens, start, N = s["lens"], [0], len(s["lens"])
    for n in lens:
        start.append(start[-1] + n)
    order = sorted(range(N), key=lambda n: -lens[n])
    live = [sum(n > t for n in lens) for t in range(max(lens))]
    base = torch.tensor([start[n] for n in order], device="cuda")
    last = torch.tensor([start[n] + lens[n] - 1 for n in order], device="cuda")
    size = (N, Hs, case["Dk"], case["Dv"])
    S = s["state_in"].double()[order] if s["state_in"] is not None else torch.zeros(size, dtype=F64, device="cuda")
    inverse = [order.index(n) for n in range(N)]
    qg = group(q)
    if case["kind"] == "fwd":
        o = torch.empty(q.shape[0], Hs, r, case["Dv"], dtype=F64, device="cuda")
        for t, n in enumerate(live):  # the n sequences that still have a token t
            at = base[:n] + t
            A = S[:n].mul_(lam)
            A += k[at][..., None] * v[at][..., None, :]
            o[at] = qg[at] @ A
        out = {"o": s["scale"] * o.flatten(1, 2)}
        return {**out, "state": S[inverse]} if case["states"] else out
    do = group(s["dout"].double())
    dq, dk, dv = torch.empty_like(qg), torch.empty_like(k), torch.empty_like(v)
    X = s["d_state"].double()[order] if s["d_state"] is not None else torch.zeros(size, dtype=F64, device="cuda")
    for t, n in enumerate(live):
        at = base[:n] + t
        A = S[:n].mul_(lam)
        A += k[at][..., None] * v[at][..., None, :]
        dq[at] = s["scale"] * do[at] @ A.transpose(-1, -2)
    for t, n in enumerate(live):
        at = last[:n] - t
        A = X[:n]
        A += s["scale"] * qg[at].transpose(-1, -2) @ do[at]
        dk[at] = (A @ v[at][..., None])[..., 0]
        dv[at] = (k[at][..., None, :] @ A)[..., 0, :]
        A.mul_(lam)
    out = {"dq": dq.flatten(1, 2), "dk": dk, "dv": dv}
    return {**out, "d_state_in": X[inverse]} if case["states"] else out


def _cut(x, unit_exp, rand16):
    """x cut to multiples of 2^unit_exp after a random part of one is added to its magnitude."""
    unit = torch.ldexp(torch.ones_like(x), unit_exp)
    return torch.sign(x) * torch.floor(x.abs() / unit + rand16 / 65536.0) * unit


def _exact_adamw(case, s):
    h, t1 = HYPER, STEP0 + 1
    clip = 1.0
    if case["clip"]:
        clip = min(1.0, 1.0 / (math.sqrt(sum(float(g.double().square().sum()) for g in s["g"])) + 1e-6))
    out = {name: [] for name in ["p", "m", "v"] + (["ms", "vs"] if case["bits"] == 8 else []) +
           (["master"] if case["master"] else [])}
    for t, g in enumerate(s["g"]):
        n, g = g.numel(), g.double() * clip
        m, v = s["m"][t].double(), s["v"][t].double()
        if case["bits"] == 8:
            m = m * s["ms"][t].double().repeat_interleave(QBLOCK)[:n]
            v = (v * s["vs"][t].double().repeat_interleave(QBLOCK)[:n]) ** 2
        m = m + (1 - h["b1"]) * (g - m)
        v = v + (1 - h["b2"]) * (g * g - v)
        p = (s["master"] if case["master"] else s["p"])[t].double()
        p = p - h["lr"] * (h["wd"] * p + m / (1 - h["b1"] ** t1) / ((v / (1 - h["b2"] ** t1)).sqrt() + h["eps"]))
        u = _random16(s["seed"], t1, t, n)
        if case["bits"] == 32:
            out["m"].append(m)
            out["v"].append(v)
        else:
            for x, rand, codes, scales in ((m, u[0], "m", "ms"), (v.sqrt(), u[1], "v", "vs")):
                top = _blocks(x).abs().amax(1)
                y = x * (448.0 / top).repeat_interleave(QBLOCK)[:n]
                exponent = (torch.frexp(y)[1] - 1).clamp(min=-6) - 3
                out[codes].append(_cut(y, exponent, rand).clamp(-448.0, 448.0))
                out[scales].append(top / 448.0)
        if case["master"]:
            out["master"].append(p)
        elif case["p"] == "bf16":
            p = _cut(p, torch.frexp(p)[1] - 8, u[2])
        out["p"].append(p)
    return out
