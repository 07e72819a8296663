"""Workloads of the operators around the layer: the router's balance loss, the AdamW step of
the adapters, and the adapters of many requests beside a shared projection.

Sizes are those of the layer's own configurations (moe_inputs.CONFIGS: hidden 128 / 2048 /
2880 / 7168, 8 to 256 experts, ranks 8 to 32) and generic odd ones.
"""
import math

import torch

own = False

BLOCK = 256          # elements of an 8-bit state that share a scale
HYPER = dict(lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.01)
TAKEN = 99           # optimizer steps taken before the timed one


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # --- balance loss: dir "forward" (loss and counts), "backward" (adds into dlogits), "both"
        # the smallest layer's batch: latency of one forward and one backward call
        dict(name="balance tiny", op="balance", dir="both", T=256, E=8, k=2, S=1, masked=False, biased=False),
        # one 4096-token sequence through 128 experts, the loss alone (evaluation, logging)
        dict(name="balance 4096x128 forward", op="balance", dir="forward", T=4096, E=128, k=8, S=1, masked=False,
             biased=False),
        # a packed batch of ragged sequences with padding, the gradient added to the router's
        dict(name="balance packed 32768x256 backward", op="balance", dir="backward", T=32768, E=256, k=8, S=29,
             masked=True, biased=True),
        # a long packed training batch, loss and gradient, an odd token count
        dict(name="balance packed 131071x128", op="balance", dir="both", T=131071, E=128, k=8, S=64, masked=False,
             biased=True),
        # --- AdamW
        # the four adapter tensors of the smallest layer
        dict(name="adamw tiny adapters", op="adamw", kind="adapters", layers=1, E=8, m=128, n=64, r=8, param="bf16",
             grad="bf16", master=False, bits=32),
        # one layer's adapters (13 M parameters) with fp32 master weights
        dict(name="adamw one layer 32-bit", op="adamw", kind="adapters", layers=1, E=128, m=2048, n=768, r=16,
             param="bf16", grad="bf16", master=True, bits=32),
        # eight layers' adapters (104 M parameters) in one step, states in 8 bits
        dict(name="adamw eight layers 8-bit", op="adamw", kind="adapters", layers=8, E=128, m=2048, n=768, r=16,
             param="bf16", grad="bf16", master=False, bits=8),
        # many small fp32 tensors of odd sizes packed back to back in a flat buffer
        dict(name="adamw 151 odd tensors", op="adamw", kind="odd", count=151, largest=90001, param="fp32", grad="fp32",
             master=False, bits=32),
        # --- adapters of many requests
        # one new token of one request
        dict(name="lora one token", op="lora", K=2048, N=2048, r=16, adapters=8, S=1, T=1, tokens="single"),
        # a decoding batch: 64 requests, each its own token and adapter
        dict(name="lora 64 single tokens", op="lora", K=7168, N=2048, r=32, adapters=64, S=64, T=64, tokens="single"),
        # prompts and decoding requests packed into one batch, some without an adapter, padding rows behind
        dict(name="lora mixed batch", op="lora", K=2880, N=2880, r=16, adapters=16, S=40, T=4133, tokens="mixed"),
        # long prompts
        dict(name="lora long prompts", op="lora", K=7168, N=4096, r=32, adapters=8, S=9, T=16384, tokens="packed"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("balance", "adamw", "lora"))
    if op == "balance":
        E = _log(rng, 3, 1024)
        T = _log(rng, 1, min(131072, 16000000 // E))
        return dict(op=op, dir=rng.choice(("forward", "backward", "both")), T=T, E=E, k=rng.randint(1, min(8, E)),
                    S=min(T, _log(rng, 1, 96)), masked=rng.random() < 0.5, biased=rng.random() < 0.5)
    if op == "adamw":
        bits = rng.choice((8, 32))
        param = rng.choice(("bf16", "fp32"))
        common = dict(op=op, param=param, grad=rng.choice(("bf16", "fp32")),
                      master=param == "bf16" and rng.random() < 0.5, bits=bits)
        if rng.random() < 0.5:
            m, n, r = 16 * rng.randint(4, 128), 16 * rng.randint(2, 48), 8 * rng.randint(1, 8)
            E = max(1, min(rng.randint(1, 128), 9000000 // (r * (2 * m + 3 * n))))
            return dict(common, kind="adapters", layers=rng.randint(1, 3), E=E, m=m, n=n, r=r)
        return dict(common, kind="odd", count=rng.randint(1, 160), largest=_log(rng, 1, 200000))
    K, N = 16 * _log(rng, 1, 448), 16 * _log(rng, 1, 256)
    r = rng.choice((8, 16, 24, 32, 64, 128))
    tokens = rng.choice(("single", "mixed", "packed"))
    adapters = rng.randint(1, max(1, min(64, 64000000 // ((K + N) * r))))
    if tokens == "single":
        S = _log(rng, 1, 256)
        return dict(op=op, K=K, N=N, r=r, adapters=adapters, S=S, T=S, tokens=tokens)
    S = rng.randint(1, 48)
    T = max(S, _log(rng, 16, 8192))
    return dict(op=op, K=K, N=N, r=r, adapters=adapters, S=S, T=T, tokens=tokens)


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _host(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _normal(g, shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _lengths(seed, total, S):
    """S ragged lengths of at most `total` tokens together; with room, some are empty and some rows are left over."""
    g = _host(seed)
    cut = torch.randint(0, total + 1, (S - 1,), generator=g).sort().values.tolist() if S > 1 else []
    end = total if S == 1 or total < 64 else total - int(torch.randint(0, 1 + total // 64, (1,), generator=g))
    off = [0] + [min(c, end) for c in cut] + [end]
    return off


def _balance(c, seed):
    g = _gen(seed)
    T, E, S = c["T"], c["E"], c["S"]
    logits = _normal(g, (T, E))
    if c["biased"]:     # routing that needs balancing: a few hot experts
        logits += -1.2 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    ids = logits.topk(c["k"], dim=1).indices.to(torch.int32)
    off = _lengths(seed, T, S)
    s = dict(c=c, logits=logits, ids=ids, off=None, mask=None,
             loss=torch.empty(S, device="cuda"), counts=torch.empty(S, E, dtype=torch.int32, device="cuda"),
             valid=torch.empty(S, dtype=torch.int32, device="cuda"))
    if S > 1:
        s["off"] = torch.tensor(off, dtype=torch.int32, device="cuda")
    if c["masked"]:
        s["mask"] = torch.rand(T, generator=g, device="cuda") > 0.1
        if S > 2:       # a sequence with nothing valid in it
            s["mask"][off[1]:off[2]] = False
    s["dloss"] = torch.rand(S, generator=g, device="cuda") * (0.01 / S) + 1e-4
    s["dlogits"] = _normal(g, (T, E), 1e-4)
    if c["dir"] == "backward":
        _, s["counts"], s["valid"], _ = _balance_forward(s)
    if own:
        import mixture_experts_lora_b200 as ml
        s["ws"] = torch.empty(ml.moe_balance_workspace_bytes(T, E, S), dtype=torch.uint8, device="cuda")
    return s


def _sizes(c):
    if c["kind"] == "adapters":
        E, m, n, r = c["E"], c["m"], c["n"], c["r"]
        return [(E, m, r), (E, r, 2 * n), (E, n, r), (E, r, m)] * c["layers"]
    g = _host(c["count"] * 1000003 + c["largest"])
    return [(1 + int(c["largest"] ** float(u)) // 1,) for u in torch.rand(c["count"], generator=g)]


def _adamw(c, seed):
    g = _gen(seed)
    shapes = _sizes(c)
    ns = [math.prod(x) for x in shapes]
    types = {"bf16": torch.bfloat16, "fp32": torch.float32}
    # parameters and gradients: one buffer each, the tensors back to back in it
    total = sum(ns)
    w = _normal(g, (total,), 0.02)
    p = w.to(types[c["param"]])
    grad = _normal(g, (total,), 1e-3, types[c["grad"]])
    # states: each tensor's part begins at a multiple of BLOCK elements
    starts, at = [], 0
    for n in ns:
        starts.append(at)
        at += -(-n // BLOCK) * BLOCK
    pad = torch.zeros(at, dtype=torch.bool, device="cuda")
    for a, n in zip(starts, ns):
        pad[a:a + n] = True
    m = _normal(g, (at,), 1e-4) * pad
    v = (_normal(g, (at,), 1e-3).square() + 1e-9) * pad
    s = dict(c=c, p=p, grad=grad, ns=ns, starts=starts, steps=TAKEN, total=total, master=None)
    cut = torch.tensor([0] + ns).cumsum(0).tolist()
    s["params"] = [p[a:b].view(x) for a, b, x in zip(cut, cut[1:], shapes)]
    s["grads"] = [grad[a:b].view(x) for a, b, x in zip(cut, cut[1:], shapes)]
    # per-state views of the same tensors, for the plain form
    if c["master"]:
        s["master"] = torch.zeros(at, device="cuda")
        for a, n, b in zip(starts, ns, cut):
            s["master"][a:a + n] = w[b:b + n]
    if c["bits"] == 8:
        noise = torch.zeros_like(m, dtype=torch.int32)
        s["m"], s["ms"] = _encode(m, noise)
        s["v"], s["vs"] = _encode(v.sqrt(), noise)
    else:
        s["m"], s["v"] = m, v
    if own:
        import mixture_experts_lora_b200 as ml
        opt = ml.AdamW(s["params"], s["grads"], lr=HYPER["lr"], betas=(HYPER["b1"], HYPER["b2"]), eps=HYPER["eps"],
                       weight_decay=HYPER["wd"], state_bits=c["bits"], master_weights=c["master"])
        opt.exp_avg.copy_(s["m"])
        opt.exp_avg_sq.copy_(s["v"])
        if c["bits"] == 8:
            opt.exp_avg_scale.copy_(s["ms"])
            opt.exp_avg_sq_scale.copy_(s["vs"])
        if c["master"]:
            opt.master.copy_(s["master"])
        opt.steps.fill_(TAKEN)
        s["opt"] = opt
    return s


def _lora(c, seed):
    g = _gen(seed)
    T, K, N, r, S, n = c["T"], c["K"], c["N"], c["r"], c["S"], c["adapters"]
    h = _host(seed + 1)
    if c["tokens"] == "single":
        off = list(range(T + 1))
        which = torch.randperm(max(n, S), generator=h)[:S] % n
    else:
        if c["tokens"] == "mixed" and S > 4:   # a few prompts, the other requests one token each
            long = max(1, S // 8)
            off = _lengths(seed, T - (S - long), long)
            off = off + [off[-1] + i + 1 for i in range(S - long)]
        else:
            off = _lengths(seed, T, S)
        which = torch.randint(-1 if c["tokens"] == "mixed" else 0, n, (S,), generator=h)
    return dict(c=c, off=off, which=which.tolist(),
                X=_normal(g, (T, K), 1.0, torch.bfloat16), Y=_normal(g, (T, N), 1.0, torch.bfloat16),
                A=_normal(g, (n, K, r), 1.0 / math.sqrt(K), torch.bfloat16),
                B=_normal(g, (n, r, N), 0.2, torch.bfloat16),
                scale=torch.rand(n, generator=g, device="cuda") + 0.5,
                adapters=which.to(device="cuda", dtype=torch.int32),
                offsets=None if c["tokens"] == "single" else torch.tensor(off, dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    return {"balance": _balance, "adamw": _adamw, "lora": _lora}[case["op"]](case, seed)


# ------------------------------------------------------------------------------- plain forms
def _segments(s):
    """Row t's sequence, and whether the row counts."""
    c = s["c"]
    t = torch.arange(c["T"], device="cuda")
    if s["off"] is None:
        seg, ok = torch.zeros_like(t), torch.ones_like(t, dtype=torch.bool)
    else:
        seg = (t[:, None] >= s["off"][None, 1:]).sum(1)
        ok = seg < c["S"]
        seg = seg.clamp(max=c["S"] - 1)
    return seg, ok if s["mask"] is None else ok & s["mask"]


def _softmax(x):
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _balance_forward(s):
    c = s["c"]
    E, S, k = c["E"], c["S"], c["k"]
    seg, ok = _segments(s)
    p = _softmax(s["logits"]) * ok[:, None]
    at = torch.where(ok[:, None], seg[:, None] * E + s["ids"], S * E).reshape(-1)
    counts = torch.zeros(S * E + 1, dtype=torch.int32, device="cuda")
    counts.index_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    counts = counts[:-1].view(S, E)
    hot = (seg[None, :] == torch.arange(S, device="cuda")[:, None]) & ok[None, :]
    valid = hot.sum(1).to(torch.int32)
    sums = hot.double() @ p.double()              # long sums
    n = valid.double().clamp(min=1)
    loss = (E / k) * (counts.double() * sums).sum(1) / (n * n)
    return loss.float(), counts, valid, (p, seg, ok)


def _balance_backward(s, counts, valid, p, seg, ok):
    c = s["c"]
    n = valid.float().clamp(min=1)
    f = counts.float() * (s["dloss"] * (c["E"] / c["k"]) / (n * n))[:, None]
    f = f[seg]
    return torch.where(ok[:, None], p * (f - (p * f).sum(1, keepdim=True)), 0.0)


def _plain_balance(s):
    c = s["c"]
    if c["dir"] == "backward":
        seg, ok = _segments(s)
        s["dlogits"] += _balance_backward(s, s["counts"], s["valid"], _softmax(s["logits"]), seg, ok)
        return {"dlogits": s["dlogits"]}
    loss, counts, valid, rest = _balance_forward(s)
    out = {"loss": loss, "counts": counts, "valid": valid}
    if c["dir"] == "both":
        out["dlogits"] = _balance_backward(s, counts, valid, *rest)
    return out


def _noise(t, n):
    """Two 16-bit random numbers for each of n elements at step t: a 32-bit integer mix of the index and the step."""
    def mix(x):
        x = x & 0xFFFFFFFF
        x = ((x ^ (x >> 16)) * 0x9E3779B9) & 0xFFFFFFFF
        x = ((x ^ (x >> 15)) * 0xBB67AE85) & 0xFFFFFFFF
        return x ^ (x >> 16)
    seed = mix(torch.tensor(t, dtype=torch.int64, device="cuda"))
    h = mix(torch.arange(n, dtype=torch.int64, device="cuda") ^ seed)
    return (h & 0xFFFF).int(), (h >> 16).int()


def _encode(x, noise):
    """Blocks of BLOCK elements to e4m3 (rounded up where the noise says so) and the blocks' scales."""
    x = torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)
    noise = torch.nn.functional.pad(noise, (0, x.numel() - noise.numel())).view(-1, BLOCK)
    top = x.abs().amax(1, keepdim=True)
    top = torch.where(top < 2.0 ** -100, 0.0, top)
    inv = torch.where(top > 0, 448.0 / top, 0.0)
    # e4m3's exponents moved to the bottom of fp32's: its subnormals are fp32's, and 20 bits go
    bits = ((x.abs() * inv) * 2.0 ** -120).view(torch.int32)
    code = ((bits + (noise << 4)) >> 20).clamp(max=0x7E)
    code = torch.where((x < 0) & (code > 0), code | 0x80, code)
    return code.to(torch.uint8).view(-1).view(torch.float8_e4m3fn), (top / 448.0).view(-1)


def _decode(code, scale):
    return (code.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def _adamw_one(s, i, t, at):
    c, n, a = s["c"], s["ns"][i], s["starts"][i]
    b = a + -(-n // BLOCK) * BLOCK
    p, g = s["p"][at:at + n], s["grad"][at:at + n].float()
    h = HYPER
    blocks = slice(a // BLOCK, b // BLOCK)
    if c["bits"] == 8:
        m = _decode(s["m"][a:b], s["ms"][blocks])[:n]
        v = _decode(s["v"][a:b], s["vs"][blocks])[:n].square()
    else:
        m, v = s["m"][a:a + n], s["v"][a:a + n]
    m = h["b1"] * m + (1 - h["b1"]) * g
    v = h["b2"] * v + (1 - h["b2"]) * (g * g)
    u = v.sqrt()
    w = p.float() if s["master"] is None else s["master"][a:a + n]
    w = w * (1 - h["lr"] * h["wd"]) - (h["lr"] / (1 - h["b1"] ** t)) * (m / (u / math.sqrt(1 - h["b2"] ** t) + h["eps"]))
    p.copy_(w)
    if s["master"] is not None:
        s["master"][a:a + n] = w
    if c["bits"] == 8:
        nm, nv = _noise(t, n)
        code, s["ms"][blocks] = _encode(m, nm)
        s["m"][a:b].view(torch.uint8).copy_(code.view(torch.uint8))
        code, s["vs"][blocks] = _encode(u, nv)
        # a positive root is never stored as zero
        least = torch.nn.functional.pad((u > 0).to(torch.uint8), (0, b - a - n)) * (s["vs"][blocks] > 0).to(
            torch.uint8).repeat_interleave(BLOCK)
        s["v"][a:b].view(torch.uint8).copy_(torch.maximum(code.view(torch.uint8), least))
    else:
        s["m"][a:a + n], s["v"][a:a + n] = m, v


def _adamw_out(s, p, m, v, ms, vs, master, steps):
    out = {"p": p, "m": m, "v": v, "steps": steps}
    if s["c"]["bits"] == 8:
        out.update(ms=ms, vs=vs)
    if s["c"]["master"]:
        out["master"] = master
    return out


def _plain_adamw(s):
    s["steps"] += 1
    ends = torch.tensor([0] + s["ns"]).cumsum(0).tolist()
    [_adamw_one(s, i, s["steps"], ends[i]) for i in range(len(s["ns"]))]
    return _adamw_out(s, s["p"], s["m"], s["v"], s.get("ms"), s.get("vs"), s["master"], s["steps"])


def _plain_lora(s):
    X, A, B, Y, scale = s["X"], s["A"], s["B"], s["Y"], s["scale"]
    if s["offsets"] is None:
        at = s["adapters"].long()
        xa = (X.float()[:, None] @ A[at].float()) * scale[at][:, None, None]
        Y.copy_(Y.float() + (xa @ B[at].float())[:, 0])
        return {"Y": Y}
    [Y[i:j].copy_(Y[i:j].float() + (X[i:j].float() @ A[a].float()) * scale[a] @ B[a].float())
     for i, j, a in zip(s["off"], s["off"][1:], s["which"]) if j > i and a >= 0]
    return {"Y": Y}


# ------------------------------------------------------------------------------- the framework's operators
def _own_balance(s):
    import mixture_experts_lora_b200 as ml
    c = s["c"]
    if c["dir"] == "backward":
        ml.moe_balance_loss_backward(s["logits"], s["counts"], s["valid"], s["dloss"], c["k"], s["dlogits"],
                                     seq_offsets=s["off"], token_mask=s["mask"], accumulate=True)
        return {"dlogits": s["dlogits"]}
    ml.moe_balance_loss(s["logits"], s["ids"], s["loss"], s["counts"], s["valid"], s["ws"], seq_offsets=s["off"],
                        token_mask=s["mask"])
    out = {"loss": s["loss"], "counts": s["counts"], "valid": s["valid"]}
    if c["dir"] == "both":
        ml.moe_balance_loss_backward(s["logits"], s["counts"], s["valid"], s["dloss"], c["k"], s["dlogits"],
                                     seq_offsets=s["off"], token_mask=s["mask"])
        out["dlogits"] = s["dlogits"]
    return out


def _own_adamw(s):
    o = s["opt"]
    o.step()
    return _adamw_out(s, s["p"], o.exp_avg, o.exp_avg_sq, o.exp_avg_scale, o.exp_avg_sq_scale, o.master, o.steps)


def _own_lora(s):
    import mixture_experts_lora_b200 as ml
    ml.moe_lora_requests(s["X"], s["adapters"], s["A"], s["B"], s["scale"], s["Y"], seq_offsets=s["offsets"])
    return {"Y": s["Y"]}


def run(state):
    op = state["c"]["op"]
    if own:
        return {"balance": _own_balance, "adamw": _own_adamw, "lora": _own_lora}[op](state)
    return {"balance": _plain_balance, "adamw": _plain_adamw, "lora": _plain_lora}[op](state)


# ------------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "balance":
        T, E, k, S = c["T"], c["E"], c["k"], c["S"]
        side = S * (4 * E + 8) + (4 * S if S > 1 else 0) + (T if c["masked"] else 0)
        fwd = 4 * T * E + 4 * T * k + side
        bwd = 4 * T * E * (3 if c["dir"] == "backward" else 2) + side + 4 * S
        return {"forward": {"bytes": fwd, "flops": 5 * T * E}, "backward": {"bytes": bwd, "flops": 8 * T * E},
                # one read of the logits serves both
                "both": {"bytes": fwd + bwd - 4 * T * E, "flops": 13 * T * E}}[c["dir"]]
    if c["op"] == "adamw":
        n = sum(math.prod(x) for x in _sizes(c))
        b = {"bf16": 2, "fp32": 4}
        each = b[c["grad"]] + b[c["param"]] + (8 if c["master"] else b[c["param"]])
        each += 16 if c["bits"] == 32 else 4 + 16 / BLOCK
        return {"bytes": n * each, "flops": 14 * n}
    T, K, N, r = c["T"], c["K"], c["N"], c["r"]
    used = min(c["S"], c["adapters"])
    return {"bytes": 2 * T * (K + 2 * N) + 2 * used * r * (K + N), "flops": 2 * T * r * (K + N)}


# ------------------------------------------------------------------------------- in 64 bits
def _exact_balance(s):
    c = s["c"]
    E, S, k = c["E"], c["S"], c["k"]
    off = [0, c["T"]] if s["off"] is None else s["off"].tolist()
    live = torch.ones(c["T"], dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    grad = s["dlogits"].double() if c["dir"] == "backward" else torch.zeros(c["T"], E, device="cuda", dtype=torch.float64)
    loss, counts, valid = [], [], []
    for i in range(S):
        rows = torch.arange(off[i], off[i + 1], device="cuda")
        rows = rows[live[rows]]
        p = torch.softmax(s["logits"][rows].double(), 1)
        n = rows.numel()
        cnt = torch.bincount(s["ids"][rows].reshape(-1).long(), minlength=E)
        f = cnt.double() * (E / (k * max(n, 1) ** 2))
        loss.append((f * p.sum(0)).sum())
        counts.append(cnt)
        valid.append(n)
        grad[rows] += s["dloss"][i].double() * p * (f - p @ f[:, None])
    if c["dir"] == "backward":
        return {"dlogits": grad}
    out = {"loss": torch.stack(loss), "counts": torch.stack(counts).int(),
           "valid": torch.tensor(valid, dtype=torch.int32, device="cuda")}
    if c["dir"] == "both":
        out["dlogits"] = grad
    return out


def _exact_codes(x, rnd, positive):
    """e4m3 values of a tensor's blocks in 64 bits (rnd: 16-bit numbers), and the scales."""
    n = x.numel()
    x = torch.cat([x, x.new_zeros(-n % BLOCK)]).view(-1, BLOCK)
    rnd = torch.cat([rnd, rnd.new_zeros(-n % BLOCK)]).view(-1, BLOCK)
    top = x.abs().max(1, keepdim=True).values
    y = x.abs() * 448 / top.clamp(min=2.0 ** -100)
    step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
    q = (torch.floor(y / step + rnd.double() / 65536) * step).clamp(max=448)
    if positive:
        q = torch.where((x > 0) & (q == 0), 2.0 ** -9, q)
    return (q * torch.sign(x)).view(-1), (top / 448).view(-1)


def _exact_adamw(s):
    c, t = s["c"], s["steps"] + 1
    h = HYPER
    at = s["m"].numel()
    f64 = dict(dtype=torch.float64, device="cuda")
    P, M, V, W = torch.zeros(s["total"], **f64), torch.zeros(at, **f64), torch.zeros(at, **f64), torch.zeros(at, **f64)
    MS, VS = torch.zeros(at // BLOCK, **f64), torch.zeros(at // BLOCK, **f64)
    o = 0
    seed = t
    for n, a in zip(s["ns"], s["starts"]):
        b = a + (n + BLOCK - 1) // BLOCK * BLOCK
        ka, kb = a // BLOCK, b // BLOCK
        m, v = s["m"][a:b].double(), s["v"][a:b].double()
        if c["bits"] == 8:
            m = m * s["ms"][ka:kb].double().repeat_interleave(BLOCK)
            v = (v * s["vs"][ka:kb].double().repeat_interleave(BLOCK)) ** 2
        g = s["grad"][o:o + n].double()
        m = m[:n] * h["b1"] + g * (1 - h["b1"])
        v = v[:n] * h["b2"] + g ** 2 * (1 - h["b2"])
        w = s["p"][o:o + n].double() if s["master"] is None else s["master"][a:a + n].double()
        step = m / (1 - h["b1"] ** t) / ((v / (1 - h["b2"] ** t)) ** 0.5 + h["eps"])
        w = w - h["lr"] * (step + h["wd"] * w)
        P[o:o + n] = w
        W[a:a + n] = w
        if c["bits"] == 8:
            h0 = seed & 0xFFFFFFFF
            for shift, k in ((16, 0x9E3779B9), (15, 0xBB67AE85)):
                h0 = ((h0 ^ (h0 >> shift)) * k) & 0xFFFFFFFF
            h0 ^= h0 >> 16
            i = torch.bitwise_xor(torch.arange(n, device="cuda"), h0)
            for shift, k in ((16, 0x9E3779B9), (15, 0xBB67AE85)):
                i = torch.remainder(torch.bitwise_xor(i, torch.div(i, 1 << shift, rounding_mode="floor")) * k, 1 << 32)
            i = torch.bitwise_xor(i, torch.div(i, 65536, rounding_mode="floor"))
            M[a:b], MS[ka:kb] = _exact_codes(m, torch.remainder(i, 65536), False)
            V[a:b], VS[ka:kb] = _exact_codes(v.sqrt(), torch.div(i, 65536, rounding_mode="floor"), True)
        else:
            M[a:a + n], V[a:a + n] = m, v
        o += n
    return _adamw_out(s, P, M, V, MS, VS, W, t)


def _exact_lora(s):
    Y = s["Y"].double()
    for i, j, a in zip(s["off"], s["off"][1:], s["which"]):
        if a >= 0 and j > i:
            Y[i:j] += s["scale"][a].double() * ((s["X"][i:j].double() @ s["A"][a].double()) @ s["B"][a].double())
    return {"Y": Y}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"balance": _exact_balance, "adamw": _exact_adamw, "lora": _exact_lora}[case["op"]](s)
