"""Cases of what stands between a decoder block's attention and its experts, and after them:

gate      router logits to k experts a token and their weights: softmax or sigmoid scores, a bias that takes part in the
          choice alone, groups of experts of which the best stay, weights renormalised and scaled;
route     the same, then the assignments sorted by expert;
norm      r = a x + g * norm(y) and the norm of r: a block's residual addition with its gate and scale, between the norm
          of what the block gave and the norm of what the next one takes;
combine   the same, where y is the weighted sum of each token's expert rows and its shared expert's row.

`own` chooses between the plain form (elementary torch operations in 32 bits; the scores that a choice goes by in 64) and
the framework's kernels.
"""
import math

import torch

own = False

EPS = 1e-6


# --------------------------------------------------------------------------- #
# cases
# --------------------------------------------------------------------------- #
def _gate(name, op, T, E, k, score, bias, groups=1, top_groups=1, group_score="top2", renorm=True, scale=1.0, out=0,
          coarse=False):
    """`out`: experts that are not available (logit -inf); `coarse`: logits that are bf16 values, many of them equal."""
    c = {"op": op, "T": T, "E": E, "k": k, "score": score, "bias": bias, "groups": groups, "top_groups": top_groups,
         "group_score": group_score, "renorm": renorm, "scale": scale, "out": out, "coarse": coarse}
    if name:
        c["name"] = name
    return c


def _norm(name, op, T, H, stream="bf16", post=True, gate="none", scale=1.0, param="bf16", offset=0.0, pad=0, k=0):
    """`stream`: type of the residual stream; `gate`: none, channel, token or full; `param`: type of weights and of the
    channels' gate; `pad`: elements between the rows of x and of y, as in views of wider tensors; `k`: experts a token
    (combine)."""
    c = {"op": op, "T": T, "H": H, "stream": stream, "post": post, "gate": gate, "scale": scale, "param": param,
         "offset": offset, "pad": pad, "k": k}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one token's choice of experts (latency counts): 8 of 256, sigmoid scores, 4 of 8 groups by their two best
        _gate("gate 1 token", "gate", 1, 256, 8, "sigmoid", True, 8, 4, "top2", True, 2.5),
        # a ragged batch through another router: odd sizes, softmax scores with a bias, groups by their best expert
        _gate("gate 777 of 160", "gate", 777, 160, 6, "softmax", True, 8, 3, "max", False, 16.0),
        # the largest: a long offline batch
        _gate("gate 262144", "gate", 262144, 256, 8, "sigmoid", True, 8, 4, "top2", True, 2.5),
        # a 4096-token prompt routed: choice and sort
        _gate("route 4096", "route", 4096, 256, 8, "sigmoid", True, 8, 4, "top2", True, 2.5),
        # four such prompts through a softmax router without bias or groups, weights not renormalised
        _gate("route 16384 softmax", "route", 16384, 256, 8, "softmax", False, 1, 1, "max", False, 1.0),
        # one token between the attention and the experts (latency counts)
        _norm("norm 1 token", "norm", 1, 2048, "bf16", True, "none"),
        # a 4096-token prompt between the attention and the experts, with gains and a gate per channel
        _norm("norm 4096", "norm", 4096, 2048, "bf16", True, "channel", 1.0, "bf16"),
        # odd sizes: a residual stream in 32 bits, rows that are not aligned, a gate per token
        _norm("norm 777 x 1999", "norm", 777, 1999, "f32", False, "token", 0.5, "f32", 1.0, 3),
        # the largest: a wide model's long prompt, the stream in 32 bits, a gate per element
        _norm("norm 16384 x 8192", "norm", 16384, 8192, "f32", True, "full", 0.7071, "f32"),
        # eight decoding sequences behind the experts
        _norm("combine 8 tokens", "combine", 8, 2048, "bf16", True, "none", k=8),
        # a 4096-token prompt behind the experts, no norm of what they gave
        _norm("combine 4096", "combine", 4096, 2048, "bf16", False, "none", k=8),
        # four such prompts, everything at once
        _norm("combine 16384", "combine", 16384, 2048, "f32", True, "channel", 0.7071, "bf16", 1.0, 0, 8),
    ]


def draw(rng):
    """A case of the listed ranges: one token to many, odd sizes among them, every score, gate, type and layout."""
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    while True:
        op = rng.choice(["gate", "gate", "route", "norm", "norm", "combine"])
        if op in ("gate", "route"):
            groups = rng.choice([1, 1, 2, 4, 8, 8, 16])
            per = log(2, max(2, 1024 // groups))
            E = groups * per
            top = rng.randint(1, groups)
            k = min(32, rng.choice([1, 2, 4, 6, 8, 8, 10, 16, 32]), top * per)
            T = log(1, 262144 if op == "gate" else 16384)
            c = _gate(None, op, T, E, k, rng.choice(["softmax", "sigmoid", "sigmoid"]), rng.random() < 0.7, groups, top,
                      rng.choice(["max", "top2", "top2"]), rng.random() < 0.7, rng.choice([1.0, 2.5, 16.0]),
                      rng.choice([0, 0, 0, rng.randint(1, E - 1)]), rng.random() < 0.3)
        else:
            H = log(64, 16384)
            T = log(1, 131072)
            if rng.random() < 0.6 or op == "combine":
                H = max(64, H // 64 * 64)
            c = _norm(None, op, T, H, rng.choice(["bf16", "f32"]), rng.random() < 0.6,
                      rng.choice(["none", "channel", "token", "full"]), rng.choice([1.0, 1.0, 0.5, 0.7071]),
                      rng.choice(["bf16", "f32"]), rng.choice([0.0, 0.0, 1.0]), rng.choice([0, 0, 3, 64]),
                      rng.choice([1, 2, 4, 6, 8, 8, 16]) if op == "combine" else 0)
            if op == "combine":
                c["pad"] = 0
        if work(c)["bytes"] <= max(work(x)["bytes"] for x in listed() if x["op"] == op):
            return c


def work(case):
    c, T = case, case["T"]
    if c["op"] in ("gate", "route"):
        E, k = c["E"], c["k"]
        n = 4 * T * E + 8 * T * k + (4 * E if c["bias"] else 0)
        if c["op"] == "route":
            n += 8 * T * k + 4 * (2 * E + 1)
        return {"bytes": n, "flops": 4 * T * E}
    H, k = c["H"], c["k"]
    s, p = (2 if c["stream"] == "bf16" else 4), (2 if c["param"] == "bf16" else 4)
    n = T * H * (2 * s + 2) + p * H * (1 + c["post"] + (c["gate"] == "channel"))  # x, r, the norm, the parameters
    n += {"token": 2 * T, "full": 2 * T * H}.get(c["gate"], 0)
    n += T * ((k + 1) * H * 2 + 8 * k) if c["op"] == "combine" else T * H * 2  # y
    return {"bytes": n, "flops": T * H * (10 + 2 * k)}


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
def prepare(case, seed):
    """What a program has before the call: a router's logits, or the residual stream, what the block gave, and the
    parameters.  With `own` also the handles on the parameters that it keeps, and the outputs that it reuses."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    c, T = case, case["T"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    if c["op"] in ("gate", "route"):
        E = c["E"]
        # experts of unlike popularity, tokens of unlike certainty
        logits = normal(T, E).mul_(normal(T, 1).mul_(0.3).exp_()).add_(normal(E) * 0.7)
        if c["coarse"]:
            logits = logits.bfloat16().float()
        if c["out"]:
            logits[:, torch.randperm(E, generator=gen, device=dev)[:c["out"]]] = -math.inf
        # a bias that has been stepped up and down by a thousandth
        bias = torch.round(normal(E) * 40) * 0.001 if c["bias"] else None
        s = {"case": dict(c), "logits": logits, "bias": bias}
        if own:
            from bit_mixture_experts_gb300 import ExpertGate
            s["gate"] = ExpertGate(c["k"], c["score"], bias, c["groups"], c["top_groups"], c["group_score"], c["renorm"],
                                   c["scale"])
            s["out"] = (torch.empty((T, c["k"]), dtype=torch.int32, device=dev),
                        torch.empty((T, c["k"]), dtype=torch.float32, device=dev))
        return s

    H, k = c["H"], c["k"]
    stream = torch.bfloat16 if c["stream"] == "bf16" else torch.float32
    param = torch.bfloat16 if c["param"] == "bf16" else torch.float32

    def rows(n, dtype):  # rows of unlike size, with some channels much larger, as in a residual stream
        x = normal(n, H + c["pad"]).mul_(normal(n, 1).mul_(0.5).exp_())
        x[:, :H:97] *= 8
        return x.to(dtype)[:, :H]

    s = {"case": dict(c), "x": rows(T, stream), "w_pre": (normal(H) * 0.2 + 1 - c["offset"]).to(param),
         "w_post": (normal(H) * 0.2 + 1 - c["offset"]).to(param) if c["post"] else None, "gate": None}
    if c["gate"] == "channel":
        s["gate"] = (normal(H) * 0.3 + 0.5).to(param)
    elif c["gate"] != "none":
        s["gate"] = torch.sigmoid(normal(T, 1 if c["gate"] == "token" else H)).bfloat16()
    if c["op"] == "norm":
        s["y"] = rows(T, torch.bfloat16)
    else:
        s["y"] = rows(T * (k + 1), torch.bfloat16)
        s["inv_perm"] = torch.randperm(T * k, generator=gen, device=dev).int()
        w = torch.softmax(normal(T, k), 1)
        s["topk_w"] = w.contiguous()
    if own:
        from bit_mixture_experts_gb300 import ResidualNorm
        s["norm"] = ResidualNorm(s["w_pre"], s["w_post"], c["scale"], EPS, c["offset"])
        s["out"] = (torch.empty((T, H), dtype=stream, device=dev), torch.empty((T, H), dtype=torch.bfloat16, device=dev))
    return s


# --------------------------------------------------------------------------- #
# one pass
# --------------------------------------------------------------------------- #
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    op = s["case"]["op"]
    if op == "gate":
        return s["gate"].choose(s["logits"], out=s["out"])
    if op == "route":
        r = s["gate"].route(s["logits"], block_n=64)
        return r.topk_ids, r.topk_w, r.counts, r.offsets, r.perm, r.inv_perm
    if op == "norm":
        return s["norm"].add(s["x"], s["y"], gate=s["gate"], out=s["out"])
    return s["norm"].combine(s["x"], s["y"], s["inv_perm"], s["topk_w"], gate=s["gate"], out=s["out"])


def _run_plain(s):
    op = s["case"]["op"]
    if op in ("gate", "route"):
        ids, w = _choose_plain(s)
        return (ids, w) if op == "gate" else (ids, w) + _sort_plain(ids, s["case"]["E"])
    return _norm_plain(s)


def _choose_plain(s):
    c, T, k = s["case"], s["case"]["T"], s["case"]["k"]
    logits = s["logits"].double()
    if c["score"] == "softmax":
        score = (logits - logits.amax(1, keepdim=True)).exp_()
        score = score / score.sum(1, keepdim=True)
    else:
        score = 1 / (1 + (-logits).exp_())
    value = score if s["bias"] is None else score + s["bias"].double()
    value = torch.where(logits == -math.inf, torch.full_like(value, -1e300), value)  # not available: behind all others
    if c["groups"] > 1:
        best = value.view(T, c["groups"], -1).sort(dim=2, descending=True).values[:, :, :2]
        total = best[:, :, 0]
        if c["group_score"] == "top2":
            total = total + torch.where(best[:, :, 1] > -1e299, best[:, :, 1], torch.zeros_like(total))
        kept = total.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        stay = torch.zeros((T, c["groups"]), dtype=torch.bool, device=value.device)
        stay[torch.arange(T, device=value.device)[:, None], kept] = True
        value = torch.where(stay.repeat_interleave(c["E"] // c["groups"], 1), value, torch.full_like(value, -math.inf))
    ids = value.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = score[torch.arange(T, device=ids.device)[:, None], ids]
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return ids.int(), (w * c["scale"]).float()


def _sort_plain(ids, E):
    flat = ids.flatten().long()
    perm = flat.sort(stable=True).indices
    n = torch.arange(len(flat), device=flat.device)
    inv = torch.empty_like(perm)
    inv[perm] = n
    counts = torch.zeros(E, dtype=torch.long, device=flat.device).index_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return counts.int(), offsets.int(), perm.int(), inv.int()


def _rms(x, w, offset):
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * (w.float() + offset)


def _norm_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        y = s["y"].float()
    else:
        T, k = c["T"], c["k"]
        y = (s["y"][s["inv_perm"].long()].float().view(T, k, -1) * s["topk_w"][:, :, None]).sum(1) + s["y"][T * k:].float()
    if s["w_post"] is not None:
        y = _rms(y, s["w_post"], c["offset"])
    if s["gate"] is not None:
        y = y * s["gate"].float()
    r = s["x"].float() * c["scale"] + y
    return r.to(s["x"].dtype), _rms(r, s["w_pre"], c["offset"]).bfloat16()


# --------------------------------------------------------------------------- #
# the definition in 64 bits
# --------------------------------------------------------------------------- #
def exact(case, seed):
    s = prepare(case, seed)
    c, T = case, case["T"]
    if c["op"] in ("norm", "combine"):
        r, n = [], []
        for lo in range(0, T, 4096):
            hi = min(T, lo + 4096)
            if c["op"] == "norm":
                z = s["y"][lo:hi].double()
            else:
                k = c["k"]
                z = s["y"][T * k + lo:T * k + hi].double()
                for j in range(k):
                    z = z + s["topk_w"][lo:hi, j, None].double() * s["y"][s["inv_perm"].view(T, k)[lo:hi, j].long()].double()
            if c["post"]:
                z = z / torch.sqrt((z * z).sum(1, keepdim=True) / c["H"] + EPS) * (s["w_post"].double() + c["offset"])
            g = s["gate"]
            if g is not None:
                z = z * (g if g.dim() == 1 else g[lo:hi]).double()
            z = z + c["scale"] * s["x"][lo:hi].double()
            r.append(z)
            n.append(z / torch.sqrt((z * z).sum(1, keepdim=True) / c["H"] + EPS) * (s["w_pre"].double() + c["offset"]))
        return torch.cat(r), torch.cat(n)

    E, k, G = c["E"], c["k"], c["groups"]
    at = torch.arange(E, device=s["logits"].device)
    ids, w = [], []
    for lo in range(0, T, 32768):
        z = s["logits"][lo:lo + 32768].double()
        off = torch.isinf(z)
        score = torch.softmax(z, 1) if c["score"] == "softmax" else torch.sigmoid(z)
        v = score.clone() if s["bias"] is None else score + s["bias"].double()
        v[off] = -1e200
        if G > 1:
            members = [v[:, g * (E // G):(g + 1) * (E // G)] for g in range(G)]
            first = torch.stack([m.amax(1) for m in members], 1)
            if c["group_score"] == "top2":
                second = torch.stack([torch.topk(m, 2, dim=1).values[:, 1] for m in members], 1)
                first = first + second.clamp(min=-1e100) * (second > -1e100)
            # a group stays if fewer than top_groups are ahead of it
            gi = torch.arange(G, device=v.device)
            ahead = (first[:, None, :] > first[:, :, None]) | ((first[:, None, :] == first[:, :, None]) & (gi < gi[:, None]))
            drop = ahead.sum(2) >= c["top_groups"]
            v[drop.repeat_interleave(E // G, 1)] = -math.inf
        taken = []
        for _ in range(k):  # the largest, of equal ones the first
            i = torch.where(v == v.amax(1, keepdim=True), at, E).amin(1)
            taken.append(i)
            v[torch.arange(len(v), device=v.device), i] = -math.inf
        taken = torch.stack(taken, 1)
        p = torch.gather(score, 1, taken)
        if c["renorm"]:
            p = torch.nan_to_num(p / p.sum(1, keepdim=True))
        ids.append(taken)
        w.append(p * c["scale"])
    ids, w = torch.cat(ids), torch.cat(w)
    if c["op"] == "gate":
        return ids.int(), w
    flat = ids.flatten()
    counts = torch.bincount(flat, minlength=E)
    perm = torch.argsort(flat * len(flat) + torch.arange(len(flat), device=flat.device))
    return (ids.int(), w, counts.int(), torch.nn.functional.pad(counts.cumsum(0), (1, 0)).int(), perm.int(),
            torch.argsort(perm).int())
