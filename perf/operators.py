"""Cases of the paged key/value cache operators: writing new tokens' keys and values into the cache (bf16, or e4m3
with one power-of-two scale per token and head), reading them back, and the attention of a chunk of new tokens over
the cache.

A sequence b of a batch has kv_len[b] tokens in the cache, its new ones included; its q_len[b] new tokens are rows
cu_q[b] .. cu_q[b + 1] - 1 of the inputs and sit at positions kv_len[b] - q_len[b] .. kv_len[b] - 1.  Position p lives
in page page_table[b, p // page_size], row p % page_size.

`own` chooses between the plain form (elementary torch operations in 32 bits) and the framework's kernels.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0


# --------------------------------------------------------------------------- #
# cases
# --------------------------------------------------------------------------- #
def _case(name, op, fmt, batch, new, past, hq, hkv, d, page, ragged, lse=False):
    """`new`: new tokens per sequence (prefill and drafts: at most, when ragged); `past`: tokens already cached (at
    most, when ragged); `ragged`: 0 for equal lengths, else the seed of the lengths."""
    c = {"op": op, "fmt": fmt, "batch": batch, "new": new, "past": past, "hq": hq, "hkv": hkv, "d": d, "page": page,
         "ragged": ragged, "lse": lse}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step of eight sequences: eight tokens' keys and values quantised into their pages and read back
        # (latency counts)
        _case("append e4m3 decode8", "append", "e4m3", 8, 1, 4095, 16, 2, 128, 64, 11),
        # a 4096-token prompt's keys and values, sliced from the fused projection, quantised and handed on dense
        _case("append e4m3 prefill4k", "append", "e4m3", 1, 4096, 0, 16, 2, 128, 64, 0),
        # the largest: a ragged prefill batch with eight KV heads, unquantised pages of 16 tokens
        _case("append bf16 ragged x8", "append", "bf16", 8, 8192, 1000, 32, 8, 128, 16, 13),
        # a long prefix read back, e.g. to move the sequence to another cache
        _case("read e4m3 131071", "read", "e4m3", 1, 131071, 0, 16, 2, 128, 64, 0),
        # batch-1 decode with a 4K context: a latency-bound call
        _case("decode1 bf16 4k", "attention", "bf16", 1, 1, 4095, 16, 2, 128, 64, 0),
        # eight sequences of ragged length decoding from a quantised cache
        _case("decode8 e4m3 ragged 32k", "attention", "e4m3", 8, 1, 32000, 16, 2, 128, 64, 17),
        # a serving batch: 64 ragged sequences, one token each; the scores' log-sum-exp kept for a later merge
        _case("decode64 bf16 ragged 8k", "attention", "bf16", 64, 1, 8191, 16, 2, 128, 32, 19, True),
        # batch-1 decode at the longest context
        _case("decode1 e4m3 131071", "attention", "e4m3", 1, 1, 131070, 16, 2, 128, 64, 0),
        # drafted tokens of eight sequences checked in one pass
        _case("draft8x6 bf16 ragged 9k", "attention", "bf16", 8, 6, 9000, 16, 2, 128, 64, 23),
        # a 512-token prompt with nothing cached before it
        _case("prefill512 bf16", "attention", "bf16", 1, 512, 0, 16, 2, 128, 64, 0),
        # a chunk of 4096 tokens over a 32K context: the largest, tensor-core bound
        _case("chunk4k over 32k bf16", "attention", "bf16", 1, 4096, 32768, 16, 2, 128, 128, 0),
        # a ragged batch of chunks over quantised contexts
        _case("chunks x6 e4m3 ragged", "attention", "e4m3", 6, 1777, 9001, 16, 2, 128, 64, 29),
    ]


def _lens(case):
    """(q_len, kv_len) of every sequence, from the case alone."""
    B, new, past = case["batch"], case["new"], case["past"]
    if not case["ragged"]:
        return [new] * B, [new + past] * B
    r = random.Random(case["ragged"])
    q = [new if new == 1 else r.randint(max(1, new // 4), new) for _ in range(B)]
    q[r.randrange(B)] = new
    return q, [n + (r.randint(past // 8, past) if past else 0) for n in q]


def _pairs(q, kv):
    """Visible (new token, key) pairs: sum over new tokens of their position + 1."""
    return sum(n * (c - n) + n * (n + 1) // 2 for n, c in zip(q, kv))


def work(case):
    q, kv = _lens(case)
    T, C = sum(q), sum(kv)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    row = d * 2 if case["fmt"] == "bf16" else d + 4  # one cached key or value row of one head, with its scale
    meta = 4 * (2 * case["batch"] + 1) + 4 * sum(-(-c // case["page"]) for c in kv)
    if case["op"] == "append":  # reads the new rows, writes the cache's; then reads the cache's and writes dense rows
        return {"bytes": 2 * T * hkv * (d * 2 + row + row + d * 2) + meta, "flops": 0}
    if case["op"] == "read":
        return {"bytes": 2 * T * hkv * (row + d * 2) + meta, "flops": 0}
    return {"bytes": 2 * T * hq * d * 2 + 2 * C * hkv * row + meta + (4 * T * hq if case["lse"] else 0),
            "flops": 4 * d * hq * _pairs(q, kv)}


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def draw(rng):
    """A case of the listed ranges: every operator, one token to thousands, contexts from none to 128K, odd lengths,
    other head layouts and page sizes."""
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    while True:
        kind = rng.choice(["append", "read", "decode", "decode", "draft", "prefill", "prefill"])
        hkv = rng.choice([1, 2, 2, 4, 8])
        g = rng.choice([1, 2, 4, 5, 8, 8, 16])
        c = _case(None, kind if kind in ("append", "read") else "attention", rng.choice(["bf16", "e4m3"]),
                  1, 1, 0, g * hkv, hkv, rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 64, 128]),
                  rng.choice([0, rng.randrange(1, 1 << 20), rng.randrange(1, 1 << 20)]), rng.random() < 0.25)
        if kind == "append":
            c["batch"], c["new"], c["past"] = log(1, 64), log(1, 8192), log(1, 9000) - 1
        elif kind == "read":
            c["batch"], c["new"] = log(1, 16), log(16, 131072)
        elif kind == "decode":
            c["batch"], c["past"] = log(1, 128), log(1, 131072) - 1
        elif kind == "draft":
            c["batch"], c["new"], c["past"] = log(1, 32), rng.randint(2, 16), log(16, 65536)
        else:
            c["batch"], c["new"], c["past"] = log(1, 8), log(17, 8192), log(1, 40000) - 1
        if c["op"] != "attention":
            c["lse"] = False
        q, kv = _lens(c)
        dense = c["batch"] * max(kv) * hkv * c["d"] * 8  # the plain form's dense keys and values in 32 bits
        scores = c["batch"] * c["hq"] * max(q) * max(kv) * 4
        if dense > 9e9 or scores > 1.0e10:
            continue
        if _cost(c) <= max(_cost(x) for x in listed() if x["op"] == c["op"]):
            return c


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
def _pow2_scale(amax):
    """The least power of two 2^e (e >= -126) with amax <= 448 * 2^e; 1 for amax = 0.  Exact: frexp and ldexp."""
    m, x = torch.frexp(amax)  # amax = m * 2^x, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, x - 9, x - 8).clamp(min=-126)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    return torch.ldexp(torch.ones_like(amax), e)


def _quantise(x):
    """float32 rows [..., d] -> (e4m3 values as float8_e4m3fn, float32 scale [...])."""
    s = _pow2_scale(x.abs().amax(-1))
    return (x / s[..., None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    """The caches, their page tables and the step's fused projection output.  With `own` also the framework's handles
    on these same tensors, which a user's program keeps from call to call."""
    dev = torch.device("cuda")
    q_len, kv_len = _lens(case)
    B, T, P = case["batch"], sum(q_len), case["page"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    need = [-(-c // P) for c in kv_len]
    n_pages = sum(need) + 3
    # pages handed out in no order, as after a while of serving; unused table entries hold 0
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros((B, max(need)), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n

    def pages():
        # rows of unlike magnitude, as keys and values are
        x = torch.randn((n_pages, hkv, P, d), generator=gen, device=dev)
        x *= torch.exp2(torch.randn((n_pages, hkv, P, 1), generator=gen, device=dev) * 0.5)
        if case["fmt"] == "bf16":
            return x.bfloat16(), None
        return _quantise(x.bfloat16().float())

    k_pages, k_scale = pages()
    v_pages, v_scale = pages()
    qkv = torch.randn((T, (hq + 2 * hkv) * d), generator=gen, device=dev).bfloat16()
    cu = [0]
    for n in q_len:
        cu.append(cu[-1] + n)
    s = {"case": dict(case), "T": T, "max_q": max(q_len), "k_pages": k_pages, "v_pages": v_pages,
         "k_scale": k_scale, "v_scale": v_scale, "page_table": table,
         "cu_q": torch.tensor(cu, dtype=torch.int32, device=dev),
         "kv_len": torch.tensor(kv_len, dtype=torch.int32, device=dev),
         "q": qkv[:, :hq * d].unflatten(1, (hq, d)),
         "k": qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
         "v": qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))}
    if own:
        from bit_mixture_experts_gb300 import PagedKVCache
        s["cache"] = PagedKVCache.from_tensors(k_pages, v_pages, k_scale, v_scale)
        s["batch"] = s["cache"].batch(table, s["cu_q"], s["kv_len"], T)
    return s


# --------------------------------------------------------------------------- #
# one pass
# --------------------------------------------------------------------------- #
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    c, cache, batch = s["case"], s["cache"], s["batch"]
    if c["op"] == "append":
        cache.append(s["k"], s["v"], batch)
        return cache.read(batch)
    if c["op"] == "read":
        return cache.read(batch)
    return cache.attention(s["q"], batch, return_lse=c["lse"])


def _token_rows(s):
    """Per new token: its page and its row in the page."""
    cu, kv = s["cu_q"].long(), s["kv_len"].long()
    t = torch.arange(s["T"], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = kv[b] - (cu[b + 1] - cu[b]) + t - cu[b]
    P = s["case"]["page"]
    return s["page_table"].long()[b, pos // P], pos % P


def _values(pages, scale):
    x = pages.float()
    return x if scale is None else x * scale[..., None]


def _run_plain(s):
    c = s["case"]
    if c["op"] == "attention":
        return _attention_plain(s)
    at = _token_rows(s)
    if c["op"] == "append":
        _write(s["k"], s["k_pages"], s["k_scale"], *at)
        _write(s["v"], s["v_pages"], s["v_scale"], *at)
    return _read(s["k_pages"], s["k_scale"], *at), _read(s["v_pages"], s["v_scale"], *at)


def _write(new, pages, scale, page, row):
    if scale is None:
        pages[page, :, row] = new
    else:
        x, sc = _quantise(new.float())
        pages.view(torch.uint8)[page, :, row] = x.view(torch.uint8)
        scale[page, :, row] = sc


def _read(pages, scale, page, row):
    if scale is None:
        return pages[page, :, row]
    x = pages.view(torch.uint8)[page, :, row].view(torch.float8_e4m3fn)
    return _values(x, scale[page, :, row]).bfloat16()


def _attention_plain(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    g, B, n = hq // hkv, c["batch"], s["max_q"]
    cu, kv, table = s["cu_q"].long(), s["kv_len"].long(), s["page_table"].long()

    def dense(pages, scale):  # [B, hkv, keys, d] in 32 bits
        x = pages.view(torch.uint8)[table].view(torch.float8_e4m3fn) if scale is not None else pages[table]
        x = _values(x, scale[table] if scale is not None else None)
        return x.transpose(1, 2).flatten(2, 3)

    k, v = dense(s["k_pages"], s["k_scale"]), dense(s["v_pages"], s["v_scale"])
    i = torch.arange(n, device=cu.device)
    q = s["q"][(cu[:-1, None] + i).clamp(max=s["T"] - 1)].float()  # [B, n, hq, d], padded
    q = q.unflatten(2, (hkv, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    scores = (q @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(d))
    q_len = cu[1:] - cu[:-1]
    seen = (kv - q_len)[:, None] + i + 1  # keys that new token i sees
    seen = seen.repeat_interleave(g, 1)[:, None, :, None]
    scores.masked_fill_(torch.arange(k.shape[2], device=cu.device) >= seen, float("-inf"))
    m = scores.amax(3, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = scores.sub_(m).exp_()
    total = p.sum(3, keepdim=True)
    o = torch.where(total > 0, (p @ v) / total, torch.zeros_like(total))
    lse = (m + total.log()).squeeze(3)
    t = torch.arange(s["T"], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    o = o.unflatten(2, (n, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)[b, t - cu[b]].bfloat16()
    if not c["lse"]:
        return o
    return o, lse.unflatten(2, (n, g)).permute(0, 2, 1, 3).flatten(2, 3)[b, t - cu[b]]


# --------------------------------------------------------------------------- #
# the definition in 64 bits
# --------------------------------------------------------------------------- #
def _e4m3_nearest(x):
    """The e4m3 value nearest to each element of a float64 tensor with |x| <= 448, ties to the even one: a grid of
    step 2^(floor(log2 |x|) - 3), no finer than 2^-9."""
    a = x.abs().clamp(min=2.0 ** -6)
    step = torch.exp2(torch.floor(torch.log2(a)) - 3)
    over = a / step  # in [8, 16] but for log2's rounding at powers of two
    step = torch.where(over >= 16, step * 2, torch.where(over < 8, step / 2, step))
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    hq, hkv, d, P = case["hq"], case["hkv"], case["d"], case["page"]
    q_len, kv_len = _lens(case)
    table = s["page_table"].cpu().tolist()

    def cached(pages, scale, b, lo, hi):
        """Rows lo .. hi - 1 of sequence b, [rows, hkv, d] in 64 bits."""
        ids = torch.tensor(table[b][lo // P:(hi + P - 1) // P], device=pages.device)
        x = (pages if scale is None else pages.view(torch.uint8)).index_select(0, ids)
        if scale is not None:
            x = x.view(torch.float8_e4m3fn).double() * scale.index_select(0, ids).double().unsqueeze(-1)
        x = x.double().permute(0, 2, 1, 3).reshape(-1, hkv, d)
        return x[lo % P:lo % P + hi - lo]

    if case["op"] == "append":
        out = []
        for x in (s["k"].double(), s["v"].double()):
            if case["fmt"] == "e4m3":
                a = x.abs().amax(2, keepdim=True)
                # the least power of two that brings the row within 448
                e = torch.ceil(torch.log2(a.clamp(min=1e-300) / E4M3_MAX)).clamp(min=-126)
                e = torch.where(a > E4M3_MAX * torch.exp2(e), e + 1, e)
                e = torch.where((a <= E4M3_MAX * torch.exp2(e - 1)) & (e > -126), e - 1, e)
                s2 = torch.where(a > 0, torch.exp2(e), torch.ones_like(a))
                x = _e4m3_nearest(x / s2) * s2
            out.append(x)
        return tuple(out)
    if case["op"] == "read":
        return tuple(torch.cat([cached(p, sc, b, kv_len[b] - n, kv_len[b]) for b, n in enumerate(q_len)])
                     for p, sc in ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"])))
    if 4 * d * hq * _pairs(q_len, kv_len) > 6e12:
        return None
    out = torch.zeros((s["T"], hq, d), dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros((s["T"], hq), dtype=torch.float64, device=s["q"].device)
    at = 0
    for b, n in enumerate(q_len):
        k = cached(s["k_pages"], s["k_scale"], b, 0, kv_len[b])
        v = cached(s["v_pages"], s["v_scale"], b, 0, kv_len[b])
        for lo in range(0, n, 1024):
            hi = min(n, lo + 1024)
            seen = kv_len[b] - n + hi
            hidden = (torch.arange(seen, device=k.device)[None, :]
                      > torch.arange(kv_len[b] - n + lo, kv_len[b] - n + hi, device=k.device)[:, None])
            for h in range(hq):
                z = s["q"][at + lo:at + hi, h].double() @ k[:seen, h // (hq // hkv)].T / math.sqrt(d)
                z[hidden] = -math.inf
                lse[at + lo:at + hi, h] = torch.logsumexp(z, 1)
                out[at + lo:at + hi, h] = torch.softmax(z, 1) @ v[:seen, h // (hq // hkv)]
        at += n
    return (out, lse) if case["lse"] else out
