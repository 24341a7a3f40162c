"""The serving operators around paged decode attention, as they are measured.

Three operators of a decode or prefill step:

* ``norm_rope``  RMS norm of every query and key head and the position
  rotation, in one pass (``decode_attn_qk_norm_rope``);
* ``append``     the same for keys on their way into the pages of an f16 paged
  cache, values beside them, optionally the queries in the same call
  (``decode_attn_append_paged_rope``);
* ``prefix``     decode attention of a batch whose sequences share the pages
  of a long prefix (``decode_attn_paged_prefix``).

``run`` computes them in elementary torch operations, or, with ``own`` set,
through the package.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
GOLDEN = 0.6180339887498949


# ------------------------------------------------------------------ the cases
def _nr(name, n, hq, hkv, d, t, rd, il=False, norm=True, far=4096):
    return dict(name=name, op="norm_rope", n=n, hq=hq, hkv=hkv, d=d, type=t, rd=rd, interleaved=il,
                norm=norm, far=far)


def _ap(name, seqs, n, hq, hkv, d, t, rd, bs, past, il=False, norm=False):
    return dict(name=name, op="append", seqs=seqs, n=n, hq=hq, hkv=hkv, d=d, type=t, rd=rd, bs=bs,
                past=past, interleaved=il, norm=norm)


def _px(name, b, t, hq, hkv, d, bs, prefix, smin, smax, window=0, softcap=0.0, short=0, empty=0):
    return dict(name=name, op="prefix", b=b, t=t, hq=hq, hkv=hkv, d=d, bs=bs, prefix=prefix,
                smin=smin, smax=smax, window=window, softcap=softcap, short=short, empty=empty)


def listed():
    return [
        # one token of a small model: latency alone
        _nr("norm_rope_token", 1, 8, 2, 64, "f16", 64),
        # a decode batch of a large grouped-query model, sliced from its fused projection
        _nr("norm_rope_batch", 128, 64, 8, 128, "bf16", 128, far=32768),
        # a long prompt's prefill (odd length)
        _nr("norm_rope_prefill", 16381, 32, 8, 128, "bf16", 128, far=131072),
        # one token of one sequence, no norm
        _ap("append_token", 1, 1, 0, 2, 64, "f16", 64, 16, 255),
        # a decode step: one token of each of 32 sequences, queries and norms in the same call
        _ap("append_batch", 32, 32, 32, 8, 128, "bf16", 128, 16, 4095, norm=True),
        # drafted tokens of 64 sequences, wide heads, half of each head rotated in adjacent pairs
        _ap("append_drafts", 64, 256, 16, 8, 256, "f32", 128, 32, 8191, il=True),
        # five prompts' ragged prefill (odd total)
        _ap("append_prefill", 5, 12287, 0, 8, 128, "bf16", 128, 16, 2000),
        # two short requests of a small model
        _px("prefix_tiny", 2, 1, 8, 2, 64, 16, 192, 8, 64),
        # 32 chats behind one system prompt; one slot empty, one sequence shorter than the prompt
        _px("prefix_chat", 32, 1, 32, 8, 128, 16, 4096, 16, 512, short=1, empty=1),
        # four drafted tokens of 24 sequences over a shared document
        _px("prefix_drafts", 24, 4, 32, 8, 128, 16, 8192, 64, 1400),
        # sliding window and softcap, wide heads; the window cuts into the prefix
        _px("prefix_window", 64, 1, 16, 8, 256, 32, 6144, 256, 2048, window=4096, softcap=50.0),
        # 128 sequences over a long shared context
        _px("prefix_long", 128, 1, 64, 8, 128, 16, 32768, 64, 2048),
    ]


def _loguniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "prefix"])
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8])
    rd = rng.choice([d, d, d // 2, d // 4])
    t = rng.choice(["f16", "bf16", "f32"])
    if op == "norm_rope":
        c = _nr("", _loguniform(rng, 1, 12000), hkv * g, hkv, d, t, rd, rng.random() < 0.5,
                rng.random() < 0.8, rng.choice([4096, 32768, 131072, 1 << 20]))
    elif op == "append":
        seqs = _loguniform(rng, 1, 96)
        c = _ap("", seqs, seqs * _loguniform(rng, 1, max(2, 12000 // seqs)),
                hkv * g if rng.random() < 0.5 else 0, hkv, d, t, rd, rng.choice([8, 16, 32, 64]),
                _loguniform(rng, 1, 6000), rng.random() < 0.5, rng.random() < 0.5)
    else:
        b, tok = _loguniform(rng, 1, 96), rng.choice([1, 1, 1, 2, 4])
        hi = _loguniform(rng, 2, 1500)
        c = _px("", b, tok, hkv * g, hkv, d, rng.choice([8, 16, 32, 64, 128]),
                _loguniform(rng, 64, 12000), max(1, hi // rng.choice([1, 4, 30])), hi,
                rng.choice([0, 0, 0, 500, 4096]), rng.choice([0.0, 0.0, 30.0, 50.0]),
                min(b - 1, rng.choice([0, 0, 1])), min(b - 1, rng.choice([0, 0, 1])))
    del c["name"]
    return c


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _inv_freq(rd):
    """Radians a position for each rotated pair: 10000^(-2i/rd), in 64 bits."""
    return 10000.0 ** (-2.0 * np.arange(rd // 2, dtype=np.float64) / rd)


def _turns(rd):
    """The rotation plan a program keeps: turns a position, in units of 2^-64."""
    f = _inv_freq(rd) / (2.0 * math.pi)
    return torch.tensor(np.rint(f * 2.0 ** 64).astype(np.uint64).view(np.int64), device=DEV)


def _projection(g, n, heads, d, t):
    """Rows as a fused projection leaves them: every head of a token side by side."""
    return torch.randn((n, heads * d), generator=g, device=DEV).mul_(1.5).to(TYPES[t])


def _weight(g, d):
    return 1.0 + 0.2 * torch.randn((d,), generator=g, device=DEV)


def _suffix_lens(c):
    """Keys a sequence has past the prefix, log-uniform over [smin, smax]; the
    same multiset for every seed."""
    b = np.arange(c["b"])
    u = np.mod(0.5 + b * GOLDEN, 1.0)
    return np.rint(c["smin"] * (c["smax"] / c["smin"]) ** u).astype(np.int64)


def _prefix_pages(c):
    return c["prefix"] // c["bs"]


def _seq_lens(c):
    lens = _prefix_pages(c) * c["bs"] + _suffix_lens(c)
    for i in range(c["short"]):  # shorter than the prefix
        lens[1 + i] = max(1, c["prefix"] // 3)
    for i in range(c["empty"]):  # a slot without a request
        lens[c["b"] - 1 - i] = 0
    return lens


def _token_split(c):
    """Tokens a sequence brings: even but for the ragged remainder."""
    n, s = c["n"], c["seqs"]
    per = np.full(s, n // s)
    per[: n - (n // s) * s] += 1
    if n > 4 * s:  # prompts are ragged
        for i in range(s // 2):
            k = per[i] // 3
            per[i] -= k
            per[s - 1 - i] += k
    return per


def prepare(case, seed):
    c, g, r = case, _gen(seed), np.random.RandomState(seed)
    if c["op"] == "norm_rope":
        h = c["hq"] + c["hkv"]
        qkv = _projection(g, c["n"], h + c["hkv"], c["d"], c["type"]).view(c["n"], -1, c["d"])
        return dict(c=c, q=qkv[:, : c["hq"]], k=qkv[:, c["hq"]: h], turns=_turns(c["rd"]),
                    pos=torch.randint(0, c["far"], (c["n"],), generator=g, device=DEV,
                                      dtype=torch.int32),
                    qw=_weight(g, c["d"]), kw=_weight(g, c["d"]))
    if c["op"] == "append":
        qkv = _projection(g, c["n"], c["hq"] + 2 * c["hkv"], c["d"], c["type"])
        qkv = qkv.view(c["n"], -1, c["d"])
        per = _token_split(c)
        past = np.maximum(0, c["past"] - r.randint(0, max(1, c["past"] // 2), c["seqs"]))
        need = -(-(past + per) // c["bs"])
        mb = -(-(c["past"] + int(per.max())) // c["bs"])
        nb = c["seqs"] * mb + 7
        perm = r.permutation(nb)
        table = np.full((c["seqs"], mb), -1, np.int32)
        for b in range(c["seqs"]):
            table[b, : need[b]] = perm[b * mb: b * mb + need[b]]
        seq = np.repeat(np.arange(c["seqs"]), per)
        pos = np.concatenate([np.arange(p, p + k) for p, k in zip(past, per)])
        shape = (nb, c["bs"], c["hkv"], c["d"])
        return dict(c=c, q=qkv[:, : c["hq"]] if c["hq"] else None,
                    k=qkv[:, c["hq"]: c["hq"] + c["hkv"]], v=qkv[:, c["hq"] + c["hkv"]:],
                    turns=_turns(c["rd"]), pos=torch.tensor(pos, dtype=torch.int32, device=DEV),
                    seq=torch.tensor(seq, dtype=torch.int32, device=DEV),
                    table=torch.tensor(table, device=DEV), qw=_weight(g, c["d"]),
                    kw=_weight(g, c["d"]),
                    k_pool=torch.randn(shape, generator=g, device=DEV, dtype=torch.float16),
                    v_pool=torch.randn(shape, generator=g, device=DEV, dtype=torch.float16))
    lens = _seq_lens(c)
    keep = c["b"] - c["empty"]
    lens[:keep] = r.permutation(lens[:keep])
    pages = _prefix_pages(c)
    own_pages = np.maximum(0, -(-lens // c["bs"]) - pages)
    mb = pages + max(1, int(own_pages.max()))
    nb = pages + int(own_pages.sum()) + 5
    perm = r.permutation(nb).astype(np.int32)
    table = np.full((c["b"], mb), -1, np.int32)
    table[:, :pages] = perm[:pages]
    at = pages
    for b in range(c["b"]):
        table[b, pages: pages + own_pages[b]] = perm[at: at + own_pages[b]]
        at += own_pages[b]
    shape = (nb, c["bs"], c["hkv"], c["d"])
    qs = (c["b"], c["t"], c["hq"], c["d"]) if c["t"] > 1 else (c["b"], c["hq"], c["d"])
    return dict(c=c, q=torch.randn(qs, generator=g, device=DEV),
                k_pool=torch.randn(shape, generator=g, device=DEV, dtype=torch.float16),
                v_pool=torch.randn(shape, generator=g, device=DEV, dtype=torch.float16),
                table=torch.tensor(table, device=DEV), max_len=int(lens.max()),
                longest=int(max(1, own_pages.max())) * c["bs"],
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV))


# ------------------------------------------------------------------ plain forms
EPS = 1e-6


def _normed(x, w, norm):
    x = x.float()
    if not norm:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _rotated(x, pos, turns, interleaved):
    """x f32 [N, H, D]; the angle of pair i is pos * turns[i] / 2^64 turns, whose whole
    turns drop out of the 64-bit product."""
    a = (pos.long()[:, None] * turns[None, :]).double() * (2.0 * math.pi / 2.0 ** 64)
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    half = turns.shape[0]
    y = x.clone()
    if interleaved:
        x0, x1 = x[..., 0: 2 * half: 2], x[..., 1: 2 * half: 2]
        y[..., 0: 2 * half: 2] = x0 * cos - x1 * sin
        y[..., 1: 2 * half: 2] = x0 * sin + x1 * cos
    else:
        x0, x1 = x[..., :half], x[..., half: 2 * half]
        y[..., :half] = x0 * cos - x1 * sin
        y[..., half: 2 * half] = x0 * sin + x1 * cos
    return y


def _plain_norm_rope(s):
    c = s["c"]
    q = _rotated(_normed(s["q"], s["qw"], c["norm"]), s["pos"], s["turns"], c["interleaved"])
    k = _rotated(_normed(s["k"], s["kw"], c["norm"]), s["pos"], s["turns"], c["interleaved"])
    return {"q": q, "k": k.half()}


def _plain_append(s):
    c = s["c"]
    k = _rotated(_normed(s["k"], s["kw"], c["norm"]), s["pos"], s["turns"], c["interleaved"])
    pos = s["pos"].long()
    page = s["table"].long()[s["seq"].long(), pos // c["bs"]]
    s["k_pool"][page, pos % c["bs"]] = k.half()
    s["v_pool"][page, pos % c["bs"]] = s["v"].float().half()
    out = {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    if c["hq"]:
        out["q"] = _rotated(_normed(s["q"], s["qw"], c["norm"]), s["pos"], s["turns"],
                            c["interleaved"])
    return out


def _scores(x, c):
    x = x * float(np.float32(1.0 / math.sqrt(c["d"])))
    return c["softcap"] * torch.tanh(x / c["softcap"]) if c["softcap"] else x


def _plain_prefix(s):
    """The prefix's scores of all rows in one product a kv head, each
    sequence's own in another, and one softmax over both."""
    c = s["c"]
    B, T, H, D, bs = c["b"], c["t"], c["hkv"], c["d"], c["bs"]
    G = c["hq"] // H
    pages = _prefix_pages(c)
    P = pages * bs
    q = s["q"].view(B, T, H, G, D)
    L = s["lens"].long()
    qp = (L - T)[:, None] + torch.arange(T, device=DEV)  # [B, T]
    lo = torch.where(qp >= c["window"], qp - c["window"] + 1, 0) if c["window"] else qp * 0
    hi = torch.minimum(qp + 1, L[:, None])

    def seen(keys):  # [B, T, keys]
        return (keys >= lo[..., None]) & (keys < hi[..., None])

    kp = s["k_pool"][s["table"][0, :pages].long()].view(P, H, D).float()
    vp = s["v_pool"][s["table"][0, :pages].long()].view(P, H, D).float()
    qh = q.permute(2, 0, 1, 3, 4).reshape(H, B * T * G, D)
    sp = _scores(torch.matmul(qh, kp.permute(1, 2, 0)), c).view(H, B, T, G, P)
    ok = seen(torch.arange(P, device=DEV))
    sp = sp.masked_fill(~ok[None, :, :, None], -math.inf)
    S = s["longest"]
    own_pages = s["table"][:, pages: pages + S // bs].long().clamp(min=0)
    ks = s["k_pool"][own_pages].view(B, S, H, D).float()
    vs = s["v_pool"][own_pages].view(B, S, H, D).float()
    qb = q.permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D)
    ss = _scores(torch.matmul(qb, ks.permute(0, 2, 3, 1)), c).view(B, H, T, G, S)
    ok = seen(P + torch.arange(S, device=DEV))
    ss = ss.masked_fill(~ok[:, None, :, None], -math.inf)
    ss = ss.permute(1, 0, 2, 3, 4)  # [H, B, T, G, S]
    m = torch.maximum(sp.amax(-1), ss.amax(-1)) if pages else ss.amax(-1)
    m0 = torch.where(m == -math.inf, 0.0, m)[..., None]
    wp, ws = torch.exp(sp - m0), torch.exp(ss - m0)
    total = wp.sum(-1) + ws.sum(-1)  # [H, B, T, G]
    o = torch.matmul(wp.view(H, B * T * G, P), vp.permute(1, 0, 2)).view(H, B, T, G, D)
    own_o = torch.matmul(ws.permute(1, 0, 2, 3, 4).reshape(B, H, T * G, S), vs.permute(0, 2, 1, 3))
    o = o + own_o.view(B, H, T, G, D).permute(1, 0, 2, 3, 4)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    lse = m + torch.log(total)
    return {"out": o.permute(1, 2, 0, 3, 4).reshape(s["q"].shape),
            "lse": lse.permute(1, 2, 0, 3).reshape(s["q"].shape[:-1])}


# ------------------------------------------------------------------ the package's calls
def _own_norm_rope(s):
    import quantized_kv_decode_paged_gb300 as qk
    c = s["c"]
    q, k = qk.decode_attn_qk_norm_rope(s["q"], s["k"], s["pos"], s["turns"], norm=c["norm"],
                                       q_weight=s["qw"] if c["norm"] else None,
                                       k_weight=s["kw"] if c["norm"] else None, eps=EPS,
                                       interleaved=c["interleaved"])
    return {"q": q, "k": k}


def _own_append(s):
    import quantized_kv_decode_paged_gb300 as qk
    c = s["c"]
    q = qk.decode_attn_append_paged_rope(s["k"], s["v"], s["pos"], s["table"], s["k_pool"],
                                         s["v_pool"], s["turns"], token_seq=s["seq"], q=s["q"],
                                         norm=c["norm"], q_weight=s["qw"] if c["norm"] else None,
                                         k_weight=s["kw"] if c["norm"] else None, eps=EPS,
                                         interleaved=c["interleaved"])
    out = {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    if c["hq"]:
        out["q"] = q
    return out


def _own_prefix(s):
    import quantized_kv_decode_paged_gb300 as qk
    c = s["c"]
    out, lse = qk.decode_attn_paged_prefix(s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"],
                                           _prefix_pages(c) * c["bs"], softcap=c["softcap"],
                                           sliding_window=c["window"], max_seq_len=s["max_len"])
    return {"out": out, "lse": lse}


def run(state):
    op = state["c"]["op"]
    if own:
        return {"norm_rope": _own_norm_rope, "append": _own_append, "prefix": _own_prefix}[op](state)
    return {"norm_rope": _plain_norm_rope, "append": _plain_append,
            "prefix": _plain_prefix}[op](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    e = 4 if c.get("type") == "f32" else 2
    if c["op"] == "norm_rope":
        rows = c["n"] * c["d"]
        return {"bytes": rows * (c["hq"] * (e + 4) + c["hkv"] * (e + 2)) + 4 * c["n"] + 4 * c["rd"],
                "flops": rows * (c["hq"] + c["hkv"]) * (7 if c["norm"] else 3)}
    if c["op"] == "append":
        rows = c["n"] * c["d"]
        return {"bytes": rows * (c["hq"] * (e + 4) + 2 * c["hkv"] * (e + 2)) + 12 * c["n"]
                + 4 * c["rd"], "flops": rows * (c["hq"] + c["hkv"]) * (7 if c["norm"] else 3)}
    P = _prefix_pages(c) * c["bs"]
    L = _seq_lens(c)
    rows = c["b"] * c["t"] * c["hq"]
    tok = np.arange(c["t"])
    qp = L[:, None] - c["t"] + tok
    lo = np.where(qp >= c["window"], qp - c["window"] + 1, 0) if c["window"] else qp * 0
    hi = np.minimum(qp + 1, L[:, None])
    keys = int(np.maximum(0, hi - lo).sum())  # keys seen, over sequences and tokens
    own_keys = int(np.maximum(0, L - np.maximum(P, lo[:, 0])).sum())
    ph, pl = min(P, int(hi.max())), min(P, int(lo[L > 0].min()) if (L > 0).any() else 0)
    kv = (max(0, ph - pl) + own_keys) * c["hkv"] * c["d"] * 4
    return {"bytes": kv + rows * (c["d"] * 8 + 4), "flops": 4 * keys * c["hq"] * c["d"]}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_rows(x, w, pos, c):
    """numpy, one pair at a time along the last axis, angles pos * 10000^(-2i/rd)."""
    y = x.double().cpu().numpy()
    if c["norm"]:
        y = y / np.sqrt(np.mean(np.square(y), axis=-1, keepdims=True) + EPS)
        y = y * w.double().cpu().numpy()
    z = y.copy()
    p = pos.cpu().numpy().astype(np.float64)
    for i, f in enumerate(_inv_freq(c["rd"])):
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + c["rd"] // 2)
        co, si = np.cos(p * f)[:, None], np.sin(p * f)[:, None]
        z[..., a] = y[..., a] * co - y[..., b] * si
        z[..., b] = y[..., a] * si + y[..., b] * co
    return z


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm_rope":
        return {"q": _exact_rows(s["q"], s["qw"], s["pos"], c),
                "k": _exact_rows(s["k"], s["kw"], s["pos"], c)}
    if c["op"] == "append":
        k = _exact_rows(s["k"], s["kw"], s["pos"], c)
        v = s["v"].double().cpu().numpy()
        kp, vp = s["k_pool"].double().cpu().numpy(), s["v_pool"].double().cpu().numpy()
        pos, seq = s["pos"].cpu().numpy(), s["seq"].cpu().numpy()
        table = s["table"].cpu().numpy()
        for n in range(c["n"]):
            page, row = table[seq[n], pos[n] // c["bs"]], pos[n] % c["bs"]
            kp[page, row], vp[page, row] = k[n], v[n]
        out = {"k_pool": kp, "v_pool": vp}
        if c["hq"]:
            out["q"] = _exact_rows(s["q"], s["qw"], s["pos"], c)
        return out
    # each sequence alone, through its own table, in 64-bit products
    T, H, D, G = c["t"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    q = s["q"].double().view(c["b"], T, c["hq"], D)
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device=DEV)
    for b, L in enumerate(s["lens"].tolist()):
        for t in range(T):
            p = L - T + t
            first = p - c["window"] + 1 if c["window"] and p >= c["window"] else 0
            if p < first:
                continue
            key = torch.arange(first, p + 1, device=DEV)
            page = s["table"][b].long()[key // c["bs"]]
            k = s["k_pool"][page, key % c["bs"]].double()
            v = s["v_pool"][page, key % c["bs"]].double()
            x = torch.einsum("hgd,khd->hgk", q[b, t].view(H, G, D), k)
            x = x * float(np.float32(1.0 / math.sqrt(D)))
            if c["softcap"]:
                x = c["softcap"] * torch.tanh(x / c["softcap"])
            lse[b, t] = torch.logsumexp(x, -1).reshape(-1)
            w = torch.softmax(x, -1)
            out[b, t] = torch.einsum("hgk,khd->hgd", w, v).reshape(c["hq"], D)
    return {"out": out.view(s["q"].shape), "lse": lse.view(s["q"].shape[:-1])}
