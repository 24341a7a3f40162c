"""The operators of a paged cache held in 4 bits, as they are measured.

A serving step over such a cache has four:

* ``plan``    pages for requests that grow and from requests that shrink or end,
  and the places of their new tokens, worked out on the GPU from the request
  lengths (``decode_attn_plan_blocks``);
* ``append``  new keys and values quantised to 4 bits into their pages, the keys
  optionally normed and rotated on the way (``decode_attn_append_paged_q4``);
* ``gather``  cached tokens back as f16 rows (``decode_attn_gather_paged_q4``);
* ``attend``  decode attention over the pages (``decode_attn_paged_q4``).

``run`` computes them in elementary torch operations, or, with ``own`` set,
through the package.

The cache: uint8 [pages, Hkv, page bytes].  A group of ``group`` neighbouring
values of a row has f16 (zero, scale): zero = min, scale = (max - min) / 15, and
a value is scale * code + zero with code = round((x - zero) / scale) in 0..15.
A page of one kv head holds the key codes of its rows (D/2 bytes each, value 2j
in the low half of byte j), the value codes, then (scale, zero) of every row and
group of the keys and of the values.  The 16-byte pieces of row t are permuted:
piece c lies at place c ^ (t / (256 / D)) % (D / 32).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
GOLDEN = 0.6180339887498949
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def _pl(name, b, bs, mb, grow, new, past, ended):
    """b requests: `grow` of them bring up to `new` tokens each, `ended` end, the rest wait."""
    return dict(name=name, op="plan", b=b, bs=bs, mb=mb, grow=grow, new=new, past=past, ended=ended)


def _ap(name, seqs, n, hq, hkv, d, group, t, rd, bs, past, il=False):
    return dict(name=name, op="append", seqs=seqs, n=n, hq=hq, hkv=hkv, d=d, group=group, type=t,
                rd=rd, bs=bs, past=past, interleaved=il)


def _ga(name, seqs, n, hkv, d, group, bs):
    return dict(name=name, op="gather", seqs=seqs, n=n, hkv=hkv, d=d, group=group, bs=bs)


def _at(name, b, t, hq, hkv, d, group, bs, lmin, lmax, window=0, softcap=0.0, empty=0):
    return dict(name=name, op="attend", b=b, t=t, hq=hq, hkv=hkv, d=d, group=group, bs=bs,
                lmin=lmin, lmax=lmax, window=window, softcap=softcap, empty=empty)


def listed():
    return [
        # a decode step: 256 requests, a token each, every sixteenth needs a page
        _pl("plan_step", 256, 16, 512, 256, 1, 4000, 0),
        # a busy server: 2000 slots, prompts come in, hundreds of requests end
        _pl("plan_busy", 2000, 16, 512, 300, 400, 6000, 500),
        # one token of a small model: latency alone
        _ap("append_token", 1, 1, 0, 2, 64, 32, "f16", 0, 16, 255),
        # a decode step of 64 sequences: keys and queries normed and rotated in the same call
        _ap("append_step", 64, 64, 32, 8, 128, 32, "bf16", 128, 16, 4095),
        # five prompts' ragged prefill (odd total); their own attention has rotated the keys
        _ap("append_prompts", 5, 12287, 0, 8, 128, 128, "bf16", 0, 16, 2000),
        # a short request's cache handed on
        _ga("gather_request", 1, 333, 2, 64, 32, 16),
        # the past of seven long requests, for the next chunk of their prompts (odd total)
        _ga("gather_past", 7, 40003, 8, 128, 64, 32),
        # two short requests of a small model
        _at("attend_tiny", 2, 1, 8, 2, 64, 32, 16, 100, 256),
        # 32 chats, one slot empty
        _at("attend_chat", 32, 1, 32, 8, 128, 64, 16, 512, 4096, empty=1),
        # four drafted tokens of 24 sequences
        _at("attend_drafts", 24, 4, 32, 8, 128, 128, 16, 1000, 9000),
        # wide heads behind a sliding window, with softcap
        _at("attend_window", 64, 1, 16, 8, 256, 128, 32, 3000, 8192, window=4096, softcap=50.0),
        # 128 long sequences of a large grouped-query model
        _at("attend_long", 128, 1, 64, 8, 128, 128, 16, 2048, 24000),
    ]


def _loguniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "gather", "attend", "attend"])
    d = rng.choice([64, 128, 256])
    group = min(d, rng.choice([32, 64, 128]))
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8])
    bs = rng.choice([8, 16, 32, 64, 128])
    if op == "plan":
        b = _loguniform(rng, 1, 2000)
        grow = _loguniform(rng, 1, b)
        past = _loguniform(rng, 10, 6000)
        new = _loguniform(rng, 1, 400)
        c = _pl("", b, bs, -(-(past + new) // bs) + rng.randint(0, 40), grow, new, past,
                rng.randint(0, b - grow))
    elif op == "append":
        seqs = _loguniform(rng, 1, 96)
        t = rng.choice(["f16", "bf16", "f32"])
        # rows that are normed and rotated are those of decode steps; prompts' come ready
        rotated = rng.random() < 0.5
        n = (seqs * rng.choice([1, 1, 2, 4]) if rotated
             else seqs * _loguniform(rng, 1, max(2, 12000 // seqs)))
        c = _ap("", seqs, n, hkv * g if rng.random() < 0.7 and rotated else 0, hkv, d,
                32 if rotated else group, t, rng.choice([d, d, d // 2, d // 4]) if rotated else 0,
                bs, _loguniform(rng, 1, 6000), rng.random() < 0.5)
    elif op == "gather":
        seqs = _loguniform(rng, 1, 40)
        c = _ga("", seqs, seqs * _loguniform(rng, 1, max(2, 30000 // seqs)), hkv, d, group, bs)
    else:
        b, tok = _loguniform(rng, 1, 96), rng.choice([1, 1, 1, 2, 4])
        hi = _loguniform(rng, 20, 12000)
        c = _at("", b, tok, hkv * g, hkv, d, group, bs, max(tok, hi // rng.choice([1, 3, 10])), hi,
                rng.choice([0, 0, 0, 500, 4096]), rng.choice([0.0, 0.0, 30.0, 50.0]),
                min(b - 1, rng.choice([0, 0, 1])))
    del c["name"]
    return c


# ------------------------------------------------------------------ the inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _spread(n, lo, hi):
    """n lengths, log-uniform over [lo, hi]; the same ones for every seed."""
    u = np.mod(0.5 + np.arange(n) * GOLDEN, 1.0)
    return np.rint(lo * (hi / lo) ** u).astype(np.int64)


def _lens(c):
    lens = _spread(c["b"], c["lmin"], c["lmax"])
    lens[c["b"] - c["empty"]:] = 0
    return lens


def _split(n, seqs):
    """Tokens a sequence brings: even but for the ragged remainder."""
    per = np.full(seqs, n // seqs)
    per[: n - (n // seqs) * seqs] += 1
    if n > 4 * seqs:  # prompts are ragged
        for i in range(seqs // 2):
            k = per[i] // 3
            per[i] -= k
            per[seqs - 1 - i] += k
    return per


def _request_lens(c):
    """(lengths before, lengths after) of a plan: the same multiset for every seed."""
    old = _spread(c["b"], max(1, c["past"] // 4), c["past"])
    new = old.copy()
    new[: c["grow"]] += _spread(c["grow"], 1, c["new"])
    new[c["b"] - c["ended"]:] = 0
    return old, new


def _page_bytes(c):
    return c["bs"] * (c["d"] + 8 * (c["d"] // c["group"]))


def _tables(r, lens, bs, spare):
    """Block table of sequences of these lengths, pages in any order, and how many pages there are."""
    need = -(-lens // bs)
    mb, nb = max(1, int(need.max())), int(need.sum()) + spare
    perm = r.permutation(nb).astype(np.int32)
    table = np.full((len(lens), mb), -1, np.int32)
    at = np.concatenate([[0], np.cumsum(need)])
    for b in range(len(lens)):
        table[b, : need[b]] = perm[at[b]: at[b + 1]]
    return table, nb


def _pool(g, c, pages):
    """A cache as appends of normal keys and values left it."""
    shape = (pages, c["hkv"], c["bs"], c["d"])
    pool = torch.empty((pages, c["hkv"], _page_bytes(c)), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // (c["hkv"] * c["bs"] * c["d"]))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        x = torch.randn((2, n) + shape[1:], generator=g, device=DEV)
        pool[i: i + n] = _pages(*_quantised(x, c["group"]), c)
    return pool


def _turns(rd):
    """The rotation plan a program keeps: turns a position, in units of 2^-64."""
    f = 10000.0 ** (-2.0 * np.arange(rd // 2, dtype=np.float64) / rd) / (2.0 * math.pi)
    return torch.tensor(np.rint(f * 2.0 ** 64).astype(np.uint64).view(np.int64), device=DEV)


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c, g, r = case, _gen(seed), np.random.RandomState(seed)
    if c["op"] == "plan":
        old, new = _request_lens(c)
        order = r.permutation(c["b"])
        old, new = old[order], new[order]
        po, pn = -(-old // c["bs"]), -(-new // c["bs"])
        pages = int(np.maximum(po, pn).sum()) + 64
        perm = r.permutation(pages).astype(np.int32)
        # table, free list and its count side by side: one copy takes the whole state
        held = int(po.sum())
        state = np.full(c["b"] * c["mb"] + pages + 1, -1, np.int32)
        table = state[: c["b"] * c["mb"]].reshape(c["b"], c["mb"])
        at = np.concatenate([[0], np.cumsum(po)])
        for b in range(c["b"]):
            table[b, : po[b]] = perm[at[b]: at[b + 1]]
        state[c["b"] * c["mb"]: c["b"] * c["mb"] + pages - held] = perm[held:]
        state[-1] = pages - held
        tokens = int(np.maximum(new - old, 0).sum())
        return dict(c=c, state=_int(state), pages=pages, old=_int(old), new=_int(new),
                    tokens=tokens + tokens // 8 + 1)
    if c["op"] == "append":
        qkv = torch.randn((c["n"], (c["hq"] + 2 * c["hkv"]) * c["d"]), generator=g, device=DEV)
        qkv = qkv.mul_(1.5).to(TYPES[c["type"]]).view(c["n"], -1, c["d"])  # a fused projection's
        per = _split(c["n"], c["seqs"])
        past = np.maximum(0, c["past"] - r.randint(0, max(1, c["past"] // 2), c["seqs"]))
        table, nb = _tables(r, past + per, c["bs"], 7)
        pos = np.concatenate([np.arange(p, p + k) for p, k in zip(past, per)])
        return dict(c=c, q=qkv[:, : c["hq"]] if c["hq"] else None,
                    k=qkv[:, c["hq"]: c["hq"] + c["hkv"]], v=qkv[:, c["hq"] + c["hkv"]:],
                    turns=_turns(c["rd"]) if c["rd"] else None, pos=_int(pos),
                    seq=_int(np.repeat(np.arange(c["seqs"]), per)), table=_int(table),
                    qw=1.0 + 0.2 * torch.randn((c["d"],), generator=g, device=DEV),
                    kw=1.0 + 0.2 * torch.randn((c["d"],), generator=g, device=DEV),
                    pool=torch.zeros((nb, c["hkv"], _page_bytes(c)), dtype=torch.uint8, device=DEV))
    if c["op"] == "gather":
        per = _split(c["n"], c["seqs"])
        table, nb = _tables(r, per, c["bs"], 3)
        return dict(c=c, pool=_pool(g, c, nb), table=_int(table),
                    seq=_int(np.repeat(np.arange(c["seqs"]), per)),
                    pos=_int(np.concatenate([np.arange(k) for k in per])))
    lens = _lens(c)
    keep = c["b"] - c["empty"]
    lens[:keep] = r.permutation(lens[:keep])
    table, nb = _tables(r, lens, c["bs"], 5)
    shape = (c["b"], c["t"], c["hq"], c["d"]) if c["t"] > 1 else (c["b"], c["hq"], c["d"])
    return dict(c=c, q=torch.randn(shape, generator=g, device=DEV), pool=_pool(g, c, nb),
                table=_int(table), lens=_int(lens), max_len=int(lens.max()))


# ------------------------------------------------------------------ plain forms
def _quantised(x, group):
    """x f32 [..., D] -> codes uint8 [..., D], params f16 [..., D / group, 2] (scale, zero)."""
    y = x.unflatten(-1, (-1, group))
    lo, hi = y.amin(-1), y.amax(-1)
    zero, scale = lo.half(), ((hi - lo) / 15).half()
    s, z = scale.float()[..., None], zero.float()[..., None]
    code = torch.where(s > 0, torch.round((y - z) / s).clamp(0, 15), 0.0)
    return code.to(torch.uint8).flatten(-2), torch.stack([scale, zero], -1)


def _dequantised(codes, params):
    """The f32 values of codes [..., D] with params [..., D / group, 2]."""
    p = params.float()
    y = codes.float().unflatten(-1, (p.shape[-2], -1))
    return (y * p[..., :1] + p[..., 1:]).flatten(-2)


def _piece_order(c):
    """[bs, D / 32]: where piece j of row t lies."""
    t = torch.arange(c["bs"], device=DEV)[:, None]
    j = torch.arange(c["d"] // 32, device=DEV)[None]
    return j ^ (t // (256 // c["d"])) % (c["d"] // 32)


def _pages(codes, params, c):
    """Pages [n, Hkv, bytes] of codes [2, n, Hkv, bs, D] and their params."""
    packed = codes[..., 0::2] | codes[..., 1::2] << 4
    n, order = codes.shape[1], _piece_order(c)
    pieces = packed.unflatten(-1, (-1, 16)).permute(1, 2, 0, 3, 4, 5)  # n, Hkv, 2, bs, piece, 16
    t = torch.arange(c["bs"], device=DEV)[:, None]
    head = pieces[:, :, :, t, order].reshape(n, c["hkv"], -1)  # the permutation is its own inverse
    tail = params.permute(1, 2, 0, 3, 4, 5).contiguous().view(torch.uint8).reshape(n, c["hkv"], -1)
    return torch.cat([head, tail], -1)


def _unpaged(pages, c):
    """codes [2, n, Hkv, bs, D], params [2, n, Hkv, bs, D / group, 2] of pages [n, Hkv, bytes]."""
    n, bs, d = pages.shape[0], c["bs"], c["d"]
    head = pages[..., : bs * d].reshape(n, c["hkv"], 2, bs, -1, 16)
    t = torch.arange(bs, device=DEV)[:, None]
    packed = head[:, :, :, t, _piece_order(c)].flatten(-2).permute(2, 0, 1, 3, 4)
    codes = torch.stack([packed & 15, packed >> 4], -1).flatten(-2)
    tail = pages[..., bs * d:].contiguous().view(torch.float16)
    return codes, tail.reshape(n, c["hkv"], 2, bs, -1, 2).permute(2, 0, 1, 3, 4, 5)


def _offsets(c, page, row, heads):
    """Byte offsets in the flat pool of the rows (page, row): code bytes [2, N, Hkv, D / 2] and
    param bytes [2, N, Hkv, 4 D / group]."""
    bs, d, rec = c["bs"], c["d"], _page_bytes(c)
    at = (page[:, None] * heads + torch.arange(heads, device=DEV)) * rec  # [N, Hkv]
    j = torch.arange(d // 2, device=DEV)
    place = (j // 16 ^ (row[:, None] // (256 // d)) % (d // 32)) * 16 + j % 16
    code = at[..., None] + (row[:, None] * (d // 2) + place)[:, None]
    w = 4 * (d // c["group"])
    param = (at + bs * d)[..., None] + (row[:, None] * w + torch.arange(w, device=DEV))[:, None]
    two = torch.arange(2, device=DEV)[:, None, None, None]
    return code + two * (bs * d // 2), param + two * (bs * w)


def _rows(s):
    """Page and row of each token."""
    pos, bs = s["pos"].long(), s["c"]["bs"]
    return s["table"].long()[s["seq"].long(), pos // bs], pos % bs


def _read(s, page, row):
    """f32 [2, N, Hkv, D]: the values that the cache stands for."""
    c, flat = s["c"], s["pool"].view(-1)
    code, param = _offsets(c, page, row, c["hkv"])
    packed = flat[code]
    codes = torch.stack([packed & 15, packed >> 4], -1).flatten(-2)
    return _dequantised(codes, flat[param].view(torch.float16).unflatten(-1, (-1, 2)))


def _normed(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _rotated(x, pos, turns, interleaved):
    """x f32 [N, H, D]; the angle of pair i is pos * turns[i] / 2^64 turns, whose whole
    turns drop out of the 64-bit product."""
    a = (pos.long()[:, None] * turns[None, :]).double() * (2.0 * math.pi / 2.0 ** 64)
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    half = turns.shape[0]
    lo, hi = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
              else (slice(0, half), slice(half, 2 * half)))
    y = x.clone()
    y[..., lo] = x[..., lo] * cos - x[..., hi] * sin
    y[..., hi] = x[..., lo] * sin + x[..., hi] * cos
    return y


def _plain_plan(s):
    c, pages = s["c"], s["pages"]
    state, B, mb, bs = s["state"].clone(), c["b"], c["mb"], c["bs"]
    table, free, count = state[: B * mb], state[B * mb: -1], state[-1:]
    old, new = s["old"].long(), s["new"].long()
    po, pn = (old + bs - 1) // bs, (new + bs - 1) // bs
    j = torch.arange(mb, device=DEV)[None]
    taken = ((j >= po[:, None]) & (j < pn[:, None])).view(-1)
    given = ((j >= pn[:, None]) & (j < po[:, None])).view(-1)
    nt, ng = torch.cumsum(taken, 0), torch.cumsum(given, 0)
    left = count.long() + ng[-1:] - nt[-1:]  # pages free afterwards
    # the free pages, then those given back, requests in order; the last ones of these are taken
    stack = torch.cat([free, torch.zeros(B * mb + 1, dtype=torch.int32, device=DEV)])
    stack[torch.where(given, count.long() + ng - 1, pages + B * mb)] = table
    got = stack[torch.where(taken, left + nt - 1, 0)]
    table.copy_(torch.where(taken, got, torch.where(given, -1, table)))
    free.copy_(torch.where(torch.arange(pages, device=DEV) < left, stack[:pages], free))
    count.copy_(left)
    cu = torch.cumsum(torch.clamp(new - old, min=0), 0)
    n = torch.arange(s["tokens"], device=DEV)
    seq = torch.searchsorted(cu, n, right=True)
    pad = seq == B
    seq = seq.clamp(max=B - 1)
    pos = new[seq] - (cu[seq] - n)
    page = table.view(B, mb)[seq, (pos // bs).clamp(0, mb - 1)].long()
    return {"table": table.view(B, mb), "free": free, "count": count,
            "positions": torch.where(pad, 0, pos).int(), "seq": torch.where(pad, -1, seq).int(),
            "slots": torch.where(pad, -1, page * bs + pos % bs),
            "cu": torch.cat([torch.zeros_like(cu[:1]), cu]).int()}


def _plain_append(s):
    c = s["c"]
    out, k = {}, s["k"].float()
    if c["rd"]:
        k = _rotated(_normed(k, s["kw"]), s["pos"], s["turns"], c["interleaved"])
        if c["hq"]:
            out["q"] = _rotated(_normed(s["q"].float(), s["qw"]), s["pos"], s["turns"],
                                c["interleaved"])
    codes, params = _quantised(torch.stack([k, s["v"].float()]), c["group"])
    page, row = _rows(s)
    code_at, param_at = _offsets(c, page, row, c["hkv"])
    flat = s["pool"].view(-1)
    flat[code_at] = codes[..., 0::2] | codes[..., 1::2] << 4
    flat[param_at] = params.view(torch.uint8).flatten(-2)
    kv = _read(s, page, row).half()
    return {**out, "k": kv[0], "v": kv[1]}


def _plain_gather(s):
    kv = _read(s, *_rows(s)).half()
    return {"k": kv[0], "v": kv[1]}


def _softmaxed(x, ok, c):
    """exp(x - max), max and sum over the last axis of scores x where ok."""
    x = x * float(np.float32(1.0 / math.sqrt(c["d"])))
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    x = x.masked_fill(~ok, -math.inf)
    m = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    return w, m[..., 0], w.sum(-1)


def _plain_attend(s):
    c = s["c"]
    B, T, H, D, bs = c["b"], c["t"], c["hkv"], c["d"], c["bs"]
    G, L = c["hq"] // H, s["lens"].long()
    codes, params = _unpaged(s["pool"], c)
    k, v = _dequantised(codes, params)  # [pages, Hkv, bs, D]
    mb = s["table"].shape[1]
    page = s["table"].long().clamp(min=0)
    keys = torch.arange(mb * bs, device=DEV)
    qp = (L - T)[:, None] + torch.arange(T, device=DEV)  # [B, T]
    lo = torch.where(qp >= c["window"], qp - c["window"] + 1, 0) if c["window"] else qp * 0
    ok = (keys >= lo[..., None]) & (keys <= qp[..., None])
    q = s["q"].view(B, T, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D)

    def padded(x):  # [B, Hkv, keys, D]
        return x[page].transpose(1, 2).reshape(B, H, mb * bs, D)

    x = torch.matmul(q, padded(k).transpose(2, 3)).view(B, H, T, G, mb * bs)
    w, m, total = _softmaxed(x, ok[:, None, :, None], c)
    del x
    o = torch.matmul(w.view(B, H, T * G, -1), padded(v)).view(B, H, T, G, D)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    lse = m + torch.log(total)
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(s["q"].shape),
            "lse": lse.permute(0, 2, 1, 3).reshape(s["q"].shape[:-1])}


# ------------------------------------------------------------------ the package's calls
def _own_plan(s):
    import quantized_kv_decode_paged_gb300 as qk
    c = s["c"]
    state, n = s["state"].clone(), c["b"] * c["mb"]
    table, free, count = state[:n].view(c["b"], c["mb"]), state[n: -1], state[-1:]
    pos, seq, slots, cu = qk.decode_attn_plan_blocks(s["old"], s["new"], table, free, count,
                                                     block_size=c["bs"], num_blocks=s["pages"],
                                                     max_tokens=s["tokens"])
    return {"table": table, "free": free, "count": count, "positions": pos, "seq": seq,
            "slots": slots, "cu": cu}


def _own_append(s):
    import quantized_kv_decode_paged_gb300 as qk
    c = s["c"]
    norm = c["rd"] > 0
    q = qk.decode_attn_append_paged_q4(s["k"], s["v"], s["pos"], s["table"], s["pool"], s["turns"],
                                       group=c["group"], token_seq=s["seq"], q=s["q"], norm=norm,
                                       q_weight=s["qw"] if norm else None,
                                       k_weight=s["kw"] if norm else None, eps=EPS,
                                       interleaved=c["interleaved"])
    k, v = qk.decode_attn_gather_paged_q4(s["pos"], s["table"], s["pool"], head_dim=c["d"],
                                          group=c["group"], token_seq=s["seq"])
    return {"k": k, "v": v, **({"q": q} if c["hq"] else {})}


def _own_gather(s):
    import quantized_kv_decode_paged_gb300 as qk
    c = s["c"]
    k, v = qk.decode_attn_gather_paged_q4(s["pos"], s["table"], s["pool"], head_dim=c["d"],
                                          group=c["group"], token_seq=s["seq"])
    return {"k": k, "v": v}


def _own_attend(s):
    import quantized_kv_decode_paged_gb300 as qk
    c = s["c"]
    out, lse = qk.decode_attn_paged_q4(s["q"], s["pool"], s["table"], s["lens"], group=c["group"],
                                       softcap=c["softcap"], sliding_window=c["window"],
                                       max_seq_len=s["max_len"])
    return {"out": out, "lse": lse}


def run(state):
    op = state["c"]["op"]
    if own:
        return {"plan": _own_plan, "append": _own_append, "gather": _own_gather,
                "attend": _own_attend}[op](state)
    return {"plan": _plain_plan, "append": _plain_append, "gather": _plain_gather,
            "attend": _plain_attend}[op](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "plan":
        old, new = _request_lens(c)
        moved = int(np.abs(-(-old // c["bs"]) + -new // c["bs"]).sum())
        tokens = int(np.maximum(new - old, 0).sum())
        return {"bytes": 12 * c["b"] + 8 * moved + 16 * tokens, "flops": 0}
    row = c["d"] // 2 + 4 * (c["d"] // c["group"])  # a cached row's bytes
    if c["op"] == "append":
        e = 4 if c["type"] == "f32" else 2
        rows = c["n"] * c["hkv"]
        # written to the cache, and read back from it
        return {"bytes": rows * 2 * (c["d"] * (e + 2) + 2 * row) + c["n"] * (c["hq"] * c["d"] * (e + 4) + 12),
                "flops": rows * 2 * c["d"] * 6}
    if c["op"] == "gather":
        return {"bytes": c["n"] * (c["hkv"] * 2 * (row + 2 * c["d"]) + 12),
                "flops": c["n"] * c["hkv"] * 4 * c["d"]}
    L, tok = _lens(c), np.arange(c["t"])
    qp = L[:, None] - c["t"] + tok
    lo = np.where(qp >= c["window"], qp - c["window"] + 1, 0) if c["window"] else qp * 0
    seen = int(np.maximum(0, np.minimum(qp + 1, L[:, None]) - lo).sum())
    keys = int(np.maximum(0, L - np.maximum(0, lo[:, 0])).sum())
    return {"bytes": keys * c["hkv"] * 2 * row + c["b"] * c["t"] * c["hq"] * (8 * c["d"] + 4),
            "flops": 4 * seen * c["hq"] * c["d"]}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_stored(x, group):
    """What the cache holds of x (numpy, float64), group by group along the last axis."""
    y = x.copy()
    for i in range(0, x.shape[-1], group):
        part = x[..., i: i + group]
        lo, hi = part.min(-1, keepdims=True), part.max(-1, keepdims=True)
        zero = lo.astype(np.float16).astype(np.float64)
        scale = ((hi - lo) / 15.0).astype(np.float16).astype(np.float64)
        safe = np.where(scale > 0, scale, 1.0)
        code = np.where(scale > 0, np.clip(np.rint((part - zero) / safe), 0, 15), 0)
        y[..., i: i + group] = code * scale + zero
    return y


def _exact_rotated(x, w, pos, c):
    y = x / np.sqrt(np.mean(np.square(x), axis=-1, keepdims=True) + EPS) * w
    z, p = y.copy(), pos.astype(np.float64)
    for i in range(c["rd"] // 2):
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + c["rd"] // 2)
        angle = p * 10000.0 ** (-2.0 * i / c["rd"])
        co, si = np.cos(angle)[:, None], np.sin(angle)[:, None]
        z[..., a] = y[..., a] * co - y[..., b] * si
        z[..., b] = y[..., a] * si + y[..., b] * co
    return z


def _exact_values(pages, c):
    """float64 [2, n, Hkv, bs, D] of pages uint8 [n, Hkv, bytes], row by row of a page."""
    n, h, bs, d = pages.shape[0], c["hkv"], c["bs"], c["d"]
    out = torch.empty((2, n, h, bs, d), dtype=torch.float64, device=pages.device)
    group = torch.arange(d, device=pages.device) // c["group"]
    ng = d // c["group"]
    for which in range(2):
        for t in range(bs):
            at = which * bs * d // 2 + t * d // 2
            par = pages[..., bs * d + (which * bs + t) * ng * 4:][..., : ng * 4].contiguous()
            par = par.view(torch.float16).double().view(n, h, ng, 2)
            byte = torch.arange(d, device=pages.device) // 2
            byte = (byte // 16 ^ (t // (256 // d)) % (d // 32)) * 16 + byte % 16
            code = pages[..., at + byte].double()
            odd = torch.arange(d, device=pages.device) % 2 == 1
            code = torch.where(odd, torch.floor(code / 16), torch.remainder(code, 16))
            out[which, :, :, t] = code * par[..., group, 0] + par[..., group, 1]
    return out


def _exact_plan(s):
    c, bs = s["c"], s["c"]["bs"]
    state, n = s["state"].cpu().numpy().copy(), c["b"] * c["mb"]
    table, free, count = state[:n].reshape(c["b"], c["mb"]), state[n: -1], int(state[-1])
    old, new = s["old"].tolist(), s["new"].tolist()
    stack, taken = list(free[:count]), sum(max(0, -(-q // bs) - -(-p // bs)) for p, q in zip(old, new))
    for b in range(c["b"]):
        for j in range(-(-new[b] // bs), -(-old[b] // bs)):
            stack.append(table[b, j])
            table[b, j] = -1
    left = len(stack) - taken
    got = iter(stack[left:])
    pos, seq, slots, cu = [], [], [], [0]
    for b in range(c["b"]):
        for j in range(-(-old[b] // bs), -(-new[b] // bs)):
            table[b, j] = next(got)
        for p in range(old[b], new[b]):
            pos.append(p)
            seq.append(b)
            slots.append(int(table[b, p // bs]) * bs + p % bs)
        cu.append(len(pos))
    free[:left] = stack[:left]
    pads = s["tokens"] - len(pos)
    return {"table": table, "free": free, "count": np.array([left], np.int32),
            "positions": np.array(pos + [0] * pads, np.int32),
            "seq": np.array(seq + [-1] * pads, np.int32),
            "slots": np.array(slots + [-1] * pads, np.int64), "cu": np.array(cu, np.int32)}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "plan":
        return _exact_plan(s)
    if c["op"] == "append":
        k, v = (s[n].double().cpu().numpy() for n in ("k", "v"))
        out, pos = {}, s["pos"].cpu().numpy()
        if c["rd"]:
            k = _exact_rotated(k, s["kw"].double().cpu().numpy(), pos, c)
            if c["hq"]:
                out["q"] = _exact_rotated(s["q"].double().cpu().numpy(),
                                          s["qw"].double().cpu().numpy(), pos, c)
        return {**out, "k": _exact_stored(k, c["group"]), "v": _exact_stored(v, c["group"])}
    if c["op"] == "gather":
        values = _exact_values(s["pool"], c)
        page, row = (x.tolist() for x in _rows(s))
        kv = torch.stack([values[:, p, :, t] for p, t in zip(page, row)], 1)
        return {"k": kv[0], "v": kv[1]}
    # each sequence alone, its pages in the order of its table, in 64-bit products
    T, H, D, G = c["t"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    q = s["q"].double().view(c["b"], T, c["hq"], D)
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device=DEV)
    for b, L in enumerate(s["lens"].tolist()):
        if L == 0:
            continue
        pages = s["pool"][s["table"][b, : -(-L // c["bs"])].long()]
        kv = _exact_values(pages, c).transpose(2, 3).flatten(1, 2)  # [2, keys, Hkv, D]
        for t in range(T):
            p = L - T + t
            first = p - c["window"] + 1 if c["window"] and p >= c["window"] else 0
            if p < first:
                continue
            k, v = kv[0, first: p + 1], kv[1, first: p + 1]
            x = torch.einsum("hgd,khd->hgk", q[b, t].view(H, G, D), k)
            x = x * float(np.float32(1.0 / math.sqrt(D)))
            if c["softcap"]:
                x = c["softcap"] * torch.tanh(x / c["softcap"])
            lse[b, t] = torch.logsumexp(x, -1).reshape(-1)
            out[b, t] = torch.einsum("hgk,khd->hgd", torch.softmax(x, -1), v).reshape(c["hq"], D)
    return {"out": out.view(s["q"].shape), "lse": lse.view(s["q"].shape[:-1])}
