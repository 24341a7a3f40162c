"""A paged cache held in 4 bits in numpy, and attention over it in 64 bits
(shared by tests; not collected)."""
import numpy as np


def quantised(x, group):
    """x f32 [..., D] -> codes uint8 [..., D], scale and zero f16 [..., D / group]; every
    step as the format defines it (f32, IEEE division, ties to even)."""
    x = np.asarray(x, np.float32)
    y = x.reshape(x.shape[:-1] + (-1, group))
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        lo = np.clip(y.min(-1), np.float32(-65504), np.float32(65504))
        hi = np.clip(y.max(-1), np.float32(-65504), np.float32(65504))
        zero, scale = lo.astype(np.float16), ((hi - lo) / np.float32(15)).astype(np.float16)
        s, z = scale.astype(np.float32)[..., None], zero.astype(np.float32)[..., None]
        code = np.clip(np.rint((y - z) / s), 0, 15)
    code = np.where(s > 0, code, 0)
    return np.nan_to_num(code).astype(np.uint8).reshape(x.shape), scale, zero


class Cache:
    """codes [2, NB, H, bs, D] (keys, values), scale and zero [2, NB, H, bs, D / group]."""

    def __init__(self, NB, H, bs, D, group):
        self.NB, self.H, self.bs, self.D, self.group = NB, H, bs, D, group
        shape = (2, NB, H, bs)
        self.codes = np.zeros(shape + (D,), np.uint8)
        self.scale = np.zeros(shape + (D // group,), np.float16)
        self.zero = np.zeros(shape + (D // group,), np.float16)

    def fill(self, rng, chunk=1 << 22):
        """Normal keys and values, page by page."""
        step = max(1, chunk // (self.H * self.bs * self.D))
        for i in range(0, self.NB, step):
            n = min(step, self.NB - i)
            x = rng.standard_normal((2, n, self.H, self.bs, self.D), np.float32)
            self.codes[:, i:i + n], self.scale[:, i:i + n], self.zero[:, i:i + n] = quantised(
                x, self.group)
        return self

    def places(self):
        """[bs, D / 32]: where piece c of row t lies."""
        t, c = np.arange(self.bs)[:, None], np.arange(self.D // 32)[None]
        return c ^ ((t // (256 // self.D)) % (self.D // 32))

    def bytes(self):
        """The pool: uint8 [NB, H, page bytes]."""
        packed = (self.codes[..., 0::2] | self.codes[..., 1::2] << 4)
        packed = packed.reshape(packed.shape[:-1] + (-1, 16))
        out = np.empty_like(packed)
        t = np.arange(self.bs)[:, None]
        out[..., t, self.places(), :] = packed
        par = np.stack([self.scale, self.zero], -1)
        parts = [out[0], out[1], par[0], par[1]]
        parts = [np.ascontiguousarray(p).view(np.uint8).reshape(self.NB, self.H, -1) for p in parts]
        return np.concatenate(parts, -1)

    @classmethod
    def of_bytes(cls, pool, bs, D, group):
        NB, H, n = pool.shape
        c = cls(NB, H, bs, D, group)
        code = pool[..., :bs * D].reshape(NB, H, 2, bs, -1, 16)
        t = np.arange(bs)[:, None]
        code = code[:, :, :, t, c.places()].reshape(NB, H, 2, bs, -1).transpose(2, 0, 1, 3, 4)
        c.codes[..., 0::2], c.codes[..., 1::2] = code & 15, code >> 4
        par = np.ascontiguousarray(pool[..., bs * D:]).view(np.float16)
        par = par.reshape(NB, H, 2, bs, -1, 2).transpose(2, 0, 1, 3, 4, 5)
        c.scale, c.zero = par[..., 0].copy(), par[..., 1].copy()
        return c

    def values(self, pages=slice(None)):
        """float64 [2, pages, H, bs, D]."""
        s, z = (np.repeat(x[:, pages].astype(np.float64), self.group, -1)
                for x in (self.scale, self.zero))
        with np.errstate(invalid="ignore"):
            return self.codes[:, pages] * s + z


def attend(q, cache, table, lens, q_pos=None, *, scale=0.0, softcap=0.0, sliding_window=0,
           causal=True):
    """(out, lse, flags) in 64 bits: q [B, Hq, D] or [B, T, Hq, D]; every sequence alone,
    its keys in the order of its table."""
    import quantized_kv_decode_paged_gb300 as qk
    shape = q.shape
    q = q.reshape(shape[0], -1, shape[-2], shape[-1]).astype(np.float64)
    B, T, Hq, D = q.shape
    H, bs, mb = cache.H, cache.bs, table.shape[1]
    sc = float(np.float32(scale if scale > 0 else 1 / np.sqrt(D)))
    out, lse = np.zeros(q.shape), np.full(q.shape[:-1], -np.inf)
    flags = 0
    for b in range(B):
        L = int(lens[b])
        if L < 0 or L > mb * bs:
            flags |= qk.DEV_BAD_SEQ_LEN
            L = min(max(L, 0), mb * bs)
        base = L - T
        if q_pos is not None:
            base = int(q_pos[b])
            if base < 0:
                flags |= qk.DEV_BAD_QPOS
                continue
        npg = -(-L // bs)
        row = table[b, :npg].astype(np.int64)
        good = (row >= 0) & (row < cache.NB)
        kv = cache.values(np.where(good, row, 0))  # [2, npg, H, bs, D]
        kv = kv.transpose(2, 0, 1, 3, 4).reshape(H, 2, npg * bs, D)
        seen_page = np.repeat(good, bs)
        for t in range(T):
            p = base + t
            first = p - sliding_window + 1 if sliding_window > 0 and p >= sliding_window else 0
            last = min(L, p + 1) if causal else L
            if last <= first:
                continue
            keys = np.arange(first, last)
            if (~good[first // bs:-(-last // bs)]).any():
                flags |= qk.DEV_BAD_BLOCK
            keys = keys[seen_page[keys]]
            if not len(keys):
                continue
            with np.errstate(invalid="ignore", over="ignore"):
                x = np.einsum("hgd,hkd->hgk", q[b, t].reshape(H, -1, D), kv[:, 0, keys]) * sc
                if softcap > 0:
                    x = softcap * np.tanh(x / softcap)
                m = x.max(-1, keepdims=True)
                w = np.exp(x - m)
                total = w.sum(-1, keepdims=True)
                o = np.einsum("hgk,hkd->hgd", w / total, kv[:, 1, keys])
                lse[b, t] = (m + np.log(total)).reshape(Hq)
            out[b, t] = o.reshape(Hq, D)
    return out.reshape(shape), lse.reshape(shape[:-1]), flags
