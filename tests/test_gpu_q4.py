"""The paged cache held in 4 bits on the GPU: append, gather and decode against
numpy forms in 64 bits."""
import numpy as np
import pytest

import quantized_kv_decode_paged_gb300 as qk
from q4_64 import Cache, attend, quantised
from rope64 import norm_rope

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    yield
    import torch
    torch.cuda.empty_cache()


def _t(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _np(t):
    return t.detach().float().cpu().numpy()


def _status():
    import torch
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _table(r, lens, bs, spare=2):
    need = -(-np.maximum(np.asarray(lens, np.int64), 0) // bs)
    perm = r.permutation(int(need.sum()) + spare).astype(np.int32)
    table = np.full((len(need), max(1, int(need.max()))), -1, np.int32)
    at = np.concatenate([[0], np.cumsum(need)])
    for b in range(len(need)):
        table[b, :need[b]] = perm[at[b]:at[b + 1]]
    return table, len(perm)


class Case:
    def __init__(self, seed, Hq, H, D, group, bs, lens, T=1, q_scale=1.0):
        r = np.random.default_rng(seed)
        self.r, self.T, self.D, self.group, self.bs = r, T, D, group, bs
        self.lens = np.asarray(lens, np.int32)
        self.table, NB = _table(r, self.lens, bs)
        self.cache = Cache(NB, H, bs, D, group).fill(r)
        B = len(self.lens)
        shape = (B, Hq, D) if T == 1 else (B, T, Hq, D)
        self.q = (r.standard_normal(shape) * q_scale).astype(np.float32)
        self.q_pos, self.kw = None, {}

    def args(self):
        return [_t(x) for x in (self.q, self.cache.bytes(), self.table, self.lens)]

    def run(self, **kw):
        import torch
        status = _status()
        kw = {"max_seq_len": int(max(0, self.lens.max())), **self.kw, **kw}
        out, lse = qk.decode_attn_paged_q4(*self.args(), None if self.q_pos is None else _t(self.q_pos),
                                           group=self.group, dev_status=status, **kw)
        torch.cuda.synchronize()
        return out.cpu().numpy(), lse.cpu().numpy(), int(status.item())

    def want(self):
        return attend(self.q, self.cache, self.table, self.lens, self.q_pos, **self.kw)

    def bounds(self):
        """(out, lse): how far f32 results may be off.

        A score is scale * (s sum q_d code_d + z sum q_d), group by group: q is held as two f16
        terms of its row scaled to a power of two (2^-22 of the value), the products
        with the codes are exact, their sums take D / 16 truncating adds a term, 2^-23 of
        the partial sum each, and a few f32 operations follow: eps = scale * sum |q_d| * (15 s
        + |z|) * (D / 8 + 16) * 2^-23; the softcap adds 8 u of the cap.
        Weights: 2^x is good to 2^-22 and x = m - s to eps; two f16 terms hold a
        weight to 2^-22: 8 u.  Values: sums of weights times codes around 8 and of
        weights times z + 8 s, n / 16 adds each and a few more for joining states: (n / 8 + 48)
        * 2^-23 of 8 s + |z + 8 s|."""
        scale = self.kw.get("scale") or 1.0 / np.sqrt(self.D)
        c, n = self.cache, max(1, int(self.lens.max()))
        s, z = c.scale.astype(np.float64), c.zero.astype(np.float64)
        fin = np.isfinite(s) & np.isfinite(z)
        s, z = np.where(fin, s, 0), np.where(fin, z, 0)
        kmag, vmag = (15 * s + np.abs(z))[0].max(), (8 * s + np.abs(z + 8 * s))[1].max()
        mag = np.abs(self.q[np.isfinite(self.q).all(-1)].astype(np.float64)).sum(-1).max(initial=0)
        eps = scale * mag * kmag * (self.D / 8 + 16) * 2.0 ** -23
        eps += self.kw.get("softcap", 0.0) * 8 * U
        chain = (n / 8 + 48) * 2.0 ** -23
        return vmag * (2 * eps + 8 * U + chain), 2 * eps + chain

    def check(self, got=None, flags=0):
        out, lse, fl = got if got is not None else self.run()
        ro, rl, rf = self.want()
        assert fl == flags == rf, (fl, rf)
        bo, bl = self.bounds()
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(lse), empty)
        assert (out[empty] == 0).all()
        err = np.abs(out - ro)
        assert not (~(err <= bo)).any(), f"out off by {np.nanmax(err):.3e}, bound {bo:.3e}"
        lerr = np.abs(lse[~empty] - rl[~empty])
        assert not (~(lerr <= bl + 2.0 ** -23 * np.abs(rl[~empty]))).any(), f"lse {lerr.max():.3e}"


FORMATS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


# ------------------------------------------------------------------ append and gather
def _rows(rng, shape, kind):
    x = rng.standard_normal(shape).astype(np.float32)
    if kind == "wide":
        x *= np.float32(5000.0)
    elif kind == "tiny":  # scales below f16's normal numbers
        x *= np.float32(3e-6)
    elif kind == "ties":  # scale 1, every half-integer a tie
        x = (rng.integers(0, 31, size=shape) / 2.0).astype(np.float32)
        x[..., ::32], x[..., 1::32] = 0, 15
    elif kind == "flat":
        x[:] = np.float32(0.3)
    elif kind == "past":  # values past f16's range and infinities
        x *= np.float32(4e4)
        x.reshape(-1)[::97] = np.inf
        x.reshape(-1)[5::97] = -np.inf
    return x


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("D,group", FORMATS)
@pytest.mark.parametrize("bs", [8, 64])
@pytest.mark.parametrize("kind", ["normal", "wide", "tiny", "ties", "flat", "past"])
def test_append_without_rotation_bit_for_bit(dtype, D, group, bs, kind):
    """A ragged call with padding and each kind of bad token: the pool's bytes are those of
    the definition, and nothing else is touched; the gather gives the values back."""
    import torch
    rng = np.random.default_rng(D + group + bs)
    B, H, npg = 5, 3, max(4, 40 // bs)
    perm = rng.permutation(B * npg + 2).astype(np.int32)
    table, NB = perm[:B * npg].reshape(B, npg).copy(), B * npg + 2
    seq = np.array([0] * 21 + [1, 2, 3, 3] + [-1, -7] + [4, 4, 4, 4, 1], np.int32)
    pos = np.array(list(range(5, 26)) + [0, npg * bs - 1, 7, 8] + [1, -3]
                   + [npg * bs, -1, 0, 2 ** 31 - 1, 3], np.int32)
    seq[-1] = B + 2
    table[4, 0] = NB
    N = len(seq)
    x = torch.from_numpy(_rows(rng, (N, 2 * H, D), kind)).cuda().to(getattr(torch, dtype))
    k, v = x[:, :H], x[:, H:]
    want = Cache(NB, H, bs, D, group).fill(rng)
    pool = _t(want.bytes())
    kept = np.zeros(N, bool)
    for n in range(N):
        s, p = seq[n], pos[n]
        if not (0 <= s < B and 0 <= p < npg * bs and 0 <= table[s, p // bs] < NB):
            continue
        kept[n] = True
        at = (table[s, p // bs], slice(None), p % bs)
        for i, rows in enumerate((_np(k), _np(v))):
            c, sc, z = quantised(rows[n], group)
            want.codes[i][at], want.scale[i][at], want.zero[i][at] = c, sc, z
    status = _status()
    args = (_t(pos), _t(table), pool)
    assert qk.decode_attn_append_paged_q4(k, v, *args, group=group, token_seq=_t(seq),
                                          dev_status=status) is None
    bad = qk.DEV_BAD_BLOCK | qk.DEV_BAD_SEQ_LEN | qk.DEV_BAD_SEQ
    assert int(status.item()) == bad
    assert np.array_equal(pool.cpu().numpy(), want.bytes())
    status.zero_()
    for dt in ("float32", "float16", "bfloat16"):
        gk, gv = qk.decode_attn_gather_paged_q4(*args, head_dim=D, group=group, token_seq=_t(seq),
                                                dtype=getattr(torch, dt), dev_status=status)
        assert int(status.item()) == bad
        for i, g in enumerate((gk, gv)):
            vals = want.values()[i]
            ref = np.zeros((N, H, D))
            for n in np.flatnonzero(kept):
                ref[n] = vals[table[seq[n], pos[n] // bs], :, pos[n] % bs]
            # one f32 rounding, then one to the type (f16's smallest step is 2^-24)
            step = {"float32": 0, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}[dt]
            tol = np.abs(ref) * (step + U) * (1 + 2.0 ** -7) + (2.0 ** -25 if dt == "float16" else 0)
            sat = np.clip(ref, -65504, 65504) if dt == "float16" else ref
            assert (np.abs(_np(g) - sat) <= tol).all()
            assert (_np(g)[~kept] == 0).all()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("D,rd,group,il", [(64, 64, 32, False), (64, 16, 64, True),
                                           (128, 128, 32, True), (128, 48, 128, False),
                                           (256, 256, 64, False), (256, 96, 128, True)])
def test_append_with_norm_and_rotation(dtype, D, rd, group, il):
    """Stored keys stand within half a step of the 64-bit rows; queries as by the f16
    append, bit for bit; padding tokens' queries are left as they were."""
    import torch
    rng = np.random.default_rng(D + rd)
    N, H, Hq, bs = 37, 2, 6, 16
    x = torch.from_numpy(rng.standard_normal((N, Hq + 2 * H, D)).astype(np.float32)).cuda()
    x = x.to(getattr(torch, dtype))
    q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    pos = rng.integers(0, 64, N).astype(np.int32)
    table = rng.permutation(N * 4).astype(np.int32).reshape(N, 4)
    seq = np.arange(N, dtype=np.int32)
    seq[5] = -1
    inv = 10000.0 ** (-2.0 * np.arange(rd // 2) / rd)
    f = qk.decode_attn_rope_freqs(rd, inv_freq=inv)
    qw, kw = ((1 + 0.1 * rng.standard_normal(D)).astype(np.float32) for _ in range(2))
    pool = torch.zeros((N * 4, H, qk.decode_attn_q4_page_bytes(bs, D, group)), dtype=torch.uint8,
                       device="cuda")
    opts = dict(token_seq=_t(seq), q=q, norm=True, q_weight=_t(qw), k_weight=_t(kw),
                weight_offset=0.5, interleaved=il)
    out = torch.full((N, Hq, D), 7.0, device="cuda")
    status = _status()
    got = qk.decode_attn_append_paged_q4(k, v, _t(pos), _t(table), pool, f, group=group, q_out=out,
                                         dev_status=status, **opts)
    assert got is out and int(status.item()) == 0
    pools = [torch.zeros((N * 4, bs, H, D), dtype=torch.float16, device="cuda") for _ in range(2)]
    other = torch.full((N, Hq, D), 7.0, device="cuda")
    qk.decode_attn_append_paged_rope(k, v, _t(pos), _t(table), *pools, f, q_out=other, **opts)
    assert torch.equal(out, other) and bool((out[5] == 7).all())
    c = Cache.of_bytes(pool.cpu().numpy(), bs, D, group)
    vals = c.values()
    y, b = norm_rope(_np(k), pos, f.cpu().numpy(), norm=True, weight=kw, offset=0.5,
                     interleaved=il)
    for i, (rows, off) in enumerate(((y, b), (_np(v).astype(np.float64), np.zeros_like(y)))):
        for n in range(N):
            at = (table[n, pos[n] // bs], slice(None), pos[n] % bs)
            s = np.repeat(c.scale[i][at].astype(np.float64), group, -1)
            z = np.repeat(c.zero[i][at].astype(np.float64), group, -1)
            if n == 5:
                assert (s == 0).all() and (c.codes[i][at] == 0).all()
                continue
            # half a step; the last code stands up to 15 of the scale's rounding (2^-11) and the
            # zero's below the largest value, the first one the zero's rounding above the least
            tol = s * (0.5 + 15 * 2.0 ** -11) + np.abs(z) * 2.0 ** -11 + 2 * off[n] + 2.0 ** -24
            assert (np.abs(vals[i][at] - rows[n]) <= tol).all()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("D,rd,group", [(64, 64, 32), (64, 16, 64), (128, 128, 32), (128, 128, 128),
                                        (128, 96, 64), (256, 256, 128), (256, 96, 32), (256, 16, 64)])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("norm,kind", [(True, "normal"), (False, "wide"), (False, "past"), (True, "nan")])
def test_append_of_rotated_keys_bit_for_bit(dtype, D, rd, group, il, norm, kind):
    """The f32 rows that the norm and rotation give, quantised as the format defines it, whichever
    threads hold a group's values; a NaN's group and no other."""
    import torch
    rng = np.random.default_rng(D + rd + group)
    N, H, bs = 333, 2, 16
    rows = _rows(rng, (N, 2 * H, D), kind)
    if kind == "nan":
        rows[::7, :, D // 3] = np.nan
    x = torch.from_numpy(rows).cuda().to(getattr(torch, dtype))
    k, v = x[:, :H], x[:, H:]
    pos = rng.integers(0, 64, N).astype(np.int32)
    table = rng.permutation(N * 4).astype(np.int32).reshape(N, 4)
    f = qk.decode_attn_rope_freqs(rd)
    w = _t((1 + 0.1 * rng.standard_normal(D)).astype(np.float32)) if norm else None
    pool = torch.zeros((N * 4, H, qk.decode_attn_q4_page_bytes(bs, D, group)), dtype=torch.uint8,
                       device="cuda")
    qk.decode_attn_append_paged_q4(k, v, _t(pos), _t(table), pool, f, group=group, norm=norm,
                                   k_weight=w, interleaved=il)
    y, _ = qk.decode_attn_qk_norm_rope(k, None, _t(pos), f, norm=norm, q_weight=w, interleaved=il)
    c = Cache.of_bytes(pool.cpu().numpy(), bs, D, group)
    at = (table[np.arange(N), pos // bs], slice(None), pos % bs)
    for i, ref in enumerate((y, v)):
        codes, scale, zero = quantised(_np(ref), group)
        assert np.array_equal(c.scale[i][at], scale, equal_nan=True)
        assert np.array_equal(c.zero[i][at], zero, equal_nan=True)
        assert np.array_equal(c.codes[i][at], codes)
    assert kind == "past" or np.isnan(c.scale).any() == (kind == "nan")


def test_append_keeps_nan_where_it_is():
    """A NaN makes its own group NaN, keys and values, and no other."""
    import torch
    D, group, H, bs = 128, 32, 2, 16
    x = torch.randn((3, 2 * H, D), device="cuda")
    x[1, 0, 40] = float("nan")
    x[2, 3, 127] = float("nan")
    pool = torch.zeros((3, H, qk.decode_attn_q4_page_bytes(bs, D, group)), dtype=torch.uint8,
                       device="cuda")
    args = (torch.tensor([3, 4, 5], dtype=torch.int32, device="cuda"),
            torch.arange(3, dtype=torch.int32, device="cuda")[:, None], pool)
    qk.decode_attn_append_paged_q4(x[:, :H], x[:, H:], *args, group=group)
    for dt in (torch.float16, torch.bfloat16, torch.float32):
        k, v = qk.decode_attn_gather_paged_q4(*args, head_dim=D, group=group, dtype=dt)
        nan = torch.zeros((2, 3, H, D), dtype=torch.bool, device="cuda")
        nan[0, 1, 0, 32:64] = nan[1, 2, 1, 96:] = True
        assert torch.equal(torch.stack([k, v]).isnan(), nan)


@pytest.mark.parametrize("N", [1, 2, 1000, 5001])
def test_append_and_gather_of_many_tokens(N):
    """One prompt, longer and longer; a call of the whole and calls of its parts agree."""
    import torch
    rng = np.random.default_rng(N)
    D, group, H, bs = 128, 64, 4, 32
    x = torch.from_numpy(rng.standard_normal((N, 2 * H, D)).astype(np.float32)).cuda().half()
    npg = -(-N // bs)
    table = _t(rng.permutation(npg).astype(np.int32)[None])
    pos, seq = torch.arange(N, dtype=torch.int32, device="cuda"), torch.zeros(
        N, dtype=torch.int32, device="cuda")
    shape = (npg, H, qk.decode_attn_q4_page_bytes(bs, D, group))
    pools = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for pool, step in zip(pools, (N, max(1, N // 3))):
        for i in range(0, N, step):
            e = slice(i, i + step)
            qk.decode_attn_append_paged_q4(x[e, :H], x[e, H:], pos[e], table, pool, group=group,
                                           token_seq=seq[e])
    assert torch.equal(*pools)
    k, v = qk.decode_attn_gather_paged_q4(pos, table, pools[0], head_dim=D, group=group,
                                          token_seq=seq, dtype=torch.float32)
    for got, rows in ((k, x[:, :H]), (v, x[:, H:])):
        c, s, z = quantised(_np(rows), group)
        ref = c * np.repeat(s.astype(np.float64), group, -1) + np.repeat(z.astype(np.float64), group, -1)
        assert (np.abs(_np(got) - ref) <= U * np.abs(ref)).all()


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("D,group", FORMATS)
@pytest.mark.parametrize("Hq,H", [(1, 1), (8, 2), (7, 1), (6, 6), (40, 4), (32, 2)])
@pytest.mark.parametrize("bs", [8, 16, 64, 256])
def test_head_layouts_formats_and_page_sizes(D, group, Hq, H, bs):
    Case(1, Hq, H, D, group, bs, [300, 1, 77, 0]).check()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_lengths_around_pages_and_tiles(D):
    lens = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513]
    Case(2, 4, 2, D, 32, 16, lens).check()
    Case(2, 4, 2, D, 64, 8, lens[::-1]).check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,Hq,H", [(2, 8, 2), (3, 5, 1), (4, 16, 2), (9, 4, 2), (17, 2, 2), (64, 3, 1)])
def test_query_tokens(D, T, Hq, H):
    """Some sequences are shorter than the query tokens: rows before their first key are empty."""
    Case(3, Hq, H, D, 64, 16, [200, T, 1, 0, T + 1, 333], T=T).check()


@pytest.mark.parametrize("B", [1, 5, 160, 1500])
def test_batches(B):
    r = np.random.default_rng(B)
    Case(4, 2, 1, 64, 32, 16, r.integers(0, 70, B)).check()


@pytest.mark.parametrize("D,L", [(64, 40000), (128, 33000), (256, 20011)])
def test_long_axes(D, L):
    Case(5, 8, 1, D, 64, 16, [L, 100]).check()
    Case(5, 2, 2, D, 32, 256, [L // 2, 3, L // 3]).check()


@pytest.mark.parametrize("D,group,T,B", [(64, 64, 1, 300), (128, 32, 1, 300), (128, 128, 4, 300),
                                         (256, 128, 1, 300), (256, 32, 3, 150), (256, 64, 17, 60)])
def test_many_tiles_a_processor(D, group, T, B):
    """Shares of many tiles and of several units: every buffer is used again and again, by
    whoever comes first.  The sequences' tables name a few pages over and over."""
    c = Case(15, 4, 2, D, group, 32, [2048], T=T)
    r = c.r
    c.lens = r.integers(1500, 2049, B).astype(np.int32)
    c.table = r.integers(0, c.cache.NB, (B, 64)).astype(np.int32)
    c.q = r.standard_normal((B,) + c.q.shape[1:]).astype(np.float32)
    got = c.run()
    c.check(got)
    again = c.run()
    assert np.array_equal(got[0], again[0]) and np.array_equal(got[1], again[1])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 15, 100, 4000])
@pytest.mark.parametrize("T", [1, 3])
def test_sliding_windows(D, window, T):
    c = Case(6, 8, 2, D, 64, 16, [5000, 30, 101, 900], T=T)
    c.kw = dict(sliding_window=window)
    c.check()


@pytest.mark.parametrize("D,group", FORMATS)
@pytest.mark.parametrize("T,Hq,H", [(1, 36, 4), (2, 32, 4), (5, 20, 4), (9, 32, 4), (16, 40, 4)])
@pytest.mark.parametrize("window,causal", [(0, True), (70, True), (200, False)])
def test_many_rows_of_many_heads(D, group, T, Hq, H, window, causal):
    """9 to 160 rows a kv head in a batch large enough for warps of 16 rows, tables with room
    for 1024 keys and more; lengths from none on."""
    c = Case(18, Hq, H, D, group, 16, [0, 1, T, 15, 16, 17, 63, 64, 65, 300, 1024, 700, 33], T=T)
    pick = np.arange(44) % 13
    pick[13:] = pick[13:][::-1]
    c.lens, c.table, c.q = c.lens[pick], c.table[pick], c.q[pick]
    c.q = c.q + np.float32(0.01) * np.arange(44, dtype=np.float32).reshape((44,) + (1,) * (c.q.ndim - 1))
    c.kw = dict(sliding_window=window, causal=causal)
    c.check()
    c.cache.scale[1, c.table[10, 3], 1, 5, -1] = np.nan  # in one value group of one key
    out, lse, _ = c.run()
    ro, _, _ = c.want()
    assert np.array_equal(np.isnan(out), np.isnan(ro)) and np.isfinite(lse[10]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,Hq,H", [(2, 2, 1), (4, 2, 2), (17, 4, 2), (40, 1, 1)])
@pytest.mark.parametrize("window", [1, 5, 40])
def test_query_tokens_behind_windows(D, T, Hq, H, window):
    """Rows of a unit that see different keys, some none of a tile that others see."""
    c = Case(17, Hq, H, D, 32, 8, [300, 3, 41, 0, T], T=T)
    c.kw = dict(sliding_window=window)
    c.check()
    c.q_pos = np.array([350, 0, 20, 5, 10 ** 6], np.int32)
    for causal in (True, False):
        c.kw = dict(sliding_window=window, causal=causal)
        c.check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("softcap,scale,q_scale", [(50.0, 0.0, 1.0), (2.0, 0.0, 4.0), (30.0, 1.0, 3.0),
                                                   (0.0, 0.3, 1.0), (1e-3, 0.0, 1.0)])
def test_softcap_and_scale(D, softcap, scale, q_scale):
    c = Case(7, 8, 2, D, 32, 16, [500, 33], q_scale=q_scale)
    c.kw = dict(softcap=softcap, scale=scale)
    c.check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("T", [1, 4])
def test_query_positions(causal, T):
    c = Case(8, 8, 2, 128, 64, 16, [300, 200, 100, 50, 0], T=T)
    c.q_pos = np.array([10, 500, 99, -1, 3], np.int32)
    c.kw = dict(causal=causal)
    c.check(flags=qk.DEV_BAD_QPOS)
    c.kw = dict(causal=causal, sliding_window=40)
    c.check(flags=qk.DEV_BAD_QPOS)


@pytest.mark.parametrize("T", [1, 4])
def test_query_positions_up_to_the_last(T):
    """Positions and windows whose sums pass 2^31: a window's first key is key 0, inside the
    sequence, or past every key."""
    far = 2 ** 31 - 1
    c = Case(16, 8, 2, 64, 32, 16, [300, 200, 300, 77, 300], T=T)
    c.q_pos = np.array([far, far - 1, far - 2, far - 150, 299], np.int32)
    for window in (0, 1, 2, far - 150, far - 3, far):
        c.kw = dict(sliding_window=window)
        c.check()


def test_bad_pages_and_lengths_are_masked_and_flagged():
    c = Case(9, 8, 2, 128, 64, 16, [300, 200, 100, 50])
    c.table[0, 3], c.table[1, 0], c.table[2, 6] = -1, c.cache.NB, 2 ** 31 - 1
    c.check(flags=qk.DEV_BAD_BLOCK)
    c.table[3, :4] = -5
    c.check(flags=qk.DEV_BAD_BLOCK)  # a sequence without a single page
    d = Case(9, 8, 2, 128, 64, 16, [304, 200, 100, 50])
    d.table[:] = d.r.permutation(d.table.size).reshape(d.table.shape) % d.cache.NB
    d.lens = np.array([-4, 305, 2 ** 31 - 1, 304], np.int32)
    d.kw = dict(sliding_window=200)
    d.check(d.run(max_seq_len=0), flags=qk.DEV_BAD_SEQ_LEN)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bs", [8, 16, 64, 256])
@pytest.mark.parametrize("B,T,Hq,H", [(4, 1, 8, 2), (4, 1, 16, 2), (40, 4, 16, 4)])
@pytest.mark.parametrize("window", [0, 333])
def test_bad_pages_of_every_place_in_a_tile(D, bs, B, T, Hq, H, window):
    """Units of 4, 8 and 16 rows, tiles of many pages and pages of many tiles: pages outside the
    pool first, last and inside of a tile, side by side, before the window and as the last
    one of a sequence."""
    c = Case(26, Hq, H, D, 32, bs, [1100, 700, 1024, 801], T=T)
    pick = np.arange(B) % 4
    c.lens, c.table = c.lens[pick], c.table[pick]
    c.q = c.r.standard_normal((B,) + c.q.shape[1:]).astype(np.float32)
    for b in range(B):
        n = -(-int(c.lens[b]) // bs)
        some = [(b // 4 + k) % n for k in (0, 5, 6, n - 1)] + c.r.integers(0, n, 1 + n // 9).tolist()
        c.table[b, some[b % 2:]] = c.r.choice([-1, c.cache.NB, 2 ** 31 - 1, -2 ** 31])
    c.kw = dict(sliding_window=window)
    c.check(flags=qk.DEV_BAD_BLOCK)
    c.table[:B // 2] = -1  # sequences without a single page
    c.check(flags=qk.DEV_BAD_BLOCK)


@pytest.mark.parametrize("D,group", FORMATS)
@pytest.mark.parametrize("poison", [np.nan, np.inf, -np.inf])
def test_nonfinite_scales_in_masked_places(D, group, poison):
    """Rows behind a sequence's last key, before its window and in other pages."""
    c = Case(10, 8, 2, D, group, 16, [300, 5, 0, 250])
    c.kw = dict(sliding_window=100)
    live = np.zeros((c.cache.NB, 16), bool)
    for b, L in enumerate(c.lens):
        for t in range(max(0, L - 100), L):
            live[c.table[b, t // 16], t % 16] = True
    dead = np.broadcast_to(~live[None, :, None, :, None], c.cache.scale.shape)
    c.cache.scale[dead] = poison
    c.cache.zero[dead] = poison
    out, lse, flags = c.run()
    assert np.isfinite(out).all()
    c.check((out, lse, flags))


@pytest.mark.parametrize("D,group", FORMATS)
def test_nan_that_is_seen(D, group):
    """A NaN value group makes its own columns NaN, a NaN key its heads' rows."""
    c = Case(11, 4, 2, D, group, 16, [300, 40])
    page, row = c.table[0, 7], 3
    c.cache.scale[1, page, 1, row, -1] = np.nan
    out, lse, _ = c.run()
    ro, rl, _ = c.want()
    assert np.array_equal(np.isnan(out), np.isnan(ro)) and np.isnan(ro).any()
    assert np.isfinite(lse).all()
    c.cache.zero[0, page, 0, row, 0] = np.nan
    out, lse, _ = c.run()
    ro, rl, _ = c.want()
    assert np.array_equal(np.isnan(out), np.isnan(ro))
    assert np.array_equal(np.isnan(lse), np.isnan(rl))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_query_values_of_any_size(D):
    """Rows from 2^-140 to 2^100 in one call, against keys that bring the scores back to order 1
    or to 0; a row with an infinity or a NaN is NaN, alone."""
    c = Case(12, 8, 1, D, 64, 16, [100])
    for j, e in enumerate([-140, -60, -20, 0]):
        c.q[0, j] = c.q[0, j].astype(np.float64) * 2.0 ** e
    c.check()
    c.q[0, 4] = c.r.standard_normal(D).astype(np.float32) * 2.0 ** 5
    c.q[0, 5, 7] = np.inf
    c.q[0, 6, 0] = np.nan
    out, lse, _ = c.run()
    assert np.isnan(out[0, 5:7]).all() and np.isnan(lse[0, 5:7]).all()
    ro, rl, _ = c.want()
    keep = np.array([0, 1, 2, 3, 4, 7])
    bo, bl = c.bounds()
    assert (np.abs(out - ro)[0, keep] <= bo).all() and (np.abs(lse - rl)[0, keep] <= bl + 1e-6).all()
    # large queries over small keys
    d = Case(12, 4, 1, D, 64, 16, [100])
    d.cache.scale[0] = (d.cache.scale[0].astype(np.float64) * 2.0 ** -8).astype(np.float16)
    d.cache.zero[0] = (d.cache.zero[0].astype(np.float64) * 2.0 ** -8).astype(np.float16)
    d.q *= np.float32(2.0 ** 100)
    d.kw = dict(scale=2.0 ** -92)
    d.check()


@pytest.mark.parametrize("D,group", FORMATS)
@pytest.mark.parametrize("B,T,Hq,H", [(3, 1, 4, 2), (3, 1, 16, 2), (48, 3, 16, 4)])
@pytest.mark.parametrize("window", [0, 300])
def test_scores_below_f32(D, group, B, T, Hq, H, window):
    """Keys whose scores are below f32's range have no weight, also those that come first: their
    rows are all -1000, the other keys 0, every q_d 10^36.  The others' scores are 0, exactly, and
    count alike: the bounds are those of q = 0."""
    c = Case(24, Hq, H, D, group, 16, [1, 40, 200, 1040, 5000], T=T)
    pick = np.arange(B) % 3 + 2
    c.lens, c.table, c.q = c.lens[pick], c.table[pick], np.zeros((B,) + c.q.shape[1:], np.float32)
    c.cache.codes[0], c.cache.scale[0], c.cache.zero[0] = 0, 0, -1000
    for b in range(B):
        for t in range(c.lens[b] - 90, c.lens[b] - T + 1):  # every query token sees some
            c.cache.zero[0, c.table[b, t // 16], :, t % 16] = 0
    c.kw = dict(sliding_window=window)
    bo, bl = c.bounds()
    c.q[:] = 1e36
    out, lse, flags = c.run()
    ro, rl, _ = c.want()
    assert flags == 0 and (np.abs(out - ro) <= bo).all()
    assert (np.abs(lse - rl) <= bl + 2.0 ** -23 * np.abs(rl)).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_softcap_below_normal_numbers(D):
    """cap * tanh(s / cap) of the least caps is 0 to any accuracy, also for s = 0."""
    c = Case(25, 8, 2, D, 32, 16, [300, 33])
    c.q[:, :2] = 0
    for cap in (1e-37, 1e-39, 1e-40, 1e-45):
        c.kw = dict(softcap=cap)
        c.check()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_softcap_past_every_score(D):
    """A cap near f32's largest number changes nothing.  s / cap is off by half of f32's least step,
    2^-150, which comes back times a cap below 2^128: 2^-22 of a score in units of log 2."""
    c = Case(27, 8, 2, D, 32, 16, [300, 33])
    bo, bl = c.bounds()
    vmag = (8 * c.cache.scale[1] + np.abs(c.cache.zero[1] + 8 * c.cache.scale[1])).max()
    for cap in (1e37, 2e38, 3.4e38):
        out, lse, _ = c.run(softcap=cap)
        ro, rl, _ = c.want()
        assert (np.abs(out - ro) <= bo + 2 * 2.0 ** -22 * vmag).all()
        assert (np.abs(lse - rl) <= bl + 2.0 ** -22 + 2.0 ** -23 * np.abs(rl)).all()


@pytest.mark.parametrize("D,group", [(64, 64), (128, 32), (128, 128), (256, 128)])
@pytest.mark.parametrize("s", [2.0 ** -20, 2.0 ** -10, 1.0, 4096.0])
def test_value_scales_of_any_size(D, group, s):
    """The values' scales go into the weights: nothing over- or underflows on the way."""
    c = Case(13, 8, 2, D, group, 16, [300, 900])
    c.cache.scale[1] = (c.cache.scale[1].astype(np.float64) * s).astype(np.float16)
    c.cache.zero[1] = (c.cache.zero[1].astype(np.float64) * s).astype(np.float16)
    c.check()


@pytest.mark.parametrize("D,group", FORMATS)
def test_value_scales_far_apart(D, group):
    """Groups, keys and heads whose scales differ by powers of two up to 2^16, a key with
    weight near 1 and tiny values beside keys of small weight and large ones."""
    c = Case(14, 8, 2, D, group, 16, [200, 64])
    e = c.r.integers(-10, 7, c.cache.scale[1].shape)
    c.cache.scale[1] = (c.cache.scale[1].astype(np.float64) * 2.0 ** e).astype(np.float16)
    c.cache.zero[1] = (c.cache.zero[1].astype(np.float64) * 2.0 ** e).astype(np.float16)
    c.q *= 3
    c.check()


ROWS = [(2, 2), (40, 4)]


@pytest.mark.parametrize("B,Hq", ROWS)
@pytest.mark.parametrize("D,group", FORMATS)
def test_low_terms_of_queries(D, group, B, Hq):
    """Scores that live in the low bits of q: every key has as many codes 11 as 5 in every pair
    of neighbours, around a zero of -8, and q_d = 1 + s_d 2^-12: a score is scale *
    2^-12 sum s_d k_d with k_d = +-3.  f16 alone sees no difference between keys."""
    r = np.random.default_rng(75)
    c = Case(75, Hq, 1, D, group, 16, 60 + r.integers(1, 14, B))
    k = np.where(r.random(c.cache.codes[0].shape) < 0.5, 11, 5)
    k[..., 1::2] = 16 - k[..., ::2]
    c.cache.codes[0], c.cache.scale[0], c.cache.zero[0] = k, 1, -8
    c.q = (1 + np.where(r.random(c.q.shape) < 0.5, 1, -1) * 2.0 ** -12).astype(np.float32)
    c.kw = dict(scale=8.0)
    out, _, _ = c.run()
    ro = c.want()[0]
    vals = c.cache.values()[1]
    flat = np.stack([vals[c.table[b]].transpose(1, 0, 2, 3).reshape(-1, D)[:c.lens[b]].mean(0)
                     for b in range(B)])[:, None]
    # without the low terms every score is 0: a quarter of what they bring to the least moved row
    assert np.abs(out - ro).max() <= np.abs(ro - flat).max((1, 2)).min() / 4


@pytest.mark.parametrize("D,group", FORMATS)
@pytest.mark.parametrize("T,L", [(1, 1000), (1, 20000), (4, 3001)])
def test_errors_are_those_of_f32(D, group, T, L):
    """The root mean square of the error against that of the result, for normal inputs.

    A score of order 1 is the difference of sums of order sqrt(D) * 8.7 / 4.6, whose D / 16 truncating
    adds leave half of 2^-23 of their size each: up to 16 * 6e-8 * 2 = 1.9e-6 for D =
    256.  Values: joined from sums of a few adds of 2^-23 each, 1e-6 at most.  Counted as 2^-18
    = 3.8e-6.  One f16 term of q or of the weights leaves 2^-12 or more."""
    c = Case(77, 16, 2, D, group, 16, [L, L // 2, L // 3 + 1], T=T)
    out, lse, _ = c.run()
    ro, rl, _ = c.want()
    rms = lambda x: np.sqrt(np.mean(np.square(x.astype(np.float64))))  # noqa: E731
    assert rms(out - ro) <= 2.0 ** -18 * rms(ro)
    assert rms(lse - rl) <= 2.0 ** -18 * max(1.0, rms(rl))


def test_workspaces_and_repeats():
    """Bit for bit the same twice, with a workspace of any content; too small ones are
    refused; rows behind the last sequence are left alone."""
    import torch
    c = Case(20, 8, 2, 128, 64, 16, [9000, 40, 0, 3000, 700])
    args = c.args()
    a = qk.decode_attn_paged_q4(*args, group=64)
    p = qk.DaParams(5, 8, 2, 128, 16, c.table.shape[1], c.cache.NB, 0, 0.0, 0.0, 0, 1)
    n = qk.decode_attn_paged_q4_workspace_size(p, 1)
    assert n > 0
    for fill in (0, 255, 127):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        out = torch.full((7, 8, 128), 7.0, device="cuda")
        lse = torch.full((7, 8), 7.0, device="cuda")
        qk.decode_attn_paged_q4(*args, group=64, workspace=ws, out=out[:5], lse=lse[:5])
        assert torch.equal(out[:5], a[0]) and torch.equal(lse[:5], a[1])
        assert bool((out[5:] == 7).all()) and bool((lse[5:] == 7).all())
    c.check((a[0].cpu().numpy(), a[1].cpu().numpy(), 0))
    with pytest.raises(qk.DecodeAttnError) as e:
        qk.decode_attn_paged_q4(*args, group=64, workspace=ws[:n - 1])
    assert e.value.status == qk.DA_ERR_WORKSPACE
    with pytest.raises(qk.DecodeAttnError) as e:
        qk.decode_attn_paged_q4(*args, group=64, out=args[0])
    assert e.value.status == qk.DA_ERR_INVALID


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_workspace_serves_smaller_calls(D):
    """Its size never falls as batch, query tokens or room grow; a call of few rows in the
    workspace of a large one."""
    import torch
    size = lambda B, T, mb: qk.decode_attn_paged_q4_workspace_size(  # noqa: E731
        qk.DaParams(B, 16, 4, D, 16, mb, 64, 0, 0.0, 0.0, 0, 1), T)
    axes = ((1, 30, 40, 2000), (1, 2, 3, 5, 40), (1, 63, 64, 4000))
    for mb in axes[2]:
        for T in axes[1]:
            for B in axes[0]:
                n = size(B, T, mb)
                assert n > 0 and all(size(B2, T2, mb2) <= n for B2 in axes[0] if B2 <= B
                                     for T2 in axes[1] if T2 <= T for mb2 in axes[2] if mb2 <= mb)
    ws = torch.empty(size(2000, 40, 4000), dtype=torch.uint8, device="cuda")
    c = Case(23, 16, 4, D, 64, 16, [700, 3, 90])
    c.check(c.run(workspace=ws))


def test_a_length_past_the_bound_is_still_right():
    """max_seq_len sizes the launch only."""
    c = Case(21, 8, 2, 128, 64, 16, [5000, 40, 900])
    for bound in (1, 100, 0, 10 ** 6):
        c.check(c.run(max_seq_len=bound))


def test_side_stream_and_two_graphs():
    import torch
    lens = np.array([5, 3000, 80, 1, 200, 7000])
    c = Case(22, 8, 2, 128, 64, 16, lens)
    args, side = c.args(), torch.cuda.Stream()
    torch.cuda.synchronize()
    o = qk.decode_attn_paged_q4(*args, group=64, stream=side)
    side.synchronize()
    c.check((o[0].cpu().numpy(), o[1].cpu().numpy(), 0))
    graphs = []
    for i in range(2):
        d = Case(30 + i, 8, 2, 128, 64, 16, lens)
        a, s = d.args(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            qk.decode_attn_paged_q4(*a, group=64)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                out = qk.decode_attn_paged_q4(*a, group=64)
        graphs.append((d, a, s, g, out))
    for i in range(3):
        for d, a, s, g, out in graphs:
            d.q = np.random.default_rng(40 + i).standard_normal(d.q.shape).astype(np.float32)
            d.lens = (np.arange(6) * 37 + 11 * i) % lens + 1
            d.lens = d.lens.astype(np.int32)
            a[0].copy_(_t(d.q))
            a[3].copy_(_t(d.lens))
        torch.cuda.synchronize()
        for _ in range(5):
            for d, a, s, g, out in graphs:
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for d, a, s, g, out in graphs:
            d.check((out[0].cpu().numpy(), out[1].cpu().numpy(), 0))


@pytest.mark.parametrize("own_workspace", [False, True])
def test_two_threads_on_one_stream(own_workspace):
    import threading
    import torch
    cases = [Case(60 + i, 8, 2, 128, 64, 16, 1000 * (i + 1) + np.arange(7 + 30 * i) * 13)
             for i in range(2)]
    stream = torch.cuda.Stream()
    args = [c.args() for c in cases]
    kw = {"stream": stream}
    if own_workspace:
        kw["workspace"] = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got, start = [[], []], threading.Barrier(2)

    def work(i):
        start.wait(60)
        for _ in range(200):
            got[i].append(qk.decode_attn_paged_q4(*args[i], group=64, **kw))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    stream.synchronize()
    for c, g in zip(cases, got):
        assert len(g) == 200
        c.check((g[0][0].cpu().numpy(), g[0][1].cpu().numpy(), 0))
        assert all(torch.equal(a, g[0][0]) and torch.equal(b, g[0][1]) for a, b in g)


def test_a_named_stream_takes_no_memory_in_use():
    import torch
    c = Case(54, 8, 2, 128, 64, 16, 256 + np.arange(64))
    args, side = c.args(), torch.cuda.Stream()
    x = torch.full(c.q.shape, 7.0, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    y = x.clone()
    del x
    out, lse = qk.decode_attn_paged_q4(*args, group=64, stream=side)
    torch.cuda.synchronize()
    assert (y == 7).all()
    c.check((out.cpu().numpy(), lse.cpu().numpy(), 0))


def test_pool_past_four_giga_bytes():
    """Offsets of pages past 32 bits: append, gather and decode in the pool's last pages."""
    import torch
    D, group, H, bs = 128, 32, 8, 256
    per = qk.decode_attn_q4_page_bytes(bs, D, group) * H
    NB = (9 << 29) // per
    pool = torch.empty((NB, H, per // H), dtype=torch.uint8, device="cuda")
    L = 3 * bs - 5
    table = np.array([[NB - 1, 0, NB - 2]], np.int32)
    r = np.random.default_rng(80)
    x = torch.from_numpy(r.standard_normal((L, 2 * H, D)).astype(np.float32)).cuda()
    pos, seq = torch.arange(L, dtype=torch.int32, device="cuda"), torch.zeros(
        L, dtype=torch.int32, device="cuda")
    qk.decode_attn_append_paged_q4(x[:, :H], x[:, H:], pos, _t(table), pool, group=group,
                                   token_seq=seq)
    k, v = qk.decode_attn_gather_paged_q4(pos, _t(table), pool, head_dim=D, group=group,
                                          token_seq=seq, dtype=torch.float32)
    c = Case(80, 16, H, D, group, bs, [L])
    for i, rows in enumerate((x[:, :H], x[:, H:])):
        codes, s, z = quantised(_np(rows), group)
        ref = codes * np.repeat(s.astype(np.float64), group, -1) + np.repeat(
            z.astype(np.float64), group, -1)
        assert (np.abs(_np((k, v)[i]) - ref) <= U * np.abs(ref)).all()
        for t in range(L):
            at = (c.table[0, t // bs], slice(None), t % bs)
            c.cache.codes[i][at], c.cache.scale[i][at], c.cache.zero[i][at] = codes[t], s[t], z[t]
    out, lse = qk.decode_attn_paged_q4(_t(c.q), pool, _t(table), _t(c.lens), group=group)
    c.check((out.cpu().numpy(), lse.cpu().numpy(), 0))


# ------------------------------------------------------------------ together
def test_calls_behind_one_another():
    """Append, read back and decode over and over without a wait between: each sees what
    the one before it wrote (a kernel may be set up while the one before it still runs)."""
    import torch
    B, Hq, H, D, group, bs, steps = 40, 8, 2, 128, 32, 16, 30
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn((steps, B, Hq + 2 * H, D), generator=g, device="cuda")
    table = torch.randperm(4 * B, generator=g, device="cuda").int().view(B, 4)
    shape = (4 * B, H, qk.decode_attn_q4_page_bytes(bs, D, group))
    runs = []
    for wait in (True, False):
        pool = torch.zeros(shape, dtype=torch.uint8, device="cuda")
        got = []
        for i in range(steps):
            pos = torch.full((B,), i, dtype=torch.int32, device="cuda")
            lens = pos + 1
            k, v = x[i, :, Hq:Hq + H], x[i, :, Hq + H:]
            calls = (lambda: qk.decode_attn_append_paged_q4(k, v, pos, table, pool, group=group,
                                                            q=x[i, :, :Hq]),
                     lambda: qk.decode_attn_gather_paged_q4(pos, table, pool, head_dim=D, group=group),
                     lambda: qk.decode_attn_paged_q4(got[-2], pool, table, lens, group=group))
            for call in calls:
                if wait:
                    torch.cuda.synchronize()
                got.append(call())
        torch.cuda.synchronize()
        runs.append([t for y in got for t in (y if isinstance(y, tuple) else (y,))])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


@pytest.mark.parametrize("what", ["append", "gather"])
def test_cache_calls_in_two_graphs(what):
    """Captured on streams of their own, replayed in turn with new inputs in place."""
    import torch
    N, H, D, group, bs = 50, 3, 64, 64, 8
    r = np.random.default_rng(91)
    runs = []
    for i in range(2):
        x = torch.zeros((N, 2 * H, D), device="cuda")
        pos = torch.zeros(N, dtype=torch.int32, device="cuda")
        table = _t(r.permutation(N * 2).astype(np.int32).reshape(N, 2))
        pool = torch.zeros((N * 2, H, qk.decode_attn_q4_page_bytes(bs, D, group)), dtype=torch.uint8,
                           device="cuda")
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()

        def call(x=x, pos=pos, table=table, pool=pool):
            if what == "append":
                return qk.decode_attn_append_paged_q4(x[:, :H], x[:, H:], pos, table, pool, group=group)
            return qk.decode_attn_gather_paged_q4(pos, table, pool, head_dim=D, group=group)

        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            call()
            with torch.cuda.graph(g, stream=s):
                out = call()
        runs.append((x, pos, table, pool, s, g, out))
    for _ in range(3):
        for x, pos, table, pool, s, g, out in runs:
            x.copy_(_t(r.standard_normal(x.shape).astype(np.float32)))
            pos.copy_(_t(r.integers(0, 16, N).astype(np.int32)))
            if what == "gather":
                pool.copy_(_t(Cache(N * 2, H, bs, D, group).fill(r).bytes()))
            else:
                pool.zero_()
        torch.cuda.synchronize()
        for x, pos, table, pool, s, g, out in runs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for x, pos, table, pool, s, g, out in runs:
            c = Cache.of_bytes(pool.cpu().numpy(), bs, D, group)
            p, t = pos.cpu().numpy(), table.cpu().numpy()
            for n in range(N):
                at = (t[n, p[n] // bs], slice(None), p[n] % bs)
                for j in range(2):
                    if what == "append":
                        want = quantised(_np(x)[n, j * H:(j + 1) * H], group)
                        for a, b in zip((c.codes, c.scale, c.zero), want):
                            assert np.array_equal(a[j][at], b)
                    else:
                        ref = c.values()[j][at]
                        assert (np.abs(_np(out[j])[n] - ref) <= 2.0 ** -11 * np.abs(ref) + 2.0 ** -25).all()


@pytest.mark.parametrize("T", [1, 3])
def test_a_serving_run(T):
    """Prompts, then steps: lengths planned, tokens appended (keys and queries rotated), attended,
    rejected drafts given back and a request ended, all captured once and replayed."""
    import torch
    r = np.random.default_rng(90)
    B, Hq, H, D, group, bs, mb, NB = 4, 8, 2, 128, 64, 16, 24, 70
    f = qk.decode_attn_rope_freqs(D)
    dev = dict(dtype=torch.int32, device="cuda")
    table = torch.full((B, mb), -1, **dev)
    free, count = torch.from_numpy(r.permutation(NB).astype(np.int32)).cuda(), torch.tensor([NB], **dev)
    pool = torch.zeros((NB, H, qk.decode_attn_q4_page_bytes(bs, D, group)), dtype=torch.uint8,
                       device="cuda")
    status = _status()
    lens = torch.zeros(B, **dev)
    ref = [[] for _ in range(B)]  # (k, v) of every token, quantised

    def plan(new, n):
        got = qk.decode_attn_plan_blocks(lens, new, table, free, count, block_size=bs,
                                         num_blocks=NB, max_tokens=n, dev_status=status)
        lens.copy_(new)
        return got

    def rows(n):
        return torch.from_numpy(r.standard_normal((n, Hq + 2 * H, D)).astype(np.float32)).cuda()

    def remember(x, pos, seq):
        k, _ = qk.decode_attn_qk_norm_rope(None, x[:, Hq:Hq + H], pos, f, norm=False)
        k64, _ = norm_rope(_np(x[:, Hq:Hq + H]), pos.cpu().numpy(), f.cpu().numpy())
        for n, (p, s) in enumerate(zip(pos.tolist(), seq.tolist())):
            if s >= 0:
                assert len(ref[s]) == p
                ref[s].append((k64[n], _np(x[n, Hq + H:])))

    prompts = torch.tensor([37, 100, 1, 250], **dev)
    pos, seq, slots, cu = plan(prompts, 400)
    assert cu.tolist() == [0, 37, 137, 138, 388] and int((seq >= 0).sum()) == 388
    x = rows(400)
    qk.decode_attn_append_paged_q4(x[:, Hq:Hq + H], x[:, Hq + H:], pos, table, pool, f, group=group,
                                   token_seq=seq, dev_status=status)
    remember(x, pos, seq)

    new = torch.zeros(B, **dev)
    x = rows(B * T)
    outs = {}

    def step():
        pos, seq, slots, cu = plan(new, B * T)
        q = qk.decode_attn_append_paged_q4(x[:, Hq:Hq + H], x[:, Hq + H:], pos, table, pool, f,
                                           group=group, token_seq=seq, q=x[:, :Hq],
                                           dev_status=status)
        outs["q"] = q.view(B, T, Hq, D)
        outs["o"], outs["l"] = qk.decode_attn_paged_q4(outs["q"], pool, table, lens, group=group,
                                                       dev_status=status)
        outs["pos"], outs["seq"] = pos, seq

    s = torch.cuda.Stream()
    saved = [t.clone() for t in (table, free, count, pool, lens)]
    new.copy_(lens + T)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        for a, b in zip((table, free, count, pool, lens), saved):
            a.copy_(b)
        with torch.cuda.graph(g, stream=s):
            step()
    torch.cuda.synchronize()
    for i in range(4):
        new.copy_(lens + T)
        x.copy_(rows(B * T))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        remember(x, outs["pos"], outs["seq"])
        # what the pages hold, against the rows that went in
        cache = Cache.of_bytes(pool.cpu().numpy(), bs, D, group)
        vals, tab = cache.values(), table.cpu().numpy()
        for b in range(B):
            for t, (k, v) in enumerate(ref[b]):
                at = (tab[b, t // bs], slice(None), t % bs)
                for j, row in enumerate((k, v)):
                    sc = np.repeat(cache.scale[j][at].astype(np.float64), group, -1)
                    assert (np.abs(vals[j][at] - row) <= sc * 0.52 + 4e-3).all()
        ro, rl, _ = attend(outs["q"].cpu().numpy(), cache, tab, lens.cpu().numpy())
        assert np.abs(outs["o"].cpu().numpy() - ro).max() <= 2e-5
        assert np.abs(outs["l"].cpu().numpy() - rl).max() <= 2e-5
        # no page is in two places
        held = np.concatenate([tab[tab >= 0], free.cpu().numpy()[:int(count.item())]])
        assert sorted(held.tolist()) == list(range(NB))
        if T > 1:  # one drafted token of each is rejected
            plan(lens - 1, 0)
            for b in range(B):
                ref[b].pop()
        if i == 1:  # request 1 ends, another takes its slot
            end = lens.clone()
            end[1] = 0
            plan(end, 0)
            ref[1].clear()
            start = lens.clone()
            start[1] = 20
            pos, seq, _, _ = plan(start, 20)
            y = rows(20)
            qk.decode_attn_append_paged_q4(y[:, Hq:Hq + H], y[:, Hq + H:], pos, table, pool, f,
                                           group=group, token_seq=seq, dev_status=status)
            remember(y, pos, seq)
