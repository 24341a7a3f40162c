"""Decode of a batch that shares a prefix, on the GPU against the oracle's
decode of every sequence alone through a table that holds the prefix."""
import numpy as np
import pytest

import oracle
import quantized_kv_decode_paged_gb300 as qk
from rope64 import half_bound, norm_rope

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    yield
    import torch
    torch.cuda.empty_cache()


def _t(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    """A pool, a prefix table and full tables (prefix first) for the oracle;
    the library's block_table holds junk in the prefix columns when
    ``junk``."""

    def __init__(self, seed, B, Hq, Hkv, D, bs, prefix_len, lens, T=1, q_scale=1.0, junk=True,
                 extra_pages=0):
        r = np.random.default_rng(seed)
        self.T, self.D, self.prefix_len, self.bs = T, D, prefix_len, bs
        self.lens = np.asarray(lens, np.int32)
        P = prefix_len // bs
        own = np.maximum(0, -(-np.maximum(self.lens, 0) // bs) - P)
        mb = max(1, P + int(own.max()), -(-prefix_len // bs)) + extra_pages
        NB = P + int(own.sum()) + 2
        perm = r.permutation(NB).astype(np.int32)
        self.full = np.full((B, mb), -1, np.int32)
        self.full[:, :P] = perm[:P]
        at = P
        for b in range(B):
            self.full[b, P:P + own[b]] = perm[at:at + own[b]]
            at += own[b]
        self.prefix_table = perm[:P].copy()
        self.table = self.full.copy()
        if junk:
            self.table[:, :P] = r.integers(-5, 2 ** 31 - 1, (B, P))
        self.k = r.standard_normal((NB, bs, Hkv, D)).astype(np.float16)
        self.v = r.standard_normal((NB, bs, Hkv, D)).astype(np.float16)
        shape = (B, Hq, D) if T == 1 else (B, T, Hq, D)
        self.q = (r.standard_normal(shape) * q_scale).astype(np.float32)
        self.q_pos = None
        self.kw = {}

    def run(self, **kw):
        import torch
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = qk.decode_attn_paged_prefix(
            _t(self.q), _t(self.k), _t(self.v), _t(self.table), _t(self.lens), self.prefix_len,
            _t(self.prefix_table), None if self.q_pos is None else _t(self.q_pos),
            max_seq_len=int(max(0, self.lens.max())), dev_status=status, **self.kw, **kw)
        torch.cuda.synchronize()
        return out.cpu().numpy(), lse.cpu().numpy(), int(status.item())

    def want(self):
        return oracle.decode_paged(self.q, self.k, self.v, self.full, self.lens, self.q_pos,
                                   **self.kw)

    def bounds(self):
        """(out, lse): how far f32 results may be off.  u = 2^-24.

        Scores: q is held as two f16 terms of its row scaled to a power of two
        (2^-22 of the row's largest value a term) and the 2 D products are added
        in f32 in groups of 16 (2 D / 16 adds, a step of 2^-23 each at most):
        eps = scale * max_j sum_d |q_d k_jd| * (D / 8 + 8) * 2^-23, and the
        softcap adds 4 u of the cap.  Weights: 2^x is good to 2^-22, two f16
        terms hold a weight to 2^-22: 8 u.  Values: the weighted sum of n keys
        adds 2 n / 16 groups, and merging states a few more roundings:
        (n / 8 + 32) * 2^-23 of sum p |v| <= max |v|."""
        scale = self.kw.get("scale") or 1.0 / np.sqrt(self.D)
        kmax = np.abs(self.k[np.isfinite(self.k)].astype(np.float64)).max()
        mag = np.abs(self.q.astype(np.float64)).sum(-1).max() * kmax * scale
        n = max(1, int(self.lens.max()))
        eps = mag * (self.D / 8 + 8) * 2.0 ** -23 + self.kw.get("softcap", 0.0) * 4 * 2.0 ** -24
        chain = (n / 8 + 32) * 2.0 ** -23
        vmax = np.abs(self.v[np.isfinite(self.v)].astype(np.float64)).max()
        return vmax * (2 * eps + 8 * 2.0 ** -24 + chain), 2 * eps + chain

    def check(self, got=None, flags=0):
        out, lse, fl = got if got is not None else self.run()
        ro, rl, rf = self.want()
        assert fl == flags == rf, (fl, rf)
        ro, rl = ro.reshape(out.shape), rl.reshape(lse.shape)
        bo, bl = self.bounds()
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(lse), empty)
        assert (out[empty] == 0).all()
        err = np.abs(out - ro)
        assert not (~(err <= bo)).any(), f"out off by {np.nanmax(err):.3e}, bound {bo:.3e}"
        lerr = np.abs(lse[~empty] - rl[~empty])
        assert not (~(lerr <= bl + 2.0 ** -23 * np.abs(rl[~empty]))).any(), f"lse {lerr.max():.3e}"


def _lens(rng, B, prefix, most):
    return prefix + rng.integers(1, most, B)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (7, 1), (6, 6), (40, 8)])
@pytest.mark.parametrize("bs", [8, 16, 64, 256])
def test_head_layouts_and_page_sizes(D, Hq, Hkv, bs):
    r = np.random.default_rng(D + Hq + bs)
    prefix = 3 * bs if bs >= 64 else 11 * bs
    Case(1, 5, Hq, Hkv, D, bs, prefix, _lens(r, 5, prefix, 150)).check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 127, 128, 129, 255, 257, 640, 1000])
def test_prefix_lengths(D, prefix):
    """Also prefixes that end inside a page (those keys come from the
    sequence's own pages) or inside a tile, and none at all."""
    r = np.random.default_rng(prefix + D)
    lens = np.concatenate([[prefix + 1], _lens(r, 3, prefix, 90), [prefix + 128, prefix + 129]])
    Case(2, 6, 8, 2, D, 16, prefix, lens).check()


@pytest.mark.parametrize("T", [2, 3, 4, 20])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 2), (128, 8, 1), (256, 4, 2)])
def test_query_tokens(T, D, Hq, Hkv):
    """Several tokens a sequence (T * G of 160 needs two row tiles for one
    sequence), some sequences shorter than T."""
    r = np.random.default_rng(T + D)
    lens = np.concatenate([_lens(r, 4, 200, 180) + T, [1, T]])
    Case(3, 6, Hq, Hkv, D, 16, 200, lens, T=T).check()


@pytest.mark.parametrize("B", [1, 2, 33, 128, 300, 520])
def test_batches(B):
    """Row tiles that cut through a sequence's heads, and batches past one
    launch's."""
    r = np.random.default_rng(B)
    Case(4, B, 15, 3, 64, 16, 320, _lens(r, B, 320, 70)).check()


@pytest.mark.parametrize("D,T", [(64, 1), (128, 1), (128, 3), (256, 1)])
@pytest.mark.parametrize("prefix,most", [(16, 40), (16, 700), (300, 20), (0, 300)])
def test_many_parts_a_processor(D, T, prefix, most):
    """So many units that every CTA goes through runs of parts with many rows,
    of parts with few, and from the ones to the others."""
    r = np.random.default_rng(prefix + most + D)
    Case(24, 160, 64, 8, D, 16, prefix, _lens(r, 160, prefix, most) + T - 1, T=T).check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("prefix,longest", [(4096, 40), (64, 3000), (0, 5000), (2048, 2048)])
def test_long_axes(D, prefix, longest):
    """One long part beside a short one: the work is split along it."""
    r = np.random.default_rng(prefix + D)
    lens = prefix + np.array([longest, 1, longest // 2 + 1, 7])
    Case(5, 4, 8, 2, D, 16, prefix, r.permutation(lens)).check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 33, 300, 5000])
@pytest.mark.parametrize("T", [1, 3])
def test_sliding_windows(D, window, T):
    """Windows that end before, inside and past the prefix."""
    c = Case(6, 4, 4, 2, D, 16, 512, [512 + T, 540, 700, 900], T=T)
    c.kw = dict(sliding_window=window)
    c.check()


@pytest.mark.parametrize("softcap", [0.5, 30.0, 50.0, 1e4])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_softcap_and_scale(softcap, D):
    c = Case(7, 3, 8, 4, D, 32, 256, [300, 257, 420], q_scale=3.0)
    c.kw = dict(softcap=softcap, scale=0.11)
    c.check()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_short_empty_and_full_sequences(D):
    """Sequences inside the prefix (one key to all of it), none, all of the
    prefix and no more; the first and the last slot empty."""
    c = Case(8, 8, 8, 2, D, 16, 640, [0, 1, 639, 640, 641, 128, 129, 0])
    c.check()
    c = Case(9, 3, 8, 2, D, 16, 640, [0, 0, 0], extra_pages=1)
    c.check()
    # every sequence ends inside the prefix
    Case(10, 3, 8, 2, D, 16, 640, [5, 100, 300]).check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("T", [1, 2])
def test_query_positions(causal, T):
    """Positions before, inside and after the prefix, past the end, and a
    negative one (flagged, the row is empty)."""
    c = Case(11, 6, 8, 2, 128, 16, 320, [400, 400, 330, 380, 400, 390], T=T)
    c.q_pos = np.array([0, 319, 320, 5000, -1, 389], np.int32)
    c.kw = dict(causal=causal)
    c.check(flags=qk.DEV_BAD_QPOS)
    c.q_pos = None
    c.kw = dict(causal=causal, sliding_window=100)
    c.check()


def test_bad_pages_and_lengths_are_masked_and_flagged():
    """Page ids outside the pool, in the prefix and in own pages, and lengths
    outside the table: masked or clamped, with their flags."""
    c = Case(12, 5, 8, 2, 128, 16, 320, [400, 330, 321, 380, 352])
    nb = len(c.k)
    for tab in (c.full, c.table):
        tab[1, 20] = nb
        tab[2, 20] = -1
    c.prefix_table[3] = -9
    c.prefix_table[19] = nb + 7
    c.full[:, 3] = -9
    c.full[:, 19] = nb + 7
    c.check(flags=qk.DEV_BAD_BLOCK)
    c = Case(13, 3, 8, 2, 64, 16, 320, [400, 400, 400])
    c.lens[0] = -4
    c.lens[2] = 10 ** 9
    want = c.want()
    assert want[2] == qk.DEV_BAD_SEQ_LEN
    out, lse, fl = c.run()
    assert fl == qk.DEV_BAD_SEQ_LEN
    c.lens[2] = c.full.shape[1] * 16  # bounds() wants the real length
    bo, bl = c.bounds()
    assert (np.abs(out - want[0].reshape(out.shape)) <= bo).all()
    assert np.isneginf(lse[0]).all() and np.abs(lse[1:] - want[1].reshape(lse.shape)[1:]).max() <= bl + 1e-6


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("poison", [np.nan, np.inf, -np.inf])
def test_nonfinite_values_in_masked_places(D, poison):
    """Rows past a sequence's end, keys below its window, prefix keys past a
    short sequence, and every page no table names: none reaches a row that
    does not see it."""
    c = Case(14, 4, 8, 2, D, 16, 320, [333, 350, 200, 375])
    c.kw = dict(sliding_window=250)
    used = np.zeros(c.k.shape[:2], bool)
    seen_all = np.zeros(c.k.shape[:2], bool)
    lo = np.maximum(0, c.lens - 250)
    for b in range(4):
        for t in range(int(lo[b]), int(c.lens[b])):
            used[c.full[b, t // 16], t % 16] = True
            if t < 200 or t >= 320 or b == 3:
                seen_all[c.full[b, t // 16], t % 16] = True
    # poison what nobody sees, and the prefix keys [210, 240) that the short
    # sequence 2 (200 keys) does not see: rows 0, 1 and 3 must turn NaN or stay
    # away from it; row 2 stays exact
    k0, v0 = c.k.copy(), c.v.copy()
    c.k[~used], c.v[~used] = poison, poison
    c.check()
    for t in range(210, 240):
        c.v[c.full[0, t // 16], t % 16] = poison
        if poison != -np.inf:
            c.k[c.full[0, t // 16], t % 16] = poison
    out, lse, fl = c.run()
    d = Case(14, 4, 8, 2, D, 16, 320, [333, 350, 200, 375])
    d.kw, d.k, d.v = c.kw, k0, v0
    ro, rl, _ = d.want()
    ro, rl = ro.reshape(out.shape), rl.reshape(lse.shape)
    bo, bl = d.bounds()
    assert fl == 0
    assert (np.abs(out[2] - ro[2]) <= bo).all() and (np.abs(lse[2] - rl[2]) <= bl + 1e-6).all()
    assert not np.isfinite(out[[0, 1, 3]]).any()


def test_query_values_of_any_size():
    """Rows of very large, very small, zero and non-finite queries; a bad row
    does not touch its neighbours in the tile."""
    c = Case(15, 6, 4, 2, 128, 16, 256, [260, 300, 290, 270, 280, 257])
    c.q[0] *= 1e-30
    c.q[1] *= 1e4
    c.q[2] = 0
    c.q[3, 0] = np.nan
    c.q[4, 1, 7] = np.inf
    out, lse, _ = c.run()
    ro, rl, _ = c.want()
    ro, rl = ro.reshape(out.shape), rl.reshape(lse.shape)
    assert np.isnan(out[3, 0]).all() and not np.isfinite(out[4, 1]).any()
    c.q[3, 0], c.q[4, 1, 7] = 0, 0  # for the bound
    big, c.q[1] = c.q[1].copy(), 0
    bo, bl = c.bounds()
    for b, h in ((0, slice(None)), (2, slice(None)), (3, slice(1, 4)), (5, slice(None))):
        assert (np.abs(out[b, h] - ro[b, h]) <= bo).all(), b
        assert (np.abs(lse[b, h] - rl[b, h]) <= bl + 1e-6).all(), b
    # scores of thousands: one key takes all, or nearly
    c.q[:] = 0
    c.q[1] = big
    bo, bl = c.bounds()
    assert (np.abs(out[1] - ro[1]) <= bo).all()
    assert (np.abs(lse[1] - rl[1]) <= bl + 2.0 ** -22 * np.abs(rl[1])).all()


def test_low_parts_of_queries_and_weights():
    """Results that live in the low bits of q (scores that cancel in f16) and
    of the weights (two nearly equal ones against opposite values)."""
    r = np.random.default_rng(16)
    c = Case(16, 2, 2, 1, 128, 16, 128, [130, 140])
    # neighbouring values of every key cancel, and every q_d is 1 + s_d 2^-12: the score is
    # scale * 2^-12 * sum s_d k_d with k = +-64, at most 2 / sqrt(128)
    k = np.where(r.random(c.k.shape) < 0.5, 1, -1)
    k[..., 1::2] = -k[..., ::2]
    c.k = (64 * k).astype(np.float16)
    c.q = (1 + np.where(r.random(c.q.shape) < 0.5, 1, -1) * 2.0 ** -12).astype(np.float32)
    out, lse, _ = c.run()
    ro, rl, _ = c.want()
    spread = np.abs(ro.reshape(out.shape) - c.v[c.full[0, :8]].astype(np.float64).mean((0, 1))[0])
    # the pairs' sums are exact, the rest's partial sums stay below 2: 32 adds of a step of 2^-23,
    # and the products with the scale
    eps = 2 * (32 + 4) * 2.0 ** -23 / np.sqrt(128)
    tol = 4.6 * (2 * eps + (140 / 8 + 40) * 2.0 ** -23)
    assert np.abs(out - ro.reshape(out.shape)).max() <= tol
    assert spread.max() > 100 * tol
    c = Case(17, 2, 2, 1, 64, 16, 16, [18, 18])
    c.q[:] = 0
    c.q[..., 0] = 1
    c.k[:] = 0
    c.v[:] = 1
    own = c.full[:, 1]
    c.v[own, 0] = -17  # 17 keys of weight w0 against one of weight 1
    c.k[own, 0, :, 0] = np.float16(2.0 ** -9)
    out, lse, _ = c.run()
    ro, _, _ = c.want()
    # 17 - 17 e^(2^-9 / 8): of the size 17 * 2^-12 / 18; weights good to 2^-21
    assert 1e-4 < np.abs(ro).max() < 1e-2
    assert np.abs(out - ro.reshape(out.shape)).max() <= 2 * 17 * 2.0 ** -21


def test_equals_the_unshared_decode():
    """The same result as decode_attn_paged and decode_attn_paged_multi on the
    same tables, row 0 of the table standing for the prefix."""
    for T in (1, 3):
        c = Case(18, 5, 8, 2, 128, 16, 640, [700, 650, 900, 641, 660], T=T, junk=False)
        args = [_t(x) for x in (c.q, c.k, c.v, c.full, c.lens)]
        a = qk.decode_attn_paged_prefix(*args, 640)
        b = (qk.decode_attn_paged if T == 1 else qk.decode_attn_paged_multi)(*args)
        bo, bl = c.bounds()
        assert (a[0] - b[0]).abs().max().item() <= bo + 1e-6
        assert (a[1] - b[1]).abs().max().item() <= bl + 1e-6


def test_repeats_bit_for_bit_and_leaves_rows_behind_alone():
    import torch
    c = Case(19, 9, 8, 2, 128, 16, 2048, 2048 + np.arange(9) * 61 + 1)
    big = torch.full((12, 8, 128), 5.0, device="cuda")
    lbig = torch.full((12, 8), 5.0, device="cuda")
    a = c.run(out=big[:9], lse=lbig[:9])
    b = c.run()
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    assert (big[9:] == 5).all() and (lbig[9:] == 5).all()
    c.check(a)


def test_own_workspace_of_any_content_and_too_small():
    import torch
    c = Case(20, 4, 8, 2, 128, 16, 512, [600, 520, 700, 513])
    p = qk.DaParams(4, 8, 2, 128, 16, c.table.shape[1], len(c.k), 0, 0.0, 0.0, 0, 1)
    n = qk.decode_attn_paged_prefix_workspace_size(p, 1, 512)
    for fill in (0, 255):
        c.check(c.run(workspace=torch.full((n,), fill, dtype=torch.uint8, device="cuda")))
    with pytest.raises(qk.DecodeAttnError) as e:
        c.run(workspace=torch.zeros(n - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == qk.DA_ERR_WORKSPACE


def test_streams_and_two_graphs():
    """On a side stream, and two captured graphs replayed at once on two
    streams, each with its own workspace, over new inputs."""
    import torch
    c = Case(21, 6, 8, 2, 128, 16, 1024, 1024 + np.array([5, 300, 80, 1, 200, 33]))
    side = torch.cuda.Stream()
    args = [_t(x) for x in (c.q, c.k, c.v, c.table, c.lens)]
    pt = _t(c.prefix_table)
    torch.cuda.synchronize()
    o = qk.decode_attn_paged_prefix(*args, 1024, pt, stream=side)
    side.synchronize()
    c.check((o[0].cpu().numpy(), o[1].cpu().numpy(), 0))
    graphs = []
    for i in range(2):
        d = Case(30 + i, 6, 8, 2, 128, 16, 1024, c.lens)
        a = [_t(x) for x in (d.q, d.k, d.v, d.table, d.lens)]
        t = _t(d.prefix_table)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            qk.decode_attn_paged_prefix(*a, 1024, t)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                out = qk.decode_attn_paged_prefix(*a, 1024, t)
        graphs.append((d, a, t, s, g, out))
    torch.cuda.synchronize()
    for i in range(3):
        for d, a, t, s, g, out in graphs:
            d.q = np.random.default_rng(40 + i).standard_normal(d.q.shape).astype(np.float32)
            d.lens = (1024 + (np.arange(6) * 37 + 11 * i) % 300 % (d.lens - 1024) + 1).astype(np.int32)
            a[0].copy_(_t(d.q))
            a[4].copy_(_t(d.lens))
        torch.cuda.synchronize()
        for _ in range(5):
            for d, a, t, s, g, out in graphs:
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for d, a, t, s, g, out in graphs:
            d.check((out[0].cpu().numpy(), out[1].cpu().numpy(), 0))


def test_pool_past_two_giga_elements():
    """Pages whose element offsets pass 32 bits."""
    import torch
    H, D, bs, P = 8, 128, 16, 256
    NB = (1 << 32) // (bs * H * D) + 40
    c = Case(22, 2, 8, 8, D, bs, P, [P + 20, P + 9])
    n = len(c.k)
    pools = []
    for x in (c.k, c.v):
        t = torch.zeros((NB, bs, H, D), dtype=torch.float16, device="cuda")
        t[NB - n:] = _t(x)
        pools.append(t)
    shift = NB - n
    out, lse = qk.decode_attn_paged_prefix(_t(c.q), *pools, _t(np.where(c.full >= 0, c.full + shift, -1).astype(np.int32)),
                                           _t(c.lens), P)
    torch.cuda.synchronize()
    c.check((out.cpu().numpy(), lse.cpu().numpy(), 0))


@pytest.mark.parametrize("T", [1, 3])
def test_a_serving_step(T):
    """The operators as a step runs them: a prompt's shared keys appended once,
    each sequence's own keys appended ragged, then T new tokens normed,
    rotated and appended with their queries in one launch, and attended to."""
    rng = np.random.default_rng(50 + T)
    B, Hq, H, D, bs, P = 4, 8, 2, 128, 16, 96
    f = qk.decode_attn_rope_freqs(D)
    fh = f.cpu().numpy()
    qw, kw = [(1 + 0.1 * rng.standard_normal(D)).astype(np.float32) for _ in range(2)]
    own = np.array([3, 40, 17, 29])
    mb = (P + int(own.max()) + T + bs - 1) // bs
    NB = mb * B + P // bs
    perm = rng.permutation(NB).astype(np.int32)
    table = perm[:B * mb].reshape(B, mb).copy()
    table[:, :P // bs] = perm[-(P // bs):]
    import torch
    kp = torch.zeros((NB, bs, H, D), dtype=torch.float16, device="cuda")
    vp = torch.zeros_like(kp)
    K, V = np.zeros((NB, bs, H, D)), np.zeros((NB, bs, H, D))
    BK = np.zeros_like(K)

    def step(seq, pos, with_q):
        N = len(seq)
        x = torch.from_numpy(rng.standard_normal((N, Hq + 2 * H, D)).astype(np.float32)).cuda()
        x = x.bfloat16()
        q = qk.decode_attn_append_paged_rope(
            x[:, Hq:Hq + H], x[:, Hq + H:], _t(pos.astype(np.int32)), _t(table), kp, vp, f,
            token_seq=_t(seq.astype(np.int32)), q=x[:, :Hq] if with_q else None, norm=True,
            k_weight=_t(kw), q_weight=_t(qw) if with_q else None)
        h = x.double().cpu().numpy()
        y, b = norm_rope(h[:, Hq:Hq + H], pos, fh, norm=True, weight=kw)
        for n in range(N):
            at = table[seq[n], pos[n] // bs], pos[n] % bs
            K[at], V[at], BK[at] = y[n], h[n, Hq + H:], half_bound(y[n], b[n])
        if with_q:
            return q, norm_rope(h[:, :Hq], pos, fh, norm=True, weight=qw)[0]

    step(np.zeros(P, int), np.arange(P), False)
    step(np.repeat(np.arange(B), own), np.concatenate([P + np.arange(n) for n in own]), False)
    seq = np.repeat(np.arange(B), T)
    q, qref = step(seq, (P + own[:, None] + np.arange(T)).reshape(-1), True)
    lens = (P + own + T).astype(np.int32)
    assert (np.abs(kp.double().cpu().numpy() - K) <= BK).all()
    shape = (B, Hq, D) if T == 1 else (B, T, Hq, D)
    out, lse = qk.decode_attn_paged_prefix(q.view(shape), kp, vp, _t(table), _t(lens), P)
    # the attention is compared on the cache's own f16 values, the queries on their 64-bit form
    ro, rl, fl = oracle.decode_paged(qref.reshape(shape).astype(np.float32), kp.cpu().numpy(),
                                     vp.cpu().numpy(), table, lens)
    assert fl == 0
    # 24 u of |q| <= sqrt(2) * 1.5 * 11.4 (a normed row's largest value) on top of the scores' bound
    mag = np.abs(qref).sum(-1).max() * kp.abs().max().item() / np.sqrt(D)
    eps = mag * (D / 8 + 8 + 24) * 2.0 ** -23
    n = int(lens.max())
    vmax = vp.abs().max().item()
    assert np.abs(out.cpu().numpy() - ro.reshape(shape)).max() <= vmax * (2 * eps + (n / 8 + 40) * 2.0 ** -23)
    assert np.abs(lse.cpu().numpy() - rl.reshape(shape[:-1])).max() <= 2 * eps + (n / 8 + 40) * 2.0 ** -23


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_wait_that_runs_out_is_reported(D):
    """CTA 0's first copy left out: its consumers' waits run out after 50 ms,
    the kernel ends with DEV_TIMEOUT, and the next call is right again."""
    lib = qk.load_library()
    # long enough for CTA 0 to hold tiles beside the entries of the list that stand for a unit's cost
    c = Case(23, 2, 8, 8, D, 64, 16384, [16385, 16450])
    with qk.tuning(wait_limit_ms=50):
        lib.decode_attn_testing_skip_first_arm(1)
        try:
            assert c.run()[2] == qk.DEV_TIMEOUT
        finally:
            lib.decode_attn_testing_skip_first_arm(0)
    c.check()


@pytest.mark.parametrize("B,T,Hq,Hkv,D", [(130, 1, 8, 4, 128), (65, 1, 16, 2, 64), (90, 2, 14, 2, 128),
                                          (60, 3, 8, 1, 128), (140, 4, 8, 2, 64), (100, 1, 16, 8, 256),
                                          (144, 2, 12, 2, 256), (130, 1, 64, 64, 64)])
@pytest.mark.parametrize("prefix,most", [(80, 2), (600, 2), (600, 400), (3000, 60)])
def test_row_tiles_side_by_side(B, T, Hq, Hkv, D, prefix, most):
    """2 to 18 tiles of the batch's rows, with next to no own keys and with as
    many as the prefix has: groups of several widths, that leave CTAs out or places of their
    last block empty, and own keys that fill runs up."""
    r = np.random.default_rng(B + prefix)
    lens = prefix + T - 1 + r.integers(1, most, B)
    lens[::7] = prefix // 2  # shorter than the prefix
    Case(50, B, Hq, Hkv, D, 16, prefix, lens, T=T).check()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_sequence_holds_all_own_keys(D):
    lens = np.full(70, 320)
    lens[69] = 9000
    Case(51, 70, 8, 2, D, 16, 320, lens).check()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_on_16_byte_boundaries(D):
    """q and out 16 bytes past a 32-byte boundary: the same bits."""
    import torch
    c = Case(52, 9, 16, 2, D, 16, 512, 512 + np.arange(9) * 31 + 1)
    want = c.run()
    c.check(want)
    args = [_t(x) for x in (c.k, c.v, c.table, c.lens)]
    buf = torch.zeros(2 * c.q.size + 64, device="cuda")
    q = buf[4:4 + c.q.size].view(c.q.shape)
    out = buf[c.q.size + 12:2 * c.q.size + 12].view(c.q.shape)
    assert q.data_ptr() % 32 == 16 and out.data_ptr() % 32 == 16
    q.copy_(_t(c.q))
    _, lse = qk.decode_attn_paged_prefix(q, *args, 512, _t(c.prefix_table), out=out)
    assert np.array_equal(out.cpu().numpy(), want[0]) and np.array_equal(lse.cpu().numpy(), want[1])


def test_two_threads_on_streams_of_their_own():
    import threading
    import torch
    cases = [Case(60 + i, 20 + i, 8, 2, 128, 16, 1024, 1024 + np.arange(20 + i) * 13 + 1)
             for i in range(2)]
    got = [None, None]

    def work(i):
        c, s = cases[i], torch.cuda.Stream()
        args = [_t(x) for x in (c.q, c.k, c.v, c.table, c.lens)]
        t = _t(c.prefix_table)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            for _ in range(20):
                out, lse = qk.decode_attn_paged_prefix(*args, 1024, t)
        s.synchronize()
        got[i] = (out.cpu().numpy(), lse.cpu().numpy(), 0)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for c, g in zip(cases, got):
        c.check(g)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_wait_that_runs_out_among_own_keys(D):
    """As above, with no prefix."""
    lib = qk.load_library()
    c = Case(53, 2, 8, 8, D, 64, 0, [16385, 9000])
    with qk.tuning(wait_limit_ms=50):
        lib.decode_attn_testing_skip_first_arm(1)
        try:
            assert c.run()[2] == qk.DEV_TIMEOUT
        finally:
            lib.decode_attn_testing_skip_first_arm(0)
    c.check()


def test_a_named_stream_takes_no_memory_in_use():
    """What a call with a stream of its own allocates is not memory whose last
    reader, on the current stream, is still to come."""
    import torch
    c = Case(54, 64, 8, 2, 128, 16, 256, 256 + np.arange(64) + 1)
    args = [_t(x) for x in (c.q, c.k, c.v, c.table, c.lens)]
    pt, side = _t(c.prefix_table), torch.cuda.Stream()
    x = torch.full(c.q.shape, 7.0, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    y = x.clone()
    del x
    out, lse = qk.decode_attn_paged_prefix(*args, 256, pt, stream=side)
    torch.cuda.synchronize()
    assert (y == 7).all()
    c.check((out.cpu().numpy(), lse.cpu().numpy(), 0))


def test_order_with_what_runs_before_and_after():
    """The kernels may be set up before the work ahead of them in the stream is
    done: copies, other kernels, each other and work joined from another stream, eager and
    captured, each with results that follow from the order alone."""
    import torch
    B, Hq, Hkv, D, bs, P = 40, 8, 2, 128, 16, 512
    r = np.random.default_rng(70)
    c = Case(71, B, Hq, Hkv, D, bs, P, P + r.integers(1, 60, B))
    src = [_t(r.standard_normal((B, Hq, D)).astype(np.float32)) for _ in range(2)]
    k, v, table, lens, pt = (_t(x) for x in (c.k, c.v, c.table, c.lens, c.prefix_table))
    want = [qk.decode_attn_paged_prefix(s, k, v, table, lens, P, pt) for s in src]
    q, lens2 = torch.zeros_like(src[0]), torch.zeros_like(lens)
    freqs = qk.decode_attn_rope_freqs(D)
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    got = [[torch.empty_like(t) for t in w] for w in want]

    def step():
        cur = torch.cuda.current_stream()
        for i in range(2):
            side.wait_stream(cur)
            with torch.cuda.stream(side):
                lens2.zero_()
                torch.cuda._sleep(20_000)
                lens2.add_(lens)
            q.copy_(src[1 - i])  # overwritten by the next, which has to come after it
            q.zero_()
            qk.decode_attn_qk_norm_rope(src[i], None, zero, freqs, norm=False, q_out=q)
            cur.wait_stream(side)
            qk.decode_attn_paged_prefix(q, k, v, table, lens2, P, pt, out=got[i][0], lse=got[i][1])
            q.zero_()

    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for _ in range(20):
            step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    for replay in range(2):
        for w, g in zip(want, got):
            assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])
            g[0].zero_()
            g[1].zero_()
        if replay == 0:
            with torch.cuda.graph(graph, stream=stream):
                step()
            for _ in range(20):
                graph.replay()
            torch.cuda.synchronize()


@pytest.mark.parametrize("path", ["C++", "Python", "own workspace"])
def test_two_threads_on_one_stream(path):
    """Calls of other sizes and inputs that go into the same stream at the same
    time: each gets its own result, bit for bit."""
    import threading
    import torch
    cases = [Case(64 + i, 7 + 30 * i, 8, 2, 128, 16, 1024 * (i + 1),
                  1024 * (i + 1) + np.arange(7 + 30 * i) * 13 + 1) for i in range(2)]
    stream = torch.cuda.Stream()
    args = [[_t(x) for x in (c.q, c.k, c.v, c.table, c.lens)] + [c.prefix_len, _t(c.prefix_table)]
            for c in cases]
    kw = {}
    if path != "C++":
        kw["stream"] = stream
    if path == "own workspace":
        kw["workspace"] = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got, start = [[], []], threading.Barrier(2)

    def work(i):
        with torch.cuda.stream(stream):
            start.wait(60)
            for _ in range(300):
                got[i].append(qk.decode_attn_paged_prefix(*args[i], **kw))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    stream.synchronize()
    for c, g in zip(cases, got):
        assert len(g) == 300
        c.check((g[0][0].cpu().numpy(), g[0][1].cpu().numpy(), 0))
        assert all(torch.equal(a, g[0][0]) and torch.equal(b, g[0][1]) for a, b in g)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_queries_next_to_the_largest_f32(D):
    """Rows whose largest value is past 2^127; every key is seen by every row."""
    c = Case(72, 3, 8, 2, D, 16, 256, [384, 384, 384])
    c.q *= 1e37
    c.q[..., 5] = np.where(c.q[..., 5] < 0, -3e38, 3e38)
    c.k = (c.k.astype(np.float32) / 64).astype(np.float16)
    c.kw = dict(scale=2e-38)
    c.check()


def test_a_query_that_is_not_finite_takes_no_longer():
    """A row that is NaN whatever its keys is not done again over all of them.  (The bound is a
    factor of ten; over 32,768 keys one at a time it was hundreds.)"""
    import torch
    c = Case(73, 4, 8, 2, 128, 16, 32768, 32768 + np.array([20, 1, 50, 33]))
    args = [_t(x) for x in (c.k, c.v, c.table, c.lens)] + [c.prefix_len, _t(c.prefix_table)]
    good = _t(c.q)
    bad = good.clone()
    bad[1], bad[2, 3, 7] = float("nan"), float("inf")

    def us(q):
        times = []
        for _ in range(9):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda.synchronize()
            a.record()
            out, _ = qk.decode_attn_paged_prefix(q, *args)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b) * 1e3)
        return sorted(times)[4], out

    t, want = us(good)
    tb, out = us(bad)
    assert torch.isnan(out[1]).all() and torch.isnan(out[2, 3]).any()
    assert torch.equal(out[[0, 3]], want[[0, 3]])
    assert tb <= 10 * t, f"{tb:.0f} us against {t:.0f}"


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [(384, 384, 384), (384, 380, 300)])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_visible_infinities(D, lens, softcap):
    """Keys whose scores are -inf have weight 0 (with a softcap that of the cap),
    infinite values are infinite in their column alone, whether or not the row
    meets tiles with masked keys."""
    def case():
        c = Case(74, 3, 8, 2, D, 16, 256, lens)
        c.kw = dict(softcap=softcap)
        c.q[..., 5] = np.abs(c.q[..., 5]) + 0.5
        return c

    c, d = case(), case()
    bounds = d.bounds()
    for b, t in ((0, 3), (0, 200), (0, 300), (1, 299)):
        at = c.full[b, t // 16], t % 16
        c.k[at][..., 5] = -np.inf
        # of the oracle: scores of -0.5 * 60000 / 16 and less, their weight e^-1800 of the others', and
        # a tanh that rounds to -1
        d.k[at][..., 5] = -60000
    for b, t, col, x in ((0, 7, 9, np.inf), (0, 310, 11, -np.inf)):
        at = c.full[b, t // 16], t % 16
        c.v[at][..., col] = x
        d.v[at][..., col] = 0
    out, lse, fl = c.run()
    ro, rl, rf = d.want()
    assert fl == rf == 0
    assert (out[..., 9] == np.inf).all()
    assert (out[0, :, 11] == -np.inf).all()
    keep = np.ones(out.shape, bool)
    keep[..., 9] = keep[0, :, 11] = False
    assert not (~(np.abs(out - ro.reshape(out.shape)) <= bounds[0]))[keep].any()
    assert not (~(np.abs(lse - rl.reshape(lse.shape)) <= bounds[1] + 1e-6)).any()


# rows of a kv head: few enough for one warp's lanes in the prefix and own keys; two tiles of the
# prefix, one of them full
ROWS = [(2, 2), (40, 4)]


@pytest.mark.parametrize("B,Hq", ROWS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_low_terms_of_queries(D, B, Hq):
    """Scores that live in the low bits of q: neighbouring values of every key
    cancel, k = +-64, and q_d = 1 + s_d 2^-12, so a score is scale * 2^-12 *
    sum s_d k_d, at most sqrt(D) / 64.  f16 alone sees no difference between keys."""
    r = np.random.default_rng(75)
    c = Case(75, B, Hq, 1, D, 16, 128, 128 + r.integers(1, 14, B))
    k = np.where(r.random(c.k.shape) < 0.5, 1, -1)
    k[..., 1::2] = -k[..., ::2]
    c.k = (64 * k).astype(np.float16)
    c.q = (1 + np.where(r.random(c.q.shape) < 0.5, 1, -1) * 2.0 ** -12).astype(np.float32)
    out, _, _ = c.run()
    ro = c.want()[0].reshape(out.shape)
    # the products of q's high term cancel within each sum of 16; those of its low one stay below
    # D / 64: D / 16 truncating adds of 2^-23 of that a term, and the products with the scale
    eps = (D / 64) * (D / 8 + 4) * 2.0 ** -23 / np.sqrt(D)
    tol = np.abs(c.v.astype(np.float64)).max() * (2 * eps + (142 / 8 + 40) * 2.0 ** -23)
    assert np.abs(out - ro).max() <= tol
    # what scores of zero would give
    flat = np.stack([c.v[c.full[b]].reshape(-1, D)[:c.lens[b]].astype(np.float64).mean(0)
                     for b in range(B)])[:, None]
    assert np.abs(ro - flat).max((1, 2)).min() > 20 * tol


@pytest.mark.parametrize("B,Hq", ROWS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("own", [False, True])
def test_low_terms_of_weights(D, B, Hq, own):
    """Weights next to each other against opposite values, in the prefix's keys
    or in own ones: 31 keys of weight w = e^(-2^-9 / sqrt(D)) and value 1, one
    of weight 1 and value -31, and a key of weight w and value 0 beside them."""
    c = Case(76, B, Hq, 1, D, 16, 32, np.full(B, 33 if not own else 64 + 32), junk=False)
    c.q[:] = 0
    c.q[..., 0] = 1
    c.k[:], c.v[:] = 0, 0
    for b in range(B):
        at = c.full[b, :2] if not own else c.full[b, 2:4]
        c.v[at] = 1
        c.v[at[0], 3] = -31
        c.k[at[0], 3, :, 0] = np.float16(2.0 ** -9)
    out, _, _ = c.run()
    ro = c.want()[0].reshape(out.shape)
    n = int(c.lens[0])
    # a weight is 2^x, good to 2^-22, in two terms, 2^-22: 62 of them times 2^-21 over n, and n / 8
    # + 32 adds of 2^-23 of partial sums of at most 31 / n
    tol = 62 / n * 2.0 ** -21 + (n / 8 + 32) * 2.0 ** -23 * 31 / n
    assert np.abs(out - ro).max() <= tol
    # one f16 term: every weight is 1, and the sum 0
    assert np.abs(ro).min() > 10 * tol


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,prefix,most", [(1, 1000, 60), (1, 96, 900), (4, 4096, 40)])
def test_errors_are_those_of_f32(D, T, prefix, most):
    """The root mean square of the error against that of the result, for
    normal inputs.

    A score: q's terms leave 2^-23 of the row's largest value, 4.5 of its
    deviation at most, in each of D products of deviation 1 / sqrt(D): 5.4e-7; its 2 D / 16
    truncating adds leave half of 2^-23 of a sum of order 1 each, D / 8 * 6e-8, up to 1.9e-6
    for D = 256.  Values: up to 16 such adds of 2^-23 in a group of two tiles, 1e-6 (D = 64:
    32 and 1.9e-6).  Together 4.5e-6 at most, counted as 2^-17 = 7.6e-6.  One f16 term of q or of
    the weights leaves 2^-12 or more: 30 times that."""
    r = np.random.default_rng(77)
    c = Case(77, 6, 16, 2, D, 16, prefix, _lens(r, 6, prefix, most) + T - 1, T=T)
    out, lse, _ = c.run()
    ro, rl, _ = c.want()
    rms = lambda x: np.sqrt(np.mean(np.square(x.astype(np.float64))))  # noqa: E731
    assert rms(out - ro.reshape(out.shape)) <= 2.0 ** -17 * rms(ro)
    assert rms(lse - rl.reshape(lse.shape)) <= 2.0 ** -17 * max(1.0, rms(rl))


def test_prefix_of_row_0_whatever_its_sequence_is():
    """Without a prefix_table row 0 holds the prefix's pages, its slot empty or its
    sequence short; pages that it lacks are masked for all and flagged."""
    import torch
    for first in (0, 3, 100):
        c = Case(78, 4, 8, 2, 128, 16, 320, [first, 400, 321, 350], junk=False)
        c.table[1:, :20] = -1  # not read
        args = [_t(x) for x in (c.q, c.k, c.v, c.table, c.lens)]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = qk.decode_attn_paged_prefix(*args, 320, dev_status=status)
        c.check((out.cpu().numpy(), lse.cpu().numpy(), int(status.item())))
        args[3][0, 7] = -1
        c.full[:, 7] = -1
        out, lse = qk.decode_attn_paged_prefix(*args, 320, dev_status=status)
        c.check((out.cpu().numpy(), lse.cpu().numpy(), int(status.item())), flags=qk.DEV_BAD_BLOCK)
