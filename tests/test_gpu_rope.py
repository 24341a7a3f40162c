"""Norm + rotation of queries and keys, and the rotating paged append, on the
GPU against 64-bit forms (rope64)."""
import numpy as np
import pytest

import quantized_kv_decode_paged_gb300 as qk
from rope64 import half_bound, norm_rope

pytestmark = pytest.mark.gpu

TYPES = ("float32", "float16", "bfloat16")


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    yield


def _t(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(getattr(torch, dtype))


def _np(t):
    return t.double().cpu().numpy()


def _close(got, want, bound, what):
    err = np.abs(_np(got) - want)
    assert err.shape == want.shape
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} off, worst ratio {np.nanmax(err / bound):.2f}"


def _freqs(rd, theta=10000.0):
    if rd == 0:
        return None, np.zeros(0, np.int64)
    f = qk.decode_attn_rope_freqs(rd, theta)
    return f, f.cpu().numpy()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,rd", [(64, 64), (64, 16), (128, 128), (128, 96), (256, 256), (256, 64),
                                  (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_matches_64_bits(dtype, D, rd, interleaved):
    rng = np.random.default_rng(D + rd)
    N, Hq, Hkv = 7, 5, 3
    x = _t(rng.standard_normal((N, Hq + Hkv, D)).astype(np.float32) * 2, dtype)
    pos = np.array([0, 1, 2, 1000, 131071, 2 ** 31 - 1, -5], np.int32)
    f, fh = _freqs(rd)
    for norm in (False, True):
        qw = (1 + rng.standard_normal(D) * 0.3).astype(np.float32) if norm else None
        kw = (rng.standard_normal(D) * 0.3).astype(np.float32) if norm else None
        q, k = qk.decode_attn_qk_norm_rope(
            x[:, :Hq], x[:, Hq:], _t(pos), f, norm=norm, q_weight=None if qw is None else _t(qw),
            k_weight=None if kw is None else _t(kw), weight_offset=0.0, eps=1e-5,
            interleaved=interleaved)
        kwargs = dict(norm=norm, eps=1e-5, interleaved=interleaved)
        y, b = norm_rope(_np(x[:, :Hq]), pos, fh, weight=qw, **kwargs)
        _close(q, y, b, "q")
        y, b = norm_rope(_np(x[:, Hq:]), pos, fh, weight=kw, **kwargs)
        _close(k, y, half_bound(y, b), "k")


@pytest.mark.parametrize("N,Hq,Hkv", [(1, 1, 1), (1, 64, 8), (3, 33, 1), (513, 7, 2), (2, 200, 100),
                                       (2433, 5, 1), (4871, 1, 2), (9999, 3, 3), (16381, 2, 1)])
def test_norm_rope_sizes_and_offset_weight(N, Hq, Hkv):
    rng = np.random.default_rng(N + Hq)
    D = 128
    q = _t(rng.standard_normal((N, Hq, D)).astype(np.float32), "bfloat16")
    k = _t(rng.standard_normal((N, Hkv, D)).astype(np.float32), "bfloat16")
    w = (rng.standard_normal(D) * 0.1).astype(np.float32)
    pos = rng.integers(0, 100000, N).astype(np.int32)
    f, fh = _freqs(D, 500000.0)
    qo, ko = qk.decode_attn_qk_norm_rope(q, k, _t(pos), f, q_weight=_t(w), weight_offset=1.0)
    y, b = norm_rope(_np(q), pos, fh, norm=True, weight=w, offset=1.0)
    _close(qo, y, b, "q")
    y, b = norm_rope(_np(k), pos, fh, norm=True)
    _close(ko, y, half_bound(y, b), "k")


def test_norm_rope_one_head_many_tokens():
    rng = np.random.default_rng(6)
    N, D = 12001, 64
    pos = rng.integers(0, 4096, N).astype(np.int32)
    f, fh = _freqs(D)
    q = _t(rng.standard_normal((N, 1, D)).astype(np.float32), "float16")
    y, b = norm_rope(_np(q), pos, fh, norm=True)
    out, _ = qk.decode_attn_qk_norm_rope(q, None, _t(pos), f)
    _close(out, y, b, "q")


def test_norm_rope_strides_one_side_and_in_place():
    """Rows of a wider tensor, head-major layouts, broadcast rows, q or k alone,
    and outputs that are the inputs."""
    import torch
    rng = np.random.default_rng(5)
    N, H, D = 9, 4, 64
    pos = rng.integers(0, 4096, N).astype(np.int32)
    f, fh = _freqs(D)
    wide = _t(rng.standard_normal((N, 3 * H + 1, D + 8)).astype(np.float32), "float16")
    for v in (wide[:, 1:1 + H, 8:], wide[:, 1:1 + 2 * H:2, :D],
              _t(rng.standard_normal((H, N, D)).astype(np.float32), "float16").transpose(0, 1),
              wide[:1, :H, :D].expand(N, H, D)):
        y, b = norm_rope(_np(v), pos, fh, norm=True)
        q, none = qk.decode_attn_qk_norm_rope(v, None, _t(pos), f)
        assert none is None
        _close(q, y, b, "q")
        none, k = qk.decode_attn_qk_norm_rope(None, v, _t(pos), f)
        assert none is None
        _close(k, y, half_bound(y, b), "k")
    q = _t(rng.standard_normal((N, H, D)).astype(np.float32))
    y, b = norm_rope(_np(q), pos, fh, norm=True)
    out, _ = qk.decode_attn_qk_norm_rope(q, None, _t(pos), f, q_out=q)
    assert out.data_ptr() == q.data_ptr()
    _close(q, y, b, "q in place")
    k = _t(rng.standard_normal((N, H, D)).astype(np.float32), "float16")
    y, b = norm_rope(_np(k), pos, fh, norm=True)
    _, out = qk.decode_attn_qk_norm_rope(None, k, _t(pos), f, k_out=k)
    assert out.data_ptr() == k.data_ptr()
    _close(k, y, half_bound(y, b), "k in place")
    # no tokens
    q, k = qk.decode_attn_qk_norm_rope(q[:0], k[:0].float(), _t(pos[:0]), f)
    assert q.shape == (0, H, D) and k.shape == (0, H, D)
    torch.cuda.synchronize()


def test_norm_rope_special_values():
    """A zero row stays zero, tiny and huge rows keep their direction, NaN and
    infinities stay in their own row, keys past f16's range become infinite."""
    N, H, D = 3, 4, 64
    x = np.ones((N, H, D), np.float32)
    x[0, 0] = 0
    x[0, 1] *= 1e-18
    x[0, 2] *= 1e18
    x[1, 0, 5] = np.nan
    x[1, 1, 6] = np.inf
    f, fh = _freqs(D)
    pos = np.array([3, 4, 5], np.int32)
    q, k = qk.decode_attn_qk_norm_rope(_t(x), _t(x), _t(pos), f, eps=1e-6)
    y, b = norm_rope(x[:, 2:], pos, fh, norm=True)
    _close(q[:, 2:], y, b, "q")
    assert (q[0, 0] == 0).all() and (k[0, 0] == 0).all()
    y, b = norm_rope(x[:1, 1:2], pos[:1], fh, norm=True)
    _close(q[:1, 1:2], y, b + 2.0 ** -126, "tiny")
    assert q[1, 0].isnan().all() and not q[1, 2:].isnan().any() and not q[2].isnan().any()
    _, k = qk.decode_attn_qk_norm_rope(None, _t(x * 1e5), _t(pos), f, norm=False)
    assert k[2].isinf().any() and not k[2].isnan().any()


def _cache(rng, B, npg, bs, H, D):
    NB = B * npg + 3
    table = rng.permutation(NB)[: B * npg].reshape(B, npg).astype(np.int32)
    return (table, rng.standard_normal((NB, bs, H, D)).astype(np.float16),
            rng.standard_normal((NB, bs, H, D)).astype(np.float16))


def _append_ref(k, v, pos, seq, table, kp, vp, bs, freqs, **kw):
    """Pools in 64 bits and their bounds after the valid tokens; untouched rows
    have bound 0."""
    y, b = norm_rope(k, pos, freqs, **kw)
    b = half_bound(y, b)
    v = v.astype(np.float64)
    K, V = kp.astype(np.float64), vp.astype(np.float64)
    bk, bv = np.zeros_like(K), np.zeros_like(V)
    for n in range(len(pos)):
        s, p = int(seq[n]), int(pos[n])
        if s < 0 or s >= table.shape[0] or p < 0 or p >= table.shape[1] * bs:
            continue
        pg = table[s, p // bs]
        if pg < 0 or pg >= kp.shape[0]:
            continue
        K[pg, p % bs], bk[pg, p % bs] = y[n], b[n]
        V[pg, p % bs], bv[pg, p % bs] = v[n], half_bound(v[n], 0.0)
    return K, bk, V, bv


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,rd,bs,il", [(64, 64, 8, False), (128, 128, 16, True),
                                        (128, 32, 16, False), (256, 256, 1, False), (256, 0, 32, False)])
@pytest.mark.parametrize("with_q", [False, True])
def test_append_matches_64_bits(dtype, D, rd, bs, il, with_q):
    """A ragged call: a prompt, single tokens, padding, and each kind of bad
    token, which writes nothing and raises its flag."""
    import torch
    rng = np.random.default_rng(D + rd + bs)
    B, H, Hq = 5, 3, 6
    npg = max(4, 40 // bs)
    table, kp, vp = _cache(rng, B, npg, bs, H, D)
    seq = np.array([0] * 21 + [1, 2, 3, 3] + [-1, -7] + [4, 4, 4, 4, 1], np.int32)
    pos = np.array(list(range(5, 26)) + [0, npg * bs - 1, 7, 8] + [1, -3]
                   + [npg * bs, -1, 0, 2 ** 31 - 1, 3], np.int32)
    seq[-1] = B + 2  # no such sequence
    table[4, 0] = len(kp)  # a page outside the pool
    N = len(seq)
    x = _t(rng.standard_normal((N, Hq + 2 * H, D)).astype(np.float32), dtype)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    f, fh = _freqs(rd)
    kw = (1 + 0.1 * rng.standard_normal(D)).astype(np.float32)
    qw = (1 + 0.1 * rng.standard_normal(D)).astype(np.float32)
    K, bk, V, bv = _append_ref(_np(k), _np(v), pos, seq, table, kp, vp, bs, fh, norm=True,
                               weight=kw, interleaved=il)
    tk, tv = _t(kp), _t(vp)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    canary = torch.full((N, Hq, D), 7.0, device="cuda")
    out = qk.decode_attn_append_paged_rope(
        k, v, _t(pos), _t(table), tk, tv, f, token_seq=_t(seq), q=q if with_q else None, norm=True,
        q_weight=_t(qw) if with_q else None, k_weight=_t(kw), interleaved=il,
        q_out=canary if with_q else None, dev_status=status)
    assert int(status.item()) == qk.DEV_BAD_BLOCK | qk.DEV_BAD_SEQ_LEN | qk.DEV_BAD_SEQ
    _close(tk, K, bk, "k pool")
    _close(tv, V, bv, "v pool")
    if with_q:
        y, b = norm_rope(_np(q), pos, fh, norm=True, weight=qw, interleaved=il)
        pad = seq < 0
        _close(out[torch.from_numpy(~pad).cuda()], y[~pad], b[~pad], "q")
        assert (out[torch.from_numpy(pad).cuda()] == 7.0).all()
    else:
        assert out is None


def test_append_of_a_long_ragged_prefill():
    """Many tokens, so that a CTA takes several at once, of three prompts and
    with padding between them."""
    rng = np.random.default_rng(13)
    B, H, D, bs = 3, 2, 64, 16
    lens = [7001, 1, 2444]
    npg = -(-max(lens) // bs)
    table, kp, vp = _cache(rng, B, npg, bs, H, D)
    seq = np.concatenate([np.full(n, b) for b, n in enumerate(lens)] + [np.full(555, -1)])
    pos = np.concatenate([np.arange(n) for n in lens] + [np.zeros(555)])
    order = rng.permutation(len(seq))
    seq, pos = seq[order].astype(np.int32), pos[order].astype(np.int32)
    x = _t(rng.standard_normal((len(seq), 2 * H, D)).astype(np.float32), "bfloat16")
    f, fh = _freqs(D)
    K, bk, V, bv = _append_ref(_np(x[:, :H]), _np(x[:, H:]), pos, seq, table, kp, vp, bs, fh)
    tk, tv = _t(kp), _t(vp)
    qk.decode_attn_append_paged_rope(x[:, :H], x[:, H:], _t(pos), _t(table), tk, tv, f,
                                     token_seq=_t(seq))
    _close(tk, K, bk, "k pool")
    _close(tv, V, bv, "v pool")


def test_append_without_rotation_equals_the_plain_append():
    """f16 rows, no norm, no frequencies, one token per sequence: bit for bit
    what decode_attn_append_paged writes."""
    import torch
    rng = np.random.default_rng(11)
    B, H, D, bs = 6, 2, 128, 16
    table, kp, vp = _cache(rng, B, 4, bs, H, D)
    pos = np.array([0, 17, 63, 30, 40, 64], np.int32)
    k = _t(rng.standard_normal((B, H, D)).astype(np.float16))
    v = _t(rng.standard_normal((B, H, D)).astype(np.float16))
    a = [_t(kp), _t(vp)]
    b = [_t(kp), _t(vp)]
    qk.decode_attn_append_paged(k, v, _t(pos), _t(table), *a)
    qk.decode_attn_append_paged_rope(k, v, _t(pos), _t(table), *b, None)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_append_past_two_giga_elements():
    """A pool whose element offsets pass 32 bits; the far page is written and
    the one 2^32 elements below it is not."""
    import torch
    H, D, bs = 8, 128, 16
    NB = (1 << 32) // (bs * H * D) + 2
    k_pool = torch.zeros((NB, bs, H, D), dtype=torch.float16, device="cuda")
    v_pool = torch.zeros((NB, bs, H, D), dtype=torch.float16, device="cuda")
    table = torch.tensor([[NB - 1]], dtype=torch.int32, device="cuda")
    k = torch.ones((1, H, D), dtype=torch.float16, device="cuda")
    qk.decode_attn_append_paged_rope(k, 2 * k, _t(np.array([5], np.int32)), table, k_pool, v_pool,
                                     None)
    assert (k_pool[NB - 1, 5] == 1).all() and (v_pool[NB - 1, 5] == 2).all()
    assert int(k_pool.view(-1, D).count_nonzero()) == H * D


def test_append_side_stream_and_graph_replay():
    """Launched on another stream, and captured once and replayed over new
    rows, positions and sequences (padding among them)."""
    import torch
    rng = np.random.default_rng(12)
    B, H, Hq, D, bs, N = 4, 2, 4, 128, 16, 6
    table, kp, vp = _cache(rng, B, 4, bs, H, D)
    f, fh = _freqs(D)
    side = torch.cuda.Stream()
    x = torch.zeros((N, Hq + 2 * H, D), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(N, dtype=torch.int32, device="cuda")
    seq = torch.zeros(N, dtype=torch.int32, device="cuda")
    tk, tv, tt = _t(kp), _t(vp), _t(table)
    torch.cuda.synchronize()

    def call(stream=None):
        return qk.decode_attn_append_paged_rope(x[:, Hq:Hq + H], x[:, Hq + H:], pos, tt, tk, tv, f,
                                                token_seq=seq, q=x[:, :Hq], norm=True,
                                                stream=stream)

    def fresh(i):
        r = np.random.default_rng(100 + i)
        x.copy_(torch.from_numpy(r.standard_normal(x.shape).astype(np.float32)))
        s = np.array([0, 1, 2, 3, 0, -1], np.int32)
        p = (np.array([3, 9, 60, 0, 4, 5]) + (i % 2)).astype(np.int32)
        pos.copy_(torch.from_numpy(p))
        seq.copy_(torch.from_numpy(s))
        tk.copy_(torch.from_numpy(kp))
        tv.copy_(torch.from_numpy(vp))
        K, bk, V, bv = _append_ref(_np(x[:, Hq:Hq + H]), _np(x[:, Hq + H:]), p, s, table, kp, vp,
                                   bs, fh, norm=True)
        y, b = norm_rope(_np(x[:, :Hq]), p, fh, norm=True)
        return K, bk, V, bv, y[:5], b[:5]

    K, bk, V, bv, y, b = fresh(0)
    torch.cuda.synchronize()
    q = call(stream=side)
    side.synchronize()
    _close(tk, K, bk, "k side")
    _close(q[:5], y, b, "q side")
    with torch.cuda.stream(side):
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            q = call()
    for i in range(1, 4):
        K, bk, V, bv, y, b = fresh(i)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _close(tk, K, bk, f"k replay {i}")
        _close(tv, V, bv, f"v replay {i}")
        _close(q[:5], y, b, f"q replay {i}")


@pytest.mark.parametrize("dtype", ["float16", "float32"])
def test_outputs_on_16_byte_boundaries(dtype):
    """q_out 16 bytes past a 32-byte boundary, from both entry points: the same bits."""
    import torch
    rng = np.random.default_rng(17)
    N, Hq, H, D = 37, 6, 2, 128
    f, fh = _freqs(D)
    pos = _t(rng.integers(0, 4096, N).astype(np.int32))
    q, k, v = (_t(rng.standard_normal((N, h, D)).astype(np.float32), dtype) for h in (Hq, H, H))
    want, _ = qk.decode_attn_qk_norm_rope(q, k, pos, f)
    buf = torch.zeros(N * Hq * D + 8, device="cuda")
    out = buf[4:-4].view(N, Hq, D)
    assert out.data_ptr() % 32 == 16
    qk.decode_attn_qk_norm_rope(q, k, pos, f, q_out=out)
    assert torch.equal(out, want)
    table = torch.arange(N, dtype=torch.int32, device="cuda").repeat_interleave(1)[:, None].repeat(1, 256)
    kp, vp = (torch.zeros((N, 16, H, D), dtype=torch.float16, device="cuda") for _ in range(2))
    out.zero_()
    qk.decode_attn_append_paged_rope(k, v, pos, table, kp, vp, f, q=q, norm=True, q_out=out)
    assert torch.equal(out, want)
    assert (buf[:4] == 0).all() and (buf[-4:] == 0).all()


def test_a_named_stream_takes_no_memory_in_use():
    """What a call with a stream of its own allocates is not memory whose last
    reader, on the current stream, is still to come."""
    import torch
    N, H, D = 64, 8, 128
    f, _ = _freqs(D)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    q, side = torch.ones((N, H, D), device="cuda"), torch.cuda.Stream()
    kp, vp = (torch.zeros((N, 16, H, D), dtype=torch.float16, device="cuda") for _ in range(2))
    table = torch.arange(N, dtype=torch.int32, device="cuda")[:, None].repeat(1, 8)
    want, _ = qk.decode_attn_qk_norm_rope(q, None, pos, f)
    for call in (lambda: qk.decode_attn_qk_norm_rope(q, None, pos, f, stream=side)[0],
                 lambda: qk.decode_attn_append_paged_rope(q, q, pos, table, kp, vp, f, q=q,
                                                          norm=True, stream=side)):
        x = torch.full((N, H, D), 7.0, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)
        y = x.clone()
        del x
        out = call()
        torch.cuda.synchronize()
        assert (y == 7).all()
        assert torch.equal(out, want)


def test_weights_of_a_side_that_is_not_given_are_not_read():
    """A program that keeps both weights passes both, whichever rows a call has."""
    import torch
    rng = np.random.default_rng(21)
    N, H, D = 5, 2, 64
    f, _ = _freqs(D)
    pos = _t(rng.integers(0, 128, N).astype(np.int32))
    x = _t(rng.standard_normal((N, H, D)).astype(np.float32))
    w = _t(1 + 0.1 * rng.standard_normal(D).astype(np.float32))
    bad = torch.full((D,), float("nan"), device="cuda")
    table = torch.arange(N, dtype=torch.int32, device="cuda")[:, None].repeat(1, 8)
    pools = [[torch.zeros((N, 16, H, D), dtype=torch.float16, device="cuda") for _ in range(2)]
             for _ in range(2)]
    for (kp, vp), qw in zip(pools, (None, bad)):
        out = qk.decode_attn_append_paged_rope(x, x, pos, table, kp, vp, f, norm=True, q_weight=qw,
                                               k_weight=w)
        assert out is None
    assert torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1])
    q, none = qk.decode_attn_qk_norm_rope(x, None, pos, f, q_weight=w, k_weight=bad)
    assert none is None and torch.isfinite(q).all()
    none, k = qk.decode_attn_qk_norm_rope(None, x, pos, f, q_weight=bad, k_weight=w)
    assert none is None and torch.isfinite(k).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_next_to_quarter_turns(interleaved):
    """Sines and cosines as the rotation of (1, 0), to their own size: the smaller
    one too, of angles at and next to every quarter of a turn and of any others.

    a, the angle's distance from the nearest quarter turn, is rounded to f32
    (2^-24 |a|), and sincospif's two results are within 2^-23 of themselves."""
    import torch
    rng = np.random.default_rng(31)
    D = 256
    near = [(k << 62) + s * (1 << e) for k in range(4) for e in (8, 30, 40, 52, 60) for s in (1, -1)]
    some = [int(x) for x in rng.integers(0, 1 << 63, D // 2 - len(near) - 4) * 2]
    turns = np.array([x % (1 << 64) for x in near + some + [k << 62 for k in range(4)]], np.uint64)
    pos = np.array([1, 2, 3, -1, 5, 4097, 131071, 2 ** 31 - 1], np.int32)
    q = torch.zeros(len(pos), 1, D, device="cuda")
    lo, hi = ((slice(0, D, 2), slice(1, D, 2)) if interleaved
              else (slice(0, D // 2), slice(D // 2, D)))
    q[..., lo] = 1
    out, _ = qk.decode_attn_qk_norm_rope(q, None, _t(pos), _t(turns.view(np.int64)), norm=False,
                                         interleaved=interleaved)
    with np.errstate(over="ignore"):
        t = pos.astype(np.int64).view(np.uint64)[:, None] * turns
        quarter = (t + np.uint64(1 << 61)) >> np.uint64(62)
        a = (t - (quarter << np.uint64(62))).view(np.int64) * (2 * np.pi / 2.0 ** 64)
    quarter = quarter.astype(int)
    sin, cos, u = np.sin(a), np.cos(a), 2.0 ** -24
    bs, bc = u * (np.abs(a) + 2 * np.abs(sin)), u * (np.abs(a * sin) + 2 * cos)
    swap = quarter % 2 == 1
    c, s = np.where(swap, -sin, cos), np.where(swap, cos, sin)
    sign = np.where(quarter >= 2, -1, 1)
    got = _np(out)[:, 0]
    for what, have, want, bound in (("cos", got[:, lo], sign * c, np.where(swap, bs, bc)),
                                    ("sin", got[:, hi], sign * s, np.where(swap, bc, bs))):
        assert not (~(np.abs(have - want) <= bound)).any(), what


def test_both_layouts_take_the_same_time():
    """The same bytes of f32 rows: with an address made of
    selected terms the half layout spilled and took 41 us where 28.8 and 28.5 are usual."""
    import torch
    N, Hq, H, D = 4096, 16, 4, 256
    xs = [torch.randn((N, Hq + H, D), device="cuda") for _ in range(6)]  # 500 MB: past L2
    w, f = torch.ones(D, device="cuda"), qk.decode_attn_rope_freqs(D)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    outs = dict(q_out=torch.empty((N, Hq, D), device="cuda"),
                k_out=torch.empty((N, H, D), dtype=torch.float16, device="cuda"))
    s, graphs, times = torch.cuda.Stream(), [], ([], [])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for il in (False, True):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                for x in xs:
                    qk.decode_attn_qk_norm_rope(x[:, :Hq], x[:, Hq:], pos, f, norm=True, q_weight=w,
                                                k_weight=w, interleaved=il, **outs)
            graphs.append(g)
        for i in range(25):
            for g, t in zip(graphs, times):
                a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
                a.record()
                g.replay()
                b.record()
                b.synchronize()
                t.append(a.elapsed_time(b))
    half, interleaved = (sorted(t[5:])[10] for t in times)
    assert half <= 1.2 * interleaved, (half, interleaved)
