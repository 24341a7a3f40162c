"""The calls of the cache held in 4 bits and of the block plan, as far as they go
without a device: sizes, refusals and the format's reference."""
import ctypes

import numpy as np
import pytest
import torch

import quantized_kv_decode_paged_gb300 as qk
from q4_64 import Cache, quantised

FAKE = ctypes.c_void_p(0x10000)  # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10004)
BYTE = ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def lib():
    qk.build()
    return qk.load_library()


def _params(**kw):
    base = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16,
                max_blocks_per_seq=4, num_blocks=8, max_seq_len=64, scale=0.0, softcap=0.0,
                sliding_window=0, causal=1)
    base.update(kw)
    return qk.DaParams(**base)


def _rope(**kw):
    base = dict(type=0, rotary_dim=0, interleaved=0, norm=0, eps=1e-6, weight_offset=0.0,
                q_token_stride=1024, q_head_stride=128, k_token_stride=256, k_head_stride=128,
                v_token_stride=256, v_head_stride=128, freqs=None, q_weight=None, k_weight=None)
    base.update(kw)
    return qk.DaRopeParams(**base)


def test_page_bytes(lib):
    for bs in (8, 16, 256):
        for D, group in ((64, 32), (64, 64), (128, 32), (256, 128)):
            n = qk.decode_attn_q4_page_bytes(bs, D, group)
            assert n == 2 * bs * (D // 2 + 4 * (D // group)) == Cache(1, 1, bs, D, group).bytes().size
            assert n % 16 == 0
    for bad in ((4, 64, 32), (512, 64, 32), (24, 64, 32), (16, 96, 32), (16, 64, 128), (16, 64, 16),
                (16, 128, 48), (0, 64, 32), (16, 64, 0), (16, 64, -32)):
        with pytest.raises(qk.DecodeAttnError):
            qk.decode_attn_q4_page_bytes(*bad)


def test_reference_packs_and_unpacks():
    r = np.random.default_rng(0)
    for D, group, bs in ((64, 32, 8), (128, 64, 16), (256, 128, 32)):
        c = Cache(3, 2, bs, D, group).fill(r)
        d = Cache.of_bytes(c.bytes(), bs, D, group)
        assert np.array_equal(c.codes, d.codes) and np.array_equal(c.zero, d.zero)
        assert np.array_equal(c.scale, d.scale)
    x = np.array([0.0, 0.5, 1.5, 2.5, 15.0] + [7.0] * 27, np.float32)
    codes, scale, zero = quantised(x, 32)
    assert codes[:5].tolist() == [0, 0, 2, 2, 15] and scale[0] == 1 and zero[0] == 0


@pytest.mark.parametrize("kw,status", [
    (dict(num_q_heads=7), qk.DA_ERR_INVALID), (dict(head_dim=96), qk.DA_ERR_UNSUPPORTED),
    (dict(block_size=12), qk.DA_ERR_UNSUPPORTED), (dict(block_size=4), qk.DA_ERR_UNSUPPORTED),
    (dict(block_size=512), qk.DA_ERR_UNSUPPORTED), (dict(scale=-1.0), qk.DA_ERR_INVALID),
    (dict(scale=float("nan")), qk.DA_ERR_INVALID), (dict(softcap=-2.0), qk.DA_ERR_INVALID),
    (dict(sliding_window=-1), qk.DA_ERR_INVALID), (dict(causal=2), qk.DA_ERR_INVALID),
    (dict(num_blocks=0), qk.DA_ERR_INVALID), (dict(max_seq_len=-1), qk.DA_ERR_INVALID)])
def test_attention_rejects_bad_params(lib, kw, status):
    def call(p, group=32, T=1, ptrs=None, ws=None, n=0, stat=None):
        a = [FAKE] * 4 + [None, ctypes.c_void_p(0x90000), None] if ptrs is None else ptrs
        return lib.decode_attn_paged_q4(ctypes.byref(p), group, T, *a, ws, n, stat, None)

    assert call(_params(**kw)) == status
    good = _params()
    assert lib.decode_attn_paged_q4_workspace_size(ctypes.byref(_params(**kw)), 1) == 0
    for group in (0, -32):
        assert call(good, group) == qk.DA_ERR_INVALID
    for group in (16, 33, 256):
        assert call(good, group) == qk.DA_ERR_UNSUPPORTED
    assert call(_params(head_dim=64), 128) == qk.DA_ERR_UNSUPPORTED
    assert call(good, T=0) == qk.DA_ERR_INVALID
    assert call(good, T=2 ** 30) == qk.DA_ERR_UNSUPPORTED
    far = ctypes.c_void_p(0x90000)
    for i in (0, 1, 2, 3, 5):
        ptrs = [FAKE] * 4 + [None, far, None]
        ptrs[i] = None
        assert call(good, ptrs=ptrs) == qk.DA_ERR_INVALID
        ptrs[i] = BYTE
        assert call(good, ptrs=ptrs) == qk.DA_ERR_INVALID
    for i in (0, 1, 5):
        ptrs = [FAKE] * 4 + [None, far, None]
        ptrs[i] = ODD
        assert call(good, ptrs=ptrs) == qk.DA_ERR_INVALID
    for i in (4, 6):
        ptrs = [FAKE] * 4 + [None, far, None]
        ptrs[i] = BYTE
        assert call(good, ptrs=ptrs) == qk.DA_ERR_INVALID
    assert call(good, n=64) == qk.DA_ERR_INVALID  # bytes without a workspace
    assert call(good, ws=ODD, n=1 << 20) == qk.DA_ERR_INVALID
    assert call(good, stat=BYTE) == qk.DA_ERR_INVALID
    # an output over the queries
    ptrs = [FAKE] * 4 + [None, ctypes.c_void_p(0x10000 + 16), None]
    assert call(good, ptrs=ptrs) == qk.DA_ERR_INVALID
    assert call(_params(batch=0)) == qk.DA_OK
    assert call(good) in (qk.DA_ERR_WORKSPACE, qk.DA_ERR_CUDA)  # none given (or no device to ask)


def test_append_and_gather_reject_bad_arguments(lib):
    def append(p, r, group=32, n=2, ptrs=None):
        a = [None, FAKE, FAKE, FAKE, None, FAKE, None, FAKE, None] if ptrs is None else ptrs
        return lib.decode_attn_append_paged_q4(ctypes.byref(p), ctypes.byref(r), group, n, *a, None)

    def gather(p, group=32, n=2, kind=1, ptrs=None):
        a = [FAKE, None, FAKE, FAKE, FAKE, FAKE, None] if ptrs is None else ptrs
        return lib.decode_attn_gather_paged_q4(ctypes.byref(p), group, n, kind, *a, None)

    for call in (lambda p, *a: append(p, _rope(), *a), gather):
        for kw, status in ((dict(head_dim=96), qk.DA_ERR_UNSUPPORTED),
                           (dict(block_size=12), qk.DA_ERR_UNSUPPORTED),
                           (dict(block_size=1), qk.DA_ERR_UNSUPPORTED),
                           (dict(block_size=0), qk.DA_ERR_INVALID),
                           (dict(num_blocks=0), qk.DA_ERR_INVALID), (dict(batch=-1), qk.DA_ERR_INVALID),
                           (dict(num_blocks=2 ** 30), qk.DA_ERR_UNSUPPORTED)):
            assert call(_params(**kw)) == status, kw
        for group, status in ((0, qk.DA_ERR_INVALID), (16, qk.DA_ERR_UNSUPPORTED),
                              (256, qk.DA_ERR_UNSUPPORTED)):
            assert call(_params(), group) == status
        assert call(_params(), 32, -1) == qk.DA_ERR_INVALID
        assert call(_params(), 32, 3) == qk.DA_ERR_INVALID  # no token_seq: a token a sequence
        assert call(_params(batch=0), 32, 0) == qk.DA_OK
    p = _params()
    for r in (_rope(type=3), _rope(k_token_stride=-1), _rope(k_token_stride=255), _rope(rotary_dim=64),
              _rope(norm=2)):
        assert append(p, r) == qk.DA_ERR_INVALID
    for i in (1, 2, 3, 5, 7):
        ptrs = [None, FAKE, FAKE, FAKE, None, FAKE, None, FAKE, None]
        ptrs[i] = None
        assert append(p, _rope(), ptrs=ptrs) == qk.DA_ERR_INVALID
        ptrs[i] = BYTE
        assert append(p, _rope(), ptrs=ptrs) == qk.DA_ERR_INVALID
    ptrs = [FAKE, FAKE, FAKE, FAKE, None, FAKE, None, FAKE, None]  # queries without a place
    assert append(p, _rope(), ptrs=ptrs) == qk.DA_ERR_INVALID
    for i in (0, 2, 3, 4, 5):
        ptrs = [FAKE, None, FAKE, FAKE, FAKE, FAKE, None]
        ptrs[i] = None
        assert gather(p, ptrs=ptrs) == qk.DA_ERR_INVALID
        ptrs[i] = BYTE
        assert gather(p, ptrs=ptrs) == qk.DA_ERR_INVALID
    assert gather(p, kind=3) == qk.DA_ERR_INVALID
    assert gather(_params(num_kv_heads=5000, num_q_heads=5000)) == qk.DA_ERR_UNSUPPORTED


def test_plan_rejects_bad_arguments(lib):
    good = dict(B=4, bs=16, mb=8, NB=64, N=10, cap=64)

    def call(ptrs=None, **kw):
        a = {**good, **kw}
        p = [FAKE] * 9 + [None] if ptrs is None else ptrs
        return lib.decode_attn_plan_blocks(a["B"], a["bs"], a["mb"], a["NB"], a["N"], a["cap"], *p,
                                           None)

    for kw, status in ((dict(B=-1), qk.DA_ERR_INVALID), (dict(bs=0), qk.DA_ERR_INVALID),
                       (dict(mb=0), qk.DA_ERR_INVALID), (dict(NB=0), qk.DA_ERR_INVALID),
                       (dict(N=-1), qk.DA_ERR_INVALID), (dict(cap=-1), qk.DA_ERR_INVALID),
                       (dict(bs=24), qk.DA_ERR_UNSUPPORTED), (dict(bs=4), qk.DA_ERR_UNSUPPORTED),
                       (dict(bs=512), qk.DA_ERR_UNSUPPORTED), (dict(B=16385), qk.DA_ERR_UNSUPPORTED),
                       (dict(NB=2 ** 28), qk.DA_ERR_UNSUPPORTED),
                       (dict(mb=2 ** 28), qk.DA_ERR_UNSUPPORTED),
                       (dict(N=2 ** 31 - 1), qk.DA_ERR_UNSUPPORTED),
                       (dict(cap=2 ** 31 - 1), qk.DA_ERR_UNSUPPORTED)):
        assert call(**kw) == status, kw
    for i in range(9):
        ptrs = [FAKE] * 9 + [None]
        ptrs[i] = None
        assert call(ptrs) == qk.DA_ERR_INVALID, i
        ptrs[i] = BYTE
        assert call(ptrs) == qk.DA_ERR_INVALID, i
    ptrs = [FAKE] * 9 + [None]
    ptrs[7] = ODD  # slots have 64 bits
    assert call(ptrs) == qk.DA_ERR_INVALID
    assert call(B=0, N=0) == qk.DA_OK


def _cpu_attend(**kw):
    a = dict(q=torch.zeros(2, 8, 64), pool=torch.zeros(5, 2, 16 * 80, dtype=torch.uint8),
             block_table=torch.zeros(2, 4, dtype=torch.int32),
             seq_lens=torch.zeros(2, dtype=torch.int32), group=32)
    a.update(kw)
    return qk.decode_attn_paged_q4(**a)


def test_binding_refuses_before_the_device(lib):
    i32 = torch.int32
    for bad, exc in ((dict(q=torch.zeros(2, 8, 64).half()), TypeError), (dict(q=torch.zeros(8, 64)), ValueError),
                     (dict(q=torch.zeros(2, 8, 128)), ValueError), (dict(group=48), qk.DecodeAttnError),
                     (dict(group=0), qk.DecodeAttnError), (dict(group=128), qk.DecodeAttnError),
                     (dict(pool=torch.zeros(5, 2, 1281, dtype=torch.uint8)), ValueError),
                     (dict(pool=torch.zeros(5, 2, 1280)), TypeError), (dict(pool=torch.zeros(5, 1280, dtype=torch.uint8)), ValueError),
                     (dict(seq_lens=torch.zeros(3, dtype=i32)), ValueError),
                     (dict(seq_lens=torch.zeros(2).long()), TypeError),
                     (dict(block_table=torch.zeros(3, 4, dtype=i32)), ValueError),
                     (dict(q_pos=torch.zeros(3, dtype=i32)), ValueError),
                     (dict(out=torch.zeros(2, 8, 128)), ValueError), (dict(lse=torch.zeros(2, 4)), ValueError),
                     (dict(workspace=3), ValueError), (dict(workspace=None), ValueError), ({}, ValueError)):
        with pytest.raises(exc):
            _cpu_attend(**bad)
    for name in ("pool", "block_table", "seq_lens", "q_pos", "out", "lse", "dev_status"):
        with pytest.raises(TypeError, match=name):
            _cpu_attend(**{name: [0, 1]})
    k, pos = torch.zeros(3, 2, 64), torch.zeros(3, dtype=i32)
    pool, table = torch.zeros(5, 2, 16 * 80, dtype=torch.uint8), torch.zeros(3, 4, dtype=i32)
    base = dict(k_new=k, v_new=k, positions=pos, block_table=table, pool=pool, group=32)
    for bad, exc in ((dict(v_new=k[:2]), ValueError), (dict(v_new=k.half()), TypeError),
                     (dict(pool=pool[:, :1].contiguous()), ValueError), (dict(token_seq=pos[:2]), ValueError),
                     (dict(q=k[:2]), ValueError), (dict(q_out=k), ValueError), (dict(group=128), qk.DecodeAttnError),
                     (dict(freqs=torch.zeros(32, dtype=i32)), TypeError),
                     (dict(k_weight=torch.ones(64)), ValueError), ({}, ValueError)):
        with pytest.raises(exc):
            qk.decode_attn_append_paged_q4(**{**base, **bad})
    for name in ("v_new", "positions", "block_table", "pool", "freqs", "token_seq", "dev_status"):
        with pytest.raises(TypeError, match=name):
            qk.decode_attn_append_paged_q4(**{**base, name: [0, 1, 2]})
    base = dict(positions=pos, block_table=table, pool=pool, head_dim=64, group=32)
    for bad, exc in ((dict(head_dim=128), ValueError), (dict(token_seq=pos[:2]), ValueError),
                     (dict(dtype=torch.float64), TypeError), (dict(k_out=torch.zeros(3, 2, 32).half()), ValueError),
                     (dict(k_out=k.half(), v_out=k), TypeError), ({}, ValueError)):
        with pytest.raises(exc):
            qk.decode_attn_gather_paged_q4(**{**base, **bad})
    for name in ("positions", "block_table", "pool", "token_seq", "k_out", "v_out", "dev_status"):
        with pytest.raises(TypeError, match=name):
            qk.decode_attn_gather_paged_q4(**{**base, name: [0, 1, 2]})
    lens = torch.zeros(3, dtype=i32)
    base = dict(old_lens=lens, new_lens=lens, block_table=table, free_list=torch.zeros(9, dtype=i32),
                free_count=torch.zeros(1, dtype=i32), block_size=16, num_blocks=9, max_tokens=4)
    for bad, exc in ((dict(new_lens=lens[:2]), ValueError), (dict(old_lens=lens.long()), TypeError),
                     (dict(block_table=table[:2]), ValueError), (dict(free_count=lens), ValueError),
                     (dict(max_tokens=-1), ValueError), (dict(slots=lens), TypeError),
                     (dict(positions=lens), ValueError), (dict(cu_tokens=lens), ValueError), ({}, ValueError)):
        with pytest.raises(exc):
            qk.decode_attn_plan_blocks(**{**base, **bad})
    for name in ("old_lens", "new_lens", "block_table", "free_list", "free_count", "positions", "token_seq",
                 "slots", "cu_tokens", "dev_status"):
        with pytest.raises(TypeError, match=name):
            qk.decode_attn_plan_blocks(**{**base, name: [0, 1, 2]})
