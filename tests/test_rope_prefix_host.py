"""Host-side checks, no GPU: the rotation frequencies, and the refusals of
the norm / rotation / append and shared-prefix calls before any launch."""
import ctypes
import math

import numpy as np
import pytest
import torch

import quantized_kv_decode_paged_gb300 as qk

FAKE = ctypes.c_void_p(0x10000)  # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    qk.build()
    return qk.load_library()


# ------------------------------------------------------------------ frequencies
@pytest.mark.parametrize("rd,theta", [(64, 10000.0), (128, 500000.0), (16, 1.0), (256, 1e6)])
def test_rope_freqs_are_turns_in_64_bit_fixed_point(lib, rd, theta):
    got = qk.decode_attn_rope_freqs(rd, theta, device="cpu").numpy().view(np.uint64)
    want = theta ** (-2.0 * np.arange(rd // 2) / rd) / (2 * math.pi)
    # pow, the quotient and the table's rounding: a few 2^-53 of the value
    err = np.abs(got.astype(np.float64) / 2.0 ** 64 - want)
    assert (err <= 8 * 2.0 ** -53 * want + 2.0 ** -65).all()


def test_rope_freqs_take_given_frequencies_modulo_a_turn(lib):
    w = [0.5, 2 * math.pi + 0.25, -0.25, 0.0]
    got = qk.decode_attn_rope_freqs(8, inv_freq=w, device="cpu").numpy().view(np.uint64)
    want = np.mod(np.array(w) / (2 * math.pi), 1.0)
    # the whole turn taken off leaves an error of the quotient before it: 2^-53 of 1.04
    assert (np.abs(got.astype(np.float64) / 2.0 ** 64 - want) <= 2.0 ** -51).all()
    assert qk.decode_attn_rope_freqs(0, device="cpu").numel() == 0


def test_rope_freqs_refusals(lib):
    for bad in (dict(rotary_dim=7), dict(rotary_dim=-2), dict(rotary_dim=8, theta=0.0),
                dict(rotary_dim=8, theta=-1.0), dict(rotary_dim=8, theta=math.inf),
                dict(rotary_dim=8, theta=math.nan),
                dict(rotary_dim=8, inv_freq=[1, 2, 3, math.inf])):
        with pytest.raises((qk.DecodeAttnError, ValueError, RuntimeError)):
            qk.decode_attn_rope_freqs(device="cpu", **bad)
    with pytest.raises(ValueError):
        qk.decode_attn_rope_freqs(8, inv_freq=[1.0, 2.0], device="cpu")


# ------------------------------------------------------------------ the C entries
def _rope(**kw):
    base = dict(type=1, rotary_dim=64, interleaved=0, norm=1, eps=1e-6, weight_offset=0.0,
                q_token_stride=512, q_head_stride=64, k_token_stride=128, k_head_stride=64,
                v_token_stride=128, v_head_stride=64, freqs=0x10000, q_weight=None, k_weight=None)
    base.update(kw)
    return qk.DaRopeParams(**base)


BAD_ROPE = [
    (dict(type=3), qk.DA_ERR_INVALID), (dict(type=-1), qk.DA_ERR_INVALID),
    (dict(rotary_dim=-16), qk.DA_ERR_INVALID), (dict(rotary_dim=80), qk.DA_ERR_INVALID),
    (dict(rotary_dim=7), qk.DA_ERR_INVALID), (dict(rotary_dim=24), qk.DA_ERR_UNSUPPORTED),
    (dict(interleaved=2), qk.DA_ERR_INVALID), (dict(norm=-1), qk.DA_ERR_INVALID),
    (dict(eps=-1.0), qk.DA_ERR_INVALID), (dict(eps=math.nan), qk.DA_ERR_INVALID),
    (dict(eps=math.inf), qk.DA_ERR_INVALID), (dict(weight_offset=math.inf), qk.DA_ERR_INVALID),
    (dict(freqs=None), qk.DA_ERR_INVALID), (dict(freqs=0x10004), qk.DA_ERR_INVALID),
    (dict(k_weight=0x10004), qk.DA_ERR_INVALID),
    (dict(k_token_stride=-64), qk.DA_ERR_INVALID), (dict(k_head_stride=3), qk.DA_ERR_INVALID),
    (dict(k_token_stride=4), qk.DA_ERR_INVALID), (dict(k_token_stride=1 << 41), qk.DA_ERR_INVALID),
]


@pytest.mark.parametrize("kw,status", BAD_ROPE)
def test_rope_entries_reject_bad_params(lib, kw, status):
    r = _rope(**kw)
    st = lib.decode_attn_qk_norm_rope(ctypes.byref(r), 4, 8, 2, 64, FAKE, FAKE, FAKE, FAKE, FAKE,
                                      None)
    assert st == status
    p = qk.DaParams(4, 8, 2, 64, 16, 4, 16, 0, 0.0, 0.0, 0, 1)
    st = lib.decode_attn_append_paged_rope(ctypes.byref(p), ctypes.byref(r), 4, FAKE, FAKE, FAKE,
                                           FAKE, None, FAKE, FAKE, FAKE, FAKE, None, None)
    assert st == status


def test_norm_rope_rejects_bad_arguments(lib):
    good = dict(n=4, hq=8, hkv=2, d=64, q=FAKE, k=FAKE, pos=FAKE, qo=FAKE, ko=FAKE)

    def call(**kw):
        a = {**good, **kw}
        return lib.decode_attn_qk_norm_rope(ctypes.byref(_rope()), a["n"], a["hq"], a["hkv"],
                                            a["d"], a["q"], a["k"], a["pos"], a["qo"], a["ko"],
                                            None)

    for bad in (dict(n=-1), dict(hq=0), dict(hkv=-1), dict(d=0), dict(q=None, k=None),
                dict(qo=None), dict(ko=None), dict(q=ODD), dict(k=ODD), dict(qo=ODD),
                dict(ko=ODD), dict(pos=None), dict(pos=ctypes.c_void_p(0x10002))):
        assert call(**bad) == qk.DA_ERR_INVALID, bad
    assert call(d=96) == qk.DA_ERR_UNSUPPORTED
    assert call(hq=4095) == qk.DA_ERR_UNSUPPORTED
    assert call(n=0) == qk.DA_OK
    assert lib.decode_attn_qk_norm_rope(None, 4, 8, 2, 64, FAKE, FAKE, FAKE, FAKE, FAKE,
                                        None) == qk.DA_ERR_INVALID


def test_append_rope_rejects_bad_arguments(lib):
    base = dict(batch=4, num_q_heads=8, num_kv_heads=2, head_dim=64, block_size=16,
                max_blocks_per_seq=4, num_blocks=16, max_seq_len=0, scale=0.0, softcap=0.0,
                sliding_window=0, causal=1)
    good = dict(n=4, q=FAKE, k=FAKE, v=FAKE, pos=FAKE, seq=FAKE, table=FAKE, qo=FAKE, kp=FAKE,
                vp=FAKE, st=None)

    def call(params=None, **kw):
        a = {**good, **kw}
        p = qk.DaParams(**{**base, **(params or {})})
        return lib.decode_attn_append_paged_rope(
            ctypes.byref(p), ctypes.byref(_rope()), a["n"], a["q"], a["k"], a["v"], a["pos"],
            a["seq"], a["table"], a["qo"], a["kp"], a["vp"], a["st"], None)

    two = ctypes.c_void_p(0x10002)
    for bad in (dict(n=-1), dict(n=5, seq=None), dict(k=None), dict(v=None), dict(pos=None),
                dict(table=None), dict(kp=None), dict(vp=None), dict(qo=None), dict(q=None),
                dict(k=ODD), dict(v=ODD), dict(q=ODD), dict(kp=ODD), dict(vp=ODD), dict(qo=ODD),
                dict(pos=two), dict(seq=two), dict(table=two), dict(st=two)):
        assert call(**bad) == qk.DA_ERR_INVALID, bad
    for bad in (dict(batch=-1), dict(num_kv_heads=0), dict(num_q_heads=0), dict(block_size=0),
                dict(max_blocks_per_seq=0), dict(num_blocks=0)):
        assert call(bad) == qk.DA_ERR_INVALID, bad
    assert call(dict(head_dim=96)) == qk.DA_ERR_UNSUPPORTED
    assert call(dict(num_blocks=1 << 28)) == qk.DA_ERR_UNSUPPORTED
    assert call(n=0) == qk.DA_OK


def test_prefix_rejects_bad_arguments(lib):
    base = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16,
                max_blocks_per_seq=4, num_blocks=8, max_seq_len=64, scale=0.0, softcap=0.0,
                sliding_window=0, causal=1)
    good = dict(t=1, plen=32, pt=FAKE, q=FAKE, kp=FAKE, vp=FAKE, table=FAKE, lens=FAKE, qpos=None,
                out=FAKE, lse=None, ws=FAKE, nb=1 << 40, st=None)

    def call(params=None, **kw):
        a = {**good, **kw}
        p = qk.DaParams(**{**base, **(params or {})})
        return lib.decode_attn_paged_prefix(
            ctypes.byref(p), a["t"], a["plen"], a["pt"], a["q"], a["kp"], a["vp"], a["table"],
            a["lens"], a["qpos"], a["out"], a["lse"], a["ws"], a["nb"], a["st"], None)

    two = ctypes.c_void_p(0x10002)
    for bad in (dict(t=0), dict(plen=-1), dict(plen=65), dict(pt=None), dict(q=None),
                dict(kp=None), dict(vp=None), dict(table=None), dict(lens=None), dict(out=None),
                dict(ws=None), dict(ws=ctypes.c_void_p(0x10010)), dict(q=ODD), dict(kp=ODD),
                dict(vp=ODD), dict(out=ODD), dict(pt=two), dict(table=two), dict(lens=two),
                dict(qpos=two), dict(lse=two), dict(st=two)):
        assert call(**bad) == qk.DA_ERR_INVALID, bad
    for bad in (dict(num_q_heads=7), dict(scale=-1.0), dict(scale=math.nan), dict(softcap=-2.0),
                dict(sliding_window=-1), dict(causal=2), dict(num_blocks=0), dict(batch=-1),
                dict(max_seq_len=-1)):
        assert call(bad) == qk.DA_ERR_INVALID, bad
    for bad in (dict(head_dim=96), dict(block_size=12), dict(block_size=512)):
        assert call(bad) == qk.DA_ERR_UNSUPPORTED, bad
    assert call(t=1 << 24) == qk.DA_ERR_UNSUPPORTED
    assert call(dict(batch=0)) == qk.DA_OK
    p = qk.DaParams(**{**base, "head_dim": 96})
    assert qk.decode_attn_paged_prefix_workspace_size(p, 1, 0) == 0
    assert qk.decode_attn_paged_prefix_workspace_size(qk.DaParams(**base), 0, 0) == 0
    assert qk.decode_attn_paged_prefix_workspace_size(qk.DaParams(**base), 1, 65) == 0


def test_prefix_refuses_an_output_over_its_queries(lib):
    p = qk.DaParams(2, 8, 2, 128, 16, 4, 8, 64, 0.0, 0.0, 0, 1)
    n = 2 * 3 * 8 * 128 * 4  # bytes of q and of out, three tokens a sequence

    def call(q, out):
        return lib.decode_attn_paged_prefix(ctypes.byref(p), 3, 32, FAKE, q, FAKE, FAKE, FAKE, FAKE,
                                            None, out, None, FAKE, 0, None, None)

    at = FAKE.value
    for d in (0, 16, n - 16):
        for a, b in ((at, at + d), (at + d, at)):
            assert call(ctypes.c_void_p(a), ctypes.c_void_p(b)) == qk.DA_ERR_INVALID
    for a, b in ((at, at + n), (at + n, at)):  # side by side: not for this reason
        assert call(ctypes.c_void_p(a), ctypes.c_void_p(b)) != qk.DA_ERR_INVALID


# ------------------------------------------------------------------ the binding
def _cpu_prefix(**kw):
    a = dict(q=torch.zeros(2, 8, 64), k_pool=torch.zeros(8, 16, 2, 64, dtype=torch.float16),
             v_pool=torch.zeros(8, 16, 2, 64, dtype=torch.float16),
             block_table=torch.zeros(2, 4, dtype=torch.int32),
             seq_lens=torch.zeros(2, dtype=torch.int32), prefix_len=32)
    a.update(kw)
    return qk.decode_attn_paged_prefix(**a)


def test_binding_refuses_before_the_device(lib):
    """Types, shapes and CPU tensors raise in the binding; no CUDA call is made
    (this runs without a device)."""
    for bad, exc in ((dict(q=torch.zeros(2, 8, 64, dtype=torch.float16)), TypeError),
                     (dict(q=torch.zeros(8, 64)), ValueError),
                     (dict(q=torch.zeros(2, 8, 128)), ValueError),
                     (dict(seq_lens=torch.zeros(3, dtype=torch.int32)), ValueError),
                     (dict(seq_lens=torch.zeros(2, dtype=torch.int64)), TypeError),
                     (dict(block_table=torch.zeros(3, 4, dtype=torch.int32)), ValueError),
                     (dict(prefix_table=torch.zeros(1, dtype=torch.int32)), ValueError),
                     (dict(q_pos=torch.zeros(3, dtype=torch.int32)), ValueError),
                     (dict(out=torch.zeros(2, 8, 128)), ValueError),
                     (dict(lse=torch.zeros(2, 4)), ValueError),
                     (dict(workspace=None), ValueError), ({}, ValueError)):
        with pytest.raises(exc):
            _cpu_prefix(**bad)
    q, k = torch.zeros(3, 8, 64), torch.zeros(3, 2, 64)
    pos = torch.zeros(3, dtype=torch.int32)
    f = qk.decode_attn_rope_freqs(64, device="cpu")
    for args, kw, exc in (((None, None, pos, f), {}, ValueError),
                          ((q.double(), k, pos, f), {}, TypeError),
                          ((q, k.half(), pos, f), {}, TypeError),
                          ((q, k[:2], pos, f), {}, ValueError),
                          ((q, k, pos.long(), f), {}, TypeError),
                          ((q, k, pos[:2], f), {}, ValueError),
                          ((q, k, None, f), {}, ValueError),
                          ((q, k, pos, f.int()), {}, TypeError),
                          ((q.transpose(1, 2), k, pos, f), {}, ValueError),
                          ((q, k, pos, f), dict(q_weight=torch.ones(32)), ValueError),
                          ((q, k, pos, f), dict(norm=False, q_weight=torch.ones(64)), ValueError),
                          ((q, k, pos, f), dict(q_out=torch.zeros(3, 8, 32)), ValueError),
                          ((q, k, pos, f), {}, ValueError)):
        with pytest.raises(exc):
            qk.decode_attn_qk_norm_rope(*args, **kw)
    pool = torch.zeros(8, 16, 2, 64, dtype=torch.float16)
    table = torch.zeros(3, 4, dtype=torch.int32)
    for args, kw, exc in (((k, k[:2], pos, table, pool, pool, f), {}, ValueError),
                          ((k, k.half(), pos, table, pool, pool, f), {}, TypeError),
                          ((k, k, pos, table, pool.float(), pool, f), {}, TypeError),
                          ((k, k, pos, table, pool, pool[:4], f), {}, ValueError),
                          ((k, k, pos, table, pool, pool, f), dict(token_seq=pos[:2]), ValueError),
                          ((k, k, pos, table, pool, pool, f), dict(q=q[:2]), ValueError),
                          ((k, k, pos, table, pool, pool, f), dict(q_out=q), ValueError),
                          ((k, k, pos, table, pool, pool, f), {}, ValueError)):
        with pytest.raises(exc):
            qk.decode_attn_append_paged_rope(*args, **kw)


# ------------------------------------------------------------------ the binding, up to the library
class _Entry:
    """Stands for an entry point of the library: keeps the calls' arguments."""

    def __init__(self, then=lambda: None):
        self.calls, self.then = [], then

    def __call__(self, *args):
        self.calls.append(args)
        self.then()
        return qk.DA_OK


@pytest.fixture
def on_host(lib, monkeypatch):
    """The calls' Python path on CPU tensors, as far as a stand-in for the library."""
    class Library:
        decode_attn_paged_prefix = _Entry()

        @staticmethod
        def decode_attn_paged_prefix_workspace_size(*args):
            return 4096

        decode_attn_status_string = lib.decode_attn_status_string

    qk._load_call()  # leaves CPU tensors to Python
    monkeypatch.setattr(qk, "_lib", Library)
    monkeypatch.setattr(qk, "_check_cuda", lambda name, t: None)
    monkeypatch.setattr(qk, "_call_guard", lambda *args: qk._NO_GUARD)
    monkeypatch.setattr(qk, "_raw_stream", lambda *args: 0)
    monkeypatch.setattr(qk, "_prefix_ws_bytes", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return Library


def test_calls_at_once_have_workspaces_of_their_own(on_host):
    """Two threads inside the entry point at the same time, on one stream."""
    import threading
    both = threading.Barrier(2)
    on_host.decode_attn_paged_prefix = entry = _Entry(lambda: both.wait(30))
    threads = [threading.Thread(target=_cpu_prefix) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    a, b = [c[12] for c in entry.calls]
    assert abs(a - b) >= 4096 and [c[13] for c in entry.calls] == [4096, 4096]


def test_binding_names_arguments_that_are_no_tensors(lib):
    q, k = torch.zeros(3, 8, 64), torch.zeros(3, 2, 64)
    pos, f = torch.zeros(3, dtype=torch.int32), qk.decode_attn_rope_freqs(64, device="cpu")
    pool, table = torch.zeros(8, 16, 2, 64, dtype=torch.float16), torch.zeros(3, 4, dtype=torch.int32)
    for name in ("positions", "freqs", "q_weight", "k_weight", "q_out"):
        args = dict(q=q, k=k, positions=pos, freqs=f)
        args[name] = [0, 1, 2]
        with pytest.raises(TypeError, match=name):
            qk.decode_attn_qk_norm_rope(**args)
    for name in ("v_new", "positions", "block_table", "k_pool", "v_pool", "freqs", "token_seq",
                 "dev_status"):
        args = dict(k_new=k, v_new=k, positions=pos, block_table=table, k_pool=pool, v_pool=pool,
                    freqs=f)
        args[name] = [0, 1, 2]
        with pytest.raises(TypeError, match=name):
            qk.decode_attn_append_paged_rope(**args)
    for name in ("k_pool", "v_pool", "block_table", "seq_lens", "prefix_table", "q_pos", "out"):
        with pytest.raises(TypeError, match=name):
            _cpu_prefix(**{name: [0, 1]})


def test_pools_without_rows_are_refused(on_host):
    on_host.decode_attn_paged_prefix = lambda *args: qk.DA_ERR_INVALID
    pool = torch.zeros(8, 0, 2, 64, dtype=torch.float16)
    with pytest.raises(qk.DecodeAttnError):
        _cpu_prefix(k_pool=pool, v_pool=pool)


def test_rope_freqs_refuse_a_power_that_overflows(lib):
    with pytest.raises(qk.DecodeAttnError):
        qk.decode_attn_rope_freqs(128, 5e-324, device="cpu")
    assert qk.decode_attn_rope_freqs(128, 1e-300, device="cpu").numel() == 64


def test_a_stream_of_another_device_is_refused():
    """Its kernels would get pointers of a device that is not theirs."""
    class Stream:
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError, match="cuda:1"):
        qk._call_guard(torch, torch.device("cuda", 0), Stream())
