"""The C++ marshalling of the norm, append and shared-prefix calls: what it takes,
what it leaves to the checks in Python, and that both give the same."""
import pytest
import torch

import quantized_kv_decode_paged_gb300 as qk


@pytest.fixture(scope="module")
def call():
    qk.build()
    return qk._load_call()


def _rope_args(q, k, pos, f, **kw):
    a = dict(norm=True, q_weight=None, k_weight=None, weight_offset=0.0, eps=1e-6,
             interleaved=False, q_out=None, k_out=None)
    a.update(kw)
    return (q, k, pos, f, a["norm"], a["q_weight"], a["k_weight"], a["weight_offset"], a["eps"],
            a["interleaved"], a["q_out"], a["k_out"])


def test_leaves_what_is_not_on_a_device_to_the_checks(call):
    x, pos = torch.zeros(2, 4, 64), torch.zeros(2, dtype=torch.int32)
    f = qk.decode_attn_rope_freqs(64, device="cpu")
    for args in ((x, x, pos, f), (None, None, pos, f), ("x", x, pos, f), (x, None, None, None)):
        assert call.norm_rope(*_rope_args(*args)) is NotImplemented
    pool, table = torch.zeros(4, 16, 4, 64, dtype=torch.float16), torch.zeros(2, 2, dtype=torch.int32)
    assert call.append(x, x, pos, table, pool, pool, f, None, None, False, None, None, 0.0, 1e-6,
                       False, None, None) is NotImplemented
    assert call.prefix(x, pool, pool, table, pos, 0, None, None, 0.0, 0.0, 0, True, 0, None, None,
                       None) is NotImplemented


def test_wrong_numbers_of_arguments_and_null_addresses_raise(call):
    for fn in (call.norm_rope, call.append, call.prefix, call.bind):
        with pytest.raises(TypeError):
            fn(None)
    with pytest.raises(ValueError):
        call.bind(0, 0, 0, 0)
    with pytest.raises(TypeError):
        call.bind("a", 1, 1, 1)


# ------------------------------------------------------------------ on a device
def _cuda(*shape, dtype=torch.float32):
    g = torch.Generator(device="cuda")
    g.manual_seed(sum(shape))
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.gpu
def test_takes_the_common_calls_with_the_same_results(cuda_lib, call):
    """A named stream goes through Python: the same bits."""
    N, Hq, H, D = 7, 6, 2, 128
    qkv = _cuda(N, Hq + 2 * H, D, dtype=torch.bfloat16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    pos = torch.arange(N, dtype=torch.int32, device="cuda") * 5
    f = qk.decode_attn_rope_freqs(D)
    w = torch.nn.Parameter(1 + 0.1 * _cuda(D))  # as a module holds it
    here = torch.cuda.current_stream()
    kw = dict(q_weight=w, k_weight=w, weight_offset=1.0, interleaved=True)
    got = call.norm_rope(*_rope_args(q, k, pos, f, **kw))
    assert type(got) is tuple and not got[0].requires_grad
    want = qk.decode_attn_qk_norm_rope(q, k, pos, f, stream=here, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = torch.zeros(N, Hq, D, device="cuda")
    got = call.norm_rope(*_rope_args(q, None, pos, f, q_out=out, **kw))
    assert got[0] is out and got[1] is None and torch.equal(out, want[0])
    got = call.norm_rope(*_rope_args(None, k, None, None, norm=False))
    assert got[0] is None and torch.equal(got[1], k.half())

    table = torch.arange(N, dtype=torch.int32, device="cuda")[:, None].repeat(1, 4)
    pools = [[torch.zeros(N, 16, H, D, dtype=torch.float16, device="cuda") for _ in range(2)]
             for _ in range(2)]
    seq = torch.arange(N, dtype=torch.int32, device="cuda")
    a = call.append(k, v, pos, table, *pools[0], f, seq, q, True, w, w, 1.0, 1e-6, True, None, None)
    b = qk.decode_attn_append_paged_rope(k, v, pos, table, *pools[1], f, token_seq=seq, q=q,
                                         norm=True, stream=here, **kw)
    assert torch.equal(a, b) and all(torch.equal(x, y) for x, y in zip(*pools))
    assert call.append(k, v, pos, table, *pools[0], f, seq, None, False, None, None, 0.0, 1e-6, True,
                       None, None) is None

    lens = pos + 1
    for T in (1, 3):
        qq = _cuda(*((N, Hq, D) if T == 1 else (N, T, Hq, D)))
        a = call.prefix(qq, *pools[0], table, lens, 16, None, None, 0.0, 30.0, 9, True, 64, None, None,
                        None)
        b = qk.decode_attn_paged_prefix(qq, *pools[0], table, lens, 16, softcap=30.0,
                                        sliding_window=9, max_seq_len=64, stream=here)
        assert type(a) is tuple and all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
def test_leaves_unusual_calls_to_python(cuda_lib, call):
    N, H, D = 4, 2, 64
    x, f = _cuda(N, H, D), qk.decode_attn_rope_freqs(D)
    pos = torch.zeros(N, dtype=torch.int32, device="cuda")
    ok = _rope_args(x, x, pos, f)
    assert type(call.norm_rope(*ok)) is tuple
    for bad in ((x.double(), x, pos, f), (x, x.half(), pos, f), (x, x[:2], pos, f),
                (x, x, pos.long(), f), (x, x, pos[:2], f), (x, x, None, f), (x, x, pos, f.int()),
                (x.transpose(1, 2), x, pos, f), (x[:0], x[:0], pos[:0], f), (x, x, pos, f.cpu())):
        assert call.norm_rope(*_rope_args(*bad)) is NotImplemented
    for kw in (dict(norm=1), dict(eps="a"), dict(q_weight=x), dict(norm=False, q_weight=x[0, 0]),
               dict(q_out=x[:, :1]), dict(q_out=x.half())):
        assert call.norm_rope(*_rope_args(x, x, pos, f, **kw)) is NotImplemented
    # an error of the entry point: its status
    assert call.norm_rope(*_rope_args(x, x, pos, f, eps=-1.0)) == qk.DA_ERR_INVALID
    with pytest.raises(qk.DecodeAttnError):
        qk.decode_attn_qk_norm_rope(x, x, pos, f, eps=-1.0)
    # a captured shared-prefix call has a workspace of its graph's
    pool = _cuda(N, 16, H, D, dtype=torch.float16)
    table = torch.arange(N, dtype=torch.int32, device="cuda")[:, None].repeat(1, 2)
    lens = torch.full((N,), 20, dtype=torch.int32, device="cuda")
    args = (x, pool, pool, table, lens, 0, None, None, 0.0, 0.0, 0, True, 0, None, None, None)
    assert type(call.prefix(*args)) is tuple
    torch.cuda.synchronize()
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        assert call.prefix(*args) is NotImplemented
        assert type(call.norm_rope(*ok)) is tuple
    torch.cuda.synchronize()
