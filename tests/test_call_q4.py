"""The C++ marshalling of the 4-bit cache's calls and of the block plan: what it
takes, what it leaves to the checks in Python, and that both give the same."""
import pytest
import torch

import quantized_kv_decode_paged_gb300 as qk

N, HQ, H, D, GROUP, BS = 7, 6, 2, 128, 64, 16


@pytest.fixture(scope="module")
def call():
    qk.build()
    return qk._load_call()


def _tensors(device):
    g = torch.Generator(device="cpu")
    g.manual_seed(3)
    qkv = torch.randn((N, HQ + 2 * H, D), generator=g).to(torch.bfloat16).to(device)
    i32 = dict(dtype=torch.int32, device=device)
    return dict(q=qkv[:, :HQ], k=qkv[:, HQ:HQ + H], v=qkv[:, HQ + H:],
                pos=torch.arange(N, **i32) * 5, seq=torch.arange(N, **i32),
                table=torch.arange(N * 4, **i32).view(N, 4),
                pool=torch.zeros((N * 4, H, BS * (D + 8 * D // GROUP)), dtype=torch.uint8,
                                 device=device))


def _append(t, f=None, **kw):
    a = {**t, "group": GROUP, "norm": False, "w": None, "eps": 1e-6, "q_out": None, "status": None, **kw}
    return (a["k"], a["v"], a["pos"], a["table"], a["pool"], f, a["group"], a["seq"], a["q"], a["norm"],
            a["w"], a["w"], 0.0, a["eps"], False, a["q_out"], a["status"])


def _gather(t, **kw):
    a = {**t, "d": D, "group": GROUP, "status": None, **kw}
    return (a["pos"], a["table"], a["pool"], a["d"], a["group"], a["seq"], a["status"])


def _attend(t, q, lens, **kw):
    a = {**t, "q_pos": None, "group": GROUP, "scale": 0.0, "out": None, "lse": None, "status": None, **kw}
    return (q, a["pool"], a["table"], lens, a["q_pos"], a["group"], a["scale"], 0.0, 0, True, 0,
            a["out"], a["lse"], a["status"])


def _plan(t, old, new, n=40, **kw):
    a = {"free": t["seq"] + 4 * N - N, "count": t["seq"][N - 1:], "bs": BS, "status": None, **kw}
    return (old, new, t["table"], a["free"], a["count"], a["bs"], 4 * N, n, a["status"])


def test_leaves_what_is_not_on_a_device_to_the_checks(call):
    t = _tensors("cpu")
    q = torch.zeros(N, HQ, D)
    for fn, args in ((call.append_q4, _append(t)), (call.gather_q4, _gather(t)),
                     (call.attend_q4, _attend(t, q, t["pos"])),
                     (call.plan, _plan(t, t["pos"], t["pos"]))):
        assert fn(*args) is NotImplemented
        assert fn(*(None for _ in args)) is NotImplemented
        assert fn(*("x" for _ in args)) is NotImplemented


def test_wrong_numbers_of_arguments_and_null_addresses_raise(call):
    for fn in (call.append_q4, call.gather_q4, call.attend_q4, call.plan, call.bind_q4):
        with pytest.raises(TypeError):
            fn(None)
    with pytest.raises(ValueError):
        call.bind_q4(0, 0, 0, 0, 0)
    with pytest.raises(TypeError):
        call.bind_q4("a", 1, 1, 1, 1)


# ------------------------------------------------------------------ on a device
@pytest.mark.gpu
def test_takes_the_common_calls_with_the_same_results(cuda_lib, call):
    """A named stream goes through Python: the same bits."""
    t, here = _tensors("cuda"), torch.cuda.current_stream()
    f = qk.decode_attn_rope_freqs(D)
    w = torch.nn.Parameter(torch.linspace(0.5, 1.5, D, device="cuda"))  # as a module holds it
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pools = [torch.zeros_like(t["pool"]) for _ in range(2)]
    a = call.append_q4(*_append(t, f, pool=pools[0], norm=True, w=w, status=status))
    assert type(a) is torch.Tensor and not a.requires_grad
    b = qk.decode_attn_append_paged_q4(t["k"], t["v"], t["pos"], t["table"], pools[1], f, group=GROUP,
                                       token_seq=t["seq"], q=t["q"], norm=True, q_weight=w, k_weight=w,
                                       stream=here)
    assert torch.equal(a, b) and torch.equal(*pools) and bool(pools[0].any())
    out = torch.zeros_like(a)
    c = call.append_q4(*_append(t, f, pool=pools[0], norm=True, w=w, q_out=out))
    assert c is out and torch.equal(out, b)
    assert call.append_q4(*_append(t, f, pool=pools[0], q=None)) is None
    t["pool"] = pools[1]

    got = call.gather_q4(*_gather(t, status=status))
    want = qk.decode_attn_gather_paged_q4(t["pos"], t["table"], t["pool"], head_dim=D, group=GROUP,
                                          token_seq=t["seq"], stream=here)
    assert type(got) is tuple and all(torch.equal(x, y) for x, y in zip(got, want))

    lens = t["pos"] + 1
    for T in (1, 3):
        q = torch.randn((N, HQ, D) if T == 1 else (N, T, HQ, D), device="cuda")
        got = call.attend_q4(*_attend(t, q, lens, q_pos=lens - 1, status=status))
        want = qk.decode_attn_paged_q4(q, t["pool"], t["table"], lens, lens - 1, group=GROUP, stream=here)
        assert type(got) is tuple and all(torch.equal(x, y) for x, y in zip(got, want))
        outs = [torch.zeros_like(x) for x in want]
        got = call.attend_q4(*_attend(t, q, lens, q_pos=lens - 1, out=outs[0], lse=outs[1]))
        assert all(x is y and torch.equal(x, z) for x, y, z in zip(got, outs, want))

    old, new = t["pos"].clone(), t["pos"] + 3  # 0, 5 ... 30; pages 0 to 2 of each row
    free = torch.arange(4 * N, dtype=torch.int32, device="cuda")
    states = []
    for i in range(2):
        table, stack = t["table"].clone(), free.clone()
        count = torch.full((1,), 2 * N, dtype=torch.int32, device="cuda")
        if i == 0:
            got = call.plan(old, new, table, stack, count, BS, 4 * N, 40, status)
            assert type(got) is tuple
        else:
            got = qk.decode_attn_plan_blocks(old, new, table, stack, count, block_size=BS,
                                             num_blocks=4 * N, max_tokens=40, stream=here)
        states.append((*got, table, stack, count))
    assert int(states[0][3][-1]) == 3 * N
    assert all(torch.equal(x, y) for x, y in zip(*states))
    assert int(status) == 0


@pytest.mark.gpu
def test_leaves_unusual_calls_to_python(cuda_lib, call):
    t = _tensors("cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, lens = torch.zeros((N, HQ, D), device="cuda"), t["pos"] + 1
    assert type(call.append_q4(*_append(t))) is torch.Tensor
    for kw in (dict(k=t["k"].float()), dict(v=t["v"][:2]), dict(q=t["q"][:2]), dict(pos=t["pos"].long()),
               dict(pos=t["pos"][:2]), dict(seq=t["seq"][:2]), dict(pool=t["pool"].int()),
               dict(pool=t["pool"][:, :1]), dict(pool=t["pool"][..., :-1].contiguous()), dict(group=48),
               dict(group=256), dict(group=0), dict(group=-64), dict(group="a"), dict(norm=1), dict(eps="a"),
               dict(w=q[0, 0]), dict(q_out=q[:, :1]), dict(q_out=q.half()), dict(table=t["table"].t()),
               dict(table=t["table"].cpu()), dict(q=None, q_out=q), dict(status=status.long())):
        assert call.append_q4(*_append(t, **kw)) is NotImplemented, kw
    assert type(call.gather_q4(*_gather(t))) is tuple
    for kw in (dict(pos=t["pos"][:0]), dict(pos=t["pos"].long()), dict(seq=t["seq"][:2]), dict(d=0),
               dict(d=-128), dict(d=2 ** 40), dict(d=96), dict(group=7), dict(pool=t["pool"].cpu()),
               dict(table=t["table"][0]), dict(status=q)):
        assert call.gather_q4(*_gather(t, **kw)) is NotImplemented, kw
    assert type(call.attend_q4(*_attend(t, q, lens))) is tuple
    for kw in (dict(q_pos=lens[:2]), dict(q_pos=lens.long()), dict(group=16), dict(scale="a"),
               dict(out=q[:, :1]), dict(lse=q), dict(table=t["table"][:2]), dict(pool=t["pool"][0])):
        assert call.attend_q4(*_attend(t, q, lens, **kw)) is NotImplemented, kw
    for bad in (q.half(), q[:, :, :64], q.transpose(0, 1), q[0], q[:0], q.cpu()):
        assert call.attend_q4(*_attend(t, bad, lens)) is NotImplemented
    old = t["pos"]
    for args in (_plan(t, old.long(), old), _plan(t, old, old[:2]), _plan(t, old, old, -1),
                 _plan(t, old[:0], old[:0]), _plan(t, old, old, count=t["seq"]),
                 _plan(t, old, old, free=t["seq"].cpu()), _plan(t, old, old, bs="a")):
        assert call.plan(*args) is NotImplemented
    # an error of the entry point: its status
    assert call.attend_q4(*_attend(t, q, lens, out=q)) == qk.DA_ERR_INVALID
    assert call.plan(*_plan(t, old, old, bs=24)) == qk.DA_ERR_UNSUPPORTED
    with pytest.raises(qk.DecodeAttnError):
        qk.decode_attn_paged_q4(q, t["pool"], t["table"], lens, group=GROUP, out=q)
    with pytest.raises(qk.DecodeAttnError):
        qk.decode_attn_plan_blocks(old, old, t["table"], t["seq"], t["seq"][:1], block_size=24,
                                   num_blocks=4 * N, max_tokens=0)
    # a captured decode has a workspace of its graph's
    torch.cuda.synchronize()
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        assert call.attend_q4(*_attend(t, q, lens)) is NotImplemented
        assert type(call.gather_q4(*_gather(t))) is tuple
    torch.cuda.synchronize()
