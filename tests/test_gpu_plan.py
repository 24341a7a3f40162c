"""Pages and places of requests on the GPU against a loop on the host: every
table entry, free page, position and slot has to match."""
import os
import subprocess
import sys

import numpy as np
import pytest

import quantized_kv_decode_paged_gb300 as qk

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    yield


def _t(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def plan(old, new, table, free, count, bs, NB, N):
    """The definition, a request at a time; (flags, table, free, count, positions, seq, slots,
    cu), the state unchanged where a flag is set."""
    B, mb = table.shape
    none = (table, free, count, np.zeros(N, np.int32), np.full(N, -1, np.int32),
            np.full(N, -1, np.int64), np.zeros(B + 1, np.int32))
    flags = 0
    ok = (old >= 0) & (new >= 0) & (old <= mb * bs) & (new <= mb * bs)
    if not ok.all():
        flags |= qk.DEV_BAD_SEQ_LEN
    o, n = np.where(ok, old, 0).astype(np.int64), np.where(ok, new, 0).astype(np.int64)
    po, pn = -(-o // bs), -(-n // bs)
    most = min(len(free), NB)
    if count < 0 or count > most:
        flags |= qk.DEV_BAD_FREE_LIST
    if np.maximum(n - o, 0).sum() > N:
        flags |= qk.DEV_TOKEN_OVERFLOW
    taken, given = int(np.maximum(pn - po, 0).sum()), int(np.maximum(po - pn, 0).sum())
    left = count + given - taken
    if left < 0:
        flags |= qk.DEV_NO_BLOCKS
    if left > most:
        flags |= qk.DEV_BAD_FREE_LIST
    if flags:
        return (flags,) + none
    table2, free2 = table.copy(), free.copy()
    stack = free[:count].tolist()
    for i in range(left, count):
        if not 0 <= free[i] < NB:
            flags |= qk.DEV_BAD_FREE_LIST
    for b in range(B):
        for j in range(pn[b], po[b]):
            if not 0 <= table[b, j] < NB:
                flags |= qk.DEV_BAD_BLOCK
            stack.append(table[b, j])
            table2[b, j] = -1
        if n[b] > o[b] and o[b] % bs and not 0 <= table[b, o[b] // bs] < NB:
            flags |= qk.DEV_BAD_BLOCK
    if flags:
        return (flags,) + none
    free2[:left] = stack[:left]
    top = iter(stack[left:])
    pos, seq, slots, cu = [], [], [], [0]
    for b in range(B):
        for j in range(po[b], pn[b]):
            table2[b, j] = next(top)
        for p in range(o[b], n[b]):
            pos.append(p)
            seq.append(b)
            slots.append(int(table2[b, p // bs]) * bs + p % bs)
        cu.append(len(pos))
    pads = N - len(pos)
    return (0, table2, free2, left, np.array(pos + [0] * pads, np.int32),
            np.array(seq + [-1] * pads, np.int32), np.array(slots + [-1] * pads, np.int64),
            np.array(cu, np.int32))


def _state(r, old, bs, mb, NB, capacity=None):
    held = -(-old // bs)
    perm = r.permutation(NB).astype(np.int32)
    table = np.full((len(old), mb), -1, np.int32)
    at = np.concatenate([[0], np.cumsum(held)])
    for b in range(len(old)):
        table[b, :held[b]] = perm[at[b]:at[b + 1]]
    free = np.full(NB if capacity is None else capacity, -7, np.int32)
    rest = perm[at[-1]:]
    free[:len(rest)] = rest
    return table, free, len(rest)


def _run(old, new, table, free, count, bs, NB, N, **kw):
    import torch
    tt, tf, tc = _t(table), _t(free), _t(np.array([count], np.int32))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = qk.decode_attn_plan_blocks(_t(old.astype(np.int32)), _t(new.astype(np.int32)), tt, tf, tc,
                                      block_size=bs, num_blocks=NB, max_tokens=N,
                                      dev_status=status, **kw)
    torch.cuda.synchronize()
    return (int(status.item()), tt.cpu().numpy(), tf.cpu().numpy(), int(tc.item()),
            *[o.cpu().numpy() for o in outs])


def _same(got, want):
    names = ("flags", "table", "free", "count", "positions", "token_seq", "slots", "cu_tokens")
    for name, g, w in zip(names, got, want):
        assert np.array_equal(g, w), (name, g, w)


@pytest.mark.parametrize("B", [1, 2, 31, 33, 1000, 1025, 5000, 16384])
@pytest.mark.parametrize("bs", [8, 16, 256])
def test_growing_shrinking_and_waiting(B, bs):
    r = np.random.default_rng(B + bs)
    cap = 40 if B > 2000 else 700
    old, new = r.integers(0, cap, B), r.integers(0, cap, B)
    wait = r.random(B) < 0.3
    new[wait] = old[wait]
    mb = -(-cap // bs) + 1
    NB = int(np.maximum(-(-old // bs), -(-new // bs)).sum()) + 3
    table, free, count = _state(r, old, bs, mb, NB)
    N = int(np.maximum(new - old, 0).sum()) + int(r.integers(0, 9))
    args = (old, new, table, free, count, bs, NB, N)
    want = plan(*args)
    assert want[0] == 0
    got = _run(*args)
    _same(got, want)
    # old and new exchanged: every page back where it was
    M = int(np.maximum(old - new, 0).sum())
    back = _run(new, old, got[1], got[2], got[3], bs, NB, M)
    assert back[0] == 0 and back[3] == count
    assert np.array_equal(back[1], table) and np.array_equal(back[2][:count], free[:count])


@pytest.mark.parametrize("old,new", [([0], [0]), ([0], [1]), ([16], [17]), ([16], [15]), ([15], [16]),
                                     ([33], [32]), ([32], [0]), ([0, 5, 0], [48, 5, 0]),
                                     ([48, 0], [0, 48]), ([0, 48], [48, 0]), ([40, 8], [8, 48])])
def test_small_steps(old, new):
    r = np.random.default_rng(3)
    old, new = np.array(old), np.array(new)
    table, free, count = _state(r, old, 16, 3, 6)
    for N in (48, 60):
        args = (old, new, table, free, count, 16, 6, N)
        _same(_run(*args), plan(*args))


@pytest.mark.parametrize("B", [6, 3000])
def test_all_or_nothing(B):
    """Each reason alone: flags as defined, nothing changed, all padding."""
    r = np.random.default_rng(4)
    bs, mb = 16, 8
    old = r.integers(17, 60, B)
    new = np.minimum(old + 20, mb * bs)
    new[1], new[2] = 3, old[2] - 16
    old[3] = 40  # inside a page
    new[3] = 45
    NB = B * mb
    table, free, count = _state(r, old, bs, mb, NB)
    N = int(np.maximum(new - old, 0).sum())
    ok = dict(old=old, new=new, table=table, free=free, count=count, bs=bs, NB=NB, N=N)
    assert plan(**ok)[0] == 0
    need = int(np.maximum(-(-new // bs) + -old // bs, 0).sum())

    def entry(a, at, v):
        a = a.copy()
        a[at] = v
        return a

    up = np.maximum(old, new)  # nothing comes back
    cases = [(dict(count=0, free=free[:0], new=up), qk.DEV_NO_BLOCKS),
             (dict(N=N - 1), qk.DEV_TOKEN_OVERFLOW),
             (dict(old=entry(old, 0, -1)), qk.DEV_BAD_SEQ_LEN),
             (dict(new=entry(new, 0, mb * bs + 1)), qk.DEV_BAD_SEQ_LEN),
             (dict(new=entry(new, B - 1, 2 ** 31 - 1)), qk.DEV_BAD_SEQ_LEN),
             (dict(table=entry(table, (1, 1), -1)), qk.DEV_BAD_BLOCK),  # given back
             (dict(table=entry(table, (3, 2), NB)), qk.DEV_BAD_BLOCK),  # goes on growing
             (dict(free=entry(free, count - 1, -1), new=up), qk.DEV_BAD_FREE_LIST),
             (dict(count=-1), qk.DEV_BAD_FREE_LIST),
             (dict(count=len(free) + 1), qk.DEV_BAD_FREE_LIST)]
    assert need > 0
    for change, flag in cases:
        args = {**ok, **change}
        want = plan(**args)
        assert want[0] & flag, (change, want[0])
        _same(_run(**args), want)
    # a stack too small for what comes back
    gone = np.zeros(B, np.int64)
    t2, f2, c2 = _state(r, old, bs, mb, NB, capacity=None)
    args = dict(old=old, new=gone, table=t2, free=f2[:c2 + 1], count=c2, bs=bs, NB=NB, N=0)
    want = plan(**args)
    assert want[0] == qk.DEV_BAD_FREE_LIST
    _same(_run(**args), want)
    # entries that the call does not read may hold anything
    t3 = entry(table, (0, mb - 1), 2 ** 31 - 1)
    args = {**ok, "table": t3}
    _same(_run(**args), plan(**args))


def test_many_tokens_of_few_requests():
    r = np.random.default_rng(5)
    old, new = np.array([5, 0, 70000, 31]), np.array([60000, 33333, 70001, 2])
    bs, mb, NB = 32, 2300, 9000
    table, free, count = _state(r, old, bs, mb, NB)
    args = (old, new, table, free, count, bs, NB, 100000)
    _same(_run(*args), plan(*args))


def test_outputs_streams_and_graph_replay():
    """Given outputs are filled, behind a pending copy on the call's stream; one capture,
    replayed from step to step."""
    import torch
    r = np.random.default_rng(6)
    B, bs, mb, NB, N = 50, 16, 12, 800, 400
    old = r.integers(0, 100, B)
    table, free, count = _state(r, old, bs, mb, NB)
    tt, tf, tc = _t(table), _t(free), _t(np.array([count], np.int32))
    told, tnew = _t(old.astype(np.int32)), _t(old.astype(np.int32))
    i32 = dict(dtype=torch.int32, device="cuda")
    outs = [torch.empty(N, **i32), torch.empty(N, **i32),
            torch.empty(N, dtype=torch.int64, device="cuda"), torch.empty(B + 1, **i32)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()

    def call(**kw):
        got = qk.decode_attn_plan_blocks(told, tnew, tt, tf, tc, block_size=bs, num_blocks=NB,
                                         max_tokens=N, positions=outs[0], token_seq=outs[1],
                                         slots=outs[2], cu_tokens=outs[3], **kw)
        assert all(a is b for a, b in zip(got, outs))

    call(stream=s)  # nothing to do
    s.synchronize()
    assert outs[3].abs().max() == 0 and (outs[1] == -1).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for i in range(6):
        new = np.clip(old + r.integers(-20, 9, B), 0, mb * bs)
        want = plan(old, new, table, free, count, bs, NB, N)
        assert want[0] == 0
        told.copy_(_t(old.astype(np.int32)))
        tnew.copy_(_t(new.astype(np.int32)))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.synchronize()
        _same((0, tt.cpu().numpy(), tf.cpu().numpy(), int(tc.item()),
               *[o.cpu().numpy() for o in outs]), want)
        _, table, free, count = want[:4]
        old = new


def test_a_large_call_in_a_graph():
    """A cluster's launch, captured and replayed: there and back, many times."""
    import torch
    r = np.random.default_rng(7)
    B, bs, mb, NB = 1500, 16, 10, 9000
    old, new = r.integers(0, 80, B), r.integers(0, 80, B)
    table, free, count = _state(r, old, bs, mb, NB)
    N = 40000
    want = plan(old, new, table, free, count, bs, NB, N)
    assert want[0] == 0
    tt, tf, tc = _t(table), _t(free), _t(np.array([count], np.int32))
    told, tnew = _t(old.astype(np.int32)), _t(new.astype(np.int32))
    kw = dict(block_size=bs, num_blocks=NB, max_tokens=N)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            outs = qk.decode_attn_plan_blocks(told, tnew, tt, tf, tc, **kw)
            kept = [t.clone() for t in (tt, tf, tc)]
            qk.decode_attn_plan_blocks(tnew, told, tt, tf, tc, **kw)
        for _ in range(5):
            g.replay()
    torch.cuda.synchronize()
    _same((0, kept[0].cpu().numpy(), kept[1].cpu().numpy(), int(kept[2].item()),
           *[o.cpu().numpy() for o in outs]), want)
    assert np.array_equal(tt.cpu().numpy(), table) and int(tc.item()) == count
    assert np.array_equal(tf.cpu().numpy()[:count], free[:count])


def test_no_requests_and_no_tokens():
    import torch
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    table = torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    free, count = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.ones(
        1, dtype=torch.int32, device="cuda")
    pos, seq, slots, cu = qk.decode_attn_plan_blocks(z, z, table, free, count, block_size=16,
                                                     num_blocks=4, max_tokens=5)
    assert pos.tolist() == [0] * 5 and seq.tolist() == slots.tolist() == [-1] * 5
    assert cu.tolist() == [0] and int(count) == 1
    args = (np.array([20]), np.array([3]), np.array([[2, 1]], np.int32), np.array([0, 9], np.int32),
            1, 16, 4, 0)
    _same(_run(*args), plan(*args))


def test_shared_memory_up_to_and_past_the_default(tmp_path):
    """A process's first calls, from 2417 requests on (48,352 bytes of sums and lengths beside the
    kernel's own; past 48 KB a kernel has to be allowed to have them), none larger before."""
    code = ("import numpy as np, test_gpu_plan as t\n"
            "r = np.random.default_rng(8)\n"
            "for B in (2417, 2418, 2440, 2457, 2458):\n"
            "    old, new = r.integers(0, 60, B), r.integers(0, 60, B)\n"
            "    table, free, count = t._state(r, old, 16, 4, 4 * B)\n"
            "    args = (old, new, table, free, count, 16, 4 * B, 60 * B)\n"
            "    t._same(t._run(*args), t.plan(*args))\n")
    here = os.path.dirname(os.path.abspath(__file__))
    env = {**os.environ, "PYTHONPATH": os.pathsep.join([here, os.path.dirname(here)])}
    ran = subprocess.run([sys.executable, "-c", code], env=env, cwd=tmp_path, capture_output=True,
                         text=True, timeout=300)
    assert ran.returncode == 0, ran.stderr[-2000:]
