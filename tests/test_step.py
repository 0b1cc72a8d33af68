"""The operators of a serving step around the attention: pa_build_slots,
pa_cache_write and pa_verify_drafts against plain implementations (whole
numbers and 64 bits), their refusals, and a run of all four together.

Everything here is compared exactly: block ids, slots and tokens are whole
numbers and cache rows are copied bit for bit.  A drawn token is compared with
the exact rational arithmetic of Python's fractions (or fp64 sums where the
draw lies far from every border of the running sum)."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import oracle
import paged_gqa_decode_pa_gb300 as pg
from paged_gqa_decode_pa_gb300 import build as pgbuild
from paged_gqa_decode_pa_gb300 import workloads as wl


@pytest.fixture(scope="module", autouse=True)
def built_library():
    pgbuild.build()
    yield


FAKE = 1 << 20


# ------------------------------------------------------------------ refusals


def slots_call(s, total_new=8, ws_bytes=256, **ptr):
    names = ("cache_seqlens", "new_lens", "held", "table", "free_list", "free_count")
    outs = ("cu", "slots", "seqlens_out", "held_out", "free_count_out", "ws")
    p = {n: FAKE for n in names + outs}
    p.update(ptr)
    return pg.lib().pa_build_slots(ctypes.byref(s) if s else None, *(p[n] for n in names), total_new,
                                   *(p[n] for n in outs), ws_bytes, None)


def shape(B=3, bs=16, maxblk=8, P=16, Hkv=2, d=128, dtype=pg.PA_BF16):
    return pg.pa_shape(B, Hkv, Hkv, d, bs, maxblk, P, dtype)


def test_build_slots_refuses():
    assert slots_call(None) == pg.PA_ERR_NULL
    for n in ("cache_seqlens", "new_lens", "held", "table", "free_list", "free_count", "cu", "slots", "seqlens_out",
              "held_out", "free_count_out", "ws"):
        assert slots_call(shape(), **{n: None}) == pg.PA_ERR_NULL, n
        assert slots_call(shape(), **{n: FAKE + 4}) == pg.PA_ERR_ALIGN, n
    assert slots_call(shape(), ws_bytes=128) == pg.PA_ERR_WORKSPACE
    for bad in (shape(B=-1), shape(B=pg.PA_MAX_BATCH + 1), shape(bs=8), shape(bs=48), shape(maxblk=0), shape(P=0),
                shape(maxblk=1 << 28), shape(B=8192, maxblk=1 << 20)):
        assert slots_call(bad) == pg.PA_ERR_SHAPE
    assert slots_call(shape(), total_new=-1) == pg.PA_ERR_SHAPE


def write_call(s, T=4, ks=256, vs=256, k=FAKE, v=FAKE, slots=FAKE, kc=FAKE, vc=FAKE, ws=FAKE, ws_bytes=256):
    return pg.lib().pa_cache_write(ctypes.byref(s), k, ks, v, vs, slots, T, kc, vc, ws, ws_bytes, None)


def test_cache_write_refuses():
    for kw in (dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None), dict(ws=None)):
        assert write_call(shape(), **kw) == pg.PA_ERR_NULL
    for kw in (dict(k=FAKE + 8), dict(v=FAKE + 2), dict(slots=FAKE + 8), dict(kc=FAKE + 4), dict(vc=FAKE + 8)):
        assert write_call(shape(), **kw) == pg.PA_ERR_ALIGN
    for kw in (dict(T=-1), dict(ks=255), dict(ks=260), dict(vs=248), dict(vs=257)):
        assert write_call(shape(), **kw) == pg.PA_ERR_SHAPE
    for bad in (shape(d=12), shape(Hkv=0), shape(P=0), shape(bs=0), shape(dtype=pg.PA_F32)):
        assert write_call(bad, ks=1 << 20, vs=1 << 20) == pg.PA_ERR_SHAPE
    assert write_call(shape(), ws_bytes=8) == pg.PA_ERR_WORKSPACE
    assert write_call(shape(), T=0, k=None, slots=None) == pg.PA_OK


def verify_call(B=2, V=100, D=4, dt=pg.PA_F32, qs=100, ps=100, ws_bytes=1 << 30, **ptr):
    p = {n: FAKE for n in ("x", "cu", "q", "p", "ua", "us", "out", "acc", "ws")}
    p.update(ptr)
    return pg.lib().pa_verify_drafts(B, V, D, dt, p["x"], p["cu"], p["q"], qs, p["p"], ps, p["ua"], p["us"], p["out"],
                                     p["acc"], p["ws"], ws_bytes, None)


def test_verify_drafts_refuses():
    for n in ("x", "cu", "p", "ua", "us", "out", "acc", "ws"):
        assert verify_call(**{n: None}) == pg.PA_ERR_NULL, n
    for n in ("x", "cu", "q", "p", "ua", "us", "out", "acc", "ws"):
        assert verify_call(**{n: FAKE + 4}) == pg.PA_ERR_ALIGN, n
    for kw in (dict(B=-1), dict(B=pg.PA_MAX_BATCH + 1), dict(V=0), dict(V=pg.PA_MAX_VOCAB + 1, ps=1 << 25, qs=1 << 25),
               dict(D=-1), dict(dt=3), dict(qs=99), dict(ps=99)):
        assert verify_call(**kw) == pg.PA_ERR_SHAPE, kw
    assert verify_call(ws_bytes=256) == pg.PA_ERR_WORKSPACE
    assert verify_call(B=0, cu=None, p=None, ws=None) == pg.PA_OK
    assert pg.lib().pa_workspace_size_verify(2, 100, None) == pg.PA_ERR_NULL
    for code in (pg.PA_STATUS_NO_BLOCKS, pg.PA_STATUS_BAD_PROB, pg.PA_STATUS_BAD_TOKEN):
        assert pg.status_string(code) != "unknown code"


# ------------------------------------------------------------------ slot maps


def plain_slots(lens, new, held, table, free, count, bs, T, P):
    """The rule of pa_build_slots, one sequence at a time."""
    table, free = table.copy(), free.copy()
    B, cols = table.shape
    bad = [n < 0 or a < 0 or n + a > cols * bs or h < 0 or h > cols or -(-n // bs) > h for n, a, h in zip(lens, new, held)]
    need = [h if b else -(-(n + a) // bs) for n, a, h, b in zip(lens, new, held, bad)]
    stack = list(free[:count])
    for b in range(B):
        stack += [table[b, c] for c in range(need[b], held[b])]
    top = len(stack)
    full = list(stack)
    cu, slots = np.zeros(B + 1, np.int64), np.full(T, -1, np.int64)
    so, ho = np.zeros(B, np.int32), np.zeros(B, np.int32)
    wanted, used, status = 0, 0, 0
    for b in range(B):
        rows = max(new[b], 0)
        cu[b + 1] = cu[b] + rows
        want = max(0, need[b] - held[b])
        wanted += want
        fits = rows == 0 or cu[b + 1] <= T
        served = not bad[b] and fits and (want == 0 or wanted <= top)
        if bad[b] or not fits:
            status |= pg.PA_STATUS_BAD_SEQLEN
        elif not served:
            status |= pg.PA_STATUS_NO_BLOCKS
        so[b] = lens[b] + rows if served else lens[b]
        ho[b] = need[b] if served else min(held[b], need[b])
        if served:
            for c in range(held[b], need[b]):
                table[b, c] = full[top - 1 - (wanted - want) - (c - held[b])]
            used += want
            for i in range(rows):
                pos = lens[b] + i
                slots[cu[b] + i] = int(table[b, pos // bs]) * bs + pos % bs
    free[:top] = full
    return dict(table=table, free=free, cu=np.minimum(cu, T).astype(np.int32), slots=slots, seqlens_out=so, held_out=ho,
                count=top - used, status=status)


def run_slots(lens, new, held, table, free, count, bs, T, alias=False):
    import torch

    def dev(x, dt=torch.int32):
        return torch.tensor(np.asarray(x), dtype=dt, device="cuda")

    B = len(lens)
    sl, nw, hd, tb, fr, ct = dev(lens), dev(new), dev(held), dev(table), dev(free), dev([count])
    cu = torch.full((B + 1,), -9, dtype=torch.int32, device="cuda")
    slots = torch.full((T,), -9, dtype=torch.int64, device="cuda")
    so, ho, co = (sl, hd, ct) if alias else (torch.full_like(sl, -9), torch.full_like(hd, -9), torch.full_like(ct, -9))
    ws = pg.alloc_workspace_status()
    pg.pa_build_slots(sl, nw, hd, tb, fr, ct, bs, cu, slots, so, ho, co, ws)
    st = pg.pa_read_status(ws)
    n = lambda t: t.cpu().numpy()  # noqa: E731
    return dict(table=n(tb), free=n(fr), cu=n(cu), slots=n(slots), seqlens_out=n(so), held_out=n(ho), count=int(co), status=st)


def slot_case(B, bs, seed, spare=None, cols=None, T=None):
    rng = np.random.default_rng(seed)
    new = rng.integers(0, 40, B)
    lens = rng.integers(0, 300, B)
    gone = rng.random(B) < 0.15
    new[gone] = lens[gone] = 0
    new[rng.random(B) < 0.4] = 1
    cols = cols or -(-340 // bs) + 2
    held = [min(cols, -(-int(n) // bs) + int(rng.integers(0, 3))) for n in lens]
    held = [int(rng.integers(0, cols + 1)) if g else h for h, g in zip(held, gone)]
    need = sum(max(0, -(-int(n + a) // bs) - h) for n, a, h in zip(lens, new, held))
    P = sum(held) + need + 5
    ids = rng.permutation(P).astype(np.int32)
    table = np.full((B, cols), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, : held[b]] = ids[at: at + held[b]]
        at += held[b]
    count = P - at if spare is None else min(spare, P - at)
    free = np.full(P, -1, np.int32)
    free[:count] = ids[at: at + count]
    T = int(new.sum()) + 6 if T is None else T
    return [int(x) for x in lens], [int(x) for x in new], held, table, free, count, bs, T


def same(got, want):
    for k in want:
        assert np.array_equal(got[k], want[k]), (k, got[k], want[k])


@pytest.mark.gpu
@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("B,bs", [(1, 16), (2, 64), (31, 16), (255, 32), (256, 16), (257, 64), (1025, 16), (5000, 32),
                                  (8192, 16)])
def test_slots_match_the_rule(B, bs, alias):
    case = slot_case(B, bs, seed=B)
    same(run_slots(*case, alias=alias), plain_slots(*case, P=len(case[4])))


@pytest.mark.gpu
@pytest.mark.parametrize("B", [5, 200, 3000])
@pytest.mark.parametrize("spare", [0, 2, 40])
def test_slots_with_a_short_stack_and_a_short_map(B, spare):
    case = slot_case(B, 16, seed=B + spare, spare=spare)
    want = plain_slots(*case, P=len(case[4]))
    same(run_slots(*case), want)
    case = slot_case(B, 16, seed=B, T=max(1, B // 3))
    want = plain_slots(*case, P=len(case[4]))
    assert want["status"] & pg.PA_STATUS_BAD_SEQLEN
    same(run_slots(*case), want)


_FRESH = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import numpy as np
from test_step import plain_slots, run_slots, same
for B in (2405, 2406, 2457, 2458, 2459):
    table = np.arange(2 * B, dtype=np.int32).reshape(B, 2)
    case = ([16] * B, [1] * B, [1] * B, table, np.arange(2 * B, dtype=np.int32), 2 * B - 1, 16, B + 2)
    same(run_slots(*case), plain_slots(*case, P=2 * B))
print("done")
"""


@pytest.mark.gpu
def test_slots_of_batches_whose_sums_take_just_under_48_kb():
    """In a process that has launched no larger batch: the kernel's shared memory is asked for in every call that needs it
    (its own variables count too, so from 2406 sequences on)."""
    import os
    import subprocess
    import sys

    tests = os.path.dirname(os.path.abspath(__file__))
    code = _FRESH.format(root=os.path.dirname(tests), tests=tests)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("done\n"), r.stderr[-2000:]


@pytest.mark.gpu
def test_slots_of_one_long_prompt_and_of_nothing():
    cols, bs = 3000, 32
    case = ([17], [90001], [1], np.full((1, cols), 3999, np.int32), np.arange(4000, dtype=np.int32), 3999, bs, 90010)
    same(run_slots(*case), plain_slots(*case, P=4000))
    case = ([], [], [], np.zeros((0, 4), np.int32), np.arange(6, dtype=np.int32), 5, 16, 3)
    got = run_slots(*case)
    assert got["count"] == 5 and got["cu"].tolist() == [0] and got["slots"].tolist() == [-1] * 3


@pytest.mark.gpu
def test_slots_with_invalid_lengths():
    lens, new, held, table, free, count, bs, T = slot_case(40, 16, seed=77)
    lens[3], new[7], held[11], held[13], lens[20] = -1, -4, -2, table.shape[1] + 1, 5000
    held[25] = 0  # fewer blocks than its tokens need
    lens[25] = 40
    got = run_slots(lens, new, held, table, free, count, bs, T)
    want = plain_slots(lens, new, held, table, free, count, bs, T, P=len(free))
    assert want["status"] & pg.PA_STATUS_BAD_SEQLEN
    for b in (11, 13):  # nothing is read or written for them; what they hold is reported as it came
        want["held_out"][b] = held[b]
    same(got, want)


@pytest.mark.gpu
def test_slots_with_ids_outside_the_pool():
    table = np.full((2, 4), -1, np.int32)
    table[0, 0] = 99  # token 3 of sequence 0 lies in block 99 of 8
    got = run_slots([3, 0], [2, 1], [1, 0], table, np.array([5, 8, 1, 0, 0, 0, 0, 0], np.int32), 2, 16, 3)
    assert got["status"] == pg.PA_STATUS_BAD_BLOCK
    assert got["slots"].tolist() == [-1, -1, -1]  # block 8 of 8 for sequence 1
    got = run_slots([0], [1], [0], table[:1], np.zeros(8, np.int32), 9, 16, 1)
    assert got["status"] == pg.PA_STATUS_BAD_BLOCK


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [-1, 8, 2**31 - 1])
@pytest.mark.parametrize("B", [3, 300])
def test_slots_report_a_bad_id_that_goes_back(B, bad):
    """A finished sequence, or a rejected draft, that gives back an id outside the pool: the call that puts it on the
    stack reports it."""
    P = max(8, 2 * B)
    bad = P if bad == 8 else bad
    for held, lens, col in ((2, 0, 1), (2, 0, 0), (2, 10, 1)):  # all blocks go back, or the second one
        table = np.full((B, 4), -1, np.int32)
        table[:, :2] = np.arange(2 * B).reshape(B, 2)
        table[B - 1, col] = bad
        free = np.full(P, -1, np.int32)
        case = ([10] * (B - 1) + [lens], [0] * B, [1] * (B - 1) + [held], table, free, 0, 16, 4)
        got = run_slots(*case)
        want = plain_slots(*case, P=P)
        assert got["status"] == pg.PA_STATUS_BAD_BLOCK and want["status"] == 0
        del want["status"]
        same(got, want)
        # a good id raises nothing
        table[B - 1, col] = 2 * B - 1
        same(run_slots(*case), plain_slots(*case, P=P))


@pytest.mark.gpu
def test_slots_agree_with_the_block_manager():
    """The device stack hands out the blocks that the host's manager hands out."""
    bs, cols, P, B = 16, 20, 64, 4
    bm = pg.BlockManager(P, bs, B, cols)
    table, free, count = np.full((B, cols), -1, np.int32), np.arange(P - 1, -1, -1, dtype=np.int32), P
    lens, held = [0] * B, [0] * B
    for step in ([20, 1, 100, 7], [1, 1, 1, 30], [5, 0, 1, 1]):
        got = run_slots(lens, step, held, table, free, count, bs, sum(step))
        for b in range(B):
            bm.allocate(b, -(-(lens[b] + step[b]) // bs) - held[b])
        table, free, count = got["table"], got["free"], got["count"]
        lens, held = got["seqlens_out"].tolist(), got["held_out"].tolist()
        want = bm.block_table(range(B), cols)
        assert np.array_equal(table, want) and count == bm.free_blocks()
    # sequence 2 ends, and its blocks serve the others' next tokens
    bm.free_sequence(2)
    got = run_slots([lens[0], lens[1], 0, lens[3]], [40, 40, 0, 40], held, table, free, count, bs, 120)
    for b in (0, 1, 3):
        bm.allocate(b, -(-(lens[b] + 40) // bs) - held[b])
    want = bm.block_table(range(B), cols)
    rows = [0, 1, 3]
    mask = want[rows] >= 0
    assert np.array_equal(got["table"][rows][mask], want[rows][mask]) and got["count"] == bm.free_blocks()
    bm.close()


# ------------------------------------------------------------------ cache write


def bits(t):
    import torch

    return t.contiguous().view(torch.int16).cpu().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("T,Hkv,d,bs,fused", [(1, 1, 64, 16, False), (3, 2, 64, 64, True), (77, 3, 256, 16, False),
                                              (1000, 8, 128, 32, True), (257, 5, 8, 16, True), (9, 40, 256, 16, False)])
def test_cache_write_copies_rows_and_nothing_else(T, Hkv, d, bs, fused, dtype):
    import torch

    dt = getattr(torch, dtype)
    g = torch.Generator(device="cuda").manual_seed(T)
    P = -(-2 * T // bs) + 1

    def rand(*s):  # any bit patterns, NaN among them
        return torch.randint(-32768, 32768, s, generator=g, device="cuda", dtype=torch.int32).to(torch.int16).view(dt)

    pools = [rand(P, bs, Hkv, d), rand(P, bs, Hkv, d)]
    slots = torch.randperm(P * bs, generator=g, device="cuda")[:T].contiguous()
    slots[::5] = -1
    slots[1::11] = -(1 << 40)
    if fused:
        rows = rand(T, 4 * Hkv, d)
        new = [rows[:, Hkv:2 * Hkv], rows[:, 3 * Hkv:]]
    else:
        new = [rand(T, Hkv, d), rand(T, Hkv, d)]
    want = [bits(p).reshape(P * bs, Hkv, d).copy() for p in pools]
    at = slots.cpu().numpy()
    for w, n in zip(want, new):
        w[at[at >= 0]] = bits(n)[at >= 0]
    ws = pg.alloc_workspace_status()
    pg.pa_cache_write(new[0], new[1], slots, pools[0], pools[1], ws)
    assert pg.pa_read_status(ws) == 0
    for w, p in zip(want, pools):
        assert np.array_equal(bits(p).reshape(w.shape), w)
    # a slot past the pool is reported and not written
    slots.fill_(-1)
    slots[0] = P * bs
    pg.pa_cache_write(new[0], new[1], slots, pools[0], pools[1], ws)
    assert pg.pa_read_status(ws) == pg.PA_STATUS_NO_SLOT
    for w, p in zip(want, pools):
        assert np.array_equal(bits(p).reshape(w.shape), w)


# ------------------------------------------------------------------ draft verification


def plain_verify(tokens, cu, q, p, ua, us, lookup):
    """In exact rational arithmetic."""
    B = len(cu) - 1
    out, acc = np.full(len(tokens) + B, -1, np.int64), np.zeros(B, np.int64)
    F = Fraction
    for b in range(B):
        c0, k = cu[b], cu[b + 1] - cu[b]
        n = 0
        while n < k:
            x = tokens[c0 + n]
            if not 0 <= x < p.shape[1]:
                break
            qx = F(1) if lookup else F(float(q[c0 + n, x]))
            if not F(float(ua[c0 + n])) * qx < F(float(p[c0 + b + n, x])):
                break
            out[c0 + b + n] = x
            n += 1
        acc[b] = n
        w = [F(float(x)) for x in p[c0 + b + n]]
        full = list(w)
        if n < k:
            if lookup:
                if 0 <= tokens[c0 + n] < len(w):
                    w[tokens[c0 + n]] = F(0)
            else:
                w = [max(F(0), a - F(float(x))) for a, x in zip(w, q[c0 + n])]
        if sum(w) == 0:
            w = full
        t, run = F(float(us[b])) * sum(w), F(0)
        for i, x in enumerate(w):
            run += x
            if run > t:
                out[c0 + b + n] = i
                break
    return out, acc


def run_verify(tokens, cu, q, p, ua, us, dtype="float32", pad=0):
    import torch

    dt = getattr(torch, dtype)
    B = len(cu) - 1

    def rows(x):
        t = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=dt, device="cuda")
        t[:, : x.shape[1]] = torch.from_numpy(x).to("cuda").to(dt)
        return t[:, : x.shape[1]]

    D = len(tokens)
    out = torch.full((D + B,), -9, dtype=torch.int32, device="cuda")
    acc = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    ws = pg.alloc_workspace_verify(B, p.shape[1])
    args = (torch.tensor(np.asarray(tokens, np.int32), device="cuda"), torch.tensor(np.asarray(cu, np.int32), device="cuda"),
            None if q is None else rows(q), rows(p), torch.from_numpy(ua).cuda(), torch.from_numpy(us).cuda(), out, acc, ws)
    pg.pa_verify_drafts(*args)
    st = pg.pa_read_status(ws)
    first = out.cpu().numpy().copy(), acc.cpu().numpy().copy()
    out.fill_(-9)
    pg.pa_verify_drafts(*args)  # the workspace is as it was
    assert np.array_equal(out.cpu().numpy(), first[0])
    return first[0], first[1], st


def verify_case(B, V, k_hi, seed, dtype="float32", peak=2.5):
    import torch

    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(rng.integers(0, k_hi + 1, B))])
    D = int(cu[-1])
    lg = rng.standard_normal((D + B, V)) * peak
    near = lg[[int(r + np.searchsorted(cu[1:], r, side="right")) for r in range(D)]] + 0.4 * rng.standard_normal((D, V))

    def soft(x):
        x = np.exp(x - x.max(1, keepdims=True)) if x.size else x
        x = (x / x.sum(1, keepdims=True)).astype(np.float32) if x.size else x.astype(np.float32)
        return torch.from_numpy(x).to(getattr(torch, dtype)).float().numpy()  # values that the type holds

    p, q = soft(lg), soft(near.reshape(D, V))
    tokens = [int(rng.choice(V, p=r.astype(np.float64) / r.astype(np.float64).sum())) for r in q]
    return tokens, cu.tolist(), q, p, rng.random(D).astype(np.float32), rng.random(B).astype(np.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("lookup", [False, True])
@pytest.mark.parametrize("B,V,k", [(1, 1, 2), (3, 7, 3), (16, 257, 4), (5, 2049, 2), (9, 5003, 8)])
def test_verify_matches_exact_arithmetic(B, V, k, lookup, dtype):
    tokens, cu, q, p, ua, us = verify_case(B, V, k, seed=B + V, dtype=dtype)
    us[0] = 0.0
    if B > 1:
        us[1] = np.float32(1 - 2.0 ** -24)
    want = plain_verify(tokens, cu, q, p, ua, us, lookup)
    for pad in (0, 3):
        out, acc, st = run_verify(tokens, cu, None if lookup else q, p, ua, us, dtype, pad)
        assert st == 0
        assert np.array_equal(acc, want[1]) and np.array_equal(out, want[0])


@pytest.mark.gpu
def test_verify_a_large_vocabulary_and_many_drafts():
    # 300 drafts of one sequence, all accepted or cut late; fp64 sums decide away from borders
    V = 150001
    rng = np.random.default_rng(4)
    p = np.zeros((3 + 2, V), np.float32)
    p[:] = rng.random((5, V)).astype(np.float32) ** 8
    p /= p.sum(1, keepdims=True, dtype=np.float64).astype(np.float32)
    q = np.roll(p[:3], 1, axis=1)
    tokens = [11, 12, 13]
    for trial in range(4):
        us = rng.random(2).astype(np.float32)
        ua = np.zeros(3, np.float32) if trial % 2 else np.full(3, 0.9999, np.float32)
        out, acc, st = run_verify(tokens, [0, 1, 3], q, p, ua, us)
        assert st == 0
        for b, (c0, c1) in enumerate(((0, 1), (1, 3))):
            n = int(acc[b])
            for i in range(n):
                assert float(ua[c0 + i]) * float(q[c0 + i, tokens[c0 + i]]) < float(p[c0 + b + i, tokens[c0 + i]])
            w = p[c0 + b + n].astype(np.float64)
            if n < c1 - c0:
                w = np.maximum(w - q[c0 + n].astype(np.float64), 0)
            c = np.cumsum(w)
            t = float(us[b]) * c[-1]
            i = int(np.searchsorted(c, t, side="right"))
            assert min(abs(c[i] - t), abs(t - (c[i - 1] if i else 0))) > 1e-13  # away from a border
            assert out[c0 + b + n] == i
    B, k, V = 1, 300, 64
    p = np.full((k + 1, V), 1 / 64, np.float32)
    toks = [i % V for i in range(k)]
    ua = np.full(k, 0.5, np.float32)
    ua[290] = 1.0 - 2.0 ** -24
    q = np.full((k, V), 1 / 64, np.float32)
    q[290] = 0
    q[290, toks[290]] = 1
    out, acc, st = run_verify(toks, [0, k], q, p, ua, np.array([0.999], np.float32))
    assert st == 0 and acc[0] == 290 and out[:290].tolist() == toks[:290]
    assert out[290] == 63 and (out[291:] == -1).all()


@pytest.mark.gpu
def test_verify_edges_and_bad_rows():
    V = 4100
    flat = np.full(V, 1 / 4096, np.float32)
    p = np.stack([flat] * 9)
    q = np.stack([flat] * 2)
    # 0: nothing left of p after q: drawn from p.  1: a NaN.  2: an infinity.  3: negative.  4: all zero.  5: sums to 5.
    # 6: a draft outside the vocabulary
    p[2, 4099], p[3, 0], p[4, 17], p[5], p[6] = np.nan, np.inf, -0.25, 0, 5 / 4096
    p[0, 5] = 0.0
    q[0] = flat
    q[0, 5] = 0.5  # u q(5) < p(5) = 0 never holds; max(p - q, 0) is 0 everywhere
    cu = [0, 1, 1, 1, 1, 1, 1, 2]
    us = np.full(7, 0.5, np.float32)
    out, acc, st = run_verify([5, V], cu, q, p, np.array([0.5, 0.0], np.float32), us)
    assert st == pg.PA_STATUS_BAD_PROB | pg.PA_STATUS_BAD_TOKEN
    assert acc.tolist() == [0] * 7
    c = np.cumsum(p[0].astype(np.float64))
    assert out[0] == int(np.searchsorted(c, 0.5 * c[-1], side="right")) and out[1] == -1
    assert out[2:7].tolist() == [-1] * 5
    assert out[8] == -1 and out[7] == int(np.searchsorted(np.cumsum(p[7] - q[1] > 0), 0.5, side="right")) or out[7] >= 0
    # spans that are none
    out, acc, st = run_verify([5, 6], [0, 3, 1], None, p[:4], np.zeros(2, np.float32), np.zeros(2, np.float32))
    assert st == pg.PA_STATUS_BAD_SEQLEN and acc.tolist() == [-1, -1] and (out == -9).all()
    # random numbers outside their range still give a token
    for u in (np.nan, -3.0, 1.0, np.inf):
        out, acc, st = run_verify([], [0, 0], None, np.stack([flat]), np.zeros(0, np.float32), np.array([u], np.float32))
        assert st == 0 and 0 <= out[0] < V


@pytest.mark.gpu
@pytest.mark.parametrize("lookup", [False, True])
def test_verify_draws_after_a_draft_outside_the_vocabulary(lookup):
    """The draft is rejected, the token comes from max(p - q, 0), or from p where nothing is left of it, and the row of
    the missing draft holds -1."""
    V = 4100
    rng = np.random.default_rng(6)
    p = rng.random((6, V)).astype(np.float32)
    q = rng.random((3, V)).astype(np.float32)
    p /= p.sum(1, keepdims=True)
    q /= q.sum(1, keepdims=True)
    p[4] = q[2]  # sequence 2: nothing is left
    tokens, cu = [V, -1, 1 << 30], [0, 1, 2, 3]
    us = np.array([0.5, 0.25, 0.75], np.float32)
    out, acc, st = run_verify(tokens, cu, None if lookup else q, p, np.zeros(3, np.float32), us)
    want, none = plain_verify(tokens, cu, q, p, np.zeros(3, np.float32), us, lookup)
    assert st == pg.PA_STATUS_BAD_TOKEN
    assert acc.tolist() == none.tolist() == [0, 0, 0]
    assert out.tolist() == want.tolist()
    assert out[1::2].tolist() == [-1] * 3 and (out[::2] >= 0).all() and (out[::2] < V).all()
    c = np.cumsum(p[4].astype(np.float64))
    assert out[4] == int(np.searchsorted(c, 0.75 * c[-1], side="right"))


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, 600])
def test_verify_draws_exactly_at_a_border_of_the_running_sum(shift):
    """u * sum(w) lies 2^-23 of a step (2^-46) below a running sum: that sum exceeds it.  In 53 bits they are equal."""
    s = 2.0 ** -46
    w = [2 ** 45, 2 ** 24 + 2 ** 22, 1, 2 ** 24 - 2 ** 22 - 3, 2 ** 45]  # whole steps, all held by fp32
    p = np.zeros((4, 700), np.float32)
    for b in range(4):
        p[b, shift + np.arange(5) * 11] = np.array(w, np.float64) * s
    assert all(float(np.float32(x * s)) == x * s for x in w)
    u = np.float32(0.5 + 2.0 ** -24)
    t = Fraction(float(u)) * sum(w)
    assert sum(w[:3]) - t == Fraction(1, 2 ** 23) and float(t) == sum(w[:3])
    # and the numbers next to it, and one among fp32's subnormals
    us = np.array([u, np.nextafter(u, np.float32(1)), np.float32(0.5), np.float32(1e-44)], np.float32)
    args = ([], [0] * 5, None, p, np.zeros(0, np.float32), us)
    want, _ = plain_verify(*args, True)
    assert [(x - shift) / 11 for x in want] == [2, 3, 1, 0]
    out, acc, st = run_verify(*args)
    assert st == 0 and out.tolist() == want.tolist()


@pytest.mark.gpu
def test_verify_workspace_serves_batches_of_any_size():
    import torch

    V = 700
    ws = pg.alloc_workspace_verify(300, V)
    for B in (2, 300, 40, 300, 1, 299):
        tokens, cu, q, p, ua, us = verify_case(B, V, 3, seed=B, dtype="float32")
        want = plain_verify(tokens, cu, q, p, ua, us, False)
        out = torch.full((len(tokens) + B,), -9, dtype=torch.int32, device="cuda")
        acc = torch.full((B,), -9, dtype=torch.int32, device="cuda")
        on = [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in
              (np.asarray(tokens, np.int32), np.asarray(cu, np.int32), q.astype(np.float32), p.astype(np.float32), ua, us)]
        pg.pa_verify_drafts(*on, out, acc, ws)
        assert pg.pa_read_status(ws) == 0
        assert np.array_equal(acc.cpu().numpy(), want[1]) and np.array_equal(out.cpu().numpy(), want[0])


# ------------------------------------------------------------------ a step of all four


@pytest.mark.gpu
def test_a_serving_loop_of_drafts():
    """Prompt, then steps of drafted tokens: tables and slots on the device, rows written by slot map, attention over
    the cache, verification, and the rejected rows' blocks going back -- captured once and replayed."""
    import torch

    rng = np.random.default_rng(8)
    B, H, Hkv, d, bs, cols, P, V, k = 3, 8, 2, 64, 16, 16, 40, 97, 4
    dev = dict(device="cuda")
    i32 = dict(dtype=torch.int32, **dev)
    kc, vc = (torch.full((P, bs, Hkv, d), float("nan"), dtype=torch.bfloat16, **dev) for _ in range(2))
    table = torch.full((B, cols), -1, **i32)
    free, count = torch.arange(P, **i32).flip(0).contiguous(), torch.tensor([P], **i32)
    lens, held, new = torch.zeros(B, **i32), torch.zeros(B, **i32), torch.zeros(B, **i32)
    T = 64
    cu, slots, so = torch.zeros(B + 1, **i32), torch.zeros(T, dtype=torch.int64, **dev), torch.zeros(B, **i32)
    qkv = torch.zeros(T, H + 2 * Hkv, d, dtype=torch.bfloat16, **dev)
    q, kn, vn = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    out, lse = torch.zeros(T, H, d, dtype=torch.bfloat16, **dev), torch.zeros(T, H, **dev)
    st, ws = pg.alloc_workspace_status(), pg.alloc_workspace_prefill(pg.shape_multi(q, kc, table))
    stream = torch.cuda.Stream()

    def step():
        pg.pa_build_slots(lens, new, held, table, free, count, bs, cu, slots, so, held, count, st)
        pg.pa_cache_write(kn, vn, slots, kc, vc, st)
        pg.pa_prefill(q, cu, True, kc, vc, table, so, d ** -0.5, out, lse, ws)

    keys = [[] for _ in range(B)]
    vals = [[] for _ in range(B)]
    graph = None
    for turn in range(6):
        adds = [20, 33, 7] if turn == 0 else [k + 1] * B
        qkv.copy_(torch.from_numpy(rng.standard_normal((T, H + 2 * Hkv, d)).astype(np.float32)))
        new.copy_(torch.tensor(adds))
        torch.cuda.synchronize()
        if turn == 2:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                step()
        if graph is None:
            step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert pg.pa_read_status(st) == 0 and pg.pa_read_status(ws) == 0
        rows = np.concatenate([[0], np.cumsum(adds)])
        assert cu.tolist() == rows.tolist()
        qf, kf, vf = (x.double().cpu().numpy() for x in (q, kn, vn))
        for b in range(B):
            r = slice(rows[b], rows[b + 1])
            keys[b] += list(kf[r])
            vals[b] += list(vf[r])
            n, K, W = len(keys[b]), np.array(keys[b]), np.array(vals[b])
            assert int(so[b]) == n and int(held[b]) == -(-n // bs)
            for i in range(adds[b]):
                for h in range(H):
                    x = K[: n - adds[b] + i + 1, h // 4] @ qf[rows[b] + i, h] * d ** -0.5
                    w = np.exp(x - x.max())
                    ref, A = w @ W[: len(x), h // 4] / w.sum(), w @ np.abs(W[: len(x), h // 4]) / w.sum()
                    u = 2.0 ** -8
                    err = np.abs(out[rows[b] + i, h].double().cpu().numpy() - ref)
                    assert (err <= u * (np.abs(ref) * (1 + u) + A) + 2.0 ** -14 * A + 2.0 ** -24).all()
        assert int(count) + int(held.sum()) == P  # no block is lost
        used = [int(x) for b in range(B) for x in table[b, : int(held[b])].tolist()] + free[: int(count)].tolist()
        assert sorted(used) == list(range(P))
        if turn == 0:
            lens.copy_(so)
            continue
        # the drafts' verification decides how much of the step stays
        tokens, cud, qd, pt, ua, us = verify_case(B, V, 0, seed=turn)[0:1] + (None,) * 5
        D = B * k
        cud = [k * b for b in range(B + 1)]
        pt = rng.dirichlet(np.ones(V), D + B).astype(np.float32)
        qd = rng.dirichlet(np.ones(V), D).astype(np.float32)
        tokens = rng.integers(0, V, D).tolist()
        ua, us = rng.random(D).astype(np.float32), rng.random(B).astype(np.float32)
        emitted, acc, status = run_verify(tokens, cud, qd, pt, ua, us)
        want = plain_verify(tokens, cud, qd, pt, ua, us, False)
        assert status == 0 and np.array_equal(emitted, want[0]) and np.array_equal(acc, want[1])
        for b in range(B):  # the last token and the accepted drafts stay in the cache
            keep = len(keys[b]) - k + int(acc[b])
            del keys[b][keep:], vals[b][keep:]
        lens.copy_(torch.tensor([len(x) for x in keys]))


class _Loop:
    """Four steps of a serving loop whose lengths, held blocks and free count are updated in place."""

    def __init__(self, seed):
        import torch

        self.B, self.T, H, Hkv, d, self.bs, cols = 300, 9000, 4, 2, 64, 16, 24
        rng = np.random.default_rng(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        P = self.B * 20
        self.new = [torch.tensor(rng.integers(0, 50 if s == 0 else 9, self.B), **i32) for s in range(4)]
        self.qkv = torch.from_numpy(rng.standard_normal((self.T, H + 2 * Hkv, d)).astype(np.float32)).cuda().bfloat16()
        self.kv = [torch.zeros(P, self.bs, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.table, self.free = torch.full((self.B, cols), -1, **i32), torch.arange(P, **i32)
        self.lens, self.held, self.count = torch.zeros(self.B, **i32), torch.zeros(self.B, **i32), torch.tensor([P], **i32)
        self.cu = torch.zeros(self.B + 1, **i32)
        self.out = [torch.zeros(self.T, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        self.lse = [torch.zeros(self.T, H, device="cuda") for _ in range(4)]
        self.maps = [torch.zeros(self.T, dtype=torch.int64, device="cuda") for _ in range(4)]
        self.q, k, v = self.qkv[:, :H], self.qkv[:, H:H + Hkv], self.qkv[:, H + Hkv:]
        self.k, self.v, self.d = k, v, d
        self.st, self.ws = pg.alloc_workspace_status(), pg.alloc_workspace_prefill(pg.shape_multi(self.q, self.kv[0], self.table))
        self.start = [x.clone() for x in self.state()]

    def state(self):
        return [*self.kv, self.table, self.free, self.lens, self.held, self.count]

    def results(self):
        return [*self.state(), *self.out, *self.lse, *self.maps]

    def reset(self):
        for x, y in zip(self.state(), self.start):
            x.copy_(y)
        for x in self.out + self.lse + self.maps:
            x.fill_(7)

    def steps(self, between=lambda: None):
        for s in range(4):
            pg.pa_build_slots(self.lens, self.new[s], self.held, self.table, self.free, self.count, self.bs, self.cu,
                              self.maps[s], self.lens, self.held, self.count, self.st)
            between()
            pg.pa_cache_write(self.k, self.v, self.maps[s], *self.kv, self.st)
            between()
            pg.pa_prefill(self.q, self.cu, True, *self.kv, self.table, self.lens, self.d ** -0.5, self.out[s], self.lse[s],
                          self.ws)
            between()


@pytest.mark.gpu
def test_steps_in_place_and_in_flight_together_give_what_they_give_one_by_one():
    """Lengths, held blocks and the free count are each call's inputs and outputs, and every call follows the one before
    without a wait of the host: on one stream, in a replayed graph, and two loops on two streams."""
    import torch

    loops = [_Loop(seed) for seed in (1, 2)]
    want = []
    for x in loops:
        x.reset()
        x.steps(torch.cuda.synchronize)
        want.append([t.clone() for t in x.results()])
        assert int(x.lens.sum()) == sum(int(n.sum()) for n in x.new)

    def compare():
        torch.cuda.synchronize()
        for x, w in zip(loops, want):
            assert pg.pa_read_status(x.st) == 0 and pg.pa_read_status(x.ws) == 0
            for a, b in zip(x.results(), w):
                assert torch.equal(a, b)

    streams, graphs = [torch.cuda.Stream() for _ in loops], []
    for _ in range(10):
        for x in loops:
            x.reset()
        torch.cuda.synchronize()
        for x, s in zip(loops, streams):
            with torch.cuda.stream(s):
                x.steps()
        compare()
    for x, s in zip(loops, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            x.steps()
        graphs.append(g)
    for _ in range(10):
        for x in loops:
            x.reset()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        compare()


@pytest.mark.gpu
def test_blocks_whose_offsets_pass_32_bits():
    """Pools of 4.9 10^9 elements each, blocks at their end: tables, slots, written rows and attention over them."""
    import torch

    P, bs, Hkv, d, n, H = 300000, 16, 8, 128, 333, 16
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    kc, vc = (torch.empty(P, bs, Hkv, d, dtype=torch.float16, device="cuda") for _ in range(2))
    free, count = torch.zeros(P, **i32), torch.tensor([40], **i32)
    free[:40] = P - 1 - 3 * torch.arange(40, device="cuda")
    table, new, held = torch.full((1, 64), -1, **i32), torch.tensor([n], **i32), torch.zeros(1, **i32)
    lens, cu, slots = torch.zeros(1, **i32), torch.zeros(2, **i32), torch.zeros(n, dtype=torch.int64, device="cuda")
    st = pg.alloc_workspace_status()
    pg.pa_build_slots(lens, new, held, table, free, count, bs, cu, slots, lens, held, count, st)
    ids = P - 1 - 3 * np.arange(39, 39 - 21, -1)  # from the top of the stack
    assert table[0, :21].tolist() == ids.tolist() and count.item() == 19
    assert slots.tolist() == [int(ids[i // bs]) * bs + i % bs for i in range(n)]
    k, v = (torch.randn(n, Hkv, d, generator=g, device="cuda").half() for _ in range(2))
    pg.pa_cache_write(k, v, slots, kc, vc, st)
    assert torch.equal(kc.view(-1, Hkv, d)[slots], k) and torch.equal(vc.view(-1, Hkv, d)[slots], v)
    q = torch.randn(n, H, d, generator=g, device="cuda").half()
    out, ws = torch.zeros_like(q), pg.alloc_workspace_prefill(pg.shape_multi(q, kc, table))
    pg.pa_prefill(q, cu, True, kc, vc, table, lens, d ** -0.5, out, None, ws)
    # the same rows in a pool of their own blocks
    small = [torch.zeros(21, bs, Hkv, d, dtype=torch.float16, device="cuda") for _ in range(2)]
    for pool, rows in zip(small, (k, v)):
        pool.view(-1, Hkv, d)[:n] = rows
    want = torch.zeros_like(q)
    pg.pa_prefill(q, cu, True, *small, torch.arange(21, **i32)[None].contiguous(), lens, d ** -0.5, want, None, ws)
    assert torch.equal(out, want)
    x = torch.einsum("qhd,khd->hqk", q.double(), k.double().repeat_interleave(H // Hkv, 1)) * d ** -0.5
    x.masked_fill_(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -float("inf"))
    w, vd = x.softmax(-1), v.double().repeat_interleave(H // Hkv, 1)
    ref, A = torch.einsum("hqk,khd->qhd", w, vd), torch.einsum("hqk,khd->qhd", w, vd.abs())
    u = 2.0 ** -11  # a rounding of the output, one of each weight; subnormal weights; fp32's exponentials and sums
    assert ((out.double() - ref).abs() <= u * (ref.abs() * (1 + u) + A) + n * 2.0 ** -25 * 5 + 2.0 ** -13 * A + 2.0 ** -24).all()
    assert pg.pa_read_status(st) == 0 and pg.pa_read_status(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "float16"])
def test_verify_the_largest_vocabulary(dtype):
    import torch

    V = pg.PA_MAX_VOCAB
    p = torch.full((3, V), 2.0 ** -24, dtype=getattr(torch, dtype), device="cuda")  # sums to 1
    us = torch.tensor([0.0, 0.5, 1 - 2.0 ** -24], device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    tokens, acc = torch.full((3,), -9, dtype=torch.int32, device="cuda"), torch.full((3,), -9, dtype=torch.int32, device="cuda")
    ws = pg.alloc_workspace_verify(3, V)
    pg.pa_verify_drafts(none, torch.zeros(4, dtype=torch.int32, device="cuda"), None, p, none.float(), us, tokens, acc, ws)
    assert pg.pa_read_status(ws) == 0
    assert tokens.tolist() == [0, V // 2, V - 1] and acc.tolist() == [0, 0, 0]
