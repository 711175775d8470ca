"""Host side of the packed attention and rotary calls (no GPU): the planner's
item table covers every visible (query, key) pair once, partial results and
their merge agree, and wrong arguments are refused before any launch."""
import ctypes
import math
import random

import numpy as np
import pytest

from token_level_sparse_pddp_b200 import build as tlsp_build


@pytest.fixture(scope="module")
def T():
    tlsp_build.build()
    from token_level_sparse_pddp_b200 import tlsp
    tlsp.lib()
    return tlsp


class Rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class RotaryTensor(ctypes.Structure):
    _fields_ = ([("src", ctypes.c_void_p), ("dst", ctypes.c_void_p)]
                + [(n, ctypes.c_int64) for n in ("in_batch", "in_token", "in_head", "out_batch",
                                                 "out_token", "out_head")]
                + [("heads", ctypes.c_int32)])


class RotaryCall(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("tokens", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("positions_64", ctypes.c_int32), ("positions", ctypes.c_void_p),
                ("position_axis", ctypes.c_int64), ("position_batch", ctypes.c_int64)]


def make(T, q, kv, heads=4, kv_heads=2, d=128, dtype=1, causal=1, prefix=0, starts=None):
    desc = T.PackedDesc(len(q), heads, kv_heads, d, dtype, causal, prefix)
    data = T.PackedPlanData()
    aq, akv = (ctypes.c_int32 * len(q))(*q), (ctypes.c_int32 * len(kv))(*kv)
    ast = None if starts is None else (ctypes.c_int64 * len(starts))(*starts)
    L = T.lib()
    code = L.tlsp_packed_make_plan(ctypes.byref(desc), aq, akv, ast, None, 0, ctypes.byref(data))
    assert code in (T.TLSP_OK, T.TLSP_ERR_WORKSPACE), code
    buf = (ctypes.c_char * max(1, data.items_bytes))()
    assert L.tlsp_packed_make_plan(ctypes.byref(desc), aq, akv, ast, buf, data.items_bytes,
                                   ctypes.byref(data)) == T.TLSP_OK
    table = np.frombuffer(bytes(buf)[:data.items_bytes], dtype=np.int32).reshape(-1, 8)
    n1 = data.tile_items
    n2 = n1 + data.token_items
    n3 = n2 + data.token_segments
    assert len(table) == n3 + data.merge_items and data.cluster in (1, 2, 4, 8)
    return data, table[:n1], token_work(table[n1:n2], table[n2:n3], dtype), table[n3:]


def token_work(tokens, segments, dtype):
    """Token items as rows (q0, nt, kv0, kv_n, pre0, pre_n, diag, slot, counts): one for each
    segment (bf16; those of sequences that share an item cover part of its tokens), or as they
    are (fp32). `counts`: whether the row stands for the item's result."""
    if dtype == 0:
        assert len(segments) == 0
        return [list(t) + [1] for t in tokens.tolist()]
    out, used = [], []
    for q0, nt, seg0, nseg, slot, *_ in tokens.tolist():
        assert 0 <= nseg <= 32
        used += range(seg0, seg0 + nseg)
        out.append([q0, nt, 0, 0, 0, 0, 0, slot, 1])
        for k0, n, tok0, ntok, diag, prefix, *_ in segments[seg0:seg0 + nseg].tolist():
            assert n > 0 and tok0 >= 0 and ntok >= 1 and tok0 + ntok <= nt
            out.append([q0 + tok0, ntok] + ([0, 0, k0, n, 0] if prefix else [k0, n, 0, 0, diag])
                       + [-1, 0])
            assert not prefix or (tok0, ntok) == (0, nt)
    assert sorted(used) == list(range(len(segments)))
    return out


def check_cover(T, q, kv, heads, kv_heads, d, dtype, causal, prefix, starts=None):
    data, tiles, tokens, merges = make(T, q, kv, heads, kv_heads, d, dtype, causal, prefix, starts)
    g = heads // kv_heads
    rows = sum(q)
    assert data.q_rows == rows and len(merges) == data.merge_items
    where = []  # of each token: own keys from, keys, how many of them it sees
    end = 0
    for s, (n, m) in enumerate(zip(q, kv)):
        k0 = end if starts is None else starts[s]
        end += m
        where += [(k0, max(0, min(m, m - n + i + 1)) if causal else m) for i in range(n)]
    own = [[] for _ in range(rows)]   # (first key, number) ranges of each token
    pre = [[] for _ in range(rows)]
    slots = {}                        # partial row -> token
    direct = [0] * rows
    for kind, table in (("tile", tiles), ("token", tokens)):
        rows_of = table if kind == "token" else [t + [1] for t in table.tolist()]
        for q0, nt, kv0, kv_n, pre0, pre_n, diag, slot, counts in rows_of:
            assert nt >= 1 and q0 >= 0 and q0 + nt <= rows
            assert nt * g <= (16 if kind == "token" else 256)
            assert 0 <= pre0 and pre0 + pre_n <= prefix and pre_n >= 0 and kv_n >= 0 and kv0 >= 0
            assert kv_n == 0 or kv0 + kv_n <= data.kv_rows
            assert -(1 << 30) <= diag <= kv_n
            for i in range(nt):
                t = q0 + i
                seen = max(0, min(kv_n, diag + i + 1))
                if seen:
                    own[t].append((kv0, seen))
                if pre_n:
                    pre[t].append((pre0, pre_n))
                if not counts:
                    continue
                if slot < 0:
                    direct[t] += 1
                else:
                    assert slot + i < data.part_rows and slot + i not in slots
                    slots[slot + i] = t
    merged = [0] * rows
    used = set()
    for q0, nt, a, ap, ast, b, bp, bst in merges.tolist():
        assert 1 <= nt and q0 + nt <= rows
        for i in range(nt):
            merged[q0 + i] += 1
            for base, parts, stride in ((a, ap, ast), (b, bp, bst)):
                for p in range(parts):
                    r = base + p * stride + i
                    assert slots[r] == q0 + i and r not in used
                    used.add(r)
    assert used == set(slots)
    for t in range(rows):
        assert (direct[t], merged[t]) in ((1, 0), (0, 1)), (t, direct[t], merged[t])

        def joined(ranges):
            at = None
            for a, n in sorted(ranges):
                assert at is None or a == at
                at = a + n
            return (min(a for a, _ in ranges), sum(n for _, n in ranges)) if ranges else (0, 0)
        assert joined(pre[t]) == (0, prefix)
        k0, seen = where[t]
        got = joined(own[t])
        assert got[1] == seen and (seen == 0 or got[0] == k0), (t, got, where[t])
    return data


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("case", [
    dict(q=[1], kv=[1]), dict(q=[1], kv=[0]), dict(q=[0], kv=[5]), dict(q=[0, 0], kv=[0, 0]),
    dict(q=[1] * 9, kv=[900, 1, 4700, 0, 128, 129, 127, 2000, 64]),
    dict(q=[300, 0, 1, 7, 2], kv=[298, 3, 1, 500, 0]),
    dict(q=[5000], kv=[9000]), dict(q=[17, 33], kv=[40000, 17]),
    dict(q=[1] * 3 + [40] + [1] * 30, kv=[10] * 34, prefix=3001),
    dict(q=[1, 2, 3], kv=[0, 0, 3], prefix=130), dict(q=[700, 1, 650], kv=[700, 9, 650], prefix=999),
    dict(q=[3, 4], kv=[5, 9], causal=0), dict(q=[600], kv=[100], causal=0),
    dict(q=[600], kv=[100]), dict(q=[5, 1], kv=[5, 70], starts=[1000, 0]),
])
def test_plan_covers_every_pair_once(T, case, dtype):
    for heads, kv_heads in ((1, 1), (6, 2), (5, 1), (7, 1), (64, 1), (12, 12)):
        check_cover(T, case["q"], case["kv"], heads, kv_heads, 128, dtype, case.get("causal", 1),
                    case.get("prefix", 0), case.get("starts"))


def test_plan_covers_random_batches(T):
    r = random.Random(4)
    for _ in range(60):
        n = r.randint(1, 30)
        q = [r.choice([0, 1, 1, 1, 2, r.randint(3, 700)]) for _ in range(n)]
        kv = [r.choice([0, a, a + r.randint(0, 3000), r.randint(0, 700)]) for a in q]
        hk = r.choice([1, 2, 8])
        check_cover(T, q, kv, hk * r.choice([1, 3, 5, 8, 16, 17]), hk, r.choice([64, 128]),
                    r.randint(0, 1), r.randint(0, 1), r.choice([0, 0, 1, 127, 5000, 30000]))


def test_short_sequences_share_a_long_prefix(T):
    """Sequences of 17 to 64 rows beside others: their rows take the prefix together."""
    r = random.Random(8)
    for _ in range(40):
        heads, kv_heads = r.choice([(8, 1), (6, 2), (12, 12), (40, 8), (17, 1), (64, 1)])
        q = [r.choice([0, 1, 2, 3, 5, 9, r.randint(1, 90)]) for _ in range(r.randint(1, 24))]
        kv = [r.choice([0, n, n + r.randint(0, 400), r.randint(0, 9)]) for n in q]
        check_cover(T, q, kv, heads, kv_heads, 128, 1, r.randint(0, 1), r.choice([2047, 2048, 9000]))
    q = [3] * 16                                        # 24 rows each, three in a query tile
    _, tiles, _, _ = make(T, q, [40] * 16, heads=8, kv_heads=1, prefix=15329)
    assert sum(-(-int(t[5]) // 128) for t in tiles) < 2 * 120 + 30  # two items' steps, cut


def test_long_caches_are_split(T):
    """A single token behind a long cache is shared out over many CTAs."""
    data, tiles, tokens, merges = make(T, [1], [60000], heads=12, kv_heads=4)
    assert len(tiles) == 0 and data.token_items * data.cluster * 4 >= 100 and len(merges) == 1
    data, tiles, tokens, merges = make(T, [100], [60000], heads=12, kv_heads=4)
    assert len(tokens) == 0 and len(tiles) * 4 >= 100


def test_plan_refusals(T):
    L, E = T.lib(), T.TLSP_ERR_INVALID_ARG
    data = T.PackedPlanData()
    one = (ctypes.c_int32 * 1)(1)
    neg = (ctypes.c_int32 * 1)(-1)
    buf = (ctypes.c_char * 4096)()

    def plan(n=1, h=4, hk=2, d=128, dt=1, causal=1, pre=0, q=one, kv=one, st=None, to=buf, size=4096):
        desc = T.PackedDesc(n, h, hk, d, dt, causal, pre)
        return L.tlsp_packed_make_plan(ctypes.byref(desc), q, kv, st, to, size, ctypes.byref(data))
    assert plan() == T.TLSP_OK
    for bad in (dict(n=0), dict(h=0), dict(hk=0), dict(h=5), dict(d=96), dict(dt=7), dict(causal=2),
                dict(pre=-1), dict(q=None), dict(kv=None), dict(q=neg), dict(kv=neg),
                dict(st=(ctypes.c_int64 * 1)(-5))):
        assert plan(**bad) == E, bad
    assert plan(h=130, hk=2) == T.TLSP_ERR_UNSUPPORTED          # 65 heads share one
    assert plan(st=(ctypes.c_int64 * 1)(1 << 31)) == T.TLSP_ERR_UNSUPPORTED
    huge = (ctypes.c_int32 * 1)(0x7ffffe00)                     # too many items, not too few bytes
    assert plan(h=64, hk=1, q=huge, kv=huge, to=None, size=0) == T.TLSP_ERR_UNSUPPORTED
    assert plan(size=16) == T.TLSP_ERR_WORKSPACE and data.items_bytes > 16
    assert plan(to=None, size=0) == T.TLSP_ERR_WORKSPACE
    assert L.tlsp_packed_make_plan(None, one, one, None, buf, 4096, ctypes.byref(data)) == E


def test_attention_refusals(T):
    """Nothing is launched by a call that fails validation."""
    L, E, E_WS = T.lib(), T.TLSP_ERR_INVALID_ARG, T.TLSP_ERR_WORKSPACE
    before = L.tlsp_launch_count()
    data, *_ = make(T, [3, 1], [3, 900], heads=4, kv_heads=2)
    pdata, *_ = make(T, [3, 1], [3, 900], heads=4, kv_heads=2, prefix=77)
    p = ctypes.c_void_p(0x10000)      # never dereferenced

    def rows(heads, ptr=0x10000, rs=None, hs=128):
        return ctypes.byref(Rows(ptr, heads * 128 if rs is None else rs, hs))
    ok = dict(plan=ctypes.byref(data), items=p, Q=rows(4), K=rows(2), V=rows(2), O=rows(4), lse=None,
              scale=0.0, ws=p, n=1 << 40)

    def call(**kw):
        a = {**ok, **kw}
        return L.tlsp_packed_attention(a["plan"], a["items"], a["Q"], a["K"], a["V"], a["O"],
                                       a["lse"], a["scale"], a["ws"], a["n"], None)
    for bad in (dict(plan=None), dict(items=None), dict(items=ctypes.c_void_p(0x10008)), dict(Q=None),
                dict(K=None), dict(V=None), dict(O=None), dict(Q=rows(4, 0)), dict(Q=rows(4, 0x10008)),
                dict(K=rows(2, rs=0)), dict(K=rows(2, hs=0)), dict(V=rows(2, rs=260)),
                dict(V=rows(2, hs=132)), dict(O=rows(4, hs=64)), dict(ws=None),
                dict(O=rows(4, rs=256, hs=128)), dict(O=rows(4, rs=128, hs=384)),
                dict(ws=ctypes.c_void_p(0x10004)), dict(scale=math.inf), dict(scale=math.nan),
                dict(lse=ctypes.c_void_p(0x10002)), dict(plan=ctypes.byref(pdata))):
        assert call(**bad) == E, bad
    assert call(n=255) == E_WS and call(n=data.ws_bytes - 1) == E_WS

    def prefix(plan=ctypes.byref(pdata), Kp=rows(2), Vp=rows(2)):
        return L.tlsp_prefix_attention(plan, p, ok["Q"], Kp, Vp, ok["K"], ok["V"], ok["O"], None,
                                       0.0, p, 64, None)
    assert prefix() == E_WS
    assert prefix(Kp=None) == E and prefix(Vp=None) == E and prefix(Kp=rows(2, 0x10004)) == E
    assert prefix(plan=ctypes.byref(data)) == E
    # no queries: nothing to launch, and that is no error
    empty, *_ = make(T, [0], [9])
    assert call(plan=ctypes.byref(empty)) == T.TLSP_OK
    assert L.tlsp_launch_count() == before


# ------------------------------------------------------------------ rotary

@pytest.mark.parametrize("kw", [
    dict(), dict(rotary_dim=64), dict(base=500000.0, scaling="linear", factor=4.0),
    dict(scaling="base", factor=8.0), dict(scaling="ramp", factor=16.0, original_len=4096),
    dict(sections=(22, 21, 21)), dict(sections=(62, 1, 1), scaling="base", factor=2.0),
    dict(layout="interleaved", rotary_dim=2),
])
def test_rotary_frequencies(T, kw):
    """Turns per position, modulo 1, against the formulas in 64-bit arithmetic."""
    plan = T.RotaryPlan(128, **kw)
    r = kw.get("rotary_dim", 128)
    sec = kw.get("sections", (r // 2,))
    f, i = kw.get("factor", 1.0), 0
    for a, s in enumerate(sec):
        for e in range(s):
            b = kw.get("base", 10000.0)
            if kw.get("scaling") == "base" and s > 1:
                b *= f ** (s / (s - 1))
            w = b ** (-e / s)
            if kw.get("scaling") == "linear":
                w /= f
            if kw.get("scaling") == "ramp":
                c = min(1, max(0, (kw["original_len"] * w / (2 * math.pi) - 1) / 31))
                w = c * w + (1 - c) * w / f
            got = plan.data.turns[i] / 2.0 ** 64
            assert abs(got - w / (2 * math.pi)) <= 4e-16 and plan.data.axis[i] == a
            i += 1
    amp = 1 + 0.1 * math.log(16) if kw.get("scaling") == "ramp" else 1.0
    assert abs(plan.data.amplitude - amp) <= 2 ** -23 * amp


def test_struct_layouts(T):
    """The bytes the binding packs are the structs' layouts."""
    assert T._ROTARY_TENSOR.size == ctypes.sizeof(RotaryTensor)
    assert T._ROTARY_CALL.size == ctypes.sizeof(RotaryCall) and T._ROWS.size == ctypes.sizeof(Rows)
    a = T._ROTARY_TENSOR.pack(*range(1, 10))
    assert a == bytes(RotaryTensor(*range(1, 10)))
    assert T._ROTARY_CALL.pack(*range(1, 8)) == bytes(RotaryCall(*range(1, 8)))


def test_rotary_refusals(T):
    for kw in (dict(head_dim=100), dict(head_dim=264), dict(head_dim=0), dict(rotary_dim=63),
               dict(rotary_dim=130), dict(rotary_dim=0), dict(base=0.0), dict(base=math.inf),
               dict(base=math.nan), dict(factor=0.5), dict(factor=math.nan), dict(sections=(1, 2)),
               dict(sections=(65, -1)), dict(scaling="ramp", factor=2.0),
               dict(scaling="ramp", factor=2.0, original_len=100, fast=1.0, slow=1.0)):
        with pytest.raises(T.TlspError) as e:
            T.RotaryPlan(**{"head_dim": 128, **kw})
        assert e.value.code == T.TLSP_ERR_INVALID_ARG, kw
    for kw in (dict(layout="x"), dict(scaling="x"), dict(amplitude=0.0), dict(amplitude=math.nan),
               dict(sections=()), dict(sections=(8,) * 8)):
        with pytest.raises(ValueError):
            T.RotaryPlan(128, **kw)
    L, E = T.lib(), T.TLSP_ERR_INVALID_ARG
    before = L.tlsp_launch_count()
    plan = T.RotaryPlan(128).data

    def call(c=None, q=None, k=None, backward=0, plan=plan):
        c = RotaryCall(1, 4, 1, 0, 0x10000, 0, 0) if c is None else c
        q = RotaryTensor(0x10000, 0x20000, 0, 128, 512, 0, 128, 512, 2) if q is None else q
        return L.tlsp_rotary(ctypes.byref(plan), ctypes.byref(c), ctypes.byref(q),
                             None if k is None else ctypes.byref(k), backward, None)
    assert call(c=RotaryCall(1, 0, 1, 0, 0x10000, 0, 0)) == T.TLSP_OK      # no tokens
    for c in (RotaryCall(-1, 4, 1, 0, 0x10000, 0, 0), RotaryCall(1, -4, 1, 0, 0x10000, 0, 0),
              RotaryCall(1, 4, 7, 0, 0x10000, 0, 0), RotaryCall(1, 4, 1, 0, 0, 0, 0),
              RotaryCall(1, 4, 1, 1, 0x10004, 0, 0)):
        assert call(c=c) == E
    for q in (RotaryTensor(0, 0x20000, 0, 128, 512, 0, 128, 512, 2),
              RotaryTensor(0x10000, 0, 0, 128, 512, 0, 128, 512, 2),
              RotaryTensor(0x10001, 0x20000, 0, 128, 512, 0, 128, 512, 2),
              RotaryTensor(0x10000, 0x10000, 0, 128, 512, 0, 256, 512, 2),   # in place, other strides
              RotaryTensor(0x10000, 0x20000, 0, 128, 512, 0, 128, 512, 0)):
        assert call(q=q) == E and call(k=q) == E
    assert call(backward=2) == E
    broken = T.RotaryPlan(128).data
    broken.axis[3] = 1
    assert call(plan=broken) == E
    assert L.tlsp_launch_count() == before


# ------------------------------------------------------------------ values out of range

@pytest.mark.parametrize("start", [2 ** 63 - 1, 2 ** 63 - 2, 2 ** 62, 0x7ffffeff - 24])
@pytest.mark.parametrize("dtype", [0, 1])
def test_starts_whose_end_is_out_of_range(T, start, dtype):
    """Sequences that would end behind the largest key row, sums that do not fit included."""
    data = T.PackedPlanData()
    desc = T.PackedDesc(1, 4, 2, 128, dtype, 1, 0)
    buf = (ctypes.c_char * 65536)()
    q, kv = (ctypes.c_int32 * 1)(20), (ctypes.c_int32 * 1)(25)

    def plan(start):
        return T.lib().tlsp_packed_make_plan(ctypes.byref(desc), q, kv, (ctypes.c_int64 * 1)(start),
                                             buf, len(buf), ctypes.byref(data))
    assert plan(start) == T.TLSP_ERR_UNSUPPORTED
    assert plan(0x7ffffeff - 25) == T.TLSP_OK and data.kv_rows == 0x7ffffeff
    desc.prefix_len = 0x7fffff00
    assert plan(0) == T.TLSP_ERR_UNSUPPORTED


# ------------------------------------------------------------------ shared memory

def test_outputs_that_share_memory(T):
    """Nothing is launched by a call whose output, lse or workspace lies on what it reads or on
    each other."""
    L = T.lib()
    before = L.tlsp_launch_count()
    data, *_ = make(T, [3, 1], [3, 900], heads=4, kv_heads=2, prefix=50)
    base, M = 1 << 32, 1 << 24                              # addresses, never dereferenced
    at = dict(Q=base, Kp=base + M, Vp=base + 2 * M, K=base + 3 * M, V=base + 4 * M, O=base + 5 * M,
              lse=base + 6 * M, ws=base + 7 * M)

    def call(strides=(512, 128), **kw):
        p = {**at, **kw}
        rows = {n: ctypes.byref(Rows(p[n], *((256, 128) if n in ("K", "V", "Kp", "Vp") else strides)))
                for n in ("Q", "Kp", "Vp", "K", "V", "O")}
        return L.tlsp_prefix_attention(
            ctypes.byref(data), ctypes.c_void_p(base + 8 * M), rows["Q"], rows["Kp"], rows["Vp"],
            rows["K"], rows["V"], rows["O"], ctypes.c_void_p(p["lse"]), 0.0, ctypes.c_void_p(p["ws"]),
            data.ws_bytes, None)
    for name, last in (("Q", 4 * 1024), ("Kp", 50 * 512), ("Vp", 50 * 512), ("K", 903 * 512),
                       ("V", 903 * 512)):
        assert call(O=at[name]) == T.TLSP_ERR_INVALID_ARG, name
        assert call(O=at[name] + last - 16) == T.TLSP_ERR_INVALID_ARG, name
        assert call(lse=at[name] + last - 4) == T.TLSP_ERR_INVALID_ARG, name
        assert call(ws=at[name] - data.ws_bytes + 16) == T.TLSP_ERR_INVALID_ARG, name
    assert call(lse=at["O"] + 16) == T.TLSP_ERR_INVALID_ARG
    assert call(ws=at["O"]) == T.TLSP_ERR_INVALID_ARG
    assert call(lse=at["ws"] + data.ws_bytes - 4) == T.TLSP_ERR_INVALID_ARG   # its last bytes
    # a part of the same channels of one wider tensor
    assert call(strides=(1024, 256), O=at["Q"] + 128) == T.TLSP_ERR_INVALID_ARG
    assert L.tlsp_launch_count() == before


def test_rotary_outputs_that_share_memory(T):
    """An output is its own input or lies apart from everything else."""
    L = T.lib()
    before = L.tlsp_launch_count()
    plan = T.RotaryPlan(128).data
    A, B, C, D = (x << 32 for x in range(1, 5))             # addresses, never dereferenced
    token = 4 * 128

    def call(q, k=None, batch=1, tokens=40):
        c = RotaryCall(batch, tokens, 1, 0, 0x10000, 0, 0)
        return L.tlsp_rotary(ctypes.byref(plan), ctypes.byref(c), ctypes.byref(q),
                             None if k is None else ctypes.byref(k), 0, None)

    def t(src, dst, src_strides=(0, token, 128), dst_strides=(0, token, 128), heads=4):
        return RotaryTensor(src, dst, *src_strides, *dst_strides, heads)
    for q, k in (
            (t(A, A + 256), None), (t(A, A + 2 * token), None), (t(A, A - 2 * token), None),
            (t(A, A + 39 * 2 * token), None),               # the last token's row
            (t(A, A, dst_strides=(0, 128, 40 * 128)), None),
            (t(A, B, dst_strides=(0, token, 64)), None),    # heads on each other
            (t(A, B, dst_strides=(0, 0, 128)), None), (t(A, B, dst_strides=(0, 256, 128)), None),
            (t(A, B), t(C, B)), (t(A, B), t(B, C)), (t(A, B), t(B, A)), (t(A, A), t(A, A)),
            (t(A, A), t(C, A + 256)), (t(A, C), t(C + 16, D))):
        assert call(q, k) == T.TLSP_ERR_INVALID_ARG, (q.src, q.dst)
    assert call(t(A, B, dst_strides=(token, token, 128)), batch=2) == T.TLSP_ERR_INVALID_ARG
    assert L.tlsp_launch_count() == before


@pytest.mark.parametrize("scale", [2.4e38, -3e38, 3.4e38])
def test_scales_beyond_the_range_of_the_exponent(T, scale):
    """Kernels work with scale log2(e): its product has to be finite too."""
    L = T.lib()
    data, *_ = make(T, [3, 1], [3, 900], heads=4, kv_heads=2)
    rows = [ctypes.byref(Rows(x << 32, h * 128, 128)) for x, h in ((1, 4), (2, 2), (3, 2), (4, 4))]
    assert L.tlsp_packed_attention(ctypes.byref(data), ctypes.c_void_p(5 << 32), *rows, None, scale,
                                   ctypes.c_void_p(6 << 32), data.ws_bytes, None) == \
        T.TLSP_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", [0, 1])
def test_merges_that_no_grid_holds(T, dtype):
    """More heads than the merging kernel's grid takes are refused by the plan, not by a call
    that has launched part of its work."""
    data = T.PackedPlanData()
    q, kv = (ctypes.c_int32 * 9)(*[1] * 9), (ctypes.c_int32 * 9)(*[5] * 9)

    def plan(heads, kv_heads):
        desc = T.PackedDesc(9, heads, kv_heads, 64, dtype, 1, 999)
        return T.lib().tlsp_packed_make_plan(ctypes.byref(desc), q, kv, None, None, 0,
                                             ctypes.byref(data))
    assert plan(4 * 65535, 65535) == T.TLSP_ERR_WORKSPACE and data.merge_items == 9
    assert plan(5 * 65535, 65535) == T.TLSP_ERR_UNSUPPORTED


def test_plans_of_many_sequences_take_time_in_proportion(T):
    """Single tokens by the ten thousand behind a prefix: eight times as many take well below
    sixty-four times as long (each the best of a few)."""
    import time

    def seconds(n, times):
        q, kv = (ctypes.c_int32 * n)(*[1] * n), (ctypes.c_int32 * n)(*[5] * n)
        desc, data, best = T.PackedDesc(n, 16, 1, 64, 1, 1, 1), T.PackedPlanData(), 1e9
        for _ in range(times):
            start = time.perf_counter()
            assert T.lib().tlsp_packed_make_plan(ctypes.byref(desc), q, kv, None, None, 0,
                                                 ctypes.byref(data)) == T.TLSP_ERR_WORKSPACE
            best = min(best, time.perf_counter() - start)
        assert data.token_items == n
        return best
    assert seconds(160000, 2) < 30 * seconds(20000, 5)
