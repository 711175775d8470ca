"""Packed causal attention with grouped heads and shared-prefix attention on the
GPU against the definition in 64 bits, within bounds that follow from the
kernels' arithmetic (tests/packed_ref.py)."""
import random

import pytest
import torch

from tests.packed_ref import Ref

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def T():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from token_level_sparse_pddp_b200 import build, tlsp
    build.build()
    return tlsp


def inputs(q, kv, heads, kv_heads, d, dtype, prefix=0, seed=0, rows=None, kv_rows=None, gain=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(n, h, a=1.0):
        return (torch.randn((n, h, d), generator=g, device="cuda") * a).to(dtype)
    Q = rand(sum(q) if rows is None else rows, heads, gain)
    n = sum(kv) if kv_rows is None else kv_rows
    K, V = rand(n, kv_heads), rand(n, kv_heads)
    Kp, Vp = (rand(prefix, kv_heads), rand(prefix, kv_heads)) if prefix else (None, None)
    return Q, K, V, Kp, Vp


def attend(T, Q, K, V, Kp, Vp, plan, ws, **kw):
    lse = torch.full(Q.shape[:2], 7.0, device="cuda")
    if Kp is not None:
        O = T.prefix_attention(Q, Kp, Vp, K, V, plan, ws, lse=lse, **kw)
    else:
        O = T.packed_attention(Q, K, V, plan, ws, lse=lse, **kw)
    return O, lse


def run(T, q, kv, heads=4, kv_heads=2, d=128, dtype=BF16, causal=True, prefix=0, starts=None,
        scale=None, tensors=None):
    Q, K, V, Kp, Vp = tensors if tensors is not None else inputs(q, kv, heads, kv_heads, d, dtype, prefix)
    plan = T.PackedPlan(q, kv, heads, kv_heads, d, dtype, causal, prefix, starts)
    ws = plan.workspace()
    O, lse = attend(T, Q, K, V, Kp, Vp, plan, ws, scale=scale)
    torch.cuda.synchronize()
    assert ws.status() == T.TLSP_OK
    Ref(Q, K, V, q, kv, starts, causal, Kp, Vp, scale).check(O, lse)
    return O, lse


HEADS = [(1, 1), (4, 4), (6, 2), (5, 1), (16, 2), (14, 2), (64, 1), (51, 3)]


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (FP32, 128), (FP32, 64)])
@pytest.mark.parametrize("heads,kv_heads", HEADS)
def test_ragged_prompts(T, dtype, d, heads, kv_heads):
    q = [1, 0, 129, 300, 2, 64, 17]
    kv = [1, 4, 129, 300, 2, 64, 17]
    run(T, q, kv, heads, kv_heads, d, dtype)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (FP32, 128), (FP32, 64)])
@pytest.mark.parametrize("heads,kv_heads", HEADS)
def test_single_tokens(T, dtype, d, heads, kv_heads):
    run(T, [1] * 8, [1, 2, 15, 16, 17, 127, 129, 1500], heads, kv_heads, d, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,m", [(1, 0), (5, 0), (200, 0), (7, 3), (300, 40), (130, 129), (129, 2)])
def test_rows_that_see_nothing(T, dtype, n, m):
    O, lse = run(T, [n, 3], [m, 3], dtype=dtype)
    empty = max(0, n - m)
    assert (O[:empty] == 0).all() and (lse[:empty] == -torch.inf).all()
    assert torch.isfinite(O).all()


@pytest.mark.parametrize("n", [1, 2, 3, 8, 31, 63, 64, 65, 127, 128, 129, 255, 256, 257, 513])
@pytest.mark.parametrize("past", [0, 1, 127, 128, 400])
def test_lengths_around_tiles(T, n, past):
    run(T, [n], [n + past], 3, 1, 128, BF16)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (FP32, 128)])
def test_long_cache_split_and_merged(T, dtype, d):
    run(T, [1, 3, 1], [20011, 5000, 100], 6, 2, d, dtype)      # token items
    run(T, [33], [9001], 6, 2, d, dtype)                       # tile items
    run(T, [300, 2], [7000, 6000], 3, 3, d, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("q,kv", [([3, 200, 1], [50, 100, 700]), ([600], [77]), ([1, 2], [0, 3])])
def test_without_causal_mask(T, dtype, q, kv):
    run(T, q, kv, 6, 2, 128, dtype, causal=False)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (FP32, 128), (FP32, 64)])
@pytest.mark.parametrize("prefix", [1, 100, 128, 129, 1560, 6001])
@pytest.mark.parametrize("q,kv", [
    ([1] * 4, [1, 9, 130, 40]),
    ([1] * 40, [5 + 3 * i for i in range(40)]),
    ([1, 300, 1, 2, 0, 150], [20, 300, 0, 2, 4, 400]),
    ([3, 2], [0, 1]),
])
def test_shared_prefix(T, dtype, d, prefix, q, kv):
    for heads, kv_heads in ((6, 2), (5, 1)):
        run(T, q, kv, heads, kv_heads, d, dtype, prefix=prefix)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(8, 1), (6, 2), (5, 5)])
@pytest.mark.parametrize("causal", [True, False])
def test_short_sequences_share_a_long_prefix(T, d, heads, kv_heads, causal):
    q = [3, 0, 1, 5, 8, 2, 3, 300, 4, 4, 90, 7, 1]
    kv = [3, 0, 500, 0, 8, 200, 3, 290, 4, 700, 95, 5, 0]
    run(T, q, kv, heads, kv_heads, d, BF16, causal, prefix=2100)


def test_prefix_without_own_keys(T):
    Q, _, _, Kp, Vp = inputs([1, 40], [0, 0], 4, 2, 128, BF16, prefix=300)
    plan = T.PackedPlan([1, 40], [0, 0], 4, 2, 128, BF16, False, 300)
    ws = plan.workspace()
    O = T.prefix_attention(Q, Kp, Vp, None, None, plan, ws)
    Ref(Q, None, None, [1, 40], [0, 0], None, False, Kp, Vp).check(O)
    assert ws.status() == T.TLSP_OK


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_given_scale_and_large_logits(T, dtype):
    """Keys that grow along the sequence raise the running maximum again and again."""
    q, kv = [400, 1], [400, 900]
    for scale in (0.3, -0.2):
        run(T, q, kv, 6, 2, 128, dtype, scale=scale)
    Q, K, V, _, _ = inputs(q, kv, 6, 2, 128, dtype, gain=1.0)
    K *= torch.linspace(0.1, 12.0, K.shape[0], device="cuda")[:, None, None].to(dtype)
    run(T, q, kv, 6, 2, 128, dtype, tensors=(Q, K, V, None, None))
    K = K.flip(0).contiguous()
    run(T, q, kv, 6, 2, 128, dtype, tensors=(Q, K, V, None, None))
    # spikes for some rows of a warp only
    Q, K, V, _, _ = inputs(q, kv, 6, 2, 128, dtype, gain=0.5)
    K *= 0.5
    for key, c, rows, val in ((70, 3, slice(5, None, 8), 45.0), (228, 2, slice(3, None, 4), 50.0),
                              (300, 0, slice(1, None, 2), 40.0)):
        Q[rows, :, c] = 8.0
        K[key, :, c] = val
        K[400 + key, :, c] = val
    run(T, q, kv, 6, 2, 128, dtype, tensors=(Q, K, V, None, None))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("prefix", [0, 200])
def test_masked_keys_have_no_influence(T, dtype, prefix):
    """Infinities and NaN in K and V of keys that a row does not see, of other sequences and of
    room between sequences."""
    q, kv = [150, 1, 5, 300], [150, 70, 133, 290]
    starts = [3, 200, 300, 500]
    t = inputs(q, kv, 6, 2, 128, dtype, prefix, kv_rows=900)
    Q, K, V, Kp, Vp = t
    keep = torch.zeros(900, dtype=torch.bool, device="cuda")
    for s, m in zip(starts, kv):
        keep[s:s + m] = True
    for x, bad in ((K, float("nan")), (V, float("nan"))):
        x[~keep] = bad
    K[160], V[160] = float("inf"), float("-inf")     # behind the first sequence
    # seen by the later rows only
    V[3 + 140, :, 5] = float("nan")
    V[3 + 100, 0, 64:] = float("inf")
    V[500 + 289, :, 0] = float("-inf")
    V[300 + 131, 1, 9] = float("nan")                # last rows of a few-token sequence
    K[3 + 149] = float("nan")                        # the last key of a prompt
    plan = T.PackedPlan(q, kv, 6, 2, 128, dtype, True, prefix, starts)
    ws = plan.workspace()
    O, lse = attend(T, Q, K, V, Kp, Vp, plan, ws)
    assert ws.status() == T.TLSP_OK
    first = slice(0, 149)                            # the rows that do not see the NaN key
    ref = Ref(Q, torch.where(torch.isnan(K), 0.0, K), V, q, kv, starts, True, Kp, Vp)
    assert torch.isnan(O[149]).all() and torch.isnan(lse[149]).all()
    O[149], lse[149] = ref.O[149].to(dtype), ref.lse[149].float()
    ref.check(O, lse)
    assert torch.isfinite(O[first][:100]).all()


@pytest.mark.parametrize("d", [64, 128])
def test_sequences_that_share_an_item(T, d):
    """A few tokens of several sequences behind one prefix: each sees its own keys only, whatever
    the others' hold."""
    q, kv, starts = [1, 2, 0, 3, 1], [40, 17, 6, 3, 0], [100, 0, 60, 200, 0]
    Q, K, V, Kp, Vp = inputs(q, kv, 4, 2, d, BF16, 333, kv_rows=260)
    keep = torch.zeros(260, dtype=torch.bool, device="cuda")
    for s, m in zip(starts, kv):
        keep[s:s + m] = True
    K[~keep], V[~keep] = float("nan"), float("inf")
    V[100 + 39, :, 3] = float("inf")         # seen by the first sequence
    V[5, 0, 7], V[6, 0, 7] = float("inf"), float("-inf")
    V[16, 1, 20] = float("nan")              # the second sequence's last key
    V[201, :, 1] = float("-inf")             # the fourth's second token on
    plan = T.PackedPlan(q, kv, 4, 2, d, BF16, True, 333, starts)
    ws = plan.workspace()
    O, lse = attend(T, Q, K, V, Kp, Vp, plan, ws)
    assert ws.status() == T.TLSP_OK
    ref = Ref(Q, K, V, q, kv, starts, True, Kp, Vp)
    ref.check(O, lse)
    assert torch.isnan(ref.O).any() and torch.isinf(ref.O).any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens,heads", [(1, 1), (1, 3), (1, 5), (3, 5), (1, 7), (1, 11), (1, 15)])
def test_odd_rows_of_a_cluster(T, d, tokens, heads):
    """Items of an odd number of rows shared by the CTAs of a cluster: with d = 64 half of a warp
    has an element less to join than the other half."""
    plan = T.PackedPlan([tokens] * 2, [1200, 700], heads, 1, d)
    assert plan.data.cluster > 1 and plan.data.tile_items == 0
    run(T, [tokens] * 2, [1200, 700], heads, 1, d)


def test_rows_behind_the_last_sequence(T):
    q, kv = [40, 1], [40, 300]
    Q, K, V, _, _ = inputs(q, kv, 4, 2, 128, BF16, rows=60, kv_rows=400)
    Q[41:], K[340:], V[340:] = float("nan"), float("nan"), float("nan")
    plan = T.PackedPlan(q, kv, 4, 2, 128)
    ws = plan.workspace()
    out = torch.full_like(Q, 3.0)
    lse = torch.full((60, 4), 5.0, device="cuda")
    T.packed_attention(Q, K, V, plan, ws, out=out, lse=lse)
    assert (out[41:] == 3.0).all() and (lse[41:] == 5.0).all()
    Ref(Q, K, V, q, kv).check(out, lse)
    assert (T.packed_attention(Q, K, V, plan, ws)[41:] == 0).all()


def test_strided_tensors(T):
    """Slices of one fused projection, head-major storage, an output inside a wider tensor."""
    q, kv, h, hk, d = [70, 1, 200], [70, 1, 200], 6, 2, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn((271, h + 2 * hk, d), generator=g, device="cuda").bfloat16()
    Q, K, V = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
    plan = T.PackedPlan(q, kv, h, hk, d)
    ws = plan.workspace()
    wide = torch.zeros((271, h, 2 * d), dtype=BF16, device="cuda")
    O = T.packed_attention(Q, K, V, plan, ws, out=wide[..., d:])
    ref = Ref(Q, K, V, q, kv)
    ref.check(O)
    assert (wide[..., :d] == 0).all()
    Qh, Kh, Vh = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (Q, K, V))
    assert torch.equal(T.packed_attention(Qh, Kh, Vh, plan, ws), O)


def test_outputs_beside_inputs(T):
    """An output among the inputs' heads or channels is taken, one on top of them refused."""
    q, kv, h, hk, d = [70, 1, 200], [70, 1, 200], 6, 2, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn((271, 2 * h + 2 * hk, d), generator=g, device="cuda").bfloat16()
    Q, K, V, O = wide[:, :h], wide[:, h:h + hk], wide[:, h + hk:h + 2 * hk], wide[:, h + 2 * hk:]
    plan = T.PackedPlan(q, kv, h, hk, d)
    ws = plan.workspace()
    want = T.packed_attention(Q, K, V, plan, ws)
    before = T.launch_count()
    for out in (Q, wide[:, 1:h + 1], wide[:, h + hk:2 * h + hk], wide[:, h + 2 * hk - 1:-1]):
        with pytest.raises(T.TlspError) as e:
            T.packed_attention(Q, K, V, plan, ws, out=out)
        assert e.value.code == T.TLSP_ERR_INVALID_ARG
    assert T.launch_count() == before
    assert torch.equal(T.packed_attention(Q, K, V, plan, ws, out=O), want)
    pair = torch.zeros((271, h, 2 * d), dtype=BF16, device="cuda")
    pair[..., :d] = Q
    T.packed_attention(pair[..., :d], K, V, plan, ws, out=pair[..., d:])
    assert torch.equal(pair[..., d:], want) and torch.equal(pair[..., :d], Q)
    heads_first = torch.zeros((2 * h, 271, d), dtype=BF16, device="cuda").transpose(0, 1)
    heads_first[:, :h] = Q
    T.packed_attention(heads_first[:, :h], K, V, plan, ws, out=heads_first[:, h:])
    assert torch.equal(heads_first[:, h:], want)


def test_same_bits_again(T):
    q, kv = [1] * 9 + [260], [3000 + 7 * i for i in range(9)] + [260]
    Q, K, V, Kp, Vp = inputs(q, kv, 6, 2, 128, BF16, 2000)
    plan = T.PackedPlan(q, kv, 6, 2, 128, prefix_len=2000)
    ws = plan.workspace()
    a = attend(T, Q, K, V, Kp, Vp, plan, ws)
    for _ in range(5):
        b = attend(T, Q, K, V, Kp, Vp, plan, ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_streams_and_captured_replays(T):
    """Two plans on two streams at once, each with its workspace; the same calls captured and
    replayed on new inputs."""
    cases = []
    for seed, (q, kv) in enumerate((([1] * 6, [700, 80, 3000, 9, 1, 400]), ([300, 20], [300, 900]))):
        t = inputs(q, kv, 6, 2, 128, BF16, 500, seed=seed)
        plan = T.PackedPlan(q, kv, 6, 2, 128, prefix_len=500)
        cases.append((q, kv, t, plan, plan.workspace(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        for q, kv, t, plan, ws, st in cases:
            with torch.cuda.stream(st):
                outs.append(attend(T, *t, plan, ws))
    torch.cuda.synchronize()
    for i, (O, lse) in enumerate(outs):
        q, kv, t, *_ = cases[i % 2]
        Ref(t[0], t[1], t[2], q, kv, Kp=t[3], Vp=t[4]).check(O, lse)
    graphs = []
    for q, kv, t, plan, ws, st in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            graphs.append((graph, attend(T, *t, plan, ws)))
    for (q, kv, t, plan, ws, st), (graph, (O, lse)) in zip(cases, graphs):
        for x in t:
            x.copy_(torch.randn_like(x))
        graph.replay()
        torch.cuda.synchronize()
        Ref(t[0], t[1], t[2], q, kv, Kp=t[3], Vp=t[4]).check(O, lse)
        assert ws.status() == T.TLSP_OK
    with pytest.raises(RuntimeError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            T.PackedPlan([1], [1], 4, 2, 128)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_each_call_reads_the_one_before(T, dtype):
    """Calls whose queries are the output before them, on one workspace per plan, back to back
    and as a captured graph: the same bits as with a synchronisation after each call. Tile and
    token items together, with and without merged parts, either of them alone, and rotary."""
    heads, kv_heads, d, rows = 8, 2, 128, 424
    batches = [([1] * 40 + [384], [900 + 37 * i for i in range(40)] + [700], 0),  # both
               ([1] * 424, [3 * i % 500 for i in range(424)], 900),  # both, merged
               ([424], [424], 0), ([424], [9000], 0),  # tile items, cut and merged
               ([4] * 106, [50 + i for i in range(106)], 0),  # token items
               ([1] * 40 + [384], [500] * 41, 300)]
    turn = T.RotaryPlan(d)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    steps = []
    for i, (q, kv, prefix) in enumerate(batches):
        plan = T.PackedPlan(q, kv, heads, kv_heads, d, dtype, prefix_len=prefix)
        _, K, V, Kp, Vp = inputs([rows], kv, heads, kv_heads, d, dtype, prefix, seed=i, kv_rows=sum(kv))
        steps.append((plan, plan.workspace(), K, V, Kp, Vp))
    first = inputs([rows], [1], heads, kv_heads, d, dtype, seed=9)[0]

    def chain(wait):
        outs = [torch.empty_like(first) for _ in range(4 * len(steps))]
        x = first
        for i, (plan, ws, K, V, Kp, Vp) in enumerate(steps + steps):
            y, turned = outs[2 * i:2 * i + 2]
            if Kp is None:
                T.packed_attention(x, K, V, plan, ws, scale=2.0, out=y)
            else:
                T.prefix_attention(x, Kp, Vp, K, V, plan, ws, scale=2.0, out=y)
            wait()
            T.rotary(y, None, pos, turn, out=turned)
            wait()
            x = turned
        return outs
    want = chain(torch.cuda.synchronize)
    runs = [chain(lambda: None) for _ in range(3)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        runs.append(chain(lambda: None))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for outs in runs:
        for a, b in zip(want, outs):
            assert torch.equal(a, b)
    for step in steps:
        assert step[1].status() == T.TLSP_OK


def test_a_dropped_workspace_of_another_stream(T):
    """Dropped while a call on the plan's stream still waits to run, a workspace that another
    stream made is not handed out there again."""
    q, kv = [1] * 2, [20000, 17]
    Q, K, V, _, _ = inputs(q, kv, 6, 2, 128, BF16)
    plan, other = T.PackedPlan(q, kv, 6, 2, 128), torch.cuda.Stream()
    assert plan.data.part_rows > 0
    with torch.cuda.stream(other):
        ws = plan.workspace()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)               # about 0.1 s of the current stream
    O = T.packed_attention(Q, K, V, plan, ws)
    at, nbytes = ws.buf.data_ptr(), ws.nbytes
    del ws
    with torch.cuda.stream(other):
        again = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    assert not torch.cuda.current_stream().query() and again.data_ptr() != at
    torch.cuda.synchronize()
    Ref(Q, K, V, q, kv).check(O)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("q,kv,prefix", [
    ([1] * 8, [900 + 37 * i for i in range(8)], 0),                # token items alone
    ([1] * 2, [20000, 17], 0),                                     # cut and merged
    ([300], [9000], 0),                                            # tile items, cut and merged
    ([1] * 40 + [384], [500] * 40 + [700], 900),                   # both, merged
])
def test_tables_written_just_before(T, dtype, q, kv, prefix):
    """A plan's table that kernels ahead in the stream write (in turn all zeros, which no kernel
    takes for items, and the table) is read as stream order has it."""
    tensors = inputs(q, kv, 8, 2, 128, dtype, prefix)
    plan = T.PackedPlan(q, kv, 8, 2, 128, dtype, prefix_len=prefix)
    ws, table = plan.workspace(), plan.items.clone()
    want = attend(T, *tensors, plan, ws)
    zero = torch.zeros_like(table)
    outs = []
    for _ in range(10):
        torch.add(zero, 0, out=plan.items)
        torch.add(table, 0, out=plan.items)
        outs.append(attend(T, *tensors, plan, ws))
        outs.append(attend(T, *tensors, plan, ws))
    torch.cuda.synchronize()
    assert ws.status() == T.TLSP_OK
    for O, lse in outs:
        assert torch.equal(O, want[0]) and torch.equal(lse, want[1])


def test_cache_beyond_32_bit_offsets(T):
    """Keys whose element offsets pass 2^32: a cache of 4.3 G elements, of which little is read."""
    kv_rows, hk, d = 4200000, 8, 128
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB of device memory")
    K = torch.empty((kv_rows, hk, d), dtype=BF16, device="cuda")
    V = torch.empty_like(K)
    q, kv, starts = [1, 200], [300, 257], [kv_rows - 300, kv_rows - 700]
    g = torch.Generator(device="cuda").manual_seed(0)
    for x in (K, V):
        x[-1000:] = torch.randn((1000, hk, d), generator=g, device="cuda").bfloat16()
    Q = torch.randn((201, 16, d), generator=g, device="cuda").bfloat16()
    plan = T.PackedPlan(q, kv, 16, hk, d, kv_starts=starts)
    ws = plan.workspace()
    O = T.packed_attention(Q, K, V, plan, ws)
    Ref(Q, K, V, q, kv, starts).check(O)
    assert ws.status() == T.TLSP_OK


def test_refusals(T):
    q, kv = [3, 1], [3, 9]
    Q, K, V, Kp, Vp = inputs(q, kv, 4, 2, 128, BF16, 5)
    plan, pplan = T.PackedPlan(q, kv, 4, 2, 128), T.PackedPlan(q, kv, 4, 2, 128, prefix_len=5)
    ws, small = pplan.workspace(), T.Workspace.status_only()
    many = inputs([300], [20000], 4, 2, 128, BF16)               # cut keys: partial results
    mplan = T.PackedPlan([300], [20000], 4, 2, 128)
    assert mplan.data.part_rows > 0
    before = T.launch_count()
    bad = [
        lambda: T.packed_attention(Q[:3], K, V, plan, ws),
        lambda: T.packed_attention(Q, K[:11], V, plan, ws),
        lambda: T.packed_attention(Q, K, V[:, :1], plan, ws),
        lambda: T.packed_attention(Q, K, V.float(), plan, ws),
        lambda: T.packed_attention(Q.cpu(), K, V, plan, ws),
        lambda: T.packed_attention(Q, None, V, plan, ws),
        lambda: T.packed_attention(Q, K, V, pplan, ws),
        lambda: T.prefix_attention(Q, Kp, Vp, K, V, plan, ws),
        lambda: T.prefix_attention(Q, None, Vp, K, V, pplan, ws),
        lambda: T.prefix_attention(Q, Kp[:4], Vp, K, V, pplan, ws),
        lambda: T.packed_attention(Q, K, V, plan, ws, scale=0.0),
        lambda: T.packed_attention(Q, K, V, plan, ws, out=Q[:2]),
        lambda: T.packed_attention(Q, K, V, plan, ws, lse=torch.empty(4, 4, device="cuda").T),
        lambda: T.packed_attention(Q, K, V, plan, ws, lse=torch.empty(4, 3, device="cuda")),
        lambda: T.packed_attention(Q.transpose(1, 2).contiguous().transpose(1, 2), K, V, plan, ws),
        lambda: T.PackedPlan(torch.tensor(q, device="cuda"), kv, 4, 2, 128),
        lambda: T.PackedPlan(q, kv[:1], 4, 2, 128),
        lambda: T.PackedPlan(q, kv, 4, 2, 128, dtype=torch.float16),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    status = [
        (T.TLSP_ERR_WORKSPACE, lambda: T.packed_attention(*many[:3], mplan, small)),
        (T.TLSP_ERR_INVALID_ARG, lambda: T.packed_attention(Q, K[:, :1].expand(12, 2, 128), V, plan, ws)),
        (T.TLSP_ERR_INVALID_ARG, lambda: T.PackedPlan([-1], [1], 4, 2, 128)),
        (T.TLSP_ERR_INVALID_ARG, lambda: T.PackedPlan([1], [1], 4, 3, 128)),
        (T.TLSP_ERR_UNSUPPORTED, lambda: T.PackedPlan([1], [1], 65, 1, 128)),
    ]
    for code, f in status:
        with pytest.raises(T.TlspError) as e:
            f()
        assert e.value.code == code
    assert T.launch_count() == before


def test_a_table_of_another_batch_is_caught(T):
    """Items outside the call's tensors are skipped and recorded, not followed."""
    q, kv = [3, 1], [3, 9]
    Q, K, V, _, _ = inputs(q, kv, 4, 2, 128, BF16)
    for other_q, other_kv in (([3, 1], [3, 5000]), ([300, 1], [300, 9])):
        plan, other = T.PackedPlan(q, kv, 4, 2, 128), T.PackedPlan(other_q, other_kv, 4, 2, 128)
        items = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
        items[:other.items.numel()] = other.items
        plan.items = items
        ws = plan.workspace()
        T.packed_attention(Q, K, V, plan, ws)
        torch.cuda.synchronize()
        assert ws.status() == T.TLSP_ERR_DEVICE_ASSERT


def test_rotary_prompt_then_shared_decoding(T):
    """The operators together: a context is rotated and attended as a prompt, then a batch of
    continuations decodes two tokens each behind its keys, against whole-sequence attention."""
    h, hk, d, P, S, steps = 6, 2, 128, 777, 5, 2
    g = torch.Generator(device="cuda").manual_seed(1)

    def rand(n, heads):
        return torch.randn((n, heads, d), generator=g, device="cuda").bfloat16()
    rope = T.RotaryPlan(d, scaling="ramp", factor=4.0, original_len=512)
    Qc, Kc, Vc = rand(P, h), rand(P, hk), rand(P, hk)
    Qc, Kc = T.rotary(Qc, Kc, torch.arange(P, dtype=torch.int32, device="cuda"), rope)
    plan = T.PackedPlan([P], [P], h, hk, d)
    Oc = T.packed_attention(Qc, Kc, Vc, plan, plan.workspace())
    Ref(Qc, Kc, Vc, [P], [P]).check(Oc)
    cap = 16
    cache_k = torch.full((S * cap, hk, d), float("nan"), dtype=BF16, device="cuda")
    cache_v = cache_k.clone()
    starts = [s * cap for s in range(S)]
    rows = torch.tensor(starts, device="cuda")
    for t in range(steps):
        Q, K, V = rand(S, h), rand(S, hk), rand(S, hk)
        Q, K = T.rotary(Q, K, torch.full((S,), P + t, dtype=torch.int32, device="cuda"), rope)
        cache_k[rows + t], cache_v[rows + t] = K, V
        plan = T.PackedPlan([1] * S, [t + 1] * S, h, hk, d, prefix_len=P, kv_starts=starts)
        ws = plan.workspace()
        O = T.prefix_attention(Q, Kc, Vc, cache_k, cache_v, plan, ws)
        Ref(Q, cache_k, cache_v, [1] * S, [t + 1] * S, starts, True, Kc, Vc).check(O)
        assert ws.status() == T.TLSP_OK


@pytest.mark.parametrize("seed", range(40))
def test_random_batches(T, seed):
    """Lengths, heads, types, masks, prefixes, cache places and strides drawn at random; a second
    call returns the same bits."""
    r = random.Random(seed)
    d, dtype = r.choice([64, 128]), r.choice([BF16, BF16, BF16, FP32])
    hk, g = r.choice([1, 2, 3, 8]), r.choice([1, 2, 3, 5, 7, 8, 13, 16])
    kind = r.choice([[0, 1, 1, 1, 2, 3], [0, 1, 64, 127, 129, 300], [0, 1, 2, 40, 200]])
    n = r.choice([1, 3, 8, 20])
    q = [r.choice(kind) for _ in range(n)]
    kv = [r.choice([a, a + r.randint(0, 1500), r.randint(0, 300), 0]) for a in q]
    prefix, causal = r.choice([0, 0, 1, 129, 2000]), r.random() < 0.75
    starts, rows = None, max(1, sum(kv))
    if r.random() < 0.4:
        starts, at = [0] * n, r.randint(0, 9)
        for s in r.sample(range(n), n):
            starts[s], at = at, at + kv[s] + r.randint(0, 40)
        rows = max(1, at)
    Q, K, V, Kp, Vp = inputs(q, kv, hk * g, hk, d, dtype, prefix, seed, rows=sum(q) + 3, kv_rows=rows)
    if r.random() < 0.3:
        Q = Q.transpose(0, 1).contiguous().transpose(0, 1)
    if starts is not None:
        keep = torch.zeros(rows, dtype=torch.bool, device="cuda")
        for s in range(n):
            keep[starts[s]:starts[s] + kv[s]] = True
        K[~keep], V[~keep] = float("nan"), float("inf")
    plan = T.PackedPlan(q, kv, hk * g, hk, d, dtype, causal, prefix, starts)
    ws = plan.workspace()
    O, lse = attend(T, Q, K, V, Kp, Vp, plan, ws, out=torch.full_like(Q, 9.0))
    again = attend(T, Q, K, V, Kp, Vp, plan, ws, out=torch.full_like(Q, 9.0))
    torch.cuda.synchronize()
    assert ws.status() == T.TLSP_OK
    assert torch.equal(O, again[0]) and torch.equal(lse, again[1])
    assert (O[sum(q):] == 9.0).all() and (lse[sum(q):] == 7.0).all()
    Ref(Q, K, V, q, kv, starts, causal, Kp, Vp).check(O, lse)
