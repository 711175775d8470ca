"""Rotary positions on the GPU against the formulas in 64 bits (bounds: tests/packed_ref.py)."""
import pytest
import torch

from tests.packed_ref import rotary_ref, rotary_tables

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def T():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from token_level_sparse_pddp_b200 import build, tlsp
    build.build()
    return tlsp


def rand(shape, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def near(y, ref_tol):
    ref, tol = ref_tol
    off = (y.double() - ref).abs()
    assert (off <= tol).all(), f"{float((off - tol).max()):.3g} over the bound"


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("d,r", [(128, 128), (128, 64), (64, 64), (64, 18), (256, 256), (8, 2), (72, 40)])
def test_packed_tokens(T, dtype, layout, backward, d, r):
    for n, h, hk in ((1, 1, 1), (77, 5, 2), (3000, 3, 1)):
        Q, K = rand((n, h, d), dtype), rand((n, hk, d), dtype, 1)
        pos = torch.randint(-50, 200000, (n,), device="cuda", dtype=torch.int32)
        plan = T.RotaryPlan(d, rotary_dim=r, layout=layout)
        f = T.rotary_backward if backward else T.rotary
        Qr, Kr = f(Q, K, pos, plan)
        tab = rotary_tables(d, r, pos[None])
        c, s = tab[0][:, None], tab[1][:, None]
        near(Qr, rotary_ref(Q, c, s, tab[2], r, layout, backward))
        near(Kr, rotary_ref(K, c, s, tab[2], r, layout, backward))


@pytest.mark.parametrize("kw", [
    dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0, base=500000.0),
    dict(scaling="ramp", factor=16.0, original_len=4096),
])
@pytest.mark.parametrize("pos_dtype", [torch.int32, torch.int64])
def test_far_positions(T, kw, pos_dtype):
    n, d = 300, 128
    Q = rand((n, 2, d), FP32)
    pos = torch.randint(0, 2 ** 31 - 1, (n,), device="cuda").to(pos_dtype)
    if pos_dtype == torch.int64:
        pos[:100] += 2 ** 33
    plan = T.RotaryPlan(d, **kw)
    y = T.rotary(Q, None, pos, plan)
    tab = rotary_tables(d, d, pos[None], **kw)
    ref, tol = rotary_ref(Q, tab[0][:, None], tab[1][:, None], tab[2], d, "half")
    # both frequencies carry 2^-53 relative (the reference) and 2^-65 turns (the plan): p = 2^34
    # positions away the angles differ by up to 2^34 2^-53 of a radian plus 2^-31 of a turn
    tol = tol + 2 * Q.double().abs().amax() * tab[2] * (2.0 ** -19 + 2.0 ** -28)
    near(y, (ref, tol))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_video_grid_heads_first(T, dtype, layout):
    """[batch, heads, tokens, channels] with (frame, row, column) sections, own positions per
    batch element and shared ones."""
    B, h, f, hh, w, d = 2, 3, 3, 5, 7, 128
    n, sec = f * hh * w, (22, 21, 21)
    i = torch.arange(n, device="cuda")
    pos = torch.stack([i // (hh * w), i % (hh * w) // w, i % w]).to(torch.int32)
    Q, K = rand((B, h, n, d), dtype), rand((B, 1, n, d), dtype, 1)
    plan = T.RotaryPlan(d, layout=layout, sections=sec)
    tab = rotary_tables(d, d, pos, sections=sec)
    Qr, Kr = T.rotary(Q, K, pos, plan)
    near(Qr, rotary_ref(Q, tab[0], tab[1], 1.0, d, layout))
    near(Kr, rotary_ref(K, tab[0], tab[1], 1.0, d, layout))
    each = torch.stack([pos, pos + 100], 1)          # [axes, batch, tokens]
    Qr, Kr = T.rotary(Q, K, each, plan)
    tab = rotary_tables(d, d, each, sections=sec)
    near(Qr, rotary_ref(Q, tab[0][:, None], tab[1][:, None], 1.0, d, layout))
    one = torch.stack([i, 3 * i])                    # [batch, tokens], one axis
    y = T.rotary(Q, None, one, T.RotaryPlan(d, layout=layout))
    tab = rotary_tables(d, d, one[None])
    near(y, rotary_ref(Q, tab[0][:, None], tab[1][:, None], 1.0, d, layout))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d,r", [(128, 128), (128, 64), (64, 18)])
def test_strides_and_in_place(T, dtype, d, r):
    n, h, hk = 130, 4, 2
    qkv = rand((n, h + 2 * hk, d), dtype)
    pos = torch.arange(n, device="cuda")
    plan = T.RotaryPlan(d, rotary_dim=r)
    want = T.rotary(qkv[:, :h].contiguous(), qkv[:, h:h + hk].contiguous(), pos, plan)
    got = T.rotary(qkv[:, :h], qkv[:, h:h + hk], pos, plan)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    v = qkv[:, h + hk:].clone()
    T.rotary(qkv[:, :h], qkv[:, h:h + hk], pos, plan, out=(qkv[:, :h], qkv[:, h:h + hk]))
    assert torch.equal(qkv[:, :h], want[0]) and torch.equal(qkv[:, h:h + hk], want[1])
    assert torch.equal(qkv[:, h + hk:], v)
    # rows that are not 16-byte aligned, and a broadcast input
    odd = torch.zeros((n, h, d + 1), dtype=dtype, device="cuda")[..., 1:]
    src = rand((n, 1, d), dtype, 5).expand(n, h, d)
    T.rotary(src, None, pos, plan, out=odd)
    assert torch.equal(odd, T.rotary(src.contiguous(), None, pos, plan))


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_outputs_beside_inputs(T, dtype):
    """Outputs in other parts of the inputs' tensor, and in place where only axes of length 1 have
    other strides; outputs on other inputs are refused."""
    n, h, d = 130, 3, 64
    pos = torch.arange(n, device="cuda")
    plan = T.RotaryPlan(d)
    wide = rand((n, 4 * h, d), dtype)
    parts = [wide[:, i * h:(i + 1) * h] for i in range(4)]
    want = T.rotary(parts[0], parts[1], pos, plan)
    before = T.launch_count()
    for out in ((parts[1], parts[0]), (parts[2], parts[2]), (parts[0], parts[0]), (parts[2], parts[0]),
                (wide[:, 1:h + 1], parts[3]), (parts[2], wide[:, 3 * h - 1:-1])):
        with pytest.raises(T.TlspError) as e:
            T.rotary(parts[0], parts[1], pos, plan, out=out)
        assert e.value.code == T.TLSP_ERR_INVALID_ARG
    assert T.launch_count() == before
    T.rotary(parts[0], parts[1], pos, plan, out=(parts[3], parts[2]))
    assert torch.equal(parts[3], want[0]) and torch.equal(parts[2], want[1])
    T.rotary(parts[0], parts[1], pos, plan, out=(parts[0], parts[3]))       # one of them in place
    assert torch.equal(parts[0], want[0]) and torch.equal(parts[3], want[1])
    pairs = rand((n, h, 2, d), dtype, 1)                                    # heads in turn
    want = T.rotary(pairs[:, :, 0], pairs[:, :, 1], pos, plan)
    T.rotary(pairs[:, :, 0], pairs[:, :, 1], pos, plan, out=(pairs[:, :, 0], pairs[:, :, 1]))
    assert torch.equal(pairs[:, :, 0], want[0]) and torch.equal(pairs[:, :, 1], want[1])
    three = rand((2, 3, h, n, d), dtype, 2)                                 # [batch, q/k/v, heads, ...]
    want = T.rotary(three[:, 0], three[:, 1], pos, plan)
    T.rotary(three[:, 0], three[:, 1], pos, plan, out=(three[:, 0], three[:, 1]))
    assert torch.equal(three[:, 0], want[0]) and torch.equal(three[:, 1], want[1])
    x = rand((1, h, n, d), dtype, 3)
    want = T.rotary(x, None, pos, plan)
    T.rotary(x, None, pos, plan, out=x.as_strided(x.shape, (7 * d, *x.stride()[1:])))
    assert torch.equal(x, want)


def test_backward_is_the_gradient(T):
    """Against differences of the forward pass: the map is linear, so <y(x + e) - y(x), g> is
    <e, gradient> up to the roundings of fp32 (n terms of a sum taken in 64 bits, each
    product's factor off by 2^-21)."""
    n, h, d = 200, 3, 128
    for layout in ("half", "interleaved"):
        plan = T.RotaryPlan(d, rotary_dim=64, layout=layout, scaling="ramp", factor=4.0, original_len=64)
        pos = torch.randint(0, 10000, (n,), device="cuda")
        x, e, g = (rand((n, h, d), FP32, s) for s in (0, 1, 2))
        dx = T.rotary_backward(g, None, pos, plan)
        dy = T.rotary(x + e, None, pos, plan).double() - T.rotary(x, None, pos, plan).double()
        left, right = (dy * g).sum(), (((x + e).double() - x) * dx).sum()
        size = ((x.abs() + e.abs()).double() * 4 * g.abs()).sum()
        assert abs(float(left - right)) <= float(size) * 2.0 ** -20
        # turning back: y / A^2 returns x
        a = plan.data.amplitude
        back = T.rotary_backward(T.rotary(x, None, pos, plan), None, pos, plan)
        back[..., :64] /= a * a
        assert (back - x).abs().max() <= 16 * 2.0 ** -21 * x.abs().max()


def test_gradient_against_the_formula(T):
    """autograd through the formula in 64 bits."""
    n, h, d, r = 90, 2, 128, 96
    pos = torch.randint(0, 5000, (n,), device="cuda")
    for layout in ("half", "interleaved"):
        plan = T.RotaryPlan(d, rotary_dim=r, layout=layout)
        cos, sin, amp = rotary_tables(d, r, pos[None])
        x = rand((n, h, d), FP32).double().requires_grad_()
        half = r // 2
        a, b = (x[..., :half], x[..., half:r]) if layout == "half" else (x[..., 0:r:2], x[..., 1:r:2])
        c, s = cos[:, None], sin[:, None]
        y1, y2 = a * c - b * s, b * c + a * s
        y = torch.cat([y1, y2], -1) if layout == "half" else torch.stack([y1, y2], -1).flatten(-2)
        g = rand((n, h, d), FP32, 3)
        (torch.cat([y, x[..., r:]], -1) * g).sum().backward()
        tol = rotary_ref(g, c, s, amp, r, layout, True)[1]
        near(T.rotary_backward(g, None, pos, plan), (x.grad, tol))


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_autograd(T, dtype):
    """Gradients through rotary() are rotary_backward()'s: of Q and K, of slices of a fused tensor,
    of a broadcast input (summed), of either alone, on another stream and in a captured step."""
    n, h, hk, d = 70, 4, 2, 128
    pos = torch.randint(0, 5000, (n,), device="cuda")
    plan = T.RotaryPlan(d, rotary_dim=64, scaling="linear", factor=2.0)
    gq, gk = rand((n, h, d), dtype, 1), rand((n, hk, d), dtype, 2)
    want = T.rotary_backward(gq, gk, pos, plan)
    qkv = rand((n, h + 2 * hk, d), dtype).requires_grad_()

    def step():
        Q, K = T.rotary(qkv[:, :h], qkv[:, h:h + hk], pos, plan)
        return torch.autograd.grad((Q, K), qkv, (gq, gk))[0]

    def same(grad):
        assert torch.equal(grad[:, :h], want[0]) and torch.equal(grad[:, h:h + hk], want[1])
        assert not grad[:, h + hk:].any()
    same(step())
    x = rand((n, 1, d), FP32, 3).to(dtype).requires_grad_()
    y = T.rotary(x.expand(n, h, d), None, pos, plan)
    dx, = torch.autograd.grad(y, x, gq)
    assert torch.equal(dx, want[0].sum(1, keepdim=True))
    k = rand((n, hk, d), dtype, 4).requires_grad_()
    Q, K = T.rotary(gq, k, pos, plan)
    assert torch.equal(torch.autograd.grad(K.sum(), k)[0],
                       T.rotary_backward(torch.ones_like(k), None, pos, plan))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            got = step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            captured = step()
    side.synchronize()
    same(got)
    captured.zero_()
    gq.copy_(rand((n, h, d), dtype, 7))
    want = T.rotary_backward(gq, gk, pos, plan)
    graph.replay()
    torch.cuda.synchronize()
    same(captured)


def test_special_values_stay_in_their_pair(T):
    n, h, d = 64, 2, 128
    x = rand((n, h, d), BF16)
    pos = torch.arange(n, device="cuda")
    plan = T.RotaryPlan(d, rotary_dim=64)
    clean = T.rotary(x, None, pos, plan)
    x[5, 1, 3], x[6, 0, 100] = float("nan"), float("inf")
    y = T.rotary(x, None, pos, plan)
    assert torch.isnan(y[5, 1, 3]) and torch.isnan(y[5, 1, 35]) and y[6, 0, 100] == float("inf")
    same = torch.ones_like(x, dtype=torch.bool)
    same[5, 1, 3] = same[5, 1, 35] = same[6, 0, 100] = False
    assert torch.equal(y[same], clean[same])


def test_empty_streams_and_graphs(T):
    plan = T.RotaryPlan(128)
    assert T.rotary(rand((0, 4, 128), BF16), None, torch.zeros(0, dtype=torch.int32, device="cuda"),
                    plan).shape == (0, 4, 128)
    Q, K = rand((50, 4, 128), BF16), rand((50, 1, 128), BF16, 1)
    pos = torch.arange(50, device="cuda", dtype=torch.int32)
    want = T.rotary(Q, K, pos, plan)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = T.rotary(Q, K, pos, plan)
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = T.rotary(Q, K, pos, plan)
    Q.copy_(rand((50, 4, 128), BF16, 9))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], T.rotary(Q, None, pos, plan))


def test_refusals(T):
    plan = T.RotaryPlan(128)
    two = T.RotaryPlan(128, sections=(32, 32))
    Q, K = rand((5, 4, 128), BF16), rand((5, 2, 128), BF16)
    pos = torch.arange(5, device="cuda")
    before = T.launch_count()
    for i, f in enumerate([
        lambda: T.rotary(Q, K[:4], pos, plan), lambda: T.rotary(Q, K.float(), pos, plan),
        lambda: T.rotary(Q, K[None], pos, plan), lambda: T.rotary(Q[..., :64], None, pos, plan),
        lambda: T.rotary(Q[0], None, pos, plan), lambda: T.rotary(Q.cpu(), None, pos.cpu(), plan),
        lambda: T.rotary(Q, K, pos[:4], plan), lambda: T.rotary(Q, K, pos.float(), plan),
        lambda: T.rotary(Q, K, pos.cpu(), plan), lambda: T.rotary(Q, K, pos, two),
        lambda: T.rotary(Q, K, torch.arange(10, device="cuda")[::2], plan),
        lambda: T.rotary(Q.half(), None, pos, plan),
        lambda: T.rotary(Q.transpose(1, 2).contiguous().transpose(1, 2), None, pos, plan),
        lambda: T.rotary(Q, None, pos, plan, out=Q[:4]),
        lambda: T.rotary(Q, K, pos, plan, out=(Q,)),
        lambda: T.rotary(Q, None, pos, plan, out=Q[:, :1].expand(5, 4, 128)),
        lambda: T.rotary(rand((2, 4, 5, 128), BF16), None, pos.expand(3, 5), plan),
    ]):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(T.TlspError):     # in place with other strides
        T.rotary(Q, None, pos, plan, out=Q.view(-1).as_strided((5, 4, 128), (128, 640, 1)))
    assert T.launch_count() == before


def test_schedule_turns_queries_and_keys(T):
    """MCSparseAttention with a rotary plan equals rotating first, and leaves its inputs alone."""
    from token_level_sparse_pddp_b200.schedule import MCSparseAttention
    n, h, d = 256, 2, 128
    pos = torch.stack([torch.arange(n, device="cuda") // 64, torch.arange(n, device="cuda") % 64])
    rope = T.RotaryPlan(d, layout="interleaved", sections=(24, 40))
    a = MCSparseAttention(64, 64, schedule="AR", rotary=rope)
    b = MCSparseAttention(64, 64, schedule="AR")
    for step in range(2):
        Q, K, V = (rand((1, h, n, d), BF16, 10 * step + i) for i in range(3))
        keep = Q.clone(), K.clone()
        O = a(Q, K, V, pos)
        Qr, Kr = T.rotary(Q, K, pos, rope)
        assert torch.equal(O, b(Qr, Kr, V))
        assert torch.equal(Q, keep[0]) and torch.equal(K, keep[1])
    few = Q[:, :, :128].contiguous()
    c, e = MCSparseAttention(64, 64, rotary=rope), MCSparseAttention(64, 64)
    O = c(few, K, V, pos[:, 128:].contiguous(), pos)
    assert torch.equal(O, e(T.rotary(few, None, pos[:, 128:].contiguous(), rope),
                            T.rotary(K, None, pos, rope), V))
    for bad in (lambda: c(few, K, V), lambda: c(few, K, V, pos[:, :128].contiguous()),
                lambda: e(few, K, V, pos)):
        with pytest.raises(ValueError):
            bad()
