"""The binding of the packed attention and rotary calls without a GPU: what it checks and keeps
before it calls the library."""
import types

import pytest
import torch

from token_level_sparse_pddp_b200 import build as tlsp_build


@pytest.fixture(scope="module")
def T():
    tlsp_build.build()
    from token_level_sparse_pddp_b200 import tlsp
    tlsp.lib()
    return tlsp


@pytest.fixture
def calls(T, monkeypatch):
    """Library calls of the binding, recorded in place of being made; a current stream that a
    test sets (`calls.stream`), on "device" -1, where CPU tensors lie."""
    made = types.SimpleNamespace(stream=5, list=[])

    def launch(device, fn, *args):
        made.list.append(fn.__name__)
        return T.TLSP_OK
    monkeypatch.setattr(T, "_launch", launch)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: made.stream, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda dev=None: types.SimpleNamespace(cuda_stream=made.stream))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return made


class Buffer:
    """Stands for a device buffer: notes the streams it is recorded on."""

    def __init__(self):
        self.recorded = []

    def get_device(self):
        return -1

    def data_ptr(self):
        return 4096

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)


def plan_of(T, q, kv, heads=4, kv_heads=2, d=64, made_on=5, prefix=0):
    return types.SimpleNamespace(q_rows=sum(q), kv_rows=sum(kv), heads=heads, kv_heads=kv_heads,
                                 head_dim=d, dtype=torch.float32, prefix_len=prefix, device="cpu",
                                 items=Buffer(), _at=0, _dev=-1, _made_on=made_on)


def workspace(T, made_on):
    ws = object.__new__(T.Workspace)
    ws.nbytes, ws.buf, ws.made_on = 1 << 20, Buffer(), made_on
    return ws


def tensors(q, kv, heads=4, kv_heads=2, d=64):
    return torch.zeros(q, heads, d), torch.zeros(kv, kv_heads, d), torch.zeros(kv, kv_heads, d)


@pytest.mark.parametrize("plan_on,ws_on,now,plan_kept,ws_kept", [
    (5, 5, 5, [], []), (5, 6, 5, [], [5]), (6, 5, 5, [5], []), (6, 7, 5, [5], [5]),
])
def test_memory_of_other_streams_is_kept(T, calls, plan_on, ws_on, now, plan_kept, ws_kept):
    """Plan and workspace are each recorded on the calling stream if they were made on another."""
    plan, ws = plan_of(T, [3], [3], made_on=plan_on), workspace(T, ws_on)
    calls.stream = now
    T.packed_attention(*tensors(3, 3), plan, ws)
    assert calls.list == ["tlsp_packed_attention"]
    assert plan.items.recorded == plan_kept and ws.buf.recorded == ws_kept


def planned(T, q=(1, 2), kv=(1, 2), heads=4, kv_heads=2, head_dim=64, prefix_len=0, kv_starts=None):
    return T.PackedPlan(list(q), list(kv), heads, kv_heads, head_dim, torch.float32,
                        prefix_len=prefix_len, kv_starts=kv_starts, device="cpu")


@pytest.mark.parametrize("kw", [
    dict(q=(2 ** 32 + 1, 1)), dict(kv=(2, 2 ** 32 + 3)), dict(q=(2 ** 31, 0)), dict(kv=(1, -2 ** 32)),
    dict(kv_starts=[0, 2 ** 64 + 4]), dict(kv_starts=[2 ** 63, 0]), dict(prefix_len=2 ** 32 + 5),
    dict(heads=2 ** 32 + 4), dict(kv_heads=2 ** 32 + 2), dict(head_dim=2 ** 32 + 64),
])
def test_numbers_that_do_not_fit(T, calls, kw):
    """A number too large for the library's types is refused, not cut to its low bits."""
    assert planned(T).q_rows == 3 and planned(T, q=torch.tensor([1, 2]).tolist()).kv_rows == 3
    with pytest.raises(ValueError):
        planned(T, **kw)


@pytest.mark.parametrize("kw", [
    dict(head_dim=2 ** 32 + 64), dict(rotary_dim=2 ** 32 + 64), dict(sections=(2 ** 32 + 16, 16)),
    dict(sections=(2 ** 32, 32)),
])
def test_rotary_numbers_that_do_not_fit(T, kw):
    with pytest.raises(ValueError):
        T.RotaryPlan(**{"head_dim": 64, **kw})


def test_numbers_that_are_not_whole(T, calls):
    for f in (lambda: planned(T, q=(1.5, 2)), lambda: planned(T, kv_starts=[0.5, 9]),
              lambda: planned(T, heads=4.0), lambda: planned(T, prefix_len=3.5),
              lambda: T.RotaryPlan(64, sections=(16.5, 15.5)), lambda: T.RotaryPlan(64.0)):
        with pytest.raises(TypeError):
            f()


# ------------------------------------------------------------------ gradients

def turned(T, x, pos, plan, sign=1.0):
    """The formula for one axis and the half layout, in elementary operations."""
    r = plan.rotary_dim
    turns = torch.tensor([plan.data.turns[i] / 2.0 ** 64 for i in range(r // 2)], dtype=torch.float64)
    a = 2 * torch.pi * pos.double()[:, None] * turns
    c, s = (plan.data.amplitude * a.cos())[:, None], (sign * plan.data.amplitude * a.sin())[:, None]
    x1, x2 = x.double()[..., :r // 2], x.double()[..., r // 2:r]
    return torch.cat([x1 * c - x2 * s, x2 * c + x1 * s, x.double()[..., r:]], -1)


@pytest.fixture
def on_host(T, monkeypatch):
    """rotary()'s launch replaced by the formula: the autograd path without a GPU."""
    def fake(Q, K, positions, plan, out, backward):
        made = [turned(T, x.detach(), positions, plan, -1.0 if backward else 1.0).to(x.dtype)
                for x in (Q, K) if x is not None]
        return made[0] if K is None else tuple(made)
    monkeypatch.setattr(T, "_rotary", fake)


def test_rotary_carries_gradients(T, on_host):
    """rotary() of tensors that require gradients returns ones that carry them; so does
    rotary_backward(), whose own gradient turns forward again."""
    plan = T.RotaryPlan(64, rotary_dim=32)
    pos = torch.tensor([3, 0, 70])
    g = torch.Generator().manual_seed(0)
    q, k, gq, gk = (torch.randn(3, h, 64, generator=g, dtype=torch.float64) for h in (2, 1, 2, 1))
    for need_q, need_k in ((True, True), (True, False), (False, True)):
        Q, K = q.clone().requires_grad_(need_q), k.clone().requires_grad_(need_k)
        yq, yk = T.rotary(Q, K, pos, plan)
        ((yq * gq).sum() + (yk * gk).sum()).backward()
        for x, grad, need in ((Q, gq, need_q), (K, gk, need_k)):
            assert (x.grad is not None) == need
            if need:
                assert torch.allclose(x.grad, turned(T, grad, pos, plan, -1.0), rtol=0, atol=1e-12)
    # one output alone takes part; broadcast gradients (of a sum)
    Q, K = q.clone().requires_grad_(), k.clone().requires_grad_()
    T.rotary(Q, K, pos, plan)[1].sum().backward()
    assert torch.allclose(K.grad, turned(T, torch.ones_like(k), pos, plan, -1.0), rtol=0, atol=1e-12)
    assert Q.grad is None or not Q.grad.any()
    Q = q.clone().requires_grad_()
    assert torch.autograd.gradcheck(lambda x: T.rotary(x, None, pos, plan), Q)
    assert torch.autograd.gradcheck(lambda x: T.rotary_backward(x, None, pos, plan), Q)
    assert torch.autograd.gradgradcheck(lambda x: T.rotary(x, None, pos, plan) ** 2, Q)
    with torch.no_grad():
        assert not T.rotary(Q, None, pos, plan).requires_grad
    assert not T.rotary(q, k, pos, plan)[0].requires_grad


def test_given_outputs_carry_no_gradients(T, on_host):
    """A gradient could not flow through memory that the caller gives: refused, unless none is
    asked for."""
    plan, pos = T.RotaryPlan(64), torch.arange(3)
    x, y = torch.zeros(3, 2, 64, requires_grad=True), torch.zeros(3, 2, 64)
    for q, k, out in ((x, None, y), (x, None, x), (y, None, x), (y, x, (y, x)), (y, y, (y, x))):
        with pytest.raises(ValueError):
            T.rotary(q, k, pos, plan, out=out)
        with pytest.raises(ValueError):
            T.rotary_backward(q, k, pos, plan, out=out)
        with torch.no_grad():
            T.rotary(q, k, pos, plan, out=out)


def test_attention_has_no_gradient(T, calls):
    """The attention calls have no backward pass and say so instead of returning a result that
    carries none."""
    Q, K, V = tensors(3, 3)
    ws = workspace(T, 5)
    prefix = torch.zeros(4, 2, 64)
    for which in range(3):
        args = [Q, K, V]
        args[which] = args[which].clone().requires_grad_()
        with pytest.raises(ValueError):
            T.packed_attention(*args, plan_of(T, [3], [3]), ws)
        with torch.no_grad():
            T.packed_attention(*args, plan_of(T, [3], [3]), ws)
    for which in range(2):
        pre = [prefix, prefix]
        pre[which] = prefix.clone().requires_grad_()
        with pytest.raises(ValueError):
            T.prefix_attention(Q, *pre, K, V, plan_of(T, [3], [3], prefix=4), ws)
    with pytest.raises(ValueError):
        T.packed_attention(Q, K, V, plan_of(T, [3], [3]), ws, out=Q.clone().requires_grad_())
    assert len(calls.list) == 3


# ------------------------------------------------------------------ scale

@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-60, -1e-50, 7e-46])
def test_scales_that_are_zero_in_32_bits(T, calls, scale):
    """The library takes a scale of 0 for 1/sqrt(d), so none may become 0 on its way there."""
    ws = workspace(T, 5)
    with pytest.raises(ValueError):
        T.packed_attention(*tensors(3, 3), plan_of(T, [3], [3]), ws, scale=scale)
    T.packed_attention(*tensors(3, 3), plan_of(T, [3], [3]), ws, scale=1e-44)
    assert len(calls.list) == 1
