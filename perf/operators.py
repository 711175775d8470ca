"""What is measured of three operators: rotary positions, causal attention over packed sequences
with grouped heads, and attention of a batch that shares a long prefix.

Each operator has a plain form in elementary torch operations (32-bit arithmetic, angles in 64)
and the call a user makes of the library (`own`). Shapes follow the library's workloads (12 or 40
heads of 128 channels, token grids 21 x 30 x 52 and 3 x 30 x 52) or are generic.

  rotary   y = A (x_1 cos a - x_2 sin a, x_2 cos a + x_1 sin a) for each rotated pair, a = position
           times the pair's frequency; the backward pass turns the other way.
  packed   sequences laid end to end; query i of a sequence with n queries and m keys sees its keys
           j <= i + m - n; query head h reads key/value head h // (heads / kv_heads).
  prefix   the same, and every query of every sequence also sees all keys of one shared prefix.
Attention returns O and the natural-log partition per row (O = 0, -inf where no key is seen).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    """Twelve cases, the smallest calls first in each operator."""
    return [
        # one decoding step of a batch: a token per sequence, far positions, ramp-scaled frequencies
        dict(name="rotary_tokens", op="rotary", form="packed", batch=1, tokens=64, frames=0, heads=12,
             kv_heads=4, head_dim=128, rotary_dim=128, layout="half", scaling="ramp", factor=8.0,
             dtype="bf16", backward=False, fused=False, start=100000),
        # Q and K of the whole 21 x 30 x 52 video grid, (frame, height, width) sections
        dict(name="rotary_video", op="rotary", form="heads", batch=1, tokens=21 * 30 * 52, frames=21,
             heads=12, kv_heads=12, head_dim=128, rotary_dim=128, layout="interleaved", scaling="none",
             factor=1.0, dtype="bf16", backward=False, fused=False, start=0),
        # Q and K as slices of one fused projection's output, half of each head rotated
        dict(name="rotary_fused", op="rotary", form="packed", batch=1, tokens=16381, frames=0, heads=40,
             kv_heads=8, head_dim=128, rotary_dim=64, layout="half", scaling="base", factor=4.0,
             dtype="bf16", backward=False, fused=True, start=7),
        # gradients of a 32-bit training step with 64-channel heads
        dict(name="rotary_backward", op="rotary", form="heads", batch=2, tokens=4680, frames=0, heads=12,
             kv_heads=12, head_dim=64, rotary_dim=64, layout="half", scaling="linear", factor=2.0,
             dtype="fp32", backward=True, fused=False, start=0),
        # one decoding step of a few sequences with caches of odd lengths
        dict(name="packed_tokens", op="packed", seqs=8, q_min=1, q_max=1, past_min=900, past_max=4700,
             heads=12, kv_heads=4, head_dim=128, dtype="bf16", lens=1),
        # a batch of prompts of very different lengths (one of them empty, one with fewer keys than queries)
        dict(name="packed_prompts", op="packed", seqs=24, q_min=1, q_max=4096, past_min=0, past_max=0,
             heads=12, kv_heads=4, head_dim=128, dtype="bf16", lens=2),
        # one prompt as long as the 21 x 30 x 52 grid
        dict(name="packed_long", op="packed", seqs=1, q_min=32760, q_max=32760, past_min=0, past_max=0,
             heads=12, kv_heads=12, head_dim=128, dtype="bf16", lens=3),
        # the next 3 x 30 x 52 chunk of an autoregressive video behind a cache of earlier frames
        dict(name="packed_chunk", op="packed", seqs=2, q_min=4680, q_max=4680, past_min=14040,
             past_max=28080, heads=40, kv_heads=8, head_dim=128, dtype="bf16", lens=4),
        # small ragged batch in 32 bits with 64-channel heads
        dict(name="packed_fp32", op="packed", seqs=6, q_min=50, q_max=1000, past_min=0, past_max=300,
             heads=8, kv_heads=2, head_dim=64, dtype="fp32", lens=5),
        # a few continuations of one frame of context, one token each
        dict(name="prefix_few", op="prefix", seqs=4, q_min=1, q_max=1, past_min=1, past_max=130,
             prefix=1560, heads=12, kv_heads=4, head_dim=128, dtype="bf16", lens=6),
        # many continuations decoding behind a long shared context
        dict(name="prefix_tokens", op="prefix", seqs=64, q_min=1, q_max=1, past_min=16, past_max=2000,
             prefix=32760, heads=40, kv_heads=8, head_dim=128, dtype="bf16", lens=7),
        # several candidate frames (30 x 52 tokens each) generated from the same earlier frames
        dict(name="prefix_frames", op="prefix", seqs=8, q_min=1560, q_max=1560, past_min=0, past_max=0,
             prefix=23400, heads=12, kv_heads=12, head_dim=128, dtype="bf16", lens=8),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


MOST_FLOPS = 3.0e12     # below the largest listed attention case
MOST_CACHE = 1.0e9      # bytes of keys and values


def draw(rng):
    op = rng.choice(["rotary", "packed", "packed", "prefix", "prefix"])
    while True:
        dtype = "fp32" if rng.random() < 0.2 else "bf16"
        head_dim = rng.choice([64, 128])
        kv_heads = rng.choice([1, 2, 3, 4, 5, 8])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
        if op == "rotary":
            axes = rng.random() < 0.3
            fused = not axes and rng.random() < 0.4
            form = "packed" if fused or rng.random() < 0.5 else "heads"
            frames = rng.randint(1, 21) if axes else 0
            tokens = frames * rng.randint(1, 45) * rng.randint(1, 52) if axes else _log_int(rng, 1, 65536)
            scaling = rng.choice(["none", "linear", "base", "ramp"])
            case = dict(op=op, form=form, batch=rng.randint(1, 3) if form == "heads" else 1, tokens=tokens,
                        frames=frames, heads=heads, kv_heads=kv_heads, head_dim=head_dim,
                        rotary_dim=head_dim if axes else rng.choice([16, 32, head_dim // 2, head_dim]),
                        layout=rng.choice(["half", "interleaved"]), scaling=scaling,
                        factor=1.0 if scaling == "none" else float(rng.choice([2, 4, 8, 16])), dtype=dtype,
                        backward=rng.random() < 0.4, fused=fused, start=0 if axes else _log_int(rng, 1, 1000000))
            if work(case)["bytes"] <= 8.0e8:
                return case
            continue
        tokens = rng.random() < 0.5   # single tokens behind caches, or prompts
        if dtype == "fp32":
            q_max, seqs = (1, rng.randint(1, 16)) if tokens else (_log_int(rng, 2, 2000), rng.randint(1, 6))
            past_max = _log_int(rng, 1, 4000)
        else:
            q_max, seqs = (rng.choice([1, 1, 2, 3]), _log_int(rng, 1, 64)) if tokens else (
                _log_int(rng, 8, 20000), _log_int(rng, 1, 24))
            past_max = _log_int(rng, 8, 12000)
        case = dict(op=op, seqs=seqs, q_min=1 if rng.random() < 0.7 else q_max, q_max=q_max,
                    past_min=rng.randint(0, past_max), past_max=past_max)
        if op == "prefix":
            case["prefix"] = _log_int(rng, 100, 4000 if dtype == "fp32" else 40000)
        case.update(heads=heads, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype, lens=rng.randint(10, 10 ** 6))
        w = work(case)
        cache = 2 * sum(_lengths(case)[1]) * kv_heads * head_dim * (4 if dtype == "fp32" else 2)
        if w["flops"] <= (3.0e10 if dtype == "fp32" else MOST_FLOPS) and cache <= MOST_CACHE and w["flops"] > 0:
            return case


def _lengths(case):
    """Queries and keys of each sequence; they belong to the case, not to the seed."""
    r = random.Random(case["lens"])
    q, kv = [], []
    for _ in range(case["seqs"]):
        n = case["q_max"] if case["q_min"] == case["q_max"] else _log_int(r, case["q_min"], case["q_max"])
        q.append(n)
        kv.append(n + r.randint(case["past_min"], case["past_max"]))
    if case["seqs"] >= 24 and case["past_max"] == 0:
        q[3], kv[3] = 0, 0            # an empty sequence
        kv[5] = max(0, q[5] - 2)      # fewer keys than queries: the first two rows see nothing
    return q, kv


def _visible(case):
    """(query, key) pairs that count, per query head."""
    pre, pairs = case.get("prefix", 0), 0
    for n, m in zip(*_lengths(case)):
        first = m - n                                   # query i sees max(0, i + first + 1) of its keys
        lo = max(0, -first)                             # queries before `lo` see none
        k = n - lo
        pairs += n * pre + k * (lo + first + 1) + k * (k - 1) // 2
    return pairs


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rotary":
        axes = 3 if case["frames"] else 1
        rows = case["batch"] * case["tokens"]
        values = rows * (case["heads"] + case["kv_heads"]) * case["head_dim"]
        turned = rows * (case["heads"] + case["kv_heads"]) * case["rotary_dim"]
        return {"bytes": 2 * values * size + 4 * axes * case["tokens"], "flops": 3 * turned}
    q, kv = _lengths(case)
    rows, keys = sum(q), sum(kv) + case.get("prefix", 0)
    d, h, hk = case["head_dim"], case["heads"], case["kv_heads"]
    return {"bytes": size * d * (2 * rows * h + 2 * keys * hk) + 4 * rows * h,
            "flops": 4 * d * h * _visible(case)}


# ------------------------------------------------------------------ inputs

def _frequencies(case):
    """64-bit frequency of each rotated pair, the axis it turns by, and the amplitude."""
    pairs = case["rotary_dim"] // 2
    if case["frames"]:
        side = pairs // 3
        sections = [pairs - 2 * side, side, side]
    else:
        sections = [pairs]
    freq, axis = [], []
    base, f, orig = 10000.0, case["factor"], 4096.0
    for a, s in enumerate(sections):
        b = base * f ** (2 * s / (2 * s - 2)) if case["scaling"] == "base" and s > 1 else base
        w = torch.tensor(b, dtype=torch.float64) ** (-torch.arange(s, dtype=torch.float64) / s)
        if case["scaling"] == "linear":
            w = w / f
        if case["scaling"] == "ramp":
            keep = ((orig * w / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
            w = keep * w + (1 - keep) * w / f
        freq.append(w)
        axis += [a] * s
    amp = 1.0 + 0.1 * math.log(f) if case["scaling"] == "ramp" else 1.0
    return torch.cat(freq).cuda(), torch.tensor(axis, device="cuda"), amp, sections


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def rand(*shape, gain=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * gain).to(dt)

    state = {"case": case}
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "rotary":
        n, b = case["tokens"], case["batch"]
        if case["fused"]:
            qkv = rand(n, h + 2 * hk, d)
            state["Q"], state["K"] = qkv[:, :h], qkv[:, h:h + hk]
        elif case["form"] == "packed":
            state["Q"], state["K"] = rand(n, h, d), rand(n, hk, d)
        else:
            state["Q"], state["K"] = rand(b, h, n, d), rand(b, hk, n, d)
        if case["frames"]:                      # frame, row and column of each token of the grid
            per = n // case["frames"]
            width = max(w for w in range(1, 53) if per % w == 0)
            i = torch.arange(n, device="cuda")
            pos = torch.stack([i // per, i % per // width, i % width])
        elif n <= 256:                          # single tokens of different sequences
            pos = torch.randint(0, case["start"] + 1, (n,), generator=g, device="cuda")
        else:
            pos = torch.arange(n, device="cuda") + case["start"]
        state["pos"] = pos.to(torch.int32)
        state["freq"], state["axis"], state["amp"], sections = _frequencies(case)
        if own:
            from token_level_sparse_pddp_b200 import tlsp
            state["plan"] = tlsp.RotaryPlan(
                d, rotary_dim=case["rotary_dim"], layout=case["layout"], scaling=case["scaling"],
                factor=case["factor"], original_len=4096, sections=sections)
        return state
    q, kv = _lengths(case)
    state["q_lens"], state["kv_lens"], state["prefix"] = q, kv, case.get("prefix", 0)
    state["Q"] = rand(sum(q), h, d, gain=2.0)           # logits of a few nats
    state["K"], state["V"] = rand(sum(kv), hk, d), rand(sum(kv), hk, d)
    if state["prefix"]:
        state["Kp"], state["Vp"] = rand(state["prefix"], hk, d), rand(state["prefix"], hk, d)
    if own:
        from token_level_sparse_pddp_b200 import tlsp
        state["plan"] = tlsp.PackedPlan(q, kv, heads=h, kv_heads=hk, head_dim=d, dtype=dt,
                                        prefix_len=state["prefix"])
        state["ws"] = state["plan"].workspace()
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if case["op"] == "rotary":
        if own:
            from token_level_sparse_pddp_b200 import tlsp
            f = tlsp.rotary_backward if case["backward"] else tlsp.rotary
            return f(state["Q"], state["K"], state["pos"], state["plan"])
        return _plain_rotary(state)
    if own:
        from token_level_sparse_pddp_b200 import tlsp
        lse = torch.empty(state["Q"].shape[:2], dtype=torch.float32, device="cuda")
        if state["prefix"]:
            O = tlsp.prefix_attention(state["Q"], state["Kp"], state["Vp"], state["K"], state["V"],
                                      state["plan"], state["ws"], lse=lse)
        else:
            O = tlsp.packed_attention(state["Q"], state["K"], state["V"], state["plan"], state["ws"], lse=lse)
        return O, lse
    return _plain_attention(state)


def _plain_rotary(state):
    case = state["case"]
    r, half = case["rotary_dim"], case["rotary_dim"] // 2
    pos = state["pos"].double().reshape(-1, state["pos"].shape[-1])
    angle = pos[state["axis"]].T * state["freq"]                     # [tokens, pairs]
    if case["backward"]:
        angle = -angle
    c, s = (angle.cos() * state["amp"]).float(), (angle.sin() * state["amp"]).float()
    if case["form"] == "packed":
        c, s = c[:, None], s[:, None]                                # broadcast over heads

    def turn(x):
        f = x.float()
        a, b = (f[..., :half], f[..., half:r]) if case["layout"] == "half" else (f[..., 0:r:2], f[..., 1:r:2])
        y = [a * c - b * s, b * c + a * s]
        y = torch.cat(y, -1) if case["layout"] == "half" else torch.stack(y, -1).flatten(-2)
        return torch.cat([y, f[..., r:]], -1).to(x.dtype)

    return turn(state["Q"]), turn(state["K"])


def _plain_softmax(s, v):
    """Rows of scores s (masked: -inf) and values: the weighted sum and the log partition."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -torch.inf, torch.zeros_like(m), m)
    e = torch.exp(s - m)
    z = e.sum(-1, keepdim=True)
    return e @ v / torch.where(z == 0, torch.ones_like(z), z), (m + torch.log(z)).squeeze(-1)


def _plain_attention(state):
    return _plain_tokens(state) if max(state["q_lens"]) <= 4 else _plain_prompts(state)


def _plain_tokens(state):
    """Few queries in each sequence: sequences padded to one length, the prefix scored for all at once."""
    Q, K, V, dev = state["Q"], state["K"], state["V"], state["Q"].device
    t, h, d = Q.shape
    hk = K.shape[1]
    n, m = (torch.tensor(state[x], device=dev) for x in ("q_lens", "kv_lens"))
    seqs, nq, nk = len(n), max(state["q_lens"]), max(max(state["kv_lens"]), 1)
    i, j = torch.arange(nq, device=dev), torch.arange(nk, device=dev)
    iq = (n.cumsum(0) - n)[:, None] + i
    ik = ((m.cumsum(0) - m)[:, None] + j).clamp(max=K.shape[0] - 1)
    q = Q[iq.clamp(max=t - 1)].float().view(seqs, nq, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(seqs, hk, -1, d)
    seen = (j < m[:, None])[:, None, :] & (j[None, None, :] <= i[None, :, None] + (m - n)[:, None, None])
    k, v = (x[ik].float().permute(0, 2, 1, 3) for x in (K, V))
    s = (q @ k.transpose(-1, -2) / math.sqrt(d)).view(seqs, hk, h // hk, nq, nk)
    s = s.masked_fill(~seen[:, None, None], -torch.inf).view(seqs, hk, -1, nk)
    o, lse = _plain_softmax(s, v)
    if state["prefix"]:
        kp, vp = state["Kp"].float().transpose(0, 1), state["Vp"].float().transpose(0, 1)
        qa = q.transpose(0, 1).reshape(hk, -1, d)
        op, lp = _plain_softmax(qa @ kp.transpose(-1, -2) / math.sqrt(d), vp)
        op, lp = (x.view(hk, seqs, -1, *x.shape[2:]).transpose(0, 1) for x in (op, lp))
        both = torch.logaddexp(lse, lp)
        o = o * torch.exp(lse - both)[..., None] + op * torch.exp(lp - both)[..., None]
        lse = both
    o, lse = (x.view(seqs, hk, h // hk, nq, *x.shape[3:]).permute(0, 3, 1, 2, *range(4, x.dim() + 1))
              .reshape(seqs, nq, h, *x.shape[3:])[i < n[:, None]] for x in (o, lse))
    return o.to(Q.dtype), lse


def _plain_prompts(state):
    """Sequence by sequence, blocks of queries against all their keys."""
    Q, K, V = state["Q"], state["K"], state["V"]
    t, h, d = Q.shape
    hk = K.shape[1]
    O, lse = torch.empty_like(Q), torch.empty((t, h), dtype=torch.float32, device=Q.device)
    pre, q0, k0 = state["prefix"], 0, 0
    for n, m in zip(state["q_lens"], state["kv_lens"]):
        k, v = K[k0:k0 + m], V[k0:k0 + m]
        if pre:
            k, v = torch.cat([state["Kp"], k]), torch.cat([state["Vp"], v])
        k, v = k.float().permute(1, 2, 0), v.float().transpose(0, 1)
        block = max(1, (1 << 30) // (h * (m + pre) + 1))
        for b in range(0, n, block):
            e = min(n, b + block)
            last = pre + e + m - n if e + m - n > 0 else pre         # no query of the block sees further
            q = Q[q0 + b:q0 + e].float().view(e - b, hk, h // hk, d).permute(1, 2, 0, 3).reshape(hk, -1, d)
            s = (q @ k[..., :last]).mul_(1 / math.sqrt(d)).view(hk, h // hk, e - b, last)
            i = torch.arange(b, e, device=Q.device)[:, None] + (pre + m - n)
            j = torch.arange(last, device=Q.device)
            s = s.masked_fill_((j > i) & (j >= pre), -torch.inf).view(hk, -1, last)
            if last:
                o, z = _plain_softmax(s, v[:, :last])
            else:
                o, z = torch.zeros_like(q), torch.full(q.shape[:2], -torch.inf, device=Q.device)
            O[q0 + b:q0 + e] = o.view(hk, h // hk, e - b, d).permute(2, 0, 1, 3).reshape(e - b, h, d)
            lse[q0 + b:q0 + e] = z.view(h, e - b).T
        q0, k0 = q0 + n, k0 + m
    return O, lse


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    return _exact_rotary(state) if case["op"] == "rotary" else _exact_attention(state)


def _exact_rotary(state):
    """Each pair as a complex number times A exp(i angle)."""
    case = state["case"]
    pairs, r = case["rotary_dim"] // 2, case["rotary_dim"]
    where = state["pos"].view(-1, case["tokens"]).double()
    turn = torch.empty(case["tokens"], pairs, dtype=torch.complex128, device="cuda")
    for p in range(pairs):
        angle = where[int(state["axis"][p])] * float(state["freq"][p])
        turn[:, p] = torch.polar(torch.full_like(angle, state["amp"]), -angle if case["backward"] else angle)
    if case["form"] == "packed":
        turn = turn.unsqueeze(1)
    outs = []
    for x in (state["Q"], state["K"]):
        y = x.double().clone()
        first = slice(0, pairs) if case["layout"] == "half" else slice(0, r, 2)
        second = slice(pairs, r) if case["layout"] == "half" else slice(1, r, 2)
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        outs.append(y)
    return tuple(outs)


def _exact_attention(state):
    Q, case = state["Q"], state["case"]
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    O = torch.zeros(Q.shape, dtype=torch.float64, device="cuda")
    L = torch.full(Q.shape[:2], -torch.inf, dtype=torch.float64, device="cuda")
    starts, at, kt = [], 0, 0
    for n, m in zip(state["q_lens"], state["kv_lens"]):
        starts.append((at, n, kt, m))
        at, kt = at + n, kt + m
    pre = state["prefix"]
    for at, n, kt, m in starts:
        if n == 0 or m + pre == 0:
            continue
        step = max(1, (1 << 28) // (m + pre))
        for head in range(h):
            kv = head // (h // hk)
            k, v = state["K"][kt:kt + m, kv].double(), state["V"][kt:kt + m, kv].double()
            if pre:
                k = torch.cat([state["Kp"][:, kv].double(), k])
                v = torch.cat([state["Vp"][:, kv].double(), v])
            for b in range(0, n, step):
                rows = torch.arange(b, min(n, b + step), device="cuda")
                logits = Q[at + rows, head].double() @ k.T / math.sqrt(d)
                own_key = torch.arange(m + pre, device="cuda") - pre
                logits[own_key[None] > rows[:, None] + (m - n)] = -torch.inf
                if pre:
                    logits[:, :pre] = Q[at + rows, head].double() @ k[:pre].T / math.sqrt(d)
                z = torch.logsumexp(logits, -1)
                w = torch.exp(logits - torch.where(z == -torch.inf, 0.0, z)[:, None])
                O[at + rows, head] = w @ v
                L[at + rows, head] = z
    return O, L
