"""Cases, inputs and plain forms of the paged-cache serving operators.

Four operators of one serving step with a paged key-value cache:

* ``rotary_multi_axis``: rotary positions with several axes (time, height, width) on q and k;
* ``paged_kv_append``: the new K/V rows of a packed batch, rotated, written into the cache's pages
  (q is rotated in the same pass);
* ``attention_packed_prefill``: attention over whole prompts packed one after another;
* ``attention_paged_decode``: attention of one new token per sequence over its pages.

With ``own`` false ``run`` computes them from elementary torch operations in 32 bits (angles in 64);
with ``own`` true it makes the library's calls.
"""
import math

import torch

own = False


def _library():
    from biased_gqa_attention_gb300 import extkv
    return extkv


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


# ---- cases -----------------------------------------------------------------------------------------


def listed():
    return [
        # one chat continuing: a single sequence, a short cache, where the call's latency is everything
        dict(name="decode_one", op="decode", type="bf16", lens="517", Hq=16, Hkv=8, D=256, page=16, window=0),
        # a small batch on a sliding-window layer: only the window's pages are live
        dict(name="decode_window", op="decode", type="bf16", lens="3291,877,4096,1024,513,2050,1999,3700",
             Hq=16, Hkv=8, D=256, page=16, window=1024),
        # a full batch on a global layer with wide heads, lengths from 1 to 8192
        dict(name="decode_wide", op="decode", type="bf16",
             lens="8192,1,4096,17,8191,333,2500,7001,64,5120,1023,6666,4097,129,3333,7777,2048,905,31,5999,"
                  "1500,8000,4444,256,6100,12,3800,7300,700,5500,2222,6401",
             Hq=16, Hkv=2, D=512, page=32, window=0),
        # a few very long documents, sixteen query heads on each key-value head
        dict(name="decode_long", op="decode", type="bf16", lens="131071,65537,12345", Hq=32, Hkv=2, D=128,
             page=64, window=0),
        # a handful of short prompts in full precision
        dict(name="prompt_f32", op="prefill", type="f32", lens="16,1,137,64", Hq=4, Hkv=2, D=64, causal=True,
             window=0, fused_qkv=False),
        # arrivals of one scheduling step: prompts of very different lengths, q, k and v slices of one projection
        dict(name="prompt_ragged", op="prefill", type="bf16",
             lens="17,1200,3,512,90,2047,1,640,333,128,1801,45", Hq=8, Hkv=4, D=128, causal=True, window=4096,
             fused_qkv=True),
        # a sliding-window layer with wide heads
        dict(name="prompt_window", op="prefill", type="bf16", lens="4096,2048,1500", Hq=16, Hkv=8, D=256,
             causal=True, window=1024, fused_qkv=False),
        # one long document
        dict(name="prompt_long", op="prefill", type="bf16", lens="16001", Hq=8, Hkv=4, D=128, causal=True,
             window=0, fused_qkv=False),
        # the rows of one decode step of a small batch
        dict(name="append_step", op="append", type="bf16", lens="1,1,1,1,1,1,1,1", past=4000, Hq=16, Hkv=8, D=256,
             page=16, R=256, axes=3, interleaved=False),
        # the rows of a packed prompt with images in it
        dict(name="append_prompt", op="append", type="bf16", lens="4096,2047,1200,801", past=0, Hq=32, Hkv=2, D=128,
             page=64, R=128, axes=3, interleaved=False),
        # a tiny step in full precision, text positions only, adjacent pairs
        dict(name="rotary_f32", op="rotary", type="f32", B=1, S=16, past=0, Hq=4, Hkv=2, D=64, R=64, axes=1,
             interleaved=True),
        # a prefill chunk of a video prompt far into a long context, three quarters of each head rotated
        dict(name="rotary_video", op="rotary", type="bf16", B=2, S=4097, past=1000000, Hq=16, Hkv=8, D=256, R=192,
             axes=3, interleaved=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, B, longest, total):
    """B lengths, log-spread up to `longest`, cut so that they sum to `total` at most."""
    out, left = [], total
    for i in range(B):
        n = max(1, min(_log_int(rng, 1, longest), left - (B - 1 - i)))
        out.append(n)
        left -= n
    rng.shuffle(out)
    return ",".join(str(n) for n in out)


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "append", "rotary"])
    kind = "f32" if rng.random() < 0.2 else "bf16"
    D = rng.choice([64, 128, 256] + ([512] if op == "decode" else []))
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 6, 8] + ([16] if Hkv <= 2 else []))
    if op == "decode":
        row = Hkv * D * _BYTES[kind] * 2
        longest = _log_int(rng, 64, 100000 if kind == "bf16" else 20000)
        B = _log_int(rng, 1, 48)
        budget = (200 << 20) if kind == "bf16" else (60 << 20)
        return dict(op=op, type=kind, lens=_lens(rng, B, longest, max(B, budget // row)), Hq=Hkv * g, Hkv=Hkv, D=D,
                    page=rng.choice([16, 32, 64, 128]), window=rng.choice([0, 0, _log_int(rng, 16, 4096)]))
    if op == "prefill":
        B = _log_int(rng, 1, 24)
        longest = _log_int(rng, 8, 6000) if kind == "bf16" else _log_int(rng, 8, 500)
        total = 9000 if kind == "bf16" else 1500
        longest = min(longest, int(math.sqrt(2e9 / (B * Hkv * g))))  # the padded scores of a plain form fit
        return dict(op=op, type=kind, lens=_lens(rng, B, longest, total), Hq=Hkv * g, Hkv=Hkv, D=D,
                    causal=rng.random() < 0.8, window=rng.choice([0, 0, _log_int(rng, 16, 4096)]),
                    fused_qkv=rng.random() < 0.5)
    R = rng.choice([D, D, D // 2])
    axes = rng.choice([1, 2, 3])
    if op == "append":
        if rng.random() < 0.5:
            lens = ",".join(["1"] * _log_int(rng, 1, 256))
        else:
            lens = _lens(rng, _log_int(rng, 1, 16), 4096, 8000)
        return dict(op=op, type=kind, lens=lens, past=rng.choice([0, _log_int(rng, 1, 5000)]), Hq=Hkv * g, Hkv=Hkv,
                    D=D, page=rng.choice([16, 32, 64, 128]), R=R, axes=axes, interleaved=rng.random() < 0.3)
    B = _log_int(rng, 1, 16)
    return dict(op=op, type=kind, B=B, S=max(1, _log_int(rng, 1, 4000) // B), past=rng.choice([0, _log_int(rng, 1, 1000000)]),
                Hq=Hkv * g, Hkv=Hkv, D=D, R=R, axes=axes, interleaved=rng.random() < 0.3)


def _lengths(case):
    return [int(n) for n in case["lens"].split(",")]


def _sections(case):
    """Pairs of each axis: two axes split evenly, three as 1/4 time, 3/8 height, 3/8 width."""
    half = case["R"] // 2
    if case["axes"] == 1:
        return (half,)
    if case["axes"] == 2:
        return (half // 2, half - half // 2)
    a = half // 4
    b = (half - a) // 2
    return (a, b, half - a - b)


def _pairs(case):
    """(query, key) pairs a prompt attends."""
    total = 0
    for n in _lengths(case):
        w = case["window"] if 0 < case["window"] < n else n
        causal = w * (w + 1) // 2 + (n - w) * w
        total += causal if case["causal"] else causal + n * (n - 1) // 2
    return total


def work(case):
    e, D, Hq, Hkv = _BYTES[case["type"]], case["D"], case["Hq"], case["Hkv"]
    if case["op"] == "decode":
        lens = _lengths(case)
        live = [min(n, case["window"]) if case["window"] > 0 else n for n in lens]
        pages = sum((n - 1) // case["page"] - (n - m) // case["page"] + 1 for n, m in zip(lens, live))
        return {"bytes": sum(live) * Hkv * D * 2 * e + 2 * len(lens) * Hq * D * e + 8 * pages + 8 * len(lens),
                "flops": 4 * D * Hq * sum(live)}
    if case["op"] == "prefill":
        T = sum(_lengths(case))
        return {"bytes": T * D * e * (2 * Hq + 2 * Hkv) + 8 * len(_lengths(case)), "flops": 4 * D * Hq * _pairs(case)}
    if case["op"] == "append":
        T = sum(_lengths(case))
        return {"bytes": T * D * e * (2 * Hq + 4 * Hkv) + 8 * T * case["axes"], "flops": 3 * T * case["R"] * (Hq + Hkv)}
    T = case["B"] * case["S"]
    return {"bytes": T * D * e * 2 * (Hq + Hkv) + 8 * T * case["axes"], "flops": 3 * T * case["R"] * (Hq + Hkv)}


# ---- inputs ----------------------------------------------------------------------------------------


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _normal(gen, shape, dtype, sigma=1.0):
    x = torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32)
    return (x * sigma if sigma != 1.0 else x).to(dtype)


def _positions(case, gen, starts, lens):
    """(axes, tokens) positions: runs of text, where all axes agree, and images, where the first axis
    stands still while the others walk over rows and columns of a grid 24 patches wide."""
    rows = []
    for s, n in zip(starts, lens):
        i = torch.arange(n, device=gen.device)
        image = (i // 577) % 2 == 1
        k = i % 577
        t = torch.where(image, i - k, i)
        rows.append(torch.stack([t, torch.where(image, t + k // 24, i), torch.where(image, t + k % 24, i)]) + s)
    return torch.cat(rows, 1)[: case["axes"]].contiguous()


def _rotary_inputs(case, gen, starts, lens):
    half = case["R"] // 2
    inv = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).to(torch.float32).to(gen.device)
    return _positions(case, gen, starts, lens), inv


def _pages_for(case, gen, lens):
    """Random pages for sequences of these lengths in a pool that holds other pages too."""
    ps = case["page"]
    need = [(n + ps - 1) // ps for n in lens]
    width = max(need) + 1
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=gen, device=gen.device)
    table = torch.full((len(lens), width), -1, dtype=torch.int64, device=gen.device)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return pool, table


def _inputs(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 11)
    dt, D, Hq, Hkv = _TYPES[case["type"]], case["D"], case["Hq"], case["Hkv"]
    s = dict(case=case, scale=1.0 / math.sqrt(D))
    if case["op"] == "decode":
        lens = _lengths(case)
        pool, table = _pages_for(case, gen, lens)
        s.update(q=_normal(gen, (len(lens), Hq, D), dt, 2.0), table=table, longest=max(lens),
                 nonpad=torch.tensor(lens, dtype=torch.int64, device=dev),
                 k=_normal(gen, (pool, Hkv, case["page"], D), dt), v=_normal(gen, (pool, Hkv, case["page"], D), dt))
        s["y"] = torch.empty_like(s["q"])
    elif case["op"] == "prefill":
        lens = _lengths(case)
        T = sum(lens)
        if case["fused_qkv"]:
            qkv = _normal(gen, (T, Hq + 2 * Hkv, D), dt)
            q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            q, k, v = (_normal(gen, (T, h, D), dt) for h in (Hq, Hkv, Hkv))
        q.mul_(2.0)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s.update(q=q, k=k, v=v, cu=torch.tensor(cu, dtype=torch.int64, device=dev), longest=max(lens),
                 y=torch.empty((T, Hq, D), dtype=dt, device=dev))
    elif case["op"] == "append":
        lens = _lengths(case)
        T = sum(lens)
        starts = [case["past"] + (37 * b) % 101 if case["past"] else 0 for b in range(len(lens))]
        pool, table = _pages_for(case, gen, [a + n for a, n in zip(starts, lens)])
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        pos, inv = _rotary_inputs(case, gen, starts, lens)
        s.update(q=_normal(gen, (T, Hq, D), dt), k_new=_normal(gen, (T, Hkv, D), dt), v_new=_normal(gen, (T, Hkv, D), dt),
                 table=table, write_idx=torch.tensor(starts, dtype=torch.int64, device=dev),
                 cu=torch.tensor(cu, dtype=torch.int64, device=dev), pos=pos, inv=inv,
                 k=_normal(gen, (pool, Hkv, case["page"], D), dt), v=_normal(gen, (pool, Hkv, case["page"], D), dt))
        s["q_out"] = torch.empty_like(s["q"])
    else:
        B, S = case["B"], case["S"]
        starts = [case["past"] + 11 * b for b in range(B)]
        pos, inv = _rotary_inputs(case, gen, starts, [S] * B)
        s.update(q=_normal(gen, (B, Hq, S, D), dt), k=_normal(gen, (B, Hkv, S, D), dt), pos=pos.reshape(-1, B, S), inv=inv)
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # the handle that a loop repeating the call over its buffers keeps
        s["call"] = _prepared(s)
    return s


# ---- the library's calls -----------------------------------------------------------------------------


def _prepared(s):
    """The operator's call with its arguments marshalled once, as a serving loop keeps it."""
    ek, case = _library(), s["case"]
    if case["op"] == "decode":
        return ek.prepare_attention_paged_decode(s["y"], s["q"], s["k"], s["v"], s["table"], s["nonpad"], s["scale"],
                                                 window=case["window"])
    if case["op"] == "prefill":
        return ek.prepare_attention_packed_prefill(s["y"], s["q"], s["k"], s["v"], s["cu"], s["scale"],
                                                   causal=case["causal"], window=case["window"])
    rotary = ek.RotarySpec(positions=s["pos"], inv_freq=s["inv"], sections=_sections(case),
                           interleaved=case["interleaved"])
    if case["op"] == "append":
        return ek.prepare_paged_kv_append(s["k"], s["v"], s["k_new"], s["v_new"], s["table"], s["write_idx"],
                                          cu_seqlens=s["cu"], rotary=rotary, q_out=s["q_out"], q=s["q"])
    return ek.prepare_rotary_multi_axis(s["q_out"], s["k_out"], s["q"], s["k"], rotary)


# ---- plain forms -------------------------------------------------------------------------------------


def _softmax_rows(score, live):
    """Softmax over the last axis of the live entries; zeros where a row has none."""
    score = torch.where(live, score, torch.full((), -math.inf, device=score.device))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, p / total, torch.zeros_like(p))


def _plain_decode(s):
    case, q = s["case"], s["q"].float()
    B, Hq, D = q.shape
    Hkv, ps = case["Hkv"], case["page"]
    n_pages = (s["longest"] + ps - 1) // ps
    pages = s["table"][:, :n_pages].clamp(min=0)
    k, v = (t[pages].transpose(1, 2).reshape(B, Hkv, n_pages * ps, D).float() for t in (s["k"], s["v"]))
    j = torch.arange(n_pages * ps, device=q.device)
    n = s["nonpad"][:, None]
    live = j < n
    if case["window"] > 0:
        live &= j >= n - case["window"]
    score = torch.matmul(q.view(B, Hkv, Hq // Hkv, D), k.transpose(2, 3)) * s["scale"]
    p = _softmax_rows(score, live[:, None, None, :])
    v = torch.where(live[:, None, :, None], v, torch.zeros_like(v))
    return torch.matmul(p, v).view(B, Hq, D).to(s["q"].dtype)


def _plain_prefill(s):
    case, cu, L = s["case"], s["cu"], s["longest"]
    T, Hq, D = s["q"].shape
    Hkv, B = case["Hkv"], cu.numel() - 1
    i = torch.arange(L, device=cu.device)
    n = cu[1:] - cu[:-1]
    row = torch.where(i < n[:, None], cu[:-1, None] + i, torch.zeros_like(i))  # (B, L) padded
    q, k, v = (s[x][row].transpose(1, 2).float() for x in ("q", "k", "v"))     # (B, H, L, D)
    score = torch.matmul(q.reshape(B, Hkv, Hq // Hkv * L, D), k.transpose(2, 3)) * s["scale"]
    live = (i < n[:, None])[:, None, :].expand(B, L, L)
    ahead = i[:, None] - i[None, :]
    if case["causal"]:
        live = live & (ahead >= 0)
    if case["window"] > 0:
        live = live & (ahead < case["window"])
    p = _softmax_rows(score.view(B, Hkv, Hq // Hkv, L, L), live[:, None, None])
    y = torch.matmul(p.view(B, Hkv, Hq // Hkv * L, L), v).view(B, Hq, L, D).transpose(1, 2)
    return y[i < n[:, None]].to(s["q"].dtype)


def _cos_sin(s):
    """cos and sin of every token's angles, (..., R/2): angles in 64 bits, rounded once."""
    case = s["case"]
    axis = torch.repeat_interleave(torch.arange(case["axes"], device=s["inv"].device),
                                   torch.tensor(_sections(case), device=s["inv"].device), output_size=case["R"] // 2)
    angle = s["pos"].double()[axis].movedim(0, -1) * s["inv"].double()
    return torch.cos(angle).float(), torch.sin(angle).float()


def _rotate(x, cos, sin, R, interleaved):
    y = x.float().clone()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    xa, xb = y[..., a].clone(), y[..., b].clone()
    y[..., a] = xa * cos - xb * sin
    y[..., b] = xb * cos + xa * sin
    return y.to(x.dtype)


def _plain_append(s):
    case, cu = s["case"], s["cu"]
    cos, sin = (x[:, None] for x in _cos_sin(s))
    t = torch.arange(s["q"].shape[0], device=cu.device)
    b = torch.bucketize(t, cu[1:], right=True)
    slot = s["write_idx"][b] + t - cu[b]
    page = s["table"][b, slot // case["page"]]
    s["k"][page, :, slot % case["page"]] = _rotate(s["k_new"], cos, sin, case["R"], case["interleaved"])
    s["v"][page, :, slot % case["page"]] = s["v_new"]
    return s["k"], s["v"], _rotate(s["q"], cos, sin, case["R"], case["interleaved"])


def _plain_rotary(s):
    case = s["case"]
    cos, sin = (x[:, None] for x in _cos_sin(s))
    return tuple(_rotate(s[x], cos, sin, case["R"], case["interleaved"]) for x in ("q", "k"))


def run(state):
    op = state["case"]["op"]
    if own:
        state["call"]()
        if op == "append":
            return state["k"], state["v"], state["q_out"]
        if op == "rotary":
            return state["q_out"], state["k_out"]
        return state["y"]
    return {"decode": _plain_decode, "prefill": _plain_prefill, "append": _plain_append, "rotary": _plain_rotary}[op](state)


# ---- the definitions in 64 bits ------------------------------------------------------------------------


def _exact_head(q, k, v, allowed, scale):
    """softmax(scale q k^T) v over the allowed keys of each row, in 64 bits."""
    w = (q.double() @ k.double().T) * scale
    w = w.masked_fill(~allowed, -math.inf)
    w = torch.exp(w - w.amax(1, keepdim=True))
    return (w @ v.double()) / w.sum(1, keepdim=True)


def _exact_turn(x, pos, inv, sections, R, interleaved):
    """x (..., D) turned pair by pair by pos[axis] * inv[pair]; pos (axes, ...) in x's leading shape."""
    out = x.double().clone()
    first = 0
    for axis, count in enumerate(sections):
        for i in range(first, first + count):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
            ang = pos[axis].double() * float(inv[i])
            c, d = torch.cos(ang), torch.sin(ang)
            out[..., a] = x[..., a].double() * c - x[..., b].double() * d
            out[..., b] = x[..., a].double() * d + x[..., b].double() * c
        first += count
    return out


def exact(case, seed):
    w = work(case)
    if w["flops"] > 6e12 or (case["op"] == "prefill" and max(_lengths(case)) > 20000):
        return None
    s = _inputs(case, seed)
    if case["op"] == "decode":
        g, ps = case["Hq"] // case["Hkv"], case["page"]
        y = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
        for b, n in enumerate(_lengths(case)):
            lo = max(0, n - case["window"]) if case["window"] > 0 else 0
            j = torch.arange(lo, n, device=y.device)
            at, off = s["table"][b][j // ps], j % ps
            for h in range(case["Hkv"]):
                rows = slice(h * g, h * g + g)
                ok = torch.ones((g, n - lo), dtype=torch.bool, device=y.device)
                y[b, rows] = _exact_head(s["q"][b, rows], s["k"][at, h, off], s["v"][at, h, off], ok, s["scale"])
        return y
    if case["op"] == "prefill":
        g = case["Hq"] // case["Hkv"]
        y = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
        t0 = 0
        for n in _lengths(case):
            at = slice(t0, t0 + n)
            p = torch.arange(n, device=y.device)
            ok = torch.ones((n, n), dtype=torch.bool, device=y.device)
            if case["causal"]:
                ok &= p[None, :] <= p[:, None]
            if case["window"] > 0:
                ok &= p[:, None] - p[None, :] < case["window"]
            for h in range(case["Hq"]):
                y[at, h] = _exact_head(s["q"][at, h], s["k"][at, h // g], s["v"][at, h // g], ok, s["scale"])
            t0 += n
        return y
    inv = s["inv"].tolist()
    turn = lambda x, pos: _exact_turn(x, pos, inv, _sections(case), case["R"], case["interleaved"])  # noqa: E731
    if case["op"] == "rotary":
        pos = s["pos"][:, :, None, :]
        return tuple(turn(s[x], pos) for x in ("q", "k"))
    pos = s["pos"][:, :, None]
    q, kr = turn(s["q"], pos), turn(s["k_new"], pos)
    k, v = s["k"].double(), s["v"].double()
    t0, ps = 0, case["page"]
    for b, n in enumerate(_lengths(case)):
        slot = int(s["write_idx"][b]) + torch.arange(n, device=k.device)
        at = s["table"][b][slot // ps]
        k[at, :, slot % ps] = kr[t0:t0 + n]
        v[at, :, slot % ps] = s["v_new"][t0:t0 + n].double()
        t0 += n
    return k, v, q
