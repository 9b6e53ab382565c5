"""What stands between the QKV projection and the output projection of a W8A8
layer, in its plain form and through the library's calls: the rotary table, the
rotation with the append to a paged 8-bit key/value cache, the cache read back,
attention of the newest tokens over that cache, and attention over whole
prompts.

A case's "op" names the operator:
  table      cos/sin of every position and frequency, scaled for long contexts
  append     rotate q and k, quantize k and v into the cache's blocks
  read       a range of every sequence's cached tokens, as values
  attend     the last `q_len` tokens of every sequence over its cached tokens
  prompt     packed prompts over themselves
Lengths of a ragged batch follow from the case alone (its "mix")."""
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the table of a short-context model, built at load
        {"name": "table 4k", "op": "table", "n_pos": 4096, "rot": 128, "theta": 1e4, "factor": 1.0,
         "low": 0.0, "high": 0.0, "orig": 0, "mag": 1.0},
        # the table of a long-context model whose slow frequencies are stretched eightfold
        {"name": "table 128k scaled", "op": "table", "n_pos": 131072, "rot": 128, "theta": 5e5, "factor": 8.0,
         "low": 1.0, "high": 4.0, "orig": 8192, "mag": 1.0},
        # one decode step of 64 users: one new token each, 70B-like heads
        {"name": "append decode 64", "op": "append", "seqs": 64, "new": 1, "ctx": 4000, "hq": 64, "hkv": 8, "d": 128,
         "rot": 128, "ps": 64, "sb": 16, "pairs": False, "dt": "bf16", "mix": 1},
        # five prompts of a 7B-like layer that arrive together, some behind a cached prefix
        {"name": "append prompts 7b", "op": "append", "seqs": 5, "new": 1300, "ctx": 500, "hq": 32, "hkv": 32, "d": 128,
         "rot": 64, "ps": 64, "sb": 64, "pairs": True, "dt": "bf16", "mix": 2},
        # the cached prefix of one short chat, read back as values
        {"name": "read one prefix", "op": "read", "seqs": 1, "ctx": 777, "hkv": 8, "d": 128, "ps": 16, "sb": 16,
         "dt": "bf16", "mix": 3},
        # prefixes of sixteen users
        {"name": "read 16 prefixes", "op": "read", "seqs": 16, "ctx": 4096, "hkv": 32, "d": 128, "ps": 64, "sb": 16,
         "dt": "bf16", "mix": 4},
        # one user's next token: latency
        {"name": "attend one user", "op": "attend", "seqs": 1, "q_len": 1, "ctx": 700, "hq": 32, "hkv": 8, "d": 128,
         "ps": 16, "sb": 16, "dt": "bf16", "mix": 5},
        # a ragged batch of 64 users, 70B-like heads
        {"name": "attend ragged 64", "op": "attend", "seqs": 64, "q_len": 1, "ctx": 8192, "hq": 64, "hkv": 8, "d": 128,
         "ps": 64, "sb": 16, "dt": "bf16", "mix": 6},
        # one very long document
        {"name": "attend 128k", "op": "attend", "seqs": 1, "q_len": 1, "ctx": 131072, "hq": 64, "hkv": 8, "d": 128,
         "ps": 128, "sb": 64, "dt": "bf16", "mix": 7},
        # four proposed tokens checked at once, fp32 activations, every head its own keys, a scale for each token
        {"name": "attend 4 proposed f32", "op": "attend", "seqs": 8, "q_len": 4, "ctx": 2000, "hq": 32, "hkv": 32,
         "d": 128, "ps": 32, "sb": 1, "dt": "f32", "mix": 8},
        # a handful of short prompts, small heads
        {"name": "prompt short d64", "op": "prompt", "seqs": 6, "len": 300, "hq": 16, "hkv": 4, "d": 64, "causal": True,
         "mix": 9},
        # two long prompts packed, 70B-like heads
        {"name": "prompt 2 long 70b", "op": "prompt", "seqs": 2, "len": 5000, "hq": 64, "hkv": 8, "d": 128,
         "causal": True, "mix": 10},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["table", "append", "append", "read", "attend", "attend", "attend", "prompt", "prompt"])
    mix = rng.randrange(1 << 20)
    if op == "table":
        scaled = rng.random() < 0.5
        return {"op": op, "n_pos": _log(rng, 1000, 131072), "rot": rng.choice([16, 32, 64, 128]),
                "theta": rng.choice([1e4, 5e5, 1e6]), "factor": rng.choice([2.0, 8.0, 32.0]) if scaled else 1.0,
                "low": 1.0 if scaled else 0.0, "high": 4.0 if scaled else 0.0, "orig": 8192 if scaled else 0,
                "mag": 1.0 + 0.1 * rng.randrange(3)}
    d = rng.choice([64, 128, 128])
    hq, hkv = rng.choice([(32, 32), (32, 8), (64, 8), (40, 40), (16, 2), (8, 1), (12, 4)])
    ps = rng.choice([16, 32, 64, 128])
    sb = rng.choice([b for b in (1, 2, 4, 8, 16, 32, 64, 128) if b <= ps])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op == "append":
        seqs = _log(rng, 1, 64)
        new = 1 if rng.random() < 0.5 else _log(rng, 2, max(2, 6000 // seqs))
        return {"op": op, "seqs": seqs, "new": new, "ctx": _log(rng, 1, 4000), "hq": hq, "hkv": hkv, "d": d,
                "rot": rng.choice([d, d // 2, d // 4]), "ps": ps, "sb": sb, "pairs": rng.random() < 0.5, "dt": dt, "mix": mix}
    if op == "read":
        seqs = _log(rng, 1, 16)
        return {"op": op, "seqs": seqs, "ctx": _log(rng, 1, 4096), "hkv": hkv, "d": d, "ps": ps, "sb": sb, "dt": dt, "mix": mix}
    if op == "attend":
        seqs = _log(rng, 1, 128)
        return {"op": op, "seqs": seqs, "q_len": rng.choice([1, 1, 1, 2, 5, 8]), "ctx": _log(rng, 20, max(20, min(131072, 500000 // seqs // (hkv // 8 + 1)))),
                "hq": hq, "hkv": hkv, "d": d, "ps": ps, "sb": sb, "dt": dt, "mix": mix}
    seqs = _log(rng, 1, 24)
    return {"op": op, "seqs": seqs, "len": _log(rng, 2, max(2, 6000 // seqs)), "hq": hq, "hkv": hkv, "d": d,
            "causal": rng.random() < 0.75, "mix": mix}


def _spread(case, most, at_least=1):
    """Lengths of the case's sequences: the first as long as can be, the others from a fifth of it up."""
    r = random.Random(case["mix"])
    return [most if i == 0 else max(at_least, r.randint(min(most, max(at_least, most // 5)), most))
            for i in range(case["seqs"])]


def _lens(case):
    """(new tokens, tokens cached before) of every sequence of an append."""
    new = [1] * case["seqs"] if case["new"] == 1 else _spread(case, case["new"])
    r = random.Random(case["mix"] + 1)
    return new, [r.randint(0, case["ctx"]) for _ in new]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _cu(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return _ints(at)


def _cache(case, g, lens):
    """A paged cache that holds `lens` tokens, its pages in random order: codes
    of normal values with a few channels that stand out, as keys have them."""
    ps, hkv, d, nsb = case["ps"], case["hkv"], case["d"], case["ps"] // case["sb"]
    most = max(1, -(-max(lens) // ps))
    need = [-(-n // ps) for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)
    cu = torch.tensor([sum(need[:i]) for i in range(len(need))], device=DEV)
    col = torch.arange(most, device=DEV)
    table = torch.where(col < torch.tensor(need, device=DEV)[:, None], order[(cu[:, None] + col).clamp(max=pages - 1)], 0)
    k = torch.randn((pages, hkv, ps, d), device=DEV, generator=g).mul_(28.0)
    k[..., torch.randperm(d, device=DEV, generator=g)[:3]] += 80.0
    k = k.round_().clamp_(-127, 127).to(torch.int8)
    v = torch.randn((pages, hkv, ps, d), device=DEV, generator=g).mul_(36.0).round_().clamp_(-127, 127).to(torch.int8)
    ks = torch.rand((pages, hkv, nsb), device=DEV, generator=g) * 0.03 + 0.02
    vs = torch.rand((pages, hkv, nsb), device=DEV, generator=g) * 0.03 + 0.02
    return (k, v, ks, vs), table.contiguous()


def _table64(n_pos, rot, theta, factor, low, high, orig, mag):
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    f = theta ** (-2.0 * i / rot)
    if high > 0:
        turns = orig * f / (2.0 * torch.pi)
        keep = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        f = (1.0 - keep) * f / factor + keep * f
    else:
        f = f / factor
    a = torch.arange(n_pos, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.stack((torch.cos(a) * mag, torch.sin(a) * mag), dim=-1)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, state = case["op"], dict(case)
    if op == "table":
        # where in the context the program's table begins is the only input that is data
        state["first"] = random.Random(seed).randrange(1, 4096)
        return state
    dt = TYPES[case.get("dt", "bf16")]
    if op == "prompt":
        lens = _spread(case, case["len"])
        t, hq, hkv, d = sum(lens), case["hq"], case["hkv"], case["d"]
        # q, k and v as they lie in the output of one QKV projection
        qkv = torch.randn((t, hq + 2 * hkv, d), device=DEV, generator=g)
        qkv[:, hq:hq + hkv, torch.randperm(d, device=DEV, generator=g)[:2]] *= 3.0
        qkv = qkv.to(dt)
        state.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], cu=_cu(lens), longest=max(lens))
        return state
    if op == "append":
        new, ctx = _lens(case)
        t, hq, hkv, d, sb = sum(new), case["hq"], case["hkv"], case["d"], case["sb"]
        state["cache"], state["pages"] = _cache(case, g, [a + b for a, b in zip(new, ctx)])
        qkv = torch.randn((t, hq + 2 * hkv, d), device=DEV, generator=g)
        qkv[:, hq:hq + hkv, torch.randperm(d, device=DEV, generator=g)[:2]] *= 6.0
        qkv = qkv.to(dt)
        first = [c // sb * sb for c in ctx]
        state.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], cu=_cu(new), ctx=_ints(ctx),
                     table=_table64(max(a + b for a, b in zip(new, ctx)), case["rot"], 1e4, 1.0, 0.0, 0.0, 0, 1.0).float(),
                     first=_ints(first), cu_read=_cu([a + b - f for a, b, f in zip(new, ctx, first)]),
                     n_read=sum(a + b - f for a, b, f in zip(new, ctx, first)))
        return state
    lens = _spread(case, case["ctx"])
    state["cache"], state["pages"] = _cache(case, g, lens)
    if op == "read":
        state.update(first=_ints([0] * len(lens)), cu_read=_cu(lens), n_read=sum(lens))
        return state
    state.update(q=torch.randn((case["seqs"], case["q_len"], case["hq"], case["d"]), device=DEV, generator=g).to(dt),
                 lens=_ints(lens))
    return state


# ---------------------------------------------------------------- plain forms
def _rotate(x, c, s, rot, pairs):
    """x [T, H, D] in fp32, its first `rot` channels turned by c, s [T, rot / 2]."""
    c, s = c[:, None, :], s[:, None, :]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    y, z = a * c - b * s, b * c + a * s
    turned = torch.stack((y, z), dim=-1).flatten(-2) if pairs else torch.cat((y, z), dim=-1)
    return torch.cat((turned, x[..., rot:]), dim=-1)


def _quantize(x, codes, scales, sid, slot, page, start_page, start_slot, old, sb):
    """x [T, H, D] fp32 into its blocks of `sb` tokens; `old` [B]: tokens that
    the first touched block of a sequence held already, in the block that
    begins at (start_page, start_slot)."""
    pages, h, ps, d = codes.shape
    nsb = ps // sb
    top = torch.full((), 127.0, device=x.device)
    flat = scales.permute(0, 2, 1).reshape(pages * nsb, h)
    start = start_page * nsb + start_slot // sb
    new = torch.full_like(flat, -1.0).index_reduce_(0, sid, x.abs().amax(-1), "amax")
    before = torch.where(old[:, None] > 0, flat[start], 0.0)
    held = torch.where(new >= 0, new / top, flat)
    held[start] = torch.maximum(held[start], before)
    # tokens that were there before, on the block's new scale
    span = torch.arange(sb, device=x.device)
    was = codes[start_page[:, None], :, start_slot[:, None] + span].float()
    now = held[start][:, None, :, None]
    again = torch.where(now > 0, was * before[:, None, :, None] / now, 0.0).round().clamp(-127, 127)
    again = torch.where((span < old[:, None])[:, :, None, None], again, was)
    codes[start_page[:, None], :, start_slot[:, None] + span] = again.to(torch.int8)
    s = held[sid][:, :, None]
    codes[page, :, slot] = torch.where(s > 0, x / s, 0.0).round().clamp(-127, 127).to(torch.int8)
    scales.copy_(held.view(pages, nsb, h).permute(0, 2, 1))


def _values(codes, scales, pages, first, cu, n, dt):
    """The cached tokens first[b] .. of every sequence, packed by cu."""
    ps, sb = codes.shape[2], codes.shape[2] // scales.shape[2]
    t = torch.arange(n, device=codes.device)
    b = torch.searchsorted(cu[1:], t, right=True)
    pos = first[b] + t - cu[b]
    page, slot = pages[b, pos // ps].long(), (pos % ps).long()
    return (codes[page, :, slot].float() * scales[page, :, slot // sb][:, :, None]).to(dt)


def _softmax_v(score, seen, v):
    """Masked softmax of score over its last axis, times v; rows that see nothing give zero."""
    score = torch.where(seen, score, -torch.inf)
    m = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(m == -torch.inf, 0.0, m))
    s = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(s > 0, s, 1.0)


def _plain(st):
    op = st["op"]
    if op == "table":
        t = _table64(st["first"] + st["n_pos"], st["rot"], st["theta"], st["factor"], st["low"], st["high"], st["orig"], st["mag"])
        return t[st["first"]:].float()
    if op == "append":
        (k, v, ks, vs), q = st["cache"], st["q"]
        ps, sb, cu, ctx, dt = st["ps"], st["sb"], st["cu"], st["ctx"], q.dtype
        t = torch.arange(q.shape[0], device=q.device)
        b = torch.searchsorted(cu[1:], t, right=True)
        pos = (ctx[b] + t - cu[b]).long()
        page, slot = st["pages"][b, pos // ps].long(), pos % ps
        cs = st["table"][pos]
        turned = [_rotate(x.float(), cs[..., 0], cs[..., 1], st["rot"], st["pairs"]) for x in (q, st["k"])]
        begin = (ctx // sb * sb).long()
        start_page = st["pages"].gather(1, (begin // ps)[:, None])[:, 0].long()
        sid = page * (ps // sb) + slot // sb
        _quantize(turned[1], k, ks, sid, slot, page, start_page, begin % ps, ctx % sb, sb)
        _quantize(st["v"].float(), v, vs, sid, slot, page, start_page, begin % ps, ctx % sb, sb)
        at = (st["pages"], st["first"], st["cu_read"], st["n_read"], torch.bfloat16)
        return {"q": turned[0].to(dt), "k": turned[1].to(dt), "k_held": _values(k, ks, *at), "v_held": _values(v, vs, *at),
                "k_scale": ks, "v_scale": vs}
    if op == "read":
        k, v, ks, vs = st["cache"]
        at = (st["pages"], st["first"], st["cu_read"], st["n_read"], TYPES[st["dt"]])
        return _values(k, ks, *at), _values(v, vs, *at)
    if op == "attend":
        (k, v, ks, vs), q = st["cache"], st["q"]
        (n, l, hq, d), hkv = q.shape, st["hkv"]
        # [pages, heads, tokens, d] -> [sequences, heads, tokens, d] in fp32
        k, v = [(c[st["pages"]].float() * s[st["pages"]].repeat_interleave(st["sb"], dim=-1)[..., None])
                .transpose(1, 2).flatten(2, 3) for c, s in ((k, ks), (v, vs))]
        q = q.float().view(n, l, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, -1, d)
        score = torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5
        i = torch.arange(l, device=q.device).repeat_interleave(hq // hkv)
        seen = torch.arange(k.shape[2], device=q.device) <= (st["lens"][:, None] - l + i)[:, None, :, None]
        out = _softmax_v(score, seen, v)
        return out.view(n, hkv, l, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(n, l, hq, d).to(st["q"].dtype)
    q, k, v, cu, m = st["q"], st["k"], st["v"], st["cu"], st["longest"]
    (t, hq, d), hkv = q.shape, st["hkv"]
    lens = cu[1:] - cu[:-1]
    col = torch.arange(m, device=q.device)
    at = (cu[:-1, None] + col).clamp(max=t - 1)
    pad = [x[at].float().transpose(1, 2) for x in (q, k, v)]  # [sequences, heads, longest, d]
    g = pad[0].reshape(len(lens), hkv, hq // hkv * m, d)
    score = torch.matmul(g, pad[1].transpose(-1, -2)).mul_(d ** -0.5)
    row = col.repeat(hq // hkv)[:, None]
    seen = col < lens[:, None, None, None]
    if st["causal"]:
        seen = seen & (col <= row)
    out = _softmax_v(score, seen, pad[2]).view(len(lens), hq, m, d).transpose(1, 2)
    tok = torch.arange(t, device=q.device)
    b = torch.searchsorted(cu[1:], tok, right=True)
    return out[b, tok - cu[b]].to(q.dtype)


# ---------------------------------------------------------------- the library's calls
def _own(st):
    from w8a8_post_quantization_calibrate_b200 import sq
    op = st["op"]
    if op == "table":
        return sq.sq_rope_table(st["n_pos"], st["rot"], st["theta"], first_pos=st["first"], factor=st["factor"],
                                low_turns=st["low"], high_turns=st["high"], original_len=st["orig"], magnitude=st["mag"])
    if op == "prompt":
        return sq.sq_prompt_attention(st["q"], st["k"], st["v"], st["cu"], causal=st["causal"])
    cache = sq.KvCache(*st["cache"])
    if op == "append":
        q, k = sq.sq_rope_kv_append(st["q"], st["k"], st["v"], cache, st["pages"], st["ctx"], st["cu"], table=st["table"],
                                    interleaved=st["pairs"], want_k=True)
        k_held, v_held = sq.sq_kv_read(cache, st["pages"], st["first"], st["cu_read"], st["n_read"])
        return {"q": q, "k": k, "k_held": k_held, "v_held": v_held, "k_scale": cache.k_scale, "v_scale": cache.v_scale}
    if op == "read":
        return sq.sq_kv_read(cache, st["pages"], st["first"], st["cu_read"], st["n_read"], dtype=TYPES[st["dt"]])
    return sq.sq_kv_attention(st["q"], cache, st["pages"], st["lens"])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op = case["op"]
    if op == "table":
        n = case["n_pos"] * case["rot"]
        return {"bytes": 4 * n, "flops": 4 * n}
    hq, hkv, d = case.get("hq", 0), case["hkv"], case["d"]
    if op == "prompt":
        lens = _spread(case, case["len"])
        seen = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens)
        return {"bytes": 2 * sum(lens) * (2 * hq + 2 * hkv) * d, "flops": 4 * d * hq * seen}
    size, nsb = (4 if case["dt"] == "f32" else 2), case["ps"] // case["sb"]
    if op == "append":
        new, ctx = _lens(case)
        t = sum(new)
        blocks = sum((c + n - 1) // case["sb"] - c // case["sb"] + 1 for n, c in zip(new, ctx))
        held = sum(n + c - c // case["sb"] * case["sb"] for n, c in zip(new, ctx))
        table = max(a + b for a, b in zip(new, ctx)) * case["rot"] * 4
        return {"bytes": t * d * (size * (2 * hq + 3 * hkv) + 2 * hkv) + min(table, t * case["rot"] * 4) + 8 * blocks * hkv
                + held * hkv * d * 2 * (1 + 2), "flops": 6 * t * d * (hq + 2 * hkv)}
    lens = _spread(case, case["ctx"])
    scales = sum(-(-n // case["sb"]) for n in lens) * hkv * 8
    held = 2 * sum(lens) * hkv * d
    if op == "read":
        return {"bytes": held * (1 + size) + scales, "flops": held}
    l = case["q_len"]
    return {"bytes": held + scales + 2 * size * case["seqs"] * l * hq * d,
            "flops": sum(4 * d * hq * max(0, n - l + 1 + i) for n in lens for i in range(l))}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "table":
        i = torch.arange(case["rot"] // 2, device=DEV, dtype=f64)
        f = torch.exp(torch.log(torch.tensor(case["theta"], dtype=f64, device=DEV)) * (-2 * i / case["rot"]))
        slow = f / case["factor"]
        if case["high"] > 0:
            wave = 2 * torch.pi / f
            blend = (case["orig"] / wave - case["low"]) / (case["high"] - case["low"])
            mixed = slow + (f - slow) * blend
            slow = torch.where(wave < case["orig"] / case["high"], f, torch.where(wave > case["orig"] / case["low"], slow, mixed))
        p = torch.arange(st["first"], st["first"] + case["n_pos"], device=DEV, dtype=f64)
        z = torch.polar(torch.full((), case["mag"], dtype=f64, device=DEV), torch.outer(p, slow))
        return torch.view_as_real(z)
    if op == "prompt":
        at, out = st["cu"].tolist(), torch.zeros(st["q"].shape, dtype=f64, device=DEV)
        for a, b in zip(at, at[1:]):
            for h in range(case["hq"]):
                kh = h // (case["hq"] // case["hkv"])
                w = st["q"][a:b, h].double() @ st["k"][a:b, kh].double().T / case["d"] ** 0.5
                if case["causal"]:
                    w.masked_fill_(torch.ones_like(w, dtype=torch.bool).triu_(1), float("-inf"))
                w = torch.exp(w - w.amax(1, keepdim=True))
                out[a:b, h] = (w / w.sum(1, keepdim=True)) @ st["v"][a:b, kh].double()
        return out
    k, v, ks, vs = st["cache"]
    pages, ps, sb = st["pages"].tolist(), case["ps"], case["sb"]

    def held(codes, scales, b, lo, hi):
        """Tokens lo..hi of sequence b, [tokens, heads, d]."""
        own_pages = pages[b][lo // ps:-(-hi // ps)]
        x = codes[own_pages].double() * scales[own_pages].double().repeat_interleave(sb, dim=2)[..., None]
        return x.transpose(1, 2).flatten(0, 1)[lo % ps:lo % ps + hi - lo]

    if op == "read":
        both = []
        for codes, scales in ((k, ks), (v, vs)):
            both.append(torch.cat([held(codes, scales, b, 0, n) for b, n in enumerate(_spread(case, case["ctx"]))]))
        return both
    if op == "attend":
        out = torch.zeros(st["q"].shape, dtype=f64, device=DEV)
        g = case["hq"] // case["hkv"]
        for b, n in enumerate(st["lens"].tolist()):
            kb, vb = held(k, ks, b, 0, n), held(v, vs, b, 0, n)
            for i in range(case["q_len"]):
                m = n - case["q_len"] + 1 + i
                if m <= 0:
                    continue
                q = st["q"][b, i].double().view(case["hkv"], g, -1)
                w = torch.einsum("hgd,thd->hgt", q, kb[:m]) / case["d"] ** 0.5
                w = torch.exp(w - w.amax(-1, keepdim=True))
                out[b, i] = torch.einsum("hgt,thd->hgd", w / w.sum(-1, keepdim=True), vb[:m]).flatten(0, 1)
        return out
    at, ctx = st["cu"].tolist(), st["ctx"].tolist()
    rot, d = case["rot"], case["d"]
    out = {"q": torch.zeros(st["q"].shape, dtype=f64, device=DEV), "k": torch.zeros(st["k"].shape, dtype=f64, device=DEV),
           "k_held": [], "v_held": [], "k_scale": ks.double(), "v_scale": vs.double()}
    lo = torch.arange(rot // 2, device=DEV)
    ia, ib = (2 * lo, 2 * lo + 1) if case["pairs"] else (lo, lo + rot // 2)
    for b, c in enumerate(ctx):
        rows = slice(at[b], at[b + 1])
        n = at[b + 1] - at[b]
        z = torch.view_as_complex(st["table"][c:c + n].double())[:, None]
        for name in ("q", "k"):
            x = st[name][rows].double()
            y = torch.complex(x[..., ia], x[..., ib]) * z
            x[..., ia], x[..., ib] = y.real, y.imag
            out[name][rows] = x
        first = c // sb * sb
        for name, codes, scales, x in (("k", k, ks, out["k"][rows]), ("v", v, vs, st["v"][rows].double())):
            got, end = [], c + n
            for s in range(first, end, sb):
                p, blk = pages[b][s // ps], s % ps // sb
                a, e = max(s, c), min(s + sb, end)
                fresh = x[a - c:e - c]
                before = scales[p, :, blk].double() if a > s else torch.zeros(case["hkv"], dtype=f64, device=DEV)
                now = torch.maximum(before, fresh.abs().amax((0, 2)) / 127)
                held_codes = codes[p, :, s % ps:s % ps + a - s].double().transpose(0, 1)
                parts = torch.cat((held_codes * before[:, None], fresh))
                step = now[:, None]
                got.append(torch.round(torch.where(step > 0, parts / step, 0.0)).clamp(-127, 127) * step)
                out[name + "_scale"][p, :, blk] = now
            out[name + "_held"].append(torch.cat(got))
    out["k_held"], out["v_held"] = torch.cat(out["k_held"]), torch.cat(out["v_held"])
    return out
