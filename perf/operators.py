"""The decode-step operators as measured work: block tables and slot maps
(`paged_slots`), attention of one new token per request over the paged K/V
cache (`paged_attention`) and sampling of the next token (`sample_tokens`).

Each case is one call on inputs of a serving step.  `run` computes it either
through the library (`own`) or in plain torch operations; `exact` computes it
again in float64 from the definition.
"""
import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one chat request: latency only
        dict(name="attention_one_request", op="attention", batch=1, hq=32, hkv=8, d=128, block=16, longest=700,
             zeros=0, out="bf16", lse=False, window=0),
        # the decode batch of the paged-cache workload: 32 requests, positions up to 4096, 16-row blocks
        dict(name="attention_decode_batch", op="attention", batch=32, hq=32, hkv=8, d=128, block=16, longest=4096,
             zeros=0, out="bf16", lse=False, window=0),
        # one KV head per query head, codes out for the next E4M3 Linear, two padded rows of a captured batch
        dict(name="attention_mha_codes", op="attention", batch=24, hq=32, hkv=32, d=128, block=32, longest=1500,
             zeros=2, out="e4m3", lse=False, window=0),
        # eight query heads on one wide KV head, a sliding window over long requests
        dict(name="attention_mqa_window", op="attention", batch=48, hq=8, hkv=1, d=256, block=64, longest=9001,
             zeros=0, out="bf16", lse=True, window=4096),
        # two very long documents: few rows, all of the cache's length to split
        dict(name="attention_long", op="attention", batch=2, hq=40, hkv=8, d=128, block=64, longest=131072,
             zeros=0, out="bf16", lse=True, window=0),
        # a full server: the largest case
        dict(name="attention_full_server", op="attention", batch=256, hq=32, hkv=8, d=128, block=16, longest=4096,
             zeros=0, out="bf16", lse=False, window=0),
        # one new token for each of 32 requests
        dict(name="slots_decode", op="slots", batch=32, block=16, longest=4096, prompts=0, longest_prompt=0, ended=0,
             pad=0),
        # decode rows beside prompts that begin, requests that end, rows behind the last token
        dict(name="slots_mixed", op="slots", batch=300, block=16, longest=4096, prompts=24, longest_prompt=4096,
             ended=9, pad=256),
        # one request, nucleus sampling on bf16 logits
        dict(name="sample_one", op="sample", batch=1, vocab=32000, dtype="bf16", kinds="nucleus", logprob=False),
        # a decode batch whose requests ask for different things
        dict(name="sample_mixed", op="sample", batch=32, vocab=151936, dtype="bf16", kinds="mixed", logprob=True),
        # an odd vocabulary: rows that do not begin on a 16-byte boundary, temperature alone
        dict(name="sample_odd_vocab", op="sample", batch=61, vocab=50257, dtype="bf16", kinds="plain", logprob=True),
        # a full server on float32 logits, nucleus
        dict(name="sample_full_server", op="sample", batch=256, vocab=128000, dtype="f32", kinds="nucleus",
             logprob=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["attention", "attention", "slots", "sample", "sample"])
    if op == "attention":
        hkv = rng.choice([1, 2, 4, 8, 8, 16, 32])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 12, 16])
        d = rng.choice([64, 96, 128, 128, 256])
        longest = _log_int(rng, 1, 131072)
        # no more cache, and no more arithmetic, than the largest listed case has
        room = max(1, (256 * 4096 * 8 * 128) // (longest * hkv * d * max(4, group) // 4))
        batch = _log_int(rng, 1, min(room, 256))
        return dict(op=op, batch=batch, hq=hkv * group, hkv=hkv, d=d, block=rng.choice([1, 8, 16, 16, 24, 64, 128]),
                    longest=longest, zeros=rng.choice([0, 0, 1]) if batch > 1 else 0,
                    out=rng.choice(["bf16", "bf16", "e4m3"]), lse=rng.random() < 0.4,
                    window=rng.choice([0, 0, 0, _log_int(rng, 1, 8192)]))
    if op == "slots":
        batch = _log_int(rng, 1, 1024)
        return dict(op=op, batch=batch, block=rng.choice([1, 8, 16, 16, 24, 64, 128]), longest=_log_int(rng, 16, 16384),
                    prompts=rng.randrange(0, min(batch, 32) + 1), longest_prompt=_log_int(rng, 1, 4096),
                    ended=rng.randrange(0, max(1, batch // 8) + 1), pad=rng.choice([0, 0, 1, 77]))
    vocab = _log_int(rng, 1000, 262144)
    batch = _log_int(rng, 1, max(1, min(512, 256 * 128000 // vocab)))
    return dict(op=op, batch=batch, vocab=vocab, dtype=rng.choice(["bf16", "bf16", "f32"]),
                kinds=rng.choice(["nucleus", "mixed", "mixed", "plain"]), logprob=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _lengths(batch, longest, zeros):
    """Lengths of a batch in the order of their size: spread over 1..longest,
    the first `zeros` of them padding rows of length 0.  The seed only
    permutes them, so a case's work does not depend on it."""
    n = batch - zeros
    spread = [0] * zeros + [max(1, round(longest * (i + 1) / n)) for i in range(n)]
    return spread


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _permuted(values, gen):
    v = torch.tensor(values, dtype=torch.int32, device="cuda")
    return v[torch.randperm(len(values), generator=gen, device="cuda")]


def _prepare_attention(c, seed):
    g = _generator(seed)
    b, hq, hkv, d, bs = c["batch"], c["hq"], c["hkv"], c["d"], c["block"]
    lens = _permuted(_lengths(b, c["longest"], c["zeros"]), g)
    width = -(-c["longest"] // bs)
    have = (lens.long() + bs - 1) // bs
    blocks = int(have.sum()) + 3
    # each request's blocks are scattered over the cache
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(b, width, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None, :] < have[:, None]] = order[:int(have.sum())]
    rows = blocks * bs
    # normalised heads: unit variance keys, queries that make a moderately peaked softmax
    q = (torch.randn(b, hq, d, generator=g, device="cuda") * 2.0).bfloat16()
    k = torch.randn(rows, hkv, d, generator=g, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(rows, hkv, d, generator=g, device="cuda", dtype=torch.bfloat16)
    out = torch.empty(b, hq, d, device="cuda", dtype=torch.uint8 if c["out"] == "e4m3" else torch.bfloat16)
    lse = torch.empty(b, hq, device="cuda") if c["lse"] else None
    # the workspace of partial results that a server keeps: enough for any batch
    workspace = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    return dict(q=q, k=k, v=v, table=table, lens=lens, out=out, lse=lse, workspace=workspace, scale=d ** -0.5,
                out_scale=0.01)


def _slots_batch(c):
    """(context length, new tokens) of each request: decode rows, prompts that
    begin (no context yet), ended requests (-1), which give their blocks back."""
    b = c["batch"]
    prompts = min(c["prompts"], b)
    lens, new = _lengths(b, c["longest"], 0), [1] * b
    for i in range(prompts):
        lens[i * b // prompts] = 0
        new[i * b // prompts] = max(1, round(c["longest_prompt"] * (i + 1) / prompts))
    living = [i for i in range(b) if lens[i] > 0]
    for i in range(min(c["ended"], len(living))):
        new[living[i * len(living) // c["ended"]]] = -1
    return lens, new


def _prepare_slots(c, seed):
    g = _generator(seed)
    b, bs = c["batch"], c["block"]
    lens, new = _slots_batch(c)
    perm = torch.randperm(b, generator=g, device="cuda")
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")[perm]
    add = torch.tensor(new, dtype=torch.int32, device="cuda")[perm]
    tokens = sum(n for n in new if n > 0)
    width = -(-max(l + max(n, 0) for l, n in zip(lens, new)) // bs)
    have = (ctx.long() + bs - 1) // bs
    want = (ctx.long() + add.clamp(min=0) + bs - 1) // bs
    held = int(have.sum())
    blocks = held + int((want - have).sum()) + 5
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None, :] < have[:, None]] = order[:held]
    # a ring of block ids that has gone round: the free ones begin somewhere in it
    head = int(torch.randint(0, blocks, (1,), generator=g, device="cuda"))
    free = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    free[(head + torch.arange(blocks - held, device="cuda")) % blocks] = order[held:]
    ring = torch.tensor([head, blocks - held], dtype=torch.int32, device="cuda")
    return dict(ctx=ctx, add=add, table=table, free=free, ring=ring, block=bs,
                seq=torch.zeros(b, dtype=torch.int32, device="cuda"), ring_out=torch.zeros_like(ring),
                slots=torch.full((tokens + c["pad"],), -1, dtype=torch.int32, device="cuda"),
                pos=torch.full((tokens + c["pad"],), -1, dtype=torch.int32, device="cuda"),
                start=torch.zeros(b + 1, dtype=torch.int32, device="cuda"))


def _prepare_sample(c, seed):
    g = _generator(seed)
    b, v = c["batch"], c["vocab"]
    # a broad body with a few strong candidates in each row, as a language model's head gives
    logits = torch.randn(b, v, generator=g, device="cuda") * 2.2
    strong = torch.randint(0, v, (b, 24), generator=g, device="cuda")
    logits.scatter_add_(1, strong, torch.rand(b, 24, generator=g, device="cuda") * 9.0 + 2.0)
    # tokens that a grammar forbids
    forbidden = torch.randint(0, v, (b, max(1, v // 50)), generator=g, device="cuda")
    logits.scatter_(1, forbidden, float("-inf"))
    if c["dtype"] == "bf16":
        logits = logits.bfloat16()
    kind = torch.arange(b, device="cuda")[torch.randperm(b, generator=g, device="cuda")] % 8
    temperature = 0.5 + torch.rand(b, generator=g, device="cuda")
    top_k = top_p = min_p = None
    if c["kinds"] == "plain":
        temperature = torch.where(kind == 1, torch.zeros_like(temperature), temperature)     # greedy requests
    elif c["kinds"] == "nucleus":
        top_p = 0.8 + 0.19 * torch.rand(b, generator=g, device="cuda")
    else:
        temperature = torch.where(kind == 1, torch.zeros_like(temperature), temperature)
        some_k = torch.randint(1, 201, (b,), generator=g, device="cuda", dtype=torch.int32)
        top_k = torch.where((kind == 2) | (kind == 3) | (kind == 4), some_k, torch.zeros_like(some_k))
        some_p = 0.7 + 0.29 * torch.rand(b, generator=g, device="cuda")
        top_p = torch.where((kind == 3) | (kind == 5), some_p, torch.ones_like(some_p))
        some_m = 0.02 + 0.1 * torch.rand(b, generator=g, device="cuda")
        min_p = torch.where((kind == 4) | (kind == 6), some_m, torch.zeros_like(some_m))
    uniform = torch.rand(b, generator=g, device="cuda")
    return dict(logits=logits, uniform=uniform, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p,
                tokens=torch.zeros(b, dtype=torch.int32, device="cuda"),
                logprob=torch.zeros(b, device="cuda") if c["logprob"] else None)


def prepare(case, seed):
    make = {"attention": _prepare_attention, "slots": _prepare_slots, "sample": _prepare_sample}[case["op"]]
    return dict(make(case, seed), case=case)


# -------------------------------------------------------------- plain forms

def _plain_attention(s):
    c = s["case"]
    b, hq, hkv, d, bs = c["batch"], c["hq"], c["hkv"], c["d"], c["block"]
    lens = s["lens"].long()
    at = torch.arange(c["longest"], device="cuda")
    first = (lens - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(lens)
    seen = (at[None, :] < lens[:, None]) & (at[None, :] >= first[:, None])           # [B, L]
    rows = s["table"].long()[:, at // bs] * bs + at % bs
    rows = torch.where(seen, rows, torch.zeros_like(rows))
    q = s["q"].float().view(b, hkv, hq // hkv, d)
    k = s["k"][rows].float().permute(0, 2, 3, 1)                                      # [B, Hkv, D, L]
    score = torch.matmul(q, k) * s["scale"]
    del k
    score = score.masked_fill(~seen[:, None, None, :], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = s["v"][rows].float().permute(0, 2, 1, 3)                                      # [B, Hkv, L, D]
    o = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
    o = o.reshape(b, hq, d)
    if c["out"] == "e4m3":
        o = (o / s["out_scale"]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    else:
        o = o.bfloat16()
    if not c["lse"]:
        return {"out": o}
    return {"out": o, "lse": (torch.log(total) + top).reshape(b, hq)}


def _plain_slots(s):
    bs, b, n = s["block"], s["ctx"].numel(), s["free"].numel()
    ctx, add = s["ctx"].long(), s["add"].long()
    ended, fresh = add < 0, add.clamp(min=0)
    have, want = (ctx + bs - 1) // bs, (ctx + fresh + bs - 1) // bs
    head, count = s["ring"][0].long(), s["ring"][1].long()
    who = torch.arange(b, device="cuda")
    # blocks taken, request by request, from the front of the ring
    need = want - have
    before = torch.cumsum(need, 0) - need
    row = torch.repeat_interleave(who, need)
    i = torch.arange(row.numel(), device="cuda")
    s["table"][row, have[row] + i - before[row]] = s["free"][(head + i) % n]
    # blocks given back, behind its end
    back = torch.where(ended, have, torch.zeros_like(have))
    before = torch.cumsum(back, 0) - back
    row = torch.repeat_interleave(who, back)
    i = torch.arange(row.numel(), device="cuda")
    s["free"][(head + count + i) % n] = s["table"][row, i - before[row]]
    taken, given = need.sum(), back.sum()
    s["ring_out"].copy_(torch.stack([(head + taken) % n, count - taken + given]))
    s["seq"].copy_(torch.where(ended, torch.zeros_like(ctx), ctx + fresh))
    end = torch.cumsum(fresh, 0)
    s["start"][1:] = end
    row = torch.repeat_interleave(who, fresh)
    t = torch.arange(row.numel(), device="cuda")
    p = ctx[row] + t - (end - fresh)[row]
    s["pos"][:row.numel()] = p.int()
    s["slots"][:row.numel()] = (s["table"][row, p // bs].long() * bs + p % bs).int()
    return _slots_out(s)


def _slots_out(s):
    return {k: s[k] for k in ("table", "free", "ring_out", "seq", "slots", "pos", "start")}


def _plain_sample(s):
    x = s["logits"].double()
    b, v = x.shape
    t = s["temperature"].double()
    greedy = t == 0
    top = x.amax(1, keepdim=True)
    w = torch.exp((x - top) / torch.where(greedy, torch.ones_like(t), t)[:, None])
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    sorted_w = w.gather(1, order)
    rank = torch.arange(v, device="cuda")[None, :]
    keep = torch.ones_like(sorted_w, dtype=torch.bool)
    if s["top_k"] is not None:
        k = s["top_k"].long()
        keep &= rank < torch.where(k > 0, k, torch.full_like(k, v))[:, None]
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        mass = torch.where(keep, sorted_w, torch.zeros_like(sorted_w))
        before = torch.cumsum(mass, 1) - mass
        keep &= (before < p * mass.sum(1, keepdim=True)) | (p >= 1)
    if s["min_p"] is not None:
        keep &= sorted_w >= s["min_p"].double()[:, None]
    kept = torch.zeros_like(keep).scatter(1, order, keep)
    w = torch.where(kept, w, torch.zeros_like(w))
    mass = torch.cumsum(w, 1)
    total = mass[:, -1:]
    token = (mass > s["uniform"].double()[:, None] * total).int().argmax(1)
    token = torch.where(greedy, order[:, 0], token)
    out = {"tokens": token.int()}
    if s["logprob"] is not None:
        p = w.gather(1, token[:, None])[:, 0] / total[:, 0]
        out["logprob"] = torch.where(greedy, torch.zeros_like(p), torch.log(p)).float()
    return out


def _own(s):
    import fusion_add_rmsnorm_gb300 as gbf
    c = s["case"]
    if c["op"] == "attention":
        gbf.paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], c["block"], s["out"], s["workspace"],
                            scale=s["scale"], window=c["window"], lse=s["lse"],
                            out_scale=s["out_scale"] if c["out"] == "e4m3" else None)
        out = s["out"].view(torch.float8_e4m3fn) if c["out"] == "e4m3" else s["out"]
        return {"out": out, "lse": s["lse"]} if c["lse"] else {"out": out}
    if c["op"] == "slots":
        gbf.paged_slots(s["ctx"], s["add"], s["table"], s["free"], s["ring"], s["block"], s["seq"], s["ring_out"],
                        s["slots"], s["pos"], s["start"])
        return _slots_out(s)
    gbf.sample_tokens(s["logits"], s["uniform"], s["tokens"], temperature=s["temperature"], top_k=s["top_k"],
                      top_p=s["top_p"], min_p=s["min_p"], logprob=s["logprob"])
    return {"tokens": s["tokens"], "logprob": s["logprob"]} if c["logprob"] else {"tokens": s["tokens"]}


def run(state):
    if own:
        return _own(state)
    plain = {"attention": _plain_attention, "slots": _plain_slots, "sample": _plain_sample}
    return plain[state["case"]["op"]](state)


# ------------------------------------------------------------- what it costs

def work(case):
    c = case
    if c["op"] == "attention":
        lens = _lengths(c["batch"], c["longest"], c["zeros"])
        if c["window"]:
            lens = [min(n, c["window"]) for n in lens]
        tokens, heads = sum(lens), c["batch"] * c["hq"]
        size = tokens * c["hkv"] * c["d"] * 4 + heads * c["d"] * (3 if c["out"] == "e4m3" else 4)
        size += 4 * sum(-(-n // c["block"]) for n in lens) + 4 * c["batch"] + (4 * heads if c["lse"] else 0)
        return {"bytes": size, "flops": 4 * c["hq"] * c["d"] * tokens}
    if c["op"] == "slots":
        b, bs = c["batch"], c["block"]
        tokens = blocks = 0
        for n, more in zip(*_slots_batch(c)):
            tokens += max(more, 0)
            # a table entry is read or written for each block that tokens go to, or that goes back
            blocks += -(-n // bs) if more < 0 else (n + more - 1) // bs - n // bs + 1 if more else 0
        return {"bytes": 12 * b + 16 + 4 * (b + 1) + 8 * tokens + 8 * blocks, "flops": 0}
    size = 2 if c["dtype"] == "bf16" else 4
    n = c["batch"] * c["vocab"]
    return {"bytes": n * size + c["batch"] * 24, "flops": 4 * n}


# ----------------------------------------------------------------- in 64 bits

def _exact_attention(c, s):
    outs, lses = [], []
    group = c["hq"] // c["hkv"]
    lens, q = s["lens"].tolist(), s["q"].double()
    for i, n in enumerate(lens):
        lo = max(0, n - c["window"]) if c["window"] else 0
        if n == 0:
            outs.append(torch.zeros(c["hq"], c["d"], dtype=torch.float64, device="cuda"))
            lses.append(torch.full((c["hq"],), float("-inf"), dtype=torch.float64, device="cuda"))
            continue
        j = torch.arange(lo, n, device="cuda")
        slot = s["table"][i, j // c["block"]].long() * c["block"] + j % c["block"]
        k, v = s["k"][slot].double(), s["v"][slot].double()                     # [n, Hkv, D]
        x = torch.einsum("hgd,nhd->hgn", q[i].view(c["hkv"], group, c["d"]), k) * s["scale"]
        lses.append(torch.logsumexp(x, -1).reshape(-1))
        outs.append(torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), v).reshape(c["hq"], c["d"]))
    out = torch.stack(outs)
    if c["out"] == "e4m3":
        out = (out / s["out_scale"]).clamp(-E4M3_MAX, E4M3_MAX)
    return {"out": out, "lse": torch.stack(lses)} if c["lse"] else {"out": out}


def _exact_slots(c, s):
    ctx, add, table, free = s["ctx"].tolist(), s["add"].tolist(), s["table"].tolist(), s["free"].tolist()
    (head, count), n, bs = s["ring"].tolist(), s["free"].numel(), s["block"]
    slots, pos, start, seq, at = [], [], [0], [], head
    for i, (have, more) in enumerate(zip(ctx, add)):
        for p in range(have, have + max(more, 0)):
            if p % bs == 0:
                table[i][p // bs] = free[at % n]
                at += 1
            slots.append(table[i][p // bs] * bs + p % bs)
            pos.append(p)
        start.append(len(slots))
        seq.append(0 if more < 0 else have + more)
    tail = head + count
    for i, more in enumerate(add):
        for j in range(-(-ctx[i] // bs) if more < 0 else 0):
            free[tail % n] = table[i][j]
            tail += 1
    rest = [-1] * (s["slots"].numel() - len(slots))
    return dict(table=table, free=free, ring_out=[at % n, tail - at], seq=seq, slots=slots + rest, pos=pos + rest,
                start=start)


def _exact_sample(c, s):
    tokens, logs = [], []
    at = lambda name, i, other: other if s[name] is None else s[name][i].item()            # noqa: E731
    for i in range(c["batch"]):
        x = s["logits"][i].double()
        t = s["temperature"][i].item()
        if t == 0:
            tokens.append(int((x == x.max()).nonzero()[0]))
            logs.append(0.0)
            continue
        w = torch.softmax((x - x.max()) / t, 0)
        ids = torch.arange(c["vocab"], device="cuda")[w > 0]
        by_size = torch.argsort(x[ids], descending=True, stable=True)
        ids, k = ids[by_size], at("top_k", i, 0)
        ids = ids[:k] if k > 0 else ids
        p = at("top_p", i, 1.0)
        if p < 1:
            share = w[ids] / w[ids].sum()
            ids = ids[:1 + int((torch.cumsum(share, 0) < p).sum())]
        ids = ids[w[ids] >= at("min_p", i, 0.0) * w.max()]
        ids = torch.sort(ids).values
        share = torch.cumsum(w[ids], 0)
        j = min(int((share <= s["uniform"][i].item() * share[-1]).sum()), len(ids) - 1)
        tokens.append(int(ids[j]))
        logs.append(float(torch.log(w[ids[j]] / share[-1])))
    out = {"tokens": torch.tensor(tokens, dtype=torch.int32)}
    if c["logprob"]:
        out["logprob"] = torch.tensor(logs, dtype=torch.float64)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "slots":
        return {k: torch.tensor(v, dtype=torch.int32) for k, v in _exact_slots(case, s).items()}
    return {"attention": _exact_attention, "sample": _exact_sample}[case["op"]](case, s)
