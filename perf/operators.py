"""The grouped-query, rotary operators over the paged cache, as a set of measured cases.

Three operators of one attention layer: rope_and_cache (rotate q and k by the
token's position and append k, v to the paged cache), decode_grouped (one new
token per sequence over its paged history) and prefill_grouped (many tokens per
sequence).  K/V heads are shared by groups of query heads; the attention's
scores may be capped by a tanh, get a bias by distance, and be limited to a
window and a prefix.

own = False runs the plain form of each operator in elementary torch
operations, fp32 throughout and rounded once; own = True calls the library.
"""
import math

import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
GOLD = 0.6180339887498949


def _spread(n, lo, hi):
    """n lengths in [lo, hi], evenly spread and unordered, from the case alone."""
    return [lo + int((hi - lo + 1) * ((0.5 + i * GOLD) % 1.0)) for i in range(n)]


def listed():
    return [
        # one running sequence's new token: the launch latency counts
        dict(name="rope_step_one", op="rope", tokens=1, seqs=1, q_heads=32, kv_heads=8, head_dim=128, rotary=128,
             block=16, dtype="fp16", interleaved=False, packed=True, far=32768, skip=0),
        # one step of a continuously batched server: a token of each of 256 sequences
        dict(name="rope_step_batch", op="rope", tokens=256, seqs=256, q_heads=32, kv_heads=8, head_dim=128, rotary=128,
             block=16, dtype="bf16", interleaved=False, packed=True, far=32768, skip=0),
        # ragged prompts of a small model that rotates half of each head; some rows are padding
        dict(name="rope_prompts_odd", op="rope", tokens=1009, seqs=5, q_heads=12, kv_heads=4, head_dim=64, rotary=32,
             block=32, dtype="bf16", interleaved=True, packed=False, far=4096, skip=7),
        # a batch of long prompts
        dict(name="rope_prompt_long", op="rope", tokens=16384, seqs=2, q_heads=32, kv_heads=8, head_dim=128, rotary=128,
             block=16, dtype="bf16", interleaved=False, packed=True, far=32768, skip=0),
        # one user, a short chat
        dict(name="decode_one", op="decode", seqs=1, ctx_min=1000, ctx_max=1000, q_heads=32, kv_heads=8, head_dim=128,
             block=16, dtype="fp16", cap=0.0, alibi=False, window=0, prefix=0),
        # the decode batch of a server, contexts of 256 to 2048 tokens
        dict(name="decode_batch", op="decode", seqs=64, ctx_min=256, ctx_max=2048, q_heads=32, kv_heads=8, head_dim=128,
             block=16, dtype="bf16", cap=0.0, alibi=False, window=0, prefix=0),
        # a sliding-window layer with capped scores and wide heads; the first tokens stay visible
        dict(name="decode_window_cap", op="decode", seqs=96, ctx_min=700, ctx_max=8191, q_heads=16, kv_heads=8,
             head_dim=256, block=16, dtype="bf16", cap=50.0, alibi=False, window=1024, prefix=4),
        # four long documents, a bias by distance, eight query heads to each K/V head
        dict(name="decode_long_alibi", op="decode", seqs=4, ctx_min=20001, ctx_max=32768, q_heads=64, kv_heads=8,
             head_dim=128, block=16, dtype="fp16", cap=0.0, alibi=True, window=0, prefix=0),
        # a few drafted tokens of three sequences, checked at once
        dict(name="prefill_few", op="prefill", seqs=3, ctx_min=301, ctx_max=640, new_min=1, new_max=17, q_heads=8,
             kv_heads=2, head_dim=128, block=16, dtype="fp16", cap=0.0, alibi=False, window=0, prefix=0),
        # whole prompts of ordinary length, packed
        dict(name="prefill_prompts", op="prefill", seqs=16, ctx_min=333, ctx_max=1024, new_min=0, new_max=0, q_heads=32,
             kv_heads=8, head_dim=128, block=16, dtype="bf16", cap=0.0, alibi=False, window=0, prefix=0),
        # prompts with a part that all tokens see, a bias by distance, three query heads to each K/V head
        dict(name="prefill_prefix_alibi", op="prefill", seqs=5, ctx_min=517, ctx_max=2500, new_min=0, new_max=0,
             q_heads=12, kv_heads=4, head_dim=64, block=32, dtype="fp16", cap=0.0, alibi=True, window=0, prefix=300),
        # one long prompt with capped scores
        dict(name="prefill_long_cap", op="prefill", seqs=1, ctx_min=8192, ctx_max=8192, new_min=0, new_max=0, q_heads=32,
             kv_heads=4, head_dim=128, block=16, dtype="bf16", cap=30.0, alibi=False, window=0, prefix=0),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope", "decode", "prefill"])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    while kv * group > 64:
        group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    c = dict(op=op, q_heads=kv * group, kv_heads=kv, block=rng.choice([8, 16, 32]), dtype=rng.choice(["fp16", "bf16"]))
    if op == "rope":
        c["head_dim"] = rng.choice([64, 128, 256])
        row = (c["q_heads"] + 2 * kv) * c["head_dim"]
        most = min(32768, 16384 * 48 * 128 // row)
        c["tokens"] = _log_uniform(rng, 1, most)
        c["seqs"] = c["tokens"] if rng.random() < 0.4 else _log_uniform(rng, 1, min(c["tokens"], 40))
        c["rotary"] = c["head_dim"] if rng.random() < 0.6 else 16 * rng.randint(1, c["head_dim"] // 16)
        c["interleaved"] = rng.random() < 0.4
        c["packed"] = rng.random() < 0.7
        c["far"] = rng.choice([4096, 32768, 131072])
        c["skip"] = rng.choice([0, 0, 5, 9])
        c["far"] = max(c["far"], 32768) if c["tokens"] > 4096 else c["far"]
        return c
    c["cap"] = rng.choice([0.0, 0.0, 20.0, 50.0])
    c["alibi"] = rng.random() < 0.3
    c["window"] = rng.choice([0, 0, 0, 1, 100, 1024, 4096])
    c["prefix"] = rng.choice([0, 0, 0, 3, 500])
    if op == "decode":
        c["head_dim"] = rng.choice([64, 128, 256])
        token = kv * c["head_dim"] * 4
        most = (4 * 24000 * 8 * 128 * 4) // token  # visible or not: the history is in the pool
        c["seqs"] = _log_uniform(rng, 1, 512)
        c["ctx_max"] = _log_uniform(rng, 1, max(1, min(40000, most // c["seqs"])))
        c["ctx_min"] = rng.randint(max(1, c["ctx_max"] // 3), c["ctx_max"])
        return c
    c["head_dim"] = rng.choice([64, 128])
    pairs = 32 * 8192 * 8192 // 4
    c["seqs"] = _log_uniform(rng, 1, 24)
    c["ctx_max"] = _log_uniform(rng, 1, max(1, min(8192, int(math.sqrt(pairs / (c["seqs"] * c["q_heads"]))))))
    c["ctx_min"] = rng.randint(max(1, c["ctx_max"] // 3), c["ctx_max"])
    whole = rng.random() < 0.5
    c["new_max"] = 0 if whole else _log_uniform(rng, 1, c["ctx_min"])
    c["new_min"] = 0 if whole else rng.randint(1, c["new_max"])
    return c


# ------------------------------------------------------------------ sizes

def _lens(case):
    return _spread(case["seqs"], case["ctx_min"], case["ctx_max"])


def _new(case):
    """Query tokens of each sequence: the whole prompt, or its last few."""
    ctx = _lens(case)
    if case["new_max"] == 0:
        return ctx
    return [min(c, n) for c, n in zip(ctx, _spread(case["seqs"], case["new_min"], case["new_max"]))]


def _visible(p, ctx, window, prefix):
    """Keys that the query at position p sees."""
    lo = max(0, p - window + 1) if window else 0
    pre = min(prefix, ctx)
    return (p + 1 - lo) + max(0, min(pre, lo)) + max(0, pre - (p + 1))


def _rope_lens(case):
    """Tokens of each sequence in a rope case."""
    T, n = case["tokens"], case["seqs"]
    w = _spread(n, 100, 300)
    total = sum(w)
    got = [max(1, T * x // total) for x in w]
    i = 0
    while sum(got) != T:
        step = 1 if sum(got) < T else -1
        if got[i % n] + step >= 1:
            got[i % n] += step
        i += 1
    return got


def work(case):
    D, Hq, Hk = case["head_dim"], case["q_heads"], case["kv_heads"]
    if case["op"] == "rope":
        T = case["tokens"]
        kept = T - (T // case["skip"] if case["skip"] else 0)
        return {"bytes": T * 2 * Hq * D * 2 + kept * 4 * Hk * D * 2 + T * (case["rotary"] * 4 + 8),
                "flops": 3 * (T * Hq + kept * Hk) * case["rotary"]}
    ctx = _lens(case)
    W, pre = case["window"], case["prefix"]
    if case["op"] == "decode":
        seen = [_visible(c - 1, c, W, pre) for c in ctx]
        return {"bytes": sum(seen) * Hk * D * 4 + case["seqs"] * (Hq * D * 4 + 4) + sum(4 * -(-v // case["block"]) for v in seen),
                "flops": 4 * D * Hq * sum(seen)}
    new = _new(case)
    pairs = sum(_visible(p, c, W, pre) for c, n in zip(ctx, new) for p in range(c - n, c))
    keys = sum(min(c, (n + W - 1 + pre) if W else c) for c, n in zip(ctx, new))
    return {"bytes": sum(new) * Hq * D * 4 + keys * Hk * D * 4 + sum(4 * -(-c // case["block"]) for c in ctx),
            "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------ inputs

def _pool(case, ctx, gen, dev):
    """A shuffled block pool that holds the sequences: caches, block tables, lengths."""
    B, Hk, D, dt = case["block"], case["kv_heads"], case["head_dim"], _DT[case["dtype"]]
    need = [-(-c // B) for c in ctx]
    N = sum(need) + max(2, sum(need) // 10)
    kc = torch.empty(N, Hk, B, D, dtype=dt, device=dev).normal_(generator=gen)
    vc = torch.empty(N, Hk, B, D, dtype=dt, device=dev).normal_(generator=gen)
    order = torch.randperm(N, generator=gen, device=dev)[:sum(need)].to(torch.int32).cpu()
    tables = torch.full((len(ctx), max(need)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = order[at:at + n]
        at += n
    return kc, vc, tables.to(dev), torch.tensor(ctx, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    D, Hq, Hk, B, dt = case["head_dim"], case["q_heads"], case["kv_heads"], case["block"], _DT[case["dtype"]]
    if case["op"] == "rope":
        T, n, r = case["tokens"], case["seqs"], case["rotary"]
        lens = _rope_lens(case)
        near = torch.randint(0, case["far"] - max(lens) + 1, (n,), generator=gen, device=dev).cpu().tolist()
        pos = torch.cat([torch.arange(a, a + m, dtype=torch.int32) for a, m in zip(near, lens)]).to(dev)
        # each sequence's new tokens lie in blocks of its own, from an offset inside the first
        first = [a % B for a in near]
        need = [-(-(f + m) // B) for f, m in zip(first, lens)]
        N = sum(-(-(B - 1 + m) // B) for m in lens) + 2  # whatever the offsets are
        order = torch.randperm(N, generator=gen, device=dev)[:sum(need)].cpu()
        slots, at = [], 0
        for f, m, k in zip(first, lens, need):
            t = torch.arange(f, f + m)
            slots.append(order[at:at + k][t // B] * B + t % B)
            at += k
        slots = torch.cat(slots).to(torch.int32)
        if case["skip"]:
            slots[case["skip"] - 1::case["skip"]] = -1
        if case["packed"]:  # one projection's output, q | k | v in each row
            qkv = torch.empty(T, Hq + 2 * Hk, D, dtype=dt, device=dev).normal_(generator=gen)
            q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        else:
            q, k, v = (torch.empty(T, h, D, dtype=dt, device=dev).normal_(generator=gen) for h in (Hq, Hk, Hk))
        ang = torch.arange(case["far"], dtype=torch.float64, device=dev)[:, None] \
            * 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device=dev) / r)
        table = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        kc = torch.zeros(N, Hk, B, D, dtype=dt, device=dev)
        return dict(op="rope", q=q, k=k, v=v, k_cache=kc, v_cache=torch.zeros_like(kc), positions=pos, table=table,
                    slots=slots.to(dev), interleaved=case["interleaved"],
                    q_out=torch.zeros(T, Hq, D, dtype=dt, device=dev))
    ctx = _lens(case)
    kc, vc, tables, lens = _pool(case, ctx, gen, dev)
    st = dict(op=case["op"], k_cache=kc, v_cache=vc, tables=tables, lens=lens, scale=D ** -0.5, cap=case["cap"],
              window=case["window"],
              prefix=torch.full((len(ctx),), case["prefix"], dtype=torch.int32, device=dev) if case["prefix"] else None,
              slopes=(2.0 ** (-8.0 * torch.arange(1, Hq + 1, dtype=torch.float32, device=dev) / Hq)) if case["alibi"] else None)
    new = [1] * len(ctx) if case["op"] == "decode" else _new(case)
    st["q"] = torch.empty(sum(new), Hq, D, dtype=dt, device=dev).normal_(generator=gen)
    if case["cap"]:
        st["q"] *= 3.0  # scores that reach the cap's bend
    st["out"] = torch.zeros_like(st["q"])
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    st["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    st["max_new"] = max(new)
    st["max_ctx"] = max(ctx)
    return st


# ------------------------------------------------------------------ plain forms

def _rotate(x, cos, sin, interleaved):
    """x [T, H, D] fp32; cos, sin [T, r / 2]."""
    h = cos.shape[1]
    c, s = cos[:, None], sin[:, None]
    rot, rest = x[..., :2 * h], x[..., 2 * h:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = rot[..., :h], rot[..., h:]
        rot = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([rot, rest], -1)


def _plain_rope(st):
    h = st["table"].shape[1] // 2
    cs = st["table"][st["positions"].long()]
    cos, sin = cs[:, :h], cs[:, h:]
    st["q_out"].copy_(_rotate(st["q"].float(), cos, sin, st["interleaved"]))
    k = _rotate(st["k"].float(), cos, sin, st["interleaved"]).to(st["k_cache"].dtype)
    B = st["k_cache"].shape[2]
    keep = st["slots"] >= 0
    slot = st["slots"][keep].long()
    st["k_cache"][slot // B, :, slot % B] = k[keep]
    st["v_cache"][slot // B, :, slot % B] = st["v"][keep]
    return [st["q_out"], st["k_cache"], st["v_cache"]]


def _plain_attention(st):
    kc, tables, starts = st["k_cache"], st["tables"], st["starts"].long()
    S, n = tables.shape[0], st["max_new"]
    _, Hk, B, D = kc.shape
    Hq = st["q"].shape[1]
    G = Hq // Hk
    idx = tables.clamp(min=0).long()
    k = kc[idx].transpose(1, 2).reshape(S, Hk, -1, D).float()         # [S, Hk, K, D]
    v = st["v_cache"][idx].transpose(1, 2).reshape(S, Hk, -1, D).float()
    K = k.shape[2]
    count = starts[1:] - starts[:-1]
    i = torch.arange(n, device=kc.device)
    row = (starts[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)     # [S, n]
    q = st["q"][row].float().view(S, n, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hk, G * n, D)
    s = torch.matmul(q, k.transpose(2, 3)).mul_(st["scale"]).view(S, Hk, G, n, K)
    if st["cap"]:
        s.div_(st["cap"]).tanh_().mul_(st["cap"])
    lens = st["lens"].long()
    pos = (lens - count)[:, None] + i                                  # [S, n]
    j = torch.arange(K, device=kc.device)
    ahead = j - pos[..., None]                                         # [S, n, K]
    if st["slopes"] is not None:
        s.sub_(st["slopes"].view(1, Hk, G, 1, 1) * ahead.abs().float()[:, None, None])
    seen = ahead <= 0
    if st["window"]:
        seen &= ahead > -st["window"]
    if st["prefix"] is not None:
        seen |= j < st["prefix"][:, None, None]
    seen &= j < lens[:, None, None]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-3e38)
    s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(S, Hk, G * n, K), v).view(S, Hk, G, n, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.permute(0, 3, 1, 2, 4).reshape(S, n, Hq, D)
    st["out"].copy_(o[i < count[:, None]])
    return st["out"]


def run(st):
    if not own:
        return _plain_rope(st) if st["op"] == "rope" else _plain_attention(st)
    import paged_kv_cache_269_gb300 as pa
    if st["op"] == "rope":
        pa.rope_and_cache(st["q_out"], st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["positions"],
                          st["table"], st["slots"], interleaved=st["interleaved"])
        return [st["q_out"], st["k_cache"], st["v_cache"]]
    if st["op"] == "decode":
        return pa.decode_grouped(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["scale"],
                                 softcap=st["cap"], alibi_slopes=st["slopes"], window=st["window"],
                                 prefix_lens=st["prefix"])
    return pa.prefill_grouped(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], st["starts"],
                              st["scale"], max_query_len=st["max_new"], softcap=st["cap"], alibi_slopes=st["slopes"],
                              window=st["window"], prefix_lens=st["prefix"])


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "rope":
        T, r = case["tokens"], case["rotary"]
        # the operator's input is the fp32 table: its rows, widened
        rows = st["table"].to(f64).index_select(0, st["positions"].long())
        turn = torch.complex(rows[:, :r // 2], rows[:, r // 2:])[:, None, :]

        def turned(x):
            x = x.to(f64)
            part = x[..., :r]
            pairs = part.unflatten(-1, (r // 2, 2)) if case["interleaved"] else part.unflatten(-1, (2, r // 2)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            z = z.reshape(part.shape) if case["interleaved"] else z.transpose(-1, -2).reshape(part.shape)
            return torch.cat([z, x[..., r:]], dim=-1)

        B = case["block"]
        out = []
        for cache, x in ((st["k_cache"], turned(st["k"])), (st["v_cache"], st["v"].to(f64))):
            flat = cache.to(f64).permute(0, 2, 1, 3).reshape(-1, case["kv_heads"], case["head_dim"])
            ok = (st["slots"] >= 0).nonzero().flatten()
            flat.index_copy_(0, st["slots"][ok].long(), x[ok])
            out.append(flat.view(-1, B, case["kv_heads"], case["head_dim"]).permute(0, 2, 1, 3).contiguous())
        return [turned(st["q"]), out[0], out[1]]
    ctx = _lens(case)
    new = [1] * len(ctx) if case["op"] == "decode" else _new(case)
    Hk, B, D = case["kv_heads"], case["block"], case["head_dim"]
    G = case["q_heads"] // Hk
    res = torch.zeros(st["q"].shape, dtype=f64, device=st["q"].device)
    at = 0
    for s, (c, n) in enumerate(zip(ctx, new)):
        blocks = st["tables"][s, :-(-c // B)].long()
        key = torch.arange(c, device=res.device, dtype=f64)
        p = torch.arange(c - n, c, device=res.device, dtype=f64)
        dist = p[:, None] - key
        hidden = dist < 0
        if case["window"]:
            hidden = hidden | (dist >= case["window"])
        if case["prefix"]:
            hidden = hidden & (key >= case["prefix"])
        for h in range(Hk):
            K = st["k_cache"][blocks, h].reshape(-1, D)[:c].to(f64)
            V = st["v_cache"][blocks, h].reshape(-1, D)[:c].to(f64)
            for g in range(G):
                x = st["q"][at:at + n, h * G + g].to(f64) @ K.T * case["head_dim"] ** -0.5
                if case["cap"]:
                    x = case["cap"] * torch.tanh(x / case["cap"])
                if case["alibi"]:
                    x = x - st["slopes"][h * G + g].to(f64) * dist.abs()
                x[hidden] = -math.inf
                res[at:at + n, h * G + g] = torch.softmax(x, dim=-1) @ V
        at += n
    return res
