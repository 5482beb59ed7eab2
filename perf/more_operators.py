"""The 8-bit paged cache as a set of measured cases: its append, its read-back
and the attention over it.

Four operators: norm_rope_and_cache (norm each head of q and k, rotate them by
the token's position, append k and v to a paged cache of 16 or 8 bits),
gather_cache_q8 (read tokens of an 8-bit cache back as 16-bit rows),
decode_grouped_q8 and prefill_grouped_q8 (one new token, or many, per sequence
over an 8-bit paged history).  A value of an 8-bit cache is its e4m3 number
times its head's scale.

own = False runs the plain form of each operator in elementary torch
operations, fp32 throughout and rounded once; own = True calls the library.
"""
import math

import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
GOLD = 0.6180339887498949
EPS = 1e-6


def _spread(n, lo, hi):
    """n lengths in [lo, hi], evenly spread and unordered, from the case alone."""
    return [lo + int((hi - lo + 1) * ((0.5 + i * GOLD) % 1.0)) for i in range(n)]


def listed():
    return [
        # one running sequence's new token: the launch latency counts
        dict(name="append_step_one", op="append", tokens=1, seqs=1, q_heads=32, kv_heads=8, head_dim=128, rotary=128,
             block=16, dtype="bf16", interleaved=False, packed=True, far=32768, skip=0, norm=True, bits=8),
        # one step of a continuously batched server that keeps a 16-bit cache
        dict(name="append_step_batch", op="append", tokens=256, seqs=256, q_heads=32, kv_heads=8, head_dim=128,
             rotary=128, block=16, dtype="bf16", interleaved=False, packed=True, far=32768, skip=0, norm=True, bits=16),
        # ragged prompts of a small model without norms that rotates half of each head; some rows are padding
        dict(name="append_prompts_odd", op="append", tokens=1009, seqs=5, q_heads=12, kv_heads=4, head_dim=64, rotary=32,
             block=32, dtype="fp16", interleaved=True, packed=False, far=4096, skip=7, norm=False, bits=8),
        # a batch of long prompts
        dict(name="append_prompt_long", op="append", tokens=16384, seqs=2, q_heads=32, kv_heads=8, head_dim=128,
             rotary=128, block=16, dtype="bf16", interleaved=False, packed=True, far=32768, skip=0, norm=True, bits=8),
        # one cached prompt read back, to be handed to another program
        dict(name="gather_prompt", op="gather", seqs=1, ctx_min=1000, ctx_max=1000, kv_heads=8, head_dim=128, block=16,
             dtype="fp16", skip=0),
        # a batch's histories read back before its pool is rebuilt; some entries are padding
        dict(name="gather_batch", op="gather", seqs=64, ctx_min=256, ctx_max=2048, kv_heads=8, head_dim=128, block=16,
             dtype="bf16", skip=9),
        # one user, a short chat
        dict(name="decode_one", op="decode", seqs=1, ctx_min=1000, ctx_max=1000, q_heads=32, kv_heads=8, head_dim=128,
             block=16, dtype="fp16", cap=0.0, alibi=False, window=0, prefix=0),
        # the decode batch of a server, twice as many sequences as its memory would hold in 16 bits
        dict(name="decode_batch", op="decode", seqs=128, ctx_min=256, ctx_max=2048, q_heads=32, kv_heads=8, head_dim=128,
             block=16, dtype="bf16", cap=0.0, alibi=False, window=0, prefix=0),
        # long documents on wide heads, capped scores
        dict(name="decode_long_cap", op="decode", seqs=6, ctx_min=20001, ctx_max=32768, q_heads=16, kv_heads=8,
             head_dim=256, block=32, dtype="bf16", cap=50.0, alibi=False, window=0, prefix=0),
        # a few drafted tokens of three sequences, checked at once
        dict(name="prefill_few", op="prefill", seqs=3, ctx_min=301, ctx_max=640, new_min=1, new_max=17, q_heads=8,
             kv_heads=2, head_dim=128, block=16, dtype="fp16", cap=0.0, alibi=False, window=0, prefix=0),
        # the next chunk of four long prompts
        dict(name="prefill_chunks", op="prefill", seqs=4, ctx_min=4097, ctx_max=8192, new_min=512, new_max=512,
             q_heads=32, kv_heads=8, head_dim=128, block=16, dtype="bf16", cap=0.0, alibi=False, window=0, prefix=0),
        # one whole long prompt, a bias by distance, small heads
        dict(name="prefill_long_alibi", op="prefill", seqs=1, ctx_min=8191, ctx_max=8191, new_min=0, new_max=0,
             q_heads=32, kv_heads=4, head_dim=64, block=16, dtype="bf16", cap=0.0, alibi=True, window=0, prefix=0),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append", "gather", "decode", "prefill"])
    kv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, kv_heads=kv, block=rng.choice([8, 16, 32]), dtype=rng.choice(["fp16", "bf16"]))
    if op == "gather":
        c["head_dim"] = rng.choice([64, 128, 256])
        most = 64 * 1152 * 8 * 128 // (kv * c["head_dim"])
        c["seqs"] = _log_uniform(rng, 1, 256)
        c["ctx_max"] = _log_uniform(rng, 1, max(1, min(32768, most // c["seqs"])))
        c["ctx_min"] = rng.randint(max(1, c["ctx_max"] // 3), c["ctx_max"])
        c["skip"] = rng.choice([0, 0, 5, 9])
        return c
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    while kv * group > 64:
        group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    c["q_heads"] = kv * group
    if op == "append":
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
        c["bits"] = rng.choice([8, 8, 16])
        c["norm"] = c["bits"] == 16 or rng.random() < 0.6
        return c
    c["cap"] = rng.choice([0.0, 0.0, 20.0, 50.0])
    c["alibi"] = rng.random() < 0.3
    c["window"] = rng.choice([0, 0, 0, 1, 100, 1024, 4096])
    c["prefix"] = rng.choice([0, 0, 0, 3, 500])
    if op == "decode":
        c["head_dim"] = rng.choice([64, 128, 256])
        most = 6 * 26000 * 8 * 256 // (kv * c["head_dim"])  # visible or not: the history is in the pool
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


def _append_lens(case):
    """Tokens of each sequence in an append case."""
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
    D, Hk = case["head_dim"], case["kv_heads"]
    if case["op"] == "gather":
        T = sum(_lens(case))
        kept = T - (T // case["skip"] if case["skip"] else 0)
        return {"bytes": kept * 2 * Hk * D * 3 + T * 4 + 8 * Hk, "flops": kept * 2 * Hk * D}
    Hq = case["q_heads"]
    if case["op"] == "append":
        T = case["tokens"]
        kept = T - (T // case["skip"] if case["skip"] else 0)
        out = case["bits"] // 8
        return {"bytes": T * 2 * Hq * D * 2 + kept * 2 * Hk * D * (2 + out) + T * (case["rotary"] * 4 + 8),
                "flops": (T * Hq + kept * Hk) * (3 * case["rotary"] + (4 * D if case["norm"] else 0))
                + (kept * 2 * Hk * D if out == 1 else 0)}
    ctx = _lens(case)
    W, pre = case["window"], case["prefix"]
    if case["op"] == "decode":
        seen = [_visible(c - 1, c, W, pre) for c in ctx]
        return {"bytes": sum(seen) * Hk * D * 2 + case["seqs"] * (Hq * D * 4 + 4)
                + sum(4 * -(-v // case["block"]) for v in seen), "flops": 4 * D * Hq * sum(seen)}
    new = _new(case)
    pairs = sum(_visible(p, c, W, pre) for c, n in zip(ctx, new) for p in range(c - n, c))
    keys = sum(min(c, (n + W - 1 + pre) if W else c) for c, n in zip(ctx, new))
    return {"bytes": sum(new) * Hq * D * 4 + keys * Hk * D * 2 + sum(4 * -(-c // case["block"]) for c in ctx),
            "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------ inputs

def _scales(heads, gen, dev):
    """A scale for each head, as amax / 448 of calibrated values would give."""
    return 0.01 + 0.01 * torch.rand(heads, generator=gen, device=dev)


def _pool(case, ctx, gen, dev):
    """A shuffled 8-bit block pool that holds the sequences: caches, block tables, lengths."""
    B, Hk, D = case["block"], case["kv_heads"], case["head_dim"]
    need = [-(-c // B) for c in ctx]
    N = sum(need) + max(2, sum(need) // 10)
    caches = []
    for _ in range(2):
        x = torch.empty(N, Hk, B, D, dtype=torch.float16, device=dev).normal_(generator=gen)
        caches.append(x.mul_(70.0).clamp_(-448.0, 448.0).to(E4M3))
    order = torch.randperm(N, generator=gen, device=dev)[:sum(need)].to(torch.int32).cpu()
    tables = torch.full((len(ctx), max(need)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = order[at:at + n]
        at += n
    return caches[0], caches[1], tables.to(dev), torch.tensor(ctx, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    D, Hk, B, dt = case["head_dim"], case["kv_heads"], case["block"], _DT[case["dtype"]]
    ks, vs = _scales(Hk, gen, dev), _scales(Hk, gen, dev)
    if case["op"] == "append":
        Hq = case["q_heads"]
        T, n, r = case["tokens"], case["seqs"], case["rotary"]
        lens = _append_lens(case)
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
        weights = [1.0 + 0.2 * torch.randn(D, generator=gen, device=dev) for _ in range(2)] if case["norm"] else [None] * 2
        kc = torch.zeros(N, Hk, B, D, dtype=torch.float16 if case["bits"] == 8 else dt, device=dev)
        kc = kc.to(E4M3) if case["bits"] == 8 else kc
        return dict(op="append", q=q, k=k, v=v, k_cache=kc, v_cache=kc.clone(), positions=pos, table=table,
                    slots=slots.to(dev), interleaved=case["interleaved"], q_weight=weights[0], k_weight=weights[1],
                    k_scales=ks if case["bits"] == 8 else None, v_scales=vs if case["bits"] == 8 else None,
                    q_out=torch.zeros(T, Hq, D, dtype=dt, device=dev))
    ctx = _lens(case)
    kc, vc, tables, lens = _pool(case, ctx, gen, dev)
    if case["op"] == "gather":
        slots = []
        for s, c in enumerate(ctx):
            t = torch.arange(c, device=dev)
            slots.append(tables[s].long()[t // B] * B + t % B)
        slots = torch.cat(slots).to(torch.int32)
        if case["skip"]:
            slots[case["skip"] - 1::case["skip"]] = -1
        T = slots.shape[0]
        return dict(op="gather", k_cache=kc, v_cache=vc, k_scales=ks, v_scales=vs, slots=slots,
                    k_out=torch.zeros(T, Hk, D, dtype=dt, device=dev), v_out=torch.zeros(T, Hk, D, dtype=dt, device=dev))
    Hq = case["q_heads"]
    st = dict(op=case["op"], k_cache=kc, v_cache=vc, k_scales=ks, v_scales=vs, tables=tables, lens=lens, scale=D ** -0.5,
              cap=case["cap"], window=case["window"],
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
    return st


# ------------------------------------------------------------------ plain forms

def _normed(x, weight):
    """x [T, H, D] fp32; every head's row by the root of its mean square."""
    return x if weight is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight


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


def _plain_append(st):
    h = st["table"].shape[1] // 2
    cs = st["table"][st["positions"].long()]
    cos, sin = cs[:, :h], cs[:, h:]
    st["q_out"].copy_(_rotate(_normed(st["q"].float(), st["q_weight"]), cos, sin, st["interleaved"]))
    keep = st["slots"] >= 0
    slot = st["slots"][keep].long()
    B = st["k_cache"].shape[2]

    def put(cache, x, scales):
        x = x[keep]
        if scales is not None:
            x = (x / scales[:, None]).clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)
            cache.view(torch.uint8)[slot // B, :, slot % B] = x
        else:
            cache[slot // B, :, slot % B] = x.to(cache.dtype)

    put(st["k_cache"], _rotate(_normed(st["k"].float(), st["k_weight"]), cos, sin, st["interleaved"]), st["k_scales"])
    put(st["v_cache"], st["v"].float(), st["v_scales"])
    return [st["q_out"], st["k_cache"], st["v_cache"]]


def _plain_gather(st):
    B = st["k_cache"].shape[2]
    keep = st["slots"] >= 0
    slot = st["slots"][keep].long()

    def take(out, cache, scales):
        x = cache.view(torch.uint8)[slot // B, :, slot % B].view(E4M3).float() * scales[:, None]
        out[keep] = x.to(out.dtype)

    take(st["k_out"], st["k_cache"], st["k_scales"])
    take(st["v_out"], st["v_cache"], st["v_scales"])
    return [st["k_out"], st["v_out"]]


def _plain_attention(st):
    tables, starts = st["tables"], st["starts"].long()
    S, n = tables.shape[0], st["max_new"]
    _, Hk, B, D = st["k_cache"].shape
    Hq = st["q"].shape[1]
    G = Hq // Hk
    idx = tables.clamp(min=0).long()

    def history(cache, scales):                                        # [S, Hk, K, D]
        x = cache.view(torch.uint8)[idx].transpose(1, 2).reshape(S, Hk, -1, D).view(E4M3).float()
        return x * scales[:, None, None]

    k, v = history(st["k_cache"], st["k_scales"]), history(st["v_cache"], st["v_scales"])
    K = k.shape[2]
    count = starts[1:] - starts[:-1]
    i = torch.arange(n, device=k.device)
    row = (starts[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)     # [S, n]
    q = st["q"][row].float().view(S, n, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hk, G * n, D)
    s = torch.matmul(q, k.transpose(2, 3)).mul_(st["scale"]).view(S, Hk, G, n, K)
    if st["cap"]:
        s.div_(st["cap"]).tanh_().mul_(st["cap"])
    lens = st["lens"].long()
    pos = (lens - count)[:, None] + i                                  # [S, n]
    j = torch.arange(K, device=k.device)
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
        return (_plain_append(st) if st["op"] == "append" else
                _plain_gather(st) if st["op"] == "gather" else _plain_attention(st))
    import paged_kv_cache_269_gb300 as pa
    if st["op"] == "append":
        pa.norm_rope_and_cache(st["q_out"], st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["positions"],
                               st["table"], st["slots"], q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS,
                               interleaved=st["interleaved"], k_scales=st["k_scales"], v_scales=st["v_scales"])
        return [st["q_out"], st["k_cache"], st["v_cache"]]
    if st["op"] == "gather":
        pa.gather_cache_q8(st["k_out"], st["v_out"], st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"],
                           st["slots"])
        return [st["k_out"], st["v_out"]]
    if st["op"] == "decode":
        return pa.decode_grouped_q8(st["out"], st["q"], st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"],
                                    st["tables"], st["lens"], st["scale"], softcap=st["cap"], alibi_slopes=st["slopes"],
                                    window=st["window"], prefix_lens=st["prefix"])
    return pa.prefill_grouped_q8(st["out"], st["q"], st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"],
                                 st["tables"], st["lens"], st["starts"], st["scale"], max_query_len=st["max_new"],
                                 softcap=st["cap"], alibi_slopes=st["slopes"], window=st["window"],
                                 prefix_lens=st["prefix"])


# ------------------------------------------------------------------ the definition, in 64 bits

def _to_e4m3(x):
    """x (fp64) at the nearest e4m3 number, ties to even, saturated at 448: a sign, 4 significant bits, steps of 2^-9 below 2^-6."""
    exponent = torch.frexp(x)[1].clamp(min=-5) - 4   # frexp's mantissa is in [1/2, 1): 4 bits of it
    step = torch.ldexp(torch.ones_like(x), exponent)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    B, Hk, D = case["block"], case["kv_heads"], case["head_dim"]
    if case["op"] == "append":
        T, r = case["tokens"], case["rotary"]
        # the operator's input is the fp32 table: its rows, widened
        rows = st["table"].to(f64).index_select(0, st["positions"].long())
        turn = torch.complex(rows[:, :r // 2], rows[:, r // 2:])[:, None, :]

        def turned(x, weight):
            x = x.to(f64)
            if weight is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["head_dim"] + 1e-6) * weight.to(f64)
            part = x[..., :r]
            pairs = part.unflatten(-1, (r // 2, 2)) if case["interleaved"] else part.unflatten(-1, (2, r // 2)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            z = z.reshape(part.shape) if case["interleaved"] else z.transpose(-1, -2).reshape(part.shape)
            return torch.cat([z, x[..., r:]], dim=-1)

        out = []
        for cache, x, scales in ((st["k_cache"], turned(st["k"], st["k_weight"]), st["k_scales"]),
                                 (st["v_cache"], st["v"].to(f64), st["v_scales"])):
            if scales is not None:
                x = _to_e4m3(x / scales.to(f64)[:, None])
            flat = cache.to(torch.float32).to(f64).permute(0, 2, 1, 3).reshape(-1, Hk, D)
            ok = (st["slots"] >= 0).nonzero().flatten()
            flat.index_copy_(0, st["slots"][ok].long(), x[ok])
            out.append(flat.view(-1, B, Hk, D).permute(0, 2, 1, 3).contiguous())
        return [turned(st["q"], st["q_weight"]), out[0], out[1]]

    def values(cache, scales):
        return cache.to(torch.float32).to(f64) * scales.to(f64)[:, None, None]

    if case["op"] == "gather":
        at = (st["slots"] >= 0).nonzero().flatten()
        out = []
        for cache, scales in ((st["k_cache"], st["k_scales"]), (st["v_cache"], st["v_scales"])):
            flat = values(cache, scales).permute(0, 2, 1, 3).reshape(-1, Hk, D)
            x = torch.zeros(st["slots"].shape[0], Hk, D, dtype=f64, device=flat.device)
            out.append(x.index_copy(0, at, flat.index_select(0, st["slots"][at].long())))
        return out
    ctx = _lens(case)
    new = [1] * len(ctx) if case["op"] == "decode" else _new(case)
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
        keys, vals = (x.view(torch.uint8).index_select(0, blocks).view(E4M3).to(torch.float32).to(f64) * y.to(f64)[:, None, None]
                      for x, y in ((st["k_cache"], st["k_scales"]), (st["v_cache"], st["v_scales"])))
        for h in range(Hk):
            K, V = keys[:, h].reshape(-1, D)[:c], vals[:, h].reshape(-1, D)[:c]
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
