"""The attention operators around the expert layer, case by case: what each one is given, computes and costs.

Three operators over a paged key/value cache held in 8 bits (E4M3 codes, one power-of-two scale per page and head):

  append     normalise (optionally) and rotate the new queries and keys, quantise the new keys and values into the cache
  gather     read a range of cached tokens of each sequence back in bf16
  attention  softmax attention of the new queries over their sequence's cached keys and values

`run` computes them either in their plain form (elementary torch operations in fp32) or, with `own`, by the framework's calls.

The cache.  Page p of head h holds `page` tokens of D codes, [n_pages, Hkv, page, D], and scale byte b = k_scale[p, h]
stands for 2^(b - 127).  With a = the largest finite magnitude among the new tokens of a page (before quantisation), the
exponent is e = max(-64, ceil(log2(a / 448))) -- the smallest power of two that keeps every code within +-448 -- and at least
the page's present exponent when the page already holds earlier tokens of its sequence; if it grows, the earlier tokens'
codes are rounded again to the new scale.
"""
import math
import random

import torch

own = False

D = 128          # head size


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one user's next token, early in a conversation: latency of the smallest append
        _case("append_one", op="append", B=1, new=(1, 1), ctx=(36, 36), Hq=32, Hkv=4, page=16, norm=False),
        # a decode batch of 64 (the decode workload's T) at ragged positions, with the query/key norms
        _case("append_decode_64", op="append", B=64, new=(1, 1), ctx=(0, 8190), Hq=64, Hkv=8, page=64, norm=True),
        # a mixed batch: prompts and chunks of odd lengths behind cached prefixes, interleaved rotation of half the head
        _case("append_ragged", op="append", B=7, new=(1, 1300), ctx=(0, 3000), Hq=32, Hkv=4, page=32, norm=True, rot=64, interleaved=True),
        # one long prompt (the long prefill workload's T)
        _case("append_prompt_16384", op="append", B=1, new=(16384, 16384), ctx=(0, 0), Hq=64, Hkv=8, page=64, norm=True),
        # a short prefix handed to another reader of the cache
        _case("gather_short", op="gather", B=1, new=(200, 200), ctx=(17, 17), Hq=32, Hkv=4, page=16),
        # cached prefixes of a batch read back whole
        _case("gather_batch", op="gather", B=16, new=(500, 9000), ctx=(0, 500), Hq=64, Hkv=8, page=64),
        # the first decode step after a short prompt: latency
        _case("attend_one", op="attention", B=1, new=(1, 1), ctx=(128, 128), Hq=32, Hkv=4, page=16),
        # the decode batch of 64 over a few thousand tokens each
        _case("attend_decode_64", op="attention", B=64, new=(1, 1), ctx=(1500, 8190), Hq=64, Hkv=8, page=64),
        # one user's decode step far into a long document
        _case("attend_decode_long", op="attention", B=1, new=(1, 1), ctx=(131000, 131000), Hq=64, Hkv=8, page=64),
        # a batch of 16 whose last few tokens are checked together (speculative decoding), sliding window
        _case("attend_verify_16", op="attention", B=16, new=(2, 5), ctx=(300, 12000), Hq=32, Hkv=8, page=128, window=4096),
        # chunked prefill: chunks of odd lengths behind prefixes
        _case("attend_ragged", op="attention", B=4, new=(100, 1900), ctx=(0, 5000), Hq=64, Hkv=8, page=32),
        # one long prompt
        _case("attend_prompt_16384", op="attention", B=1, new=(16384, 16384), ctx=(0, 0), Hq=32, Hkv=4, page=64),
    ]


def _case(name, op, B, new, ctx, Hq, Hkv, page, norm=False, rot=D, interleaved=False, causal=True, window=0, spread=1):
    c = dict(op=op, B=B, new_lo=new[0], new_hi=new[1], ctx_lo=ctx[0], ctx_hi=ctx[1], Hq=Hq, Hkv=Hkv, page=page, spread=spread)
    if op == "append":
        c.update(norm=norm, rot=rot, interleaved=interleaved)
    if op == "attention":
        c.update(causal=causal, window=window)
    return dict(c, name=name) if name else c


_HEADS = [(64, 8), (32, 4), (32, 8), (16, 2), (8, 8), (20, 4), (28, 4), (12, 1)]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    Hq, Hkv = rng.choice(_HEADS)
    page = rng.choice([16, 32, 64, 128])
    spread = rng.randrange(1, 1 << 20)
    op = rng.choice(["append", "append", "gather", "attention", "attention", "attention", "attention"])
    if op == "append":
        kind = rng.choice(["decode", "mixed", "prompt"])
        if kind == "decode":
            B, new, ctx = _log(rng, 1, 128), (1, 1), (0, _log(rng, 1, 8000))
        elif kind == "mixed":
            B, new, ctx = rng.randint(2, 12), (0, _log(rng, 2, 1500)), (0, _log(rng, 1, 4000))
        else:
            n = _log(rng, 100, 16000)
            B, new, ctx = 1, (n, n), (0, 0)
        return _case(None, op, B, new, ctx, Hq, Hkv, page, norm=rng.random() < 0.6, rot=rng.choice([128, 128, 64, 32, 96]),
                     interleaved=rng.random() < 0.4, spread=spread)
    if op == "gather":
        B = _log(rng, 1, 16)
        return _case(None, op, B, (0, _log(rng, 8, 9000)), (0, _log(rng, 1, 3000)), Hq, Hkv, page, spread=spread)
    kind = rng.choice(["decode", "decode", "long", "verify", "prefill", "prefill"])
    window = rng.choice([0, 0, 0, _log(rng, 32, 4096)])
    causal = True
    if kind == "decode":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, 8000)
        new, ctx = (1, 1), (rng.randint(0, hi), hi)
    elif kind == "long":
        B = rng.randint(1, 2)
        n = _log(rng, 10000, 131000)
        new, ctx = (1, 1), (n // 2, n)
    elif kind == "verify":
        B = _log(rng, 1, 32)
        new, ctx = (0, rng.randint(2, 8)), (0, _log(rng, 10, 8000))
    else:
        B = rng.randint(1, 4)
        new, ctx = (0, _log(rng, 20, 2000)), (0, _log(rng, 1, 5000))
        causal = rng.random() < 0.8
    return _case(None, op, B, new, ctx, Hq, Hkv, page, causal=causal, window=window if causal else 0, spread=spread)


def _lengths(case):
    """(new tokens, tokens before them) of each sequence: part of the case, the same for every seed."""
    r = random.Random(case["spread"])
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    if not sum(new):
        new[0] = max(1, case["new_hi"])
    return new, ctx


# ------------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    rnd = random.Random(seed)
    new, ctx = _lengths(case)
    B, Hq, Hkv, page = case["B"], case["Hq"], case["Hkv"], case["page"]
    total = [a + b for a, b in zip(new, ctx)]
    T = sum(new)
    used = [-(-t // page) for t in total]
    width = max(1, max(used)) + 1
    n_pages = sum(used) + 3
    order = list(range(n_pages))
    rnd.shuffle(order)                       # a pool in use hands its pages out in no order
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    starts = torch.tensor([0] + new, dtype=torch.int64).cumsum(0)
    s = dict(case=dict(case), T=T, page_table=table.to(dev), q_start=starts.to(torch.int32).to(dev),
             kv_len=torch.tensor(total, dtype=torch.int32, device=dev), max_q=max(new), keep={})
    seq = torch.repeat_interleave(torch.arange(B), torch.tensor(new))
    s["seq"] = seq.to(dev)                   # sequence of each new token
    s["pos"] = (torch.arange(T) - starts[:-1][seq] + torch.tensor(ctx)[seq]).to(dev)

    # the cache as earlier appends left it: keys with a few strong channels, values of a size that drifts from page to page
    gain = torch.exp(0.5 * torch.randn(Hkv, 1, D, device=dev, generator=g))
    drift = torch.exp(0.7 * torch.randn(n_pages, 1, 1, 1, device=dev, generator=g))
    for name, mul in (("k", gain), ("v", drift)):
        codes = torch.empty(n_pages, Hkv, page, D, dtype=torch.uint8, device=dev)
        scale = torch.empty(n_pages, Hkv, dtype=torch.uint8, device=dev)
        for i in range(0, n_pages, 2048):
            x = torch.randn(min(2048, n_pages - i), Hkv, page, D, device=dev, generator=g)
            x *= mul if name == "k" else drift[i:i + 2048]
            e = _exponent(x.abs().amax((2, 3)))
            scale[i:i + 2048] = (e + 127).to(torch.uint8)
            codes[i:i + 2048] = (x * torch.exp2(-e)[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        s[name + "_codes"], s[name + "_scale"] = codes, scale

    if case["op"] == "append":
        # the rows of a merged projection [query heads | key heads | value heads]
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, device=dev, generator=g)
        qkv[:, :(Hq + Hkv) * D] *= 3.0
        s["qkv"] = qkv.to(torch.bfloat16)
        if case["norm"]:
            s["q_norm"] = (1 + 0.3 * torch.randn(D, device=dev, generator=g)).to(torch.bfloat16)
            s["k_norm"] = (1 + 0.3 * torch.randn(D, device=dev, generator=g)).to(torch.bfloat16)
        rot = case["rot"]
        angle = torch.arange(max(1, max(total)), device=dev, dtype=torch.float64)[:, None] * \
            1e6 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
        part = [b for b in range(B) if new[b] and ctx[b] % page]
        s["part_seq"] = torch.tensor(part, dtype=torch.int64, device=dev)
        s["part_page"] = torch.tensor([ctx[b] // page for b in part], dtype=torch.int64, device=dev)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        # what is read back: every page that the call touched, from its first token
        begin = [c // page * page if n else 0 for n, c in zip(new, ctx)]
        count = [t - b if n else 0 for n, t, b in zip(new, total, begin)]
    else:
        s["q"] = (torch.randn(T, Hq, D, device=dev, generator=g) * 1.5).to(torch.bfloat16) if case["op"] == "attention" else None
        begin, count = ctx, new
    s["g_start"] = torch.tensor(begin, dtype=torch.int32, device=dev)
    out_start = torch.tensor([0] + count, dtype=torch.int64).cumsum(0)
    s["g_out_start"] = out_start.to(torch.int32).to(dev)
    s["g_rows"] = int(out_start[-1])
    gseq = torch.repeat_interleave(torch.arange(B), torch.tensor(count))
    s["g_seq"] = gseq.to(dev)
    s["g_pos"] = (torch.arange(s["g_rows"]) - out_start[:-1][gseq] + torch.tensor(begin)[gseq]).to(dev)
    return s


def _exponent(amax):
    """max(-64, ceil(log2(amax / 448))), exactly: amax = m 2^x with m in [0.5, 1), and 448 = 0.875 * 2^9."""
    m, x = torch.frexp(amax)
    e = (x - 9 + (m > 0.875)).float()
    return torch.where(amax > 0, e, -64.0).clamp(min=-64)


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op == "append":
        q = _append(s)
        k, v = _gather(s)
        return {"q": q, "k": k, "v": v}
    if op == "gather":
        k, v = _gather(s)
        return {"k": k, "v": v}
    return {"out": _attention(s)}


def _run_own(s):
    import moe_expert_layer_fwd_gb300 as moe
    c, keep = s["case"], s["keep"]
    cache = moe.KVCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    if "ws" not in keep:
        keep["ws"] = moe.moe_paged_attention_workspace(s["T"], c["B"], c["Hq"], c["Hkv"], D, s["max_q"], s["page_table"].device)
    if c["op"] == "attention":
        return {"out": moe.moe_paged_attention(s["q"], cache, s["q_start"], s["kv_len"], s["page_table"], max_q=s["max_q"],
                                               causal=c["causal"], window=c["window"], ws=keep["ws"])}
    out = {}
    if c["op"] == "append":
        q, k, v = s["qkv"].view(s["T"], -1, D).split([c["Hq"], c["Hkv"], c["Hkv"]], dim=1)
        out["q"] = moe.moe_kv_append(q, k, v, cache, s["q_start"], s["kv_len"], s["page_table"], s["cos_sin"], rot_dim=c["rot"],
                                     interleaved=c["interleaved"], q_norm_weight=s.get("q_norm"), k_norm_weight=s.get("k_norm"),
                                     eps=1e-6, ws=keep["ws"])
    out["k"], out["v"] = moe.moe_kv_gather(cache, s["g_start"], s["g_out_start"], s["page_table"], s["g_rows"], ws=keep["ws"])
    return out


def _norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()


def _rotate(x, cos, sin, rot, interleaved):
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = (a * cos - b * sin, a * sin + b * cos)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat([y, x[..., rot:]], -1)


def _append(s):
    c = s["case"]
    page, Hkv, rot = c["page"], c["Hkv"], c["rot"]
    q, k, v = s["qkv"].view(s["T"], -1, D).float().split([c["Hq"], Hkv, Hkv], dim=1)
    if c["norm"]:
        q, k = _norm(q, s["q_norm"]), _norm(k, s["k_norm"])
    cs = s["cos_sin"][s["pos"]][:, None]
    q = _rotate(q, cs[..., :rot // 2], cs[..., rot // 2:], rot, c["interleaved"])
    k = _rotate(k, cs[..., :rot // 2], cs[..., rot // 2:], rot, c["interleaved"])
    pages = s["page_table"][s["seq"], s["pos"] // page].long()       # page of each new token
    slot = s["pos"] % page
    # pages that hold earlier tokens of their sequence: at most the first one that a sequence touches
    part = s["page_table"][s["part_seq"], s["part_page"]].long()
    for name, x in (("k", k), ("v", v)):
        codes, scale = s[name + "_codes"], s[name + "_scale"]
        n = codes.shape[0]
        old = scale[part].float() - 127
        least = torch.full((n, Hkv), -64.0, device=x.device)
        least[part] = old
        top = torch.zeros(n, Hkv, device=x.device).scatter_reduce_(0, pages[:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
        e = torch.maximum(_exponent(top), least)
        scale[pages] = (e[pages] + 127).to(torch.uint8)
        earlier = codes[part].view(torch.float8_e4m3fn).float() * torch.exp2(old - e[part])[:, :, None, None]
        codes[part] = earlier.to(torch.float8_e4m3fn).view(torch.uint8)
        codes[pages, :, slot] = (x * torch.exp2(-e[pages])[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.to(torch.bfloat16)


def _values(codes, scale):
    return codes.view(torch.float8_e4m3fn).float() * torch.exp2(scale.float() - 127)[..., None]


def _gather(s):
    page = s["case"]["page"]
    pages, slot = s["page_table"][s["g_seq"], s["g_pos"] // page].long(), s["g_pos"] % page
    return tuple(_values(s[n + "_codes"][pages, :, slot], s[n + "_scale"][pages]).to(torch.bfloat16) for n in "kv")


def _attention(s):
    c = s["case"]
    B, Hq, Hkv, page, Tq = c["B"], c["Hq"], c["Hkv"], c["page"], s["max_q"]
    G = Hq // Hkv
    pages = s["page_table"][:, :-1].long().clamp(min=0)
    S = pages.shape[1] * page
    j = torch.arange(S, device=pages.device)
    there = j < s["kv_len"][:, None]                                  # [B, S]

    def rows(name):                                                   # [B, Hkv, S, D]
        x = _values(s[name + "_codes"][pages], s[name + "_scale"][pages][..., None])
        x = x.transpose(1, 2).reshape(B, Hkv, S, D)
        return x.masked_fill_(~there[:, None, :, None], 0.0)

    # queries padded to the longest sequence's
    i = torch.arange(Tq, device=pages.device)
    n_new = s["q_start"][1:] - s["q_start"][:-1]
    token = (s["q_start"][:-1, None] + i).long().clamp(max=s["T"] - 1)
    q = s["q"].float()[token].view(B, Tq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Tq, D)
    p = torch.matmul(q * D ** -0.5, rows("k").transpose(-1, -2)).view(B, Hkv, G, Tq, S)
    pos = (s["kv_len"] - n_new)[:, None] + i                          # [B, Tq]
    seen = there[:, None, :].expand(B, Tq, S)
    if c["causal"]:
        seen = seen & (j <= pos[..., None])
    if c["window"]:
        seen = seen & (j > pos[..., None] - c["window"])
    p.masked_fill_(~seen[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, Hkv, G * Tq, S), rows("v")).view(B, Hkv, G, Tq, D)
    out = out / torch.where(total > 0, total, 1.0)
    out = out[s["seq"], :, :, (torch.arange(s["T"], device=pages.device) - s["q_start"][s["seq"]])]
    return out.reshape(s["T"], Hq, D).to(torch.bfloat16)


# ------------------------------------------------------------------------------------------------ costs
def _visible(case):
    """Over the sequences: query-key pairs that the masks leave, and keys that some query of the sequence sees."""
    pairs = keys = 0
    for n, c in zip(*_lengths(case)):
        if not n:
            continue
        if not case["causal"]:
            pairs, keys = pairs + n * (c + n), keys + c + n
            continue
        w = case["window"] or c + n
        keys += min(c + n, w + n - 1)
        full = max(0, min(n, w - c))          # queries that see everything before them
        pairs += full * c + full * (full + 1) // 2 + (n - full) * w
    return pairs, keys


def work(case):
    new, ctx = _lengths(case)
    T, Hq, Hkv, page = sum(new), case["Hq"], case["Hkv"], case["page"]
    if case["op"] == "attention":
        pairs, keys = _visible(case)
        return {"bytes": 2 * keys * Hkv * D + 4 * T * Hq * D, "flops": 4 * pairs * Hq * D}
    if case["op"] == "gather":
        return {"bytes": 6 * T * Hkv * D, "flops": 2 * T * Hkv * D}
    back = sum(n + c - c // page * page for n, c in zip(new, ctx) if n)
    table = T * case["rot"] * 4
    return {"bytes": T * (4 * Hq + 4 * Hkv + 2 * Hkv) * D + table + 6 * back * Hkv * D, "flops": 8 * T * (Hq + 2 * Hkv) * D}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _e4m3(x):
    """The nearest E4M3 value, ties to even: 3 fraction bits down to 2^-6, then multiples of 2^-9."""
    _, ex = torch.frexp(x.abs())
    step = torch.exp2((ex - 4).clamp(min=-9).double())
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    page, Hq, Hkv = case["page"], case["Hq"], case["Hkv"]
    new, ctx = _lengths(case)
    table = s["page_table"].long()

    def cached(name, b, lo, hi, codes=None):
        """Tokens [lo, hi) of sequence b, [Hkv, hi - lo, D] in 64 bits."""
        at = table[b, lo // page:-(-hi // page)]
        x = s[name + "_codes"][at].view(torch.float8_e4m3fn).double() * torch.exp2(s[name + "_scale"][at].double() - 127)[:, :, None, None]
        return x.transpose(0, 1).flatten(1, 2)[:, lo - lo // page * page:][:, :hi - lo]

    if case["op"] == "gather":
        parts = {n: [cached(n, b, c, c + t).transpose(0, 1) for b, (t, c) in enumerate(zip(new, ctx)) if t] for n in "kv"}
        return {n: torch.cat(parts[n]) for n in "kv"}

    if case["op"] == "attention":
        pairs, _ = _visible(case)
        if pairs * Hq * D * 8 > 1.2e13:
            return None
        outs, at = [], 0
        for b, (t, c) in enumerate(zip(new, ctx)):
            if not t:
                continue
            k, v = cached("k", b, 0, c + t), cached("v", b, 0, c + t)
            j = torch.arange(c + t, device=k.device)
            for i in range(0, t, 1024):
                n = min(1024, t - i)
                q = s["q"][at + i:at + i + n].double().view(n, Hkv, Hq // Hkv, D)
                hi = c + i + n if case["causal"] else c + t
                z = torch.einsum("ihgd,hjd->higj", q, k[:, :hi]) / math.sqrt(D)
                here = (c + i + torch.arange(n, device=k.device))[:, None]
                no = torch.zeros(n, hi, dtype=torch.bool, device=k.device)
                if case["causal"]:
                    no |= j[:hi] > here
                if case["window"]:
                    no |= j[:hi] <= here - case["window"]
                z.masked_fill_(no[:, None], -math.inf)
                outs.append(torch.einsum("higj,hjd->ihgd", torch.softmax(z, -1), v[:, :hi]).reshape(n, Hq, D))
            at += t
        return {"out": torch.cat(outs)}

    rot = case["rot"]
    qs, ks, vs, at = [], [], [], 0
    for b, (t, c) in enumerate(zip(new, ctx)):
        if not t:
            continue
        q, k, v = s["qkv"][at:at + t].double().view(t, -1, D).split([Hq, Hkv, Hkv], dim=1)
        if case["norm"]:
            q = q / torch.sqrt(q.square().mean(-1, keepdim=True) + 1e-6) * s["q_norm"].double()
            k = k / torch.sqrt(k.square().mean(-1, keepdim=True) + 1e-6) * s["k_norm"].double()
        cs = s["cos_sin"][c:c + t].double()
        turn = torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])[:, None]
        done = []
        for x in (q, k):
            r = x[..., :rot]
            pair = r.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else r.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
            z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
            done.append(torch.cat([z, x[..., rot:]], -1))
        qs.append(done[0])
        first = c // page * page
        for name, x, to in (("k", done[1], ks), ("v", v, vs)):
            before = cached(name, b, first, c).transpose(0, 1) if c > first else x[:0]
            for p in range(first, c + t, page):                       # page by page
                lo, hi = max(p, c), min(p + page, c + t)
                y = x[lo - c:hi - c]
                a = y.abs().amax((0, 2))
                m, ex = torch.frexp(a)
                e = torch.where(a > 0, (ex - 9 + (m > 0.875)).double(), -64.0).clamp(min=-64)
                if p < c:
                    e = torch.maximum(e, s[name + "_scale"][table[b, p // page]].double() - 127)
                    to.append(_e4m3(before / torch.exp2(e)[:, None]) * torch.exp2(e)[:, None])
                to.append(_e4m3(y / torch.exp2(e)[:, None]) * torch.exp2(e)[:, None])
        at += t
    return {"q": torch.cat(qs), "k": torch.cat(ks), "v": torch.cat(vs)}
