"""Operators around the attention cache for long conversations, case by case: what each one is given, computes and costs.

Four operators over the paged 8-bit key/value cache (E4M3 codes, one power-of-two scale per page and head):

  append   rotate the new queries and keys by positions on several axes (time, height, width) that the caller gives, and
           quantise the new keys and values into the cache
  shared   softmax attention of a batch whose groups of sequences share a long prefix, read once for all of a group, with the
           logarithm of every row's denominator
  weights  add up, for every cached key of a head, the attention weights that the new queries give it
  evict    keep the tokens of the largest accumulated weights, each head its own, packed into new pages

`run` computes them either in their plain form (elementary torch operations in fp32) or, with `own`, by the framework's calls.

The cache.  Page p of head h holds `page` tokens of D codes, [n_pages, Hkv, page, D], and scale byte b = k_scale[p, h]
stands for 2^(b - 127).  Append: with a = the largest finite magnitude among the new tokens of a page, the exponent is
e = max(-64, ceil(log2(a / 448))), and at least the page's present exponent when the page already holds earlier tokens of its
sequence; if it grows, the earlier tokens' codes are rounded again to the new scale.  Evict: the exponent of a new page is
the largest of those that its tokens had, and the codes are rounded again to it.
"""
import math
import random

import torch

own = False

D = 128          # head size
MAX_POS = 32768  # rows of the rotation table


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the next token of one conversation whose prompt held images: latency
        _append("append_one", B=1, new=(1, 1), ctx=(77, 77), Hq=32, Hkv=4, page=16),
        # a decode batch of 64 (the decode workload's T) after evictions: positions on one axis, far from the slots
        _append("append_decode_64", B=64, new=(1, 1), ctx=(0, 2100), Hq=64, Hkv=8, page=64, axes=1),
        # prompts of text and images of odd sizes behind cached turns, axes dealt out one by one
        _append("append_images", B=5, new=(300, 4100), ctx=(0, 900), Hq=32, Hkv=4, page=32, strided=True),
        # four answers sampled from one short prompt: latency
        _shared("shared_few", groups=1, B=4, new=(1, 1), own=(0, 40), prefix=(500, 500), Hq=32, Hkv=4, page=16),
        # a decode batch of 64 behind one long system prompt
        _shared("shared_decode_64", groups=1, B=64, new=(1, 1), own=(50, 1000), prefix=(8200, 8200), Hq=64, Hkv=8, page=64),
        # three documents, a few readers of each, whose last few tokens are checked together (speculative decoding)
        _shared("shared_documents", groups=3, B=21, new=(0, 5), own=(0, 700), prefix=(1000, 30000), Hq=64, Hkv=8, page=128),
        # questions of odd lengths sent behind one long prompt
        _shared("shared_questions", groups=1, B=16, new=(20, 250), own=(0, 300), prefix=(4001, 4001), Hq=32, Hkv=4, page=64),
        # one decode step of a short conversation: latency
        _weights("weights_one", B=1, new=(1, 1), ctx=(130, 130), Hq=32, Hkv=4, page=16),
        # the decode batch of 64 over a few thousand tokens each
        _weights("weights_decode_64", B=64, new=(1, 1), ctx=(1500, 8190), Hq=64, Hkv=8, page=64),
        # the last tokens of long prompts, whose weights choose what of the prompt stays
        _weights("weights_prompt_end", B=4, new=(40, 64), ctx=(5000, 16000), Hq=64, Hkv=8, page=32),
        # one short conversation cut to its budget: latency
        _evict("evict_one", B=1, ctx=(700, 700), keep=(200, 200), sink=4, recent=32, Hkv=4, page=16),
        # a batch of long conversations cut to a quarter
        _evict("evict_batch", B=32, ctx=(3000, 9000), keep=(1500, 2200), sink=4, recent=256, Hkv=8, page=64),
    ]


def _case(name, **c):
    return dict(c, name=name) if name else c


def _append(name, B, new, ctx, Hq, Hkv, page, axes=3, strided=False, norm=True, rot=D, interleaved=False, spread=1):
    return _case(name, op="append", B=B, new_lo=new[0], new_hi=new[1], ctx_lo=ctx[0], ctx_hi=ctx[1], Hq=Hq, Hkv=Hkv, page=page,
                 axes=axes, strided=strided, norm=norm, rot=rot, interleaved=interleaved, spread=spread)


def _shared(name, groups, B, new, own, prefix, Hq, Hkv, page, spread=1):
    return _case(name, op="shared", groups=groups, B=B, new_lo=new[0], new_hi=new[1], ctx_lo=own[0], ctx_hi=own[1],
                 prefix_lo=prefix[0], prefix_hi=prefix[1], Hq=Hq, Hkv=Hkv, page=page, spread=spread)


def _weights(name, B, new, ctx, Hq, Hkv, page, window=0, fresh=False, spread=1):
    return _case(name, op="weights", B=B, new_lo=new[0], new_hi=new[1], ctx_lo=ctx[0], ctx_hi=ctx[1], Hq=Hq, Hkv=Hkv, page=page,
                 window=window, fresh=fresh, spread=spread)


def _evict(name, B, ctx, keep, sink, recent, Hkv, page, spread=1):
    return _case(name, op="evict", B=B, new_lo=0, new_hi=0, ctx_lo=ctx[0], ctx_hi=ctx[1], keep_lo=keep[0], keep_hi=keep[1], sink=sink,
                 recent=recent, Hq=Hkv, Hkv=Hkv, page=page, spread=spread)


_HEADS = [(64, 8), (32, 4), (32, 8), (16, 2), (8, 8), (20, 4), (28, 4), (12, 1)]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    Hq, Hkv = rng.choice(_HEADS)
    page = rng.choice([16, 32, 64, 128])
    spread = rng.randrange(1, 1 << 20)
    op = rng.choice(["append", "shared", "shared", "weights", "weights", "evict", "evict"])
    if op == "append":
        kind = rng.choice(["decode", "mixed", "prompt"])
        if kind == "decode":
            B, new, ctx = _log(rng, 1, 128), (1, 1), (0, _log(rng, 1, 8000))
        elif kind == "mixed":
            B, new, ctx = rng.randint(2, 12), (0, _log(rng, 2, 1500)), (0, _log(rng, 1, 4000))
        else:
            n = _log(rng, 100, 14000)
            B, new, ctx = 1, (n, n), (0, 0)
        return _append(None, B, new, ctx, Hq, Hkv, page, axes=rng.choice([1, 2, 3, 3, 4]), strided=rng.random() < 0.4,
                       norm=rng.random() < 0.6, rot=rng.choice([128, 128, 64, 32, 96]), interleaved=rng.random() < 0.4, spread=spread)
    if op == "shared":
        groups = _log(rng, 1, 6)
        if rng.random() < 0.7:
            B, new = groups * _log(rng, 1, 32 // groups), (1, 1)
            if rng.random() < 0.4:
                new = (0, rng.randint(2, 8))
        else:
            B, new = groups * rng.randint(1, 2), (0, _log(rng, 20, 250))
        hi = _log(rng, 16, 8200)
        return _shared(None, groups, B, new, (0, _log(rng, 1, 1500)), (rng.randint(0, hi), hi), Hq, Hkv, page, spread=spread)
    if op == "weights":
        kind = rng.choice(["decode", "decode", "verify", "end", "prompt"])
        window = rng.choice([0, 0, 0, _log(rng, 32, 4096)])
        if kind == "decode":
            B, new, hi = _log(rng, 1, 64), (1, 1), _log(rng, 1, 8000)
        elif kind == "verify":
            B, new, hi = _log(rng, 1, 32), (0, rng.randint(2, 8)), _log(rng, 10, 8000)
        elif kind == "end":
            B, new, hi = rng.randint(1, 4), (8, 64), _log(rng, 100, 16000)
        else:
            B, new, hi = rng.randint(1, 3), (0, _log(rng, 20, 1200)), _log(rng, 1, 3000)
        return _weights(None, B, new, (rng.randint(0, hi), hi), Hq, Hkv, page, window=window, fresh=rng.random() < 0.3, spread=spread)
    B = _log(rng, 1, 24)
    hi = _log(rng, 64, 9000 if B > 2 else 100000)
    keep = _log(rng, 1, min(hi, 6000))
    return _evict(None, B, (rng.randint(0, hi), hi), (rng.randint(0, keep), keep), rng.choice([0, 1, 4]), rng.choice([0, 8, _log(rng, 8, 500)]),
                  Hkv, page, spread=spread)


def _lengths(case):
    """Of each sequence: new tokens, tokens before them; of each group: sequences, prefix; of each sequence: tokens kept.
    Part of the case, the same for every seed."""
    r = random.Random(case["spread"])
    B = case["B"]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(B)]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(B)]
    if not sum(new):
        new[0] = 0 if case["op"] == "evict" else max(1, case["new_hi"])
    if case["op"] == "evict":
        return new, ctx, [r.randint(case["keep_lo"], case["keep_hi"]) for _ in range(B)]
    if case["op"] == "shared":
        n = case["groups"]
        cuts = sorted(r.randint(0, B) for _ in range(n - 1))
        members = [b - a for a, b in zip([0] + cuts, cuts + [B])]
        return new, ctx, members, [r.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(n)]
    return new, ctx


# ------------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    rnd = random.Random(seed)
    op = case["op"]
    new, ctx = _lengths(case)[:2]
    B, Hq, Hkv, page = case["B"], case["Hq"], case["Hkv"], case["page"]
    total = [a + b for a, b in zip(new, ctx)]
    T = sum(new)
    s = dict(case=dict(case), T=T, max_q=max(new), keep={})
    if op == "shared":
        members, prefix = _lengths(case)[2:]
        tokens = [sum(new[sum(members[:i]):sum(members[:i + 1])]) for i in range(len(members))]
        more = prefix
    elif op == "evict":
        keeps = _lengths(case)[2]
        more = [min(a, b) for a, b in zip(keeps, total)]
    else:
        more = []

    # one pool; a pool in use hands its pages out in no order
    lists = [-(-t // page) for t in total] + [-(-t // page) for t in more]
    n_pages = sum(lists) + 3
    order = list(range(n_pages))
    rnd.shuffle(order)
    rows, at = [], 0
    for n in lists:
        rows.append(order[at:at + n])
        at += n

    def table(rows):
        t = torch.full((len(rows), max(1, max(len(r) for r in rows)) + (op != "evict")), -1, dtype=torch.int32)
        for i, r in enumerate(rows):
            t[i, :len(r)] = torch.tensor(r, dtype=torch.int32)
        return t.to(dev)

    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    starts = torch.tensor([0] + new, dtype=torch.int64).cumsum(0)
    s.update(page_table=table(rows[:B]), q_start=starts.to(torch.int32).to(dev), kv_len=i32(total))
    seq = torch.repeat_interleave(torch.arange(B), torch.tensor(new))
    s["seq"] = seq.to(dev)                   # sequence of each new token
    s["slot"] = (torch.arange(T) - starts[:-1][seq] + torch.tensor(ctx)[seq]).to(dev)

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

    if op in ("shared", "weights"):
        s["q"] = (torch.randn(T, Hq, D, device=dev, generator=g) * 1.5).to(torch.bfloat16)
    if op == "shared":
        s["prefix_table"], s["prefix_len"] = table(rows[B:]), i32(prefix)
        s["prefix_start"] = i32([sum(tokens[:i]) for i in range(len(tokens) + 1)])
        s["max_prefix_q"] = max(tokens)
        s["tokens"], s["prefix"] = tokens, prefix
    if op == "weights":
        # weights that earlier steps added up, and the denominators that the attention before this call left
        s["weight"] = torch.exp(2.0 * torch.randn(n_pages, Hkv, page, device=dev, generator=g) - 2.0)
        s["weight_out"] = s["weight"].clone()
        s["lse"] = torch.empty(T, Hq, device=dev)
        for b, z in _scores(s, new):
            s["lse"][int(starts[b]):int(starts[b + 1])] = torch.logsumexp(z, -1).permute(2, 0, 1).reshape(new[b], Hq)
    if op == "append":
        # the rows of a merged projection [query heads | key heads | value heads]
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, device=dev, generator=g)
        qkv[:, :(Hq + Hkv) * D] *= 3.0
        s["qkv"] = qkv.to(torch.bfloat16)
        if case["norm"]:
            s["q_norm"] = (1 + 0.3 * torch.randn(D, device=dev, generator=g)).to(torch.bfloat16)
            s["k_norm"] = (1 + 0.3 * torch.randn(D, device=dev, generator=g)).to(torch.bfloat16)
        rot, A = case["rot"], case["axes"]
        s["axes"] = [f % A if case["strided"] else f * A // (rot // 2) for f in range(rot // 2)]
        s["positions"] = torch.cat([_positions(rnd, n, A) for n in new], 1).to(torch.int32).to(dev)
        angle = torch.arange(MAX_POS, device=dev, dtype=torch.float64)[:, None] * \
            1e6 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        part = [b for b in range(B) if new[b] and ctx[b] % page]
        s["part_seq"] = torch.tensor(part, dtype=torch.int64, device=dev)
        s["part_page"] = torch.tensor([ctx[b] // page for b in part], dtype=torch.int64, device=dev)
        # what is read back: every page that the call touched, from its first token
        begin = [c // page * page if n else 0 for n, c in zip(new, ctx)]
        count = [t - b if n else 0 for n, t, b in zip(new, total, begin)]
        back = s["page_table"]
    if op == "evict":
        # many tokens with next to no weight, a few with much, equal ones among them
        w = torch.exp(2.0 * torch.randn(n_pages, Hkv, page, device=dev, generator=g) - 3.0)
        w = torch.where(torch.rand(w.shape, device=dev, generator=g) < 0.3, (w * 64).floor() / 64, w)
        s["weight"] = w
        s["keep_n"], s["new_table"] = i32(keeps), table(rows[B:])
        s["new_n"] = more
        begin, count, back = [0] * B, more, s["new_table"]
    if op in ("append", "evict"):
        s["g_start"], s["g_table"] = i32(begin), back
        out_start = torch.tensor([0] + count, dtype=torch.int64).cumsum(0)
        s["g_out_start"] = out_start.to(torch.int32).to(dev)
        s["g_rows"] = int(out_start[-1])
        gseq = torch.repeat_interleave(torch.arange(B), torch.tensor(count))
        s["g_seq"] = gseq.to(dev)
        s["g_slot"] = (torch.arange(s["g_rows"]) - out_start[:-1][gseq] + torch.tensor(begin)[gseq]).to(dev)
    return s


def _positions(rnd, n, axes):
    """[axes, n]: a turn of text (the same position on every axis) and of images (the first axis stands still, the others run over
    the image's rows and columns), after a past of any length."""
    at, parts, left = rnd.randint(0, MAX_POS // 2), [], n
    while left:
        if axes > 1 and rnd.random() < 0.5:
            h, w = rnd.randint(1, 40), rnd.randint(1, 40)
            grid = [torch.full((h * w,), at), at + torch.arange(h).repeat_interleave(w), at + torch.arange(w).repeat(h), torch.full((h * w,), at)]
            part, step = torch.stack((grid if axes != 2 else grid[1:3])[:axes]), max(h, w)
        else:
            step = rnd.randint(1, 600)
            part = (at + torch.arange(step)).expand(axes, -1)
        parts.append(part[:, :left])
        left -= parts[-1].shape[1]
        at += step
    return torch.cat(parts, 1).clamp(max=MAX_POS - 1) if parts else torch.zeros(axes, 0, dtype=torch.int64)


def _exponent(amax):
    """max(-64, ceil(log2(amax / 448))), exactly: amax = m 2^x with m in [0.5, 1), and 448 = 0.875 * 2^9."""
    m, x = torch.frexp(amax)
    e = (x - 9 + (m > 0.875)).float()
    return torch.where(amax > 0, e, -64.0).clamp(min=-64)


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import moe_expert_layer_fwd_gb300 as moe
    c, keep, op = s["case"], s["keep"], s["case"]["op"]
    cache = moe.KVCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    if op == "shared":
        prefix = (s["prefix_start"], s["prefix_len"], s["prefix_table"], s["max_prefix_q"])
        if "ws" not in keep:
            keep["ws"] = moe.moe_paged_attention_shared_workspace(s["T"], c["B"], c["Hq"], c["Hkv"], D, s["max_q"], c["groups"],
                                                                  s["max_prefix_q"], s["q"].device)
        out, lse = moe.moe_paged_attention_shared(s["q"], cache, s["q_start"], s["kv_len"], s["page_table"], max_q=s["max_q"],
                                                  prefix=prefix, ws=keep["ws"])
        return {"out": out, "lse": lse}
    if op == "weights":
        if "ws" not in keep:
            keep["ws"] = moe.moe_kv_workspace(s["q"].device)
        w = moe.moe_kv_weights(s["q"], s["lse"], cache, s["q_start"], s["kv_len"], s["page_table"], max_q=s["max_q"],
                               weight=None if c["fresh"] else s["weight"], out=s["weight_out"], window=c["window"], ws=keep["ws"])
        return {"weight": w}
    if op == "evict":
        if "ws" not in keep:
            keep["ws"] = moe.moe_kv_workspace(s["weight"].device)
        n, kept = moe.moe_kv_evict(cache, s["weight"], s["kv_len"], s["page_table"], s["keep_n"], s["new_table"], sink=c["sink"],
                                   recent=c["recent"], ws=keep["ws"])
        out = {"len": n, "kept": kept, "weight": s["weight"]}
    else:
        if "ws" not in keep:
            keep["ws"] = moe.moe_kv_workspace(s["qkv"].device)
        q, k, v = s["qkv"].view(s["T"], -1, D).split([c["Hq"], c["Hkv"], c["Hkv"]], dim=1)
        rows = moe.moe_rope_rows(s["positions"], s["axes"], s["cos_sin"], ws=keep["ws"])
        out = {"q": moe.moe_kv_append_at(q, k, v, cache, s["q_start"], s["kv_len"], s["page_table"], rows, interleaved=c["interleaved"],
                                         q_norm_weight=s.get("q_norm"), k_norm_weight=s.get("k_norm"), eps=1e-6, ws=keep["ws"])}
    out["k"], out["v"] = moe.moe_kv_gather(cache, s["g_start"], s["g_out_start"], s["g_table"], s["g_rows"], ws=keep["ws"])
    return out


def _run_plain(s):
    op = s["case"]["op"]
    if op == "shared":
        return _shared_attention(s)
    if op == "weights":
        return {"weight": _weights_plain(s)}
    out = _evict_plain(s) if op == "evict" else {"q": _append_plain(s)}
    out["k"], out["v"] = _gather(s)
    return out


def _values(codes, scale):
    return codes.view(torch.float8_e4m3fn).float() * torch.exp2(scale.float() - 127)[..., None]


def _gather(s):
    page = s["case"]["page"]
    pages, slot = s["g_table"][s["g_seq"], s["g_slot"] // page].long(), s["g_slot"] % page
    return tuple(_values(s[n + "_codes"][pages, :, slot], s[n + "_scale"][pages]).to(torch.bfloat16) for n in "kv")


def _norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()


def _rotate(x, cos, sin, rot, interleaved):
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = (a * cos - b * sin, a * sin + b * cos)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat([y, x[..., rot:]], -1)


def _append_plain(s):
    c = s["case"]
    page, Hkv, rot = c["page"], c["Hkv"], c["rot"]
    q, k, v = s["qkv"].view(s["T"], -1, D).float().split([c["Hq"], Hkv, Hkv], dim=1)
    if c["norm"]:
        q, k = _norm(q, s["q_norm"]), _norm(k, s["k_norm"])
    axes = torch.tensor(s["axes"], device=q.device)
    at = s["positions"].long()[axes].T                               # [T, rot / 2]
    f = torch.arange(rot // 2, device=q.device)
    cos, sin = s["cos_sin"][at, f][:, None], s["cos_sin"][at, rot // 2 + f][:, None]
    q, k = _rotate(q, cos, sin, rot, c["interleaved"]), _rotate(k, cos, sin, rot, c["interleaved"])
    pages = s["page_table"][s["seq"], s["slot"] // page].long()      # page of each new token
    slot = s["slot"] % page
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


def _padded(s, name, table, length):
    """Cached rows [B, Hkv, S, D] of the sequences of a page table, zeros behind their ends, and which are there [B, S]."""
    pages = table[:, :-1].long().clamp(min=0)
    B, S = pages.shape[0], pages.shape[1] * s["case"]["page"]
    there = torch.arange(S, device=pages.device) < length[:, None]
    x = _values(s[name + "_codes"][pages], s[name + "_scale"][pages][..., None])
    return x.transpose(1, 2).reshape(B, -1, S, D).masked_fill_(~there[:, None, :, None], 0.0), there


def _own_scores(s, window=0):
    """Scores [B, Hkv, G, Tq, S] of the new queries, padded to the longest sequence's, against their sequence's own keys; -inf
    where a key is not seen.  And the padded query of each token."""
    c = s["case"]
    B, Hq, Hkv, Tq = c["B"], c["Hq"], c["Hkv"], s["max_q"]
    G = Hq // Hkv
    k, there = _padded(s, "k", s["page_table"], s["kv_len"])
    S = k.shape[2]
    i, j = torch.arange(Tq, device=k.device), torch.arange(S, device=k.device)
    n_new = s["q_start"][1:] - s["q_start"][:-1]
    token = (s["q_start"][:-1, None] + i).long().clamp(max=s["T"] - 1)
    q = s["q"].float()[token].view(B, Tq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Tq, D)
    z = torch.matmul(q * D ** -0.5, k.transpose(-1, -2)).view(B, Hkv, G, Tq, S)
    pos = (s["kv_len"] - n_new)[:, None] + i
    seen = there[:, None, :] & (j <= pos[..., None])
    if window:
        seen = seen & (j > pos[..., None] - window)
    z.masked_fill_(~seen[:, None, None], -math.inf)
    return z, torch.arange(s["T"], device=k.device) - s["q_start"][s["seq"]]


def _shared_attention(s):
    c = s["case"]
    B, Hq, Hkv, Tq, T = c["B"], c["Hq"], c["Hkv"], s["max_q"], s["T"]
    G = Hq // Hkv
    z, i = _own_scores(s)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = z.sub_(top).exp_()
    o = torch.matmul(p.view(B, Hkv, G * Tq, -1), _padded(s, "v", s["page_table"], s["kv_len"])[0]).view(B, Hkv, G, Tq, D)
    pick = lambda x: x[s["seq"], :, :, i]                             # [T, Hkv, G, ...]
    o, total, top = pick(o), pick(p.sum(-1)), pick(top.squeeze(-1))
    # the prefixes, each once for all tokens of its group
    at = 0
    for g, (n, length) in enumerate(zip(s["tokens"], s["prefix"])):
        if n and length:
            rows = slice(at, at + n)
            pages = s["prefix_table"][g, :-(-length // c["page"])].long()
            k, v = (_values(s[x + "_codes"][pages], s[x + "_scale"][pages][..., None]).transpose(0, 1).reshape(Hkv, -1, D)[:, :length]
                    for x in "kv")
            q = s["q"][rows].float().view(n, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * n, D)
            z = torch.matmul(q * D ** -0.5, k.transpose(-1, -2))
            m = z.amax(-1, keepdim=True)
            p = z.sub_(m).exp_()
            back = lambda x: x.view(Hkv, G, n, -1).permute(2, 0, 1, 3)
            o1, t1, m1 = back(torch.matmul(p, v)), back(p.sum(-1, keepdim=True))[..., 0], back(m)[..., 0]
            ref = torch.where(total[rows] > 0, torch.maximum(top[rows], m1), m1)
            f, f1 = torch.exp(top[rows] - ref) * (total[rows] > 0), torch.exp(m1 - ref)
            o[rows] = o[rows] * f[..., None] + o1 * f1[..., None]
            total[rows] = total[rows] * f + t1 * f1
            top[rows] = ref
        at += n
    out = o / torch.where(total > 0, total, 1.0)[..., None]
    lse = torch.where(total > 0, top + total.log(), -math.inf)
    return {"out": out.reshape(T, Hq, D).to(torch.bfloat16), "lse": lse.reshape(T, Hq)}


def _weights_plain(s):
    c = s["case"]
    B, Hkv, page = c["B"], c["Hkv"], c["page"]
    z, i = _own_scores(s, c["window"])
    lse = torch.full(z.shape[:-1], math.inf, device=z.device)
    lse[s["seq"], :, :, i] = s["lse"].view(s["T"], Hkv, -1)
    add = torch.exp(z.sub_(lse[..., None])).sum((2, 3))               # [B, Hkv, S]
    n_new = (s["q_start"][1:] - s["q_start"][:-1])[:, None]
    slot = torch.arange(add.shape[-1], device=add.device)
    first = s["kv_len"][:, None] - n_new
    # tokens that some query sees, or that are new; the others keep what they have
    lo = (first - c["window"] + 1).clamp(min=0) if c["window"] else torch.zeros_like(first)
    touched = (slot < s["kv_len"][:, None]) & (slot >= lo) & (n_new > 0)
    b, j = touched.nonzero(as_tuple=True)
    pages = s["page_table"][b, j // page].long()
    old = s["weight"][pages, :, j % page] * (j < first[b, 0])[:, None]
    s["weight_out"][pages, :, j % page] = add[b, :, j] + (0.0 if c["fresh"] else old)
    return s["weight_out"]


def _evict_plain(s):
    c = s["case"]
    B, Hkv, page = c["B"], c["Hkv"], c["page"]
    pages = s["page_table"].long().clamp(min=0)
    w = s["weight"][pages].transpose(1, 2).reshape(B, Hkv, -1)       # [B, Hkv, S]
    S = w.shape[-1]
    j = torch.arange(S, device=w.device)
    n = s["kv_len"][:, None, None]
    rank = w.masked_fill((j < c["sink"]) | (j >= n - c["recent"]), math.inf).masked_fill(j >= n, -1.0)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    count = torch.minimum(s["keep_n"], s["kv_len"])
    width = s["new_table"].shape[1] * page
    chosen = order[..., :width].masked_fill(torch.arange(min(width, S), device=w.device) >= count[:, None, None], S)
    kept = torch.sort(chosen, -1).values                              # tokens in their order, then S
    if kept.shape[-1] < width:
        kept = torch.cat([kept, kept.new_full((B, Hkv, width - kept.shape[-1]), S)], -1)
    b, h, i = (kept < S).nonzero(as_tuple=True)
    tok = kept[b, h, i]
    src, dst = pages[b, tok // page], s["new_table"][b, i // page].long()
    s["weight"][dst, h, i % page] = s["weight"][src, h, tok % page]
    for name in "kv":
        codes, scale = s[name + "_codes"], s[name + "_scale"]
        old = scale[src, h].float() - 127
        e = torch.full(scale.shape, -math.inf, device=w.device).view(-1)
        e = e.scatter_reduce_(0, dst * Hkv + h, old, "amax").view(scale.shape)
        x = codes[src, h, tok % page].view(torch.float8_e4m3fn).float() * torch.exp2(old - e[dst, h])[:, None]
        codes[dst, h, i % page] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        scale[dst, h] = (e[dst, h] + 127).to(torch.uint8)
    return {"len": count, "kept": kept.masked_fill(kept == S, -1).to(torch.int32), "weight": s["weight"]}


# ------------------------------------------------------------------------------------------------ costs
def _visible(case):
    """Over the sequences: query-key pairs that the masks leave among their own tokens, and keys that some query sees."""
    pairs = keys = 0
    for n, c in zip(*_lengths(case)[:2]):
        if not n:
            continue
        w = case.get("window") or c + n
        keys += min(c + n, w + n - 1)
        full = max(0, min(n, w - c))          # queries that see everything before them
        pairs += full * c + full * (full + 1) // 2 + (n - full) * w
    return pairs, keys


def work(case):
    lengths = _lengths(case)
    new, ctx = lengths[:2]
    T, Hq, Hkv, page = sum(new), case["Hq"], case["Hkv"], case["page"]
    if case["op"] == "append":
        back = sum(n + c - c // page * page for n, c in zip(new, ctx) if n)
        turn = T * (case["rot"] * 4 + case["axes"] * 4)
        return {"bytes": T * (4 * Hq + 4 * Hkv + 2 * Hkv) * D + turn + 6 * back * Hkv * D, "flops": 8 * T * (Hq + 2 * Hkv) * D}
    if case["op"] == "evict":
        kept = sum(min(a, b) for a, b in zip(lengths[2], ctx))
        return {"bytes": 4 + Hkv * (sum(ctx) * 4 + kept * (8 + 4 * D + 6 * D)), "flops": Hkv * (sum(ctx) + 4 * kept * D)}
    pairs, keys = _visible(case)
    if case["op"] == "weights":
        return {"bytes": keys * Hkv * (D + (4 if case["fresh"] else 8)) + T * Hq * (2 * D + 4), "flops": 2 * pairs * Hq * D}
    at = 0
    for m, length in zip(*lengths[2:]):
        n = sum(new[at:at + m])
        at += m
        pairs, keys = pairs + n * length, keys + (length if n else 0)
    return {"bytes": 2 * keys * Hkv * D + T * Hq * (4 * D + 4), "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _e4m3(x):
    """The nearest E4M3 value, ties to even: 3 fraction bits down to 2^-6, then multiples of 2^-9."""
    _, ex = torch.frexp(x.abs())
    step = torch.exp2((ex - 4).clamp(min=-9).double())
    return (torch.round(x / step) * step).clamp(-448, 448)


def _cached(s, name, table, lo, hi):
    """Tokens [lo, hi) of a row of a page table, [Hkv, hi - lo, D] in 64 bits."""
    page = s["case"]["page"]
    at = table[lo // page:-(-hi // page)].long()
    x = s[name + "_codes"][at].view(torch.float8_e4m3fn).double() * torch.exp2(s[name + "_scale"][at].double() - 127)[:, :, None, None]
    return x.transpose(0, 1).flatten(1, 2)[:, lo - lo // page * page:][:, :hi - lo]


def _scores(s, new):
    """(sequence, scores [Hkv, G, n, keys] in 64 bits, -inf where unseen) of each sequence with new tokens, over its own keys."""
    c, at = s["case"], 0
    ctx = _lengths(c)[1]
    for b, n in enumerate(new):
        if n:
            k = _cached(s, "k", s["page_table"][b], 0, ctx[b] + n)
            q = s["q"][at:at + n].double().view(n, c["Hkv"], -1, D)
            z = torch.einsum("ihgd,hjd->hgij", q, k) / math.sqrt(D)
            j, here = torch.arange(ctx[b] + n, device=k.device), ctx[b] + torch.arange(n, device=k.device)[:, None]
            no = j > here
            if c.get("window"):
                no = no | (j <= here - c["window"])
            yield b, z.masked_fill_(no, -math.inf)
        at += n


def exact(case, seed):
    s = prepare(case, seed)
    op, page, Hq, Hkv = case["op"], case["page"], case["Hq"], case["Hkv"]
    lengths = _lengths(case)
    new, ctx = lengths[:2]
    if op == "weights":
        out = s["weight"].double()
        at = 0
        for b, z in _scores(s, new):
            n, first = new[b], ctx[b]
            at = sum(new[:b])
            lse = s["lse"][at:at + n].double().view(n, Hkv, -1).permute(1, 2, 0)
            add = torch.exp(z - lse[..., None]).sum((1, 2))           # [Hkv, keys]
            for j in range(max(0, first - case["window"] + 1) // page * page if case["window"] else 0, first + n, page):
                lo, hi = max(j, first - case["window"] + 1 if case["window"] else 0), min(j + page, first + n)
                p = int(s["page_table"][b, j // page])
                old = torch.zeros_like(out[p, :, lo - j:hi - j])
                if not case["fresh"] and lo < first:
                    old[:, :first - lo] = out[p, :, lo - j:min(hi, first) - j]
                out[p, :, lo - j:hi - j] = old + add[:, lo:hi]
        return {"weight": out}

    if op == "shared":
        outs, lses, at, b = [], [], 0, 0
        group = [g for g, m in enumerate(lengths[2]) for _ in range(m)]
        for b, z in _scores(s, new):
            n, g = new[b], group[b]
            at = sum(new[:b])
            v = _cached(s, "v", s["page_table"][b], 0, ctx[b] + n)
            length = lengths[3][g]
            if length:
                k1, v1 = (_cached(s, x, s["prefix_table"][g], 0, length) for x in "kv")
                q = s["q"][at:at + n].double().view(n, Hkv, -1, D)
                z = torch.cat([torch.einsum("ihgd,hjd->hgij", q, k1) / math.sqrt(D), z], -1)
                v = torch.cat([v1, v], 1)
            outs.append(torch.einsum("hgij,hjd->ihgd", torch.softmax(z, -1), v).reshape(n, Hq, D))
            lses.append(torch.logsumexp(z, -1).permute(2, 0, 1).reshape(n, Hq))
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}

    if op == "evict":
        width = s["new_table"].shape[1] * page
        kept = torch.full((case["B"], Hkv, width), -1, dtype=torch.int32)
        weight, ks, vs = s["weight"].double(), [], []
        source = s["weight"].cpu()
        table, new_table = s["page_table"].cpu(), s["new_table"].cpu()
        for b, n in enumerate(ctx):
            m = min(lengths[2][b], n)
            at = table[b, :-(-n // page)].long()
            w = source[at].transpose(0, 1).flatten(1)[:, :n].double()
            w[:, :case["sink"]] = math.inf
            w[:, max(0, n - case["recent"]):] = math.inf
            got = {x: torch.zeros(m, Hkv, D, dtype=torch.float64, device="cuda") for x in "kv"}
            for h in range(Hkv):
                value = w[h].tolist()
                tok = sorted(sorted(range(n), key=lambda j: (-value[j], j))[:m])
                kept[b, h, :m] = torch.tensor(tok, dtype=torch.int32)
                t = torch.tensor(tok, dtype=torch.int64)
                src, i = at[t // page], torch.arange(m)
                dst = new_table[b, i // page].long()
                weight[dst, h, i % page] = source[src, h, t % page].double().to(weight.device)
                for x in "kv":
                    e = s[x + "_scale"][src, h].double() - 127
                    tops = torch.stack([part.max() for part in e.split(page)])[i // page] if m else e
                    raw = s[x + "_codes"][src, h, t % page].view(torch.float8_e4m3fn).double()
                    got[x][:, h] = _e4m3(raw * torch.exp2(e - tops)[:, None]) * torch.exp2(tops)[:, None]
            ks.append(got["k"])
            vs.append(got["v"])
        return {"len": torch.tensor([min(a, b) for a, b in zip(lengths[2], ctx)], dtype=torch.int32), "kept": kept, "weight": weight,
                "k": torch.cat(ks), "v": torch.cat(vs)}

    rot = case["rot"]
    qs, ks, vs, at = [], [], [], 0
    f = 1e6 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    for b, (t, c) in enumerate(zip(new, ctx)):
        if not t:
            continue
        q, k, v = s["qkv"][at:at + t].double().view(t, -1, D).split([Hq, Hkv, Hkv], dim=1)
        if case["norm"]:
            q = q / torch.sqrt(q.square().mean(-1, keepdim=True) + 1e-6) * s["q_norm"].double()
            k = k / torch.sqrt(k.square().mean(-1, keepdim=True) + 1e-6) * s["k_norm"].double()
        angle = torch.stack([s["positions"][a, at:at + t].double() * f[i] for i, a in enumerate(s["axes"])], 1)
        # the table holds cosines and sines in fp32
        turn = torch.complex(angle.cos().float().double(), angle.sin().float().double())[:, None]
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
            before = _cached(s, name, s["page_table"][b], first, c).transpose(0, 1) if c > first else x[:0]
            for p in range(first, c + t, page):                       # page by page
                lo, hi = max(p, c), min(p + page, c + t)
                y = x[lo - c:hi - c]
                a = y.abs().amax((0, 2))
                m, ex = torch.frexp(a)
                e = torch.where(a > 0, (ex - 9 + (m > 0.875)).double(), -64.0).clamp(min=-64)
                if p < c:
                    e = torch.maximum(e, s[name + "_scale"][s["page_table"][b, p // page].long()].double() - 127)
                    to.append(_e4m3(before / torch.exp2(e)[:, None]) * torch.exp2(e)[:, None])
                to.append(_e4m3(y / torch.exp2(e)[:, None]) * torch.exp2(e)[:, None])
        at += t
    return {"q": torch.cat(qs), "k": torch.cat(ks), "v": torch.cat(vs)}
