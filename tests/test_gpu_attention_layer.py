"""AttentionLayer against the float64 oracle, its arguments, its workspaces and their status words (GPU)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

from test_gpu_attention import D, bf16, env, f64  # noqa: E402,F401
from oracle import attention as oa  # noqa: E402

HQ, HKV, PAGE = 8, 2, 16


def i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kw", [
    dict(), dict(window=25, interleaved=True, rot_dim=64, scale=0.05, norms=True), dict(window=7, rot_dim=32, rope_base=500.0),
    dict(rot_dim=0, scale=0.2, norms=True, eps=0.5), dict(interleaved=True, rope_base=1e4, norms=True)])
def test_layer_against_the_oracle(env, kw):  # noqa: F811
    """Prompts, single tokens and chunks in turn.  Queries and cached keys are compared with rotations in 64 bits that know nothing of
    the layer, its outputs with the oracle's attention over the cache that it left.  Tolerances: queries are rounded once to bf16; a
    cached number is rounded to E4M3 (2^-4 of it, 2^-10 of the page's scale at least) and once more, to smaller numbers' absolute
    steps, whenever the page's scale grows: 2^-10 (1 + 1/2 + 1/4 ..) of the last scale."""
    moe, torch = env
    rng = np.random.default_rng(len(kw))
    args = dict(kw)
    norms = [bf16(rng, D).cuda(), bf16(rng, D).cuda()] if args.pop("norms", False) else [None, None]
    layer = moe.AttentionLayer(16, HQ, HKV, page=PAGE, max_pos=128, q_norm_weight=norms[0], k_norm_weight=norms[1], **args)
    rot, il, base, eps = args.get("rot_dim", D), args.get("interleaved", False), args.get("rope_base", 1e6), args.get("eps", 1e-6)
    angles = oa.rope_table(128, rot, base) if rot else np.zeros((128, 0))
    weights = [None if w is None else f64(w) for w in norms]
    table = rng.permutation(16).reshape(2, 8).astype(np.int32)
    d_table = torch.from_numpy(table).cuda()
    other = moe.KVCache.empty(16, HKV, PAGE)          # the same tokens by moe_kv_append alone, for its queries
    keys = [np.zeros((0, HKV, D))] * 2
    lens = [0, 0]
    for new in ([50, 13], [1, 1], [5, 2], [0, 1], [40, 60]):
        T = sum(new)
        first, lens = list(lens), [a + n for a, n in zip(lens, new)]
        starts = np.cumsum([0] + new).astype(np.int32)
        pos = np.concatenate([np.arange(a, a + n) for a, n in zip(first, new)])
        x = bf16(rng, T, HQ + 2 * HKV, D, mul=2.0)
        out = layer.forward(x.view(T, -1).cuda(), i32(starts), i32(lens), d_table, max(new))
        assert layer.status() == moe.MOE_OK and out.shape == (T, HQ * D)
        q, k, v = x.cuda().split([HQ, HKV, HKV], dim=1)
        cos_sin = torch.from_numpy(angles.astype(np.float32)).cuda() if rot else None
        rq = moe.moe_kv_append(q, k, v, other, i32(starts), i32(lens), d_table, cos_sin, interleaved=il, q_norm_weight=norms[0],
                               k_norm_weight=norms[1], eps=eps)
        turned = [oa.norm_rotate(f64(x)[:, a:b], pos, angles, rot, il, w, eps)
                  for a, b, w in ((0, HQ, weights[0]), (HQ, HQ + HKV, weights[1]))]
        size = np.abs(turned[0]).max(-1, keepdims=True)
        assert (np.abs(f64(rq) - turned[0]) <= 2.0 ** -8 * np.abs(turned[0]) + 2.0 ** -18 * size).all()
        host = {n: getattr(layer.cache, n).cpu().numpy() for n in ("k_codes", "v_codes", "k_scale", "v_scale")}
        for b in range(2):
            keys[b] = np.concatenate([keys[b], turned[1][starts[b]:starts[b + 1]]])
            got = oa.read(host, "k", b, 0, lens[b], table)
            unit = 2.0 ** (host["k_scale"][table[b, np.arange(lens[b]) // PAGE]].astype(int) - 127)[..., None]
            size = np.abs(keys[b]).max(-1, keepdims=True)
            assert (np.abs(got - keys[b]) <= 2.0 ** -4 * np.abs(keys[b]) + 2.0 ** -9 * unit + 2.0 ** -18 * size).all()
        ref, spread = oa.attention(f64(rq), host, starts, lens, table, args.get("scale", D ** -0.5), True, args.get("window", 0))
        assert (np.abs(f64(out).reshape(T, HQ, D) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * spread).all()


def test_more_than_all_tokens_as_the_most(env):  # noqa: F811
    """max_q is an upper bound: a program that knows only that no sequence brings more than 40 tokens gives 40, also with 3."""
    moe, torch = env
    rng = np.random.default_rng(1)
    layers = [moe.AttentionLayer(16, HQ, HKV, page=PAGE, max_pos=128) for _ in range(2)]
    table = torch.from_numpy(rng.permutation(16).reshape(2, 8).astype(np.int32)).cuda()
    lens = [0, 0]
    for new in ([20, 9], [2, 1], [0, 1]):
        lens = [a + n for a, n in zip(lens, new)]
        x = bf16(rng, sum(new), (HQ + 2 * HKV) * D).cuda()
        args = x, i32([0, new[0], sum(new)]), i32(lens), table
        assert torch.equal(layers[0].forward(*args, sum(new)), layers[1].forward(*args, 400 if lens[0] > 20 else 40))
    q = bf16(rng, 1, HQ, D).cuda()
    call = lambda m: moe.moe_paged_attention(q, layers[0].cache, i32([0, 0, 1]), i32(lens), table, max_q=m)
    assert torch.equal(call(1), call(7))


@pytest.mark.parametrize("kw", [dict(max_q=0), dict(max_q=-1), dict(max_q=2), dict(out=(5, 3)), dict(out=(5, HQ * D), dtype="float32")])
def test_refused_calls_leave_the_cache_alone(env, kw):  # noqa: F811
    """What the attention refuses, the layer refuses before it appends.  (5 tokens of 2 sequences: one of them brings 3.)"""
    moe, torch = env
    rng = np.random.default_rng(2)
    layer = moe.AttentionLayer(16, HQ, HKV, page=PAGE, max_pos=128)
    for t in layer.cache:
        t.fill_(3)
    before = [t.clone() for t in layer.cache]
    table = torch.from_numpy(rng.permutation(16).reshape(2, 8).astype(np.int32)).cuda()
    out = torch.empty(kw["out"], dtype=getattr(torch, kw.get("dtype", "bfloat16")), device="cuda") if "out" in kw else None
    with pytest.raises((ValueError, moe.MoEError)):
        layer.forward(bf16(rng, 5, (HQ + 2 * HKV) * D).cuda(), i32([0, 2, 5]), i32([2, 3]), table, kw.get("max_q", 3), out=out)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, layer.cache))


def test_layer_arguments_are_checked(env):  # noqa: F811
    moe, torch = env
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(window=-1)):
        with pytest.raises(ValueError):
            moe.AttentionLayer(4, HQ, HKV, **kw)


def capture(torch, f):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f()
    return g, out


def test_status_of_a_graph_whose_workspace_was_outgrown(env):  # noqa: F811
    """A decode graph goes on using the workspace that it was captured with: what it reports there reaches layer.status()."""
    moe, torch = env
    rng = np.random.default_rng(3)
    layer = moe.AttentionLayer(40, HQ, HKV, page=PAGE, max_pos=1024)
    table = torch.from_numpy(rng.permutation(40).reshape(1, 40).astype(np.int32)).cuda()
    start, lens, x = i32([0, 1]), i32([1]), bf16(rng, 1, (HQ + 2 * HKV) * D).cuda()
    layer.forward(x, start, lens, table, 1)
    g, _ = capture(torch, lambda: layer.forward(x, start, lens, table, 1))
    layer.forward(bf16(rng, 300, (HQ + 2 * HKV) * D).cuda(), i32([0, 300]), i32([300]), table, 300)
    lens.fill_(301)
    g.replay()
    assert layer.status() == moe.MOE_OK
    table[0, 4] = 1 << 20
    g.replay()
    assert layer.status() == moe.MOE_ERR_DEVICE_CHECK
    layer.clear_status()
    assert layer.status() == moe.MOE_OK


def test_first_call_inside_a_capture(env):  # noqa: F811
    """A graph captured before any other call: right, and what its replays report stays, as the eager calls' around them does."""
    moe, torch = env
    rng = np.random.default_rng(4)
    layers = [moe.AttentionLayer(40, HQ, HKV, page=PAGE, max_pos=1024) for _ in range(2)]
    table = torch.from_numpy(rng.permutation(40).reshape(1, 40).astype(np.int32)).cuda()
    start, lens, x = i32([0, 1]), i32([1]), bf16(rng, 1, (HQ + 2 * HKV) * D).cuda()
    junk = [torch.full((8 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    del junk
    g, out = capture(torch, lambda: layers[0].forward(x, start, lens, table, 1))
    assert layers[0].status() == moe.MOE_OK
    g.replay()
    assert torch.equal(out, layers[1].forward(x, start, lens, table, 1)) and layers[0].status() == moe.MOE_OK
    prompt = bf16(rng, 300, (HQ + 2 * HKV) * D).cuda(), i32([0, 300]), i32([301]), table, 300
    assert torch.equal(layers[0].forward(*prompt), layers[1].forward(*prompt)) and layers[0].status() == moe.MOE_OK
    lens.fill_(302)
    good = int(table[0, 4])
    table[0, 4] = 1 << 20
    g.replay()
    table[0, 4] = good
    g.replay()
    assert layers[0].status() == moe.MOE_ERR_DEVICE_CHECK
    layers[1].forward(x, start, lens, table, 1)
    assert torch.equal(out, layers[1].forward(x, start, lens, table, 1))


def test_strides_of_a_single_token(env):  # noqa: F811
    """One token's rows have no stride: any will do."""
    moe, torch = env
    rng = np.random.default_rng(5)
    cache = moe.KVCache.empty(4, HKV, PAGE)
    table = i32([[2, 0]])
    q, k = bf16(rng, 1, HQ, D).cuda(), bf16(rng, 1, HKV, D).cuda()
    odd = lambda t: torch.as_strided(t, t.shape, (10001, D, 1))
    plain = moe.moe_kv_append(q, k, k, cache, i32([0, 1]), i32([1]), table)
    assert torch.equal(moe.moe_kv_append(odd(q), odd(k), odd(k), cache, i32([0, 1]), i32([1]), table), plain)
    one = moe.moe_paged_attention(plain, cache, i32([0, 1]), i32([1]), table, max_q=1)
    assert torch.equal(moe.moe_paged_attention(odd(plain), cache, i32([0, 1]), i32([1]), table, max_q=1), one)
