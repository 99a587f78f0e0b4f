"""The measured cases of rotary positions with several axes, windowed attention with sinks, and an e4m3 cache with block scales.

Four operators of one attention layer of a serving step over a paged cache:

turn   the step's queries and new keys are rotated to positions with several axes (time, height, width), keys and
       values written into the cache (bf16, or e4m3 codes of value / scale). Outputs: the rotated queries, both caches.
sinks  attention with a sliding window in which the first tokens of each sequence stay visible. Output: bf16 rows.
fill   the step's new keys (rotated, or as they are) and values are written into an e4m3 cache with a scale for each
       block of tokens (a page) and KV head. A block without earlier tokens takes the least power of two that brings
       its largest magnitude to 448 or below; one with earlier tokens keeps its scale, or doubles it (and divides the
       earlier codes) as often as the new tokens need. Outputs: both caches' codes, their scales, the rotated queries.
read   attention over such a cache, decoding and in chunks of prompts. Output: bf16 rows.

A case's sequence lengths come from the case alone ("lens" seeds them), the values, the page order and the
weights of the cache from the seed of `prepare`.
"""
import math
import random

import torch

own = False

BLOCK_GAP = 3  # physical blocks beyond the ones in use
LEAST, MOST = 2.0 ** -100, 2.0 ** 100  # block scales that an append makes

# ---------------------------------------------------------------- cases


def listed():
    turn = dict(op="turn", window=0, sinks=0, power=True)
    sinks = dict(op="sinks", axes=1, cycle=False, rot=0, interleaved=False, fused=False, fp8=False, power=True)
    fill = dict(op="fill", axes=1, cycle=False, window=0, sinks=0, fp8=True, power=True)
    read = dict(op="read", axes=1, cycle=False, rot=0, interleaved=False, fused=False, fp8=True)
    return [
        # one user's next token after text and images: launch latency
        turn | dict(name="axes_one_token", seqs=1, q_lo=1, q_hi=1, ctx_lo=8191, ctx_hi=8191, hq=32, hkv=8, d=128, bs=16,
                    fp8=False, lens=21, rot=128, axes=3, cycle=False, interleaved=False, fused=False),
        # images and text in chunks of odd sizes, rows of a fused projection, e4m3 cache, the axes taking turns over the pairs
        turn | dict(name="axes_chunks_fp8", seqs=9, q_lo=100, q_hi=1500, ctx_lo=0, ctx_hi=3000, hq=24, hkv=4, d=96, bs=32,
                    fp8=True, lens=22, rot=96, axes=3, cycle=True, interleaved=True, fused=True),
        # whole prompts of video frames
        turn | dict(name="axes_prompts", seqs=4, q_lo=4096, q_hi=4096, ctx_lo=0, ctx_hi=0, hq=32, hkv=32, d=128, bs=16,
                    fp8=False, lens=23, rot=128, axes=3, cycle=False, interleaved=False, fused=True),
        # one user's next token in a session without end: latency
        sinks | dict(name="sinks_one_token", seqs=1, q_lo=1, q_hi=1, ctx_lo=131071, ctx_hi=131071, hq=32, hkv=8, d=128,
                     bs=16, lens=24, window=1024, sinks=4),
        # a batch of decoding users with long sessions
        sinks | dict(name="sinks_decode", seqs=64, q_lo=1, q_hi=1, ctx_lo=2000, ctx_hi=16000, hq=32, hkv=8, d=128, bs=16,
                     lens=25, window=4096, sinks=4),
        # whole prompts under a window
        sinks | dict(name="sinks_prompts", seqs=4, q_lo=4096, q_hi=4096, ctx_lo=0, ctx_hi=0, hq=32, hkv=8, d=128, bs=16,
                     lens=26, window=1024, sinks=64),
        # decoding users: one new token each, in blocks that hold earlier ones
        fill | dict(name="fill_decode", seqs=64, q_lo=1, q_hi=1, ctx_lo=512, ctx_hi=16000, hq=64, hkv=8, d=128, bs=16,
                    lens=27, rot=128, interleaved=False, fused=True),
        # chunks of odd sizes into larger blocks, keys as they are
        fill | dict(name="fill_chunks", seqs=9, q_lo=100, q_hi=700, ctx_lo=0, ctx_hi=2000, hq=24, hkv=4, d=96, bs=64,
                    lens=28, rot=0, interleaved=False, fused=False),
        # whole prompts
        fill | dict(name="fill_prompts", seqs=4, q_lo=4096, q_hi=4096, ctx_lo=0, ctx_hi=0, hq=32, hkv=8, d=128, bs=16,
                    lens=29, rot=128, interleaved=False, fused=True),
        # a batch of decoding users, ragged lengths
        read | dict(name="read_decode", seqs=64, q_lo=1, q_hi=1, ctx_lo=511, ctx_hi=8191, hq=32, hkv=8, d=128, bs=16,
                    lens=30, window=0, sinks=0, power=True),
        # few users with very long contexts, scales of any value
        read | dict(name="read_decode_long", seqs=8, q_lo=1, q_hi=1, ctx_lo=131071, ctx_hi=131071, hq=64, hkv=8, d=128,
                    bs=16, lens=31, window=0, sinks=0, power=False),
        # chunks of prompts over earlier tokens, with a window and sinks
        read | dict(name="read_chunks", seqs=5, q_lo=300, q_hi=1100, ctx_lo=100, ctx_hi=2500, hq=32, hkv=8, d=128, bs=16,
                    lens=32, window=1000, sinks=4, power=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hkv, qpk = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 3, 4, 8])
    d = 32 * rng.randint(1, 8)
    case = dict(op=rng.choice(["turn", "sinks", "fill", "read"]), hq=hkv * qpk, hkv=hkv, d=d,
                bs=rng.choice([16, 32, 64, 128, 256]), lens=rng.randrange(1 << 20), window=0, sinks=0, axes=1, cycle=False,
                rot=0, interleaved=False, fused=False, fp8=True, power=rng.random() < 0.5)
    if case["op"] in ("turn", "fill"):
        tokens = _log(rng, 1, 16384)
        case["seqs"] = min(tokens, _log(rng, 1, 128))
        case["q_hi"] = max(1, tokens // case["seqs"])
        case["ctx_hi"] = _log(rng, 1, max(2, min(100000, 200000 // case["seqs"])))
        case |= dict(interleaved=rng.random() < 0.5, rot=2 * rng.randint(1, d // 2) if rng.random() < 0.4 else d,
                     fused=rng.random() < 0.5)
        if case["op"] == "turn":
            case |= dict(axes=rng.randint(2, 4), cycle=rng.random() < 0.5, fp8=rng.random() < 0.4)
        elif rng.random() < 0.4:
            case |= dict(rot=0, fused=False)
    else:
        decode = rng.random() < 0.5
        case["q_hi"] = rng.randint(1, 4) if decode else _log(rng, 5, 2000)
        case["seqs"] = _log(rng, 1, 100 if decode else max(2, min(16, 6000 // case["q_hi"])))
        case["ctx_hi"] = _log(rng, 1, max(2, min(60000, 200000 // case["seqs"])) if decode else 3500)
        if case["op"] == "sinks" or rng.random() < 0.3:
            case |= dict(window=_log(rng, 1, 4000), sinks=_log(rng, 1, 300))
        if case["op"] == "sinks":
            case["fp8"] = rng.random() < 0.3
    case["q_lo"] = rng.choice([1, case["q_hi"]])
    case["ctx_lo"] = rng.choice([0, case["ctx_hi"]])
    return case


def _lengths(case):
    rng = random.Random(case["lens"])
    q = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["seqs"])]
    return q, [n + rng.randint(case["ctx_lo"], case["ctx_hi"]) for n in q]


def _pair_axes(case):
    """The position axis of each pair: in turns, or in runs with a third fewer pairs for the first axis."""
    n, axes = case["rot"] // 2, case["axes"]
    if case["cycle"]:
        return [i % axes for i in range(n)]
    first = n * 2 // (3 * axes)
    return [0 if i < first else min(axes - 1, 1 + (i - first) * (axes - 1) // max(1, n - first)) for i in range(n)]


def _frequencies(case):
    return [500000.0 ** (-2 * i / case["rot"]) for i in range(case["rot"] // 2)]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=gen, device=dev)  # noqa: E731
    qlens, kvlens = _lengths(case)
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    total, need = sum(qlens), [-(-n // bs) for n in kvlens]
    blocks = sum(need) + BLOCK_GAP
    order = torch.randperm(blocks, generator=gen, device=dev).to(torch.int32)
    first = torch.tensor([sum(need[:i]) for i in range(len(need))], device=dev)
    col = torch.arange(max(need), device=dev)
    tables = torch.where(col < torch.tensor(need, device=dev)[:, None],
                         order[(first[:, None] + col).clamp(max=blocks - 1)], order[-1]).to(torch.int32).contiguous()
    cu = [0]
    for n in qlens:
        cu.append(cu[-1] + n)
    s = dict(case=case, cu=cu, kv=kvlens, blocks=blocks, max_q=max(qlens), max_kv=max(kvlens), tables=tables,
             cu_dev=torch.tensor(cu, dtype=torch.int32, device=dev),
             kv_dev=torch.tensor(kvlens, dtype=torch.int32, device=dev), k_scale=1.0, v_scale=1.0, scale=d ** -0.5)
    scaled = case["op"] in ("fill", "read")
    if case["fp8"] and not scaled:
        s["k_scale"], s["v_scale"] = 0.0113, 0.0087

    def cache(scale):
        """The cache's elements, and its block scales: blocks and heads of different magnitudes."""
        x = torch.empty(blocks, bs, hkv, d, dtype=torch.float8_e4m3fn if case["fp8"] else torch.bfloat16, device=dev)
        scales = torch.empty(blocks, hkv, device=dev)
        step = max(1, (1 << 26) // (bs * hkv * d))
        for b in range(0, blocks, step):  # in parts: 32-bit copies of a long cache would not fit beside it
            part = randn(*x[b:b + step].shape)
            if scaled:
                part *= torch.exp2(randn(len(part), 1, hkv, 1))
                top = part.abs().amax((1, 3)) / 448
                scales[b:b + step] = torch.exp2(top.log2().ceil()) if case["power"] else top
                part /= scales[b:b + step, None, :, None]
            elif case["fp8"]:
                part /= scale
            x[b:b + step] = (part.clamp(-448, 448) if case["fp8"] else part).to(x.dtype)
        return x, scales

    s["k_cache"], k_scales = cache(s["k_scale"])
    s["v_cache"], v_scales = cache(s["v_scale"])
    if scaled:
        s["k_scales"], s["v_scales"] = k_scales, v_scales
    if case["op"] in ("turn", "fill"):
        if case["fused"]:  # rows of one projection's output
            rows = randn(total, hq + 2 * hkv, d).to(torch.bfloat16)
            s["q"], s["k_new"], s["v_new"] = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        else:
            s["q"], s["k_new"], s["v_new"] = (randn(total, h, d).to(torch.bfloat16) for h in (hq, hkv, hkv))
        s["inv_freq"], s["pair_axes"] = _frequencies(case), _pair_axes(case)
        s["inv_freq_dev"] = torch.tensor(s["inv_freq"], dtype=torch.float64, device=dev)
        s["pair_axes_dev"] = torch.tensor(s["pair_axes"], dtype=torch.int64, device=dev)
        at = torch.cat([torch.arange(kv - n, kv, device=dev) for n, kv in zip(qlens, kvlens)])
        if case["axes"] > 1:
            # runs of 96 text tokens, whose positions agree on all axes, and frames of 12 x 16 patches, which stand at
            # one time and at places of their own
            patch, place = at % 288 - 96, torch.stack((at // 288 * 100, at % 192 // 16, at % 16, at % 7))[:case["axes"]]
            s["positions"] = torch.where(patch < 0, at // 288 * 100 + at % 288, place).to(torch.int32).contiguous()
        # the blocks that the step writes to, and the first slot it writes in each
        places = [(i, b, max(0, kv - n - b * bs)) for i, (n, kv) in enumerate(zip(qlens, kvlens)) if n
                  for b in range((kv - n) // bs, -(-kv // bs))]
        row, b, slot = torch.tensor(places, device=dev).T
        s["touched"], s["first_slot"] = tables[row, b].long(), slot
    else:
        # queries that agree with some keys: scores of a few units, as trained heads have
        s["q"] = 2.0 * randn(total, hq, d)
        if case["sinks"] and case["op"] == "sinks":
            # the first tokens draw attention whatever the query is, and say little
            lean = randn(hkv, 1, d)
            s["q"] = (s["q"].view(total, hkv, -1, d) + lean).view(total, hq, d)
            t = torch.arange(min(case["sinks"], 4, min(kvlens)), device=dev)
            page, slot = tables[:, t // bs].long(), (t % bs).expand(case["seqs"], -1)
            for x, y, scale in ((s["k_cache"], 0.4 * lean.view(hkv, d).expand(*page.shape, -1, -1), s["k_scale"]),
                                (s["v_cache"], 0.1 * randn(*page.shape, hkv, d), s["v_scale"])):
                x[page, slot] = ((y / scale).clamp(-448, 448) if case["fp8"] else y).to(x.dtype)
        s["q"] = s["q"].to(torch.bfloat16)
    s["out"] = torch.empty(total, hq, d, dtype=torch.bfloat16, device=dev)
    if own:
        import paged_kv_attention_unified_gb300 as ua
        s["plan"] = ua.Plan(cu, kvlens, hq, hkv, d, bs, tables.shape[1],
                            kv_dtype=ua.UA_KV_FP8_E4M3 if case["fp8"] else ua.UA_KV_BF16, window=case["window"],
                            sink_tokens=case["sinks"])
        if scaled:
            s["plan"].set_block_scales(k_scales, v_scales)
        if case["rot"]:
            s["rope"] = ua.Rope(s["inv_freq"], interleaved=case["interleaved"], axes=s["pair_axes"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if case["op"] in ("sinks", "read"):
        if own:
            s["plan"].forward(s["q"], s["k_cache"], s["v_cache"], s["out"], s["cu_dev"], s["kv_dev"], s["tables"],
                              s["blocks"], s["max_q"], s["max_kv"], s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"])
            return s["out"]
        return _plain_attend(s)
    if own and case["rot"]:
        s["plan"].rope_append_kv(s["rope"], s["q"], s["k_new"], s["v_new"], s["out"], s["k_cache"], s["v_cache"],
                                 s["tables"], s["blocks"], positions=s.get("positions"), k_scale=s["k_scale"],
                                 v_scale=s["v_scale"])
    elif own:
        s["plan"].append_kv(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["tables"], s["blocks"])
    else:
        _plain_append(s)
    done = {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if case["op"] == "fill":
        done |= {"k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    if case["rot"]:
        done["q"] = s["out"]
    return done


def _tokens(s):
    """For each query token: its sequence, its index in it, its position in the sequence's cache."""
    tok = torch.arange(s["cu"][-1], device=s["q"].device)
    seq = torch.searchsorted(s["cu_dev"][1:], tok, right=True)
    i = tok - s["cu_dev"][seq]
    return seq, i, s["kv_dev"][seq] - (s["cu_dev"][seq + 1] - s["cu_dev"][seq]) + i


def _plain_append(s):
    case, rot = s["case"], s["case"]["rot"]
    seq, _, pos = _tokens(s)
    page, slot = s["tables"][seq, pos // case["bs"]].long(), pos % case["bs"]
    k, v = s["k_new"].float(), s["v_new"].float()
    if rot:
        at = s["positions"][s["pair_axes_dev"]].T if "positions" in s else pos[:, None]
        angle = at.double() * s["inv_freq_dev"]
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

        def turned(x):
            if case["interleaved"]:
                a, b = x[..., :rot:2], x[..., 1:rot:2]
                head = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
            else:
                a, b = x[..., :rot // 2], x[..., rot // 2:rot]
                head = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
            return torch.cat((head, x[..., rot:]), -1)

        k = turned(k)
        s["out"].copy_(turned(s["q"].float()))
    if case["op"] == "fill":
        _plain_fill(s, s["k_cache"], s["k_scales"], k, page, slot)
        _plain_fill(s, s["v_cache"], s["v_scales"], v, page, slot)
        return
    if case["fp8"]:
        k, v = (k / s["k_scale"]).clamp(-448, 448), (v / s["v_scale"]).clamp(-448, 448)
    s["k_cache"][page, slot] = k.to(s["k_cache"].dtype)
    s["v_cache"][page, slot] = v.to(s["v_cache"].dtype)


def _plain_fill(s, cache, scales, x, page, slot):
    touched, first = s["touched"], s["first_slot"][:, None]
    size = x.abs().amax(-1)
    top = torch.zeros_like(scales).scatter_reduce_(0, page[:, None].expand_as(size), size, "amax")[touched]
    part, power = torch.frexp(top)  # top = part 2^power, 448 = 7/8 2^9
    fresh = torch.ldexp(torch.ones_like(top), power - 9 + (part > 0.875).int()).clamp(LEAST, MOST)
    fresh = torch.where(top > 0, fresh, LEAST)
    old = scales[touched]
    old_part, old_power = torch.frexp(448 * old)
    doublings = (power - old_power + (part > old_part).int()).clamp(min=0)
    scale = torch.where(first == 0, fresh, torch.where(top > 0, torch.ldexp(old, doublings), old))
    kept = (cache[touched].float() * (old / scale)[:, None, :, None]).to(cache.dtype).view(torch.uint8)
    earlier = torch.arange(cache.shape[1], device=x.device) < first
    cache[touched] = torch.where(earlier[:, :, None, None], kept, cache[touched].view(torch.uint8)).view(cache.dtype)
    scales[touched] = scale
    cache[page, slot] = (x / scales[page][..., None]).clamp(-448, 448).to(cache.dtype)


def _plain_attend(s):
    case = s["case"]
    hkv, d, n, window = case["hkv"], case["d"], case["seqs"], case["window"]
    seq, i, _ = _tokens(s)
    q = torch.zeros(n, s["max_q"], case["hq"], d, device=s["q"].device)
    q[seq, i] = s["q"].float()
    q = q.view(n, s["max_q"], hkv, -1, d).permute(0, 2, 3, 1, 4)  # sequence, KV head, query of the group, token, dim
    # the keys that some query of a sequence sees: its first ones, then those from the first query's window on
    ctx = s["kv_dev"] - (s["cu_dev"][1:] - s["cu_dev"][:-1])
    begin = (ctx - window + 1).clamp(min=case["sinks"]) if window else torch.zeros_like(ctx)
    head = case["sinks"] if window else 0
    col = torch.arange(min(s["max_kv"], head + window + s["max_q"]) if window else s["max_kv"], device=q.device)
    t = torch.where(col < head, col, begin[:, None] + col - head)  # [sequence, key]
    inside = t < s["kv_dev"][:, None]
    t = torch.where(inside, t, 0)
    page, slot = s["tables"].gather(1, t // case["bs"]).long(), t % case["bs"]

    def rows(cache, scales, scale):
        x = cache[page, slot].float()
        return x.mul_(scales[page][..., None]) if scales is not None else x.mul_(scale) if case["fp8"] else x

    k = rows(s["k_cache"], s.get("k_scales"), s["k_scale"]).permute(0, 2, 3, 1).unsqueeze(2)
    x = torch.matmul(q, k) * s["scale"]
    del k
    pos = (ctx[:, None] + torch.arange(s["max_q"], device=x.device))[:, :, None]
    seen = inside[:, None] & (t[:, None] <= pos)
    if window:
        seen = seen & ((t[:, None] > pos - window) | (t[:, None] < case["sinks"]))
    x.masked_fill_(~seen[:, None, None], -math.inf)
    x -= x.amax(-1, keepdim=True)
    x.exp_()
    x /= x.sum(-1, keepdim=True)
    x.nan_to_num_(0.0)  # the padding tokens of the shorter sequences
    v = rows(s["v_cache"], s.get("v_scales"), s["v_scale"]).permute(0, 2, 1, 3).unsqueeze(2)
    out = torch.matmul(x, v).permute(0, 3, 1, 2, 4).reshape(n, s["max_q"], case["hq"], d)
    return s["out"].copy_(out[seq, i])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    qlens, kvlens = _lengths(case)
    hq, hkv, d, bs, elt, total = case["hq"], case["hkv"], case["d"], case["bs"], 1 if case["fp8"] else 2, sum(qlens)
    if case["op"] in ("turn", "fill"):
        pages = sum(-(-kv // bs) - (kv - n) // bs for n, kv in zip(qlens, kvlens) if n)
        queries = 4 * total * hq * d if case["rot"] else 0
        more = 8 * hkv * pages if case["op"] == "fill" else 4 * case["axes"] * total
        return {"bytes": queries + 2 * total * hkv * d * (2 + elt) + more, "flops": 3 * total * (hq + hkv) * case["rot"]}
    keys = pairs = pages = 0
    for n, kv in zip(qlens, kvlens):
        ctx = kv - n
        if not case["window"]:
            keys, pages, pairs = keys + kv, pages - (-kv // bs), pairs + n * ctx + n * (n + 1) // 2
            continue
        low = max(0, ctx - case["window"] + 1)
        head = min(case["sinks"], low)
        keys, pages = keys + head + kv - low, pages - (-kv // bs) - low // bs + min(-(-head // bs), low // bs)
        for i in range(ctx, kv):
            lo = max(0, i - case["window"] + 1)
            pairs += i + 1 - lo + min(case["sinks"], lo)
    more = 8 * hkv * pages if case["op"] == "read" else 0
    return {"bytes": 4 * total * hq * d + 2 * hkv * d * elt * keys + more, "flops": 4 * hq * d * pairs}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    qlens, kvlens = _lengths(case)
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    if case["op"] in ("turn", "fill"):
        return _exact_append(s, qlens, kvlens)
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    if (4.0 * hq * d + 200.0) * sum(n * kv for n, kv in zip(qlens, kvlens)) > 6e12:
        return None
    for j, (n, kv) in enumerate(zip(qlens, kvlens)):
        begin = s["cu"][j]
        t = torch.arange(kv, device=out.device)
        i = torch.arange(kv - n, kv, device=out.device)[:, None]
        hide = t > i
        if case["window"]:
            hide |= (t <= i - case["window"]) & (t >= case["sinks"])
        page, slot = s["tables"][j].long()[t // bs], t % bs
        for g in range(hkv):
            k, v = s["k_cache"][page, slot, g].double(), s["v_cache"][page, slot, g].double()
            if case["op"] == "read":
                k, v = k * s["k_scales"][page, g].double()[:, None], v * s["v_scales"][page, g].double()[:, None]
            else:
                k, v = k * s["k_scale"], v * s["v_scale"]
            for h in range(g * (hq // hkv), (g + 1) * (hq // hkv)):
                score = s["q"][begin:begin + n, h].double() @ k.T * s["scale"]
                out[begin:begin + n, h] = torch.softmax(score.masked_fill(hide, -math.inf), -1) @ v
    return out


def _exact_append(s, qlens, kvlens):
    case, bs, rot = s["case"], s["case"]["bs"], s["case"]["rot"]
    dev = s["q"].device
    done = {"k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
    new_k, new_v = s["k_new"].double(), s["v_new"].double()
    logical = torch.cat([torch.arange(kv - n, kv, device=dev) for n, kv in zip(qlens, kvlens)])
    pages = torch.cat([x[torch.arange(kv - n, kv, device=dev) // bs] for n, kv, x in zip(qlens, kvlens, s["tables"].long())])
    if rot:
        done["q"] = s["q"].double()
        where = torch.arange(rot // 2, device=dev)
        a, b = (2 * where, 2 * where + 1) if case["interleaved"] else (where, where + rot // 2)
        w = torch.tensor(_frequencies(case), dtype=torch.float64, device=dev)
        axis = torch.tensor(_pair_axes(case), device=dev)
        places = s["positions"].double() if case["axes"] > 1 else logical.double()[None]
        for lo in range(0, len(logical), 1024):
            turn = torch.exp(1j * places[:, lo:lo + 1024][axis].T * w)[:, None]
            for x in (done["q"][lo:lo + 1024], new_k[lo:lo + 1024]):
                z = torch.complex(x[..., a], x[..., b]) * turn
                x[..., a], x[..., b] = z.real, z.imag
    if case["op"] == "turn":
        for to, x, scale in ((done["k_cache"], new_k, s["k_scale"]), (done["v_cache"], new_v, s["v_scale"])):
            to[pages, logical % bs] = (x / scale).clamp(-448, 448) if case["fp8"] else x
        return done
    for name, x in (("k", new_k), ("v", new_v)):
        codes, scales = done[name + "_cache"], s[name + "_scales"].double()
        top = torch.zeros_like(scales).index_reduce_(0, pages, x.abs().amax(-1), "amax")
        for page, slot in zip(s["touched"].tolist(), s["first_slot"].tolist()):
            if slot:
                grown = (top[page] / (448 * scales[page])).clamp(min=1).log2().ceil().exp2()
                codes[page, :slot] /= grown[:, None]
                scales[page] *= grown
            else:
                scales[page] = (top[page] / 448).log2().ceil().clamp(-100, 100).exp2()
        codes[pages, logical % bs] = (x / scales[pages][..., None]).clamp(-448, 448)
        done[name + "_scales"] = scales
    return done
