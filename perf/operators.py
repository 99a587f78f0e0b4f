"""The measured cases of rotary append and of attention with shaped scores over a paged cache.

Two operators of one attention layer of a serving step:

rope    the step's queries and new keys are rotated to their positions, the keys and values written into the
        paged cache (bf16, or e4m3 codes of value / scale). Outputs: the rotated queries and both whole caches.
attend  attention of the step's queries over the cache, with scores capped by a tanh, a bias that falls with the
        distance, or a prefix that every query sees. Output: bf16 rows.

A case's sequence lengths come from the case alone ("lens" seeds them), the values, the page order and the
weights of the cache from the seed of `prepare`.
"""
import math
import random

import torch

own = False

BLOCK_GAP = 3  # physical blocks beyond the ones in use


# ---------------------------------------------------------------- cases

def listed():
    rope = dict(op="rope", window=0, causal=True, cap=0.0, alibi=False, prefix=0)
    attend = dict(op="attend", interleaved=False, rot=0, scaling="plain", fused=False, shift=0, window=0, causal=True,
                  prefix=0, cap=0.0, alibi=False)
    return [
        # one user's next token after a long context: launch latency
        rope | dict(name="rope_one_token", seqs=1, q_lo=1, q_hi=1, ctx_lo=131071, ctx_hi=131071, hq=32, hkv=8, d=128,
                    bs=16, fp8=False, lens=1, rot=128, interleaved=False, scaling="plain", fused=False, shift=0),
        # a batch of decoding users, e4m3 cache, half of each head rotated, frequencies scaled by bands
        rope | dict(name="rope_decode_batch_fp8", seqs=64, q_lo=1, q_hi=1, ctx_lo=512, ctx_hi=16000, hq=64, hkv=8, d=128,
                    bs=16, fp8=True, lens=2, rot=64, interleaved=False, scaling="bands", fused=True, shift=0),
        # prompts in chunks of odd sizes, rows inside a fused projection, pairs interleaved, positions given (a cache
        # whose oldest part was dropped)
        rope | dict(name="rope_chunks", seqs=9, q_lo=100, q_hi=700, ctx_lo=0, ctx_hi=2000, hq=24, hkv=4, d=96, bs=32,
                    fp8=False, lens=3, rot=96, interleaved=True, scaling="linear", fused=True, shift=100003),
        # whole prompts, all heads, stretched for long contexts
        rope | dict(name="rope_prompts", seqs=4, q_lo=4096, q_hi=4096, ctx_lo=0, ctx_hi=0, hq=32, hkv=32, d=128, bs=128,
                    fp8=False, lens=4, rot=128, interleaved=False, scaling="yarn", fused=False, shift=0),
        # one user's next token with capped scores: latency
        attend | dict(name="capped_one_token", seqs=1, q_lo=1, q_hi=1, ctx_lo=500, ctx_hi=500, hq=32, hkv=8, d=128, bs=16,
                      fp8=False, lens=5, cap=50.0),
        # a batch of decoding users, ragged lengths
        attend | dict(name="capped_decode", seqs=64, q_lo=1, q_hi=1, ctx_lo=511, ctx_hi=4095, hq=32, hkv=8, d=128, bs=16,
                      fp8=False, lens=6, cap=50.0),
        # few users with very long contexts, e4m3 cache
        attend | dict(name="capped_decode_long_fp8", seqs=8, q_lo=1, q_hi=1, ctx_lo=131071, ctx_hi=131071, hq=64, hkv=8,
                      d=128, bs=16, fp8=True, lens=7, cap=30.0),
        # whole prompts with capped scores
        attend | dict(name="capped_prompts", seqs=4, q_lo=4096, q_hi=4096, ctx_lo=0, ctx_hi=0, hq=32, hkv=32, d=128, bs=128,
                      fp8=False, lens=8, cap=50.0),
        # distance bias: decoding users, all heads separate, narrow heads
        attend | dict(name="alibi_decode", seqs=33, q_lo=1, q_hi=1, ctx_lo=700, ctx_hi=9000, hq=16, hkv=16, d=64, bs=32,
                      fp8=False, lens=9, alibi=True),
        # distance bias: chunks of new tokens over earlier ones, e4m3 cache
        attend | dict(name="alibi_chunks_fp8", seqs=5, q_lo=300, q_hi=1100, ctx_lo=100, ctx_hi=2500, hq=32, hkv=8, d=128,
                      bs=16, fp8=True, lens=10, alibi=True),
        # prompts whose first part every token sees (an image or an instruction), wide heads
        attend | dict(name="prefix_prompts", seqs=6, q_lo=900, q_hi=2100, ctx_lo=0, ctx_hi=0, hq=16, hkv=8, d=256, bs=64,
                      fp8=False, lens=11, prefix=700),
        # all of them with a window: chunks over earlier tokens
        attend | dict(name="capped_alibi_prefix_window", seqs=7, q_lo=1, q_hi=900, ctx_lo=0, ctx_hi=1800, hq=32, hkv=8, d=64,
                      bs=16, fp8=False, lens=12, cap=20.0, alibi=True, prefix=333, window=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hkv, qpk = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 3, 4, 8])
    d = 32 * rng.randint(1, 8)
    case = dict(op=rng.choice(["rope", "attend"]), hq=hkv * qpk, hkv=hkv, d=d, bs=rng.choice([16, 32, 64, 128, 256]),
                fp8=rng.random() < 0.4, lens=rng.randrange(1 << 20), causal=True, window=0, cap=0.0, alibi=False,
                prefix=0, interleaved=False, rot=0, scaling="plain", fused=False, shift=0)
    if case["op"] == "rope":
        tokens = _log(rng, 1, 16384)
        case["seqs"] = min(tokens, _log(rng, 1, 128))
        case["q_hi"] = max(1, tokens // case["seqs"])
        case["ctx_hi"] = _log(rng, 1, max(2, min(100000, 200000 // case["seqs"])))
        case |= dict(interleaved=rng.random() < 0.5, rot=2 * rng.randint(1, d // 2) if rng.random() < 0.4 else d,
                     scaling=rng.choice(["plain", "linear", "ntk", "yarn", "bands"]), fused=rng.random() < 0.5,
                     shift=_log(rng, 1, 1000000) if rng.random() < 0.3 else 0)
    else:
        decode = rng.random() < 0.5
        case["q_hi"] = rng.randint(1, 4) if decode else _log(rng, 5, 2000)
        case["seqs"] = _log(rng, 1, 100 if decode else max(2, min(16, 6000 // case["q_hi"])))
        case["ctx_hi"] = _log(rng, 1, max(2, min(60000, 200000 // case["seqs"])) if decode else 3000)
        kind = rng.randrange(1, 8)  # at least one of cap, bias and prefix
        case["cap"] = float(rng.choice([10, 20, 30, 50, 100])) if kind & 1 else 0.0
        case["alibi"] = bool(kind & 2)
        case["prefix"] = _log(rng, 1, case["q_hi"] + case["ctx_hi"]) if kind & 4 else 0
        if not kind & 4:
            case["causal"] = rng.random() < 0.8
        case["window"] = _log(rng, 1, 4000) if rng.random() < 0.3 else 0
    case["q_lo"] = rng.choice([1, case["q_hi"]])
    case["ctx_lo"] = rng.choice([0, case["ctx_hi"]])
    return case


def _lengths(case):
    rng = random.Random(case["lens"])
    q = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["seqs"])]
    return q, [n + rng.randint(case["ctx_lo"], case["ctx_hi"]) for n in q]


def _prefixes(case):
    rng = random.Random(case["lens"] + 1)
    return [rng.randint(case["prefix"] // 2, case["prefix"]) for _ in range(case["seqs"])]


def _frequencies(case):
    """Rotation frequencies (radians a position) and the amplitude of the sines, as a model's configuration states them."""
    n, base, factor, far = case["rot"] // 2, 500000.0, 8.0, 8192.0
    kind = case["scaling"]
    if kind == "ntk":
        base *= factor ** (case["rot"] / max(1, case["rot"] - 2))
    w = [base ** (-i / n) for i in range(n)]
    if kind == "linear":
        w = [x / factor for x in w]
    if kind == "bands":  # slow pairs stretched, fast ones left, those between blended
        share = [min(1.0, max(0.0, (far * x / (2 * math.pi) - 1.0) / (4.0 - 1.0))) for x in w]
        w = [x * (s + (1 - s) / factor) for x, s in zip(w, share)]
    if kind == "yarn":
        at = lambda turns: case["rot"] * math.log(far / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(at(32.0))), min(case["rot"] - 1, math.ceil(at(1.0)))
        ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(n)]
        w = [x * (1 - r) + x / factor * r for x, r in zip(w, ramp)]
        return w, 0.1 * math.log(factor) + 1.0
    return w, 1.0


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
    if case["fp8"]:
        s["k_scale"], s["v_scale"] = 0.0113, 0.0087

    def cache(scale):
        x = torch.empty(blocks, bs, hkv, d, dtype=torch.float8_e4m3fn if case["fp8"] else torch.bfloat16, device=dev)
        step = max(1, (1 << 26) // (bs * hkv * d))
        for b in range(0, blocks, step):  # in parts: 32-bit copies of a long cache would not fit beside it
            part = randn(*x[b:b + step].shape)
            x[b:b + step] = ((part / scale).clamp(-448, 448) if case["fp8"] else part).to(x.dtype)
        return x

    s["k_cache"], s["v_cache"] = cache(s["k_scale"]), cache(s["v_scale"])
    if case["op"] == "rope":
        if case["fused"]:  # rows of one projection's output
            rows = randn(total, hq + 2 * hkv, d).to(torch.bfloat16)
            s["q"], s["k_new"], s["v_new"] = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        else:
            s["q"], s["k_new"], s["v_new"] = (randn(total, h, d).to(torch.bfloat16) for h in (hq, hkv, hkv))
        s["inv_freq"], s["amplitude"] = _frequencies(case)
        if case["shift"]:  # positions other than the places in the cache
            s["positions"] = torch.cat([torch.arange(kv - n, kv, device=dev) for n, kv in zip(qlens, kvlens)])
            s["positions"] = (s["positions"] + case["shift"]).to(torch.int32)
        s["inv_freq_dev"] = torch.tensor(s["inv_freq"], dtype=torch.float64, device=dev)
    else:
        # queries that agree with some keys: scores of a few units, as trained heads have
        s["q"] = (2.0 * randn(total, hq, d)).to(torch.bfloat16)
        if case["alibi"]:
            s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], dtype=torch.float32, device=dev)
        if case["prefix"]:
            s["prefix"] = _prefixes(case)
            s["prefix_dev"] = torch.tensor(s["prefix"], dtype=torch.int32, device=dev)
    s["out"] = torch.empty(total, hq, d, dtype=torch.bfloat16, device=dev)
    if own:
        import paged_kv_attention_unified_gb300 as ua
        s["plan"] = ua.Plan(cu, kvlens, hq, hkv, d, bs, tables.shape[1],
                            kv_dtype=ua.UA_KV_FP8_E4M3 if case["fp8"] else ua.UA_KV_BF16, causal=int(case["causal"]),
                            window=case["window"], prefix_lens=s.get("prefix"))
        if case["op"] == "rope":
            s["rope"] = ua.Rope(s["inv_freq"], interleaved=case["interleaved"], amplitude=s["amplitude"])
        else:
            s["plan"].set_scores(softcap=case["cap"], alibi_slopes=s.get("slopes"))
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if s["case"]["op"] == "rope":
        if own:
            s["plan"].rope_append_kv(s["rope"], s["q"], s["k_new"], s["v_new"], s["out"], s["k_cache"], s["v_cache"],
                                     s["tables"], s["blocks"], positions=s.get("positions"), k_scale=s["k_scale"],
                                     v_scale=s["v_scale"])
        else:
            _plain_rope(s)
        return {"q": s["out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if own:
        s["plan"].forward(s["q"], s["k_cache"], s["v_cache"], s["out"], s["cu_dev"], s["kv_dev"], s["tables"], s["blocks"],
                          s["max_q"], s["max_kv"], s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["out"]
    return _plain_attend(s)


def _tokens(s):
    """For each query token: its sequence, its index in it, its position in the sequence's cache."""
    tok = torch.arange(s["cu"][-1], device=s["q"].device)
    seq = torch.searchsorted(s["cu_dev"][1:], tok, right=True)
    i = tok - s["cu_dev"][seq]
    return seq, i, s["kv_dev"][seq] - (s["cu_dev"][seq + 1] - s["cu_dev"][seq]) + i


def _plain_rope(s):
    case, rot = s["case"], s["case"]["rot"]
    seq, _, pos = _tokens(s)
    angle = s.get("positions", pos).double()[:, None] * s["inv_freq_dev"]
    cos, sin = (s["amplitude"] * angle.cos()).float()[:, None], (s["amplitude"] * angle.sin()).float()[:, None]

    def turned(x):
        x = x.float()
        if case["interleaved"]:
            a, b = x[..., :rot:2], x[..., 1:rot:2]
            head = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            head = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((head, x[..., rot:]), -1)

    page, slot = s["tables"][seq, pos // case["bs"]].long(), pos % case["bs"]
    k, v = turned(s["k_new"]), s["v_new"].float()
    if case["fp8"]:
        k, v = (k / s["k_scale"]).clamp(-448, 448), (v / s["v_scale"]).clamp(-448, 448)
    s["k_cache"][page, slot] = k.to(s["k_cache"].dtype)
    s["v_cache"][page, slot] = v.to(s["v_cache"].dtype)
    s["out"].copy_(turned(s["q"]))


def _plain_attend(s):
    case = s["case"]
    hkv, d = case["hkv"], case["d"]
    seq, i, _ = _tokens(s)
    n = case["seqs"]
    q = torch.zeros(n, s["max_q"], case["hq"], d, device=s["q"].device)
    q[seq, i] = s["q"].float()
    q = q.view(n, s["max_q"], hkv, -1, d).permute(0, 2, 3, 1, 4)  # sequence, KV head, query of the group, token, dim
    rows = lambda cache, scale: (cache[s["tables"].long()].float() * scale).flatten(1, 2)  # noqa: E731
    k = rows(s["k_cache"], s["k_scale"]).permute(0, 2, 3, 1).unsqueeze(2)
    x = torch.matmul(q, k) * s["scale"]
    del k
    if case["cap"]:
        x.div_(case["cap"]).tanh_().mul_(case["cap"])
    t = torch.arange(x.shape[-1], device=x.device)
    pos = (s["kv_dev"] - (s["cu_dev"][1:] - s["cu_dev"][:-1]))[:, None] + torch.arange(s["max_q"], device=x.device)
    pos = pos[:, None, None, :, None]
    if case["alibi"]:
        x -= s["slopes"].view(1, hkv, -1, 1, 1) * (pos - t).abs().float()
    seen = (t < s["kv_dev"].view(-1, 1, 1, 1, 1)).expand(-1, -1, -1, s["max_q"], -1)
    if case["prefix"]:
        seen = seen & ((t <= pos) | (t < s["prefix_dev"].view(-1, 1, 1, 1, 1)))
    elif case["causal"]:
        seen = seen & (t <= pos)
    if case["window"]:
        seen = seen & (t > pos - case["window"])
    x.masked_fill_(~seen, -math.inf)
    x -= x.amax(-1, keepdim=True)
    x.exp_()
    x /= x.sum(-1, keepdim=True)
    x.nan_to_num_(0.0)  # the padding tokens of the shorter sequences
    v = rows(s["v_cache"], s["v_scale"]).permute(0, 2, 1, 3).unsqueeze(2)
    out = torch.matmul(x, v).permute(0, 3, 1, 2, 4).reshape(n, s["max_q"], case["hq"], d)
    return s["out"].copy_(out[seq, i])


# ---------------------------------------------------------------- what a pass cannot do without

def _visible(case, n, kv, prefix):
    """Visible (query, key) pairs of one sequence, and the keys that any query sees."""
    pairs, first, last, ctx = 0, kv, 0, kv - n
    for i in range(n):
        hi = min(kv, max(ctx + i + 1, prefix)) if case["causal"] else kv
        lo = max(0, ctx + i - case["window"] + 1) if case["window"] else 0
        pairs, first, last = pairs + hi - lo, min(first, lo), max(last, hi)
    return pairs, max(0, last - first)


def work(case):
    qlens, kvlens = _lengths(case)
    hq, hkv, d, elt, total = case["hq"], case["hkv"], case["d"], 1 if case["fp8"] else 2, sum(qlens)
    if case["op"] == "rope":
        return {"bytes": total * d * (4 * hq + 2 * hkv * (2 + elt)), "flops": 3 * total * (hq + hkv) * case["rot"]}
    seen = [_visible(case, n, kv, prefix) for n, kv, prefix in zip(qlens, kvlens, _prefixes(case))]
    return {"bytes": 4 * total * hq * d + 2 * hkv * d * elt * sum(k for _, k in seen),
            "flops": 4 * hq * d * sum(p for p, _ in seen)}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    qlens, kvlens = _lengths(case)
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    group = hq // hkv
    if case["op"] == "rope":
        done = {"q": s["q"].double(), "k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
        new_k, new_v = s["k_new"].double(), s["v_new"].double()
        w, rot = torch.tensor(s["inv_freq"], dtype=torch.float64, device=s["q"].device), case["rot"]
        at = torch.arange(rot // 2, device=w.device)
        a, b = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + rot // 2)
        for n, kv, begin, table in zip(qlens, kvlens, s["cu"], s["tables"].long()):
            pos = torch.arange(kv - n, kv, device=w.device)
            turn = torch.polar(torch.full((n, 1, rot // 2), s["amplitude"], dtype=torch.float64, device=w.device),
                               torch.outer((pos + case["shift"]).double(), w)[:, None])
            for x in (done["q"][begin:begin + n], new_k[begin:begin + n]):
                z = torch.complex(x[..., a], x[..., b]) * turn
                x[..., a], x[..., b] = z.real, z.imag
            for to, x, scale in ((done["k_cache"], new_k, s["k_scale"]), (done["v_cache"], new_v, s["v_scale"])):
                x = x[begin:begin + n]
                to[table[pos // bs], pos % bs] = (x / scale).clamp(-448, 448) if case["fp8"] else x
        return done
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    per_pair = 4.0 * hq * d + 200.0
    if per_pair * sum(n * kv for n, kv in zip(qlens, kvlens)) > 6e12:
        return None
    for j, (n, kv) in enumerate(zip(qlens, kvlens)):
        begin = s["cu"][j]
        t = torch.arange(kv, device=out.device)
        i = torch.arange(kv - n, kv, device=out.device)[:, None]
        hide = torch.zeros(n, kv, dtype=torch.bool, device=out.device)
        if case["causal"]:
            hide |= t > i
        if case["prefix"]:
            hide &= t >= s["prefix"][j]
        if case["window"]:
            hide |= t <= i - case["window"]
        page, slot = s["tables"][j].long()[t // bs], t % bs
        for g in range(hkv):
            k = s["k_cache"][page, slot, g].double() * s["k_scale"]
            v = s["v_cache"][page, slot, g].double() * s["v_scale"]
            for h in range(g * group, (g + 1) * group):
                score = s["q"][begin:begin + n, h].double() @ k.T * s["scale"]
                if case["cap"]:
                    score = case["cap"] * torch.tanh(score / case["cap"])
                if case["alibi"]:
                    score -= s["slopes"][h].double() * (i - t).abs()
                weight = torch.softmax(score.masked_fill(hide, -math.inf), -1)
                out[begin:begin + n, h] = weight @ v
    return out
