"""The serving operators of the latent cache, as they are measured: appending new
rows to the paged cache (normalisation, position rotation and rounding on the
way) and attention of one or a few new tokens per request over it (decode).

``run`` computes each in its plain form, elementary torch operations in 32 bits
rounded once at the end, or, where ``own`` is true, through the framework's
entry points.  ``exact`` computes the same from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

D_C, D_R, D_NOPE, D_V, BLOCK = 512, 64, 128, 128, 64
THETA = 10000.0
EPS = 1e-6
#: Columns of the fused down-projection whose last 576 are the new cache rows.
FUSED = 1536 + D_C + D_R
#: Most (key, head, query) score products and most cached tokens of a decode case.
MOST_WORK = 600_000 * 128
MOST_KEYS = 600_000


def listed():
    d = lambda name, **k: dict({"name": name, "op": "decode", "kv": "bf16", "heads": 128, "q": 1, "docs": 0, "spread": 1}, **k)  # noqa: E731
    a = lambda name, **k: dict({"name": name, "op": "append", "kv": "bf16", "norm": True, "spread": 1}, **k)  # noqa: E731
    return [
        # the first tokens of one short chat: launch and latency are all there is
        d("decode_1x500", reqs=1, lo=500, hi=500),
        # one user's next token over a 32K prompt (the short-extend workload's cache with one new token)
        d("decode_1x32k", reqs=1, lo=32769, hi=32769),
        # a full serving batch with ragged contexts, the largest case
        d("decode_64_mixed", reqs=64, lo=2048, hi=32768),
        # the same with an FP8 cache and medium contexts
        d("decode_64_fp8", reqs=64, lo=4000, hi=16384, kv="fp8"),
        # two 128K FP8 prompts, one drafted token verified with the next one
        d("decode_2x128k_fp8_draft", reqs=2, lo=131074, hi=131074, q=2, kv="fp8"),
        # 16 documents of 16K cached at their own positions, then the answer's tokens
        d("decode_docs_256k", reqs=1, lo=262144 + 77, hi=262144 + 77, docs=16),
        # one tensor-parallel shard of 16 heads, many short chats
        d("decode_96_heads16", reqs=96, lo=700, hi=6000, heads=16),
        # a shard of 32 heads with three drafted tokens per request
        d("decode_24_heads32_draft", reqs=24, lo=1000, hi=12000, heads=32, q=4),
        # one new row per request of a decode step
        a("append_64x1", reqs=64, lo=1, hi=1),
        # the same into an FP8 cache, a large batch with two tokens each
        a("append_200x2_fp8", reqs=200, lo=2, hi=2, kv="fp8"),
        # a prefill batch of ragged new extents
        a("append_8_prefill", reqs=8, lo=512, hi=4096),
        # a long prefill into an FP8 cache
        a("append_4x16k_fp8", reqs=4, lo=15000, hi=16384, kv="fp8"),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    kv = rng.choice(["bf16", "fp8"])
    spread = rng.randrange(1 << 20)
    if rng.random() < 0.3:
        reqs = log(1, 256)
        hi = log(1, max(1, min(16384, 65536 // reqs)))
        return {"op": "append", "kv": kv, "norm": rng.random() < 0.8, "reqs": reqs, "lo": log(1, hi), "hi": hi, "spread": spread}
    heads = rng.choice([128, 128, 64, 32, 16, 8, rng.randrange(1, 129)])
    q = rng.choice([1, 1, 1, 2, 3, 4, 8])
    reqs = log(1, 128)
    most = min(MOST_KEYS, MOST_WORK // (heads * q)) // reqs
    hi = log(max(q, 64), max(128, min(131072, most)))
    lo = log(max(q, hi / 16), hi)
    docs = rng.choice([0, 0, 0, rng.randrange(1, 9)])
    if hi < 16 * docs + q:
        docs = 0
    return {"op": "decode", "kv": kv, "heads": heads, "q": q, "reqs": reqs, "lo": lo, "hi": hi, "docs": docs if lo > 16 * docs + q else 0, "spread": spread}


def _lens(case):
    """The case's lengths, spread over their logarithm: of the contexts (decode), of the new extents (append)."""
    r = random.Random(case["spread"])
    lo, hi = case["lo"], case["hi"]
    if lo == hi:
        return [lo] * case["reqs"]
    return [min(hi, max(lo, int(round(math.exp(r.uniform(math.log(lo), math.log(hi))))))) for _ in range(case["reqs"])]


def _segments(case, n):
    """(start, length, rope offset) of the documents of a request of n tokens: equal parts of what its new tokens leave."""
    docs, q = case["docs"], case["q"]
    if not docs:
        return []
    tail = 76 + q if n > 16 * (77 + q) else q
    each = (n - tail) // docs
    return [(d * each, each, d * each) for d in range(docs)]


def _before(case):
    """Tokens that an append's requests have in the cache already."""
    r = random.Random(case["spread"] + 1)
    return [r.randrange(0, 200) for _ in range(case["reqs"])]


def _paged(lens, g, dev):
    """A block table over a pool in random order with a tenth to spare, and the pool's size."""
    need = [-(-n // BLOCK) for n in lens]
    pool = sum(need) + -(-sum(need) // 10) + 1
    perm = torch.randperm(pool, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    cols = torch.arange(max(need), device=dev)
    needs = torch.tensor(need, device=dev)
    first = torch.cumsum(needs, 0) - needs
    at = (first[:, None] + cols[None, :]).clamp_(max=pool - 1)
    table = torch.where(cols[None, :] < needs[:, None], perm[at], torch.full_like(at, -1, dtype=torch.int32))
    return table.contiguous(), pool


def _cache(pool, kv, g, dev):
    """Cached rows: normalised latents and rotated keys, both of unit variance."""
    if kv == "bf16":
        c = torch.empty((pool, BLOCK, D_C + D_R), dtype=torch.bfloat16, device=dev)
        for part in c.split(4096):
            part.normal_(generator=g)
        return c, 1.0
    c = torch.empty((pool, BLOCK, D_C + 2 * D_R), dtype=torch.uint8, device=dev)
    scale = 5.5 / 448.0
    for part in c.split(4096):
        x = torch.randn(part.shape[:2] + (D_C + D_R,), generator=g, device=dev)
        part[..., :D_C] = (x[..., :D_C] / scale).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        part[..., D_C:] = x[..., D_C:].to(torch.bfloat16).view(torch.uint8)
    return c, scale


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"case": case}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    if case["op"] == "append":
        new, before = _lens(case), _before(case)
        lens = [a + b for a, b in zip(new, before)]
        rows = sum(new)
        s["block_table"], pool = _paged(lens, g, dev)
        s["kv_cache"], s["kv_scale"] = _cache(pool, case["kv"], g, dev)
        # the rows are the last columns of the fused down-projection's output, and stay strided
        s["kv"] = torch.randn((rows, FUSED), generator=g, device=dev, dtype=torch.float32).mul_(3.0).to(torch.bfloat16)[:, FUSED - D_C - D_R:]
        s["norm_weight"] = (1.0 + 0.2 * torch.randn(D_C, generator=g, device=dev)).to(torch.bfloat16) if case["norm"] else None
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s["cu_q"], s["seq_lens"] = i32(cu), i32(lens)
        s["pos"] = torch.cat([torch.arange(b, b + n, device=dev) for b, n in zip(before, new)]).to(torch.int32)
        return s
    lens, q, H = _lens(case), case["q"], case["heads"]
    s["block_table"], pool = _paged(lens, g, dev)
    s["kv_cache"], s["kv_scale"] = _cache(pool, case["kv"], g, dev)
    rows = len(lens) * q
    s["q"] = torch.randn((rows, H, D_NOPE + D_R), generator=g, device=dev).to(torch.bfloat16)
    s["kv_b_proj"] = (torch.randn((D_C, H * (D_NOPE + D_V)), generator=g, device=dev) / math.sqrt(D_C)).to(torch.bfloat16)
    s["seq_lens"] = i32(lens)
    s["q_pos"] = (s["seq_lens"][:, None] - q + torch.arange(q, device=dev)[None, :]).to(torch.int32).reshape(-1).contiguous()
    if case["docs"]:
        segs = [_segments(case, n) for n in lens]
        s["segments"] = torch.tensor([x for r in segs for x in r], dtype=torch.int64, device=dev)
        s["seg_ptr"] = i32([case["docs"] * k for k in range(len(lens) + 1)])
    s["out"] = torch.empty((rows, H, D_V), dtype=torch.bfloat16, device=dev)
    s["softmax_scale"] = (D_NOPE + D_R) ** -0.5
    return s


def _turn(x, angle):
    """Pairs (2k, 2k + 1) of x's last axis turned by angle (one for each pair, in 64 bits)."""
    c, n = torch.cos(angle).to(x.dtype), torch.sin(angle).to(x.dtype)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * c - b * n, a * n + b * c), -1).flatten(-2)


def _angles(pos):
    k = torch.arange(D_R // 2, device=pos.device, dtype=torch.float64)
    return pos.to(torch.float64)[..., None] * torch.pow(torch.tensor(THETA, dtype=torch.float64, device=pos.device), -2 * k / D_R)


def _append_outputs(s):
    c = s["kv_cache"]
    if s["case"]["kv"] == "bf16":
        return {"cache": c}
    return {"codes": c[..., :D_C].view(torch.float8_e4m3fn), "k_rope": c[..., D_C:].view(torch.bfloat16)}


def _plain_append(s):
    x = s["kv"].float()
    c = x[:, :D_C]
    if s["norm_weight"] is not None:
        c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * s["norm_weight"].float()
    k = _turn(x[:, D_C:], _angles(s["pos"]))
    row = torch.arange(x.shape[0], device=x.device)
    req = torch.bucketize(row, s["cu_q"][1:].long(), right=True)
    tok = s["seq_lens"].long()[req] - s["cu_q"].long()[req + 1] + row
    block = s["block_table"][req, tok // BLOCK].long()
    if s["case"]["kv"] == "bf16":
        s["kv_cache"][block, tok % BLOCK] = torch.cat((c, k), -1).to(torch.bfloat16)
    else:
        codes = (c / s["kv_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["kv_cache"][block, tok % BLOCK] = torch.cat((codes, k.to(torch.bfloat16).view(torch.uint8)), -1)
    return _append_outputs(s)


def _plain_decode(s):
    case, H, q = s["case"], s["case"]["heads"], s["case"]["q"]
    lens = s["seq_lens"].long()
    B, L, dev = lens.shape[0], s["block_table"].shape[1] * BLOCK, lens.device
    tok = torch.arange(L, device=dev)
    rows = s["kv_cache"][s["block_table"].long().clamp_min(0)].reshape(B, L, -1)
    if case["kv"] == "bf16":
        c, k = rows[..., :D_C].float(), rows[..., D_C:].float()
    else:
        c = rows[..., :D_C].view(torch.float8_e4m3fn).float() * s["kv_scale"]
        k = rows[..., D_C:].view(torch.bfloat16).float()
    live = tok[None, :] < lens[:, None]
    c = torch.where(live[..., None], c, torch.zeros((), device=dev))
    k = torch.where(live[..., None], k, torch.zeros((), device=dev))
    seen = tok[None, None, :] <= (lens[:, None] - q + torch.arange(q, device=dev)[None, :])[..., None]
    if case["docs"]:
        # a document's keys are attended with the query turned back by its offset: the same as turning its keys on
        seg = s["segments"].reshape(B, -1, 3)
        inside = (tok >= seg[:, :, :1]) & (tok < seg[:, :, :1] + seg[:, :, 1:2])
        k = _turn(k, _angles((inside * seg[:, :, 2:]).sum(1)))
        seen = seen & (inside.any(1) | (tok >= (seg[:, :, 0] + seg[:, :, 1]).amax(1, keepdim=True)))[:, None]
    w = s["kv_b_proj"].float().reshape(D_C, 2, H, D_NOPE)
    x = s["q"].float().reshape(B, q, H, -1)
    lat = torch.einsum("bqhd,chd->bqhc", x[..., :D_NOPE], w[:, 0]).reshape(B, q * H, D_C)
    rot = _turn(x[..., D_NOPE:], _angles(s["q_pos"].reshape(B, q, 1))).reshape(B, q * H, D_R)
    score = (lat @ c.transpose(1, 2) + rot @ k.transpose(1, 2)) * s["softmax_scale"]
    score = score.reshape(B, q, H, L).masked_fill(~seen[:, :, None], float("-inf"))
    p = torch.exp(score - score.amax(-1, keepdim=True))
    o = (p.reshape(B, q * H, L) @ c).reshape(B, q, H, D_C) / p.sum(-1)[..., None]
    return {"out": torch.einsum("bqhc,chd->bqhd", o, w[:, 1]).to(torch.bfloat16).reshape(B * q, H, D_V)}


def run(state):
    s = state
    if not own:
        return _plain_append(s) if s["case"]["op"] == "append" else _plain_decode(s)
    from mla_prefix_cache_gb300 import api
    if s["case"]["op"] == "append":
        api.cache_append(s["kv"], s["pos"], s["kv_cache"], s["block_table"], s["seq_lens"], cu_q=s["cu_q"],
                         norm_weight=s["norm_weight"], norm_eps=EPS, rope_theta=THETA, kv_scale=s["kv_scale"])
        return _append_outputs(s)
    if "workspace" not in s:
        n = api.decode_workspace_size(s["seq_lens"].shape[0], s["q"].shape[0], s["q"].shape[1])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=s["q"].device)
    out = api.decode(s["q"], s["q_pos"], s["kv_cache"], s["block_table"], s["seq_lens"], s["kv_b_proj"],
                     segments=s.get("segments"), seg_ptr=s.get("seg_ptr"), softmax_scale=s["softmax_scale"], rope_theta=THETA,
                     kv_scale=s["kv_scale"], out=s["out"], workspace=s["workspace"])
    return {"out": out}


def work(case):
    lens = _lens(case)
    row = 2 * (D_C + D_R) if case["kv"] == "bf16" else D_C + 2 * D_R
    if case["op"] == "append":
        n = sum(lens)
        return {"bytes": n * (2 * (D_C + D_R) + row + 4) + (2 * D_C if case["norm"] else 0), "flops": n * (5 * D_C + 3 * D_R)}
    H, q, docs = case["heads"], case["q"], case["docs"]
    rows = len(lens) * q
    keys = pairs = 0
    for n in lens:
        seg = _segments(case, n)
        hidden = seg[-1][0] + seg[-1][1] - sum(x[1] for x in seg) if docs else 0
        keys += n - hidden
        pairs += sum(n - hidden - (q - 1 - i) for i in range(q))
    proj = 2 * D_C * (D_NOPE + D_V) * H * rows
    return {"bytes": keys * row + 2 * D_C * H * (D_NOPE + D_V) + rows * H * 2 * (D_NOPE + D_R + D_V) + 4 * sum(-(-n // BLOCK) for n in lens),
            "flops": 2 * (D_C + D_R + D_C) * H * pairs + proj}


def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    table, lens = s["block_table"].tolist(), s["seq_lens"].tolist()
    if case["op"] == "append":
        cache, cu = s["kv_cache"], s["cu_q"].tolist()
        if case["kv"] == "bf16":
            lat, rope = cache[..., :D_C].to(f), cache[..., D_C:].to(f)
        else:
            lat, rope = cache[..., :D_C].view(torch.float8_e4m3fn).to(f), cache[..., D_C:].view(torch.bfloat16).to(f)
        z = torch.polar(torch.ones((), dtype=f, device=cache.device), _exact_angle(s["pos"]))
        for r, n in enumerate(lens):
            x = s["kv"][cu[r]:cu[r + 1]].to(f)
            t = range(n - x.shape[0], n)
            b, o = torch.tensor([table[r][i // BLOCK] for i in t], device=x.device), torch.tensor([i % BLOCK for i in t], device=x.device)
            y = x[:, :D_C]
            if case["norm"]:
                y = y / torch.sqrt((y * y).sum(1, keepdim=True) / D_C + EPS) * s["norm_weight"].to(f)
            lat[b, o] = y if case["kv"] == "bf16" else (y / s["kv_scale"]).clamp(-448, 448)
            rope[b, o] = torch.view_as_real(torch.view_as_complex(x[:, D_C:].reshape(-1, D_R // 2, 2)) * z[cu[r]:cu[r + 1]]).flatten(1)
        return {"cache": torch.cat((lat, rope), -1)} if case["kv"] == "bf16" else {"codes": lat, "k_rope": rope}
    H, q = case["heads"], case["q"]
    wk, wv = s["kv_b_proj"][:, :H * D_NOPE].to(f).reshape(D_C, H, D_NOPE), s["kv_b_proj"][:, H * D_NOPE:].to(f).reshape(D_C, H, D_V)
    out = []
    for r, n in enumerate(lens):
        rows = s["kv_cache"][torch.tensor(table[r][:-(-n // BLOCK)], device=wk.device)].flatten(0, 1)[:n]
        if case["kv"] == "bf16":
            c, k = rows[:, :D_C].to(f), rows[:, D_C:].to(f)
        else:
            c, k = rows[:, :D_C].view(torch.float8_e4m3fn).to(f) * s["kv_scale"], rows[:, D_C:].view(torch.bfloat16).to(f)
        seg = _segments(case, n)
        parts = seg + [(seg[-1][0] + seg[-1][1] if seg else 0, n, 0)]
        for i in range(q):
            x, pos = s["q"][r * q + i].to(f), int(s["q_pos"][r * q + i])
            score, value = [], []
            for start, length, offset in parts:
                e = min(start + length, n - q + i + 1)
                if e <= start:
                    continue
                z = torch.polar(torch.ones((), dtype=f, device=c.device), _exact_angle(torch.tensor(pos - offset, device=c.device)))
                xr = torch.view_as_real(torch.view_as_complex(x[:, D_NOPE:].reshape(H, -1, 2).contiguous()) * z).flatten(1)
                if n * H <= 1 << 17:   # each key up-projected, as it is defined
                    nope = torch.einsum("hd,thd->ht", x[:, :D_NOPE], torch.einsum("tc,chd->thd", c[start:e], wk))
                else:                  # the same product, taken the other way round
                    nope = torch.einsum("hd,chd->hc", x[:, :D_NOPE], wk) @ c[start:e].T
                score.append(s["softmax_scale"] * (nope + xr @ k[start:e].T))
                value.append(c[start:e])
            a = torch.softmax(torch.cat(score, 1), 1)
            out.append(torch.einsum("hc,chd->hd", a @ torch.cat(value), wv))
    return {"out": torch.stack(out)}


def _exact_angle(pos):
    k = torch.arange(D_R // 2, device=pos.device, dtype=torch.float64)
    return pos.to(torch.float64).unsqueeze(-1) * torch.exp(-2 * k / D_R * math.log(THETA))
