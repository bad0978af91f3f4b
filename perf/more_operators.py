"""The operators of a sparse decoding step, as they are measured: block tables
and slot maps from the requests' lengths, the mean row of every block that new
rows fill, a cheap score of every block for every query, and the choice of the
blocks that a query attends.

``run`` computes each in its plain form, elementary torch operations in 32 bits
rounded once at the end, or, where ``own`` is true, through the framework's
entry points.  ``exact`` computes the numbers among them from the definitions in
64 bits.
"""
import math
import random

import torch

own = False

D_C, D_R, D_NOPE, D_V, BLOCK = 512, 64, 128, 128, 64
ROW = D_C + D_R
THETA = 10000.0
#: Most rows of a step, (query, head, block) products and (query, block) pairs of a case.
MOST_ROWS = 65536
MOST_PRODUCTS = 32 * 2048 * 128
MOST_PAIRS = 128 * 16384


def listed():
    t = lambda name, **k: dict({"name": name, "op": "tables", "shared": 0, "short": False, "spread": 1}, **k)  # noqa: E731
    m = lambda name, **k: dict({"name": name, "op": "means", "kv": "bf16", "spread": 1}, **k)  # noqa: E731
    s = lambda name, **k: dict({"name": name, "op": "scores", "heads": 128, "q": 1, "spread": 1}, **k)  # noqa: E731
    c = lambda name, **k: dict({"name": name, "op": "select", "scores": "fp32", "q": 1, "sinks": 1, "recent": 2, "spread": 1}, **k)  # noqa: E731
    return [
        # a decoding step with four drafted tokens each, and the cut back to the accepted ones
        t("tables_64_drafts", kind="drafts", reqs=64, lo=2048, hi=32768, new=5),
        # prompts admitted (their slots are those of a whole prefill batch), and retired
        t("tables_32_prompts", kind="prompts", reqs=32, lo=512, hi=4096, new=4096),
        # a large continuous batch: sequences end, others begin, behind a shared prefix of 16 blocks
        t("tables_512_mixed", kind="mixed", reqs=512, lo=1024, hi=32768, new=128, shared=16),
        # a decoding step with three drafted tokens each: one request in 16 fills a block
        m("means_64_step", reqs=64, lo=2048, hi=32768, new_lo=4, new_hi=4),
        # a prefill batch of ragged new extents, FP8 cache
        m("means_8_prefill_fp8", reqs=8, lo=512, hi=8192, new_lo=512, new_hi=4096, kv="fp8"),
        # a long prefill
        m("means_4x16k", reqs=4, lo=16384, hi=16384, new_lo=15000, new_hi=16384),
        # one user's next token over a 32K prompt
        s("scores_1x32k", reqs=1, lo=32769, hi=32769),
        # a shard of 32 heads with three drafted tokens per request
        s("scores_24_heads32_draft", reqs=24, lo=1000, hi=12000, heads=32, q=4),
        # a full serving batch with ragged contexts
        s("scores_64_mixed", reqs=64, lo=2048, hi=32768),
        # long prompts
        s("scores_32x128k", reqs=32, lo=131074, hi=131074),
        # the choice in a full serving batch: 2048 of up to 32768 tokens
        c("select_64_mixed", reqs=64, lo=2048, hi=32768, keep=32),
        # a million tokens each
        c("select_128x1m", reqs=128, lo=1 << 20, hi=1 << 20, keep=64),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    spread = rng.randrange(1 << 20)
    op = rng.choice(["tables", "means", "scores", "scores", "select"])
    if op == "tables":
        kind = rng.choice(["drafts", "prompts", "mixed"])
        reqs = log(1, 512)
        hi = log(256, min(131072, 512 * 32768 // reqs) if kind != "prompts" else max(257, MOST_ROWS // reqs))
        new = {"drafts": rng.randrange(1, 9), "prompts": hi, "mixed": log(1, MOST_ROWS // reqs)}[kind]
        shared = rng.choice([0, 0, log(1, 32)]) if kind != "prompts" else 0
        return {"op": op, "kind": kind, "reqs": reqs, "lo": log(max(1, hi / 16), hi), "hi": hi, "new": new, "shared": min(shared, hi // BLOCK),
                "short": rng.random() < 0.15, "spread": spread}
    if op == "means":
        reqs = log(1, 256)
        new_hi = log(1, max(1, min(16384, MOST_ROWS // reqs)))
        hi = max(new_hi, log(64, max(64, min(131072, 512 * 2048 // reqs))))
        return {"op": op, "kv": rng.choice(["bf16", "fp8"]), "reqs": reqs, "lo": log(max(1, hi / 16), hi), "hi": hi, "new_lo": log(1, new_hi), "new_hi": new_hi,
                "spread": spread}
    q = rng.choice([1, 1, 1, 2, 3, 4, 8])
    if op == "scores":
        heads = rng.choice([128, 128, 64, 32, 16, 8, rng.randrange(1, 129)])
        reqs = log(1, 128)
        hi = log(512, max(513, min(1 << 19, BLOCK * MOST_PRODUCTS // (128 * reqs * q))))
        return {"op": op, "heads": heads, "q": q, "reqs": reqs, "lo": log(max(256, hi / 16), hi), "hi": hi, "spread": spread}
    reqs = log(1, 256)
    hi = log(64, max(64, min(1 << 20, BLOCK * MOST_PAIRS // (reqs * q))))
    sinks, recent = rng.randrange(0, 4), rng.randrange(1, 4)
    return {"op": op, "scores": rng.choice(["fp32", "bf16"]), "q": q, "reqs": reqs, "lo": log(max(q, hi / 16), hi), "hi": hi,
            "keep": max(sinks + recent, log(1, 256)), "sinks": sinks, "recent": recent, "spread": spread}


def _spread(r, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm."""
    return lo if lo >= hi else min(hi, max(lo, int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))))


def _lens(case):
    """The contexts' lengths, at least the new rows of each."""
    r = random.Random(case["spread"])
    return [_spread(r, case["lo"], case["hi"]) for _ in range(case["reqs"])]


def _new(case):
    """The new rows of a means case's requests, at most their lengths."""
    r = random.Random(case["spread"] + 1)
    return [min(n, _spread(r, case["new_lo"], case["new_hi"])) for n in _lens(case)]


def _steps(case):
    """The two steps that a tables case goes to and fro between: (lengths, new rows) of its requests."""
    r = random.Random(case["spread"])
    least = BLOCK * case["shared"]
    a, b = [], []
    for _ in range(case["reqs"]):
        n = max(least, _spread(r, case["lo"], case["hi"]))
        if case["kind"] == "drafts":        # drafted, and cut back by what was rejected
            k = r.randrange(0, case["new"])
            a.append((n + case["new"], case["new"]))
            b.append((n + k, 0))
        elif case["kind"] == "prompts":     # admitted, and retired
            a.append((n, min(n, case["new"])))
            b.append((least, 0))
        else:                               # every sequence ends, begins, goes on or is cut back by chance
            m = max(least, _spread(r, case["lo"], case["hi"]))
            n, m = (n, m) if r.random() < 0.3 else (n, n + r.randrange(0, 200))
            n, m = (least if r.random() < 0.2 else n), (least if r.random() < 0.2 else m)
            a.append((n, min(case["new"], max(0, n - m))))
            b.append((m, min(case["new"], max(0, m - n))))
    return [[n for n, _ in a], [k for _, k in a]], [[n for n, _ in b], [k for _, k in b]]


def _blocks(n):
    return -(-n // BLOCK)


def _paged(lens, g, dev):
    """A block table over a pool in random order with a tenth to spare, and the pool's size."""
    need = [_blocks(n) for n in lens]
    pool = sum(need) + _blocks(sum(need)) + 1
    perm = torch.randperm(pool, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    cols = torch.arange(max(need), device=dev)
    needs = torch.tensor(need, device=dev)
    first = torch.cumsum(needs, 0) - needs
    at = (first[:, None] + cols[None, :]).clamp_(max=pool - 1)
    return torch.where(cols[None, :] < needs[:, None], perm[at], torch.full_like(at, -1, dtype=torch.int32)).contiguous(), pool


def _cu(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return cu


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"case": case}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    if case["op"] == "tables":
        steps, sh = _steps(case), case["shared"]
        need = [[_blocks(n) for n in lens] for lens, _ in steps]
        most = max(sum(n) for n in need)
        short = case["short"] and sum(need[0]) > sum(need[1])
        pool = sum(need[1]) + (sum(need[0]) - sum(need[1])) // 2 + 1 if short else most + _blocks(most) + 64
        # the table as the second step left it: shared blocks first, the same for all, then each request's own
        width = max(max(n) for n in need) + 3
        perm = torch.randperm(pool + sh, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
        cols, held = torch.arange(width, device=dev), torch.tensor(need[1], device=dev)
        mine = (held - sh).clamp_min(0)
        first = torch.cumsum(mine, 0) - mine + sh
        at = torch.where(cols < sh, cols.expand(len(need[1]), -1), first[:, None] + cols - sh).clamp_(max=pool + sh - 1)
        s["block_table"] = torch.where(cols < held[:, None], perm[at], torch.full_like(at, -1, dtype=torch.int32)).contiguous()
        s["held"], s["shared"] = held.to(torch.int32), i32([sh] * case["reqs"]) if sh else None
        used = int(mine.sum()) + sh
        s["free_blocks"] = torch.full((pool,), -1, dtype=torch.int32, device=dev)
        s["free_blocks"][:pool + sh - used] = perm[used:]
        s["free_count"] = i32([pool + sh - used])
        s["steps"] = [(i32(lens), i32(_cu(new)), torch.empty(sum(new), dtype=torch.int64, device=dev)) for lens, new in steps]
        s["turn"] = 0
        return s
    lens, q = _lens(case), case.get("q", 0)
    s["block_table"], pool = _paged(lens, g, dev)
    s["seq_lens"] = i32(lens)
    rows = len(lens) * q
    if case["op"] == "means":
        new = _new(case)
        s["rows"], s["cu_q"] = sum(new), i32(_cu(new))
        s["means"] = torch.randn((pool, ROW), generator=g, device=dev).to(torch.bfloat16)
        # normalised latents and rotated keys, both of unit variance
        if case["kv"] == "bf16":
            s["kv_cache"], s["kv_scale"] = torch.empty((pool, BLOCK, ROW), dtype=torch.bfloat16, device=dev), 1.0
            for part in s["kv_cache"].split(4096):
                part.normal_(generator=g)
            return s
        s["kv_cache"], s["kv_scale"] = torch.empty((pool, BLOCK, D_C + 2 * D_R), dtype=torch.uint8, device=dev), 5.5 / 448.0
        for part in s["kv_cache"].split(4096):
            x = torch.randn(part.shape[:2] + (ROW,), generator=g, device=dev)
            part[..., :D_C] = (x[..., :D_C] / s["kv_scale"]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            part[..., D_C:] = x[..., D_C:].to(torch.bfloat16).view(torch.uint8)
        return s
    width = s["block_table"].shape[1]
    if case["op"] == "select":
        # shares of attention: positive, over orders of magnitude, many of the least ones 0; not seen, -infinite
        x = torch.randn((rows, width), generator=g, device=dev)
        x = torch.where(x < -1.5, torch.zeros((), device=dev), torch.exp(2.5 * x)) / (24 * width)
        s["scores"] = x.masked_fill_(~_seen(s), float("-inf")).to(torch.float32 if case["scores"] == "fp32" else torch.bfloat16)
        s["table"], s["lens"] = torch.empty((rows, case["keep"]), dtype=torch.int32, device=dev), torch.empty(rows, dtype=torch.int32, device=dev)
        return s
    H = case["heads"]
    # means of a block's rows keep what its tokens share: less than unit variance, and queries that tell blocks apart
    s["means"] = (0.4 * torch.randn((pool, ROW), generator=g, device=dev)).to(torch.bfloat16)
    s["q"] = (2.5 * torch.randn((rows, H, D_NOPE + D_R), generator=g, device=dev)).to(torch.bfloat16)
    s["kv_b_proj"] = (torch.randn((D_C, H * (D_NOPE + D_V)), generator=g, device=dev) / math.sqrt(D_C)).to(torch.bfloat16)
    s["q_pos"] = (s["seq_lens"][:, None] - q + torch.arange(q, device=dev)[None, :]).to(torch.int32).reshape(-1).contiguous()
    s["out"] = torch.empty((rows, width), dtype=torch.bfloat16, device=dev)
    s["softmax_scale"] = (D_NOPE + D_R) ** -0.5
    return s


def _own_block(s):
    """The block that each query's own token lies in."""
    q = s["case"]["q"]
    return (s["seq_lens"].long()[:, None] - q + torch.arange(q, device=s["seq_lens"].device)).reshape(-1) // BLOCK


def _seen(s):
    """[query][block]: the block is complete and before the query's own."""
    return torch.arange(s["block_table"].shape[1], device=s["block_table"].device) < _own_block(s)[:, None]


def _turn(x, angle):
    """Pairs (2k, 2k + 1) of x's last axis turned by angle (one for each pair, in 64 bits)."""
    c, n = torch.cos(angle).to(x.dtype), torch.sin(angle).to(x.dtype)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * c - b * n, a * n + b * c), -1).flatten(-2)


def _angles(pos):
    k = torch.arange(D_R // 2, device=pos.device, dtype=torch.float64)
    return pos.to(torch.float64)[..., None] * torch.pow(torch.tensor(THETA, dtype=torch.float64, device=pos.device), -2 * k / D_R)


def _tables_outputs(s, slots):
    return {"table": s["block_table"], "held": s["held"], "free": s["free_blocks"], "count": s["free_count"], "slots": slots}


def _plain_tables(s, lens, cu, slots):
    table, stack = s["block_table"], s["free_blocks"]
    dev, cap = table.device, stack.shape[0]
    j = torch.arange(table.shape[1], device=dev)
    held, need = s["held"].long(), (lens.long() + BLOCK - 1) // BLOCK
    shared = s["shared"].long() if s["shared"] is not None else torch.zeros_like(held)
    # blocks behind the new length, all but the shared ones, go onto the stack, the last one first
    back = (j >= torch.maximum(need, shared)[:, None]) & (j < held[:, None])
    order = torch.cumsum(back.reshape(-1), 0).reshape(back.shape)
    top = s["free_count"].long() + order[-1, -1]
    stack = torch.cat((stack, stack[:1]))     # one place more for what is not written
    stack[torch.where(back, top - order, cap)] = table
    # requests that the free blocks suffice for, in order, take theirs from the top
    more = (need - held).clamp_min(0)
    ends = torch.cumsum(more, 0)
    served = (ends <= top) | (more == 0)
    kept = torch.where(served, need, held)
    fresh = (j >= held[:, None]) & (j < kept[:, None])
    at = top - 1 - ((ends - more)[:, None] + j - held[:, None])
    table = torch.where(fresh, stack[torch.where(fresh, at, cap)], torch.where((j >= need[:, None]) & (j < held[:, None]), -1, table))
    s["block_table"].copy_(table)
    s["free_blocks"].copy_(stack[:cap])
    s["held"].copy_(kept)
    s["free_count"].copy_(top - torch.where(served, more, 0).sum())
    row = torch.arange(slots.shape[0], device=dev)
    r = torch.bucketize(row, cu[1:].long(), right=True)
    t = lens.long()[r] - cu.long()[r + 1] + row
    b = t // BLOCK
    ok = (t >= 0) & (b < kept[r])
    slots.copy_(torch.where(ok, table[r, torch.where(ok, b, 0)].long() * BLOCK + t % BLOCK, -1))
    return _tables_outputs(s, slots)


def _rows(s, blocks):
    c = s["kv_cache"][blocks]
    if s["case"]["kv"] == "bf16":
        return c.float()
    return torch.cat((c[..., :D_C].view(torch.float8_e4m3fn).float() * s["kv_scale"], c[..., D_C:].view(torch.bfloat16).float()), -1)


def _filled(s):
    """The blocks that the new rows of a means case fill, found in a list with room for any (their places repeat the last one where it is longer)."""
    cu, lens = s["cu_q"].long(), s["seq_lens"].long()
    lo = (lens - cu.diff()) // BLOCK
    n = lens // BLOCK - lo
    ends = torch.cumsum(n, 0)
    i = torch.arange(s["rows"] // BLOCK + lens.shape[0], device=lens.device)
    r = torch.bucketize(i, ends, right=True)
    ok = r < lens.shape[0]
    r = r.clamp_max(lens.shape[0] - 1)
    b = torch.where(ok, lo[r] + i - (ends - n)[r], 0)
    return torch.where(ok, s["block_table"][r, b].long(), s["means"].shape[0])


def _plain_means(s):
    blocks, n = _filled(s), s["means"].shape[0]
    mean = _rows(s, blocks.clamp_max(n - 1)).sum(1) / BLOCK
    more = torch.cat((s["means"], s["means"][:1]))     # one place more for what is not written
    more[blocks] = mean.to(torch.bfloat16)
    s["means"].copy_(more[:n])
    return {"means": s["means"]}


def _plain_scores(s):
    H, q, B = s["case"]["heads"], s["case"]["q"], s["seq_lens"].shape[0]
    m = s["means"][s["block_table"].long().clamp_min(0)].float()
    x = s["q"].float().reshape(B, q, H, -1)
    w = s["kv_b_proj"][:, :H * D_NOPE].float().reshape(D_C, H, D_NOPE)
    lat = torch.einsum("bqhd,chd->bqhc", x[..., :D_NOPE], w)
    rot = _turn(x[..., D_NOPE:], _angles(s["q_pos"].reshape(B, q, 1)))
    score = (torch.cat((lat, rot), -1).reshape(B, q * H, ROW) @ m.transpose(1, 2) * s["softmax_scale"]).reshape(B * q, H, -1)
    seen = _seen(s)
    score = score.masked_fill(~seen[:, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    share = (p / p.sum(-1, keepdim=True).clamp_min(1e-30)).sum(1) / H
    s["out"].copy_(share.masked_fill(~seen, float("-inf")))
    return {"scores": s["out"]}


def _plain_select(s):
    case, scores = s["case"], s["scores"].float()
    mine, width = _own_block(s), s["block_table"].shape[1]
    j = torch.arange(width, device=scores.device)
    always = (j < case["sinks"]) | (j > mine[:, None] - case["recent"])
    key = torch.where(j > mine[:, None], float("-inf"), torch.where(always, float("inf"), scores))
    best = torch.sort(key, dim=1, descending=True, stable=True).indices     # equal ones: the lowest first
    n = torch.minimum(mine + 1, torch.tensor(case["keep"], device=scores.device))
    best = torch.nn.functional.pad(best[:, :case["keep"]], (0, max(0, case["keep"] - width)))
    i = torch.arange(case["keep"], device=scores.device)
    blocks = torch.sort(torch.where(i < n[:, None], best, width)).values
    req = torch.arange(scores.shape[0], device=scores.device) // case["q"]
    table = s["block_table"][req[:, None], blocks.clamp_max(width - 1)]
    t = s["seq_lens"].long()[req] - case["q"] + torch.arange(scores.shape[0], device=scores.device) % case["q"]
    s["table"].copy_(torch.where(i < n[:, None], table, -1))
    s["lens"].copy_(torch.where(n > 0, (n - 1) * BLOCK + t % BLOCK + 1, 0))
    return {"table": s["table"], "lens": s["lens"]}


def run(state):
    s, op = state, state["case"]["op"]
    if op == "tables":
        lens, cu, slots = s["steps"][s["turn"]]
        s["turn"] ^= 1
    if not own:
        return _plain_tables(s, lens, cu, slots) if op == "tables" else {"means": _plain_means, "scores": _plain_scores, "select": _plain_select}[op](s)
    from mla_prefix_cache_gb300 import api
    if op == "tables":
        api.assign_blocks(s["block_table"], s["held"], lens, s["free_blocks"], s["free_count"], shared=s["shared"], cu_q=cu, slots=slots)
        return _tables_outputs(s, slots)
    if op == "means":
        return {"means": api.block_means(s["kv_cache"], s["block_table"], s["seq_lens"], s["means"], rows=s["rows"], cu_q=s["cu_q"], kv_scale=s["kv_scale"])}
    if op == "scores":
        if "workspace" not in s:
            n = api.block_scores_workspace_size(s["q"].shape[0], s["q"].shape[1], s["block_table"].shape[1])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=s["q"].device)
        return {"scores": api.block_scores(s["q"], s["q_pos"], s["means"], s["block_table"], s["seq_lens"], s["kv_b_proj"], softmax_scale=s["softmax_scale"],
                                           rope_theta=THETA, out=s["out"], workspace=s["workspace"])}
    case = s["case"]
    table, lens = api.select_blocks(s["scores"], s["block_table"], s["seq_lens"], keep=case["keep"], sinks=case["sinks"], recent=case["recent"],
                                    table=s["table"], lens=s["lens"])
    return {"table": table, "lens": lens}


def work(case):
    if case["op"] == "tables":
        (a, new_a), (b, new_b) = _steps(case)
        moved = sum(abs(_blocks(n) - _blocks(m)) for n, m in zip(a, b))
        # each way by turns: an id is read and written once when it is taken, and once more, as -1, when it is given back
        return {"bytes": (8 + 8 + 12) * case["reqs"] / 2 + moved * (8 + 12) / 2 + 8 * (sum(new_a) + sum(new_b)) / 2, "flops": 0}
    lens = _lens(case)
    if case["op"] == "means":
        n = sum(x // BLOCK - (x - k) // BLOCK for x, k in zip(lens, _new(case)))
        return {"bytes": n * (BLOCK * (2 * ROW if case["kv"] == "bf16" else D_C + 2 * D_R) + 2 * ROW) + 8 * len(lens), "flops": n * BLOCK * ROW}
    q, width = case["q"], max(_blocks(n) for n in lens)
    seen = [[max(0, n - q + i) // BLOCK for i in range(q)] for n in lens]
    pairs, rows = sum(map(sum, seen)), len(lens) * q
    if case["op"] == "select":
        kept = sum(min(case["keep"], x + 1) for r in seen for x in r)
        return {"bytes": pairs * (4 if case["scores"] == "fp32" else 2) + 4 * rows * (case["keep"] + 1) + 4 * kept, "flops": 0}
    H = case["heads"]
    return {"bytes": sum(max(r) for r in seen) * (2 * ROW + 4) + 2 * D_C * H * D_NOPE + rows * (2 * H * (D_NOPE + D_R) + 2 * width),
            "flops": 2 * ROW * H * pairs + 2 * D_C * D_NOPE * H * rows}


def exact(case, seed):
    if case["op"] in ("tables", "select"):
        return None
    s = prepare(case, seed)
    f, lens = torch.float64, s["seq_lens"].tolist()
    if case["op"] == "means":
        mean, cu = s["means"].to(f), s["cu_q"].tolist()
        for r, n in enumerate(lens):
            for j in range((n - (cu[r + 1] - cu[r])) // BLOCK, n // BLOCK):
                b = int(s["block_table"][r, j])
                x = s["kv_cache"][b]
                if case["kv"] == "fp8":
                    mean[b] = torch.cat((x[:, :D_C].view(torch.float8_e4m3fn).to(f).mean(0) * s["kv_scale"], x[:, D_C:].view(torch.bfloat16).to(f).mean(0)))
                else:
                    mean[b] = x.to(f).mean(0)
        return {"means": mean}
    H, q = case["heads"], case["q"]
    w = s["kv_b_proj"][:, :H * D_NOPE].to(f).reshape(D_C, H, D_NOPE)
    out = torch.full((len(lens) * q, s["block_table"].shape[1]), float("-inf"), dtype=f, device=w.device)
    k = torch.arange(D_R // 2, device=w.device, dtype=f)
    for r, n in enumerate(lens):
        for i in range(q):
            b = (n - q + i) // BLOCK
            if b < 1:
                continue
            m = s["means"][s["block_table"][r, :b].long()].to(f)
            x, pos = s["q"][r * q + i].to(f), int(s["q_pos"][r * q + i])
            z = torch.polar(torch.ones((), dtype=f, device=w.device), pos * torch.exp(-2 * k / D_R * math.log(THETA)))
            rot = torch.view_as_real(torch.view_as_complex(x[:, D_NOPE:].reshape(H, -1, 2).contiguous()) * z).flatten(1)
            lat = torch.einsum("hd,chd->hc", x[:, :D_NOPE], w)
            out[r * q + i, :b] = torch.softmax(s["softmax_scale"] * (lat @ m[:, :D_C].T + rot @ m[:, D_C:].T), 1).mean(0)
    return {"scores": out}
