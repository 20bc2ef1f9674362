"""The paged-cache operators, in their plain form and through the framework's entry points, over the cases that stand for their use.

Three operators of a server that answers many requests about one long document, its key/value cache kept in pages of 64 tokens:
``plan`` (block tables and slot maps from request lengths), ``append`` (new key/value rows into their slots) and ``decode`` (the
attention of a batch whose requests share a long prefix and have tokens of their own).
"""
import math

import torch

own = False

PAGE = 64
BF16 = torch.bfloat16


# ---- cases ----
def listed():
    return [
        # one decode step of a serving loop: every request adds one token, a few finish
        {"name": "plan_step_b64", "op": "plan", "B": 64, "prompts": 0, "prompt": 0, "done": 3, "cached": 4000},
        # the same for a large padded batch, ragged histories
        {"name": "plan_step_b1500", "op": "plan", "B": 1500, "prompts": 0, "prompt": 0, "done": 40, "cached": 9001},
        # prompts and running requests in one step
        {"name": "plan_prompts_b256", "op": "plan", "B": 256, "prompts": 32, "prompt": 8192, "done": 16, "cached": 20000},
        # one token for each of 64 running requests, 8 key heads
        {"name": "append_step_n64", "op": "append", "n": 64, "Hkv": 8, "D": 128, "G": 1, "run": 1},
        # an odd number of prompt rows, sliced from a fused projection with grouped heads
        {"name": "append_prompt_n3001", "op": "append", "n": 3001, "Hkv": 4, "D": 64, "G": 4, "run": 300},
        # the rows of one long prompt chunk
        {"name": "append_prompt_n32768", "op": "append", "n": 32768, "Hkv": 8, "D": 128, "G": 1, "run": 32768},
        # a short system prompt and a handful of young requests: latency
        {"name": "decode_p1000_b4", "op": "decode", "B": 4, "H": 4, "Hkv": 4, "Tq": 1, "D": 64, "prefix": 1000, "own": 60, "idle": 0},
        # a batch of questions about a 32K document
        {"name": "decode_p32768_b16", "op": "decode", "B": 16, "H": 8, "Hkv": 8, "Tq": 1, "D": 128, "prefix": 32768, "own": 700, "idle": 1},
        # many requests, 16 query heads to a key head: the prefix is a wide matrix product
        {"name": "decode_p65536_b64_g16", "op": "decode", "B": 64, "H": 32, "Hkv": 2, "Tq": 1, "D": 128, "prefix": 65536, "own": 1500, "idle": 5},
        # drafted tokens checked together, ragged everywhere, grouped heads
        {"name": "decode_p20011_b24_q4", "op": "decode", "B": 24, "H": 16, "Hkv": 4, "Tq": 4, "D": 64, "prefix": 20011, "own": 3000, "idle": 2},
        # long answers after a short shared prompt: the requests' own pages dominate
        {"name": "decode_p2048_b32_own16k", "op": "decode", "B": 32, "H": 16, "Hkv": 4, "Tq": 1, "D": 128, "prefix": 2048, "own": 16384, "idle": 0},
        # a million-token document
        {"name": "decode_p1m_b8", "op": "decode", "B": 8, "H": 8, "Hkv": 8, "Tq": 1, "D": 128, "prefix": 1048576, "own": 1000, "idle": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "decode", "decode"])
    if op == "plan":
        B = _log(rng, 1, 3000)
        prompts = min(B, rng.choice([0, 0, 1, B // 8, B // 3]), 40)
        done = rng.randint(0, (B - prompts) // 8)
        return {"op": op, "B": B, "prompts": prompts, "prompt": _log(rng, 20, 8192) if prompts else 0, "done": done,
                "cached": _log(rng, 50, 20000)}
    if op == "append":
        n = _log(rng, 1, 32768)
        return {"op": op, "n": n, "Hkv": rng.choice([1, 2, 4, 8]), "D": rng.choice([64, 128]), "G": rng.choice([1, 2, 4, 8]),
                "run": rng.choice([1, rng.randint(1, n), n])}
    Hkv, G, Tq = rng.choice([1, 2, 4, 8]), rng.choice([1, 1, 2, 4, 8, 16]), rng.choice([1, 1, 1, 2, 3, 5])
    B = max(1, min(_log(rng, 1, 96), 4096 // (Hkv * G * Tq)))
    rows = B * Hkv * G * Tq
    return {"op": op, "B": B, "H": Hkv * G, "Hkv": Hkv, "Tq": Tq, "D": rng.choice([64, 128, 128]),
            "prefix": rng.choice([0, _log(rng, 1, 64), *[_log(rng, 64, min(300000, (1 << 27) // rows))] * 6]),
            "own": _log(rng, 5, min(12000, (1 << 22) // rows + 5)), "idle": rng.randint(0, B // 4)}


def _spread(n, top):
    """n lengths from 1 to top, most of them short: what a batch of running requests looks like."""
    return [1 + int((top - 1) * ((i + 0.5) / n) ** 2) for i in range(n)]


def _pages(tokens):
    return (tokens + PAGE - 1) // PAGE


def _plan_lengths(case):
    """(cached, new) of each request, before they are put in the seed's order."""
    B, P, done = case["B"], case["prompts"], case["done"]
    new = _spread(P, case["prompt"]) + [-1] * done + [1] * (B - P - done)
    return [0] * P + (_spread(B - P, case["cached"])[::-1] if B > P else []), new


def _own_lengths(case):
    live = case["B"] - case["idle"]
    return [max(case["Tq"], x) for x in _spread(live, case["own"])] + [-1] * case["idle"]


# ---- inputs ----
def _order(n, gen):
    return torch.randperm(n, generator=gen)


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed)
    dev = torch.Generator(device="cuda").manual_seed(seed)
    return {"op": case["op"], **{"plan": _prepare_plan, "append": _prepare_append, "decode": _prepare_decode}[case["op"]](case, gen, dev)}


def _prepare_plan(case, gen, dev):
    cached, new = (torch.tensor(x) for x in _plan_lengths(case))
    order = _order(case["B"], gen)
    cached, new = cached[order], new[order]
    after = cached + new.clamp(min=0)
    held, width = _pages(cached), int(_pages(int(after.max()))) + 2
    F = int(_pages(after).sum()) + 17
    ids = _order(F, gen).to(torch.int32)
    table = torch.full((case["B"], width), -1, dtype=torch.int32)
    has = torch.arange(width)[None] < held[:, None]
    used = int(held.sum())
    table[has] = ids[:used]
    taken = F + int(torch.randint(0, F, (1,), generator=gen))  # a pool in mid-life: its ring has wrapped
    ring = torch.full((F,), -1, dtype=torch.int32)
    ring[(taken + torch.arange(F - used)) % F] = ids[used:]
    tokens = int(new.clamp(min=0).sum())
    return {"cache_len": cached.cuda(), "new_len": new.to(torch.int32).cuda(), "table": table.cuda(), "ring": ring.cuda(),
            "pool": torch.tensor([taken, taken + F - used, 0]).cuda(), "pool_out": torch.zeros(3, dtype=torch.int64).cuda(),
            "max_tokens": tokens + 5}


def _prepare_append(case, gen, dev):
    n, Hkv, D, run = case["n"], case["Hkv"], case["D"], case["run"]
    heads = case["G"] * Hkv
    qkv = torch.randn((n, heads + 2 * Hkv, D), generator=dev, device="cuda", dtype=torch.float32).to(BF16)
    runs = -(-n // run)
    per = _pages(run)
    pages = runs * per + 3
    ids = _order(pages, gen)[:runs * per].view(runs, per)
    i = torch.arange(n)
    # a run of one token sits somewhere in its page; a longer one starts at a page
    at = torch.randint(0, PAGE, (n,), generator=gen) if run == 1 else i % run
    slots = ids[i // run, at // PAGE] * PAGE + at % PAGE
    slots[_order(n, gen)[:n // 50]] = -1  # rows of refused requests, and padding
    pool = torch.randn((2, pages, Hkv, PAGE, D), generator=dev, device="cuda", dtype=torch.float32).to(BF16)
    return {"K": qkv[:, heads:heads + Hkv], "V": qkv[:, heads + Hkv:], "slots": slots.cuda(), "Kp": pool[0], "Vp": pool[1]}


def _prepare_decode(case, gen, dev):
    B, H, Hkv, Tq, D = (case[k] for k in ("B", "H", "Hkv", "Tq", "D"))
    lens = torch.tensor(_own_lengths(case))[_order(B, gen)]
    npre, held = _pages(case["prefix"]), _pages(lens.clamp(min=0))
    width = int(held.max()) + 1
    total = npre + int(held.sum()) + 2
    ids = _order(total, gen).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    table[torch.arange(width)[None] < held[:, None]] = ids[npre:npre + int(held.sum())]
    pool = torch.empty((2, total, Hkv, PAGE, D), device="cuda", dtype=BF16).normal_(generator=dev)
    q = torch.randn((B, H, Tq, D), generator=dev, device="cuda", dtype=torch.float32).to(BF16)
    return {"q": q, "Kp": pool[0], "Vp": pool[1], "prefix_table": ids[:npre].clone().cuda(), "table": table.cuda(),
            "prefix_len": torch.tensor([case["prefix"]]).cuda(), "own_len": lens.cuda()}


# ---- one pass ----
def run(state):
    if own:
        from ultra_long_context_b200 import hsa
        if state["op"] == "plan":
            cu, slots, total = hsa.hsa_page_plan(state["cache_len"], state["new_len"], state["table"], state["ring"], state["pool"],
                                                 state["max_tokens"], pool_out=state["pool_out"])
            return {"cu": cu, "slots": slots, "total": total, "table": state["table"], "ring": state["ring"], "pool": state["pool_out"]}
        if state["op"] == "append":
            hsa.hsa_page_append(state["K"], state["V"], state["slots"], state["Kp"], state["Vp"])
            return {"Kp": state["Kp"], "Vp": state["Vp"]}
        out, lse = hsa.hsa_prefix_decode(state["q"], state["Kp"], state["Vp"], state["prefix_table"], state["prefix_len"], state["table"],
                                         state["own_len"])
        return {"out": out, "lse": lse}
    return {"plan": _plain_plan, "append": _plain_append, "decode": _plain_decode}[state["op"]](state)


def _plain_plan(s):
    cached, new, table, ring, pool = s["cache_len"], s["new_len"].long(), s["table"], s["ring"], s["pool"]
    (B, width), F, T = table.shape, ring.numel(), s["max_tokens"]
    add = new.clamp(min=0)
    ends = add.cumsum(0)
    held, after = (cached + 63) // PAGE, (cached + add + 63) // PAGE
    known = (cached >= 0) & (cached <= width * PAGE)
    fits = known & (new > 0) & (after <= width) & (ends <= T)
    need = torch.where(fits, after - held, 0)
    upto = need.cumsum(0)
    admitted = fits & ((need == 0) | (upto <= pool[1] - pool[0]))
    leaves = known & (new < 0)
    total = torch.where(admitted, cached + add, torch.where(leaves, 0, cached))
    # tokens: request, position, page
    t = torch.arange(T, device=cached.device)
    b = torch.searchsorted(ends, t, right=True).clamp(max=B - 1)
    pos = cached[b] + t - (ends - add)[b]
    page = pos // PAGE
    old = table[b, page.clamp(0, width - 1)].long()
    fresh = ring[(pool[0] + (upto - need)[b] + page - held[b]) % F].long()
    page_id = torch.where(page < held[b], old, fresh)
    live = admitted[b] & (t < ends[-1])
    slots = torch.where(live, page_id * PAGE + pos % PAGE, -1)
    # table entries of new pages; a spare place takes what is not written
    spare = B * width
    place = torch.where(live & (page >= held[b]), b * width + page, spare)
    table = torch.cat([table.view(-1), table.new_zeros(1)]).index_put((place,), page_id.to(torch.int32))[:spare].view(B, width)
    # pages of finished requests to the ring's end
    back = torch.where(leaves, held, 0)
    j = torch.arange(width, device=cached.device)[None]
    at = (pool[1] + (back.cumsum(0) - back)[:, None] + j) % F
    at = torch.where(j < back[:, None], at, F)
    ring = torch.cat([ring, ring.new_zeros(1)]).index_put((at.view(-1),), s["table"].view(-1))[:F]
    used = torch.where(admitted, need, 0).sum()
    refused = ((new > 0) & ~admitted).sum() + ((new <= 0) & ~known).sum()
    cu = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
    return {"cu": cu, "slots": slots, "total": total, "table": table, "ring": ring, "pool": torch.stack([pool[0] + used, pool[1] + back.sum(), refused])}


def _plain_append(s):
    ok = s["slots"] >= 0
    page, at = s["slots"][ok] // PAGE, s["slots"][ok] % PAGE
    s["Kp"][page, :, at] = s["K"][ok]
    s["Vp"][page, :, at] = s["V"][ok]
    return {"Kp": s["Kp"], "Vp": s["Vp"]}


def _plain_decode(s):
    q, Kp, Vp = s["q"].float(), s["Kp"], s["Vp"]
    B, H, Tq, D = q.shape
    Hkv = Kp.shape[1]
    G = H // Hkv
    q = q.view(B, Hkv, G * Tq, D) / math.sqrt(D)
    own_len, i = s["own_len"], torch.arange(Tq, device=q.device).repeat(G)
    last = own_len[:, None] - Tq + i[None]  # position behind the prefix; it sees the tokens up to itself
    live = (own_len >= 0)[:, None]
    see_own = torch.where(live, (last + 1).clamp(min=0), 0)
    see_pre = torch.where(live, (s["prefix_len"] + (last + 1).clamp(max=0)).clamp(min=0), 0)
    # the shared pages, once for all requests
    kp, vp = (x[s["prefix_table"].long()].float().transpose(0, 1).reshape(Hkv, -1, D) for x in (Kp, Vp))
    qp = q.transpose(0, 1).reshape(Hkv, B * G * Tq, D)
    sp = (qp @ kp.transpose(1, 2)).view(Hkv, B, G * Tq, -1).transpose(0, 1)
    sp = sp.masked_fill(torch.arange(kp.shape[1], device=q.device) >= see_pre[:, None, :, None], -math.inf)
    # each request's own
    table = s["table"].long().clamp(min=0)
    ko, vo = (x[table].float().transpose(1, 2).reshape(B, Hkv, -1, D) for x in (Kp, Vp))
    so = (q @ ko.transpose(2, 3)).masked_fill(torch.arange(ko.shape[2], device=q.device) >= see_own[:, None, :, None], -math.inf)
    top = so.amax(-1, keepdim=True)
    top = torch.maximum(top, sp.amax(-1, keepdim=True)) if sp.shape[-1] else top
    top = torch.where(top == -math.inf, 0.0, top)
    pp, po = torch.exp(sp - top), torch.exp(so - top)
    z = pp.sum(-1, keepdim=True) + po.sum(-1, keepdim=True)
    o = po @ vo + (pp.transpose(0, 1).reshape(Hkv, B * G * Tq, -1) @ vp).view(Hkv, B, G * Tq, D).transpose(0, 1)
    out = torch.where(z > 0, o / z, 0.0)
    return {"out": out.reshape(B, H, Tq, D).to(BF16), "lse": (top + torch.log(z)).reshape(B, H, Tq)}


# ---- what a pass cannot do without ----
def work(case):
    if case["op"] == "plan":
        cached, new = _plan_lengths(case)
        tokens = sum(x for x in new if x > 0)
        fresh = sum(_pages(c + n) - _pages(c) for c, n in zip(cached, new) if n > 0)
        back = sum(_pages(c) for c, n in zip(cached, new) if n < 0)
        return {"bytes": case["B"] * (8 + 4 + 8 + 4) + 8 * (tokens + 5) + 8 * (fresh + back) + 4 * sum(1 for c, n in zip(cached, new) if n > 0 and c % PAGE) + 48,
                "flops": 0}
    if case["op"] == "append":
        rows = case["n"] - case["n"] // 50
        return {"bytes": 2 * 2 * rows * case["Hkv"] * case["D"] * 2 + 8 * case["n"], "flops": 0}
    B, H, Hkv, Tq, D = (case[k] for k in ("B", "H", "Hkv", "Tq", "D"))
    lens = [x for x in _own_lengths(case) if x > 0]
    keys = case["prefix"] + sum(lens)
    seen = sum(case["prefix"] * Tq + sum(max(0, n - Tq + i + 1) for i in range(Tq)) for n in lens)
    return {"bytes": keys * Hkv * D * 4 + B * H * Tq * (D * 4 + 4) + 4 * (_pages(case["prefix"]) + sum(_pages(n) for n in lens)) + 8 * B,
            "flops": 4 * D * H * seen}


# ---- the definitions in 64 bits ----
def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "append": _exact_append, "decode": _exact_decode}[case["op"]](s)


def _exact_plan(s):
    """The serving loop's bookkeeping, request by request."""
    table, ring = s["table"].cpu().tolist(), s["ring"].cpu().tolist()
    width, F, T = len(table[0]), len(ring), s["max_tokens"]
    taken, given, refused = s["pool"].cpu().tolist()
    avail, asked, refused, at = given - taken, 0, 0, 0
    start = taken
    cu, slots, total = [0], [-1] * T, []
    for b, (c, n) in enumerate(zip(s["cache_len"].tolist(), s["new_len"].tolist())):
        known = 0 <= c <= width * PAGE
        if n < 0 and known:
            for page in table[b][:-(-c // PAGE)]:
                ring[given % F] = page
                given += 1
            total.append(0)
        elif n > 0:
            need = -(-(c + n) // PAGE) - -(-c // PAGE)
            fits = known and c + n <= width * PAGE and at + n <= T
            asked += need if fits else 0
            if fits and (need == 0 or asked <= avail):
                for k in range(need):
                    table[b][-(-c // PAGE) + k] = ring[(start + asked - need + k) % F]
                taken += need
                for i in range(n):
                    slots[at + i] = table[b][(c + i) // PAGE] * PAGE + (c + i) % PAGE
                total.append(c + n)
            else:
                refused += 1
                total.append(c)
            at += n
        else:
            refused += not known
            total.append(c)
        cu.append(at)
    as_int = lambda x, t=torch.int64: torch.tensor(x, dtype=t)  # noqa: E731
    return {"cu": as_int(cu, torch.int32), "slots": as_int(slots), "total": as_int(total), "table": as_int(table, torch.int32),
            "ring": as_int(ring, torch.int32), "pool": as_int([taken, given, refused])}


def _exact_append(s):
    """Rows to slots, as one long list of rows."""
    res = {}
    for name, pool, rows in (("Kp", s["Kp"], s["K"]), ("Vp", s["Vp"], s["V"])):
        flat = pool.transpose(1, 2).reshape(-1, *rows.shape[1:]).double()
        for lo in range(0, rows.shape[0], 8192):
            part = s["slots"][lo:lo + 8192]
            keep = torch.nonzero(part >= 0)[:, 0]
            flat.index_copy_(0, part[keep], rows[lo:lo + 8192][keep].double())
        res[name] = flat.view(pool.shape[0], PAGE, *rows.shape[1:]).transpose(1, 2).contiguous()
    return res


def _exact_decode(s):
    """Softmax attention of each request over its whole sequence, the prefix's tokens and then its own, head by head."""
    q, Kp, Vp = s["q"], s["Kp"], s["Vp"]
    B, H, Tq, D = q.shape
    Hkv = Kp.shape[1]
    G, plen = H // Hkv, int(s["prefix_len"])
    out = torch.zeros((B, H, Tq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((B, H, Tq), -math.inf, dtype=torch.float64, device=q.device)
    lens = s["own_len"].tolist()
    for h in range(Hkv):
        kp, vp = (x[s["prefix_table"].long(), h].reshape(-1, D)[:plen].double() for x in (Kp, Vp))
        for b in range(B):
            if lens[b] < 0:
                continue
            pages = s["table"][b, :-(-lens[b] // PAGE)].long()
            ko, vo = (x[pages, h].reshape(-1, D)[:lens[b]].double() for x in (Kp, Vp))
            rows = q[b, h * G:(h + 1) * G].double().reshape(G * Tq, D)
            logits = torch.cat([rows @ kp.T, rows @ ko.T], 1) * D ** -0.5
            pos = torch.arange(plen + lens[b], device=q.device)
            seen = plen + lens[b] - Tq + torch.arange(Tq, device=q.device).repeat(G)
            logits[pos[None] > seen[:, None]] = -math.inf
            any_seen = seen >= 0
            z = torch.logsumexp(logits, 1)
            p = torch.where(any_seen[:, None], torch.exp(logits - z[:, None]), 0.0)
            out[b, h * G:(h + 1) * G] = (p[:, :plen] @ vp + p[:, plen:] @ vo).view(G, Tq, D)
            lse[b, h * G:(h + 1) * G] = z.view(G, Tq)
    return {"out": out, "lse": lse}
