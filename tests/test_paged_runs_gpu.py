"""The shared-prefix decode over long runs: segments of more than 32 tiles of keys, whose partial sums, references and rings
of buffers go round, in both kernels and in the launch order that a user's call has. The plain form here runs in fp64 on the GPU,
and page ids repeat in the prefix's table, so that a long prefix needs a small pool only. At the end, large calls of the plan and the
append."""
import math

import numpy as np
import pytest
import torch

from oracle import paged
from ultra_long_context_b200 import hsa

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16
TILE = 128   # keys that the kernels take at a time


def _tokens(pool, ids, n, h):
    """The first n tokens of one key head in the pages `ids` [..., pages], fp64, and whether they are there."""
    ok = (ids >= 0) & (ids < pool.shape[0])
    rows = pool[torch.where(ok, ids, 0), h].double().flatten(-3, -2)
    there = ok.repeat_interleave(64, -1) & (torch.arange(rows.shape[-2], device=DEV) < n)
    return torch.where(there[..., None], rows, 0.0), there


def plain_decode(q, Kp, Vp, pre, P, table, own, run=0):
    """Row by row over the visible tokens, fp64. `run` > 0: also the share of (row, run of `run` prefix tiles) in which a tile
    after the first holds a logit that is over the one of the run's first key by more than 2^64."""
    B, H, Tq, D = q.shape
    Hkv = Kp.shape[1]
    G = H // Hkv
    pre, table, own = pre.long(), table.long(), own.clamp(max=table.shape[1] * 64)
    P = min(max(P, 0), 64 * pre.numel())
    pre = pre[:-(-P // 64)]
    scale = D ** -0.5
    res = {k: torch.zeros((B, H, Tq) + ((D,) if k in ("out", "mean_abs") else ()), dtype=torch.float64, device=DEV)
           for k in ("out", "mean_abs", "lse", "reach", "keys")}
    moved = []
    last = P + own[:, None] - Tq + torch.arange(Tq, device=DEV)                  # [B, Tq]: the last token that a row sees
    last = torch.where(own[:, None] < 0, -1, last)
    step = max(1, (1 << 27) // (G * Tq * max(1, P)))                              # requests at a time
    for h in range(Hkv):
        kp, there = _tokens(Kp, pre, P, h)
        vp = _tokens(Vp, pre, P, h)[0]
        for b in range(0, B, step):
            e = min(B, b + step)
            rows = q[b:e, h * G:(h + 1) * G].double()                             # [b, G, Tq, D]
            ko, owned = _tokens(Kp, table[b:e], own[b:e, None], h)
            vo = _tokens(Vp, table[b:e], own[b:e, None], h)[0]
            see_p = there & (torch.arange(kp.shape[0], device=DEV) <= last[b:e, None, :, None])
            see_o = owned[:, None, None] & (P + torch.arange(ko.shape[1], device=DEV) <= last[b:e, None, :, None])
            sp = scale * rows @ kp.T
            so = scale * rows @ ko.transpose(1, 2)[:, None]
            if run:
                first = sp[..., ::run * TILE]
                top = torch.where(see_p, sp, -math.inf)
                top[..., torch.arange(top.shape[-1], device=DEV) // TILE % run == 0] = -math.inf
                pad = -top.shape[-1] % (run * TILE)
                top = torch.nn.functional.pad(top, (0, pad), value=-math.inf).unflatten(-1, (-1, run * TILE)).amax(-1)
                moved.append((((top - first) * math.log2(math.e) > 64)).double().mean())
            s = torch.cat([torch.where(see_p, sp, -math.inf), torch.where(see_o, so, -math.inf)], -1)
            lse = torch.logsumexp(s, -1)
            w = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None])
            wp, wo = w[..., :kp.shape[0]], w[..., kp.shape[0]:]
            at = np.s_[b:e, h * G:(h + 1) * G]
            res["out"][at] = wp @ vp + wo @ vo[:, None]
            res["mean_abs"][at] = wp @ vp.abs() + wo @ vo.abs()[:, None]
            res["lse"][at] = lse
            far = torch.cat([torch.where(see_p, rows.abs() @ kp.abs().T, 0.0), torch.where(see_o, rows.abs() @ ko.abs().transpose(1, 2)[:, None], 0.0)], -1)
            res["reach"][at] = scale * far.amax(-1)
            res["keys"][at] = (see_p.expand_as(sp).sum(-1) + see_o.expand_as(so).sum(-1)).double()
            del s, w, wp, wo, far, sp, so, see_p
    ref = {k: v.cpu().numpy() for k, v in res.items()}
    ref["moved"] = float(torch.stack(moved).mean()) if moved else 0.0
    return ref


def run_case(seed, B, H, Hkv, D, prefix, own, Tq=1, shape="flat", pages=48, bad=()):
    """A prefix of `pages` pages in an order that repeats them. shape: flat (normal logits); up and down (logits that climb, or
    fall, by 2^160 over 20 tiles and jump back, for a third of the rows; that do the opposite for another third).
    bad: places of the prefix's table that hold no page."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    own = torch.as_tensor(own).expand(B).clone()
    held = (own.clamp(min=0) + 63) // 64
    npre, width = (prefix + 63) // 64, int(held.max()) + 1
    total = pages + int(held.sum()) + 2
    pool = torch.randn(2, total, Hkv, 64, D, generator=g, device=DEV)
    q = torch.randn(B, H, Tq, D, generator=g, device=DEV)
    table = torch.full((B, width), -1, dtype=torch.int32)
    has = torch.arange(width)[None] < held[:, None]
    table[has] = (pages + 1 + torch.arange(int(held.sum()))).to(torch.int32)
    if shape == "flat":
        pre = torch.randint(0, pages, (npre,), generator=cpu)
    else:
        # the logit of a row with sign 1 in page p: 2^160 in all, by the first column alone, beside half of the noise
        assert pages >= 40
        level = torch.arange(40, device=DEV) / 39 * 160 / math.log2(math.e)
        pool[0, :40] *= 0.5
        pool[0, :40, :, :, 0] = (level * D ** 0.5 / 8)[:, None, None]
        q[..., 0] = 8.0 * (torch.arange(B * H * Tq, device=DEV).view(B, H, Tq) % 3 - 1)
        pre = torch.arange(npre) % 40
        if shape == "down":
            pre = 39 - pre
    last = pages    # the prefix's last page is one of its own: what follows its tokens is NaN
    if prefix % 64:
        pre[-1] = last
        pool[:, last, :, prefix % 64:] = math.nan
    for b in range(B):
        if own[b] > 0 and own[b] % 64:
            pool[:, int(table[b, held[b] - 1]), :, int(own[b]) % 64:] = math.nan
    for k, p in enumerate(bad):
        pre[p] = (-1, total, 2**31 - 1, -2**31)[k % 4]
    pool = pool.to(BF16)
    return q.to(BF16), pool[0].contiguous(), pool[1].contiguous(), pre.to(torch.int32).to(DEV), prefix, table.to(DEV), own.to(DEV)


def workspace(q, Kp, pre, table):
    B, H, Tq, D = q.shape
    n = hsa.hsa_prefix_decode_workspace_size(B, H, Kp.shape[1], D, pre.numel(), table.shape[1], Tq)
    ws = torch.empty(n + 256, dtype=torch.uint8, device=DEV)
    return ws[-ws.data_ptr() % 256:]


def division(ws):
    """How the last call cut its prefix: (tiles, tiles per segment, segments), which stand behind the workspace's first block."""
    _, _, tiles, run, _, items = ws[256:256 + 24].view(torch.int32).tolist()
    return tiles, run, items


def kernels_of(call):
    hsa.hsa_profile_enable(True)
    try:
        res = call()
        torch.cuda.synchronize()
        return res, hsa.hsa_profile_summary()
    finally:
        hsa.hsa_profile_enable(False)


def check(case, wide, room=0, min_run=33, moved=False):
    q, Kp, Vp, pre, P, table, own = case
    D = q.shape[-1]
    if room:
        pre = torch.cat([pre, torch.full((room,), -1, dtype=torch.int32, device=DEV)])
    ws = workspace(q, Kp, pre, table)
    plen = torch.tensor([P], device=DEV)

    def call():
        return hsa.hsa_prefix_decode(q, Kp, Vp, pre, plen, table, own, workspace=ws)

    out, lse = call()     # as a user calls it, the kernels starting under one another
    hsa.hsa_workspace_status(ws)
    tiles, run, items = division(ws)
    assert tiles == -(-P // TILE) and run >= min_run, (tiles, run, items)
    again, names = kernels_of(call)
    assert ("prefix_wide" in names) == wide, names
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    ref = plain_decode(q, Kp, Vp, pre, P, table, own, run=run if moved else 0)
    if moved:
        assert ref["moved"] > 0.05, ref["moved"]
    tol, tol_lse = paged.prefix_tolerance(ref, D)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    none = ref["keys"] == 0
    assert (got[none] == 0).all() and np.isneginf(got_lse[none]).all()
    off = np.abs(got - ref["out"]) - tol
    assert np.isfinite(got).all() and (off <= 0).all(), (int((off > 0).sum()), float(off.max()), np.argwhere(off > 0)[:4].tolist())
    off = np.abs(got_lse[~none] - ref["lse"][~none]) - tol_lse[~none]
    assert (off <= 0).all(), (int((off > 0).sum()), float(off.max()))
    return run, items


# Row groups of the few-rows kernel (at most 64 rows a key head, by eights over two warpgroups); 16, 32 and 64 columns.
FEW = [dict(B=3, H=2, Hkv=2), dict(B=5, H=2, Hkv=1), dict(B=16, H=8, Hkv=8), dict(B=9, H=6, Hkv=2), dict(B=32, H=4, Hkv=4), dict(B=31, H=4, Hkv=2),
       dict(B=64, H=2, Hkv=2), dict(B=7, H=6, Hkv=2, Tq=3)]
# Row groups of the wide kernel: one stream an item (up to 128 rows), two, and groups that end early
WIDE = [dict(B=65, H=2, Hkv=2), dict(B=25, H=16, Hkv=4), dict(B=128, H=2, Hkv=2), dict(B=43, H=6, Hkv=2), dict(B=64, H=16, Hkv=4),
        dict(B=75, H=8, Hkv=2), dict(B=48, H=16, Hkv=2), dict(B=20, H=12, Hkv=2, Tq=3)]


def long_prefix(c, D, wide):
    """Tokens that make runs of more than 32 tiles over 148 SMs, an odd number, not whole pages."""
    rows = c["B"] * (c["H"] // c["Hkv"]) * c.get("Tq", 1)
    units = c["Hkv"] * (-(-rows // 256) if wide else 1)
    return 150 // units * 37 * TILE + 61


def own_of(c, seed):
    own = torch.randint(0, 300, (c["B"],), generator=torch.Generator().manual_seed(seed))
    own[::7] = 0
    own[3::11] = -1
    return own


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", ["flat", "up", "down"])
@pytest.mark.parametrize("c", FEW)
def test_few_rows_over_long_runs(c, shape, D):
    P = long_prefix(c, D, False)
    check(run_case(51, D=D, prefix=P, own=own_of(c, 1), shape=shape, **c), wide=False, moved=shape != "flat")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", ["flat", "up", "down"])
@pytest.mark.parametrize("c", WIDE)
def test_wide_batches_over_long_runs(c, shape, D):
    P = long_prefix(c, D, True)
    check(run_case(52, D=D, prefix=P, own=own_of(c, 2), shape=shape, **c), wide=True, room=60000, moved=shape != "flat")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("c,wide", [(FEW[4], False), (WIDE[5], True)])
def test_values_up_to_their_bound(c, wide, D):
    """|V| just below 2^28 with logits that climb over the references by as much as they may."""
    case = list(run_case(57, D=D, prefix=long_prefix(c, D, wide), own=own_of(c, 6), shape="up", **c))
    case[2] = (case[2].float() * 2.0**26).clamp(-2.0**27.9, 2.0**27.9).to(BF16)
    check(case, wide=wide, room=60000 if wide else 0, moved=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", ["flat", "up"])
@pytest.mark.parametrize("c,wide", [(FEW[2], False), (FEW[4], False), (WIDE[1], True), (WIDE[4], True), (WIDE[5], True)])
def test_bad_pages_late_in_long_runs(c, wide, shape, D):
    """Places without a page in every part of the runs: their first pages, the second of a tile, whole tiles, behind the 16 tiles
    whose pages are looked up together, the last one."""
    P = long_prefix(c, D, wide)
    n = -(-P // 64)
    bad = sorted({*range(0, n, 149), *range(1, n, 83), *range(66, n, 132), *range(67, n, 132), *range(34, n, 97), n - 1})
    check(run_case(53, D=D, prefix=P, own=own_of(c, 3), shape=shape, bad=bad, **c), wide=wide, room=60000 if wide else 0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", ["flat", "up", "down"])
@pytest.mark.parametrize("B,Hkv,rows", [(80, 32, 32), (300, 64, 2)])
def test_more_segments_than_sms(B, Hkv, rows, shape, D):
    """Several segments one after the other on an SM, their queries and sums in turn in the same buffers: 2560 rows in groups of
    256 (two streams a tile) and 600 (the last group 88, one stream a tile)."""
    c = dict(B=B, H=Hkv * rows, Hkv=Hkv)
    run, items = check(run_case(54, D=D, prefix=35 * TILE - 17, own=own_of(c, 4), shape=shape, **c), wide=True, room=60000, min_run=1)
    assert items > 148


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("wide", [False, True])
def test_calls_back_to_back_equal_the_plain_form(wide, D):
    """Sixty calls without a pause, over queries and lengths that the stream changes between them; each of the answers as when it
    is computed alone, and as the plain form has it."""
    c = WIDE[5] if wide else FEW[4]
    q, Kp, Vp, pre, P, table, own = run_case(55, D=D, prefix=9000, own=own_of(c, 5), **c)
    pre = torch.cat([pre, torch.full((60000 if wide else 0,), -1, dtype=torch.int32, device=DEV)])
    ws = workspace(q, Kp, pre, table)
    lens = [(9000, own), (4097, own.clamp(max=64)), (1, own.clamp(max=1)), (8999, own.flip(0).minimum(own))]
    queries = [torch.roll(q, k, 0) for k in range(3)]
    plens = [torch.tensor([n], device=DEV) for n, _ in lens]
    x, plen, mine = torch.empty_like(q), torch.empty_like(plens[0]), torch.empty_like(own)
    torch.cuda.synchronize()
    got = []
    for k in range(60):
        x.copy_(queries[k % 3])
        plen.copy_(plens[k % 4])
        mine.copy_(lens[k % 4][1])
        got.append(hsa.hsa_prefix_decode(x, Kp, Vp, pre, plen, table, mine, workspace=ws))
    torch.cuda.synchronize()
    for k in range(12):
        P, o = lens[k % 4]
        (out, lse), names = kernels_of(lambda: hsa.hsa_prefix_decode(queries[k % 3], Kp, Vp, pre, plens[k % 4], table, o))
        assert ("prefix_wide" in names) == wide
        for n in range(k, 60, 12):
            assert torch.equal(got[n][0], out) and torch.equal(got[n][1], lse), n
        ref = plain_decode(queries[k % 3], Kp, Vp, pre, P, table, o)
        tol, tol_lse = paged.prefix_tolerance(ref, D)
        some = ref["keys"] > 0
        assert (np.abs(out.double().cpu().numpy() - ref["out"]) <= tol).all()
        assert (np.abs(lse.double().cpu().numpy()[some] - ref["lse"][some]) <= tol_lse[some]).all()


@pytest.mark.parametrize("graph", [False, True])
def test_serving_loop_of_a_wide_batch_without_a_pause(graph):
    """Steps of plan, append and decode whose prefix goes to the wide kernel, in one stream with nothing between them: the early
    start of the few-rows kernel under the wide one must see what the append before them wrote."""
    B, H, Hkv, D, width, T = 70, 8, 2, 128, 6, 70
    F, steps, doc = 900, 12, 5000
    gen = torch.Generator(device=DEV).manual_seed(7)
    Kp, Vp = (torch.full((F, Hkv, 64, D), math.nan, dtype=BF16, device=DEV) for _ in range(2))
    ring = torch.randperm(F, generator=torch.Generator().manual_seed(2)).to(torch.int32).to(DEV)
    pool = torch.tensor([0, F, 0], device=DEV)
    doc_table = torch.full((1, 60000), -1, dtype=torch.int32, device=DEV)
    kv = torch.randn(2, doc, Hkv, D, generator=gen, device=DEV).to(BF16)
    _, slots, doc_len = hsa.hsa_page_plan(torch.zeros(1, dtype=torch.int64, device=DEV), torch.tensor([doc], dtype=torch.int32, device=DEV),
                                          doc_table, ring, pool, doc)
    hsa.hsa_page_append(kv[0], kv[1], slots, Kp, Vp)
    lens = torch.zeros(B, dtype=torch.int64, device=DEV)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    new = torch.ones(B, dtype=torch.int32, device=DEV)
    rows = torch.randn(steps, 2, T, Hkv, D, generator=gen, device=DEV).to(BF16)
    qs = torch.randn(steps, B, H, D, generator=gen, device=DEV).to(BF16)
    row, q = torch.empty_like(rows[0]), torch.empty_like(qs[0])
    cu, slots = torch.empty(B + 1, dtype=torch.int32, device=DEV), torch.empty(T, dtype=torch.int64, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(B, H, device=DEV)
    ws = workspace(q[:, :, None], Kp, doc_table, table)

    def step():
        hsa.hsa_page_plan(lens, new, table, ring, pool, T, cu_new=cu, slots=slots, total_len=lens)
        hsa.hsa_page_append(row[0], row[1], slots, Kp, Vp)
        hsa.hsa_prefix_decode(q, Kp, Vp, doc_table.view(-1), doc_len, table, lens, out=out, lse=lse, workspace=ws)

    torch.cuda.synchronize()
    if graph:
        recorded = torch.cuda.CUDAGraph()
        with torch.cuda.graph(recorded):
            step()
    got = []
    for k in range(steps):
        row.copy_(rows[k])
        q.copy_(qs[k])
        recorded.replay() if graph else step()
        got.append((out.clone(), lse.clone()))
    hsa.hsa_workspace_status(ws)
    assert lens.tolist() == [steps] * B and int(pool[2]) == 0
    for k in (0, 1, 5, steps - 1):
        ref = plain_decode(qs[k][:, :, None], Kp, Vp, doc_table.view(-1)[:79], doc, table, torch.full((B,), k + 1, device=DEV))
        tol, tol_lse = paged.prefix_tolerance(ref, D)
        assert (np.abs(got[k][0].double().cpu().numpy()[:, :, None] - ref["out"]) <= tol).all()
        assert (np.abs(got[k][1].double().cpu().numpy()[:, :, None] - ref["lse"]) <= tol_lse).all()


@pytest.mark.parametrize("limit,after,arrive,ok", [(50000, 10000, 1, True), (50000, 0, 1, True), (4000, 0, 0, False), (1, 0, 0, False)])
def test_timed_wait_ends_with_the_arrival_or_at_its_limit(limit, after, arrive, ok):
    ws = torch.empty(4096, dtype=torch.uint8, device=DEV)
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ev[0].record()
    assert hsa.lib().hsa_selftest_timed_wait(ws.data_ptr(), 4096, limit, after, arrive, torch.cuda.current_stream().cuda_stream) == 0
    ev[1].record()
    if ok:
        hsa.hsa_workspace_status(ws)
    else:
        with pytest.raises(hsa.HSAError, match="HSA_ERR_TIMEOUT"):
            hsa.hsa_workspace_status(ws)
    torch.cuda.synchronize()
    # (64 probes stand between two looks at the time, each some tens of microseconds at most)
    assert (after if ok else limit) * 0.9 <= ev[0].elapsed_time(ev[1]) * 1e3 <= (after if ok else limit) + 50000


@pytest.mark.parametrize("B,H,tokens", [(4, 8, 1 << 28), (24, 32, 1 << 26)])
def test_prefix_of_many_millions_of_tokens(B, H, tokens):
    """Runs that take tens of milliseconds each, in many pieces: the warp that copies queries waits through every piece, and at the end of
    all of them copies those of the requests' own tokens. The prefix is 64 pages in turn; the own tokens outweigh it by far in half of the
    requests, so that they are held to their rounding, and count for nothing in the others, which are held to the rounding of
    sums of that many terms."""
    D, Hkv, pages = 128, 8, 64
    q, Kp, Vp, pre, _, table, own = run_case(56, B=B, H=H, Hkv=Hkv, D=D, prefix=pages * 64, own=torch.arange(B) % 5 * 70 + 60, pages=pages)
    pre = torch.arange(tokens // 64, device=DEV, dtype=torch.int32) % pages
    ws = workspace(q, Kp, pre, table)
    big = torch.arange(B, device=DEV) % 2 == 0
    mine = torch.unique(table[big][table[big] >= 0].long())
    Kp[mine, :, :, 1] = 100.0 * D ** 0.5 / 8
    q[..., 1] = 8.0
    out, lse = hsa.hsa_prefix_decode(q, Kp, Vp, pre, torch.tensor([tokens], device=DEV), table, own, workspace=ws)
    hsa.hsa_workspace_status(ws)    # no wait ran out
    _, run, _ = division(ws)
    more = math.log(tokens / (pages * 64))
    rows = np.arange(B) % 2 == 0
    # a request whose own tokens outweigh the prefix: the prefix seen once, or as often as it is there, makes no difference
    ref = plain_decode(q, Kp, Vp, pre[:pages], pages * 64, table, own)
    tol, tol_lse = paged.prefix_tolerance(ref, D)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (np.abs(got[rows] - ref["out"][rows]) <= tol[rows]).all() and (np.abs(got_lse[rows] - ref["lse"][rows]) <= tol_lse[rows]).all()
    # the others: own tokens are a few parts in a million of the sum. A thread's sums grow by one term a tile, the output's by
    # eight products of sixteen keys, whose accumulator may cut instead of rounding
    alone = plain_decode(q[~big], Kp, Vp, pre[:pages], pages * 64, table[~big], torch.zeros(B // 2, dtype=torch.int64, device=DEV))
    assert (np.abs(got_lse[~rows] - alone["lse"] - more) <= run * 2.0**-24 + 1e-4).all()
    tol = paged.prefix_tolerance(alone, D)[0] + (run * (8 * 2.0**-23 + 2.0**-24) + 1e-4) * alone["mean_abs"]
    assert (np.abs(got[~rows] - alone["out"]) <= tol).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("c,wide", [(FEW[1], False), (FEW[4], False), (WIDE[1], True), (WIDE[5], True)])
def test_queries_that_are_no_numbers_stay_in_their_rows(c, wide, D):
    """NaN and infinities in the queries of a live request, of the empty rows of a padded batch and of rows that see nothing."""
    own = own_of(c, 7)
    q, Kp, Vp, pre, P, table, own = run_case(58, D=D, prefix=5000, own=own, **c)
    pre = torch.cat([pre, torch.full((60000 if wide else 0,), -1, dtype=torch.int32, device=DEV)])
    plen, nothing = torch.tensor([P], device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
    want = hsa.hsa_prefix_decode(q, Kp, Vp, pre, plen, table, own)
    bad = q.clone()
    bad[own < 0] = math.nan
    bad[2] = math.nan
    bad[4, :, :, ::3] = math.inf
    got = hsa.hsa_prefix_decode(bad, Kp, Vp, pre, plen, table, own)
    none = hsa.hsa_prefix_decode(torch.full_like(q, math.nan), Kp, Vp, pre, nothing, table, own.clamp(max=0))
    torch.cuda.synchronize()
    keep = torch.ones(c["B"], dtype=torch.bool, device=DEV)
    keep[[2, 4]] = False
    assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1][keep], want[1][keep])
    assert (got[0][own < 0] == 0).all() and (got[1][own < 0] == -math.inf).all()
    assert (none[0] == 0).all() and (none[1] == -math.inf).all()


@pytest.mark.parametrize("wide", [False, True])
def test_captured_call_that_allocates_its_own_workspace(wide):
    """Two calls of one graph, each with outputs and a workspace out of the graph's memory, replayed over changed lengths."""
    c = WIDE[5] if wide else FEW[4]
    q, Kp, Vp, pre, P, table, own = run_case(59, D=128, prefix=7001, own=own_of(c, 8), **c)
    pre = torch.cat([pre, torch.full((60000 if wide else 0,), -1, dtype=torch.int32, device=DEV)])
    plen, mine, x = torch.tensor([P], device=DEV), own.clone(), torch.roll(q, 1, 0)
    hsa.hsa_prefix_decode(q, Kp, Vp, pre, plen, table, mine)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = hsa.hsa_prefix_decode(q, Kp, Vp, pre, plen, table, mine)
        b = hsa.hsa_prefix_decode(x, Kp, Vp, pre, plen, table, mine)
    for n, lens in ((P, own), (64, own.clamp(max=40)), (0, own), (6999, own.clamp(max=0))):
        plen.fill_(n)
        mine.copy_(lens)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        for y, got in ((q, a), (x, b)):
            want = hsa.hsa_prefix_decode(y, Kp, Vp, pre, plen, table, mine)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H,prefix,own,wide", [
    (4, 8, 1 << 26, 0, False), (24, 32, 1 << 26, 0, True), (32, 64, 1 << 26, 0, True),    # the prefix
    (2, 8, 0, 1 << 27, False), (1, 16, 100, (1 << 27) + 77, False),                       # a request's own tokens
])
def test_sums_over_very_many_tokens_do_not_drift(B, H, prefix, own, wide, D):
    """V is one everywhere, so the output is one: products accumulate in fp32 by cutting, which took 0.8% off 2^26 tokens summed in one
    go. In runs of 512 tiles, eight products a tile, each cut by 2^-23 at most, 2^-11 are lost at most, which with the rounding to
    bf16 (half a step below one is 2^-9) leaves no other number."""
    Hkv, pages = 8, 64
    q, Kp, Vp, _, _, table, _ = run_case(60, B=B, H=H, Hkv=Hkv, D=D, prefix=pages * 64, own=torch.zeros(B, dtype=torch.int64), pages=pages)
    Vp.fill_(1.0)
    Kp.mul_(0.5)
    pre = torch.arange(-(-prefix // 64), device=DEV, dtype=torch.int32) % pages
    if own:
        table = (torch.arange(B * -(-own // 64), device=DEV, dtype=torch.int32) % pages).view(B, -1)
    lens = torch.full((B,), own, device=DEV)
    ws = workspace(q, Kp, pre, table)

    def call():
        return hsa.hsa_prefix_decode(q, Kp, Vp, pre, torch.tensor([prefix], device=DEV), table, lens, workspace=ws)

    (out, lse), names = kernels_of(call)
    hsa.hsa_workspace_status(ws)
    assert ("prefix_wide" in names) == wide
    assert (out == 1).all(), (float(out.float().min()), float(out.float().max()))
    # the sum of the exponentials: 64 pages, as often as they are there (what is over counts for less than a part in 100,000)
    few = torch.arange(pages, device=DEV, dtype=torch.int32)
    ref = plain_decode(q, Kp, Vp, few, pages * 64, table[:, :0], torch.zeros(B, dtype=torch.int64, device=DEV))
    more = math.log((prefix + own) / (pages * 64))
    assert (np.abs(lse.double().cpu().numpy() - ref["lse"] - more) <= 512 * 2.0**-24 + 1e-4).all()


@pytest.mark.parametrize("shape", ["flat", "up", "down"])
@pytest.mark.parametrize("D,B,H,wide", [(64, 3, 8, False), (128, 5, 24, False), (64, 10, 72, True), (128, 6, 136, True)])
def test_pieces_of_runs_longer_than_the_accumulator_sums(D, B, H, wide, shape):
    """Runs of 700 tiles are walked in pieces of 512 and what is left: the second is added to the first, both with references that
    moved, with bad pages at the joint; some requests see all, some nothing."""
    c = dict(B=B, H=H, Hkv=8)
    P = 37 * 700 * TILE + 61
    n = -(-P // 64)
    bad = sorted({*range(1023, n, 1400), *range(1024, n, 2800), *range(7, n, 9001)})
    check(run_case(61, D=D, prefix=P, own=own_of(c, 9), shape=shape, bad=bad, **c), wide=wide, room=0, min_run=513, moved=shape != "flat")


def test_threads_that_call_at_once():
    """Four host threads with a stream each and batches of several kernels and sizes: each gets what it gets alone."""
    import threading

    cases = [run_case(62 + k, D=D, prefix=P, own=own_of(c, 10 + k), **c) + (room,)
             for k, (c, D, P, room) in enumerate([(FEW[0], 64, 700, 0), (FEW[4], 128, 9000, 0), (WIDE[5], 128, 4000, 60000), (WIDE[2], 64, 9000, 60000)])]
    calls = []
    for q, Kp, Vp, pre, P, table, own, room in cases:
        pre = torch.cat([pre, torch.full((room,), -1, dtype=torch.int32, device=DEV)])
        calls.append((q, Kp, Vp, pre, torch.tensor([P], device=DEV), table, own))
    want = [hsa.hsa_prefix_decode(*a) for a in calls]
    torch.cuda.synchronize()
    got, errors = [[] for _ in calls], []

    def work(k):
        try:
            s = torch.cuda.Stream()
            for _ in range(25):
                got[k].append(hsa.hsa_prefix_decode(*calls[k], stream=s))
            s.synchronize()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for w, g in zip(want, got):
        assert len(g) == 25 and all(torch.equal(o, w[0]) and torch.equal(l, w[1]) for o, l in g)


def test_append_of_rows_past_two_to_the_30_vectors():
    """Rows of 8.6e9 elements, where vectors are counted in 64 bits; all but a few rows are skipped."""
    n, Hkv, D, pages = (1 << 22) + 3, 16, 128, 3
    K = torch.empty(n, Hkv, D, dtype=BF16, device=DEV)
    rows = torch.tensor([0, 1, (1 << 20) - 1, 1 << 20, (1 << 21) + 5, (1 << 22) - 1, 1 << 22, n - 1], device=DEV)
    K[rows] = torch.randn(len(rows), Hkv, D, device=DEV).to(BF16)
    slots = torch.full((n,), -1, dtype=torch.int64, device=DEV)
    at = torch.tensor([191, 0, 64, 5, 63, 127, 100, 130], device=DEV)
    slots[rows] = at
    Kp, Vp = (torch.zeros(pages, Hkv, 64, D, dtype=BF16, device=DEV) for _ in range(2))
    hsa.hsa_page_append(K, K, slots, Kp, Vp)
    torch.cuda.synchronize()
    want = torch.zeros_like(Kp)
    want[at // 64, :, at % 64] = K[rows]
    assert torch.equal(Kp, want) and torch.equal(Vp, want)


def test_plan_of_a_prompt_that_fills_its_table_and_more():
    """One request of 2^24 tokens and one that does not fit behind it: as many slots as a map holds, in one call."""
    n = 1 << 24
    width = n // 64
    table = torch.full((2, width), -1, dtype=torch.int32, device=DEV)
    ring = torch.randperm(width + 5, device=DEV).to(torch.int32)
    pool = torch.tensor([3, 3 + width + 5, 0], device=DEV)
    before = ring.clone()
    cu, slots, total = hsa.hsa_page_plan(torch.zeros(2, dtype=torch.int64, device=DEV), torch.tensor([n, 6 * 64], dtype=torch.int32, device=DEV),
                                         table, ring, pool, n + 6 * 64)
    torch.cuda.synchronize()
    ids = before.roll(-3)[:width]
    assert torch.equal(table[0], ids) and (table[1] == -1).all() and torch.equal(ring, before)
    assert torch.equal(slots[:n], (ids.long()[:, None] * 64 + torch.arange(64, device=DEV)).view(-1)) and (slots[n:] == -1).all()
    assert cu.tolist() == [0, n, n + 384] and total.tolist() == [n, 0] and pool.tolist() == [3 + width, 3 + width + 5, 1]
