"""The paged-cache operators on the GPU against the plain fp64 forms: the page plan (whole numbers, equal), the
append (bits, equal) and the shared-prefix decode (elementwise bounds from the rounding of its types)."""
import math

import numpy as np
import pytest
import torch

from oracle import paged
from ultra_long_context_b200 import hsa

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16


def npy(t):
    return (t.float() if t.dtype == BF16 else t).cpu().numpy()


# ---- page plan ----
def plan_case(seed, B, width, F, tokens=3, prompts=0, done=0, idle=0, bad=0, short=False):
    """Lengths, tables and a pool in mid-life whose ring has wrapped; bad: requests with impossible lengths."""
    rng = np.random.default_rng(seed)
    cap = width * 64
    cached = np.minimum((rng.random(B) ** 2 * cap).astype(np.int64), cap - 1)
    new = rng.integers(1, tokens + 1, B).astype(np.int32)
    who = rng.permutation(B)
    for k, val in ((done, -1), (idle, 0)):
        new[who[:k]] = val
        who = who[k:]
    cached[who[:prompts]] = 0
    new[who[:prompts]] = rng.integers(1, cap // 2 + 1, prompts)
    who = who[prompts:]
    cached[who[:bad]] = rng.choice([-3, cap + 1, 1 << 40], bad)
    held = np.where((cached >= 0) & (cached <= cap), paged.pages(cached), 0)
    free = 0 if short is None else int(B // 3) if short else F
    ids = rng.permutation(int(held.sum()) + free).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    ring = np.full(max(1, len(ids)), -1, np.int32)
    taken = int(rng.integers(0, 5 * len(ring) + 1))
    ring[(taken + np.arange(len(ids) - at)) % len(ring)] = ids[at:]
    total = int(np.maximum(new, 0).sum())
    return cached, new, table, ring, np.array([taken, taken + len(ids) - at, 0]), total


def run_plan(cached, new, table, ring, pool, T, in_place=False):
    t = [torch.tensor(x, device=DEV) for x in (cached, new, table, ring, pool)]
    kw = {} if not in_place else dict(total_len=t[0])
    if not in_place:
        kw["pool_out"] = torch.full((3,), -7, dtype=torch.int64, device=DEV)
    cu, slots, total = hsa.hsa_page_plan(*t[:4], t[4], T, **kw)
    torch.cuda.synchronize()
    if not in_place:
        assert np.array_equal(npy(t[4]), pool) and np.array_equal(npy(t[0]), cached)
    got = (cu, slots, total, t[2], t[3], t[4] if in_place else kw["pool_out"])
    return [npy(x) for x in got]


PLANS = [
    dict(B=1, width=1, F=3), dict(B=1, width=200, F=150, prompts=1), dict(B=5, width=3, F=20, done=1, idle=1),
    dict(B=64, width=70, F=100, done=5, idle=3), dict(B=130, width=40, F=2000, prompts=40, done=20, idle=9, bad=7),
    dict(B=130, width=40, F=2000, prompts=40, done=20, bad=7, short=True), dict(B=33, width=9, F=0, done=30, idle=3),
    dict(B=513, width=30, F=4000, prompts=100, tokens=130, done=60), dict(B=700, width=5, F=0, short=None, tokens=1),
    dict(B=8192, width=4, F=9000, done=500, idle=500, bad=20), dict(B=20, width=2000, F=30000, prompts=15, done=4),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", PLANS)
def test_page_plan_equals_the_request_by_request_form(case, in_place):
    cached, new, table, ring, pool, total = plan_case(11, **case)
    for T in (total + 9, max(0, total - 5)):   # the second leaves the last rows without room
        want = paged.page_plan(cached, new, table, ring, pool, T)
        got = run_plan(cached, new, table, ring, pool, T, in_place)
        for w, g, name in zip(want, got, ("cu_new", "slots", "total_len", "block_table", "free_pages", "pool")):
            assert np.array_equal(w, g), name


def test_page_plan_saturates_row_sums():
    cached, new = np.array([0, 0, 5]), np.array([2**31 - 1, 2**31 - 1, 1], np.int32)
    table, ring = np.full((3, 4), 2, np.int32), np.arange(9, dtype=np.int32)
    want = paged.page_plan(cached, new, table, ring, np.array([0, 9, 0]), 10)
    got = run_plan(cached, new, table, ring, np.array([0, 9, 0]), 10)
    for w, g in zip(want, got):
        assert np.array_equal(w, g)


def test_page_plan_leaves_neighbouring_memory_alone():
    cached, new, table, ring, pool, total = plan_case(3, B=40, width=12, F=200, prompts=9, done=4)
    guard = {}

    def fenced(shape, dtype):
        n = int(np.prod(shape))
        g = torch.full((n + 64,), 77, dtype=dtype, device=DEV)
        guard[len(guard)] = g
        return g[32:32 + n].view(shape)

    t = [torch.tensor(x, device=DEV) for x in (cached, new, table, ring, pool)]
    tab, rng_ = fenced(table.shape, torch.int32), fenced(ring.shape, torch.int32)
    tab.copy_(t[2])
    rng_.copy_(t[3])
    hsa.hsa_page_plan(t[0], t[1], tab, rng_, t[4], total + 3, cu_new=fenced((41,), torch.int32),
                      slots=fenced((total + 3,), torch.int64), total_len=fenced((40,), torch.int64),
                      pool_out=fenced((3,), torch.int64))
    torch.cuda.synchronize()
    for g in guard.values():
        assert (g[:32] == 77).all() and (g[-32:] == 77).all()


# ---- append ----
@pytest.mark.parametrize("n,Hkv,D,extra", [(1, 1, 64, 0), (7, 3, 128, 0), (129, 8, 128, 16), (1000, 2, 64, 8), (4097, 4, 64, 128),
                                           (0, 2, 128, 0)])
def test_append_writes_rows_into_their_slots(n, Hkv, D, extra):
    rng = np.random.default_rng(n)
    pages = n // 40 + 3
    big = torch.randn(n, 2 * Hkv * D + 2 * extra, device=DEV).to(BF16)
    K, V = big[:, extra:extra + Hkv * D].view(n, Hkv, D), big[:, extra + Hkv * D:2 * Hkv * D + extra].view(n, Hkv, D)
    slots = rng.permutation(pages * 64)[:n].astype(np.int64)
    slots[rng.permutation(n)[:n // 10]] = rng.choice([-1, -2**40, pages * 64, 2**45], n // 10)
    pool = torch.randn(2, pages, Hkv, 64, D, device=DEV).to(BF16)
    Kp, Vp = pool[0].clone(), pool[1].clone()
    wk, wv = paged.page_append(npy(K), npy(V), slots, npy(Kp), npy(Vp))
    hsa.hsa_page_append(K, V, torch.tensor(slots, device=DEV), Kp, Vp)
    torch.cuda.synchronize()
    assert np.array_equal(npy(Kp), wk) and np.array_equal(npy(Vp), wv)


def test_append_reaches_slots_past_two_to_the_31_elements():
    pages, Hkv, D = 140000, 2, 128          # 2.3e9 elements a pool
    Kp, Vp = (torch.zeros(pages, Hkv, 64, D, dtype=BF16, device=DEV) for _ in range(2))
    K, V = (torch.randn(3, Hkv, D, device=DEV).to(BF16) for _ in range(2))
    slots = torch.tensor([pages * 64 - 1, 131072 * 64 + 5, 0], device=DEV)
    hsa.hsa_page_append(K, V, slots, Kp, Vp)
    torch.cuda.synchronize()
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(Kp[s // 64, :, s % 64], K[t]) and torch.equal(Vp[s // 64, :, s % 64], V[t])
    assert int((Kp != 0).sum()) == int((K != 0).sum()) and int((Vp != 0).sum()) == int((V != 0).sum())


# ---- shared-prefix decode ----
def decode_case(seed, B, H, Hkv, Tq, D, prefix, own, scale=0.0, poison=True, sharp=1.0):
    """Pools with scattered pages; rows behind a length, and pages nobody owns, hold NaN and infinities."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    own = np.asarray(own, np.int64)
    held = paged.pages(np.maximum(own, 0))
    npre = paged.pages(prefix)
    total = int(npre + held.sum()) + 2
    ids = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).numpy().astype(np.int32)
    width = int(held.max()) + 1
    table = np.full((B, width), -1, np.int32)
    at = npre
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    pool = torch.randn(2, total, Hkv, 64, D, generator=g, device=DEV).to(BF16)
    if poison:
        for last, n in [(ids[npre - 1] if npre else -1, prefix)] + [(table[b, held[b] - 1] if held[b] else -1, own[b]) for b in range(B)]:
            if last >= 0 and n % 64:
                pool[:, last, :, n % 64:] = torch.tensor([math.nan, math.inf], device=DEV, dtype=BF16)[:, None, None, None]
        pool[:, torch.tensor(ids[at:].astype(np.int64), device=DEV)] = math.nan
    q = (torch.randn(B, H, Tq, D, generator=g, device=DEV) * sharp).to(BF16)
    return q, pool[0].contiguous(), pool[1].contiguous(), ids[:npre].copy(), prefix, table, own, scale


def check_decode(q, Kp, Vp, pre, prefix, table, own, scale, squeeze=False, room=0, **kw):
    """room: pages that the prefix's table has beyond the prefix (the kernels are chosen by the table's size)."""
    D = q.shape[-1]
    pre = np.concatenate([pre, np.full(room, -1, np.int32)])
    args = [torch.tensor(x, device=DEV) for x in (pre, [prefix], table, own)]
    hsa.hsa_profile_enable(room > 0)
    out, lse = hsa.hsa_prefix_decode(q.squeeze(2) if squeeze else q, Kp, Vp, args[0], args[1], args[2], args[3], scale=scale, **kw)
    torch.cuda.synchronize()
    if room:
        assert "prefix_wide" in hsa.hsa_profile_summary()
        hsa.hsa_profile_enable(False)
    ref = paged.prefix_decode(npy(q), npy(Kp), npy(Vp), pre, prefix, table, own, scale if scale > 0 else D ** -0.5)
    got, got_lse = npy(out).astype(np.float64).reshape(ref["out"].shape), npy(lse).astype(np.float64).reshape(ref["lse"].shape)
    tol, tol_lse = paged.prefix_tolerance(ref, D)
    assert np.isfinite(got).all()
    assert np.array_equal(np.isneginf(got_lse), np.isneginf(ref["lse"]))
    bad = np.abs(got - ref["out"]) > tol
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - ref["out"]).max()), np.argwhere(bad)[:4].tolist())
    fin = np.isfinite(ref["lse"])
    off = np.abs(got_lse[fin] - ref["lse"][fin])
    assert (off <= tol_lse[fin]).all(), (float(off.max()), float((off / tol_lse[fin]).max()))
    assert (got[ref["keys"] == 0] == 0).all()
    return out, lse


DECODES = [
    # no prefix, no own tokens, single tokens, page and tile borders
    dict(B=1, H=1, Hkv=1, Tq=1, D=64, prefix=1, own=[0]),
    dict(B=1, H=1, Hkv=1, Tq=1, D=128, prefix=0, own=[1]),
    dict(B=2, H=2, Hkv=1, Tq=1, D=128, prefix=0, own=[0, -1]),
    dict(B=3, H=4, Hkv=4, Tq=1, D=64, prefix=64, own=[1, 64, 65]),
    dict(B=4, H=4, Hkv=2, Tq=1, D=128, prefix=63, own=[127, 128, 129, -1]),
    dict(B=5, H=3, Hkv=3, Tq=1, D=128, prefix=129, own=[0, 3, 191, 192, 193]),
    dict(B=4, H=8, Hkv=8, Tq=1, D=128, prefix=1000, own=[17, 300, 1, 0]),
    # several tokens a step, some requests shorter than them (and the prefix too)
    dict(B=4, H=4, Hkv=2, Tq=3, D=64, prefix=130, own=[3, 64, 2, 0]),
    dict(B=3, H=2, Hkv=1, Tq=5, D=128, prefix=3, own=[0, 1, 7]),
    dict(B=2, H=4, Hkv=1, Tq=64, D=64, prefix=40, own=[70, 10]),
    # row counts around a tile of 128 rows and a group of 256, grouped heads
    dict(B=32, H=4, Hkv=1, Tq=1, D=128, prefix=700, own=[5 + 3 * i for i in range(32)]),
    dict(B=43, H=3, Hkv=1, Tq=1, D=64, prefix=500, own=[i for i in range(43)]),
    dict(B=17, H=32, Hkv=2, Tq=1, D=128, prefix=400, own=[-1 if i % 5 == 2 else 4 * i for i in range(17)]),
    dict(B=3, H=16, Hkv=1, Tq=16, D=128, prefix=300, own=[200, 16, 333]),
    dict(B=1, H=32, Hkv=1, Tq=32, D=64, prefix=257, own=[500]),
    # one long request among short ones
    dict(B=9, H=2, Hkv=2, Tq=1, D=128, prefix=200, own=[1, 2, 9000, 4, 0, 6, 7, -1, 9]),
    dict(B=2, H=2, Hkv=2, Tq=2, D=64, prefix=20000, own=[5, 70]),
    # a longer prefix than the wave of key ranges has tiles, many heads
    dict(B=2, H=16, Hkv=16, Tq=1, D=64, prefix=2500, own=[40, 500]),
]


@pytest.mark.parametrize("case", DECODES)
def test_prefix_decode_equals_the_plain_form(case):
    check_decode(*decode_case(21, **case))


WIDE = 60000   # with a table this long, batches of more than 64 rows per key head take the kernel for wide products


@pytest.mark.parametrize("case", [c for c in DECODES if c["B"] * c["H"] * c["Tq"] // c["Hkv"] > 64] + [
    dict(B=65, H=1, Hkv=1, Tq=1, D=64, prefix=129, own=[2] * 65),
    dict(B=129, H=2, Hkv=2, Tq=1, D=128, prefix=1, own=[i % 3 - 1 for i in range(129)]),
    dict(B=100, H=4, Hkv=1, Tq=1, D=128, prefix=64, own=[i % 70 for i in range(100)]),
    dict(B=86, H=3, Hkv=1, Tq=3, D=64, prefix=1000, own=[i % 5 for i in range(86)]),
    dict(B=257, H=2, Hkv=1, Tq=1, D=128, prefix=3333, own=[i for i in range(257)]),
    dict(B=16, H=16, Hkv=1, Tq=1, D=128, prefix=0, own=[3] * 16),
])
def test_prefix_decode_of_wide_batches_equals_the_plain_form(case):
    check_decode(*decode_case(41, **case), room=WIDE)


@pytest.mark.parametrize("room", [0, WIDE])
@pytest.mark.parametrize("B", [20, 40, 45])
@pytest.mark.parametrize("sharp,scale", [(8.0, 0.0), (1.0, 2.0), (0.02, 0.0)])
def test_prefix_decode_of_peaked_and_flat_rows_in_groups(sharp, scale, B, room):
    """Row groups that end early: 80, 160 and 180 rows per key head, in groups of 64 or of 256."""
    for D in (64, 128):
        check_decode(*decode_case(42, B=B, H=8, Hkv=2, Tq=1, D=D, prefix=2500, own=[i for i in range(B)], sharp=sharp, scale=scale), room=room)


@pytest.mark.parametrize("room", [0, WIDE])
def test_prefix_decode_maxima_that_keep_growing_in_groups(room):
    """Rows of which some move their reference in every tile while others of the same tile do not."""
    for D, flip in ((64, False), (128, True), (128, False)):
        q, Kp, Vp, pre, prefix, table, own, scale = decode_case(43, B=90, H=2, Hkv=2, Tq=1, D=D, prefix=1500, own=[1] * 90, poison=False)
        size = torch.linspace(0.0, 40.0, len(pre), device=DEV)
        if flip:
            size = size.flip(0)
        Kp[torch.tensor(pre.astype(np.int64), device=DEV)] = (q[::2].float().mean(0)[:, 0][None, :, None] * 8 * size[:, None, None, None]).to(BF16)
        check_decode(q, Kp, Vp, pre, prefix, table, own, scale, room=room)


def test_wide_prefix_decode_leaves_out_bad_pages():
    q, Kp, Vp, pre, prefix, table, own, scale = decode_case(44, B=70, H=4, Hkv=2, Tq=1, D=128, prefix=1900, own=[5] * 70)
    pre[[0, 1, 5, 14, 29]] = [-1, Kp.shape[0], Kp.shape[0], 2**31 - 1, -9]
    check_decode(q, Kp, Vp, pre, prefix, table, own, scale, room=WIDE)
    pre[:] = -1
    check_decode(q, Kp, Vp, pre, prefix, table, own, scale, room=WIDE)


def test_wide_and_few_row_kernels_back_to_back():
    """Many calls without a pause, the two kernels of each overlapping; the same answer every time."""
    q, Kp, Vp, pre, prefix, table, own, scale = decode_case(45, B=48, H=16, Hkv=2, Tq=1, D=128, prefix=9000, own=[1 + 61 * i % 700 for i in range(48)])
    args = [torch.tensor(x, device=DEV) for x in (np.concatenate([pre, np.full(WIDE, -1, np.int32)]), [prefix], table, own)]
    got = [hsa.hsa_prefix_decode(q, Kp, Vp, *args) for _ in range(60)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, got[0][0]) and torch.equal(l, got[0][1]) for o, l in got)
    check_decode(q, Kp, Vp, pre, prefix, table, own, scale, room=WIDE)


@pytest.mark.parametrize("sharp,scale", [(8.0, 0.0), (1.0, 2.0), (0.02, 0.0)])
def test_prefix_decode_of_peaked_and_flat_rows(sharp, scale):
    """Maxima that move far along the keys (every rescaling happens) and rows that are nearly uniform."""
    check_decode(*decode_case(22, B=6, H=4, Hkv=2, Tq=2, D=128, prefix=3000, own=[2, 100, 700, 9, 1500, 64], sharp=sharp, scale=scale))


def test_prefix_decode_maxima_that_keep_growing():
    """Keys sorted so that every tile holds a larger logit than the one before it, by far more than the softmax's
    range in one step; and the other way round."""
    for flip in (False, True):
        q, Kp, Vp, pre, prefix, table, own, scale = decode_case(23, B=3, H=2, Hkv=2, Tq=1, D=64, prefix=2048, own=[300, 64, 0], poison=False)
        size = torch.linspace(0.0, 30.0, len(pre), device=DEV)
        if flip:
            size = size.flip(0)
        Kp[torch.tensor(pre.astype(np.int64), device=DEV)] = (q[0, :, 0][None, :, None] * size[:, None, None, None]).to(BF16)
        check_decode(q, Kp, Vp, pre, prefix, table, own, scale)


def test_prefix_decode_leaves_out_bad_pages():
    q, Kp, Vp, pre, prefix, table, own, scale = decode_case(24, B=4, H=4, Hkv=2, Tq=1, D=128, prefix=900, own=[400, 130, 64, 300])
    pre[[0, 5, 14]] = [-1, Kp.shape[0], 2**31 - 1]
    table[0, [1, 3]] = [-(2**31), Kp.shape[0] + 7]
    table[2, 0] = -1
    check_decode(q, Kp, Vp, pre, prefix, table, own, scale)
    # a prefix without one good page, and requests without one either
    pre[:] = -1
    table[1:] = -1
    check_decode(q, Kp, Vp, pre, prefix, table, own, scale)


def test_prefix_decode_cuts_lengths_to_the_tables():
    q, Kp, Vp, pre, prefix, table, own, scale = decode_case(25, B=2, H=2, Hkv=2, Tq=1, D=64, prefix=128, own=[64, 128], poison=False)
    a = check_decode(q, Kp, Vp, pre, 1 << 50, table[:, :1].copy(), np.array([1 << 45, 1 << 33]), scale)
    b = check_decode(q, Kp, Vp, pre, 128, table[:, :1].copy(), np.array([64, 64]), scale)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_decode(q, Kp, Vp, pre, -5, table, np.array([7, 0]), scale)


def test_prefix_decode_without_tables():
    q, Kp, Vp, pre, prefix, table, own, scale = decode_case(26, B=3, H=4, Hkv=2, Tq=1, D=128, prefix=300, own=[100, 20, 90])
    check_decode(q, Kp, Vp, pre, prefix, table[:, :0].copy(), np.array([100, 0, -1]), scale)
    check_decode(q, Kp, Vp, pre[:0].copy(), 0, table, own, scale)
    check_decode(q, Kp, Vp, pre[:0].copy(), 0, table[:, :0].copy(), own, scale)
    check_decode(q, Kp, Vp, pre, prefix, table, own, scale, squeeze=True)


def test_prefix_decode_batch_of_8192():
    rng = np.random.default_rng(4)
    own = rng.integers(-1, 3, 8192)
    own[[0, 4000, 8191]] = (500, 130, 64)
    case = decode_case(27, B=8192, H=1, Hkv=1, Tq=1, D=64, prefix=200, own=own, poison=False)
    check_decode(*case)
    check_decode(*case, room=WIDE)


def test_prefix_decode_pools_past_two_to_the_31_elements():
    """The last pages of pools of 2.4e9 elements."""
    pages, D = 9200, 128
    q, Kp0, Vp0, pre, prefix, table, own, scale = decode_case(28, B=2, H=32, Hkv=32, Tq=1, D=D, prefix=150, own=[70, 64], poison=False)
    n = Kp0.shape[0]
    Kp, Vp = (torch.full((pages, 32, 64, D), math.nan, dtype=BF16, device=DEV) for _ in range(2))
    Kp[pages - n:], Vp[pages - n:] = Kp0, Vp0
    small = [torch.tensor(x, device=DEV) for x in (pre, [prefix], table, own)]
    want = hsa.hsa_prefix_decode(q, Kp0, Vp0, *small)
    far = [small[0] + (pages - n), small[1], small[2] + (pages - n), small[3]]
    got = hsa.hsa_prefix_decode(q, Kp, Vp, *far)
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    check_decode(q, Kp0, Vp0, pre, prefix, table, own, scale)


def test_prefix_decode_repeats_bit_for_bit_and_ignores_the_workspace():
    q, Kp, Vp, pre, prefix, table, own, scale = decode_case(29, B=20, H=8, Hkv=2, Tq=1, D=128, prefix=5000, own=[37 * i for i in range(20)])
    args = [torch.tensor(x, device=DEV) for x in (pre, [prefix], table, own)]
    size = hsa.hsa_prefix_decode_workspace_size(20, 8, 2, 128, len(pre), table.shape[1]) + 256
    outs = []
    for fill in (0, 255, 127):
        ws = torch.full((size,), fill, dtype=torch.uint8, device=DEV)
        outs.append(hsa.hsa_prefix_decode(q, Kp, Vp, *args, workspace=ws))
        hsa.hsa_workspace_status(ws[(-ws.data_ptr()) % 256:])
    for o, l in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1])


@pytest.mark.parametrize("D", [64, 128])
def test_prefix_decode_long_runs_and_many_short_segments_back_to_back(D):
    """Runs of many tiles and segments of an odd number of them, so that the copies' ring goes round many times with
    its slots changing hands between the two streams; many calls without a pause between them."""
    own = [1 + 61 * i % 700 for i in range(40)]
    q, Kp, Vp, pre, prefix, table, own, scale = decode_case(33, B=40, H=2, Hkv=2, Tq=1, D=D, prefix=40000, own=own)
    args = [torch.tensor(x, device=DEV) for x in (pre, [prefix], table, own)]
    got = [hsa.hsa_prefix_decode(q, Kp, Vp, *args) for _ in range(60)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, got[0][0]) and torch.equal(l, got[0][1]) for o, l in got)
    check_decode(q, Kp, Vp, pre, prefix, table, own, scale)


def test_prefix_decode_follows_its_lengths_in_a_captured_graph():
    """Two graphs share a workspace and are replayed in turn while lengths and tables change on the device."""
    q, Kp, Vp, pre, prefix, table, own, scale = decode_case(30, B=6, H=8, Hkv=2, Tq=1, D=64, prefix=3000, own=[5, 64, 900, 1, 130, -1], poison=False)
    args = [torch.tensor(x, device=DEV) for x in (pre, [prefix], table, own)]
    q2 = torch.randn_like(q)
    ws = torch.empty(hsa.hsa_prefix_decode_workspace_size(6, 8, 2, 64, len(pre), table.shape[1]) + 256, dtype=torch.uint8, device=DEV)
    outs = [(torch.empty_like(q), torch.empty(q.shape[:-1], device=DEV)) for _ in range(2)]
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x, (o, l) in zip((q, q2), outs):
            hsa.hsa_prefix_decode(x, Kp, Vp, *args, out=o, lse=l, workspace=ws)
    torch.cuda.synchronize()
    for x, (o, l) in zip((q, q2), outs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            hsa.hsa_prefix_decode(x, Kp, Vp, *args, out=o, lse=l, workspace=ws)
        graphs.append(gr)
    for P, lens in ((3000, [5, 64, 900, 1, 130, -1]), (77, [0, -1, 901, 2, 131, 3]), (0, [1, 1, 1, 1, 1, 1])):
        args[1].fill_(P)
        args[3].copy_(torch.tensor(lens))
        for o, l in outs:
            o.fill_(7)
            l.fill_(7)
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for x, (o, l) in zip((q, q2), outs):
            want = hsa.hsa_prefix_decode(x, Kp, Vp, *args)
            assert torch.equal(want[0], o) and torch.equal(want[1], l)
            check_decode(x, Kp, Vp, pre, P, table, np.array(lens), scale)


def test_prefix_decode_on_another_stream():
    q, Kp, Vp, pre, prefix, table, own, scale = decode_case(31, B=6, H=8, Hkv=8, Tq=1, D=128, prefix=3000, own=[5, 64, 900, 1, 130, -1])
    args = [torch.tensor(x, device=DEV) for x in (pre, [prefix], table, own)]
    want = hsa.hsa_prefix_decode(q, Kp, Vp, *args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a = hsa.hsa_prefix_decode(q, Kp, Vp, *args, stream=s)
    b = hsa.hsa_prefix_decode(q, Kp, Vp, *args)       # overlaps the other, each with its own workspace
    torch.cuda.synchronize()
    for o in (a, b):
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])


def test_bindings_refuse_wrong_tensors():
    q, Kp, Vp, pre, prefix, table, own, scale = decode_case(32, B=2, H=2, Hkv=1, Tq=1, D=64, prefix=64, own=[5, 6])
    args = [torch.tensor(x, device=DEV) for x in (pre, [prefix], table, own)]
    with pytest.raises(TypeError, match="prefix_len"):
        hsa.hsa_prefix_decode(q, Kp, Vp, args[0], args[1].int(), args[2], args[3])
    with pytest.raises(ValueError, match="Vp"):
        hsa.hsa_prefix_decode(q, Kp, Vp[:-1], *args)
    with pytest.raises(ValueError, match="contiguous"):
        hsa.hsa_prefix_decode(q.expand(2, 2, 4, 64), Kp, Vp, *args)
    with pytest.raises(ValueError, match="cpu"):
        hsa.hsa_prefix_decode(q, Kp, Vp, args[0], args[1], args[2], args[3].cpu())
    with pytest.raises(hsa.HSAError, match="HSA_ERR_WORKSPACE"):
        hsa.hsa_prefix_decode(q, Kp, Vp, *args, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    K = torch.randn(4, 1, 64, device=DEV).to(BF16)
    slots = torch.arange(4, device=DEV)
    with pytest.raises(ValueError, match="V must have shape"):
        hsa.hsa_page_append(K, K[:3], slots, Kp, Vp)
    with pytest.raises(ValueError, match="contiguously"):
        hsa.hsa_page_append(K.transpose(0, 2).contiguous().transpose(0, 2), K, slots, Kp, Vp)
    with pytest.raises(ValueError, match="slots"):
        hsa.hsa_page_append(K, K, slots[:3], Kp, Vp)
    with pytest.raises(hsa.HSAError, match="strides"):
        hsa.hsa_page_append(torch.randn(4, 68, device=DEV).to(BF16)[:, :64].view(4, 1, 64), K, slots, Kp, Vp)
    with pytest.raises(TypeError, match="new_len"):
        hsa.hsa_page_plan(args[3], args[3], args[2], args[0], torch.zeros(3, dtype=torch.int64, device=DEV), 4)


# ---- together ----
@pytest.mark.parametrize("graph", [False, True])
def test_serving_loop_over_a_shared_document(graph):
    """A document is planned and appended as one request; then several steps of plan, append and decode, with
    prompts, single tokens, a request that finishes and its row taken by a new one."""
    B, H, Hkv, D, width, F, T = 5, 4, 2, 64, 8, 64, 200
    gen = torch.Generator(device=DEV).manual_seed(9)
    Kp, Vp = (torch.full((F, Hkv, 64, D), math.nan, dtype=BF16, device=DEV) for _ in range(2))
    ring = torch.randperm(F, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    pool = torch.tensor([0, F, 0], device=DEV)
    doc = 700
    doc_table = torch.full((1, 12), -1, dtype=torch.int32, device=DEV)
    kv = torch.randn(2, doc, Hkv, D, generator=gen, device=DEV).to(BF16)
    _, slots, doc_len = hsa.hsa_page_plan(torch.zeros(1, dtype=torch.int64, device=DEV), torch.tensor([doc], dtype=torch.int32, device=DEV),
                                          doc_table, ring, pool, doc)
    hsa.hsa_page_append(kv[0], kv[1], slots, Kp, Vp)

    lens = torch.zeros(B, dtype=torch.int64, device=DEV)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    new = torch.zeros(B, dtype=torch.int32, device=DEV)
    rows = torch.zeros(2, T, Hkv, D, dtype=BF16, device=DEV)
    q = torch.zeros(B, H, D, dtype=BF16, device=DEV)
    cu, slots = torch.empty(B + 1, dtype=torch.int32, device=DEV), torch.empty(T, dtype=torch.int64, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(B, H, device=DEV)
    ws = torch.empty(hsa.hsa_prefix_decode_workspace_size(B, H, Hkv, D, 12, width) + 256, dtype=torch.uint8, device=DEV)

    def step():
        hsa.hsa_page_plan(lens, new, table, ring, pool, T, cu_new=cu, slots=slots, total_len=lens)
        hsa.hsa_page_append(rows[0], rows[1], slots, Kp, Vp)
        hsa.hsa_prefix_decode(q, Kp, Vp, doc_table.view(-1), doc_len, table, lens, out=out, lse=lse, workspace=ws)

    if graph:
        torch.cuda.synchronize()
        recorded = torch.cuda.CUDAGraph()
        with torch.cuda.graph(recorded):
            step()
    history = [np.zeros((2, 0, Hkv, D)) for _ in range(B)]
    for adds in ([10, 64, 0, 100, 1], [1, 1, 63, 1, 1], [1, -1, 1, 60, 1], [0, 130, 1, 1, -1], [1, 1, 1, 1, 2]):
        new.copy_(torch.tensor(adds, dtype=torch.int32))
        rows.copy_(torch.randn(rows.shape, generator=gen, device=DEV).to(BF16))
        q.copy_(torch.randn(q.shape, generator=gen, device=DEV).to(BF16))
        recorded.replay() if graph else step()
        torch.cuda.synchronize()
        at = 0
        for b, n in enumerate(adds):
            if n < 0:
                history[b] = np.zeros((2, 0, Hkv, D))
            else:
                history[b] = np.concatenate([history[b], npy(rows[:, at:at + n])], 1)
                at += n
        assert int(pool[2]) == 0 and lens.tolist() == [h.shape[1] for h in history]
        assert int(pool[1] - pool[0]) == F - 11 - sum(-(-h.shape[1] // 64) for h in history)
        # the same attention over plainly laid out sequences: request b's tokens in pages of its own
        pages = [paged.pages(h.shape[1]) for h in history]
        plain = np.zeros((2, 11 + sum(pages), Hkv, 64, D))
        flat = np.zeros((2, 11 * 64, Hkv, D))
        flat[:, :doc] = npy(kv)
        plain[:, :11] = flat.reshape(2, 11, 64, Hkv, D).swapaxes(2, 3)
        tab = np.full((B, width), -1)
        at = 11
        for b, h in enumerate(history):
            flat = np.zeros((2, pages[b] * 64, Hkv, D))
            flat[:, :h.shape[1]] = h
            plain[:, at:at + pages[b]] = flat.reshape(2, pages[b], 64, Hkv, D).swapaxes(2, 3)
            tab[b, :pages[b]] = np.arange(at, at + pages[b])
            at += pages[b]
        ref = paged.prefix_decode(npy(q)[:, :, None], plain[0], plain[1], np.arange(11), doc, tab, [h.shape[1] for h in history], D ** -0.5)
        tol, tol_lse = paged.prefix_tolerance(ref, D)
        assert (np.abs(npy(out)[:, :, None] - ref["out"]) <= tol).all()
        assert (np.abs(npy(lse)[:, :, None] - ref["lse"]) <= tol_lse).all()
