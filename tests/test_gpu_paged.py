"""The receiver's paged cache on the GPU (mf_paged_decode, mf_kv_append, mf_kv_evict,
mf_map_key_scores) against plain float64 loops.

Bounds.  dx bounds a score's error: d products of magnitude sum |q k| scale, rounded and summed in
float32 (plus the scale).  A weight exp(x - lse) is then off by a relative 2 dx (its own x and the
lse), by the rounding of x and lse as stored numbers (|x| 2^-22 covers two roundings in the base-2
domain) and by the base-2 exponential (2^-22) and the sums (one rounding per 16 keys and warp, and
one per joined part); the bf16 pair that carries it into P.V is off by 2^-17.  O adds its own
rounding, half a step."""
import ctypes
import math

import pytest
import torch

import paged_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _mf():
    import cross_model_attention_mf_b200 as mf
    return mf


def _kv(mf, c, both=None, max_len=None):
    """Device copy of a cache (keeping interleaved K and V slices of one tensor)."""
    if both is not None:
        b = both.cuda()
        K, V = b[:, 0], b[:, 1]
    else:
        K, V = c.K.cuda(), c.V.cuda()
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    return mf.PagedKV(K, V, c.table.cuda(), lens, max(c.lens) if max_len is None else max_len)


def _clean(mf):
    rc, bits = mf.mf_get_status()
    assert rc == mf.MF_OK and bits == 0, (rc, bits)


def check_decode(c, Q, O, lse=None, gathered=None, scale=None, dtype=F32):
    """gathered: (score before, score after)."""
    wantO, want_lse, w, dx, A, xmax = ref.decode(c, Q, scale)
    n = max(1, max(c.lens))
    rel = 2 * dx + xmax * 2.0 ** -22 + 2.0 ** -21 + (n / 16 + 64) * 2.0 ** -24
    tol = (A * (rel + 2.0 ** -17)[..., None]) + 1e-30
    if O.dtype == BF:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * wantO.abs()
    err = (O.double().cpu() - wantO).abs()
    assert torch.isfinite(O.double()).all()
    assert (err <= tol).all(), (err - tol).max()
    if lse is not None:
        lo = lse.double().cpu()
        dead = want_lse == -math.inf
        assert (lo[dead] == -math.inf).all()
        assert ((lo - want_lse).abs()[~dead] <= (rel + want_lse.abs() * 2.0 ** -22)[~dead]).all()
    if gathered is not None:
        before, after = (t.double().cpu() for t in gathered)
        G = Q.shape[1] // c.K.shape[2]
        worst = rel.view(rel.shape[0], -1, G).amax(2)[..., None]
        for s, L in enumerate(c.lens):
            want = before[s, :, :L] + w[s, :, :L]
            t = w[s, :, :L] * worst[s] + 2.0 ** -23 * want.abs() + 1e-30
            assert ((after[s, :, :L] - want).abs() <= t).all(), s
            assert torch.equal(after[s, :, L:], before[s, :, L:])  # slots past the length: untouched


DECODE = [
    # lens, h_kv, group, d, page, dtype
    ((1,), 1, 1, 64, 16, BF),
    ((0, 1, 15, 16, 17, 33), 2, 4, 128, 16, BF),
    ((100,), 8, 4, 128, 16, BF),
    ((300, 0, 1), 8, 3, 128, 64, BF),
    ((2500, 1, 0, 777), 3, 5, 80, 12, BF),
    ((257, 4000), 2, 8, 64, 1, BF),
    ((900, 40), 1, 16, 256, 20, BF),
    ((513,), 2, 9, 192, 7, BF),
    ((600, 31), 1, 40, 96, 32, BF),
    ((1000, 5), 2, 1, 8, 16, BF),
    ((1,), 1, 1, 64, 16, F32),
    ((0, 1, 7, 8, 9, 65), 2, 4, 128, 16, F32),
    ((1001, 0, 143), 3, 5, 80, 12, F32),
    ((700,), 1, 11, 256, 20, F32),
    ((300, 299), 2, 2, 192, 5, F32),
    ((2100,), 4, 3, 64, 64, F32),
    ((333,), 2, 1, 8, 3, F32),
]


@pytest.mark.parametrize("lens,h_kv,group,d,page,dtype", DECODE)
@pytest.mark.parametrize("mode", ["plain", "scores", "loose_bound"])
def test_decode(lens, h_kv, group, d, page, dtype, mode):
    mf = _mf()
    # every row that no sequence holds is NaN: reading one would show
    c, both = ref.make_cache(lens, h_kv, d, page, dtype, seed=len(lens) + d, interleaved=mode == "scores",
                             stale=float("nan"))
    g = torch.Generator().manual_seed(7)
    h_r = group * h_kv
    qkv = (2.0 * torch.randn(len(lens), h_r * d + 64, generator=g)).to(dtype)
    Q = qkv[:, :h_r * d].unflatten(1, (h_r, d))
    Qd = qkv.cuda()[:, :h_r * d].unflatten(1, (h_r, d))
    # a loose length bound takes the split path even for short sequences
    kv = _kv(mf, c, both if mode == "scores" else None,
             max_len=max(lens) + 300 if mode == "loose_bound" else None)
    lse = torch.full((len(lens), h_r), 7.0, device="cuda")
    if mode == "scores":
        before = torch.rand(len(lens), h_kv, max(lens) + 3, generator=g).cuda()
        after = before.clone()
        O = mf.mf_paged_decode(kv, Qd, lse=lse, score=after, o_f32=dtype == BF)
        gathered = (before, after)
        out = torch.full_like(before, 5.0)
        mf.mf_paged_decode(kv, Qd, score=before, score_out=out)
        for s, L in enumerate(lens):
            assert torch.equal(out[s, :, :L], after[s, :, :L])
            assert (out[s, :, L:] == 5.0).all()
    else:
        O = mf.mf_paged_decode(kv, Qd, lse=lse)
        gathered = None
    _clean(mf)
    assert O.dtype == (F32 if mode == "scores" else dtype)
    check_decode(c, Q, O, lse, gathered)
    again = mf.mf_paged_decode(kv, Qd, o_f32=O.dtype == F32 and dtype == BF)
    if mode != "scores":
        assert torch.equal(again, O)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_many_sequences_share_pages(dtype):
    """600 short sequences over a shared prefix page: more units than CTAs, and many per CTA."""
    mf = _mf()
    n, page, h_kv, d = 600, 8, 2, 64
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 40, (n,), generator=g).tolist()
    K = torch.randn(50, page, h_kv, d, generator=g).to(dtype)
    V = torch.randn(50, page, h_kv, d, generator=g).to(dtype)
    table = torch.randint(1, 50, (n, 40), generator=g).to(torch.int32)
    table[:, 0] = 0
    c = ref.Cache(K, V, table, lens, page)
    Q = torch.randn(n, 4, d, generator=g).to(dtype)
    kv = mf.PagedKV(K.cuda(), V.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), 320)
    before = torch.rand(n, h_kv, 320, generator=g).cuda()
    after = before.clone()
    lse = torch.empty(n, 4, device="cuda")
    O = mf.mf_paged_decode(kv, Q.cuda(), lse=lse, score=after)
    _clean(mf)
    check_decode(c, Q, O, lse, (before, after))


def test_decode_extreme_values():
    """Scores of +-inf and NaN keys: a row whose every score is -inf is empty, a NaN or +inf key
    makes its head's row NaN, other heads and sequences stay finite."""
    mf = _mf()
    c, _ = ref.make_cache((40, 40, 40, 40), 2, 64, 16, F32, seed=1)
    Q = torch.ones(4, 2, 64)
    slots = torch.arange(40)
    rows = lambda s: (c.table[s].long()[slots // 16], slots % 16)
    p, r = rows(0)
    c.K[p, r, 0] = 0.0
    c.K[p, r, 0, 0] = -math.inf          # every score of (0, head 0) is -inf
    p, r = rows(1)
    c.K[p[5], r[5], 1, 3] = math.nan
    p, r = rows(2)
    c.K[p[39], r[39], 0] = 0.0
    c.K[p[39], r[39], 0, 0] = math.inf   # one +inf
    for dtype in (F32, BF):
        kv = mf.PagedKV(c.K.to(dtype).cuda(), c.V.to(dtype).cuda(), c.table.cuda(),
                        torch.tensor(c.lens, dtype=torch.int32, device="cuda"), 40)
        for max_len in (40, 48):
            kv.max_len = max_len
            lse = torch.empty(4, 2, device="cuda")
            score = torch.zeros(4, 2, 64, device="cuda")
            O = mf.mf_paged_decode(kv, Q.to(dtype).cuda(), lse=lse, score=score)
            _clean(mf)
            assert (O[0, 0] == 0).all() and lse[0, 0] == -math.inf and (score[0, 0] == 0).all()
            assert O[1, 1].isnan().all() and O[2, 0].isnan().all()
            for s, h in ((0, 1), (1, 0), (2, 1), (3, 0), (3, 1)):
                assert torch.isfinite(O[s, h]).all() and torch.isfinite(lse[s, h])
                assert abs(score[s, h].sum().item() - 1.0) < 1e-4


def test_decode_reports_bad_lengths_and_pages():
    mf = _mf()
    c, _ = ref.make_cache((40, 20), 1, 64, 16, BF, seed=2)
    kv = _kv(mf, c)
    Q = torch.randn(2, 1, 64).to(BF)
    O = mf.mf_paged_decode(kv, Q.cuda())
    _clean(mf)
    # a page id out of range reads as zeros
    bad = c.table.clone()
    bad[0, 1] = 1000
    kv.block_table = bad.cuda()
    got = mf.mf_paged_decode(kv, Q.cuda(), o_f32=True)
    rc, bits = mf.mf_get_status()
    assert rc == mf.MF_ERR_DEVICE_INDEX and bits == 16
    slots = torch.arange(16, 32)
    z, _ = ref.make_cache((40, 20), 1, 64, 16, BF, seed=2)
    z.K[c.table[0].long()[slots // 16], slots % 16] = 0
    z.V[c.table[0].long()[slots // 16], slots % 16] = 0
    check_decode(z, Q, got)
    # lengths outside [0, max_len]: taken as the nearest bound
    kv = _kv(mf, c)
    kv.seq_lens = torch.tensor([41, -3], dtype=torch.int32, device="cuda")
    got = mf.mf_paged_decode(kv, Q.cuda())
    rc, bits = mf.mf_get_status()
    assert rc == mf.MF_ERR_DEVICE_INDEX and bits == 1
    assert torch.equal(got[0], O[0]) and (got[1] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_splits_agree_over_batches(dtype):
    """One sequence alone and among others: another split of the same keys, the same result
    within the bound; the largest scale and a given one."""
    mf = _mf()
    c, _ = ref.make_cache((3000, 2000, 10), 2, 128, 16, dtype, seed=5)
    Q = torch.randn(3, 8, 128).to(dtype)
    kv = _kv(mf, c)
    O = mf.mf_paged_decode(kv, Q.cuda(), scale=0.5)
    check_decode(c, Q, O, scale=0.5)
    one = ref.Cache(c.K, c.V, c.table[1:2], c.lens[1:2], c.page)
    O1 = mf.mf_paged_decode(_kv(mf, one), Q[1:2].cuda(), scale=0.5)
    _clean(mf)
    check_decode(one, Q[1:2], O1, scale=0.5)


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("new,lens,h_kv,d,page", [
    ((1, 1, 1), (1, 17, 64), 8, 128, 16),
    ((0, 5, 300, 1), (9, 5, 301, 100), 3, 80, 12),
    ((2000,), (2100,), 2, 64, 64),
    ((7, 0), (7, 0), 64, 256, 3),
])
def test_append(new, lens, h_kv, d, page, dtype):
    mf = _mf()
    c, both = ref.make_cache(lens, h_kv, d, page, dtype, seed=d, interleaved=True)
    kv = _kv(mf, c, both)
    g = torch.Generator().manual_seed(1)
    T = sum(new)
    wide = torch.randn(T + 1, 3 * h_kv * d, generator=g).to(dtype)
    Kn, Vn = (wide[:, k * h_kv * d:(k + 1) * h_kv * d].unflatten(1, (h_kv, d)) for k in (1, 2))
    wd = wide.cuda()
    Kd, Vd = (wd[:, k * h_kv * d:(k + 1) * h_kv * d].unflatten(1, (h_kv, d)) for k in (1, 2))
    cu = torch.tensor([0, *new]).cumsum(0).to(torch.int32).cuda()
    seen = torch.tensor([L + 11 * s for s, L in enumerate(lens)], dtype=torch.int32)
    W = max(lens) + 2
    score = torch.rand(len(lens), h_kv, W, generator=g)
    pos = torch.randint(0, 99, (len(lens), h_kv, W), generator=g, dtype=torch.int32)
    sd, pd = score.cuda(), pos.cuda()
    mf.mf_kv_append(kv, Kd, Vd, cu, max(new), n_seen=seen.cuda(), score=sd, pos=pd)
    _clean(mf)
    at = 0
    for s, (n, L) in enumerate(zip(new, lens)):
        j = torch.arange(L - n, L)
        idx = (c.table[s].long()[j // page], j % page)
        c.K[idx], c.V[idx] = Kn[at:at + n], Vn[at:at + n]
        score[s, :, L - n:L] = 0
        pos[s, :, L - n:L] = torch.arange(n, dtype=torch.int32) + seen[s] - n
        at += n
    assert torch.equal(kv.K.cpu(), c.K) and torch.equal(kv.V.cpu(), c.V)
    assert torch.equal(sd.cpu(), score) and torch.equal(pd.cpu(), pos)
    # without scores and positions only the rows are written, the same ones
    kv.K.zero_()
    mf.mf_kv_append(kv, Kd, Vd, cu, max(new))
    _clean(mf)
    assert int((kv.K != 0).any(-1).sum()) == T * h_kv


def test_append_skips_bad_sequences():
    mf = _mf()
    c, _ = ref.make_cache((20, 20, 20), 1, 64, 16, F32, seed=4)
    kv = _kv(mf, c)
    K0 = kv.K.clone()
    new = torch.randn(24, 1, 64, device="cuda")
    # more new tokens than the sequence holds; past max_new; backwards
    for cu in ([0, 21, 22, 23], [0, 9, 10, 11], [0, 5, 4, 6], [0, 5, 6, 30]):
        kv.K.copy_(K0)
        mf.mf_kv_append(kv, new, new, torch.tensor(cu, dtype=torch.int32, device="cuda"),
                        20 if cu[1] != 9 else 8)
        rc, bits = mf.mf_get_status()
        assert rc == mf.MF_ERR_DEVICE_INDEX and bits == 1, cu
        changed = [int((kv.K != K0)[c.table[s].long().cuda()].any(-1).sum()) for s in range(3)]
        n = [b - a for a, b in zip(cu, cu[1:])]
        ok = [0 <= k <= min(20, 8 if cu[1] == 9 else 20) and b <= 24 for k, b in zip(n, cu[1:])]
        assert changed == [k if good else 0 for k, good in zip(n, ok)], (cu, changed)


# ------------------------------------------------------------------ eviction

def _score_case(kind, shape, g):
    if kind == "random":
        return torch.rand(shape, generator=g)
    if kind == "ties":
        return torch.randint(0, 3, shape, generator=g).float() * 0.5
    if kind == "zeros":
        return torch.where(torch.rand(shape, generator=g) < 0.5, -0.0, 0.0)
    x = torch.randn(shape, generator=g) * 1e3
    special = torch.tensor([math.inf, -math.inf, math.nan, 0.0, -0.0, 3.4028235e38, -3.4028235e38, 1e-45])
    pick = torch.randint(0, 16, shape, generator=g)
    return torch.where(pick < 8, special[pick % 8], x)


EVICT = [
    # lens, budget, sink, window, h_kv, d, page, dtype
    ((65,), 64, 4, 16, 2, 128, 16, BF),
    ((1, 0, 3), 1, 0, 0, 1, 64, 16, BF),
    ((300, 10, 64, 65), 64, 2, 8, 3, 80, 12, F32),
    ((5000, 4097, 777), 1000, 4, 64, 2, 64, 64, BF),
    ((9000,), 8999, 0, 1, 1, 64, 16, BF),
    ((2000, 1999), 1, 0, 1, 2, 256, 7, BF),
    ((40000,), 128, 0, 0, 1, 8, 32, BF),
    ((70, 70), 70, 10, 60, 2, 64, 1, F32),
    ((90,), 20, 10, 10, 1, 64, 16, BF),
    # rows that a CTA of 512 threads takes whole (many of them), and that a cluster of them shares
    ((16384, 15000), 300, 4, 20, 33, 8, 256, BF),
    ((20000, 16385), 12000, 4, 64, 33, 8, 64, BF),
    ((70001,), 20000, 4, 64, 2, 64, 64, F32),
]


@pytest.mark.parametrize("lens,budget,sink,window,h_kv,d,page,dtype", EVICT)
@pytest.mark.parametrize("kind", ["random", "ties", "zeros", "special"])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(lens, budget, sink, window, h_kv, d, page, dtype, kind, in_place):
    mf = _mf()
    c, both = ref.make_cache(lens, h_kv, d, page, dtype, seed=budget, interleaved=True)
    kv = _kv(mf, c, both)
    g = torch.Generator().manual_seed(budget)
    W = max(lens) + 3
    score = _score_case(kind, (len(lens), h_kv, W), g)
    pos = torch.rand(len(lens), h_kv, W, generator=g).argsort(-1).to(torch.int32)
    seen = [W + s for s in range(len(lens))]
    ns = torch.tensor(seen, dtype=torch.int32, device="cuda")
    sd, pd = score.cuda(), pos.cuda()
    if in_place:
        out = mf.mf_kv_evict(kv, sd, pd, budget, sink, window, n_seen=ns)
        assert out is kv.seq_lens
        so, po = sd, pd
        before = (score, pos)
    else:
        so, po = torch.full_like(sd, 9.0), torch.full_like(pd, 9)
        out = mf.mf_kv_evict(kv, sd, pd, budget, sink, window, n_seen=ns, score_out=so, pos_out=po,
                             seq_lens_out=torch.empty_like(kv.seq_lens))
        assert torch.equal(sd.cpu().view(torch.int32), score.view(torch.int32)) and torch.equal(pd.cpu(), pos)
        assert kv.seq_lens.tolist() == list(lens)
    _clean(mf)
    wscore, wpos, wlens = ref.evict(c, score, pos, seen, budget, sink, window)
    assert out.tolist() == wlens
    assert torch.equal(kv.K.cpu(), c.K) and torch.equal(kv.V.cpu(), c.V)
    for s, L in enumerate(lens):
        assert torch.equal(so[s, :, :L].cpu().view(torch.int32), wscore[s, :, :L].contiguous().view(torch.int32))
        assert torch.equal(po[s, :, :L].cpu(), wpos[s, :, :L])
        if in_place:
            assert torch.equal(so[s, :, L:].cpu().view(torch.int32), before[0][s, :, L:].contiguous().view(torch.int32))
        else:
            assert (so[s, :, L:] == 9).all() and (po[s, :, L:] == 9).all()


def test_evict_more_protected_than_budget_and_default_seen():
    """Repeated positions can protect more slots than the budget: the first of them stay.  Without
    n_seen the window counts from the length."""
    mf = _mf()
    c, _ = ref.make_cache((50, 30), 1, 64, 16, F32, seed=9)
    kv = _kv(mf, c)
    score = torch.rand(2, 1, 50)
    pos = torch.zeros(2, 1, 50, dtype=torch.int32)
    sd, pd = score.cuda(), pos.cuda()
    mf.mf_kv_evict(kv, sd, pd, 20, sink=1, window=5)
    _clean(mf)
    wscore, wpos, wlens = ref.evict(c, score, pos, [50, 30], 20, 1, 5)
    assert kv.seq_lens.tolist() == wlens == [20, 20]
    assert torch.equal(sd.cpu(), wscore) and torch.equal(pd.cpu(), wpos) and torch.equal(kv.K.cpu(), c.K)


def test_evict_very_long_row():
    """More slots than a cluster keeps in shared memory: the rest are read again in every round."""
    mf = _mf()
    L, budget = 8 * 32768 + 12345, 5000
    page = 256
    n_pages = -(-L // page)
    K = torch.randn(n_pages, page, 1, 8, device="cuda").to(BF)
    V = torch.randn(n_pages, page, 1, 8, device="cuda").to(BF)
    table = torch.randperm(n_pages, device="cuda").to(torch.int32)[None]
    g = torch.Generator().manual_seed(0)
    score = torch.randint(0, 100000, (1, 1, L), generator=g).float()
    pos = torch.arange(L, dtype=torch.int32)[None, None].contiguous()
    c = ref.Cache(K.cpu(), V.cpu(), table.cpu(), [L], page)
    kv = mf.PagedKV(K, V, table, torch.tensor([L], dtype=torch.int32, device="cuda"), L)
    sd, pd = score.cuda(), pos.cuda()
    mf.mf_kv_evict(kv, sd, pd, budget, 3, 50)
    _clean(mf)
    wscore, wpos, wlens = ref.evict(c, score, pos, [L], budget, 3, 50)
    assert kv.seq_lens.tolist() == wlens
    assert torch.equal(sd.cpu(), wscore) and torch.equal(pd.cpu(), wpos)
    assert torch.equal(K.cpu(), c.K) and torch.equal(V.cpu(), c.V)


# ------------------------------------------------------------------ key scores

SCORES = [
    # lens, B, h_s, h_kv, group, dtype
    ((256,), 32, 4, 1, 2, F32),
    ((300, 0, 77), 64, 32, 8, 4, BF),
    ((130, 1), 128, 40, 3, 1, BF),
    ((200,), 64, 7, 2, 3, F32),
    ((150, 129), 128, 3, 1, 16, F32),
    ((64, 65, 63), 32, 33, 4, 2, BF),
    ((1000,), 64, 70, 64, 1, BF),
    ((500,), 64, 256, 2, 2, BF),
]


@pytest.mark.parametrize("lens,B,h_s,h_kv,group,dtype", SCORES)
@pytest.mark.parametrize("junk", [None, float("nan")])
def test_key_scores(lens, B, h_s, h_kv, group, dtype, junk):
    mf = _mf()
    values, row_ptr, cols, base = ref.make_bsr(lens, B, h_s, dtype, seed=B + h_s, junk=junk, gap=2)
    W = torch.randn(h_kv * group, h_s, generator=torch.Generator().manual_seed(2)) / math.sqrt(h_s)
    # a BSR with spare capacity
    spare = 3
    bsr = mf.BSR(row_ptr.cuda(), torch.cat([cols, torch.full((spare,), 999, dtype=torch.int32)]).cuda(),
                 torch.cat([values, torch.full((spare,) + tuple(values.shape[1:]), float("nan"), dtype=dtype)]).cuda(),
                 row_ptr[-1:].cuda())
    cu = torch.tensor([0, *lens]).cumsum(0).to(torch.int32).cuda()
    score = torch.full((len(lens), h_kv, max(lens) + 2), 3.0, device="cuda")
    mf.mf_map_key_scores(bsr, W.cuda(), cu, torch.tensor(base, dtype=torch.int32, device="cuda"),
                         max(lens), h_kv, score=score)
    _clean(mf)
    want, mag = ref.key_scores(values, row_ptr, cols, W, lens, base, B, h_kv)
    # float32: B additions down a column, h_s terms of the mix (group weights rounded first), one rounding
    tol = (B + h_s + group + 8) * 2.0 ** -23 * mag + 1e-30
    for s, L in enumerate(lens):
        err = (score[s, :, :L].double().cpu() - want[s, :, :L]).abs()
        assert (err <= tol[s, :, :L]).all(), (s, (err - tol[s, :, :L]).max())
        assert (score[s, :, L:] == 3.0).all()
    again = mf.mf_map_key_scores(bsr, W.cuda(), cu, torch.tensor(base, dtype=torch.int32, device="cuda"),
                                 max(lens) + 100, h_kv)
    for s, L in enumerate(lens):
        assert torch.equal(again[s, :, :L], score[s, :, :L])


def test_key_scores_reports_bad_indices():
    mf = _mf()
    values, row_ptr, cols, base = ref.make_bsr((200,), 64, 4, BF, seed=1)
    W = torch.ones(2, 4, device="cuda")
    cu = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    b = torch.tensor(base, dtype=torch.int32, device="cuda")

    def run(rp=row_ptr, ci=cols, cu=cu, b=b):
        mf.mf_map_key_scores(mf.BSR(rp.cuda(), ci.cuda(), values.cuda(), rp[-1:].cuda()), W, cu, b, 200, 1)
        return mf.mf_get_status()

    assert run() == (mf.MF_OK, 0)
    bad = cols.clone()
    bad[-1] = 77
    assert run(ci=bad) == (mf.MF_ERR_DEVICE_INDEX, 1)
    bad = row_ptr.clone()
    bad[-1] += 5
    assert run(rp=bad) == (mf.MF_ERR_DEVICE_INDEX, 1)
    assert run(cu=torch.tensor([0, 300], dtype=torch.int32, device="cuda")) == (mf.MF_ERR_DEVICE_INDEX, 1)
    assert run(b=torch.tensor([2], dtype=torch.int32, device="cuda")) == (mf.MF_ERR_DEVICE_INDEX, 1)


# ------------------------------------------------------------------ streams and graphs

def test_decode_step_captured_and_replayed():
    """append + decode + evict captured once, replayed with new inputs: lengths, scores and
    positions live on the device, so the graph needs no host values."""
    mf = _mf()
    lens, cap, budget = [60, 64, 33], 65, 64
    h_kv, G, d, page = 2, 4, 64, 16
    c, _ = ref.make_cache(lens, h_kv, d, page, BF, seed=11, capacity=[cap] * 3)
    kv = _kv(mf, c, max_len=cap)
    Q = torch.zeros(3, h_kv * G, d, dtype=BF, device="cuda")
    Kn, Vn = (torch.zeros(3, h_kv, d, dtype=BF, device="cuda") for _ in range(2))
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    seen = kv.seq_lens.clone()
    score = torch.zeros(3, h_kv, cap, device="cuda")
    pos = torch.arange(cap, dtype=torch.int32, device="cuda").expand(3, h_kv, cap).contiguous()
    O = torch.empty(3, h_kv * G, d, dtype=F32, device="cuda")
    wd = torch.empty(mf.mf_paged_decode_workspace_size(kv, h_kv * G, scores=True), dtype=torch.uint8, device="cuda")
    we = torch.empty(mf.mf_kv_evict_workspace_size(kv, budget), dtype=torch.uint8, device="cuda")

    def step():
        kv.seq_lens.add_(1)
        seen.add_(1)
        mf.mf_kv_append(kv, Kn, Vn, cu, 1, n_seen=seen, score=score, pos=pos)
        mf.mf_paged_decode(kv, Q, O=O, score=score, o_f32=True, workspace=wd)
        mf.mf_kv_evict(kv, score, pos, budget, sink=2, window=8, n_seen=seen, workspace=we)

    state = [t.clone() for t in (kv.K, kv.V, kv.seq_lens, seen, score, pos)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, v in zip((kv.K, kv.V, kv.seq_lens, seen, score, pos), state):
        t.copy_(v)
    g = torch.Generator().manual_seed(5)
    hseen = list(lens)
    hpos = pos.cpu()
    for _ in range(8):
        q, k, v = (torch.randn(t.shape, generator=g).to(BF) for t in (Q, Kn, Vn))
        Q.copy_(q)
        Kn.copy_(k)
        Vn.copy_(v)
        before = score.clone().cpu()
        graph.replay()
        torch.cuda.synchronize()
        # the same step on the host: the eviction goes by the device's own scores
        c.lens = [L + 1 for L in c.lens]
        hseen = [n + 1 for n in hseen]
        for s in range(3):
            j = c.lens[s] - 1
            c.K[c.table[s, j // page], j % page] = k[s]
            c.V[c.table[s, j // page], j % page] = v[s]
            before[s, :, j] = 0
            hpos[s, :, j] = hseen[s] - 1
        check_decode(c, q, O)
        _, _, w, dx, _, _ = ref.decode(c, q)
        total = before.double()
        total[:, :, :w.shape[2]] += w
        hscore, hpos, c.lens = ref.evict(c, total.float(), hpos, hseen, budget, 2, 8)
        assert kv.seq_lens.tolist() == c.lens
        assert torch.equal(pos.cpu(), hpos)
        assert torch.equal(kv.K.cpu(), c.K) and torch.equal(kv.V.cpu(), c.V)
        assert ((score.cpu() - hscore).abs() <= 1e-5).all()
    _clean(mf)


def test_side_streams_and_two_calls_at_once():
    """Two decodes at the same time on two streams, each with its own workspace, and calls that
    allocate their own on a stream that is not current."""
    mf = _mf()
    cases = []
    for k in range(2):
        c, _ = ref.make_cache((3000, 500), 4, 128, 16, BF, seed=20 + k)
        Q = torch.randn(2, 16, 128, generator=torch.Generator().manual_seed(k)).to(BF)
        cases.append((c, Q, _kv(mf, c), Q.cuda(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[mf.mf_paged_decode(kv, Qd, stream=st) for _ in range(3)] for _ in range(2) for _, _, kv, Qd, st in cases]
    torch.cuda.synchronize()
    _clean(mf)
    for i, o in enumerate(outs):
        c, Q = cases[i % 2][:2]
        check_decode(c, Q, o[0])
        assert all(torch.equal(o[0], x) for x in o)


# ------------------------------------------------------------------ the operators together

def test_receiver_decodes_after_reused_prefill():
    """A receiver's path: the sender's maps compressed from Q and K, the prefill attention
    retrieved through the pages that mf_kv_append filled, the weights gathered by the prefill, the
    cache cut back by them, then decode steps that gather on and evict, against float64."""
    mf = _mf()
    from synth.qk import gen_qk
    lens, h_s, B, tau = (300, 77), 8, 64, 1.0
    h_kv, G, d, page, budget = 2, 4, 128, 16, 48
    h_r = h_kv * G
    Qs, Ks = gen_qk(lens, h_s, 2, d, 8, 0)
    cu = torch.tensor([0, 300, 377], dtype=torch.int32, device="cuda")
    nqb = [-(-L // B) for L in lens]
    n_c = sum(n * (n + 1) // 2 for n in nqb)
    bsr = mf.alloc_bsr(sum(nqb), n_c, h_s, B, BF, "cuda")
    mf.mf_compress_qk(Qs.cuda(), Ks.cuda(), cu, max(lens), B, tau, bsr)
    g = torch.Generator().manual_seed(3)
    W = (torch.rand(1, h_r, h_s, generator=g) / h_s)
    base = torch.tensor([0, nqb[0]], dtype=torch.int32, device="cuda")
    # the receiver's own keys and values go into the pages, the prefill reads its V from them
    cap = [L + 8 for L in lens]
    c, _ = ref.make_cache(list(lens), h_kv, d, page, BF, seed=8, capacity=cap)
    kv = _kv(mf, c, max_len=max(cap))
    Kp, Vp = (torch.randn(377, h_kv, d, generator=g).to(BF) for _ in range(2))
    pos = torch.full((2, h_kv, max(cap)), -1, dtype=torch.int32, device="cuda")
    mf.mf_kv_append(kv, Kp.cuda(), Vp.cuda(), cu, 300, pos=pos)
    O = mf.mf_map_retrieve([bsr], [0], W.cuda(), kv.V, cu, cu, base, max(lens), h_r, h_kv, total_q=377,
                           paged=(kv.block_table, page))[0]
    score = torch.zeros(2, h_kv, max(cap), device="cuda")
    mf.mf_map_key_scores(bsr, W[0].cuda(), cu, base, max(lens), h_kv, score=score)
    _clean(mf)
    n = int(bsr.nnz.item())
    rp, ci, vals = bsr.row_ptr.cpu(), bsr.col_idx.cpu()[:n], bsr.values.cpu()[:n]
    want, mag = ref.key_scores(vals, rp, ci, W[0], lens, [0, nqb[0]], B, h_kv)
    assert ((score.cpu().double()[:, :, :300] - want).abs() <= (B + h_s + G + 8) * 2.0 ** -23 * mag + 1e-30).all()
    # the weights are those of the prefill that retrieval computed: with V = 1 for one key and 0
    # elsewhere its output would sum to that key's score; here on the first key of sequence 1
    at = 0
    for s, L in enumerate(lens):
        j = torch.arange(L)
        idx = (c.table[s].long()[j // page], j % page)
        c.K[idx], c.V[idx] = Kp[at:at + L], Vp[at:at + L]
        assert torch.equal(pos[s, :, :L].cpu(), j.to(torch.int32).expand(h_kv, L))
        at += L
    assert torch.equal(kv.V.cpu(), c.V) and O.shape == (377, h_r, d)
    one = torch.zeros_like(kv.V)
    one[c.table[1, 0].item(), 0] = 1
    O1 = mf.mf_map_retrieve([bsr], [0], W.cuda(), one, cu, cu, base, max(lens), h_r, h_kv, total_q=377,
                            paged=(kv.block_table, page), o_f32=True)[0]
    got = O1[300:, :, 0].double().sum(0).view(h_kv, G).sum(1).cpu()
    # the retrieval takes W and P as bf16 pairs: 2^-15 of the terms covers both
    assert ((got - want[1, :, 0]).abs() <= 2.0 ** -15 * mag[1, :, 0]).all()
    # decode
    seen = kv.seq_lens.clone()
    hseen, hpos = list(lens), pos.cpu()
    for step in range(5):
        q = torch.randn(2, h_r, d, generator=g).to(BF)
        k, v = (torch.randn(2, h_kv, d, generator=g).to(BF) for _ in range(2))
        kv.seq_lens.add_(1)
        seen.add_(1)
        mf.mf_kv_append(kv, k.cuda(), v.cuda(), torch.arange(3, dtype=torch.int32, device="cuda"), 1,
                        n_seen=seen, score=score, pos=pos)
        before = score.clone()
        lse = torch.empty(2, h_r, device="cuda")
        O = mf.mf_paged_decode(kv, q.cuda(), lse=lse, score=score)
        gathered = score.clone()
        c.lens = [L + 1 for L in c.lens]
        hseen = [x + 1 for x in hseen]
        for s in range(2):
            j = c.lens[s] - 1
            c.K[c.table[s, j // page], j % page], c.V[c.table[s, j // page], j % page] = k[s], v[s]
            hpos[s, :, j] = hseen[s] - 1
        check_decode(c, q, O, lse, (before, gathered))
        mf.mf_kv_evict(kv, score, pos, budget, sink=4, window=16, n_seen=seen)
        hscore, hpos, c.lens = ref.evict(c, gathered.cpu(), hpos, hseen, budget, 4, 16)
        assert kv.seq_lens.tolist() == c.lens
        assert torch.equal(score.cpu(), hscore) and torch.equal(pos.cpu(), hpos)
        assert torch.equal(kv.K.cpu(), c.K) and torch.equal(kv.V.cpu(), c.V)
    _clean(mf)


def test_key_scores_of_shared_rows():
    """Two sequences over the same rows of the maps: equally long they both get the scores; where
    they disagree on what a row holds it is reported, and no kept entry past an end is used."""
    mf = _mf()
    values, row_ptr, cols, base = ref.make_bsr((200,), 64, 4, BF, seed=1)
    bsr = mf.BSR(row_ptr.cuda(), cols.cuda(), values.cuda(), row_ptr[-1:].cuda())
    W = torch.rand(2, 4, generator=torch.Generator().manual_seed(1))
    b = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    score = mf.mf_map_key_scores(bsr, W.cuda(), torch.tensor([0, 200, 400], dtype=torch.int32, device="cuda"), b, 200, 1)
    _clean(mf)
    want, mag = ref.key_scores(values, row_ptr, cols, W, (200,), base, 64, 1)
    tol = (64 + 4 + 2 + 8) * 2.0 ** -23 * mag + 1e-30
    for s in range(2):
        assert ((score[s].double().cpu() - want[0]).abs() <= tol[0]).all()
    mf.mf_map_key_scores(bsr, W.cuda(), torch.tensor([0, 200, 390], dtype=torch.int32, device="cuda"), b, 200, 1)
    assert mf.mf_get_status() == (mf.MF_ERR_DEVICE_INDEX, 1)


def test_key_scores_without_blocks():
    """No rows, no kept blocks, no tokens."""
    mf = _mf()
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    empty = torch.zeros(0, 2, 32, 32, device="cuda")
    W = torch.ones(2, 2, device="cuda")
    cu = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    for top in (0, 40):
        score = torch.full((1, 1, 40), 2.0, device="cuda")
        mf.mf_map_key_scores(mf.BSR(zero, none, empty, zero), W, cu, zero, top, 1, score=score)
        _clean(mf)
        assert (score == 2.0).all()
    # rows without a kept block: the keys gathered nothing
    score = torch.full((1, 1, 45), 2.0, device="cuda")
    rows = torch.zeros(3, dtype=torch.int32, device="cuda")
    mf.mf_map_key_scores(mf.BSR(rows, none, empty, zero), W, torch.tensor([0, 40], dtype=torch.int32, device="cuda"), zero, 40, 1,
                         score=score)
    _clean(mf)
    assert (score[..., :40] == 0).all() and (score[..., 40:] == 2.0).all()


# ------------------------------------------------------------------ what the binding refuses

def test_binding_refusals():
    mf = _mf()
    c, _ = ref.make_cache((40, 20), 2, 64, 16, BF, seed=2, spare=3)
    kv = _kv(mf, c)
    Q = torch.zeros(2, 8, 64, dtype=BF, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    score, pos = torch.zeros(2, 2, 40, device="cuda"), torch.zeros(2, 2, 40, dtype=torch.int32, device="cuda")
    new = torch.zeros(2, 2, 64, dtype=BF, device="cuda")

    def with_kv(**kw):
        f = dict(K=kv.K, V=kv.V, block_table=kv.block_table, seq_lens=kv.seq_lens, max_len=40)
        f.update(kw)
        return mf.PagedKV(**f)

    def no(match, call, error=ValueError):
        with pytest.raises(error, match=match):
            call()

    for bad, match in ((dict(V=kv.V[:-1]), "shape"), (dict(V=kv.V.float()), "must be"), (dict(K=kv.K.cpu()), "CUDA"),
                       (dict(K=kv.K[0]), "dimensions"), (dict(K=kv.K[:, :, :, ::2], V=kv.V[:, :, :, ::2]), "dense"),
                       (dict(V=torch.cat([kv.V, kv.V], 1)[:, :16]), "same stride"), (dict(seq_lens=i32(1)), "shape"),
                       (dict(seq_lens=kv.seq_lens.long()), "must be"), (dict(block_table=kv.block_table.t()), "contiguous|shape"),
                       (dict(max_len=1 << 31), "32 bits"), (dict(K=None), "CUDA")):
        for call in (lambda: mf.mf_paged_decode(with_kv(**bad), Q), lambda: mf.mf_kv_evict(with_kv(**bad), score, pos, 5),
                     lambda: mf.mf_kv_append(with_kv(**bad), new, new, i32(0, 1, 2), 1), lambda: with_kv(**bad).desc()):
            no(match, call)
    no("dtype", lambda: mf.mf_paged_decode(with_kv(K=kv.K.half(), V=kv.V.half()), Q.half()), TypeError)
    no("int", lambda: mf.mf_paged_decode(with_kv(max_len="40"), Q), TypeError)
    no("K", lambda: mf.mf_paged_decode(object(), Q), AttributeError)
    for args, match in ((dict(Q=Q.float()), "must be"), (dict(Q=Q[:1]), "shape"), (dict(Q=Q[..., :32]), "shape"),
                        (dict(Q=Q.transpose(1, 2).contiguous().transpose(1, 2)), "dense"), (dict(O=Q.float()), "must be"),
                        (dict(O=Q[:, ::2]), "shape"), (dict(O=Q, o_f32=True), "must be"), (dict(lse=score), "shape"),
                        (dict(score=score[:, :, ::2]), "contiguous"), (dict(score=score, score_out=score[:, :, 1:]), "shape|contiguous"),
                        (dict(score=pos), "must be"), (dict(workspace=torch.empty(9)), "CUDA"),
                        (dict(workspace=torch.empty(4, 4, device="cuda").t()), "contiguous")):
        a = dict(Q=Q)
        a.update(args)
        no(match, lambda: mf.mf_paged_decode(kv, **a))
    for args in (dict(Q=Q[:, :7].contiguous()), dict(scale=-1.0), dict(score=torch.zeros(2, 2, 39, device="cuda")),
                 dict(workspace=torch.empty(16, device="cuda"))):
        a = dict(Q=Q)
        a.update(args)
        no("mf status 1", lambda: mf.mf_paged_decode(kv, **a), mf.MFError)
    no("shape", lambda: mf.mf_kv_append(kv, new, new[:1], i32(0, 1, 2), 1))
    no("shape", lambda: mf.mf_kv_append(kv, new, new, i32(0, 1), 1))
    no("mf status 1", lambda: mf.mf_kv_append(kv, new, new, i32(0, 1, 2), 41), mf.MFError)
    no("32 bits", lambda: mf.mf_kv_append(kv, new, new, i32(0, 1, 2), -(1 << 40)))
    no("shape", lambda: mf.mf_kv_evict(kv, score, pos[:, :, 1:], 5))
    no("32 bits", lambda: mf.mf_kv_evict(kv, score, pos, (1 << 32) + 5))
    no("mf status 1", lambda: mf.mf_kv_evict(kv, score, pos, 5, 3, 3), mf.MFError)
    no("int|attribute", lambda: mf.mf_kv_evict(kv, score, pos, 5, stream=7), AttributeError)
    values, row_ptr, cols, base = ref.make_bsr((40,), 32, 2, BF)
    bsr = mf.BSR(row_ptr.cuda(), cols.cuda(), values.cuda(), row_ptr[-1:].cuda())
    W = torch.zeros(4, 2, device="cuda")
    for args, match in ((dict(W=W[:, :1].contiguous()), "shape"), (dict(W=W.to(BF)), "must be"), (dict(h_kv=0), "h_kv"),
                        (dict(cu_seqlens=i32()), "cu_seqlens"), (dict(qblock_base=i32(0, 1)), "shape"),
                        (dict(score=score), "shape"), (dict(max_seqlen=1 << 33), "32 bits"),
                        (dict(bsr=mf.BSR(row_ptr.cuda(), cols[:1].cuda(), values.cuda(), row_ptr[-1:].cuda())), "capacity")):
        a = dict(bsr=bsr, W=W, cu_seqlens=i32(0, 40), qblock_base=i32(0), max_seqlen=40, h_kv=2)
        a.update(args)
        no(match, lambda: mf.mf_map_key_scores(**a))
    _clean(mf)
    assert (score == 0).all() and (pos == 0).all()


def test_calls_on_a_stream_that_is_not_current():
    """Outputs, zeros and workspaces that a call allocates belong to the call's stream: work that is
    still queued on the current stream does not disturb them."""
    mf = _mf()
    c, _ = ref.make_cache((700, 90), 2, 64, 16, BF, seed=31)
    kv = _kv(mf, c)
    Q = torch.randn(2, 8, 64, generator=torch.Generator().manual_seed(1)).to(BF)
    Qd = Q.cuda()
    values, row_ptr, cols, base = ref.make_bsr((200,), 64, 4, BF, seed=1)
    bsr = mf.BSR(row_ptr.cuda(), cols.cuda(), values.cuda(), row_ptr[-1:].cuda())
    W = torch.rand(2, 4, generator=torch.Generator().manual_seed(1))
    Wd = W.cuda()
    cu = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    big = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(8):
        big = big @ big * 1e-3  # the current stream is busy, and frees what it used
    O = mf.mf_paged_decode(kv, Qd, stream=side)
    score = mf.mf_map_key_scores(bsr, Wd, cu, zero, 200, 1, stream=side)
    side.synchronize()
    check_decode(c, Q, O)
    want, mag = ref.key_scores(values, row_ptr, cols, W, (200,), base, 64, 1)
    assert ((score.double().cpu() - want).abs() <= (64 + 4 + 2 + 8) * 2.0 ** -23 * mag + 1e-30).all()
    torch.cuda.synchronize()
    _clean(mf)


@pytest.mark.parametrize("lens,h_kv,group,d,dtype", [
    ((5, 0, 33, 1), 2, 4, 128, BF), ((16, 64, 65, 130), 3, 3, 80, BF), ((9, 40, 0, 3), 1, 20, 96, BF),
    ((7, 8, 9, 0), 2, 5, 72, F32), ((200, 1, 64, 500), 2, 4, 96, F32), ((63,), 1, 12, 64, F32),
    (tuple(range(0, 150)), 4, 2, 64, BF), ((400,) * 40, 2, 1, 104, F32)])
def test_decode_short_sequences_under_a_long_bound(lens, h_kv, group, d, dtype):
    """The length bound of a serving loop is far above the lengths: the keys are split all the same,
    into units of their own where there are few, and the weights go through the second kernel."""
    mf = _mf()
    c, _ = ref.make_cache(lens, h_kv, d, 16, dtype, seed=d, stale=float("nan"))
    Q = torch.randn(len(lens), h_kv * group, d, generator=torch.Generator().manual_seed(4)).to(dtype)
    kv = _kv(mf, c, max_len=6000)
    before = torch.rand(len(lens), h_kv, 6000, generator=torch.Generator().manual_seed(5)).cuda()
    after = before.clone()
    lse = torch.empty(len(lens), h_kv * group, device="cuda")
    O = mf.mf_paged_decode(kv, Q.cuda(), lse=lse, score=after)
    _clean(mf)
    check_decode(c, Q, O, lse, (before, after))
    assert torch.equal(O, mf.mf_paged_decode(kv, Q.cuda()))


# ------------------------------------------------------------------ borders

@pytest.mark.parametrize("dtype", [BF, F32])
def test_nothing_held(dtype):
    """max_len 0: every call succeeds, empty rows get O = 0 and lse = -inf, nothing else changes."""
    mf = _mf()
    K, V = torch.ones(2, 4, 2, 64, device="cuda").to(dtype), torch.ones(2, 4, 2, 64, device="cuda").to(dtype)
    kv = mf.PagedKV(K, V, torch.full((3, 1), -1, dtype=torch.int32, device="cuda"),
                    torch.zeros(3, dtype=torch.int32, device="cuda"), 0)
    for G in (1, 4, 20):
        lse = torch.zeros(3, 2 * G, device="cuda")
        score = torch.full((3, 2, 1), 5.0, device="cuda")
        O = mf.mf_paged_decode(kv, torch.ones(3, 2 * G, 64, device="cuda").to(dtype), lse=lse, score=score)
        _clean(mf)
        assert (O == 0).all() and (lse == -math.inf).all() and (score == 5.0).all()
    pos = torch.full((3, 2, 1), 7, dtype=torch.int32, device="cuda")
    mf.mf_kv_append(kv, K[0, :0], V[0, :0], torch.zeros(4, dtype=torch.int32, device="cuda"), 0, score=score, pos=pos)
    out = mf.mf_kv_evict(kv, score, pos, 3)
    _clean(mf)
    assert out.tolist() == [0, 0, 0] and (score == 5.0).all() and (pos == 7).all() and (K == 1).all() and (V == 1).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_largest_batch(dtype):
    """4096 sequences, with the keys split and with a CTA to a unit."""
    mf = _mf()
    n, page, d = 4096, 4, 64
    g = torch.Generator().manual_seed(6)
    lens = torch.randint(0, 9, (n,), generator=g).tolist()
    lens[7], lens[4095] = 700, 40
    K, V = (torch.randn(300, page, 1, d, generator=g).to(dtype) for _ in range(2))
    table = torch.randint(0, 300, (n, 175), generator=g).to(torch.int32)
    c = ref.Cache(K, V, table, lens, page)
    Q = torch.randn(n, 2, d, generator=g).to(dtype)
    kv = mf.PagedKV(K.cuda(), V.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), 700)
    lse = torch.empty(n, 2, device="cuda")
    O = mf.mf_paged_decode(kv, Q.cuda(), lse=lse)
    _clean(mf)
    check_decode(c, Q, O, lse)
    c.lens = [min(L, 40) for L in lens]
    kv.seq_lens.clamp_(max=40)
    kv.max_len = 40
    before = torch.zeros(n, 1, 40, device="cuda")
    after = before.clone()
    O = mf.mf_paged_decode(kv, Q.cuda(), score=after)
    _clean(mf)
    check_decode(c, Q, O, None, (before, after))


@pytest.mark.parametrize("lens,h_kv,group,dtype", [((300, 17), 1, 256, BF), ((100,), 1, 256, F32), ((250, 40, 3), 2, 20, BF),
                                                   ((120, 9), 3, 9, F32), ((511, 512), 64, 4, BF), ((900,), 64, 2, F32)])
def test_decode_many_heads(lens, h_kv, group, dtype):
    """Groups of several blocks of heads, with and without a second launch; 64 key heads."""
    mf = _mf()
    c, _ = ref.make_cache(lens, h_kv, 64, 16, dtype, seed=group, stale=float("nan"))
    Q = torch.randn(len(lens), h_kv * group, 64, generator=torch.Generator().manual_seed(4)).to(dtype)
    for top in (max(lens), 3000):
        kv = _kv(mf, c, max_len=top)
        before = torch.rand(len(lens), h_kv, top, generator=torch.Generator().manual_seed(5)).cuda()
        after = before.clone()
        lse = torch.empty(len(lens), h_kv * group, device="cuda")
        O = mf.mf_paged_decode(kv, Q.cuda(), lse=lse, score=after)
        _clean(mf)
        check_decode(c, Q, O, lse, (before, after))


def test_evict_extreme_positions():
    """Windows and positions at the ends of 32 bits."""
    mf = _mf()
    top, low = 2 ** 31 - 1, -2 ** 31
    for seen, sink, window in ((low, 0, 5), (top, 3, 5), (5, 0, 0), (0, 2, 5), (low, 4, 0)):
        c, _ = ref.make_cache((50,), 1, 64, 16, F32, seed=9)
        kv = _kv(mf, c)
        g = torch.Generator().manual_seed(1)
        score = torch.rand(1, 1, 50, generator=g)
        pos = torch.tensor([low, low + 1, -1, 0, 1, 2, top - 4, top - 1, top] + list(range(10, 51)), dtype=torch.int32)[None, None].contiguous()
        sd, pd = score.cuda(), pos.cuda()
        mf.mf_kv_evict(kv, sd, pd, 20, sink=sink, window=window, n_seen=torch.tensor([seen], dtype=torch.int32, device="cuda"))
        _clean(mf)
        wscore, wpos, wlens = ref.evict(c, score, pos, [seen], 20, sink, window)
        assert kv.seq_lens.tolist() == wlens
        assert torch.equal(sd.cpu(), wscore) and torch.equal(pd.cpu(), wpos) and torch.equal(kv.K.cpu(), c.K)


def test_evict_reports_bad_lengths_and_pages():
    """A length out of range counts as the nearest bound; rows on a page that does not exist read as
    zeros and are not written."""
    mf = _mf()
    c, _ = ref.make_cache((40, 40), 1, 64, 16, F32, seed=3)
    kv = _kv(mf, c)
    score = torch.arange(40).float().expand(2, 1, 40).contiguous()
    pos = torch.arange(40, dtype=torch.int32).expand(2, 1, 40).contiguous()
    sd, pd = score.cuda(), pos.cuda()
    kv.seq_lens = torch.tensor([55, -2], dtype=torch.int32, device="cuda")
    mf.mf_kv_evict(kv, sd, pd, 10)
    assert mf.mf_get_status() == (mf.MF_ERR_DEVICE_INDEX, 1)
    wscore, wpos, _ = ref.evict(ref.Cache(c.K, c.V, c.table, [40, 0], c.page), score, pos, [40, 0], 10, 0, 0)
    assert kv.seq_lens.tolist() == [10, 0]
    assert torch.equal(sd.cpu(), wscore) and torch.equal(pd.cpu(), wpos) and torch.equal(kv.K.cpu(), c.K)
    # the movers' page is missing: they arrive as zeros
    c, _ = ref.make_cache((40,), 1, 64, 16, F32, seed=3)
    kv = _kv(mf, c)
    kv.block_table[0, 2] = 99
    sd, pd = score[:1].cuda(), pos[:1].cuda()
    K0 = kv.K.clone()
    mf.mf_kv_evict(kv, sd, pd, 10)
    assert mf.mf_get_status() == (mf.MF_ERR_DEVICE_INDEX, 16)
    first = c.table[0, 0].item()
    got = kv.K.cpu()
    # kept: slots 30 .. 39; 30 and 31 lie on the second page, 32 .. 39 on the missing one
    assert torch.equal(got[first, 0], K0.cpu()[c.table[0, 1].item(), 14]) and torch.equal(got[first, 1], K0.cpu()[c.table[0, 1].item(), 15])
    assert (got[first, 2:10] == 0).all() and pd[0, 0, :10].tolist() == list(range(30, 40))
    got[first, :10] = K0.cpu()[first, :10]
    assert torch.equal(got, K0.cpu())


def test_pages_beyond_four_gigabytes():
    """Rows whose offsets pass 32 bits, in bytes and in elements: append, decode and eviction on the
    last pages of a pool of 9 GB for K and for V."""
    mf = _mf()
    page, h_kv, d, n_pages = 16, 8, 128, 280000
    K, V = (torch.empty(n_pages, page, h_kv, d, dtype=BF, device="cuda") for _ in range(2))
    assert K.numel() > 2 ** 32
    small, _ = ref.make_cache((70, 33), h_kv, d, page, BF, seed=17, spare=0)
    n = small.K.shape[0]
    first = n_pages - n
    K[:n].zero_(), V[:n].zero_()
    table = torch.where(small.table >= 0, small.table + first, small.table).cuda()
    kv = mf.PagedKV(K, V, table, torch.tensor(small.lens, dtype=torch.int32, device="cuda"), 70)
    idx = [(small.table[s].long()[torch.arange(L) // page], torch.arange(L) % page) for s, L in enumerate(small.lens)]
    Kn, Vn = (torch.cat([t[i] for i in idx]).cuda() for t in (small.K, small.V))
    score, pos = torch.rand(2, h_kv, 70, device="cuda"), torch.zeros(2, h_kv, 70, dtype=torch.int32, device="cuda")
    mf.mf_kv_append(kv, Kn, Vn, torch.tensor([0, 70, 103], dtype=torch.int32, device="cuda"), 70, score=score, pos=pos)
    Q = torch.randn(2, 4 * h_kv, d, generator=torch.Generator().manual_seed(2)).to(BF)
    check_decode(small, Q, mf.mf_paged_decode(kv, Q.cuda(), score=score))
    kv.max_len = 4000  # split
    wide = torch.zeros(2, h_kv, 4000, device="cuda")
    check_decode(small, Q, mf.mf_paged_decode(kv, Q.cuda(), score=wide), None, (torch.zeros_like(wide), wide))
    before = score.cpu()
    kv.max_len = 70
    mf.mf_kv_evict(kv, score, pos, 40, 2, 8)
    _clean(mf)
    hpos = torch.zeros(2, h_kv, 70, dtype=torch.int32)
    for s, L in enumerate(small.lens):
        hpos[s, :, :L] = torch.arange(L, dtype=torch.int32)
    wscore, wpos, wlens = ref.evict(small, before, hpos, [70, 33], 40, 2, 8)
    assert kv.seq_lens.tolist() == wlens and torch.equal(score.cpu(), wscore) and torch.equal(pos.cpu(), wpos)
    for s, L in enumerate(wlens):
        p, r = small.table[s].long()[torch.arange(L) // page], torch.arange(L) % page
        assert torch.equal(K[(p + first).cuda(), r.cuda()].cpu(), small.K[p, r])
        assert torch.equal(V[(p + first).cuda(), r.cuda()].cpu(), small.V[p, r])
    assert (K[:n] == 0).all() and (V[:n] == 0).all()


# ------------------------------------------------------------------ order among kernels

def _order_case(mf):
    """The four calls over one cache, and what they read, as one list of tensors."""
    lens, h_kv, G, d, page, cap = [600, 77, 1, 0], 2, 4, 64, 16, 640
    c, _ = ref.make_cache(lens, h_kv, d, page, BF, seed=41, capacity=[cap] * 4)
    kv = _kv(mf, c, max_len=cap)
    g = torch.Generator().manual_seed(8)
    Q, Kn, Vn = (torch.randn(4, n, d, generator=g).to(BF).cuda() for n in (h_kv * G, h_kv, h_kv))
    score = torch.rand(4, h_kv, cap, generator=g).cuda()
    pos = torch.arange(cap, dtype=torch.int32, device="cuda").expand(4, h_kv, cap).contiguous()
    seen = kv.seq_lens.clone()
    values, row_ptr, cols, base = ref.make_bsr((600, 77, 1), 64, 4, BF, seed=1)
    bsr = mf.BSR(row_ptr.cuda(), cols.cuda(), values.cuda(), row_ptr[-1:].cuda())
    W = torch.rand(h_kv * G, 4, generator=g).cuda()
    cu = torch.tensor([0, 600, 677, 678], dtype=torch.int32, device="cuda")
    qb = torch.tensor(base, dtype=torch.int32, device="cuda")
    one = torch.arange(5, dtype=torch.int32, device="cuda")
    outs = dict(O=torch.zeros(4, h_kv * G, d, device="cuda"), lse=torch.zeros(4, h_kv * G, device="cuda"),
                keys=torch.zeros(3, h_kv, 600, device="cuda"), so=torch.zeros_like(score), po=torch.zeros_like(pos),
                lo=torch.zeros_like(kv.seq_lens), after=torch.zeros_like(score))
    inputs = [kv.K, kv.V, kv.block_table, kv.seq_lens, Q, Kn, Vn, score, pos, seen, bsr.row_ptr, bsr.col_idx, bsr.values, W, cu, qb]
    ws = torch.empty(max(mf.mf_paged_decode_workspace_size(kv, h_kv * G, True), mf.mf_kv_evict_workspace_size(kv, 64),
                         mf.mf_map_key_scores_workspace_size(bsr.capacity, 64, h_kv)), dtype=torch.uint8, device="cuda")

    def step():  # one workspace for all: each call may use it once the one before is done
        kv.seq_lens.add_(1)
        seen.add_(1)
        mf.mf_kv_append(kv, Kn, Vn, one, 1, n_seen=seen, score=score, pos=pos)
        mf.mf_map_key_scores(bsr, W, cu, qb, 600, h_kv, score=outs["keys"], workspace=ws)
        mf.mf_paged_decode(kv, Q, O=outs["O"], lse=outs["lse"], score=score, score_out=outs["after"], o_f32=True, workspace=ws)
        mf.mf_kv_evict(kv, outs["after"], pos, 64, 2, 8, n_seen=seen, score_out=outs["so"], pos_out=outs["po"],
                       seq_lens_out=outs["lo"], workspace=ws)
    return inputs, outs, step


def test_calls_wait_for_what_they_read():
    """Inputs written by a kernel just before the call, outputs read and overwritten just after it,
    and two inputs' values in turn: every result equals that of a run with a wait around each call."""
    mf = _mf()
    inputs, outs, step = _order_case(mf)
    first = [t.clone() for t in inputs]
    second = [t.clone() for t in first]
    for i in (4, 5, 6, 7, 12, 13):  # Q, new rows, scores, map values, W
        second[i] = (first[i].float() * 0.5 + 0.1).to(first[i].dtype)
    want = []
    for src in (first, second):
        for t, v in zip(inputs, src):
            t.copy_(v)
        torch.cuda.synchronize()
        for o in outs.values():
            o.zero_()
        torch.cuda.synchronize()
        step()
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs.values()] + [inputs[0].clone(), inputs[1].clone()])
    torch.cuda.synchronize()
    assert any(not torch.equal(a, b) for a, b in zip(*want))
    got = []
    for n in range(40):
        for t, v in zip(inputs, (first, second)[n % 2]):
            t.copy_(v)
        for o in outs.values():
            o.zero_()
        step()
        got.append([o.clone() for o in outs.values()] + [inputs[0].clone(), inputs[1].clone()])
    torch.cuda.synchronize()
    _clean(mf)
    for n, r in enumerate(got):
        for a, b in zip(r, want[n % 2]):
            assert torch.equal(a, b), n


def test_captured_calls_after_a_joined_stream():
    """A captured step whose first calls depend on two streams, replayed with new inputs."""
    mf = _mf()
    inputs, outs, step = _order_case(mf)
    first = [t.clone() for t in inputs]
    for o in outs.values():
        o.zero_()
    torch.cuda.synchronize()
    step()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs.values()] + [inputs[0].clone()]
    side, main = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        with torch.cuda.stream(side):  # half of the inputs are restored beside the others
            for t, v in list(zip(inputs, first))[::2]:
                t.copy_(v)
        for t, v in list(zip(inputs, first))[1::2]:
            t.copy_(v)
        for o in outs.values():
            o.zero_()
        main.wait_stream(side)
        step()
    for _ in range(5):
        for t in inputs[4:8]:
            t.zero_()
        graph.replay()
        got = [o.clone() for o in outs.values()] + [inputs[0].clone()]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    _clean(mf)


def test_calls_wait_for_every_layer_of_a_retrieval():
    """A retrieval of several layers launches them without a wait in between; the append and the
    eviction right behind it write the first layer's pages, and come after all of it."""
    mf = _mf()
    L, B, h_s, h_kv, h_r, d, page, n_layers = 4096, 64, 32, 8, 32, 128, 16, 5
    values, row_ptr, cols, base = ref.make_bsr((L,), B, h_s, BF, seed=3, share=0.05)
    bsr = mf.BSR(row_ptr.cuda(), cols.cuda(), values.cuda(), row_ptr[-1:].cuda())
    g = torch.Generator(device="cuda").manual_seed(1)
    n_pages = L // page
    V0 = torch.randn(n_layers, n_pages, page, h_kv, d, generator=g, device="cuda").to(BF)
    V, K = V0.clone(), torch.zeros_like(V0[0])
    W = torch.rand(n_layers, h_r, h_s, generator=g, device="cuda") / h_s
    table = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)[None]
    cu = torch.tensor([0, L], dtype=torch.int32, device="cuda")
    qb = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = mf.PagedKV(K, V[0], table, torch.tensor([L], dtype=torch.int32, device="cuda"), L)
    zeros = torch.zeros(L, h_kv, d, dtype=BF, device="cuda")
    score = torch.rand(1, h_kv, L, generator=g, device="cuda")
    pos = torch.arange(L, dtype=torch.int32, device="cuda").expand(1, h_kv, L).contiguous()
    so, po, lo = torch.empty_like(score), torch.empty_like(pos), torch.empty_like(kv.seq_lens)
    O = torch.empty(n_layers, L, h_r, d, dtype=BF, device="cuda")

    def retrieve():
        mf.mf_map_retrieve([bsr], [0] * n_layers, W, V, cu, cu, qb, L, h_r, h_kv, O=O, paged=(table, page),
                           v_layer_stride=V[0].numel())

    retrieve()
    torch.cuda.synchronize()
    want = O.clone()
    got = []
    for n in range(12):
        V.copy_(V0)
        O.zero_()
        retrieve()
        if n % 2:
            mf.mf_kv_append(kv, zeros, zeros, cu, L)
        else:
            mf.mf_kv_evict(kv, score, pos, L // 2, score_out=so, pos_out=po, seq_lens_out=lo)
        got.append(O.clone())
    torch.cuda.synchronize()
    _clean(mf)
    for n, o in enumerate(got):
        assert torch.equal(o, want), n


def test_two_caches_at_once():
    """All four calls on two caches, each on a stream of its own with its own workspace, enqueued in
    turn, from two host threads too: the results are those of one after the other."""
    import threading
    mf = _mf()
    cases = [_order_case(mf) for _ in range(2)]
    cases[1][0][4].mul_(0.5)  # other queries
    first = [[t.clone() for t in inputs] for inputs, _, _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]

    def reset():
        torch.cuda.synchronize()
        for (inputs, outs, _), src in zip(cases, first):
            for t, v in zip(inputs, src):
                t.copy_(v)
            for o in outs.values():
                o.zero_()
        torch.cuda.synchronize()

    def steps(k, n=3):
        with torch.cuda.stream(streams[k]):
            for _ in range(n):
                cases[k][2]()

    def results():
        torch.cuda.synchronize()
        return [[o.clone() for o in outs.values()] + [inputs[0].clone(), inputs[1].clone()] for inputs, outs, _ in cases]

    reset()
    for k in range(2):
        steps(k)
        torch.cuda.synchronize()
    want = results()
    assert not torch.equal(want[0][0], want[1][0])
    for way in ("in turn", "threads"):
        reset()
        if way == "in turn":
            for _ in range(3):
                for k in range(2):
                    steps(k, 1)
        else:
            threads = [threading.Thread(target=steps, args=(k,)) for k in range(2)]
            for t in threads:
                t.start()
            for t in threads:
                t.join()
        for a, b in zip(results(), want):
            for x, y in zip(a, b):
                assert torch.equal(x, y), way
    _clean(mf)
