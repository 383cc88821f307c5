"""The receiver's paged cache at the edges of what its calls allow: rows that overlap, bounds far
above the lengths, calls of different sizes from several threads, and non-finite keys in sequences
that are split over the GPU.  Inputs and float64 loops are paged_ref's."""
import math

import pytest
import torch

import paged_ref as ref
from test_gpu_paged import BF, F32, _clean, _kv, _mf, check_decode

pytestmark = pytest.mark.gpu


def test_expanded_rows_are_refused():
    """Rows of an expanded tensor lie 0 elements apart, which the C calls take for dense rows: a
    call that went on would read past the one row there is."""
    mf = _mf()
    c, _ = ref.make_cache((40, 20, 9), 2, 64, 16, BF, seed=2)
    kv = _kv(mf, c)
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    q, new = torch.zeros(1, 8, 64, dtype=BF, device="cuda"), torch.zeros(1, 2, 64, dtype=BF, device="cuda")
    Q, three = q.expand(3, -1, -1), new.expand(3, -1, -1)
    score, pos = torch.zeros(3, 2, 40, device="cuda"), torch.zeros(3, 2, 40, dtype=torch.int32, device="cuda")
    page = kv.K[:1].expand(kv.K.shape[0], -1, -1, -1)
    flat = mf.PagedKV(page, page, kv.block_table, kv.seq_lens, 40)
    before = kv.K.clone(), kv.V.clone()
    for call in (lambda: mf.mf_paged_decode(kv, Q),
                 lambda: mf.mf_paged_decode(kv, torch.cat([q, q]).as_strided((3, 8, 64), (8, 64, 1))),
                 lambda: mf.mf_kv_append(kv, three, three, cu, 1),
                 lambda: mf.mf_kv_append(kv, three, three.contiguous(), cu, 1),
                 lambda: mf.mf_kv_append(kv, three.contiguous(), three, cu, 1),
                 lambda: mf.mf_paged_decode(flat, Q.contiguous()),
                 lambda: mf.mf_kv_append(flat, three.contiguous(), three.contiguous(), cu, 1),
                 lambda: mf.mf_kv_evict(flat, score, pos, 5), flat.desc):
        with pytest.raises(ValueError, match="overlap"):
            call()
    _clean(mf)
    assert torch.equal(kv.K, before[0]) and torch.equal(kv.V, before[1])
    # one row has no neighbour, whatever its stride
    one = mf.PagedKV(kv.K, kv.V, kv.block_table[:1], kv.seq_lens[:1], 40)
    got = mf.mf_paged_decode(one, q.as_strided((1, 8, 64), (0, 64, 1)))
    assert torch.equal(got, mf.mf_paged_decode(one, q))
    _clean(mf)


@pytest.mark.parametrize("h_kv,d,dtype,max_new", [(64, 256, F32, 600000), (8, 128, BF, (1 << 24) + 40)])
def test_append_under_a_bound_far_above_the_new_tokens(h_kv, d, dtype, max_new):
    """max_new sizes the grid.  A CTA that starts t0 tokens in finds (n - t0) * vectors per token
    left to copy, which passes -2^31 from t0 = 524290 (64 heads of 256 float32, one token to a CTA)
    and t0 = 16777224 (8 heads of 128 bf16, 8 tokens) on: it has to stop before that product."""
    mf = _mf()
    lens, new = (9, 3, 16), (1, 0, 2)
    c, _ = ref.make_cache(lens, h_kv, d, 4, dtype, seed=3)
    kv = _kv(mf, c, max_len=max_new)
    g = torch.Generator().manual_seed(1)
    Kn, Vn = (torch.randn(3, h_kv, d, generator=g).to(dtype) for _ in range(2))
    cu = torch.tensor([0, 1, 1, 3], dtype=torch.int32, device="cuda")
    mf.mf_kv_append(kv, Kn.cuda(), Vn.cuda(), cu, max_new)
    _clean(mf)
    at = 0
    for s, (n, L) in enumerate(zip(new, lens)):
        j = torch.arange(L - n, L)
        idx = (c.table[s].long()[j // 4], j % 4)
        c.K[idx], c.V[idx] = Kn[at:at + n], Vn[at:at + n]
        at += n
    assert torch.equal(kv.K.cpu(), c.K) and torch.equal(kv.V.cpu(), c.V)


def test_key_scores_of_two_sizes_from_two_threads():
    """Calls that share a kernel but not its shared memory, 50 KB apart, enqueued by two host threads:
    neither may lower the limit that the other one's launch needs."""
    import threading
    mf = _mf()
    B, L = 64, 300
    cases = []
    for h_s, h_kv, h_r in ((256, 64, 64), (3, 1, 2)):
        values, row_ptr, cols, base = ref.make_bsr((L,), B, h_s, BF, seed=h_s)
        g = torch.Generator().manual_seed(h_s)
        bsr = mf.BSR(row_ptr.cuda(), cols.cuda(), values.cuda(), row_ptr[-1:].cuda())
        W = torch.randn(h_r, h_s, generator=g)
        want, mag = ref.key_scores(values, row_ptr, cols, W, (L,), base, B, h_kv)
        tol = (B + h_s + h_r // h_kv + 8) * 2.0 ** -23 * mag + 1e-30
        need = mf.mf_map_key_scores_workspace_size(bsr.capacity, B, h_kv)
        cases.append((bsr, W.cuda(), h_kv, torch.zeros(1, h_kv, L, device="cuda"), want, tol,
                      torch.empty(need, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()))
    cu = torch.tensor([0, L], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    errors = []

    def calls(case):
        bsr, W, h_kv, score, _, _, ws, stream = case
        for _ in range(2000):
            try:
                mf.mf_map_key_scores(bsr, W, cu, zero, L, h_kv, score=score, workspace=ws, stream=stream)
            except mf.MFError as e:
                errors.append(str(e))

    threads = [threading.Thread(target=calls, args=(c,)) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    _clean(mf)
    assert not errors, (len(errors), errors[0])
    for _, _, _, score, want, tol, _, _ in cases:
        assert ((score.cpu().double() - want).abs() <= tol).all()


def test_float32_retrieval_of_two_sizes_from_two_threads():
    """mf_map_retrieve's float32 kernel takes B^2 + B d + h_s floats of shared memory: as above."""
    import ctypes
    import threading
    mf = _mf()
    L = 200
    cases = []
    for B, d in ((128, 128), (32, 8)):
        values, row_ptr, cols, base = ref.make_bsr((L,), B, 3, F32, seed=B)
        bsr = mf.BSR(row_ptr.cuda(), cols.cuda(), values.cuda(), row_ptr[-1:].cuda())
        g = torch.Generator().manual_seed(B)
        W, V = torch.randn(1, 2, 3, generator=g), torch.randn(1, L, 1, d, generator=g)
        want, mag = torch.zeros(2, 2, L, d, dtype=torch.float64)
        for qb in range(-(-L // B)):
            rows = min(B, L - qb * B)
            for n in range(int(row_ptr[qb]), int(row_ptr[qb + 1])):
                kb = int(cols[n])
                A, v = values[n].double()[:, :rows], V[0, kb * B:(kb + 1) * B, 0].double()
                to = slice(qb * B, qb * B + rows)
                want[:, to] += torch.einsum("rs,sij,jd->rid", W[0].double(), A[:, :, :len(v)], v)
                mag[:, to] += torch.einsum("rs,sij,jd->rid", W[0].double().abs(), A[:, :, :len(v)], v.abs())
        # sums of 3 heads and of L keys, each product and sum rounded once
        tol = (L + 8) * 2.0 ** -23 * mag + 1e-30
        cases.append((bsr, W.cuda(), V.cuda(), torch.zeros(1, L, 2, d, device="cuda"), want, tol, torch.cuda.Stream()))
    cu = torch.tensor([0, L], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    errors = []

    def calls(case):
        # through the C call, descriptors at hand: what a call does in Python would keep them apart
        bsr, W, V, O, _, _, stream = case
        d, keep = mf._retrieve_desc([bsr], [0], (0, 1), W, V, O, cu, cu, zero, L, 3, bsr.values.shape[2], 2, 1, 0, 0, None, 0)
        for _ in range(20000):
            if mf._lib.mf_map_retrieve(ctypes.byref(d), stream.cuda_stream) != mf.MF_OK:
                errors.append(mf._lib.mf_last_error().decode())

    threads = [threading.Thread(target=calls, args=(c,)) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    _clean(mf)
    assert not errors, (len(errors), errors[0])
    for _, _, _, O, want, tol, _ in cases:
        assert ((O[0].cpu().double().transpose(0, 1) - want).abs() <= tol).all()


@pytest.mark.parametrize("group", [4, 9])
def test_weights_enter_the_product_in_float32(group):
    """O[j] = w_j for values that are unit vectors: the weights as P.V takes them.  Scores are exact
    (one product of small numbers) and 0, the largest, in every tile of 16 keys, so that nothing is
    rescaled.  Off are: x in the base-2 domain (its factor and product rounded once each, 2^-23 |x|)
    and the base-2 exponential (2^-22), in w_j and in the sum of the weights, and one rounding for
    each of the sums' steps, 2^-24: two tiles of two keys, three exchanges and four warps in l; three
    terms, the four warps and 1 / l in O, those of the tensor cores taken twice.  A weight of 16 bits
    would be off by up to 2^-18."""
    mf = _mf()
    n, h_kv, d = 128, 4, 128
    g = torch.Generator().manual_seed(group)
    K, V = (torch.zeros(1, n, h_kv, d) for _ in range(2))
    K[0, :, :, 0] = -torch.randint(0, 129, (n, h_kv), generator=g) / 64.0  # x in [-2, 0]
    K[0, ::16, :, 0] = 0.0
    V[0] = torch.eye(n)[:, None, :]
    q = torch.zeros(1, h_kv * group, d)
    q[..., 0] = 1.0
    for max_len in (n, 5000):  # one CTA to a unit, and split
        kv = mf.PagedKV(K.to(BF).cuda(), V.to(BF).cuda(), torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                        torch.tensor([n], dtype=torch.int32, device="cuda"), min(max_len, n))
        kv.block_table = torch.zeros(1, -(-max_len // n), dtype=torch.int32, device="cuda")
        kv.max_len = max_len
        O = mf.mf_paged_decode(kv, q.to(BF).cuda(), scale=1.0, o_f32=True)
        _clean(mf)
        want = torch.softmax(K[0, :, :, 0].double(), 0).T.repeat_interleave(group, 0)[None]
        rel = 2 * (2 * 2.0 ** -23 + 2.0 ** -22) + (2 * 2 + 3 + 4 + 2 * 3 + 4 + 2) * 2.0 ** -24
        assert rel < 2.0 ** -18
        assert ((O.double().cpu() - want).abs() <= rel * want).all(), ((O.double().cpu() - want).abs() / want).max()


@pytest.mark.parametrize("group", [4, 9])
def test_long_sums_are_rounded_to_nearest(group):
    """Equal weights (Q = 0: scores 0, weights 1, their sum exact) over 8192 positive values of 12
    powers of two, so that the sums have bits to lose.  With every addition over the tiles rounded
    to nearest, a result is off by the sum of up to 128 errors, each within 2^-24 of a partial sum
    and as often up as down: relative to the result their standard deviation is at most
    2^-24 sqrt(128 / 3) = 6.6 * 2^-24, that of the mean over 1024 columns 2^-24 / 4.8, and six of
    those are 1.3 * 2^-24.  Only the products of single tiles, cut off once per term at 2^-23 of the
    tile's sum, go one way, 3 * 2^-23; the joins' few roundings are 2^-23.  Sums over the tiles that
    are cut off towards zero are off by some 40 * 2^-24 on average."""
    mf = _mf()
    n, L, h_kv, d, page = 64, 8192, 8, 128, 16
    g = torch.Generator().manual_seed(group)
    V = torch.randn(L // page, page, h_kv, d, generator=g).abs()
    V = (V * 2.0 ** -torch.randint(0, 12, V.shape, generator=g)).to(BF).cuda()
    K = torch.randn(L // page, page, h_kv, d, generator=g).to(BF).cuda()
    # 64 sequences of the same pages: every CTA walks through whole units
    table = torch.arange(L // page, dtype=torch.int32, device="cuda").expand(n, -1).contiguous()
    kv = mf.PagedKV(K, V, table, torch.full((n,), L, dtype=torch.int32, device="cuda"), L)
    O = mf.mf_paged_decode(kv, torch.zeros(n, h_kv * group, d, dtype=BF, device="cuda"), o_f32=True)
    _clean(mf)
    want = V.double().flatten(0, 1).mean(0).repeat_interleave(group, 0)[None]
    off = (O.double() - want) / want
    assert off.abs().max() <= 128 * 2.0 ** -24
    assert off.view(n, -1).mean(1).abs().max() <= 1.3 * 2.0 ** -24 + 4 * 2.0 ** -23, off.mean()


def test_scales_that_are_no_float32_are_refused():
    """A scale that rounds to 0 as a float32 must not be taken for the default, 1 / sqrt(d)."""
    mf = _mf()
    c, _ = ref.make_cache((40, 20), 2, 64, 16, BF, seed=2)
    kv = _kv(mf, c)
    Q = torch.randn(2, 8, 64, generator=torch.Generator().manual_seed(1)).to(BF)
    for scale in (1e-60, -1e-60, 5e-324):
        with pytest.raises(ValueError, match="too small"):
            mf.mf_paged_decode(kv, Q.cuda(), scale=scale)
    for scale in (1e39, 3e38, -1.0, float("nan")):
        with pytest.raises(mf.MFError, match="scale"):
            mf.mf_paged_decode(kv, Q.cuda(), scale=scale)
    # the smallest float32: equal weights
    O = mf.mf_paged_decode(kv, Q.cuda(), scale=1e-45, o_f32=True)
    _clean(mf)
    for s, L in enumerate(c.lens):
        want = torch.stack([c.rows(c.V, s, g, range(L)).double().mean(0) for g in range(2)])
        assert ((O[s].cpu().double() - want.repeat_interleave(4, 0)).abs() <= 2.0 ** -20).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("group", [1, 3, 9])
@pytest.mark.parametrize("max_len", [3000, 6000])
def test_non_finite_keys_of_split_sequences(dtype, group, max_len):
    """Sequences long enough to be cut between CTAs, so that empty and NaN parts are joined and the
    second kernel adds the weights.  Head 0 of sequence 0: every score -inf; of 1: one NaN; of 2:
    one +inf; of 3: -inf up to slot 2000; of 4: only slot 1700 above -inf; sequence 5 is empty.
    Every other row, and those of 3 and 4, are those of the keys above -inf alone."""
    mf = _mf()
    lens, d, page = (3000, 3000, 3000, 3000, 3000, 0), 64, 16
    c, _ = ref.make_cache(lens, 2, d, page, F32, seed=group)
    c.K, c.V = c.K.to(BF).float(), c.V.to(BF).float()  # the same numbers in both types
    g = torch.Generator().manual_seed(group)
    h_r = 2 * group
    Q = (torch.rand(6, h_r, d, generator=g) + 0.5).to(BF).float()  # positive: -inf stays -inf

    def put(s, slots, value):
        slots = torch.as_tensor(slots)
        c.K[c.table[s].long()[slots // page], slots % page, 0, 3] = value

    put(0, range(3000), -math.inf)
    put(1, [2222], math.nan)
    put(2, [2999], math.inf)
    put(3, range(2000), -math.inf)
    put(4, [j for j in range(3000) if j != 1700], -math.inf)
    kv = mf.PagedKV(c.K.to(dtype).cuda(), c.V.to(dtype).cuda(), c.table.cuda(),
                    torch.tensor(lens, dtype=torch.int32, device="cuda"), max_len)
    lse = torch.empty(6, h_r, device="cuda")
    before = torch.rand(6, 2, max_len, generator=g).cuda()
    after = torch.full_like(before, 5.0)
    O = mf.mf_paged_decode(kv, Q.to(dtype).cuda(), lse=lse, score=before, score_out=after, o_f32=True)
    _clean(mf)
    O, lse, before, after = (t.cpu().double() for t in (O, lse, before, after))
    for s, L in enumerate(lens):
        for h in range(2):
            heads = slice(h * group, (h + 1) * group)
            if L == 0 or (s, h) == (0, 0):
                assert (O[s, heads] == 0).all() and (lse[s, heads] == -math.inf).all()
                assert torch.equal(after[s, h, :L], before[s, h, :L])
            elif (s, h) in ((1, 0), (2, 0)):
                assert O[s, heads].isnan().all() and lse[s, heads].isnan().all() and after[s, h, :L].isnan().all()
            else:
                K, V = (c.rows(t, s, h, range(L)).double() for t in (c.K, c.V))
                some = K[:, 3] > -math.inf
                K, V, q = K[some], V[some], Q[s, heads].double()
                x = q @ K.T * d ** -0.5
                want = torch.logsumexp(x, 1, keepdim=True)
                w = torch.exp(x - want)
                # as test_gpu_paged states it
                dx = (d + 8) * 2.0 ** -23 * d ** -0.5 * (q @ K.abs().T).max()
                rel = 2 * dx + x.abs().max() * 2.0 ** -22 + 2.0 ** -21 + (L / 16 + 64) * 2.0 ** -24
                assert ((O[s, heads] - w @ V).abs() <= rel * (w @ V.abs())).all()
                assert ((lse[s, heads] - want[:, 0]).abs() <= rel + want[:, 0].abs() * 2.0 ** -22).all()
                gained = torch.zeros(L, dtype=torch.float64)
                gained[some] = w.sum(0)
                new = before[s, h, :L] + gained
                assert ((after[s, h, :L] - new).abs() <= rel * gained + 2.0 ** -23 * new).all()
                assert torch.equal(after[s, h, :L][~some], before[s, h, :L][~some])
            assert (after[s, h, L:] == 5.0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,h_kv,group,d,page", [
    ((1,), 1, 1, 64, 16), ((0, 1, 15, 16, 17, 33), 2, 4, 128, 16), ((100,), 8, 4, 128, 16),
    ((300, 0, 1), 8, 3, 128, 64), ((90, 40), 1, 16, 256, 20), ((60, 31), 1, 40, 96, 32),
])
def test_short_sequences_under_a_bound_far_above_them(lens, h_kv, group, d, page, dtype):
    """A captured loop passes its capacity as max_len: short sequences then take the split path."""
    mf = _mf()
    c, _ = ref.make_cache(lens, h_kv, d, page, dtype, seed=d, stale=float("nan"))
    Q = torch.randn(len(lens), h_kv * group, d, generator=torch.Generator().manual_seed(1)).to(dtype)
    kv = _kv(mf, c, max_len=max(lens) + 4000)
    kv.block_table = torch.cat([kv.block_table, torch.full((len(lens), 4000 // page + 1), -1, dtype=torch.int32, device="cuda")], 1)
    lse = torch.empty(len(lens), h_kv * group, device="cuda")
    before = torch.rand(len(lens), h_kv, kv.max_len, device="cuda")
    after = before.clone()
    O = mf.mf_paged_decode(kv, Q.cuda(), lse=lse, score=after)
    _clean(mf)
    check_decode(c, Q, O, lse, (before[..., :max(lens) + 1], after[..., :max(lens) + 1]))
    assert torch.equal(after[..., max(lens):], before[..., max(lens):])


@pytest.mark.parametrize("own", ["score_out", "pos_out", "seq_lens_out"])
@pytest.mark.parametrize("lens,budget,h_kv", [((300, 10, 65), 64, 3), ((20000, 16385), 12000, 3), ((140000,), 9000, 1)])
def test_evict_with_one_output_of_its_own(lens, budget, h_kv, own):
    """Any of the outputs may be apart from its input while the others are updated in place, and
    n_seen may be seq_lens itself; rows of one CTA, of a cluster, and of several tiles."""
    mf = _mf()
    c, _ = ref.make_cache(lens, h_kv, 64, 16, BF, seed=budget)
    kv = _kv(mf, c)
    g = torch.Generator().manual_seed(budget)
    W = max(lens) + 3
    score = torch.rand(len(lens), h_kv, W, generator=g)
    pos = torch.rand(len(lens), h_kv, W, generator=g).argsort(-1).to(torch.int32)
    sd, pd = score.cuda(), pos.cuda()
    outs = {"score_out": torch.full_like(sd, 9.0), "pos_out": torch.full_like(pd, 9),
            "seq_lens_out": torch.full_like(kv.seq_lens, 9)}
    got = mf.mf_kv_evict(kv, sd, pd, budget, 4, 16, n_seen=kv.seq_lens, **{own: outs[own]})
    _clean(mf)
    wscore, wpos, wlens = ref.evict(c, score, pos, list(lens), budget, 4, 16)
    assert got.tolist() == wlens
    assert torch.equal(kv.K.cpu(), c.K) and torch.equal(kv.V.cpu(), c.V)
    so = outs["score_out"] if own == "score_out" else sd
    po = outs["pos_out"] if own == "pos_out" else pd
    for s, L in enumerate(lens):
        assert torch.equal(so[s, :, :L].cpu(), wscore[s, :, :L]) and torch.equal(po[s, :, :L].cpu(), wpos[s, :, :L])
        assert (so[s, :, L:].cpu() == (9.0 if own == "score_out" else score[s, :, L:])).all()
        assert (po[s, :, L:].cpu() == (9 if own == "pos_out" else pos[s, :, L:])).all()
    assert torch.equal(sd.cpu(), score) or own != "score_out"
    assert torch.equal(pd.cpu(), pos) or own != "pos_out"
    assert kv.seq_lens.tolist() == list(lens) or own != "seq_lens_out"
