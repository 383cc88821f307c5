"""The paged-cache operators of a receiver model, as cases that can be timed and compared.

A receiver that took its prefill attention from a sender's maps goes on with its own paged
key-value cache.  Four operators carry it from there:

    append   new tokens' keys and values (slices of a fused projection) into the cache's pages
    scores   the attention weight every key gathered during the prefill, from the kept blocks of
             the sender's maps and the receiver's head map
    decode   attention of one new token per sequence over the pages, with the row's
             log-sum-exp and the gathered weights carried on
    evict    the cache cut back to a budget of slots per sequence and head: first tokens and the
             recent window stay, the rest go by gathered weight

`run` computes each in plain torch operations (`own` false) or through the package (`own` true).
Every pass leaves its inputs as they were (updated scores, positions and lengths go to buffers of
their own; evicting or appending twice writes the same rows again), so passes can be repeated.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one user, a short chat turn: the smallest call, where the launch counts
        _decode("decode_short", nseq=1, max_len=100, low=100, h_kv=8, group=4, d=128, page=16),
        # the routing batch: 16 conversations of 1024 to 8192 tokens on 16-token pages
        _decode("decode_routing", nseq=16, max_len=8192, low=1024, h_kv=8, group=4, d=128, page=16),
        # one long document, the long-context receiver's 24 query heads, weights gathered
        _decode("decode_long", nseq=1, max_len=131072, low=131072, h_kv=8, group=3, d=128, page=64,
                scores=True),
        # a full serving batch, weights gathered for a later eviction: the largest call
        _decode("decode_batch", nseq=64, max_len=8192, low=8192, h_kv=8, group=4, d=128, page=16,
                scores=True),
        # a float32 cache of odd sizes: empty and one-token sequences, pages that end inside a tile
        _decode("decode_f32_odd", nseq=7, max_len=1001, low=0, h_kv=3, group=5, d=80, page=12,
                dtype="f32", scores=True),
        # every sequence of a serving batch adds its new token
        _append("append_step", nseq=64, max_len=4096, low=64, max_new=1, h_kv=8, group=4, d=128, page=16),
        # a prefill pack's keys and values go into the pages at once
        _append("append_prefill", nseq=4, max_len=6144, low=2048, max_new=6144, h_kv=8, group=4, d=128,
                page=16),
        # one sequence whose maps keep 3% of the causal blocks, as the 8192-token workload does
        _scores("scores_sparse", nseq=1, max_len=8192, low=8192, B=64, h_s=32, h_kv=8, group=4, percent=3),
        # a ragged pack of denser maps with 40 sender heads
        _scores("scores_pack", nseq=4, max_len=6144, low=2048, B=64, h_s=40, h_kv=8, group=4, percent=30),
        # each decode step evicts one token from every full cache of a batch
        _evict("evict_step", nseq=64, max_len=2049, low=2049, budget=2048, sink=4, window=256, h_kv=8,
               d=128, page=16, aged=True),
        # a batch of prefilled prompts cut back once before decoding
        _evict("evict_prefill", nseq=16, max_len=8192, low=1024, budget=2048, sink=4, window=64, h_kv=8,
               d=128, page=16),
        # one long document cut back to an eighth
        _evict("evict_long", nseq=1, max_len=131072, low=131072, budget=16384, sink=4, window=1024, h_kv=8,
               d=128, page=64),
    ]


def draw(rng):
    kind = rng.choice(["decode", "decode", "append", "scores", "evict", "evict"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    e = 2 if dtype == "bf16" else 4
    h_kv, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8, 16])
    d = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
    page = rng.choice([8, 12, 16, 16, 32, 64])
    nseq = _log_int(rng, 1, 64)
    if kind == "scores":
        B, h_s, percent = rng.choice([32, 64, 64, 128]), rng.choice([4, 7, 16, 32, 40]), rng.randint(2, 40)
        nseq = rng.randint(1, 4)
        top = 8192 if B > 32 else 4096
        max_len = _log_int(rng, 64, top // nseq if dtype == "f32" else top)
        case = _scores("", nseq=nseq, max_len=max_len, low=_low(rng, max_len, 1), B=B, h_s=h_s, h_kv=h_kv,
                       group=group, percent=percent, dtype=dtype)
    else:
        # at most as many cache bytes as the largest listed call
        room = 64 * 8192 * 8 * 128 * 2 // (nseq * h_kv * d * e)
        if kind == "append":
            max_new = _log_int(rng, 1, min(8192, room // 8))
            max_len = max_new + _log_int(rng, 1, min(8192, room // 8))
            case = _append("", nseq=nseq, max_len=max_len, low=_low(rng, max_len, 0), max_new=max_new,
                           h_kv=h_kv, group=group, d=d, page=page, dtype=dtype)
        elif kind == "decode":
            max_len = _log_int(rng, 1, min(131072, room))
            case = _decode("", nseq=nseq, max_len=max_len, low=_low(rng, max_len, 0), h_kv=h_kv, group=group,
                           d=d, page=page, dtype=dtype, scores=rng.random() < 0.5)
        else:
            max_len = _log_int(rng, 16, min(131072, room // 4))
            budget = rng.randint(max(1, max_len // 8), max_len)
            sink = rng.choice([0, 0, 4])
            window = rng.randint(0, max(0, (budget - sink) // 2)) if budget > sink else 0
            case = _evict("", nseq=nseq, max_len=max_len, low=_low(rng, max_len, 0), budget=budget,
                          sink=min(sink, budget), window=window, h_kv=h_kv, d=d, page=page, dtype=dtype,
                          aged=rng.random() < 0.5)
    del case["name"]
    return case


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def _low(rng, max_len, least):
    return rng.choice([max_len, max(least, max_len // 8), least])


def _decode(name, nseq, max_len, low, h_kv, group, d, page, dtype="bf16", scores=False):
    return dict(name=name, op="decode", nseq=nseq, max_len=max_len, low=low, h_kv=h_kv, group=group, d=d,
                page=page, dtype=dtype, scores=scores)


def _append(name, nseq, max_len, low, max_new, h_kv, group, d, page, dtype="bf16"):
    return dict(name=name, op="append", nseq=nseq, max_len=max_len, low=low, max_new=max_new, h_kv=h_kv,
                group=group, d=d, page=page, dtype=dtype)


def _scores(name, nseq, max_len, low, B, h_s, h_kv, group, percent, dtype="bf16"):
    return dict(name=name, op="scores", nseq=nseq, max_len=max_len, low=low, B=B, h_s=h_s, h_kv=h_kv,
                group=group, percent=percent, dtype=dtype)


def _evict(name, nseq, max_len, low, budget, sink, window, h_kv, d, page, dtype="bf16", aged=False):
    return dict(name=name, op="evict", nseq=nseq, max_len=max_len, low=low, budget=budget, sink=sink,
                window=window, h_kv=h_kv, d=d, page=page, dtype=dtype, aged=aged)


def lengths(case):
    """Sequence lengths of a case: spread over [low, max_len], the first at max_len."""
    lo, hi = case["low"], case["max_len"]
    return [hi if s == 0 else lo + (((s * 2654435761 + 40503) % 2 ** 32) * (hi - lo + 1) >> 32)
            for s in range(case["nseq"])]


def new_tokens(case):
    return [min(L, case["max_new"]) for L in lengths(case)]


def kept_counts(case):
    """Kept blocks of each query-block row, per sequence: the diagonal and a share of the others."""
    return [[max(1, (qb + 1) * case["percent"] // 100) for qb in range(-(-L // case["B"]))]
            for L in lengths(case)]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    h_kv, lens = case["h_kv"], lengths(case)
    T = sum(lens)
    if case["op"] == "decode":
        h_r, d = h_kv * case["group"], case["d"]
        pages = sum(-(-L // case["page"]) for L in lens)
        b = 2 * T * h_kv * d * e + case["nseq"] * h_r * (2 * d * e + 4) + 4 * pages + 4 * case["nseq"]
        if case["scores"]:
            b += 8 * T * h_kv
        return {"bytes": b, "flops": 4 * T * h_r * d}
    if case["op"] == "append":
        n = sum(new_tokens(case))
        return {"bytes": n * h_kv * (4 * case["d"] * e + 8) + 8 * case["nseq"], "flops": n * h_kv}
    if case["op"] == "scores":
        nnz = sum(sum(k) for k in kept_counts(case))
        els = nnz * case["h_s"] * case["B"] ** 2
        return {"bytes": els * e + 4 * nnz + 4 * T * h_kv + 4 * case["h_s"] * h_kv * case["group"], "flops": els}
    # evict: every score and position is read, the kept ones written; of the kept rows only those
    # whose slot lies past the budget have to move (read and written once, key and value)
    moved = 0
    for L in lens:
        if L > case["budget"]:
            recent = case["window"] // 2 if case["aged"] else case["window"]
            free, rest = case["budget"] - recent - case["sink"], L - recent - case["sink"]
            moved += min(recent, L - case["budget"]) + max(0, L - case["budget"] - recent) * free // max(1, rest)
    kept = sum(min(L, case["budget"]) for L in lens)
    return {"bytes": h_kv * (8 * T + 8 * kept + 4 * moved * case["d"] * e), "flops": T * h_kv}


# ------------------------------------------------------------------ inputs

def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _cache(case, g, lens):
    """Pages in a shuffled order with a few spare ones; unused table entries are -1."""
    ps, dt = case["page"], DTYPES[case["dtype"]]
    counts = [-(-L // ps) for L in lens]
    n_pages = sum(counts) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(counts))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(counts):
        table[s, :n] = order[at:at + n]
        at += n
    K = _randn(g, n_pages, ps, case["h_kv"], case["d"], dtype=dt)
    V = _randn(g, n_pages, ps, case["h_kv"], case["d"], dtype=dt)
    return dict(K=K, V=V, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = lengths(case)
    n, h_kv = len(lens), case["h_kv"]
    st = dict(case=case)
    if case["op"] == "scores":
        st.update(_maps(case, g, lens))
    else:
        st.update(_cache(case, g, lens))
    wide = case["max_len"] + 5  # rows of the score and position buffers are wider than any length
    if case["op"] == "decode":
        h_r, d = h_kv * case["group"], case["d"]
        # the query heads of a fused projection's output; peaked scores, as attention has
        qkv = _randn(g, n, (h_r + 2 * h_kv) * d) * 2.0
        st["Q"] = qkv.to(DTYPES[case["dtype"]])[:, :h_r * d].unflatten(1, (h_r, d))
        st["O"] = torch.zeros(n, h_r, d, dtype=DTYPES[case["dtype"]], device="cuda")
        st["lse"] = torch.zeros(n, h_r, device="cuda")
        if case["scores"]:
            st["score"] = torch.rand(n, h_kv, wide, generator=g, device="cuda")
            st["score_out"] = torch.zeros_like(st["score"])
    elif case["op"] == "append":
        new = new_tokens(case)
        h_r, d = h_kv * case["group"], case["d"]
        qkv = _randn(g, max(1, sum(new)), (h_r + 2 * h_kv) * d, dtype=DTYPES[case["dtype"]])
        st["K_new"] = qkv[:, h_r * d:(h_r + h_kv) * d].unflatten(1, (h_kv, d))
        st["V_new"] = qkv[:, (h_r + h_kv) * d:].unflatten(1, (h_kv, d))
        cu = torch.tensor([0] + new).cumsum(0)
        st["cu_new"] = cu.to(device="cuda", dtype=torch.int32)
        # tokens seen so far: more than the cache holds where an eviction came before
        st["seen"] = st["lens"] + torch.randint(0, 1000, (n,), generator=g, device="cuda", dtype=torch.int32)
        st["score"] = torch.rand(n, h_kv, wide, generator=g, device="cuda")
        st["pos"] = torch.zeros(n, h_kv, wide, dtype=torch.int32, device="cuda")
    elif case["op"] == "evict":
        # gathered weights: a few large ones, many small ones, some exactly 0 (never attended)
        st["score"] = torch.exp(3.0 * _randn(g, n, h_kv, wide))
        st["score"] *= torch.rand(n, h_kv, wide, generator=g, device="cuda") > 0.05
        slot = torch.arange(wide, dtype=torch.int32, device="cuda")
        if case["aged"]:
            # earlier evictions left gaps and a mixed order; the newest token sits in the last slot
            last = (st["lens"] - 1)[:, None, None]
            key = torch.rand(n, h_kv, wide, generator=g, device="cuda")
            key = torch.where(slot == last, 2.0, torch.where(slot > last, 3.0, key))
            st["pos"] = (2 * key.argsort(-1).argsort(-1)).to(torch.int32)
            st["seen"] = (2 * st["lens"] - 1).clamp(min=0)
        else:
            st["pos"] = slot.expand(n, h_kv, wide).contiguous()
            st["seen"] = st["lens"].clone()
        st["score_out"] = torch.zeros_like(st["score"])
        st["pos_out"] = torch.zeros_like(st["pos"])
        st["lens_out"] = torch.zeros_like(st["lens"])
    if own:
        _prepare_own(st, lens)
    return st


def _maps(case, g, lens):
    """Kept blocks of causal maps: the diagonal and random earlier blocks of every query-block row,
    values as a peaked softmax over the kept keys leaves them."""
    B, h_s, dt = case["B"], case["h_s"], DTYPES[case["dtype"]]
    cols, row_ptr = [], [0]
    qb_of, len_of, base = [], [], [0]
    for L, counts in zip(lens, kept_counts(case)):
        nqb = len(counts)
        r = torch.rand(nqb, nqb, generator=g, device="cuda")
        at = torch.arange(nqb, device="cuda")
        r[at[None, :] > at[:, None]] = -1.0
        r[at, at] = 2.0
        rank = r.argsort(1, descending=True).argsort(1)
        keep = rank < torch.tensor(counts, device="cuda")[:, None]
        qb, kb = keep.nonzero(as_tuple=True)
        cols.append(kb)
        qb_of.append(qb)
        len_of.append(torch.full_like(qb, L))
        for c in counts:
            row_ptr.append(row_ptr[-1] + c)
        base.append(base[-1] + nqb)
    cols, qb_of, len_of = torch.cat(cols), torch.cat(qb_of), torch.cat(len_of)
    nnz = cols.numel()
    values = torch.empty(nnz, h_s, B, B, dtype=dt, device="cuda")
    lane = torch.arange(B, device="cuda")
    per_row = torch.tensor([c for k in kept_counts(case) for c in k], device="cuda")
    count = torch.repeat_interleave(per_row, per_row)
    step = max(1, (1 << 27) // (h_s * B * B))
    for a in range(0, nnz, step):
        b = min(nnz, a + step)
        i = qb_of[a:b, None] * B + lane
        j = cols[a:b, None] * B + lane
        live = (j[:, None, :] <= i[:, :, None]) & (i[:, :, None] < len_of[a:b, None, None])
        v = torch.exp(1.5 * _randn(g, b - a, h_s, B, B)) / (3.08 * B * count[a:b, None, None, None])
        values[a:b] = (v * live[:, None]).to(dt)
    h_r = case["h_kv"] * case["group"]
    return dict(values=values, cols=cols.to(torch.int32), qb_of=qb_of,
                row_ptr=torch.tensor(row_ptr, dtype=torch.int32, device="cuda"),
                base=torch.tensor(base[:-1], dtype=torch.int32, device="cuda"),
                seq_of=torch.repeat_interleave(torch.arange(len(lens), device="cuda"),
                                               torch.tensor([sum(k) for k in kept_counts(case)], device="cuda")),
                cu=torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32),
                W=_randn(g, h_r, h_s) / math.sqrt(h_s),
                score=torch.zeros(len(lens), case["h_kv"], case["max_len"] + 5, device="cuda"))


def _prepare_own(st, lens):
    import cross_model_attention_mf_b200 as mf

    case = st["case"]
    if case["op"] == "scores":
        st["bsr"] = mf.BSR(st["row_ptr"], st["cols"], st["values"], st["row_ptr"][-1:])
        need = mf.mf_map_key_scores_workspace_size(st["bsr"].capacity, case["B"], case["h_kv"])
    else:
        st["kv"] = mf.PagedKV(st["K"], st["V"], st["table"], st["lens"], max_len=case["max_len"])
        if case["op"] == "decode":
            need = mf.mf_paged_decode_workspace_size(st["kv"], case["h_kv"] * case["group"],
                                                     scores=case["scores"])
        elif case["op"] == "evict":
            need = mf.mf_kv_evict_workspace_size(st["kv"], case["budget"])
        else:
            need = 0
    st["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    return {"decode": _own_decode, "append": _own_append, "scores": _own_scores, "evict": _own_evict}[op](state) \
        if own else {"decode": _decode_plain, "append": _append_plain, "scores": _scores_plain,
                     "evict": _evict_plain}[op](state)


def _own_decode(st):
    import cross_model_attention_mf_b200 as mf

    mf.mf_paged_decode(st["kv"], st["Q"], O=st["O"], lse=st["lse"], score=st.get("score"),
                       score_out=st.get("score_out"), workspace=st["workspace"])
    return {"O": st["O"], "lse": st["lse"], **({"score": st["score_out"]} if "score" in st else {})}


def _own_append(st):
    import cross_model_attention_mf_b200 as mf

    mf.mf_kv_append(st["kv"], st["K_new"], st["V_new"], st["cu_new"], st["case"]["max_new"],
                    n_seen=st["seen"], score=st["score"], pos=st["pos"])
    return {"K": st["K"], "V": st["V"], "score": st["score"], "pos": st["pos"]}


def _own_scores(st):
    import cross_model_attention_mf_b200 as mf

    case = st["case"]
    return mf.mf_map_key_scores(st["bsr"], st["W"], st["cu"], st["base"], case["max_len"], case["h_kv"],
                                score=st["score"], workspace=st["workspace"])


def _own_evict(st):
    import cross_model_attention_mf_b200 as mf

    case = st["case"]
    mf.mf_kv_evict(st["kv"], st["score"], st["pos"], case["budget"], sink=case["sink"], window=case["window"],
                   n_seen=st["seen"], score_out=st["score_out"], pos_out=st["pos_out"],
                   seq_lens_out=st["lens_out"], workspace=st["workspace"])
    return {"K": st["K"], "V": st["V"], "score": st["score_out"], "pos": st["pos_out"], "lens": st["lens_out"]}


def _slots(st):
    """Flat row (page * page_size + offset) of every slot of the table, and which slots are held."""
    ps = st["case"]["page"]
    slot = torch.arange(st["table"].shape[1] * ps, device="cuda")
    page = st["table"].long().clamp(min=0)[:, slot // ps]
    return page * ps + slot % ps, slot < st["lens"][:, None]


def _decode_plain(st):
    case = st["case"]
    row, held = _slots(st)
    h_kv, group, d = case["h_kv"], case["group"], case["d"]
    K = st["K"].flatten(0, 1)[row].float().transpose(1, 2)  # [n, h_kv, slots, d]
    V = st["V"].flatten(0, 1)[row].float().transpose(1, 2)
    q = st["Q"].float().unflatten(1, (h_kv, group))
    s = (q @ K.transpose(2, 3)) / math.sqrt(d)
    s = torch.where(held[:, None, None], s, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, 0.0)
    O = p @ torch.where(held[:, None, :, None], V, 0.0)
    st["O"].copy_(O.flatten(1, 2))
    st["lse"].copy_((torch.log(total) + top).flatten(1))
    out = {"O": st["O"], "lse": st["lse"]}
    if case["scores"]:
        w, n = p.sum(2), min(p.shape[3], st["score"].shape[2])
        at = held[:, None, :n]
        st["score_out"][:, :, :n] = torch.where(at, st["score"][:, :, :n] + w[:, :, :n], st["score_out"][:, :, :n])
        out["score"] = st["score_out"]
    return out


def _append_plain(st):
    ps = st["case"]["page"]
    cu = st["cu_new"].long()
    n = cu[1:] - cu[:-1]
    T = int(cu[-1])
    token = torch.arange(T, device="cuda")
    seq = torch.searchsorted(cu[1:], token, right=True)
    back = n[seq] - (token - cu[seq])  # 1 for a sequence's last token
    slot = st["lens"].long()[seq] - back
    row = st["table"].long()[seq, slot // ps] * ps + slot % ps
    st["K"].flatten(0, 1)[row] = st["K_new"][:T]
    st["V"].flatten(0, 1)[row] = st["V_new"][:T]
    st["score"][seq, :, slot] = 0.0
    st["pos"][seq, :, slot] = (st["seen"].long()[seq] - back).to(torch.int32)[:, None]
    return {"K": st["K"], "V": st["V"], "score": st["score"], "pos": st["pos"]}


def _scores_plain(st):
    case = st["case"]
    B, h_kv = case["B"], case["h_kv"]
    Wg = st["W"].unflatten(0, (h_kv, case["group"])).sum(1)
    nnz = st["cols"].numel()
    width = -(-case["max_len"] // B) * B
    acc = torch.zeros(len(st["cu"]) - 1, width // B, h_kv, B, device="cuda")
    step = max(1, (1 << 28) // (case["h_s"] * B * B))
    for a in range(0, nnz, step):
        b = min(nnz, a + step)
        part = torch.einsum("gs,nsj->ngj", Wg, st["values"][a:b].float().sum(2))
        acc.index_put_((st["seq_of"][a:b], st["cols"][a:b].long()), part, accumulate=True)
    total = acc.transpose(1, 2).flatten(2)[:, :, :case["max_len"]]
    lens = (st["cu"][1:] - st["cu"][:-1])[:, None, None]
    live = torch.arange(case["max_len"], device="cuda") < lens
    st["score"][:, :, :case["max_len"]] = torch.where(live, total, st["score"][:, :, :case["max_len"]])
    return st["score"]


def _evict_plain(st):
    case = st["case"]
    ps, budget = case["page"], case["budget"]
    n, h, wide = st["score"].shape
    slot = torch.arange(wide, device="cuda")
    lens = st["lens"].long()[:, None, None]
    seen = st["seen"].long()[:, None, None]
    held = slot < lens
    safe = (st["pos"] < case["sink"]) | (st["pos"] >= seen - case["window"])
    rank = torch.where(held, torch.where(safe, math.inf, st["score"]), -math.inf)
    order = rank.sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros(n, h, wide, dtype=torch.bool, device="cuda").scatter_(2, order[:, :, :budget], True) & held
    left = torch.minimum(lens, torch.full_like(lens, budget))
    holes = ~kept & (slot < left)
    movers = kept & (slot >= left)
    s, g, dst = holes.nonzero(as_tuple=True)
    src = movers.nonzero(as_tuple=True)[2]
    table = st["table"].long()
    for pages in (st["K"], st["V"]):
        pages[table[s, dst // ps], dst % ps, g] = pages[table[s, src // ps], src % ps, g]
    for name, empty in (("score", 0.0), ("pos", -1)):
        new = st[name].clone()
        new[s, g, dst] = st[name][s, g, src]
        new = torch.where(slot < left, new, torch.full_like(new, empty))
        st[name + "_out"].copy_(torch.where(held, new, st[name + "_out"]))
    st["lens_out"].copy_(left[:, 0, 0])
    return {"K": st["K"], "V": st["V"], "score": st["score_out"], "pos": st["pos_out"], "lens": st["lens_out"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"decode": _exact_decode, "append": _exact_append, "scores": _exact_scores,
            "evict": _exact_evict}[case["op"]](case, st)


def _held_rows(pages, table_row, L, g):
    """Rows 0 .. L-1 of one sequence and head, in float64."""
    n = -(-L // pages.shape[1])
    return pages[table_row[:n].long(), :, g].double().flatten(0, 1)[:L]


def _exact_decode(case, st):
    lens = lengths(case)
    n, h_r, d = st["Q"].shape
    O = torch.zeros(n, h_r, d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, h_r), -math.inf, dtype=torch.float64, device="cuda")
    score = st["score_out"].double() if case["scores"] else None
    for s, L in enumerate(lens):
        if L == 0:
            continue
        for g in range(case["h_kv"]):
            heads = slice(g * case["group"], (g + 1) * case["group"])
            K = _held_rows(st["K"], st["table"][s], L, g)
            x = st["Q"][s, heads].double() @ K.T * d ** -0.5
            lse[s, heads] = torch.logsumexp(x, 1)
            w = torch.exp(x - lse[s, heads, None])
            O[s, heads] = w @ _held_rows(st["V"], st["table"][s], L, g)
            if score is not None:
                score[s, g, :L] = st["score"][s, g, :L].double() + w.sum(0)
    return {"O": O, "lse": lse, **({"score": score} if score is not None else {})}


def _exact_append(case, st):
    lens, new = lengths(case), new_tokens(case)
    seen = st["seen"].tolist()
    ps, table = case["page"], st["table"].cpu()
    K, V, score, pos = st["K"].clone(), st["V"].clone(), st["score"].double(), st["pos"].clone()
    at = 0
    for s, (L, n) in enumerate(zip(lens, new)):
        slot = torch.arange(L - n, L)
        page, row = table[s].long()[slot // ps].cuda(), (slot % ps).cuda()
        K[page, row] = st["K_new"][at:at + n]
        V[page, row] = st["V_new"][at:at + n]
        score[s, :, L - n:L] = 0.0
        pos[s, :, L - n:L] = torch.arange(seen[s] - n, seen[s], dtype=torch.int32, device="cuda")
        at += n
    return {"K": K, "V": V, "score": score, "pos": pos}


def _exact_scores(case, st):
    out = st["score"].double()
    lens, B, group = lengths(case), case["B"], case["group"]
    row_ptr, cols = st["row_ptr"].tolist(), st["cols"].tolist()
    W = st["W"].double()
    row = 0
    for s, L in enumerate(lens):
        total = torch.zeros(case["h_kv"], -(-L // B) * B, dtype=torch.float64, device="cuda")
        for _ in range(-(-L // B)):
            a, b = row_ptr[row], row_ptr[row + 1]
            column = st["values"][a:b].double().sum(2)  # [kept, h_s, B]
            for k in range(a, b):
                mixed = (W @ column[k - a]).unflatten(0, (case["h_kv"], group)).sum(1)
                total[:, cols[k] * B:(cols[k] + 1) * B] += mixed
            row += 1
        out[s, :, :L] = total[:, :L]
    return out


def _exact_evict(case, st):
    lens, budget, ps = lengths(case), case["budget"], case["page"]
    score, pos, seen = st["score"].cpu(), st["pos"].cpu(), st["seen"].tolist()
    table = st["table"].cpu().long()
    new_score, new_pos = st["score_out"].cpu().double(), st["pos_out"].cpu()
    dst_all, src_all = [], []
    for s, L in enumerate(lens):
        for g in range(case["h_kv"]):
            sc, po = score[s, g, :L].double().numpy(), pos[s, g, :L].numpy()
            if L > budget:
                safe = (po < case["sink"]) | (po >= seen[s] - case["window"])
                ranked = sorted(range(L), key=lambda j: (not safe[j], 0.0 if safe[j] else -sc[j], j))
                kept = set(ranked[:budget])
                dst = [j for j in range(budget) if j not in kept]
                src = sorted(j for j in kept if j >= budget)
            else:
                dst, src = [], []
            left = min(L, budget)
            a, b = torch.from_numpy(sc.copy()), torch.from_numpy(po.copy())
            a[dst], b[dst] = a[src], b[src]
            a[left:], b[left:] = 0.0, -1
            new_score[s, g, :L], new_pos[s, g, :L] = a, b
            for j, i in zip(dst, src):
                dst_all.append((s, g, j))
                src_all.append((s, g, i))
    K, V = st["K"].clone(), st["V"].clone()
    if dst_all:
        d, f = torch.tensor(dst_all), torch.tensor(src_all)
        to = (table[d[:, 0], d[:, 2] // ps].cuda(), (d[:, 2] % ps).cuda(), d[:, 1].cuda())
        at = (table[f[:, 0], f[:, 2] // ps].cuda(), (f[:, 2] % ps).cuda(), f[:, 1].cuda())
        K[to], V[to] = st["K"][at], st["V"][at]
    return {"K": K, "V": V, "score": new_score.cuda(), "pos": new_pos.cuda(),
            "lens": torch.tensor([min(L, budget) for L in lens], dtype=torch.int32, device="cuda")}
