"""The paged cache's entry points without a GPU: struct mirrors, refusals, workspace sizes, the
binding's checks of tensors, and the float64 loops the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import paged_ref as ref


@pytest.fixture(scope="module")
def mf():
    import __graft_entry__
    __graft_entry__.load_builder().build()
    import cross_model_attention_mf_b200 as mf
    return mf


A = 4096  # a pointer that is never read


def kv_desc(mf, d):
    kv = d.kv
    kv.K = kv.V = kv.block_table = kv.seq_lens = A
    kv.dtype, kv.n_pages, kv.page_size, kv.max_pages = 1, 10, 16, 4
    kv.h_kv, kv.d, kv.nseq, kv.max_len = 2, 64, 3, 64


def decode_desc(mf):
    d = mf.PagedDecodeDesc()
    kv_desc(mf, d)
    d.Q = d.O = A
    d.h_r = 8
    return d


def append_desc(mf):
    d = mf.KvAppendDesc()
    kv_desc(mf, d)
    d.K_new = d.V_new = d.cu_seqlens_new = A
    d.total_new, d.max_new = 3, 1
    return d


def evict_desc(mf):
    d = mf.KvEvictDesc()
    kv_desc(mf, d)
    d.score_in = d.pos_in = d.score_out = d.pos_out = d.seq_lens_out = A
    d.score_stride, d.budget, d.sink, d.window = 64, 32, 4, 8
    return d


def scores_desc(mf):
    d = mf.KeyScoresDesc()
    d.bsr = mf.BsrDesc(A, A, A, 5)
    d.n_rows, d.map_dtype, d.h_s, d.B, d.h_r, d.h_kv = 4, 1, 8, 64, 8, 2
    d.W = d.cu_seqlens = d.qblock_base = d.score = A
    d.nseq, d.max_seqlen, d.score_stride = 1, 256, 256
    return d


CALLS = {"mf_paged_decode": decode_desc, "mf_kv_append": append_desc, "mf_kv_evict": evict_desc,
         "mf_map_key_scores": scores_desc}


def call(mf, name, d, ws=A, ws_bytes=1 << 40):
    fn = getattr(mf._lib, name)
    if name == "mf_kv_append":
        return fn(ctypes.byref(d), None)
    return fn(ctypes.byref(d), ctypes.c_void_p(ws), ws_bytes, None)


def test_struct_mirrors(mf):
    for k, s in ((5, mf.PagedDecodeDesc), (6, mf.KvAppendDesc), (8, mf.KvEvictDesc), (9, mf.KeyScoresDesc)):
        assert mf._lib.mf_abi_struct_size(k) == ctypes.sizeof(s)


KV_BAD = [("K", 0, 1), ("V", 0, 1), ("block_table", 0, 1), ("seq_lens", 0, 1), ("dtype", 2, 1),
          ("n_pages", 0, 1), ("page_size", 0, 1), ("max_pages", 0, 1), ("nseq", 0, 1), ("max_len", -1, 1),
          ("h_kv", 0, 1), ("d", 0, 1), ("nseq", 4097, 2), ("max_len", 1 << 30, 2), ("h_kv", 65, 2),
          ("d", 20, 2), ("d", 264, 2), ("page_stride", 16 * 2 * 64 - 8, 1),
          ("page_stride", 16 * 2 * 64 + 4, 1), ("page_stride", -8, 1), ("K", A + 8, 1), ("V", A + 2, 1),
          ("seq_lens", A + 1, 1), ("page_stride", (1 << 58) - 8, 1), ("page_stride", (1 << 56) + 8, 1)]


def test_page_offsets_that_pass_64_bits_are_refused(mf):
    d = decode_desc(mf)
    d.kv.page_stride, d.kv.n_pages = 1 << 50, 1 << 20
    assert call(mf, "mf_paged_decode", d) == 2


@pytest.mark.parametrize("name", ["mf_paged_decode", "mf_kv_append", "mf_kv_evict"])
@pytest.mark.parametrize("field,value,status", KV_BAD)
def test_bad_cache_is_refused(mf, name, field, value, status):
    d = CALLS[name](mf)
    setattr(d.kv, field, value)
    assert call(mf, name, d) == status
    assert mf._lib.mf_last_error()


BAD = [
    ("mf_paged_decode", "Q", 0, 1), ("mf_paged_decode", "O", 0, 1), ("mf_paged_decode", "h_r", 7, 1),
    ("mf_paged_decode", "h_r", 0, 1), ("mf_paged_decode", "h_r", 258, 2), ("mf_paged_decode", "scale", -1.0, 1),
    ("mf_paged_decode", "scale", math.inf, 1), ("mf_paged_decode", "scale", math.nan, 1),
    ("mf_paged_decode", "flags", 2, 1), ("mf_paged_decode", "q_stride", 8 * 64 - 8, 1),
    ("mf_paged_decode", "q_stride", 8 * 64 + 4, 1), ("mf_paged_decode", "Q", A + 4, 1),
    ("mf_paged_decode", "O", A + 8, 1), ("mf_paged_decode", "score_in", A, 1),
    ("mf_paged_decode", "score_out", A, 1), ("mf_paged_decode", "lse", A + 2, 1),
    ("mf_kv_append", "K_new", 0, 1), ("mf_kv_append", "V_new", A + 8, 1), ("mf_kv_append", "cu_seqlens_new", 0, 1),
    ("mf_kv_append", "total_new", -1, 1), ("mf_kv_append", "max_new", -1, 1), ("mf_kv_append", "max_new", 65, 1),
    ("mf_kv_append", "new_stride", 127, 1), ("mf_kv_append", "new_stride", 132, 1),
    ("mf_kv_append", "score", A, 1), ("mf_kv_append", "pos", A, 1), ("mf_kv_append", "n_seen", A + 1, 1),
    ("mf_kv_evict", "score_in", 0, 1), ("mf_kv_evict", "pos_in", 0, 1), ("mf_kv_evict", "score_out", 0, 1),
    ("mf_kv_evict", "pos_out", 0, 1), ("mf_kv_evict", "seq_lens_out", 0, 1), ("mf_kv_evict", "budget", 0, 1),
    ("mf_kv_evict", "sink", -1, 1), ("mf_kv_evict", "window", -1, 1), ("mf_kv_evict", "window", 29, 1),
    ("mf_kv_evict", "score_stride", 63, 1), ("mf_kv_evict", "score_in", A + 2, 1),
    ("mf_map_key_scores", "map_dtype", 3, 1), ("mf_map_key_scores", "B", 48, 1), ("mf_map_key_scores", "h_s", 0, 1),
    ("mf_map_key_scores", "h_s", 257, 1), ("mf_map_key_scores", "h_r", 7, 1), ("mf_map_key_scores", "h_kv", 0, 1),
    ("mf_map_key_scores", "W", 0, 1), ("mf_map_key_scores", "score", 0, 1), ("mf_map_key_scores", "nseq", 0, 1),
    ("mf_map_key_scores", "nseq", 4097, 2), ("mf_map_key_scores", "max_seqlen", -1, 1),
    ("mf_map_key_scores", "max_seqlen", 4097 * 64, 2), ("mf_map_key_scores", "n_rows", -1, 1),
    ("mf_map_key_scores", "n_rows", 1 << 24, 1), ("mf_map_key_scores", "score_stride", 255, 1),
    ("mf_map_key_scores", "cu_seqlens", A + 2, 1),
]


@pytest.mark.parametrize("name,field,value,status", BAD)
def test_bad_descriptor_is_refused(mf, name, field, value, status):
    d = CALLS[name](mf)
    setattr(d, field, value)
    assert call(mf, name, d) == status
    assert mf._lib.mf_last_error()


def test_bad_bsr_is_refused(mf):
    for bsr in (mf.BsrDesc(0, A, A, 5), mf.BsrDesc(A, 0, A, 5), mf.BsrDesc(A, A, 0, 5),
                mf.BsrDesc(A, A, A + 8, 5), mf.BsrDesc(A, A, A, -1)):
        d = scores_desc(mf)
        d.bsr = bsr
        assert call(mf, "mf_map_key_scores", d) == 1


@pytest.mark.parametrize("name", ["mf_paged_decode", "mf_kv_evict", "mf_map_key_scores"])
def test_workspace_is_checked(mf, name):
    d = CALLS[name](mf)
    n = ctypes.c_size_t(0)
    size = getattr(mf._lib, name + "_workspace_size")
    assert size(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value > 0
    assert size(ctypes.byref(d), None) == 1 and size(None, ctypes.byref(n)) == 1
    assert call(mf, name, d, ws_bytes=n.value - 1) == 1 and b"workspace" in mf._lib.mf_last_error()
    assert call(mf, name, d, ws=A + 128) == 1 and b"aligned" in mf._lib.mf_last_error()
    assert call(mf, name, d, ws=0) == 1
    assert getattr(mf._lib, name)(None, ctypes.c_void_p(A), 1 << 40, None) == 1


def test_workspace_sizes(mf):
    d = decode_desc(mf)
    d.h_r = 6  # groups of 3: a key's scores take 4 places
    n = ctypes.c_size_t(0)
    sizes = []
    for d.score_out in (0, A):
        d.score_stride = 64
        assert mf._lib.mf_paged_decode_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0
        sizes.append(n.value)
    assert sizes[1] - sizes[0] == 3 * 2 * 64 * 4 * 4
    e = evict_desc(mf)
    assert mf._lib.mf_kv_evict_workspace_size(ctypes.byref(e), ctypes.byref(n)) == 0
    assert n.value >= 2 * 4 * 3 * 2 * 32


@pytest.mark.parametrize("name", list(CALLS))
def test_null_descriptor(mf, name):
    fn = getattr(mf._lib, name)
    assert (fn(None, None) if name == "mf_kv_append" else fn(None, None, 0, None)) == 1


def test_binding_refuses_tensors_off_the_device(mf):
    c, _ = ref.make_cache((5,), 1, 64, 16, torch.float32)
    kv = mf.PagedKV(c.K, c.V, c.table, torch.tensor(c.lens, dtype=torch.int32), 5)
    with pytest.raises(ValueError, match="CUDA"):
        mf.mf_paged_decode(kv, torch.zeros(1, 1, 64))
    with pytest.raises(TypeError):
        mf.PagedKV(c.K.half(), c.V.half(), c.table, kv.seq_lens, 5).desc()


# ------------------------------------------------------------------ the float64 loops themselves

def test_reference_decode_matches_dense_softmax():
    c, _ = ref.make_cache((9, 0, 33), 2, 16, 4, torch.float32, seed=1)
    Q = torch.randn(3, 6, 16)
    O, lse, w, *_ = ref.decode(c, Q)
    for s, L in enumerate(c.lens):
        for r in range(6):
            if L == 0:
                assert (O[s, r] == 0).all() and lse[s, r] == -math.inf
                continue
            j = torch.arange(L)
            K = c.K[c.table[s].long()[j // 4], j % 4, r // 3].double()
            V = c.V[c.table[s].long()[j // 4], j % 4, r // 3].double()
            p = torch.softmax(Q[s, r].double() @ K.T / 4.0, -1)
            assert torch.allclose(O[s, r], p @ V, atol=1e-12)
        if L:
            assert torch.allclose(w[s].sum(-1), torch.full((2,), 3.0, dtype=torch.float64))


def test_reference_evict_keeps_the_right_rows():
    c, _ = ref.make_cache((6,), 1, 8, 2, torch.float32, seed=2)
    rows = [c.rows(c.K, 0, 0, [j])[0].clone() for j in range(6)]
    score = torch.tensor([[[0.0, 5.0, math.nan, 5.0, -math.inf, 0.0]]])
    pos = torch.arange(6, dtype=torch.int32)[None, None].contiguous()
    s, p, lens = ref.evict(c, score, pos, [6], 3, 1, 1)
    # position 0 (sink) and 5 (window) are protected, then the first of the two 5.0
    assert lens == [3] and p[0, 0].tolist() == [0, 1, 5, -1, -1, -1]
    assert s[0, 0].tolist() == [0.0, 5.0, 0.0, 0.0, 0.0, 0.0]
    for j, want in enumerate((0, 1, 5)):
        assert torch.equal(c.rows(c.K, 0, 0, [j])[0], rows[want])


def test_reference_key_scores_match_the_dense_sum():
    values, row_ptr, cols, base = ref.make_bsr((70,), 32, 3, torch.float32, seed=4, share=1.0)
    W = torch.randn(4, 3)
    out, _ = ref.key_scores(values, row_ptr, cols, W, (70,), base, 32, 2)
    dense = torch.zeros(3, 96, 96, dtype=torch.float64)
    for qb in range(3):
        for n in range(int(row_ptr[qb]), int(row_ptr[qb + 1])):
            dense[:, qb * 32:qb * 32 + 32, int(cols[n]) * 32:int(cols[n]) * 32 + 32] = values[n]
    P = torch.einsum("rs,sij->rij", W.double(), dense)
    assert torch.allclose(out[0], P.sum(1).view(2, 2, 96).sum(1)[:, :70])


def test_binding_refuses_overlapping_pages(mf):
    """Expanded pages lie 0 elements apart, which the C calls would take for dense ones."""
    from torch._subclasses import FakeTensorMode
    with FakeTensorMode():
        t = lambda *shape, dtype=torch.int32: torch.empty(*shape, dtype=dtype, device="cuda")
        one = t(1, 16, 2, 64, dtype=torch.bfloat16)
        dense = t(4, 16, 2, 64, dtype=torch.bfloat16)
        apart = t(4, 2, 16, 2, 64, dtype=torch.bfloat16)[:, 0]
        desc = lambda K, V: mf.PagedKV(K, V, t(3, 2), t(3), 30).desc()
        for K, V in ((one.expand(4, -1, -1, -1),) * 2, (dense, one.expand(4, -1, -1, -1)),
                     (one.expand(4, -1, -1, -1), apart), (dense.as_strided((4, 16, 2, 64), (2040, 128, 64, 1)),) * 2):
            with pytest.raises(ValueError, match="overlap"):
                desc(K, V)
        assert desc(apart, apart).page_stride == 2 * 16 * 2 * 64
        assert desc(dense, dense).page_stride == 0 and desc(one, one).page_stride == 0


@pytest.mark.parametrize("binding", [None, b"not a library"])
def test_import_without_the_paged_binding(mf, tmp_path, binding):
    """Only the paged cache's calls need _mf_bind.so, which fits one PyTorch: without it the package
    imports, the other calls run, and those raise the reason."""
    import os
    import shutil
    import subprocess
    import sys
    here = os.path.dirname(mf.__file__)
    to = tmp_path / "cross_model_attention_mf_b200"
    to.mkdir()
    for name in ("__init__.py", "libmf.so"):
        shutil.copy(os.path.join(here, name), to / name)
    if binding:
        (to / "_mf_bind.so").write_bytes(binding)
    code = """
import torch, cross_model_attention_mf_b200 as mf
assert mf.mf_version() and mf.mf_map_key_scores_workspace_size(4, 64, 2) > 0
assert mf.mf_prefix_hashes([1, 2, 3], 2).size == 2
t = torch.zeros(1)
kv = mf.PagedKV(t, t, t, t, 1)
for call in (kv.desc, lambda: mf.mf_paged_decode(kv, t), lambda: mf.mf_kv_append(kv, t, t, t, 1),
             lambda: mf.mf_kv_evict(kv, t, t, 1), lambda: mf.mf_map_key_scores(None, t, t, t, 1, 1)):
    try:
        call()
    except ImportError as e:
        assert "_mf_bind.so" in str(e) and isinstance(e.__cause__, ImportError), e
    else:
        raise AssertionError("no error")
print("ok")
"""
    run = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True,
                         env={k: v for k, v in os.environ.items() if k != "MF_LIBRARY"})
    assert run.returncode == 0 and run.stdout.strip() == "ok", run.stderr


def test_import_without_the_library_names_a_way_to_build_it(mf, tmp_path):
    import os
    import re
    import shutil
    import subprocess
    import sys
    to = tmp_path / "cross_model_attention_mf_b200"
    to.mkdir()
    for name in ("__init__.py", "build.py"):
        shutil.copy(os.path.join(os.path.dirname(mf.__file__), name), to / name)
    run = subprocess.run([sys.executable, "-c", "import cross_model_attention_mf_b200"], cwd=tmp_path,
                         capture_output=True, text=True, env={k: v for k, v in os.environ.items() if k != "MF_LIBRARY"})
    script = re.search(r"libmf.so is missing: build it with `python (\S+)`", run.stderr)
    # the script that it names starts without the package
    assert run.returncode and script, run.stderr
    run = subprocess.run([sys.executable, "-c", f"import runpy; print(runpy.run_path({script[1]!r})['LIB'])"],
                         cwd=tmp_path, capture_output=True, text=True)
    assert run.stdout.strip() == str(to / "libmf.so"), run.stderr


def test_scales_of_the_base_two_domain_are_bounded(mf):
    """Scores are multiplied by scale log2 e, a float32: a scale above 2^128 / log2 e would make it
    infinite, and scores of 0 NaN."""
    d = decode_desc(mf)
    n = ctypes.c_size_t(0)
    for scale, status in ((2.0 ** 127, 0), (1e-45, 0), (0.0, 0), (2.0 ** 127 * 1.0001, 1), (3.4e38, 1)):
        d.scale = scale
        assert mf._lib.mf_paged_decode_workspace_size(ctypes.byref(d), ctypes.byref(n)) == status, scale


@pytest.mark.parametrize("h_r", [2, 4, 6, 8, 18])
def test_decode_workspace_is_as_documented(mf, h_r):
    """The scores x_j take nseq * max_len * h_kv * (group rounded up to even) * 4 bytes; groups above
    8 take more scratch for bf16 (16 heads to a unit) than for float32 (8)."""
    n, got = ctypes.c_size_t(0), {}
    for dtype in (0, 1):
        for scores in (0, A):
            d = decode_desc(mf)
            d.kv.dtype, d.kv.max_pages, d.kv.max_len, d.h_r = dtype, 64, 1024, h_r
            d.score_out, d.score_stride = scores, 1024
            assert mf._lib.mf_paged_decode_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0
            got[dtype, scores] = n.value
        G = h_r // 2
        assert got[dtype, A] - got[dtype, 0] == 3 * 1024 * 2 * (G + G % 2) * 4
    assert (got[1, 0] > got[0, 0]) == (h_r > 16)
