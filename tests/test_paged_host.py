"""The paged-cache entry points without a GPU: refusals that the host makes
before any CUDA call, workspace sizes, the binding's checks, and the 64-bit
reference the GPU tests compare with."""
import ctypes

import pytest
import torch

import paged_ref as ref

FAKE = 0x10000            # aligned, never dereferenced: validation fails first
MIS = 0x10004
OK_BUT_NO_GPU = (1, 4)    # past the host's checks: no GPU here (4), or not device memory (1)


@pytest.fixture(scope="module")
def lib():
    from gqa_kv_head_gb300 import build
    build.build()
    import gqa_kv_head_gb300 as fr
    return fr.load()


def _strides(*s):
    return (ctypes.c_int64 * 3)(*s)


def _kv(lib, type=0, k=FAKE, v=FAKE, ks=None, vs=None, k_st=(2 * 64 * 128, 64 * 128, 128), v_st=None, n_pages=9, ps=64,
        H=2, hd=128, desc=True):
    from gqa_kv_head_gb300._abi import FrPagedKV
    d = FrPagedKV()
    return lib.fr_paged_kv_init(ctypes.addressof(d) if desc else None, type, k, _strides(*k_st), v,
                                _strides(*(v_st or k_st)), ks, vs, n_pages, ps, H, hd)


def test_cache_descriptor_refusals(lib):
    assert _kv(lib) in OK_BUT_NO_GPU
    assert _kv(lib, desc=False) == 1
    assert _kv(lib, k=None) == 1 and _kv(lib, v=None) == 1
    assert _kv(lib, k=MIS) == 1 and _kv(lib, v=MIS) == 1
    assert _kv(lib, type=2) == 1 and _kv(lib, type=-1) == 1
    assert _kv(lib, n_pages=0) == 1 and _kv(lib, H=0) == 1 and _kv(lib, ps=0) == 1 and _kv(lib, hd=0) == 1
    for hd in (32, 80, 96, 192, 512):
        assert _kv(lib, hd=hd) == 2
    for ps in (1, 8, 24, 48, 100, 512):
        assert _kv(lib, ps=ps) == 2
    # scales: with e4m3, and only with e4m3
    assert _kv(lib, ks=FAKE) == 1 and _kv(lib, vs=FAKE) == 1
    assert _kv(lib, type=1) == 1 and _kv(lib, type=1, ks=FAKE) == 1
    assert _kv(lib, type=1, ks=FAKE, vs=FAKE) in OK_BUT_NO_GPU
    assert _kv(lib, type=1, ks=FAKE + 2, vs=FAKE) == 1 and _kv(lib, type=1, ks=FAKE, vs=FAKE + 1) == 1


def test_cache_strides(lib):
    # [pages][rows][heads][hd] pools and padded rows are fine
    assert _kv(lib, k_st=(64 * 2 * 128, 128, 2 * 128)) in OK_BUT_NO_GPU
    assert _kv(lib, k_st=(2 * 64 * 136, 64 * 136, 136)) in OK_BUT_NO_GPU
    assert _kv(lib, k_st=(128, 9 * 128, 2 * 9 * 128)) in OK_BUT_NO_GPU       # pages innermost
    # rows that overlap, heads that overlap, pages that overlap, expanded dims
    assert _kv(lib, k_st=(2 * 64 * 128, 64 * 128, 64)) == 1
    assert _kv(lib, k_st=(2 * 64 * 128, 32 * 128, 128)) == 1
    assert _kv(lib, k_st=(64 * 128, 64 * 128, 128)) == 1
    assert _kv(lib, k_st=(0, 64 * 128, 128)) == 1
    assert _kv(lib, k_st=(2 * 64 * 128, 0, 128)) == 1
    assert _kv(lib, k_st=(-2 * 64 * 128, 64 * 128, 128)) == 1
    # more than any memory
    assert _kv(lib, n_pages=2 ** 31 - 1, k_st=(1 << 38, 64 * 128, 128)) == 1
    # not multiples of 16 bytes
    assert _kv(lib, k_st=(2 * 64 * 132, 64 * 132, 132)) == 1
    assert _kv(lib, type=1, ks=FAKE, vs=FAKE, k_st=(2 * 64 * 136, 64 * 136, 136)) == 1
    assert _kv(lib, v_st=(2 * 64 * 128, 64 * 128, 64)) == 1
    # a size-1 dimension's stride is not used
    assert _kv(lib, H=1, k_st=(64 * 128, 7, 128)) in OK_BUT_NO_GPU
    assert _kv(lib, n_pages=1, k_st=(0, 64 * 128, 128)) in OK_BUT_NO_GPU


def test_batch_descriptor_refusals(lib):
    from gqa_kv_head_gb300._abi import FrPagedBatch

    def call(ts=FAKE, kl=FAKE, tab=FAKE, stride=4, n_seq=3, n_tok=3, max_pages=4, desc=True):
        d = FrPagedBatch()
        return lib.fr_paged_batch_init(ctypes.addressof(d) if desc else None, ts, kl, tab, stride, n_seq, n_tok, max_pages)
    assert call() in OK_BUT_NO_GPU
    assert call(desc=False) == 1
    assert call(ts=None) == 1 and call(kl=None) == 1 and call(tab=None) == 1
    assert call(ts=FAKE + 2) == 1
    assert call(n_seq=0) == 1 and call(n_tok=0) == 1 and call(max_pages=0) == 1
    assert call(stride=3) == 1
    assert call(n_seq=65537) == 2 and call(n_tok=(1 << 20) + 1) == 2 and call(max_pages=(1 << 22) + 1, stride=1 << 23) == 2


def test_calls_want_filled_descriptors(lib):
    from gqa_kv_head_gb300 import rope_params
    from gqa_kv_head_gb300._abi import FrPagedBatch, FrPagedKV
    kv, bt, rp = FrPagedKV(), FrPagedBatch(), rope_params(128)
    for a, b in ((None, ctypes.addressof(bt)), (ctypes.addressof(kv), None), (ctypes.addressof(kv), ctypes.addressof(bt))):
        assert lib.fr_paged_attn(a, b, FAKE, 1024, 8, 1, 0, 1.0, FAKE, FAKE, 1 << 30, None) == 1
        assert lib.fr_kv_append_paged(a, b, 0, FAKE, 256, FAKE, 256, FAKE, ctypes.addressof(rp), None, None) == 1
    # a refused fill leaves a descriptor that no call takes
    kv.opaque[0] = 5
    assert lib.fr_paged_kv_init(ctypes.addressof(kv), 0, FAKE, _strides(1, 1, 1), FAKE, _strides(1, 1, 1), None, None, 4, 16,
                                1, 128) == 1
    assert not any(kv.opaque)


def test_workspace_size(lib):
    ws = lib.fr_paged_attn_workspace_size
    assert ws(8, 1, 256) > 0 and ws(32, 8, 128) > 0 and ws(7, 7, 64) > 0
    assert ws(8, 3, 128) == 0 and ws(0, 1, 128) == 0 and ws(8, 0, 128) == 0 and ws(8, 1, 96) == 0
    # two states of a row tile (16 rows at hd 256) for each of 152 CTAs and more
    assert ws(8, 1, 256) >= 2 * 152 * 16 * (256 * 4 + 8)
    assert max(ws(8, 1, hd) for hd in (64, 128, 256)) < 64 << 20
    assert lib.fr_status_string(6).startswith(b"FR_ERR_DEVICE_INPUT")


def test_binding_refuses_cpu_tensors():
    import gqa_kv_head_gb300 as fr
    p = torch.zeros((4, 1, 16, 64), dtype=torch.float16)
    with pytest.raises(ValueError):
        fr.PagedKV(p, p)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        fr.PagedBatch(i, i[:1], i[None, :])


# ---- the reference itself -----------------------------------------------------

def test_reference_scale_is_the_smallest_power_of_two():
    for a in (1e-3, 0.5, 1.0, 223.9, 224.0, 447.9, 448.0, 448.1, 1e6, 3e38):
        s = ref.pow2_scale(a)
        assert a <= 448.0 * s and (a > 224.0 * s or s == 2.0 ** -100)
    assert ref.pow2_scale(0.0) == 2.0 ** -100 and ref.pow2_scale(1e-40) == 2.0 ** -100


def test_reference_attention_against_one_softmax():
    """One sequence in pages in order: the plain masked softmax over the contiguous keys."""
    g = torch.Generator().manual_seed(0)
    ps, hd, H, G, n, n_kv = 16, 64, 2, 3, 4, 37
    k = torch.randn((3, H, ps, hd), generator=g, dtype=torch.float64)
    v = torch.randn((3, H, ps, hd), generator=g, dtype=torch.float64)
    q = torch.randn((n, H * G, hd), generator=g).half()
    table = torch.tensor([[0, 1, 2]], dtype=torch.int32)
    for kw in ({}, {"causal": False}, {"window": 5}, {"kq_scale": 0.3}):
        out, tol = ref.attention(q, k, v, [0, n], [n_kv], table, H * G, **kw)
        kc = k.permute(1, 0, 2, 3).reshape(H, -1, hd)[:, :n_kv].repeat_interleave(G, dim=0)
        vc = v.permute(1, 0, 2, 3).reshape(H, -1, hd)[:, :n_kv].repeat_interleave(G, dim=0)
        s = kw.get("kq_scale", 1.0) * torch.einsum("thd,hjd->thj", q.double(), kc)
        j, p = torch.arange(n_kv), (n_kv - n + torch.arange(n))[:, None]
        see = torch.ones((n, n_kv), dtype=torch.bool) if kw.get("causal") is False else j <= p
        if kw.get("window"):
            see &= j > p - kw["window"]
        s = s.masked_fill(~see[:, None, :], float("-inf"))
        want = torch.einsum("thj,hjd->thd", torch.softmax(s, dim=2), vc)
        assert float((out - want).abs().max()) < 1e-13
        assert 0 < float(tol.max()) < 1e-2


def test_reference_append_against_scalar_steps():
    """f16 rounding and e4m3 codes one value at a time, with e4m3's values listed."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    finite = codes[torch.isfinite(codes)]
    g = torch.Generator().manual_seed(1)
    rows = torch.randn((3, 1, 64), generator=g) * 5
    k = torch.zeros((2, 1, 16, 64), dtype=torch.float8_e4m3fn)
    sc = torch.full((2, 1), 2.0 ** -3)
    out, _, s, _ = ref.append(rows, rows, [0, 3], [18], torch.tensor([[1, 0]], dtype=torch.int32), k, k, sc, sc)
    # cache rows 15, 16, 17: one at the end of page 1 (which goes on), two at the start of page 0 (which begins)
    assert float(s[1, 0]) == max(2.0 ** -3, ref.pow2_scale(float(rows[0].abs().max())))
    assert float(s[0, 0]) == ref.pow2_scale(float(rows[1:].abs().max()))
    for r, (page, row) in enumerate(((1, 15), (0, 0), (0, 1))):
        for d in range(64):
            x = float(rows[r, 0, d]) / float(s[page, 0])
            got = float(out[page, 0, row, d].float())
            assert abs(got - x) <= float((finite - x).abs().min()) + 1e-12
