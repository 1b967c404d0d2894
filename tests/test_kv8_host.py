"""Host-side refusals of the 8-bit cache's entry points and of eviction (no GPU: fake pointers,
every call carries an argument that is refused before any CUDA call), the binding's checks, and the
plain 64-bit forms that the GPU tests compare with."""
import math

import numpy as np
import pytest
import torch

import kv8_util as ref

FAKE = 1 << 20
MIS = FAKE + 2
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer calls run only on hosts without a CUDA device")


@pytest.fixture(scope="module")
def pkg():
    from block_sparse_long_uocr_b200 import build
    build.build()
    import block_sparse_long_uocr_b200 as m
    return m


SPEC = {
    "rope_append_kv8": dict(q=FAKE, idx_q=FAKE, k_new=FAKE, v_new=FAKE, idx_k_new=FAKE, tok=FAKE, page=FAKE, start=FAKE, bt=FAKE,
                            sl=FAKE, n=4, B=4, H=10, mb=64, P=256, q_out=FAKE, idx_q_out=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE,
                            idx_k=FAKE, err=None, stream=None),
    "sparse_attn_kv8": dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, sl=FAKE, q_seq=None, q_pos=None, sel=FAKE, n=4, B=4,
                            H=10, mb=64, P=256, scale=0.1, out=FAKE, mass=None, err=None, stream=None),
    "sparse_decode_kv8": dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, idx_q=FAKE, idx_k=FAKE, bt=FAKE, sl=FAKE, B=4, H=10, mb=64,
                              P=256, out=FAKE, sel=FAKE, mass=None, ws=FAKE, wsn=1 << 40, err=None, stream=None),
    "dense_decode_kv8": dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, sl=FAKE, refb=3, B=4, H=10, mb=64, P=256, out=FAKE,
                             mass=None, ws=FAKE, wsn=1 << 40, err=None, stream=None),
    "sparse_attn_seq_kv8": dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, sl=FAKE, seq=0, q_pos=FAKE, sel=FAKE, n=4, B=4,
                                H=10, mb=64, P=256, scale=0.1, out=FAKE, mass=None, ws=FAKE, wsn=1 << 40, err=None, stream=None),
    "sparse_prefill_kv8": dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, idx_q=FAKE, idx_k=FAKE, bt=FAKE, sl=FAKE, seq=0, q_pos=FAKE,
                               n=4, B=4, H=10, mb=64, P=256, out=FAKE, sel=FAKE, mass=None, ws=FAKE, wsn=1 << 40, err=None,
                               stream=None),
    "evict_blocks": dict(mass=FAKE, bt=FAKE + (1 << 30), sl=FAKE + (2 << 30), B=4, H=10, mb=64, keep=16, sink=2,
                         new_mass=FAKE + (3 << 30), new_table=FAKE + (4 << 30), new_lens=FAKE + (5 << 30), freed=FAKE + (6 << 30),
                         n_freed=FAKE + (7 << 30), ws=FAKE + (8 << 30), wsn=1 << 40, err=None, stream=None),
}


def call(pkg, fn, **over):
    a = dict(SPEC[fn])
    assert set(over) <= set(a)
    a.update(over)
    return getattr(pkg.lib, "uocr_" + fn)(*a.values())


POINTERS = {"q", "idx_q", "k_new", "v_new", "idx_k_new", "tok", "page", "bt", "sl", "q_out", "idx_q_out", "k", "v", "ks", "vs", "idx_k",
            "sel", "out", "new_mass", "new_table", "new_lens", "freed", "n_freed"}


@no_gpu
@pytest.mark.parametrize("fn", list(SPEC))
def test_null_and_misaligned_pointers_are_refused(pkg, fn):
    for name in POINTERS & set(SPEC[fn]):
        assert call(pkg, fn, **{name: None}) == 1, name
        assert call(pkg, fn, **{name: MIS}) == 1, name
    if fn in ("sparse_attn_seq_kv8", "sparse_prefill_kv8"):
        assert call(pkg, fn, q_pos=None) == 1
    if fn != "evict_blocks" and "mass" in SPEC[fn]:
        assert call(pkg, fn, mass=MIS) == 1
    assert call(pkg, fn, err=MIS) == 1
    if "ws" in SPEC[fn]:
        assert call(pkg, fn, ws=None) == 3 and call(pkg, fn, ws=FAKE + 16) == 3 and call(pkg, fn, wsn=8) == 3


@no_gpu
@pytest.mark.parametrize("fn", list(SPEC))
def test_sizes_are_refused(pkg, fn):
    for over in (dict(B=0), dict(mb=0)):
        assert call(pkg, fn, **over) == 1, over
    assert call(pkg, fn, H=0) == 2 and call(pkg, fn, H=65) == 2
    assert call(pkg, fn, mb=1 << 27) == 2
    if "P" in SPEC[fn]:
        assert call(pkg, fn, P=0) == 1
    if "scale" in SPEC[fn]:
        assert call(pkg, fn, scale=math.nan) == 1 and call(pkg, fn, scale=math.inf) == 1
    if "seq" in SPEC[fn]:
        assert call(pkg, fn, seq=-1) == 1 and call(pkg, fn, seq=4) == 1
        assert call(pkg, fn, n=1 << 28) == 2


@no_gpu
def test_specific_refusals(pkg):
    assert call(pkg, "rope_append_kv8", n=-1) == 1
    assert call(pkg, "rope_append_kv8", start=None, n=5) == 1            # one token per sequence needs n == B
    assert call(pkg, "rope_append_kv8", q_out=FAKE + 256) == 1           # partial overlap with q
    assert call(pkg, "rope_append_kv8", idx_q_out=FAKE + 256) == 1
    assert call(pkg, "sparse_attn_kv8", mass=FAKE, q_seq=FAKE) == 1      # two queries could share a total
    assert call(pkg, "dense_decode_kv8", refb=-1) == 1
    for over in (dict(keep=5, sink=2), dict(keep=3, sink=0), dict(sink=-1), dict(sink=65), dict(keep=-1),
                 dict(new_mass=FAKE + 64), dict(new_table=FAKE), dict(freed=FAKE + (1 << 30)),
                 dict(n_freed=FAKE + (6 << 30)), dict(new_lens=FAKE + (2 << 30) + 4), dict(freed=FAKE + (4 << 30) + 512)):
        assert call(pkg, "evict_blocks", **over) == 1, over


@no_gpu
def test_zero_rows_are_a_no_op(pkg):
    assert call(pkg, "rope_append_kv8", n=0, q=None, k_new=None) == 0
    assert call(pkg, "sparse_attn_kv8", n=0, q=None, out=None) == 0
    assert call(pkg, "sparse_attn_seq_kv8", n=0, q=None, ws=None) == 0
    assert call(pkg, "sparse_prefill_kv8", n=0, q=None, ws=None) == 0


def test_workspace_sizes(pkg):
    for fn in (pkg.dense_kv8_workspace_bytes, pkg.sparse_attn_seq_kv8_workspace_bytes, pkg.prefill_kv8_workspace_bytes,
               pkg.evict_workspace_bytes):
        assert fn(0, 10, 64) == 0 and fn(4, 0, 64) == 0 and fn(4, 10, 0) == 0
        assert fn(4, 10, 64) % 256 == 0 and 0 < fn(4, 10, 64) <= fn(8, 10, 64) <= fn(8, 10, 128)


def test_binding_refuses_before_any_launch(pkg):
    """CPU tensors, wrong types and shapes raise in the binding."""
    q = torch.zeros((2, 3, 128), dtype=torch.bfloat16)
    k = torch.zeros((4, 3, 32, 128), dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones((4, 3))
    bt, sl = torch.zeros((2, 4), dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.dense_decode_kv8(q, k, k, s, s, bt, sl)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.evict_blocks(torch.zeros((2, 3, 4)), bt, sl, 4)
    with pytest.raises(TypeError):
        pkg.sparse_attn_kv8(None, k, k, s, s, bt, sl, torch.zeros((2, 16), dtype=torch.int32))


def test_what_the_checks_refuse_is_never_launched(pkg, monkeypatch):
    """Where the quick expression says no and the search for the culprit finds nothing, the call still ends there."""
    launched = []
    monkeypatch.setattr(pkg, "_refuse", lambda *a: None)
    monkeypatch.setattr(pkg, "_dev", lambda t, *a: t)
    monkeypatch.setattr(pkg, "_space", lambda *a: torch.empty(1, dtype=torch.uint8))
    monkeypatch.setattr(pkg, "_launch", lambda *a: launched.append(a[1]))
    q, x = torch.zeros((2, 3, 128), dtype=torch.bfloat16), torch.zeros((2, 128), dtype=torch.bfloat16)
    k, s = torch.zeros((4, 3, 32, 128), dtype=torch.uint8).view(torch.float8_e4m3fn), torch.ones((4, 3))
    bt, sl, ik = torch.zeros((2, 4), dtype=torch.int32), torch.ones(2, dtype=torch.int32), torch.zeros((4, 32, 128), dtype=torch.bfloat16)
    sel, mass = torch.zeros((2, 16), dtype=torch.int32), torch.zeros((2, 3, 4))
    out = dict(new_mass=mass.clone(), new_table=bt.clone(), new_lens=sl.clone(), freed=bt.clone(), n_freed=sl.clone())
    for call in (lambda: pkg.rope_append_kv8(q, x, q, q, x, sl, sl, bt, sl, k, k, s, s, ik),
                 lambda: pkg.sparse_attn_kv8(q, k, k, s, s, bt, sl, sel, out=q.clone()),
                 lambda: pkg.dense_decode_kv8(q, k, k, s, s, bt, sl, out=q.clone()),
                 lambda: pkg.sparse_attn_seq_kv8(q, k, k, s, s, bt, sl, 0, sl, sel, out=q.clone()),
                 lambda: pkg.evict_blocks(mass, bt, sl, 4, **out)):
        with pytest.raises(ValueError, match="do not fit together"):
            call()
    assert not launched


# --------------------------------------------------------------------------- the plain forms themselves
def test_encode_matches_torch_and_the_grid():
    x = torch.cat((torch.randn(4000) * 3, torch.randn(4000) * 1e-3, torch.linspace(-448, 448, 5001)))
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.encode(x.double().numpy()), want)
    codes = np.array([c for c in range(256) if c & 127 != 127], dtype=np.uint8)
    assert np.array_equal(ref.encode(ref.GRID[codes]), codes)
    # ties to the even code, both sides of a midpoint
    mid = (ref.GRID[8:126] + ref.GRID[9:127]) / 2
    got = ref.encode(mid)
    assert (got % 2 == 0).all() and (np.abs(got.astype(int) - np.arange(8, 126)) <= 1).all()
    assert np.array_equal(ref.encode(np.nextafter(mid, 1e9)), np.arange(9, 127))
    assert np.array_equal(ref.encode(np.nextafter(mid, 0)), np.arange(8, 126))
    assert (ref.encode(np.array([math.inf, -math.inf, math.nan])) & 127 == 127).all()


def test_scales_hold_their_rows():
    for amax in (0.0, 1e-45, 1e-30, 0.3, 447.9, 448.0, 448.1, 896.0, 3e38):
        s = ref.need_scale(np.array([amax, -amax / 2]))
        assert amax <= 448 * s and math.frexp(s)[0] == 0.5
        assert s == 2.0 ** -126 or amax > 224 * s
    assert ref.pow2_at_least(0.25) == 0.25 and ref.pow2_at_least(0.3) == 0.5 and ref.pow2_at_least(0.0) == 2.0 ** -126


def test_evict_by_hand():
    mass = torch.tensor([[[5, 1, 0, 1, 7, 0, 2, 2, 2, 2, 9, 9]], [[1.0] * 12]])
    table = torch.arange(24, dtype=torch.int32).reshape(2, 12)
    lens = torch.tensor([32 * 9 + 1, 64], dtype=torch.int32)      # 10 blocks and two pages ahead; 2 blocks
    m, t, n, f, c = ref.evict(mass, table, lens, 7, 1)
    # candidates 1..5 of totals 1 0 1 7 0: the two highest are 4 and (lower id on a tie) 1
    assert t[0].tolist() == [0, 1, 4, 6, 7, 8, 9, 10, 11, -1, -1, -1]
    assert f[0].tolist()[:4] == [2, 3, 5, -1] and c.tolist() == [3, 0] and n.tolist() == [32 * 6 + 1, 64]
    assert m[0, 0].tolist() == [5, 1, 7, 2, 2, 2, 2, 9, 9, 0, 0, 0]
    assert t[1].tolist() == table[1].tolist() and torch.equal(m[1], mass[1])
